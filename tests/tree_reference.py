"""Draft trees for the tests, and what their nodes must get: the oracle's
decode steps along each node's own path, one token after another."""

import numpy as np
import torch

from oracle import csahca_oracle as O
from tests.helpers import npy

NONE = -2


def parents_of(shape: str, B: int, T: int, seed: int = 0) -> list:
    """parents [B][T]: "chain", "flat" (every node a first token), "wide"
    (random, some further first tokens), "padded" (wide, the last places and one
    inner place without a node, its descendants orphans)."""
    rng = np.random.RandomState(seed)
    rows = []
    for b in range(B):
        row = []
        for i in range(T):
            if shape == "chain" or (i == 0 and shape != "flat"):
                row.append(i - 1)
            elif shape == "flat":
                row.append(-1)
            else:
                row.append(int(rng.randint(max(-1, i - 6), i)))
        if shape == "padded":
            live = max(1, T - 1 - b % 3)
            row[live:] = [NONE] * (T - live)
            if live > 4:
                row[3] = NONE
        rows.append(row)
    return rows


def path_of(parents, i):
    """Nodes from the first drafted token to node i, or None if i is no node."""
    up = []
    while i >= 0:
        if parents[i] < -1:
            return None
        up.append(i)
        i = parents[i]
    return up[::-1]


def node_position(parents, pos, i):
    path = path_of(parents, i)
    return -1 if path is None or pos < 0 else pos + len(path) - 1


def entry_of_node(kind, b, i, parents, pos, streams, ring, biases, m, **finish):
    """The oracle's entry of node i of sequence b: (entry, pooled, finished) or
    None, by decode_compress_step over the path's tokens."""
    names = ("a", "b", "za", "zb") if kind == "csa" else ("a", "za")
    path = path_of(parents[b], i)
    if path is None or pos[b] < 0:
        return None
    state = {n: npy(ring[b, :, j]) for j, n in enumerate(names)}
    entry = None
    for o, node in enumerate(path):
        new = {n: npy(streams[j][b, node]) for j, n in enumerate(names)}
        state, entry, _ = O.decode_compress_step(kind, pos[b] + o, new, state, biases, m, **finish)
    return entry


def attend_node(kind, b, i, parents, pos, q, kv, win, kv_raw, draft, sinks, *, m, w, r, q_gain, kv_gain, sel=None,
                q_norm=True, kv_norm=True, tau=None):
    """The oracle's decode attention of node i after its path's tokens: their
    window rows in the ring, their entries (rows of draft) in the cache."""
    path = path_of(parents[b], i)
    if path is None or pos[b] < 0:
        return None
    t = pos[b] + len(path) - 1
    N = kv.shape[1]
    cache = np.zeros((N, kv.shape[2]))
    v = min(N, pos[b] // m)
    cache[:v] = npy(kv[b, :v])
    ring = np.zeros((w, kv.shape[2]))
    for p in range(max(0, pos[b] - w), pos[b]):
        ring[p % w] = npy(win[b, p % w])
    local = {}
    for o, node in enumerate(path):
        p = pos[b] + o
        if w > 0:
            ring[p % w] = O.finish_rows(npy(kv_raw[b, node]), p, None if kv_gain is None else npy(kv_gain), r,
                                        normalize=kv_norm)
        if draft is not None and (p + 1) % m == 0 and (p + 1) // m - 1 < N:
            cache[(p + 1) // m - 1] = npy(draft[b, node])
            local[node] = (p + 1) // m - 1
    if kind == "hca" and draft is None:
        cache, kind_v = cache[:v], v
    rows = None
    if kind == "csa":
        rows = []
        for e in np.asarray(sel):
            if 0 <= e < N:
                rows.append(npy(kv[b, int(e)]))
            elif e >= N:
                rows.append(npy(draft[b, int(e) - N]))
        cache = np.stack(rows) if rows else np.zeros((0, kv.shape[2]))
        sel = np.arange(len(rows))
    return O.decode_attention(kind, npy(q[b, i]), t, cache, ring, npy(sinks), m=m, w=w, r=r,
                              q_gain=None if q_gain is None else npy(q_gain), sel=sel, q_norm=q_norm, tau=tau)


def select_node(b, i, parents, pos, qI, wI, kI, draft_kI, m, k, N):
    """The oracle's top-k over committed entries and the path's own, in the
    call's indices (N + j: drafted entry j)."""
    path = path_of(parents[b], i)
    if path is None or pos[b] < 0:
        return np.full(k, -1, np.int64)
    v = min(N, pos[b] // m)
    names = list(range(v))
    keys = [npy(kI[b, :v])]
    if draft_kI is not None:
        for o, node in enumerate(path):
            p = pos[b] + o
            if (p + 1) % m == 0 and (p + 1) // m - 1 < N:
                names.append(N + node)
                keys.append(npy(draft_kI[b, node])[None])
    scores = O.indexer_scores(npy(qI[b, i]), npy(wI[b, i]), np.concatenate(keys))
    got = O.top_k_select(scores, k)
    return np.array([names[e] if e >= 0 else -1 for e in got], np.int64)


def ints(rows, dev):
    return torch.tensor(rows, dtype=torch.int32, device=dev)
