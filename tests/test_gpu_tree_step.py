"""A verification step over interleaved layers (runtime.TreeStep) as it is used:
every node's output against the library's own decode steps along the node's
path, from the same state; then the accepted path committed, the state against
the decode steps' bit for bit, and the next step from there.

Tolerances: tests/helpers.py's (both sides are bf16 kernels with the same
roundings, so their difference is at most two of theirs: the oracle tests hold
each to 2e-2 and 5e-3)."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api, runtime, synth
from tests import tree_reference as R
from tests.helpers import check_close, npy

pytestmark = pytest.mark.gpu
DEV = "cuda"


def clone(layers):
    return [{n: (v.clone() if isinstance(v, torch.Tensor) else v) for n, v in L.items()} for L in layers]


def decode_path(wl, L, b, path, pos):
    """Decode steps of sequence b's path on its own copy of layer L's state
    (a batch of one): the outputs and the state."""
    one = {n: (v[b:b + 1].clone() if isinstance(v, torch.Tensor) and n in ("kv", "win", "ring", "iring", "kI", "kI_scale") else v)
           for n, v in L.items()}
    csa = L["kind"] == "csa"
    outs, sels = [], []
    for o, node in enumerate(path):
        p = R.ints([pos + o], DEV)
        row = lambda x: x[b, node][None].contiguous()                       # noqa: E731
        kw = {}
        if csa:
            kw = dict(istreams=tuple(row(x) for x in L["tis"]), ibias_a=L["ibias_a"], ibias_b=L["ibias_b"], iring=one["iring"],
                      kI=one["kI"], kI_scale=one["kI_scale"])
        api.decode_compress(L["kind"], p, tuple(row(x) for x in L["ts"]), one["ring"], one["kv"], m=L["m"], bias_a=L["bias_a"],
                            bias_b=L["bias_b"], kv_raw=row(L["tkv_raw"]), win=one["win"], kv_gain=L["kv_gain"], rope_dims=wl.r, **kw)
        kw = {}
        sel = None
        if csa:
            sel = torch.empty(1, wl.k, dtype=torch.int32, device=DEV)
            kw = dict(k=wl.k, qI=row(L["tqI"]), wI=row(L["tw"]), kI=one["kI"], kI_scale=one["kI_scale"], idx_out=sel)
        outs.append(api.compressed_attn_decode(L["kind"], row(L["tq"]), p, one["kv"], one["win"], L["sinks"], m=L["m"],
                                               rope_dims=wl.r, q_gain=L["q_gain"], **kw))
        sels.append(sel)
    return outs, sels, one


def same_selection(tree_idx, seq_idx, path, pos, m, N):
    """The node's selection names drafted entry j where the decode step names
    its place in the cache; scores that differ by a rounding may swap entries
    at the k-th place."""
    place = {N + node: (pos + o + 1) // m - 1 for o, node in enumerate(path)}
    a = {place.get(int(e), int(e)) for e in tree_idx.tolist() if e >= 0}
    b = {int(e) for e in seq_idx.tolist() if e >= 0}
    return len(a ^ b)


@pytest.mark.parametrize("name,ctx,B,T", [("decode_256k", 8189, 2, 12), ("decode_1m", 16383, 2, 7), ("decode_1m", 200, 1, 3),
                                           ("decode_1m_fp8kv", 16381, 2, 9)])
def test_step_is_the_decode_steps_of_each_path(name, ctx, B, T):
    wl = synth.WORKLOADS[name]
    layers = synth.tree_inputs(wl, T, DEV, ctx=ctx, B=B, layers=("csa", "hca"), room=2 * T)
    if B > 1:
        for L in layers:
            L["pos"][1] -= 130                                              # ragged: behind a block's end in both kinds
    before = clone(layers)
    stream = torch.cuda.Stream()
    step = runtime.TreeStep(wl, layers, stream, keep_idx=True)
    step()
    stream.synchronize()
    parents, pos = layers[0]["parents"].tolist(), layers[0]["pos"].tolist()
    first = [o.clone() for o in step.outputs]
    for li, L in enumerate(before):
        assert all(torch.equal(L[n], layers[li][n]) for n in ("kv", "win", "ring"))   # the caches are only read
        for b in range(B):
            for i in {T - 1, T // 2, 0}:
                path = R.path_of(parents[b], i)
                outs, sels, _ = decode_path(wl, L, b, path, pos[b])
                if L["kind"] == "csa":
                    swapped = same_selection(step.idx[li][b, i], sels[-1][0], path, pos[b], L["m"], L["kv"].shape[1])
                    assert swapped <= 2, f"layer {li} node {b},{i}: {swapped} entries differ"
                    if swapped:
                        continue                                            # near ties at the k-th place: other keys
                check_close(npy(first[li][b, i]), npy(outs[-1][0]), "bf16", f"layer {li} node {b},{i}")
    # accept the deepest path of each sequence but the last one's second half
    paths = [max((R.path_of(parents[b], i) for i in range(T)), key=len) for b in range(B)]
    paths[-1] = paths[-1][:max(1, len(paths[-1]) // 2)]
    n = max(len(p) for p in paths)
    step.commit(R.ints([p + [-1] * (n - len(p)) for p in paths], DEV))
    stream.synchronize()
    for li, L in enumerate(before):
        for b in range(B):
            _, _, one = decode_path(wl, L, b, paths[b], pos[b])
            for key in ("kv", "win", "ring", "iring", "kI", "kI_scale"):
                if L.get(key) is not None:
                    assert torch.equal(layers[li][key][b], one[key][0]), f"layer {li} {key} of sequence {b}"
            assert int(layers[li]["pos"][b]) == pos[b] + len(paths[b])
    # the next trees from the committed state, replayed as a graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    graph.replay()
    stream.synchronize()
    for li, L in enumerate(layers):
        outs, sels, _ = decode_path(wl, L, 0, R.path_of(parents[0], T - 1), int(L["pos"][0]))
        if L["kind"] == "csa" and same_selection(step.idx[li][0, T - 1], sels[-1][0], R.path_of(parents[0], T - 1),
                                                 int(L["pos"][0]), L["m"], L["kv"].shape[1]):
            continue
        check_close(npy(step.outputs[li][0, T - 1]), npy(outs[-1][0]), "bf16", f"next step, layer {li}")
    assert api.device_error() == 0


def test_commit_leaves_inactive_sequences_alone():
    """Nodes named for a sequence without committed tokens are not taken, and
    paths made on the current stream are waited for."""
    wl = synth.WORKLOADS["decode_1m"]
    layers = synth.tree_inputs(wl, 3, DEV, ctx=254, B=2, layers=("csa", "hca"), room=6)
    for L in layers:
        L["pos"][0] = -1
    before = clone(layers)
    step = runtime.TreeStep(wl, layers, torch.cuda.Stream())
    step()
    slow = torch.randn(4096, 4096, device=DEV)
    for _ in range(8):
        slow = slow @ slow * 1e-3
    path = R.path_of(layers[0]["parents"].tolist()[1], 2)
    paths = torch.full((2, len(path)), -1, device=DEV, dtype=torch.int32)
    paths[0] = 0
    paths[1] = R.ints(path, DEV)
    step.commit(paths)
    step.stream.synchronize()
    for li, (L, was) in enumerate(zip(layers, before)):
        _, _, one = decode_path(wl, was, 1, path, 254)
        assert L["pos"].tolist() == [-1, 254 + len(path)]
        for key in ("kv", "win", "ring", "iring", "kI", "kI_scale"):
            if L.get(key) is not None:
                assert torch.equal(L[key][0], was[key][0]), f"layer {li} {key} of the inactive sequence"
                assert torch.equal(L[key][1], one[key][0]), f"layer {li} {key}"
    assert api.device_error() == 0
