"""A verification step over interleaved layers, node by node: every CSA node's
selection obeys the top-k rule over the committed entries and its own path's,
and every node's output is the decode step's over the same keys, ties or not;
then the same for the next trees, from the committed state and a replayed graph.

Tolerances: tests/helpers.py's (selections: entries within 1e-3 of the k-th score
may be swapped; outputs: both sides are bf16 kernels of the same roundings)."""

import numpy as np
import pytest
import torch

from long_context_compressed_overlapped_b200 import api, runtime, synth
from oracle import csahca_oracle as O
from tests import tree_reference as R
from tests.helpers import check_close, check_topk, npy
from tests.test_gpu_tree_step import DEV, clone, decode_path

pytestmark = pytest.mark.gpu


def indexer_keys(rows, scale):
    if scale is None:
        return npy(rows)
    return npy(rows.view(torch.float8_e4m3fn).float()) * np.repeat(npy(scale), 128, axis=-1)


def check_step(wl, layers, before, step, what):
    """Returns how many CSA nodes were compared, and how many of them had drafted entries to choose from."""
    parents, pos = layers[0]["parents"].tolist(), before[0]["pos"].tolist()
    B, T = layers[0]["tq"].shape[:2]
    compared = mixed = 0
    for li, L in enumerate(before):
        m, N = L["m"], L["kv"].shape[1]
        if L["kind"] == "csa":
            f8 = L["kI_scale"] is not None
            dks = torch.zeros(B, T, wl.dI // 128, device=DEV) if f8 else None
            dk = torch.zeros(B, T, wl.dI, dtype=torch.uint8, device=DEV) if f8 else None
            dk = api.tree_compress("csa", L["tis"], L["iring"], L["pos"], L["parents"], L["ibias_a"], m, bias_b=L["ibias_b"],
                                   rms_norm=False, out=dk, out_scale=dks)
        for b in range(B):
            for i in sorted({T - 1, T // 2, 1, 0}):
                name = f"{what}, layer {li} node {b},{i}"
                path = R.path_of(parents[b], i)
                outs, _, state = decode_path(wl, L, b, path, pos[b])
                want = outs[-1][0]
                if L["kind"] == "csa":
                    v = min(N, pos[b] // m)
                    own = [j for o, j in enumerate(path) if (pos[b] + o + 1) % m == 0 and (pos[b] + o + 1) // m - 1 < N]
                    place = {N + j: v + x for x, j in enumerate(own)}
                    sel = [place.get(e, e) for e in step.idx[li][b, i].tolist()]
                    keys = indexer_keys(L["kI"][b, :v], L["kI_scale"][b, :v] if f8 else None)
                    mine = indexer_keys(dk[b, own], dks[b, own] if f8 else None)
                    scores = O.indexer_scores(npy(L["tqI"][b, i]), npy(L["tw"][b, i]), np.concatenate([keys, mine]))
                    check_topk(sel, scores, wl.k, name)
                    mixed += len(own) > 0
                    compared += 1
                    want = api.compressed_attn_decode("csa", L["tq"][b, i][None].contiguous(), R.ints([pos[b] + len(path) - 1], DEV),
                                                      state["kv"], state["win"], L["sinks"], m=m, rope_dims=wl.r, k=wl.k,
                                                      idx_in=R.ints([sel], DEV), q_gain=L["q_gain"])[0]
                check_close(npy(step.outputs[li][b, i]), npy(want), "bf16", name)
    return compared, mixed


@pytest.mark.parametrize("name,ctx,B,T", [("decode_256k", 8187, 2, 12), ("decode_1m", 16381, 2, 7), ("decode_1m", 199, 1, 3),
                                          ("decode_1m_fp8kv", 16383, 2, 9)])
def test_every_node_is_the_decode_step_over_its_keys(name, ctx, B, T):
    wl = synth.WORKLOADS[name]
    layers = synth.tree_inputs(wl, T, DEV, ctx=ctx, B=B, layers=("csa", "hca", "csa"), room=2 * T)
    if B > 1:
        for L in layers:
            L["pos"][1] -= 130
    before = clone(layers)
    stream = torch.cuda.Stream()
    step = runtime.TreeStep(wl, layers, stream, keep_idx=True)
    step()
    stream.synchronize()
    compared, mixed = check_step(wl, layers, before, step, "first step")
    assert compared >= 2 * min(3, T) * B and mixed > 0
    paths = [max((R.path_of(row, i) for i in range(T)), key=len) for row in layers[0]["parents"].tolist()]
    n = max(map(len, paths))
    step.commit(R.ints([p + [-1] * (n - len(p)) for p in paths], DEV))
    stream.synchronize()
    before = clone(layers)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    graph.replay()
    stream.synchronize()
    compared, _ = check_step(wl, layers, before, step, "next step")
    assert compared >= 2 * min(3, T) * B and api.device_error() == 0
