"""The argument structs of the decode and tree calls hold device pointers: the tensors that
they point to stay alive with the list that comes with the struct, and a
TreeStep's buffers are its own."""

import gc
import weakref

import pytest
import torch

from long_context_compressed_overlapped_b200 import api, runtime, synth
from tests.test_gpu_tree import DEV, SMALL, attn_case, compress_case
from tests import tree_reference as R

pytestmark = pytest.mark.gpu


def tensors(*xs):
    return [x for x in xs if isinstance(x, torch.Tensor)]


def test_structs_keep_their_tensors():
    c = compress_case("csa", torch.bfloat16, 2, 4, 128, 4, [7, 9], "chain")
    pos, parents = R.ints(c["pos"], DEV), R.ints(c["parents"], DEV)
    out, scale = torch.zeros(2, 4, 128, dtype=torch.uint8, device=DEV), torch.zeros(2, 4, 1, device=DEV)
    refs = [weakref.ref(t) for t in tensors(*c["streams"], c["ring"], pos, parents, c["bias_a"], c["bias_b"], c["gain"], out, scale)]
    held = api.tree_compress_args("csa", c["streams"], c["ring"], pos, parents, c["bias_a"], 4, bias_b=c["bias_b"], gain=c["gain"],
                                  out=out, out_scale=scale)
    del c, pos, parents, out, scale
    gc.collect()
    assert all(r() is not None for r in refs)
    del held
    s = attn_case("csa", 2, 4, [900, 800], "chain", 4, 16, 32, **SMALL)
    pos, parents = R.ints(s["pos"], DEV), R.ints(s["parents"], DEV)
    qI, wI = torch.randn(2, 4, 2, 32, device=DEV), torch.randn(2, 4, 2, device=DEV)
    kI, dk = torch.randn(2, s["N"], 32, device=DEV), torch.randn(2, 4, 32, device=DEV)
    idx = torch.empty(2, 4, 32, dtype=torch.int32, device=DEV)
    kw = dict(draft=s["draft"], qI=qI, wI=wI, kI=kI, draft_kI=dk, idx_out=idx, q_gain=s["q_gain"], kv_gain=s["kv_gain"])
    refs = [weakref.ref(t) for t in tensors(*kw.values(), pos, parents, s["q"], s["kv"], s["win"], s["kv_raw"], s["sinks"])]
    held = api.tree_attn_args("csa", s["q"], pos, parents, s["kv"], s["win"], s["kv_raw"], s["sinks"], m=4, rope_dims=16, k=32, **kw)
    del s, pos, parents, qI, wI, kI, dk, idx, kw
    gc.collect()
    assert all(r() is not None for r in refs)
    del held


def test_decode_structs_keep_their_tensors():
    wl = synth.WORKLOADS["decode_1m"]
    L = synth.decode_inputs(wl, DEV, ctx=1003, B=2, layers=("csa",))[0]
    idx, out = torch.empty(2, wl.k, dtype=torch.int32, device=DEV), torch.empty_like(L["q"])
    names = ("q", "pos", "kv", "win", "sinks", "qI", "w", "kI", "kI_scale", "q_gain")
    refs = [weakref.ref(L[n]) for n in names] + [weakref.ref(idx), weakref.ref(out)]
    held = api.decode_args("csa", L["q"], L["pos"], L["kv"], L["win"], L["sinks"], m=L["m"], rope_dims=wl.r, k=wl.k, qI=L["qI"], wI=L["w"],
                           kI=L["kI"], kI_scale=L["kI_scale"], idx_out=idx, out=out, q_gain=L["q_gain"])
    names = ("pos", "kv", "win", "ring", "iring", "ca", "cb", "cza", "czb", "ia", "ib", "iza", "izb", "kv_raw", "kI", "kI_scale",
             "bias_a", "bias_b", "ibias_a", "ibias_b", "kv_gain")
    refs += [weakref.ref(L[n]) for n in names]
    comp = runtime.compress_args(wl, L)
    del L, idx, out
    gc.collect()
    assert all(r() is not None for r in refs)
    del held, comp


def test_a_step_writes_its_own_buffers_only():
    """Small tensors made on the step's stream after the step (where the
    allocator hands out what is free) keep their contents."""
    wl = synth.WORKLOADS["decode_1m"]
    layers = synth.tree_inputs(wl, 8, DEV, ctx=1003, B=2, layers=("csa", "hca", "csa"))
    stream = torch.cuda.Stream()
    step = runtime.TreeStep(wl, layers, stream)
    gc.collect()
    with torch.cuda.stream(stream):
        mine = [torch.full((16,), 7.0, device=DEV) for _ in range(64)]
    step()
    stream.synchronize()
    assert all((x == 7).all() for x in mine)
    assert api.device_error() == 0
