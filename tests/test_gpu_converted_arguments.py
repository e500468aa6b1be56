"""Gains, sinks and scales that the wrappers convert to fp32: a call with bf16 or
fp64 tensors gives the bits of the same values in fp32 (each converted copy lives
until the call's kernels have been queued)."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("other", [torch.bfloat16, torch.float64])
@pytest.mark.parametrize("dt,H,d,r", [(torch.float32, 4, 64, 16), (torch.bfloat16, 64, 512, 64), (torch.bfloat16, 16, 128, 64)])
@pytest.mark.parametrize("kind", ["csa", "hca"])
def test_prefill(kind, dt, H, d, r, other):
    n, m, w = 70, 4, 16
    g = torch.Generator(device=DEV).manual_seed(d)
    q, kv, win = (torch.randn(*s, generator=g, device=DEV).to(dt) for s in ((1, n, H, d), (1, n // m, d), (1, n, d)))
    few = [torch.randn(x, generator=g, device=DEV).bfloat16() for x in (H, d, d)]
    kw = dict(m=m, w=w, rope_dims=r)
    if kind == "csa":
        kw["idx"] = torch.arange(8, device=DEV, dtype=torch.int32).expand(1, n, 8).contiguous()
    call = lambda sinks, qg, kg: api.compressed_attn_prefill(kind, q, kv, win, sinks, q_gain=qg, kv_gain=kg, **kw)   # noqa: E731
    want = call(*(x.float() for x in few))
    for _ in range(4):
        assert torch.equal(call(*(x.to(other) for x in few)), want)
    assert api.device_error() == 0


@pytest.mark.parametrize("N,nq", [(300, 2), (40000, 1)])
def test_indexer_scales(N, nq):
    g = torch.Generator(device=DEV).manual_seed(N)
    qI, w = torch.randn(1, nq, 64, 128, generator=g, device=DEV).bfloat16(), torch.randn(1, nq, 64, generator=g, device=DEV)
    codes, scale = synth.quantize_e4m3_rows(torch.randn(1, N, 128, generator=g, device=DEV).bfloat16())
    pos = torch.full((1, nq), N - 1, device=DEV, dtype=torch.int32)
    want = api.indexer_topk(qI, w, codes, pos, 1, 64, kI_scale=scale)
    for _ in range(4):
        assert torch.equal(api.indexer_topk(qI, w.double(), codes, pos.long(), 1, 64, kI_scale=scale.double()), want)
    assert api.device_error() == 0
