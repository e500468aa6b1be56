"""qk_norm_rope without output tensors: the rows of padding tokens (pos < 0) of
the new outputs are zeros, whatever their memory held, and the others what a
given output receives; rows of a given output are left as they were."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,n,HQ,HK,d,r", [(2, 3, 64, 1, 512, 64), (1, 1, 5, 3, 96, 32), (1, 1301, 3, 1, 64, 16), (3, 2001, 1, 2, 128, 64),
                                           (1, 900, 0, 5, 40, 8), (1, 650, 2, 0, 256, 0)])
def test_padding_rows_of_new_outputs_are_zeros(dt, B, n, HQ, HK, d, r):
    g = torch.Generator(device=DEV).manual_seed(n)
    wide = torch.randn(B, n, HQ + HK + 1, d, generator=g, device=DEV).to(dt)
    q, k = (wide[:, :, :HQ] if HQ else None), (wide[:, :, HQ:HQ + HK] if HK else None)
    pos = torch.randint(0, 1 << 20, (B, n), generator=g, device=DEV, dtype=torch.int32)
    for hide in (torch.rand(B, n, generator=g, device=DEV) < 0.3, torch.ones(B, n, device=DEV, dtype=torch.bool)):
        pos = torch.where(hide, torch.where(pos % 2 == 0, -1, -(1 << 31)), pos).int()       # (any negative position)
        given = [None if x is None else torch.full((B, n, x.shape[2], d), 7.0, device=DEV, dtype=dt) for x in (q, k)]
        api.qk_norm_rope(q, k, pos, rope_dims=r, q_out=given[0], k_out=given[1])
        junk = torch.full((64 << 20,), float("nan"), device=DEV)                            # (what the allocator hands out next)
        del junk
        new = api.qk_norm_rope(q, k, pos, rope_dims=r)
        for y, z in zip(new, given):
            if z is None:
                assert y is None
                continue
            live = pos >= 0
            assert not y[~live].any() and (z[~live] == 7).all()
            assert torch.equal(y[live], z[live])
    if HQ and HK:                                                                           # one side new, one given
        k_out = torch.full((B, n, HK, d), 7.0, device=DEV, dtype=dt)
        y, z = api.qk_norm_rope(q, k, pos, rope_dims=r, k_out=k_out)
        assert z is k_out and (z == 7).all() and not y.any()
        q_out = torch.full((B, n, HQ, d), 7.0, device=DEV, dtype=dt)
        y, z = api.qk_norm_rope(q, k, pos, rope_dims=r, q_out=q_out)
        assert y is q_out and (y == 7).all() and not z.any()
    assert api.device_error() == 0
