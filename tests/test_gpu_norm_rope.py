"""qk_norm_rope against the formula in 64 bits (complex rotation, angles in
long double).

Tolerance: the arithmetic is fp32 (sum of d squares, one rsqrt, two products, a
rotation by fp32 cosines): below d eps/2 + 8 eps relative to the largest value
of the pair, eps = 2^-23, with fp32 stores; bf16 stores add half a step, 2^-8
relative at the most, of the value itself."""

import numpy as np
import pytest
import torch

from long_context_compressed_overlapped_b200 import api
from tests.helpers import npy

pytestmark = pytest.mark.gpu
DEV = "cuda"


def reference(x, pos, r, gain, norm, eps=1e-6, base=10000.0):
    x = npy(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else x.copy()
    if norm and gain is not None:
        y = y * npy(gain)
    d = x.shape[-1]
    if r:
        ang = npy(pos).astype(np.longdouble)[..., None, None] * np.longdouble(base) ** (-2 * np.arange(r // 2, dtype=np.longdouble) / r)
        z = (y[..., d - r::2] + 1j * y[..., d - r + 1::2]) * (np.cos(ang) + 1j * np.sin(ang)).astype(np.complex128)
        y = y.copy()
        y[..., d - r::2], y[..., d - r + 1::2] = z.real, z.imag
    return y


def check(got, ref, dt, d, live):
    got = npy(got)[live]
    ref = ref[live]
    pair = np.maximum(np.abs(ref), np.abs(ref.reshape(*ref.shape[:-1], -1, 2)[..., ::-1].reshape(ref.shape)))
    tol = (d / 2 + 8) * 2.0**-23 * pair + 1e-30
    if dt == torch.bfloat16:
        tol = tol + 2.0**-8 * np.abs(ref) * (1 + 2.0**-8)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)


CASES = [
    # dtype, B, n, HQ, HK, d, r, gains, q_norm, k_norm
    (torch.bfloat16, 2, 1, 64, 1, 512, 64, True, True, True),
    (torch.bfloat16, 1, 37, 64, 1, 512, 64, True, True, True),
    (torch.bfloat16, 3, 5, 16, 2, 128, 64, True, True, False),
    (torch.bfloat16, 1, 3, 1, 0, 1024, 512, False, True, True),
    (torch.bfloat16, 2, 9, 0, 3, 8, 8, True, True, True),
    (torch.bfloat16, 1, 11, 5, 3, 96, 32, False, False, True),
    (torch.bfloat16, 1, 700, 3, 1, 200, 0, True, True, True),
    (torch.float32, 3, 17, 4, 1, 64, 16, True, True, True),
    (torch.float32, 1, 2, 7, 1, 512, 512, True, True, True),
    (torch.float32, 2, 3, 33, 9, 4, 2, False, True, True),
    (torch.float32, 1, 1301, 2, 2, 36, 10, True, True, False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("far", [64, 1 << 20, (1 << 31) - 64])
def test_values(case, far):
    dt, B, n, HQ, HK, d, r, gains, qn, kn = case
    g = torch.Generator(device=DEV).manual_seed(d + n)
    q = torch.randn(B, n, HQ, d, generator=g, device=DEV).to(dt) if HQ else None
    k = (3 * torch.randn(B, n, HK, d, generator=g, device=DEV)).to(dt) if HK else None
    pos = far - 1 - torch.randint(0, 64, (B, n), generator=g, device=DEV, dtype=torch.int32)
    pos[0, 0] = 0
    if n > 2:
        pos[0, 2] = -1                                   # padding: left as it was
    qg = 1 + 0.1 * torch.randn(d, generator=g, device=DEV) if gains else None
    kg = 1 + 0.1 * torch.randn(d, generator=g, device=DEV) if gains else None
    q_out = torch.full_like(q, 7.0) if HQ else None
    k_out = torch.full_like(k, 7.0) if HK else None
    got = api.qk_norm_rope(q, k, pos, rope_dims=r, q_gain=qg, k_gain=kg, q_norm=qn, k_norm=kn, q_out=q_out, k_out=k_out)
    live = npy(pos) >= 0
    for x, y, gain, norm in ((q, got[0], qg, qn), (k, got[1], kg, kn)):
        if x is None:
            assert y is None
            continue
        check(y, reference(x, pos, r, gain, norm), dt, d, live)
        assert (npy(y)[~live] == 7.0).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_strided_slices_of_one_projection_and_in_place(dt):
    """Heads as slices of a fused projection, tokens with a gap, and in place."""
    g = torch.Generator(device=DEV).manual_seed(3)
    wide = torch.randn(2, 13, 9, 72, generator=g, device=DEV).to(dt)
    q, k = wide[:, ::2, 1:5, 8:], wide[:, ::2, 6:7, 8:]
    pos = torch.arange(14, device=DEV, dtype=torch.int32).view(2, 7) * 1000
    oq, ok = api.qk_norm_rope(q, k, pos, rope_dims=32)
    for x, y in ((q, oq), (k, ok)):
        assert y.is_contiguous()
        check(y, reference(x, pos, 32, None, True), dt, 64, np.ones((2, 7), bool))
    qc, kc = q.contiguous(), k.contiguous()
    got = api.qk_norm_rope(qc, kc, pos, rope_dims=32, q_out=qc, k_out=kc)
    assert got[0] is qc and torch.equal(qc, oq) and torch.equal(kc, ok)
    with pytest.raises(ValueError):
        api.qk_norm_rope(wide.transpose(2, 3), None, torch.zeros(2, 13, device=DEV, dtype=torch.int32), rope_dims=0)


def test_broadcast_rows():
    """Expanded inputs: strides of 0 along any dims, all three among them."""
    g = torch.Generator(device=DEV).manual_seed(4)
    pos = torch.arange(6, device=DEV, dtype=torch.int32).view(2, 3) * 77
    for x in (torch.randn(1, 1, 1, 64, generator=g, device=DEV), torch.randn(2, 1, 5, 64, generator=g, device=DEV),
              torch.randn(1, 3, 1, 64, generator=g, device=DEV)):
        y, _ = api.qk_norm_rope(x.expand(2, 3, 5, 64), None, pos, rope_dims=16)
        check(y, reference(x.expand(2, 3, 5, 64), pos, 16, None, True), torch.float32, 64, np.ones((2, 3), bool))


def test_strides_of_dims_of_size_one():
    """A dim of size 1 may carry any stride; in place is contiguous all the same."""
    g = torch.Generator(device=DEV).manual_seed(5)
    base = torch.randn(4096, generator=g, device=DEV)
    pos = torch.arange(3, device=DEV, dtype=torch.int32).view(1, 3) * 501
    x = base.as_strided((1, 3, 2, 64), (7, 256, 96, 1))
    y, _ = api.qk_norm_rope(x, None, pos, rope_dims=16)
    check(y, reference(x, pos, 16, None, True), torch.float32, 64, np.ones((1, 3), bool))
    x = base.as_strided((3, 1, 1, 64), (128, 13, 5, 1))
    y, _ = api.qk_norm_rope(x, None, pos.view(3, 1), rope_dims=16)
    check(y, reference(x, pos.view(3, 1), 16, None, True), torch.float32, 64, np.ones((3, 1), bool))
    x = base.clone().as_strided((1, 1, 2, 64), (9, 11, 64, 1))
    ref = reference(x, pos[:, 1:2], 16, None, True)
    with pytest.raises(RuntimeError):                       # (positions at an address that is no multiple of 16)
        api.qk_norm_rope(x, None, pos[:, 1:2], rope_dims=16, q_out=x)
    y, _ = api.qk_norm_rope(x, None, pos[:, 1:2].clone(), rope_dims=16, q_out=x)
    check(y, ref, torch.float32, 64, np.ones((1, 1), bool))


def test_rows_past_32_bit_offsets():
    """The last of 2.6e9 elements: the same bits as from a call on them alone."""
    n, last = 80_000, 50
    q = torch.randn(1, n, 64, 512, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV, dtype=torch.bfloat16)
    pos = torch.arange(n, device=DEV, dtype=torch.int32)[None]
    y, _ = api.qk_norm_rope(q, None, pos, rope_dims=64)
    z, _ = api.qk_norm_rope(q[:, -last:].contiguous(), None, pos[:, -last:].clone(), rope_dims=64)
    assert torch.equal(y[:, -last:], z)


def test_zero_rows_and_large_rows():
    x = torch.zeros(1, 3, 2, 64, device=DEV)
    x[0, 1] = 1e15
    x[0, 2] = 1e-12
    pos = torch.tensor([[5, 6, 7]], device=DEV, dtype=torch.int32)
    y, _ = api.qk_norm_rope(x, None, pos, rope_dims=16)
    check(y, reference(x, pos, 16, None, True), torch.float32, 64, np.ones((1, 3), bool))
    assert (y[0, 0] == 0).all()


def test_matches_the_attention_rows():
    """Window rows: the same finished rows as the decode compressor writes."""
    B, d, w, r = 3, 512, 8, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    raw = torch.randn(B, 1, 1, d, generator=g, device=DEV).bfloat16()
    gain = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
    pos = torch.tensor([[0], [12345], [1048575]], device=DEV, dtype=torch.int32)
    _, rows = api.qk_norm_rope(None, raw, pos, rope_dims=r, k_gain=gain)
    win = torch.zeros(B, w, d, dtype=torch.bfloat16, device=DEV)
    z = torch.zeros(B, d, dtype=torch.bfloat16, device=DEV)
    api.decode_compress("hca", pos[:, 0], (z, z), torch.zeros(B, 128, 2, d, dtype=torch.bfloat16, device=DEV),
                        torch.zeros(B, 8192, d, dtype=torch.bfloat16, device=DEV), m=128,
                        bias_a=torch.zeros(128, d, device=DEV), kv_raw=raw.view(B, d), win=win, kv_gain=gain, rope_dims=r)
    for b in range(B):
        a, c = npy(rows[b, 0, 0]), npy(win[b, int(pos[b, 0]) % w])
        assert np.abs(a - c).max() <= 2.0**-8 * np.abs(c).max()


def test_other_stream_and_graph():
    x = torch.randn(2, 3, 4, 128, device=DEV).bfloat16()
    pos = torch.arange(6, device=DEV, dtype=torch.int32).view(2, 3)
    want, _ = api.qk_norm_rope(x, None, pos, rope_dims=64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = api.qk_norm_rope(x, None, pos, rope_dims=64, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.qk_norm_rope(x, None, pos, rope_dims=64, q_out=out)
    x.mul_(2)
    pos.add_(3)
    graph.replay()
    assert torch.equal(out, api.qk_norm_rope(x, None, pos, rope_dims=64)[0])
    assert api.device_error() == 0
