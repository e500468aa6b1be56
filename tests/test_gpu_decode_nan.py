"""Decode steps of queries that hold NaN, and over cache rows that hold
infinities, in both kernels and however the keys are split over CTAs: a NaN
query's row is NaN; a key with an infinite value scores +inf (inf - inf: the row
is NaN) or -inf (no weight).  Finite values: tolerances of tests/helpers.py."""

import numpy as np
import pytest
import torch

from long_context_compressed_overlapped_b200 import api
from oracle import csahca_oracle as O
from tests import tree_reference as R
from tests.helpers import check_close, npy
from tests.test_gpu_tree import DEV, SMALL, TC, gen, name_of

pytestmark = pytest.mark.gpu
DIM = 5                                                     # (not a rope dim in either shape)


@pytest.mark.parametrize("heads", [SMALL, TC], ids=["f32", "tc"])
@pytest.mark.parametrize("kind", ["hca", "csa"])
def test_decode_step_of_a_nan_query(kind, heads):
    """A NaN in one head of one sequence's query: that row is NaN, the others
    keep their bits."""
    B, m, w, k, pos = 2, (16 if kind == "hca" else 4), 128, 1000, [29998, 20001]
    dt, H, d, r = heads["dt"], heads["H"], heads["d"], heads["r"]
    g = gen(31)

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=DEV) * (d ** -0.5 if dt == torch.float32 else 1.0)).to(dt)
    kv, win, q = normal(B, pos[0] // m + 1, d), normal(B, w, d), normal(B, H, d)
    sinks = torch.randn(H, generator=g, device=DEV)
    kw = {}
    if kind == "csa":
        kw = dict(k=k, idx_in=torch.stack([torch.randperm(pos[1] // m, generator=g, device=DEV)[:k].sort().values for _ in range(B)]).int())
    for q_norm in (True, False):
        call = lambda x: api.compressed_attn_decode(kind, x, R.ints(pos, DEV), kv, win, sinks, m=m, rope_dims=r, q_norm=q_norm, **kw)  # noqa: E731
        clean = call(q)
        bad = q.clone()
        bad[1, 2, DIM] = float("nan")
        got = call(bad)
        assert torch.isfinite(clean).all() and got[1, 2].isnan().all()
        got[1, 2] = clean[1, 2]
        assert torch.equal(got, clean)
    assert api.device_error() == 0


@pytest.mark.parametrize("heads", [SMALL, TC], ids=["f32", "tc"])
@pytest.mark.parametrize("n", [1, 130, 400])
def test_decode_step_over_infinite_entries(heads, n):
    """Heads that score the infinite keys -inf give them no weight (their dim
    aside, which may hold 0 x inf), the others are NaN."""
    m, w, pos = 16, 128, 29998
    dt, H, d, r = heads["dt"], heads["H"], heads["d"], heads["r"]
    g = gen(33)

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=DEV) * (d ** -0.5 if dt == torch.float32 else 1.0)).to(dt)
    kv, win, q = normal(1, pos // m + 1, d), normal(1, w, d), normal(1, H, d)
    sinks = torch.randn(H, generator=g, device=DEV)
    kv[0, :n, DIM] = float("inf")
    got = npy(api.compressed_attn_decode("hca", q, R.ints([pos], DEV), kv, win, sinks, m=m, rope_dims=r)[0])
    with np.errstate(invalid="ignore"):
        ref = O.decode_attention("hca", npy(q[0]), pos, npy(kv[0]), npy(win[0]), npy(sinks), m=m, w=w, r=r)
    low = npy(q[0, :, DIM]) < 0
    assert low.any() and not low.all()
    assert np.isnan(got[~low]).all() and np.isnan(ref[~low]).all()
    rest = np.arange(d) != DIM
    check_close(got[low][:, rest], ref[low][:, rest], name_of(dt))
    assert api.device_error() == 0
