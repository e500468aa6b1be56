"""NaN scores rank below every other score, ties to the lower index, in every
form of the selection: few rows and more rows than SMs, short rows and long
ones, scores routed out of the scan or read back, and the merge of several shards.

Every finite score is a small multiple of a quarter, exact in all types, and
every value is copied or compared, so that selections match exactly."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


def queries(kind, *lead):
    """qI, w whose heads read a key's dim 1 (weight 1) and dim 2 (weight -1), and
    dim 0 with both weights: 0, or inf - inf where its double overflows."""
    HI, dI, dt = (4, 32, torch.float32) if kind == "f32" else (64, 128, torch.bfloat16)
    qI, w = torch.zeros(*lead, HI, dI, device=DEV, dtype=dt), torch.zeros(*lead, HI, device=DEV)
    qI[..., 0, 0] = qI[..., 1, 0] = 2
    qI[..., 2, 1] = qI[..., 3, 2] = 1
    w[..., 0], w[..., 1], w[..., 2], w[..., 3] = 1, -1, 1, -1
    return qI, w


def keys(kind, scores):
    """Keys (and scales) that score as given."""
    dI = 32 if kind == "f32" else 128
    s = torch.nan_to_num(scores, nan=0.0)
    k = torch.zeros(*scores.shape, dI, device=DEV)
    k[..., 1], k[..., 2] = s.clamp(min=0), (-s).clamp(min=0)
    if kind == "e4m3":
        scale = torch.where(scores.isnan(), torch.nan, 1.0)[..., None].contiguous()
        return k.to(torch.float8_e4m3fn).view(torch.uint8), scale
    k[..., 0] = torch.where(scores.isnan(), 3e38, 0.0)
    return k.to(torch.float32 if kind == "f32" else torch.bfloat16), None


def some_scores(g, N, live):
    s = torch.randint(-28, 29, (N,), generator=g, device=DEV) / 4.0         # (exact in e4m3 below 8)
    s = torch.where(s.abs() >= 4, s.round(), s)
    s[torch.randperm(N, generator=g, device=DEV)[live:]] = torch.nan
    return s


def ranking(s):
    order = torch.sort(torch.nan_to_num(s, nan=-1e30), descending=True, stable=True).indices
    nan = s[order].isnan()
    return torch.cat([order[~nan], order[nan]])


def same(a, b):
    return torch.equal(a.nan_to_num(nan=-1e30), b.nan_to_num(nan=-1e30))


@pytest.mark.parametrize("kind,nq,N", [
    ("f32", 3, 3000), ("f32", 200, 3000), ("f32", 1, 40000), ("f32", 3, 40000), ("f32", 160, 20000),
    ("bf16", 1, 5000), ("bf16", 200, 5000), ("bf16", 1, 40000), ("bf16", 4, 40000),
    ("e4m3", 1, 5000), ("e4m3", 1, 40000), ("e4m3", 4, 40000), ("e4m3", 200, 20000)])
@pytest.mark.parametrize("k,live", [(64, 40), (64, 2500), (1024, 1000), (2048, 7)])
def test_nan_ranks_last(kind, nq, N, k, live):
    g = torch.Generator(device=DEV).manual_seed(N + nq + k)
    s = some_scores(g, N, live)
    kI, scale = keys(kind, s[None])
    qI, w = queries(kind, 1, nq)
    pos = torch.full((1, nq), N - 1, device=DEV, dtype=torch.int32)
    pos[0, 0] = N - 301                                                     # (not the last entries)
    for with_scores in (False, True):                                       # (rows in one pass, or read back)
        sel = torch.empty(1, nq, k, device=DEV) if with_scores else None
        idx = api.indexer_topk(qI, w, kI, pos, 1, k, kI_scale=scale, sel_scores=sel)
        for q in sorted({0, nq // 2, nq - 1}):
            v = int(pos[0, q]) + 1
            want = ranking(s[:v])[:k].sort().values
            assert torch.equal(idx[0, q, :len(want)], want.int()), f"query {q}"
            if with_scores:
                assert same(sel[0, q, :len(want)], s[want])
    assert api.device_error() == 0


@pytest.mark.parametrize("live", [70, 20])                                  # (of 2 x 500: more than k = 96, and fewer)
def test_nan_ranks_last_in_the_merge_of_shards(live):
    g = torch.Generator(device=DEV).manual_seed(3)
    n, k = 500, 96
    s = some_scores(g, n, live), some_scores(g, n, live)
    qI, w = queries("f32", 1, 1)
    pos = torch.full((1, 1), 2 * n - 1, device=DEV, dtype=torch.int32)
    ci, cs = torch.empty(2, 1, k, dtype=torch.int32, device=DEV), torch.empty(2, 1, k, device=DEV)
    for r in range(2):
        api.indexer_topk(qI, w, keys("f32", s[r][None])[0], pos, 1, k, idx=ci[r][None], sel_scores=cs[r][None], entry_base=r * n)
    got, _ = api.cp_topk_merge(ci, cs, [0, n], 0)
    assert torch.equal(got[0], ranking(torch.cat(s))[:k].sort().values.int())
    assert api.device_error() == 0
