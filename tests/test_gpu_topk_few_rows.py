"""Top-k of rows up to 32,768 scores in calls of few rows (a CTA of 1,024
threads each) and of more rows than SMs, on the same rows: the k largest of the
GPU's own scores, ties to the lower index, and their scores; every value is
copied or compared, so both must match exactly.

The rows: random scores, few distinct ones, equal ones, ones that rise with the
index, infinite ones, all large ones in the segments that a sample takes (the
bound it gives is then too high), all in one warp's range, and NaN (below every
score)."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
DI = 32


def rows_of(N, seed):
    """[rows, N] fp32."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    j = torch.arange(N, device=DEV)
    a = torch.randn(N, generator=g, device=DEV)
    rows = [a, (a * 2).round(), torch.full_like(a, -0.25), torch.zeros_like(a), j * 0.5 - 77, 100.0 - j * 0.5,
            torch.where((j // 32) % 8 == 0, a.abs() + 1000, a), torch.where((j // 32) % 8 == 0, -a.abs() - 1000, a),
            torch.where(j < N // 32, a.abs() + 9, -a.abs()), torch.where(j % 7 == 0, torch.inf, a),
            torch.where(j % 5 == 0, -torch.inf, a)]
    return torch.stack(rows)


def run(rows, visible, k):
    """Top-k over given scores: a key's two dims are the score's positive and
    negative part, and two heads of weights 1 and -1 read one each."""
    nq, N = rows.shape
    idx = torch.empty(1, nq, k, dtype=torch.int32, device=DEV)
    sel = torch.empty(1, nq, k, device=DEV)
    # (one set of keys a call: every row its own sequence)
    kI = torch.zeros(nq, N, DI, device=DEV)
    kI[..., 0], kI[..., 1] = rows.clamp(min=0), (-rows).clamp(min=0)
    qI = torch.zeros(nq, 1, 2, DI, device=DEV)
    qI[:, 0, 0, 0] = qI[:, 0, 1, 1] = 1.0
    w = torch.tensor([1.0, -1.0], device=DEV).expand(nq, 1, 2).contiguous()
    pos = torch.as_tensor(visible, device=DEV, dtype=torch.int32).view(nq, 1) - 1
    api.indexer_topk(qI, w, kI, pos, 1, k, idx=idx.view(nq, 1, k), sel_scores=sel.view(nq, 1, k))
    return idx[0], sel[0]


def expected(row, v, k):
    s = row[:v]
    # NaN behind everything; stable, so that ties go to the lower index
    order = torch.sort(torch.where(s.isnan(), -torch.inf, s), descending=True, stable=True).indices
    nan = s[order].isnan()
    order = torch.cat([order[~nan], order[nan]])
    pick = order[:k].sort().values
    idx = torch.full((k,), -1, dtype=torch.int32, device=DEV)
    sel = torch.full((k,), -torch.inf, device=DEV)
    idx[:len(pick)] = pick.to(torch.int32)
    sel[:len(pick)] = s[pick]
    return idx, sel


@pytest.mark.parametrize("N,k", [(40, 7), (700, 512), (4096, 1024), (4097, 64), (9001, 1024), (16384, 1024), (16384, 5000),
                                 (16385, 1), (20000, 2048), (32768, 1024), (32768, 32767), (300, 512)])
def test_few_rows_and_many_rows(N, k):
    rows = rows_of(N, N + k)
    inf = rows.isinf()
    rows = torch.where(inf, rows.sign() * 3e38, rows)          # (0 x inf in a dot product is NaN: the largest values instead)
    n = rows.shape[0]
    g = torch.Generator(device=DEV).manual_seed(5)
    visible = torch.randint(1, N + 1, (n,), generator=g, device=DEV)
    visible[: n // 2] = N
    few = run(rows, visible, k)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    many = sms // n + 1
    if n * many * N * DI * 4 > 24 << 30:
        many = 0
    for r in range(n):
        want = expected(rows[r], int(visible[r]), k)
        assert torch.equal(few[0][r], want[0]), f"row {r}"
        assert torch.equal(few[1][r], want[1]), f"scores of row {r}"
    if many:
        idx, sel = run(rows.repeat(many, 1), visible.repeat(many), k)
        assert torch.equal(idx, few[0].repeat(many, 1)) and torch.equal(sel, few[1].repeat(many, 1))
    assert api.device_error() == 0


@pytest.mark.parametrize("N,k,live", [(3000, 100, 80), (16384, 1024, 9000), (16384, 1024, 1000), (32768, 8, 4)])
def test_nan_scores_rank_last(N, k, live):
    """A head of infinite weight: keys that it sees score infinity, the others
    0 x inf.  The `live` ones come first, then the NaN ones by index."""
    g = torch.Generator(device=DEV).manual_seed(N + live)
    alive = torch.zeros(N, dtype=torch.bool, device=DEV)
    alive[torch.randperm(N, generator=g, device=DEV)[:live]] = True
    kI = torch.zeros(1, N, DI, device=DEV)
    kI[0, alive, 0] = 1.0
    qI = torch.zeros(1, 1, 2, DI, device=DEV)
    qI[..., 0] = 1.0
    w = torch.tensor([[[float("inf"), 0.0]]], device=DEV)
    idx = api.indexer_topk(qI, w, kI, torch.tensor([[N - 1]], device=DEV, dtype=torch.int32), 1, k)
    want, _ = expected(torch.where(alive, torch.inf, torch.nan), N, k)
    assert torch.equal(idx[0, 0], want)
    assert api.device_error() == 0
