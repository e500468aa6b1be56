"""Drafted entries beside committed ones where either score NaN: a NaN ranks
below every other score, ties go to the lower index (the committed entry)."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api
from tests.test_gpu_nan_rank import DEV, keys, queries, ranking, some_scores
from tests.test_gpu_tree import SMALL, attn_case, run_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("v,k,live,drafted", [
    (20, 8, 5, [0.5, 3.0]),                      # three candidates are NaN: both drafted entries come in
    (20, 8, 7, [-5.0, 3.0]),                     # one is: the better of them does
    (20, 8, 8, [-6.5, -6.75]),                   # none is
    (20, 8, 5, [float("nan"), 1.0]),
    (20, 8, 5, [float("nan"), float("nan")]),    # NaN against NaN: the lower index, the committed one
    (6, 8, 3, [float("nan"), float("nan")]),     # free places take them all the same
    (7, 8, 3, [1.0, float("nan")]),              # the one free place, and no further
    (40000, 64, 30, [0.25, -1.0]), (40000, 64, 63, [-6.5, float("nan")]), (20000, 64, 20, [0.25, -1.0])])
@pytest.mark.parametrize("sign", [0, 1])
def test_drafted_entries_among_nan(v, k, live, drafted, sign):
    T, m = 9, 4
    s = attn_case("csa", 1, T, [m * v], "chain", m, 0, 1, seed=1, **SMALL)
    s["draft"].normal_()
    g = torch.Generator(device=DEV).manual_seed(v + live)
    N = s["N"]
    score = some_scores(g, N, N)
    score[:v] = some_scores(g, v, live)
    if drafted[0] == -6.5:
        score[:v] = score[:v].abs()
    own = torch.zeros(T, device=DEV)
    own[3], own[7] = drafted[0], drafted[1]
    qI, w = queries("f32", 1, T)
    if sign:
        w[..., :2] *= -1                                                    # the other NaN, if signs differ
    idx = torch.empty(1, T, k, dtype=torch.int32, device=DEV)
    run_attn(s, k=k, qI=qI, wI=w, kI=keys("f32", score[None])[0], draft_kI=keys("f32", own[None])[0], idx_out=idx)
    for i in range(T):
        mine = [j for j in (3, 7) if j <= i]
        names = torch.cat([torch.arange(v, device=DEV), torch.tensor([N + j for j in mine], device=DEV, dtype=torch.int64)])
        all_scores = torch.cat([score[:v], own[mine]])
        want = names[ranking(all_scores)[:k]].sort().values.int()
        assert torch.equal(idx[0, i, :len(want)], want), f"node {i}"
        assert (idx[0, i, len(want):] == -1).all()
    assert api.device_error() == 0
