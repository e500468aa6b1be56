"""NaN and infinities in what a tree node sees: its output holds NaN where the
definition does in IEEE arithmetic, however the call splits the keys over CTAs.

A NaN score makes the whole row NaN; a key with an infinite value scores +inf
(inf - inf: the row is NaN) or -inf (weight 0, but 0 x inf is NaN in that dim).
The other values are the oracle's, within the tolerances of tests/helpers.py."""

import numpy as np
import pytest
import torch

from long_context_compressed_overlapped_b200 import api
from tests import tree_reference as R
from tests.helpers import check_close, npy
from tests.test_gpu_tree import DEV, HEADS16, SMALL, TC, attn_case, name_of, run_attn

pytestmark = pytest.mark.gpu
DIM = 5                                                     # (not a rope dim in any of the shapes)


def check_with_nan(got, ref, dtype, what):
    assert (np.isnan(got) == np.isnan(ref)).all(), f"{what}: NaN in {np.isnan(got).sum()} places, {np.isnan(ref).sum()} expected"
    check_close(np.where(np.isnan(got), 0.0, got), np.where(np.isnan(ref), 0.0, ref), dtype, what)


TREES = [
    # few nodes over many keys (their tiles are split over the SMs), and many nodes over few (one CTA a node)
    ("hca", 1, 3, [29998], "chain", 16, 16, 0),
    ("hca", 2, 40, [2990, 2990], "chain", 16, 16, 0),
    ("csa", 2, 6, [9002, 9006], "wide", 4, 128, 1000),
    ("csa", 3, 60, [602, 602, 602], "chain", 4, 16, 64),
]


@pytest.mark.parametrize("heads", [SMALL, TC, HEADS16], ids=["f32", "tc", "16h"])
@pytest.mark.parametrize("case", TREES)
@pytest.mark.parametrize("poison", ["entry", "window", "path", "draft", "query", "infinite entry", "infinite entries"])
def test_tree_nodes(case, heads, poison):
    kind, B, T, pos, shape, m, w, k = case
    s = attn_case(kind, B, T, pos, shape, m, w, k, seed=21, **heads)
    nan = float("nan")
    if poison == "entry":
        s["kv"][0, 7, DIM] = nan
    elif poison == "window":
        s["win"][0, (pos[0] - 1) % w, DIM] = nan
    elif poison == "path":
        s["kv_raw"][0, 1, DIM] = nan
    elif poison == "draft":
        s["draft"][0, :, DIM] = nan
    elif poison == "query":
        s["q"][0, 1, 2, DIM] = nan
    elif poison == "infinite entry":
        s["kv"][0, 7, DIM] = float("inf")
    else:
        s["kv"][0, :130, DIM] = float("inf")                # whole tiles: a split may hold no others
    if kind == "csa" and "entr" in poison:
        n = 1 if poison != "infinite entries" else min(130, k - 8)
        s["idx"][0, :, :n] = torch.arange(7, 7 + n, device=DEV, dtype=torch.int32) % 130
    out = run_attn(s)
    sel = npy(s["idx"]) if kind == "csa" else None
    seen = 0
    for b in range(B):
        for i in sorted({0, 1, 2, T // 2, T - 1}):
            with np.errstate(invalid="ignore"):
                ref = R.attend_node(kind, b, i, s["parents"], s["pos"], s["q"], s["kv"], s["win"], s["kv_raw"], s["draft"],
                                    s["sinks"], m=m, w=w, r=s["r"], q_gain=s["q_gain"], kv_gain=s["kv_gain"],
                                    sel=None if sel is None else sel[b, i])
            check_with_nan(npy(out[b, i]), ref, name_of(s["q"].dtype), f"node {b},{i}")
            seen += np.isnan(ref).sum()
    assert seen > 0 and api.device_error() == 0
