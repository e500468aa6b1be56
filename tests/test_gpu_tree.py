"""tree_compress and compressed_attn_tree against the oracle's decode steps
along each node's own path.

Tolerances are the path's (tests/helpers.py): fp32 max-abs 1e-5; bf16 max-abs
2e-2 and relative L2 5e-3.  The bf16 path rounds the finished queries, the
drafted window rows, the weights and the output once each (split partials are
fp32), every rounding at most half a step: 2^-8 relative, and over a binade's
values 1.7e-3 rms.  All four at that rms in quadrature are 3.4e-3."""

import numpy as np
import pytest
import torch

from long_context_compressed_overlapped_b200 import api, synth
from oracle import csahca_oracle as O
from tests import tree_reference as R
from tests.helpers import check_close, npy

pytestmark = pytest.mark.gpu
DEV = "cuda"
TC = dict(dt=torch.bfloat16, H=64, d=512, r=64)
SMALL = dict(dt=torch.float32, H=4, d=64, r=16)
HEADS16 = dict(dt=torch.bfloat16, H=16, d=128, r=64)


def name_of(dt):
    return "f32" if dt == torch.float32 else "bf16"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---------------------------------------------------------------- compress ----

def compress_case(kind, dt, B, T, c, m, pos, shape, seed=0):
    g = gen(seed)
    S, Rn = (4, 2 * m) if kind == "csa" else (2, m)
    std = c ** -0.5 if dt == torch.float32 else 1.0
    return dict(kind=kind, m=m, parents=R.parents_of(shape, B, T, seed), pos=pos,
                streams=tuple((torch.randn(B, T, c, generator=g, device=DEV) * (std if i < S // 2 else 1)).to(dt) for i in range(S)),
                ring=torch.randn(B, Rn, S, c, generator=g, device=DEV).mul(std).to(dt),
                bias_a=0.1 * torch.randn(m, c, generator=g, device=DEV),
                bias_b=0.1 * torch.randn(m, c, generator=g, device=DEV) if S == 4 else None,
                gain=1 + 0.1 * torch.randn(c, generator=g, device=DEV))


def run_compress(s, norm=True, r=0, **kw):
    return api.tree_compress(s["kind"], s["streams"], s["ring"], R.ints(s["pos"], DEV), R.ints(s["parents"], DEV), s["bias_a"],
                             s["m"], bias_b=s["bias_b"], gain=s["gain"], rms_norm=norm, rope_dims=r, **kw)


def oracle_entry(s, b, i, norm, r):
    biases = (npy(s["bias_a"]), None if s["bias_b"] is None else npy(s["bias_b"]))
    return R.entry_of_node(s["kind"], b, i, s["parents"], s["pos"], s["streams"], s["ring"], biases, s["m"],
                           gain=npy(s["gain"]), r=r, normalize=norm)


@pytest.mark.parametrize("kind,dt,B,T,c,m,pos,shape,norm,r", [
    ("csa", torch.bfloat16, 3, 13, 512, 4, [1048571, 0, 5], "wide", True, 64),
    ("csa", torch.bfloat16, 2, 64, 512, 4, [262143, 2], "chain", True, 64),         # tokens all drafted
    ("csa", torch.bfloat16, 2, 9, 128, 4, [77, 3], "padded", False, 0),
    ("csa", torch.float32, 2, 7, 64, 4, [0, 510], "wide", True, 16),
    ("csa", torch.float32, 1, 5, 36, 1, [9], "flat", True, 10),                      # every token a block
    ("csa", torch.float32, 1, 40, 32, 16, [31], "chain", True, 0),
    ("csa", torch.bfloat16, 1, 3, 1024, 4, [1021], "chain", True, 512),
    ("hca", torch.bfloat16, 4, 32, 512, 128, [262142, 127, 126, 100], "chain", True, 64),
    ("hca", torch.bfloat16, 2, 6, 512, 128, [1048575, 255], "padded", True, 64),
    ("hca", torch.float32, 2, 5, 64, 16, [15, 47], "flat", True, 16),
    ("hca", torch.float32, 1, 2, 32, 512, [511], "flat", True, 0),
])
def test_compress(kind, dt, B, T, c, m, pos, shape, norm, r):
    s = compress_case(kind, dt, B, T, c, m, pos, shape)
    out = torch.full((B, T, c), 7.0, dtype=dt, device=DEV)
    run_compress(s, norm, r, out=out)
    done = 0
    for b in range(B):
        for i in range(T):
            entry = oracle_entry(s, b, i, norm, r)
            if entry is None:
                assert (out[b, i] == 7).all(), (b, i)
            else:
                check_close(npy(out[b, i]), entry[2], name_of(dt), f"node {b},{i}")
                done += 1
    assert done > 0 and api.device_error() == 0


def test_compress_e4m3_keys_are_the_decode_compressors():
    """Codes and scales of a drafted indexer key = those that decode_compress
    stores once the same tokens are committed."""
    B, T, dI, m, d = 2, 8, 128, 4, 64
    pos = [1021, 4]
    s = compress_case("csa", torch.bfloat16, B, T, dI, m, pos, "chain", seed=4)
    codes = torch.zeros(B, T, dI, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(B, T, 1, device=DEV)
    run_compress(s, False, 0, out=codes, out_scale=scale)
    ring, iring = torch.zeros(B, 2 * m, 4, d, dtype=torch.bfloat16, device=DEV), s["ring"].clone()
    kv = torch.zeros(B, 300, d, dtype=torch.bfloat16, device=DEV)
    kI, kI_scale = torch.zeros(B, 300, dI, dtype=torch.uint8, device=DEV), torch.zeros(B, 300, 1, device=DEV)
    z = torch.zeros(B, d, dtype=torch.bfloat16, device=DEV)
    seen = 0
    for i in range(T):
        p = R.ints([x + i for x in pos], DEV)
        api.decode_compress("csa", p, (z, z, z, z), ring, kv, m=m, bias_a=torch.zeros(m, d, device=DEV),
                            bias_b=torch.zeros(m, d, device=DEV), istreams=tuple(x[:, i].contiguous() for x in s["streams"]),
                            ibias_a=s["bias_a"], ibias_b=s["bias_b"], iring=iring, kI=kI, kI_scale=kI_scale)
        for b in range(B):
            if (pos[b] + i + 1) % m == 0:
                e = (pos[b] + i + 1) // m - 1
                # both pool in fp32, in different orders: the scale to a few ulps, a code at most one step off
                assert abs(float(scale[b, i, 0] / kI_scale[b, e, 0]) - 1) <= 16 * 2.0**-23
                a, c = codes[b, i].view(torch.float8_e4m3fn).float(), kI[b, e].view(torch.float8_e4m3fn).float()
                assert (a - c).abs().le(torch.maximum(a.abs(), c.abs()) * 2.0**-3 + 2.0**-9).all()
                assert (codes[b, i] == kI[b, e]).float().mean() >= 0.99
                seen += 1
    assert seen == 4


def test_compress_infinite_logits():
    """A token whose logit is -inf has no weight; one that hides a NaN row
    behind another branch changes nothing."""
    s = compress_case("csa", torch.float32, 1, 4, 32, 4, [4], "chain", seed=1)
    s["streams"][2][0, 1] = float("-inf")
    s["ring"][0, :, 3] = float("-inf")                                              # zb of the preceding block
    got = run_compress(s, False, 0)[0, 3]
    z = npy(s["streams"][2][0, :4]) + npy(s["bias_a"])
    e = np.exp(z - z.max(0))
    check_close(npy(got), (e * npy(s["streams"][0][0, :4])).sum(0) / e.sum(0), "f32")


# --------------------------------------------------------------- attention ----

def attn_case(kind, B, T, pos, shape, m, w, k=0, N=None, dt=None, H=None, d=None, r=None, seed=0, drafted=True):
    g = gen(seed)
    N = max((max(pos) + T + 1) // m, 1) if N is None else N
    std = d ** -0.5 if dt == torch.float32 else 1.0

    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)
    s = dict(kind=kind, m=m, w=w, r=r, N=N, parents=R.parents_of(shape, B, T, seed), pos=list(pos), q=normal(B, T, H, d),
             kv=normal(B, N, d), win=normal(B, w, d) if w else None, kv_raw=normal(B, T, d),
             draft=normal(B, T, d) if drafted else None, sinks=torch.randn(H, generator=g, device=DEV),
             q_gain=1 + 0.1 * torch.randn(d, generator=g, device=DEV), kv_gain=1 + 0.1 * torch.randn(d, generator=g, device=DEV))
    # what no node may see holds NaN: entries that are not committed, ring slots not yet written
    for b in range(B):
        s["kv"][b, max(0, pos[b]) // m:] = float("nan")
        if w:
            for p in range(w):
                if p >= pos[b]:
                    s["win"][b, p] = float("nan")
        for i in range(T):
            if R.path_of(s["parents"][b], i) is None:
                for n in ("q", "kv_raw", "draft"):
                    if s[n] is not None:
                        s[n][b, i] = float("nan")
            elif s["draft"] is not None and (R.node_position(s["parents"][b], pos[b], i) + 1) % m:
                s["draft"][b, i] = float("nan")                                     # it completes no entry
    if kind == "csa":
        rng = np.random.RandomState(seed + 1)
        idx = np.full((B, T, k), -1, np.int64)
        for b in range(B):
            v = min(N, max(0, pos[b]) // m)
            for i in range(T):
                path = R.path_of(s["parents"][b], i)
                own = [] if path is None or not drafted else [N + j for o, j in enumerate(path) if (pos[b] + o + 1) % m == 0]
                pick = np.sort(rng.permutation(v)[:max(0, k - len(own))])
                row = list(pick) + own
                idx[b, i, :len(row[:k])] = row[:k]
        s["idx"] = R.ints(idx.tolist(), DEV)
    return s


def run_attn(s, **kw):
    kw = dict(dict(draft=s["draft"], q_gain=s["q_gain"], kv_gain=s["kv_gain"]), **kw)
    if s["kind"] == "csa" and "qI" not in kw:
        kw.setdefault("idx_in", s["idx"])
    return api.compressed_attn_tree(s["kind"], s["q"], R.ints(s["pos"], DEV), R.ints(s["parents"], DEV), s["kv"], s["win"],
                                    s["kv_raw"], s["sinks"], m=s["m"], rope_dims=s["r"], **kw)


def check_attn(s, out, idx=None, nodes=None, left=7.0, **kw):
    B, T = s["q"].shape[:2]
    sel = npy(s["idx"] if idx is None else idx) if s["kind"] == "csa" else None
    for b in range(B):
        for i in range(T):
            if nodes is not None and (b, i) not in nodes:
                continue
            ref = R.attend_node(s["kind"], b, i, s["parents"], s["pos"], s["q"], s["kv"], s["win"], s["kv_raw"], s["draft"],
                                s["sinks"], m=s["m"], w=s["w"], r=s["r"], q_gain=s["q_gain"], kv_gain=s["kv_gain"],
                                sel=None if sel is None else sel[b, i], **kw)
            if ref is None:
                assert (out[b, i] == left).all(), f"node {b},{i} is none"
            else:
                check_close(npy(out[b, i]), ref, name_of(s["q"].dtype), f"node {b},{i}")


ATTN = [
    # kind, B, T, pos, shape, m, w, k
    ("hca", 1, 1, [300], "chain", 128, 128, 0),
    ("hca", 3, 7, [2047, 126, 0], "wide", 128, 128, 0),          # a completed block, nothing committed
    ("hca", 2, 64, [1000, 3], "chain", 16, 128, 0),
    ("hca", 2, 9, [5000, 4999], "padded", 16, 16, 0),
    ("hca", 2, 5, [640, 255], "flat", 1, 130, 0),                # whole tiles only, two window tiles
    ("hca", 2, 3, [64, 0], "chain", 128, 0, 0),                  # no window: rows without any key
    ("csa", 1, 1, [4096], "chain", 4, 128, 1024),
    ("csa", 3, 6, [9000, 10, 0], "wide", 4, 128, 200),
    ("csa", 2, 17, [600, 601], "padded", 4, 16, 64),
    ("csa", 2, 64, [3, 70], "chain", 4, 128, 5),
    ("csa", 1, 4, [37], "flat", 1, 0, 1),
]


@pytest.mark.parametrize("heads", [SMALL, TC, HEADS16], ids=["f32", "tc", "16h"])
@pytest.mark.parametrize("case", ATTN)
def test_attention(case, heads):
    kind, B, T, pos, shape, m, w, k = case
    s = attn_case(kind, B, T, pos, shape, m, w, k, **heads)
    out = torch.full_like(s["q"], 7.0)
    got = run_attn(s, out=out)
    assert got is out
    check_attn(s, out)
    assert api.device_error() == 0


@pytest.mark.parametrize("B,T,pos,kind", [(2, 40, [70000, 69999], "hca"), (1, 2, [130000], "hca"), (4, 64, [9001, 9000, 8999, 40], "csa")])
def test_attention_many_items(B, T, pos, kind):
    """Several items a CTA (one split each), and many splits of few nodes."""
    s = attn_case(kind, B, T, pos, "wide", 4 if kind == "csa" else 16, 128, 300 if kind == "csa" else 0, **TC)
    out = run_attn(s, out=torch.full_like(s["q"], 7.0))
    rng = np.random.RandomState(0)
    nodes = {(b, i) for b in range(B) for i in {0, T - 1, *rng.randint(0, T, 5).tolist()}}
    check_attn(s, out, nodes=nodes)
    assert api.device_error() == 0


@pytest.mark.parametrize("heads", [SMALL, HEADS16, dict(dt=torch.float32, H=5, d=512, r=512)], ids=["f32", "16h", "f32-512"])
def test_attention_on_cuda_cores_in_splits(heads):
    """Few nodes over many keys: the splits of the CUDA-core path and their join."""
    for kind, pos, k in (("hca", [5000, 4700], 0), ("csa", [40000, 9], 4000)):
        s = attn_case(kind, 2, 3, pos, "padded", 1 if kind == "hca" else 4, 16, k, seed=8, **heads)
        out = run_attn(s, out=torch.full_like(s["q"], 7.0))
        check_attn(s, out)
    assert api.device_error() == 0


@pytest.mark.parametrize("heads", [SMALL, TC], ids=["f32", "tc"])
def test_entries_past_the_capacity_are_no_keys(heads):
    """A full cache: what the path completes beyond N_cap is not stored by a
    decode step, so no node sees it, and the indexer does not offer it."""
    s = attn_case("hca", 1, 9, [60], "chain", 4, 16, N=16, seed=5, **heads)             # entries 15 | 16, 17 are past it
    out = run_attn(s)
    check_attn(s, out)
    s = attn_case("csa", 1, 9, [60], "chain", 4, 16, 20, N=16, seed=5, **heads)
    g, dt = gen(3), heads["dt"]
    qI, wI = whole(g, 1, 3, dt, 1, 9, 2, 32), whole(g, 1, 4, torch.float32, 1, 9, 2)
    kI, dk = whole(g, 0, 3, dt, 1, 16, 32), whole(g, 4, 5, dt, 1, 9, 32)
    idx = torch.empty(1, 9, 20, dtype=torch.int32, device=DEV)
    run_attn(s, k=20, qI=qI, wI=wI, kI=kI, draft_kI=dk, idx_out=idx)
    got = npy(idx)[0]
    assert (got[2] == list(range(15)) + [-1] * 5).all() and (got[8] == list(range(15)) + [16 + 3] + [-1] * 4).all()


def test_nan_scores_stay_in_the_row():
    """Drafted keys of NaN rank last; no row of the selection runs over."""
    s = attn_case("csa", 1, 12, [2], "chain", 1, 0, 1, seed=1, **SMALL)
    s["draft"].normal_()
    qI, wI = torch.ones(1, 12, 2, 32, device=DEV), torch.ones(1, 12, 2, device=DEV)
    kI, dk = torch.ones(1, s["N"], 32, device=DEV), torch.full((1, 12, 32), float("nan"), device=DEV)
    idx = torch.full((1, 13, 3), -9, dtype=torch.int32, device=DEV)
    run_attn(s, k=3, qI=qI, wI=wI, kI=kI, draft_kI=dk, idx_out=idx[:, :12])
    assert (idx[0, 12] == -9).all() and (idx[0, :12, :2] == torch.tensor([0, 1], device=DEV)).all()
    assert (idx[0, :12, 2] >= s["N"]).all()                                            # the one free place: a drafted entry
    assert api.device_error() == 0


@pytest.mark.parametrize("heads", [SMALL, TC], ids=["f32", "tc"])
def test_without_drafted_entries_gains_or_norms(heads):
    for kind, k in (("hca", 0), ("csa", 30)):
        s = attn_case(kind, 2, 6, [254, 40], "wide", 4, 16, k, drafted=False, seed=3, **heads)
        s["q_gain"] = s["kv_gain"] = None
        out = run_attn(s, q_norm=False, kv_norm=False, scale=0.125, out=torch.full_like(s["q"], 7.0))
        B, T = s["q"].shape[:2]
        for b in range(B):
            for i in range(T):
                # (the reference's HCA visibility counts drafted entries: keep the committed ones only)
                t = R.node_position(s["parents"][b], s["pos"][b], i)
                path = R.path_of(s["parents"][b], i)
                v = s["pos"][b] // s["m"]
                comp = npy(s["kv"][b, :v]) if kind == "hca" else npy(s["kv"][b, s["idx"][b, i][s["idx"][b, i] >= 0].long()])
                wp = O.window_positions(t, 16)
                win = [npy(s["win"][b, p % 16]) if p < s["pos"][b] else O.finish_rows(npy(s["kv_raw"][b, path[p - s["pos"][b]]]), p, None, s["r"], normalize=False) for p in wp]
                qf = O.finish_rows(npy(s["q"][b, i]), t, None, s["r"], normalize=False)
                ref = O.attend_query(qf, np.concatenate([comp, np.stack(win)]), npy(s["sinks"]), t, s["r"], 0.125)
                check_close(npy(out[b, i]), ref, name_of(s["q"].dtype), f"{kind} {b},{i}")


@pytest.mark.parametrize("heads", [SMALL, TC], ids=["f32", "tc"])
@pytest.mark.parametrize("T", [3, 64])
def test_infinite_sinks(heads, T):
    """A sink of -inf is no sink; one of +inf takes all the weight."""
    s = attn_case("hca", 2, T, [700, 0], "chain", 128, 0, **heads)
    s["sinks"][0], s["sinks"][1] = float("-inf"), float("inf")
    out = run_attn(s)
    assert torch.isfinite(out).all() and (out[:, :, 1] == 0).all()
    assert (out[1, :, 0] == 0).all()                                                # neither key nor sink
    s["sinks"][1] = 0.0
    ref = R.attend_node("hca", 0, 0, s["parents"], s["pos"], s["q"], s["kv"], None, s["kv_raw"], s["draft"], s["sinks"], m=128, w=0,
                        r=s["r"], q_gain=s["q_gain"], kv_gain=s["kv_gain"])
    check_close(npy(out[0, 0, 0]), ref[0], name_of(s["q"].dtype))
    check_close(npy(out[0, 0, 2:]), ref[2:], name_of(s["q"].dtype))


@pytest.mark.parametrize("heads", [SMALL, TC], ids=["f32", "tc"])
def test_selection_with_holes_and_bad_entries(heads):
    """-1 anywhere in idx_in is skipped; an index past the drafted rows is
    skipped and reported."""
    s = attn_case("csa", 1, 3, [2000], "chain", 4, 16, 150, **heads)
    s["idx"][0, :, 3:20] = -1
    s["idx"][0, 1, 100:] = -1
    out = run_attn(s)
    check_attn(s, out)
    assert api.device_error() == 0
    clean = s["idx"].clone()
    s["idx"][0, 2, 5] = s["N"] + 3
    s["idx"][0, 2, 6] = 2**31 - 1
    out = run_attn(s)
    assert api.device_error() == 2
    check_attn(s, out, idx=clean)


@pytest.mark.parametrize("heads", [SMALL, TC], ids=["f32", "tc"])
def test_an_entry_named_twice_is_two_keys(heads):
    s = attn_case("csa", 1, 3, [2000], "chain", 4, 16, 150, **heads)
    s["idx"][0, :, 70:90] = s["idx"][0, :, 10:30].clone()
    s["idx"][0, 1] = s["idx"][0, 1, 3]
    out = run_attn(s)
    check_attn(s, out)
    assert api.device_error() == 0


@pytest.mark.parametrize("heads", [64, 5])
def test_rows_past_32_bit_offsets(heads):
    """Selected rows at the end of a 6 GB cache: the same bits as from a cache
    that holds those rows alone."""
    B, N, tail, T, k = 2, 3_000_000, 5000, 3, 256
    g = gen(12)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV).bfloat16()
    kv = torch.zeros(B, N, 512, device=DEV, dtype=torch.bfloat16)
    kv[:, -tail:] = normal(B, tail, 512)
    args = (normal(B, 16, 512), normal(B, T, 512), torch.randn(heads, generator=g, device=DEV))
    q, draft, parents = normal(B, T, heads, 512), normal(B, T, 512), R.ints([[-1, 0, 1]] * B, DEV)
    idx = torch.stack([torch.randperm(tail, generator=g, device=DEV)[:k].sort().values for _ in range(B * T)]).view(B, T, k).int()
    pos = R.ints([4 * N - 1000] * B, DEV)
    kw = dict(m=4, rope_dims=64, draft=draft)
    want = api.compressed_attn_tree("csa", q, pos, parents, kv[:, -tail:].contiguous(), *args, idx_in=idx, **kw)
    got = api.compressed_attn_tree("csa", q, pos, parents, kv, *args, idx_in=idx + (N - tail), **kw)
    assert torch.equal(got, want) and got.any() and api.device_error() == 0


def test_bad_parent_is_reported():
    s = attn_case("hca", 1, 5, [300], "chain", 128, 16, **SMALL)
    s["parents"][0][2] = 2                                                          # its own parent: a walk that must end
    out = run_attn(s, out=torch.full_like(s["q"], 7.0))
    assert api.device_error() == 2
    s["parents"][0][2:] = [R.NONE] * 3
    check_attn(s, out)
    c = compress_case("hca", torch.float32, 1, 5, 32, 4, [3], "chain")
    c["parents"][0][1] = 63
    got = run_compress(c, out=torch.full((1, 5, 32), 7.0, device=DEV))
    assert api.device_error() == 2
    assert (got[0, 1:] == 7).all() and (got[0, 0] != 7).any()


def test_inactive_sequences_are_left_alone():
    s = attn_case("hca", 3, 4, [500, 500, 500], "chain", 128, 16, **TC)
    s["pos"][1] = -1
    out = run_attn(s, out=torch.full_like(s["q"], 7.0))
    assert (out[1] == 7).all()
    check_attn(s, out)
    assert api.device_error() == 0


def pack_fp8(rows, r):
    """FP8 KV rows of bf16 rows, and the rows they stand for; a row with NaN in
    it becomes NaN codes, NaN RoPE dims and NaN scales."""
    bad = rows.isnan().any(-1)
    packed = synth.pack_kv_rows_fp8(torch.where(bad[..., None], torch.zeros_like(rows), rows), r)
    packed[bad] = 0xff                                                              # e4m3 and bf16 and fp32 NaN alike
    codes, scales, rope = synth.unpack_kv_rows_fp8(packed, rows.shape[-1], r)
    body = codes.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 64)) * scales[..., None]
    return packed, torch.cat([body.flatten(-2), rope.float()], -1)


@pytest.mark.parametrize("r", [64, 128])
@pytest.mark.parametrize("case", [("hca", 3, 7, [2047, 126, 0], "wide", 128, 128, 0), ("hca", 2, 40, [9000, 77], "padded", 16, 128, 0),
                                  ("hca", 2, 3, [2047, 600], "chain", 16, 16, 0),        # (few nodes: widened in the gather)
                                  ("csa", 3, 6, [9000, 10, 0], "wide", 4, 128, 200), ("csa", 1, 64, [5000], "chain", 4, 16, 70)])
def test_fp8_kv_rows(case, r):
    """FP8 KV caches and drafted entries, against the oracle on the rows they
    stand for."""
    kind, B, T, pos, shape, m, w, k = case
    s = attn_case(kind, B, T, pos, shape, m, w, k, seed=4, dt=torch.bfloat16, H=64, d=512, r=r)
    ref = dict(s)
    s["kv"], ref["kv"] = pack_fp8(s["kv"], r)
    s["draft"], ref["draft"] = pack_fp8(s["draft"], r)
    out = run_attn(s, out=torch.full_like(s["q"], 7.0))
    check_attn(ref, out)
    assert api.device_error() == 0


def test_compress_fp8_kv_rows_are_the_decode_compressors():
    B, T, d, m, r = 2, 9, 512, 4, 64
    pos = [1021, 4]
    s = compress_case("csa", torch.bfloat16, B, T, d, m, pos, "chain", seed=12)
    rows = run_compress(s, True, r, kv_fp8=True)
    ring, kv = s["ring"].clone(), torch.zeros(B, 300, 640, dtype=torch.uint8, device=DEV)
    seen = 0
    for i in range(T):
        api.decode_compress("csa", R.ints([x + i for x in pos], DEV), tuple(x[:, i].contiguous() for x in s["streams"]), ring, kv, m=m,
                            bias_a=s["bias_a"], bias_b=s["bias_b"], kv_gain=s["gain"], rope_dims=r)
        for b in range(B):
            if (pos[b] + i + 1) % m == 0:
                e = (pos[b] + i + 1) // m - 1
                a, c = synth.unpack_kv_rows_fp8(rows[b, i], d, r), synth.unpack_kv_rows_fp8(kv[b, e], d, r)
                # pooled in fp32 in different orders: scales to a few ulps, codes and RoPE dims to a step, nearly all equal
                assert ((a[1] / c[1] - 1).abs() <= 32 * 2.0**-23).all()
                fa, fc = (x[0].contiguous().view(torch.float8_e4m3fn).float() for x in (a, c))
                assert (fa - fc).abs().le(torch.maximum(fa.abs(), fc.abs()) * 2.0**-3 + 2.0**-9).all()
                assert (a[0] == c[0]).float().mean() >= 0.98
                assert (a[2].float() - c[2].float()).abs().le(c[2].float().abs() * 2.0**-7 + 1e-6).all()
                seen += 1
            else:
                assert (rows[b, i] == 0).all()
    assert seen == 4


def whole(g, lo, hi, dt, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).to(dt)


@pytest.mark.parametrize("keys", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("B,T,pos,shape,k", [(2, 9, [4099, 30], "wide", 256), (1, 1, [2000], "chain", 512), (1, 33, [150], "chain", 40),
                                             (2, 5, [0, 3], "flat", 3), (1, 6, [140000], "padded", 64)])
def test_indexer_selects_committed_and_drafted(keys, B, T, pos, shape, k):
    """Scores are exact (small whole numbers), so the selection must be the
    oracle's to the last tie; and the output is the attention over it."""
    heads = SMALL if keys == "f32" else TC
    s = attn_case("csa", B, T, pos, shape, 4, 16, 1, seed=2, **heads)
    for b in range(B):                                                              # any drafted entry may be asked for
        s["draft"][b] = torch.randn(T, heads["d"], device=DEV).to(heads["dt"])
    g = gen(11)
    dt = torch.float32 if keys == "f32" else torch.bfloat16
    HI, dI = (64, 128) if keys != "f32" else (2, 32)
    qI, wI = whole(g, -3, 3, dt, B, T, HI, dI), whole(g, -4, 4, torch.float32, B, T, HI) / 4
    kI, dk = whole(g, -3, 3, dt, B, s["N"], dI), whole(g, -5, 5, dt, B, T, dI)
    kw, ref_k, ref_d = {}, kI, dk
    if keys == "e4m3":
        code = lambda x: x.float().to(torch.float8_e4m3fn).view(torch.uint8)       # noqa: E731
        one = lambda x: torch.full((*x.shape[:2], 1), 0.5, device=DEV)             # noqa: E731
        kw = dict(kI_scale=one(kI), draft_kI_scale=one(dk))
        ref_k, ref_d = kI.float() / 2, dk.float() / 2
        kI, dk = code(kI), code(dk)
    idx = torch.full((B, T, k), -9, dtype=torch.int32, device=DEV)
    out = run_attn(s, k=k, qI=qI, wI=wI, kI=kI, draft_kI=dk, idx_out=idx, out=torch.full_like(s["q"], 7.0), **kw)
    got, mixed = npy(idx), 0
    for b in range(B):
        for i in range(T):
            want = R.select_node(b, i, s["parents"], s["pos"], qI, wI, ref_k, ref_d, 4, k, s["N"])
            assert (got[b, i] == want).all(), f"node {b},{i}"
            mixed += (want >= s["N"]).sum()
    if T > 8:
        assert mixed > 0
    nodes = {(0, 0), (B - 1, T - 1), (0, T // 2)}
    check_attn(s, out, idx=idx, nodes=nodes)
    again = run_attn(s, k=k, qI=qI, wI=wI, kI=kI, draft_kI=dk, out=torch.full_like(s["q"], 7.0), **kw)   # selection in the workspace
    assert torch.equal(again, out) and api.device_error() == 0
    plain = torch.empty_like(idx)
    run_attn(s, k=k, qI=qI, wI=wI, kI=kI, idx_out=plain, **{n: v for n, v in kw.items() if n == "kI_scale"})
    for b in range(B):
        want = R.select_node(b, 0, s["parents"], s["pos"], qI, wI, ref_k, None, 4, k, s["N"])
        assert (npy(plain)[b, 0] == want).all()


def test_one_node_is_a_decode_step():
    """T = 1 after decode_compress of the same token: the decode call's output."""
    B, m, w, d, r, H, k = 2, 4, 128, 512, 64, 64, 100
    pos = [4095, 2001]
    s = attn_case("csa", B, 1, pos, "chain", m, w, k, seed=6, **TC)
    s["kv"] = torch.randn(B, s["N"], d, device=DEV).bfloat16()
    c = compress_case("csa", torch.bfloat16, B, 1, d, m, pos, "chain", seed=6)
    c["gain"] = s["kv_gain"]
    s["draft"] = run_compress(c, True, r)
    s["idx"] = R.ints([[list(range(0, 4 * k, 4))], [list(range(0, 4 * k, 4))]], DEV)
    s["idx"][0, 0, -1] = s["N"]                                                     # sequence 0 completes entry 1023
    tree = run_attn(s)
    kv, win, ring = s["kv"].clone(), s["win"].clone(), c["ring"].clone()
    p = R.ints(pos, DEV)
    api.decode_compress("csa", p, tuple(x[:, 0].contiguous() for x in c["streams"]), ring, kv, m=m, bias_a=c["bias_a"],
                        bias_b=c["bias_b"], kv_raw=s["kv_raw"][:, 0].contiguous(), win=win, kv_gain=s["kv_gain"], rope_dims=r)
    idx = s["idx"][:, 0].clone()
    idx[0, -1] = 1023
    one = api.compressed_attn_decode("csa", s["q"][:, 0].contiguous(), p, kv, win, s["sinks"], m=m, rope_dims=r, k=k, idx_in=idx.contiguous(), q_gain=s["q_gain"])
    check_close(npy(tree[:, 0]), npy(one), "bf16")


@pytest.mark.parametrize("kind", ["csa", "hca"])
def test_streams_graphs_and_workspaces(kind):
    """Another stream, two calls in flight at once, a captured call whose
    inputs change, and a workspace that held other contents."""
    cases = [attn_case(kind, 2, 6, [3000, 2999 + j], "wide", 4 if kind == "csa" else 16, 128, 70, seed=j, **TC) for j in range(2)]
    want = [run_attn(s) for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for j, (s, st) in enumerate(zip(cases, streams)):
            got[j].append(run_attn(s, stream=st))
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(x, want[j]) for x in got[j])                         # and each run gives the same bits
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(run_attn(cases[0], workspace=ws), want[0])
    s = cases[0]
    pos, parents = R.ints(s["pos"], DEV), R.ints(s["parents"], DEV)
    out = torch.zeros_like(s["q"])
    kw = dict(m=s["m"], rope_dims=s["r"], draft=s["draft"], q_gain=s["q_gain"], kv_gain=s["kv_gain"], out=out, workspace=ws)
    if kind == "csa":
        kw["idx_in"] = s["idx"]
    args = (kind, s["q"], pos, parents, s["kv"], s["win"], s["kv_raw"], s["sinks"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.compressed_attn_tree(*args, **kw)
    graph.replay()
    assert torch.equal(out, want[0])
    s["q"].copy_(cases[1]["q"])
    parents.copy_(R.ints(R.parents_of("chain", 2, 6), DEV))
    graph.replay()
    replayed = out.clone()
    assert torch.equal(replayed, api.compressed_attn_tree(*args, **{**kw, "out": torch.zeros_like(out), "workspace": None}))
    assert api.device_error() == 0


def test_inputs_live_until_the_stream_has_read_them():
    """Arguments that the caller drops after a call on another stream: their
    memory is not handed out again before that stream has read it."""
    st = torch.cuda.Stream()
    s = attn_case("hca", 2, 6, [3000, 2999], "wide", 16, 128, 0, **TC)
    pos, parents = R.ints(s["pos"], DEV), R.ints(s["parents"], DEV)
    g = gen(9)
    streams = [torch.randn(2, 6, 512, generator=g, device=DEV).bfloat16() for _ in range(2)]
    ring, bias = torch.randn(2, 16, 2, 512, generator=g, device=DEV).bfloat16(), torch.randn(16, 512, generator=g, device=DEV)
    node_pos = torch.arange(12, device=DEV, dtype=torch.int32).view(2, 6) * 100

    def attn(pos, parents, **kw):
        return api.compressed_attn_tree("hca", s["q"], pos, parents, s["kv"], s["win"], s["kv_raw"], s["sinks"], m=16, rope_dims=64,
                                        draft=s["draft"], **kw)

    def comp(pos, parents, **kw):
        return api.tree_compress("hca", streams, ring, pos, parents, bias, 16, rope_dims=64, **kw)

    def norm(pos, parents, **kw):
        return api.qk_norm_rope(s["q"], None, pos, rope_dims=64, q_out=torch.zeros_like(s["q"]), **kw)[0]
    slow = torch.randn(4096, 4096, device=DEV)
    for call, p in ((attn, pos), (comp, pos), (norm, node_pos)):
        want = call(p, parents)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(10):
                slow = slow @ slow * 1e-3
        args = [p.clone(), parents.clone()]
        torch.cuda.current_stream().synchronize()
        got = call(*args, stream=st)
        del args
        junk = [torch.full_like(x, -1) for x in (p, parents) for _ in range(200)]      # (-1: a sequence, token or node that is left alone)
        st.synchronize()
        assert torch.equal(got, want), call.__name__
        del junk


@pytest.mark.parametrize("heads", [SMALL, TC, HEADS16], ids=["f32", "tc", "16h"])
@pytest.mark.parametrize("B,T,pos", [(2, 9, [300, -1]), (1, 24, [5000])])
def test_new_outputs_are_zero_where_there_is_no_node(heads, B, T, pos):
    """A new out holds zeros in the rows of places without a node, whatever its
    memory held; the other rows are what a given out receives."""
    m = 4
    s = attn_case("hca", B, T, pos, "padded", m, 16, 0, seed=6, **heads)
    live = torch.tensor([[pos[b] >= 0 and R.path_of(s["parents"][b], i) is not None for i in range(T)] for b in range(B)], device=DEV)
    assert not live.all()
    want = run_attn(s, out=torch.zeros_like(s["q"]))
    junk = torch.full((64 << 20,), float("nan"), device=DEV)                # (what the allocator hands out next)
    del junk
    got = run_attn(s)
    assert torch.equal(got, want) and not got[~live].any()
    dt, c = s["q"].dtype, 128
    g = gen(7)
    streams = [torch.randn(B, T, c, generator=g, device=DEV).to(dt) for _ in range(4)]
    ring = torch.randn(B, 2 * m, 4, c, generator=g, device=DEV).to(dt)
    bias = [torch.randn(m, c, generator=g, device=DEV) for _ in range(2)]
    args = ("csa", streams, ring, R.ints(pos, DEV), R.ints(s["parents"], DEV), bias[0], m)
    for f8 in (False, True) if dt == torch.bfloat16 else (False,):
        kw = dict(bias_b=bias[1], rope_dims=64, kv_fp8=f8)
        shape = api.tree_compress(*args, **kw).shape
        want = api.tree_compress(*args, out=torch.zeros(shape, dtype=torch.uint8 if f8 else dt, device=DEV), **kw)
        junk = torch.full((4 << 20,), float("nan"), device=DEV)
        del junk
        got = api.tree_compress(*args, **kw)
        assert torch.equal(got, want)
        for b in range(B):
            for i in range(T):
                done = bool(live[b, i]) and (R.node_position(s["parents"][b], pos[b], i) + 1) % m == 0
                assert done == bool(got[b, i].any())
    assert api.device_error() == 0


def test_wrapper_refusals():
    s = attn_case("csa", 1, 3, [100], "chain", 4, 16, 8, **SMALL)
    for kw, err in ((dict(idx_in=s["idx"].long()), TypeError), (dict(idx_in=s["idx"][:, :2]), ValueError),
                    (dict(draft=s["draft"].bfloat16()), TypeError), (dict(draft=s["draft"][:, :, :32]), ValueError),
                    (dict(out=s["q"]), RuntimeError), (dict(idx_in=None), ValueError)):
        with pytest.raises(err):
            run_attn(s, **kw)
    with pytest.raises(ValueError):
        api.compressed_attn_tree("csa", s["q"], R.ints(s["pos"], DEV), R.ints(s["parents"], DEV), s["kv"], s["win"],
                                 s["kv_raw"][:, :, :32].contiguous(), s["sinks"], m=4, rope_dims=16, idx_in=s["idx"])
    with pytest.raises(ValueError):
        api.compressed_attn_tree("csa", s["q"], R.ints(s["pos"], DEV), R.ints(s["parents"], "cpu"), s["kv"], s["win"],
                                 s["kv_raw"], s["sinks"], m=4, rope_dims=16, idx_in=s["idx"])
