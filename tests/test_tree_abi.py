"""Host-side checks of qk_norm_rope, tree_compress and compressed_attn_tree:
every refusal comes before any launch, and empty work needs no device."""

import ctypes as C

import pytest
import torch

from long_context_compressed_overlapped_b200 import api, build, native as N, synth
from tests import tree_reference as R


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.lib()


def norm(**kw):
    a = dict(dtype=N.BF16, B=1, n=2, HQ=4, HK=1, d=64, rope_dims=16, q=64, k=64, pos=64, q_out=128, k_out=128)
    return N.NormRopeArgs(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=N.E4M3), N.ERR_INVALID_ARG),
    (dict(n=-1), N.ERR_INVALID_ARG),
    (dict(d=0), N.ERR_INVALID_ARG),
    (dict(rope_dims=15), N.ERR_INVALID_ARG),
    (dict(rope_dims=66), N.ERR_INVALID_ARG),
    (dict(d=68), N.ERR_UNSUPPORTED),
    (dict(d=1032), N.ERR_UNSUPPORTED),
    (dict(d=1024, rope_dims=514), N.ERR_UNSUPPORTED),
    (dict(dtype=N.F32, d=516), N.ERR_UNSUPPORTED),
    (dict(HQ=65535), N.ERR_UNSUPPORTED),
    (dict(B=1 << 16, n=1 << 16), N.ERR_UNSUPPORTED),
    (dict(q=None), N.ERR_INVALID_ARG),
    (dict(k_out=None), N.ERR_INVALID_ARG),
    (dict(pos=None), N.ERR_INVALID_ARG),
    (dict(q=72), N.ERR_ALIGNMENT),
    (dict(q_stride=(N.i64 * 3)(512, 256, -64)), N.ERR_INVALID_ARG),
    (dict(q_stride=(N.i64 * 3)(512, 260, 64)), N.ERR_ALIGNMENT),
    (dict(q_out=64, q_stride=(N.i64 * 3)(2048, 512, 64)), N.ERR_INVALID_ARG),      # in place, strided
])
def test_norm_rope_refusals(lib, kw, status):
    assert lib.qk_norm_rope(C.byref(norm(**kw)), None) == status


def test_norm_rope_empty(lib):
    assert lib.qk_norm_rope(None, None) == N.ERR_INVALID_ARG
    for kw in (dict(B=0), dict(n=0), dict(HQ=0, HK=0, q=None, k=None)):
        assert lib.qk_norm_rope(C.byref(norm(**kw)), None) == N.OK


def comp(**kw):
    a = dict(kind=N.CSA, dtype=N.BF16, out_dtype=N.BF16, B=1, T=4, c=128, m=4, rms_norm=1, rope_dims=64, pos=64,
             parents=64, a=64, b=64, za=64, zb=64, ring=64, bias_a=64, bias_b=64, out=64)
    return N.TreeCompressArgs(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(kind=2), N.ERR_INVALID_ARG),
    (dict(dtype=5), N.ERR_INVALID_ARG),
    (dict(T=-1), N.ERR_INVALID_ARG),
    (dict(m=0), N.ERR_INVALID_ARG),
    (dict(rope_dims=63), N.ERR_INVALID_ARG),
    (dict(out_dtype=N.F32), N.ERR_UNSUPPORTED),
    (dict(out_dtype=N.E4M3, c=64), N.ERR_UNSUPPORTED),
    (dict(out_dtype=N.E4M3), N.ERR_INVALID_ARG),                                    # no out_scale
    (dict(dtype=N.F32, out_dtype=N.E4M3), N.ERR_UNSUPPORTED),
    (dict(kv_rows=1), N.ERR_UNSUPPORTED),                                           # FP8 rows are an E4M3 output
    (dict(out_dtype=N.E4M3, kv_rows=1, c=128, rope_dims=32), N.ERR_UNSUPPORTED),
    (dict(c=132), N.ERR_UNSUPPORTED),
    (dict(T=65), N.ERR_UNSUPPORTED),
    (dict(m=257), N.ERR_UNSUPPORTED),
    (dict(kind=N.HCA, m=513), N.ERR_UNSUPPORTED),
    (dict(zb=None), N.ERR_INVALID_ARG),
    (dict(ring=None), N.ERR_INVALID_ARG),
    (dict(parents=None), N.ERR_INVALID_ARG),
    (dict(out=68), N.ERR_ALIGNMENT),
])
def test_tree_compress_refusals(lib, kw, status):
    assert lib.tree_compress(C.byref(comp(**kw)), None) == status


def test_tree_compress_empty(lib):
    assert lib.tree_compress(None, None) == N.ERR_INVALID_ARG
    for kw in (dict(B=0), dict(T=0)):
        assert lib.tree_compress(C.byref(comp(**kw)), None) == N.OK


def attn(**kw):
    a = dict(kind=N.CSA, dtype=N.BF16, B=2, T=4, H=64, d=512, N_cap=300, m=4, w=128, k=64, rope_dims=64, q=64, pos=64,
             parents=64, kv_cache=64, win=64, kv_raw=64, draft=64, sinks=64, idx_in=64, out=128)
    return N.TreeAttnArgs(**{**a, **kw})


INDEXER = dict(idx_in=None, HI=4, dI=128, qI_dtype=N.BF16, kI_dtype=N.BF16, qI=64, wI=64, kI=64)


@pytest.mark.parametrize("kw,status", [
    (dict(kind=3), N.ERR_INVALID_ARG),
    (dict(dtype=N.E4M3), N.ERR_INVALID_ARG),
    (dict(H=0), N.ERR_INVALID_ARG),
    (dict(w=-1), N.ERR_INVALID_ARG),
    (dict(rope_dims=513), N.ERR_INVALID_ARG),
    (dict(T=65), N.ERR_UNSUPPORTED),
    (dict(d=48, rope_dims=0), N.ERR_UNSUPPORTED),
    (dict(d=544), N.ERR_UNSUPPORTED),
    (dict(kv_dtype=N.E4M3, d=128), N.ERR_UNSUPPORTED),
    (dict(kv_dtype=N.E4M3, rope_dims=32), N.ERR_UNSUPPORTED),
    (dict(kv_dtype=N.E4M3, dtype=N.F32), N.ERR_UNSUPPORTED),
    (dict(k=0), N.ERR_INVALID_ARG),
    (dict(k=2**31 - 1), N.ERR_UNSUPPORTED),
    (dict(N_cap=2**31 - 1), N.ERR_UNSUPPORTED),
    (dict(w=1 << 28), N.ERR_UNSUPPORTED),
    (dict(H=65536), N.ERR_UNSUPPORTED),
    (dict(q=None), N.ERR_INVALID_ARG),
    (dict(out=64), N.ERR_INVALID_ARG),                                              # out is q
    (dict(parents=None), N.ERR_INVALID_ARG),
    (dict(kv_cache=None), N.ERR_INVALID_ARG),
    (dict(win=None), N.ERR_INVALID_ARG),
    (dict(kv_raw=None), N.ERR_INVALID_ARG),
    (dict(kv_raw=72), N.ERR_ALIGNMENT),
    (dict(INDEXER, qI=None), N.ERR_INVALID_ARG),
    (dict(INDEXER, kI=None), N.ERR_INVALID_ARG),
    (dict(INDEXER, kI_dtype=N.F32), N.ERR_UNSUPPORTED),
    (dict(INDEXER, kI_dtype=N.E4M3), N.ERR_INVALID_ARG),                            # no kI_scale
    (dict(INDEXER, kI_dtype=N.E4M3, kI_scale=64, draft_kI=64), N.ERR_INVALID_ARG),  # no draft_kI_scale
    (dict(INDEXER, draft_kI=64, draft=None), N.ERR_INVALID_ARG),
    (dict(INDEXER, draft_kI=64, k=4097), N.ERR_UNSUPPORTED),
])
def test_tree_attn_refusals(lib, kw, status):
    assert lib.compressed_attn_tree(C.byref(attn(**kw)), None) == status


def test_tree_attn_empty_and_workspace(lib):
    assert lib.compressed_attn_tree(None, None) == N.ERR_INVALID_ARG
    for kw in (dict(B=0), dict(T=0)):
        assert lib.compressed_attn_tree(C.byref(attn(**kw)), None) == N.OK
        assert lib.csahca_tree_workspace_size(C.byref(attn(**kw))) == 0
    assert lib.csahca_tree_workspace_size(C.byref(attn(d=48))) == 0
    # the plan (positions, row lists of w + T codes), finished rows and queries at the least
    need = lib.csahca_tree_workspace_size(C.byref(attn()))
    assert need >= 8 * (4 + 4 + 16 + 4 * (128 + 4) + 2 * 512 + 2 * 64 * 512)


def test_wrappers_refuse_on_the_host():
    x = torch.zeros(1, 2, 4, 64)
    pos = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.qk_norm_rope(x, None, pos, rope_dims=16)                                # not on a CUDA device
    with pytest.raises(ValueError):
        api.qk_norm_rope(None, None, pos, rope_dims=16)
    with pytest.raises(TypeError):
        api.qk_norm_rope(x.half(), None, pos, rope_dims=16)
    s = tuple(torch.zeros(1, 4, 64) for _ in range(2))
    with pytest.raises(ValueError):
        api.tree_compress("csa", s, None, None, None, None, 4)                      # two streams for csa


def test_reference_paths():
    """The tests' own trees: parents come first, padding cuts descendants off."""
    for shape in ("chain", "flat", "wide", "padded"):
        for b, row in enumerate(R.parents_of(shape, 3, 9, seed=5)):
            assert all(p < i for i, p in enumerate(row))
            for i, p in enumerate(row):
                path = R.path_of(row, i)
                assert (path is None) == (p == R.NONE or (p >= 0 and R.path_of(row, p) is None))
                assert path is None or (path[-1] == i and len(path) == R.node_position(row, 10, i) - 9)


def test_tree_inputs_are_seeded():
    wl = synth.WORKLOADS["decode_256k"]
    a = synth.tree_inputs(wl, 5, "cpu", ctx=300, B=1)
    b = synth.tree_inputs(wl, 5, "cpu", ctx=300, B=1)
    assert torch.equal(a[0]["tq"], b[0]["tq"]) and torch.equal(a[1]["parents"], b[0]["parents"])
    assert a[0]["parents"].lt(torch.arange(5)).all()
