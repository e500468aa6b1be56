"""Torch-facing wrappers of the C-ABI entry points (same names).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, outputs and workspaces are allocated with torch when the caller
does not pass them, and the call goes to libcsahca.so on the current CUDA
stream.  Every step of the path runs in the library's kernels.
"""

from __future__ import annotations

import ctypes as C
import functools

import torch

from . import native as N

_DT = {torch.float32: N.F32, torch.bfloat16: N.BF16, torch.uint8: N.E4M3}


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the CUDA library must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the CUDA library must be contiguous")
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _f32(t):
    return None if t is None else t.contiguous().float()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _keep_for(stream, x):
    """Tensors among x (nested): their memory stays theirs until the stream has read it."""
    if isinstance(x, torch.Tensor):
        if x.is_cuda:
            x.record_stream(stream)
    elif isinstance(x, (tuple, list, dict)):
        for y in x.values() if isinstance(x, dict) else x:
            _keep_for(stream, y)


def _on(stream, dev, call, *args):
    """call(*args) with the tensors' device current and the given stream (or
    the device's current one) as the stream of its allocations and kernels.
    On a stream that is not the current one the caller may drop the tensors
    as soon as the call returns."""
    if dev.type != "cuda":
        raise ValueError("tensors passed to the CUDA library must live on a CUDA device")
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream on {stream.device}, tensors on {dev}")
        _keep_for(stream, args)
        with torch.cuda.stream(stream):
            return call(*args)
    if torch.cuda.current_device() == dev.index:
        return call(*args)
    with torch.cuda.device(dev):
        return call(*args)


def _streamed(call):
    """A wrapper whose stream argument is handled by _on (the first tensor among
    its arguments says which device): its workspace and converted copies belong
    to the stream that reads them."""
    @functools.wraps(call)
    def on(*args, stream=None, **kw):
        dev = next((x.device for x in (*args, *kw.values()) if isinstance(x, torch.Tensor)), None)
        if dev is None or dev.type != "cuda":
            return call(*args, stream=stream, **kw)          # (refused there)
        return _on(stream, dev, lambda a, k: call(*a, **k), args, kw)
    return on


@_streamed
def _compress(kind, a, za, bias_a, m, *, b=None, zb=None, bias_b=None, gain=None,
              rms_norm=True, rope_dims=0, rope_base=10000.0, eps=1e-6, first_block=0,
              num_blocks=-1, out=None, stream=None):
    B, n, c = a.shape
    nb = (n // m - first_block) if num_blocks < 0 else num_blocks
    if out is None:
        out = torch.empty(B, max(nb, 0), c, dtype=a.dtype, device=a.device)
    bias_a = _f32(bias_a)
    bias_b = _f32(bias_b)
    gain = _f32(gain)
    args = N.CompressArgs(dtype=_dt(a), B=B, n=n, c=c, m=m, first_block=first_block,
                          num_blocks=num_blocks, rms_norm=int(bool(rms_norm)),
                          rope_dims=rope_dims, rope_base=rope_base, eps=eps,
                          a=_ptr(a), b=_ptr(b), za=_ptr(za), zb=_ptr(zb), bias_a=_ptr(bias_a),
                          bias_b=_ptr(bias_b), gain=_ptr(gain), out=_ptr(out))
    fn = N.lib().csa_compress if kind == "csa" else N.lib().hca_compress
    N.check(fn(C.byref(args), _stream(stream)), f"{kind}_compress")
    return out


def csa_compress(a, b, za, zb, bias_a, bias_b, m, **kw):
    """Overlapped two-stream compression (ratio 1/m, 2m tokens per entry),
    then optional RMSNorm * gain and RoPE at position i*m.  [B, n, c] -> [B, n/m, c]."""
    return _compress("csa", a, za, bias_a, m, b=b, zb=zb, bias_b=bias_b, **kw)


def hca_compress(a, za, bias_a, m, **kw):
    """Non-overlapped single-stream compression (ratio 1/m'), then optional
    RMSNorm * gain and RoPE at position i*m'."""
    return _compress("hca", a, za, bias_a, m, **kw)


@_streamed
def indexer_topk(qI, w, kI, q_pos, m, k, *, kI_scale=None, idx=None, scores_out=None,
                 sel_scores=None, entry_base=0, stream=None):
    """Lightning-indexer scores over the visible compressed keys and the
    per-query top-k (ties to the lower index), sorted ascending, -1 padded.

    qI [B, nq, HI, dI]; w [B, nq, HI] f32; kI [B, N, dI] (f32/bf16, or uint8
    e4m3 codes with kI_scale [B, N, dI/128]); q_pos [B, nq] int32.
    Context parallelism: kI holds the global entries entry_base ..
    entry_base + N - 1 (idx then holds local rows), and sel_scores
    [B, nq, k] f32 receives the score of each selected row."""
    B, nq, HI, dI = qI.shape
    Nk = kI.shape[1]
    if idx is None:
        idx = torch.empty(B, nq, k, dtype=torch.int32, device=qI.device)
    w, kI_scale = _f32(w), _f32(kI_scale)        # (locals: converted copies live until the launches)
    q_pos = q_pos.to(torch.int32).contiguous()
    args = N.IndexerArgs(q_dtype=_dt(qI), k_dtype=_dt(kI), B=B, nq=nq, HI=HI, dI=dI, N=Nk, m=m,
                         k=k, qI=_ptr(qI), w=_ptr(w), kI=_ptr(kI),
                         kI_scale=_ptr(kI_scale), q_pos=_ptr(q_pos), idx=_ptr(idx),
                         scores_out=_ptr(scores_out), sel_scores=_ptr(sel_scores),
                         entry_base=int(entry_base))
    L = N.lib()
    ws_bytes = L.csahca_indexer_workspace_size(C.byref(args))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=qI.device) if ws_bytes else None
    args.workspace = _ptr(ws)
    args.workspace_bytes = ws_bytes
    N.check(L.indexer_topk(C.byref(args), _stream(stream)), "indexer_topk")
    return idx


@_streamed
def compressed_attn_prefill(kind, q, kv_comp, kv_win, sinks, *, m, w, rope_dims, idx=None,
                            q_gain=None, kv_gain=None, q_norm=True, kv_norm=True,
                            rope_base=10000.0, eps=1e-6, scale=0.0, out=None, stream=None):
    """CSA (selected entries) or HCA (every visible entry) attention plus the
    sliding window and per-head sink, for every query of a prefill.

    q [B, n, H, d] raw; kv_comp [B, N, d] final rows; kv_win [B, n, d] raw
    per-token rows; idx [B, n, k] int32 (CSA)."""
    B, n, H, d = q.shape
    Nc = kv_comp.shape[1]
    if out is None:
        out = torch.empty_like(q)
    kk = idx.shape[2] if idx is not None else 0
    q_gain, kv_gain, sinks = _f32(q_gain), _f32(kv_gain), _f32(sinks)
    args = N.AttnArgs(kind=N.CSA if kind == "csa" else N.HCA, dtype=_dt(q), B=B, n=n, H=H, d=d,
                      N=Nc, m=m, k=kk, w=w, rope_dims=rope_dims, rope_base=rope_base, eps=eps,
                      scale=scale, q_norm=int(bool(q_norm)), kv_norm=int(bool(kv_norm)),
                      q=_ptr(q), kv_comp=_ptr(kv_comp) if Nc > 0 else None, kv_win=_ptr(kv_win),
                      q_gain=_ptr(q_gain), kv_gain=_ptr(kv_gain),
                      idx=_ptr(idx), sinks=_ptr(sinks), out=_ptr(out))
    L = N.lib()
    ws_bytes = L.csahca_prefill_workspace_size(C.byref(args))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    args.workspace = _ptr(ws)
    args.workspace_bytes = ws_bytes
    N.check(L.compressed_attn_prefill(C.byref(args), _stream(stream)), "compressed_attn_prefill")
    return out


def decode_args(kind, q, pos, kv_cache, win, sinks, *, m, rope_dims, k=0, qI=None, wI=None,
                kI=None, kI_scale=None, idx_in=None, idx_out=None, q_gain=None, q_norm=True,
                rope_base=10000.0, eps=1e-6, scale=0.0, out=None, entry_base=0, partial_out=None,
                skip_window=False):
    """Build the DecodeArgs struct (and keep the tensors it points to alive in
    the returned list)."""
    B, H, d = q.shape
    keep = []

    def f(t):
        t = _f32(t)
        keep.append(t)
        return t

    pos = pos.to(torch.int32).contiguous()
    keep.append(pos)
    if out is None and partial_out is None:
        out = torch.empty_like(q)
    keep.append((q, kv_cache, win, qI, kI, idx_in, idx_out, out, partial_out))
    HI = dI = 0
    qI_dt = kI_dt = 0
    if qI is not None:
        _, HI, dI = qI.shape
        qI_dt, kI_dt = _dt(qI), _dt(kI)
    # a uint8 cache holds FP8 KV rows (include/csahca.h: e4m3 non-RoPE dims with
    # one fp32 scale per 64, bf16 RoPE dims)
    kv_dt = N.E4M3 if kv_cache.dtype == torch.uint8 else _dt(q)
    args = N.DecodeArgs(kind=N.CSA if kind == "csa" else N.HCA, dtype=_dt(q), B=B, H=H, d=d,
                        N_cap=kv_cache.shape[1], m=m, w=win.shape[1] if win is not None else 0,
                        kv_dtype=kv_dt,
                        rope_dims=rope_dims, rope_base=rope_base, eps=eps, scale=scale,
                        q_norm=int(bool(q_norm)), k=k, HI=HI, dI=dI, qI_dtype=qI_dt,
                        kI_dtype=kI_dt, q=_ptr(q), pos=_ptr(pos), q_gain=_ptr(f(q_gain)),
                        kv_cache=_ptr(kv_cache), win=_ptr(win), sinks=_ptr(f(sinks)),
                        qI=_ptr(qI), wI=_ptr(f(wI)), kI=_ptr(kI), kI_scale=_ptr(f(kI_scale)),
                        idx_in=_ptr(idx_in), idx_out=_ptr(idx_out), out=_ptr(out),
                        entry_base=int(entry_base), partial_out=_ptr(partial_out),
                        skip_window=int(bool(skip_window)))
    return args, out, keep


@_streamed
def compressed_attn_decode(kind, q, pos, kv_cache, win, sinks, *, m, rope_dims, k=0, qI=None,
                           wI=None, kI=None, kI_scale=None, idx_in=None, idx_out=None,
                           q_gain=None, q_norm=True, rope_base=10000.0, eps=1e-6, scale=0.0,
                           out=None, entry_base=0, partial_out=None, skip_window=False,
                           workspace=None, stream=None):
    """One decode step of one CSA or HCA layer for B sequences (one new query
    each at pos[b]); CSA selects with the lightning indexer unless idx_in is
    given.  Returns out [B, H, d], or partial_out [B, 2H + H*d] f32 (this
    rank's share of a context-parallel layer whose cache shard starts at
    global entry entry_base) when that is given."""
    args, out, keep = decode_args(kind, q, pos, kv_cache, win, sinks, m=m, rope_dims=rope_dims,
                                  k=k, qI=qI, wI=wI, kI=kI, kI_scale=kI_scale, idx_in=idx_in,
                                  idx_out=idx_out, q_gain=q_gain, q_norm=q_norm,
                                  rope_base=rope_base, eps=eps, scale=scale, out=out,
                                  entry_base=entry_base, partial_out=partial_out,
                                  skip_window=skip_window)
    L = N.lib()
    ws_bytes = L.csahca_decode_workspace_size(C.byref(args))
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    args.workspace = _ptr(workspace)
    args.workspace_bytes = workspace.numel()
    N.check(L.compressed_attn_decode(C.byref(args), _stream(stream)), "compressed_attn_decode")
    del keep
    return out if partial_out is None else partial_out


def decode_compress_args(kind, pos, streams, ring, kv_cache, *, m, bias_a, bias_b=None, kv_raw=None,
                         win=None, kv_gain=None, kv_norm=True, rope_dims=0, rope_base=10000.0,
                         eps=1e-6, istreams=None, ibias_a=None, ibias_b=None, iring=None, kI=None,
                         kI_scale=None, entry_base=0):
    """Build the DecodeCompressArgs struct (and the list of tensors it points to).

    streams: (a, b, za, zb) for "csa" or (a, za) for "hca", each [B, d];
    ring [B, R, S, d]; istreams: (ia, ib, iza, izb) [B, dI] with iring
    [B, 2m, 4, dI] and kI / kI_scale (csa only, optional)."""
    B, d = streams[0].shape
    keep = []

    def f(t):
        t = _f32(t)
        keep.append(t)
        return t

    pos = pos.to(torch.int32).contiguous()
    keep.append(pos)
    csa = kind == "csa"
    a, b, za, zb = (streams if csa else (streams[0], None, streams[1], None))
    dI = 0
    ia = ib = iza = izb = None
    if csa and istreams is not None:
        ia, ib, iza, izb = istreams
        dI = ia.shape[1]
        if kI is None or iring is None or ibias_a is None or ibias_b is None:
            raise ValueError("decode_compress: indexer streams need iring, ibias_a, ibias_b and kI")
    keep.append((a, b, za, zb, kv_raw, ring, kv_cache, win, ia, ib, iza, izb, iring, kI, kI_scale))
    args = N.DecodeCompressArgs(
        kind=N.CSA if csa else N.HCA, dtype=_dt(a), B=B, d=d, m=m, N_cap=kv_cache.shape[1],
        w=win.shape[1] if win is not None else 0, rope_dims=rope_dims, rope_base=rope_base, eps=eps,
        kv_norm=int(bool(kv_norm)), dI=dI, kI_dtype=_dt(kI) if dI else 0,
        kv_dtype=N.E4M3 if kv_cache.dtype == torch.uint8 else _dt(a), entry_base=int(entry_base),
        pos=_ptr(pos), kv_raw=_ptr(kv_raw), a=_ptr(a), b=_ptr(b), za=_ptr(za), zb=_ptr(zb),
        bias_a=_ptr(f(bias_a)), bias_b=_ptr(f(bias_b)), kv_gain=_ptr(f(kv_gain)), ring=_ptr(ring),
        kv_cache=_ptr(kv_cache), win=_ptr(win), ia=_ptr(ia), ib=_ptr(ib), iza=_ptr(iza), izb=_ptr(izb),
        ibias_a=_ptr(f(ibias_a)), ibias_b=_ptr(f(ibias_b)), iring=_ptr(iring), kI=_ptr(kI),
        kI_scale=_ptr(kI_scale))
    return args, keep


@_streamed
def decode_compress(kind, pos, streams, ring, kv_cache, *, m, bias_a, stream=None, **kw):
    """One decode step of one layer's compressors: the new token's raw streams
    into the ring, its window row (if kv_raw and win are given) and, when the
    token completes a block, the new compressed entry (and indexer key) into
    the caches.  Updates ring, win, kv_cache, iring, kI, kI_scale in place."""
    args, keep = decode_compress_args(kind, pos, streams, ring, kv_cache, m=m, bias_a=bias_a, **kw)
    N.check(N.lib().decode_compress(C.byref(args), _stream(stream)), "decode_compress")
    del keep


def cp_partial_floats(H: int, d: int) -> int:
    """Floats of one row's context-parallel attention share: mx[H], l[H], o[H][d]."""
    return 2 * H + H * d


@_streamed
def cp_topk_merge(cand_idx, cand_scores, bases, rank, *, idx_global=None, idx_local=None, stream=None):
    """Stage 1 of context parallelism: the global top-k from every rank's
    candidates.  cand_idx / cand_scores [R, rows, k] (local rows and their
    scores, as indexer_topk writes idx / sel_scores); bases: the R shards'
    first global entries (host ints).  Returns (idx_global, idx_local), each
    [rows, k] int32 in ascending global order, -1 padded; idx_local holds the
    rows of rank `rank` and -1 for the other ranks' entries."""
    R, rows, k = cand_idx.shape
    dev = cand_idx.device
    if idx_global is None:
        idx_global = torch.empty(rows, k, dtype=torch.int32, device=dev)
    if idx_local is None:
        idx_local = torch.empty(rows, k, dtype=torch.int32, device=dev)
    b = (C.c_int32 * R)(*[int(x) for x in bases])
    args = N.CpTopkMergeArgs(R=R, rows=rows, k=k, rank=int(rank), bases=C.cast(b, C.c_void_p),
                             cand_idx=_ptr(cand_idx), cand_scores=_ptr(cand_scores),
                             idx_global=_ptr(idx_global), idx_local=_ptr(idx_local))
    N.check(N.lib().cp_topk_merge(C.byref(args), _stream(stream)), "cp_topk_merge")
    return idx_global, idx_local


@_streamed
def cp_attn_merge(partials, sinks, pos, *, H, d, rope_dims, dtype=torch.bfloat16, rope_base=10000.0,
                  out=None, stream=None):
    """Stage 2 of context parallelism: the layer output [rows, H, d] from the
    ranks' shares partials [R, rows, 2H + H*d] f32, with the sink and the
    output de-rotation by -pos."""
    R, rows, _ = partials.shape
    if out is None:
        out = torch.empty(rows, H, d, dtype=dtype, device=partials.device)
    keep = _f32(sinks)
    pos = pos.to(torch.int32).contiguous()
    args = N.CpMergeArgs(dtype=_dt(out), R=R, rows=rows, H=H, d=d, rope_dims=rope_dims, rope_base=rope_base,
                         partials=_ptr(partials), sinks=_ptr(keep), pos=_ptr(pos), out=_ptr(out))
    N.check(N.lib().cp_attn_merge(C.byref(args), _stream(stream)), "cp_attn_merge")
    return out


def _arg(name, t, dev, shape, dtype, optional=False):
    """Pointer of an argument tensor, checked for device, shape, dtype and contiguity."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and t.is_contiguous():
        return t.data_ptr()
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _ints(name, t, dev, shape, keep):
    """Pointer of an int32 argument (other integer tensors are converted)."""
    if t.dtype is not torch.int32 or not t.is_contiguous():
        if t.dtype.is_floating_point or t.device != dev:
            raise TypeError(f"{name} must be an integer tensor on {dev}")
        t = t.to(torch.int32).contiguous()
        keep.append(t)
    return _arg(name, t, dev, shape, torch.int32)


def _floats(name, t, dev, shape, keep, optional=True):
    """Pointer of an fp32 argument (other floating tensors are converted)."""
    if t is not None and (t.dtype is not torch.float32 or not t.is_contiguous()):
        t = t.contiguous().float()
        keep.append(t)
    return _arg(name, t, dev, shape, torch.float32, optional)


def _heads(name, t, out, gain, dev, dt, B, n, d, keep):
    """One side of qk_norm_rope: (heads, strides or None, pointers of rows, output and gain, output, output is new)."""
    shape = t.shape
    if t.dtype is not dt or t.device != dev or len(shape) != 4 or shape[0] != B or shape[1] != n or shape[3] != d:
        raise ValueError(f"{name}: {tuple(shape)} {t.dtype} on {t.device} does not match the other rows")
    strides = None
    if not t.is_contiguous():
        strides = t.stride()
        if d > 1 and strides[3] != 1:
            raise ValueError(f"{name}: the dims of a head must be contiguous")
        if not any(strides[:3]):                 # one row for every head (the library's mark of contiguous rows)
            t, strides = t.contiguous(), None
            keep.append(t)
    fresh = out is None
    if fresh:
        out = torch.empty_like(t, memory_format=torch.contiguous_format)
        o = out.data_ptr()
    else:
        o = _arg(name + "_out", out, dev, shape, dt)
    return shape[2], strides, t.data_ptr(), o, _floats(name + "_gain", gain, dev, (d,), keep), out, fresh


def _norm_rope(q, k, pos, rope_dims, q_gain, k_gain, q_norm, k_norm, rope_base, eps, q_out, k_out):
    x = q if q is not None else k
    dev, dt, keep = x.device, x.dtype, []
    B, n, _, d = x.shape
    a = N.NormRopeArgs(_dt(x), B, n, 0, 0, d, rope_dims, rope_base, eps, bool(q_norm), bool(k_norm))
    a.pos = _ints("pos", pos, dev, (B, n), keep)
    if q is not None:
        a.HQ, st, a.q, a.q_out, a.q_gain, q_out, fresh = _heads("q", q, q_out, q_gain, dev, dt, B, n, d, keep)
        a.zero_rest = int(fresh)
        if st is not None:
            a.q_stride[:] = st[:3]
    if k is not None:
        a.HK, st, a.k, a.k_out, a.k_gain, k_out, fresh = _heads("k", k, k_out, k_gain, dev, dt, B, n, d, keep)
        a.zero_rest |= 2 * fresh
        if st is not None:
            a.k_stride[:] = st[:3]
    N.check(N.lib().qk_norm_rope(C.byref(a), _raw_stream(dev.index)), "qk_norm_rope")
    return (q_out if q is not None else None, k_out if k is not None else None)


def qk_norm_rope(q, k, pos, *, rope_dims, q_gain=None, k_gain=None, q_norm=True, k_norm=True, rope_base=10000.0,
                 eps=1e-6, q_out=None, k_out=None, stream=None):
    """RMSNorm * gain of every query and key head and RoPE at the token's
    position on the last rope_dims, in one pass.

    q [B, n, HQ, d] and k [B, n, HK, d] (either may be None): the dims of a head
    contiguous, the other strides free (multiples of 16 bytes), so heads may be
    slices of one projection; pos [B, n] int32 (at an address that is a
    multiple of 16, as every argument), negative for padding (the rows of such a
    token are left as they were, zero in a new output).  q_out / k_out:
    contiguous, by default new; a contiguous input may be its own output.
    Returns (q_out, k_out)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is required")
    _dt(x)
    return _on(stream, x.device, _norm_rope, q, k, pos, rope_dims, q_gain, k_gain, q_norm, k_norm, rope_base, eps, q_out,
               k_out)


def tree_compress_args(kind, streams, ring, pos, parents, bias_a, m, *, bias_b=None, gain=None, rms_norm=True,
                       rope_dims=0, rope_base=10000.0, eps=1e-6, out=None, out_scale=None, kv_fp8=False):
    """Build the TreeCompressArgs struct (and keep the tensors it points to
    alive in the returned list).  Returns (args, out, keep)."""
    csa = kind == "csa"
    if len(streams) != (4 if csa else 2):
        raise ValueError("csa takes four streams (a, b, za, zb), hca two (a, za)")
    x = streams[0]
    dev, dt, keep = x.device, x.dtype, []
    code = _dt(x)
    B, T, c = shape = x.shape
    f8 = kv_fp8 or out_scale is not None
    odt = torch.uint8 if f8 else dt
    oshape = (B, T, N.lib().csahca_kv_row_bytes(N.E4M3, c, rope_dims)) if kv_fp8 else shape
    fresh = out is None
    if fresh:
        out = torch.empty(oshape, dtype=odt, device=dev)
    p = [_arg("streams", t, dev, shape, dt) for t in streams]
    keep.append((*streams, ring, pos, parents, bias_a, bias_b, gain, out, out_scale))
    # (in the struct's order)
    a = N.TreeCompressArgs(
        N.CSA if csa else N.HCA, code, N.E4M3 if f8 else code, B, T, c, m, bool(rms_norm), rope_dims, rope_base, eps,
        bool(kv_fp8), fresh, 0, _ints("pos", pos, dev, (B,), keep), _ints("parents", parents, dev, (B, T), keep),
        p[0], p[1] if csa else None, p[2 if csa else 1], p[3] if csa else None,
        _arg("ring", ring, dev, (B, 2 * m, 4, c) if csa else (B, m, 2, c), dt),
        _floats("bias_a", bias_a, dev, (m, c), keep, False),
        _floats("bias_b", bias_b, dev, (m, c), keep, False) if csa else None,
        None if gain is None else _floats("gain", gain, dev, (c,), keep), _arg("out", out, dev, oshape, odt),
        None if out_scale is None else _arg("out_scale", out_scale, dev, (B, T, c // 128), torch.float32))
    return a, out, keep


def _tree_compress(args, kw):
    a, out, keep = tree_compress_args(*args, **kw)
    N.check(N.lib().tree_compress(C.byref(a), _raw_stream(out.device.index)), "tree_compress")
    del keep
    return out


def tree_compress(kind, streams, ring, pos, parents, bias_a, m, *, stream=None, **kw):
    """The compressed entries that the nodes of draft trees complete.

    streams: (a, b, za, zb) for "csa" or (a, za) for "hca", each [B, T, c], the
    drafted tokens' raw streams; ring [B, R, S, c] as decode_compress keeps it;
    pos [B] the first drafted token's position; parents [B, T] (parent node, -1
    for a node that follows the last committed token, < -1 for no node).
    out [B, T, c]: row i is written iff node i's token ends a block, the others
    are left as they were (zero in a new out).  With out_scale
    [B, T, c / 128] f32, out holds e4m3 codes (uint8), as for indexer keys; with
    kv_fp8, FP8 KV rows (uint8 [B, T, csahca_kv_row_bytes]).
    bias_b, gain, rms_norm, rope_dims, rope_base, eps as in csa_compress."""
    if len(streams) != (4 if kind == "csa" else 2):
        raise ValueError("csa takes four streams (a, b, za, zb), hca two (a, za)")
    return _on(stream, streams[0].device, _tree_compress, (kind, streams, ring, pos, parents, bias_a, m), kw)


def tree_attn_args(kind, q, pos, parents, kv_cache, win, kv_raw, sinks, *, m, rope_dims, draft=None, k=0, qI=None,
                   wI=None, kI=None, kI_scale=None, draft_kI=None, draft_kI_scale=None, idx_in=None, idx_out=None,
                   q_gain=None, kv_gain=None, q_norm=True, kv_norm=True, rope_base=10000.0, eps=1e-6, scale=0.0,
                   out=None):
    """Build the TreeAttnArgs struct (and keep the tensors it points to alive
    in the returned list).  Returns (args, out, keep)."""
    csa = kind == "csa"
    dev, dt, keep = q.device, q.dtype, []
    code = _dt(q)
    shape = q.shape
    B, T, H, d = shape
    Nc = kv_cache.shape[1]
    w = win.shape[1] if win is not None else 0
    fresh = out is None
    if fresh:
        out = torch.empty(shape, dtype=dt, device=dev)
    row = (B, T, d)
    # a uint8 cache holds FP8 KV rows, and so do the drafted entries
    f8 = kv_cache.dtype is torch.uint8
    cdt, cd = (torch.uint8, N.lib().csahca_kv_row_bytes(N.E4M3, d, rope_dims)) if f8 else (dt, d)
    keep.append((q, pos, parents, kv_cache, win, kv_raw, sinks, draft, qI, wI, kI, kI_scale, draft_kI, draft_kI_scale, idx_in,
                 idx_out, q_gain, kv_gain, out))
    # (in the struct's order)
    a = N.TreeAttnArgs(
        N.CSA if csa else N.HCA, code, B, T, H, d, Nc, m, w, k, rope_dims, rope_base, eps, scale, bool(q_norm),
        bool(kv_norm), 0, 0, 0, 0, N.E4M3 if f8 else code, fresh,
        _arg("q", q, dev, shape, dt), _ints("pos", pos, dev, (B,), keep), _ints("parents", parents, dev, (B, T), keep),
        None if q_gain is None else _floats("q_gain", q_gain, dev, (d,), keep),
        None if kv_gain is None else _floats("kv_gain", kv_gain, dev, (d,), keep),
        _arg("kv_cache", kv_cache, dev, (B, Nc, cd), cdt) if Nc else None,
        _arg("win", win, dev, (B, w, d), dt) if w else None,
        _arg("kv_raw", kv_raw, dev, row, dt) if w else None,
        None if draft is None else _arg("draft", draft, dev, (B, T, cd), cdt),
        _floats("sinks", sinks, dev, (H,), keep, False))
    a.out = _arg("out", out, dev, shape, dt)
    if csa:
        if idx_in is not None:
            a.k = k = idx_in.shape[2]
            a.idx_in = _arg("idx_in", idx_in, dev, (B, T, k), torch.int32)
        else:
            if qI is None or wI is None or kI is None:
                raise ValueError("csa needs idx_in, or qI, wI and kI for the indexer")
            HI, dI = qI.shape[2:]
            a.HI, a.dI, a.qI_dtype, a.kI_dtype = HI, dI, _dt(qI), _dt(kI)
            a.qI = _arg("qI", qI, dev, (B, T, HI, dI), qI.dtype)
            a.wI = _floats("wI", wI, dev, (B, T, HI), keep, False)
            a.kI = _arg("kI", kI, dev, (B, Nc, dI), kI.dtype) if Nc else None
            a.kI_scale = _floats("kI_scale", kI_scale, dev, (B, Nc, dI // 128), keep)
            a.draft_kI = _arg("draft_kI", draft_kI, dev, (B, T, dI), kI.dtype, True)
            a.draft_kI_scale = _floats("draft_kI_scale", draft_kI_scale, dev, (B, T, dI // 128), keep)
        if idx_out is not None:
            a.idx_out = _arg("idx_out", idx_out, dev, (B, T, k), torch.int32)
    return a, out, keep


def _attn_tree(args, kw, workspace):
    a, out, keep = tree_attn_args(*args, **kw)
    dev = out.device
    L = N.lib()
    ref = C.byref(a)
    nbytes = L.csahca_tree_workspace_size(ref)
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        a.workspace = _arg("workspace", workspace, dev, workspace.shape, workspace.dtype)
    else:
        workspace = torch.empty(nbytes + 1, dtype=torch.uint8, device=dev)
        a.workspace = workspace.data_ptr()
    a.workspace_bytes = nbytes
    st = L.compressed_attn_tree(ref, _raw_stream(dev.index))
    if st:
        N.check(st, "compressed_attn_tree")
    del keep
    return out


def compressed_attn_tree(kind, q, pos, parents, kv_cache, win, kv_raw, sinks, *, m, rope_dims, workspace=None,
                         stream=None, **kw):
    """Attention of every node of draft trees over one CSA or HCA layer's caches:
    what decode steps along each node's own path would return, in one call.

    q [B, T, H, d] raw queries of the drafted tokens; pos [B] the first drafted
    token's position; parents [B, T] as in tree_compress; kv_cache [B, N_cap, d],
    win [B, w, d] (the committed tokens'); kv_raw [B, T, d] the drafted tokens'
    raw window rows; draft [B, T, d] the entries they complete (tree_compress);
    uint8 kv_cache and draft: FP8 KV rows.
    CSA: idx_in [B, T, k] (N_cap + j names draft row j), or k with qI, wI, kI
    (kI_scale) and draft_kI (draft_kI_scale) for the lightning indexer; idx_out
    [B, T, k] receives the selection.  Rows of places without a node are left as
    they were (zero in a new out).  Returns out [B, T, H, d]."""
    return _on(stream, q.device, _attn_tree, (kind, q, pos, parents, kv_cache, win, kv_raw, sinks),
               dict(kw, m=m, rope_dims=rope_dims), workspace)


def device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    code = N.i32(0)
    N.check(N.lib().csahca_device_error(_stream(stream), C.byref(code)), "csahca_device_error")
    return int(code.value)


def selftest_bounded_wait(stream=None) -> None:
    """Launch the library's failure-path self-test: a kernel whose bounded
    wait gives up; device_error() on the same stream then reports code 1."""
    N.check(N.lib().csahca_selftest_bounded_wait(_stream(stream)), "csahca_selftest_bounded_wait")


def trace_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with CUDA events (see trace_collect)."""
    N.check(N.lib().csahca_trace_enable(int(bool(on))), "csahca_trace_enable")


def trace_collect() -> dict:
    """Per-kernel {name: (launches, total_ms)} of the launches traced since
    the last collect (synchronises their events)."""
    buf = (N.TraceEntry * 64)()
    n = C.c_int(0)
    N.check(N.lib().csahca_trace_collect(buf, 64, C.byref(n)), "csahca_trace_collect")
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms))
            for i in range(n.value)}
