"""Thin PyTorch binding of the GCA C ABI (argument marshalling only).

Each ``gca_*`` function has the name and argument order of its C entry point
and passes ``data_ptr()`` of CUDA tensors plus the current CUDA stream; every
step of the computation runs in libgca.so.  The convenience functions
``score_topk``, ``fwd``, ``bwd`` and ``decode_retrieve`` only allocate the
outputs (and workspace) with PyTorch, then call the same entry points.

GCA itself ("Efficient Length-Generalizable Attention via Causal Retrieval
for Long-Context Language Modeling", ICML 2025) is documented in
include/gca.h next to each entry point.
"""
from __future__ import annotations

import ctypes
import functools
import operator

import torch

from . import _lib
from ._lib import (GCA_BF16, GCA_F32, GcaError, GcaPagedParams, GcaParams, GcaSwaParams,
                   GcaSwaSinkParams)

_DT = {torch.bfloat16: GCA_BF16, torch.float32: GCA_F32}


def dtype_code(t: torch.dtype) -> int:
    if t not in _DT:
        raise TypeError("GCA supports bfloat16 and float32 tensors, got %s" % t)
    return _DT[t]


def make_params(*, B, Lq, S, H, d, topk, n_pool_chunks=None, landmark_dim=0, dtype=torch.bfloat16,
                off_by_one=False, include_self=False, score_scale=0.0, attn_scale=0.0) -> GcaParams:
    return GcaParams(B=B, Lq=Lq, S=S, H=H, d=d, topk=topk,
                     n_pool_chunks=(Lq // S if n_pool_chunks is None else n_pool_chunks),
                     landmark_dim=landmark_dim, dtype=dtype_code(dtype),
                     softmax_off_by_one=int(bool(off_by_one)), include_self=int(bool(include_self)),
                     score_scale=float(score_scale), attn_scale=float(attn_scale))


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("GCA entry points take CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("GCA entry points take contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, code):
    if code != 0:
        raise GcaError(fn, code)


# --- the C entry points, same names --------------------------------------------------
def gca_score_topk(params: GcaParams, landmarks, idx, score, weight, stream=None):
    _check("gca_score_topk", _lib.load().gca_score_topk(ctypes.byref(params), _p(landmarks), _p(idx),
                                                        _p(score), _p(weight), _stream(stream)))


def gca_score_topk_noisy(params: GcaParams, landmarks, noise, idx, score, weight, stream=None):
    _check("gca_score_topk_noisy", _lib.load().gca_score_topk_noisy(
        ctypes.byref(params), _p(landmarks), _p(noise), _p(idx), _p(score), _p(weight),
        _stream(stream)))


def gca_landmark_bwd_workspace_size(params: GcaParams) -> int:
    return int(_lib.load().gca_landmark_bwd_workspace_size(ctypes.byref(params)))


def gca_landmark_bwd(params: GcaParams, landmarks, idx, dscore, dlandmarks, workspace, stream=None):
    _check("gca_landmark_bwd", _lib.load().gca_landmark_bwd(
        ctypes.byref(params), _p(landmarks), _p(idx), _p(dscore), _p(dlandmarks), _p(workspace),
        workspace.numel(), _stream(stream)))


def gca_fwd(params: GcaParams, q, k, v, idx, weight, o, lse=None, stream=None):
    _check("gca_fwd", _lib.load().gca_fwd(ctypes.byref(params), _p(q), _p(k), _p(v), _p(idx),
                                          _p(weight), _p(o), _p(lse), _stream(stream)))


def gca_bwd_workspace_size(params: GcaParams) -> int:
    return int(_lib.load().gca_bwd_workspace_size(ctypes.byref(params)))


def gca_bwd(params: GcaParams, q, k, v, idx, weight, lse, dout, dq, dk, dv, dscore, workspace,
            stream=None):
    _check("gca_bwd", _lib.load().gca_bwd(ctypes.byref(params), _p(q), _p(k), _p(v), _p(idx),
                                          _p(weight), _p(lse), _p(dout), _p(dq), _p(dk), _p(dv),
                                          _p(dscore), _p(workspace), workspace.numel(),
                                          _stream(stream)))


def gca_decode_workspace_size(n_landmarks: int, D: int, topk: int) -> int:
    return int(_lib.load().gca_decode_workspace_size(n_landmarks, D, topk))


def gca_decode_retrieve(landmarks, query_landmark, N, D, topk, dtype, off_by_one, score_scale,
                        idx, score, weight, workspace, stream=None):
    _check("gca_decode_retrieve", _lib.load().gca_decode_retrieve(
        _p(landmarks), _p(query_landmark), N, D, topk, dtype_code(dtype), int(bool(off_by_one)),
        float(score_scale), _p(idx), _p(score), _p(weight), _p(workspace), workspace.numel(),
        _stream(stream)))


def gca_decode_retrieve_noalloc(landmarks, query_landmark, N, D, topk, dtype, off_by_one,
                                score_scale, idx, score, weight, stream=None):
    """Decode retrieval without a workspace argument, for callers that may not
    allocate device memory (the library's own fixed device array is used)."""
    _check("gca_decode_retrieve_noalloc", _lib.load().gca_decode_retrieve_noalloc(
        _p(landmarks), _p(query_landmark), N, D, topk, dtype_code(dtype), int(bool(off_by_one)),
        float(score_scale), _p(idx), _p(score), _p(weight), _stream(stream)))


def _pa(t):
    """Pointer of a CUDA tensor, or of a pinned host tensor (device-addressable)."""
    if t.is_cuda:
        return _p(t)
    if not t.is_pinned():
        raise ValueError("offloaded caches must be in page-locked (pinned) host memory")
    if not t.is_contiguous():
        raise ValueError("GCA entry points take contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def gca_gather_chunks(src_k, src_v, n_src, chunk_bytes, idx, topk, dst_k, dst_v, dst_idx,
                      stream=None):
    _check("gca_gather_chunks", _lib.load().gca_gather_chunks(
        _pa(src_k), _pa(src_v), n_src, chunk_bytes, _p(idx), topk, _p(dst_k), _p(dst_v),
        _p(dst_idx), _stream(stream)))


def make_swa_params(*, B, L, H, d, window, dtype=torch.bfloat16, attn_scale=0.0) -> GcaSwaParams:
    return GcaSwaParams(B=B, L=L, H=H, d=d, window=window, dtype=dtype_code(dtype),
                        attn_scale=float(attn_scale))


def gca_swa_fwd(params: GcaSwaParams, q, k, v, o, lse, stream=None):
    _check("gca_swa_fwd", _lib.load().gca_swa_fwd(ctypes.byref(params), _p(q), _p(k), _p(v), _p(o),
                                                  _p(lse), _stream(stream)))


def swa_fwd(q, k, v, *, window, attn_scale=0.0, with_lse=True):
    """Sliding-window self-attention: q, k, v [B, L, H, d] -> (o, lse [B, L, H])."""
    B, L, H, d = q.shape
    p = make_swa_params(B=B, L=L, H=H, d=d, window=window, dtype=q.dtype, attn_scale=attn_scale)
    o = torch.empty_like(q)
    lse = torch.empty(B, L, H, dtype=torch.float32, device=q.device) if with_lse else None
    gca_swa_fwd(p, q, k, v, o, lse)
    return o, lse


def gca_swa_bwd_workspace_size(params: GcaSwaParams) -> int:
    return int(_lib.load().gca_swa_bwd_workspace_size(ctypes.byref(params)))


def gca_swa_bwd(params: GcaSwaParams, q, k, v, o, lse, dout, dq, dk, dv, workspace, stream=None):
    _check("gca_swa_bwd", _lib.load().gca_swa_bwd(
        ctypes.byref(params), _p(q), _p(k), _p(v), _p(o), _p(lse), _p(dout), _p(dq), _p(dk), _p(dv),
        _p(workspace), workspace.numel(), _stream(stream)))


def swa_bwd(q, k, v, o, lse, dout, *, window, attn_scale=0.0, workspace=None):
    """Gradients of the sliding-window self-attention: returns (dq, dk, dv)."""
    B, L, H, d = q.shape
    p = make_swa_params(B=B, L=L, H=H, d=d, window=window, dtype=q.dtype, attn_scale=attn_scale)
    if workspace is None:
        workspace = torch.empty(gca_swa_bwd_workspace_size(p), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    gca_swa_bwd(p, q, k, v, o, lse, dout, dq, dk, dv, workspace)
    return dq, dk, dv


# --- windowed attention with sinks, and its paged K/V cache ----------------------------
def _token_stride(shape, stride):
    """Elements between consecutive tokens of a [..., tokens, heads, d] tensor whose heads
    are dense and whose batch rows follow each other (a dense tensor, or a slice of a
    packed projection)."""
    h, d = shape[-2], shape[-1]
    batched = len(shape) == 4 and shape[0] > 1
    step = stride[-3] if shape[-3] > 1 else (stride[0] if batched else h * d)
    if (d > 1 and stride[-1] != 1) or (h > 1 and stride[-2] != d) or step < h * d or \
            (batched and stride[0] != shape[1] * step):
        raise ValueError("token tensors need dense heads and equally spaced tokens")
    return step


def _same_device(*ts):
    """The entries launch on the current device's stream: tensors of another device (or of
    none) would be read through a foreign address.  Returns the device index."""
    dev = ts[0].get_device()
    ok = dev >= 0 and dev == torch._C._cuda_getDevice()     # (current_device() without its setup)
    for t in ts:
        ok = ok and (t is None or t.get_device() == dev)
    if not ok:
        raise ValueError("tensors must be CUDA tensors on the current device")
    return dev


def _empty_like(t):
    """A dense tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _dense(t, shape, dtype, what):
    if t is None:
        raise ValueError("%s is needed" % what)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s" % (what, tuple(shape)))


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _raw_stream(stream, dev):
    # (the stream's handle alone: building a torch.cuda.Stream costs more than a launch)
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


_INT_MAX = 2 ** 31 - 1


def _params(cls, **fields):
    """The C struct; its integers have 32 bits, of which ctypes would keep a larger one's lowest.
    (A call's window, sinks or max_q beyond that are all tokens, as the largest that fits.)"""
    for name, x in fields.items():
        if name != "attn_scale" and not -_INT_MAX <= operator.index(x) <= _INT_MAX:
            raise ValueError("%s does not fit 32 bits: %d" % (name, x))
    return cls(**fields)


def make_swa_sink_params(*, B, L, H, d, window, Hkv=None, sinks=0, dtype=torch.bfloat16,
                         attn_scale=0.0, q_stride=0, kv_stride=0) -> GcaSwaSinkParams:
    return _params(GcaSwaSinkParams, B=B, L=L, H=H, Hkv=H if Hkv is None else Hkv, d=d, window=window,
                   sinks=sinks, dtype=dtype_code(dtype), attn_scale=attn_scale, q_stride=q_stride,
                   kv_stride=kv_stride)


def gca_swa_sink_fwd_workspace_size(params: GcaSwaSinkParams) -> int:
    return int(_lib.load().gca_swa_sink_fwd_workspace_size(ctypes.byref(params)))


def gca_swa_sink_fwd(params: GcaSwaSinkParams, q, k, v, o, lse, workspace, stream=None):
    _check("gca_swa_sink_fwd", _lib.load().gca_swa_sink_fwd(
        ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(workspace),
        workspace.numel() if workspace is not None else 0, _raw_stream(stream, q.get_device())))


def gca_swa_sink_bwd_workspace_size(params: GcaSwaSinkParams) -> int:
    return int(_lib.load().gca_swa_sink_bwd_workspace_size(ctypes.byref(params)))


def gca_swa_sink_bwd(params: GcaSwaSinkParams, q, k, v, o, lse, dout, dq, dk, dv, workspace,
                     stream=None):
    _check("gca_swa_sink_bwd", _lib.load().gca_swa_sink_bwd(
        ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
        _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(),
        _raw_stream(stream, q.get_device())))


@functools.lru_cache(maxsize=256)
def _swa_sink_plan(qs, qst, ks, kst, vs, vst, qt, kt, vt, window, sinks, attn_scale):
    """What a call derives from its arguments' shapes, strides and types alone."""
    if len(qs) != 4 or len(ks) != 4 or ks != vs or ks[:2] != qs[:2] or ks[3] != qs[3]:
        raise ValueError("q must be [B, L, H, d] and k, v [B, L, Hkv, d]")
    if qt != kt or qt != vt:
        raise TypeError("q, k and v must have one dtype")
    step = _token_stride(ks, kst)
    if step != _token_stride(vs, vst):
        raise ValueError("k and v must have one token stride")
    B, L, H, d = qs
    p = make_swa_sink_params(B=B, L=L, H=H, Hkv=ks[2], d=d, window=min(window, _INT_MAX),
                             sinks=min(sinks, _INT_MAX), dtype=qt, attn_scale=attn_scale,
                             q_stride=_token_stride(qs, qst), kv_stride=step)
    return p, gca_swa_sink_fwd_workspace_size(p), gca_swa_sink_bwd_workspace_size(p)


def _swa_sink_args(q, k, v, window, sinks, attn_scale):
    # (a plan is kept by these numbers' values, never by a tensor's identity, and 30.0 is not 30)
    if type(window) is not int or type(sinks) is not int:
        window, sinks = operator.index(window), operator.index(sinks)
    return _swa_sink_plan(q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride(), q.dtype,
                          k.dtype, v.dtype, window, sinks, float(attn_scale))


_UNTOUCHED = 256       # the size of a workspace that a call does not touch
_untouched = {}


def _workspace(given, need, dev):
    if given is None:
        if need != _UNTOUCHED:
            return torch.empty(need, dtype=torch.uint8, device=dev)
        given = _untouched.get(dev)
        if given is None:
            given = _untouched[dev] = torch.empty(need, dtype=torch.uint8, device=dev)
    if given.dtype != torch.uint8 or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    return given


def swa_sink_fwd(q, k, v, *, window, sinks, attn_scale=0.0, with_lse=True, workspace=None):
    """Windowed self-attention with sinks: q [B, L, H, d], k, v [B, L, Hkv, d] (token strides
    may be those of a packed projection) -> (o [B, L, H, d], lse [B, L, H])."""
    _same_device(q, k, v, workspace)
    p, need, _ = _swa_sink_args(q, k, v, window, sinks, attn_scale)
    dev = q.device
    ws = _workspace(workspace, need, dev)
    o = _empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev) if with_lse else None
    gca_swa_sink_fwd(p, q, k, v, o, lse, ws)
    return o, lse


def swa_sink_bwd(q, k, v, o, lse, dout, *, window, sinks, attn_scale=0.0, workspace=None):
    """Gradients of swa_sink_fwd: returns dense (dq, dk, dv)."""
    _same_device(q, k, v, o, lse, dout, workspace)
    p, _, need = _swa_sink_args(q, k, v, window, sinks, attn_scale)
    _dense(o, q.shape, q.dtype, "o")
    _dense(dout, q.shape, q.dtype, "dout")
    _dense(lse, q.shape[:3], torch.float32, "lse")
    dev = q.device
    ws = _workspace(workspace, need, dev)
    dq, dk, dv = _empty_like(q), _empty_like(k), _empty_like(v)
    gca_swa_sink_bwd(p, q, k, v, o, lse, dout, dq, dk, dv, ws)
    return dq, dk, dv


def make_paged_params(*, B, total_q, Hkv, d, page, n_pages, table_width, H=None, max_q=0, window=0,
                      sinks=0, dtype=torch.bfloat16, attn_scale=0.0, q_stride=0,
                      kv_stride=0) -> GcaPagedParams:
    return _params(GcaPagedParams, B=B, total_q=total_q, max_q=max_q, H=Hkv if H is None else H,
                   Hkv=Hkv, d=d, page=page, n_pages=n_pages, table_width=table_width, window=window,
                   sinks=sinks, dtype=dtype_code(dtype), attn_scale=attn_scale, q_stride=q_stride,
                   kv_stride=kv_stride)


def gca_paged_append(params: GcaPagedParams, k_new, v_new, cu_q, kv_len, table, k_cache, v_cache,
                     stream=None):
    _check("gca_paged_append", _lib.load().gca_paged_append(
        ctypes.byref(params), _ptr(k_new), _ptr(v_new), _ptr(cu_q), _ptr(kv_len), _ptr(table),
        _ptr(k_cache), _ptr(v_cache), _raw_stream(stream, k_cache.get_device())))


def gca_paged_attn_workspace_size(params: GcaPagedParams) -> int:
    return int(_lib.load().gca_paged_attn_workspace_size(ctypes.byref(params)))


def gca_paged_attn(params: GcaPagedParams, q, k_cache, v_cache, cu_q, kv_len, table, o, lse,
                   workspace, stream=None):
    _check("gca_paged_attn", _lib.load().gca_paged_attn(
        ctypes.byref(params), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_q), _ptr(kv_len),
        _ptr(table), _ptr(o), _ptr(lse), _ptr(workspace),
        workspace.numel() if workspace is not None else 0, _raw_stream(stream, q.get_device())))


@functools.lru_cache(maxsize=256)
def _paged_plan(ts, tst, cache, v_cache, table, cu_q, kv_len, dt, k_dt, v_dt, attend, max_q, window,
                sinks, attn_scale):
    """What a paged call derives from shapes, strides and types alone: parameters and
    workspace size."""
    if k_dt != dt or v_dt != dt:
        raise TypeError("the caches must have the token tensors' dtype")
    if len(cache) != 4 or len(table) != 2:
        raise ValueError("caches must be [n_pages, page, Hkv, d] and table [B, table_width]")
    n_pages, page, Hkv, d = cache
    B, width = table
    if v_cache != cache or tuple(cu_q) != (B + 1,) or tuple(kv_len) != (B,):
        raise ValueError("v_cache must be like k_cache, cu_q [%d] and kv_len [%d]" % (B + 1, B))
    if len(ts) != 3 or ts[2] != d or (not attend and ts[1] != Hkv):
        raise ValueError("token tensors must be [T, heads, d] like the cache")
    step = _token_stride(ts, tst)
    p = make_paged_params(B=B, total_q=ts[0], max_q=min(max_q, _INT_MAX), H=ts[1], Hkv=Hkv, d=d,
                          page=page, n_pages=n_pages, table_width=width,
                          window=min(window, _INT_MAX), sinks=min(sinks, _INT_MAX), dtype=dt,
                          attn_scale=attn_scale, q_stride=step if attend else 0,
                          kv_stride=0 if attend else step)
    return p, gca_paged_attn_workspace_size(p) if attend else 0


def _paged_args(tok, k_cache, v_cache, table, cu_q, kv_len, attend, max_q, window=0, sinks=0, attn_scale=0.0):
    if type(max_q) is not int or type(window) is not int or type(sinks) is not int:
        max_q, window, sinks = operator.index(max_q), operator.index(window), operator.index(sinks)
    i32 = torch.int32
    if table.dtype != i32 or cu_q.dtype != i32 or kv_len.dtype != i32:
        raise TypeError("table, cu_q and kv_len must be int32")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and table.is_contiguous() and
            cu_q.is_contiguous() and kv_len.is_contiguous()):
        raise ValueError("the caches, table, cu_q and kv_len must be contiguous")
    return _paged_plan(tok.shape, tok.stride(), k_cache.shape, v_cache.shape, table.shape, cu_q.shape,
                       kv_len.shape, tok.dtype, k_cache.dtype, v_cache.dtype, attend, max_q, window,
                       sinks, float(attn_scale))


def paged_append(k_new, v_new, k_cache, v_cache, table, cu_q, kv_len, *, max_q=0):
    """Write new tokens into the paged cache, in place: k_new, v_new [T, Hkv, d]; caches
    [n_pages, page, Hkv, d]; table [B, table_width], cu_q [B + 1], kv_len [B] int32 on the
    device.  ``kv_len`` counts the new tokens."""
    _same_device(k_cache, v_cache, table, cu_q, kv_len, k_new, v_new)
    p, _ = _paged_args(k_new, k_cache, v_cache, table, cu_q, kv_len, False, max_q)
    if v_new.dtype != k_new.dtype:
        raise TypeError("k_new and v_new must have one dtype")
    if v_new.shape != k_new.shape or (v_new.stride() != k_new.stride() and
                                      _token_stride(v_new.shape, v_new.stride()) != p.kv_stride):
        raise ValueError("k_new and v_new must have one shape and one token stride")
    gca_paged_append(p, k_new, v_new, cu_q, kv_len, table, k_cache, v_cache)


def paged_attn(q, k_cache, v_cache, table, cu_q, kv_len, *, max_q=0, window=0, sinks=0,
               attn_scale=0.0, with_lse=False, out=None, workspace=None):
    """Attention of the new tokens q [T, H, d] over the paged cache -> (o [T, H, d], lse [T, H]
    or None).  ``max_q`` bounds the new tokens of one sequence (0: T); a host that knows it
    saves work.  Rows of o behind cu_q[B] are left as they were (``out`` supplies o)."""
    _same_device(q, k_cache, v_cache, table, cu_q, kv_len, out, workspace)
    p, need = _paged_args(q, k_cache, v_cache, table, cu_q, kv_len, True, max_q, window, sinks, attn_scale)
    dev = q.device
    ws = _workspace(workspace, need, dev)
    if out is None:
        out = _empty_like(q)
    else:
        _dense(out, q.shape, q.dtype, "out")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev) if with_lse else None
    gca_paged_attn(p, q, k_cache, v_cache, cu_q, kv_len, table, out, lse, ws)
    return out, lse


def gather_chunks(cache_k, cache_v, idx):
    """cache_k/v [n_chunks, S, H, d] (device or pinned host) -> compact
    pools [1, topk*S, H, d] on the device and the remapped idx [1, 1, topk]."""
    n, S, H, d = cache_k.shape
    topk = idx.numel()
    dev = idx.device
    dk = torch.empty(topk * S, H, d, dtype=cache_k.dtype, device=dev)
    dv = torch.empty_like(dk)
    di = torch.empty(topk, dtype=torch.int32, device=dev)
    chunk_bytes = S * H * d * cache_k.element_size()
    gca_gather_chunks(cache_k, cache_v, n, chunk_bytes, idx, topk, dk, dv, di)
    return dk.view(1, topk * S, H, d), dv.view(1, topk * S, H, d), di.view(1, 1, topk)


def gca_get_status(stream=None) -> int:
    return int(_lib.load().gca_get_status(_stream(stream)))


def gca_debug_stall_next_decode(wait_ns: int):
    """Test-only: the next decode launch on this thread withholds one stage and
    bounds its waits by ``wait_ns`` (include/gca_debug.h)."""
    _check("gca_debug_stall_next_decode", _lib.load().gca_debug_stall_next_decode(int(wait_ns)))


def gca_last_launch_count() -> int:
    return int(_lib.load().gca_last_launch_count())


def gca_synth_fill_hash(dst, seed: int, tensor_id: int, first_elem: int = 0, stream=None):
    _check("gca_synth_fill_hash", _lib.load().gca_synth_fill_hash(
        _p(dst), dst.numel(), dtype_code(dst.dtype), seed, tensor_id, first_elem, _stream(stream)))


# --- allocating helpers ----------------------------------------------------------------
def score_topk(landmarks, *, S, H, d, topk, off_by_one=False, include_self=False, score_scale=0.0):
    """landmarks [B, nC, D] -> idx int32, score fp32, weight fp32, each [B, nC, topk]."""
    B, nC, D = landmarks.shape
    p = make_params(B=B, Lq=nC * S, S=S, H=H, d=d, topk=topk, landmark_dim=D,
                    dtype=landmarks.dtype, off_by_one=off_by_one, include_self=include_self,
                    score_scale=score_scale)
    dev = landmarks.device
    idx = torch.empty(B, nC, topk, dtype=torch.int32, device=dev)
    score = torch.empty(B, nC, topk, dtype=torch.float32, device=dev)
    weight = torch.empty(B, nC, topk, dtype=torch.float32, device=dev)
    gca_score_topk(p, landmarks, idx, score, weight)
    return idx, score, weight


def score_topk_noisy(landmarks, noise, *, S, H, d, topk, off_by_one=False, include_self=False,
                     score_scale=0.0):
    """Like score_topk, selecting by score + noise (noise [B, nC, nC] fp32)."""
    B, nC, D = landmarks.shape
    p = make_params(B=B, Lq=nC * S, S=S, H=H, d=d, topk=topk, landmark_dim=D,
                    dtype=landmarks.dtype, off_by_one=off_by_one, include_self=include_self,
                    score_scale=score_scale)
    dev = landmarks.device
    idx = torch.empty(B, nC, topk, dtype=torch.int32, device=dev)
    score = torch.empty(B, nC, topk, dtype=torch.float32, device=dev)
    weight = torch.empty(B, nC, topk, dtype=torch.float32, device=dev)
    gca_score_topk_noisy(p, landmarks, noise, idx, score, weight)
    return idx, score, weight


def landmark_bwd(landmarks, idx, dscore, *, S, H, d, score_scale=0.0):
    """dLoss/dlandmarks [B, nC, D] from dLoss/dr."""
    B, nC, D = landmarks.shape
    p = make_params(B=B, Lq=nC * S, S=S, H=H, d=d, topk=idx.shape[-1], landmark_dim=D,
                    dtype=landmarks.dtype, score_scale=score_scale)
    ws = torch.empty(gca_landmark_bwd_workspace_size(p), dtype=torch.uint8, device=landmarks.device)
    dl = torch.empty_like(landmarks)
    gca_landmark_bwd(p, landmarks, idx, dscore, dl, ws)
    return dl


def fwd(q, k, v, idx, weight, *, S, attn_scale=0.0, with_lse=True):
    """q [B, Lq, H, d]; k, v [B, nP*S, H, d]; idx, weight [B, Lq/S, topk] -> (o, lse)."""
    B, Lq, H, d = q.shape
    topk = idx.shape[-1]
    p = make_params(B=B, Lq=Lq, S=S, H=H, d=d, topk=topk, n_pool_chunks=k.shape[1] // S,
                    dtype=q.dtype, attn_scale=attn_scale)
    o = torch.empty_like(q)
    lse = torch.empty(B, Lq, H, topk, dtype=torch.float32, device=q.device) if with_lse else None
    gca_fwd(p, q, k, v, idx, weight, o, lse)
    return o, lse


def bwd(q, k, v, idx, weight, lse, dout, *, S, attn_scale=0.0, workspace=None):
    """Returns (dq, dk, dv, dscore)."""
    B, Lq, H, d = q.shape
    topk = idx.shape[-1]
    p = make_params(B=B, Lq=Lq, S=S, H=H, d=d, topk=topk, n_pool_chunks=k.shape[1] // S,
                    dtype=q.dtype, attn_scale=attn_scale)
    need = gca_bwd_workspace_size(p)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    dscore = torch.empty(B, Lq // S, topk, dtype=torch.float32, device=q.device)
    gca_bwd(p, q, k, v, idx, weight, lse, dout, dq, dk, dv, dscore, workspace)
    return dq, dk, dv, dscore


def decode_retrieve(landmarks, query_landmark, *, topk, off_by_one=False, score_scale=0.0,
                    workspace=None):
    """landmarks [N, D], query_landmark [D] -> idx, score, weight [topk]."""
    N, D = landmarks.shape
    need = gca_decode_workspace_size(N, D, topk)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=landmarks.device)
    dev = landmarks.device
    idx = torch.empty(topk, dtype=torch.int32, device=dev)
    score = torch.empty(topk, dtype=torch.float32, device=dev)
    weight = torch.empty(topk, dtype=torch.float32, device=dev)
    gca_decode_retrieve(landmarks, query_landmark, N, D, topk, landmarks.dtype, off_by_one,
                        score_scale, idx, score, weight, workspace)
    return idx, score, weight
