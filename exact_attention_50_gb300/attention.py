"""PyTorch-facing API over the C ABI.  PyTorch supplies device memory and the current stream;
every step of the computation runs in libattn_gb300.so's kernels.

- ``flash_attention(q, k, v, causal=True, scale=None)``: [batch, heads, seq, head_dim] tensors,
  GQA when k/v have fewer heads, differentiable (Aule-Attention API, jeff.news/article/688:
  causal defaults to True, scale to 1/sqrt(head_dim)).
- ``flash_attn_varlen_qkvpacked_func(qkv, cu_seqlens, max_seqlen, ...)``: packed variable-length
  forward with the flash_attn signature (Turing varlen article, ewbang.com/...1000323363:
  causal defaults to False; window_size, softcap, alibi_slopes and return_attn_probs are
  rejected; dropout is not provided).
- ``fwd``, ``bwd``, ``fwd_varlen``: explicit calls that also return the LSE / take workspaces.
- ``kvcache8_append``, ``fwd_kvcache8``: a KV cache held in 8 bits with a scale per block of
  tokens and head, and attention over it; ``kvcache_weights``, ``kvcache_evict``: the attention
  weight that each cached key has received, and eviction by it.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _lib

_DT8 = {torch.int8: _lib.ATTN_CACHE_I8, torch.float8_e4m3fn: _lib.ATTN_CACHE_E4M3}
_DT = {torch.float32: _lib.ATTN_F32, torch.float16: _lib.ATTN_F16, torch.bfloat16: _lib.ATTN_BF16}


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}: float16, bfloat16 or float32")
    return _DT[t.dtype]


def _require(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _scale_arg(scale) -> float:
    if scale is None:
        return 0.0
    scale = float(scale)
    if not (scale > 0.0) or math.isinf(scale):
        raise ValueError("scale must be a positive finite number (None = 1/sqrt(head_dim))")
    return scale


def get_device_status() -> int:
    """Synchronises the current stream and returns/clears the device status word."""
    return _lib.attn_get_device_status(_stream())


def fwd(q, k, v, causal: bool, scale=None, out_f32: bool = False, with_lse: bool = True):
    """Dense forward.  q [B,Hq,N,d]; k, v [B,Hkv,N,d].  Returns (o, lse or None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, q.dtype)
    if q.dim() != 4 or k.shape != v.shape or k.dim() != 4:
        raise ValueError("q must be [B,Hq,N,d] and k, v [B,Hkv,N,d]")
    B, Hq, N, d = q.shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError("q and k/v disagree on batch, sequence length or head_dim")
    Hkv = k.shape[1]
    o = torch.empty(q.shape, dtype=torch.float32 if out_f32 else q.dtype, device=q.device)
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if with_lse else None
    st = _lib.attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                       lse.data_ptr() if lse is not None else None, B, Hq, Hkv, N, d, causal,
                       _scale_arg(scale), _dtype_code(q), _lib.ATTN_FLAG_OUT_F32 if out_f32 else 0, _stream())
    _lib._check(st, "attn_fwd")
    return o, lse


def _bwd_flags(out_f32: bool, deterministic: bool) -> int:
    return (_lib.ATTN_FLAG_OUT_F32 if out_f32 else 0) | (_lib.ATTN_FLAG_DETERMINISTIC if deterministic else 0)


def bwd(q, k, v, o, lse, dout, causal: bool, scale=None, out_f32: bool = False, workspace=None,
        deterministic: bool = False):
    """Dense backward.  Returns (dq, dk, dv).  deterministic: dq bitwise reproducible (slower)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _require(t, n, q.dtype)
    _require(lse, "lse", torch.float32)
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if o.shape != q.shape or dout.shape != q.shape or lse.shape != (B, Hq, N):
        raise ValueError("o and dout must be shaped like q, lse [B,Hq,N]")
    odt = torch.float32 if out_f32 else q.dtype
    dq = torch.empty(q.shape, dtype=odt, device=q.device)
    dk = torch.empty(k.shape, dtype=odt, device=q.device)
    dv = torch.empty(v.shape, dtype=odt, device=q.device)
    nbytes = _lib.attn_bwd_workspace_bytes(B, Hq, N, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    st = _lib.attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                       dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.numel(),
                       B, Hq, Hkv, N, d, causal, _scale_arg(scale), _dtype_code(q),
                       _bwd_flags(out_f32, deterministic), _stream())
    _lib._check(st, "attn_bwd")
    return dq, dk, dv


def bwd_cross(q, k, v, o, lse, dout, causal: bool, scale=None, out_f32: bool = False, workspace=None,
              deterministic: bool = False):
    """Cross-attention backward (any Nq, Nk; bottom-right causal alignment: query i sees key j
    iff j <= i + Nk - Nq).  q, o, dout [B,Hq,Nq,d]; k, v [B,Hkv,Nk,d]; lse [B,Hq,Nq] from
    fwd_kvcache without cache lengths.  Query rows that see no key get dq = 0.
    Returns (dq, dk, dv)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _require(t, n, q.dtype)
    _require(lse, "lse", torch.float32)
    B, Hq, Nq, d = q.shape
    _, Hkv, Nk, _ = k.shape
    if v.shape != k.shape or o.shape != q.shape or dout.shape != q.shape or lse.shape != (B, Hq, Nq):
        raise ValueError("o and dout must be shaped like q, v like k, lse [B,Hq,Nq]")
    odt = torch.float32 if out_f32 else q.dtype
    dq = torch.empty(q.shape, dtype=odt, device=q.device)
    dk = torch.empty(k.shape, dtype=odt, device=q.device)
    dv = torch.empty(v.shape, dtype=odt, device=q.device)
    flags = _bwd_flags(out_f32, deterministic)
    nbytes = _lib.attn_bwd_cross_workspace_bytes(B, Hq, Nq, Nk, d, _dtype_code(q), flags)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    st = _lib.attn_bwd_cross(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.numel(),
                             B, Hq, Hkv, Nq, Nk, d, causal, _scale_arg(scale), _dtype_code(q), flags, _stream())
    _lib._check(st, "attn_bwd_cross")
    return dq, dk, dv


def fwd_varlen(qkv, cu_seqlens, max_seqlen: int, causal: bool, scale=None, out_f32: bool = False,
               with_lse: bool = True):
    """Packed varlen forward.  qkv [T,3,H,d], cu_seqlens int32 [nseq+1] (device).
    Returns (out [T,H,d], lse [H,T] or None)."""
    _require(qkv, "qkv")
    _require(cu_seqlens, "cu_seqlens", torch.int32)
    if qkv.dim() != 4 or qkv.shape[1] != 3:
        raise ValueError("qkv must be [total_tokens, 3, heads, head_dim]")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be 1-D with batch_size + 1 entries")
    T, _, H, d = qkv.shape
    nseq = cu_seqlens.numel() - 1
    out = torch.empty((T, H, d), dtype=torch.float32 if out_f32 else qkv.dtype, device=qkv.device)
    lse = torch.empty((H, T), dtype=torch.float32, device=qkv.device) if with_lse else None
    st = _lib.attn_fwd_varlen(qkv.data_ptr(), cu_seqlens.data_ptr(), nseq, T, int(max_seqlen), out.data_ptr(),
                              lse.data_ptr() if lse is not None else None, H, d, causal, _scale_arg(scale),
                              _dtype_code(qkv), _lib.ATTN_FLAG_OUT_F32 if out_f32 else 0, _stream())
    _lib._check(st, "attn_fwd_varlen")
    return out, lse


def bwd_varlen(qkv, out, lse, dout, cu_seqlens, max_seqlen: int, causal: bool, scale=None, out_f32: bool = False,
               workspace=None, deterministic: bool = False):
    """Packed varlen backward.  qkv [T,3,H,d], out / dout [T,H,d], lse [H,T] (from fwd_varlen),
    cu_seqlens int32 [nseq+1] (device).  Returns dqkv [T,3,H,d]."""
    _require(qkv, "qkv")
    for t, n in ((out, "out"), (dout, "dout")):
        _require(t, n, qkv.dtype)
    _require(lse, "lse", torch.float32)
    _require(cu_seqlens, "cu_seqlens", torch.int32)
    T, _, H, d = qkv.shape
    if out.shape != (T, H, d) or dout.shape != (T, H, d) or lse.shape != (H, T):
        raise ValueError("out and dout must be [T,H,d], lse [H,T]")
    nseq = cu_seqlens.numel() - 1
    dqkv = torch.zeros(qkv.shape, dtype=torch.float32 if out_f32 else qkv.dtype, device=qkv.device)
    nbytes = _lib.attn_bwd_varlen_workspace_bytes(T, H, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=qkv.device)
    st = _lib.attn_bwd_varlen(qkv.data_ptr(), out.data_ptr(), dout.data_ptr(), lse.data_ptr(), cu_seqlens.data_ptr(),
                              nseq, T, int(max_seqlen), dqkv.data_ptr(), workspace.data_ptr(), workspace.numel(), H,
                              d, causal, _scale_arg(scale), _dtype_code(qkv),
                              _bwd_flags(out_f32, deterministic), _stream())
    _lib._check(st, "attn_bwd_varlen")
    return dqkv


def kvcache_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int, num_splits: int = 0) -> int:
    """Bytes of the device workspace fwd_kvcache needs for these sizes and num_splits."""
    return _lib.attn_fwd_kvcache_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits)


def fwd_kvcache(q, k_cache, v_cache, cache_seqlens=None, causal: bool = False, scale=None, num_splits: int = 0,
                out_f32: bool = False, with_lse: bool = True, workspace=None):
    """KV-cache / cross-attention forward.  q [B,Hq,Nq,d]; k_cache, v_cache [B,Hkv,Nk,d];
    cache_seqlens int32 [B] on the device (None: Nk keys each).  causal aligns the queries with
    the last Nq keys of each cache.  num_splits: key ranges per (batch, kv head), 0 = chosen
    from the sizes.  Returns (o [B,Hq,Nq,d], lse [B,Hq,Nq] or None)."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n, q.dtype)
    if q.dim() != 4 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("q must be [B,Hq,Nq,d] and k_cache, v_cache [B,Hkv,Nk,d]")
    B, Hq, Nq, d = q.shape
    _, Hkv, Nk, dk = k_cache.shape
    if k_cache.shape[0] != B or dk != d:
        raise ValueError("q and the caches disagree on batch or head_dim")
    lens_ptr = None
    if cache_seqlens is not None:
        _require(cache_seqlens, "cache_seqlens", torch.int32)
        if cache_seqlens.shape != (B,) or cache_seqlens.device != q.device:
            raise ValueError("cache_seqlens must be int32 [B] on q's device")
        lens_ptr = cache_seqlens.data_ptr()
    o = torch.empty(q.shape, dtype=torch.float32 if out_f32 else q.dtype, device=q.device)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if with_lse else None
    need = _lib.attn_fwd_kvcache_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits) if B * Nq > 0 else 0
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    elif workspace.numel() < need:
        raise ValueError(f"workspace too small: {workspace.numel()} < {need} bytes")
    st = _lib.attn_fwd_kvcache(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), lens_ptr, o.data_ptr(),
                               lse.data_ptr() if lse is not None else None, workspace.data_ptr(), workspace.numel(),
                               B, Hq, Hkv, Nq, Nk, d, causal, _scale_arg(scale), num_splits, _dtype_code(q),
                               _lib.ATTN_FLAG_OUT_F32 if out_f32 else 0, _stream())
    _lib._check(st, "attn_fwd_kvcache")
    return o, lse


def _fit(dev: int, *tensors) -> bool:
    """Contiguous tensors on GPU `dev`; None stands for an optional one that is not given."""
    for t in tensors:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            return False
    return dev >= 0


def _check_sizes(*shapes):
    """C takes sizes in 32 bits."""
    for s in shapes:
        if max(s) >= 2 ** 31:
            raise ValueError("every size must be below 2**31")


def _explain(*named):
    """Raises what is wrong with the arguments of a cache call: (tensor, name, dtype, optional) each,
    contiguous tensors on the first one's GPU."""
    for t, name, dtype, optional in named:
        if t is None and optional:
            continue
        _require(t, name, dtype)
        if t.device != named[0][0].device:
            raise ValueError(f"{name} must be on {named[0][1]}'s device")
    raise TypeError("the tensors' types do not fit together")


def _on_device(dev: int, call, *args) -> int:
    """call(*args, stream) with `dev` as the current device, on its current stream."""
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        return call(*args, stream)
    with torch.cuda.device(dev):
        return call(*args, stream)


def _lens_ptr(t, name: str, B: int):
    if t is None:
        return None
    if t.shape != (B,):
        raise ValueError(f"{name} must be int32 [B]")
    return t.data_ptr()


def _check_cache8(k8, v8, k_scale, v_scale, block: int):
    """Shapes of an 8-bit cache; returns them and the C code of its type."""
    code = _DT8.get(k8.dtype)
    if code is None:
        raise TypeError(f"unsupported cache dtype {k8.dtype}: int8 or float8_e4m3fn")
    if block not in (16, 32, 64, 128):
        raise ValueError("block must be 16, 32, 64 or 128")
    shape = k8.shape
    if len(shape) != 4 or shape != v8.shape:
        raise ValueError("k8 and v8 must be [B,Hkv,Nk,d]")
    B, Hkv, Nk, d = shape
    scales = (B, Hkv, -(-Nk // block))
    if k_scale.shape != scales or v_scale.shape != scales:
        raise ValueError("k_scale and v_scale must be [B,Hkv,ceil(Nk/block)]")
    return B, Hkv, Nk, d, code


def kvcache8_append(k8, v8, k_scale, v_scale, k_new, v_new, cache_seqlens=None, new_seqlens=None, block: int = 64):
    """Writes tokens into an 8-bit cache, in place.  k8, v8 [B,Hkv,Nk,d] int8 or float8_e4m3fn;
    k_scale, v_scale float32 [B,Hkv,ceil(Nk/block)]; k_new, v_new [B,Hkv,Nn,d].  Batch b's tokens
    go behind its first cache_seqlens[b] (int32 [B] on the device; None: an empty cache), the
    first new_seqlens[b] of them (None: Nn); the caller advances the lengths.  block: tokens per
    scale, 16, 32, 64 or 128."""
    f32, i32 = torch.float32, torch.int32
    try:
        dev = k8.get_device()
        fit = (_fit(dev, k8, v8, k_scale, v_scale, k_new, v_new, cache_seqlens, new_seqlens) and v8.dtype is k8.dtype
               and k_scale.dtype is f32 and v_scale.dtype is f32 and v_new.dtype is k_new.dtype
               and (cache_seqlens is None or cache_seqlens.dtype is i32) and (new_seqlens is None or new_seqlens.dtype is i32))
    except AttributeError:  # not a tensor
        fit = False
    if not fit:
        _explain((k8, "k8", None, False), (v8, "v8", getattr(k8, "dtype", None), False), (k_scale, "k_scale", f32, False),
                 (v_scale, "v_scale", f32, False), (k_new, "k_new", None, False),
                 (v_new, "v_new", getattr(k_new, "dtype", None), False), (cache_seqlens, "cache_seqlens", i32, True),
                 (new_seqlens, "new_seqlens", i32, True))
    B, Hkv, Nk, d, code = _check_cache8(k8, v8, k_scale, v_scale, block)
    shape = k_new.shape
    if len(shape) != 4 or shape != v_new.shape or shape[0] != B or shape[1] != Hkv or shape[3] != d:
        raise ValueError("k_new and v_new must be [B,Hkv,Nn,d]")
    _check_sizes(k8.shape, shape)
    st = _on_device(dev, _lib.attn_kvcache8_append, k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                    k_new.data_ptr(), v_new.data_ptr(), _lens_ptr(cache_seqlens, "cache_seqlens", B),
                    _lens_ptr(new_seqlens, "new_seqlens", B), B, Hkv, shape[2], Nk, d, block, _dtype_code(k_new),
                    code)
    _lib._check(st, "attn_kvcache8_append")


@functools.lru_cache(maxsize=1024)
def kvcache8_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    """Bytes of the device workspace fwd_kvcache8 needs for these sizes."""
    return _lib.attn_fwd_kvcache8_workspace_bytes(B, Hq, Hkv, Nq, Nk, d)


def fwd_kvcache8(q, k8, v8, k_scale, v_scale, cache_seqlens=None, causal: bool = False, scale=None, block: int = 64,
                 out_f32: bool = False, with_lse: bool = True, workspace=None):
    """fwd_kvcache over an 8-bit cache.  q [B,Hq,Nq,d] float16 or bfloat16; k8, v8, k_scale,
    v_scale and block as kvcache8_append writes them; cache_seqlens int32 [B] on the device (None:
    Nk tokens each).  Calls that may run at the same time need a workspace each; with more than 64
    rows per kv head (Hq / Hkv * Nq) it takes up to 1 GB, or 4 * Nk * d bytes where a single kv head has
    more.  Returns (o [B,Hq,Nq,d], lse [B,Hq,Nq] or None)."""
    f32, i32 = torch.float32, torch.int32
    try:
        dev = q.get_device()
        fit = (_fit(dev, q, k8, v8, k_scale, v_scale, cache_seqlens, workspace) and v8.dtype is k8.dtype
               and k_scale.dtype is f32 and v_scale.dtype is f32 and (cache_seqlens is None or cache_seqlens.dtype is i32))
    except AttributeError:  # not a tensor
        fit = False
    if not fit:
        _explain((q, "q", None, False), (k8, "k8", None, False), (v8, "v8", getattr(k8, "dtype", None), False),
                 (k_scale, "k_scale", f32, False), (v_scale, "v_scale", f32, False),
                 (cache_seqlens, "cache_seqlens", i32, True), (workspace, "workspace", None, True))
    B, Hkv, Nk, d, code = _check_cache8(k8, v8, k_scale, v_scale, block)
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != d:
        raise ValueError("q must be [B,Hq,Nq,d], with the cache's batch and head_dim")
    _check_sizes(shape, k8.shape)
    Hq, Nq = shape[1], shape[2]
    device = q.device
    o = torch.empty_like(q, dtype=torch.float32) if out_f32 else torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=device) if with_lse else None
    if workspace is None:
        need = kvcache8_workspace_bytes(B, Hq, Hkv, Nq, Nk, d)
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    st = _on_device(dev, _lib.attn_fwd_kvcache8, q.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
                    v_scale.data_ptr(), _lens_ptr(cache_seqlens, "cache_seqlens", B), o.data_ptr(),
                    lse.data_ptr() if with_lse else None, None if workspace is None else workspace.data_ptr(),
                    0 if workspace is None else workspace.nbytes, B, Hq, Hkv, Nq, Nk, d, block, causal,
                    _scale_arg(scale), _dtype_code(q), code, _lib.ATTN_FLAG_OUT_F32 if out_f32 else 0)
    _lib._check(st, "attn_fwd_kvcache8")
    return o, lse


def kvcache_weights(q, k_cache, lse, cache_seqlens=None, causal: bool = False, scale=None, weights=None, out=None):
    """The attention weight that each cached key receives from these queries, added up over them
    and over the query heads of its kv head.  q [B,Hq,Nq,d], k_cache [B,Hkv,Nk,d], cache_seqlens,
    causal and scale as given to fwd_kvcache (or fwd), and lse [B,Hq,Nq] as it returned it.
    weights float32 [B,Hkv,Nk]: what earlier queries added up to (None: zeros).  out: where to
    write (may be weights).  Returns float32 [B,Hkv,Nk]."""
    f32, i32 = torch.float32, torch.int32
    try:
        dev = q.get_device()
        fit = (_fit(dev, q, k_cache, lse, cache_seqlens, weights, out) and k_cache.dtype is q.dtype and lse.dtype is f32
               and (cache_seqlens is None or cache_seqlens.dtype is i32) and (weights is None or weights.dtype is f32)
               and (out is None or out.dtype is f32))
    except AttributeError:  # not a tensor
        fit = False
    if not fit:
        _explain((q, "q", None, False), (k_cache, "k_cache", getattr(q, "dtype", None), False), (lse, "lse", f32, False),
                 (cache_seqlens, "cache_seqlens", i32, True), (weights, "weights", f32, True), (out, "out", f32, True))
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q must be [B,Hq,Nq,d] and k_cache [B,Hkv,Nk,d]")
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k_cache.shape
    if Bk != B or dk != d:
        raise ValueError("q and the cache disagree on batch or head_dim")
    _check_sizes(q.shape, k_cache.shape)
    if lse.shape != (B, Hq, Nq):
        raise ValueError("lse must be [B,Hq,Nq]")
    for t, n in ((weights, "weights"), (out, "out")):
        if t is not None and t.shape != (B, Hkv, Nk):
            raise ValueError(f"{n} must be [B,Hkv,Nk]")
    if out is None:
        out = torch.empty((B, Hkv, Nk), dtype=torch.float32, device=q.device)
    st = _on_device(dev, _lib.attn_kvcache_weights, q.data_ptr(), k_cache.data_ptr(), lse.data_ptr(),
                    _lens_ptr(cache_seqlens, "cache_seqlens", B), None if weights is None else weights.data_ptr(),
                    out.data_ptr(), B, Hq, Hkv, Nq, Nk, d, causal, _scale_arg(scale), _dtype_code(q))
    _lib._check(st, "attn_kvcache_weights")
    return out


def kvcache_evict(k_cache, v_cache, weights, keep: int, recent: int, cache_seqlens=None, out=None):
    """Cuts caches down to their last `recent` keys and, of the others, the `keep` of the largest
    weights (per batch and kv head; equal weights: the lowest positions), in the order of their
    positions.  k_cache, v_cache [B,Hkv,Nk,d]; weights float32 [B,Hkv,Nk]; cache_seqlens int32 [B]
    on the device (None: Nk each).  out: (k_out, v_out) [B,Hkv,capacity,d] to write into, capacity
    >= keep + recent; rows past the kept ones are left as they are (None: new caches of capacity
    keep + recent, zeros past the kept ones).  Returns (k_out, v_out, weights
    [B,Hkv,capacity], index int32 [B,Hkv,keep+recent] with -1 past the kept keys, lengths int32
    [B])."""
    _require(k_cache, "k_cache")
    keep, recent = int(keep), int(recent)
    if keep < 0 or recent < 0 or keep + recent < 1:
        raise ValueError("keep and recent must not be negative, nor both zero")
    if k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [B,Hkv,Nk,d]")
    B, Hkv, Nk, d = k_cache.shape
    device = k_cache.device
    if out is None:
        out = tuple(torch.zeros((B, Hkv, keep + recent, d), dtype=k_cache.dtype, device=device) for _ in range(2))
    k_out, v_out = out
    dt, f32, i32 = k_cache.dtype, torch.float32, torch.int32
    try:
        dev = k_cache.get_device()
        fit = (_fit(dev, k_cache, v_cache, weights, k_out, v_out, cache_seqlens) and v_cache.dtype is dt and weights.dtype is f32
               and k_out.dtype is dt and v_out.dtype is dt and (cache_seqlens is None or cache_seqlens.dtype is i32))
    except AttributeError:  # not a tensor
        fit = False
    if not fit:
        _explain((k_cache, "k_cache", None, False), (v_cache, "v_cache", dt, False), (weights, "weights", f32, False),
                 (k_out, "k_out", dt, False), (v_out, "v_out", dt, False), (cache_seqlens, "cache_seqlens", i32, True))
    if v_cache.shape != k_cache.shape or weights.shape != (B, Hkv, Nk):
        raise ValueError("k_cache and v_cache must be [B,Hkv,Nk,d] and weights [B,Hkv,Nk]")
    if k_out.dim() != 4 or k_out.shape != v_out.shape or k_out.shape[:2] != (B, Hkv) or k_out.shape[3] != d:
        raise ValueError("k_out and v_out must be [B,Hkv,capacity,d]")
    _check_sizes(k_cache.shape, k_out.shape)
    cap = k_out.shape[2]
    if cap < keep + recent:
        raise ValueError("the capacity of k_out and v_out must be at least keep + recent")
    w_out = torch.empty((B, Hkv, cap), dtype=torch.float32, device=device)
    index = torch.empty((B, Hkv, keep + recent), dtype=torch.int32, device=device)
    lens = torch.empty((B,), dtype=torch.int32, device=device)
    st = _on_device(dev, _lib.attn_kvcache_evict, k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(),
                    _lens_ptr(cache_seqlens, "cache_seqlens", B), k_out.data_ptr(), v_out.data_ptr(), w_out.data_ptr(),
                    index.data_ptr(), lens.data_ptr(), B, Hkv, Nk, cap, d, keep, recent, _dtype_code(k_cache))
    _lib._check(st, "attn_kvcache_evict")
    return k_out, v_out, w_out, index, lens


class _AttnFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, deterministic):
        # queries and keys of different lengths: cross-attention (bottom-right causal alignment)
        ctx.cross = q.dim() == 4 and k.dim() == 4 and q.shape[2] != k.shape[2]
        if ctx.cross:
            o, lse = fwd_kvcache(q, k, v, None, causal, scale)
        else:
            o, lse = fwd(q, k, v, causal, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale, ctx.deterministic = causal, scale, deterministic
        return o

    @staticmethod
    def backward(ctx, dout):
        q, k, v, o, lse = ctx.saved_tensors
        call = bwd_cross if ctx.cross else bwd
        dq, dk, dv = call(q, k, v, o, lse, dout.contiguous(), ctx.causal, ctx.scale, deterministic=ctx.deterministic)
        return dq, dk, dv, None, None, None


def flash_attention(q, k, v, causal: bool = True, scale=None, deterministic: bool = False):
    """Exact attention of [B,Hq,Nq,d] queries over [B,Hkv,Nk,d] keys/values (Hq % Hkv == 0).
    Nq != Nk is cross-attention, with the causal mask aligned to the last Nq keys.
    deterministic makes the backward's dq bitwise reproducible (slower)."""
    return _AttnFn.apply(q, k, v, causal, scale, bool(deterministic))


class _VarlenFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qkv, cu_seqlens, max_seqlen, causal, scale, deterministic):
        out, lse = fwd_varlen(qkv, cu_seqlens, max_seqlen, causal, scale)
        ctx.save_for_backward(qkv, out, lse, cu_seqlens)
        ctx.max_seqlen, ctx.causal, ctx.scale, ctx.deterministic = max_seqlen, causal, scale, deterministic
        return out

    @staticmethod
    def backward(ctx, dout):
        qkv, out, lse, cu_seqlens = ctx.saved_tensors
        dqkv = bwd_varlen(qkv, out, lse, dout.contiguous(), cu_seqlens, ctx.max_seqlen, ctx.causal, ctx.scale,
                          deterministic=ctx.deterministic)
        return dqkv, None, None, None, None, None


def flash_attn_varlen_qkvpacked_func(qkv, cu_seqlens, max_seqlen, dropout_p=0.0, softmax_scale=None,
                                     causal=False, window_size=(-1, -1), softcap=0.0, alibi_slopes=None,
                                     deterministic=False, return_attn_probs=False):
    """flash_attn's packed varlen call: qkv [total_tokens,3,H,d], cu_seqlens [batch+1] -> [total_tokens,H,d]."""
    if tuple(window_size) != (-1, -1):
        raise ValueError("window_size is not supported (must be (-1, -1))")
    if softcap != 0.0:
        raise ValueError("softcap is not supported (must be 0.0)")
    if alibi_slopes is not None:
        raise ValueError("alibi_slopes is not supported (must be None)")
    if return_attn_probs:
        raise ValueError("return_attn_probs is not supported (must be False)")
    if dropout_p != 0.0:
        raise ValueError("dropout is not supported (dropout_p must be 0.0)")
    if not isinstance(qkv, torch.Tensor) or qkv.dim() != 4 or qkv.shape[1] != 3:
        raise ValueError("Bad qkv shape")
    if cu_seqlens is None or cu_seqlens.dim() != 1:
        raise ValueError("Bad cu_seqlens")
    if cu_seqlens.numel() - 1 <= 0:
        raise ValueError("Bad batch size")
    if qkv.shape[0] != int(cu_seqlens[-1].item()):
        raise ValueError("Token count mismatch")
    return _VarlenFn.apply(qkv, cu_seqlens.to(torch.int32), int(max_seqlen), bool(causal), softmax_scale,
                           bool(deterministic))
