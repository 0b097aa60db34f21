"""Thin Python binding of libidx.so (the C ABI in include/idx.h).

Argument marshalling only: every step of the indexer runs in the CUDA
library.  The functions keep the C names; tensors are torch CUDA tensors (bf16
inputs may be given as bfloat16, int16 or uint16 tensors), and the stream
defaults to torch's current stream on the tensor's device.

If libidx.so is missing the first call raises ``RuntimeError``: there is no
fallback of any kind.
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libidx.so")

IDX_OK, IDX_EINVAL, IDX_EUNSUPPORTED, IDX_ENOWORKSPACE, IDX_ECUDA, IDX_EDEVICE = 0, -1, -2, -3, -4, -5
IDX_MAX_K = 2048

# Every symbol include/idx.h declares, with its ctypes signature.
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
SIGNATURES = {
    "idx_init": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I]),
    "idx_destroy": (_I, [_P]),
    "centroid_score": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _L, _P, _P]),
    "topk_select": (_I, [_P, _P, _P, _I, _I, _L, _I, _P, _P, _P]),
    "score_topk_fused": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _L, _I, _P, _P, _P]),
    "centroid_score_tokens": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _L, _P, _P]),
    "score_topk_fused_tokens": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _L, _I, _P, _P, _P]),
    "centroid_pool": (_I, [_P, _P, _P, _I, _I, _I, _I, _L, _P, _L, _P]),
    "centroid_score_paged": (_I, [_P, _P, _P, _I, _P, _L, _P, _I, _I, _I, _I, _I, _P, _P]),
    "score_topk_fused_paged": (_I, [_P, _P, _P, _I, _P, _L, _P, _I, _I, _I, _I, _I, _I, _P, _P,
                                    _P]),
    "idx_get_status": (_I, [_P, _P, ctypes.POINTER(_I)]),
    "idx_strerror": (ctypes.c_char_p, [_I]),
    "idx_num_sms": (_I, [_P]),
    "topk_select_noalloc": (_I, [_P, _P, _I, _I, _L, _I, _P, _P, _P]),
    "kmeans_assign": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "kmeans_scores": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "kv_block_tables": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _L, _I, _P, _I, _P, _P, _P, _P, _P,
                             _P]),
    "kv_append": (_I, [_P, _P, _P, _L, _L, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "kv_attention": (_I, [_P, _P, _L, _P, _P, _P, _P, _I, _I, _P, _L, _I, _P, _P, _I, _I, _I, _I,
                          _I, _I, _I, ctypes.c_float, _P, _P, _P]),
}

_lib = None


class IdxError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (what, strerror(code), code))


def lib():
    """The loaded CDLL with argtypes set (raises if libidx.so was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libidx.so not found at %s: build it with "
                               "`python -m page_scoring_top_b200.build`" % LIB_PATH)
        dll = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(dll, name)
            fn.restype = res
            fn.argtypes = args
        _lib = dll
    return _lib


def strerror(code):
    return lib().idx_strerror(int(code)).decode()


def _check(rc, what):
    if rc != IDX_OK:
        raise IdxError(rc, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


class Context:
    """An idx_ctx: device, limits and the workspace allocated once by idx_init."""

    def __init__(self, device=0, max_rows=1, max_n=1, max_k=1):
        if isinstance(device, torch.device):
            device = device.index if device.index is not None else torch.cuda.current_device()
        self.device = int(device)
        self.max_rows, self.max_n, self.max_k = int(max_rows), int(max_n), int(max_k)
        handle = ctypes.c_void_p()
        _check(lib().idx_init(ctypes.byref(handle), self.device, self.max_rows, self.max_n,
                              self.max_k), "idx_init")
        self.handle = handle

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _check(lib().idx_destroy(self.handle), "idx_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def num_sms(self):
        return lib().idx_num_sms(self.handle)


def idx_init(device, max_rows, max_n, max_k):
    return Context(device, max_rows, max_n, max_k)


def idx_destroy(ctx):
    ctx.close()


def _score_shapes(q, c):
    if q.dim() != 4 or c.dim() != 3:
        raise ValueError("q must be [B][T][Q][D] and c [B][N][D]")
    B, T, Q, D = q.shape
    Bc, N, Dc = c.shape
    if Bc != B or Dc != D:
        raise ValueError("q and c disagree on B or D")
    if not q.is_contiguous() or c.stride(2) != 1 or c.stride(1) != D:
        raise ValueError("q must be contiguous and c's pages contiguous rows of D")
    return B, T, Q, D, N, c.stride(0)


def centroid_score(ctx, q, c, lengths, scores, stream=None):
    """scores[b][t][p] (fp32 [B][T][N]) = sum_h q[b,t,h,:] . c[b,p,:]; -inf past lengths."""
    B, T, Q, D, N, ldc = _score_shapes(q, c)
    if tuple(scores.shape) != (B, T, N) or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous fp32 [B][T][N]")
    _check(lib().centroid_score(ctx.handle, _ptr(q), _ptr(c), _ptr(lengths), B, T, Q, D, N, ldc,
                                _ptr(scores), _stream(stream, q.device)), "centroid_score")
    return scores


def topk_select(ctx, scores, lengths, K, idx_out, val_out=None, stream=None):
    """Top-K of each row of a 2-D fp32 tensor (row stride = scores.stride(0))."""
    if scores.dim() != 2 or scores.stride(1) != 1:
        raise ValueError("scores must be 2-D with unit column stride")
    rows, N = scores.shape
    _check(lib().topk_select(ctx.handle, _ptr(scores), _ptr(lengths), rows, N, scores.stride(0), K,
                             _ptr(idx_out), _ptr(val_out), _stream(stream, scores.device)),
           "topk_select")
    return idx_out, val_out


def topk_select_noalloc(scores, lengths, K, idx_out, val_out=None, stream=None):
    """topk_select without a context: scratch in a static device array (see idx.h)."""
    if scores.dim() != 2 or scores.stride(1) != 1:
        raise ValueError("scores must be 2-D with unit column stride")
    rows, N = scores.shape
    # the C call works on the current device: make it the one holding the data
    with torch.cuda.device(scores.device):
        _check(lib().topk_select_noalloc(_ptr(scores), _ptr(lengths), rows, N, scores.stride(0),
                                         K, _ptr(idx_out), _ptr(val_out),
                                         _stream(stream, scores.device)),
               "topk_select_noalloc")
    return idx_out, val_out


def score_topk_fused(ctx, q, c, lengths, K, idx_out, val_out=None, stream=None):
    """idx_out[b*T+t] = top-K pages of request b for token t (int32 [B*T][K])."""
    B, T, Q, D, N, ldc = _score_shapes(q, c)
    _check(lib().score_topk_fused(ctx.handle, _ptr(q), _ptr(c), _ptr(lengths), B, T, Q, D, N, ldc,
                                  K, _ptr(idx_out), _ptr(val_out), _stream(stream, q.device)),
           "score_topk_fused")
    return idx_out, val_out


def _token_lengths(token_lengths, B, T):
    if (tuple(token_lengths.shape) not in ((B, T), (B * T,)) or token_lengths.dtype != torch.int32
            or not token_lengths.is_contiguous()):
        raise ValueError("token_lengths must be contiguous int32 [B][T]")
    return token_lengths


def centroid_score_tokens(ctx, q, c, token_lengths, scores, stream=None):
    """centroid_score with a valid page count per (request, token) row."""
    B, T, Q, D, N, ldc = _score_shapes(q, c)
    _token_lengths(token_lengths, B, T)
    if tuple(scores.shape) != (B, T, N) or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous fp32 [B][T][N]")
    _check(lib().centroid_score_tokens(ctx.handle, _ptr(q), _ptr(c), _ptr(token_lengths), B, T, Q,
                                       D, N, ldc, _ptr(scores), _stream(stream, q.device)),
           "centroid_score_tokens")
    return scores


def score_topk_fused_tokens(ctx, q, c, token_lengths, K, idx_out, val_out=None, stream=None):
    """score_topk_fused with a valid page count per (request, token) row."""
    B, T, Q, D, N, ldc = _score_shapes(q, c)
    _token_lengths(token_lengths, B, T)
    _check(lib().score_topk_fused_tokens(ctx.handle, _ptr(q), _ptr(c), _ptr(token_lengths), B, T,
                                         Q, D, N, ldc, K, _ptr(idx_out), _ptr(val_out),
                                         _stream(stream, q.device)),
           "score_topk_fused_tokens")
    return idx_out, val_out


def idx_get_status(ctx, stream=None):
    """(status code, raised bits) of the context; synchronises the stream."""
    bits = ctypes.c_int(0)
    rc = lib().idx_get_status(ctx.handle, _stream(stream, torch.device("cuda", ctx.device)),
                              ctypes.byref(bits))
    return rc, bits.value


def centroid_pool(ctx, keys, key_counts, P, c, stream=None):
    """c[b,p,:] = bf16 mean of the valid keys of page p (P keys per page).
    keys: bf16 bits (int16) [B][L][D]; key_counts: int32 [B]; c: int16 [B][N][D]."""
    if keys.dim() != 3 or keys.dtype != torch.int16 or not keys.is_contiguous():
        raise ValueError("keys must be contiguous bf16 bits (int16) [B][L][D]")
    B, Lk, D = keys.shape
    if c.dim() != 3 or c.dtype != torch.int16 or not c.is_contiguous() or c.shape[0] != B \
            or c.shape[2] != D:
        raise ValueError("c must be contiguous bf16 bits (int16) [B][N][D]")
    N = c.shape[1]
    if tuple(key_counts.shape) != (B,) or key_counts.dtype != torch.int32:
        raise ValueError("key_counts must be int32 [B]")
    _check(lib().centroid_pool(ctx.handle, _ptr(keys), _ptr(key_counts), B, D, P, N, Lk * D,
                               _ptr(c), N * D, _stream(stream, keys.device)), "centroid_pool")
    return c


def _kmeans_shapes(x, centroids):
    for name, t in (("x", x), ("centroids", centroids)):
        if t.dim() != 2 or t.dtype not in (torch.int16, torch.bfloat16) or not t.is_contiguous():
            raise ValueError("%s must be contiguous bf16 (or its int16 bits) [rows][D]" % name)
    M, D = x.shape
    C, Dc = centroids.shape
    if Dc != D:
        raise ValueError("x and centroids differ in D")
    return M, C, D


def kmeans_assign(ctx, x, centroids, assign_out, score_out=None, stream=None):
    """assign_out[i] = nearest centroid of point i (int32 [M]); score_out, if
    given, gets the winning x.c - |c|^2/2 (fp32 [M])."""
    M, C, D = _kmeans_shapes(x, centroids)
    _check(lib().kmeans_assign(ctx.handle, _ptr(x), _ptr(centroids), M, C, D, _ptr(assign_out),
                               _ptr(score_out), _stream(stream, x.device)), "kmeans_assign")
    return assign_out, score_out


def kmeans_scores(ctx, x, centroids, scores, stream=None):
    """scores[i, c] = x_i.c - |c|^2/2 (fp32 [M][C])."""
    M, C, D = _kmeans_shapes(x, centroids)
    if tuple(scores.shape) != (M, C) or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous fp32 [M][C]")
    _check(lib().kmeans_scores(ctx.handle, _ptr(x), _ptr(centroids), M, C, D, _ptr(scores),
                               _stream(stream, x.device)), "kmeans_scores")
    return scores


def _paged_shapes(q, pool, page_table):
    if q.dim() != 4 or q.dtype != torch.int16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 bits (int16) [B][T][Q][D]")
    if pool.dim() != 2 or pool.dtype != torch.int16 or not pool.is_contiguous():
        raise ValueError("pool must be contiguous bf16 bits (int16) [n_blocks][D]")
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_contiguous():
        raise ValueError("page_table must be contiguous int32 [B][N]")
    B, T, Q, D = q.shape
    if pool.shape[1] != D or page_table.shape[0] != B:
        raise ValueError("shape mismatch")
    return B, T, Q, D, page_table.shape[1], pool.shape[0]


def centroid_score_paged(ctx, q, pool, page_table, lengths, scores, stream=None):
    """centroid_score with page p of request b read from pool[page_table[b, p]]."""
    B, T, Q, D, N, nb = _paged_shapes(q, pool, page_table)
    if tuple(scores.shape) != (B, T, N) or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous fp32 [B][T][N]")
    _check(lib().centroid_score_paged(ctx.handle, _ptr(q), _ptr(pool), nb, _ptr(page_table), N,
                                      _ptr(lengths), B, T, Q, D, N, _ptr(scores),
                                      _stream(stream, q.device)), "centroid_score_paged")
    return scores


def score_topk_fused_paged(ctx, q, pool, page_table, lengths, K, idx_out, val_out=None,
                           stream=None):
    """score_topk_fused with page p of request b read from pool[page_table[b, p]]."""
    B, T, Q, D, N, nb = _paged_shapes(q, pool, page_table)
    _check(lib().score_topk_fused_paged(ctx.handle, _ptr(q), _ptr(pool), nb, _ptr(page_table), N,
                                        _ptr(lengths), B, T, Q, D, N, K, _ptr(idx_out),
                                        _ptr(val_out), _stream(stream, q.device)),
           "score_topk_fused_paged")
    return idx_out, val_out


# 8-bit paged KV cache (see idx.h).  The format of a cache is its tensors' dtype.
KV_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _kv_refuse(ctx, name, t, dtypes, shape, contiguous):
    """Says what is wrong with a tensor (nothing: returns)."""
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if t.device.type != "cuda" or t.device.index != ctx.device:
        raise ValueError("%s must be on cuda:%d" % (name, ctx.device))
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s" % (name, " or ".join(str(d) for d in dtypes)))
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError("%s must be of shape %s" % (name, tuple("*" if n is None else n for n in shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _kv_tensor(ctx, name, t, dtype, shape):
    """The address of t, a contiguous tensor of this dtype and shape on the context's device.
    (A call checks ten tensors: the one comparison here is what it costs, the reasons come from
    _kv_refuse.)"""
    if t.dtype != dtype or t.shape != shape or t.get_device() != ctx.device or not t.is_contiguous():
        _kv_refuse(ctx, name, t, dtype, shape, True)
    return t.data_ptr()


def _kv_rows(name, t, lead):
    """The row stride of t [..rows][heads][D] whose rows are contiguous and evenly spaced."""
    shape = t.shape
    heads, D = shape[-2:]
    if t.is_contiguous():
        return heads * D
    stride = t.stride()
    if stride[-1] != 1 or (heads > 1 and stride[-2] != D):
        raise ValueError("%s's rows must be contiguous" % name)
    ld, below = None, 1
    for d in range(lead - 1, -1, -1):  # dimensions of one row tell nothing
        if shape[d] > 1:
            if stride[d] % below or ld not in (None, stride[d] // below):
                raise ValueError("%s's rows must be evenly spaced" % name)
            ld = stride[d] // below
        below *= shape[d]
    return heads * D if ld is None else ld


def _kv_bf16(ctx, name, t, shape, lead):
    """Address and row stride of bf16 rows [..lead dims][heads][D]."""
    if t.dtype not in _BF16 or t.shape != shape or t.get_device() != ctx.device:
        _kv_refuse(ctx, name, t, _BF16, shape, False)
    return t.data_ptr(), _kv_rows(name, t, lead)


def _kv_cache(ctx, k_cache, v_cache, k_scale, v_scale):
    fmt = KV_FORMATS.get(k_cache.dtype)
    if fmt is None or k_cache.dim() != 4:
        _kv_refuse(ctx, "k_cache", k_cache, tuple(KV_FORMATS), (None,) * 4, True)
    shape = k_cache.shape
    per = shape[:2]
    return (shape, fmt, _kv_tensor(ctx, "k_cache", k_cache, k_cache.dtype, shape),
            _kv_tensor(ctx, "v_cache", v_cache, k_cache.dtype, shape),
            _kv_tensor(ctx, "k_scale", k_scale, torch.float32, per),
            _kv_tensor(ctx, "v_scale", v_scale, torch.float32, per))


def _kv_table(ctx, page_table, B):
    """Address, width and row stride of an int32 [B][N] table of contiguous rows."""
    shape = page_table.shape
    if page_table.dtype != torch.int32 or len(shape) != 2 or shape[0] != B \
            or page_table.get_device() != ctx.device:
        _kv_refuse(ctx, "page_table", page_table, torch.int32, (B, None), False)
    N = shape[1]
    ld, one = page_table.stride()
    if (N > 1 and one != 1) or (B > 1 and ld < N):
        raise ValueError("page_table's rows must be contiguous")
    return page_table.data_ptr(), N, ld if B > 1 else N


def _kv_stream(ctx, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(ctx.device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def kv_block_tables(ctx, cached, fresh, P, n_blocks, page_table, free_list, free_head,
                    free_head_out, slots, key_counts, page_counts, stream=None):
    """Pages for fresh[b] (None: T) new tokens behind cached[b] keys, taken from free_list from
    entry free_head[0] (None: 0) on and written into page_table [B][N]; slots, key_counts and
    page_counts [B][T] of the new tokens; free_head_out[0] (may be None) = the entry after the
    last one taken.  All tensors int32."""
    i32 = torch.int32
    shape = slots.shape
    if len(shape) != 2:
        _kv_refuse(ctx, "slots", slots, i32, (None, None), True)
    B, T = shape
    table, N, ld = _kv_table(ctx, page_table, B)
    n_free = free_list.numel()
    _check(lib().kv_block_tables(
        ctx.handle, _kv_tensor(ctx, "cached", cached, i32, (B,)),
        None if fresh is None else _kv_tensor(ctx, "fresh", fresh, i32, (B,)), B, T, P, N, table,
        ld, n_blocks, _kv_tensor(ctx, "free_list", free_list, i32, (n_free,)), n_free,
        None if free_head is None else _kv_tensor(ctx, "free_head", free_head, i32, (1,)),
        None if free_head_out is None else _kv_tensor(ctx, "free_head_out", free_head_out, i32, (1,)),
        _kv_tensor(ctx, "slots", slots, i32, shape),
        _kv_tensor(ctx, "key_counts", key_counts, i32, shape),
        _kv_tensor(ctx, "page_counts", page_counts, i32, shape), _kv_stream(ctx, stream)),
        "kv_block_tables")
    return slots, key_counts, page_counts


def kv_append(ctx, k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Rows k, v (bf16 [R][H][D], rows may be strided) into the cache's slots[r] (int32 [R], or any
    shape of R elements; -1: none), with the scales of the pages they reach."""
    (n_blocks, H, P, D), fmt, kc, vc, ks, vs = _kv_cache(ctx, k_cache, v_cache, k_scale, v_scale)
    R = slots.numel()
    k_at, ldk = _kv_bf16(ctx, "k", k, (R, H, D), 1)
    v_at, ldv = _kv_bf16(ctx, "v", v, (R, H, D), 1)
    _check(lib().kv_append(ctx.handle, k_at, v_at, ldk, ldv,
                           _kv_tensor(ctx, "slots", slots, torch.int32, slots.shape), R, H, D, P,
                           n_blocks, fmt, kc, vc, ks, vs, _kv_stream(ctx, stream)), "kv_append")


def kv_attention(ctx, q, k_cache, v_cache, k_scale, v_scale, page_table, key_counts, out, lse=None,
                 page_idx=None, scale=None, stream=None):
    """out (bf16 [B][T][Q][D]) = attention of q (bf16 [B][T][Q][D], rows may be strided) over the
    first key_counts[b, t] keys of the request: of the pages page_idx[b*T+t] (int32 [B*T][K], -1:
    none), or of all its pages.  lse: fp32 [B][T][Q] or None; scale: 1/sqrt(D) if None."""
    (n_blocks, H, P, D), fmt, kc, vc, ks, vs = _kv_cache(ctx, k_cache, v_cache, k_scale, v_scale)
    shape = q.shape
    if len(shape) != 4 or shape[3] != D:
        _kv_refuse(ctx, "q", q, _BF16, (None, None, None, D), False)
    B, T, Q, _ = shape
    q_at, ldq = _kv_bf16(ctx, "q", q, shape, 2)
    if out.dtype not in _BF16:
        _kv_refuse(ctx, "out", out, _BF16, shape, True)
    table, N, ld = _kv_table(ctx, page_table, B)
    if key_counts.numel() != B * T:
        raise ValueError("key_counts must have B*T elements")
    K, idx = 0, None
    if page_idx is not None:
        if page_idx.dim() != 2 or page_idx.shape[1] == 0:
            raise ValueError("page_idx must be int32 [B*T][K] with K > 0")
        K = page_idx.shape[1]
        idx = _kv_tensor(ctx, "page_idx", page_idx, torch.int32, (B * T, K))
    _check(lib().kv_attention(
        ctx.handle, q_at, ldq, kc, vc, ks, vs, n_blocks, fmt, table, ld, N,
        _kv_tensor(ctx, "key_counts", key_counts, torch.int32, key_counts.shape), idx, K, B, T, Q,
        H, D, P, D ** -0.5 if scale is None else scale, _kv_tensor(ctx, "out", out, out.dtype, shape),
        None if lse is None else _kv_tensor(ctx, "lse", lse, torch.float32, (B, T, Q)),
        _kv_stream(ctx, stream)), "kv_attention")
    return out, lse
