"""Serving the Compressor's rows: norm into a paged cache, page tables, attention over the cache.

Argument checks and marshalling for the entry points of include/csa_serving.h; the arithmetic runs in the CUDA kernels
of libcsa.so.  The helpers allocate their outputs with torch and launch on ``stream`` (a torch.cuda.Stream, a raw
cudaStream_t integer, or None for torch's current stream); no call synchronises.  Tensors live on the current CUDA
device; ValueError / TypeError name an argument that does not fit, CSAError a call that the library refuses.

    out, scales, stream, rstd = rms_norm_forward(x, weight, eps, residual=..., out_dtype=..., slots=...)
    grad_x, grad_weight       = rms_norm_backward(grad_out, h, weight, rstd, grad_residual=...)
    table, cu_rows, slots, counts = page_tables(before, after, ratio, page_size, free_pages, block_table, capacity)
    out, lse                  = latent_attention(q, cache, block_table, cu_q, seq_lens, ratio, scale, ...)
"""
from __future__ import annotations

import contextlib
import ctypes

__all__ = ["csa_rms_norm_fwd", "csa_rms_norm_bwd", "csa_page_tables", "csa_latent_attention", "rms_norm_forward",
           "rms_norm_backward", "page_tables", "latent_attention"]

_lib = None
_raise = None

BF16, F16, F32, E4M3 = 0, 1, 2, 3
_CODES = {}


def _bind(lib, check):
    """Declares the entry points of the loaded library (called once by the package)."""
    global _lib, _raise
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.csa_rms_norm_fwd.argtypes = [P, i64, P, i64, P, i64, i32, f32, i32, P, i64, P, i64, i32, P, i32, P, P, P]
    lib.csa_rms_norm_bwd.argtypes = [P, i64, P, i64, P, i64, P, P, i64, i32, i32, P, P, P]
    lib.csa_page_tables.argtypes = [P, P, i32, i32, i32, P, i32, P, P, i64, i32, i64, P, P, P, P, P]
    lib.csa_latent_attention.argtypes = [P, i64, i64, P, i32, i64, i32, i32, i32, P, i64, i32, P, i64, i32, P, i64, i32,
                                         P, i32, f32, P, P, P, P]
    for f in ("csa_rms_norm_fwd", "csa_rms_norm_bwd", "csa_page_tables", "csa_latent_attention"):
        getattr(lib, f).restype = ctypes.c_int
    _lib, _raise = lib, check


def _addr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return s if isinstance(s, int) else s.cuda_stream


def _on(stream):
    """Outputs are allocated on the stream that writes them."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


# ------------------------------------------------------------ the C entry points

def csa_rms_norm_fwd(x, x_stride, residual, residual_stride, weight, n_rows, dim, eps, dtype, slots, n_slots, out,
                     out_stride, out_dtype, scales, scale_group, residual_out, rstd, stream=None) -> None:
    _raise(_lib.csa_rms_norm_fwd(_addr(x), x_stride, _addr(residual), residual_stride, _addr(weight), n_rows, dim, eps,
                                 dtype, _addr(slots), n_slots, _addr(out), out_stride, out_dtype, _addr(scales),
                                 scale_group, _addr(residual_out), _addr(rstd), _stream(stream)))


def csa_rms_norm_bwd(h, h_stride, grad_out, grad_out_stride, grad_residual, grad_residual_stride, weight, rstd, n_rows,
                     dim, dtype, grad_x, grad_weight, stream=None) -> None:
    _raise(_lib.csa_rms_norm_bwd(_addr(h), h_stride, _addr(grad_out), grad_out_stride, _addr(grad_residual),
                                 grad_residual_stride, _addr(weight), _addr(rstd), n_rows, dim, dtype, _addr(grad_x),
                                 _addr(grad_weight), _stream(stream)))


def csa_page_tables(before, after, n_req, ratio, page_size, free_pages, n_free, taken, table, table_stride, width,
                    capacity, table_out, cu_rows, slots, counts, stream=None) -> None:
    _raise(_lib.csa_page_tables(_addr(before), _addr(after), n_req, ratio, page_size, _addr(free_pages), n_free,
                                _addr(taken), _addr(table), table_stride, width, capacity, _addr(table_out),
                                _addr(cu_rows), _addr(slots), _addr(counts), _stream(stream)))


def csa_latent_attention(q, q_token_stride, q_head_stride, cu_q, n_req, n_tokens, n_heads, head_dim, v_dim, cache,
                         cache_stride, cache_dtype, row_scales, n_pages, page_size, block_table, table_stride, width,
                         seq_lens, ratio, scale, sink, out, lse, stream=None) -> None:
    _raise(_lib.csa_latent_attention(_addr(q), q_token_stride, q_head_stride, _addr(cu_q), n_req, n_tokens, n_heads,
                                     head_dim, v_dim, _addr(cache), cache_stride, cache_dtype, _addr(row_scales),
                                     n_pages, page_size, _addr(block_table), table_stride, width, _addr(seq_lens),
                                     ratio, scale, _addr(sink), _addr(out), _addr(lse), _stream(stream)))


# ------------------------------------------------------------ checks

def _codes():
    if not _CODES:
        import torch
        _CODES.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32, torch.float8_e4m3fn: E4M3})
    return _CODES


def _check(name, t, dtype, shape=None, like=None, contiguous=True):
    """t is a tensor of dtype and shape (None: any extent) on like's device."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if shape is not None and (t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape))):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple("*" if w is None else w for w in shape), tuple(t.shape)))
    if like is not None and t.device != like.device:
        raise ValueError("%s must be on %s (got %s)" % (name, like.device, t.device))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _check_device(t, name):
    import torch
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError("%s must be on the current CUDA device (got %s)" % (name, t.device))


def _rows(name, t, dtype, shape, like):
    """A matrix whose rows are contiguous: checked; returns its row stride."""
    _check(name, t, dtype, shape, like, contiguous=False)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s's last dimension must be contiguous" % name)
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


# ------------------------------------------------------------ helpers

def rms_norm_forward(x, weight=None, eps=1e-6, residual=None, out_dtype=None, scale_group=0, slots=None, out=None,
                     scales=None, stream=None):
    """Root-mean-square norm of x [n_rows, dim] (bf16, f16 or f32; + residual), see csa_rms_norm_fwd.

    out_dtype: x's (default) or torch.float8_e4m3fn with a scale a row (scale_group 0) or every 128 columns.  slots
    (int64 [n_rows], needs ``out`` and for 8 bits ``scales``): row i goes to out[slots[i]], nowhere when negative.
    Returns (out, scales or None, x + residual or None, rstd fp32 [n_rows]).
    """
    import torch
    codes = _codes()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    if x.dim() != 2 or x.dtype not in codes or x.dtype == torch.float8_e4m3fn:
        raise ValueError("x must be [n_rows, dim] in bf16, f16 or f32 (got %s, %s)" % (tuple(x.shape), x.dtype))
    _check_device(x, "x")
    n, dim = x.shape
    xs = _rows("x", x, x.dtype, (n, dim), x)
    rs = 0 if residual is None else _rows("residual", residual, x.dtype, (n, dim), x)
    if weight is not None:
        _check("weight", weight, torch.float32, (dim,), x)
    if out is not None:
        out_dtype = out.dtype if out_dtype is None else out_dtype
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype != x.dtype and out_dtype != torch.float8_e4m3fn:
        raise ValueError("out_dtype must be %s or torch.float8_e4m3fn (got %s)" % (x.dtype, out_dtype))
    bits8 = out_dtype == torch.float8_e4m3fn
    if scale_group not in (0, 128) or (scale_group and (dim % 128 or not bits8)):
        raise ValueError("scale_group must be 0, or 128 for an 8-bit output of a width that it divides (got %s)" % (scale_group,))
    groups = dim // scale_group if scale_group else 1
    if slots is not None:
        _check("slots", slots, torch.int64, (n,), x)
        if out is None or (bits8 and scales is None):
            raise ValueError("slots need out (and scales for an 8-bit output)")
    with _on(stream):
        if out is None:
            out = torch.empty((n, dim), dtype=out_dtype, device=x.device)
        os_ = _rows("out", out, out_dtype, (n if slots is None else None, dim), x)
        if bits8:
            if scales is None:
                scales = torch.empty((n, groups), dtype=torch.float32, device=x.device)
            if scales.dim() == 1 and groups == 1:
                _check("scales", scales, torch.float32, (out.shape[0],), x)
            else:
                _check("scales", scales, torch.float32, (out.shape[0], groups), x)
        elif scales is not None:
            raise ValueError("scales go with an 8-bit output")
        total = None if residual is None else torch.empty((n, dim), dtype=x.dtype, device=x.device)
        rstd = torch.empty((n,), dtype=torch.float32, device=x.device)
    csa_rms_norm_fwd(x, xs, residual, rs, weight, n, dim, eps, codes[x.dtype], slots, out.shape[0], out, os_,
                     codes[out_dtype], scales, scale_group, total, rstd, stream)
    return out, scales, total, rstd


def rms_norm_backward(grad_out, h, weight, rstd, grad_residual=None, stream=None):
    """Gradient of rms_norm_forward: (grad_x [n_rows, dim] -- the residual's too -- and grad_weight fp32 [dim]).

    h is the forward's x + residual (x without a residual), rstd its fourth result; grad_residual the gradient that
    reaches x + residual directly.
    """
    import torch
    codes = _codes()
    if not isinstance(h, torch.Tensor):
        raise TypeError("h must be a tensor")
    if h.dim() != 2 or h.dtype not in codes or h.dtype == torch.float8_e4m3fn:
        raise ValueError("h must be [n_rows, dim] in bf16, f16 or f32 (got %s, %s)" % (tuple(h.shape), h.dtype))
    _check_device(h, "h")
    n, dim = h.shape
    hs = _rows("h", h, h.dtype, (n, dim), h)
    gs = _rows("grad_out", grad_out, h.dtype, (n, dim), h)
    rs = 0 if grad_residual is None else _rows("grad_residual", grad_residual, h.dtype, (n, dim), h)
    if weight is not None:
        _check("weight", weight, torch.float32, (dim,), h)
    _check("rstd", rstd, torch.float32, (n,), h)
    with _on(stream):
        grad_x = torch.empty((n, dim), dtype=h.dtype, device=h.device)
        grad_weight = torch.empty((dim,), dtype=torch.float32, device=h.device)
    csa_rms_norm_bwd(h, hs, grad_out, gs, grad_residual, rs, weight, rstd, n, dim, codes[h.dtype], grad_x, grad_weight, stream)
    return grad_x, grad_weight


def page_tables(before, after, ratio, page_size, free_pages, block_table, capacity, taken=None, out=None, stream=None):
    """Pages and slots for the rows that requests gain from before to after tokens, see csa_page_tables.

    before, after int32 [n_req]; free_pages int32 [n_free]; taken int32 [1] or None: entries of free_pages already
    used; block_table int32 [n_req, width]; capacity: how many slots to return.  ``out``: where the new table goes
    (block_table itself for an update in place), a new tensor by default.
    Returns (table, cu_rows int32 [n_req + 1], slots int64 [capacity], counts int32 [4]: new rows, pages taken, pages
    short, pages of the widest request).
    """
    import torch
    i32 = torch.int32
    _check("before", before, i32, (None,))
    n = before.shape[0]
    _check_device(before, "before")
    _check("after", after, i32, (n,), before)
    _check("free_pages", free_pages, i32, (None,), before)
    if taken is not None:
        _check("taken", taken, i32, (1,), before)
    stride = _rows("block_table", block_table, i32, (n, None), before)
    width = block_table.shape[1]
    if capacity < 0:
        raise ValueError("capacity must be >= 0 (got %s)" % (capacity,))
    with _on(stream):
        if out is None:
            out = torch.empty((n, width), dtype=i32, device=before.device)
        else:
            _check("out", out, i32, (n, width), before)
        cu_rows = torch.empty((n + 1,), dtype=i32, device=before.device)
        slots = torch.empty((capacity,), dtype=torch.int64, device=before.device)
        counts = torch.empty((4,), dtype=i32, device=before.device)
    csa_page_tables(before, after, n, ratio, page_size, free_pages, free_pages.shape[0], taken, block_table, stride, width,
                    capacity, out, cu_rows, slots, counts, stream)
    return out, cu_rows, slots, counts


def latent_attention(q, cache, block_table, cu_q, seq_lens, ratio, scale, v_dim=None, row_scales=None, sink=None,
                     out=None, stream=None):
    """Attention of q [n_tokens, n_heads, head_dim] (bf16) over a paged cache of rows that are keys and values in one.

    cache [n_pages, page_size, head_dim], bf16, or float8_e4m3fn with row_scales fp32 [n_pages, page_size]; block_table
    int32 [n_req, width]; cu_q int32 [n_req + 1]; seq_lens int32 [n_req], tokens of each request with the new ones;
    ratio: tokens a row; v_dim: leading columns that are the values (all by default); sink fp32 [n_heads] or None.
    Returns (out bf16 [n_tokens, n_heads, v_dim], lse fp32 [n_tokens, n_heads]); see csa_latent_attention.
    """
    import torch
    _check("q", q, torch.bfloat16, (None, None, None), contiguous=False)
    _check_device(q, "q")
    n, heads, dim = q.shape
    if q.stride(2) != 1 and dim > 1:
        raise ValueError("q's last dimension must be contiguous")
    if not isinstance(cache, torch.Tensor):
        raise TypeError("cache must be a tensor")
    bits8 = cache.dtype == torch.float8_e4m3fn
    if not bits8 and cache.dtype != torch.bfloat16:
        raise ValueError("cache must be bf16 or float8_e4m3fn (got %s)" % cache.dtype)
    _check("cache", cache, cache.dtype, (None, None, dim), q, contiguous=False)
    pages, page_size = cache.shape[0], cache.shape[1]
    if page_size < 1:
        raise ValueError("cache must have at least one row a page")
    row = cache.stride(1) if page_size > 1 else cache.stride(0) if pages > 1 else dim
    if cache.numel() and (cache.stride(2) != 1 or (pages > 1 and cache.stride(0) != row * page_size)):
        raise ValueError("cache's rows must be contiguous and evenly spaced")
    if bits8 != (row_scales is not None):
        raise ValueError("row_scales go with a float8_e4m3fn cache, and it with them")
    if bits8:
        _check("row_scales", row_scales, torch.float32, (pages, page_size), q)
    _check("cu_q", cu_q, torch.int32, (None,), q)
    n_req = cu_q.shape[0] - 1
    if n_req < 0:
        raise ValueError("cu_q must be [n_req + 1]")
    _check("seq_lens", seq_lens, torch.int32, (n_req,), q)
    stride = _rows("block_table", block_table, torch.int32, (n_req, None), q)
    if sink is not None:
        _check("sink", sink, torch.float32, (heads,), q)
    v_dim = dim if v_dim is None else v_dim
    with _on(stream):
        if out is None:
            out = torch.empty((n, heads, v_dim), dtype=torch.bfloat16, device=q.device)
        else:
            _check("out", out, torch.bfloat16, (n, heads, v_dim), q)
        lse = torch.empty((n, heads), dtype=torch.float32, device=q.device)
    csa_latent_attention(q, q.stride(0) if n > 1 else max(q.stride(0), dim), q.stride(1) if heads > 1 else max(q.stride(1), dim),
                         cu_q, n_req, n, heads, dim, v_dim, cache, row, E4M3 if bits8 else BF16, row_scales, pages,
                         page_size, block_table, stride, block_table.shape[1], seq_lens, ratio, scale, sink, out, lse,
                         stream)
    return out, lse
