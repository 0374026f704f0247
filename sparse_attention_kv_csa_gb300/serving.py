"""Serving the Compressor's rows: norm into a paged cache, page tables, attention over the cache.

Argument checks and marshalling for the entry points of include/csa_serving.h; the arithmetic runs in the CUDA kernels
of libcsa.so.  Ordinary calls (contiguous tensors, the current stream) go through csa_torch, which checks, allocates and
calls in C++; everything else, and every refusal, through the checks here, as does every call where csa_torch cannot be
built or loaded.  The helpers allocate their outputs with torch and launch on ``stream`` (a torch.cuda.Stream, a raw
cudaStream_t integer, or None for torch's current stream); no call synchronises, and inputs handed to another stream than
their own have to live until it has read them.  Tensors live on the current CUDA device; ValueError / TypeError name an
argument that does not fit, CSAError a call that the library refuses.

    out, scales, stream, rstd = rms_norm_forward(x, weight, eps, residual=..., out_dtype=..., slots=...)
    grad_x, grad_weight       = rms_norm_backward(grad_out, h, weight, rstd, grad_residual=...)
    table, cu_rows, slots, counts = page_tables(before, after, ratio, page_size, free_pages, block_table, capacity)
    out, lse                  = latent_attention(q, cache, block_table, cu_q, seq_lens, ratio, scale, ...)
"""
from __future__ import annotations

import ctypes
import importlib.util
import warnings

from . import _build

__all__ = ["csa_rms_norm_fwd", "csa_rms_norm_bwd", "csa_page_tables", "csa_latent_attention", "rms_norm_forward",
           "rms_norm_backward", "page_tables", "latent_attention"]

_lib = None
_raise = None
_torch = None
_Tensor = None
_raw_stream = None
_short = None  # csa_torch: the ordinary case of each helper in one call (None where it is not to be had)
_e4m3 = None

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


def _load_torch():
    """torch is imported on first use, like in the rest of the package."""
    global _torch, _Tensor, _raw_stream, _short, _e4m3
    import torch
    try:
        spec = importlib.util.spec_from_file_location("csa_torch", _build.build_binding())
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(_lib, f), ctypes.c_void_p).value for f in
                      ("csa_rms_norm_fwd", "csa_rms_norm_bwd", "csa_page_tables", "csa_latent_attention")))
        _short = module
    except Exception as e:  # no compiler or headers, or a library that this torch does not load
        warnings.warn("csa_torch is not to be had (%s): calls are checked and made in Python, some 8 us longer each"
                      % (str(e) or type(e).__name__).splitlines()[0], RuntimeWarning, stacklevel=3)
    _e4m3 = torch.float8_e4m3fn
    _torch, _Tensor = torch, torch.Tensor
    # the current stream's handle without building a Stream object (some 3 us of a call of 10)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _CODES.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32, torch.float8_e4m3fn: E4M3})


def _addr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def _stream(s):
    if s is None:
        if _torch is None:
            _load_torch()
        if _raw_stream is not None:
            return _raw_stream(_torch.cuda.current_device())
        return _torch.cuda.current_stream().cuda_stream
    return s if isinstance(s, int) else s.cuda_stream


def _empty(shape, dtype, device, stream):
    """An output, allocated on the stream that writes it."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(_torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _fit(bits, **numbers):
    """The numbers fit the entry points' integers (ctypes would cut them off silently)."""
    for name, v in numbers.items():
        if not -1 << (bits - 1) <= v < 1 << (bits - 1):
            raise ValueError("%s must fit %d bits (got %s)" % (name, bits, v))


# ------------------------------------------------------------ the C entry points

def csa_rms_norm_fwd(x, x_stride, residual, residual_stride, weight, n_rows, dim, eps, dtype, slots, n_slots, out,
                     out_stride, out_dtype, scales, scale_group, residual_out, rstd, stream=None) -> None:
    _fit(32, dim=dim, dtype=dtype, out_dtype=out_dtype, scale_group=scale_group)
    _fit(64, x_stride=x_stride, residual_stride=residual_stride, n_rows=n_rows, n_slots=n_slots, out_stride=out_stride)
    _raise(_lib.csa_rms_norm_fwd(_addr(x), x_stride, _addr(residual), residual_stride, _addr(weight), n_rows, dim, eps,
                                 dtype, _addr(slots), n_slots, _addr(out), out_stride, out_dtype, _addr(scales),
                                 scale_group, _addr(residual_out), _addr(rstd), _stream(stream)))


def csa_rms_norm_bwd(h, h_stride, grad_out, grad_out_stride, grad_residual, grad_residual_stride, weight, rstd, n_rows,
                     dim, dtype, grad_x, grad_weight, stream=None) -> None:
    _fit(32, dim=dim, dtype=dtype)
    _fit(64, h_stride=h_stride, grad_out_stride=grad_out_stride, grad_residual_stride=grad_residual_stride, n_rows=n_rows)
    _raise(_lib.csa_rms_norm_bwd(_addr(h), h_stride, _addr(grad_out), grad_out_stride, _addr(grad_residual),
                                 grad_residual_stride, _addr(weight), _addr(rstd), n_rows, dim, dtype, _addr(grad_x),
                                 _addr(grad_weight), _stream(stream)))


def csa_page_tables(before, after, n_req, ratio, page_size, free_pages, n_free, taken, table, table_stride, width,
                    capacity, table_out, cu_rows, slots, counts, stream=None) -> None:
    _fit(32, n_req=n_req, ratio=ratio, page_size=page_size, n_free=n_free, width=width)
    _fit(64, table_stride=table_stride, capacity=capacity)
    _raise(_lib.csa_page_tables(_addr(before), _addr(after), n_req, ratio, page_size, _addr(free_pages), n_free,
                                _addr(taken), _addr(table), table_stride, width, capacity, _addr(table_out),
                                _addr(cu_rows), _addr(slots), _addr(counts), _stream(stream)))


def csa_latent_attention(q, q_token_stride, q_head_stride, cu_q, n_req, n_tokens, n_heads, head_dim, v_dim, cache,
                         cache_stride, cache_dtype, row_scales, n_pages, page_size, block_table, table_stride, width,
                         seq_lens, ratio, scale, sink, out, lse, stream=None) -> None:
    _fit(32, n_req=n_req, n_heads=n_heads, head_dim=head_dim, v_dim=v_dim, cache_dtype=cache_dtype, page_size=page_size,
         width=width, ratio=ratio)
    _fit(64, q_token_stride=q_token_stride, q_head_stride=q_head_stride, n_tokens=n_tokens, cache_stride=cache_stride,
         n_pages=n_pages, table_stride=table_stride)
    _raise(_lib.csa_latent_attention(_addr(q), q_token_stride, q_head_stride, _addr(cu_q), n_req, n_tokens, n_heads,
                                     head_dim, v_dim, _addr(cache), cache_stride, cache_dtype, _addr(row_scales),
                                     n_pages, page_size, _addr(block_table), table_stride, width, _addr(seq_lens),
                                     ratio, scale, _addr(sink), _addr(out), _addr(lse), _stream(stream)))


# ------------------------------------------------------------ checks

def _check(name, t, dtype, shape, device):
    """t is a contiguous tensor of dtype and shape (None: any extent) on the device (its number, None: any)."""
    if (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and (device is None or t.get_device() == device)):
        return
    _fits(name, t, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _fits(name, t, dtype, shape, device):
    if not isinstance(t, _torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple("*" if w is None else w for w in shape), tuple(t.shape)))
    if device is not None and t.get_device() != device:
        raise ValueError("%s must be on cuda:%d (got %s)" % (name, device, t.device))


def _check_device(t, name):
    """The number of t's device, which is the current one."""
    d = t.get_device()
    if d < 0 or d != _torch.cuda.current_device():
        raise ValueError("%s must be on the current CUDA device (got %s)" % (name, t.device))
    return d


def _rows(name, t, dtype, shape, device):
    """A matrix whose rows are contiguous: checked; returns its row stride."""
    if type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return shape[1]
    _fits(name, t, dtype, shape, device)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s's last dimension must be contiguous" % name)
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _vector(name, t, dtype, device):
    """t's length: a contiguous vector of dtype on the device."""
    if type(t) is _Tensor and t.dtype is dtype and t.dim() == 1 and t.is_contiguous() and t.get_device() == device:
        return t.shape[0]
    _check(name, t, dtype, (None,), device)
    return t.shape[0]


def _table(name, t, rows, device):
    """The row stride and width of an int32 matrix of so many rows."""
    if type(t) is _Tensor and t.dtype is _torch.int32 and t.dim() == 2 and t.is_contiguous() and t.get_device() == device:
        n, width = t.shape
        if n == rows:
            return width, width
    _fits(name, t, _torch.int32, (rows, None), device)
    return _rows(name, t, _torch.int32, tuple(t.shape), device), t.shape[1]


def _handle(stream, device):
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream(stream)


def _pointer(t):
    return None if t is None else t.data_ptr()


def _matrix(name, t):
    """t's shape, code and device: a matrix in bf16, f16 or f32 on the current device."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    code = _CODES.get(t.dtype, E4M3)
    if code == E4M3 or t.dim() != 2:
        raise ValueError("%s must be [n_rows, dim] in bf16, f16 or f32 (got %s, %s)" % (name, tuple(t.shape), t.dtype))
    return t.shape, code, _check_device(t, name)


# ------------------------------------------------------------ helpers

def rms_norm_forward(x, weight=None, eps=1e-6, residual=None, out_dtype=None, scale_group=0, slots=None, out=None,
                     scales=None, stream=None):
    """Root-mean-square norm of x [n_rows, dim] (bf16, f16 or f32; + residual), see csa_rms_norm_fwd.

    out_dtype: x's (default) or torch.float8_e4m3fn with a scale a row (scale_group 0) or every 128 columns.  slots
    (int64 [n_rows], needs ``out`` and for 8 bits ``scales``): row i goes to out[slots[i]], nowhere when negative.
    Returns (out, scales or None, x + residual or None, rstd fp32 [n_rows]).
    """
    if _torch is None:
        _load_torch()
    if _short is not None and stream is None and (out_dtype is None or out_dtype is _e4m3):
        bits8 = out_dtype is _e4m3 or (out is not None and getattr(out, "dtype", None) is _e4m3)
        r = _short.rms_norm_forward(x, weight, eps, residual, bits8, scale_group, slots, out, scales)
        if r is not None:
            return r if type(r) is tuple else _raise(r)
    shape, code, d = _matrix("x", x)
    n, dim = shape
    _fit(32, dim=dim)
    dtype, device, f32 = x.dtype, x.device, _torch.float32
    xs = dim if x.is_contiguous() else _rows("x", x, dtype, shape, d)
    rs = 0 if residual is None else _rows("residual", residual, dtype, shape, d)
    if weight is not None:
        _check("weight", weight, f32, (dim,), d)
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    bits8 = out_dtype == _torch.float8_e4m3fn
    if out_dtype != dtype and not bits8:
        raise ValueError("out_dtype must be %s or torch.float8_e4m3fn (got %s)" % (dtype, out_dtype))
    if scale_group and (scale_group != 128 or dim % 128 or not bits8):
        raise ValueError("scale_group must be 0, or 128 for an 8-bit output of a width that it divides (got %s)" % (scale_group,))
    groups = dim // scale_group if scale_group else 1
    if slots is not None:
        _check("slots", slots, _torch.int64, (n,), d)
        if out is None or (bits8 and scales is None):
            raise ValueError("slots need out (and scales for an 8-bit output)")
    if out is None:
        out, out_stride = _empty(shape, out_dtype, device, stream), dim
    else:
        out_stride = _rows("out", out, out_dtype, (n if slots is None else None, dim), d)
    if bits8:
        if scales is None:
            scales = _empty((n, groups), f32, device, stream)
        elif groups == 1 and isinstance(scales, _torch.Tensor) and scales.dim() == 1:
            _check("scales", scales, f32, (out.shape[0],), d)
        else:
            _check("scales", scales, f32, (out.shape[0], groups), d)
    elif scales is not None:
        raise ValueError("scales go with an 8-bit output")
    total = None if residual is None else _empty(shape, dtype, device, stream)
    rstd = _empty((n,), f32, device, stream)
    rc = _lib.csa_rms_norm_fwd(x.data_ptr(), xs, _pointer(residual), rs, _pointer(weight), n, dim, eps, code, _pointer(slots),
                               out.shape[0], out.data_ptr(), out_stride, E4M3 if bits8 else code, _pointer(scales),
                               scale_group, _pointer(total), rstd.data_ptr(), _handle(stream, d))
    if rc:
        _raise(rc)
    return out, scales, total, rstd


def rms_norm_backward(grad_out, h, weight, rstd, grad_residual=None, stream=None):
    """Gradient of rms_norm_forward: (grad_x [n_rows, dim] -- the residual's too -- and grad_weight fp32 [dim]).

    h is the forward's x + residual (x without a residual), rstd its fourth result; grad_residual the gradient that
    reaches x + residual directly.
    """
    if _torch is None:
        _load_torch()
    if _short is not None and stream is None:
        r = _short.rms_norm_backward(grad_out, h, weight, rstd, grad_residual)
        if r is not None:
            return r if type(r) is tuple else _raise(r)
    shape, code, d = _matrix("h", h)
    n, dim = shape
    _fit(32, dim=dim)
    dtype, device, f32 = h.dtype, h.device, _torch.float32
    hs = dim if h.is_contiguous() else _rows("h", h, dtype, shape, d)
    gs = _rows("grad_out", grad_out, dtype, shape, d)
    rs = 0 if grad_residual is None else _rows("grad_residual", grad_residual, dtype, shape, d)
    if weight is not None:
        _check("weight", weight, f32, (dim,), d)
    _check("rstd", rstd, f32, (n,), d)
    grad_x = _empty(shape, dtype, device, stream)
    grad_weight = _empty((dim,), f32, device, stream)
    rc = _lib.csa_rms_norm_bwd(h.data_ptr(), hs, grad_out.data_ptr(), gs, _pointer(grad_residual), rs, _pointer(weight),
                               rstd.data_ptr(), n, dim, code, grad_x.data_ptr(), grad_weight.data_ptr(), _handle(stream, d))
    if rc:
        _raise(rc)
    return grad_x, grad_weight


def page_tables(before, after, ratio, page_size, free_pages, block_table, capacity, taken=None, out=None, stream=None):
    """Pages and slots for the rows that requests gain from before to after tokens, see csa_page_tables.

    before, after int32 [n_req]; free_pages int32 [n_free]; taken int32 [1] or None: entries of free_pages already
    used; block_table int32 [n_req, width]; capacity: how many slots to return.  ``out``: where the new table goes
    (block_table itself for an update in place), a new tensor by default.
    Returns (table, cu_rows int32 [n_req + 1], slots int64 [capacity], counts int32 [4]: new rows, pages taken, pages
    short, pages of the widest request).  Where the last exceeds block_table's width, add nothing to ``taken``: widen the
    table and call again, or the pages past its columns are lost.
    """
    if _torch is None:
        _load_torch()
    if _short is not None and stream is None:
        r = _short.page_tables(before, after, ratio, page_size, free_pages, block_table, capacity, taken, out)
        if r is not None:
            return r if type(r) is tuple else _raise(r)
    _fit(32, ratio=ratio, page_size=page_size)
    i32 = _torch.int32
    if not isinstance(before, _torch.Tensor):
        raise TypeError("before must be a tensor")
    d, device = _check_device(before, "before"), before.device
    n = _vector("before", before, i32, d)
    _check("after", after, i32, (n,), d)
    n_free = _vector("free_pages", free_pages, i32, d)
    if taken is not None:
        _check("taken", taken, i32, (1,), d)
    stride, width = _table("block_table", block_table, n, d)
    _fit(32, n_req=n, n_free=n_free, width=width)
    if capacity < 0:
        raise ValueError("capacity must be >= 0 (got %s)" % (capacity,))
    if out is None:
        out = _empty((n, width), i32, device, stream)
    else:
        _check("out", out, i32, (n, width), d)
    cu_rows = _empty((n + 1,), i32, device, stream)
    slots = _empty((capacity,), _torch.int64, device, stream)
    counts = _empty((4,), i32, device, stream)
    rc = _lib.csa_page_tables(before.data_ptr(), after.data_ptr(), n, ratio, page_size, free_pages.data_ptr(), n_free,
                              _pointer(taken), block_table.data_ptr(), stride, width, capacity, out.data_ptr(),
                              cu_rows.data_ptr(), slots.data_ptr(), counts.data_ptr(), _handle(stream, d))
    if rc:
        _raise(rc)
    return out, cu_rows, slots, counts


def latent_attention(q, cache, block_table, cu_q, seq_lens, ratio, scale, v_dim=None, row_scales=None, sink=None,
                     out=None, stream=None):
    """Attention of q [n_tokens, n_heads, head_dim] (bf16) over a paged cache of rows that are keys and values in one.

    cache [n_pages, page_size, head_dim], bf16, or float8_e4m3fn with row_scales fp32 [n_pages, page_size]; block_table
    int32 [n_req, width]; cu_q int32 [n_req + 1]; seq_lens int32 [n_req], tokens of each request with the new ones;
    ratio: tokens a row; v_dim: leading columns that are the values (all by default); sink fp32 [n_heads] or None.
    Multiples of 64 up to 576 columns with a v_dim of up to 512 run on the tensor cores, other widths (576 columns with
    the default v_dim among them) on the fp32 units, more than a hundred times slower.  Tokens outside of cu_q are left unwritten.
    Returns (out bf16 [n_tokens, n_heads, v_dim], lse fp32 [n_tokens, n_heads]); see csa_latent_attention.
    """
    if _torch is None:
        _load_torch()
    if _short is not None and stream is None:
        r = _short.latent_attention(q, cache, block_table, cu_q, seq_lens, ratio, scale, v_dim, row_scales, sink, out)
        if r is not None:
            return r if type(r) is tuple else _raise(r)
    _fit(32, ratio=ratio, v_dim=0 if v_dim is None else v_dim)
    bf16, f32, i32 = _torch.bfloat16, _torch.float32, _torch.int32
    if type(q) is not _Tensor or q.dtype is not bf16 or q.dim() != 3:
        _fits("q", q, bf16, (None, None, None), None)
    d, device = _check_device(q, "q"), q.device
    n, heads, dim = q.shape
    q_token, q_head, q_column = q.stride()
    if q_column != 1 and dim > 1:
        raise ValueError("q's last dimension must be contiguous")
    if not isinstance(cache, _torch.Tensor):
        raise TypeError("cache must be a tensor")
    bits8 = cache.dtype == _torch.float8_e4m3fn
    if not bits8 and cache.dtype != bf16:
        raise ValueError("cache must be bf16 or float8_e4m3fn (got %s)" % cache.dtype)
    if cache.dim() != 3 or cache.shape[2] != dim or cache.get_device() != d:
        _fits("cache", cache, cache.dtype, (None, None, dim), d)
    pages, page_size, _ = cache.shape
    if page_size < 1:
        raise ValueError("cache must have at least one row a page")
    if cache.is_contiguous():
        row = dim
    else:
        row = cache.stride(1) if page_size > 1 else cache.stride(0) if pages > 1 else dim
        if cache.stride(2) != 1 or (pages > 1 and cache.stride(0) != row * page_size):
            raise ValueError("cache's rows must be contiguous and evenly spaced")
    if bits8 != (row_scales is not None):
        raise ValueError("row_scales go with a float8_e4m3fn cache, and it with them")
    if bits8:
        _check("row_scales", row_scales, f32, (pages, page_size), d)
    n_req = _vector("cu_q", cu_q, i32, d) - 1
    if n_req < 0:
        raise ValueError("cu_q must be [n_req + 1]")
    _check("seq_lens", seq_lens, i32, (n_req,), d)
    stride, width = _table("block_table", block_table, n_req, d)
    _fit(32, n_req=n_req, n_heads=heads, head_dim=dim, page_size=page_size, width=width)
    if sink is not None:
        _check("sink", sink, f32, (heads,), d)
    v_dim = dim if v_dim is None else v_dim
    if out is None:
        out = _empty((n, heads, v_dim), bf16, device, stream)
    else:
        _check("out", out, bf16, (n, heads, v_dim), d)
    lse = _empty((n, heads), f32, device, stream)
    rc = _lib.csa_latent_attention(q.data_ptr(), q_token if n > 1 else max(q_token, dim), q_head if heads > 1 else max(q_head, dim),
                                   cu_q.data_ptr(), n_req, n, heads, dim, v_dim, cache.data_ptr(), row,
                                   E4M3 if bits8 else BF16, _pointer(row_scales), pages, page_size, block_table.data_ptr(),
                                   stride, width, seq_lens.data_ptr(), ratio, scale, _pointer(sink), out.data_ptr(),
                                   lse.data_ptr(), _handle(stream, d))
    if rc:
        _raise(rc)
    return out, lse
