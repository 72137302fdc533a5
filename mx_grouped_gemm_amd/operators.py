"""Binding of the operators around the grouped GEMM (``include/bsgemm.h``, second part): norm,
sort, rows there and back, SwiGLU and quantisation, and the MX product for few rows.

Argument marshalling only, as in the package's other functions. Every tensor is compared with the
sizes of the call, since the C ABI sees bare pointers: ValueError where its shape, type, device or
layout is not what the call needs (``check_*`` make the same checks without a call, on any device).
Sizes the library itself rejects come back as :class:`BsgemmError`. Outputs that are not given are
allocated on the stream the call runs on.

Results have no autograd history, also where an input requires a gradient: the gradients are calls of
their own (``*_backward``; that of ``bsgemm_permute_rows`` is ``bsgemm_combine_rows`` without weights), which
a ``torch.autograd.Function`` or a hand-written backward pass makes.
"""

import ctypes
import functools

import torch

ACT = {"none": 0, "swiglu": 1}
ROW_DTYPE = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}
QUANTS = (("e4m3", "blockwise"), ("e4m3", "mx"), ("e2m1", "mx"), ("e2m1", "nv"))
_QUANT_WORDS = dict(zip(QUANTS, (1 | (1 << 8), 1 | (2 << 8), 2 | (2 << 8), 2 | (3 << 8))))

EXPORTED = ("bsgemm_quantize", "bsgemm_swiglu_backward", "bsgemm_rms_norm_quantize", "bsgemm_rms_norm_backward",
            "bsgemm_rms_norm_backward_workspace_size", "bsgemm_route_sort", "bsgemm_route_sort_workspace_size",
            "bsgemm_permute_rows", "bsgemm_combine_rows", "bsgemm_combine_backward", "bsgemm_grouped_few_rows")


def declare(lib):
    """Declare the C signatures of ``EXPORTED`` on a loaded library."""
    vp, i32, u32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float, ctypes.c_size_t
    psz = ctypes.POINTER(sz)
    args = {
        "bsgemm_quantize": [vp, u32, u32, i32, i32, u32, vp, vp, vp],
        "bsgemm_swiglu_backward": [vp, vp, u32, i32, i32, vp, vp],
        "bsgemm_rms_norm_quantize": [vp, vp, vp, u32, i32, i32, f32, u32, vp, vp, vp, vp, vp],
        "bsgemm_rms_norm_backward": [vp, vp, vp, vp, vp, u32, i32, i32, vp, vp, vp, sz, vp],
        "bsgemm_rms_norm_backward_workspace_size": [i32, i32, psz],
        "bsgemm_route_sort": [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp],
        "bsgemm_route_sort_workspace_size": [i32, i32, psz],
        "bsgemm_permute_rows": [vp, i32, vp, i32, i32, vp, vp, i32, i32, vp, vp],
        "bsgemm_combine_rows": [vp, u32, vp, vp, i32, i32, i32, i32, vp, vp],
        "bsgemm_combine_backward": [vp, vp, u32, vp, vp, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp],
        "bsgemm_grouped_few_rows": [vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, u32, vp],
    }
    for name, types in args.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = types, ctypes.c_int


# q_fmt word -> (elements per code byte, elements per scale, scale type)
_QUANT_LAYOUT = {1 | (1 << 8): (1, 128, torch.float32), 1 | (2 << 8): (1, 32, torch.uint8),
                 2 | (2 << 8): (2, 32, torch.uint8), 2 | (3 << 8): (2, 16, torch.uint8)}


def make_quant(elem, scale):
    """Pack a quantised form's element format and scale kind into the C ABI's ``q_fmt`` word."""
    q_fmt = _QUANT_WORDS.get((elem, scale))
    if q_fmt is None:
        raise ValueError(f"unsupported quantised form ({elem}, {scale}); one of {QUANTS}")
    return q_fmt


def quant_shapes(q_fmt, rows, K):
    """((codes shape), (scales shape), scales dtype) of ``rows`` x ``K`` values in form ``q_fmt``."""
    layout = _QUANT_LAYOUT.get(q_fmt)
    if layout is None:
        raise ValueError(f"unknown q_fmt {q_fmt:#x}")
    return (rows, K // layout[0]), (rows, K // layout[1]), layout[2]


# --------------------------------------------------------------------------------------
# helpers
#
# A decode step makes several of these calls on kernels of a few microseconds, so what a call does on
# the host counts: messages are only formatted when a check fails, a tensor's attributes are read once,
# and its checks and its pointer come from one function.
# --------------------------------------------------------------------------------------
_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32

# The bare forms of torch.cuda.current_device() and current_stream() where torch has them (0.1 and 0.1 us a
# call; the public ones 0.2 and, building a Stream object, 2.9 us).
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _matrix(t, name):
    """(rows, columns, row type code, type) of a row matrix."""
    shape, dtype = t.shape, t.dtype
    code = ROW_DTYPE.get(dtype)
    if len(shape) != 2 or code is None:
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 matrix, got {dtype} of shape {tuple(shape)}")
    return shape[0], shape[1], code, dtype


def _placed(t, name, here):
    """The pointer of a contiguous tensor on device ``here``."""
    if t.get_device() != here or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on device {here}, got one on {t.device} with strides {t.stride()}")
    return t.data_ptr()


def _arg(t, name, shape, dtype, here):
    """The pointer of a contiguous tensor of this shape and type on device ``here``; None of None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of shape {tuple(t.shape)}")
    if t.get_device() != here or not t.is_contiguous():
        return _placed(t, name, here)
    return t.data_ptr()


def _new(shape, dtype, like, stream):
    """A new tensor on ``like``'s device, in the memory pool of the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


_functions = {}


def _function(name):
    fn = _functions.get(name)
    if fn is None:
        from . import load_library

        fn = _functions[name] = getattr(load_library(), name)
    return fn


def _failed(name, status):
    from . import BsgemmError

    return BsgemmError(name, status)


def _handle(stream, here):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(here)
    return torch.cuda.current_stream().cuda_stream


@functools.lru_cache(maxsize=1024)
def _size(name, device, *args):
    """Bytes that a size function of the library gives for ``args`` on ``device`` (the current one)."""
    n = ctypes.c_size_t(0)
    status = _function(name)(*args, ctypes.byref(n))
    if status != 0:
        raise _failed(name, status)
    return n.value


def _workspace(ws, need, like, stream, here):
    """(tensor, pointer, bytes) of ``ws``, or of a workspace of ``need`` bytes for this call (none for 0)."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = _new(need, _U8, like, stream)
    nbytes = ws.numel() * ws.element_size()
    if nbytes < need:
        raise ValueError(f"workspace holds {nbytes} bytes, the call needs {need}")
    return ws, _placed(ws, "workspace", here), nbytes


# --------------------------------------------------------------------------------------
# quantisation
# --------------------------------------------------------------------------------------
def _quantize_args(here, x, q_fmt, act, q, scales):
    rows, K, code, _ = _matrix(x, "x")
    if act == "swiglu":
        if K % 2:
            raise ValueError(f"x must be [rows, 2 K] for swiglu, got {K} columns")
        K //= 2
    elif act != "none":
        raise ValueError(f"act must be one of {tuple(ACT)}, got {act!r}")
    layout = quant_shapes(q_fmt, rows, K)
    return (code, rows, K, layout, _placed(x, "x", here), _arg(q, "q", layout[0], _U8, here),
            _arg(scales, "scales", layout[1], layout[2], here))


def check_quantize_args(x, q_fmt, act, q=None, scales=None):
    """The checks of a ``bsgemm_quantize`` call."""
    _quantize_args(x.get_device(), x, q_fmt, act, q, scales)


def bsgemm_quantize(x, q_fmt, act="none", q=None, scales=None, stream=None):
    """Rows ``x`` [rows, K], or the SwiGLU of ``x`` [rows, 2 K], in the quantised form ``q_fmt``
    (:func:`make_quant`). Returns (codes uint8, scales), detached from autograd: SwiGLU's gradient is
    ``bsgemm_swiglu_backward``."""
    here = _device()
    code, rows, K, layout, px, pq, ps = _quantize_args(here, x, q_fmt, act, q, scales)
    if q is None:
        q = _new(layout[0], _U8, x, stream)
        pq = q.data_ptr()
    if scales is None:
        scales = _new(layout[1], layout[2], x, stream)
        ps = scales.data_ptr()
    status = _function("bsgemm_quantize")(px, code, ACT[act], rows, K, q_fmt, pq, ps, _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_quantize", status)
    return q, scales


def _swiglu_backward_args(here, dy, x, dx):
    rows, K, code, dtype = _matrix(dy, "dy")
    shape = (rows, 2 * K)
    return (code, rows, K, _placed(dy, "dy", here), _arg(x, "x", shape, dtype, here), _arg(dx, "dx", shape, dtype, here))


def check_swiglu_backward_args(dy, x, dx=None):
    """The checks of a ``bsgemm_swiglu_backward`` call."""
    _swiglu_backward_args(dy.get_device(), dy, x, dx)


def bsgemm_swiglu_backward(dy, x, dx=None, stream=None):
    """Gradient of the SwiGLU of ``x`` [rows, 2 K] from that of its unquantised output, ``dy`` [rows, K].
    Returns ``dx`` [rows, 2 K], which may be given as ``x`` itself."""
    here = _device()
    code, rows, K, pdy, px, pdx = _swiglu_backward_args(here, dy, x, dx)
    if dx is None:
        dx = _new((rows, 2 * K), x.dtype, x, stream)
        pdx = dx.data_ptr()
    status = _function("bsgemm_swiglu_backward")(pdy, px, code, rows, K, pdx, _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_swiglu_backward", status)
    return dx


# --------------------------------------------------------------------------------------
# norm
# --------------------------------------------------------------------------------------
def _norm_args(here, x, weight, q_fmt, residual, residual_out, rstd, q, scales):
    rows, K, code, dtype = _matrix(x, "x")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out is given without residual")
    layout, shape = quant_shapes(q_fmt, rows, K), (rows, K)
    return (code, rows, K, layout, _placed(x, "x", here), _arg(weight, "weight", (K,), dtype, here),
            _arg(residual, "residual", shape, dtype, here), _arg(residual_out, "residual_out", shape, dtype, here),
            _arg(rstd, "rstd", (rows,), _F32, here), _arg(q, "q", layout[0], _U8, here),
            _arg(scales, "scales", layout[1], layout[2], here))


def check_norm_args(x, weight, q_fmt, residual=None, residual_out=None, rstd=None, q=None, scales=None):
    """The checks of a ``bsgemm_rms_norm_quantize`` call."""
    _norm_args(x.get_device(), x, weight, q_fmt, residual, residual_out, rstd, q, scales)


def bsgemm_rms_norm_quantize(x, weight, q_fmt, eps=1e-6, residual=None, residual_out=None, rstd=None, q=None,
                             scales=None, stream=None):
    """RMS norm of ``x + residual`` (``x`` without one) in the quantised form ``q_fmt``. Returns
    (codes, scales, residual_out, rstd); residual_out, the rounded sum, is None without a residual
    and may be given as ``residual`` itself. Detached from autograd: the gradient is ``bsgemm_rms_norm_backward``."""
    here = _device()
    code, rows, K, layout, px, pw, pr, po, pd, pq, ps = _norm_args(here, x, weight, q_fmt, residual, residual_out, rstd,
                                                                   q, scales)
    if po is None and residual is not None:
        residual_out = _new((rows, K), x.dtype, x, stream)
        po = residual_out.data_ptr()
    if rstd is None:
        rstd = _new((rows,), _F32, x, stream)
        pd = rstd.data_ptr()
    if q is None:
        q = _new(layout[0], _U8, x, stream)
        pq = q.data_ptr()
    if scales is None:
        scales = _new(layout[1], layout[2], x, stream)
        ps = scales.data_ptr()
    status = _function("bsgemm_rms_norm_quantize")(px, pr, pw, code, rows, K, eps, q_fmt, po, pd, pq, ps,
                                                   _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_rms_norm_quantize", status)
    return q, scales, residual_out, rstd


def _norm_backward_args(here, dy, h, weight, rstd, dresidual, dx, dweight):
    rows, K, code, dtype = _matrix(dy, "dy")
    shape = (rows, K)
    return (code, rows, K, _placed(dy, "dy", here), _arg(h, "h", shape, dtype, here),
            _arg(weight, "weight", (K,), dtype, here), _arg(rstd, "rstd", (rows,), _F32, here),
            _arg(dresidual, "dresidual", shape, dtype, here), _arg(dx, "dx", shape, dtype, here),
            _arg(dweight, "dweight", (K,), _F32, here))


def check_norm_backward_args(dy, h, weight, rstd, dresidual=None, dx=None, dweight=None):
    """The checks of a ``bsgemm_rms_norm_backward`` call."""
    _norm_backward_args(dy.get_device(), dy, h, weight, rstd, dresidual, dx, dweight)


def bsgemm_rms_norm_backward_workspace_size(rows, K):
    """Bytes of workspace ``bsgemm_rms_norm_backward`` needs on the current device."""
    return _size("bsgemm_rms_norm_backward_workspace_size", _device(), rows, K)


def bsgemm_rms_norm_backward(dy, h, weight, rstd, dresidual=None, dx=None, dweight=None, workspace=None, stream=None):
    """Gradient of the norm: (dx, dweight float32) from the gradient ``dy`` of its unquantised output,
    the stored sum ``h`` and ``rstd``, plus ``dresidual`` where the sum is used elsewhere too."""
    here = _device()
    code, rows, K, pdy, ph, pw, pr, pres, pdx, pdw = _norm_backward_args(here, dy, h, weight, rstd, dresidual, dx, dweight)
    need = _size("bsgemm_rms_norm_backward_workspace_size", here, rows, K)
    workspace, pws, nbytes = _workspace(workspace, need, dy, stream, here)
    if dx is None:
        dx = _new((rows, K), dy.dtype, dy, stream)
        pdx = dx.data_ptr()
    if dweight is None:
        dweight = _new((K,), _F32, dy, stream)
        pdw = dweight.data_ptr()
    status = _function("bsgemm_rms_norm_backward")(pdy, ph, pw, pr, pres, code, rows, K, pdx, pdw, pws, nbytes,
                                                   _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_rms_norm_backward", status)
    return dx, dweight


# --------------------------------------------------------------------------------------
# picks sorted by expert, rows there and back
# --------------------------------------------------------------------------------------
def _route_sort_args(here, topk_ids, E, T, dest, counts, expert_offsets, tile_offsets, expert_ids):
    if topk_ids.dtype != _I32:
        raise ValueError(f"topk_ids must be int32, got {topk_ids.dtype}")
    return (_placed(topk_ids, "topk_ids", here), _arg(dest, "dest", topk_ids.shape, _I32, here),
            _arg(counts, "counts", (E,), _I32, here), _arg(expert_offsets, "expert_offsets", (E + 1,), _I32, here),
            _arg(tile_offsets, "tile_offsets", (T + 1,), _I32, here), _arg(expert_ids, "expert_ids", (T,), _I32, here))


def check_route_sort_args(topk_ids, num_experts, num_tiles, dest=None, counts=None, expert_offsets=None,
                          tile_offsets=None, expert_ids=None):
    """The checks of a ``bsgemm_route_sort`` call."""
    _route_sort_args(topk_ids.get_device(), topk_ids, num_experts, num_tiles, dest, counts, expert_offsets, tile_offsets,
                     expert_ids)


def bsgemm_route_sort_workspace_size(num_picks, num_experts):
    """Bytes of workspace ``bsgemm_route_sort`` needs (0 for a decode batch)."""
    return _size("bsgemm_route_sort_workspace_size", None, num_picks, num_experts)


def bsgemm_route_sort(topk_ids, num_experts, num_tiles, M, padded=True, dest=None, counts=None, expert_offsets=None,
                      tile_offsets=None, expert_ids=None, workspace=None, stream=None):
    """Sort int32 top-k ids (any shape) by expert. Returns (dest, counts, expert_offsets, tile_offsets,
    expert_ids): the row of every pick, and what ``bsgemm_route_counts`` and ``bsgemm_build_tiles`` give."""
    here = _device()
    pi, pd, pc, po, pt, pe = _route_sort_args(here, topk_ids, num_experts, num_tiles, dest, counts, expert_offsets,
                                              tile_offsets, expert_ids)
    n = topk_ids.numel()
    need = _size("bsgemm_route_sort_workspace_size", None, n, num_experts)
    workspace, pws, nbytes = _workspace(workspace, need, topk_ids, stream, here)
    if dest is None:
        dest = _new(topk_ids.shape, _I32, topk_ids, stream)
        pd = dest.data_ptr()
    if counts is None:
        counts = _new((num_experts,), _I32, topk_ids, stream)
        pc = counts.data_ptr()
    if expert_offsets is None:
        expert_offsets = _new((num_experts + 1,), _I32, topk_ids, stream)
        po = expert_offsets.data_ptr()
    if tile_offsets is None:
        tile_offsets = _new((num_tiles + 1,), _I32, topk_ids, stream)
        pt = tile_offsets.data_ptr()
    if expert_ids is None:
        expert_ids = _new((num_tiles,), _I32, topk_ids, stream)
        pe = expert_ids.data_ptr()
    status = _function("bsgemm_route_sort")(pi, n, num_experts, num_tiles, 1 if padded else 0, M, pc, po, pt, pe, pd, pws,
                                            nbytes, _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_route_sort", status)
    return dest, counts, expert_offsets, tile_offsets, expert_ids


def _picks(dest, tokens, here):
    """(top_k, pointer) of ``dest`` [tokens, top_k]."""
    shape = dest.shape
    if len(shape) != 2 or shape[0] != tokens or shape[1] < 1 or dest.dtype != _I32:
        raise ValueError(f"dest must be int32 [tokens={tokens}, top_k], got {dest.dtype} of shape {tuple(shape)}")
    return shape[1], _placed(dest, "dest", here)


def _groups(counts, expert_offsets, here):
    """(experts, pointers) of the sort's counts and group offsets."""
    shape = counts.shape
    if len(shape) != 1:
        raise ValueError(f"counts must be 1-D, got shape {tuple(shape)}")
    return (shape[0], _arg(counts, "counts", shape, _I32, here),
            _arg(expert_offsets, "expert_offsets", (shape[0] + 1,), _I32, here))


def _permute_rows_args(here, x, dest, counts, expert_offsets, M, out):
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError(f"x must be [tokens, K], got shape {tuple(shape)}")
    tokens, K = shape
    return (tokens, K * dtype.itemsize, _placed(x, "x", here), *_picks(dest, tokens, here),
            *_groups(counts, expert_offsets, here), _arg(out, "out", (M, K), dtype, here))


def check_permute_rows_args(x, dest, counts, expert_offsets, M, out=None):
    """The checks of a ``bsgemm_permute_rows`` call."""
    _permute_rows_args(x.get_device(), x, dest, counts, expert_offsets, M, out)


def bsgemm_permute_rows(x, dest, counts, expert_offsets, M, out=None, stream=None):
    """Rows of ``x`` [tokens, K] (any element type, rows of whole 4-byte words) at the rows of their picks
    in ``out`` [M, K]; padding rows of the groups are zero, other rows untouched. Returns ``out``
    (zeros outside the groups if it is allocated here), detached from autograd: the gradient is
    ``bsgemm_combine_rows`` without weights."""
    here = _device()
    tokens, row_bytes, px, top_k, pd, E, pc, po, pout = _permute_rows_args(here, x, dest, counts, expert_offsets, M, out)
    if out is None:
        out = _new((M, x.shape[1]), x.dtype, x, stream)
        with torch.cuda.stream(stream):
            out.zero_()
        pout = out.data_ptr()
    status = _function("bsgemm_permute_rows")(px, row_bytes, pd, tokens, top_k, pc, po, E, M, pout, _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_permute_rows", status)
    return out


def _combine_args(here, y, dest, weights, out):
    M, K, code, dtype = _matrix(y, "y")
    picks = dest.shape
    tokens = picks[0] if picks else 0
    return (M, K, code, tokens, _placed(y, "y", here), *_picks(dest, tokens, here),
            _arg(weights, "weights", picks, _F32, here), _arg(out, "out", (tokens, K), dtype, here))


def check_combine_args(y, dest, weights=None, out=None):
    """The checks of a ``bsgemm_combine_rows`` call."""
    _combine_args(y.get_device(), y, dest, weights, out)


def bsgemm_combine_rows(y, dest, weights=None, out=None, stream=None):
    """Weighted sum of the rows of each token's picks: ``y`` [M, K] -> [tokens, K]. Without ``weights``
    (float32 [tokens, top_k]) the plain sum, which is the gradient of ``bsgemm_permute_rows``. The result is detached
    from autograd: the gradient is ``bsgemm_combine_backward``, without weights ``bsgemm_permute_rows``."""
    here = _device()
    M, K, code, tokens, py, top_k, pd, pw, po = _combine_args(here, y, dest, weights, out)
    if out is None:
        out = _new((tokens, K), y.dtype, y, stream)
        po = out.data_ptr()
    status = _function("bsgemm_combine_rows")(py, code, pd, pw, tokens, top_k, K, M, po, _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_combine_rows", status)
    return out


def _combine_backward_args(here, dout, y, dest, weights, counts, expert_offsets, dy, dweights):
    M, K, code, dtype = _matrix(y, "y")
    picks = dest.shape
    tokens = picks[0] if picks else 0
    return (M, K, code, tokens, _arg(dout, "dout", (tokens, K), dtype, here), _placed(y, "y", here),
            *_picks(dest, tokens, here), _arg(weights, "weights", picks, _F32, here),
            *_groups(counts, expert_offsets, here), _arg(dy, "dy", (M, K), dtype, here),
            _arg(dweights, "dweights", picks, _F32, here))


def check_combine_backward_args(dout, y, dest, weights, counts, expert_offsets, dy=None, dweights=None):
    """The checks of a ``bsgemm_combine_backward`` call."""
    _combine_backward_args(y.get_device(), dout, y, dest, weights, counts, expert_offsets, dy, dweights)


def bsgemm_combine_backward(dout, y, dest, weights, counts, expert_offsets, dy=None, dweights=None, stream=None):
    """Gradient of the weighted ``bsgemm_combine_rows``: (dy [M, K], dweights). Padding rows of the groups
    are zero in ``dy``, other rows without a pick untouched (zeros if ``dy`` is allocated here)."""
    here = _device()
    M, K, code, tokens, pdo, py, top_k, pd, pw, E, pc, po, pdy, pdw = _combine_backward_args(
        here, dout, y, dest, weights, counts, expert_offsets, dy, dweights)
    if dy is None:
        dy = _new((M, K), y.dtype, y, stream)
        with torch.cuda.stream(stream):
            dy.zero_()
        pdy = dy.data_ptr()
    if dweights is None:
        dweights = _new((tokens, top_k), _F32, y, stream)
        pdw = dweights.data_ptr()
    status = _function("bsgemm_combine_backward")(pdo, py, code, pd, pw, tokens, top_k, K, pc, po, E, M, pdy, pdw,
                                                  _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_combine_backward", status)
    return dy, dweights


# --------------------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------------------
def bsgemm_grouped_few_rows(A, a_scales, B, b_scales, expert_ids, tile_offsets, C, M, N, K, fmt, num_tiles=None,
                            num_experts=None, stream=None):
    """``bsgemm_grouped`` with an MX ``fmt`` (A or B e2m1) for M-tiles of few rows (a decode batch): the
    weights are streamed once and only the rows that are there are computed. Arguments as there."""
    from . import check_grouped_args

    if num_tiles is None:
        num_tiles = expert_ids.numel() if expert_ids is not None else 0
    if num_experts is None:
        shape = B.shape
        num_experts = shape[0] if len(shape) == 3 else 1
    check_grouped_args(A, a_scales, B, b_scales, expert_ids, tile_offsets, C, M, N, K, fmt, num_tiles, num_experts)
    here = _device()
    status = _function("bsgemm_grouped_few_rows")(
        _placed(A, "A", here), _placed(a_scales, "a_scales", here), _placed(B, "B", here),
        _placed(b_scales, "b_scales", here), None if expert_ids is None else _placed(expert_ids, "expert_ids", here),
        None if tile_offsets is None else _placed(tile_offsets, "tile_offsets", here), num_tiles, _placed(C, "C", here), M, N, K,
        num_experts, fmt, _handle(stream, here))
    if status != 0:
        raise _failed("bsgemm_grouped_few_rows", status)
    return C
