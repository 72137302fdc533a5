"""The operators around the grouped GEMM by their definitions, in fp64 (oracle; test
infrastructure, see the package docstring).

* ``encode_e2m1`` / ``quantize`` - codes and scales of the four quantised forms of
  ``include/bsgemm.h``. The scales' and elements' divisions are the defined fp32 ones, so these
  are exact for given fp32 values.
* ``silu_mul``, ``rms_norm`` and its gradient, ``permute_rows``, ``combine`` and its gradient - plain
  formulas on fp64 arrays.

Pins: ``tests/test_oracle_operators.py`` (nearest-value brute force, the workload encoders, torch's
own functions, differences).
"""

import numpy as np

from .formats import decode_e2m1, decode_e4m3fn
from .permute import encode_e4m3fn

EMAX = {"e4m3": 8, "e2m1": 2}
MOST = {"e4m3": 448.0, "e2m1": 6.0}
FORMS = (("e4m3", "blockwise"), ("e4m3", "mx"), ("e2m1", "mx"), ("e2m1", "nv"))
BLOCK = {"blockwise": 128, "mx": 32, "nv": 16}


def encode_e2m1(values):
    """|v| <= 6 -> 4-bit codes, nearest value, ties to the even code, sign kept (-0 included)."""
    v = np.asarray(values, np.float64)
    grid = decode_e2m1(np.arange(8))
    upper = np.searchsorted(grid, np.abs(v), side="left").clip(0, 7)       # first grid value >= |v|
    lower = np.maximum(upper - 1, 0)
    up, down = grid[upper] - np.abs(v), np.abs(v) - grid[lower]
    code = np.where(up < down, upper, np.where(down < up, lower, np.where(upper % 2 == 0, upper, lower)))
    code = np.where(np.abs(v) == grid[upper], upper, code)
    return (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def pack_nibbles(codes):
    """Codes [..., K] -> bytes [..., K/2], the even index in the low nibble."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def quantize(y, elem, kind):
    """fp32 values [R, K] -> (codes as stored, scales) of the form (elem, kind)."""
    y = np.asarray(y, np.float32)
    R, K = y.shape
    b = y.reshape(R, K // BLOCK[kind], BLOCK[kind])
    amax = np.abs(b).max(-1)
    most = np.float32(MOST[elem])
    if kind == "mx":
        exponent = np.frexp(amax.astype(np.float64))[1] - 1
        scales = np.where(amax > 0, np.clip(exponent - EMAX[elem] + 127, 0, 254), 127).astype(np.uint8)
        z = b.astype(np.float64) * np.exp2(127.0 - scales)[..., None]      # exact
    elif kind == "nv":
        code = encode_e4m3fn(np.minimum(amax / np.float32(6), np.float32(448)))
        scales = np.where(amax > 0, np.maximum(code, 1), 0x38).astype(np.uint8)
        z = b / decode_e4m3fn(scales).astype(np.float32)[..., None]
    else:
        scales = np.where(amax > 0, np.maximum(amax / np.float32(448), np.float32(2.0 ** -149)), np.float32(1)).astype(np.float32)
        z = b / scales[..., None]
    z = np.clip(z, -most, most).reshape(R, K)
    return (encode_e4m3fn(z) if elem == "e4m3" else pack_nibbles(encode_e2m1(z))), scales


def silu_mul(x):
    """[R, 2 K] -> silu of the first K columns times the last K, fp64."""
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    # g sigmoid(g) without overflow for either sign
    s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
    return g * s * u


def silu_mul_backward(dy, x):
    """Gradient of ``silu_mul`` at x, fp64."""
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    e = np.exp(-np.abs(g))
    s, rest = np.where(g >= 0, 1, e) / (1 + e), np.where(g >= 0, e, 1) / (1 + e)      # sigmoid, 1 - sigmoid
    dy = np.asarray(dy, np.float64)
    return np.concatenate([dy * u * s * (1 + g * rest), dy * g * s], axis=1)


def rms_norm(h, weight, eps):
    """(y, rstd) of rows h, fp64."""
    h = np.asarray(h, np.float64)
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * np.asarray(weight, np.float64), rstd


def rms_norm_backward(dy, h, weight, rstd, dresidual=None):
    """(dx, dweight) by the chain rule, rstd a function of h."""
    dy, h, w, r = (np.asarray(a, np.float64) for a in (dy, h, weight, rstd))
    r = r[:, None]
    g = dy * w
    dr = (g * h).sum(1, keepdims=True)                       # dL/drstd
    dx = g * r - dr * r ** 3 * h / h.shape[1]                # drstd/dh = -rstd^3 h / K
    return dx + (0 if dresidual is None else np.asarray(dresidual, np.float64)), (dy * h * r).sum(0)


def permute_rows(x, dest, counts, expert_offsets, out):
    """``out`` with the token rows at their picks' rows and zeros at the groups' padding rows."""
    out = np.array(out)
    M = out.shape[0]
    for e, c in enumerate(counts):
        out[min(expert_offsets[e] + c, M):min(expert_offsets[e + 1], M)] = 0
    for t, j in np.argwhere((dest >= 0) & (dest < M)):
        out[dest[t, j]] = x[t]
    return out


def combine(y, dest, weights=None):
    """Weighted sum of each token's rows, fp64."""
    y = np.asarray(y, np.float64)
    out = np.zeros((dest.shape[0], y.shape[1]))
    for t, j in np.argwhere((dest >= 0) & (dest < y.shape[0])):
        out[t] += (1.0 if weights is None else float(weights[t, j])) * y[dest[t, j]]
    return out


def combine_backward(dout, y, dest, weights, counts, expert_offsets, dy):
    """(``dy`` with the picks' rows and zero padding rows, dweights), fp64."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    dy = permute_rows(np.zeros_like(dout), dest, counts, expert_offsets, np.asarray(dy, np.float64))
    dw = np.zeros(dest.shape)
    for t, j in np.argwhere((dest >= 0) & (dest < y.shape[0])):
        dy[dest[t, j]] = float(weights[t, j]) * dout[t]
        dw[t, j] = dout[t] @ y[dest[t, j]]
    return dy, dw
