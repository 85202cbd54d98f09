"""MXFP8 (e4m3 values in groups of 32, one power-of-two scale each) in plain numpy, float64.

Test infrastructure only (see the package docstring). The element and scale
formats are the OCP Microscaling specification's MXFP8: e4m3 ("fn": no
infinities, 0x7F / 0xFF are NaN, largest finite 448, smallest subnormal 2^-9)
and e8m0 (code c stands for 2^(c - 127), 0xFF for NaN).

Reading of the quantiser, which the specification leaves open: the scale of a
group is the smallest power of two 2^j, j in [-127, 127], with amax <= 448 2^j
(no value saturates); the values are v / 2^j rounded to e4m3, nearest, ties
to even. An all-zero group has code 0. A group that holds an infinity or a NaN
has code 0xFF and stands for 32 NaN.
"""

from __future__ import annotations

import numpy as np

from . import moe_oracle as mo

GROUP = 32
E4M3_MAX = 448.0


def e4m3_round(v) -> np.ndarray:
    """v (|v| <= 448) rounded to the nearest e4m3 value, ties to the even mantissa."""
    v = np.asarray(v, np.float64)
    _, ex = np.frexp(v)  # |v| = f 2^ex, f in [0.5, 1)
    step = np.exp2(np.maximum(ex - 1, -6) - 3.0)
    return np.round(v / step) * step


def scale_exponent(amax) -> np.ndarray:
    """The smallest j in [-127, 127] with amax <= 448 2^j (-127 for 0)."""
    amax = np.asarray(amax, np.float64)
    f, ex = np.frexp(amax)  # 448 = 0.875 2^9
    j = np.where(f <= 0.875, ex - 9, ex - 8)
    return np.clip(np.where(amax == 0, -127, j), -127, 127)


def quantize(v) -> tuple[np.ndarray, np.ndarray]:
    """(e4m3 values, scale exponents) of the last dimension of finite v (a multiple of 32 long)."""
    v = np.asarray(v, np.float64)
    g = v.reshape(*v.shape[:-1], v.shape[-1] // GROUP, GROUP)
    j = scale_exponent(np.abs(g).max(-1))
    return e4m3_round(g / np.exp2(j.astype(np.float64))[..., None]).reshape(v.shape), j


def values(v) -> np.ndarray:
    """v as MXFP8 holds it."""
    q, j = quantize(v)
    return q * np.repeat(np.exp2(j.astype(np.float64)), GROUP, axis=-1)


def weight_values(w) -> np.ndarray:
    """[..., K, N] weights as MXFP8 along K holds them."""
    return np.swapaxes(values(np.swapaxes(mo.f64(w), -1, -2)), -1, -2)


def scale_tile_offset(row: int, group: int, K: int) -> int:
    """Byte of the scale of (row, 32-group) in the [ceil(N/128)][ceil(K/128)][512] tiles."""
    kb = -(-K // 128)
    return ((row // 128) * kb + group // 4) * 512 + 16 * (row % 32) + 4 * (row % 128 // 32) + group % 4


def ffn(x, wg, wu, wd) -> np.ndarray:
    """x (already MXFP8 values) through one GeGLU feed-forward whose weights are given as values."""
    z = x @ wg
    return values(mo.gelu_tanh(z) * (x @ wu)) @ wd


def block(x, w_router, wg, wu, wd, sg, su, sd, k, bias=None, routing=None, xv=None) -> np.ndarray:
    """The MXFP8 block in float64 from bf16 weights (bit patterns): quantises them, and x unless its values xv are given."""
    x = mo.f64(x)
    idx, wt = routing if routing is not None else mo.route(x, w_router, k, bias)[:2]
    xv = values(x) if xv is None else np.asarray(xv, np.float64)
    out = ffn(xv, weight_values(sg), weight_values(su), weight_values(sd))
    for e in np.unique(idx):
        tok, slot = np.nonzero(idx == e)
        y = ffn(xv[tok], weight_values(wg[e]), weight_values(wu[e]), weight_values(wd[e]))
        out[tok] += np.asarray(wt, np.float64)[tok, slot][:, None] * y
    return out
