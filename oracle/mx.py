"""Microscaled storage (oracle; test infrastructure only): MXFP4 blocks of the
frozen base and MXFP8 blocks of the optimiser's states.

Defined by the OCP Microscaling Formats specification v1.0 (block of 32, one
E8M0 scale; E2M1, E4M3 and E5M2 elements) with these readings:
  * MXFP4 scale exponent: floor(log2 amax) - 2, at least -127 (the
    specification's conversion, 2 being E2M1's largest exponent); elements
    nearest with ties to even, saturating at 6; an all-zero block has scale
    byte 0; a block with a NaN or an infinity has scale byte 255 and codes 0;
  * byte j of a row holds element 2j in bits 3..0 and 2j + 1 in bits 7..4; a
    row of scales is padded with zeros to a multiple of 16 bytes;
  * MXFP8 state scale exponent: floor(log2 amax) - 7 for E4M3 and - 14 for E5M2
    (no saturation even after rounding up), at least -127; an element that is not
    finite is stored as code 0x7F (NaN in both).

Elements are enumerated from the format's own definition and rounded by
searching the list of representable values in fp64.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32


def _minifloat(ebits, mbits, bias, top=None):
    """Ascending non-negative values of a sign/ebits/mbits format by code."""
    vals = []
    for c in range(1 << (ebits + mbits)):
        e, m = c >> mbits, c & ((1 << mbits) - 1)
        vals.append(math.ldexp(m, 1 - bias - mbits) if e == 0 else math.ldexp((1 << mbits) + m, e - bias - mbits))
    return np.array(vals[:top], np.float64)


E2M1 = _minifloat(2, 1, 1)
E4M3 = _minifloat(4, 3, 7, top=127)   # code 0x7F is NaN
E5M2 = _minifloat(5, 2, 15, top=124)  # codes 0x7C.. are infinity and NaN
TOP = {id(E4M3): 7, id(E5M2): 14}     # exponent that a block's largest element is brought to


def scale_stride(in_f):
    return -(-(in_f // BLOCK) // 16) * 16


def floor_log2(x):
    """floor(log2 x) of positive fp64 values, exact."""
    return np.frexp(x)[1] - 1


def nearest(table, a):
    """Index of the table value nearest to each a >= 0, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(pick_hi, hi, lo)


def mx4_quantize(W):
    """W fp32 [out, in] -> (codes uint8 [out, in/2], scales uint8 [out, stride])."""
    W = np.asarray(W, np.float32)
    out_f, in_f = W.shape
    x = W.astype(np.float64).reshape(out_f, in_f // BLOCK, BLOCK)
    bad = ~np.isfinite(x).all(-1)
    xs = np.where(bad[..., None], 0.0, x)
    amax = np.abs(xs).max(-1)
    e = np.where(amax > 0, np.maximum(floor_log2(np.where(amax > 0, amax, 1.0)) - 2, -127), -127)
    code = nearest(E2M1, np.abs(xs) / np.exp2(e)[..., None]).astype(np.uint8)
    code |= (np.signbit(x) & ~bad[..., None]).astype(np.uint8) << 3
    flat = code.reshape(out_f, in_f)
    scales = np.zeros((out_f, scale_stride(in_f)), np.uint8)
    scales[:, :in_f // BLOCK] = np.where(bad, 255, e + 127)
    return (flat[:, 0::2] | (flat[:, 1::2] << 4)).astype(np.uint8), scales


def mx4_dequant(codes, scales):
    """fp64 values (NaN blocks as NaN)."""
    out_f, half = codes.shape
    n = np.empty((out_f, 2 * half), np.uint8)
    n[:, 0::2] = codes & 15
    n[:, 1::2] = codes >> 4
    v = np.where(n >= 8, -1.0, 1.0) * E2M1[n & 7]
    s = scales[:, :2 * half // BLOCK].astype(np.float64)
    s = np.where(s == 255, np.nan, np.exp2(s - 127))
    return v * np.repeat(s, BLOCK, axis=1)


# ------------------------------------------------------------- MXFP8 states
def _mix(h):
    h = h ^ (h >> np.uint32(16))
    h = h * np.uint32(0x85EBCA6B)
    h = h ^ (h >> np.uint32(13))
    h = h * np.uint32(0xC2B2AE35)
    return h ^ (h >> np.uint32(16))


def random16(n, tensor, seed, t):
    """The 16 random bits of each of a tensor's n elements at step t."""
    with np.errstate(over="ignore"):
        key = _mix(np.array([tensor], np.uint32) + np.uint32((0x9E3779B9 * t) & 0xFFFFFFFF))
        key = _mix(key + np.uint32(seed & 0xFFFFFFFF))
        i = np.arange(n, dtype=np.uint64)
        h = _mix((i >> np.uint64(1)).astype(np.uint32) + key)
    return np.where(i % 2 == 1, h >> np.uint32(16), h & np.uint32(0xFFFF)).astype(np.int64)


def decode(code, table):
    c = np.asarray(code).astype(np.int64)
    n = len(table)
    v = np.where((c & 127) >= n, np.nan, table[np.minimum(c & 127, n - 1)])
    return np.where(c >= 128, -v, v)


def state_decode(code, scale, table):
    n = len(code)
    return decode(code, table) * np.repeat(np.exp2(scale.astype(np.float64) - 127), BLOCK)[:n]


def _blocks(x):
    n = len(x)
    p = np.zeros(-(-n // BLOCK) * BLOCK, np.float64)
    p[:n] = x
    return p.reshape(-1, BLOCK)


def state_scale(x, table):
    """Scale bytes of the blocks of |x|, from its finite elements."""
    a = np.abs(_blocks(np.where(np.isfinite(x), x, 0.0))).max(-1)
    e = np.maximum(floor_log2(np.where(a > 0, a, 1.0)) - TOP[id(table)], -127)
    return np.where(a > 0, e + 127, 0).astype(np.uint8)


def _scaled(x, table):
    s = state_scale(x, table)
    return np.abs(x) / np.repeat(np.exp2(s.astype(np.float64) - 127), BLOCK)[:len(x)], s


def _signed(c, x):
    fin = np.isfinite(x)
    return np.where(fin, c + np.signbit(x) * 128, 0x7F).astype(np.uint8)


def state_encode_nearest(x, table):
    y, s = _scaled(x, table)
    return _signed(nearest(table, np.where(np.isfinite(y), y, 0.0)), x), s


def state_encode_stochastic(x, rnd16, table, keep_nonzero=False):
    """The neighbour below |x|, or the one above when the part of the step above the lower neighbour plus
    rnd / 2^16 reaches a whole step; keep_nonzero: a nonzero x keeps at least the smallest code."""
    y, s = _scaled(x, table)
    yf = np.where(np.isfinite(y), y, 0.0)
    lo = np.searchsorted(table, yf, side="right") - 1
    part = (yf - table[lo]) / (table[np.minimum(lo + 1, len(table) - 1)] - table[lo])
    c = lo + (part + rnd16 / 65536.0 >= 1.0)
    if keep_nonzero:
        c = np.where((c == 0) & (yf > 0), 1, c)
    return _signed(c, x), s
