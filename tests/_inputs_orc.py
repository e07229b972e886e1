"""64-bit forms of the operators that make the indexer's inputs (MXFP4 rows and products,
per-head norm and rotation, stored query heads and keys), in numpy on the CPU.  Test
infrastructure only; ml_dtypes' casts are the rounding to e2m1 and e4m3."""
from __future__ import annotations

import ml_dtypes
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e2m1_codes(y):
    """Codes of the nearest e2m1 values (ties to the even code, past 6 to 6; -0 kept)."""
    a = np.abs(y)
    mid = (LEVELS[1:] + LEVELS[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    mag = np.where(lo % 2 == 0, lo, hi)
    return (mag | (np.signbit(y).astype(np.int64) << 3)).astype(np.uint8)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[:-1] + (-1,))


def mxfp4(y):
    """(packed codes, scale bytes) of fp64 rows."""
    b = y.reshape(y.shape[:-1] + (-1, 32))
    with np.errstate(invalid="ignore"):
        top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1) | (top >= 2.0 ** 130)
    ex = np.frexp(np.where(bad, 1.0, top))[1] - 1          # floor(log2(top)); -1 for 0
    e = np.where(top > 0, np.maximum(ex - 2 + 127, 0), 0)
    with np.errstate(invalid="ignore"):
        q = np.where(bad[..., None], 0.0, b) * np.exp2(127.0 - e)[..., None]
    sf = np.where(bad, 255, e).astype(np.uint8)
    return pack(e2m1_codes(q).reshape(y.shape)), sf


def mxfp4_values(packed, sf):
    c = unpack(packed)
    v = np.where(c >= 8, -1.0, 1.0) * LEVELS[c & 7]
    s = np.where(sf == 255, np.nan, np.exp2(sf.astype(np.float64) - 127))
    return v * np.repeat(s, 32, -1)


def tile_scales(sf, fill=0):
    """Rows layout -> tiled layout, byte by byte from its definition."""
    r, n = sf.shape
    kt = -(-n // 4)
    out = np.full(-(-r // 128) * kt * 512, fill, np.uint8)
    i, j = np.meshgrid(np.arange(r), np.arange(n), indexing="ij")
    out[512 * ((i // 128) * kt + j // 4) + 16 * (i % 32) + 4 * (i % 128 // 32) + j % 4] = sf
    return out


def e4m3_round(z):
    """Nearest e4m3 values in fp64 (ties to even, past 448 to 448): spacing 2^-3 of the binade,
    least binade -6.  A library cast from fp64 may round to fp32 first, and 12.5 (1 + 2^-30)
    becomes the tie 12.5 and then 12 instead of 13."""
    ulp = np.exp2(np.maximum(np.frexp(z)[1] - 1, -6) - 3.0)
    return np.clip(np.round(z / ulp) * ulp, -448, 448)


def fp8(y):
    """(e4m3 codes, fp32 scales) of fp64 rows, one scale per row."""
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(y).max(-1)
        scale = (top / 448).astype(np.float32)
    bad = ~np.isfinite(y).all(-1) | ~np.isfinite(scale)
    scale = np.where((scale > 0) & ~bad, scale, np.float32(1))
    z = np.where(bad[..., None], 0.0, y) / scale.astype(np.float64)[..., None]
    codes = e4m3_round(z).astype(ml_dtypes.float8_e4m3fn).view(np.uint8)
    return codes, np.where(bad, np.float32(np.nan), scale).astype(np.float32)


def norm_rope(x, pos, weight=None, norm=True, rope=64, theta=10000.0, eps=1e-6):
    """Rows [.., heads, D] in fp64; pos of the leading dims."""
    D = x.shape[-1]
    y = x.astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        if norm:
            y = y / np.sqrt((y * y).sum(-1, keepdims=True) / D + np.float64(np.float32(eps)))
        if weight is not None:
            y = y * weight.astype(np.float64)
        if rope:
            j = np.arange(rope // 2)
            a = np.asarray(pos, np.float64)[..., None] * theta ** (-2.0 * j / rope)
            c, s = np.cos(a)[..., None, :], np.sin(a)[..., None, :]
            u, v = y[..., D - rope::2].copy(), y[..., D - rope + 1::2].copy()
            y = y.copy()
            y[..., D - rope::2] = u * c - v * s
            y[..., D - rope + 1::2] = u * s + v * c
    return y
