"""TEST INFRASTRUCTURE -- CPU oracle of the microscaled 4-bit formats.

Only ``tests/`` may import this module.  It shares no code with the CUDA library.

Values are E2M1 (sign, 2 exponent bits with bias 1, 1 mantissa bit: 0 0.5 1 1.5 2 3
4 6) with one 8-bit scale per block along a row:
  mxfp4: blocks of 32; byte = max(floor(log2 amax) - 2, -127) + 127, s = 2^(byte-127),
         q = E2M1(x / s), value = q s;
  nvfp4: blocks of 16, a tensor factor ts (fp32); byte = E4M3(fl(amax / fl(6 ts))) with
         value sb, q = E2M1(fl(x fl(1 / fl(sb ts)))), value = q sb ts;
nearest, ties to even, saturating (E2M1 at 6, E4M3 at 448); fl rounds to fp32.  A
block with a NaN or an infinity has the NaN scale (255 / 127) and codes 0; a scale
that rounds to 0 gives codes 0.
"""
from __future__ import annotations

import numpy as np

BLOCK = {"mxfp4": 32, "nvfp4": 16}
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
NAN_BYTE = {"mxfp4": 255, "nvfp4": 127}


def _nearest(grid, a):
    """Index of the nearest grid value (ascending grid), ties to the even index."""
    a = np.minimum(a, grid[-1])
    hi = np.searchsorted(grid, a, side="left")
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def e2m1_codes(v):
    """E2M1 codes of v (the sign of a zero is kept)."""
    v = np.asarray(v, np.float64)
    return (_nearest(GRID, np.abs(v)) + np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def e4m3_grid():
    """Finite non-negative E4M3 values by code 0..126."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def scale_values(byte, fmt):
    byte = np.asarray(byte).astype(np.int64)
    if fmt == "mxfp4":
        return np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))
    return np.where(byte == 127, np.nan, e4m3_grid()[np.minimum(byte, 126)])


def scale_bytes(amax, fmt, ts=1.0):
    """Scale bytes of blocks with largest magnitude amax (fp32 values; NaN/inf allowed)."""
    amax = np.asarray(amax, np.float32)
    bad = ~np.isfinite(amax)
    a = np.where(bad, np.float32(0), amax)
    if fmt == "mxfp4":
        e = np.where(a > 0, np.frexp(a.astype(np.float64))[1] - 1, -10 ** 6)
        byte = np.maximum(e - 2, -127) + 127
    else:
        with np.errstate(over="ignore"):
            t = a / (np.float32(6) * np.float32(ts))
        byte = _nearest(e4m3_grid(), t.astype(np.float64))
    return np.where(bad, NAN_BYTE[fmt], byte).astype(np.uint8)


def blocks(x, fmt):
    x = np.asarray(x)
    pad = -x.shape[1] % 32
    return np.pad(x, ((0, 0), (0, pad))).reshape(x.shape[0], -1, BLOCK[fmt])


def quantize(x, fmt, ts=1.0):
    """x [rows, cols] fp32 -> (codes [rows, cols to 32], scale bytes [rows, blocks])."""
    xb = blocks(np.asarray(x, np.float32), fmt)
    with np.errstate(invalid="ignore"):
        amax = np.max(np.abs(xb), axis=2) if xb.size else np.zeros(xb.shape[:2], np.float32)
        amax = np.where(np.isnan(xb).any(2), np.float32(np.nan), amax)
    byte = scale_bytes(amax, fmt, ts)
    s = scale_values(byte, fmt)
    if fmt == "mxfp4":
        with np.errstate(invalid="ignore"):
            y = xb.astype(np.float64) / s[..., None]
        zero = np.isnan(s)
    else:
        d = s.astype(np.float32) * np.float32(ts)
        zero = np.isnan(s) | (byte == 0)
        with np.errstate(invalid="ignore"):
            r = np.float32(1) / np.where(zero, np.float32(1), d)
            y = (xb * r[..., None]).astype(np.float64)
    y = np.where(zero[..., None], 0.0, y)
    return e2m1_codes(y).reshape(xb.shape[0], -1), byte


def values(codes, byte, fmt, ts=1.0, cols=None):
    """What the codes stand for, in 64 bits: [rows, cols]."""
    mag = GRID[codes & 7]
    q = np.where(codes >= 8, -mag, mag).reshape(codes.shape[0], -1, BLOCK[fmt])
    f = 1.0 if fmt == "mxfp4" else float(np.float32(ts))
    v = (q * scale_values(byte, fmt)[..., None] * f).reshape(codes.shape[0], -1)
    return v if cols is None else v[:, :cols]


def rounded(x, fmt, ts=1.0):
    """The 64-bit values of the 4-bit form of x."""
    c, b = quantize(x, fmt, ts)
    return values(c, b, fmt, ts, np.asarray(x).shape[1])


def pack(codes, byte, fmt):
    """Storage form: packed codes [rows, cols / 2], scale tiles [row tiles, tiles, 512]
    (padding bytes 0)."""
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    rows, nb = byte.shape
    tiles = -(-codes.shape[1] // 256) * 256 // BLOCK[fmt] // 4
    out = np.zeros((-(-rows // 128), tiles, 512), np.uint8)
    for r in range(rows):
        for b in range(nb):
            out[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte[r, b]
    return packed, out


def unpack(packed, tiles, rows, cols, fmt):
    """Storage form -> (codes, scale bytes)."""
    packed, tiles = np.asarray(packed), np.asarray(tiles)
    codes = np.empty((rows, packed.shape[1] * 2), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    nb = codes.shape[1] // BLOCK[fmt]
    r, b = np.arange(rows)[:, None], np.arange(nb)[None, :]
    return codes, tiles[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def gelu(x):
    return 0.5 * x * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)))
