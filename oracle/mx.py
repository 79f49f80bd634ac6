"""fp64 reference of the microscaled (MX) operators and the RMS norm (numpy, tests only).

Shares no code with the CUDA path.  Formats after OCP Microscaling Formats (MX)
v1.0: blocks of 32 columns with a scale byte s (2^(s - 127), 255 = NaN) and
e2m1 or e4m3 elements; rounding to nearest, ties to the even code, by search in
the table of the format's values.
"""
from __future__ import annotations

import numpy as np

E2M1, E4M3 = 0, 1
TOP = {E2M1: 2, E4M3: 8}


def values(fmt):
    """The value of each code without its sign bit, in order (e4m3 without its NaN)."""
    if fmt == E2M1:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))


def pitch(cols):
    return -(-cols // 128) * 128


def scale_byte(amax, fmt):
    """The scale byte of blocks with these largest magnitudes (0 and subnormals of fp32: byte 0)."""
    amax = np.asarray(amax, np.float64)
    out = np.zeros(amax.shape, np.int64)
    ok = np.isfinite(amax) & (amax > 0)
    out[ok] = np.clip(np.frexp(amax[ok])[1] - 1 - TOP[fmt], -127, 127) + 127
    out[~np.isfinite(amax)] = 255
    return out


def factor(byte):
    return np.where(byte == 255, np.nan, np.ldexp(1.0, np.asarray(byte, np.int64) - 127))


def round_codes(u, fmt):
    """|u| -> the nearest code (ties to even, saturating); u >= 0."""
    grid = values(fmt)
    up = np.clip(np.searchsorted(grid, u), 1, len(grid) - 1)
    low, high = u - grid[up - 1], grid[up] - u
    return np.where((low < high) | ((low == high) & (up % 2 == 1)), up - 1, up)


def blocks(v):
    """rows x cols -> rows x blocks x 32, zero behind the last column (to a multiple of 128 columns)."""
    v = np.asarray(v, np.float64)
    full = np.zeros((v.shape[0], pitch(v.shape[1])))
    full[:, :v.shape[1]] = v
    return full.reshape(v.shape[0], -1, 32)


def quantize(v, fmt):
    """rows x cols -> (codes rows x pitch with sign, scale bytes rows x pitch/32)."""
    b = blocks(v)
    byte = scale_byte(np.where(np.isnan(b), np.inf, np.abs(b)).max(2), fmt)
    bad = (byte == 255)[:, :, None]
    with np.errstate(invalid="ignore"):
        u = np.where(bad, 0.0, b / factor(byte)[:, :, None])
    code = round_codes(np.abs(u), fmt)
    sign = np.signbit(u) & ~np.broadcast_to(bad, u.shape)
    code = code | (sign.astype(np.int64) << (3 if fmt == E2M1 else 7))
    return code.reshape(b.shape[0], -1), byte


def code_values(code, fmt):
    grid = values(fmt)
    if fmt == E4M3:
        grid = np.append(grid, np.nan)
    top = 3 if fmt == E2M1 else 7
    v = grid[code & ((1 << top) - 1)]
    return np.where(code >> top, -v, v)


def dequantize(code, byte, cols, fmt):
    v = code_values(code, fmt).reshape(code.shape[0], -1, 32) * factor(byte)[:, :, None]
    return v.reshape(code.shape[0], -1)[:, :cols]


def pack_codes(code, fmt):
    """The codes buffer: two e2m1 to a byte, the even column low."""
    if fmt == E4M3:
        return code.astype(np.uint8).reshape(-1)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8).reshape(-1)


def unpack_codes(buf, rows, cols, fmt):
    buf = np.asarray(buf).astype(np.int64)
    if fmt == E2M1:
        n = rows * pitch(cols) // 2
        return np.stack((buf[:n] & 15, buf[:n] >> 4), 1).reshape(rows, -1)
    return buf[: rows * pitch(cols)].reshape(rows, -1)


def scale_index(rows, cols):
    """Where the scale byte of (row, block) lies in the scales buffer."""
    r, k = np.arange(rows)[:, None], np.arange(pitch(cols) // 32)[None, :]
    return ((r // 128) * (pitch(cols) // 128) + k // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4


def scale_bytes(rows, cols):
    return -(-rows // 128) * (pitch(cols) // 128) * 512


def pack_scales(byte, rows, cols):
    buf = np.zeros(scale_bytes(rows, cols), np.uint8)
    buf[scale_index(rows, cols)] = byte
    return buf


def unpack_scales(buf, rows, cols):
    return np.asarray(buf)[scale_index(rows, cols)].astype(np.int64)


def rmsnorm(h, weight, eps):
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rmsnorm_grads(dy, h, weight, eps, dh=None):
    """(dx, dweight) of the norm, from the formula."""
    dy, h, w = (np.asarray(t, np.float64) for t in (dy, h, weight))
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    g = dy * w
    dx = r * g - h * r ** 3 * (g * h).mean(1, keepdims=True)
    return dx + (0 if dh is None else np.asarray(dh, np.float64)), (dy * h * r).sum(0)
