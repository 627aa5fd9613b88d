"""CPU oracle of the microscaled operators: numpy, 64-bit sums, written from the
definitions in include/skgemm.h (test infrastructure only; no code shared with
the CUDA path).

The block scales and codes are defined down to the bit, so quantize() returns
the bytes themselves; "nvfp4" is defined in 32-bit arithmetic, which numpy's
float32 follows operation by operation.
"""
from __future__ import annotations

import numpy as np

BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
BITS = {"mxfp8": 8, "mxfp4": 4, "nvfp4": 4}


def _table(exp_bits: int, man_bits: int, bias: int) -> np.ndarray:
    """Magnitudes of all non-negative codes, ascending."""
    out = []
    for e in range(1 << exp_bits):
        for m in range(1 << man_bits):
            f = m / (1 << man_bits)
            out.append(f * 2.0 ** (1 - bias) if e == 0 else (1 + f) * 2.0 ** (e - bias))
    return np.array(out, dtype=np.float64)


E2M1 = _table(2, 1, 1)
E4M3 = _table(4, 3, 7)[:127]  # 0x7f is NaN


def nearest_code(y: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Number of the table entry nearest to |y| (|y| <= the last one, or
    saturating), ties to the even number."""
    a = np.abs(np.asarray(y, dtype=np.float64))
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def pad_k(x: np.ndarray) -> np.ndarray:
    rows, k = x.shape
    kp = -(-k // 32) * 32
    return np.pad(x, ((0, 0), (0, kp - k)))


def quantize(x: np.ndarray, fmt: str, g: float = 1.0):
    """(codes rows x padded k, one code per element; scale bytes rows x blocks)."""
    n = BLOCK[fmt]
    xp = pad_k(np.asarray(x, dtype=np.float32))
    xb = xp.reshape(xp.shape[0], -1, n)
    bad = ~np.isfinite(xb).all(-1)
    xs = np.where(bad[..., None], np.float32(0), xb)
    amax = np.abs(xs).max(-1)
    table = E4M3 if fmt == "mxfp8" else E2M1
    with np.errstate(all="ignore"):
        if fmt == "nvfp4":
            t = np.minimum(amax / (np.float32(6) * np.float32(g)), np.float32(448))
            s = nearest_code(t, E4M3)
            sg = E4M3[s].astype(np.float32) * np.float32(g)
            inv = np.where(sg > 0, np.float32(1) / sg, np.float32(0))
            y = xs * inv[..., None]
            bad_byte = 0x7F
        else:
            most = table[-1]
            e = np.full(amax.shape, -127, dtype=np.int64)
            nz = amax > 0
            m, ex = np.frexp(amax[nz].astype(np.float64) / most)  # in [1/2, 1) * 2^ex
            e[nz] = np.where(m > 0.5, ex, ex - 1)
            e = np.maximum(e, -127)
            s = e + 127
            y = xs.astype(np.float64) * np.exp2(-e.astype(np.float64))[..., None]
            bad_byte = 0xFF
    codes = nearest_code(y, table) | (np.signbit(y).astype(np.int64) << (BITS[fmt] - 1))
    codes = np.where(bad[..., None], 0, codes)
    return (codes.reshape(xp.shape).astype(np.uint8),
            np.where(bad, bad_byte, s).astype(np.uint8))


def pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "mxfp8":
        return codes
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(stored: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "mxfp8":
        return stored
    return np.stack((stored & 15, stored >> 4), -1).reshape(stored.shape[0], -1)


def scale_offset(r: int, b: int, groups: int) -> int:
    """Byte of row r's scale of block b."""
    return ((r // 128) * groups + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def tile_scales(s: np.ndarray) -> np.ndarray:
    rows, nb = s.shape
    groups = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * groups * 512, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[scale_offset(r, b, groups)] = s
    return out


def scale_values(s: np.ndarray, fmt: str) -> np.ndarray:
    s = s.astype(np.int64)
    if fmt == "nvfp4":
        return np.where((s & 0x7F) == 0x7F, np.nan, np.append(E4M3, np.nan)[s & 0x7F])
    return np.where(s == 0xFF, np.nan, np.exp2(s.astype(np.float64) - 127))


def code_values(codes: np.ndarray, fmt: str) -> np.ndarray:
    bits = BITS[fmt]
    table = np.append(E4M3, np.nan) if fmt == "mxfp8" else E2M1
    c = codes.astype(np.int64)
    v = table[c & ((1 << (bits - 1)) - 1)]
    return np.where(c >> (bits - 1) == 1, -v, v)


def values(codes: np.ndarray, scales: np.ndarray, fmt: str, g: float, k: int) -> np.ndarray:
    """What codes (one per element) and scales (rows x blocks) stand for."""
    v = code_values(codes, fmt).reshape(codes.shape[0], -1, BLOCK[fmt])
    return (v * scale_values(scales, fmt)[..., None] * g).reshape(codes.shape[0], -1)[:, :k]


def rmsnorm(x, weight, eps, residual=None):
    """(y, h, rstd) in 64 bits."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * np.asarray(weight, dtype=np.float64), h, rstd


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None):
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, weight))
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    xhat, u = h * r, dy * w
    dx = r * (u - xhat * (u * xhat).mean(1, keepdims=True))
    if dresidual is not None:
        dx = dx + np.asarray(dresidual, dtype=np.float64)
    return dx, (dy * xhat).sum(0)
