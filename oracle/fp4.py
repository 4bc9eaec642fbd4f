"""Microscaled 4-bit floating point (MXFP4, and NVFP4 with a factor for each
row): quantisation, the values held, and the product, in plain NumPy.

Codes are integers decided by 32-bit floating point, so the decisions are
taken in np.float32 step by step; everything after them is fp64.
"""

from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def e2m1_codes(q: np.ndarray) -> np.ndarray:
    """The nearest E2M1 code of each value, ties to the even code, beyond 6
    to 6; bit 3 is the sign (of a zero too)."""
    a = np.abs(q.astype(np.float64))
    # distance to each magnitude; on a tie the even code wins
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    mag = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    mag = np.where(a >= 6.0, 7, mag)
    return (mag + 8 * np.signbit(q)).astype(np.uint8)


def e4m3_values() -> np.ndarray:
    """Values of the bytes 0..126 of unsigned e4m3 (127 is NaN)."""
    b = np.arange(127)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0**-9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))


def e4m3_codes(t: np.ndarray) -> np.ndarray:
    """The nearest e4m3 byte of values >= 0, ties to the even byte, beyond
    448 to 448."""
    v = e4m3_values()
    t = t.astype(np.float64)
    hi = np.clip(np.searchsorted(v, t, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.abs(t - v[lo]), np.abs(v[hi] - t)
    pick_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where(pick_lo, lo, hi).astype(np.uint8)


def quantize(X: np.ndarray, fmt: str):
    """X [M, K] float32 -> (codes uint8 [M, K], scale bytes uint8 [M, blocks],
    row factors float32 [M] or None)."""
    X = np.asarray(X, np.float32)
    M, K = X.shape
    B = BLOCK[fmt]
    nb = -(-K // B)
    x = np.zeros((M, nb * B), np.float32)
    x[:, :K] = X
    x = x.reshape(M, nb, B)
    top = np.abs(x).max(-1)  # NaN where the block has one
    with np.errstate(all="ignore"):
        if fmt == "mxfp4":
            bad = ~np.isfinite(top)
            E = (np.where(bad, 0, top).astype(np.float32).view(np.uint32) >> 23).astype(np.int64)
            s = np.maximum(E - 2, 0)
            q = np.ldexp(x.astype(np.float64), (127 - s)[..., None].astype(np.int32))
            codes = np.where(bad[..., None], 0, e2m1_codes(np.where(bad[..., None], 0, q)))
            return codes.reshape(M, -1)[:, :K].astype(np.uint8), np.where(bad, 255, s).astype(np.uint8), None
        row = top.max(-1)
        bad = ~np.isfinite(row)
        r = np.maximum(np.where(bad, 0, row).astype(np.float32) * np.float32(1 / 2688), np.float32(2.0**-100))
        inv_r = np.float32(1) / r
        t = (np.where(bad[:, None], 0, top).astype(np.float32) * np.float32(1 / 6)) * inv_r[:, None]
        sb = e4m3_codes(t)
        p = e4m3_values()[sb].astype(np.float32) * r[:, None]
        inv = np.where(p > 0, np.float32(1) / np.where(p > 0, p, np.float32(1)), np.float32(0)).astype(np.float32)
        live = (p > 0)[..., None] & ~bad[:, None, None]
        q = np.where(live, x, np.float32(0)) * inv[..., None]
        codes = np.where(live, e2m1_codes(q), 0)
        return (codes.reshape(M, -1)[:, :K].astype(np.uint8), np.where(bad[:, None], 0, sb).astype(np.uint8),
                np.where(bad, np.float32(np.nan), r).astype(np.float32))


def scale_values(scales: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "mxfp4":
        return np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int32) - 127))
    v = np.append(e4m3_values(), np.nan)
    return v[scales & 127]


def dequantize(codes, scales, row_scale, fmt: str) -> np.ndarray:
    """The values held, fp64 [M, K]."""
    K = codes.shape[1]
    v = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    v = v * np.repeat(scale_values(scales, fmt), BLOCK[fmt], axis=1)[:, :K]
    return v if row_scale is None else v * row_scale.astype(np.float64)[:, None]


def pack(codes: np.ndarray, scales: np.ndarray, fmt: str):
    """Codes and scales in the library's bytes: two codes in a byte, the even
    column low; rows padded with zeros to whole 16-byte units."""
    M, K = codes.shape
    c = np.zeros((M, -(-K // 32) * 32), np.uint8)
    c[:, :K] = codes
    s = np.zeros((M, -(-scales.shape[1] // 16) * 16), np.uint8)
    s[:, :scales.shape[1]] = scales
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def linear(x64: np.ndarray, w64: np.ndarray):
    """(Y, sum of |terms|) of Y = x W^T in fp64."""
    return x64 @ w64.T, np.abs(x64) @ np.abs(w64).T
