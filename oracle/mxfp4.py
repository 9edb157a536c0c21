"""MXFP4 in numpy and 64 bits: blocks of 32 along a row, E2M1 codes, E8M0 scales.

The definition of include/fs4.h's MXFP4 section, element by element; test infrastructure only.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
COLUMN_SEED = 0xD1B54A32D192ED03


def _up(v: int, a: int) -> int:
    return (v + a - 1) // a * a


def draws(rows: int, cols: int, seed: int) -> np.ndarray:
    """The 16-bit draw of every element of a rows x cols view, as Python integers give it."""
    mask = (1 << 64) - 1
    groups = (cols + 3) // 4
    out = np.zeros((rows, 4 * groups), np.int64)
    for i in range(rows * groups):
        z = (seed + (i + 1) * 0x9E3779B97F4A7C15) & mask
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        z ^= z >> 31
        for j in range(4):
            out[i // groups, 4 * (i % groups) + j] = (z >> (16 * j)) & 0xFFFF
    return out[:, :cols]


def quantize(x: np.ndarray, rule: str = "floor", seed: int | None = None):
    """(codes [rows, K] as integers 0..15, scale bytes [rows, ceil(K/32)]) of the row view of x."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, (cols + 31) // 32), np.uint8)
    f = None if seed is None else draws(rows, cols, seed)
    for b in range(scales.shape[1]):
        s = slice(32 * b, min(32 * b + 32, cols))
        v = x[:, s]
        bad = ~np.isfinite(v).all(1)
        amax = np.where(bad, 1.0, np.abs(np.where(np.isfinite(v), v, 0)).max(1))
        m, e = np.frexp(np.where(amax > 0, amax, 1.0))            # amax = m 2^e, m in [1/2, 1)
        e = e - 3 + (m > 0.75) * (rule == "ceil")
        e = np.where(amax > 0, np.maximum(e, -127), -127)
        with np.errstate(invalid="ignore"):
            q = np.abs(v) * 2.0 ** -e[:, None].astype(np.float64)
        q = np.where(bad[:, None], 0.0, q)
        lo = np.searchsorted(GRID, q, side="right") - 1
        hi = np.minimum(lo + 1, 7)
        gap = np.where(hi > lo, GRID[hi] - GRID[lo], 1.0)
        frac = np.where(hi > lo, (q - GRID[lo]) / gap, 0.0)
        if f is None:
            up = (frac > 0.5) | ((frac == 0.5) & (lo % 2 == 1))
        else:
            up = (f[:, s] + 0.5) / 65536 <= frac
        c = np.where(up, hi, lo) + 8 * np.signbit(v)
        codes[:, s] = np.where(bad[:, None], 0, c)
        scales[:, b] = np.where(bad, 255, e + 127)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    e = np.repeat(scales.astype(np.float64) - 127, 32, axis=1)[:, :codes.shape[1]]
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7] * 2.0 ** e
    return np.where(np.repeat(scales == 255, 32, axis=1)[:, :codes.shape[1]], np.nan, v)


def pack_plain(codes: np.ndarray, scales: np.ndarray):
    rows, cols = codes.shape
    c = np.zeros((rows, _up(cols, 2)), np.uint8)
    c[:, :cols] = codes
    return c[:, 0::2] | (c[:, 1::2] << 4), scales


def pack_tiled(codes: np.ndarray, scales: np.ndarray):
    """The TILED bytes, placed one element at a time by the header's offsets."""
    rows, cols = codes.shape
    rp, kp = _up(rows, 128), _up(cols, 256)
    cb, sb = np.zeros(rp * kp // 2, np.uint8), np.zeros(rp * kp // 32, np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
    at = (r // 128 * (kp // 256) + c // 256) * 16384 + 128 * (r % 128) + 16 * ((c % 256 // 32) ^ (r % 8)) + c % 32 // 2
    np.add.at(cb, at.ravel(), (codes.astype(np.uint32) << (4 * (c % 2))).ravel().astype(np.uint8))
    r, b = np.meshgrid(np.arange(rows), np.arange(scales.shape[1]), indexing="ij")
    at = (r // 128 * (kp // 128) + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    sb[at.ravel()] = scales.ravel()
    return cb, sb
