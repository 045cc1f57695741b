"""Plain forms of the 8-bit cache in numpy, for the tests: codes and their values, the scale
rule, and a page's append. Values are exact in float64; quotients are taken in float32, as
the rule says, and rounded by a search over the table of code values."""
from __future__ import annotations

import numpy as np

TINY = np.float32(2.0 ** -126)


def e4m3_values() -> np.ndarray:
    """Value of every E4M3 code (1 sign, 4 exponent bits biased by 7, 3 mantissa bits; 0x7F and 0xFF NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e.astype(float) - 7))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >> 7, -mag, mag)


E4M3 = e4m3_values()


def decode(codes: np.ndarray, kind: str) -> np.ndarray:
    """float64 values of uint8-stored codes."""
    codes = np.ascontiguousarray(codes)
    if kind == "int8":
        return codes.view(np.int8).astype(np.float64)
    return E4M3[codes.view(np.uint8)]


def round_half_even(y: np.ndarray, kind: str) -> np.ndarray:
    """uint8-stored codes nearest to y, ties to even, cut to the largest magnitude; NaN as the rule says."""
    y = np.asarray(y, dtype=np.float64)
    nan = np.isnan(y)
    z = np.where(nan, 0.0, y)
    if kind == "int8":
        return np.rint(np.clip(z, -127, 127)).astype(np.int8).view(np.uint8)
    pos = E4M3[:127]                               # ascending, 0 .. 448
    a = np.minimum(np.abs(z), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    below, above = a - pos[lo], pos[hi] - a
    pick = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    out = pick.astype(np.uint8) | (np.signbit(z).astype(np.uint8) << 7)
    return np.where(nan, np.uint8(0x7F), out).astype(np.uint8)


def scale_for(a, kind: str) -> np.float32:
    a = np.float32(a)
    if a == 0:
        return np.float32(0)
    if kind == "int8":
        return max(np.float32(a / np.float32(127)), TINY)
    e = -126
    while np.float64(a) / 448.0 > 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def append_page(codes, scale, kept: int, new: np.ndarray, kind: str):
    """One page after ``new`` (float32 [n][d]) follows its first ``kept`` tokens: (codes, scale)."""
    codes = codes.copy()
    new = np.asarray(new, dtype=np.float32)
    fin = np.abs(new[np.isfinite(new)])
    need = scale_for(fin.max() if fin.size else 0.0, kind)
    to = need if kept == 0 else max(np.float32(scale), need)
    if kept and to > scale:
        old = decode(codes[:kept], kind).astype(np.float32) * np.float32(scale)
        codes[:kept] = round_half_even(old / to, kind)
    if to > 0:
        with np.errstate(over="ignore", invalid="ignore"):
            codes[kept:kept + len(new)] = round_half_even(new / to, kind)
    else:
        codes[kept:kept + len(new)] = 0
    return codes, to


def same_codes(a: np.ndarray, b: np.ndarray, kind: str) -> bool:
    """Equal codes (any NaN code equals any other)."""
    if kind == "int8":
        return np.array_equal(a.view(np.uint8), b.view(np.uint8))
    x, y = a.view(np.uint8), b.view(np.uint8)
    return bool(np.all((x == y) | (((x & 127) == 127) & ((y & 127) == 127))))


def dequant_unit(pool: np.ndarray, scale: np.ndarray, row: np.ndarray, T: int, kind: str) -> np.ndarray:
    """Tokens [0, T) of a unit in float64. pool: uint8 [n_pages][16][d]; row: its page table."""
    pages = row[:-(-T // 16)]
    return (decode(pool[pages], kind) * scale[pages].astype(np.float64)[:, None, None]).reshape(-1, pool.shape[2])[:T]
