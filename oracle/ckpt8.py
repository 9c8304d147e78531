"""The 8-bit checkpoint format, from its definition, in float64.

Test infrastructure only (see the package header). Per 32 neighbours of a row: the smallest e >= -126
under which the largest finite magnitude times 2^-e is at most 448 (E4M3) or below 127.5 (INT8); scale
byte e + 127; code = the nearest code value to x 2^-e, ties to the even code; not finite -> NaN code.

Pins: tests/test_oracle_around.py."""

from __future__ import annotations

import numpy as np

GROUP = 32


def e4m3_values() -> np.ndarray:
    """Value of each of the 256 E4M3 codes."""
    out = np.zeros(256)
    for c in range(256):
        ex, man = (c >> 3) & 15, c & 7
        v = (1 + man / 8) * 2.0 ** (ex - 7) if ex else man / 8 * 2.0 ** -6
        if ex == 15 and man == 7:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


def _code_e4m3(v: float) -> int:
    table = e4m3_values()[:127]
    a = abs(v)
    hi = int(np.searchsorted(table, a))
    if hi == 0:
        c = 0
    elif hi == 127:
        c = 126
    else:
        lo, up = a - table[hi - 1], table[hi] - a
        c = hi - 1 if lo < up or (lo == up and (hi - 1) % 2 == 0) else hi
    return c | (128 if np.signbit(v) else 0)


def _fits(amax: float, e: int, fmt: str) -> bool:
    u = amax * 2.0 ** -e
    return u <= 448.0 if fmt == "e4m3" else u < 127.5


def save(x, fmt: str):
    """(codes uint8 [rows, width], scale bytes uint8 [rows, ceil(width / 32)])."""
    x = np.asarray(x, dtype=np.float64)
    rows, width = x.shape
    n = -(-width // GROUP)
    codes = np.zeros((rows, width), dtype=np.uint8)
    scales = np.zeros((rows, n), dtype=np.uint8)
    for r in range(rows):
        for g in range(n):
            part = x[r, g * GROUP:(g + 1) * GROUP]
            fin = np.abs(part[np.isfinite(part)])
            amax = float(fin.max()) if fin.size else 0.0
            e = -126
            if amax > 0:
                e = max(-126, int(np.floor(np.log2(amax))) - 10)
                while not _fits(amax, e, fmt):
                    e += 1
            scales[r, g] = e + 127
            for j, v in enumerate(part):
                if not np.isfinite(v):
                    c = 0x7F if fmt == "e4m3" else 0x80
                elif fmt == "e4m3":
                    c = _code_e4m3(v * 2.0 ** -e)
                else:
                    c = int(np.rint(v * 2.0 ** -e)) & 0xFF
                codes[r, g * GROUP + j] = c
    return codes, scales


def load(codes, scales, fmt: str, limit: float = np.inf) -> np.ndarray:
    """Values in float64; finite ones at most `limit` in magnitude."""
    codes = np.asarray(codes)
    if fmt == "e4m3":
        v = e4m3_values()[codes]
    else:
        v = codes.astype(np.int8).astype(np.float64)
        v[codes == 0x80] = np.nan
    s = 2.0 ** (np.asarray(scales).astype(np.float64) - 127)
    v = v * np.repeat(s, GROUP, axis=1)[:, :codes.shape[1]]
    return np.clip(v, -limit, limit)
