"""CPU restatements for the 8-bit cache and the eviction of COLD tokens.  TEST INFRASTRUCTURE ONLY.

Quantising rounds each exact quotient once (a float64 quotient of float32 values is halfway between two
codes only if the exact one is: codes have 4 significant bits), so codes and scales can be compared
bit for bit; attention over the cache is that of
``oracle.attention`` on the dequantised values in float64.
"""

from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

BLOCK = 64
E4M3_MAX = np.float32(448.0)
AMAX_MIN = np.float32(2.0 ** -96)


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes (sign, 4 exponent bits of bias 7, 3 mantissa bits;
    0x7f and 0xff are NaN, there is no infinity)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if (e, m) == (15, 7) else x
        out[c] = -out[c] if c & 128 else out[c]
    return out


_VALUES = e4m3_values()


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest code of values held in float64: ties to the even code, saturated at +-448, NaN 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    grid = _VALUES[:127]  # the non-negative finite values, ascending
    with np.errstate(invalid="ignore"):
        hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    below = a - grid[lo]
    above = grid[hi] - a
    code = np.where(below < above, lo, np.where(below > above, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a >= 448.0, 126, code).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code).astype(np.uint8)


def quantise(x: np.ndarray, block: int) -> Tuple[np.ndarray, np.ndarray]:
    """Codes [n, n_kv, d] (uint8) and scales [n, n_kv] (float32) of float32 rows x [n, n_kv, d]:
    one scale for each `block` consecutive tokens and head (BLOCK in a slab, 1 for COLD tokens)."""
    x = np.asarray(x, dtype=np.float32)
    a = np.abs(x)
    amax = np.where(np.isfinite(a), a, np.float32(0)).max(axis=2).astype(np.float32)
    for t in range(0, x.shape[0], block):
        amax[t:t + block] = amax[t:t + block].max(axis=0)
    amax = np.maximum(amax, AMAX_MIN)
    with np.errstate(invalid="ignore", over="ignore"):
        codes = e4m3_codes(x.astype(np.float64) * 448.0 / amax.astype(np.float64)[..., None])
    return codes, amax / E4M3_MAX


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of codes [n, n_kv, d] with scales [n, n_kv]."""
    return _VALUES[codes] * scales.astype(np.float64)[..., None]


def through_cache(x: np.ndarray, block: int) -> np.ndarray:
    """The values a cache holds after rows x were written to it."""
    return values(*quantise(x, block))


def evict(seq_len: Sequence[int], n_evict: Sequence[int], keep_first: Optional[Sequence[int]], keep_last: int,
          table: np.ndarray, weight: np.ndarray) -> Tuple[np.ndarray, np.ndarray, List[int], np.ndarray]:
    """(table, weight, new lengths, slots that left) after the lightest tokens left each row."""
    table, weight = table.copy(), weight.copy()
    gone: List[int] = []
    lens = []
    for b, (n, e) in enumerate(zip(seq_len, n_evict)):
        first = keep_first[b] if keep_first is not None else 0
        places = range(first, max(first, n - keep_last))
        order = sorted(places, key=lambda t: (np.isnan(weight[b, t]), 0.0 if np.isnan(weight[b, t]) else weight[b, t], t))
        out = set(order[:e])
        stay = [t for t in range(n) if t not in out]
        gone += [int(table[b, t]) for t in sorted(out)]
        table[b, :n - e], weight[b, :n - e] = table[b, stay], weight[b, stay]
        weight[b, n - e:n] = 0.0
        lens.append(n - e)
    return table, weight, lens, np.array(gone, dtype=np.int32)
