"""CPU restatement of the 4-bit cache.  TEST INFRASTRUCTURE ONLY.

Quantising rounds each exact quotient once.  The float64 quotients below are those: a quotient of float32
values by 6 or by an e4m3 value, times a power of two, is halfway between two e4m3 or e2m1 values only if the
exact one is.  A value has 2 + 4 significant bits over a power of two, so float64 holds it exactly."""

from __future__ import annotations

from typing import Tuple

import numpy as np

from . import kv8 as K8

BLOCK = 64
GROUP = 16
EXP_MIN, EXP_MAX = -100, 116
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(n_kv: int, d: int) -> int:
    up = lambda x: (x + 15) // 16 * 16
    return up(up(n_kv * d // 2 + n_kv * d // GROUP) + n_kv)


def e2m1_codes(x: np.ndarray) -> np.ndarray:
    """Nearest code of float64 values: ties to the even code, saturated at +-6 (a NaN: any)."""
    a = np.where(np.isnan(x), 0.0, np.abs(x))
    hi = np.clip(np.searchsorted(E2M1, a), 1, 7)
    below, above = a - E2M1[hi - 1], E2M1[hi] - a
    code = np.where(below < above, hi - 1, np.where(below > above, hi, np.where(hi % 2 == 0, hi, hi - 1)))
    return np.where(np.signbit(x), code | 8, code).astype(np.uint8)


def quantise(x: np.ndarray, block: int) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """Codes [n, n_kv, d], scale bytes [n, n_kv, d / 16] and exponent bytes [n, n_kv] of float32 rows
    [n, n_kv, d]: one exponent for each `block` consecutive tokens and head (BLOCK in a slab, 1 for COLD tokens)."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    n, n_kv, d = x.shape
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = a.max(axis=2)
    for t in range(0, n, block):
        amax[t:t + block] = amax[t:t + block].max(axis=0)
    m, e = np.frexp(amax / 2688.0)
    e = np.where(m == 0.5, e - 1, e)
    e = np.clip(np.where(m == 0.0, EXP_MIN, e), EXP_MIN, EXP_MAX)
    unit = np.ldexp(1.0, e)[..., None]
    groups = x.reshape(n, n_kv, d // GROUP, GROUP)
    top = a.reshape(groups.shape).max(axis=3)
    scale = np.maximum(K8.e4m3_codes(top / (6.0 * unit)), 1).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        codes = e2m1_codes(groups / (K8.e4m3_values()[scale] * unit)[..., None]).reshape(n, n_kv, d)
    scale[np.isnan(groups).any(axis=3)] = 0x7F
    return codes, scale, (e + 127).astype(np.uint8)


def values(codes: np.ndarray, scale: np.ndarray, e: np.ndarray) -> np.ndarray:
    """float64 values of what quantise returns."""
    n, n_kv, d = codes.shape
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    v = v.reshape(n, n_kv, d // GROUP, GROUP) * (K8.e4m3_values()[scale] * np.ldexp(1.0, e.astype(np.int64) - 127)[..., None])[..., None]
    return v.reshape(n, n_kv, d)


def through_cache(x: np.ndarray, block: int) -> np.ndarray:
    """The values a cache holds after rows x were written to it."""
    return values(*quantise(x, block))


def units(x: np.ndarray, block: int) -> np.ndarray:
    """2^e of each row and head [n, n_kv]."""
    return np.ldexp(1.0, quantise(x, block)[2].astype(np.int64) - 127)


def unpack_rows(rows: np.ndarray, n_kv: int, d: int) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(codes, scale bytes, exponent bytes) of packed rows [n, row_bytes]."""
    n, a, b = rows.shape[0], n_kv * d // 2, n_kv * d // 2 + n_kv * d // GROUP
    codes = np.stack([rows[:, :a] & 15, rows[:, :a] >> 4], axis=2).reshape(n, n_kv, d)
    at = (b + 15) // 16 * 16
    return codes, rows[:, a:b].reshape(n, n_kv, d // GROUP), rows[:, at:at + n_kv]


def padding(n_kv: int, d: int) -> np.ndarray:
    """Which bytes of a row hold nothing."""
    b = n_kv * d // 2 + n_kv * d // GROUP
    at = (b + 15) // 16 * 16
    out = np.ones(row_bytes(n_kv, d), dtype=bool)
    out[:b] = False
    out[at:at + n_kv] = False
    return out
