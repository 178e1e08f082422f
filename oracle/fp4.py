"""Plain float64 CPU oracle of the 4-bit cache.

TEST INFRASTRUCTURE ONLY. A row of d elements is kept as e2m1 codes, two a byte (the
element with the even index in bits 0-3), and one biased exponent byte e for every 32
elements; element i stands for value(code_i) * 2**(e - 127), with a factor of 0 for
e = 0 and of infinity for e = 255. An e2m1 code s.ee.f is (-1)^s * 2^(ee - 1) * (1 + f / 2)
for ee = 1 .. 3, and (-1)^s * f / 2 for ee = 0. Everything here is written from that
definition: the code nearest to a value is looked up in the table of all values.
"""
from __future__ import annotations

import numpy as np

from .paged_attention import to_float64

GROUP = 32


def _values() -> np.ndarray:
    v = np.empty(16)
    for c in range(16):
        sign, ee, f = (-1.0 if c & 8 else 1.0), (c >> 1) & 3, c & 1
        v[c] = sign * (f / 2 if ee == 0 else 2.0 ** (ee - 1) * (1 + f / 2))
    return v


E2M1 = _values()
_POSITIVE = E2M1[:8]  # 0 .. 6 in rising order


def nearest_code(y: np.ndarray) -> np.ndarray:
    """The e2m1 code nearest to each finite y (ties to the even code, above 6 the code of 6)."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.abs(a - _POSITIVE[lo]), np.abs(_POSITIVE[hi] - a)
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.signbit(y), code | 8, code).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def factors(scales: np.ndarray) -> np.ndarray:
    f = np.exp2(scales.astype(np.float64) - 127.0)
    return np.where(scales == 0, 0.0, np.where(scales == 255, np.inf, f))


def quantise_rows(x: np.ndarray):
    """(packed codes [.., d / 2], exponent bytes [.., d / 32]) of rows x [.., d] (float64)."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lost = ~np.all(np.isfinite(g), axis=-1)
    g = np.where(lost[..., None], 0.0, g)
    top = np.max(np.abs(g), axis=-1)
    e = np.full(top.shape, 1, dtype=np.int64)
    for b in range(1, 252):  # the smallest byte of whose factor 7 reaches the group
        e = np.where(top > 7.0 * 2.0 ** (b - 127), b + 1, e)
    codes = nearest_code(g * np.exp2(127.0 - e)[..., None])
    codes = np.where(lost[..., None], 0, codes).astype(np.uint8)
    e = np.where(lost, 255, np.where(top > 0, e, 0))
    return pack(codes.reshape(x.shape)), e.astype(np.uint8)


def row_values(packed: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values [.., d] of packed codes [.., d / 2] and bytes [.., d / 32]."""
    v = E2M1[unpack(packed)]
    with np.errstate(invalid="ignore"):
        return (v.reshape(*v.shape[:-1], -1, GROUP) * factors(scales)[..., None]).reshape(v.shape)


def pool_values(packed: np.ndarray, scales: np.ndarray, which: int) -> np.ndarray:
    """float64 values [NB, B, Hkv, d] of K (which = 0) or V (1)."""
    return row_values(packed, scales[:, :, which].transpose(0, 2, 1, 3))


def write_fp4(key, value, key_cache, value_cache, scales, slot_mapping, block_size: int, dtype: str):
    """Copies of the pool (uint8) with the rows written."""
    kc, vc, sc = key_cache.copy(), value_cache.copy(), scales.copy()
    for which, (rows, cache) in enumerate(((key, kc), (value, vc))):
        codes, e = quantise_rows(to_float64(rows, dtype))
        for i, slot in enumerate(np.asarray(slot_mapping).tolist()):
            if slot < 0:
                continue
            blk, off = divmod(int(slot), block_size)
            cache[blk, off] = codes[i]
            sc[blk, :, which, off] = e[i]
    return kc, vc, sc
