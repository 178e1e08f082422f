"""Plain float64 CPU oracle of the 8-bit cache and of decode over a shared prefix.

TEST INFRASTRUCTURE ONLY. A row of d elements is kept as e4m3 codes c_i and one
biased exponent byte e; it stands for the values value(c_i) * 2**(e - 127). An
e4m3 code s.eeee.fff is (-1)^s * 2^(E - 7) * (1 + f / 8) for E = 1 .. 15, and
(-1)^s * 2^-6 * f / 8 for E = 0; E = 15 with f = 7 is NaN, so 448 is the largest
value. Everything here is written from that definition: the code nearest to a
value is looked up in the table of all values.
"""
from __future__ import annotations

import numpy as np

from .paged_attention import gather_kv, single_query_attention, to_float64


def _values() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        sign, E, f = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        if E == 15 and f == 7:
            v[c] = np.nan
        elif E == 0:
            v[c] = sign * 2.0 ** -6 * f / 8
        else:
            v[c] = sign * 2.0 ** (E - 7) * (1 + f / 8)
    return v


E4M3 = _values()
_POSITIVE = E4M3[:127]  # codes 0 .. 126 in rising order: 0 .. 448


def nearest_code(y: np.ndarray) -> np.ndarray:
    """The e4m3 code nearest to each y (|y| <= 448; ties to the even code); NaN for NaN."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(np.where(np.isnan(y), 0.0, y))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.signbit(y), code | 0x80, code)
    return np.where(np.isnan(y), 0x7F, code).astype(np.uint8)


def quantise_rows(x: np.ndarray):
    """(codes, exponent bytes) of rows x [..., d] (float64; not finite counts as NaN)."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    top = np.max(np.where(ok, np.abs(x), 0.0), axis=-1)
    e = np.full(top.shape, 1, dtype=np.int64)
    for b in range(1, 255):  # the smallest byte whose factor lets 448 reach the row
        e = np.where(top > 448.0 * 2.0 ** (b - 127), b + 1, e)
    e = np.minimum(e, 254)
    y = np.where(ok, x, np.nan) * np.exp2(127.0 - e)[..., None]
    return nearest_code(y), e.astype(np.uint8)


def pool_values(codes: np.ndarray, scales: np.ndarray, which: int) -> np.ndarray:
    """float64 values [NB, B, Hkv, d] of K (which = 0) or V (1); codes uint8."""
    f = np.exp2(scales[:, :, which, :].astype(np.float64) - 127.0)  # [NB, Hkv, B]
    return E4M3[codes] * f.transpose(0, 2, 1)[..., None]


def write_fp8(key, value, key_cache, value_cache, scales, slot_mapping, block_size: int, dtype: str):
    """Copies of the pool (uint8 codes, uint8 scales) with the rows written."""
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


def attend(query, K_pool, V_pool, block_tables, seq_lens, block_size: int, scale: float, dtype: str):
    """paged_decode over pools of float64 values."""
    S, Hq, _ = query.shape
    Hkv = K_pool.shape[2]
    G = Hq // Hkv
    out = np.zeros(query.shape)
    for s in range(S):
        L = int(seq_lens[s])
        K, V = (gather_kv(p, block_tables[s], L, block_size) for p in (K_pool, V_pool))
        q = to_float64(query[s], dtype)
        for h in range(Hkv):
            out[s, h * G:(h + 1) * G], _ = single_query_attention(q[h * G:(h + 1) * G], K[:, h], V[:, h],
                                                                  scale)
    return out


def shared_prefix_values(cache, block_tables, seq_lens, group_start, prefix_lens, block_size: int):
    """Per sequence, its rows with the group's prefix read through the first member's table.

    A sequence shorter than the prefix has its own rows alone.
    """
    rows = []
    for g in range(len(prefix_lens)):
        a, b, n = int(group_start[g]), int(group_start[g + 1]), int(prefix_lens[g])
        for s in range(a, b):
            L = int(seq_lens[s])
            mine = gather_kv(cache, block_tables[s], L, block_size)
            if L >= n > 0:
                mine = np.concatenate([gather_kv(cache, block_tables[a], n, block_size), mine[n:]])
            rows.append(mine)
    return rows


def shared_prefix_decode(query, key_cache, value_cache, block_tables, seq_lens, group_start, prefix_lens,
                         block_size: int, scale: float, dtype: str):
    """Decode attention with the prefix of every group read through its first member's table."""
    Hkv = key_cache.shape[2]
    G = query.shape[1] // Hkv
    out = np.zeros(query.shape)
    Ks = shared_prefix_values(key_cache, block_tables, seq_lens, group_start, prefix_lens, block_size)
    Vs = shared_prefix_values(value_cache, block_tables, seq_lens, group_start, prefix_lens, block_size)
    for s, (K, V) in enumerate(zip(Ks, Vs)):
        K, V, q = to_float64(K, dtype), to_float64(V, dtype), to_float64(query[s], dtype)
        for h in range(Hkv):
            out[s, h * G:(h + 1) * G], _ = single_query_attention(q[h * G:(h + 1) * G], K[:, h], V[:, h],
                                                                  scale)
    return out


def decode_bound(query, K_rows, V_rows, scale: float, weight_error: float) -> float:
    """How far an fp32 decode of these rows may be from the exact one.

    query [Hq, d] and rows [L, Hkv, d] in float64. With u = 2^-24:
    * a score is d products summed in fp32 (the tensor core may truncate: 2 u an
      addition) and a handful of fp32 multiplications, so it is off by at most
      (2 d + 8) u times the sum of the magnitudes of its terms; add the rounding
      of the exponent's argument, 4 u times the largest |score| in base 2;
    * a weight is then off by that, relative, plus 2^-20 for exp2 and rescaling,
      plus `weight_error` for its 16-bit parts;
    * sums of n weighted rows in fp32 are off by 2 n u, relative to the sum of
      magnitudes, and the result is a quotient of two such sums.
    Everything relative to the largest |V|, twice (numerator and denominator).
    """
    if K_rows.shape[0] == 0:
        return 0.0
    u = 2.0 ** -24
    Hkv, d = K_rows.shape[1:]
    G = query.shape[0] // Hkv
    worst = 0.0
    for h in range(Hkv):
        q = np.abs(query[h * G:(h + 1) * G])
        terms = float(np.max(q @ np.abs(K_rows[:, h]).T)) * abs(scale)
        ds = (2 * d + 8) * u * terms + 4 * u * terms * 1.4427
        rel = ds + 2.0 ** -20 + weight_error + 2 * K_rows.shape[0] * u
        worst = max(worst, 2 * rel * float(np.max(np.abs(V_rows[:, h]))))
    return worst
