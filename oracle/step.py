"""Plain CPU oracle of what stands in front of a step's attention: tables and slots of new
tokens, norms of heads, rotation by position.

TEST INFRASTRUCTURE ONLY. Written from the definitions: the rotation in float64 with the
fraction of a turn in whole numbers, the tables one token after the other.
"""
from __future__ import annotations

import numpy as np

NO_BLOCKS, OUT_OF_RANGE = 1, 2


def angles(positions, frequencies) -> np.ndarray:
    """Radians [T, n]: 2 pi times the fraction of position * frequency / 2**64 turns, in [-pi, pi)."""
    out = np.empty((len(positions), len(frequencies)))
    for t, p in enumerate(positions):
        for i, f in enumerate(frequencies):
            x = int(p) * int(f) % 2 ** 64
            out[t, i] = 2 * np.pi * ((x - 2 ** 64 if x >= 2 ** 63 else x) / 2.0 ** 64)
    return out


def pairs(n: int, interleaved: bool):
    i = np.arange(n)
    return (2 * i, 2 * i + 1) if interleaved else (i, n + i)


def rotate(x, angle, interleaved=False, factor=1.0, weight=None, eps=1e-6) -> np.ndarray:
    """Rows x [T, H, d] (float64) rotated by angle [T, n], behind the norm where there are weights."""
    y = np.array(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        if weight is not None:
            y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * weight
        ia, ib = pairs(angle.shape[1], interleaved)
        a, b = y[..., ia].copy(), y[..., ib].copy()
        c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def rotate_bound(x, n, interleaved, factor, weight, eps, ref, dtype) -> np.ndarray:
    """How far a fp32 computation, rounded once to dtype, may be from `ref` (finite results).

    The fraction of a turn is rounded to fp32 (2^-25 of half a turn, pi 2^-25 in the angle), cosine and
    sine are good to 2 units in the last place (2^-23), the products and their sum add 3 2^-24: under 2^-21
    of |a| + |b|. The norm: a sum of d squares in steps of at most 19 roundings, a reciprocal root good to
    2 units, three products: under 2^-19. Then half a step of the type, 2^-25 where fp16 has no smaller one.
    """
    y = np.abs(rotate(x, np.zeros((x.shape[0], n)), interleaved, 1.0, weight, eps))
    size = y.copy()
    ia, ib = pairs(n, interleaved)
    size[..., ia] = size[..., ib] = (y[..., ia] + y[..., ib]) * abs(factor)
    own = 2.0 ** -21 + (2.0 ** -19 if weight is not None else 0.0)
    half = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    return size * own + np.abs(ref) * half * (1 + own) + (2.0 ** -25 if dtype == "fp16" else 2.0 ** -134)


def append_tokens(tables, lens, starts, free, num_free, rows, block_size, num_blocks):
    """(tables, new lengths, new height, slots, positions, status, rejected) of one step."""
    tables, S = np.array(tables), len(lens)
    MB = tables.shape[1]
    slots, positions = np.full(rows, -1, np.int64), np.zeros(rows, np.int64)
    new = [int(starts[s + 1]) - int(starts[s]) for s in range(S)]
    held = lambda n: -(-n // block_size)  # noqa: E731
    status = 0
    if not 0 <= num_free <= len(free) or any(
            lens[s] < 0 or new[s] < 0 or starts[s] < 0 or starts[s + 1] > rows
            or int(lens[s]) + new[s] > MB * block_size for s in range(S)):
        status = OUT_OF_RANGE
    elif sum(held(int(lens[s]) + new[s]) - held(int(lens[s])) for s in range(S)) > num_free:
        status = NO_BLOCKS
    if status:
        return tables, np.array(lens), num_free, slots, positions, status, 0
    stack, rejected = list(free[:num_free]), 0
    for s in range(S):
        for i in range(new[s]):
            p = int(lens[s]) + i
            if p % block_size == 0:
                tables[s, p // block_size] = stack.pop()
            block, row = int(tables[s, p // block_size]), int(starts[s]) + i
            positions[row] = p
            if 0 <= block < num_blocks:
                slots[row] = block * block_size + p % block_size
            else:
                rejected += 1
    return tables, np.array([int(lens[s]) + new[s] for s in range(S)]), len(stack), slots, positions, 0, rejected
