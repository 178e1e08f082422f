"""Frequencies of rotary positions (host side, 64-bit).

:func:`rotary_inverse_frequencies` gives radians a position for the pairs of a head, plain or
scaled for long contexts; :func:`rotary_frequencies` turns any such list into what ``rotate`` and
``rotate_and_cache`` take: turns a position as 64-bit binary fractions, whose product with the
position modulo 2**64 is the fraction of a turn, exactly.
"""
from __future__ import annotations

import math
from fractions import Fraction
from typing import List, Optional, Sequence, Tuple

import torch

# 2**192 / (2 pi), from more digits of pi than the 64 bits that are asked for need
_UNIT = round(2 ** 191 / Fraction(3141592653589793238462643383279502884197, 10 ** 39))


def rotary_inverse_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
                               factor: float = 1.0, original_length: int = 8192, low: Optional[float] = None,
                               high: Optional[float] = None) -> Tuple[List[float], float]:
    """Radians a position for the pairs i < rotary_dim / 2, and the factor of rotated elements.

    Plain: w_i = base ** (-2 i / rotary_dim), factor 1. Scaled for contexts ``factor`` times
    ``original_length``, by ``scaling``:

    * ``"linear"``  every frequency is divided by ``factor`` (positions are interpolated);
    * ``"base"``    the base is multiplied by factor ** (d / (d - 2)), d = rotary_dim: the highest
      frequency stays, the lowest is divided by ``factor``;
    * ``"parts"``   by the turns that a pair makes over ``original_length`` tokens: above ``high`` (4
      unless given) it stays, below ``low`` (1) it is divided by ``factor``, in between the two are
      mixed in proportion to the turns;
    * ``"yarn"``    the same ends, mixed in proportion to the pair's index between the indexes (rounded
      outwards) at which a pair makes ``high`` and ``low`` turns (32 and 1 unless given), and rotated
      elements are multiplied by 1 + 0.1 ln(factor).
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim {rotary_dim} must be even and at least 2")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base {base} must be above 1")
    if scaling not in (None, "linear", "base", "parts", "yarn"):
        raise ValueError(f"scaling {scaling!r} is none of linear, base, parts, yarn")
    if scaling is not None and not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"factor {factor} must be at least 1")
    low = 1.0 if low is None else low
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if scaling in ("parts", "yarn") and not (0.0 < low < high and original_length > 0):
        raise ValueError(f"low {low} and high {high} must be positive and rise, original_length {original_length} positive")
    n = rotary_dim // 2
    if scaling == "base":
        if rotary_dim == 2:
            raise ValueError("scaling the base needs more than one pair")
        base *= factor ** (rotary_dim / (rotary_dim - 2))
    w = [base ** (-i / n) for i in range(n)]
    if scaling == "linear":
        w = [f / factor for f in w]
    if scaling == "parts":
        turns = [original_length * f / (2 * math.pi) for f in w]
        keep = [min(max((t - low) / (high - low), 0.0), 1.0) for t in turns]
        w = [f * k + f / factor * (1 - k) for f, k in zip(w, keep)]
    if scaling == "yarn":
        def index_of(turns: float) -> float:  # the pair that makes so many turns
            return n * math.log(original_length / (2 * math.pi * turns)) / math.log(base)
        first, last = max(math.floor(index_of(high)), 0), min(math.ceil(index_of(low)), rotary_dim - 1)
        keep = [1 - min(max((i - first) / max(last - first, 0.001), 0.0), 1.0) for i in range(n)]
        w = [f * k + f / factor * (1 - k) for f, k in zip(w, keep)]
        return w, 1.0 + 0.1 * math.log(factor)
    return w, 1.0


def rotary_frequencies(inverse: Sequence[float], device="cuda") -> torch.Tensor:
    """int64 [n]: the frequencies ``inverse`` (radians a position) as turns a position times 2**64."""
    turns = []
    for f in inverse:
        f = float(f)
        if not math.isfinite(f):
            raise ValueError("a frequency is not finite")
        n, d = f.as_integer_ratio()
        t = ((n * _UNIT * 2 // (d << 128)) + 1 >> 1) % 2 ** 64  # nearest
        turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    return torch.tensor(turns, dtype=torch.int64, device=device)
