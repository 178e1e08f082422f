"""Rotation, norms and slots without a GPU: frequencies against their formulas, the oracle
against what defines it, and the refusals of the entry points and of their Python binding
(nothing here launches a kernel)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_305_gb300 as pa
from oracle import step
from paged_kv_cache_305_gb300 import build as pbuild


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load_library()


# ------------------------------------------------------------ frequencies --
def test_plain_frequencies():
    w, f = pa.rotary_inverse_frequencies(8, 10000.0)
    assert f == 1.0 and np.allclose(w, [1.0, 0.1, 0.01, 0.001], rtol=1e-15)


def test_linear_and_base_scaling():
    w, _ = pa.rotary_inverse_frequencies(128, 500000.0)
    lin, _ = pa.rotary_inverse_frequencies(128, 500000.0, "linear", 4.0)
    assert np.allclose(np.array(lin) * 4, w, rtol=1e-15)
    b, _ = pa.rotary_inverse_frequencies(128, 500000.0, "base", 8.0)
    assert b[0] == 1.0 and math.isclose(b[-1], w[-1] / 8.0, rel_tol=1e-12)
    assert all(x >= y for x, y in zip(w, b))


@pytest.mark.parametrize("scaling,low,high", [("parts", 1.0, 4.0), ("yarn", 1.0, 32.0)])
def test_scaling_by_parts(scaling, low, high):
    w, _ = pa.rotary_inverse_frequencies(128, 500000.0)
    s, f = pa.rotary_inverse_frequencies(128, 500000.0, scaling, 8.0, 8192, low, high)
    assert f == (1.0 if scaling == "parts" else 1.0 + 0.1 * math.log(8.0))
    turns = 8192 * np.array(w) / (2 * np.pi)
    ratio = np.array(w) / np.array(s)
    assert np.allclose(ratio[turns > high * 1.3], 1.0) and np.allclose(ratio[turns < low / 1.3], 8.0)
    assert np.all(np.diff(ratio) > -1e-12) and ratio.max() <= 8.0 + 1e-9 and ratio.min() >= 1 - 1e-12
    same, f = pa.rotary_inverse_frequencies(128, 500000.0, scaling, 1.0, 8192, low, high)
    assert np.allclose(same, w, rtol=1e-14) and f == 1.0


def test_defaults_of_scaling_by_parts():
    # the usual ones, against plain restatements: "parts" mixes by the turns between 1 and 4, "yarn" by the
    # index between those that make 32 and 1
    d, base, s, L = 128, 10000.0, 4.0, 4096
    w = base ** (-np.arange(64) / 64)
    keep = np.clip((L * w / (2 * math.pi) - 1.0) / 3.0, 0, 1)
    got, f = pa.rotary_inverse_frequencies(d, base, "parts", s, L)
    assert f == 1.0 and np.allclose(got, w * keep + w / s * (1 - keep), rtol=1e-12)
    first, last = (64 * math.log(L / (2 * math.pi * t)) / math.log(base) for t in (32, 1))
    first, last = math.floor(first), math.ceil(last)
    keep = 1 - np.clip((np.arange(64) - first) / (last - first), 0, 1)
    got, f = pa.rotary_inverse_frequencies(d, base, "yarn", s, L)
    assert f == 1.0 + 0.1 * math.log(s) and np.allclose(got, w * keep + w / s * (1 - keep), rtol=1e-12)
    # either may be given alone
    assert pa.rotary_inverse_frequencies(d, base, "yarn", s, L, low=2.0) == \
        pa.rotary_inverse_frequencies(d, base, "yarn", s, L, 2.0, 32.0)
    assert pa.rotary_inverse_frequencies(d, base, "parts", s, L, high=8.0) == \
        pa.rotary_inverse_frequencies(d, base, "parts", s, L, 1.0, 8.0)


def test_frequencies_are_turns_in_64_bits():
    w, _ = pa.rotary_inverse_frequencies(128, 10000.0, "linear", 3.7)
    t = pa.rotary_frequencies(w + [0.0, -w[3], 2 * math.pi + 1e-3, 3.5], device="cpu")
    assert t.dtype == torch.int64
    got = [Fraction(int(x) % 2 ** 64, 2 ** 64) for x in t]
    for f, x in zip(w, got):
        # half a unit of 2^-64, and pi to more digits than that
        assert abs(x - Fraction(f) / (2 * Fraction(math.pi))) <= Fraction(1, 2 ** 65) + Fraction(f) * Fraction(1, 2 ** 53)
    assert got[64] == 0 and got[65] == 1 - got[3]
    assert math.isclose(float(got[66]), (2 * math.pi + 1e-3) / (2 * math.pi) - 1, rel_tol=1e-9)
    assert math.isclose(float(got[67]), 3.5 / (2 * math.pi), rel_tol=1e-15)


@pytest.mark.parametrize("args", [(7,), (0,), (16, 1.0), (16, math.inf), (16, 1e4, "cubic"), (16, 1e4, "linear", 0.5),
                                  (16, 1e4, "linear", math.nan), (16, 1e4, "parts", 2.0, 8192, 4.0, 4.0),
                                  (16, 1e4, "yarn", 2.0, 0), (2, 1e4, "base", 2.0)])
def test_frequency_refusals(args):
    with pytest.raises(ValueError):
        pa.rotary_inverse_frequencies(*args)


def test_frequency_refuses_what_is_not_finite():
    with pytest.raises(ValueError):
        pa.rotary_frequencies([1.0, math.nan], device="cpu")


# ----------------------------------------------------------------- oracle --
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_one(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    f = [int(v) for v in rng.integers(0, 2 ** 62, 16)]
    p = rng.integers(0, 10 ** 6, 5)
    y = step.rotate(x, step.angles(p, f), interleaved)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose(step.rotate(y, -step.angles(p, f), interleaved), x)
    # scores depend on the distance alone
    q, k = x[:1], x[1:2]
    dots = []
    for a, b in ((3, 10), (103, 110), (900007, 900014)):
        qa, kb = (step.rotate(v, step.angles([t], f), interleaved) for v, t in ((q, a), (k, b)))
        dots.append(np.sum(qa * kb, -1))
    assert np.allclose(dots[0], dots[1]) and np.allclose(dots[0], dots[2])


def test_oracle_append_agrees_with_the_block_manager(lib):
    rng = np.random.default_rng(1)
    bm = pa.BlockManager(64, 4, 16)
    ids = [bm.new_sequence() for _ in range(3)]
    tables, lens = np.zeros((3, 16), np.int32), np.zeros(3, np.int64)
    free = None
    for _ in range(6):
        new = rng.integers(0, 6, 3)
        starts = np.concatenate([[0], np.cumsum(new)])
        before = bm.num_free_blocks()
        slots, _ = bm.append([(i, int(n)) for i, n in zip(ids, new)])
        want, held = bm.block_tables(ids)
        # the same blocks through a stack that has them in the order in which they were taken
        taken = [int(want[s, j]) for s in range(3) for j in range(-(-int(lens[s]) // 4), -(-int(held[s]) // 4))]
        free = [99] * 2 + taken[::-1]
        tables, lens, left, got, pos, status, bad = step.append_tokens(tables, lens, starts, free, len(free),
                                                                      int(starts[-1]), 4, 64)
        assert status == 0 and bad == 0 and left == 2 and before - bm.num_free_blocks() == len(taken)
        assert np.array_equal(got, slots) and np.array_equal(lens, held)
        for s in range(3):
            assert np.array_equal(tables[s, :-(-int(lens[s]) // 4)], want[s, :-(-int(lens[s]) // 4)])
    bm.close()


# --------------------------------------------------------------- refusals --
OK, INVALID, UNSUPPORTED = 0, -1, -2


def _rotate(lib, T=2, Hq=4, Hkv=2, d=64, rot=64, inter=0, factor=1.0, eps=1e-6, qo=16, ko=16, q=16, k=16, pos=16,
            freq=16, qw=0, kw=0, qos=256, kos=128, qs=256, ks=128, dtype=1):
    return lib.pa_rotate(qo, ko, q, k, pos, freq, qw, kw, T, Hq, Hkv, d, rot, inter, factor, eps, qos, kos, qs, ks,
                         dtype, None)


def _cached(lib, T=2, Hq=4, Hkv=2, d=64, B=16, NB=4, rot=64, inter=0, factor=1.0, eps=1e-6, qo=16, q=16, k=16, v=16,
            kc=16, vc=16, slots=16, pos=16, freq=16, qw=0, kw=0, qos=256, qs=256, ks=128, vs=128, dtype=1):
    return lib.pa_rotate_and_cache(qo, q, k, v, kc, vc, slots, pos, freq, qw, kw, T, Hq, Hkv, d, B, NB, rot, inter,
                                   factor, eps, qos, qs, ks, vs, dtype, None)


def _append(lib, S=2, rows=4, F=8, B=16, MB=4, NB=8, nl=16, nf=16, slots=16, pos=16, bt=16, sl=16, qs=16, free=16,
            num=16, status=16):
    return lib.pa_append_tokens(nl, nf, slots, pos, bt, sl, qs, free, num, status, S, rows, F, B, MB, NB, None)


@pytest.mark.parametrize("call,kw,code", [
    (_rotate, dict(dtype=2), INVALID), (_rotate, dict(T=-1), INVALID), (_rotate, dict(Hq=0), INVALID),
    (_rotate, dict(Hkv=0), INVALID), (_rotate, dict(d=80), UNSUPPORTED), (_rotate, dict(rot=0), INVALID),
    (_rotate, dict(rot=63), INVALID), (_rotate, dict(rot=72), INVALID), (_rotate, dict(rot=24), UNSUPPORTED),
    (_rotate, dict(inter=2), INVALID), (_rotate, dict(factor=math.inf), INVALID), (_rotate, dict(qw=16), INVALID),
    (_rotate, dict(qw=16, kw=16, eps=0.0), INVALID), (_rotate, dict(qw=16, kw=16, eps=math.nan), INVALID),
    (_rotate, dict(qw=16, kw=24), INVALID), (_rotate, dict(qs=255), INVALID), (_rotate, dict(ks=120), INVALID),
    (_rotate, dict(qos=252), INVALID), (_rotate, dict(q=0), INVALID), (_rotate, dict(ko=8), INVALID),
    (_rotate, dict(pos=0), INVALID), (_rotate, dict(freq=12), INVALID), (_rotate, dict(Hq=70000, qs=1 << 24, qos=1 << 24), UNSUPPORTED),
    (_rotate, dict(T=0, q=0, ko=0, pos=0), OK),
    (_cached, dict(B=24), UNSUPPORTED), (_cached, dict(NB=0), INVALID), (_cached, dict(kc=0), INVALID),
    (_cached, dict(vc=24), INVALID), (_cached, dict(slots=0), INVALID), (_cached, dict(slots=20), INVALID),
    (_cached, dict(v=0), INVALID), (_cached, dict(vs=64), INVALID), (_cached, dict(qo=4), INVALID),
    (_cached, dict(T=0, kc=0), OK),
    (_append, dict(S=-1), INVALID), (_append, dict(S=16385), UNSUPPORTED), (_append, dict(rows=-1), INVALID),
    (_append, dict(F=-1), INVALID), (_append, dict(B=12), UNSUPPORTED), (_append, dict(MB=0), INVALID),
    (_append, dict(MB=1 << 28), UNSUPPORTED), (_append, dict(NB=0), INVALID), (_append, dict(nf=0), INVALID),
    (_append, dict(num=0), INVALID), (_append, dict(status=0), INVALID), (_append, dict(slots=0), INVALID),
    (_append, dict(pos=20), INVALID), (_append, dict(nl=0), INVALID), (_append, dict(bt=18), INVALID),
    (_append, dict(free=0), INVALID), (_append, dict(qs=0), INVALID),
])
def test_entry_points_refuse(lib, call, kw, code):
    assert call(lib, **kw) == code
    assert (pa.last_error() == "") == (code == OK)


def test_binding_refuses():
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos, freq = torch.zeros(3, dtype=torch.int64), torch.zeros(32, dtype=torch.int64)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.rotate(q, k, q, k, pos, freq)
    with pytest.raises(ValueError, match="both or neither"):
        pa.rotate(q, k, q, k, pos, freq, query_weight=w)
    with pytest.raises(ValueError, match="of query's dtype"):
        pa.rotate(q, k, q, k, pos, freq, query_weight=w.float(), key_weight=w.float())
    with pytest.raises(ValueError, match="positions"):
        pa.rotate(q, k, q, k, pos.int(), freq)
    with pytest.raises(ValueError, match="frequencies"):
        pa.rotate(q, k, q, k, pos, freq.double())
    n = torch.zeros(1, dtype=torch.int32)
    lens, bt, st = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    slots = torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pa.append_tokens(lens, n, slots, slots, bt, lens, st, lens, n, n, 16, 8)
    with pytest.raises(ValueError, match="query_start"):
        pa.append_tokens(lens, n, slots, slots, bt, lens, lens, lens, n, n, 16, 8)
    with pytest.raises(ValueError, match="slot_mapping"):
        pa.append_tokens(lens, n, slots, slots[:4], bt, lens, st, lens, n, n, 16, 8)
    with pytest.raises(ValueError, match="block_tables"):
        pa.append_tokens(lens, n, slots, slots, bt[:1], lens, st, lens, n, n, 16, 8)


def test_append_refuses_counts_beyond_32_bits():
    i32, i64 = dict(dtype=torch.int32, device="meta"), dict(dtype=torch.int64, device="meta")
    n, far = torch.zeros(1, **i32), 2 ** 32 + 4
    for rows, capacity, MB in ((far, 4, 4), (4, far, 4), (4, 4, far)):
        lens, slots = torch.empty(2, **i32), torch.empty(rows, **i64)
        with pytest.raises(ValueError, match="2\\^31"):
            pa.append_tokens(lens, n, slots, slots, torch.empty(2, MB, **i32), lens, torch.empty(3, **i32),
                             torch.empty(capacity, **i32), n, n, 16, 8)


def test_sizes_beyond_32_bits_are_refused():
    # ctypes would cut each of them to a small one that the call takes
    i32, i64, u8, bf16 = (dict(dtype=t, device="meta") for t in (torch.int32, torch.int64, torch.uint8, torch.bfloat16))
    far = 2 ** 32 + 16
    lens, n, slots = torch.empty(2, **i32), torch.zeros(1, **i32), torch.empty(2, **i64)
    for sizes in ((far, 8), (16, far), (16 - 2 ** 32, 8)):
        with pytest.raises(ValueError, match="2\\^31"):
            pa.append_tokens(lens, n, slots, slots, torch.empty(2, 4, **i32), lens, torch.empty(3, **i32),
                             torch.empty(4, **i32), n, n, *sizes)
    q, k = torch.empty(2, 4, 64, **bf16), torch.empty(2, 2, 64, **bf16)
    with pytest.raises(ValueError, match="2\\^31"):
        pa.rotate(q, k, q, k, slots, torch.empty(2 ** 31 + 16, **i64))
    pool4 = *(torch.empty(8, 16, 2, 32, **u8) for _ in range(2)), torch.empty(8, 2, 2, 16, 2, **u8)
    pool8 = *(torch.empty(8, 16, 2, 64, dtype=torch.float8_e4m3fn, device="meta") for _ in range(2)), \
        torch.empty(8, 2, 2, 16, **u8)
    bt, wide = torch.empty(2, 4, **i32), torch.empty(2, far, **i32)
    many = torch.empty(far, **i32)
    for pool, decode, gather, copy in ((pool4, pa.decode_fp4, pa.gather_cache_fp4, pa.copy_blocks_fp4),
                                       (pool8, pa.decode_fp8, pa.gather_cache_fp8, pa.copy_blocks_fp8)):
        for table, pt in ((wide, 0), (bt, far)):
            with pytest.raises(ValueError, match="2\\^31"):
                decode(q, q, *pool, table, lens, 0.1, pt)
        with pytest.raises(ValueError, match="2\\^31"):
            gather(k, k, *pool, wide, lens, slots)
        with pytest.raises(ValueError, match="2\\^31"):
            copy(*pool, many, many)
    caches = [torch.empty(8, 16, 2, 64, **bf16) for _ in range(2)]
    start = torch.empty(3, **i32)
    for bounds in ((far, 4), (4, far)):
        with pytest.raises(ValueError, match="2\\^31"):
            pa.decode_shared_prefix(q, q, *caches, bt, lens, start, lens, *bounds, 0.1)
    for table, pt in ((wide, 0), (bt, far)):
        with pytest.raises(ValueError, match="2\\^31"):
            pa.decode(q, q, *caches, table, lens, 0.1, pt)
    for table, length in ((wide, 1), (bt, far)):
        with pytest.raises(ValueError, match="2\\^31"):
            pa.prefill(q, q, *caches, table, lens, start, length, 0.1)
