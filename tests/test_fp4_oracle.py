"""The 4-bit cache without a GPU: the oracle's number format and quantiser against the
properties that define them, and the refusals of the entry points and of their Python
binding (nothing here launches a kernel)."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from oracle import fp4
from paged_kv_cache_305_gb300 import build as pbuild


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load_library()


def test_e2m1_values():
    assert fp4.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_nearest_code_is_nearest():
    y = np.concatenate([np.linspace(-7, 7, 4001), fp4.E2M1, [-0.0]])
    got = fp4.E2M1[fp4.nearest_code(y)]
    best = np.min(np.abs(y[:, None] - fp4.E2M1), axis=1)
    assert np.array_equal(np.abs(got - y), best)
    assert np.array_equal(np.signbit(got), np.signbit(y))


def test_ties_go_to_even_codes():
    ties = (fp4.E2M1[:7] + fp4.E2M1[1:8]) / 2
    assert np.all(fp4.nearest_code(ties) % 2 == 0)
    assert np.all(fp4.nearest_code(-ties) % 2 == 0)


def test_pack_and_unpack():
    c = np.arange(64).reshape(2, 32).astype(np.uint8) % 16
    p = fp4.pack(c)
    assert p.shape == (2, 16) and p[0, 0] == 0x10 and p[0, 1] == 0x32
    assert np.array_equal(fp4.unpack(p), c)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantised_rows_keep_what_the_format_promises(dtype):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((400, 128)) * np.exp2(rng.integers(-12, 12, (400, 1)))
    x = oracle.to_float64(W.f32_to_bits(x.astype(np.float32), dtype), dtype)
    codes, e = fp4.quantise_rows(x)
    f = np.exp2(e.astype(np.float64) - 127.0)
    g = np.abs(x.reshape(400, 4, 32))
    top = g.max(-1)
    assert np.all(top <= 7 * f) and np.all(top > 3.5 * f)
    err = np.abs(fp4.row_values(codes, e) - x).reshape(g.shape)
    # half a step: the steps are 1/2 up to 2, 1 up to 4, 2 above, and 7 lies half a step above 6
    step = np.where(g <= 2 * f[..., None], 0.5, np.where(g <= 4 * f[..., None], 1.0, 2.0)) * f[..., None]
    assert np.all(err <= step / 2)


def test_groups_are_their_own():
    x = np.zeros((1, 128))
    x[0, 0], x[0, 40], x[0, 70], x[0, 127] = 7.0, 2.0 ** -30, np.nan, -1e30
    codes, e = fp4.quantise_rows(x)
    v = fp4.row_values(codes, e)
    assert v[0, 0] == 6.0 and v[0, 40] == 2.0 ** -30
    assert e[0, 2] == 255 and np.all(np.isnan(v[0, 64:96]))
    assert abs(v[0, 127] / -1e30 - 1) <= 1 / 6 and np.all(v[0, 1:32] == 0)


def test_quantised_special_groups():
    x = np.zeros((6, 32))
    x[1] = -0.0
    x[2, 3] = np.inf
    x[3, 0] = 2.0 ** -140
    x[4, 0], x[4, 1] = np.float64(np.float32(3.3895314e38)), 2.0 ** 125  # the largest bf16
    x[5, 0], x[5, 1] = 7.0, 0.25
    codes, e = fp4.quantise_rows(x)
    assert e[:, 0].tolist() == [0, 0, 255, 1, 252, 127]
    v = fp4.row_values(codes, e)
    assert np.all(v[0] == 0) and np.all(v[1] == 0) and np.all(np.signbit(v[1]))
    assert np.all(np.isnan(v[2])) and np.all(v[3] == 0)
    assert v[4, 0] == 6 * 2.0 ** 125 < 3.4e38 and v[4, 1] == 2.0 ** 125
    assert v[5, 0] == 6.0 and v[5, 1] == 0.0  # 0.25 is a tie: to the even code


def test_written_rows_land_at_their_slots():
    rng = np.random.default_rng(3)
    key, value = (W.f32_to_bits(rng.standard_normal((5, 2, 64)).astype(np.float32), "bf16") for _ in range(2))
    kc = np.full((3, 4, 2, 32), 0x21, np.uint8)
    sc = np.full((3, 2, 2, 4, 2), 7, np.uint8)
    slots = np.array([9, -1, 0, 11, 4], np.int64)
    k, v, s = fp4.write_fp4(key, value, kc, kc, sc, slots, 4, "bf16")
    x = oracle.to_float64(key, "bf16")
    codes, e = fp4.quantise_rows(x)
    for i, slot in enumerate(slots):
        if slot >= 0:
            assert np.array_equal(k[slot // 4, slot % 4], codes[i])
            assert np.array_equal(s[slot // 4, :, 0, slot % 4], e[i])
    assert np.all(k[0, 1:] == 0x21) and np.all(s[2, :, :, 0] == 7)
    assert np.array_equal(fp4.pool_values(k, s, 0)[2, 1], fp4.row_values(codes[0], e[0]))


# ---------------------------------------------------------------- refusals --
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


def _write(lib, T=4, H=2, d=64, B=16, NB=4, dtype=1, key=16, value=16, kc=16, vc=16, sc=16, slots=16):
    return lib.pa_reshape_and_cache_fp4(key, value, kc, vc, sc, slots, T, H, d, B, NB, dtype, None)


def _copy(lib, n=1, H=2, d=64, B=16, NB=4, kc=16, vc=16, sc=16, src=16, dst=16):
    return lib.pa_copy_blocks_fp4(kc, vc, sc, src, dst, n, H, d, B, NB, None)


def _gather(lib, S=2, H=2, d=64, B=16, MB=4, NB=4, rows=8, dtype=1, ko=16, vo=16, kc=16, vc=16, sc=16, bt=16, sl=16,
            st=16):
    return lib.pa_gather_cache_fp4(ko, vo, kc, vc, sc, bt, sl, st, rows, S, H, d, B, MB, NB, dtype, None)


@pytest.mark.parametrize("call,kw,code", [
    (_write, dict(dtype=2), INVALID), (_write, dict(T=-1), INVALID), (_write, dict(H=0), INVALID),
    (_write, dict(d=96), UNSUPPORTED), (_write, dict(B=24), UNSUPPORTED), (_write, dict(NB=0), INVALID),
    (_write, dict(key=0), INVALID), (_write, dict(slots=0), INVALID), (_write, dict(kc=8), INVALID),
    (_write, dict(sc=8), INVALID), (_write, dict(value=24), INVALID), (_write, dict(slots=20), INVALID),
    (_write, dict(H=1 << 20, d=128), UNSUPPORTED), (_write, dict(T=0, key=0), OK),
    (_copy, dict(n=-1), INVALID), (_copy, dict(d=32), UNSUPPORTED), (_copy, dict(src=0), INVALID),
    (_copy, dict(dst=18), INVALID), (_copy, dict(sc=0), INVALID), (_copy, dict(n=0, src=0), OK),
    (_gather, dict(S=-1), INVALID), (_gather, dict(S=70000), UNSUPPORTED), (_gather, dict(rows=-1), INVALID),
    (_gather, dict(MB=0), INVALID), (_gather, dict(MB=1 << 28), UNSUPPORTED), (_gather, dict(ko=0), INVALID),
    (_gather, dict(vo=8), INVALID), (_gather, dict(st=20), INVALID), (_gather, dict(bt=18), INVALID),
    (_gather, dict(dtype=7), INVALID), (_gather, dict(rows=0, ko=0), OK), (_gather, dict(S=0, bt=0), OK),
])
def test_entry_points_refuse(lib, call, kw, code):
    assert call(lib, **kw) == code
    assert (pa.last_error() == "") == (code == OK)


def _pool(NB=4, B=16, H=2, d=64):
    return pa.alloc_fp4_cache(NB, B, H, d, device="cpu")


def test_alloc_shapes():
    k, v, s = _pool(d=128)
    assert k.shape == v.shape == (4, 16, 2, 64) and k.dtype == torch.uint8
    assert s.shape == (4, 2, 2, 16, 4) and s.dtype == torch.uint8


def test_binding_refuses():
    k, v, s = _pool()
    key = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pa.reshape_and_cache_fp4(key, key, k, v, s, slots)
    with pytest.raises(ValueError, match="uint8"):
        pa.reshape_and_cache_fp4(key, key, k.view(torch.int8), v.view(torch.int8), s, slots)
    with pytest.raises(ValueError, match="cache_scales"):
        pa.reshape_and_cache_fp4(key, key, k, v, s[..., :1], slots)
    with pytest.raises(ValueError, match="cache shape"):
        pa.copy_blocks_fp4(k, v[:2], s, slots.int(), slots.int())
    with pytest.raises(ValueError):
        pa.gather_cache_fp4(key, key, k, v, s, torch.zeros(1, 2, dtype=torch.int32),
                            torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64))
