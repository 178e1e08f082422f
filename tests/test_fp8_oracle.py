"""The 8-bit cache without a GPU: the oracle's number format against PyTorch's,
its quantiser against the properties that define it, and the refusals of the
entry points and of their Python binding (nothing here launches a kernel)."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from oracle import fp8
from paged_kv_cache_305_gb300 import build as pbuild


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.load_library()


def test_e4m3_values_match_the_type():
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.E4M3, want, equal_nan=True)


def test_nearest_code_matches_a_cast():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 2.0 ** -7,
                        (fp8.E4M3[:126] + fp8.E4M3[1:127]) / 2, fp8.E4M3[:127], -fp8.E4M3[:127]])
    y = y.astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.nearest_code(y), want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantised_rows_keep_what_the_format_promises(dtype):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((400, 64)) * np.exp2(rng.integers(-12, 12, (400, 1)))
    x = oracle.to_float64(W.f32_to_bits(x.astype(np.float32), dtype), dtype)
    codes, e = fp8.quantise_rows(x)
    f = np.exp2(e.astype(np.float64) - 127.0)[:, None]
    top = np.abs(x).max(-1)
    assert np.all(top <= 448 * f[:, 0]) and np.all(top > 224 * f[:, 0])
    # four significant bits (2^-4 of the value), or half a step at the bottom
    assert np.all(np.abs(fp8.E4M3[codes] * f - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * f))


def test_quantised_special_rows():
    x = np.zeros((5, 64))
    x[1, 3], x[2, 0], x[2, 1] = np.inf, np.nan, 3.0
    x[3, 5] = 448.0 * 2.0 ** 4     # 448 exactly at a factor of 2^4
    x[4, 5] = 448.0 * 2.0 ** 4 * (1 + 2.0 ** -7)
    codes, e = fp8.quantise_rows(x)
    assert e[0] == 1 and not codes[0].any()
    assert e[1] == 1 and codes[1, 3] == 0x7F
    assert codes[2, 0] == 0x7F and fp8.E4M3[codes[2, 1]] * 2.0 ** (int(e[2]) - 127) == 3.0
    assert e[3] == 131 and codes[3, 5] == 0x7E
    assert e[4] == 132


def test_pool_values_of_a_written_row():
    key = W.normal_bits((2, 3, 64), "bf16", 1, 1)
    kc = np.zeros((4, 8, 3, 64), np.uint8)
    sc = np.zeros((4, 3, 2, 8), np.uint8)
    kc, vc, sc = fp8.write_fp8(key, key, kc, kc, sc, [17, -1], 8, "bf16")
    got = fp8.pool_values(kc, sc, 0)[2, 1]
    x = oracle.to_float64(key[0], "bf16")
    assert np.all(np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.abs(x).max() * 2.0 ** -17))
    assert not kc[3].any() and np.array_equal(kc, vc)


FAKE = 0x10000  # a 16-byte-aligned non-null address; never dereferenced by these calls


def _write(lib, **kw):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, slots=FAKE, T=3, Hkv=2, d=64, B=16, NB=10, dtype=0)
    a.update(kw)
    return lib.pa_reshape_and_cache_fp8(a["k"], a["v"], a["kc"], a["vc"], a["sc"], a["slots"], a["T"],
                                        a["Hkv"], a["d"], a["B"], a["NB"], a["dtype"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=2), -1, "dtype"), (dict(T=-1), -1, "num_tokens"), (dict(Hkv=0), -1, "num_kv_heads"),
    (dict(Hkv=1 << 20), -2, "2^24"), (dict(d=96), -2, "head_dim"), (dict(B=24), -2, "block_size"),
    (dict(NB=0), -1, "num_blocks"), (dict(sc=None), -1, "NULL"), (dict(slots=None), -1, "NULL"),
    (dict(sc=FAKE + 8), -1, "aligned"), (dict(k=FAKE + 8), -1, "aligned"), (dict(slots=FAKE + 4), -1, "aligned"),
])
def test_write_refusals(lib, kw, code, msg):
    assert _write(lib, **kw) == code
    assert msg in pa.last_error()


def test_empty_calls_are_no_ops(lib):
    assert _write(lib, T=0, k=None, kc=None, sc=None) == 0
    assert lib.pa_copy_blocks_fp8(None, None, None, None, None, 0, 2, 64, 16, 10, None) == 0
    assert _gather(lib, S=0, kc=None, ko=None) == 0
    assert _gather(lib, rows=0, kc=None, ko=None) == 0
    assert _decode(lib, S=0, out=None, sc=None) == 0
    assert _prefix(lib, S=0, NG=0, gs=None) == 0
    assert pa.last_error() == ""


@pytest.mark.parametrize("kw,code,msg", [
    (dict(n=-1), -1, "num_copies"), (dict(d=32), -2, "head_dim"), (dict(sc=None), -1, "NULL"),
    (dict(src=None), -1, "NULL"), (dict(dst=FAKE + 2), -1, "aligned"), (dict(vc=FAKE + 4), -1, "aligned"),
])
def test_copy_refusals(lib, kw, code, msg):
    a = dict(kc=FAKE, vc=FAKE, sc=FAKE, src=FAKE, dst=FAKE, n=2, Hkv=2, d=64, B=16, NB=10)
    a.update(kw)
    assert lib.pa_copy_blocks_fp8(a["kc"], a["vc"], a["sc"], a["src"], a["dst"], a["n"], a["Hkv"], a["d"],
                                  a["B"], a["NB"], None) == code
    assert msg in pa.last_error()


def _gather(lib, **kw):
    a = dict(ko=FAKE, vo=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, sl=FAKE, st=FAKE, rows=100, S=2, Hkv=2,
             d=128, B=16, MB=4, NB=10, dtype=1)
    a.update(kw)
    return lib.pa_gather_cache_fp8(a["ko"], a["vo"], a["kc"], a["vc"], a["sc"], a["bt"], a["sl"], a["st"],
                                   a["rows"], a["S"], a["Hkv"], a["d"], a["B"], a["MB"], a["NB"], a["dtype"],
                                   None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=7), -1, "dtype"), (dict(S=-1), -1, "num_seqs"), (dict(S=65536), -2, "num_seqs"),
    (dict(rows=-1), -1, "num_out_rows"), (dict(MB=0), -1, "max_blocks_per_seq"), (dict(d=256), -2, "head_dim"),
    (dict(MB=1 << 28), -2, "overflows"), (dict(st=None), -1, "NULL"), (dict(st=FAKE + 4), -1, "out_start"),
    (dict(vo=FAKE + 2), -1, "aligned"), (dict(bt=FAKE + 1), -1, "aligned"),
])
def test_gather_refusals(lib, kw, code, msg):
    assert _gather(lib, **kw) == code
    assert msg in pa.last_error()


def _decode(lib, **kw):
    a = dict(out=FAKE, query=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, sl=FAKE, S=2, Hq=8, Hkv=2, d=128,
             B=16, scale=0.1, MB=4, NB=100, pt=0, dtype=1, odt=None, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_decode_fp8(a["out"], a["query"], a["kc"], a["vc"], a["sc"], a["bt"], a["sl"], a["S"],
                             a["Hq"], a["Hkv"], a["d"], a["B"], a["scale"], a["MB"], a["NB"], a["pt"],
                             a["dtype"], a["dtype"] if a["odt"] is None else a["odt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=2), -1, "dtype"), (dict(odt=0), -1, "out_dtype"), (dict(S=-1), -1, "num_seqs"),
    (dict(Hq=6, Hkv=4), -1, "multiple"), (dict(Hq=34, Hkv=2), -2, "query heads per kv head"),
    (dict(d=96), -2, "head_dim"), (dict(B=12), -2, "block_size"), (dict(scale=float("nan")), -1, "scale"),
    (dict(pt=24), -1, "partition_tokens"), (dict(sc=None), -1, "NULL"), (dict(sc=FAKE + 4), -1, "aligned"),
    (dict(query=FAKE + 8), -1, "aligned"), (dict(NB=1 << 27, B=64), -2, "slots"),
    (dict(MB=4096, pt=512), -3, "workspace"), (dict(MB=4096, pt=512, ws=FAKE, wsb=100), -3, "workspace"),
])
def test_decode_refusals(lib, kw, code, msg):
    assert _decode(lib, **kw) == code
    assert msg in pa.last_error()


def _prefix(lib, **kw):
    a = dict(out=FAKE, query=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, sl=FAKE, gs=FAKE, pl=FAKE, S=4, NG=2, Hq=8,
             Hkv=2, d=128, B=16, scale=0.1, MB=4, NB=100, mp=32, mg=4, dtype=1, odt=None, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.pa_decode_shared_prefix(a["out"], a["query"], a["kc"], a["vc"], a["bt"], a["sl"], a["gs"],
                                       a["pl"], a["S"], a["NG"], a["Hq"], a["Hkv"], a["d"], a["B"], a["scale"],
                                       a["MB"], a["NB"], a["mp"], a["mg"], a["dtype"],
                                       a["dtype"] if a["odt"] is None else a["odt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(NG=0), -1, "num_groups"), (dict(NG=65536), -2, "num_groups"), (dict(mp=-1), -1, "max_prefix_len"),
    (dict(mg=-1), -1, "max_group_size"), (dict(gs=None), -1, "NULL"), (dict(pl=FAKE + 2), -1, "aligned"),
    (dict(dtype=2), -1, "dtype"), (dict(odt=0), -1, "out_dtype"), (dict(S=-1), -1, "num_seqs"),
    (dict(Hq=6, Hkv=4), -1, "multiple"), (dict(Hkv=0), -1, "must be >= 1"), (dict(Hq=34, Hkv=2), -2, "per kv head"),
    (dict(d=96), -2, "head_dim"), (dict(B=12), -2, "block_size"), (dict(MB=0), -1, "max_blocks_per_seq"),
    (dict(NB=1 << 27, B=16), -2, "2^31"), (dict(scale=float("inf")), -1, "scale"), (dict(out=None), -1, "NULL"),
    (dict(MB=400, ws=None), -3, "workspace"), (dict(MB=400, wsb=64), -3, "workspace"),
    (dict(MB=400, ws=FAKE + 8), -1, "aligned"), (dict(S=200, mp=64, mg=200, Hkv=8, ws=None), -3, "workspace"),
])
def test_shared_prefix_refusals(lib, kw, code, msg):
    assert _prefix(lib, **kw) == code
    assert msg in pa.last_error()


def test_decode_workspace_holds_the_pieces_where_rows_may_be_cut(lib):
    f = pa.decode_fp8_workspace_bytes
    assert f(8, 8, 2, 128, 16, 16) == 0 and f(8, 8, 2, 128, 256, 1) == 0  # 256 tokens: rows stay whole
    assert f(8, 8, 2, 128, 17, 16) > 0
    assert f(100, 8, 2, 128, 32, 16) == 0 and f(100, 8, 2, 128, 33, 16) > 0  # more rows than SMs: up to 512
    a = f(8, 8, 2, 128, 33, 16)
    assert a > 0 and f(16, 8, 2, 128, 33, 16) > a and f(8, 16, 2, 128, 33, 16) > a
    for bad in [(-1, 8, 2, 128, 64, 16), (8, 0, 2, 128, 64, 16), (8, 8, 0, 128, 64, 16), (8, 8, 3, 128, 64, 16),
                (8, 8, 2, 96, 64, 16), (8, 8, 2, 128, 0, 16), (8, 8, 2, 128, 64, 12)]:
        assert f(*bad) == 0


@pytest.mark.parametrize("kw,code,msg", [
    (dict(pt=-16), -1, "partition_tokens"), (dict(pt=32, B=64), -1, "partition_tokens"),
    (dict(pt=1 << 30), -2, "partition_tokens"), (dict(S=65536), -2, "65535"), (dict(Hq=65536, Hkv=65536), -2, "65535"),
    (dict(MB=1 << 28), -2, "overflows"), (dict(S=65535, Hq=4096, Hkv=4096, MB=100), -2, "too large"),
    (dict(MB=0), -1, "max_blocks_per_seq"), (dict(NB=0), -1, "num_blocks"), (dict(bt=FAKE + 2), -1, "aligned"),
])
def test_decode_refusals_of_sizes(lib, kw, code, msg):
    assert _decode(lib, **kw) == code
    assert msg in pa.last_error()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(S=65536), -2, "65535"), (dict(MB=1 << 28), -2, "overflows"),
    (dict(S=65535, Hq=2048, Hkv=2048, MB=100), -2, "too large"), (dict(gs=FAKE + 1), -1, "aligned"),
])
def test_shared_prefix_refusals_of_sizes(lib, kw, code, msg):
    assert _prefix(lib, **kw) == code
    assert msg in pa.last_error()


def test_shared_prefix_workspace_grows_with_what_it_holds(lib):
    f = pa.decode_shared_prefix_workspace_bytes
    a = f(8, 1, 8, 2, 128, 64, 16, 512, 8)
    assert a > pa.decode_workspace_bytes(8, 8, 128, 64, 16)
    # a prefix pass adds a piece for each query row and chunk; few members have none
    assert f(100, 1, 8, 2, 128, 64, 16, 1000, 100) >= f(100, 1, 8, 2, 128, 64, 16, 0, 100) + 100 * 8 * 128 * 4
    assert a == f(8, 1, 8, 2, 128, 64, 16, 0, 8)
    assert f(16, 1, 8, 2, 128, 64, 16, 512, 8) > a
    # one chunk at least holds any prefix; no chunk without a prefix or members
    assert f(8, 1, 8, 2, 128, 64, 16, 1, 8) >= f(8, 1, 8, 2, 128, 64, 16, 0, 8) > 0
    assert f(8, 1, 8, 2, 128, 64, 16, 512, 0) == f(8, 1, 8, 2, 128, 64, 16, 0, 8)
    for bad in [(8, 0, 8, 2, 128, 64, 16, 512, 8), (8, 1, 8, 3, 128, 64, 16, 512, 8),
                (8, 1, 8, 2, 96, 64, 16, 512, 8), (8, 1, 8, 2, 128, 64, 3, 512, 8),
                (8, 1, 8, 2, 128, 64, 16, -1, 8)]:
        assert f(*bad) == 0


def _cpu_pool(NB=3, B=4, H=2, d=64):
    return pa.alloc_fp8_cache(NB, B, H, d, device="cpu")


def test_binding_refuses_wrong_tensors():
    kc, vc, sc = _cpu_pool()
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        pa.reshape_and_cache_fp8(k, k, kc.view(torch.uint8), vc, sc, slots)
    with pytest.raises(ValueError, match="cache_scales"):
        pa.reshape_and_cache_fp8(k, k, kc, vc, sc[:, :1], slots)
    with pytest.raises(ValueError, match="CUDA"):
        pa.reshape_and_cache_fp8(k, k, kc, vc, sc, slots)
    with pytest.raises(ValueError, match="shape"):
        pa.copy_blocks_fp8(kc, vc[:2], sc, slots.int(), slots.int())
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    bt, sl = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="shape"):
        pa.decode_fp8(q, q, kc, vc, sc, bt, sl, 1.0)
    kc16 = torch.zeros(3, 4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="group_start"):
        pa.decode_shared_prefix(q, q, kc16, kc16, bt, sl, sl, sl, 4, 2, 1.0)
    with pytest.raises(ValueError, match="int32"):
        pa.decode_shared_prefix(q, q, kc16, kc16, bt.long(), sl, sl, sl[:1], 4, 2, 1.0)
