"""The 4-bit cache on the GPU: write, block copy and read-back bit for bit against the
oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from gpu_util import dev_bits, host_bits
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_305_gb300 import build
    build.build()
    pa.bad_index_count(clear=True)
    yield
    torch.cuda.synchronize()


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def random_pool(rng, NB, B, Hkv, d, spread=3):
    """A pool with every code, factors over 2 * spread binades, and some groups of factor zero."""
    codes = [rng.integers(0, 256, (NB, B, Hkv, d // 2)).astype(np.uint8) for _ in range(2)]
    scales = rng.integers(125 - spread, 125 + spread + 1, (NB, Hkv, 2, B, d // 32)).astype(np.uint8)
    scales[rng.random(scales.shape) < 0.03] = 0
    return codes[0], codes[1], scales


def tables_for(rng, lens, B, NB, MB=None):
    held = [-(-int(n) // B) for n in lens]
    MB = MB or max(1, max(held))
    perm = rng.permutation(NB)
    bt = rng.integers(0, NB, (len(lens), MB)).astype(np.int32)
    at = 0
    for s, n in enumerate(held):
        bt[s, :n] = perm[at:at + n]
        at += n
    assert at <= NB
    return bt


# ------------------------------------------------------------------ write --
@pytest.mark.parametrize("dtype,Hkv,d,B,T", [("bf16", 8, 128, 16, 97), ("fp16", 4, 64, 16, 1),
                                             ("bf16", 1, 64, 1, 33), ("fp16", 3, 128, 64, 200),
                                             ("bf16", 5, 64, 8, 7)])
def test_write_bit_exact(dtype, Hkv, d, B, T):
    rng = np.random.default_rng(T)
    NB = -(-T // B) + 3
    x = [rng.standard_normal((T, Hkv, d)) * np.exp2(rng.integers(-20, 14, (T, Hkv, 1))) for _ in range(2)]
    key, value = (W.f32_to_bits(v.astype(np.float32), dtype) for v in x)
    slots = rng.choice(NB * B, size=T, replace=False).astype(np.int64)
    slots[3::5] = -1
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    kd, vd, sd = up(kc), up(vc), up(sc)
    pa.reshape_and_cache_fp4(dev_bits(key, dtype), dev_bits(value, dtype), kd, vd, sd, up(slots))
    wk, wv, ws = fp4.write_fp4(key, value, kc, vc, sc, slots, B, dtype)
    assert np.array_equal(kd.cpu().numpy(), wk) and np.array_equal(vd.cpu().numpy(), wv)
    assert np.array_equal(sd.cpu().numpy(), ws)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_special_groups(dtype):
    # zeros of both signs, subnormals, ties, infinities, NaN, the end of the type's range: each
    # in one group of its row, beside a group of ordinary values
    d = 64
    x = np.zeros((10, 1, d), np.float32)
    x[:, 0, 32:] = np.linspace(-3, 5, 32)
    x[1, 0, :32] = -0.0
    x[2, 0, :4] = [2.0 ** -24, -3 * 2.0 ** -24, 2.0 ** -20, 0]
    x[3, 0, :2] = [65504, -1]
    x[4, 0, :3] = [np.inf, -2.5, 1]
    x[5, 0, 31] = np.nan
    x[6, 0, :8] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    x[7, 0, :3] = [7.0625, 1, 0.5]  # just above 7: the next factor
    x[8, 0, :4] = [6.5, -6.9375, 6, -5.0]
    x[9, 0, :3] = [-np.inf, np.nan, np.inf]
    bits = W.f32_to_bits(x, dtype)
    if dtype == "bf16":
        bits = np.concatenate([bits, np.zeros((3, 1, d), np.uint16)])
        bits[10, 0, :2] = [0x7F7F, 0x0080]   # the largest bf16 and the smallest normal
        bits[11, 0, :2] = [0x0001, 0x8003]   # subnormals
        bits[12, 0, :2] = [0x0080, 0x8060]   # the smallest normal, and subnormal halves of it
    T = bits.shape[0]
    kc = np.full((2, 16, 1, d // 2), 0x55, np.uint8)
    sc = np.full((2, 1, 2, 16, 2), 9, np.uint8)
    kd, vd, sd = up(kc), up(kc), up(sc)
    slots = np.arange(T, dtype=np.int64) + 3
    pa.reshape_and_cache_fp4(dev_bits(bits, dtype), dev_bits(bits[::-1].copy(), dtype), kd, vd, sd, up(slots))
    wk, wv, ws = fp4.write_fp4(bits, bits[::-1], kc, kc, sc, slots, 16, dtype)
    assert np.array_equal(kd.cpu().numpy(), wk) and np.array_equal(vd.cpu().numpy(), wv)
    assert np.array_equal(sd.cpu().numpy(), ws)


def test_write_every_16_bit_value():
    # each of the 2^16 bf16 patterns beside each of two neighbours that set the factor
    pat = np.arange(1 << 16, dtype=np.uint16).reshape(-1, 1, 64)
    pat = np.concatenate([pat, pat], 0)
    pat[:1024, :, 0::32] = 0x4120  # 10.0
    T = pat.shape[0]
    kd, vd, sd = pa.alloc_fp4_cache(T // 64, 64, 1, 64)
    slots = np.arange(T, dtype=np.int64)
    pa.reshape_and_cache_fp4(dev_bits(pat, "bf16"), dev_bits(pat, "bf16"), kd, vd, sd, up(slots))
    codes, e = fp4.quantise_rows(oracle.to_float64(pat, "bf16"))
    assert np.array_equal(kd.cpu().numpy().reshape(codes.shape), codes)
    assert np.array_equal(vd.cpu().numpy().reshape(codes.shape), codes)
    assert np.array_equal(sd[:, 0, 0].cpu().numpy().reshape(T, 2), e.reshape(T, 2))


def test_write_out_of_range_slots_are_skipped_and_counted():
    kd, vd, sd = pa.alloc_fp4_cache(2, 8, 2, 64)
    k = dev_bits(W.normal_bits((4, 2, 64), "bf16", 1, 1), "bf16")
    pa.bad_index_count(clear=True)
    pa.reshape_and_cache_fp4(k, k, kd, vd, sd, torch.tensor([16, -1, 10 ** 12, -7], device="cuda"))
    assert pa.bad_index_count(clear=True) == 2
    assert not kd.any() and not vd.any() and not sd.any()


# ------------------------------------------------------------------- copy --
@pytest.mark.parametrize("B,Hkv,d,NB", [(16, 8, 128, 40), (1, 1, 64, 40), (64, 3, 64, 12), (2, 5, 128, 40)])
def test_copy_blocks_bit_exact(B, Hkv, d, NB):
    rng = np.random.default_rng(B)
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    kd, vd, sd = up(kc), up(vc), up(sc)
    pairs = [(3, 10), (11, 0), (NB - 1, 5), (7, 7), (3, 6)]
    bad = [(NB, 1), (2, -1)]
    pa.bad_index_count(clear=True)
    src, dst = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in zip(*(pairs + bad)))
    pa.copy_blocks_fp4(kd, vd, sd, src, dst)
    assert pa.bad_index_count(clear=True) == 2
    for got, want in ((kd, kc), (vd, vc), (sd, sc)):
        ref = want.copy()
        for a, b in pairs:
            ref[b] = want[a]
        assert np.array_equal(got.cpu().numpy(), ref)


# ----------------------------------------------------------------- gather --
@pytest.mark.parametrize("dtype,Hkv,d,B,lens", [("bf16", 8, 128, 16, [1, 17, 0, 300]),
                                                ("fp16", 3, 64, 8, [63, 64, 65]), ("bf16", 1, 128, 1, [5]),
                                                ("fp16", 2, 128, 64, [200, 1, 129]), ("fp16", 5, 64, 2, [0, 0])])
def test_gather_bit_exact_and_nothing_else(dtype, Hkv, d, B, lens):
    rng = np.random.default_rng(len(lens) + B)
    NB = sum(-(-n // B) for n in lens) + 2
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d, spread=9)
    bt = tables_for(rng, lens, B, NB)
    starts = np.cumsum([3] + [n + 2 for n in lens])[:-1].astype(np.int64)
    rows = int(starts[-1] + lens[-1] + 4)
    fill = W.normal_bits((rows, Hkv, d), dtype, 4, 4)
    ko, vo = dev_bits(fill, dtype), dev_bits(fill, dtype)
    pa.gather_cache_fp4(ko, vo, up(kc), up(vc), up(sc), up(bt), up(np.array(lens, np.int32)), up(starts))
    for which, (got, codes) in enumerate(((ko, kc), (vo, vc))):
        want = fill.copy()
        values = fp4.pool_values(codes, sc, which)
        for s, n in enumerate(lens):
            v = oracle.gather_kv(values, bt[s], n, B)
            want[starts[s]:starts[s] + n] = oracle.round_to_dtype(v.reshape(n, Hkv, d), dtype)
        assert np.array_equal(host_bits(got), want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_gather_factors_of_every_size(dtype):
    # every byte: zero, subnormal and infinite 16-bit values, and 255 as NaN where codes are zero
    rng = np.random.default_rng(8)
    kc, vc, sc = random_pool(rng, 4, 64, 1, 64)
    sc[:, 0, :, :, 0] = np.arange(256).reshape(4, 1, 64)
    sc[:, 0, :, :, 1] = np.arange(256)[::-1].reshape(4, 1, 64)
    kc[3, 63, 0, :16] = 0
    ko = torch.zeros(256, 1, 64, dtype=torch.float16 if dtype == "fp16" else torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    pa.gather_cache_fp4(ko, vo, up(kc), up(vc), up(sc), torch.arange(4, dtype=torch.int32, device="cuda")[None],
                        torch.tensor([256], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"))
    for which, (got, codes) in enumerate(((ko, kc), (vo, vc))):
        want = torch.from_numpy(fp4.pool_values(codes, sc, which).reshape(256, 1, 64)).to(got.dtype).cuda()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(1.5), want.nan_to_num(1.5))
    assert ko[255, 0, :32].isnan().all()


def test_gather_bad_indices():
    rng = np.random.default_rng(5)
    kc, vc, sc = random_pool(rng, 4, 4, 1, 64)
    bt = np.array([[0, 9, 1, -1], [2, 3, 0, 0]], np.int32)
    ko = torch.full((20, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    pa.bad_index_count(clear=True)
    # sequence 0: blocks 9 and -1 are rejected; its length is above the table's
    # 16 tokens; sequence 1: rows -2, -1 and no others are out of range
    pa.gather_cache_fp4(ko, vo, up(kc), up(vc), up(sc), up(bt), up(np.array([99, 5], np.int32)),
                        up(np.array([3, -2], np.int64)))
    assert pa.bad_index_count(clear=True) == 2 + 1 + 2
    got = ko.float().cpu().numpy()
    assert not got[7:11].any() and not got[15:19].any() and np.all(got[19] == 7.0)
    values = fp4.pool_values(kc, sc, 0)
    assert np.array_equal(got[11:15, 0].astype(np.float64), oracle.to_float64(
        oracle.round_to_dtype(values[1, :, 0], "bf16"), "bf16"))
