"""The 8-bit cache on the GPU: write, block copy and read-back bit for bit
against the oracle, decode against exact attention over the pool's values with
a bound derived from the arithmetic (oracle.fp8.decode_bound), and the pieces
together as a serving loop uses them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from gpu_util import TORCH_DTYPE, dev_bits, host_bits
from oracle import fp8

pytestmark = pytest.mark.gpu

# decode_fp8 splits a weight into two fp16 parts: relative error below 2^-20
WEIGHT_ERROR = 2.0 ** -20


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


def up8(codes):
    return up(codes).view(torch.float8_e4m3fn)


def down8(t):
    return t.view(torch.uint8).cpu().numpy()


def random_pool(rng, NB, B, Hkv, d, spread=3):
    """A pool with every code that is not NaN and factors over 2 * spread binades."""
    codes = [rng.integers(0, 256, (NB, B, Hkv, d)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0x38
    scales = rng.integers(127 - 8 - spread, 127 - 8 + spread + 1, (NB, Hkv, 2, B)).astype(np.uint8)
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
    kd, vd, sd = up8(kc), up8(vc), up(sc)
    pa.reshape_and_cache_fp8(dev_bits(key, dtype), dev_bits(value, dtype), kd, vd, sd, up(slots))
    wk, wv, ws = fp8.write_fp8(key, value, kc, vc, sc, slots, B, dtype)
    assert np.array_equal(down8(kd), wk) and np.array_equal(down8(vd), wv)
    assert np.array_equal(sd.cpu().numpy(), ws)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_special_rows(dtype):
    # zeros, negative zeros, subnormals, the type's largest value, infinities,
    # NaN, a row without a finite element, 448 and ties of the code grid
    d = 64
    x = np.zeros((10, 1, d), np.float32)
    x[1] = -0.0
    x[2, 0, :4] = [2.0 ** -24, -3 * 2.0 ** -24, 2.0 ** -20, 0]
    x[3, 0, :2] = [65504, -1]
    x[4, 0, :3] = [np.inf, -2.5, -np.inf]
    x[5, 0, :3] = [np.nan, 7.0, -7.25]
    x[6] = np.inf
    x[7, 0, :3] = [448, 17, 19]          # factor 1: ties between 16, 18 and 20
    x[8, 0, :4] = [448, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11]  # ties at the bottom of the grid
    x[9, 0, :2] = [449 if dtype == "fp16" else 450, 1]
    bits = W.f32_to_bits(x, dtype)
    if dtype == "bf16":
        bits = np.concatenate([bits, np.zeros((2, 1, d), np.uint16)])
        bits[10, 0, :2] = [0x7F7F, 0x0080]   # the largest bf16 and the smallest normal
        bits[11, 0, :2] = [0x0001, 0x8003]   # subnormals
    T = bits.shape[0]
    kc = np.full((2, 16, 1, d), 0x55, np.uint8)
    sc = np.full((2, 1, 2, 16), 9, np.uint8)
    kd, vd, sd = up8(kc), up8(kc), up(sc)
    slots = np.arange(T, dtype=np.int64) + 3
    pa.reshape_and_cache_fp8(dev_bits(bits, dtype), dev_bits(bits[::-1].copy(), dtype), kd, vd, sd, up(slots))
    wk, wv, ws = fp8.write_fp8(bits, bits[::-1], kc, kc, sc, slots, 16, dtype)
    nan = (wk & 0x7F) == 0x7F  # a NaN's sign is not kept
    assert np.array_equal((down8(kd) & 0x7F) == 0x7F, nan)
    assert np.array_equal(down8(kd)[~nan], wk[~nan])
    nan = (wv & 0x7F) == 0x7F
    assert np.array_equal((down8(vd) & 0x7F) == 0x7F, nan) and np.array_equal(down8(vd)[~nan], wv[~nan])
    assert np.array_equal(sd.cpu().numpy(), ws)


def test_write_out_of_range_slots_are_skipped_and_counted():
    kd, vd, sd = pa.alloc_fp8_cache(2, 8, 2, 64)
    k = dev_bits(W.normal_bits((4, 2, 64), "bf16", 1, 1), "bf16")
    pa.bad_index_count(clear=True)
    pa.reshape_and_cache_fp8(k, k, kd, vd, sd, torch.tensor([16, -1, 10 ** 12, -7], device="cuda"))
    assert pa.bad_index_count(clear=True) == 2
    assert not down8(kd).any() and not down8(vd).any() and not sd.any()


# ------------------------------------------------------------------- copy --
@pytest.mark.parametrize("B,Hkv,d,NB", [(16, 8, 128, 40), (1, 1, 64, 40), (64, 3, 64, 12), (2, 5, 128, 40)])
def test_copy_blocks_bit_exact(B, Hkv, d, NB):
    rng = np.random.default_rng(B)
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    kd, vd, sd = up8(kc), up8(vc), up(sc)
    pairs = [(3, 10), (11, 0), (NB - 1, 5), (7, 7), (3, 6)]
    bad = [(NB, 1), (2, -1)]
    pa.bad_index_count(clear=True)
    src, dst = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in zip(*(pairs + bad)))
    pa.copy_blocks_fp8(kd, vd, sd, src, dst)
    assert pa.bad_index_count(clear=True) == 2
    for got, want in ((down8(kd), kc), (down8(vd), vc), (sd.cpu().numpy(), sc)):
        ref = want.copy()
        for a, b in pairs:
            ref[b] = want[a]
        assert np.array_equal(got, ref)


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
    pa.gather_cache_fp8(ko, vo, up8(kc), up8(vc), up(sc), up(bt), up(np.array(lens, np.int32)), up(starts))
    for which, (got, codes) in enumerate(((ko, kc), (vo, vc))):
        want = fill.copy()
        values = fp8.pool_values(codes, sc, which)
        for s, n in enumerate(lens):
            v = oracle.gather_kv(values, bt[s], n, B)
            want[starts[s]:starts[s] + n] = oracle.round_to_dtype(v.reshape(n, Hkv, d), dtype)
        assert np.array_equal(host_bits(got), want)


def test_gather_bad_indices():
    rng = np.random.default_rng(5)
    kc, vc, sc = random_pool(rng, 4, 4, 1, 64)
    bt = np.array([[0, 9, 1, -1], [2, 3, 0, 0]], np.int32)
    ko = torch.full((20, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    pa.bad_index_count(clear=True)
    # sequence 0: blocks 9 and -1 are rejected; its length is above the table's
    # 16 tokens; sequence 1: rows -2, -1 and no others are out of range
    pa.gather_cache_fp8(ko, vo, up8(kc), up8(vc), up(sc), up(bt), up(np.array([99, 5], np.int32)),
                        up(np.array([3, -2], np.int64)))
    assert pa.bad_index_count(clear=True) == 2 + 1 + 2
    got = ko.float().cpu().numpy()
    assert not got[7:11].any() and not got[15:19].any() and np.all(got[19] == 7.0)
    values = fp8.pool_values(kc, sc, 0)
    assert np.array_equal(got[11:15, 0].astype(np.float64), oracle.to_float64(
        oracle.round_to_dtype(values[1, :, 0], "bf16"), "bf16"))


# ----------------------------------------------------------------- decode --
def check_decode(query, kc, vc, sc, bt, lens, B, scale, dtype, pt=0, ws=None, what=""):
    """Both output types against the oracle; returns the fp32 output."""
    q = dev_bits(query, dtype)
    kd, vd, sd, btd, sl = up8(kc), up8(vc), up(sc), up(bt), up(np.asarray(lens, np.int32))
    if ws is None:
        ws = pa.alloc_workspace(q, kd, btd, pt)
    o32 = torch.full(query.shape, float("nan"), dtype=torch.float32, device="cuda")
    o16 = torch.empty_like(q)
    pa.decode_fp8(o32, q, kd, vd, sd, btd, sl, scale, pt, ws)
    pa.decode_fp8(o16, q, kd, vd, sd, btd, sl, scale, pt, ws)
    got = o32.double().cpu().numpy()
    Kp, Vp = fp8.pool_values(kc, sc, 0), fp8.pool_values(vc, sc, 1)
    used = np.minimum(lens, bt.shape[1] * B)
    ref = fp8.attend(query, Kp, Vp, bt, used, B, scale, dtype)
    for s, n in enumerate(used):
        K, V = (oracle.gather_kv(p, bt[s], int(n), B) for p in (Kp, Vp))
        tol = fp8.decode_bound(oracle.to_float64(query[s], dtype), K, V, scale, WEIGHT_ERROR)
        err = np.max(np.abs(got[s] - ref[s]))
        assert err <= tol, f"{what} sequence {s} of {n} tokens: {err} > {tol}"
    assert np.array_equal(oracle.round_to_dtype(got, dtype), host_bits(o16)), what
    return o32


GRID = [
    # dtype, d, Hq, Hkv, B, lengths, partition_tokens, factor spread
    ("fp16", 64, 4, 4, 16, [1, 128, 57, 33], 0, 3),
    ("bf16", 128, 32, 8, 16, [700, 1, 64, 65, 513], 64, 3),
    ("fp16", 128, 16, 1, 8, [300, 31, 32, 33], 0, 3),
    ("bf16", 64, 6, 3, 4, [90, 0, 16, 17], 32, 3),
    ("fp16", 128, 8, 8, 1, [200, 5], 0, 8),
    ("bf16", 128, 14, 2, 32, [1100, 1023], 0, 0),
    ("fp16", 64, 8, 2, 64, [1500, 1025, 3], 128, 3),
    ("bf16", 128, 12, 4, 2, [100, 99], 16, 3),
    ("fp16", 128, 64, 8, 16, [2100, 600], 512, 3),
    ("bf16", 64, 2, 1, 16, [40, 0, 0, 1], 0, 3),
    ("bf16", 64, 13, 1, 16, [3000, 2999], 0, 3),
    ("fp16", 128, 5, 5, 16, [5000], 0, 3),
]


@pytest.mark.parametrize("idx", range(len(GRID)))
def test_decode_grid(idx):
    dtype, d, Hq, Hkv, B, lens, pt, spread = GRID[idx]
    rng = np.random.default_rng(idx)
    NB = sum(-(-n // B) for n in lens) + 3
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d, spread)
    bt = tables_for(rng, lens, B, NB, MB=max(-(-max(lens) // B) + 1, 1))
    query = W.normal_bits((len(lens), Hq, d), dtype, idx, 2)
    check_decode(query, kc, vc, sc, bt, lens, B, 1 / np.sqrt(d), dtype, pt, what=str(GRID[idx]))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_never_reads_past_the_length(d):
    # NaN codes and an infinite factor in every slot that no sequence holds
    rng = np.random.default_rng(2)
    lens, B, Hkv = [1, 15, 16, 17, 31, 32, 33, 47, 0, 130], 16, 2
    NB = 40
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    bt = tables_for(rng, lens, B, NB)
    used = np.zeros((NB, B), bool)
    for s, n in enumerate(lens):
        for t in range(n):
            used[bt[s, t // B], t % B] = True
    kc[~used], vc[~used] = 0x7F, 0xFF
    sc.transpose(0, 3, 1, 2)[~used] = 255
    query = W.normal_bits((len(lens), 8, d), "bf16", 3, 2)
    check_decode(query, kc, vc, sc, bt, lens, B, 1 / np.sqrt(d), "bf16", 32)


def test_decode_far_apart_factors():
    # V's factors over 200 binades, the large ones at tokens of small weight:
    # the weights' 16-bit parts keep their bits relative to the largest product
    rng = np.random.default_rng(3)
    B, n, d = 16, 200, 64
    kc, vc, sc = random_pool(rng, 20, B, 1, d, 2)
    bt = tables_for(rng, [n], B, 20)
    sc[:, 0, 1] = rng.integers(20, 220, sc[:, 0, 1].shape)
    query = W.normal_bits((1, 4, d), "fp16", 3, 2)
    K, V = fp8.pool_values(kc, sc, 0), fp8.pool_values(vc, sc, 1)
    q, btd, sl = dev_bits(query, "fp16"), up(bt), up(np.array([n], np.int32))
    out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
    pa.decode_fp8(out, q, up8(kc), up8(vc), up(sc), btd, sl, 0.125)
    ref = fp8.attend(query, K, V, bt, [n], B, 0.125, "fp16")
    got = out.double().cpu().numpy()
    Kr, Vr = (oracle.gather_kv(p, bt[0], n, B) for p in (K, V))
    # the bound with the weighted rows in the place of max |V|: sum p |V|, twice the terms' error
    qf = oracle.to_float64(query[0], "fp16")
    p = oracle.attention_weights(qf @ Kr[:, 0].T * 0.125)
    size = (p @ np.abs(Vr[:, 0])).max()
    rel = fp8.decode_bound(qf, Kr, np.ones_like(Vr), 0.125, WEIGHT_ERROR)
    # parts below fp16's normal range: each of n terms loses at most 2^-25 of the
    # largest weight, times a code of at most 448, where the row of the largest
    # weight has an element of at least 1 (in units of its factor)
    assert np.max(np.abs(got - ref)) <= size * (rel + n * 2.0 ** -25 * 448)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 60])
def test_decode_bf16_queries_of_any_size(size):
    # a bf16 query far outside fp16's range keeps its bits
    rng = np.random.default_rng(4)
    B, n, d = 8, 70, 128
    kc, vc, sc = random_pool(rng, 12, B, 2, d, 2)
    bt = tables_for(rng, [n], B, 12)
    q = rng.standard_normal((1, 6, d)).astype(np.float32)
    query = W.f32_to_bits((q * np.float32(size)).astype(np.float32), "bf16")
    check_decode(query, kc, vc, sc, bt, [n], B, 1 / (np.sqrt(d) * size), "bf16")


@pytest.mark.parametrize("size", [2.0 ** -118, 2.0 ** -125])
def test_decode_bf16_queries_next_to_the_smallest(size):
    rng = np.random.default_rng(24)
    B, n, d = 16, 50, 64
    kc, vc, sc = random_pool(rng, 6, B, 1, d, 2)
    bt = tables_for(rng, [n], B, 6)
    q = rng.uniform(1, 2, (1, 3, d)) * rng.choice([-1, 1], (1, 3, d))  # normal bf16 numbers
    query = W.f32_to_bits((q * size).astype(np.float32), "bf16")
    check_decode(query, kc, vc, sc, bt, [n], B, 0.125 / size, "bf16")


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.5])
@pytest.mark.parametrize("dtype,Hq,B", [("bf16", 8, 16), ("fp16", 14, 2)])
def test_decode_scales(scale, dtype, Hq, B):
    rng = np.random.default_rng(25)
    lens = [130, 1, 600]
    NB = sum(-(-n // B) for n in lens)
    kc, vc, sc = random_pool(rng, NB, B, 2, 64, 0)
    bt = tables_for(rng, lens, B, NB)
    check_decode(W.normal_bits((3, Hq, 64), dtype, 25, 2), kc, vc, sc, bt, lens, B, scale, dtype)


def test_decode_zero_query_and_zero_pool():
    kd, vd, sd = pa.alloc_fp8_cache(4, 16, 1, 64)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((1, 1, 64), 3.0, dtype=torch.float32, device="cuda")
    bt, sl = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([50], dtype=torch.int32, device="cuda")
    pa.decode_fp8(out, q, kd, vd, sd, bt, sl, 1.0)
    assert not out.any()


def test_decode_bad_blocks_read_as_zeros_and_are_counted():
    rng = np.random.default_rng(6)
    B, d, lens = 16, 64, [40, 40]
    kc, vc, sc = random_pool(rng, 6, B, 1, d)
    bt = np.array([[0, 77, 1], [2, 3, -1]], np.int32)
    query = W.normal_bits((2, 2, d), "bf16", 6, 2)
    pa.bad_index_count(clear=True)
    out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
    pa.decode_fp8(out, dev_bits(query, "bf16"), up8(kc), up8(vc), up(sc), up(bt),
                  up(np.array(lens, np.int32)), 0.125)
    assert pa.bad_index_count(clear=True) > 0
    kz, vz = np.concatenate([kc, np.zeros_like(kc[:1])]), np.concatenate([vc, np.zeros_like(vc[:1])])
    scz = np.concatenate([sc, np.full_like(sc[:1], 127)])
    btz = np.where((bt < 0) | (bt >= 6), 6, bt)
    K, V = fp8.pool_values(kz, scz, 0), fp8.pool_values(vz, scz, 1)
    ref = fp8.attend(query, K, V, btz, lens, B, 0.125, "bf16")
    for s in range(2):
        tol = fp8.decode_bound(oracle.to_float64(query[s], "bf16"), oracle.gather_kv(K, btz[s], 40, B),
                               oracle.gather_kv(V, btz[s], 40, B), 0.125, WEIGHT_ERROR)
        assert np.max(np.abs(out[s].double().cpu().numpy() - ref[s])) <= tol


def test_decode_bit_identical_however_placed_and_repeated():
    rng = np.random.default_rng(7)
    lens, B, Hkv, d = [1200, 700, 2048], 16, 2, 128
    NB = 300
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    bt = tables_for(rng, lens, B, NB)
    query = W.normal_bits((3, 8, d), "bf16", 7, 2)
    a = check_decode(query, kc, vc, sc, bt, lens, B, 0.09, "bf16", 64)
    perm = rng.permutation(NB)
    inv = np.argsort(perm)
    b = check_decode(query, kc[perm], vc[perm], sc[perm], inv[bt].astype(np.int32), lens, B, 0.09, "bf16", 64)
    assert torch.equal(a, b)


def test_workspace_shared_with_16_bit_decode_and_other_sizes():
    rng = np.random.default_rng(8)
    B, d, Hkv = 16, 64, 2
    n = max(pa.decode_workspace_bytes(6, 8, d, 64, B, 16), pa.decode_fp8_workspace_bytes(6, 8, Hkv, d, 64, B))
    big = torch.zeros(n, dtype=torch.uint8, device="cuda")
    case = W.random_case(num_seqs=4, num_q_heads=8, num_kv_heads=Hkv, head_dim=d, block_size=B,
                         len_range=(1, 900), dtype="fp16", seed=9)
    ref16 = oracle.paged_decode(case.query, case.key_cache, case.value_cache, case.block_tables,
                                case.seq_lens, B, case.scale, "fp16")
    for S in (2, 6, 3):
        lens = rng.integers(1, 1000, S)
        kc, vc, sc = random_pool(rng, int(sum(-(-lens // B))), B, Hkv, d)
        bt = tables_for(rng, lens, B, kc.shape[0], MB=64)
        check_decode(W.normal_bits((S, 8, d), "fp16", S, 2), kc, vc, sc, bt, lens, B, 0.125, "fp16", 16, big)
        o = torch.empty(case.query.shape, dtype=torch.float32, device="cuda")
        pa.decode(o, dev_bits(case.query, "fp16"), dev_bits(case.key_cache, "fp16"),
                  dev_bits(case.value_cache, "fp16"), up(case.block_tables), up(case.seq_lens), case.scale, 32, big)
        assert np.max(np.abs(o.cpu().numpy() - ref16)) <= 2e-3


def test_write_and_decode_in_a_captured_graph_on_another_stream():
    rng = np.random.default_rng(9)
    lens, B, Hkv, d = [300, 41], 16, 2, 128
    kc, vc, sc = random_pool(rng, 30, B, Hkv, d)
    bt = tables_for(rng, lens, B, 30)
    kd, vd, sd, btd = up8(kc), up8(vc), up(sc), up(bt)
    sl = up(np.array(lens, np.int32))
    query = W.normal_bits((2, 8, d), "bf16", 9, 2)
    new = [W.normal_bits((2, Hkv, d), "bf16", 9, 3 + i) for i in range(2)]
    q, nk, nv = dev_bits(query, "bf16"), dev_bits(new[0], "bf16"), dev_bits(new[1], "bf16")
    slots = np.array([bt[s, (n - 1) // B] * B + (n - 1) % B for s, n in enumerate(lens)], np.int64)
    slot_t = up(slots)
    out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
    ws = pa.alloc_workspace(q, kd, btd, 32)

    def step():
        pa.reshape_and_cache_fp8(nk, nv, kd, vd, sd, slot_t)
        pa.decode_fp8(out, q, kd, vd, sd, btd, sl, 0.09, 32, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    # new inputs into the captured buffers: lengths shrink, rows change
    nk.copy_(nv)
    for n in ([300, 41], [77, 16]):
        sl.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        wk, wv, wsc = fp8.write_fp8(new[1], new[1], kc, vc, sc, slots, B, "bf16")
        assert np.array_equal(down8(kd), wk)
        K, V = fp8.pool_values(wk, wsc, 0), fp8.pool_values(wv, wsc, 1)
        ref = fp8.attend(query, K, V, bt, n, B, 0.09, "bf16")
        for s in range(2):
            tol = fp8.decode_bound(oracle.to_float64(query[s], "bf16"), oracle.gather_kv(K, bt[s], n[s], B),
                                   oracle.gather_kv(V, bt[s], n[s], B), 0.09, WEIGHT_ERROR)
            assert np.max(np.abs(out[s].double().cpu().numpy() - ref[s])) <= tol
    assert torch.isfinite(want).all()


# wide tables: neighbouring kv heads are taken 4 and 2 at a time
GROUPED = [
    # dtype, d, Hq, Hkv, B, lengths, table tokens
    ("bf16", 128, 32, 8, 16, [900, 33, 0, 1, 257, 64], 19456),
    ("fp16", 64, 12, 12, 8, [31, 700, 5, 64, 65], 16384),
    ("bf16", 128, 42, 6, 64, [1500, 1, 129, 0, 63, 64, 300], 11264),
    ("fp16", 64, 24, 2, 32, [40, 1030, 96, 513], 58880),
    ("bf16", 128, 16, 4, 4, [333, 20, 0, 129, 77, 3, 64, 65], 29184),
    ("fp16", 64, 4, 2, 1, [50, 260, 31, 33], 58880),
]


@pytest.mark.parametrize("idx", range(len(GROUPED)))
def test_decode_with_neighbouring_heads_together(idx):
    dtype, d, Hq, Hkv, B, lens, width = GROUPED[idx]
    rng = np.random.default_rng(100 + idx)
    NB = sum(-(-n // B) for n in lens) + 3
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    bt = tables_for(rng, lens, B, NB, MB=width // B)
    query = W.normal_bits((len(lens), Hq, d), dtype, 100 + idx, 2)
    check_decode(query, kc, vc, sc, bt, lens, B, 1 / np.sqrt(d), dtype, what=str(GROUPED[idx][:5]))


def test_decode_workspace_may_hold_anything():
    rng = np.random.default_rng(21)
    lens, B, Hkv, d = [2000, 1, 0, 513, 1024], 16, 2, 128
    kc, vc, sc = random_pool(rng, 300, B, Hkv, d)
    bt = tables_for(rng, lens, B, 300)
    query = W.normal_bits((5, 8, d), "bf16", 21, 2)
    n = pa.decode_fp8_workspace_bytes(5, 8, Hkv, d, bt.shape[1], B)
    first = None
    for byte in (0, 0xFF, 0x7F, 0x80):
        ws = torch.full((n,), byte, dtype=torch.uint8, device="cuda")
        o = check_decode(query, kc, vc, sc, bt, lens, B, 0.09, "bf16", ws=ws)
        first = o if first is None else first
        assert torch.equal(o, first)


def test_two_captured_graphs_on_one_workspace():
    rng = np.random.default_rng(22)
    B, Hkv, d = 16, 2, 64
    kc, vc, sc = random_pool(rng, 200, B, Hkv, d)
    kd, vd, sd = up8(kc), up8(vc), up(sc)
    made = []
    ws = torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device="cuda")
    for lens in ([1500, 40, 700], [1100, 0]):
        bt = tables_for(rng, lens, B, 200)
        q = dev_bits(W.normal_bits((len(lens), 8, d), "fp16", 22, len(lens)), "fp16")
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        args = (out, q, kd, vd, sd, up(bt), up(np.array(lens, np.int32)), 0.125, 0, ws)
        pa.decode_fp8(*args)
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.decode_fp8(*args)
        made.append((g, out, want, args))
    for _ in range(3):
        for g, out, want, _ in made:
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(out, want)


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(23)
    B, Hkv, d, lens = 16, 2, 128, [3000, 900, 2500]
    kc, vc, sc = random_pool(rng, 450, B, Hkv, d)
    bt = tables_for(rng, lens, B, 450)
    q = dev_bits(W.normal_bits((3, 8, d), "bf16", 23, 2), "bf16")
    kd, vd, sd, btd, sl = up8(kc), up8(vc), up(sc), up(bt), up(np.array(lens, np.int32))
    want = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pa.decode_fp8(want, q, kd, vd, sd, btd, sl, 0.09, 0, pa.alloc_workspace(q, kd, btd))
    outs = [torch.empty_like(want) for _ in range(2)]
    spaces = [pa.alloc_workspace(q, kd, btd) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, w, st in zip(outs, spaces, streams):
            pa.decode_fp8(o, q, kd, vd, sd, btd, sl, 0.09, 0, w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


# ------------------------------------------------------------ all together --
@pytest.mark.parametrize("dtype,B,Hq,Hkv,d", [("bf16", 16, 8, 2, 128), ("fp16", 8, 4, 4, 64), ("bf16", 2, 6, 3, 64)])
def test_serving_loop_on_an_8_bit_pool(dtype, B, Hq, Hkv, d):
    """Prompts written in chunks, each chunk's prefill over the context that is
    read back; forked candidates with copy-on-write; decode steps straight from
    the pool. Every output is checked against the values that the rows stand for."""
    rng = np.random.default_rng(B)
    NB, MB = 300, 256 // B
    bm = pa.BlockManager(NB, B, MB)
    kd, vd, sd = pa.alloc_fp8_cache(NB, B, Hkv, d)
    scale = 1 / np.sqrt(d)
    hist, made = {}, [0]

    def rows(n):
        made[0] += 2
        return [W.normal_bits((n, Hkv, d), dtype, 50, made[0] + i) for i in range(2)]

    def held(bits):
        codes, e = fp8.quantise_rows(oracle.to_float64(bits, dtype))
        return fp8.E4M3[codes] * np.exp2(e.astype(np.float64) - 127)[..., None]

    def write(requests, ks, vs):
        slots, copies = bm.append(requests)
        if copies:
            src, dst = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in zip(*copies))
            pa.copy_blocks_fp8(kd, vd, sd, src, dst)
        pa.reshape_and_cache_fp8(dev_bits(ks, dtype), dev_bits(vs, dtype), kd, vd, sd, up(slots))
        return len(copies)

    def decode(live):
        bt, lens = bm.block_tables(live)
        made[0] += 1
        query = W.normal_bits((len(live), Hq, d), dtype, 51, made[0])
        q, btd = dev_bits(query, dtype), up(bt)
        out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
        pa.decode_fp8(out, q, kd, vd, sd, btd, up(lens), scale, 32, pa.alloc_workspace(q, kd, btd, 32))
        G = Hq // Hkv
        for i, s in enumerate(live):
            K, V = (np.concatenate(x) for x in zip(*hist[s]))
            qf = oracle.to_float64(query[i], dtype)
            ref = np.concatenate([oracle.single_query_attention(qf[h * G:(h + 1) * G], K[:, h], V[:, h], scale)[0]
                                  for h in range(Hkv)])
            assert np.max(np.abs(out[i].double().cpu().numpy() - ref)) <= fp8.decode_bound(qf, K, V, scale, WEIGHT_ERROR)

    def prefill(s, ks, vs):
        """The chunk's causal attention over the whole context, read back as 16-bit blocks."""
        n = ks.shape[0]
        bt, lens = bm.block_tables([s])
        L = int(lens[0])
        blocks = -(-L // B)
        ctx = [torch.zeros(blocks * B, Hkv, d, dtype=TORCH_DTYPE[dtype], device="cuda") for _ in range(2)]
        pa.gather_cache_fp8(*ctx, kd, vd, sd, up(bt), up(lens), torch.zeros(1, dtype=torch.int64, device="cuda"))
        made[0] += 1
        query = W.normal_bits((n, Hq, d), dtype, 52, made[0])
        out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
        pools = [c.view(blocks, B, Hkv, d) for c in ctx]
        table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
        pa.prefill(out, dev_bits(query, dtype), *pools, table, up(lens), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                   n, scale)
        K, V = (oracle.round_to_dtype(np.concatenate(x), dtype).reshape(blocks and 1, L, Hkv, d) for x in zip(*hist[s]))
        ref = oracle.paged_prefill(query, K, V, np.zeros((1, 1), np.int32), [L], [0, n], L, scale, dtype)
        assert np.max(np.abs(out.cpu().numpy() - ref)) <= 2e-3

    live, copied = [], 0
    for n in (1, 37, 90):
        s = bm.new_sequence()
        hist[s] = []
        for part in (n // 2, n - n // 2):
            if part:
                ks, vs = rows(part)
                write([(s, part)], ks, vs)
                hist[s].append((held(ks), held(vs)))
                prefill(s, ks, vs)
        live.append(s)
    for p in list(live):
        c = bm.fork(p)
        hist[c] = list(hist[p])
        live.append(c)
    decode(live)
    for step in range(6):
        ks, vs = rows(len(live))
        copied += write([(s, 1) for s in live], ks, vs)
        for i, s in enumerate(live):
            hist[s].append((held(ks[i:i + 1]), held(vs[i:i + 1])))
        decode(live)
    assert copied > 0
    bm.close()
