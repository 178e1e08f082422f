"""Decode from the 4-bit cache on the GPU, against exact attention over the pool's values
with a bound derived from the arithmetic, and the 4-bit cache's pieces together as a
serving loop uses them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from gpu_util import TORCH_DTYPE, dev_bits, host_bits
from oracle import fp4, fp8
from test_fp4_cache_gpu import random_pool, tables_for, up

pytestmark = pytest.mark.gpu

# Weights' two parts. V's factors within 2^15 of the largest: fp16 parts of weights that are at least 2^6
# at the top, off by 2^-22 of themselves or 2^-25, 2^-31 of the largest weight; multiplied by the factor over
# half the largest, 2^(1 - 2 spread) or more, they are off by 2^-25 again, 2^(2 spread - 32) of what the largest
# weight leaves there. Over n tokens that is n times as much of the largest value (the sum of weights is at
# least the largest one). Otherwise the parts are bf16.
FAR = 2.0 ** -17


def weight_error(n, spread):
    return 2.0 ** -20 + n * (2.0 ** -31 + 2.0 ** (2 * spread - 32)) if 2 * spread <= 12 else FAR


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_305_gb300 import build
    build.build()
    pa.bad_index_count(clear=True)
    yield
    torch.cuda.synchronize()


def check_rows(got, query, K, V, scale, dtype, we, what=""):
    """One sequence's output [Hq, d] against exact attention over K, V [n, Hkv, d], every head and
    group of 32 dims by the bound of its own rows."""
    n, Hkv, d = K.shape
    q = oracle.to_float64(query, dtype)
    G = q.shape[0] // Hkv
    if n == 0:
        assert not got.any(), what
        return
    for h in range(Hkv):
        qh = q[h * G:(h + 1) * G]
        ref, _ = oracle.single_query_attention(qh, K[:, h], V[:, h], scale)
        for g in range(0, d, 32):
            tol = fp8.decode_bound(qh, K[:, h:h + 1], V[:, h:h + 1, g:g + 32], scale, we)
            err = np.max(np.abs(got[h * G:(h + 1) * G, g:g + 32] - ref[:, g:g + 32]))
            assert err <= tol, f"{what} head {h} dims {g}: {err} > {tol} ({n} tokens)"


def check_decode(query, kc, vc, sc, bt, lens, B, scale, dtype, pt=0, ws=None, what="", spread=3):
    """Both output types against the oracle; returns the fp32 output."""
    q = dev_bits(query, dtype)
    kd, vd, sd, btd, sl = up(kc), up(vc), up(sc), up(bt), up(np.asarray(lens, np.int32))
    if ws is None:
        ws = pa.alloc_workspace(q, kd, btd, pt)
    o32 = torch.full(query.shape, float("nan"), dtype=torch.float32, device="cuda")
    o16 = torch.empty_like(q)
    pa.decode_fp4(o32, q, kd, vd, sd, btd, sl, scale, pt, ws)
    pa.decode_fp4(o16, q, kd, vd, sd, btd, sl, scale, pt, ws)
    got = o32.double().cpu().numpy()
    Kp, Vp = fp4.pool_values(kc, sc, 0), fp4.pool_values(vc, sc, 1)
    for s, n in enumerate(np.minimum(lens, bt.shape[1] * B)):
        K, V = (oracle.gather_kv(p, bt[s], int(n), B) for p in (Kp, Vp))
        check_rows(got[s], query[s], K, V, scale, dtype, weight_error(n, spread), f"{what} sequence {s}")
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
    ("bf16", 64, 2, 1, 16, [40, 0, 0, 1], 0, 6),
    ("bf16", 64, 13, 1, 16, [3000, 2999], 0, 20),
    ("fp16", 128, 5, 5, 16, [5000], 0, 3),
    ("bf16", 128, 24, 3, 8, [1, 2, 63, 900], 0, 8),
    ("fp16", 64, 16, 2, 16, [770, 128], 0, 12),
]


@pytest.mark.parametrize("idx", range(len(GRID)))
def test_decode_grid(idx):
    dtype, d, Hq, Hkv, B, lens, pt, spread = GRID[idx]
    rng = np.random.default_rng(idx)
    NB = sum(-(-n // B) for n in lens) + 3
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d, spread)
    sc[:, :, 0] = np.where(sc[:, :, 0] > 0, rng.integers(123, 127, sc[:, :, 0].shape), 0)  # scores of ordinary size
    bt = tables_for(rng, lens, B, NB, MB=max(-(-max(lens) // B) + 1, 1))
    query = W.normal_bits((len(lens), Hq, d), dtype, idx, 2)
    check_decode(query, kc, vc, sc, bt, lens, B, 1 / np.sqrt(d), dtype, pt, what=str(GRID[idx]), spread=spread)


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
    check_decode(query, kc, vc, sc, bt, lens, B, 0.3 / np.sqrt(d), dtype, what=str(GROUPED[idx][:5]))


@pytest.mark.parametrize("d,B", [(64, 16), (128, 16), (128, 4), (64, 64)])
def test_decode_never_reads_past_the_length(d, B):
    # the largest codes and infinite factors in every slot that no sequence holds
    rng = np.random.default_rng(2)
    lens, Hkv = [1, 15, 16, 17, 31, 32, 33, 47, 0, 130], 2
    NB = sum(-(-n // B) for n in lens) + 3
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    bt = tables_for(rng, lens, B, NB)
    used = np.zeros((NB, B), bool)
    for s, n in enumerate(lens):
        for t in range(n):
            used[bt[s, t // B], t % B] = True
    kc[~used], vc[~used] = 0x7F, 0x70
    sc.transpose(0, 3, 1, 2, 4)[~used] = 255
    query = W.normal_bits((len(lens), 8, d), "bf16", 3, 2)
    check_decode(query, kc, vc, sc, bt, lens, B, 0.3 / np.sqrt(d), "bf16", max(32, B))


# every token counts: equal scores and whole values, so that one left out, taken twice or taken
# from another place shifts the sum by about 1 or more
EVERY = [
    # dtype, d, Hq, Hkv, B, lengths, table tokens, partition_tokens
    ("bf16", 128, 8, 2, 16, [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 0, 500], 512, 0),
    ("fp16", 64, 4, 4, 16, [5000, 1, 2047, 2048, 2049, 777], 8192, 64),
    ("bf16", 128, 32, 8, 16, [900, 33, 0, 1, 257, 64, 3000], 19456, 0),
    ("fp16", 64, 6, 6, 8, [31, 700, 5, 64, 65], 16384, 0),
    ("bf16", 64, 42, 6, 64, [1500, 1, 129, 0, 63, 64, 300], 11264, 0),
    ("fp16", 128, 16, 1, 32, [40, 1030, 96, 513], 2048, 0),
    ("bf16", 128, 16, 4, 4, [333, 20, 0, 129, 77, 3, 64, 65, 4000], 29184, 0),
    ("fp16", 64, 4, 2, 1, [50, 260, 31, 33, 1025], 58880, 0),
    ("bf16", 64, 5, 1, 2, [511, 513, 2, 1, 66], 1024, 0),
    ("bf16", 128, 4, 1, 16, [60000, 1], 65536, 0),
]


@pytest.mark.parametrize("idx", range(len(EVERY)))
def test_decode_takes_every_token_once(idx):
    dtype, d, Hq, Hkv, B, lens, width, pt = EVERY[idx]
    rng = np.random.default_rng(200 + idx)
    NB = sum(-(-n // B) for n in lens) + 3
    kc, _, sc = random_pool(rng, NB, B, Hkv, d)
    codes = rng.choice([2, 4, 5, 6, 7, 10, 12, 13, 14, 15], size=(NB, B, Hkv, d))  # +-1, 2, 3, 4, 6
    vc = fp4.pack(codes.astype(np.uint8))
    kc[:], sc[:, :, 0], sc[:, :, 1] = 0x22, 120, 127  # keys all alike
    bt = tables_for(rng, lens, B, NB, MB=width // B)
    query = W.normal_bits((len(lens), Hq, d), dtype, 200 + idx, 2)
    q, btd = dev_bits(query, dtype), up(bt)
    kd = up(kc)
    out = torch.full(query.shape, float("nan"), dtype=torch.float32, device="cuda")
    pa.decode_fp4(out, q, kd, up(vc), up(sc), btd, up(np.array(lens, np.int32)), 0.05, pt, pa.alloc_workspace(q, kd, btd))
    got, V = out.double().cpu().numpy(), fp4.pool_values(vc, sc, 1)
    for s, n in enumerate(lens):
        if n == 0:
            assert not got[s].any()
            continue
        total = oracle.gather_kv(V, bt[s], n, B).sum(0)  # whole numbers below 2^24
        off = np.abs(got[s] * n - np.repeat(total, Hq // Hkv, axis=0))
        # equal weights are exact and so are sums of whole numbers; joins and the quotient round: a few
        # times 2^-23 of the result, times n: 60000 * 6 * 2^-21 = 0.17
        assert np.max(off) <= 0.3, f"{EVERY[idx]} sequence {s}: {np.max(off)}"


def one_sequence(rng, n, d, Hkv=1, B=16, spread=2):
    NB = -(-n // B) + 2
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d, spread)
    sc[:, :, 0] = 125
    sc[sc == 0] = 125
    return kc, vc, sc, tables_for(rng, [n], B, NB)


def run(query, kc, vc, sc, bt, n, scale, dtype, ws=None):
    q, btd = dev_bits(query, dtype), up(bt)
    kd = up(kc)
    out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
    pa.decode_fp4(out, q, kd, up(vc), up(sc), btd, up(np.array([n], np.int32)), scale, 0,
                  ws if ws is not None else pa.alloc_workspace(q, kd, btd))
    return out.double().cpu().numpy()


def weighted_sizes(query, K, V, scale, dtype):
    """The exact result and sum p |V| of every output, and twice the relative error of a term."""
    q = oracle.to_float64(query[0], dtype)
    G = q.shape[0] // K.shape[1]
    ref, size = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(K.shape[1]):
        qh = q[h * G:(h + 1) * G]
        p = oracle.attention_weights(qh @ K[:, h].T * scale)
        ref[h * G:(h + 1) * G] = p @ V[:, h]
        size[h * G:(h + 1) * G] = p @ np.abs(V[:, h])
    return ref, size, fp8.decode_bound(q, K, np.ones_like(V), scale, FAR)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 1), (128, 8, 1), (128, 16, 1), (128, 6, 2)])
def test_decode_far_apart_factors(d, Hq, Hkv):
    # V's factors over 90 binades, each group for itself: every term keeps its bits
    rng = np.random.default_rng(d + Hq)
    n = 200
    kc, vc, sc, bt = one_sequence(rng, n, d, Hkv)
    sc[:, :, 1] = rng.integers(80, 170, sc[:, :, 1].shape)
    query = W.normal_bits((1, Hq, d), "fp16", 3, 2)
    got = run(query, kc, vc, sc, bt, n, 0.125, "fp16")
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, 16) for i, c in enumerate((kc, vc)))
    ref, size, rel = weighted_sizes(query, K, V, 0.125, "fp16")
    assert np.all(np.abs(got[0] - ref) <= size * rel)


@pytest.mark.parametrize("dtype,Hq", [("fp16", 4), ("bf16", 8), ("bf16", 12)])
@pytest.mark.parametrize("orders", [-60, -20, 30])
def test_decode_groups_of_unequal_size(dtype, Hq, orders):
    # one group of dims far smaller or larger than the others in every token
    rng = np.random.default_rng(4)
    n, d = 300, 128
    kc, vc, sc, bt = one_sequence(rng, n, d)
    sc[:, :, 1, :, 2] = 125 + orders
    query = W.normal_bits((1, Hq, d), dtype, 4, 2)
    got = run(query, kc, vc, sc, bt, n, 0.09, dtype)
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, 16) for i, c in enumerate((kc, vc)))
    check_rows(got[0], query[0], K, V, 0.09, dtype, FAR, f"{orders}")


@pytest.mark.parametrize("at", [0, 50, 299])
@pytest.mark.parametrize("orders", [13, 24, 80])
def test_decode_a_huge_row_of_no_weight_takes_no_bits(at, orders):
    rng = np.random.default_rng(5)
    n, d, B = 300, 64, 16
    kc, vc, sc, bt = one_sequence(rng, n, d)
    blk, off = bt[0, at // B], at % B
    sc[blk, 0, 1, off] = 125 + orders
    query = np.abs(oracle.to_float64(W.normal_bits((1, 3, d), "bf16", 5, 2), "bf16"))
    query = W.f32_to_bits((query + 1).astype(np.float32), "bf16")
    kc[blk, off] = 0xFF          # -6 in every element: the lowest score by far
    sc[blk, 0, 0, off] = 127
    got = run(query, kc, vc, sc, bt, n, 0.25, "bf16")
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, B) for i, c in enumerate((kc, vc)))
    ref, size, rel = weighted_sizes(query, K, V, 0.25, "bf16")
    assert np.all(np.abs(got[0] - ref) <= size * rel)


@pytest.mark.parametrize("n,Hq", [(40, 2), (700, 4), (700, 11)])
def test_decode_nan_reaches_its_own_outputs_alone(n, Hq):
    rng = np.random.default_rng(6)
    d, Hkv, B = 128, 2, 16
    Hq *= Hkv
    kc, vc, sc, bt = one_sequence(rng, n, d, Hkv)
    query = W.normal_bits((1, Hq, d), "bf16", 6, 2)
    clean = run(query, kc, vc, sc, bt, n, 0.09, "bf16")
    blk, off = bt[0, 17 // B], 17 % B
    v2, s2 = vc.copy(), sc.copy()
    v2[blk, off, 1, 16:32], s2[blk, 1, 1, off, 1] = 0, 255   # dims 32-63 of kv head 1
    got = run(query, kc, v2, s2, bt, n, 0.09, "bf16")
    hit = np.zeros(clean.shape, bool)
    hit[0, Hq // 2:, 32:64] = True
    assert np.array_equal(np.isnan(got), hit)
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, B) for i, c in enumerate((kc, vc)))
    V[17, 1, 32:64] = 0
    ref, size, rel = weighted_sizes(query, K, V, 0.09, "bf16")
    assert np.all((np.abs(got[0] - ref) <= size * rel)[~hit[0]])
    k2, s2 = kc.copy(), sc.copy()
    k2[blk, off, 0, 48:], s2[blk, 0, 0, off, 3] = 0, 255     # a key of kv head 0
    got = run(query, k2, vc, s2, bt, n, 0.09, "bf16")
    assert np.isnan(got[0, :Hq // 2]).all() and np.array_equal(got[0, Hq // 2:], clean[0, Hq // 2:])


@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -100, 2.0 ** 60, 2.0 ** 122])
def test_decode_bf16_queries_of_any_size(size):
    # a bf16 query far outside fp16's range keeps its bits, and K's factors meet it
    rng = np.random.default_rng(7)
    n, d = 70, 128
    kc, vc, sc, bt = one_sequence(rng, n, d, 2, 8)
    sc[:, :, 0] = np.clip(125 - int(np.log2(size)), 4, 250)
    q = rng.uniform(1, 2, (1, 6, d)) * rng.choice([-1, 1], (1, 6, d))
    query = W.f32_to_bits((q * size).astype(np.float32), "bf16")
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, 8) for i, c in enumerate((kc, vc)))
    got = run(query, kc, vc, sc, bt, n, 0.05, "bf16")
    check_rows(got[0], query[0], K, V, 0.05, "bf16", weight_error(n, 2), f"{size}")


@pytest.mark.parametrize("B", [16, 4])
def test_decode_slots_behind_a_sequence_do_not_reach_its_scores(B):
    # small keys with large queries, and the largest factors in the slots behind the last token
    rng = np.random.default_rng(17)
    n, d = 37, 64
    kc, vc, sc, bt = one_sequence(rng, n, d, 1, B)
    sc[:, :, 0] = 40
    last = bt[0, (n - 1) // B]
    sc[last, :, :, (n - 1) % B + 1:] = 250
    kc[last, (n - 1) % B + 1:] = 0x77
    q = rng.uniform(1, 2, (1, 4, d)) * rng.choice([-1, 1], (1, 4, d)) * 2.0 ** 85
    query = W.f32_to_bits(q.astype(np.float32), "bf16")
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, B) for i, c in enumerate((kc, vc)))
    got = run(query, kc, vc, sc, bt, n, 0.05, "bf16")
    check_rows(got[0], query[0], K, V, 0.05, "bf16", weight_error(n, 2))


def test_decode_queries_of_heads_far_apart():
    rng = np.random.default_rng(8)
    n, d = 100, 64
    kc, vc, sc, bt = one_sequence(rng, n, d)
    q = rng.standard_normal((1, 4, d)) * np.array([1, 2.0 ** -40, 2.0 ** 8, 2.0 ** -90])[None, :, None]
    query = W.f32_to_bits(q.astype(np.float32), "bf16")
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, 16) for i, c in enumerate((kc, vc)))
    got = run(query, kc, vc, sc, bt, n, 0.02, "bf16")
    for h in range(4):
        check_rows(got[0, h:h + 1], query[0, h:h + 1], K, V, 0.02, "bf16", weight_error(n, 2), f"{h}")


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.5])
@pytest.mark.parametrize("dtype,Hq,B", [("bf16", 8, 16), ("fp16", 14, 2)])
def test_decode_scales(scale, dtype, Hq, B):
    rng = np.random.default_rng(25)
    lens = [130, 1, 600]
    NB = sum(-(-n // B) for n in lens)
    kc, vc, sc = random_pool(rng, NB, B, 2, 64, 0)
    bt = tables_for(rng, lens, B, NB)
    check_decode(W.normal_bits((3, Hq, 64), dtype, 25, 2), kc, vc, sc, bt, lens, B, scale, dtype, spread=0)


@pytest.mark.parametrize("order", [4, 20, 60, 100])
def test_decode_equal_scores_weigh_the_same_however_large(order):
    rng = np.random.default_rng(9)
    n, d = 1000, 128
    kc, vc, sc, bt = one_sequence(rng, n, d)
    kc[:] = kc[0, 0]
    sc[:, :, 0] = 127 + order
    query = W.normal_bits((1, 4, d), "bf16", 9, 2)
    got = run(query, kc, vc, sc, bt, n, 1.0, "bf16")
    V = oracle.gather_kv(fp4.pool_values(vc, sc, 1), bt[0], n, 16)[:, 0]
    # n weights of 1, exact in every part; sums of n terms in fp32
    assert np.max(np.abs(got[0] - V.mean(0))) <= 2 * n * 2.0 ** -24 * np.abs(V).mean(0).max() + 2.0 ** -22 * np.abs(V).max()


def test_decode_zero_query_and_zero_pool():
    kd, vd, sd = pa.alloc_fp4_cache(4, 16, 1, 64)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((1, 1, 64), 3.0, dtype=torch.float32, device="cuda")
    bt, sl = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([50], dtype=torch.int32, device="cuda")
    pa.decode_fp4(out, q, kd, vd, sd, bt, sl, 1.0)
    assert not out.any()


def test_decode_length_one_returns_the_value_row():
    rng = np.random.default_rng(10)
    lens = [1, 1, 1]
    kc, vc, sc = random_pool(rng, 4, 16, 2, 128, 30)
    bt = tables_for(rng, lens, 16, 4)
    out = torch.empty(3, 6, 128, dtype=torch.float32, device="cuda")
    pa.decode_fp4(out, dev_bits(W.normal_bits((3, 6, 128), "fp16", 1, 1), "fp16"), up(kc), up(vc), up(sc), up(bt),
                  up(np.array(lens, np.int32)), 0.09)
    V = fp4.pool_values(vc, sc, 1)
    for s in range(3):
        assert np.array_equal(out[s].double().cpu().numpy(), np.repeat(V[bt[s, 0], 0], 3, axis=0))


def test_decode_bad_blocks_read_as_zeros_and_are_counted():
    rng = np.random.default_rng(6)
    for B in (16, 4):
        d, n = 64, 2 * B + 3
        kc, vc, sc = random_pool(rng, 6, B, 1, d)
        bt = np.array([[0, 77, 1], [2, 3, -1]], np.int32)
        query = W.normal_bits((2, 2, d), "bf16", 6, 2)
        pa.bad_index_count(clear=True)
        out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
        pa.decode_fp4(out, dev_bits(query, "bf16"), up(kc), up(vc), up(sc), up(bt),
                      up(np.array([n, n], np.int32)), 0.125)
        assert pa.bad_index_count(clear=True) > 0
        kz, vz, scz = (np.concatenate([x, np.zeros_like(x[:1])]) for x in (kc, vc, sc))
        btz = np.where((bt < 0) | (bt >= 6), 6, bt)
        K, V = fp4.pool_values(kz, scz, 0), fp4.pool_values(vz, scz, 1)
        for s in range(2):
            rows = [oracle.gather_kv(p, btz[s], n, B) for p in (K, V)]
            check_rows(out[s].double().cpu().numpy(), query[s], *rows, 0.125, "bf16", weight_error(n, 3))


def test_decode_lengths_out_of_range_are_clamped_and_counted():
    rng = np.random.default_rng(16)
    kc, vc, sc, bt = one_sequence(rng, 64, 64)
    bt2 = np.repeat(bt, 2, 0)
    query = W.normal_bits((2, 2, 64), "fp16", 6, 2)
    out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
    pa.bad_index_count(clear=True)
    pa.decode_fp4(out, dev_bits(query, "fp16"), up(kc), up(vc), up(sc), up(bt2), up(np.array([-3, 9999], np.int32)), 0.1)
    assert pa.bad_index_count(clear=True) == 2
    assert not out[0].any()
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], 64, 16) for i, c in enumerate((kc, vc)))
    check_rows(out[1].double().cpu().numpy(), query[1], K, V, 0.1, "fp16", weight_error(64, 3))


def test_decode_bit_identical_however_placed_and_repeated():
    rng = np.random.default_rng(7)
    lens, B, Hkv, d = [1200, 700, 2048], 16, 2, 128
    NB = 300
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    bt = tables_for(rng, lens, B, NB)
    query = W.normal_bits((3, 8, d), "bf16", 7, 2)
    a = check_decode(query, kc, vc, sc, bt, lens, B, 0.03, "bf16", 64)
    perm = rng.permutation(NB)
    inv = np.argsort(perm)
    b = check_decode(query, kc[perm], vc[perm], sc[perm], inv[bt].astype(np.int32), lens, B, 0.03, "bf16", 64)
    assert torch.equal(a, b)


@pytest.mark.parametrize("B", [64, 4])
def test_blocks_behind_32_bit_offsets(B):
    """The last blocks of a pool whose codes and exponent bytes both pass 2^32 bytes: written, copied, read
    back and attended as in a small pool, and nothing where their offsets would fall in 32 bits."""
    Hkv, d, dtype = 8, 128, "bf16"
    codes, exps = B * Hkv * d // 2, B * Hkv * d // 16  # bytes a block
    NB = 2 ** 32 // exps + 200
    if torch.cuda.mem_get_info()[0] < NB * (2 * codes + exps) + 2 ** 32:
        pytest.skip("too little free memory")
    big = (*(torch.empty(NB, B, Hkv, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)),
           torch.empty(NB, Hkv, 2, B, d // 32, dtype=torch.uint8, device="cuda"))
    few = 100
    small = pa.alloc_fp4_cache(few, B, Hkv, d)
    for x in small:
        x.fill_(0x77)
    last = NB - few  # block i of the small pool is block last + i of the large one
    wrapped = [(last * n % 2 ** 32) // n for n in (codes, codes, exps)]
    for x, at in zip(big, wrapped):
        x[last:].fill_(0x77)
        assert at + few < last
        x[at:at + few + 1].fill_(0x5A)

    lens = [B * 30 + 3, B * 25 + 1]
    rng = np.random.default_rng(B)
    bt = tables_for(rng, lens, B, few - 20)
    slots = np.concatenate([bt[s, np.arange(n) // B].astype(np.int64) * B + np.arange(n) % B for s, n in enumerate(lens)])
    T = len(slots)
    key, value = (dev_bits(W.normal_bits((T, Hkv, d), dtype, 51, i), dtype) for i in range(2))
    query = dev_bits(W.normal_bits((2, 32, d), dtype, 52, 0), dtype)
    src, dst = (np.arange(20) + x for x in (0, few - 20))
    lens_d, starts = up(np.array(lens, np.int32)), up(np.array([0, lens[0]], np.int64))
    seen = []
    for pool, first in ((small, 0), (big, last)):
        pa.reshape_and_cache_fp4(key, value, *pool, up(slots + first * B))
        pa.copy_blocks_fp4(*pool, up((src + first).astype(np.int32)), up((dst + first).astype(np.int32)))
        table = up((bt + first).astype(np.int32))
        rows = [torch.empty_like(key) for _ in range(2)]
        pa.gather_cache_fp4(*rows, *pool, table, lens_d, starts)
        out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
        pa.decode_fp4(out, query, *pool, table, lens_d, 0.1, workspace=pa.alloc_workspace(query, pool[0], table))
        seen.append((out, *rows, *(x[first:first + few] for x in pool)))
    assert all(torch.equal(a, b) for a, b in zip(*seen)) and not seen[0][0].isnan().any()
    for x, at in zip(big, wrapped):
        assert (x[at:at + few + 1] == 0x5A).all()


def test_workspace_may_hold_anything_and_is_shared():
    rng = np.random.default_rng(21)
    lens, B, Hkv, d = [2000, 1, 0, 513, 1024], 16, 2, 128
    kc, vc, sc = random_pool(rng, 300, B, Hkv, d)
    bt = tables_for(rng, lens, B, 300)
    query = W.normal_bits((5, 8, d), "bf16", 21, 2)
    n = max(pa.decode_fp4_workspace_bytes(5, 8, Hkv, d, bt.shape[1], B), pa.decode_workspace_bytes(4, 8, 64, 64, 16, 32))
    case = W.random_case(num_seqs=4, num_q_heads=8, num_kv_heads=Hkv, head_dim=64, block_size=B,
                         len_range=(1, 900), dtype="fp16", seed=9)
    ref16 = oracle.paged_decode(case.query, case.key_cache, case.value_cache, case.block_tables,
                                case.seq_lens, B, case.scale, "fp16")
    first = None
    for byte in (0, 0xFF, 0x7F, 0x80):
        ws = torch.full((n,), byte, dtype=torch.uint8, device="cuda")
        o = check_decode(query, kc, vc, sc, bt, lens, B, 0.03, "bf16", ws=ws)
        first = o if first is None else first
        assert torch.equal(o, first)
        o = torch.empty(case.query.shape, dtype=torch.float32, device="cuda")
        pa.decode(o, dev_bits(case.query, "fp16"), dev_bits(case.key_cache, "fp16"),
                  dev_bits(case.value_cache, "fp16"), up(case.block_tables), up(case.seq_lens), case.scale, 32, ws)
        assert np.max(np.abs(o.cpu().numpy() - ref16)) <= 2e-3


def test_two_captured_graphs_on_one_workspace():
    rng = np.random.default_rng(22)
    B, Hkv, d = 16, 2, 64
    kc, vc, sc = random_pool(rng, 200, B, Hkv, d)
    kd, vd, sd = up(kc), up(vc), up(sc)
    made = []
    ws = torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device="cuda")
    for lens in ([1500, 40, 700], [1100, 0]):
        bt = tables_for(rng, lens, B, 200)
        q = dev_bits(W.normal_bits((len(lens), 8, d), "fp16", 22, len(lens)), "fp16")
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        args = (out, q, kd, vd, sd, up(bt), up(np.array(lens, np.int32)), 0.05, 0, ws)
        pa.decode_fp4(*args)
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.decode_fp4(*args)
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
    kd, vd, sd, btd, sl = up(kc), up(vc), up(sc), up(bt), up(np.array(lens, np.int32))
    want = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pa.decode_fp4(want, q, kd, vd, sd, btd, sl, 0.03, 0, pa.alloc_workspace(q, kd, btd))
    outs = [torch.empty_like(want) for _ in range(2)]
    spaces = [pa.alloc_workspace(q, kd, btd) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, w, st in zip(outs, spaces, streams):
            pa.decode_fp4(o, q, kd, vd, sd, btd, sl, 0.03, 0, w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_stalled_ring_winds_down():
    # no stage is handed back: waits give up and are counted, and the library works on
    rng = np.random.default_rng(24)
    n, d = 4000, 128
    kc, vc, sc, bt = one_sequence(rng, n, d)
    q = dev_bits(W.normal_bits((1, 4, d), "bf16", 23, 2), "bf16")
    kd, vd, sd, btd, sl = up(kc), up(vc), up(sc), up(bt), up(np.array([n], np.int32))
    ws = pa.alloc_workspace(q, kd, btd)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    want = pa.decode_fp4(out.clone(), q, kd, vd, sd, btd, sl, 0.03, 1024, ws)
    pa.testing_decode_fp4_stalled(out, q, kd, vd, sd, btd, sl, 0.03, 1024, ws)
    torch.cuda.synchronize()
    assert pa.wait_timeout_count(clear=True) > 0
    pa.decode_fp4(out, q, kd, vd, sd, btd, sl, 0.03, 1024, ws)
    assert torch.equal(out, want) and pa.wait_timeout_count() == 0


@pytest.mark.parametrize("dtype,d,Hq,Hkv,B", [("bf16", 128, 8, 2, 16), ("fp16", 64, 4, 4, 16), ("bf16", 64, 11, 1, 8),
                                              ("fp16", 128, 6, 1, 4)])
def test_decode_values_under_exponent_zero_are_zeros(dtype, d, Hq, Hkv, B):
    # codes of every kind whose exponents alone were cleared
    rng = np.random.default_rng(30)
    lens = [1, 31, 64, 65, 700]
    NB = sum(-(-n // B) for n in lens)
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d)
    sc[:, :, 1] = 0
    bt = tables_for(rng, lens, B, NB)
    o32 = check_decode(W.normal_bits((5, Hq, d), dtype, 30, 2), kc, vc, sc, bt, lens, B, 0.05, dtype)
    assert not o32.any()


@pytest.mark.parametrize("d,Hq,B", [(128, 4, 16), (64, 8, 16), (128, 12, 4)])
@pytest.mark.parametrize("top", [1, 5, 10, 15, 16, 17])
def test_decode_exponents_next_to_zero(d, Hq, B, top):
    # V's bytes 0 .. top with the largest code under every byte 0; equal weights, so that a factor of 2^-127 in the
    # place of zero shows: half of 6 2^-127 against a bound of about 2^-17 of 6 2^(top - 127)
    rng = np.random.default_rng(31)
    n = 40
    kc, vc, sc, bt = one_sequence(rng, n, d, 1, B)
    e = rng.integers(0, top + 1, sc[:, :, 1].shape).astype(np.uint8)
    sc[:, :, 1] = np.where(rng.random(e.shape) < 0.5, 0, e)
    codes = fp4.unpack(vc).reshape(*vc.shape[:-1], d // 32, 32)
    codes[sc[:, :, 1].transpose(0, 2, 1, 3) == 0] = 7
    codes[bt[0, 0], 0], sc[bt[0, 0], :, 1, 0] = 7, top  # the largest value, in every group
    vc = fp4.pack(codes.reshape(*vc.shape[:-1], d))
    query = W.f32_to_bits(np.zeros((1, Hq, d), np.float32), "bf16")
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, B) for i, c in enumerate((kc, vc)))
    # every group of V holds the largest factor: errors of 2^-31 and 2^-32 a token, of the largest value
    got = run(query, kc, vc, sc, bt, n, 0.1, "bf16")
    check_rows(got[0], query[0], K, V, 0.1, "bf16", weight_error(n, 0), f"{top}")


@pytest.mark.parametrize("Hq,B", [(4, 16), (8, 16), (11, 4)])
def test_decode_exponent_255_is_nan_whatever_its_codes(Hq, B):
    rng = np.random.default_rng(32)
    n, d, at = 100, 128, 37
    kc, vc, sc, bt = one_sequence(rng, n, d, 1, B)
    query = np.abs(oracle.to_float64(W.normal_bits((1, Hq, d), "bf16", 32, 2), "bf16"))
    query = W.f32_to_bits(query.astype(np.float32), "bf16")
    blk, off = bt[0, at // B], at % B
    hit = np.zeros((1, Hq, d), bool)
    hit[..., 64:96] = True
    random = rng.integers(0, 256, 16).astype(np.uint8)
    for codes in (random, 0x77, 0xFF, 0):
        v2, s2 = vc.copy(), sc.copy()
        v2[blk, off, 0, 32:48], s2[blk, 0, 1, off, 2] = codes, 255
        assert np.array_equal(np.isnan(run(query, kc, v2, s2, bt, n, 0.09, "bf16")), hit)
        k2, s2 = kc.copy(), sc.copy()
        k2[blk, off, 0, 32:48], s2[blk, 0, 0, off, 2] = codes, 255
        assert np.isnan(run(query, k2, vc, s2, bt, n, 0.09, "bf16")).all()


@pytest.mark.parametrize("order", [30, 80, 95, 115])
@pytest.mark.parametrize("Hq,at", [(4, 5), (8, 33), (12, 63)])
def test_decode_a_huge_key_leaves_the_others_their_scores(Hq, at, order):
    # bf16 queries of about 2^order and keys that make scores of ordinary size with them, beside one key
    # whose score is far below any that counts, and one whose huge group meets zeros of the query
    rng = np.random.default_rng(33)
    n, d, B, far = 64, 128, 16, 20
    kc, vc, sc, bt = one_sequence(rng, n, d)
    sc[:, :, 0] = 125 - order
    q = rng.uniform(1, 2, (1, Hq, d)) * 2.0 ** order
    q[..., 96:] = 0
    query = W.f32_to_bits(q.astype(np.float32), "bf16")
    blk, off = bt[0, at // B], at % B
    kc[blk, off], sc[blk, 0, 0, off] = 0xFF, 200   # -6 2^73 in every element
    sc[bt[0, far // B], 0, 0, far % B, 3] = 230
    K, V = (oracle.gather_kv(fp4.pool_values(c, sc, i), bt[0], n, B) for i, c in enumerate((kc, vc)))
    got = run(query, kc, vc, sc, bt, n, 0.05, "bf16")
    ref, _ = oracle.single_query_attention(q := oracle.to_float64(query[0], "bf16"), K[:, 0], V[:, 0], 0.05)
    rest = np.delete(K, at, 0)
    rest[..., 96:] = 0  # their products are zeros
    tol = fp8.decode_bound(q, rest, np.delete(V, at, 0), 0.05, weight_error(n, 2))
    assert np.max(np.abs(got[0] - ref)) <= tol


# ------------------------------------------------------------ all together --
@pytest.mark.parametrize("dtype,B,Hq,Hkv,d", [("bf16", 16, 8, 2, 128), ("fp16", 8, 4, 4, 64), ("bf16", 2, 6, 3, 64)])
def test_serving_loop_on_a_4_bit_pool(dtype, B, Hq, Hkv, d):
    """Prompts written in chunks, each chunk's prefill over the context that is read back; forked
    candidates with copy-on-write; decode steps straight from the pool. Every output is checked
    against the values that the rows stand for."""
    rng = np.random.default_rng(B)
    NB, MB = 300, 256 // B
    bm = pa.BlockManager(NB, B, MB)
    pool = pa.alloc_fp4_cache(NB, B, Hkv, d)
    scale = 1 / np.sqrt(d)
    hist, made = {}, [0]

    def rows(n):
        made[0] += 2
        return [W.normal_bits((n, Hkv, d), dtype, 50, made[0] + i) for i in range(2)]

    def held(bits):
        return fp4.row_values(*fp4.quantise_rows(oracle.to_float64(bits, dtype)))

    def write(requests, ks, vs):
        slots, copies = bm.append(requests)
        if copies:
            src, dst = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in zip(*copies))
            pa.copy_blocks_fp4(*pool, src, dst)
        pa.reshape_and_cache_fp4(dev_bits(ks, dtype), dev_bits(vs, dtype), *pool, up(slots))
        return len(copies)

    def decode(live):
        bt, lens = bm.block_tables(live)
        made[0] += 1
        query = W.normal_bits((len(live), Hq, d), dtype, 51, made[0])
        q, btd = dev_bits(query, dtype), up(bt)
        out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
        pa.decode_fp4(out, q, *pool, btd, up(lens), scale, 32, pa.alloc_workspace(q, pool[0], btd, 32))
        for i, s in enumerate(live):
            K, V = (np.concatenate(x) for x in zip(*hist[s]))
            check_rows(out[i].double().cpu().numpy(), query[i], K, V, scale, dtype, weight_error(len(K), 5))

    def prefill(s, ks):
        """The chunk's causal attention over the whole context, read back as 16-bit blocks."""
        n = ks.shape[0]
        bt, lens = bm.block_tables([s])
        L = int(lens[0])
        blocks = -(-L // B)
        ctx = [torch.zeros(blocks * B, Hkv, d, dtype=TORCH_DTYPE[dtype], device="cuda") for _ in range(2)]
        pa.gather_cache_fp4(*ctx, *pool, up(bt), up(lens), torch.zeros(1, dtype=torch.int64, device="cuda"))
        made[0] += 1
        query = W.normal_bits((n, Hq, d), dtype, 52, made[0])
        out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
        pools = [c.view(blocks, B, Hkv, d) for c in ctx]
        table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
        pa.prefill(out, dev_bits(query, dtype), *pools, table, up(lens), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                   n, scale)
        K, V = (oracle.round_to_dtype(np.concatenate(x), dtype).reshape(1, L, Hkv, d) for x in zip(*hist[s]))
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
                prefill(s, ks)
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
