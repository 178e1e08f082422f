"""The streaming decode kernel, the prefix pass and the merge where they could go wrong
unseen: waits that run out, the ends of the types' ranges, small weights beside large ones,
long sums, single tokens, NaN."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from gpu_util import dev_bits
from oracle import fp8
from test_fp8_cache_gpu import down8, random_pool, tables_for, up, up8
from test_shared_prefix_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_305_gb300 import build
    build.build()
    pa.wait_timeout_count(clear=True)
    yield
    torch.cuda.synchronize()
    assert pa.wait_timeout_count(clear=True) == 0


# ------------------------------------------------------ waits that run out --
def rows_in_range(ws, rows, slots):
    """Every row's entry (first slot, number of pieces) at the start of the workspace names slots that exist."""
    first, pieces = ws[:8 * rows].view(torch.int32).view(rows, 2).long().unbind(1)
    cut = pieces != 0
    return bool(((pieces >= 0) & (pieces <= 456)).all()) and bool(
        ((first >= 0) & (first + pieces <= slots))[cut].all())


@pytest.mark.parametrize("B", [16, 4])
def test_8_bit_decode_whose_waits_run_out_ends_and_is_counted(B):
    # some 90 short rows a CTA: the wait gives up in the first rows of its share, and
    # the merge kernel has to find an entry for the others too, whatever the workspace held
    rng = np.random.default_rng(B)
    S, Hq, Hkv, d, NB = 40000, 2, 1, 64, 64
    lens = rng.integers(1, 40, S).astype(np.int32)
    lens[::1000] = 700
    kc, vc, sc = random_pool(rng, NB, B, Hkv, d, 1)
    bt = torch.randint(0, NB, (S, 1024 // B), dtype=torch.int32, device="cuda")
    q = dev_bits(W.normal_bits((S, Hq, d), "bf16", B, 2), "bf16")
    n = pa.decode_fp8_workspace_bytes(S, Hq, Hkv, d, 1024 // B, B)
    assert n > 0
    args = (q, up8(kc), up8(vc), up(sc), bt, up(lens), 0.125, 0)
    fresh = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pa.decode_fp8(fresh, *args, torch.zeros(n, dtype=torch.uint8, device="cuda"))
    pa.wait_timeout_count(clear=True)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    pa.testing_decode_fp8_stalled(torch.empty_like(fresh), *args, ws)
    assert pa.wait_timeout_count(clear=True) >= 1
    assert rows_in_range(ws, S * Hkv, S * Hkv + 456)
    out = torch.full_like(fresh, float("nan"))
    pa.decode_fp8(out, *args, ws)
    assert torch.equal(out, fresh)
    assert pa.wait_timeout_count(clear=True) == 0


def test_shared_prefix_decode_whose_waits_run_out_ends_and_is_counted():
    case = Case("bf16", 128, 8, 2, 16, [0, 100, 103], [600, 50], [600 + 20 * i for i in range(100)] + [50, 51, 900])
    assert case.passes()
    fresh = case.run()
    n = pa.decode_shared_prefix_workspace_bytes(103, 2, 8, 2, 128, case.bt.shape[1], 16, 600, 100)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    pa.wait_timeout_count(clear=True)
    pa.testing_decode_shared_prefix_stalled(torch.empty_like(fresh), case.q, case.kd, case.vd, case.btd, case.sl,
                                            case.gs, case.pl, 600, 100, case.scale, ws)
    assert pa.wait_timeout_count(clear=True) >= 1
    assert rows_in_range(ws, 103 * 2, 103 * 2 + 456)
    assert torch.equal(case.run(ws), fresh)
    assert pa.wait_timeout_count(clear=True) == 0


# -------------------------------------------------- the ends of the ranges --
def decode8(query, kc, vc, sc, bt, lens, B, scale, dtype):
    """fp32 outputs of the kernel and the exact ones, both float64."""
    q, kd, btd = dev_bits(query, dtype), up8(kc), up(bt)
    out = torch.full(query.shape, float("nan"), dtype=torch.float32, device="cuda")
    pa.decode_fp8(out, q, kd, up8(vc), up(sc), btd, up(np.asarray(lens, np.int32)), scale, 0,
                  pa.alloc_workspace(q, kd, btd))
    ref = fp8.attend(query, fp8.pool_values(kc, sc, 0), fp8.pool_values(vc, sc, 1), bt, lens, B, scale, dtype)
    return out.double().cpu().numpy(), ref


@pytest.mark.parametrize("dtype,Hq,B,n", [("bf16", 4, 16, 90), ("fp16", 9, 4, 700)])
def test_8_bit_values_next_to_the_smallest(dtype, Hq, B, n):
    # V rows with exponent bytes 1 to 7, as rows of bf16 numbers below 3.4e-34 have
    rng = np.random.default_rng(n)
    d = 64
    kc, vc, sc = random_pool(rng, -(-n // B), B, 1, d, 1)
    sc[:, :, 1] = rng.integers(1, 8, sc[:, :, 1].shape)
    bt = tables_for(rng, [n], B, kc.shape[0])
    query = W.normal_bits((1, Hq, d), dtype, n, 2)
    got, ref = decode8(query, kc, vc, sc, bt, [n], B, 0.01, dtype)
    K, V = (oracle.gather_kv(fp8.pool_values(c, sc, i), bt[0], n, B) for i, c in enumerate((kc, vc)))
    bound = fp8.decode_bound(oracle.to_float64(query[0], dtype), K, V, 0.01, 2.0 ** -20)
    # pieces, their products with the merge's weights and the sum round to the subnormal
    # grid: 2^-150 each, of at most two stages a piece (64 tokens a stage at least)
    assert np.max(np.abs(got - ref)) <= bound + (3 * (-(-n // 64)) + 2) * 2.0 ** -150
    assert np.max(np.abs(ref)) > 10 * bound  # zeros in the place of the result would be seen


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,size,B", [("fp16", 2.0 ** 15, 16), ("bf16", 2.0 ** 20, 4), ("bf16", 2.0 ** 58, 16)])
def test_8_bit_decode_of_equal_scores_of_any_size(dtype, size, B, sign):
    # the scores of all tokens are 2^30 and more, and equal: the result is the mean of V
    rng = np.random.default_rng(B)
    lens, Hkv, d = [1, 33, 700], 2, 64
    kc, vc, sc = random_pool(rng, sum(-(-n // B) for n in lens), B, Hkv, d, 1)
    kc[:] = 0x78 | (0x80 if sign < 0 else 0)  # 256
    sc[:, :, 0] = 127 - 8 + int(np.log2(size))
    bt = tables_for(rng, lens, B, kc.shape[0])
    query = W.f32_to_bits(np.full((3, 4, d), size, np.float32), dtype)
    got, ref = decode8(query, kc, vc, sc, bt, lens, B, 0.125, dtype)
    V = np.max(np.abs(fp8.pool_values(vc, sc, 1)))
    # equal weights: sums of n rows, which the tensor core may cut off, and pieces joined by
    # the sums of their weights
    assert np.max(np.abs(got - ref)) <= V * (2 * 700 * 2.0 ** -23 + 2.0 ** -18)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("members", [3, 150])
@pytest.mark.parametrize("dtype,size", [("fp16", 2.0 ** 15), ("bf16", 2.0 ** 20), ("bf16", 2.0 ** 57)])
def test_shared_prefix_of_equal_scores_of_any_size(dtype, size, members, sign):
    case = Case(dtype, 64, 8, 2, 16, [0, members], [700], [700 + i % 70 for i in range(members)])
    assert case.passes() == (members > 3)
    case.scale = 0.125
    case.query = W.f32_to_bits(np.full(case.query.shape, size, np.float32), dtype)
    case.kc = W.f32_to_bits(np.full(case.kc.shape, sign * size, np.float32), dtype)
    got = case.run().double().cpu().numpy()
    ref = fp8.shared_prefix_decode(case.query, case.kc, case.vc, case.bt, case.lens, case.starts, case.prefixes,
                                   case.B, case.scale, dtype)
    V = np.max(np.abs(oracle.to_float64(case.vc, dtype)))
    assert np.max(np.abs(got - ref)) <= V * (2 * 770 * 2.0 ** -23 + 2.0 ** -18)


@pytest.mark.parametrize("B,Hq", [(16, 4), (2, 10)])
def test_8_bit_decode_of_small_bf16_queries_and_large_keys(B, Hq):
    # scores of ordinary size from queries near 2^-118 and keys near 2^118
    rng = np.random.default_rng(B)
    lens, d = [70, 600], 64
    kc, vc, sc = random_pool(rng, sum(-(-n // B) for n in lens), B, 1, d, 2)
    sc[:, :, 0] += 118
    bt = tables_for(rng, lens, B, kc.shape[0])
    query = W.f32_to_bits((rng.standard_normal((2, Hq, d)) * 2.0 ** -118).astype(np.float32), "bf16")
    got, ref = decode8(query, kc, vc, sc, bt, lens, B, 0.125, "bf16")
    for s, n in enumerate(lens):
        K, V = (oracle.gather_kv(fp8.pool_values(c, sc, i), bt[s], n, B) for i, c in enumerate((kc, vc)))
        assert np.max(np.abs(got[s] - ref[s])) <= fp8.decode_bound(oracle.to_float64(query[s], "bf16"), K, V, 0.125,
                                                                   2.0 ** -20)


@pytest.mark.parametrize("B,Hq", [(16, 4), (2, 10)])
def test_8_bit_decode_of_large_bf16_queries_and_small_keys(B, Hq):
    rng = np.random.default_rng(B)
    lens, d = [70, 600], 64
    kc, vc, sc = random_pool(rng, sum(-(-n // B) for n in lens), B, 1, d, 2)
    sc[:, :, 0] = 1 + sc[:, :, 0] % 3
    bt = tables_for(rng, lens, B, kc.shape[0])
    query = W.f32_to_bits((rng.standard_normal((2, Hq, d)) * 2.0 ** 122).astype(np.float32), "bf16")
    got, ref = decode8(query, kc, vc, sc, bt, lens, B, 0.125, "bf16")
    for s, n in enumerate(lens):
        K, V = (oracle.gather_kv(fp8.pool_values(c, sc, i), bt[s], n, B) for i, c in enumerate((kc, vc)))
        assert np.max(np.abs(got[s] - ref[s])) <= fp8.decode_bound(oracle.to_float64(query[s], "bf16"), K, V, 0.125,
                                                                   2.0 ** -20)


# ---------------------------------------------------- weights of any size --
LN2 = float(np.float32(np.log(2.0)))  # this scale makes whole scores powers of two


@pytest.mark.parametrize("at", [0, 150, -1])
@pytest.mark.parametrize("dtype,B,n,Hq", [("bf16", 16, 200, 4), ("fp16", 4, 200, 9), ("fp16", 16, 1500, 3)])
@pytest.mark.parametrize("binades", [12, 24, 40])
def test_8_bit_decode_with_a_huge_row_of_negligible_weight(binades, dtype, B, n, Hq, at):
    # one token has a V factor 2^binades above the others' and a softmax weight of 2^-60
    # of theirs: the others keep their bits
    rng = np.random.default_rng(n + binades)
    d = 64
    kc, vc, sc = random_pool(rng, -(-n // B), B, 1, d, 0)
    bt = tables_for(rng, [n], B, kc.shape[0])
    sc[:, :, 0] = 127 - 10  # scores of others: of the order of one
    kc[..., 0] = 0
    t = at % n
    blk, off = bt[0, t // B], t % B
    kc[blk, off] = 0
    kc[blk, off, 0, 0] = 0xF4          # -192
    sc[blk, 0, 0, off] = 127
    sc[blk, 0, 1, off] += binades
    q = rng.standard_normal((1, Hq, d)) * 0.02
    q[..., 0] = 0.3125                 # 0.3125 * -192 = -60
    query = W.f32_to_bits(q.astype(np.float32), dtype)
    got, ref = decode8(query, kc, vc, sc, bt, [n], B, LN2, dtype)
    K, V = (oracle.gather_kv(fp8.pool_values(c, sc, i), bt[0], n, B) for i, c in enumerate((kc, vc)))
    qf = oracle.to_float64(query[0], dtype)
    p = oracle.attention_weights(qf @ K[:, 0].T * LN2)
    assert np.all(p[:, t] < 2.0 ** -55 * p.max(axis=1))
    size = np.max(p @ np.abs(V[:, 0]))
    factor = np.exp2(np.array([float(sc[bt[0, i // B], 0, 1, i % B]) for i in range(n)]) - 127)
    # the bound with the weighted rows' size in the place of max |V|; what falls below fp16's
    # grid, 2^-31 of the largest weighted factor for each token, times a code
    rel = fp8.decode_bound(qf, K, np.ones_like(V), LN2, 2.0 ** -20)
    assert np.max(np.abs(got - ref)) <= size * rel + n * 2.0 ** -31 * np.max(p * factor) * 448
    assert np.max(np.abs(ref)) > 0.01 * size


@pytest.mark.parametrize("low", [-27, -31])
@pytest.mark.parametrize("members,dtype", [(2, "fp16"), (60, "fp16"), (60, "bf16"), (2, "bf16")])
def test_shared_prefix_with_a_dominating_token_without_a_value(members, dtype, low):
    # the first token takes nearly all of the weight and has V = 0: the result is
    # the small weights of all others, 2^-27 and 2^-31 of the first one's
    n, d = 3000, 64
    case = Case(dtype, d, 16, 2, 16, [0, members], [2500], [n + i for i in range(members)])
    assert case.passes() == (members > 2)
    K, V = np.zeros(case.kc.shape), np.random.default_rng(1).integers(1, 9, case.vc.shape).astype(np.float64)
    K[..., 0] = low
    for s in range(members):
        K[case.bt[s, 0], 0], V[case.bt[s, 0], 0] = 0, 0
    q = np.zeros(case.query.shape)
    q[..., 0] = 1
    case.scale = LN2
    case.query, case.kc, case.vc = (W.f32_to_bits(x.astype(np.float32), dtype) for x in (q, K, V))
    got = case.run().double().cpu().numpy()
    ref = fp8.shared_prefix_decode(case.query, case.kc, case.vc, case.bt, case.lens, case.starts, case.prefixes,
                                   case.B, case.scale, dtype)
    # a weight's relative error (exponent, exp2, parts), sums of n terms twice, and
    # pieces joined at references of up to 32 in size (2^-18)
    rel = 2 * (32 * 2.0 ** -24 + 2.0 ** -21 + 2 * (n + 60) * 2.0 ** -24 + 2.0 ** -18)
    assert np.max(np.abs(got - ref)) <= rel * np.max(ref)


# ------------------------------------------------------------- long sums --
@pytest.mark.parametrize("op,dtype", [("8-bit", "bf16"), ("8-bit", "fp16"), ("prefix", "fp16")])
def test_sums_of_long_rows_do_not_drift(op, dtype):
    # positive values of many bits: 456 rows, one for each CTA, which a warp adds up in
    # n / 128 (16-bit: n / 64) steps. Rounded to nearest, a sum of k terms is off by
    # 6 sqrt(k) 2^-24 of itself at most but once in 10^7 (the roundings are as good as
    # independent, each below half an ulp); sums that are cut off at every step are too
    # small by about k 2^-25.
    S, d, B, n, NB = 456, 64, 16, 131072, 64
    steps = n // 128 if op == "8-bit" else n // 64
    rng = np.random.default_rng(3)
    bt = (torch.arange(n // B, device="cuda") % NB).to(torch.int32).repeat(S, 1)
    lens = torch.full((S,), n, dtype=torch.int32, device="cuda")
    K = np.zeros((NB, B, 1, d), np.float32)
    K[..., 0] = rng.uniform(-3, 0, K.shape[:3])
    V = rng.uniform(0.5, 2, K.shape).astype(np.float32)
    q = np.zeros((S, 1, d), np.float32)
    q[..., 0] = 1
    q, k, v = (dev_bits(W.f32_to_bits(x, dtype), dtype) for x in (q, K, V))
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    if op == "8-bit":
        pool = pa.alloc_fp8_cache(NB, B, 1, d)
        pa.reshape_and_cache_fp8(k.view(-1, 1, d), v.view(-1, 1, d), *pool, torch.arange(NB * B, device="cuda"))
        pa.decode_fp8(out, q, *pool, bt, lens, LN2, 0, pa.alloc_workspace(q, pool[0], bt))
        kc, vc, sc = down8(pool[0]), down8(pool[1]), pool[2].cpu().numpy()
        K, V = fp8.pool_values(kc, sc, 0), fp8.pool_values(vc, sc, 1)
    else:
        starts, none = torch.arange(S + 1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
        pa.decode_shared_prefix(out, q, k, v, bt, lens, starts, none, 0, 1, LN2,
                                pa.alloc_shared_prefix_workspace(q, k, bt, starts, 0, 1))
        K, V = (x.double().cpu().numpy() for x in (k, v))
    p = np.exp(K[:, :, 0, 0] * LN2)[..., None]
    ref = (p * V[:, :, 0]).sum((0, 1)) / p.sum()
    rel = np.abs(out.double().cpu().numpy() / ref - 1)
    # both sums, the products of a tile (2^-21), a weight and its parts (2^-21), the
    # joining of warps and pieces and the quotient
    assert np.max(rel) <= 2 * 6 * np.sqrt(steps) * 2.0 ** -24 + 2 * 2.0 ** -21 + 8 * 2.0 ** -23


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_sums_of_long_prefixes_do_not_drift(dtype):
    # 300 pairs of sequences behind 131072 tokens, in whole waves of CTAs of any chunk
    # length. A piece of at most 8192 tokens adds up 8 products for each 64 of them, and
    # the tensor core may cut off: 2^-23 of the sum at each addition, as decode_bound has it
    S, d, B, n, NB = 600, 64, 16, 131072, 64
    rng = np.random.default_rng(4)
    bt = (torch.arange(n // B, device="cuda") % NB).to(torch.int32).repeat(S, 1)
    lens = torch.full((S,), n, dtype=torch.int32, device="cuda")
    K = np.zeros((NB, B, 1, d), np.float32)
    K[..., 0] = rng.uniform(-3, 0, K.shape[:3])
    V = rng.uniform(0.5, 2, K.shape).astype(np.float32)
    q = np.zeros((S, 1, d), np.float32)
    q[..., 0] = 1
    q, k, v = (dev_bits(W.f32_to_bits(x, dtype), dtype) for x in (q, K, V))
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    starts = torch.arange(0, S + 1, 2, dtype=torch.int32, device="cuda")
    prefixes = torch.full((S // 2,), n, dtype=torch.int32, device="cuda")
    pa.decode_shared_prefix(out, q, k, v, bt, lens, starts, prefixes, n, 2, LN2,
                            pa.alloc_shared_prefix_workspace(q, k, bt, starts, n, 2))
    K, V = (x.double().cpu().numpy() for x in (k, v))
    p = np.exp(K[:, :, 0, 0] * LN2)[..., None]
    ref = (p * V[:, :, 0]).sum((0, 1)) / p.sum()
    rel = np.abs(out.double().cpu().numpy() / ref - 1)
    # a weight's parts: 2^-16 at most for bf16, of random sign for each token
    assert np.max(rel) <= 1024 * 2.0 ** -23 + (2.0 ** -18 if dtype == "bf16" else 2.0 ** -21) + 8 * 2.0 ** -23


# ------------------------------------------------------- every token once --
# All scores are equal and the values whole numbers from -8 to 8: a result is the mean of
# its tokens' values, and one token left out, or taken twice, moves it by |V_t - mean| / n.
# Each test checks that every token's part is well above the tolerance. Slots that do not
# belong to the row hold a score 2^5 higher and NaN.
def mean_tolerance(n, chain):
    """For sums of n weights and rows in chains of n / chain additions, each off by
    6 sqrt(steps) 2^-24 (see above), pieces joined likewise; exp2, parts, quotient."""
    return 8 * (2 * 6 * (np.sqrt(n / chain) + np.sqrt(n / 64)) * 2.0 ** -24 + 4 * 2.0 ** -21 + 8 * 2.0 ** -23)


def check_means(got, values, chain, what, cut=0.0):
    """got [Hq, d] against the means of values [n, Hkv, d]."""
    n, Hkv, d = values.shape
    mean = values.mean(0) if n else np.zeros((Hkv, d))
    tol = mean_tolerance(n, chain) + 8 * cut
    if n > 1:
        part = np.abs(values - mean).max(2).min() / (n - 1)
        assert part > 1.5 * tol, (what, part, tol)
    err = np.max(np.abs(got - np.repeat(mean, got.shape[0] // Hkv, axis=0)))
    assert err <= tol, (what, err, tol)


ONCE = [
    # dtype, d, Hq, Hkv, B, lengths, partition_tokens, table tokens
    ("fp16", 128, 5, 5, 16, [5000], 0, None),
    ("bf16", 64, 13, 1, 16, [3000, 2999], 0, None),
    ("fp16", 128, 64, 8, 16, [2100, 600], 512, None),
    ("bf16", 128, 14, 2, 32, [1100, 1023], 0, None),
    ("fp16", 64, 8, 2, 64, [1500, 1025, 3], 128, None),
    ("bf16", 128, 16, 4, 16, [12000], 0, None),
    # neighbouring heads together; small blocks, copied by the computing warps
    ("bf16", 128, 32, 8, 16, [900, 33, 0, 1, 257, 64, 9000], 0, 20480),
    ("fp16", 64, 12, 12, 8, [31, 700, 5, 64, 65, 4001], 0, 16384),
    ("bf16", 128, 32, 8, 4, [3333, 20, 0, 129, 777], 0, 19456),
    ("fp16", 64, 4, 2, 1, [50, 2600, 31, 33], 0, 58880),
    ("bf16", 64, 32, 2, 2, [7000, 1], 0, None),
]


@pytest.mark.parametrize("idx", range(len(ONCE)))
def test_8_bit_decode_takes_every_token_once(idx):
    dtype, d, Hq, Hkv, B, lens, pt, width = ONCE[idx]
    rng = np.random.default_rng(300 + idx)
    NB = sum(-(-n // B) for n in lens) + 3
    bt = tables_for(rng, lens, B, NB, MB=width // B if width else max(-(-max(lens) // B) + 1, 1))
    V = rng.integers(-8, 9, (NB, B, Hkv, d)).astype(np.float64)
    kc, vc = np.zeros(V.shape, np.uint8), fp8.nearest_code(V)
    sc = np.full((NB, Hkv, 2, B), 127, np.uint8)
    used = np.zeros((NB, B), bool)
    for s, n in enumerate(lens):
        t = np.arange(n)
        used[bt[s, t // B], t % B] = True
    kc[..., 0] = np.where(used[..., None], 0x38, 0x60)  # 1 and 32
    vc[~used] = 0x7F
    q = np.zeros((len(lens), Hq, d), np.float32)
    q[..., 0] = 1
    qd, kd, btd = dev_bits(W.f32_to_bits(q, dtype), dtype), up8(kc), up(bt)
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
    pa.decode_fp8(out, qd, kd, up8(vc), up(sc), btd, up(np.array(lens, np.int32)), LN2, pt,
                  pa.alloc_workspace(qd, kd, btd, pt))
    for s, n in enumerate(lens):
        check_means(out[s].double().cpu().numpy(), oracle.gather_kv(V, bt[s], n, B), 32, (ONCE[idx], s))


SHARED_ONCE = [
    # dtype, d, Hq, Hkv, B, group starts, prefixes, lengths, table tokens
    ("bf16", 64, 16, 1, 16, [0, 60], [4001], [4001 + 5 * i for i in range(60)], None),
    ("fp16", 128, 8, 2, 16, [0, 100, 104], [600, 300], [600 + 3 * i for i in range(100)] + [300, 301, 499, 600], None),
    ("bf16", 128, 8, 8, 16, [0, 40], [1000], [1000 + 5 * i for i in range(40)], 20480),
    ("fp16", 64, 6, 3, 4, [0, 120], [777], [777 + i % 90 for i in range(120)], None),
    # without a pass
    ("fp16", 128, 4, 4, 4, [0, 3], [2050], [2051, 2300, 2099], None),
    ("bf16", 128, 8, 8, 16, [0, 4, 6], [300, 40], [301, 400, 555, 300, 41, 99], 20480),
    ("bf16", 64, 20, 2, 16, [0, 1, 2], [64, 0], [64, 4399], None),
]


@pytest.mark.parametrize("idx", range(len(SHARED_ONCE)))
def test_shared_prefix_takes_every_token_once(idx):
    *sizes, width = SHARED_ONCE[idx]
    case = Case(*sizes, seed=400 + idx, MB=width // sizes[4] if width else None)
    assert case.passes() == (idx < 4)
    B, V = case.B, np.random.default_rng(idx).integers(-8, 9, case.vc.shape).astype(np.float64)
    used = np.zeros(V.shape[:2], bool)
    for g, n in enumerate(case.prefixes):
        for s in range(case.starts[g], case.starts[g + 1]):
            t = np.arange(0 if s == case.starts[g] else min(n, case.lens[s]), case.lens[s])
            used[case.bt[s, t // B], t % B] = True
    K = np.zeros(V.shape)
    K[..., 0] = np.where(used[..., None], 1, 32)
    q = np.zeros(case.query.shape)
    q[..., 0] = 1
    case.scale = LN2
    case.query, case.kc, case.vc = (W.f32_to_bits(x.astype(np.float32), case.dtype)
                                    for x in (q, K, np.where(used[..., None, None], V, np.nan)))
    out = case.run().double().cpu().numpy()
    values = fp8.shared_prefix_values(V, case.bt, case.lens, case.starts, case.prefixes, B)
    # the pass's sums may be cut off, by 2^-23 at each of the 8 products for 64 tokens
    cut = case.max_prefix / 8 * 2.0 ** -23 if case.passes() else 0.0
    for s in range(len(case.lens)):
        check_means(out[s], values[s], 16, (SHARED_ONCE[idx][:5], s), cut)


# ------------------------------------------------------ values that are NaN --
@pytest.mark.parametrize("B", [16, 4])
def test_8_bit_nan_reaches_its_own_outputs_alone(B):
    rng = np.random.default_rng(B)
    lens, Hkv, d = [700, 50, 1500, 33], 2, 64
    kc, vc, sc = random_pool(rng, sum(-(-n // B) for n in lens), B, Hkv, d, 1)
    bt = tables_for(rng, lens, B, kc.shape[0])
    query = W.normal_bits((4, 10, d), "bf16", B, 2)
    clean, _ = decode8(query, kc, vc, sc, bt, lens, B, 0.05, "bf16")
    kc[bt[0, 650 // B], 650 % B, 1, 7] = 0x7F
    vc[bt[2, 3 // B], 3 % B, 0, 5] = 0x7F
    vc[bt[3, 32 // B], 32 % B, 1, 60] = 0xFF
    got, _ = decode8(query, kc, vc, sc, bt, lens, B, 0.05, "bf16")
    nan = np.zeros(got.shape, bool)
    nan[0, 5:] = True
    nan[2, :5, 5] = True
    nan[3, 5:, 60] = True
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[~nan], clean[~nan])


@pytest.mark.parametrize("members", [3, 150])
def test_shared_prefix_nan_reaches_its_own_outputs_alone(members):
    case = Case("fp16", 64, 8, 2, 16, [0, members, members + 2], [700, 20], [700 + i % 70 for i in range(members)] + [40, 900])
    assert case.passes() == (members > 3)
    clean = case.run().double().cpu().numpy()
    case.kd[int(case.bt[0, 333 // 16]), 333 % 16, 1, 7] = float("nan")               # of the first prefix
    case.vd[int(case.bt[members + 1, 850 // 16]), 850 % 16, 0, 5] = float("nan")     # of the last sequence
    got = case.run().double().cpu().numpy()
    nan = np.zeros(got.shape, bool)
    nan[:members, 4:] = True
    nan[members + 1, :4, 5] = True
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[~nan], clean[~nan])


def test_pieces_inside_a_chunk_of_a_shared_prefix():
    # 300 groups fill the machine with one chunk each: a CTA leaves two pieces of 6016
    # tokens. Whole numbers add up exactly, also where sums are cut off
    S, Hq, d, B, n = 600, 2, 64, 16, 12000
    NB = n // B + 1
    V = np.random.default_rng(5).integers(-8, 9, (NB, B, 1, d)).astype(np.float64)
    K, q = np.zeros(V.shape), np.zeros((S, Hq, d))
    K[..., 0], q[..., 0] = 1, 1
    bt = np.random.default_rng(6).permutation(NB).astype(np.int32)[None].repeat(S, 0)
    lens = (n + np.arange(S) % 3).astype(np.int32)
    qd, k, v = (dev_bits(W.f32_to_bits(x.astype(np.float32), "bf16"), "bf16") for x in (q, K, V))
    starts = torch.arange(0, S + 1, 2, dtype=torch.int32, device="cuda")
    prefixes = torch.full((S // 2,), n, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
    btd = up(bt)
    for bound in (n, NB * B):
        pa.decode_shared_prefix(out, qd, k, v, btd, up(lens), starts, prefixes, bound, 2, LN2,
                                pa.alloc_shared_prefix_workspace(qd, k, btd, starts, bound, 2))
        got = out.double().cpu().numpy()
        for s in range(S):
            check_means(got[s], oracle.gather_kv(V, bt[s], int(lens[s]), B), 16, (bound, s))


# ------------------------------------------------------------------ shares --
@pytest.mark.parametrize("bits,pt", [(4, 160), (4, 1008), (4, 64), (8, 144), (8, 1008)])
def test_shares_are_not_under_partition_tokens(bits, pt):
    # four kv heads at a time (a wide table), so that a share is counted in tiles of one warp; all shares
    # but a row's last have at least pt tokens
    Hq, Hkv, d, B, width, n = 4, 4, 64, 16, 1 << 18, 10 * pt
    alloc, decode = (pa.alloc_fp4_cache, pa.decode_fp4) if bits == 4 else (pa.alloc_fp8_cache, pa.decode_fp8)
    pool = alloc(8, B, Hkv, d)
    q = dev_bits(W.normal_bits((1, Hq, d), "bf16", pt, 2), "bf16")
    bt = torch.zeros(1, width // B, dtype=torch.int32, device="cuda")
    ws = pa.alloc_workspace(q, pool[0], bt)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    decode(out, q, *pool, bt, torch.tensor([n], dtype=torch.int32, device="cuda"), 0.1, pt, ws)
    pieces = ws[:8 * Hkv].view(torch.int32).view(Hkv, 2)[:, 1].tolist()
    assert pieces == [pieces[0]] * Hkv and 2 <= pieces[0] <= 10
    assert not out.any()


# ------------------------------------------------------- the end of the range --
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("S,Hq", [(1, 4), (2, 40), (60, 32)])
def test_pieces_of_the_largest_values_are_joined_in_range(bits, S, Hq):
    # V 6 2^125 (4-bit) or 448 2^119 in every element, equal scores: any sum of two pieces with weights of about one
    # is out of range, their mean is not. Few rows (a CTA merges each) and many (a warp each)
    rng = np.random.default_rng(S)
    Hkv, d, B, NB = 4, 64, 16, 64
    code, byte = ((0x77, 252) if bits == 4 else (0x7E, 246))
    pool = (pa.alloc_fp4_cache if bits == 4 else pa.alloc_fp8_cache)(NB, B, Hkv, d)
    pool[1].view(torch.uint8).fill_(code)
    pool[2][:, :, 1] = byte
    pool[2][:, :, 1, 3, ...] = byte - 5
    lens = rng.integers(3000, 9000, S)
    bt = torch.randint(0, NB, (S, 600), dtype=torch.int32, device="cuda")
    q = dev_bits(W.normal_bits((S, Hq, d), "bf16", S, 2), "bf16")
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    (pa.decode_fp4 if bits == 4 else pa.decode_fp8)(out, q, *pool, bt, up(lens.astype(np.int32)), 0.1,
                                                    workspace=pa.alloc_workspace(q, pool[0], bt))
    top = (6.0 if bits == 4 else 448.0) * 2.0 ** (byte - 127)
    small = (lens + 12) // 16  # one token of 16 is 2^-5 as large
    want = top * (1 - small / lens * (1 - 2.0 ** -5))
    # sums of n positive terms in fp32, twice, and a handful of roundings
    rel = np.abs(out.double().cpu().numpy() / want[:, None, None] - 1)
    assert np.all(rel <= (2 * lens[:, None, None] + 32) * 2.0 ** -24)
