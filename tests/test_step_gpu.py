"""Slots of new tokens, norms of heads and rotation by position on the GPU against the
oracle, and a whole step around each kind of cache, captured and replayed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from gpu_util import TORCH_DTYPE, dev_bits, host_bits
from oracle import fp4, fp8, step
from test_fp4_cache_gpu import up
from test_fp4_decode_gpu import check_rows, weight_error

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


def values(t, dtype):
    return oracle.to_float64(host_bits(t), dtype)


def random_frequencies(rng, n):
    w = 10000.0 ** (-np.arange(n) / n) * rng.uniform(0.9, 1.1, n)
    return pa.rotary_frequencies(w)


def check_rotated(got, x, positions, freq, dtype, interleaved, factor=1.0, weight=None, eps=1e-6, what=""):
    """Device rows against the oracle on float64 rows x."""
    angle = step.angles(positions, [int(f) for f in freq])
    w = None if weight is None else values(weight, dtype)
    ref = step.rotate(x, angle, interleaved, factor, w, eps)
    tol = step.rotate_bound(x, angle.shape[1], interleaved, factor, w, eps, ref, dtype)
    err = np.abs(values(got, dtype) - ref)
    assert np.all(err <= tol), f"{what}: {np.max(err / tol)} of the bound"


GRID = [
    # dtype, T, Hq, Hkv, d, rotary_dim, interleaved, norm, factor
    ("bf16", 1, 1, 1, 64, 64, False, False, 1.0),
    ("fp16", 5, 4, 4, 64, 16, True, False, 1.0),
    ("bf16", 33, 32, 8, 128, 128, False, True, 1.0),
    ("fp16", 130, 6, 3, 128, 64, True, True, 1.25),
    ("bf16", 7, 7, 1, 64, 48, False, True, 0.5),
    ("fp16", 64, 5, 5, 128, 80, False, False, 1.0),
    ("bf16", 9, 64, 8, 128, 32, True, True, 1.0),
    ("fp16", 257, 2, 1, 64, 32, True, False, 1.1),
    ("fp16", 3, 40, 40, 128, 112, False, True, 1.0),
    ("bf16", 18, 16, 2, 128, 16, False, True, 1.0),
]


@pytest.mark.parametrize("idx", range(len(GRID)))
def test_rotate_grid(idx):
    dtype, T, Hq, Hkv, d, rot, inter, norm, factor = GRID[idx]
    rng = np.random.default_rng(idx)
    # slices of one projection's output, with something behind them
    qkv = dev_bits(W.normal_bits((T, Hq + 2 * Hkv + 1, d), dtype, idx, 1), dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:Hq + 2 * Hkv]
    pos = rng.integers(0, 200000, T)
    freq = random_frequencies(rng, rot // 2)
    w = [dev_bits(W.normal_bits((d,), dtype, idx, 2 + i), dtype) if norm else None for i in range(2)]
    kw = dict(interleaved=inter, factor=factor, query_weight=w[0], key_weight=w[1], eps=1e-5)
    qo = torch.full((T, Hq, d), 9.0, dtype=q.dtype, device="cuda")
    ko = torch.full((T, Hkv + 2, d), 9.0, dtype=q.dtype, device="cuda")
    pa.rotate(qo, ko[:, 1:1 + Hkv], q, k, up(pos), freq, **kw)
    args = (pos, freq, dtype, inter, factor)
    check_rotated(qo, values(q, dtype), *args, w[0], 1e-5, "query")
    check_rotated(ko[:, 1:1 + Hkv], values(k, dtype), *args, w[1], 1e-5, "key")
    assert torch.all(ko[:, 0] == 9.0) and torch.all(ko[:, -1] == 9.0)
    # with the caches: the same rows at their slots, and nothing else
    B = int(rng.choice([1, 4, 16, 64]))
    NB = -(-T // B) + 2
    kc, vc = (torch.full((NB, B, Hkv, d), 7.0 + i, dtype=q.dtype, device="cuda") for i in range(2))
    slots = rng.permutation(NB * B)[:T]
    slots[2::5] = -1 - rng.integers(0, 9)
    qo2 = torch.empty_like(qo)
    pa.rotate_and_cache(qo2, q, k, v, kc, vc, up(slots), up(pos), freq, **kw)
    assert torch.equal(qo2, qo)
    wk, wv = torch.full_like(kc, 7.0), torch.full_like(vc, 8.0)
    keep = up(np.flatnonzero(slots >= 0))
    wk.view(-1, Hkv, d)[up(slots)[keep]] = ko[keep, 1:1 + Hkv]
    wv.view(-1, Hkv, d)[up(slots)[keep]] = v[keep]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    # in place, in the projection's output
    pa.rotate(q, k, q, k, up(pos), freq, **kw)
    assert torch.equal(q, qo) and torch.equal(k, ko[:, 1:1 + Hkv])


def test_far_and_negative_positions():
    # one position at a time, against whole-number turns: no drift however far
    T, d = 12, 64
    pos = np.array([0, 1, 2 ** 20, 2 ** 31 - 1, 2 ** 40 + 3, 2 ** 62 + 12345, -1, -77, -2 ** 33, 10 ** 6, 131071, -2 ** 63])
    w, _ = pa.rotary_inverse_frequencies(d, 10000.0)
    freq = pa.rotary_frequencies(w)
    x = W.normal_bits((T, 2, d), "fp16", 3, 1)
    q = dev_bits(x, "fp16")
    out = torch.empty_like(q)
    pa.rotate(out, torch.empty_like(q), q, q, up(pos), freq)
    check_rotated(out, values(q, "fp16"), pos, freq, "fp16", False)
    # and the definition: position times frequency radians, where float64 can hold it
    i = np.flatnonzero(np.abs(pos.astype(np.float64)) < 2 ** 32)
    ref = step.rotate(values(q, "fp16")[i], pos[i, None] * np.array(w), False)
    assert np.max(np.abs(values(out, "fp16")[i] - ref)) <= 2e-3 * np.abs(ref).max()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_norms_of_rows_of_any_size(dtype):
    # rows whose squares are out of fp32's range or next to nothing, zeros, beside ordinary ones
    T, H, d = 3, 8, 128
    rng = np.random.default_rng(2)
    x = rng.standard_normal((T, H, d))
    if dtype == "bf16":
        x *= np.array([1, 2.0 ** 70, 2.0 ** 120, 2.0 ** -70, 2.0 ** -30, 0, 2.0 ** 62, 2.0 ** 64])[None, :, None]
        x[2, 2] = 3.3e38
    else:
        x *= np.array([1, 2.0 ** 13, 60, 2.0 ** -14, 2.0 ** -20, 0, 2.0 ** 10, 5])[None, :, None]
    q = dev_bits(W.f32_to_bits(x.astype(np.float32), dtype), dtype)
    w = dev_bits(W.normal_bits((d,), dtype, 1, 2), dtype)
    freq = random_frequencies(rng, 32)
    pos = np.array([5, 77, 9000])
    qo, ko = torch.empty_like(q), torch.empty_like(q)
    pa.rotate(qo, ko, q, q, up(pos), freq, query_weight=w, key_weight=w)
    check_rotated(qo, values(q, dtype), pos, freq, dtype, False, 1.0, w)
    assert torch.equal(qo, ko)


MANY = [
    # dtype, T, Hq, Hkv, d, rotary_dim, interleaved, norm: rows that take a warp more rounds than it has under way
    # together. 912 tokens or more: one warp a token; just below: two; few: eight
    ("bf16", 913, 32, 8, 128, 128, False, False),
    ("bf16", 913, 32, 8, 128, 128, False, True),
    ("fp16", 913, 29, 3, 128, 64, True, True),
    ("fp16", 912, 29, 3, 128, 128, False, False),
    ("bf16", 1000, 64, 8, 64, 64, False, True),
    ("fp16", 913, 64, 8, 64, 32, True, False),
    ("bf16", 911, 64, 8, 128, 96, False, True),
    ("fp16", 911, 61, 7, 128, 128, True, False),
    ("bf16", 3, 200, 10, 128, 128, False, True),
    ("fp16", 2, 431, 5, 64, 64, False, False),
]


@pytest.mark.parametrize("idx", range(len(MANY)))
def test_rotate_rows_of_many_rounds(idx):
    dtype, T, Hq, Hkv, d, rot, inter, norm = MANY[idx]
    rng = np.random.default_rng(40 + idx)
    bits = W.normal_bits((T, Hq + 2 * Hkv, d), dtype, 40 + idx, 1)
    # rows of a NaN or an infinity among the first: nothing of them may reach rows behind
    odd = rng.choice(T, min(T, 40), replace=False)
    bits[odd[0::2], 1, 3::40] = {"bf16": 0x7FC0, "fp16": 0x7E00}[dtype]
    bits[odd[1::2], 2, 5] = {"bf16": 0xFF80, "fp16": 0xFC00}[dtype]
    qkv = dev_bits(bits, dtype)
    q, k, v = qkv.split((Hq, Hkv, Hkv), 1)
    pos, freq = rng.integers(0, 200000, T), random_frequencies(rng, rot // 2)
    w = [dev_bits(W.normal_bits((d,), dtype, 41 + idx, 2 + i), dtype) if norm else None for i in range(2)]
    kw = dict(interleaved=inter, query_weight=w[0], key_weight=w[1])
    qo, ko = torch.empty(T, Hq, d, dtype=q.dtype, device="cuda"), torch.empty(T, Hkv, d, dtype=q.dtype, device="cuda")
    pa.rotate(qo, ko, q, k, up(pos), freq, **kw)
    angle = step.angles(pos, [int(f) for f in freq])
    for got, x, weight in ((qo, q, w[0]), (ko, k, w[1])):
        x, weight = values(x, dtype), None if weight is None else values(weight, dtype)
        ref, got = step.rotate(x, angle, inter, 1.0, weight), values(got, dtype)
        fine = np.isfinite(ref)
        with np.errstate(invalid="ignore"):
            tol = step.rotate_bound(x, rot // 2, inter, 1.0, weight, 1e-6, ref, dtype)
        assert np.all(np.abs(got[fine] - ref[fine]) <= tol[fine])
        assert np.array_equal(got[~fine], ref[~fine], equal_nan=True)
    B, NB = 16, T // 16 + 3
    kc, vc = (torch.full((NB, B, Hkv, d), 7.0 + i, dtype=q.dtype, device="cuda") for i in range(2))
    slots = rng.permutation(NB * B)[:T]
    slots[2::5] = -1  # a padded batch
    qo2 = torch.empty_like(qo)
    pa.rotate_and_cache(qo2, q, k, v, kc, vc, up(slots), up(pos), freq, **kw)
    wk, wv = torch.full_like(kc, 7.0), torch.full_like(vc, 8.0)
    keep = up(np.flatnonzero(slots >= 0))
    wk.view(-1, Hkv, d)[up(slots)[keep]] = ko[keep]
    wv.view(-1, Hkv, d)[up(slots)[keep]] = v[keep]
    assert np.array_equal(host_bits(qo2), host_bits(qo))
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    # in place, in the projection's output
    pa.rotate(q, k, q, k, up(pos), freq, **kw)
    assert np.array_equal(host_bits(q), host_bits(qo)) and np.array_equal(host_bits(k), host_bits(ko))
    assert torch.equal(v, dev_bits(bits, dtype)[:, Hq + Hkv:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_nan_and_infinity_stay_in_their_pairs(interleaved, norm):
    T, H, d, rot = 2, 4, 64, 32
    rng = np.random.default_rng(3)
    x = W.normal_bits((T, H, d), "bf16", 4, 1)
    q = dev_bits(x, "bf16")
    w = dev_bits(W.normal_bits((d,), "bf16", 4, 2), "bf16") if norm else None
    freq, pos = random_frequencies(rng, rot // 2), np.array([3, 1000])
    clean = torch.empty_like(q)
    kw = dict(interleaved=interleaved, query_weight=w, key_weight=w)
    pa.rotate(clean, torch.empty_like(q), q, q, up(pos), freq, **kw)
    bad = q.clone()
    bad[0, 1, 3], bad[1, 2, 50], bad[1, 0, 63] = float("nan"), float("inf"), float("nan")
    out = torch.empty_like(q)
    pa.rotate(out, torch.empty_like(q), bad, bad, up(pos), freq, **kw)
    if norm:  # a norm spreads over its head, and no further
        hit = torch.zeros_like(q, dtype=torch.bool)
        hit[0, 1] = hit[1, 2] = hit[1, 0] = True
        assert torch.equal(out[~hit], clean[~hit])
        ref = step.rotate(values(bad, "bf16"), step.angles(pos, [int(f) for f in freq]), interleaved, 1.0, values(w, "bf16"))
        assert np.array_equal(np.isnan(ref), out.isnan().cpu().numpy())
    else:
        ia, ib = step.pairs(rot // 2, interleaved)
        partner = [int(ib[i]) if ia[i] == 3 else int(ia[i]) for i in range(rot // 2) if 3 in (ia[i], ib[i])][0]
        hit = torch.zeros_like(q, dtype=torch.bool)
        hit[0, 1, [3, partner]] = hit[1, 2, 50] = hit[1, 0, 63] = True
        assert torch.equal(out[~hit], clean[~hit])
        assert out[0, 1, [3, partner]].isnan().all() and out[1, 2, 50] == float("inf") and out[1, 0, 63].isnan()


def test_slots_above_the_pool_are_skipped_and_counted():
    T, H, d = 5, 2, 64
    q = dev_bits(W.normal_bits((T, H, d), "bf16", 5, 1), "bf16")
    kc, vc = (torch.zeros(2, 4, H, d, dtype=q.dtype, device="cuda") for _ in range(2))
    qo = torch.empty_like(q)
    pa.bad_index_count(clear=True)
    freq = random_frequencies(np.random.default_rng(0), 32)
    pos = torch.arange(T, device="cuda")
    pa.rotate_and_cache(qo, q, q, q, kc, vc, torch.tensor([8, -1, 2 ** 40, 3, -2 ** 50], device="cuda"), pos, freq)
    assert pa.bad_index_count(clear=True) == 2
    check_rotated(qo, values(q, "bf16"), range(T), freq, "bf16", False)
    assert torch.equal(kc.view(8, H, d)[3], qo[3]) and torch.equal(vc.view(8, H, d)[3], q[3])
    kc.view(8, H, d)[3] = 0
    vc.view(8, H, d)[3] = 0
    assert not kc.any() and not vc.any()


def test_no_tokens():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pa.rotate(q, q, q, q, torch.empty(0, dtype=torch.int64, device="cuda"), pa.rotary_frequencies([1.0] * 8))


# ----------------------------------------------------------------- append --
def run_append(tables, lens, starts, free, num_free, rows, B, NB, alias=False):
    t, ln, nf = up(np.array(tables, np.int32)), up(np.array(lens, np.int32)), up(np.array([num_free], np.int32))
    new_lens, new_free = (ln, nf) if alias else (torch.full_like(ln, 55), torch.full_like(nf, 55))
    slots, positions = (torch.full((rows,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.append_tokens(new_lens, new_free, slots, positions, t, ln, up(np.array(starts, np.int32)),
                     up(np.array(free, np.int32)), nf, status, B, NB)
    if not alias:
        assert np.array_equal(ln.cpu().numpy(), lens) and int(nf) == num_free
    return (t.cpu().numpy(), new_lens.cpu().numpy(), int(new_free), slots.cpu().numpy(), positions.cpu().numpy(),
            int(status))


def check_append(tables, lens, starts, free, num_free, rows, B, NB, rejected=None):
    want = step.append_tokens(tables, lens, starts, free, num_free, rows, B, NB)
    for alias in (False, True):
        pa.bad_index_count(clear=True)
        got = run_append(tables, lens, starts, free, num_free, rows, B, NB, alias)
        assert pa.bad_index_count(clear=True) == want[6]
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
    return want


@pytest.mark.parametrize("S,B,most_len,most_new,pad", [
    (1, 16, 0, 1, 0), (4, 16, 128, 1, 3), (7, 1, 40, 3, 0), (256, 64, 5000, 1, 1), (33, 2, 9, 40, 5),
    (64, 16, 4096, 400, 3), (1024, 16, 100, 2, 0), (3000, 8, 300, 3, 9), (5, 4, 60, 5000, 0), (16384, 16, 40, 1, 7)])
def test_append_against_the_oracle(S, B, most_len, most_new, pad):
    rng = np.random.default_rng(S + B)
    lens = rng.integers(0, most_len + 1, S)
    new = rng.integers(0, most_new + 1, S) if most_new > 1 else np.ones(S, int)
    starts = np.concatenate([[0], np.cumsum(new)])
    MB = -(-(most_len + most_new) // B) + 1
    spare = int(sum(-(-(a + b) // B) - -(-a // B) for a, b in zip(lens, new)))
    NB = 4 * spare + 100
    tables = rng.integers(0, NB, (S, MB))
    free = rng.integers(0, NB, spare + 4)
    check_append(tables, lens, starts, free, spare + int(rng.integers(0, 5)), int(starts[-1]) + pad, B, NB)


def test_append_one_block_short_and_exactly_enough():
    tables = np.zeros((3, 4), int)
    lens, starts = np.array([4, 7, 0]), np.array([0, 1, 3, 8])
    # new blocks: 1 (5 tokens), 1 (9), 2 (5)
    for have, status in ((4, 0), (3, step.NO_BLOCKS), (0, step.NO_BLOCKS)):
        assert check_append(tables, lens, starts, [9, 8, 7, 6, 5], have, 10, 4, 16)[5] == status


@pytest.mark.parametrize("lens,starts,num_free,rows", [
    ([-1, 3], [0, 1, 2], 4, 4), ([3, 3], [0, 2, 1], 4, 4), ([3, 3], [0, 1, 9], 4, 4), ([3, 3], [-1, 0, 1], 4, 4),
    ([3, 16], [0, 1, 2], 4, 4), ([3, 3], [0, 1, 2], -1, 4), ([3, 3], [0, 1, 2], 6, 4),
    ([3, 2 ** 31 - 2], [0, 1, 4], 4, 4)])
def test_append_out_of_range_changes_nothing(lens, starts, num_free, rows):
    want = check_append(np.full((2, 4), 3), np.array(lens), np.array(starts), [1, 2, 3, 4, 5], num_free, rows, 4, 16)
    assert want[5] == step.OUT_OF_RANGE


def test_append_out_of_range_changes_nothing_in_a_large_step():
    tables = np.full((2, 4000), 3)
    check_append(tables, np.array([5, 0]), np.array([0, 9000, 8000]), np.arange(9000), 9000, 9000, 4, 9999)
    check_append(tables, np.array([5, 0]), np.array([0, 4000, 9000]), np.arange(9000), 2000, 9000, 4, 9999)


def test_append_rejects_ids_outside_the_pool():
    # a bad id in the stack, and one in a table's last, partly filled block
    want = check_append(np.array([[2, -7, 0], [99, 0, 0]]), np.array([4, 2]), np.array([0, 6, 9]), [5, 16, -1, 3], 4, 9, 4, 16)
    assert want[6] > 0


def test_append_starts_behind_row_zero_and_empty_batches():
    check_append(np.zeros((2, 4), int), np.array([0, 5]), np.array([3, 4, 6]), [1, 2, 3], 3, 9, 4, 16)
    check_append(np.zeros((2, 4), int), np.array([0, 5]), np.array([2, 2, 2]), [1, 2, 3], 3, 4, 4, 16)
    check_append(np.zeros((0, 4), int), np.zeros(0, int), np.array([0]), [1, 2, 3], 3, 4, 4, 16)
    check_append(np.zeros((0, 4), int), np.zeros(0, int), np.array([0]), [], 0, 0, 4, 16)


def test_append_status_stays_raised():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens, free = torch.tensor([4], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    slots, pos = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    bt = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    height = torch.tensor([1], dtype=torch.int32, device="cuda")
    seen = []
    for _ in range(6):  # tokens 4 to 7 fit, 8 does not fit the table
        pa.append_tokens(lens, height, slots, pos, bt, lens, starts, free, height, status, 4, 8)
        seen.append((int(lens), int(slots), int(status)))
    assert seen == [(5, 12, 0), (6, 13, 0), (7, 14, 0), (8, 15, 0), (8, -1, 2), (8, -1, 2)]


# ------------------------------------------------------------ all together --
class Model:
    """The rows that a small model would make of each position, and what the caches then stand for."""

    def __init__(self, S, Hq, Hkv, d, dtype, rot, interleaved, pool):
        self.S, self.Hq, self.Hkv, self.d, self.dtype, self.pool = S, Hq, Hkv, d, dtype, pool
        self.interleaved = interleaved
        w, self.factor = pa.rotary_inverse_frequencies(rot, 10000.0, "yarn", 4.0, 64, 1.0, 32.0)
        self.freq = pa.rotary_frequencies(w)
        self.weights = [dev_bits(W.normal_bits((d,), dtype, 70, i), dtype) for i in range(2)]
        self.hist = [[] for _ in range(S)]

    def rows(self, T, seed):
        bits = W.normal_bits((T, self.Hq + 2 * self.Hkv, self.d), self.dtype, 71, seed)
        return dev_bits(bits, self.dtype)

    def split(self, qkv):
        return qkv.split((self.Hq, self.Hkv, self.Hkv), 1)

    def enqueue(self, qkv, qo, ko, caches, slots, positions):
        q, k, v = self.split(qkv)
        kw = dict(interleaved=self.interleaved, factor=self.factor, query_weight=self.weights[0],
                  key_weight=self.weights[1])
        if self.pool == 16:
            pa.rotate_and_cache(qo, q, k, v, *caches, slots, positions, self.freq, **kw)
        else:
            pa.rotate(qo, ko, q, k, positions, self.freq, **kw)
            (pa.reshape_and_cache_fp8 if self.pool == 8 else pa.reshape_and_cache_fp4)(ko, v.contiguous(), *caches, slots)

    def decode(self, out, qo, caches, bt, lens, ws):
        f = {16: pa.decode, 8: pa.decode_fp8, 4: pa.decode_fp4}[self.pool]
        f(out, qo, *caches, bt, lens, 0.1, workspace=ws)

    def held(self, rows):
        x = values(rows, self.dtype)
        if self.pool == 16:
            return x
        if self.pool == 8:
            c, e = fp8.quantise_rows(x)
            return fp8.E4M3[c] * np.exp2(e.astype(np.float64) - 127)[..., None]
        return fp4.row_values(*fp4.quantise_rows(x))

    def record(self, qkv, seqs, positions):
        """The rotated query rows of the oracle's inputs: rows as the library rounds them, checked."""
        q, k, v = self.split(qkv)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        kw = dict(interleaved=self.interleaved, factor=self.factor, query_weight=self.weights[0],
                  key_weight=self.weights[1])
        pa.rotate(qo, ko, q, k, up(np.array(positions)), self.freq, **kw)
        check_rotated(qo, values(q, self.dtype), positions, self.freq, self.dtype, self.interleaved, self.factor, self.weights[0])
        check_rotated(ko, values(k, self.dtype), positions, self.freq, self.dtype, self.interleaved, self.factor, self.weights[1])
        K, V = self.held(ko), self.held(v)
        for i, s in enumerate(seqs):
            self.hist[s].append((K[i], V[i]))
        return host_bits(qo)

    def check(self, out, query, what):
        for s in range(self.S):
            K, V = (np.stack(x) for x in zip(*self.hist[s]))
            got = out[s].double().cpu().numpy()
            if self.pool == 16:
                G = self.Hq // self.Hkv
                q = oracle.to_float64(query[s], self.dtype)
                ref = np.concatenate([oracle.single_query_attention(q[h * G:(h + 1) * G], K[:, h], V[:, h], 0.1)[0]
                                      for h in range(self.Hkv)])
                assert np.max(np.abs(got - ref)) <= 2e-3, what
            else:
                check_rows(got, query[s], K, V, 0.1, self.dtype, weight_error(len(K), 5), what)


@pytest.mark.parametrize("pool", [16, 8, 4])
@pytest.mark.parametrize("dtype,Hq,Hkv,d,B,rot,inter", [("bf16", 8, 2, 128, 16, 128, False),
                                                        ("fp16", 6, 3, 64, 8, 32, True)])
def test_a_captured_step_goes_on_by_itself(pool, dtype, Hq, Hkv, d, B, rot, inter):
    """Ragged prompts through append, rotation and write; then one graph of a whole decode step (slots,
    rotation, write, attention) replayed with nothing in between but new rows: every step's output is
    checked, and the tables never come from the host."""
    rng = np.random.default_rng(pool)
    S, MB, NB, steps = 5, 12, 64, 20
    m = Model(S, Hq, Hkv, d, dtype, rot, inter, pool)
    T16 = TORCH_DTYPE[dtype]
    if pool == 16:
        caches = [torch.zeros(NB, B, Hkv, d, dtype=T16, device="cuda") for _ in range(2)]
    else:
        caches = (pa.alloc_fp8_cache if pool == 8 else pa.alloc_fp4_cache)(NB, B, Hkv, d)
    i32 = dict(dtype=torch.int32, device="cuda")
    bt = torch.zeros(S, MB, **i32)
    lens, status = torch.zeros(S, **i32), torch.zeros(1, **i32)
    free, height = up(rng.permutation(NB).astype(np.int32)), torch.tensor([NB], **i32)

    prompts = [1, 33, 7, 64, 20]
    T = sum(prompts) + 3  # a padded batch
    starts = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    slots, positions = (torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2))
    pa.append_tokens(lens, height, slots, positions, bt, lens, up(starts), free, height, status, B, NB)
    qkv = m.rows(T, 1)
    qo, ko = torch.empty(T, Hq, d, dtype=T16, device="cuda"), torch.empty(T, Hkv, d, dtype=T16, device="cuda")
    m.enqueue(qkv, qo, ko, caches, slots, positions)
    seqs = [s for s, n in enumerate(prompts) for _ in range(n)]
    pos = [i for n in prompts for i in range(n)]
    query = m.record(qkv[:T - 3], seqs, pos)
    if pool == 16:  # the prompts' own attention
        out = torch.empty(T - 3, Hq, d, dtype=torch.float32, device="cuda")
        pa.prefill(out, qo[:T - 3], *caches, bt, lens, up(starts), max(prompts), 0.1)
        for s, n in enumerate(prompts):
            K, V = (np.stack(x) for x in zip(*m.hist[s]))
            bits = lambda x: W.f32_to_bits(x.astype(np.float32), dtype)  # noqa: E731
            ref = oracle.paged_prefill(query[starts[s]:starts[s + 1]], bits(K)[None], bits(V)[None], np.zeros((1, 1), np.int32),
                                       [n], [0, n], n, 0.1, dtype)
            assert np.max(np.abs(out[starts[s]:starts[s + 1]].cpu().numpy() - ref)) <= 2e-3

    step_starts = torch.arange(S + 1, **i32)
    slots, positions = (torch.zeros(S, dtype=torch.int64, device="cuda") for _ in range(2))
    row = m.rows(S, 2)
    qo, ko = torch.empty(S, Hq, d, dtype=T16, device="cuda"), torch.empty(S, Hkv, d, dtype=T16, device="cuda")
    out = torch.empty(S, Hq, d, dtype=torch.float32, device="cuda")
    ws = pa.alloc_workspace(qo, caches[0], bt)

    def whole_step():
        pa.append_tokens(lens, height, slots, positions, bt, lens, step_starts, free, height, status, B, NB)
        m.enqueue(row, qo, ko, caches, slots, positions)
        m.decode(out, qo, caches, bt, lens, ws)

    state = [t.clone() for t in (lens, height, bt)]
    whole_step()  # before the capture: first calls look up the device
    torch.cuda.synchronize()
    for t, was in zip((lens, height, bt), state):
        t.copy_(was)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        whole_step()
    used = set()
    for k in range(steps):
        row.copy_(m.rows(S, 10 + k))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        now = [n + k for n in prompts]
        assert lens.tolist() == [n + 1 for n in now] and positions.tolist() == now and int(status) == 0
        query = m.record(row, range(S), now)
        m.check(out, query, f"step {k}")
    table = bt.cpu().numpy()
    for s, n in enumerate(lens.tolist()):
        mine = set(table[s, :-(-n // B)].tolist())
        assert len(mine) == -(-n // B) and not used & mine
        used |= mine
    assert int(height) == NB - len(used)


def test_a_large_append_captured_and_replayed():
    """Lengths and the stack's height written over those read, by the second of its two launches; the
    table is read by what follows in the graph."""
    rng = np.random.default_rng(12)
    S, B, MB, new, rounds = 40, 16, 60, 150, 5
    NB = S * MB
    lens, starts = rng.integers(0, 90, S).astype(np.int32), np.arange(S + 1, dtype=np.int32) * new
    want = (rng.integers(0, NB, (S, MB)), lens, NB)
    free = rng.permutation(NB)
    t, ln, height = up(want[0].astype(np.int32)), up(lens), up(np.array([NB], np.int32))
    status, free_d, starts_d = torch.zeros_like(height), up(free.astype(np.int32)), up(starts)
    slots, positions = (torch.zeros(S * new, dtype=torch.int64, device="cuda") for _ in range(2))
    state = [x.clone() for x in (t, ln, height)]

    def call():
        pa.append_tokens(ln, height, slots, positions, t, ln, starts_d, free_d, height, status, B, NB)
        return t.clone(), slots + 0, positions + 0

    call()  # before the capture: first calls look up the device
    for x, was in zip((t, ln, height), state):
        x.copy_(was)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for k in range(rounds):
        g.replay()
        *want, w_slots, w_positions, w_status, _ = step.append_tokens(want[0], want[1], starts, free, want[2], S * new, B, NB)
        assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(ln.cpu().numpy(), want[1])
        assert int(height) == want[2] and int(status) == w_status == 0
        assert np.array_equal(got[1].cpu().numpy(), w_slots) and np.array_equal(got[2].cpu().numpy(), w_positions)


def test_on_other_streams_at_once():
    rng = np.random.default_rng(9)
    T, Hq, Hkv, d = 300, 8, 2, 128
    q, k = dev_bits(W.normal_bits((T, Hq, d), "bf16", 1, 1), "bf16"), dev_bits(W.normal_bits((T, Hkv, d), "bf16", 1, 2), "bf16")
    pos, freq = up(rng.integers(0, 5000, T)), random_frequencies(rng, 64)
    want = [torch.empty_like(q), torch.empty_like(k)]
    pa.rotate(*want, q, k, pos, freq)
    lens, starts = up(rng.integers(0, 90, 64).astype(np.int32)), up(np.arange(65, dtype=np.int32) * 90)
    free = up(rng.permutation(2000).astype(np.int32))
    num = torch.tensor([2000], dtype=torch.int32, device="cuda")
    def made():
        return [torch.empty_like(lens), torch.empty_like(num), *(torch.empty(5760, dtype=torch.int64, device="cuda") for _ in range(2)),
                torch.zeros(64, 16, dtype=torch.int32, device="cuda")]
    first, status = made(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.append_tokens(*first, lens, starts, free, num, status, 16, 2000)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [(torch.empty_like(q), torch.empty_like(k), made()) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for (a, b, c), st in zip(outs, streams):
            pa.rotate(a, b, q, k, pos, freq, stream=st)
            pa.append_tokens(*c, lens, starts, free, num, status, 16, 2000, stream=st)
    torch.cuda.synchronize()
    for a, b, c in outs:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        assert all(torch.equal(x, y) for x, y in zip(c, first)) and int(status) == 0
