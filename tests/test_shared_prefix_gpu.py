"""Decode over a shared prefix on the GPU against exact attention in which the
prefix of each group is read through its first member's table, with a bound
derived from the arithmetic (oracle.fp8.decode_bound)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import paged_kv_cache_305_gb300 as pa
import workloads as W
from gpu_util import dev_bits, host_bits
from oracle import fp8

pytestmark = pytest.mark.gpu

# a weight enters as two 16-bit parts: relative error below 2^-15 for bf16
WEIGHT_ERROR = {"bf16": 2.0 ** -15, "fp16": 2.0 ** -19}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_305_gb300 import build
    build.build()
    pa.bad_index_count(clear=True)
    pa.wait_timeout_count(clear=True)
    yield
    torch.cuda.synchronize()
    assert pa.wait_timeout_count(clear=True) == 0


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Case:
    """Sequences of `lens` tokens, each with blocks of its own; prefix entries
    of the tables of all but a group's first member are -1: they must not be read."""

    def __init__(self, dtype, d, Hq, Hkv, B, starts, prefixes, lens, seed=0, hide=True, MB=None):
        rng = np.random.default_rng(seed)
        self.dtype, self.B, self.d = dtype, B, d
        self.starts, self.prefixes = np.array(starts, np.int32), np.array(prefixes, np.int32)
        self.lens = np.array(lens, np.int32)
        held = -(-self.lens // B)
        NB = int(held.sum()) + 3
        MB = MB or max(1, int(held.max()))
        self.bt = rng.integers(0, NB, (len(lens), MB)).astype(np.int32)
        perm, at = rng.permutation(NB), 0
        for s, n in enumerate(held):
            self.bt[s, :n] = perm[at:at + n]
            at += n
        self.kc = W.normal_bits((NB, B, Hkv, d), dtype, seed, 1)
        self.vc = W.normal_bits((NB, B, Hkv, d), dtype, seed, 2)
        self.query = W.normal_bits((len(lens), Hq, d), dtype, seed, 3)
        self.scale = 1 / np.sqrt(d)
        self.table = self.bt.copy()
        if hide:
            for g, n in enumerate(prefixes):
                for s in range(starts[g] + 1, starts[g + 1]):
                    if self.lens[s] >= n:
                        self.table[s, :n // B] = -1
        self.max_prefix = int(max(prefixes)) if len(prefixes) else 0
        self.max_group = int(max(np.diff(starts)))

    def passes(self):
        """Whether the prefix is computed for its group at once: the reading that this saves, in
        bytes, against a bound that is higher where a chunk takes many CTAs of 128 rows."""
        S, Hq, d = self.query.shape
        Hkv, groups = self.kc.shape[2], len(self.prefixes)
        ctas = -(-self.max_group // (128 // (Hq // Hkv))) * groups * Hkv
        return (S - groups) * self.max_prefix * Hkv * d * 4 > (32e6 if ctas <= 38 else 128e6)

    def upload(self):
        self.q, self.kd, self.vd = (dev_bits(x, self.dtype) for x in (self.query, self.kc, self.vc))
        self.btd, self.sl, self.gs, self.pl = up(self.table), up(self.lens), up(self.starts), up(self.prefixes)

    def run(self, ws=None, max_prefix=None, max_group=None, f32=True):
        if not hasattr(self, "q"):
            self.upload()
        mp = self.max_prefix if max_prefix is None else max_prefix
        mg = self.max_group if max_group is None else max_group
        if ws is None:
            ws = pa.alloc_shared_prefix_workspace(self.q, self.kd, self.btd, self.gs, mp, mg)
        out = torch.full(self.query.shape, float("nan"), dtype=torch.float32 if f32 else self.q.dtype, device="cuda")
        pa.decode_shared_prefix(out, self.q, self.kd, self.vd, self.btd, self.sl, self.gs, self.pl, mp, mg,
                                self.scale, ws)
        return out

    def check(self, out, prefixes=None, what=""):
        prefixes = self.prefixes if prefixes is None else prefixes
        args = (self.bt, self.lens, self.starts, prefixes, self.B)
        ref = fp8.shared_prefix_decode(self.query, self.kc, self.vc, *args, self.scale, self.dtype)
        Ks, Vs = fp8.shared_prefix_values(self.kc, *args), fp8.shared_prefix_values(self.vc, *args)
        got = out.double().cpu().numpy()
        for s in range(len(self.lens)):
            K, V, q = (oracle.to_float64(x, self.dtype) for x in (Ks[s], Vs[s], self.query[s]))
            tol = fp8.decode_bound(q, K, V, self.scale, WEIGHT_ERROR[self.dtype])
            err = np.max(np.abs(got[s] - ref[s]))
            assert err <= tol, f"{what} sequence {s}: {err} > {tol}"


GRID = [
    # dtype, d, Hq, Hkv, B, group starts, prefixes, lengths
    ("bf16", 128, 8, 2, 16, [0, 5], [256], [300, 256, 257, 400, 511]),
    ("fp16", 64, 4, 4, 16, [0, 3, 4], [64, 100], [64, 65, 200, 130]),
    ("bf16", 64, 6, 3, 4, [0, 4], [333], [340, 333, 401, 350]),
    ("fp16", 128, 16, 1, 8, [0, 9], [500], [500 + 7 * i for i in range(9)]),
    ("bf16", 128, 4, 4, 1, [0, 2, 5], [40, 77], [41, 60, 77, 90, 130]),
    ("fp16", 64, 14, 2, 64, [0, 20], [700], [700 + 31 * i for i in range(20)]),
    ("bf16", 128, 12, 4, 2, [0, 1, 2, 6], [30, 65, 0], [31, 70, 9, 0, 1, 100]),
    # groups that are empty, of one member, and a prefix of one token
    ("fp16", 128, 8, 8, 32, [0, 0, 1, 1, 4, 4], [50, 20, 9, 1, 3], [33, 1, 2, 64]),
    # more members than one tile of 128 rows holds, chunked prefix
    ("bf16", 64, 16, 1, 16, [0, 30], [1500], [1500 + i for i in range(30)]),
]


# the same for groups whose prefix is computed for all members at once
PASS = [
    ("bf16", 128, 8, 2, 16, [0, 100, 104], [600, 300], [600 + 3 * i for i in range(100)] + [300, 301, 499, 600]),
    # more members than one tile of 128 rows holds
    ("fp16", 64, 4, 4, 16, [0, 130, 133], [500, 77], [500 + i % 70 for i in range(130)] + [77, 78, 200]),
    ("bf16", 64, 6, 3, 4, [0, 120], [777], [777 + i % 90 for i in range(120)]),
    ("fp16", 128, 16, 1, 8, [0, 90, 91], [1000, 5], [1000 + 2 * i for i in range(90)] + [6]),
    ("bf16", 128, 4, 4, 1, [0, 140, 145], [257, 40], [257 + i % 20 for i in range(140)] + [40, 41, 60, 99, 299]),
    ("fp16", 64, 14, 2, 64, [0, 150], [700], [700 + i for i in range(150)]),
    ("bf16", 128, 12, 4, 2, [0, 1, 2, 110], [30, 65, 400], [31, 70] + [400 + i % 33 for i in range(108)]),
    # groups that are empty, and of one member; more CTAs a chunk
    ("fp16", 128, 8, 8, 32, [0, 0, 1, 1, 130, 130], [50, 20, 9, 300, 3], [33] + [300 + i % 65 for i in range(129)]),
    ("fp16", 128, 2, 2, 16, [0, 140, 150], [129, 515], [130 + i % 3 for i in range(140)] + [515] * 10),
    # chunks of a long prefix
    ("bf16", 64, 16, 1, 16, [0, 40], [6001], [6001 + 5 * i for i in range(40)]),
]


@pytest.mark.parametrize("idx", range(len(GRID) + len(PASS)))
def test_grid(idx):
    case = Case(*(GRID + PASS)[idx], seed=idx)
    assert case.passes() == (idx >= len(GRID))
    pa.bad_index_count(clear=True)
    out = case.run()
    assert pa.bad_index_count(clear=True) == 0  # the hidden entries were never read
    case.check(out, what=str((GRID + PASS)[idx][:5]))
    o16 = case.run(f32=False)
    want = oracle.round_to_dtype(out.double().cpu().numpy(), case.dtype)
    assert np.array_equal(host_bits(o16), want)


# long prefixes, and neighbouring heads of the suffixes together
LONG = [
    # with a pass
    ("bf16", 128, 8, 8, 16, [0, 40], [1000], [1000 + 5 * i for i in range(40)], 20480),
    ("fp16", 64, 24, 6, 8, [0, 60], [900], [900 + 3 * i for i in range(60)], 8192),
    # dtype, d, Hq, Hkv, B, group starts, prefixes, lengths, table tokens
    ("bf16", 128, 8, 2, 16, [0, 5], [2100], [2100, 2101, 2200, 2731, 2115], None),
    ("fp16", 64, 16, 2, 64, [0, 2, 6], [2300, 2048], [2301, 2400, 2048, 2050, 2111, 2600], None),
    ("fp16", 128, 4, 4, 4, [0, 3], [2050], [2051, 2300, 2099], None),
    ("bf16", 128, 8, 8, 16, [0, 4, 6], [300, 40], [301, 400, 555, 300, 41, 99], 20480),
    ("fp16", 64, 24, 6, 8, [0, 6], [100], [100, 101, 340, 163, 164, 229], 8192),
    ("bf16", 64, 20, 2, 16, [0, 4], [64], [64, 100, 399, 80], 32768),
    ("bf16", 128, 4, 4, 2, [0, 4, 8], [33, 5], [34, 90, 129, 33, 5, 6, 70, 200], 16384),
    # a long prefix of a large table, with both
    ("fp16", 64, 8, 4, 16, [0, 7], [2500], [2500 + 33 * i for i in range(7)], 20480),
]


@pytest.mark.parametrize("idx", range(len(LONG)))
def test_long_prefixes_and_wide_tables(idx):
    *sizes, width = LONG[idx]
    case = Case(*sizes, seed=50 + idx, MB=width // sizes[4] if width else None)
    pa.bad_index_count(clear=True)
    out = case.run()
    assert pa.bad_index_count(clear=True) == 0
    case.check(out, what=str(sizes[:5]))
    # the bounds given size the grid and the cuts, never what is computed
    case.check(case.run(max_prefix=case.max_prefix + 1000, max_group=10 ** 6), what=str(sizes[:5]))
    assert pa.bad_index_count(clear=True) == 0


@pytest.mark.parametrize("more", [0, 80])
def test_workspace_may_hold_anything(more):
    case = Case("bf16", 128, 8, 2, 16, [0, 4 + more, 7 + more], [600, 100],
                [601, 1500, 600, 900] + [605 + i for i in range(more)] + [100, 5, 2000])
    assert case.passes() == (more > 0)
    case.upload()
    n = pa.decode_shared_prefix_workspace_bytes(7 + more, 2, 8, 2, 128, case.bt.shape[1], 16, 600, 4 + more)
    first = None
    for byte in (0, 0xFF, 0x7F, 0x80):
        out = case.run(torch.full((n,), byte, dtype=torch.uint8, device="cuda"))
        first = out if first is None else first
        assert torch.equal(out, first)
    case.check(first)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.5])
@pytest.mark.parametrize("dtype,Hq,B,more", [("bf16", 8, 16, 0), ("fp16", 14, 2, 0), ("bf16", 8, 16, 200),
                                             ("fp16", 10, 2, 200)])
def test_scales(scale, dtype, Hq, B, more):
    case = Case(dtype, 64, Hq, 2, B, [0, 3 + more, 5 + more], [400, 33],
                [400, 533, 401] + [400 + i % 50 for i in range(more)] + [40, 700], seed=70)
    assert case.passes() == (more > 0)
    case.scale = scale
    case.check(case.run())


@pytest.mark.parametrize("more", [0, 400])
def test_sequences_shorter_than_the_prefix_are_computed_alone(more):
    case = Case("bf16", 128, 8, 2, 16, [0, 6 + more], [100],
                [120, 40, 0, 100, 99, 101] + [90 + i % 30 for i in range(more)])
    assert case.passes() == (more > 0)
    case.check(case.run())


@pytest.mark.parametrize("prefix,more", [(64, 0), (512, 150)])
def test_first_member_shorter_than_the_prefix(prefix, more):
    # its table still names the prefix's blocks for the others
    case = Case("fp16", 64, 4, 2, 8, [0, 3 + more], [prefix], [prefix + 16, prefix + 26, prefix] + [prefix + 3] * more)
    assert case.passes() == (more > 0)
    case.lens[0] = 17
    case.check(case.run())


@pytest.mark.parametrize("more", [0, 160])
def test_prefixes_and_groups_above_the_bounds_given(more):
    case = Case("bf16", 128, 8, 2, 16, [0, 5, 7 + more], [300, 280],
                [301, 320, 333, 400, 350, 280, 285] + [281 + i % 40 for i in range(more)], hide=False)
    # members' tables agree with the first one's where a prefix is cut short
    for g in range(2):
        a, b, n = case.starts[g], case.starts[g + 1], case.prefixes[g]
        j = -(-n // 16)
        case.bt[a:b, :j] = case.bt[a, :j]
    case.table = case.bt.copy()
    pa.bad_index_count(clear=True)
    assert case.passes() == (more > 0)
    for mp, mg in ((100, 5), (300, 2), (0, 5), (300, 0), (64, 1), (250, 2 + more)):
        case.check(case.run(max_prefix=mp, max_group=mg), what=f"max_prefix {mp}, max_group {mg}")
        assert pa.bad_index_count(clear=True) > 0


def test_equals_decode_where_the_tables_agree():
    case = W.make_workload("shared_prefix", num_seqs=16, block_size=16)
    starts = np.array([0, 8, 16], np.int32)
    q, kd, vd = (dev_bits(x, case.dtype) for x in (case.query, case.key_cache, case.value_cache))
    bt, sl = up(case.block_tables), up(case.seq_lens)
    a, b = (torch.empty(case.query.shape, dtype=torch.float32, device="cuda") for _ in range(2))
    pa.decode(a, q, kd, vd, bt, sl, case.scale, 0, pa.alloc_workspace(q, kd, bt))
    gs, pl = up(starts), up(np.array([1024, 1024], np.int32))
    pa.decode_shared_prefix(b, q, kd, vd, bt, sl, gs, pl, 1024, 8, case.scale,
                            pa.alloc_shared_prefix_workspace(q, kd, bt, gs, 1024, 8))
    # two results, each within the bound (about 1000 tokens of N(0, 1) rows)
    assert torch.max(torch.abs(a - b)).item() <= 2e-3


def test_infinite_and_nan_slots_behind_the_lengths_are_not_read():
    case = Case("fp16", 128, 4, 2, 16, [0, 3], [70], [70, 71, 95])
    used = np.zeros(case.kc.shape[:2], bool)
    for s, n in enumerate(case.lens):
        for t in range(n):
            used[case.bt[s, t // 16], t % 16] = True
    case.kc[~used], case.vc[~used] = W.nan_bits("fp16"), W.inf_bits("fp16")
    case.check(case.run())


@pytest.mark.parametrize("prefix,more", [(64, 0), (512, 150)])
def test_bad_blocks_in_prefix_and_suffix_read_as_zeros(prefix, more):
    case = Case("bf16", 64, 4, 2, 16, [0, 3 + more], [prefix],
                [prefix + 16, prefix + 26, prefix + 36] + [prefix + 9] * more)
    assert case.passes() == (more > 0)
    case.table[0, 1] = 10 ** 6   # in the prefix, of the first member: for the whole group
    last = case.lens[2] // 16 - 1
    case.table[2, last] = -5     # in a suffix
    NB = case.kc.shape[0]
    case.upload()
    pa.bad_index_count(clear=True)
    out = case.run()
    assert pa.bad_index_count(clear=True) > 0
    case.kc, case.vc = (np.concatenate([x, np.zeros_like(x[:1])]) for x in (case.kc, case.vc))
    case.bt[0, 1], case.bt[2, last] = NB, NB
    case.check(out)


@pytest.mark.parametrize("prefix,more", [(32, 0), (512, 150)])
def test_group_starts_that_make_no_sense_touch_nothing_else(prefix, more):
    case = Case("bf16", 64, 4, 2, 16, [0, 2, 4 + more], [prefix, prefix],
                [prefix + 8, prefix + 18, prefix + 28, prefix + 1] + [prefix + 2] * more, hide=False)
    assert case.passes() == (more > 0)
    case.upload()
    case.gs = up(np.array([3, -7, 99], np.int32))
    case.pl = up(np.array([-4, 10 ** 9], np.int32))
    pa.bad_index_count(clear=True)
    out = case.run()
    assert pa.bad_index_count(clear=True) > 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("more", [0, 40])
def test_repeated_calls_and_other_calls_on_one_workspace(more):
    case = Case("bf16", 128, 8, 2, 16, [0, 12 + more], [900], [900 + 97 * i for i in range(12)] + [931] * more)
    assert case.passes() == (more > 0)
    case.upload()
    S = 12 + more
    n = pa.decode_shared_prefix_workspace_bytes(S, 1, 8, 2, 128, case.bt.shape[1], 16, 900, S)
    ws = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    first = case.run(ws)
    case.check(first)
    other = Case("fp16", 64, 4, 4, 16, [0, 40], [64], [64 + i for i in range(40)], MB=16)
    plain = torch.empty(case.query.shape, dtype=torch.float32, device="cuda")
    for _ in range(3):
        other.check(other.run(ws))
        pa.decode(plain, case.q, case.kd, case.vd, up(case.bt), case.sl, case.scale, 64,
                  torch.zeros(pa.decode_workspace_bytes(S, 8, 128, case.bt.shape[1], 16, 64), dtype=torch.uint8,
                              device="cuda"))
        assert torch.equal(case.run(ws), first)


@pytest.mark.parametrize("more", [0, 160])
def test_captured_and_replayed_with_other_lengths(more):
    case = Case("bf16", 128, 8, 2, 16, [0, 4 + more, 6 + more], [256, 64],
                [300, 280, 257, 500] + [260 + i % 33 for i in range(more)] + [70, 64])
    assert case.passes() == (more > 0)
    case.upload()
    ws = pa.alloc_shared_prefix_workspace(case.q, case.kd, case.btd, case.gs, 256, 4 + more)
    out = torch.empty(case.query.shape, dtype=torch.float32, device="cuda")

    def step():
        pa.decode_shared_prefix(out, case.q, case.kd, case.vd, case.btd, case.sl, case.gs, case.pl, 256, 4 + more,
                                case.scale, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    case.check(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens, prefixes in (([300, 280, 257, 500, 70, 64], [256, 64]), ([290, 256, 257, 300, 66, 65], [128, 33]),
                           ([10, 20, 30, 0, 70, 64], [0, 64])):
        case.lens[:4], case.lens[4 + more:], case.prefixes[:] = lens[:4], lens[4:], prefixes
        case.btd.copy_(torch.from_numpy(case.bt))
        case.sl.copy_(torch.from_numpy(case.lens))
        case.pl.copy_(torch.from_numpy(case.prefixes))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        case.check(out)


def test_candidates_of_forked_prompts():
    """The block manager's forks give the groups: candidates of a prompt share
    its blocks, diverge by copy-on-write, and are decoded with the prompt as prefix."""
    rng = np.random.default_rng(1)
    dtype, B, Hq, Hkv, d, NB, MB = "bf16", 16, 8, 2, 64, 120, 16
    bm = pa.BlockManager(NB, B, MB)
    kc = torch.zeros(NB, B, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    made, hist, live, starts, prefixes = [0], {}, [], [0], []

    def write(requests):
        total = sum(n for _, n in requests)
        made[0] += 2
        rows = [W.normal_bits((total, Hkv, d), dtype, 60, made[0] + i) for i in range(2)]
        slots, copies = bm.append(requests)
        if copies:
            src, dst = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in zip(*copies))
            pa.copy_blocks(kc, vc, src, dst)
        pa.reshape_and_cache(*(dev_bits(r, dtype) for r in rows), kc, vc, up(slots))
        at = 0
        for s, n in requests:
            hist.setdefault(s, []).append([r[at:at + n] for r in rows])
            at += n

    for prompt, candidates in ((37, 4), (64, 1), (100, 6)):
        s = bm.new_sequence()
        write([(s, prompt)])
        group = [s]
        for _ in range(candidates - 1):
            c = bm.fork(s)
            hist[c] = list(hist[s])
            group.append(c)
        live += group
        starts.append(len(live))
        prefixes.append(prompt)
    gs, pl = up(np.array(starts, np.int32)), up(np.array(prefixes, np.int32))
    scale = 1 / np.sqrt(d)
    for step in range(5):
        write([(s, 1) for s in live])
        bt, lens = bm.block_tables(live)
        query = W.normal_bits((len(live), Hq, d), dtype, 61, step)
        q, btd = dev_bits(query, dtype), up(bt)
        out = torch.empty(query.shape, dtype=torch.float32, device="cuda")
        pa.decode_shared_prefix(out, q, kc, vc, btd, up(lens), gs, pl, 100, 6, scale,
                                pa.alloc_shared_prefix_workspace(q, kc, btd, gs, 100, 6))
        G = Hq // Hkv
        for i, s in enumerate(live):
            K, V = (oracle.to_float64(np.concatenate(x), dtype) for x in zip(*hist[s]))
            qf = oracle.to_float64(query[i], dtype)
            ref = np.concatenate([oracle.single_query_attention(qf[h * G:(h + 1) * G], K[:, h], V[:, h], scale)[0]
                                  for h in range(Hkv)])
            tol = fp8.decode_bound(qf, K, V, scale, WEIGHT_ERROR[dtype])
            assert np.max(np.abs(out[i].double().cpu().numpy() - ref)) <= tol
    bm.close()
