"""Cases of the operators around a serving step's attention, and of the 4-bit cache.

A case is one call as a serving loop makes it:

* ``append``  append_tokens: block tables, slots and positions of a step's new tokens, on the GPU
* ``rotate``  rotate / rotate_and_cache: norms of Q's and K's heads and their rotation by position
  in one pass, with K and V written into the 16-bit pool (``cache``) or K given back
* ``write``   reshape_and_cache_fp4: new K/V rows are quantised into the 4-bit pool
* ``gather``  gather_cache_fp4: whole sequences are read back as 16-bit rows
* ``decode``  decode_fp4: decode attention straight from the 4-bit pool

The 4-bit pool holds e2m1 codes [blocks, block_size, kv_heads, head_dim / 2] for K and for V, element
2 i in the low half of byte i and 2 i + 1 in the high half, and one byte for every 32 elements of a row:
byte e of ``scales`` [blocks, kv_heads, 2 (K, V), block_size, head_dim / 32] stands for 2**(e - 127).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 32  # elements of a row that share a power of two
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    gqa = dict(kv_heads=8, head_dim=128, block_size=16)
    return [
        # one decode step of a small batch takes its slots: the smallest call
        dict(name="append_step", op="append", seqs=4, min_len=1, max_len=128, min_new=1, max_new=1, block_size=16),
        # ragged prompts and chunks of a batch, 32 K tokens in all
        dict(name="append_prompts", op="append", seqs=64, min_len=0, max_len=4096, min_new=1, max_new=1023,
             block_size=16),
        # one decode step of 128 sequences, norms of the heads, straight into the pool
        dict(name="rotate_step", op="rotate", dtype="bf16", cache=True, norm=True, layout="half", tokens=128, q_heads=32,
             rotary_dim=128, last=8192, scaled=False, **gqa),
        # the prompts of a batch at far positions, frequencies scaled for a long context
        dict(name="rotate_prompts", op="rotate", dtype="bf16", cache=True, norm=False, layout="half", tokens=32768,
             q_heads=32, rotary_dim=128, last=131072, scaled=True, **gqa),
        # half of every head, neighbours as pairs, odd sizes; K is given back for a quantising write
        dict(name="rotate_partial", op="rotate", dtype="fp16", cache=False, norm=True, layout="interleaved", tokens=777,
             q_heads=6, kv_heads=3, head_dim=64, block_size=16, rotary_dim=32, last=2048, scaled=False),
        # one decode step of a small batch writes its new rows
        dict(name="write4_step", op="write", dtype="fp16", tokens=4, kv_heads=4, head_dim=64, block_size=16),
        # the prompts of a batch enter the cache in one call
        dict(name="write4_prompts", op="write", dtype="bf16", tokens=32768, **gqa),
        # short ragged contexts are read back for the next prompt chunk
        dict(name="gather4_short", op="gather", dtype="fp16", seqs=5, min_len=1, max_len=333, kv_heads=4, head_dim=64,
             block_size=8),
        # 16 contexts of about 4K tokens are read back for chunked prefill
        dict(name="gather4_chunks", op="gather", dtype="bf16", seqs=16, min_len=2049, max_len=6143, **gqa),
        # the tiny workload: 4 heads of 64, at most 128 tokens
        dict(name="decode4_tiny", op="decode", dtype="fp16", seqs=4, min_len=1, max_len=128, q_heads=4, kv_heads=4,
             head_dim=64, block_size=16),
        # 128 sequences of 1K to 8K tokens, 4 query heads a kv head
        dict(name="decode4_gqa", op="decode", dtype="bf16", seqs=128, min_len=1024, max_len=8192, q_heads=32, **gqa),
        # 8 sequences of 32K to 128K tokens, 8 query heads a kv head
        dict(name="decode4_long", op="decode", dtype="bf16", seqs=8, min_len=32768, max_len=131072, q_heads=64, **gqa),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "rotate", "rotate", "write", "gather", "decode", "decode"))
    c = dict(op=op, block_size=rng.choice((1, 2, 4, 8, 16, 16, 32, 64)))
    if op == "append":
        c["seqs"] = _log(rng, 1, 1024)
        c["max_len"] = _log(rng, 1, 16384)
        c["min_len"] = rng.randint(0, c["max_len"])
        c["max_new"] = _log(rng, 1, max(1, min(8192, 65536 // c["seqs"])))
        c["min_new"] = rng.randint(0, c["max_new"])
        return c
    c |= dict(kv_heads=rng.choice((1, 2, 3, 4, 5, 8, 16)), head_dim=rng.choice((64, 128, 128)))
    slot = c["kv_heads"] * c["head_dim"]  # values of one tensor's row of a token
    c["dtype"] = rng.choice(("bf16", "fp16"))
    if op == "write":
        c["tokens"] = _log(rng, 1, min(32768, (1 << 25) // slot))
        return c
    if op == "gather":
        c["seqs"] = _log(rng, 1, 64)
        c["max_len"] = _log(rng, 1, max(1, min(16384, (1 << 26) // slot // c["seqs"])))
        c["min_len"] = rng.randint(0, c["max_len"])
        return c
    c["q_heads"] = c["kv_heads"] * rng.choice((1, 2, 3, 4, 7, 8, 16))
    if op == "rotate":
        d = c["head_dim"]
        c["tokens"] = _log(rng, 1, max(1, min(32768, (1 << 27) // ((c["q_heads"] + 2 * c["kv_heads"]) * d))))
        c["rotary_dim"] = rng.choice((16, d // 4, d // 2, d // 2 + 16, d, d, d))
        c |= dict(cache=rng.random() < 0.6, norm=rng.random() < 0.5, layout=rng.choice(("half", "interleaved")),
                  last=_log(rng, c["tokens"], 1 << 20), scaled=rng.random() < 0.5)
        return c
    c["seqs"] = _log(rng, 1, 200)
    c["max_len"] = _log(rng, 1, max(1, min(65536, (1 << 27) // slot // c["seqs"])))
    c["min_len"] = rng.randint(0, c["max_len"])
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers, evenly from lo to hi: the same sum whatever the order."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _rows(gen, n, case, dtype, heads=None):
    """n rows of queries, keys or values: normal, with a gain for each channel as projections have."""
    heads = heads or case["kv_heads"]
    gain = torch.exp(0.5 * torch.randn(heads, case["head_dim"], device="cuda", generator=gen))
    x = torch.randn(n, heads, case["head_dim"], device="cuda", generator=gen)
    return x.mul_(gain).to(dtype)


def _factors(e):
    """2**(e - 127) for bytes 1 to 254, zero for 0 and infinity for 255: the exponent field of an fp32 number."""
    return (e.int() << 23).view(torch.float32)


def _quantise4(x):
    """Codes [.., d] (0 to 15) and bytes [.., d / 32] of rows x: the smallest factor of which 7 reaches the group."""
    x = x.float().unflatten(-1, (-1, GROUP))
    top = x.abs().amax(-1)
    f, e = torch.frexp(top)
    e = (e + 127 - 3 + (f > 0.875)).clamp(1, 252)  # 7 = 0.875 * 2**3; 6 times the largest factor is finite
    e = torch.where(top > 0, e, 0)
    lost = ~torch.isfinite(x).all(-1)
    y = (x * _factors(254 - e).unsqueeze(-1)).masked_fill(lost.unsqueeze(-1), 0.0)
    a = y.abs()
    # nearest code, ties to the even one
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    code = code + 8 * torch.signbit(y)
    return code.to(torch.uint8).flatten(-2), torch.where(lost, 255, e).to(torch.uint8)


def _pack(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def _pool4(gen, blocks, case, dtype=torch.bfloat16):
    """A 4-bit pool whose every row has been written."""
    B, H, d = case["block_size"], case["kv_heads"], case["head_dim"]
    packed, bytes_ = [], []
    for _ in range(2):
        k, e = zip(*(_quantise4(r) for r in _rows(gen, blocks * B, case, dtype).split(1 << 17)))
        packed.append(torch.cat([_pack(c) for c in k]).view(blocks, B, H, d // 2))
        bytes_.append(torch.cat(e).view(blocks, B, H, -1).transpose(1, 2))
    return packed[0], packed[1], torch.stack(bytes_, 2).contiguous()


def _inverse_frequencies(case):
    """Radians a position of every pair, 64-bit; scaled: wavelengths above a context of 8192 slowed down eightfold,
    those under a quarter of it kept, in between by parts."""
    n = case["rotary_dim"] // 2
    w = [10000.0 ** (-i / n) for i in range(n)]
    if case["scaled"]:
        for i, f in enumerate(w):
            turns = 8192.0 * f / (2.0 * math.pi)
            keep = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            w[i] = f * keep + f / 8.0 * (1.0 - keep)
    return w


def _tables(gen, lens, room, case):
    """Random distinct blocks for every sequence (room[s] of them), and the pool's size."""
    S, width = len(lens), max(1, max(room))
    blocks = sum(room) + sum(room) // 5 + 1
    order = torch.randperm(blocks, device="cuda", generator=gen).int()
    first = torch.tensor([sum(room[:s]) for s in range(S)], device="cuda").unsqueeze(1)
    at = torch.arange(width, device="cuda")
    return order[(first + at) % blocks].contiguous(), blocks, order


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    op, B = case["op"], case["block_size"]
    st = dict(op=op, block_size=B)
    if op == "append":
        lens = _spread(case["min_len"], case["max_len"], case["seqs"])
        new = _spread(case["min_new"], case["max_new"], case["seqs"])
        rng.shuffle(lens)
        rng.shuffle(new)
        S = len(lens)
        held = [-(-n // B) for n in lens]
        more = [-(-(n + m) // B) - h for n, m, h in zip(lens, new, held)]
        starts = [sum(new[:s]) for s in range(S + 1)]
        tables, blocks, order = _tables(gen, lens, held, case)
        width = -(-(case["max_len"] + case["max_new"]) // B) + 3  # what the longest may come to, and more
        st["tables"] = torch.zeros(S, width, dtype=torch.int32, device="cuda")
        st["tables"][:, :tables.shape[1]] = tables
        # the free list holds more than the step needs; a padded batch has rows behind the last token
        spare = sum(more) + sum(more) // 4 + 2
        st["free"] = torch.cat([torch.randperm(spare, device="cuda", generator=gen).int() + blocks,
                                torch.zeros(5, dtype=torch.int32, device="cuda")])
        st["num_blocks"] = blocks + spare
        st["num_free"] = torch.tensor([spare], dtype=torch.int32, device="cuda")
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        rows = starts[-1] + 3
        st["slots"] = torch.zeros(rows, dtype=torch.int64, device="cuda")
        st["positions"] = torch.zeros(rows, dtype=torch.int64, device="cuda")
        st["new_lens"] = torch.zeros_like(st["lens"])
        st["new_free"] = torch.zeros_like(st["num_free"])
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return st
    H, d = case["kv_heads"], case["head_dim"]
    dtype = DTYPES[case["dtype"]]
    if op == "rotate":
        T, Hq = case["tokens"], case["q_heads"]
        # one projection's output: Q, K and V of a token beside each other
        qkv = torch.cat([_rows(gen, T, case, dtype, h) for h in (Hq, H, H)], 1)
        st["query"], st["key"], st["value"] = qkv.split((Hq, H, H), 1)
        st["query_out"] = torch.empty(T, Hq, d, dtype=dtype, device="cuda")
        first = torch.randint(0, case["last"] - T + 1, (1,), device="cuda", generator=gen)
        st["positions"] = first + torch.arange(T, device="cuda")
        if T <= 256:  # a decode step: every token is another sequence's
            st["positions"] = torch.randint(0, case["last"], (T,), device="cuda", generator=gen)
        st |= dict(inverse=_inverse_frequencies(case), interleaved=case["layout"] == "interleaved",
                   factor=1.0 + 0.1 * math.log(8.0) if case["scaled"] else 1.0)
        st["weights"] = tuple((1.0 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(dtype) for _ in range(2)) \
            if case["norm"] else (None, None)
        if case["cache"]:
            blocks = -(-T // B) * 5 // 4 + 1
            st["pool"] = [_rows(gen, blocks * B, case, dtype).view(blocks, B, H, d) for _ in range(2)]
            order = torch.randperm(blocks, device="cuda", generator=gen)
            t = torch.arange(T, device="cuda")
            st["slots"] = order[t // B] * B + t % B
            if T > 8:
                st["slots"][7::64] = -1  # padded tokens have no slot
        else:
            st["key_out"] = torch.empty(T, H, d, dtype=dtype, device="cuda")
        return st
    if op == "write":
        T = case["tokens"]
        blocks = -(-T // B) * 5 // 4 + 1
        st["pool"] = _pool4(gen, blocks, case)
        st["key"], st["value"] = _rows(gen, T, case, dtype), _rows(gen, T, case, dtype)
        # whole blocks in random order, filled one after the other; a padded token has no slot
        order = torch.randperm(blocks, device="cuda", generator=gen)
        t = torch.arange(T, device="cuda")
        st["slots"] = order[t // B] * B + t % B
        if T > 8:
            st["slots"][7::64] = -1
        return st
    lens = _spread(case["min_len"], case["max_len"], case["seqs"])
    rng.shuffle(lens)
    held = [-(-n // B) for n in lens]
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["tables"], blocks, _ = _tables(gen, lens, held, case)
    st["pool"] = _pool4(gen, blocks, case)
    if op == "gather":
        # each sequence's rows start at a whole block of the output
        starts = [B * sum(held[:s]) for s in range(len(lens))]
        st["starts"] = torch.tensor(starts, dtype=torch.int64, device="cuda")
        st["key"], st["value"] = (torch.zeros(max(1, B * sum(held)), H, d, dtype=dtype, device="cuda") for _ in range(2))
        return st
    st["scale"] = 1.0 / math.sqrt(d)
    st["query"] = torch.randn(len(lens), case["q_heads"], d, device="cuda", generator=gen).to(dtype)
    st["out"] = torch.empty_like(st["query"])
    return st


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _plain_append(st):
    B, lens, starts, tables = st["block_size"], st["lens"].long(), st["starts"].long(), st["tables"]
    new_lens = lens + starts.diff()
    held, want = (lens + B - 1) // B, (new_lens + B - 1) // B
    more = want - held
    before = more.cumsum(0) - more
    left = st["num_free"].long() - more.sum()
    # new entries of the tables: the free list from its end, in the sequences' order
    at = torch.arange(tables.shape[1], device=lens.device)
    popped = st["num_free"].long() - 1 - (before.unsqueeze(1) + at - held.unsqueeze(1))
    fresh = (at >= held.unsqueeze(1)) & (at < want.unsqueeze(1))
    tables = torch.where(fresh, st["free"][popped.clamp(0, st["free"].shape[0] - 1)], tables)
    row = torch.arange(st["slots"].shape[0], device=lens.device)
    s = torch.searchsorted(starts, row, right=True).sub(1).clamp(max=lens.shape[0] - 1)
    live = row < starts[-1]
    position = torch.where(live, lens[s] + row - starts[s], 0)
    slot = tables[s, (position // B).clamp(max=tables.shape[1] - 1)].long() * B + position % B
    return {"tables": tables, "lens": new_lens.int(), "free": left.int(), "slots": torch.where(live, slot, -1),
            "positions": position}


def _norm(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _turn(x, cos, sin, interleaved):
    """The first 2 n elements of every head rotated in pairs, n = cos.shape[-1]."""
    n = cos.shape[-1]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    else:
        a, b = x[..., :n], x[..., n:2 * n]
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _plain_rotate(st):
    # angles of far positions need 64 bits, their sines do not
    if "turn" not in st:
        st["turn"] = torch.tensor(st["inverse"], dtype=torch.float64, device="cuda")
    angle = st["positions"].double().unsqueeze(1) * st["turn"]
    cos, sin = (angle.cos() * st["factor"]).float(), (angle.sin() * st["factor"]).float()
    dtype = st["query"].dtype
    q = _turn(_norm(st["query"], st["weights"][0]), cos, sin, st["interleaved"]).to(dtype)
    k = _turn(_norm(st["key"], st["weights"][1]), cos, sin, st["interleaved"]).to(dtype)
    if "pool" not in st:
        return {"query": q, "key": k}
    keep = st["slots"] >= 0
    for pool, rows in zip(st["pool"], (k, st["value"])):
        pool.flatten(0, 1)[st["slots"][keep]] = rows[keep]
    return {"query": q, "key": st["pool"][0], "value": st["pool"][1]}


def _plain_write(st):
    kc, vc, scales = st["pool"]
    B, slots = kc.shape[1], st["slots"]
    keep = slots >= 0
    block, at = slots[keep] // B, slots[keep] % B
    for which, (pool, rows) in enumerate(((kc, st["key"]), (vc, st["value"]))):
        codes, e = _quantise4(rows[keep])
        pool[block, at] = _pack(codes)
        scales[block, :, which, at] = e
    return {"key": kc, "value": vc, "scales": scales}


def _slots(tables, tokens, B):
    """Slot of every token 0 .. tokens - 1 of every sequence."""
    t = torch.arange(tokens, device=tables.device)
    return tables[:, t // B].long() * B + t % B


def _read4(st, which, slots):
    """Rows of K (0) or V (1) at these slots as fp32 values."""
    codes, scales = st["pool"][which], st["pool"][2]
    B = codes.shape[1]
    c = codes.flatten(0, 1)[slots].int()
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=c.device)
    x = torch.stack([value[c & 15], value[c >> 4]], -1).flatten(-2)
    f = _factors(scales[slots // B, :, which, slots % B])
    return (x.unflatten(-1, (-1, GROUP)) * f.unsqueeze(-1)).flatten(-2)


def _plain_gather(st):
    B, L = st["block_size"], st["seq_lens"]
    tokens = st["tables"].shape[1] * B
    t = torch.arange(tokens, device=L.device)
    here = t < L.unsqueeze(1)
    slots = _slots(st["tables"], tokens, B)[here]
    rows = (st["starts"].unsqueeze(1) + t)[here]
    st["key"][rows] = _read4(st, 0, slots).to(st["key"].dtype)
    st["value"][rows] = _read4(st, 1, slots).to(st["value"].dtype)
    return {"key": st["key"], "value": st["value"]}


def _plain_decode(st):
    """softmax(scale * q K) V of every sequence over its first seq_lens tokens, in 32 bits."""
    q, L = st["query"], st["seq_lens"]
    slots = _slots(st["tables"], st["tables"].shape[1] * st["block_size"], st["block_size"])
    S, Hq, d = q.shape
    K = _read4(st, 0, slots)
    H = K.shape[2]
    x = torch.einsum("shgd,sthd->shgt", q.float().view(S, H, Hq // H, d), K) * st["scale"]
    del K
    here = (torch.arange(slots.shape[1], device=L.device) < L.unsqueeze(1)).view(S, 1, 1, -1)
    x = torch.where(here, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.where(here, torch.exp(x - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("shgt,sthd->shgd", p, _read4(st, 1, slots)) / torch.where(total > 0, total, 1.0)
    return o.reshape(S, Hq, d).to(q.dtype)


def _own(st):
    import paged_kv_cache_305_gb300 as pa
    op = st["op"]
    if op == "append":
        pa.append_tokens(st["new_lens"], st["new_free"], st["slots"], st["positions"], st["tables"], st["lens"],
                         st["starts"], st["free"], st["num_free"], st["status"], st["block_size"], st["num_blocks"])
        return {"tables": st["tables"], "lens": st["new_lens"], "free": st["new_free"], "slots": st["slots"],
                "positions": st["positions"]}
    if op == "rotate":
        if "frequencies" not in st:
            st["frequencies"] = pa.rotary_frequencies(st["inverse"], device="cuda")
        more = dict(interleaved=st["interleaved"], factor=st["factor"], query_weight=st["weights"][0],
                    key_weight=st["weights"][1], eps=EPS)
        if "pool" not in st:
            pa.rotate(st["query_out"], st["key_out"], st["query"], st["key"], st["positions"], st["frequencies"], **more)
            return {"query": st["query_out"], "key": st["key_out"]}
        pa.rotate_and_cache(st["query_out"], st["query"], st["key"], st["value"], *st["pool"], st["slots"],
                            st["positions"], st["frequencies"], **more)
        return {"query": st["query_out"], "key": st["pool"][0], "value": st["pool"][1]}
    if op == "write":
        pa.reshape_and_cache_fp4(st["key"], st["value"], *st["pool"], st["slots"])
        return dict(zip(("key", "value", "scales"), st["pool"]))
    if op == "gather":
        pa.gather_cache_fp4(st["key"], st["value"], *st["pool"], st["tables"], st["seq_lens"], st["starts"])
        return {"key": st["key"], "value": st["value"]}
    if "workspace" not in st:
        st["workspace"] = pa.alloc_workspace(st["query"], st["pool"][0], st["tables"])
    return pa.decode_fp4(st["out"], st["query"], *st["pool"], st["tables"], st["seq_lens"], st["scale"],
                         workspace=st["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "rotate": _plain_rotate, "write": _plain_write, "gather": _plain_gather,
            "decode": _plain_decode}[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    B = case["block_size"]
    if case["op"] == "append":
        # the order in which lengths and new tokens meet is the seed's: blocks on the average
        S = case["seqs"]
        T = sum(_spread(case["min_new"], case["max_new"], S))
        fresh = -(-T // B)
        return {"bytes": 4 * (2 * S + 1) + 4 * S + 4 * fresh + 4 * S + 4 * fresh + 16 * (T + 3) + 8, "flops": 0}
    H, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "rotate":
        T, Hq = case["tokens"], case["q_heads"]
        n = T - (len(range(7, T, 64)) if T > 8 and case["cache"] else 0)  # tokens whose K and V are written
        heads = T * Hq + n * H
        rows = heads + (n * H if case["cache"] else 0)
        return {"bytes": 4 * d * rows + 8 * T * (2 if case["cache"] else 1) + 4 * case["rotary_dim"]
                + (4 * d if case["norm"] else 0),
                "flops": heads * (3 * case["rotary_dim"] + (4 * d if case["norm"] else 0))}
    row4 = 2 * H * (d // 2 + d // GROUP)  # K and V codes of a token and their exponents
    if case["op"] == "write":
        n = case["tokens"] - (len(range(7, case["tokens"], 64)) if case["tokens"] > 8 else 0)
        return {"bytes": n * (2 * H * d * 2 + row4) + 8 * case["tokens"], "flops": 4 * n * H * d}
    lens = _spread(case["min_len"], case["max_len"], case["seqs"])
    n = sum(lens)
    tables = 4 * sum(-(-x // B) for x in lens) + 4 * len(lens)
    if case["op"] == "gather":
        return {"bytes": n * (row4 + 2 * H * d * 2) + tables + 8 * len(lens), "flops": 2 * n * H * d}
    ends = 2 * len(lens) * case["q_heads"] * d * 2  # queries and outputs
    return {"bytes": n * row4 + tables + ends, "flops": 4 * n * case["q_heads"] * d}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_rotate(st, case):
    out = {}
    n = case["rotary_dim"] // 2
    angle = torch.tensor([[p * w for w in st["inverse"]] for p in st["positions"].tolist()], dtype=torch.float64,
                         device="cuda")
    spin = torch.polar(torch.full_like(angle, st["factor"]), angle).unsqueeze(1)  # a pair is a complex number
    for name, weight in zip(("query", "key"), st["weights"]):
        x = st[name].double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
        head = x[..., :2 * n]
        pair = head.unflatten(-1, (n, 2)) if case["layout"] == "interleaved" else head.unflatten(-1, (2, n)).mT
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * spin)
        z = z if case["layout"] == "interleaved" else z.mT
        out[name] = torch.cat([z.flatten(-2), x[..., 2 * n:]], -1)
    if not case["cache"]:
        return out
    key, keep = out["key"], st["slots"] >= 0
    for name, pool, rows in (("key", st["pool"][0], key), ("value", st["pool"][1], st["value"].double())):
        v = pool.double()
        v.view(-1, *v.shape[2:])[st["slots"][keep]] = rows[keep]
        out[name] = v
    return out


def _exact_value(st, block, at, which):
    """Rows of K (0) or V (1) in 64 bits: both halves of every byte, in order, times the power of two of their 32."""
    c = st["pool"][which][block, at].long()
    c = torch.stack([c % 16, c // 16], -1).flatten(-2)
    m, e = c % 2, c // 2 % 4
    x = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * torch.exp2(e.double() - 1.0))
    x = torch.where(c >= 8, -x, x)
    f = torch.exp2(st["pool"][2][block, :, which, at].double() - 127.0)
    return x * f.repeat_interleave(GROUP, -1)


def exact(case, seed):
    op, B = case["op"], case["block_size"]
    if op in ("append", "write"):
        return None  # whole numbers: bytes of two codes, exponents, tables and slots
    st = prepare(case, seed)
    if op == "rotate":
        return _exact_rotate(st, case)
    lens = st["seq_lens"].tolist()
    out = {"key": st["key"].double(), "value": st["value"].double()} if op == "gather" else []
    for s, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        K, V = (_exact_value(st, st["tables"][s, t // B].long(), t % B, i) for i in range(2))
        if op == "gather":
            a = int(st["starts"][s])
            out["key"][a:a + n], out["value"][a:a + n] = K, V
        else:
            q = st["query"][s].double()
            if n == 0:
                out.append(torch.zeros_like(q))
                continue
            x = torch.matmul(q.view(K.shape[1], -1, q.shape[-1]), K.permute(1, 2, 0)) * st["scale"]
            out.append(torch.matmul(torch.softmax(x, -1), V.transpose(0, 1)).reshape(q.shape))
    return out if op == "gather" else torch.stack(out)
