"""What the operators around a smaller K/V cache cost: the cache held in 4 bits (its write, its read-back and
the decode attention over it), the decode that accumulates each cached token's attention weight, and the
eviction that keeps the tokens with the most of it.

The 4-bit format: 16 elements share a scale in e4m3, each element is an e2m1 code, and a pool has a scale that
is a power of two; the value is code * scale * pool scale.  A pool is uint8
[num_blocks, num_kv_heads, block_size, head_dim * 9 / 16]; the bytes of one (block, kv head) hold block_size
rows of head_dim / 2 code bytes (element 2i in the low half of byte i) and then block_size rows of
head_dim / 16 scale bytes.

A case names its operator in "op":
  store    new tokens' K/V into a 4-bit pool, and the same slots read back (the values that the pool holds)
  decode   one query a sequence over a 4-bit pool
  weights  the decode over a 16-bit pool ("kv": "16") or a 4-bit one ("kv": "fp4") that adds every cached
           token's attention weight, summed over the query heads of its kv head, to the sequence's row
  evict    the tokens with the most weight kept, between the first `sinks` and the last `recent` ones, and
           moved together in their order, in place or into fresh blocks
"""

import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decode step's new tokens, a few of them padding
        {"name": "store_step", "op": "store", "tokens": 256, "pad": 5, "heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16"},
        # an odd count of new tokens of a small head, small blocks
        {"name": "store_odd", "op": "store", "tokens": 777, "pad": 0, "heads": 4, "dim": 64, "block": 8,
         "dtype": "fp16"},
        # a prefill chunk of 64 sequences, 256 tokens each
        {"name": "store_chunk", "op": "store", "tokens": 16384, "pad": 0, "heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16"},
        # one user's short chat: latency
        {"name": "decode_one", "op": "decode", "seqs": 1, "median": 1027, "sigma": 0.0, "most": 1027, "empty": 0,
         "lens_seed": 1, "q_heads": 32, "heads": 8, "dim": 128, "block": 16, "dtype": "bf16"},
        # the benchmark's decode step: 256 sequences of ragged lengths, grouped heads
        {"name": "decode_ragged", "op": "decode", "seqs": 256, "median": 1024, "sigma": 0.75, "most": 8192, "empty": 0,
         "lens_seed": 2, "q_heads": 32, "heads": 8, "dim": 128, "block": 16, "dtype": "bf16"},
        # long contexts with a kv head for every query head
        {"name": "decode_long", "op": "decode", "seqs": 8, "median": 32768, "sigma": 0.0, "most": 32768, "empty": 0,
         "lens_seed": 3, "q_heads": 40, "heads": 40, "dim": 128, "block": 16, "dtype": "fp16"},
        # a tiny batch with an empty slot and small heads: latency
        {"name": "weights_tiny", "op": "weights", "kv": "16", "seqs": 5, "median": 60, "sigma": 0.9, "most": 100,
         "empty": 1, "lens_seed": 4, "q_heads": 4, "heads": 4, "dim": 64, "block": 16, "dtype": "fp16"},
        # the benchmark's decode step, its weights accumulated
        {"name": "weights_ragged", "op": "weights", "kv": "16", "seqs": 256, "median": 1024, "sigma": 0.75,
         "most": 8192, "empty": 0, "lens_seed": 2, "q_heads": 32, "heads": 8, "dim": 128, "block": 16,
         "dtype": "bf16"},
        # eight query heads a kv head, over the 4-bit pool
        {"name": "weights_fp4", "op": "weights", "kv": "fp4", "seqs": 128, "median": 2304, "sigma": 0.1, "most": 2561,
         "empty": 0, "lens_seed": 5, "q_heads": 64, "heads": 8, "dim": 128, "block": 16, "dtype": "bf16"},
        # the steady state: a block's worth of new tokens over the budget
        {"name": "evict_step", "op": "evict", "kv": "16", "seqs": 64, "median": 1040, "sigma": 0.0, "most": 1040,
         "empty": 0, "lens_seed": 6, "budget": 1024, "sinks": 4, "recent": 256, "skip": 0, "fresh": False, "heads": 8,
         "dim": 128, "block": 16, "dtype": "bf16"},
        # prompts cut down after their prefill, into fresh blocks (theirs are shared)
        {"name": "evict_prompt", "op": "evict", "kv": "16", "seqs": 16, "median": 5000, "sigma": 0.5, "most": 8192,
         "empty": 0, "lens_seed": 7, "budget": 1024, "sinks": 4, "recent": 128, "skip": 1, "fresh": True, "heads": 8,
         "dim": 128, "block": 16, "dtype": "bf16"},
        # two long contexts cut to a quarter, in place
        {"name": "evict_long", "op": "evict", "kv": "16", "seqs": 2, "median": 65536, "sigma": 0.0, "most": 65536,
         "empty": 0, "lens_seed": 8, "budget": 16384, "sinks": 16, "recent": 1024, "skip": 0, "fresh": False,
         "heads": 8, "dim": 128, "block": 32, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "decode", "decode", "weights", "weights", "evict"])
    case = {"op": op, "dim": rng.choice([64, 128, 128, 128]), "block": rng.choice([8, 16, 16, 32]),
            "dtype": rng.choice(["bf16", "fp16"]), "heads": rng.choice([1, 2, 4, 5, 8, 8, 16, 32])}
    if op == "store":
        case["tokens"] = _log(rng, 1, 16384 * 8 // max(case["heads"], 8))
        case["pad"] = rng.choice([0, 0, case["tokens"] // 7])
        return case
    if op != "decode":
        case["kv"] = rng.choice(["16", "16", "fp4"])
    if op in ("decode", "weights"):
        case["q_heads"] = case["heads"] * rng.choice([1, 2, 4, 4, 8])
        budget = (10_000_000 if op == "decode" else 2_500_000) // case["heads"]  # tokens of the whole batch
    else:
        budget = 1_048_576 // case["heads"]
    case["seqs"] = _log(rng, 1, 256)
    most = max(16, min(65536, budget // case["seqs"]))
    case["median"] = _log(rng, 1, most)
    case["sigma"] = rng.choice([0.0, 0.4, 0.75])
    case["most"] = min(most, 4 * case["median"])
    case["empty"] = rng.choice([0, 0, 1]) if case["seqs"] > 1 else 0
    case["lens_seed"] = rng.randrange(1 << 30)
    if op == "evict":
        case["budget"] = _log(rng, 1, max(1, case["median"]))
        case["sinks"] = rng.choice([0, 1, 4, 17])
        case["recent"] = rng.choice([0, 1, case["budget"] // 8, case["budget"] // 2])
        case["skip"] = rng.choice([0, 0, 1])
        case["fresh"] = rng.random() < 0.4
    return case


def _lens(case):
    """The batch's lengths: the same for every seed, `empty` sequences of none first."""
    rng = random.Random(case["lens_seed"])
    lens = [max(1, min(case["most"], round(case["median"] * math.exp(case["sigma"] * rng.gauss(0.0, 1.0)))))
            for _ in range(case["seqs"])]
    for i in range(case["empty"]):
        lens[i] = 0
    return lens


def _kept_lens(case):
    """Tokens that each sequence keeps; None for one that is left as it is."""
    lens = _lens(case)
    left = set(range(case["seqs"] - case["skip"], case["seqs"]))
    return [None if s in left else min(n, case["budget"]) for s, n in enumerate(lens)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _quantise(x, pool_scale):
    """Codes (uint8, 0 to 15) and scale bytes of float32 x [..., dim]: per 16 elements, the scale is the largest
    magnitude over 6 in e4m3, and each element over it rounds to the nearest e2m1 value, ties to the even code."""
    y = (x / pool_scale).unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    r = torch.where(s > 0, y.abs() / s, torch.zeros_like(y))
    code = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0))
    code = code + 8 * ((y < 0) & (s > 0))
    return code.to(torch.uint8).flatten(-2), scale.view(torch.uint8)


def _values(codes, scales, pool_scale):
    """float32 values of codes [..., dim] and scale bytes [..., dim / 16]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    s = scales.view(torch.float8_e4m3fn).float() * pool_scale
    return (table[codes.int()].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _pack(codes, scales):
    """The tile bytes [..., block, dim * 9 / 16] of codes [..., block, dim] and scale bytes [..., block, dim / 16]."""
    data = codes[..., 0::2] | (codes[..., 1::2] << 4)
    block, row = codes.shape[-2], codes.shape[-1] * 9 // 16
    return torch.cat([data.flatten(-2), scales.flatten(-2)], -1).unflatten(-1, (block, row)).contiguous()


def _unpack(tiles, dim):
    """Codes [..., block, dim] and scale bytes [..., block, dim / 16] of tile bytes [..., block, dim * 9 / 16]."""
    block = tiles.shape[-2]
    flat = tiles.flatten(-2)
    data = flat[..., : block * dim // 2].unflatten(-1, (block, dim // 2))
    scales = flat[..., block * dim // 2:].unflatten(-1, (block, dim // 16))
    return torch.stack([data & 15, data >> 4], -1).flatten(-2), scales.contiguous()


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _gain(g, heads, dim):
    """Keys have channels that are larger than the rest in every token."""
    gain = torch.exp(0.4 * torch.randn((heads, 1, dim), generator=g, device="cuda"))
    return gain / gain.square().mean(-1, keepdim=True).sqrt()


def _pools(case, g, num_blocks):
    """K and V pools: 16-bit, or 4-bit with the pools' scales."""
    heads, block, dim = case["heads"], case["block"], case["dim"]
    fp4 = case["op"] in ("store", "decode") or case["kv"] == "fp4"
    row = dim * 9 // 16 if fp4 else dim
    gain = _gain(g, heads, dim)
    pools = []
    step = max(1, (1 << 27) // (heads * block * dim))
    for part in range(2):
        pool = torch.empty((num_blocks, heads, block, row), dtype=torch.uint8 if fp4 else DTYPES[case["dtype"]],
                           device="cuda")
        for b in range(0, num_blocks, step):
            n = min(step, num_blocks - b)
            x = torch.randn((n, heads, block, dim), generator=g, device="cuda")
            x = x * gain if part == 0 else x
            pool[b: b + n] = _pack(*_quantise(x, 1.0)) if fp4 else x
        pools.append(pool)
    return pools


def _tables(g, lens, block, spare=0):
    """Block tables over a shuffled pool a tenth larger than needed, -1 past the last block, with a fresh block
    for `spare` entries of each row and one block that no table holds."""
    count = [-(-n // block) for n in lens]
    width = max(max(count), 1)
    total = sum(count) + len(lens) * spare
    num_blocks = total + total // 10 + 2
    perm = torch.randperm(num_blocks - 1, generator=g, device="cuda").int()
    offset = torch.tensor([sum(count[:s]) for s in range(len(lens))], device="cuda").unsqueeze(1)
    have = torch.tensor(count, device="cuda").unsqueeze(1)
    entry = torch.arange(width, device="cuda").unsqueeze(0)
    table = torch.where(entry < have, perm[(offset + entry).clamp(max=num_blocks - 2)], torch.full_like(entry, -1).int())
    fresh = perm[sum(count): total].reshape(len(lens), spare) if spare else None
    return table.int().contiguous(), fresh, num_blocks


def prepare(case, seed):
    g = _generator(seed)
    dt, block, dim, heads = DTYPES[case["dtype"]], case["block"], case["dim"], case["heads"]
    if case["op"] == "store":
        tokens = case["tokens"]
        num_blocks = -(-tokens // block) + 3
        slots = torch.randperm((num_blocks - 1) * block, generator=g, device="cuda")[:tokens]
        slots[torch.randperm(tokens, generator=g, device="cuda")[: case["pad"]]] = -1
        row = dim * 9 // 16
        return {"case": case, "slots": slots.contiguous(),
                "k": (torch.randn((tokens, heads, dim), generator=g, device="cuda") * _gain(g, heads, dim).squeeze(1)).to(dt),
                "v": torch.randn((tokens, heads, dim), generator=g, device="cuda").to(dt),
                "k_pool": torch.zeros((num_blocks, heads, block, row), dtype=torch.uint8, device="cuda"),
                "v_pool": torch.zeros((num_blocks, heads, block, row), dtype=torch.uint8, device="cuda"),
                "k_scale": 0.5, "v_scale": 0.25,
                "k_out": torch.empty((tokens, heads, dim), dtype=dt, device="cuda"),
                "v_out": torch.empty((tokens, heads, dim), dtype=dt, device="cuda")}
    lens = _lens(case)
    seqs = case["seqs"]
    spare = -(-case["budget"] // block) if case["op"] == "evict" and case["fresh"] else 0
    tables, fresh, num_blocks = _tables(g, lens, block, spare)
    k_pool, v_pool = _pools(case, g, num_blocks)
    state = {"case": case, "tables": tables, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "k_pool": k_pool, "v_pool": v_pool, "k_scale": 1.0, "v_scale": 1.0}
    width = tables.shape[1] * block
    if case["op"] != "decode":
        # what some hundred steps have added up: few tokens hold most of it
        w = torch.exp(1.5 * torch.randn((seqs, heads, width), generator=g, device="cuda"))
        state["weights"] = w.contiguous()
    if case["op"] == "evict":
        kept = _kept_lens(case)
        state["budgets"] = torch.tensor([-1 if m is None else case["budget"] for m in kept], dtype=torch.int32,
                                        device="cuda")
        state["kept"] = torch.full((seqs, heads, case["budget"]), -1, dtype=torch.int32, device="cuda")
        state["new_lens"] = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        state["new_weights"] = torch.zeros_like(state["weights"])
        state["to"] = tables
        if case["fresh"]:
            # a sequence that is left as it is keeps its blocks
            have = min(spare, tables.shape[1])
            state["to"] = tables.clone()
            state["to"][:, :have] = torch.where((tables[:, :have] >= 0) & (state["budgets"] >= 0).unsqueeze(1),
                                                fresh[:, :have], tables[:, :have])
        if case["kv"] == "fp4":
            # the slots of the kept tokens, to read them back
            at = [(s, j) for s, m in enumerate(kept) for j in range(m or 0)] or [(0, 0)]
            at = torch.tensor(at, device="cuda")
            entry = state["to"][at[:, 0], at[:, 1] // block].long()
            state["slots"] = torch.where(entry >= 0, entry * block + at[:, 1] % block, -1).contiguous()
            n = state["slots"].shape[0]
            state["k_out"] = torch.empty((n, heads, dim), dtype=dt, device="cuda")
            state["v_out"] = torch.empty((n, heads, dim), dtype=dt, device="cuda")
        return state
    state["scale"] = 1.0 / math.sqrt(dim)
    state["q"] = (1.5 * torch.randn((seqs, case["q_heads"], dim), generator=g, device="cuda")).to(dt)
    state["out"] = torch.empty((seqs, case["q_heads"], dim), dtype=dt, device="cuda")
    state["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import paged_kv_cache_357_b200 as pa

        if case["op"] == "decode":
            state["workspace"] = pa.alloc_decode_fp4_workspace(seqs, case["q_heads"], k_pool)
        elif case["kv"] == "fp4":
            state["workspace"] = pa.alloc_decode_fp4_workspace(seqs, case["q_heads"], k_pool, tables.shape[1])
        else:
            state["workspace"] = pa.alloc_decode_weights_workspace(seqs, case["q_heads"], k_pool, tables.shape[1])
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _plain_store(st):
    case = st["case"]
    block, dim = case["block"], case["dim"]
    slots = st["slots"]
    # padding goes to the last block, which no slot names
    to = torch.where(slots >= 0, slots, (st["k_pool"].shape[0] - 1) * block)
    outs = []
    for x, pool, scale in ((st["k"], st["k_pool"], st["k_scale"]), (st["v"], st["v_pool"], st["v_scale"])):
        codes, scales = _quantise(x.float(), scale)
        data = codes[..., 0::2] | (codes[..., 1::2] << 4)
        pool_data, pool_scales = _areas(pool, dim)
        pool_data[to // block, :, to % block] = data
        pool_scales[to // block, :, to % block] = scales
        outs.append(_plain_read(pool, slots, dim, scale).to(x.dtype))
    return {"k": outs[0], "v": outs[1]}


def _plain_read(pool, slots, dim, scale):
    """float32 values of the rows at the slots, zero for a negative one."""
    block, at = pool.shape[2], slots.clamp(min=0)
    data, scales = (area[at // block, :, at % block] for area in _areas(pool, dim))
    values = _values(torch.stack([data & 15, data >> 4], -1).flatten(-2), scales.contiguous(), scale)
    return torch.where((slots >= 0)[:, None, None], values, torch.zeros_like(values))


def _plain_rows(st, pool, scale):
    """float32 [seqs, heads, width, dim] of every table entry's rows."""
    got = pool[st["tables"].clamp(min=0)]
    x = got.float() if got.dtype != torch.uint8 else _values(*_unpack(got, st["case"]["dim"]), scale)
    return x.transpose(1, 2).flatten(2, 3)


def _plain_decode(st):
    case = st["case"]
    group = case["q_heads"] // case["heads"]
    width = st["tables"].shape[1] * case["block"]
    valid = torch.arange(width, device="cuda") < st["lens"].unsqueeze(1)  # [seqs, width]
    k = _plain_rows(st, st["k_pool"], st["k_scale"])
    q = st["q"].float().unflatten(1, (-1, group)) * st["scale"]
    scores = torch.matmul(q, k.transpose(2, 3)).masked_fill(~valid[:, None, None], -math.inf)
    del k
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    v = torch.where(valid[:, None, :, None], _plain_rows(st, st["v_pool"], st["v_scale"]), 0.0)
    out = torch.matmul(p, v).flatten(1, 2).to(st["q"].dtype)
    if case["op"] == "decode":
        return {"out": out}
    added = p.sum(2)
    newest = torch.arange(width, device="cuda") == (st["lens"] - 1).unsqueeze(1)
    w = torch.where(newest.unsqueeze(1), added, st["weights"] + added)
    st["weights"].copy_(torch.where(valid.unsqueeze(1), w, st["weights"]))
    return {"out": out, "weights": st["weights"]}


def _plain_evict(st):
    case = st["case"]
    block, dim, stride = case["block"], case["dim"], case["budget"]
    weights, n = st["weights"], st["lens"].long()
    seqs, heads, width = weights.shape
    left = st["budgets"] < 0
    m = torch.where(left, n, torch.minimum(n, st["budgets"].long()))
    recent = m.clamp(max=case["recent"])
    sinks = (m - recent).clamp(max=case["sinks"])
    pos = torch.arange(width, device="cuda")
    valid = pos < n.unsqueeze(1)
    forced = valid & ((pos < sinks.unsqueeze(1)) | (pos >= (n - recent).unsqueeze(1)))
    key = torch.where(valid.unsqueeze(1), weights, -math.inf).masked_fill(forced.unsqueeze(1), math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, pos.expand_as(order))
    chosen = rank < m[:, None, None]
    # the j-th chosen token of a head, in the order of the sequence; column `stride` takes what is not listed
    to = torch.where(chosen & ~left[:, None, None], chosen.cumsum(-1) - 1, stride)
    listed_ = torch.full((seqs, heads, stride + 1), -1, dtype=torch.int32, device="cuda")
    listed_.scatter_(-1, to, pos.int().expand_as(to))
    j = torch.arange(stride, device="cuda")
    live = (j < m.unsqueeze(1)) & ~left.unsqueeze(1)  # [seqs, stride]
    live = live.unsqueeze(1)
    kept = torch.where(live, listed_[..., :stride], st["kept"])
    st["kept"].copy_(kept)
    st["new_lens"].copy_(m)
    # rows that are not moved stand at the block that no table holds, and stay there
    unused = st["k_pool"].shape[0] - 1
    src = kept.long().clamp(min=0)
    row = torch.arange(seqs, device="cuda")[:, None, None]
    head = torch.arange(heads, device="cuda")[None, :, None]
    src_block = torch.where(live, st["tables"][row, src // block].long(), unused)
    src_row = torch.where(live, src % block, 0)
    jj = j.expand(seqs, heads, stride)
    dst_block = torch.where(live, st["to"][row, (jj // block).clamp(max=st["to"].shape[1] - 1)].long(), unused)
    dst_row = torch.where(live, jj % block, 0)
    for pool in (st["k_pool"], st["v_pool"]):
        parts = [pool] if case["kv"] == "16" else _areas(pool, dim)
        for part in parts:
            part[dst_block, head, dst_row] = part[src_block, head, src_row]
    most = min(stride, width)
    new = st["new_weights"][..., :most]
    new.copy_(torch.where(live[..., :most], weights.gather(-1, src)[..., :most], new))
    return _evicted(st)


def _areas(pool, dim):
    """Views of a 4-bit pool's code rows and scale rows."""
    block = pool.shape[2]
    flat = pool.view(pool.shape[0], pool.shape[1], -1)
    return (flat[..., : block * dim // 2].unflatten(-1, (block, dim // 2)),
            flat[..., block * dim // 2:].unflatten(-1, (block, dim // 16)))


def _evicted(st):
    out = {"kept": st["kept"], "new_lens": st["new_lens"], "weights": st["new_weights"]}
    if st["case"]["kv"] == "16":
        return {**out, "k": st["k_pool"], "v": st["v_pool"]}
    if own:
        return {**out, "k": st["k_out"], "v": st["v_out"]}
    dim, dt = st["case"]["dim"], st["k_out"].dtype
    return {**out, "k": _plain_read(st["k_pool"], st["slots"], dim, st["k_scale"]).to(dt),
            "v": _plain_read(st["v_pool"], st["slots"], dim, st["v_scale"]).to(dt)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if not own:
        return {"store": _plain_store, "decode": _plain_decode, "weights": _plain_decode,
                "evict": _plain_evict}[case["op"]](state)
    import paged_kv_cache_357_b200 as pa

    st = state
    if case["op"] == "store":
        pa.pa_cache_write_fp4(st["k"], st["v"], st["slots"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"])
        pa.pa_cache_read_fp4(st["slots"], st["k_pool"], st["v_pool"], st["k_out"], st["v_out"], st["k_scale"],
                             st["v_scale"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if case["op"] == "decode":
        pa.pa_decode_fp4(st["q"], st["k_pool"], st["v_pool"], st["tables"], st["lens"], st["scale"], st["out"],
                         st["workspace"], k_scale=st["k_scale"], v_scale=st["v_scale"], dev_status=st["status"])
        return {"out": st["out"]}
    if case["op"] == "weights":
        if case["kv"] == "fp4":
            pa.pa_decode_fp4(st["q"], st["k_pool"], st["v_pool"], st["tables"], st["lens"], st["scale"], st["out"],
                             st["workspace"], k_scale=st["k_scale"], v_scale=st["v_scale"], weights=st["weights"],
                             dev_status=st["status"])
        else:
            pa.pa_decode_weights(st["q"], st["k_pool"], st["v_pool"], st["tables"], st["lens"], st["scale"],
                                 st["weights"], st["out"], st["workspace"], dev_status=st["status"])
        return {"out": st["out"], "weights": st["weights"]}
    pa.pa_evict(st["tables"], st["lens"], st["budgets"], st["weights"], st["kept"], st["new_lens"], st["k_pool"],
                st["v_pool"], sinks=case["sinks"], recent=case["recent"], dst_tables=st["to"],
                new_weights=st["new_weights"])
    if case["kv"] == "fp4":
        pa.pa_cache_read_fp4(st["slots"], st["k_pool"], st["v_pool"], st["k_out"], st["v_out"], st["k_scale"],
                             st["v_scale"])
    return _evicted(st)


def work(case):
    heads, dim, block = case["heads"], case["dim"], case["block"]
    if case["op"] == "store":
        rows = (case["tokens"] - case["pad"]) * heads
        values = case["tokens"] * heads * dim * 2 * 2
        packed = rows * 2 * dim * 9 // 16
        return {"bytes": rows * dim * 2 * 2 + 2 * packed + values + case["tokens"] * 8, "flops": 4 * rows * dim}
    lens = _lens(case)
    rows = sum(lens) * heads
    if case["op"] == "evict":
        kept = _kept_lens(case)
        read = sum(n for n, m in zip(lens, kept) if m is not None) * heads * 4
        moved = sum(m or 0 for m in kept) * heads
        row = 2 * dim * (2 if case["kv"] == "16" else 9 / 16)
        back = (dim * 9 / 16 + 2 * dim) * 2 if case["kv"] == "fp4" else 0
        return {"bytes": read + moved * (2 * row + 4 + 4 + back) + 16 * len(lens), "flops": rows}
    fp4 = case["op"] == "decode" or case["kv"] == "fp4"
    row = 2 * dim * (9 / 16 if fp4 else 2)
    io = 2 * case["seqs"] * case["q_heads"] * dim * 2 + sum(-(-n // block) for n in lens) * 4
    return {"bytes": rows * row + io + (rows * 8 if case["op"] == "weights" else 0),
            "flops": 4 * sum(lens) * case["q_heads"] * dim}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _e4m3_values():
    """The 127 non-negative values of e4m3 (4 exponent bits of bias 7, 3 mantissa bits, the last code a NaN)."""
    small = [m * 2.0 ** -9 for m in range(8)]
    return small + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:119]


def _nearest(x, values):
    """Index of the nearest of the ascending values for x >= 0, ties to the even index, the last one at most."""
    grid = torch.tensor(values, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, x).clamp(1, len(values) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def _exact_stored(x, pool_scale):
    """The float64 values that the 4-bit pool holds for x."""
    y = x.double().reshape(*x.shape[:-1], x.shape[-1] // 16, 16) / pool_scale
    scales = torch.tensor(_e4m3_values(), dtype=torch.float64, device=x.device)
    s = scales[_nearest(y.abs().amax(-1) / 6, _e4m3_values())].unsqueeze(-1)
    codes = _nearest(y.abs() / torch.where(s == 0, 1.0, s), E2M1)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (torch.sign(y) * grid[codes] * s * pool_scale).reshape(x.shape)


def _exact_tile(tile, dim, pool_scale):
    """float64 [..., block, dim] of tile bytes [..., block, dim * 9 / 16]."""
    grid = torch.tensor([v for v in E2M1] + [-v for v in E2M1], dtype=torch.float64, device=tile.device)
    scales = torch.tensor(_e4m3_values() + [math.nan], dtype=torch.float64, device=tile.device)
    block = tile.shape[-2]
    raw = tile.reshape(*tile.shape[:-2], -1).long()
    codes, groups = raw[..., : block * dim // 2], raw[..., block * dim // 2:]
    value = torch.empty(*raw.shape[:-1], block * dim, dtype=torch.float64, device=tile.device)
    value[..., 0::2] = grid[codes % 16]
    value[..., 1::2] = grid[codes // 16]
    value = value * scales[groups].repeat_interleave(16, -1) * pool_scale
    return value.reshape(*raw.shape[:-1], block, dim)


def _exact_decode(st):
    case = st["case"]
    block, dim, heads = case["block"], case["dim"], case["heads"]
    group = case["q_heads"] // heads
    lens = _lens(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    weights = st["weights"].double() if case["op"] == "weights" else None
    for s, n in enumerate(lens):
        if n == 0:
            continue
        blocks = st["tables"][s, : -(-n // block)].long()
        for h in range(heads):
            rows = []
            for pool, scale in ((st["k_pool"], st["k_scale"]), (st["v_pool"], st["v_scale"])):
                tile = pool[blocks, h]
                x = _exact_tile(tile, dim, scale) if tile.dtype == torch.uint8 else tile.double()
                rows.append(x.reshape(-1, dim)[:n])
            q = st["q"][s, h * group: (h + 1) * group].double()
            p = torch.softmax(q @ rows[0].T * st["scale"], -1)
            out[s, h * group: (h + 1) * group] = p @ rows[1]
            if weights is not None:
                weights[s, h, : n - 1] += p[:, : n - 1].sum(0)
                weights[s, h, n - 1] = p[:, n - 1].sum()
    return {"out": out} if weights is None else {"out": out, "weights": weights}


def _exact_evict(st):
    import numpy as np

    case = st["case"]
    block, dim, heads = case["block"], case["dim"], case["heads"]
    weights, tables, to = (st[k].cpu().numpy() for k in ("weights", "tables", "to"))
    kept, new_lens = st["kept"].cpu().numpy(), np.zeros(case["seqs"], np.int32)
    new_weights = st["new_weights"].cpu().double().numpy()
    src, dst = [], []  # (block, head, row) of each move
    for s, (n, m) in enumerate(zip(_lens(case), _kept_lens(case))):
        new_lens[s] = n if m is None else m
        if not m:
            continue
        last = min(case["recent"], m)
        first = min(case["sinks"], m - last)
        for h in range(heads):
            middle = np.arange(first, n - last)
            by_weight = middle[np.lexsort((middle, -weights[s, h, middle].astype(np.float64)))]
            ids = np.concatenate([np.arange(first), np.sort(by_weight[: m - first - last]), np.arange(n - last, n)])
            kept[s, h, :m] = ids
            new_weights[s, h, :m] = weights[s, h, ids]
            j = np.arange(m)
            src.append(np.stack([tables[s, ids // block], np.full(m, h), ids % block]))
            dst.append(np.stack([to[s, j // block], np.full(m, h), j % block]))
    pools = []
    for pool, scale in ((st["k_pool"], st["k_scale"]), (st["v_pool"], st["v_scale"])):
        before = pool.view(pool.shape) if case["kv"] == "16" else _exact_tile(pool, dim, scale)
        after = before.clone()
        if src:
            a, b = (torch.from_numpy(np.concatenate(x, 1).astype(np.int64)).cuda() for x in (src, dst))
            after[b[0], b[1], b[2]] = before[a[0], a[1], a[2]]
        if case["kv"] == "fp4":
            at = st["slots"]
            got = after[at.clamp(min=0) // block, :, at.clamp(min=0) % block]
            after = torch.where((at >= 0)[:, None, None], got, 0.0)
        pools.append(after)
    return {"kept": kept, "new_lens": new_lens, "weights": new_weights, "k": pools[0], "v": pools[1]}


def exact(case, seed):
    if case["op"] in ("decode", "weights") and case["seqs"] * case["heads"] > 12000:
        return None
    st = prepare(case, seed)
    if case["op"] == "store":
        live = (st["slots"] >= 0)[:, None, None]
        return {"k": torch.where(live, _exact_stored(st["k"], st["k_scale"]), 0.0),
                "v": torch.where(live, _exact_stored(st["v"], st["v_scale"]), 0.0)}
    return _exact_evict(st) if case["op"] == "evict" else _exact_decode(st)
