"""The paged KV-cache operators of the library, case by case: their inputs, their plain
form in torch, the library's calls, and what one pass of each cannot do without.

A paged cache holds a layer's keys and values in pages of `page` slots,
[pages][kv_heads][page][head_dim * bits / 8] bytes of codes and one {min, scale} fp16 pair
per group of `group` values, in the codec's form. Sequence b's slot s is slot s % page of
page page_table[b][s // page]; it holds ctx_len[b] slots. The operators:

  attend  new tokens of a ragged batch attend to the cached slots and, causally, to their
          own fresh fp16 keys and values (or, cross attention, to the cached slots alone),
          optionally adding every slot's attention weight to the cache's running sum;
  store   new keys and values are quantised into the slots behind ctx_len, and
  load    slots are dequantised into rows again (one pass does both);
  evict   each head keeps `budget` slots: its `recent` latest positions and, of the rest,
          those with the largest accumulated weight.

The value a code c stands for: for load fp16(fp32(fp32(c * fp32(1/scale)) + min)), the
codec's; for attention fp16(c * fp16(1/scale) + min), one fp16 multiply-add, which is what
the library's products with compressed operands take.
"""
import math

import numpy as np
import torch

own = False

TAIL = 3     # rows behind the last sequence, which stay as they were


def listed():
    def attend(name, **kw):
        return dict(dict(name=name, op="attend", group=64, q_lo=1, q_hi=1, cross=False, weights=False), **kw)

    return [
        # one token for each of four short sequences at opt-125m's heads: latency
        attend("decode_small", batch=4, heads=12, kv_heads=12, dim=64, bits=4, page=16, ctx_lo=90, ctx_hi=128),
        # a whole decode batch at opt-175b's heads, prompt 512 and up to 31 tokens more
        attend("decode_batch", batch=144, heads=96, kv_heads=96, dim=128, bits=4, page=16, ctx_lo=512, ctx_hi=543),
        # few long sequences of unequal length, eight query heads to a key head, 8-bit codes
        attend("decode_long", batch=4, heads=64, kv_heads=8, dim=128, bits=8, page=64, ctx_lo=3001, ctx_hi=60001),
        # a decode step of opt-1.3b's heads that also keeps the running weights, groups of 32
        attend("decode_weights", batch=32, heads=32, kv_heads=32, dim=64, bits=4, group=32, page=32, ctx_lo=500,
               ctx_hi=1999, weights=True),
        # prompts arriving in pieces beside single tokens, ragged on both sides, with weights
        attend("chunk_ragged", batch=12, heads=32, kv_heads=32, dim=64, bits=4, page=16, ctx_lo=0, ctx_hi=1500,
               q_lo=1, q_hi=97, weights=True),
        # a late piece of two long prompts, four query heads to a key head
        attend("chunk_long", batch=2, heads=32, kv_heads=8, dim=128, bits=4, page=64, ctx_lo=8191, ctx_hi=16000,
               q_lo=2000, q_hi=2048),
        # one generated token per sequence over encoder states, some without any
        attend("cross_token", batch=32, heads=16, kv_heads=16, dim=64, bits=8, group=32, page=32, ctx_lo=0,
               ctx_hi=1500, cross=True),
        # whole target texts over encoder states of another length
        attend("cross_chunk", batch=6, heads=20, kv_heads=20, dim=64, bits=8, page=128, ctx_lo=0, ctx_hi=1500,
               q_lo=3, q_hi=448, cross=True),
        # the token of a decode step stored and read back: latency
        dict(name="store_token", op="store", batch=32, kv_heads=32, dim=64, bits=4, group=64, page=16, ctx_lo=1,
             ctx_hi=543, q_lo=1, q_hi=1),
        # prompts of opt-175b's heads stored and read back
        dict(name="store_prompt", op="store", batch=4, kv_heads=96, dim=128, bits=4, group=64, page=64, ctx_lo=0,
             ctx_hi=64, q_lo=301, q_hi=1024),
        # sixteen tokens over the budget after a few decode steps: little to move
        dict(name="evict_step", op="evict", batch=32, kv_heads=32, dim=64, bits=4, group=64, page=16, ctx_lo=1000,
             ctx_hi=1040, budget=1024, recent=512),
        # prompts cut to a quarter right after they were read
        dict(name="evict_prompt", op="evict", batch=4, kv_heads=56, dim=128, bits=4, group=64, page=64, ctx_lo=500,
             ctx_hi=2048, budget=512, recent=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "chunk", "chunk", "cross", "store", "evict"])
    bits, dim = rng.choice([4, 4, 8]), rng.choice([64, 128])
    c = dict(op="attend" if kind in ("decode", "chunk", "cross") else kind, bits=bits, dim=dim,
             group=rng.choice([32, 64]), page=rng.choice([16, 32, 64, 128]))
    share = rng.choice([1, 1, 2, 4, 8]) if c["op"] == "attend" else 1
    c["kv_heads"] = rng.randint(1, 40)
    c["batch"] = _spread(rng, 1, 144)
    c["ctx_hi"] = _spread(rng, 1, 30000 if kind == "decode" else 6000)
    c["ctx_lo"] = rng.choice([0, c["ctx_hi"] // 3, c["ctx_hi"]])
    if c["op"] == "attend":
        c["heads"] = c["kv_heads"] * share
        c["cross"] = kind == "cross"
        c["weights"] = rng.random() < 0.4
    if kind == "evict":
        c["ctx_hi"] += 1
        c["budget"] = rng.randint(1, c["ctx_hi"] - 1)
        c["recent"] = rng.randint(0, c["budget"])
    else:
        c["q_hi"] = 1 if kind == "decode" else _spread(rng, 1, 1024)
        c["q_lo"] = rng.randint(1, c["q_hi"])

    # fewer sequences, then heads, until it costs no more than the largest listed cases
    def cost():
        w = work(c)
        rows = c["batch"] * c["kv_heads"] * share * c.get("q_hi", 1)
        return max(w["bytes"] / 6e8, w["flops"] / 3e11,
                   rows * (c["ctx_hi"] + c.get("q_hi", 1)) / 1e9 if c["op"] == "attend" else 0)
    while cost() > 1 and c["batch"] > 1:
        c["batch"] = max(1, c["batch"] * 2 // 3)
    while cost() > 1 and c["kv_heads"] > 1:
        c["kv_heads"] = max(1, c["kv_heads"] * 2 // 3)
        if "heads" in c:
            c["heads"] = c["kv_heads"] * share
    return c


def _lengths(case):
    """Slots held and new tokens of each sequence: spread over the case's ranges, the ends
    of both ranges always among them. The same for every seed, as shapes are."""
    r = np.random.RandomState(case["batch"] * 1009 + case["ctx_hi"])
    n = case["batch"]
    ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, n)
    q = r.randint(case.get("q_lo", 1), case.get("q_hi", 1) + 1, n)
    ctx[0], ctx[-1] = case["ctx_lo"], case["ctx_hi"]
    q[0], q[-1] = case.get("q_hi", 1), case.get("q_lo", 1)
    return ctx.tolist(), q.tolist()


def _slot_bytes(case):
    return case["dim"] * case["bits"] // 8 + case["dim"] // case["group"] * 4


def work(case):
    ctx, q = _lengths(case)
    slot, kvh, dim = _slot_bytes(case), case["kv_heads"], case["dim"]
    if case["op"] == "store":       # rows read, slots written; slots read, rows written
        return {"bytes": sum(q) * kvh * 2 * (2 * slot + 2 * dim * 2), "flops": 0}
    if case["op"] == "evict":       # weights and positions read; what lies behind the budget and is kept moves
        b = sum(8 * n for n in ctx if n > case["budget"])
        moved = sum(case["budget"] * (n - case["budget"]) / n for n in ctx if n > case["budget"])
        return {"bytes": 8 * len(ctx) + kvh * (b + moved * 2 * (2 * slot + 8)), "flops": 0}
    heads = case["heads"]
    seen = [n * m if case["cross"] else n * m + m * (m + 1) // 2 for n, m in zip(ctx, q)]
    b = sum(ctx) * kvh * 2 * slot + sum(q) * heads * (dim * 4 + 4)
    flops = 4 * dim * heads * sum(seen)
    if not case["cross"]:
        b += sum(q) * kvh * dim * 4
    if case["weights"]:
        b += kvh * (8 * sum(ctx) + (0 if case["cross"] else 4 * sum(q)))
    return {"bytes": b, "flops": flops}


# ---- inputs ---------------------------------------------------------------------------

def _quantise(x, bits, group):
    """The codec's min/max form along the last dimension: codes (one number each) and
    {min, scale} fp16 pairs. Each fp32 operation is rounded by itself."""
    g = x.float().unflatten(-1, (-1, group))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    lo = lo + 0.0                                         # a zero minimum is +0
    top = float(2 ** bits - 1)
    span = hi - lo
    scale = torch.where(span > 0, top / span, 0).clamp(max=65504.0).half()
    c = ((g - lo) * scale.float()).round().clamp(0, top).to(torch.uint8)
    return c.flatten(-2), torch.cat([lo.half(), scale], -1)


def _pack(c, bits):
    return c if bits == 8 else c[..., 0::2] | c[..., 1::2] << 4


def _unpack(codes, bits):
    return codes if bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = dict(device="cuda")

    def randn(*shape):
        return torch.randn(shape, generator=gen, **dev)

    ctx, q = _lengths(case)
    page, kvh, dim = case["page"], case["kv_heads"], case["dim"]
    per = [-(-(n + (0 if case["op"] == "evict" else m)) // page) for n, m in zip(ctx, q)]
    pages, widest = sum(per) + 2, max(max(per), 1)
    order = torch.randperm(pages, generator=gen, **dev).to(torch.int32)
    table = torch.full((len(ctx), widest), -1, dtype=torch.int32, **dev)     # no page behind a sequence's last
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    s = {"case": case, "table": table, "ctx": torch.tensor(ctx, dtype=torch.int32, **dev),
         "cu": torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32, **dev),
         "q_hi": max(q), "total": sum(q)}
    # keys of a layer have channels of their own level and spread; values do not
    level, spread = randn(kvh, 1, dim), 0.5 + torch.rand((kvh, 1, dim), generator=gen, **dev)
    step = max(1, (1 << 26) // (kvh * page * dim))
    for name in ("k", "v"):
        parts = []
        for p in range(0, pages, step):
            x = randn(min(step, pages - p), kvh, page, dim)
            x = (x * spread + level if name == "k" else x).half()
            c, meta = _quantise(x, case["bits"], case["group"])
            parts.append((_pack(c, case["bits"]), meta))
        s[name + "_codes"], s[name + "_meta"] = (torch.cat([x[i] for x in parts]) for i in (0, 1))
    rows = sum(q) + TAIL
    if case["op"] == "store":
        s["k_new"] = (randn(rows, kvh, dim) * spread[:, 0] + level[:, 0]).half()
        s["v_new"] = randn(rows, kvh, dim).half()
        s["k_out"], s["v_out"] = randn(rows, kvh, dim).half(), randn(rows, kvh, dim).half()
        return s
    if case["op"] == "evict" or case["weights"]:
        # accumulated weights have a long tail: a few slots take most of it
        s["weight"] = torch.exp(2 * randn(pages, kvh, page) - 4)
        s["slot_pos"] = torch.zeros((pages, kvh, page), dtype=torch.int32, **dev)
    if case["op"] == "evict":
        # a cache that was cut before: its slots are not in the order of their positions
        for b, n in enumerate(ctx):
            old = torch.rand((kvh, n), generator=gen, **dev).argsort(-1)
            pos = torch.where(old < n // 2, old, old + 100).int()
            pad = torch.zeros((kvh, per[b] * page), dtype=torch.int32, **dev)
            pad[:, :n] = pos
            s["slot_pos"][table[b, :per[b]].long()] = pad.unflatten(-1, (per[b], page)).transpose(0, 1)
        s["weight_now"], s["slot_pos_now"] = torch.empty_like(s["weight"]), torch.empty_like(s["slot_pos"])
        s["new_len"] = torch.zeros(len(ctx), dtype=torch.int32, **dev)
        return s
    heads = case["heads"]
    # one row of a fused projection: queries (already scaled), keys and values side by side
    x = randn(rows, (heads + 2 * kvh) * dim).half()
    x[:, :heads * dim] *= dim ** -0.5
    k = x[:, heads * dim:(heads + kvh) * dim]
    k.copy_((k.float().unflatten(-1, (kvh, dim)) * spread[:, 0] + level[:, 0]).flatten(-2).half())
    s["qkv"] = x
    s["o"] = randn(rows, heads * dim).half()
    s["lse"] = randn(rows, heads)
    return s


# ---- the library's calls --------------------------------------------------------------

def _run_own(s):
    import group_wise_int4_b200 as fq
    case = s["case"]
    if "cache" not in s:        # the handle that a user's program keeps
        s["cache"] = fq.FlexPagedCache(s["table"], s["ctx"], pools=(s["k_codes"], s["k_meta"], s["v_codes"], s["v_meta"]),
                                       weight=s.get("weight_now", s.get("weight")),
                                       slot_pos=s.get("slot_pos_now", s.get("slot_pos")),
                                       num_bits=case["bits"], group_size=case["group"])
    cache, dim, kvh = s["cache"], case["dim"], case["kv_heads"]
    if case["op"] == "store":
        fq.flex_paged_store_kv(cache, s["k_new"], s["v_new"], kvh * dim, s["cu"], s["q_hi"], total=s["total"])
        fq.flex_paged_load_kv(cache, s["k_out"], s["v_out"], kvh * dim, s["cu"], s["q_hi"], start=s["ctx"],
                              total=s["total"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if case["op"] == "evict":
        s["weight_now"].copy_(s["weight"])
        s["slot_pos_now"].copy_(s["slot_pos"])
        if "ws" not in s:
            s["ws"] = torch.empty(fq.flex_paged_evict_ws_bytes(cache, case["budget"]), dtype=torch.uint8, device="cuda")
        fq.flex_paged_evict(cache, case["budget"], case["recent"], s["new_len"], s["ws"])
        return {"new_len": s["new_len"], "weight": s["weight_now"], "slot_pos": s["slot_pos_now"],
                "k_codes": s["k_codes"], "k_meta": s["k_meta"], "v_codes": s["v_codes"], "v_meta": s["v_meta"]}
    heads, x = case["heads"], s["qkv"]
    if "ws" not in s:
        s["ws"] = torch.empty(fq.flex_paged_attention_ws_bytes(cache, heads, s["total"], s["q_hi"], case["weights"]),
                              dtype=torch.uint8, device="cuda")
    k, v = (None, None) if case["cross"] else (x[:, heads * dim:], x[:, (heads + kvh) * dim:])
    fq.flex_paged_attention(cache, x, x.shape[1], heads, k, v, x.shape[1], s["o"], s["lse"], s["cu"], s["q_hi"],
                            s["ws"], accumulate=case["weights"], total=s["total"])
    out = {"o": s["o"], "lse": s["lse"]}
    if case["weights"]:
        out["weight"] = s["weight"]
    return out


# ---- the plain form -------------------------------------------------------------------

def _gather(pool, table):
    """[pages][kvh][page]... -> [batch][kvh][slots]..."""
    x = pool[table.long().clamp(min=0)]
    return x.transpose(1, 2).flatten(2, 3)


def _scatter(pool, table, new, count):
    """Writes new[b][h][s] to the pool for s < count[b]."""
    page = pool.shape[2]
    b, at = (torch.arange(new.shape[2], device=pool.device)[None] < count[:, None]).nonzero(as_tuple=True)
    pool[table[b, at // page].long(), :, at % page] = new[b, :, at]


def _values(codes, meta, case):
    """What attention takes a code for: one fp16 multiply-add."""
    c = _unpack(codes, case["bits"]).unflatten(-1, (-1, case["group"])).float()
    lo, scale = meta[..., 0:1].float(), meta[..., 1:2].float()
    step = torch.where(scale > 0, 1 / scale, 0).half().float()
    return (c * step + lo).half().float().flatten(-2)


def _rows(x, s):
    """Rows of a ragged batch -> [batch][most rows]..., and which of them there are."""
    at = torch.arange(s["q_hi"], device=x.device)[None]
    live = at < (s["cu"][1:] - s["cu"][:-1])[:, None]
    return x[torch.where(live, s["cu"][:-1, None] + at, 0).long()], live


def _attend(s):
    case, table = s["case"], s["table"]
    heads, kvh, dim = case["heads"], case["kv_heads"], case["dim"]
    x, live = _rows(s["qkv"], s)
    n, m = x.shape[:2]
    q = x[..., :heads * dim].float().reshape(n, m, kvh, heads // kvh, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = _values(_gather(s["k_codes"], table), _gather(s["k_meta"], table), case)
    v = _values(_gather(s["v_codes"], table), _gather(s["v_meta"], table), case)
    slots = k.shape[2]
    seen = (torch.arange(slots, device=x.device)[None] < s["ctx"][:, None])[:, None].expand(n, m, slots)
    if not case["cross"]:
        new = x[..., heads * dim:].float().reshape(n, m, 2, kvh, dim).permute(2, 0, 3, 1, 4)
        k, v = torch.cat([k, new[0]], 2), torch.cat([v, new[1]], 2)
        at = torch.arange(m, device=x.device)
        seen = torch.cat([seen, (at[None] <= at[:, None])[None].expand(n, m, m)], 2)
    seen = (seen & live[:, :, None])[:, None, None]
    sc = torch.matmul(q, k.transpose(-1, -2)).unflatten(2, (-1, m)).masked_fill(~seen, float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top > float("-inf"), top, 0)
    p = torch.exp(sc - top)
    del sc
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, m))
    lse = (top + torch.log(total))[..., 0]
    s["o"][:s["total"]] = o.permute(0, 3, 1, 2, 4).flatten(2)[live].half()
    s["lse"][:s["total"]] = lse.permute(0, 3, 1, 2).flatten(2)[live]
    out = {"o": s["o"], "lse": s["lse"]}
    if case["weights"]:
        w = p.sum((2, 3))
        old = _gather(s["weight"], table)
        w[:, :, :slots] += torch.where(torch.arange(slots, device=x.device) < s["ctx"][:, None, None], old, 0)
        if not case["cross"]:      # the fresh tokens' weights belong behind the last slot held
            at = torch.arange(slots, device=x.device)[None]
            i = (at - s["ctx"][:, None]).clamp(0, m - 1) + slots
            w = torch.where((at < s["ctx"][:, None])[:, None], w[..., :slots],
                            w.gather(2, i.long()[:, None].expand(n, kvh, slots)))
        fresh = 0 if case["cross"] else s["cu"][1:] - s["cu"][:-1]
        _scatter(s["weight"], table, w, s["ctx"] + fresh)
        out["weight"] = s["weight"]
    return out


def _store(s):
    case, table = s["case"], s["table"]
    page = case["page"]
    count = s["cu"][1:] - s["cu"][:-1]
    rows = torch.arange(s["total"], device="cuda")
    b = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count, output_size=s["total"])
    slot = s["ctx"][b] + rows - s["cu"][b]
    where = table[b, slot // page].long(), slot % page
    for name in ("k", "v"):
        c, meta = _quantise(s[name + "_new"][:s["total"]], case["bits"], case["group"])
        s[name + "_codes"][where[0], :, where[1]] = _pack(c, case["bits"])
        s[name + "_meta"][where[0], :, where[1]] = meta
        codes, meta = s[name + "_codes"][where[0], :, where[1]], s[name + "_meta"][where[0], :, where[1]].float()
        c = _unpack(codes, case["bits"]).unflatten(-1, (-1, case["group"])).float()
        step = torch.where(meta[..., 1:2] > 0, 1 / meta[..., 1:2], 0)
        s[name + "_out"][:s["total"]] = (c * step + meta[..., 0:1]).half().flatten(-2)
    return {"k": s["k_out"], "v": s["v_out"]}


def _evict(s):
    case, table, budget = s["case"], s["table"], s["case"]["budget"]
    weight, pos = _gather(s["weight"], table), _gather(s["slot_pos"], table)
    at = torch.arange(weight.shape[2], device="cuda")
    held = (at < s["ctx"][:, None])[:, None].expand_as(weight)
    latest = pos.masked_fill(~held, -2 ** 31).amax(-1, keepdim=True)
    rank = torch.where(pos.long() > latest.long() - case["recent"], 2, 1).masked_fill(~held, 0)
    # largest weight first, then the latest positions before all: stable, so ties keep slot order
    w = torch.where(weight.isnan(), float("-inf"), weight).masked_fill(rank == 2, 0)
    by = w.sort(dim=-1, descending=True, stable=True)[1]
    by = by.gather(-1, rank.gather(-1, by).sort(dim=-1, descending=True, stable=True)[1])
    new = s["ctx"].clamp(max=budget)
    kept = torch.zeros_like(held).scatter(-1, by, (at < new[:, None])[:, None].expand_as(held))
    inside = (at < new[:, None])[:, None]
    # the i-th slot to be filled, in order, takes the i-th kept slot behind the budget
    holes, movers = inside & ~kept, ~inside & kept
    to, come = (x.int().sort(dim=-1, descending=True, stable=True)[1] for x in (holes, movers))
    count = holes.sum(-1, keepdim=True)
    source = at.expand_as(held).scatter(-1, to, torch.where(at < count, come, to))
    out = {"new_len": new}
    s["weight_now"].copy_(s["weight"])
    s["slot_pos_now"].copy_(s["slot_pos"])
    for name, pool in (("weight", s["weight_now"]), ("slot_pos", s["slot_pos_now"])) + tuple(
            (name, s[name]) for name in ("k_codes", "k_meta", "v_codes", "v_meta")):
        x = _gather(pool, table)
        i = source.reshape(source.shape + (1,) * (x.dim() - 3)).expand_as(x)
        _scatter(pool, table, x.gather(2, i), new)
        out[name] = pool
    s["new_len"].copy_(new)
    out["new_len"] = s["new_len"]
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _attend, "store": _store, "evict": _evict}[state["case"]["op"]](state)


# ---- in 64 bits, sequence by sequence -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    ctx, q = _lengths(case)
    page, kvh, dim, group, bits = case["page"], case["kv_heads"], case["dim"], case["group"], case["bits"]

    def slots(name, b, n):
        """The first n slots of sequence b, head first."""
        ids = s["table"][b, :-(-n // page)].long()
        x = s[name][ids]
        return torch.cat(list(x.unbind(0)), 1)[:, :n] if len(ids) else x.new_zeros((kvh, 0) + tuple(x.shape[3:]))

    def code_numbers(x):
        if bits == 8:
            return x.double()
        two = torch.empty(x.shape + (2,), dtype=torch.float64, device=x.device)
        two[..., 0], two[..., 1] = x % 16, torch.div(x, 16, rounding_mode="floor")
        return two.reshape(x.shape[:-1] + (2 * x.shape[-1],))

    if case["op"] == "store":
        out = {}
        at = 0
        for name in ("k", "v"):
            y = s[name + "_out"].double()
            x = s[name + "_new"][:sum(q)].double().reshape(sum(q), kvh, dim // group, group)
            lo, span = x.amin(-1, True), x.amax(-1, True) - x.amin(-1, True)
            # the definition's own roundings: the scale to fp16, difference and product to fp32
            scale = torch.where(span > 0, ((2 ** bits - 1) / span.float().double()).float().clamp(max=65504.0).half().double(), 0)
            c = ((x - lo).float().double() * scale).float().double().round().clamp(0, 2 ** bits - 1)
            inverse = torch.where(scale > 0, (1 / scale).float().double(), 0)
            y[:sum(q)] = ((c * inverse).float().double() + lo).float().half().double().reshape(sum(q), kvh, dim)
            out[name] = y
        return out
    if case["op"] == "evict":
        weight = s["weight"].double()
        for b, n in enumerate(ctx):
            if n <= case["budget"]:
                continue
            ids = s["table"][b, :-(-n // page)].long()
            w, pos = slots("weight", b, n).cpu().numpy(), slots("slot_pos", b, n).cpu().numpy().astype(np.int64)
            for h in range(kvh):
                first = pos[h] > pos[h].max() - case["recent"]
                keep = np.lexsort((np.arange(n), -np.where(first, 0, w[h]), ~first))[:case["budget"]]
                keep.sort()
                stay = keep[keep < case["budget"]]
                free = np.setdiff1d(np.arange(case["budget"]), stay)
                w[h, free] = w[h, keep[keep >= case["budget"]]]
            pad = weight[ids].transpose(0, 1).reshape(kvh, -1)
            pad[:, :n] = torch.from_numpy(w).to(pad)
            weight[ids] = pad.reshape(kvh, len(ids), page).transpose(0, 1)
        return {"new_len": None, "weight": weight, "slot_pos": None, "k_codes": None, "k_meta": None,
                "v_codes": None, "v_meta": None}
    heads = case["heads"]
    share = heads // kvh
    o, lse = s["o"].double(), s["lse"].double()
    weight = s["weight"].double() if case["weights"] else None
    at = 0
    for b, (n, m) in enumerate(zip(ctx, q)):
        x = s["qkv"][at:at + m].double()
        kv = []
        for name in ("k", "v"):
            c = code_numbers(slots(name + "_codes", b, n)).reshape(kvh, n, dim // group, group)
            meta = slots(name + "_meta", b, n).double()
            scale = meta[..., 1:]
            step = torch.where(scale > 0, (1 / scale).half().double(), 0)
            kv.append((c * step + meta[..., :1]).half().double().reshape(kvh, n, dim))
        if not case["cross"]:
            for i in (0, 1):
                new = x[:, (heads + i * kvh) * dim:(heads + (i + 1) * kvh) * dim].reshape(m, kvh, dim).transpose(0, 1)
                kv[i] = torch.cat([kv[i], new], 1)
        keys = kv[0].shape[1]
        sums = torch.zeros(kvh, keys, dtype=torch.float64, device=x.device)
        hidden = torch.zeros(m, keys, dtype=torch.bool, device=x.device)
        if not case["cross"]:
            hidden[:, n:] = torch.ones(m, m, dtype=torch.bool, device=x.device).triu(1)
        for h in range(heads):
            g = h // share
            sc = (x[:, h * dim:(h + 1) * dim] @ kv[0][g].T).masked_fill(hidden, float("-inf"))
            z = torch.logsumexp(sc, 1)
            p = torch.exp(sc - torch.where(z > float("-inf"), z, 0)[:, None])
            o[at:at + m, h * dim:(h + 1) * dim] = p @ kv[1][g]
            lse[at:at + m, h] = z
            sums[g] += p.sum(0)
        if weight is not None:
            held = n if case["cross"] else n + m
            old = slots("weight", b, held).double()
            old[:, n:] = 0
            old += sums
            for i in range(-(-held // page)):
                part = old[:, i * page:(i + 1) * page]
                weight[int(s["table"][b, i]), :, :part.shape[1]] = part
        at += m
    out = {"o": o, "lse": lse}
    if weight is not None:
        out["weight"] = weight
    return out
