"""The cases that the serving-step operators are measured on, their plain forms and their exact values.

One step of a serving loop over a paged key-value cache: `plan` (block tables and slot maps from the
requests' lengths), `rope` (rotary positions), `write` (rotary positions and the write into a 16-bit
or FP8 paged cache) and `decode` (attention of one new token per sequence over that cache)."""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------


def _decode(name, B, Hq, Hk, D, low, high, dtype="bf16", cache="bf16", bs=16, layout="apart", window=0, softcap=0.0,
            alibi=False, sinks=False):
    return {"name": name, "op": "decode", "B": B, "Hq": Hq, "Hk": Hk, "D": D, "low": low, "high": high, "dtype": dtype,
            "cache": cache, "bs": bs, "layout": layout, "window": window, "softcap": softcap, "alibi": alibi,
            "sinks": sinks}


def _rotary(name, op, T, Hq, Hk, D, R, first, dtype="bf16", cache="bf16", interleaved=False, scaling="none",
            factor=1.0, original=8192, base=10000.0, pad=0, bs=16, layout="apart"):
    return {"name": name, "op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "first": first, "dtype": dtype,
            "cache": cache, "interleaved": interleaved, "scaling": scaling, "factor": factor, "original": original,
            "base": base, "pad": pad, "bs": bs, "layout": layout}


def _plan(name, B, low, high, prefill, chunk, pad=0, bs=16, spare=8):
    return {"name": name, "op": "plan", "B": B, "low": low, "high": high, "prefill": prefill, "chunk": chunk, "pad": pad,
            "bs": bs, "spare": spare}


def listed():
    return [
        # two short requests: what one call costs when there is next to nothing to read
        _decode("decode short", 2, 4, 2, 64, 37, 100),
        # a serving batch of an 8B-parameter model with grouped heads, mixed lengths
        _decode("decode batch bf16", 32, 32, 8, 128, 1024, 8192),
        # few requests with very long contexts: the length has to be split to fill the GPU
        _decode("decode long f16", 4, 64, 8, 128, 131072, 131072, "f16", "f16"),
        # the same cache in 8 bits with a scale for each head, a larger batch of equal lengths
        _decode("decode batch fp8", 64, 32, 8, 128, 4096, 4096, "bf16", "e4m3", 64),
        # a layer with a sliding window, capped scores and sinks; five kv heads, wide heads, larger blocks
        _decode("decode window", 13, 30, 5, 256, 301, 9001, "bf16", "bf16", 32, "paired", 4096, 30.0, False, True),
        # one new token for each sequence of that batch, rotated and written (eight rows of padding)
        _rotary("write decode", "write", 40, 32, 8, 128, 128, 1024, base=500000.0, pad=8),
        # a prefill of 16384 tokens
        _rotary("write prefill", "write", 16384, 32, 8, 128, 128, 0, base=500000.0, scaling="bands", factor=8.0),
        # a chunk of a long prefill into an FP8 cache, pairs side by side, half of the head rotated
        _rotary("write fp8", "write", 5003, 24, 6, 64, 32, 100003, "f16", "e4m3", True, bs=32, layout="heads"),
        # the rotation alone, as it stands before the INT4 cache write
        _rotary("rope chunk", "rope", 777, 32, 8, 128, 128, 4097, scaling="linear", factor=4.0),
        # far positions under the long-context scaling, many heads
        _rotary("rope far", "rope", 8192, 64, 8, 128, 64, 1000003, "f16", scaling="yarn", factor=32.0),
        # the table and slots of one decode step
        _plan("plan decode", 32, 1024, 8192, 0, 1),
        # a large mixed batch: prefill chunks between single tokens
        _plan("plan mixed", 256, 0, 8192, 64, 512, 100),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "write", "rope", "plan"])
    if op == "plan":
        B, bs = _log(rng, 1, 700), rng.choice([16, 16, 32, 64])
        prefill = rng.randint(0, B)
        high = _log(rng, 10, 12000)
        chunk = _log(rng, 1, max(2, min(4000, 60000 // (prefill + 1))))
        case = _plan("", B, rng.randint(0, high), high, prefill, chunk, rng.randint(0, 40), bs, rng.randint(0, 50))
    elif op == "decode":
        Hk, G, D = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), rng.choice([64, 128, 128, 256])
        dtype = rng.choice(["bf16", "f16"])
        cache = rng.choice([dtype, "e4m3"])
        high = _log(rng, 1, 40000)
        most = max(1, min(128, int(6e8 / (2 * high * Hk * D * 2))))
        case = _decode("", _log(rng, 1, most), Hk * G, Hk, D, rng.randint(max(1, high // 8), high), high, dtype, cache,
                       rng.choice([16, 16, 32, 64, 128]), rng.choice(["apart", "paired", "heads"]), rng.choice([0, 0, 0, _log(rng, 1, 5000)]),
                       rng.choice([0.0, 0.0, 30.0]), rng.random() < 0.2, rng.random() < 0.3)
    else:
        D = rng.choice([64, 80, 96, 128, 256])
        dtype = rng.choice(["bf16", "f16"] + (["f32"] if op == "rope" else []))
        Hk = rng.choice([1, 2, 3, 5, 8])
        Hq = Hk * rng.choice([1, 3, 4, 7])
        T = _log(rng, 1, min(16384, 400000000 // (3 * Hq * D * 4)))
        case = _rotary("", op, T, Hq, Hk, D, rng.choice([D, D, D // 2, D - 16]), _log(rng, 1, 1000000), dtype,
                       rng.choice([dtype, "e4m3"]) if op == "write" else dtype, rng.random() < 0.5,
                       rng.choice(["none", "linear", "bands", "yarn"]), rng.choice([2.0, 8.0, 32.0]), rng.choice([4096, 8192]),
                       rng.choice([10000.0, 500000.0]), rng.randint(0, min(9, T - 1)), rng.choice([16, 32, 64]),
                       rng.choice(["apart", "paired", "heads"]))
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------


def _spread(low, high, n):
    """n whole numbers spread evenly over [low, high]."""
    return [low + (high - low) * i // max(1, n - 1) if n > 1 else high for i in range(n)]


def _plan_lens(case):
    """Context and new tokens of each request: the first `prefill` requests bring a chunk, the rest one token."""
    new = _spread(max(1, case["chunk"] // 4), case["chunk"], case["prefill"]) + [1] * (case["B"] - case["prefill"])
    return _spread(case["low"], case["high"], case["B"]), new


def _blocks(lens, bs):
    return [-(-n // bs) for n in lens]


def _cache(nb, bs, Hk, D, layout, dtype, g):
    """A pool of nb blocks and its two views [nb, bs, Hk, D]: K and V apart, side by side in each
    block, or with the head before the token."""
    def fill(shape):
        x = torch.empty(shape, device="cuda", dtype=torch.float16 if dtype == torch.float8_e4m3fn else dtype)
        x.normal_(generator=g)
        return x.to(dtype)
    if layout == "paired":
        kv = fill((nb, 2, bs, Hk, D))
        return kv, kv[:, 0], kv[:, 1]
    if layout == "heads":
        k, v = fill((nb, Hk, bs, D)), fill((nb, Hk, bs, D))
        return (k, v), k.transpose(1, 2), v.transpose(1, 2)
    k, v = fill((nb, bs, Hk, D)), fill((nb, bs, Hk, D))
    return (k, v), k, v


def _inv_freq(case):
    """Radians a position of each pair, in 64 bits, and the factor on cos and sin."""
    R, s, n = case["R"], case["factor"], case["original"]
    f = case["base"] ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if case["scaling"] == "linear":
        return f / s, 1.0
    turns = n * f / (2 * math.pi)  # turns over the original context
    if case["scaling"] == "bands":  # below 1 turn: all of the scaling, above 4 turns: none
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f / s * (1 - keep) + f * keep, 1.0
    if case["scaling"] == "yarn":  # a ramp over the pairs, between the ones that make 32 turns and 1 turn
        at = [R * math.log(n / (t * 2 * math.pi)) / (2 * math.log(case["base"])) for t in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = ((torch.arange(R // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    i32 = dict(device="cuda", dtype=torch.int32)
    s = {"case": dict(case)}
    if case["op"] == "plan":
        context, new = _plan_lens(case)
        B, bs = case["B"], case["bs"]
        mix = torch.randperm(B, generator=cpu)
        context, new = torch.tensor(context)[mix], torch.tensor(new)[mix[torch.randperm(B, generator=cpu)]]
        have, need = (context + bs - 1) // bs, (context + new + bs - 1) // bs
        rows, width = B + 5, int(context.max() + new.max() + bs - 1) // bs + 3
        first = 17  # blocks of the free list that earlier steps took
        held, total = int(have.sum()), int(need.sum())
        ids = torch.randperm(total + case["spare"] + first, generator=g, device="cuda").to(torch.int32)
        row = torch.randperm(rows, generator=cpu)[:B]
        table = torch.full((rows, width), -1, **i32)
        used = torch.arange(width)[None] < have[:, None]
        table[row.cuda()] = table[row.cuda()].masked_scatter(used.cuda(), ids[:held])
        T = int(new.sum()) + case["pad"]
        s.update(context=context.to(**i32), new=new.to(**i32), rows=row.to(**i32), table=table, free=ids[held:].contiguous(),
                 cursor=torch.tensor([first], device="cuda"), cursor_out=torch.zeros(1, dtype=torch.int64, device="cuda"),
                 batch=torch.full((B, width), -1, **i32), T=T, bs=bs, blocks=ids.numel(),
                 lens=torch.empty(B, **i32), starts=torch.empty(B + 1, **i32), positions=torch.empty(T, **i32),
                 slots=torch.empty(T, dtype=torch.int64, device="cuda"))
        return s
    Hq, Hk, D, dtype = case["Hq"], case["Hk"], case["D"], DTYPES[case["dtype"]]
    cache = DTYPES[case["cache"]]
    scales = {}
    if case["cache"] == "e4m3":
        scales = {k: torch.rand(Hk, device="cuda", generator=g) * 0.05 + 0.02 for k in ("k_scale", "v_scale")}
    s.update({"k_scale": None, "v_scale": None}, **scales)
    if case["op"] == "decode":
        B, bs = case["B"], case["bs"]
        lens = torch.tensor(_spread(case["low"], case["high"], B))[torch.randperm(B, generator=cpu)]
        pages = (lens + bs - 1) // bs
        nb = int(pages.sum()) + 3
        ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((B, int(pages.max())), **i32)
        used = (torch.arange(table.shape[1])[None] < pages[:, None]).cuda()
        table = table.masked_scatter(used, ids[: int(pages.sum())])
        pool, k, v = _cache(nb, bs, Hk, D, case["layout"], cache, g)
        q = torch.randn((B, Hq, D), device="cuda", generator=g)
        if scales:  # the cache holds what its scales make of ordinary keys: scores as without them
            q = q / s["k_scale"].repeat_interleave(Hq // Hk)[None, :, None]
        s.update(q=q.to(dtype), pool=pool, k=k, v=v, table=table, lens=lens.to(**i32), scale=1.0 / math.sqrt(D),
                 out=torch.empty((B, Hq, D), device="cuda", dtype=dtype), lse=torch.empty((B, Hq), device="cuda"),
                 sinks=torch.randn(Hq, device="cuda", generator=g) if case["sinks"] else None,
                 slopes=torch.rand(Hq, device="cuda", generator=g) * 0.01 if case["alibi"] else None)
        return s
    T, live = case["T"], case["T"] - case["pad"]
    x = torch.randn((T, (Hq + 2 * Hk) * D), device="cuda", generator=g).to(dtype)  # the projection's output
    q, k, v = (y.unflatten(1, (-1, D)) for y in x.split([Hq * D, Hk * D, Hk * D], 1))
    inv_freq, factor = _inv_freq(case)
    positions = torch.arange(case["first"], case["first"] + T)
    if case["T"] <= 512:  # one token each of as many sequences
        positions = torch.randint(case["first"], case["first"] + 7168, (T,), generator=cpu)
    positions[live:] = -1
    s.update(x=x, q=q, k=k, v=v, positions=positions.to(**i32), inv_freq=inv_freq.cuda(), factor=factor,
             freqs=(inv_freq / (2 * math.pi) * 2.0**64).round().to(torch.int64).cuda(),
             q_out=torch.zeros((T, Hq, D), device="cuda", dtype=dtype))
    if case["op"] == "rope":
        s["k_out"] = torch.zeros((T, Hk, D), device="cuda", dtype=dtype)
        return s
    bs = case["bs"]
    nb = -(-T // bs) + 3
    s["pool"], s["kc"], s["vc"] = _cache(nb, bs, Hk, D, case["layout"], cache, g)
    blocks = torch.randperm(nb, generator=g, device="cuda")
    at = torch.arange(T, device="cuda")
    s["slots"] = blocks[at // bs] * bs + at % bs
    s["slots"][live:] = -1
    return s


def work(case):
    if case["op"] == "plan":
        context, new = _plan_lens(case)
        B, T, entries = case["B"], sum(new) + case["pad"], sum(_blocks([c + n for c, n in zip(context, new)], case["bs"]))
        return {"bytes": 20 * B + 12 * T + 8 * entries, "flops": 0}
    Hq, Hk, D, e = case["Hq"], case["Hk"], case["D"], SIZE[case["dtype"]]
    if case["op"] == "decode":
        lens = _spread(case["low"], case["high"], case["B"])
        keys = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        return {"bytes": 2 * keys * Hk * D * SIZE[case["cache"]] + case["B"] * Hq * (2 * D * e + 4) + 4 * keys // case["bs"],
                "flops": 4 * keys * Hq * D}
    live = case["T"] - case["pad"]
    if case["op"] == "rope":
        return {"bytes": live * (2 * (Hq + Hk) * D * e + 4), "flops": 3 * live * (Hq + Hk) * case["R"]}
    return {"bytes": live * ((2 * Hq + 2 * Hk) * D * e + 2 * Hk * D * SIZE[case["cache"]] + 12),
            "flops": 3 * live * (Hq + Hk) * case["R"]}


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------


def run(s):
    return {"plan": _run_plan, "rope": _run_rope, "write": _run_write, "decode": _run_decode}[s["case"]["op"]](s)


def _run_plan(s):
    if own:
        from quantized_paged_kv_int4_gb300 import kvq
        kvq.kvq_plan_step(s["context"], s["new"], s["table"], s["free"], s["cursor"], s["bs"], s["blocks"], rows=s["rows"],
                          batch_table=s["batch"], cursor_out=s["cursor_out"], seq_lens=s["lens"],
                          query_start_loc=s["starts"], positions=s["positions"], slot_mapping=s["slots"])
        return {k: s[k] for k in ("table", "batch", "cursor_out", "lens", "starts", "positions", "slots")}
    context, new, bs, T = s["context"].long(), s["new"].long(), s["bs"], s["T"]
    lens = context + new
    have, need = (context + bs - 1) // bs, (lens + bs - 1) // bs
    taken = (need - have).cumsum(0)
    j = torch.arange(s["table"].shape[1], device="cuda")[None]
    rows = s["rows"].long()
    old = s["table"][rows]
    at = s["cursor"] + (taken - (need - have))[:, None] + j - have[:, None]
    ids = torch.where((j >= have[:, None]) & (j < need[:, None]), s["free"][at.clamp(0, s["free"].numel() - 1)], old)
    s["table"][rows] = ids
    s["batch"].copy_(torch.where(j < need[:, None], ids, s["batch"]))
    starts = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts[1:], i, right=True)
    live = b < new.numel()
    b = b.clamp(max=new.numel() - 1)
    pos = torch.where(live, context[b] + i - starts[b], 0)
    slots = torch.where(live, ids[b, pos // bs].long() * bs + pos % bs, -1)
    return {"table": s["table"], "batch": s["batch"], "cursor_out": s["cursor"] + taken[-1:], "lens": lens.int(),
            "starts": starts.int(), "positions": torch.where(live, pos, -1).int(), "slots": slots}


def _angles(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    return (angle.cos() * s["factor"]).float()[:, None], (angle.sin() * s["factor"]).float()[:, None]


def _rotated(x, cos, sin, R, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., R:]), -1)
    a, b = x[..., : R // 2], x[..., R // 2 : R]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), -1)


def _run_rope(s):
    c = s["case"]
    if own:
        from quantized_paged_kv_int4_gb300 import kvq
        return kvq.kvq_rope(s["q"], s["k"], s["positions"], s["freqs"], interleaved=c["interleaved"], attn_factor=s["factor"],
                            q_out=s["q_out"], k_out=s["k_out"])
    cos, sin = _angles(s)
    live = (s["positions"] >= 0)[:, None, None]
    return tuple(torch.where(live, _rotated(x, cos, sin, c["R"], c["interleaved"]).to(x.dtype), y)
                 for x, y in ((s["q"], s["q_out"]), (s["k"], s["k_out"])))


def _run_write(s):
    c = s["case"]
    if own:
        from quantized_paged_kv_int4_gb300 import kvq
        q_out = kvq.kvq_write_kv(s["k"], s["v"], s["kc"], s["vc"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                 q=s["q"], positions=s["positions"], freqs=s["freqs"], interleaved=c["interleaved"],
                                 attn_factor=s["factor"], q_out=s["q_out"])
        return q_out, s["kc"], s["vc"]
    cos, sin = _angles(s)
    live = s["positions"] >= 0
    q_out = torch.where(live[:, None, None], _rotated(s["q"], cos, sin, c["R"], c["interleaved"]).to(s["q"].dtype), s["q_out"])
    _scatter(s["kc"], _rotated(s["k"], cos, sin, c["R"], c["interleaved"]), s["k_scale"], s["slots"])
    _scatter(s["vc"], s["v"].float(), s["v_scale"], s["slots"])
    return q_out, s["kc"], s["vc"]


def _scatter(cache, x, scale, slots):
    keep = slots >= 0
    x, slots, bs = x[keep], slots[keep], cache.shape[1]
    if scale is None:
        cache[slots // bs, slots % bs] = x.to(cache.dtype)
    else:
        codes = (x / scale[None, :, None]).clamp(-448.0, 448.0).to(cache.dtype)
        cache.view(torch.uint8)[slots // bs, slots % bs] = codes.view(torch.uint8)


def _paged(cache, table, scale):
    """[B, Hk, tokens, D] in 32 bits of the blocks that the table names."""
    x = cache.view(torch.uint8)[table].view(cache.dtype) if scale is not None else cache[table]
    x = x.flatten(1, 2).transpose(1, 2).float()
    return x if scale is None else x * scale[None, :, None, None]


def _run_decode(s):
    c = s["case"]
    if own:
        from quantized_paged_kv_int4_gb300 import kvq
        kvq.kvq_decode_kv(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                          out=s["out"], lse_out=s["lse"], sliding_window=c["window"], softcap=c["softcap"], sinks=s["sinks"],
                          alibi_slopes=s["slopes"])
        return s["out"], s["lse"]
    q, lens, table = s["q"].float(), s["lens"].long()[:, None, None, None], s["table"].long()
    B, Hq, D = q.shape
    k, v = _paged(s["k"], table, s["k_scale"]), _paged(s["v"], table, s["v_scale"])
    Hk, n = k.shape[1], torch.arange(k.shape[2], device="cuda")
    score = (q.view(B, Hk, Hq // Hk, D) @ k.transpose(2, 3)) * s["scale"]
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    if s["slopes"] is not None:
        score = score + s["slopes"].view(1, Hk, Hq // Hk, 1) * (n - (lens - 1))
    live = n < lens
    if c["window"]:
        live = live & (n >= lens - c["window"])
    score = score.masked_fill(~live, -math.inf)
    top = score.amax(-1, keepdim=True)
    sinks = s["sinks"]
    if sinks is not None:
        sinks = sinks.view(1, Hk, Hq // Hk, 1)
        top = torch.maximum(top, sinks)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - top)
    out = (p @ v) / total
    return out.view(B, Hq, D).to(s["q"].dtype), (top + total.log()).view(B, Hq)


# ------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "write": _exact_write, "decode": _exact_decode}[case["op"]](s)


def _exact_plan(s):
    """Request by request on the host."""
    bs, context, new, rows, free = s["bs"], s["context"].tolist(), s["new"].tolist(), s["rows"].tolist(), s["free"].tolist()
    table, batch, cursor = s["table"].cpu(), s["batch"].cpu(), int(s["cursor"])
    starts, positions, slots = [0], [], []
    for b, (c, n, r) in enumerate(zip(context, new, rows)):
        have, need = math.ceil(c / bs), math.ceil((c + n) / bs)
        for j in range(have, need):
            table[r, j] = free[cursor]
            cursor += 1
        batch[b, :need] = table[r, :need]
        line = table[r].tolist()
        positions += range(c, c + n)
        slots += [line[p // bs] * bs + p % bs for p in range(c, c + n)]
        starts.append(starts[-1] + n)
    rest = [-1] * (s["T"] - len(slots))
    ints = dict(dtype=torch.int32)
    return {"table": table, "batch": batch, "cursor_out": torch.tensor([cursor]),
            "lens": torch.tensor([c + n for c, n in zip(context, new)], **ints), "starts": torch.tensor(starts, **ints),
            "positions": torch.tensor(positions + rest, **ints), "slots": torch.tensor(slots + rest)}


def _turn(x, s):
    """Each pair as a complex number times factor * e^(i angle)."""
    c, R = s["case"], s["case"]["R"]
    x = x.double()
    turn = torch.polar(torch.full_like(s["inv_freq"], s["factor"]).expand(x.shape[0], -1).contiguous(),
                       s["positions"].double()[:, None] * s["inv_freq"][None])[:, None]
    if c["interleaved"]:
        z = torch.view_as_real(torch.view_as_complex(x[..., :R].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(x[..., : R // 2].contiguous(), x[..., R // 2 : R].contiguous()) * turn
        z = torch.cat((z.real, z.imag), -1)
    return torch.cat((z, x[..., R:]), -1)


def _exact_rope(s):
    live = s["case"]["T"] - s["case"]["pad"]
    found = []
    for x, y in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = y.double()
        y[:live] = _turn(x, s)[:live]
        found.append(y)
    return tuple(found)


def _exact_write(s):
    live = s["case"]["T"] - s["case"]["pad"]
    q = s["q_out"].double()
    q[:live] = _turn(s["q"], s)[:live]
    found = [q]
    for cache, x, scale in ((s["kc"], _turn(s["k"], s), s["k_scale"]), (s["vc"], s["v"].double(), s["v_scale"])):
        y = cache.to(torch.float64, memory_format=torch.preserve_format)
        slots, bs = s["slots"][:live], cache.shape[1]
        if scale is not None:
            x = (x / scale.double()[None, :, None]).clamp(-448, 448)
        y[slots // bs, slots % bs] = x[:live]
        found.append(y)
    return tuple(found)


def _exact_decode(s):
    """Sequence by sequence."""
    c = s["case"]
    B, Hq, D = s["q"].shape
    Hk = s["k"].shape[2]
    out, lse = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda"), torch.zeros((B, Hq), dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        low = max(0, L - c["window"]) if c["window"] else 0
        n = torch.arange(low, L, device="cuda")
        block = s["table"][b].long()[n // c["bs"]]
        for h in range(Hk):
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k, v = (_rows(x, block, n % c["bs"], h) for x in (s["k"], s["v"]))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            z = s["q"][b, heads].double() @ k.T * s["scale"]
            if c["softcap"]:
                z = torch.tanh(z / c["softcap"]) * c["softcap"]
            if s["slopes"] is not None:
                z = z + s["slopes"][heads, None].double() * (n - (L - 1))
            norm = torch.logsumexp(z, 1)
            if s["sinks"] is not None:
                norm = torch.logaddexp(norm, s["sinks"][heads].double())
            out[b, heads], lse[b, heads] = torch.exp(z - norm[:, None]) @ v, norm
    return out, lse


def _rows(cache, block, row, head):
    if cache.dtype == torch.float8_e4m3fn:
        return cache.view(torch.uint8)[block, row, head].view(cache.dtype).double()
    return cache[block, row, head].double()
