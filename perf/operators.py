"""Cases of the 8-bit key/value cache operators: attention of a decoding step
over a paged cache with one scale for each block of tokens and head, the
append that fills such a cache, and the eviction that bounds it.

A cache is codes K, V [page][head][slot][dim] in int8 or e4m3, scales
[page][head], a page table [sequence][n], lens [sequence] (tokens held) and
the accumulated attention weight [sequence][head][token].  A code stands for
code * scale.

Lengths of a case spread evenly from "short" to "tokens" over its sequences;
the seed decides which sequence has which, the pages, and every value.
"""

import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
TINY = 2.0 ** -64  # the smallest scale of a block that holds anything


def listed():
    return [
        # one user's first turns: everything is latency
        dict(name="attend first turn", op="attend", batch=1, q_heads=8, heads=8, dim=64, page=16,
             short=203, tokens=203, queries=1, window=0, fmt="int8", dtype="bf16", weights=False),
        # a small model with a cache head for each query head, mixed lengths, fine blocks
        dict(name="attend own heads", op="attend", batch=24, q_heads=16, heads=16, dim=64, page=32,
             short=1, tokens=1009, queries=1, window=0, fmt="int8", dtype="fp16", weights=True),
        # an ordinary decoding batch with grouped heads, weights kept for eviction
        dict(name="attend batch", op="attend", batch=16, q_heads=32, heads=8, dim=128, page=64,
             short=500, tokens=4096, queries=1, window=0, fmt="e4m3", dtype="bf16", weights=True),
        # five drafted tokens checked at once by a model with a sliding window and an odd head size
        dict(name="attend drafts", op="attend", batch=6, q_heads=24, heads=2, dim=96, page=64,
             short=3, tokens=5001, queries=5, window=1024, fmt="int8", dtype="fp16", weights=True),
        # one very long document
        dict(name="attend document", op="attend", batch=1, q_heads=64, heads=8, dim=128, page=128,
             short=131071, tokens=131071, queries=1, window=0, fmt="int8", dtype="bf16", weights=True),
        # a full server: a gigabyte of cache in one step
        dict(name="attend server", op="attend", batch=64, q_heads=32, heads=8, dim=128, page=64,
             short=8000, tokens=8192, queries=1, window=0, fmt="e4m3", dtype="bf16", weights=False),
        # every sequence of a decoding batch gains its next token
        dict(name="append step", op="append", batch=32, heads=8, dim=128, page=64, short=100,
             tokens=3001, new=1, fewest=1, fmt="e4m3", dtype="bf16"),
        # a few prompts of unlike length behind what the cache holds already
        dict(name="append prompts", op="append", batch=4, heads=4, dim=96, page=32, short=1009,
             tokens=2500, new=1000, fewest=17, fmt="int8", dtype="fp16"),
        # long prompts into an empty cache
        dict(name="append documents", op="append", batch=8, heads=8, dim=128, page=64, short=8192,
             tokens=8192, new=8192, fewest=8192, fmt="int8", dtype="bf16"),
        # two short talks, cut to a window of recent and heavy tokens
        dict(name="evict talks", op="evict", batch=2, heads=4, dim=64, page=16, short=90,
             tokens=301, budget=128, recent=32, sinks=4, fmt="int8"),
        # a decoding batch cut to a quarter
        dict(name="evict batch", op="evict", batch=16, heads=8, dim=128, page=64, short=500,
             tokens=4096, budget=1024, recent=128, sinks=4, fmt="e4m3"),
        # a very long document cut to an eighth
        dict(name="evict document", op="evict", batch=1, heads=8, dim=128, page=128, short=131071,
             tokens=131071, budget=16384, recent=1024, sinks=4, fmt="int8"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    case = dict(op=op, heads=rng.choice([1, 2, 3, 4, 8, 16]), dim=rng.choice([64, 96, 128, 192, 256]),
                page=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["int8", "e4m3"]))
    room = 1 << 28  # bytes of cache a drawn case may hold
    case["batch"] = _spread(rng, 1, 64)
    most = min(131072, room // (2 * case["batch"] * case["heads"] * case["dim"]))
    if op == "attend":
        case["tokens"] = _spread(rng, 1, most)
        case["short"] = rng.choice([case["tokens"], rng.randint(0, case["tokens"])])
        case["q_heads"] = case["heads"] * rng.choice([1, 2, 4, 5, 7, 8])
        case["queries"] = rng.choice([1, 1, 1, 2, 3, 8])
        case["window"] = rng.choice([0, 0, _spread(rng, 16, 4096)])
        case["dtype"] = rng.choice(["bf16", "fp16"])
        case["weights"] = rng.random() < 0.5
    elif op == "append":
        case["tokens"] = _spread(rng, 1, min(most, 16384))
        case["new"] = rng.choice([1, _spread(rng, 1, case["tokens"])])
        case["short"] = rng.randint(case["new"], case["tokens"])
        case["fewest"] = rng.choice([case["new"], rng.randint(0, case["new"])])
        case["dtype"] = rng.choice(["bf16", "fp16"])
    else:
        case["tokens"] = _spread(rng, 32, max(32, most))
        case["short"] = rng.randint(1, case["tokens"])
        case["budget"] = _spread(rng, 16, case["tokens"])
        case["sinks"] = rng.choice([0, 4])
        case["recent"] = rng.randint(0, case["budget"] - case["sinks"])
    return case


def _even(batch, low, high):
    """`batch` whole numbers spread evenly from high down to low."""
    return [high - (high - low) * i // max(1, batch - 1) for i in range(batch)]


def _codes(shape, fmt, gen):
    spread = torch.randn(shape, generator=gen, device="cuda")
    if fmt == "int8":
        return (spread * 32).round().clamp(-127, 127).to(torch.int8)
    return (spread * 96).clamp(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, batch, heads, dim, page, fmt = (case[k] for k in ("op", "batch", "heads", "dim", "page", "fmt"))
    width = max(1, -(-case["tokens"] // page))  # pages a sequence may have
    out_width = -(-case["budget"] // page) if op == "evict" else 0
    # one page more than the sequences can use, as a pool has
    pages = batch * (width + out_width) + 1
    order = torch.randperm(pages - 1, generator=gen, device="cuda").to(torch.int32)
    mixed = torch.randperm(batch, generator=gen, device="cuda")
    lens = torch.tensor(_even(batch, case["short"], case["tokens"]), dtype=torch.int32, device="cuda")[mixed]
    unit = 0.02 if fmt == "int8" else 0.007
    st = {
        "case": case,
        "k": _codes((pages, heads, page, dim), fmt, gen),
        "v": _codes((pages, heads, page, dim), fmt, gen),
        "k_scale": (0.5 + torch.rand((pages, heads), generator=gen, device="cuda")) * unit,
        "v_scale": (0.5 + torch.rand((pages, heads), generator=gen, device="cuda")) * unit,
        "table": order[:batch * width].reshape(batch, width).contiguous(),
        "lens": lens.contiguous(),
        "weight": None,
    }
    if op != "attend" or case["weights"]:
        # a few tokens draw most of the attention, many have none; an attending
        # step comes early, so that what it adds weighs as much as what is there
        w = torch.rand((batch, heads, width * page), generator=gen, device="cuda")
        st["weight"] = torch.where(w < 0.25, torch.zeros_like(w), (w ** 8) * (0.01 if op == "attend" else 20))
    if op == "attend":
        q = torch.randn((batch, case["queries"], case["q_heads"], dim), generator=gen, device="cuda")
        st["q"] = (q * 2).to(TYPES[case["dtype"]])
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((batch, case["queries"], case["q_heads"]), dtype=torch.float32, device="cuda")
    elif op == "append":
        shape = (batch, case["new"], heads, dim)
        loud = 1 + 3 * (torch.rand((1, 1, heads, dim), generator=gen, device="cuda") < 0.02)
        for name in ("k_new", "v_new"):
            st[name] = (torch.randn(shape, generator=gen, device="cuda") * loud).to(TYPES[case["dtype"]])
        st["counts"] = torch.tensor(_even(batch, case["fewest"], case["new"]), dtype=torch.int32,
                                    device="cuda")[torch.randperm(batch, generator=gen, device="cuda")].contiguous()
        # where the read after the append starts: a page before the new tokens
        st["first"] = (st["lens"] - st["counts"] - page).contiguous()
    else:
        st["out_table"] = order[batch * width:].reshape(batch, out_width).contiguous()
        st["out_lens"] = torch.empty_like(st["lens"])
        st["out_weight"] = torch.empty((batch, heads, out_width * page), dtype=torch.float32, device="cuda")
        st["kept"] = torch.empty((batch, heads, case["budget"]), dtype=torch.int32, device="cuda")
    if own:  # the handles that a program keeps for as long as it keeps the tensors
        from cross_core_barrier_amd import kv8
        st["cache"] = kv8.Kv8Cache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"], st["lens"],
                                   st["weight"])
        if op == "attend":
            st["workspace"] = st["cache"].attend_workspace(case["q_heads"], case["queries"], case["weights"])
        elif op == "evict":
            st["workspace"] = st["cache"].evict_workspace(case["budget"])
            st["out_cache"] = kv8.Kv8Cache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["out_table"],
                                           st["out_lens"], st["out_weight"])
    return st


def run(st):
    case = st["case"]
    if own:
        cache = st["cache"]
        if case["op"] == "attend":
            cache.attend(st["q"], window=case["window"], accumulate=case["weights"], out=st["out"], lse=st["lse"],
                         workspace=st["workspace"])
            return {"out": st["out"], "lse": st["lse"], "weight": st["weight"]}
        if case["op"] == "append":
            cache.append(st["k_new"], st["v_new"], st["counts"])
            k, v = cache.read(case["new"] + case["page"], first=st["first"])
            return {"k": k, "v": v, "weight": st["weight"]}
        cache.evict(st["out_cache"], case["budget"], recent=case["recent"], sinks=case["sinks"], kept=st["kept"],
                    workspace=st["workspace"])
        k, v = st["out_cache"].read(case["budget"])
        width = case["budget"]
        return {"kept": st["kept"], "lens": st["out_lens"], "weight": st["out_weight"][..., :width], "k": k, "v": v}
    return {"attend": _attend, "append": _append, "evict": _evict}[case["op"]](st, case)


def _take(codes, scales, pages, slots):
    """The values at (pages[b, t], slots[b, t]) as [batch, token, head, dim]."""
    got = codes.view(torch.uint8)[pages, :, slots].view(codes.dtype).float()
    return got * scales[pages].unsqueeze(-1)


def _attend(st, case):
    q, lens, table = st["q"], st["lens"].long(), st["table"].long()
    batch, queries, q_heads, dim = q.shape
    heads, page, window = case["heads"], case["page"], case["window"]
    group = q_heads // heads
    t = torch.arange(table.shape[1] * page, device=q.device)
    pages, slots = table[:, t // page], (t % page).expand(batch, -1)
    k = _take(st["k"], st["k_scale"], pages, slots).permute(0, 2, 1, 3)
    # rows of a cache head: query i, member g
    rows = q.float().reshape(batch, queries, heads, group, dim).permute(0, 2, 1, 3, 4)
    rows = rows.reshape(batch, heads, queries * group, dim)
    s = torch.matmul(rows, k.transpose(2, 3)) / math.sqrt(dim)
    del k
    last = (lens.view(-1, 1) - queries + torch.arange(queries, device=q.device)).repeat_interleave(group, dim=1)
    seen = t.view(1, 1, -1) <= last.unsqueeze(-1)
    if window:
        seen = seen & (t.view(1, 1, -1) > last.unsqueeze(-1) - window)
    seen = seen.unsqueeze(1)
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(s - m), torch.zeros_like(s))
    del s
    total = p.sum(-1, keepdim=True)
    v = _take(st["v"], st["v_scale"], pages, slots).permute(0, 2, 1, 3)
    out = torch.matmul(p, v)
    del v
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = torch.where(total > 0, m + torch.log(total), torch.full_like(m, -math.inf)).squeeze(-1)
    if st["weight"] is not None:
        share = torch.where(total > 0, p / total, torch.zeros_like(p))
        st["weight"] += share.sum(2)
    out = out.reshape(batch, heads, queries, group, dim).permute(0, 2, 1, 3, 4).reshape(q.shape)
    lse = lse.reshape(batch, heads, queries, group).permute(0, 2, 1, 3).reshape(batch, queries, q_heads)
    return {"out": out.to(q.dtype), "lse": lse, "weight": st["weight"]}


def _block_scale(a, fmt):
    """The scale of blocks whose largest value is a (float32)."""
    s = (a.double() / torch.full_like(a, QMAX[fmt], dtype=torch.float64)).float()
    return torch.where(a > 0, s.clamp(min=TINY), torch.zeros_like(s))


def _quantised(ratio, fmt):
    """The codes next to `ratio` (float64, so that no value lands on the wrong side of a border)."""
    ratio = torch.nan_to_num(ratio, nan=0.0, posinf=QMAX[fmt], neginf=-QMAX[fmt])
    if fmt == "int8":
        return ratio.round().clamp(-127, 127).to(torch.int8)
    _, e = torch.frexp(ratio.abs())
    step = (((e - 1).clamp(min=-6) - 3 + 1023).long() << 52).view(torch.float64)  # 2^(exponent - 3), by its bits
    return ((ratio / step).round() * step).clamp(-448, 448).float().to(torch.float8_e4m3fn)


def _append(st, case):
    fmt, page, heads, dim, new = (case[k] for k in ("fmt", "page", "heads", "dim", "new"))
    lens, counts, table = st["lens"].long(), st["counts"].long(), st["table"].long()
    batch, dev = lens.numel(), lens.device
    start = lens - counts
    i = torch.arange(new, device=dev)
    pos = start.view(-1, 1) + i
    fresh = i.view(1, -1) < counts.view(-1, 1)
    # the pages that may be touched, from the one that `start` lies in
    span = -(-new // page) + 1
    number = (start // page).view(-1, 1) + torch.arange(span, device=dev)
    touched = (number * page < lens.view(-1, 1)) & ((number + 1) * page > start.view(-1, 1)) & (counts.view(-1, 1) > 0)
    spare = st["k"].shape[0] - 1
    pages = torch.where(touched, table.gather(1, number.clamp(max=table.shape[1] - 1)), torch.full_like(number, spare))
    slot_pos = number.unsqueeze(-1) * page + torch.arange(page, device=dev)
    old = (slot_pos < start.view(-1, 1, 1)).view(batch, span, 1, page, 1)
    isnew = ((slot_pos >= start.view(-1, 1, 1)) & (slot_pos < lens.view(-1, 1, 1))).view(batch, span, 1, page, 1)
    held = (number * page < start.view(-1, 1)).view(batch, span, 1)
    seq = torch.arange(batch, device=dev).view(-1, 1).expand(-1, new)
    local = torch.where(fresh, pos // page - (start // page).view(-1, 1), torch.full_like(pos, span))
    for codes, scales, x in ((st["k"], st["k_scale"], st["k_new"]), (st["v"], st["v_scale"], st["v_new"])):
        block = torch.zeros((batch, span + 1, heads, page, dim), dtype=x.dtype, device=dev)
        block[seq, local, :, pos % page] = x
        block = block[:, :span]
        size = torch.where(isnew & torch.isfinite(block), block.float().abs(), torch.zeros((), device=dev))
        s0 = torch.where(held, scales[pages], torch.zeros((), device=dev))
        s1 = torch.maximum(s0, _block_scale(size.amax((3, 4)), fmt))
        by = s1.double().view(batch, span, heads, 1, 1)
        have = codes.view(torch.uint8)[pages].view(codes.dtype)
        scaled = have.float().double() * s0.double().view(batch, span, heads, 1, 1) / by
        moved = torch.where((s1 > s0).view(batch, span, heads, 1, 1), _quantised(scaled, fmt).view(torch.uint8),
                            have.view(torch.uint8))
        written = _quantised(block.double() / by, fmt).view(torch.uint8)
        codes.view(torch.uint8)[pages] = torch.where(isnew, written, torch.where(old, moved, have.view(torch.uint8)))
        scales[pages] = s1
    t = torch.arange(st["weight"].shape[-1], device=dev).view(1, 1, -1)
    st["weight"].masked_fill_((t >= start.view(-1, 1, 1)) & (t < lens.view(-1, 1, 1)), 0.0)
    # what the pages hold now, from a page before the new tokens
    at = st["first"].long().view(-1, 1) + torch.arange(new + page, device=dev)
    inside = (at >= 0) & (at < lens.view(-1, 1))
    at = at.clamp(0, table.shape[1] * page - 1)
    where, slots = table.gather(1, at // page), at % page
    zero = torch.zeros((), device=dev)
    k = torch.where(inside.view(batch, -1, 1, 1), _take(st["k"], st["k_scale"], where, slots), zero)
    v = torch.where(inside.view(batch, -1, 1, 1), _take(st["v"], st["v_scale"], where, slots), zero)
    return {"k": k, "v": v, "weight": st["weight"]}


def _evict(st, case):
    fmt, page, budget = case["fmt"], case["page"], case["budget"]
    lens, table, weight = st["lens"].long(), st["table"].long(), st["weight"]
    batch, heads, room = weight.shape
    dev = weight.device
    t = torch.arange(room, device=dev).view(1, 1, -1)
    held = lens.view(-1, 1, 1)
    stay = lens.clamp(max=budget)
    key = torch.where((t < case["sinks"]) | (t >= held - case["recent"]), torch.full_like(weight, math.inf), weight)
    key = torch.where(t < held, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, t.expand_as(order).contiguous())
    mask = rank < stay.view(-1, 1, 1)
    goes = torch.where(mask, mask.long().cumsum(-1) - 1, torch.full_like(order, budget))
    kept = torch.full((batch, heads, budget + 1), -1, dtype=torch.int64, device=dev)
    kept.scatter_(2, goes, t.expand_as(goes).contiguous())
    kept = kept[..., :budget]
    there = kept >= 0
    at = kept.clamp(min=0)
    new_weight = torch.where(there, weight.gather(2, at), torch.zeros((), device=dev))
    width = st["out_table"].shape[1]
    pad = width * page - budget
    at, there = torch.nn.functional.pad(at, (0, pad)), torch.nn.functional.pad(there, (0, pad))
    src = table.view(batch, 1, -1).expand(-1, heads, -1).gather(2, at // page)
    slot = at % page
    head = torch.arange(heads, device=dev).view(1, -1, 1)
    outs = {}
    for name in ("k", "v"):
        codes, scales = st[name], st[name + "_scale"]
        got = codes.view(torch.uint8)[src, head, slot].view(codes.dtype).float()
        by = torch.where(there, scales[src, head], torch.zeros((), device=dev))
        dim = got.shape[-1]
        size = (got.abs().amax(-1) * by).reshape(batch, heads, width, page).amax(-1)
        s1 = _block_scale(size, fmt)
        each = s1.repeat_interleave(page, dim=2).unsqueeze(-1)
        new = _quantised(got.double() * by.double().unsqueeze(-1) / each.double(), fmt)
        blocks = new.view(torch.uint8).reshape(batch, heads, width, page, dim).transpose(1, 2)
        codes.view(torch.uint8)[st["out_table"].long()] = blocks
        scales[st["out_table"].long()] = s1.transpose(1, 2)
        value = torch.where(there.unsqueeze(-1), new.float() * each, torch.zeros((), device=dev))
        outs[name] = value[:, :, :budget].transpose(1, 2).contiguous()
    return {"kept": kept.int(), "lens": stay.int(), "weight": new_weight, **outs}


def work(case):
    batch, heads, dim, page = case["batch"], case["heads"], case["dim"], case["page"]
    lens = _even(batch, case["short"], case["tokens"])
    if case["op"] == "attend":
        queries, rows = case["queries"], case["queries"] * case["q_heads"] // heads
        seen = [min(n, case["window"] + queries - 1) if case["window"] else n for n in lens]
        moved = sum(heads * n * 2 * dim for n in seen) + sum(heads * -(-n // page) * 8 for n in seen)
        moved += batch * case["q_heads"] * queries * (4 * dim + 4)
        if case["weights"]:
            moved += sum(seen) * heads * 8
        pairs = sum(max(0, min(n - queries + i + 1, case["window"] or n)) for n in lens for i in range(queries))
        return {"bytes": moved, "flops": 4 * dim * pairs * rows // queries * heads}
    if case["op"] == "append":
        counts = _even(batch, case["fewest"], case["new"])
        cells = sum(counts) * heads * 2 * dim
        # the new values in, their codes out, and the read of `new + page` places
        shown = batch * (case["new"] + page) * heads * 2 * dim
        return {"bytes": cells * 3 + shown * 4 + sum(counts) * heads * 4, "flops": 2 * cells}
    stay = [min(n, case["budget"]) for n in lens]
    cells = sum(stay) * heads * 2 * dim
    shown = batch * case["budget"] * heads * 2 * dim
    return {"bytes": sum(lens) * heads * 4 + cells * 2 + shown * 4 + sum(stay) * heads * 8, "flops": 2 * cells}


# The same results from the definitions, one sequence at a time and in 64 bits.


def _e4m3_values():
    """The values of the 256 e4m3 codes: sign, 4 exponent bits biased by 7, 3 mantissa bits; 0x7F is no number."""
    values = []
    for code in range(256):
        exponent, mantissa = (code >> 3) & 15, code & 7
        size = mantissa / 8 * 2.0 ** -6 if exponent == 0 else (1 + mantissa / 8) * 2.0 ** (exponent - 7)
        values.append(math.nan if code & 127 == 127 else -size if code & 128 else size)
    return values


def _numbers(codes):
    if codes.dtype == torch.int8:
        return codes.double()
    return torch.tensor(_e4m3_values(), dtype=torch.float64, device=codes.device)[codes.view(torch.uint8).long()]


def _dense(st, which, b, n, table="table"):
    """Sequence b's first n tokens: the codes' values and the scales, [token, head, dim] and [token, head]."""
    page = st["case"]["page"]
    used = st[table][b, :max(1, -(-n // page))].long()
    codes = _numbers(st[which].view(torch.uint8)[used].view(st[which].dtype))
    codes = codes.transpose(1, 2).flatten(0, 1)[:n]
    scales = st[which + "_scale"][used].double().repeat_interleave(page, dim=0)[:n]
    return codes, scales


def _nearest(x, fmt):
    """x [..] (64 bits) to the nearest value of the format, ties to the even code."""
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    grid = torch.tensor(_e4m3_values()[:127], dtype=torch.float64, device=x.device)
    size = x.abs().clamp(max=448.0)
    above = torch.searchsorted(grid, size).clamp(1, 126)
    low, high = grid[above - 1], grid[above]
    up = (size - low > high - size) | ((size - low == high - size) & (above % 2 == 0))
    return torch.where(up, high, low) * torch.sign(x)


def _scale_of(a, fmt):
    s = (a / QMAX[fmt]).float().double().clamp(min=TINY)
    return torch.where(a > 0, s, torch.zeros_like(s))


def exact(case, seed):
    st = prepare(case, seed)
    lens = st["lens"].tolist()
    batch, heads, dim, page, fmt = (case[k] for k in ("batch", "heads", "dim", "page", "fmt"))
    dev = st["k"].device
    if case["op"] == "attend":
        queries, q_heads = case["queries"], case["q_heads"]
        out = torch.zeros((batch, queries, q_heads, dim), dtype=torch.float64, device=dev)
        lse = torch.full((batch, queries, q_heads), -math.inf, dtype=torch.float64, device=dev)
        weight = st["weight"].double() if case["weights"] else None
        for b, n in enumerate(lens):
            (kc, ks), (vc, vs) = _dense(st, "k", b, n), _dense(st, "v", b, n)
            k, v = kc * ks.unsqueeze(-1), vc * vs.unsqueeze(-1)
            for i in range(queries):
                end = n - queries + i + 1
                begin = max(0, end - case["window"]) if case["window"] else 0
                if end <= begin:
                    continue
                q = st["q"][b, i].double().reshape(heads, -1, dim)
                s = torch.matmul(q, k[begin:end].permute(1, 2, 0).contiguous()) / math.sqrt(dim)
                lse[b, i] = torch.logsumexp(s, -1).flatten()
                p = torch.softmax(s, -1)
                out[b, i] = torch.matmul(p, v[begin:end].transpose(0, 1).contiguous()).reshape(q_heads, dim)
                if weight is not None:
                    weight[b, :, begin:end] += p.sum(1)
        return {"out": out, "lse": lse, "weight": weight}
    if case["op"] == "append":
        counts, first = st["counts"].tolist(), st["first"].tolist()
        outs = {}
        for which in ("k", "v"):
            got = torch.zeros((batch, case["new"] + page, heads, dim), dtype=torch.float64, device=dev)
            for b, n in enumerate(lens):
                start = n - counts[b]
                codes, scales = _dense(st, which, b, n)
                value = codes * scales.unsqueeze(-1)
                value[start:n] = st[which + "_new"][b, :counts[b]].double()
                # whole pages of the touched part: [page, slot, head, dim]
                base = start // page * page
                over = -(n - base) % page
                if counts[b]:
                    part = torch.nn.functional.pad(value[base:n], (0, 0, 0, 0, 0, over)).reshape(-1, page, heads, dim)
                    fresh = torch.arange(base, n + over, device=dev).reshape(-1, page, 1, 1) >= start
                    s1 = _scale_of((part.abs() * fresh).amax((1, 3)), fmt)
                    if start > base:
                        s1[0] = torch.maximum(s1[0], scales[base])
                    grid = s1.reshape(-1, 1, heads, 1)
                    back = torch.where(grid > 0, _nearest(part / grid, fmt) * grid, torch.zeros_like(part))
                    value[base:n] = back.flatten(0, 1)[:n - base]
                low, high = max(0, first[b]), min(n, first[b] + case["new"] + page)
                got[b, low - first[b]:high - first[b]] = value[low:high]
            outs[which] = got
        weight = st["weight"].double()
        for b, n in enumerate(lens):
            weight[b, :, n - counts[b]:n] = 0
        return {**outs, "weight": weight}
    budget = case["budget"]
    kept = torch.full((batch, heads, budget), -1, dtype=torch.int32, device=dev)
    weight = torch.zeros((batch, heads, budget), dtype=torch.float64, device=dev)
    outs = {w: torch.zeros((batch, budget, heads, dim), dtype=torch.float64, device=dev) for w in ("k", "v")}
    for b, n in enumerate(lens):
        stay = min(n, budget)
        held = {w: _dense(st, w, b, n) for w in ("k", "v")}
        for h in range(heads):
            if n <= budget:
                index = torch.arange(n, device=dev)
            else:
                low, high = case["sinks"], n - case["recent"]
                free = budget - case["sinks"] - case["recent"]
                best = torch.argsort(st["weight"][b, h, low:high].double(), descending=True, stable=True)[:free] + low
                ends = [torch.arange(low, device=dev), best, torch.arange(high, n, device=dev)]
                index = torch.cat(ends).sort().values
            kept[b, h, :stay] = index.int()
            weight[b, h, :stay] = st["weight"][b, h, index].double()
            for w in ("k", "v"):
                codes, scales = held[w]
                value = codes[index, h] * scales[index, h].unsqueeze(-1)
                blocks = torch.nn.functional.pad(value, (0, 0, 0, -stay % page)).reshape(-1, page, dim)
                s1 = _scale_of(blocks.abs().amax((1, 2)).float().double(), fmt).reshape(-1, 1, 1)
                back = torch.where(s1 > 0, _nearest(blocks / s1, fmt) * s1, torch.zeros_like(blocks))
                outs[w][b, :stay, h] = back.flatten(0, 1)[:stay]
    return {"kept": kept, "lens": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32, device=dev),
            "weight": weight, **outs}
