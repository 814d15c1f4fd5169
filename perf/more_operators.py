"""Cases of the 4-bit key/value cache and of the page pool that serves a
paged cache: pages handed out and taken back on the GPU with the slot map of
a step's new tokens, the append that writes those tokens, and attention over
what the pages hold.

A 4-bit cache is codes K, V [page][head][slot][dim / 2], two to a byte (the
even dimension in the low half), in e2m1 (sign, 2 exponent bits, 1 mantissa
bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), and one scale byte for every 32 dimensions
[page][head][slot][dim / 32], e8m0: a code stands for
code * 2^(scale - 127).  A page table [sequence][n] and lens [sequence] say
which pages a sequence holds, and how many tokens.

A pool keeps the numbers of its free pages as a stack: free[0 .. count - 1].

Lengths of a case spread evenly from "short" to "tokens" over its sequences;
the seed decides which sequence has which, the pages, and every value.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALVES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
VALUES = HALVES + tuple(-x for x in HALVES)  # of the 16 codes
GROUP = 32  # dimensions of a scale
LEAST, MOST = -64, 125  # exponents of the scales that an append writes


def listed():
    return [
        # one user's first turns: everything is latency
        dict(name="attend first turn", op="attend", batch=1, q_heads=8, heads=2, dim=64, page=16,
             short=259, tokens=259, queries=1, window=0, dtype="bf16"),
        # an ordinary decoding batch with grouped heads
        dict(name="attend batch", op="attend", batch=32, q_heads=32, heads=8, dim=128, page=64,
             short=100, tokens=4096, queries=1, window=0, dtype="bf16"),
        # four drafted tokens checked at once by a model with a sliding window and an odd head size
        dict(name="attend drafts", op="attend", batch=6, q_heads=24, heads=2, dim=96, page=32,
             short=3, tokens=6001, queries=4, window=1000, dtype="fp16"),
        # one book, as long as the cache lets a sequence be here
        dict(name="attend book", op="attend", batch=1, q_heads=64, heads=8, dim=128, page=128,
             short=262143, tokens=262143, queries=1, window=0, dtype="bf16"),
        # wide heads
        dict(name="attend wide heads", op="attend", batch=8, q_heads=16, heads=4, dim=256, page=64,
             short=1500, tokens=16384, queries=1, window=0, dtype="fp16"),
        # a full card: many long conversations
        dict(name="attend many long", op="attend", batch=64, q_heads=32, heads=8, dim=128, page=64,
             short=16000, tokens=16384, queries=1, window=0, dtype="bf16"),
        # a decoding step's tokens, one for each sequence
        dict(name="append one each", op="append", batch=32, heads=8, dim=128, page=64, short=64, tokens=4096,
             fewest=1, new=1, padded=0, dtype="bf16"),
        # pieces of prompts of unlike lengths, packed, in a buffer that is longer than they are
        dict(name="append prompts", op="append", batch=5, heads=6, dim=96, page=16, short=1003, tokens=1501,
             fewest=17, new=1003, padded=77, dtype="fp16"),
        # long prompts
        dict(name="append long prompts", op="append", batch=8, heads=8, dim=128, page=64, short=8192, tokens=8192,
             fewest=8192, new=8192, padded=0, dtype="bf16"),
        # a decoding step: a token each, a few requests end and others take their places
        dict(name="pages of a step", op="pages", batch=64, page=16, short=1, tokens=2000, fewest=1, new=1,
             leave=4, spare=40),
        # prompts and decoding steps together; the pool does not suffice for the last of them
        dict(name="pages of prompts", op="pages", batch=256, page=64, short=0, tokens=8000, fewest=1, new=1900,
             leave=16, spare=-1700),
        # a million tokens of prompts at once, in fine pages
        dict(name="pages of a million", op="pages", batch=1000, page=16, short=0, tokens=4000, fewest=97, new=2003,
             leave=100, spare=9000),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "pages"])
    case = dict(op=op, page=rng.choice([16, 32, 64, 128]))
    if op == "pages":
        case["batch"] = _spread(rng, 1, 2000)
        case["tokens"] = _spread(rng, 1, min(16384, 4000000 // case["batch"]))
        case["short"] = rng.randint(0, case["tokens"])
        case["new"] = rng.choice([1, _spread(rng, 1, max(1, 2000000 // case["batch"] // 2))])
        case["fewest"] = rng.randint(0, case["new"])
        case["leave"] = rng.randint(0, case["batch"])
        case["spare"] = rng.choice([0, 100, -_spread(rng, 1, 1000)])
        return case
    case.update(heads=rng.choice([1, 2, 3, 4, 8, 16]), dim=rng.choice([64, 96, 128, 192, 256]))
    case["batch"] = _spread(rng, 1, 64)
    # at most half a gigabyte of codes
    most = min(262144, (1 << 29) // (case["batch"] * case["heads"] * case["dim"]))
    case["dtype"] = rng.choice(["bf16", "fp16"])
    if op == "attend":
        case["tokens"] = _spread(rng, 1, most)
        case["short"] = rng.choice([case["tokens"], rng.randint(0, case["tokens"])])
        case["q_heads"] = case["heads"] * rng.choice([1, 2, 4, 5, 7, 8])
        case["queries"] = rng.choice([1, 1, 1, 2, 3, 8])
        case["window"] = rng.choice([0, 0, _spread(rng, 16, 4096)])
    else:
        case["tokens"] = _spread(rng, 1, max(1, min(most // 2, 16384)))
        case["new"] = rng.choice([1, _spread(rng, 1, case["tokens"])])
        case["short"] = rng.randint(case["new"], case["tokens"])
        case["fewest"] = rng.choice([case["new"], rng.randint(0, case["new"])])
        case["padded"] = rng.choice([0, rng.randint(1, 64)])
    return case


def _even(batch, low, high):
    """`batch` whole numbers spread evenly from high down to low."""
    return [high - (high - low) * i // max(1, batch - 1) for i in range(batch)]


def _mixed(values, gen):
    order = torch.randperm(len(values), generator=gen, device="cuda")
    return torch.tensor(values, dtype=torch.int32, device="cuda")[order].contiguous()


def _starts(counts):
    """[0, and the running sums of counts], 64 bits."""
    zero = torch.zeros(1, dtype=torch.int64, device=counts.device)
    return torch.cat([zero, torch.cumsum(counts.long(), 0)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, gen)
    op, batch, heads, dim, page = (case[k] for k in ("op", "batch", "heads", "dim", "page"))
    width = max(1, -(-case["tokens"] // page))  # pages a sequence may have
    pages = batch * width + 1  # one page more than the sequences can use, as a pool has
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    st = {"case": case, "table": order[:batch * width].reshape(batch, width).contiguous(),
          "lens": _mixed(_even(batch, case["short"], case["tokens"]), gen)}
    for name in ("k", "v"):
        # every code alike: values of 0.37 to 1.5 root mean square, heavier tails than a normal's
        st[name] = torch.randint(0, 256, (pages, heads, page, dim // 2), generator=gen, device="cuda",
                                 dtype=torch.uint8)
        st[name + "_scale"] = torch.randint(124, 127, (pages, heads, page, dim // GROUP), generator=gen,
                                            device="cuda", dtype=torch.uint8)
    if op == "attend":
        q = torch.randn((batch, case["queries"], case["q_heads"], dim), generator=gen, device="cuda")
        st["q"] = (q * 2).to(TYPES[case["dtype"]])
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((batch, case["queries"], case["q_heads"]), dtype=torch.float32, device="cuda")
    else:
        counts = _mixed(_even(batch, case["fewest"], case["new"]), gen)
        starts = _starts(counts)
        packed = sum(_even(batch, case["fewest"], case["new"])) + case["padded"]
        i = torch.arange(packed, device="cuda")
        b = torch.searchsorted(starts[1:].contiguous(), i, right=True).clamp(max=batch - 1)
        t = (st["lens"].long() - counts.long())[b] + i - starts[b]
        there = i < starts[-1]
        t = torch.where(there, t, torch.zeros_like(t))
        slot = st["table"].long()[b, t // page] * page + t % page
        st["slots"] = torch.where(there, slot, torch.full_like(slot, -1))
        loud = 1 + 7 * (torch.rand((1, heads, dim), generator=gen, device="cuda") < 0.02)
        for name in ("k_new", "v_new"):
            x = torch.randn((packed, heads, dim), generator=gen, device="cuda")
            st[name] = (x * loud).to(TYPES[case["dtype"]])
        # where the read after the append starts: a page before the new tokens
        st["first"] = (st["lens"] - counts - page).contiguous()
    if own:  # the handle that a program keeps for as long as it keeps the tensors
        from cross_core_barrier_amd import kv4
        st["cache"] = kv4.Kv4Cache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
        if op == "attend":
            st["workspace"] = st["cache"].attend_workspace(case["q_heads"], case["queries"])
    return st


def _prepare_pages(case, gen):
    batch, page = case["batch"], case["page"]
    lens = _mixed(_even(batch, case["short"], case["tokens"]), gen)
    counts = _mixed(_even(batch, case["fewest"], case["new"]), gen)
    width = -(-(case["tokens"] + case["new"]) // page)
    held = -(-lens.long() // page)
    # room for what the step asks if nothing is given back, and so many pages more or fewer
    counted = [-(-n // page) for n in _even(batch, case["short"], case["tokens"])]
    ask = [-(-n // page) + 1 for n in _even(batch, case["fewest"], case["new"])]
    pages = max(1, sum(counted) + max(0, sum(ask) + case["spare"]))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = _starts(held)
    j = torch.arange(width, device="cuda")
    inside = j < held.unsqueeze(1)
    index = torch.where(inside, at[:-1].unsqueeze(1) + j, torch.zeros((), dtype=torch.int64, device="cuda"))
    taken = sum(counted)
    free = torch.zeros(pages, dtype=torch.int32, device="cuda")
    free[:pages - taken] = order[taken:]
    # requests that end keep nothing, the others drop up to three drafted tokens
    ends = torch.randperm(batch, generator=gen, device="cuda") < case["leave"]
    drop = torch.randint(0, 4, (batch,), generator=gen, device="cuda")
    keep = torch.where(ends, torch.zeros_like(drop), (lens.long() - drop).clamp(min=0)).to(torch.int32)
    tokens = sum(_even(batch, case["fewest"], case["new"])) + 5  # the buffers of a program are a little longer
    st = {"case": case, "lens": lens, "counts": counts, "keep": keep, "free": free, "tokens": tokens,
          "table": torch.where(inside, order[index], torch.full_like(index, -1).int()).contiguous(),
          "count": torch.full((1,), pages - taken, dtype=torch.int32, device="cuda")}
    if own:
        from cross_core_barrier_amd import pages as pools
        st["pool"] = pools.PagePool(page, st["free"], st["count"])
        st["maps"] = st["pool"].maps(batch, tokens)
    return st


def run(st):
    case = st["case"]
    if own:
        if case["op"] == "pages":
            # the step's accounts: what ended or was rejected goes back, then every request gets its pages
            pool, maps = st["pool"], st["maps"]
            pool.trim(st["table"], st["lens"], st["keep"])
            pool.grow(st["table"], st["lens"], st["counts"], maps)
            return _accounts(st, maps.slots, maps.positions, maps.sequences, maps.starts, maps.granted)
        cache = st["cache"]
        if case["op"] == "attend":
            cache.attend(st["q"], window=case["window"], out=st["out"], lse=st["lse"], workspace=st["workspace"])
            return {"out": st["out"], "lse": st["lse"]}
        cache.append(st["k_new"], st["v_new"], st["slots"])
        k, v = cache.read(case["new"] + case["page"], first=st["first"])
        return {"k": k, "v": v}
    return {"attend": _attend, "append": _append, "pages": _pages}[case["op"]](st, case)


def _accounts(st, slots, positions, sequences, starts, granted):
    return {"table": st["table"], "lens": st["lens"], "free": st["free"], "count": st["count"], "slots": slots,
            "positions": positions, "sequences": sequences, "starts": starts, "granted": granted}


def _values(codes, scales):
    """The values of codes [.., dim / 2] under scales [.., dim / 32], float32."""
    table = torch.tensor(VALUES, dtype=torch.float32, device=codes.device)
    pair = torch.stack([table.repeat(16), table.repeat_interleave(16)], dim=1)  # of a byte: low half, high half
    x = pair.index_select(0, codes.reshape(-1).int()).reshape(*codes.shape[:-1], -1, GROUP)
    x *= _power(scales).unsqueeze(-1)
    return x.flatten(-2)


def _power(biased):
    """2^(biased - 127) for 1 to 254, by the bits of a float32."""
    return (biased.int() << 23).view(torch.float32)


def _dense(st, name, pages, slots):
    """The values at (pages[b, t], slots[b, t]) as [batch, token, head, dim]."""
    return _values(st[name][pages, :, slots], st[name + "_scale"][pages, :, slots])


def _attend(st, case):
    q, lens, table = st["q"], st["lens"].long(), st["table"].long()
    batch, queries, q_heads, dim = q.shape
    heads, page, window = case["heads"], case["page"], case["window"]
    group = q_heads // heads
    t = torch.arange(table.shape[1] * page, device=q.device)
    pages, slots = table[:, t // page], (t % page).expand(batch, -1)
    k = _dense(st, "k", pages, slots).permute(0, 2, 1, 3)
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
    out = torch.matmul(p, _dense(st, "v", pages, slots).permute(0, 2, 1, 3))
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = torch.where(total > 0, m + torch.log(total), torch.full_like(m, -math.inf)).squeeze(-1)
    out = out.reshape(batch, heads, queries, group, dim).permute(0, 2, 1, 3, 4).reshape(q.shape)
    lse = lse.reshape(batch, heads, queries, group).permute(0, 2, 1, 3).reshape(batch, queries, q_heads)
    return {"out": out.to(q.dtype), "lse": lse}


def _quantise(x):
    """x [.., dim] as (codes [.., dim / 2], scales [.., dim / 32])."""
    x = x.float().unflatten(-1, (-1, GROUP))
    size = torch.where(torch.isfinite(x), x.abs(), torch.zeros((), device=x.device)).amax(-1)
    m, e = torch.frexp(size)  # size = m 2^e with m in [0.5, 1): 7 * 2^(e - 3) is 0.875 * 2^e
    e = torch.where(m <= 0.875, e - 3, e - 2).clamp(LEAST, MOST)
    e = torch.where(size > 0, e, torch.full_like(e, LEAST))
    y = x * _power(127 - e).unsqueeze(-1)
    y = torch.nan_to_num(y, nan=0.0, posinf=6.0, neginf=-6.0)
    a = y.abs()
    # steps of 0.5 up to 2, of 1 up to 4, of 2 up to 6; torch.round takes halves to the even one
    r = torch.where(a <= 2, torch.round(a * 2) / 2, torch.where(a <= 4, torch.round(a), torch.round(a / 2) * 2))
    r = r.clamp(max=6.0)
    code = (r * 2 - (r - 2).clamp(min=0) - (r - 4).clamp(min=0) * 0.5).to(torch.uint8)
    code = code + torch.where(y < 0, 8, 0).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _append(st, case):
    page, heads, dim, new = (case[k] for k in ("page", "heads", "dim", "new"))
    lens, table, slots = st["lens"].long(), st["table"].long(), st["slots"]
    batch, dev = lens.numel(), lens.device
    # rows without a slot go where no sequence looks: the pool's page that no table names
    used = torch.zeros(st["k"].shape[0], dtype=torch.int64, device=dev)
    used.scatter_(0, table.flatten(), torch.ones_like(table).flatten())
    nowhere = torch.argmin(used)
    where = torch.where(slots >= 0, slots // page, nowhere)
    for name in ("k", "v"):
        codes, scales = _quantise(st[name + "_new"])
        st[name][where, :, slots % page] = codes
        st[name + "_scale"][where, :, slots % page] = scales
    # what the pages hold now, from a page before the new tokens
    at = st["first"].long().view(-1, 1) + torch.arange(new + page, device=dev)
    inside = (at >= 0) & (at < lens.view(-1, 1))
    at = at.clamp(0, table.shape[1] * page - 1)
    pages, places = table.gather(1, at // page), at % page
    zero = torch.zeros((), device=dev)
    return {name: torch.where(inside.view(batch, -1, 1, 1), _dense(st, name, pages, places), zero)
            for name in ("k", "v")}


def _pages(st, case):
    page, tokens = case["page"], st["tokens"]
    table, free, count = st["table"], st["free"], st["count"]
    batch, width = table.shape
    pages, dev = free.numel(), table.device
    j = torch.arange(width, device=dev)
    # what goes back: the pages behind the kept tokens, the last of them at the bottom
    n = st["lens"].long()
    keep = torch.where(st["keep"] < 0, n, torch.minimum(n, st["keep"].long()))
    low, high = -(-keep // page), -(-n // page)
    before = _starts(high - low)
    inside = (j >= low.unsqueeze(1)) & (j < high.unsqueeze(1))
    goes = count.long() + before[-1] - 1 - (before[:-1] - low).unsqueeze(1) - j
    goes = torch.where(inside, goes, torch.full_like(goes, pages))
    stack = torch.cat([free, free[:1]])
    stack.scatter_(0, goes.flatten(), table.flatten())
    free.copy_(stack[:pages])
    have = count.long() + before[-1]
    # what every sequence gets, in their order, from the top
    n, c = keep, st["counts"].long()
    low, high = -(-n // page), -(-(n + c) // page)
    need = high - low
    after = torch.cumsum(need, 0)
    given = (need == 0) | (after <= have)
    inside = (j >= low.unsqueeze(1)) & (j < high.unsqueeze(1)) & given.unsqueeze(1)
    comes = have - 1 - ((after - need - low).unsqueeze(1) + j)
    table.copy_(torch.where(inside, stack[comes.clamp(0, pages)], table))
    count.copy_(have - torch.where(after <= have, after, torch.zeros_like(after)).amax(0, keepdim=True))
    granted = torch.where(given, c, torch.zeros_like(c))
    st["lens"].copy_(n + granted)
    # the map of the new tokens
    starts = _starts(c)
    i = torch.arange(tokens, device=dev)
    b = torch.searchsorted(starts[1:].contiguous(), i, right=True).clamp(max=batch - 1)
    t = n[b] + i - starts[b]
    there = i < starts[-1]
    placed = there & given[b]
    t = torch.where(placed, t, torch.zeros_like(t))
    none = torch.full_like(t, -1)
    slots = torch.where(placed, table[b, t // page].long() * page + t % page, none)
    return _accounts(st, slots, torch.where(placed, t, none).int(), torch.where(there, b, none).int(), starts.int(),
                     granted.int())


def work(case):
    batch, page = case["batch"], case["page"]
    if case["op"] == "pages":
        new = sum(_even(batch, case["fewest"], case["new"]))
        # a token's slot, place and sequence; a page read, and written to the table or the stack; six numbers a sequence
        return {"bytes": 16 * new + 8 * (new // page) + 24 * batch, "flops": 0}
    heads, dim = case["heads"], case["dim"]
    lens = _even(batch, case["short"], case["tokens"])
    each = dim // 2 + dim // GROUP  # bytes of a token's key, and of its value
    if case["op"] == "attend":
        queries, rows = case["queries"], case["queries"] * case["q_heads"] // heads
        seen = [min(n, case["window"] + queries - 1) if case["window"] else n for n in lens]
        moved = sum(seen) * heads * 2 * each + batch * case["q_heads"] * queries * (4 * dim + 4)
        pairs = sum(max(0, min(n - queries + i + 1, case["window"] or n)) for n in lens for i in range(queries))
        return {"bytes": moved, "flops": 4 * dim * pairs * rows // queries * heads}
    counts = _even(batch, case["fewest"], case["new"])
    # the new values in, their codes out; then places read, and their values out
    shown = [min(n, c + page) for n, c in zip(lens, counts)]
    moved = sum(counts) * heads * 2 * (2 * dim + each) + sum(shown) * heads * 2 * each
    moved += batch * (case["new"] + page) * heads * 2 * dim * 4
    return {"bytes": moved, "flops": 2 * sum(counts) * heads * 2 * dim}


# The same results from the definitions, one sequence at a time and in 64 bits.


def _number(codes, scales):
    """Codes [.., dim / 2] and scales [.., dim / 32] as numbers, from the bits of sign, exponent and mantissa."""
    half = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    exponent, mantissa = (half >> 1) & 3, (half & 1).double()
    size = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * _two_to(exponent - 1))
    x = torch.where(half >= 8, -size, size)
    return x * _two_to(scales.long() - 127).repeat_interleave(GROUP, dim=-1)


def _two_to(e):
    """2^e (whole numbers) in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _held(st, name, b, n):
    """Sequence b's first n tokens, [token, head, dim]."""
    page = st["case"]["page"]
    used = st["table"][b, :max(1, -(-n // page))].long()
    x = _number(st[name][used], st[name + "_scale"][used])
    return x.transpose(1, 2).flatten(0, 1)[:n]


def _rounded(x):
    """x [.., dim] (64 bits) as the values that a 4-bit cache keeps of it."""
    grid = torch.tensor(HALVES, dtype=torch.float64, device=x.device)
    x = x.unflatten(-1, (-1, GROUP))
    size = x.abs().amax(-1, keepdim=True)
    # the least power of two that leaves nothing off by more than half a step: values up to 7 become 6
    e = torch.ceil(torch.log2(size / 7)).clamp(LEAST - 1, MOST + 1)
    e = torch.where(7 * _two_to(e) < size, e + 1, torch.where(7 * _two_to(e - 1) >= size, e - 1, e))
    unit = _two_to(e.clamp(LEAST, MOST))
    a = (x.abs() / unit).clamp(max=6.0)
    above = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    low, high = grid[above - 1], grid[above]
    up = (a - low > high - a) | ((a - low == high - a) & (above % 2 == 0))
    return (torch.where(up, high, low) * torch.sign(x) * unit).flatten(-2)


def exact(case, seed):
    if case["op"] == "pages":
        return _exact_pages(case, seed)
    st = prepare(case, seed)
    lens = st["lens"].tolist()
    batch, heads, dim, page = (case[k] for k in ("batch", "heads", "dim", "page"))
    dev = st["k"].device
    if case["op"] == "attend":
        queries, q_heads = case["queries"], case["q_heads"]
        out = torch.zeros((batch, queries, q_heads, dim), dtype=torch.float64, device=dev)
        lse = torch.full((batch, queries, q_heads), -math.inf, dtype=torch.float64, device=dev)
        for b, n in enumerate(lens):
            k, v = _held(st, "k", b, n), _held(st, "v", b, n)
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
        return {"out": out, "lse": lse}
    first, slots = st["first"].tolist(), st["slots"].tolist()
    # a row's sequence and token, from the table
    table = st["table"].tolist()
    owner = {number: (b, j) for b, row in enumerate(table) for j, number in enumerate(row)}
    rows = [(owner[s // page][0], owner[s // page][1] * page + s % page, i) for i, s in enumerate(slots) if s >= 0]
    outs = {}
    for name in ("k", "v"):
        new = _rounded(st[name + "_new"].double())
        got = torch.zeros((batch, case["new"] + page, heads, dim), dtype=torch.float64, device=dev)
        for b, n in enumerate(lens):
            value = _held(st, name, b, n)
            mine = [(t, i) for o, t, i in rows if o == b]
            if mine:
                at, of = torch.tensor(mine, device=dev).unbind(1)
                value[at] = new[of]
            low, high = max(0, first[b]), min(n, first[b] + case["new"] + page)
            got[b, low - first[b]:high - first[b]] = value[low:high]
        outs[name] = got
    return outs


def _exact_pages(case, seed):
    """Sequence by sequence, with lists."""
    st = prepare(case, seed)
    page = case["page"]
    table, free, have = st["table"].tolist(), st["free"].tolist(), int(st["count"])
    lens, keep, counts = st["lens"].tolist(), st["keep"].tolist(), st["counts"].tolist()
    back = []
    for b, n in enumerate(lens):
        lens[b] = n if keep[b] < 0 else min(n, keep[b])
        back += table[b][-(-lens[b] // page):-(-n // page)]
    for number in reversed(back):
        free[have] = number
        have += 1
    slots, positions, sequences, starts, granted = [], [], [], [0], []
    asked = room = have
    for b, c in enumerate(counts):
        n = lens[b]
        low, high = -(-n // page), -(-(n + c) // page)
        asked -= high - low
        fits = high == low or asked >= 0  # nobody passes one who has to wait
        if fits:
            for j in range(low, high):
                have -= 1
                table[b][j] = free[have]
            lens[b] = n + c
        granted.append(c if fits else 0)
        for t in range(n, n + c):
            slots.append(table[b][t // page] * page + t % page if fits else -1)
            positions.append(t if fits else -1)
            sequences.append(b)
        starts.append(starts[-1] + c)
    assert 0 <= have <= room
    more = [-1] * (st["tokens"] - len(slots))
    dev = st["table"].device
    whole = {"table": table, "lens": lens, "free": free, "count": [have], "positions": positions + more,
             "sequences": sequences + more, "starts": starts, "granted": granted}
    out = {name: torch.tensor(x, dtype=torch.int32, device=dev) for name, x in whole.items()}
    out["slots"] = torch.tensor(slots + more, dtype=torch.int64, device=dev)
    return out
