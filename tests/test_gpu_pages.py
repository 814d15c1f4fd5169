"""The page pool on the GPU against the oracle (oracle/pages.py): every number
is compared exactly, the ones that nothing may touch among them."""

import random

import numpy as np
import pytest

from oracle.pages import Pool

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _say(msg):
    print(f"[gpu case] {msg}", flush=True)


@pytest.fixture(scope="module")
def pages():
    from cross_core_barrier_amd import ccb, pages as module
    st, _, _, _ = ccb.ccb_device_info()
    assert st == 0, ccb.ccb_status_string(st)
    return module


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pair:
    """A pool with a table on the GPU, and the oracle of both."""

    def __init__(self, pages, rng, page_size, lens, width, spare, wide=0):
        held = [-(-n // page_size) for n in lens]
        numbers = list(range(sum(held) + spare))
        rng.shuffle(numbers)
        table = [[rng.randrange(-5, 1 << 20) for _ in range(width)] for _ in lens]  # behind the held ones: anything
        at = 0
        for row, n in zip(table, held):
            row[:n] = numbers[at:at + n]
            at += n
        free = numbers[at:] + [rng.randrange(-5, 1 << 20) for _ in range(at)]
        self.oracle = Pool(page_size, free, spare, table, lens)
        self.pool = pages.PagePool(page_size, _ints(free), _ints([spare]))
        whole = _ints(table) if lens else torch.zeros((0, width), dtype=torch.int32, device="cuda")
        # rows of a wider table
        self.table = torch.full((len(lens), width + wide), -77, dtype=torch.int32, device="cuda")[:, :width]
        self.table.copy_(whole)
        self.lens = _ints(lens) if lens else torch.zeros(0, dtype=torch.int32, device="cuda")

    def same(self):
        o = self.oracle
        assert self.table.tolist() == o.table
        assert self.lens.tolist() == o.lens
        assert self.pool.count.tolist() == [o.count]
        assert self.pool.free.tolist() == o.free
        assert not self.pool._state.any()
        from cross_core_barrier_amd import ccb
        assert (self.pool.err.item() == ccb.CCB_ERR_INVALID_VALUE) == o.bad and self.pool.err.item() >= 0
        self.pool.err.zero_()
        o.bad = False

    def trim(self, keep, **kw):
        self.pool.trim(self.table, self.lens, _ints(keep), **kw)
        self.oracle.trim(keep)
        self.same()

    def grow(self, counts, tokens, **kw):
        maps = self.pool.maps(len(counts), tokens)
        for t in (maps.slots, maps.positions, maps.sequences, maps.starts, maps.granted):
            t.fill_(-99)
        self.pool.grow(self.table, self.lens, _ints(counts), maps, **kw)
        want = self.oracle.grow(counts, tokens)
        for got, x, name in zip((maps.slots, maps.positions, maps.sequences, maps.starts, maps.granted), want,
                                ("slots", "positions", "sequences", "starts", "granted")):
            assert got.tolist() == x, name
        self.same()
        return maps


@pytest.mark.parametrize("page_size", [1, 16, 64, 128, 4096])
@pytest.mark.parametrize("batch", [1, 2, 7, 64, 255, 256, 257, 1000, 1024, 1025, 3000])
def test_steps(pages, page_size, batch):
    rng = random.Random(page_size * 10007 + batch)
    width = 9
    room = width * page_size
    lens = [rng.choice([0, rng.randint(0, room // 2)]) for _ in range(batch)]
    p = Pair(pages, rng, page_size, lens, width, batch * 3, wide=rng.choice([0, 3]))
    _say(f"pages: steps, P={page_size} batch={batch}")
    for _ in range(3):
        p.trim([rng.choice([-1, -1, 0, max(0, n - rng.randint(0, 3)), n, n + 5]) for n in p.oracle.lens])
        small = rng.random() < 0.5
        most = min(room, 1 + 40000 // batch)
        counts = [min(room - n, 1 if small else rng.choice([0, 1, rng.randint(0, most)])) for n in p.oracle.lens]
        p.grow(counts, max(0, sum(counts) + rng.choice([0, 1, 2, 3, 70])))


def test_everything_at_its_limits(pages):
    _say("pages: empty stacks, full tables, nothing asked, one of 8192 sequences")
    rng = random.Random(5)
    p = Pair(pages, rng, 16, [0, 17, 160], 10, 0)
    p.grow([0, 15, 0], 15)     # room in the last page: needs none
    p.grow([1, 0, 0], 4)       # the stack is empty
    p.trim([0, 0, 0])
    p.grow([160, 0, 32], 192)  # to the table's end, and the stack's
    p.grow([0, 0, 0], 0)
    p.grow([0, 0, 0], 5)
    p.trim([-1, -1, -1])
    p.trim([0, 5, 31])
    p = Pair(pages, rng, 32, [rng.randint(0, 64) for _ in range(8192)], 3, 9000)
    p.grow([rng.randint(0, 32) if n <= 64 else 0 for n in p.oracle.lens], 8192 * 32)
    p.trim([rng.choice([-1, 0, 20]) for _ in range(8192)])
    p = Pair(pages, rng, 32, [], 3, 7)
    p.pool.trim(p.table, p.lens, p.lens)
    maps = p.pool.maps(0, 6)
    maps.slots.fill_(5)
    p.pool.grow(p.table, p.lens, p.lens, maps)
    assert maps.slots.tolist() == [-1] * 6 and maps.starts.tolist() == [0]
    p.same()


def test_waits_in_line(pages):
    """Nobody passes a sequence that has to wait, but one that needs no page."""
    _say("pages: first come, first served")
    rng = random.Random(6)
    for spare in range(0, 12):
        p = Pair(pages, rng, 8, [0, 3, 8, 16, 0, 5], 6, spare)
        p.grow([17, 5, 9, 24, 0, 4], 70)
    p = Pair(pages, rng, 16, [rng.randint(0, 100) for _ in range(700)], 40, 900)
    p.grow([rng.randint(0, 300) for _ in range(700)], 700 * 300)


def test_trim_undoes_grow(pages):
    _say("pages: a trim that undoes a grow")
    rng = random.Random(7)
    lens = [rng.randint(0, 200) for _ in range(100)]
    p = Pair(pages, rng, 16, lens, 40, 2000)
    before, count = p.pool.free.clone(), p.pool.count.clone()
    p.grow([rng.randint(0, 300) for _ in lens], 30000)
    p.trim(lens)
    assert torch.equal(p.pool.free, before) and torch.equal(p.pool.count, count)


def test_a_million_tokens(pages):
    _say("pages: a million tokens")
    rng = random.Random(8)
    p = Pair(pages, rng, 16, [rng.randint(0, 4000) for _ in range(500)], 400, 70000)
    p.grow([rng.randint(1500, 2300) for _ in range(500)], 500 * 2300 + 3)
    p.trim([rng.choice([0, 1700, -1]) for _ in range(500)])


def test_bad_numbers_are_met(pages):
    _say("pages: bad lengths, counts, pages and stacks")
    rng = random.Random(9)

    def make(lens=(5, 20, 0, 60), spare=8):
        return Pair(pages, rng, 16, list(lens), 5, spare)

    def set_lens(p, lens):
        p.lens.copy_(_ints(lens))
        p.oracle.lens = list(lens)
    for lens in ([-1, 20, 0, 60], [5, 81, 0, 60], [5, 20, 0, 2 ** 31 - 1], [-2 ** 31, 20, 0, 60]):
        p = make()
        set_lens(p, lens)
        p.grow([1, 2, 3, 4], 12)
        p = make()
        set_lens(p, lens)
        p.trim([0, 0, 0, 0])
    for counts in ([-1, 2, 3, 4], [1, 61, 3, 4], [2 ** 31 - 1, 2, 3, 2 ** 31 - 1], [-2 ** 31, 2, 3, 4], [76, 3, 2, 1]):
        make().grow(counts, 100)
    for tokens in (0, 1, 9, 10):  # too few places
        make().grow([1, 2, 3, 4], tokens)
    for bad in (-1, 1 << 30, 2 ** 31 - 1):
        p = make()  # a page that is held already, and one from the stack
        p.table[0, 0] = bad
        p.oracle.table[0][0] = bad
        p.pool.free[6] = bad
        p.oracle.free[6] = bad
        p.grow([1, 20, 20, 4], 50)
        p.trim([0, 0, 0, 0])
    for count in (-1, -2 ** 31, 100, 2 ** 31 - 1):
        p = make()
        p.pool.count.fill_(count)
        p.oracle.count = count
        p.grow([1, 20, 3, 4], 50)
        p.trim([0, 0, 0, 0])
    p = make()  # pages given back twice
    p.trim([0, 0, 0, 0])
    set_lens(p, [5, 20, 0, 60])
    p.trim([0, 0, 0, 0])
    with pytest.raises(Exception, match="page pool"):
        p.pool.err.fill_(1)
        p.pool.check()
    p.pool.check()


def test_maps_may_be_left_out(pages):
    from cross_core_barrier_amd import ccb
    _say("pages: grow without maps")
    rng = random.Random(10)
    p = Pair(pages, rng, 16, [5, 20, 0, 60], 5, 8)
    counts = [20, 1, 17, 3]
    none = ccb.ccbSlotMaps(0, 0, 0, 0, 0, 41, 0)
    asked = _ints(counts)
    assert ccb.ccb_pages_grow(p.pool._c, p.pool._table(p.table, p.lens, asked, "counts"), asked, none, p.pool.err) == 0
    p.oracle.grow(counts, 41)
    torch.cuda.synchronize()
    p.same()


def test_side_stream_and_graph(pages):
    """A step's accounts captured once and replayed with other counts, eager
    work between; and on a stream of the caller's."""
    rng = random.Random(11)
    lens = [rng.randint(0, 100) for _ in range(300)]
    p = Pair(pages, rng, 16, lens, 30, 3000)
    s = torch.cuda.Stream()
    _say("pages: a side stream")
    p.trim([rng.choice([-1, 0, 50]) for _ in lens], stream=s)
    p.grow([rng.randint(0, 40) for _ in lens], 300 * 40, stream=s)
    keep, counts, maps = _ints([-1] * 300), _ints([0] * 300), p.pool.maps(300, 12000)
    p.pool.trim(p.table, p.lens, keep)
    p.pool.grow(p.table, p.lens, counts, maps)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.pool.trim(p.table, p.lens, keep)
        p.pool.grow(p.table, p.lens, counts, maps)
    p.same()
    for rep in range(5):
        _say(f"pages: replay {rep}")
        k = [rng.choice([-1, 0, max(0, n - 2)]) for n in p.oracle.lens]
        keep.copy_(_ints(k))
        p.oracle.trim(k)
        c = [min(40, 480 - n) for n in p.oracle.lens]
        counts.copy_(_ints(c))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = p.oracle.grow(c, 12000)
        assert maps.slots.tolist() == want[0] and maps.granted.tolist() == want[4]
        p.same()


def test_serves_the_8_bit_cache(pages):
    """The tables that a pool makes, under a Kv8Cache: granted tokens as counts."""
    from cross_core_barrier_amd.kv8 import Kv8Cache
    _say("pages: under an 8-bit cache")
    pool = pages.PagePool.allocate(10, 16)
    cache = Kv8Cache.allocate(12, 2, 16, 64, 3, 6, "int8")
    maps = pool.maps(3, 100)
    gen = torch.Generator(device="cuda").manual_seed(3)
    held = [torch.zeros((0, 2, 64), device="cuda") for _ in range(3)]
    for counts in ([20, 3, 33], [1, 1, 1], [0, 40, 2], [5, 45, 1]):
        pool.grow(cache.page_table, cache.lens, _ints(counts), maps)
        n = max(counts)
        x = torch.randn((3, n, 2, 64), generator=gen, device="cuda").half()
        cache.append(x, x, maps.granted)
        got = maps.granted.tolist()
        for b in range(3):
            held[b] = torch.cat([held[b], x[b, :got[b]].float()])
    assert got == [5, 0, 1]
    k, _ = cache.read(96)
    for b in range(3):
        n = held[b].shape[0]
        assert cache.lens[b].item() == n
        # scales grow with the block: a code is within a step of the largest value's 127th
        assert torch.all((k[b, :n] - held[b]).abs() <= held[b].abs().amax() / 127 * 1.5)
        assert not k[b, n:].any()
    cache.check()
    pool.check()
