"""The page pool on the CPU: the oracle on worked values, refusals of the C
entry points before anything is enqueued, and the class's checks."""

import ctypes

import pytest

from oracle.pages import Pool

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ccb():
    from cross_core_barrier_amd import ccb as lib
    return lib


def test_oracle_on_worked_values():
    p = Pool(4, [9, 8, 7, 6, 5, 0, 0, 0, 0, 0], 5, [[1, 2, -1], [3, -1, -1], [-1, -1, -1]], [7, 4, 0])
    slots, positions, sequences, starts, granted = p.grow([1, 2, 5], 10)
    assert p.table == [[1, 2, -1], [3, 5, -1], [6, 7, -1]] and p.lens == [8, 6, 5] and p.count == 2
    assert slots == [11, 20, 21, 24, 25, 26, 27, 28, -1, -1]
    assert positions == [7, 4, 5, 0, 1, 2, 3, 4, -1, -1] and sequences == [0, 1, 1, 2, 2, 2, 2, 2, -1, -1]
    assert starts == [0, 1, 3, 8] and granted == [1, 2, 5] and not p.bad
    p.trim([7, 4, 0])
    assert p.free[:5] == [9, 8, 7, 6, 5] and p.count == 5 and p.lens == [7, 4, 0]
    p.trim([0, -1, 0])  # a sequence's last page goes back first
    assert p.free[:7] == [9, 8, 7, 6, 5, 2, 1] and p.count == 7 and p.lens == [0, 4, 0]


def test_oracle_first_come_first_served():
    p = Pool(2, [0, 1, 2, 3], 3, [[-1] * 4, [-1] * 4, [3, -1, -1, -1], [-1] * 4], [0, 0, 1, 0])
    slots, _, _, _, granted = p.grow([4, 3, 1, 1], 9)
    # two pages, two that are not there, room in a page, and one that has to wait behind the second
    assert granted == [4, 0, 1, 0] and p.count == 1 and p.lens == [4, 0, 2, 0]
    assert slots == [4, 5, 2, 3, -1, -1, -1, 7, -1]


def test_struct_sizes(ccb):
    assert ctypes.sizeof(ccb.ccbPagePool) == 3 * 8 + 2 * 4
    assert ctypes.sizeof(ccb.ccbPageTable) == 3 * 8 + 2 * 4
    assert ctypes.sizeof(ccb.ccbSlotMaps) == 5 * 8 + 2 * 4


def _pool(ccb, **change):
    f = dict(free=1 << 20, count=2 << 20, state=3 << 20, numPages=64, pageSize=16)
    f.update(change)
    return ccb.ccbPagePool(**f)


def _table(ccb, **change):
    f = dict(pages=4 << 20, lens=5 << 20, stride=4, batch=3, maxPages=4)
    f.update(change)
    return ccb.ccbPageTable(**f)


def _maps(ccb, **change):
    f = dict(slots=6 << 20, positions=7 << 20, sequences=8 << 20, starts=9 << 20, granted=10 << 20, tokens=100,
             reserved=0)
    f.update(change)
    return ccb.ccbSlotMaps(**f)


@pytest.mark.parametrize("change", [dict(numPages=0), dict(numPages=1 << 30), dict(pageSize=0), dict(pageSize=24),
                                    dict(pageSize=65536), dict(free=2), dict(count=2), dict(state=64)], ids=str)
def test_refuses_a_bad_pool(ccb, change):
    p, t, numbers = _pool(ccb, **change), _table(ccb), 11 << 20
    assert ccb.ccb_pages_trim(p, t, numbers) == ccb.CCB_ERR_INVALID_VALUE
    assert ccb.ccb_pages_grow(p, t, numbers, _maps(ccb)) == ccb.CCB_ERR_INVALID_VALUE


@pytest.mark.parametrize("change", [dict(batch=-1), dict(batch=8193), dict(maxPages=0), dict(stride=3), dict(pages=2),
                                    dict(lens=2), dict(maxPages=(1 << 26) + 1, stride=1 << 27)], ids=str)
def test_refuses_a_bad_table(ccb, change):
    p, t, numbers = _pool(ccb), _table(ccb, **change), 11 << 20
    assert ccb.ccb_pages_trim(p, t, numbers) == ccb.CCB_ERR_INVALID_VALUE
    assert ccb.ccb_pages_grow(p, t, numbers, _maps(ccb)) == ccb.CCB_ERR_INVALID_VALUE


@pytest.mark.parametrize("change", [dict(tokens=-1), dict(tokens=1 << 30), dict(reserved=1), dict(slots=8),
                                    dict(positions=8), dict(sequences=8), dict(starts=2), dict(granted=2)], ids=str)
def test_refuses_bad_maps(ccb, change):
    assert ccb.ccb_pages_grow(_pool(ccb), _table(ccb), 11 << 20, _maps(ccb, **change)) == ccb.CCB_ERR_INVALID_VALUE


def test_refuses_missing_pointers(ccb):
    null, inv, ok = ccb.CCB_ERR_NULL_POINTER, ccb.CCB_ERR_INVALID_VALUE, ccb.CCB_OK
    p, t, m, x = _pool(ccb), _table(ccb), _maps(ccb), 11 << 20
    assert ccb.ccb_pages_trim(None, t, x) == null and ccb.ccb_pages_trim(p, None, x) == null
    assert ccb.ccb_pages_trim(p, t, None) == null and ccb.ccb_pages_trim(p, t, 2) == inv
    assert ccb.ccb_pages_trim(p, t, x, err=2) == inv
    assert ccb.ccb_pages_grow(None, t, x, m) == null and ccb.ccb_pages_grow(p, None, x, m) == null
    assert ccb.ccb_pages_grow(p, t, None, m) == null and ccb.ccb_pages_grow(p, t, x, None) == null
    assert ccb.ccb_pages_grow(p, t, x, m, err=2) == inv
    for name in ("free", "count", "state"):
        assert ccb.ccb_pages_trim(_pool(ccb, **{name: 0}), t, x) == null, name
        assert ccb.ccb_pages_grow(_pool(ccb, **{name: 0}), t, x, m) == null, name
    for name in ("pages", "lens"):
        assert ccb.ccb_pages_trim(p, _table(ccb, **{name: 0}), x) == null, name
        assert ccb.ccb_pages_grow(p, _table(ccb, **{name: 0}), x, m) == null, name
    assert ccb.ccb_pages_trim(p, _table(ccb, batch=0, pages=0, lens=0), None) == ok  # nothing to do


def test_class_checks_its_tensors(monkeypatch):
    from cross_core_barrier_amd import ccb, kv8, pages
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    for args in ((24, ints(8), ints(1)), (0, ints(8), ints(1)), (16, ints(8).long(), ints(1)), (16, ints(2, 4), ints(1)),
                 (16, ints(8), ints(2)), (16, ints(8), ints(1).long()), (16, ints(16)[::2], ints(1)),
                 (16, ints(0), ints(1))):
        with pytest.raises(ValueError):
            pages.PagePool(*args)
    pool = pages.PagePool.allocate(8, 16, device="cpu")
    assert pool.free.tolist() == [7, 6, 5, 4, 3, 2, 1, 0] and pool.count.tolist() == [8]
    maps = pool.maps(3, 10)
    for call in (lambda: pool.trim(ints(3, 2), ints(3), ints(3)),
                 lambda: pool.grow(ints(3, 2), ints(3), ints(3), maps)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
    for name in ("free", "count", "err", "_state", "_c"):
        with pytest.raises(AttributeError):
            setattr(pool, name, None)
    with pytest.raises(AttributeError):
        maps.slots = None
    for batch, tokens in ((8193, 1), (-1, 1), (1, -1), (1, 1 << 30)):
        with pytest.raises(ValueError):
            pool.maps(batch, tokens)
    # with the checks of the device out of the way: shapes and types
    reached = []
    for name in ("trim", "grow"):
        monkeypatch.setattr(ccb, f"ccb_pages_{name}", lambda *a, _n=name: reached.append(_n) or 0)
    monkeypatch.setattr(kv8, "_current_stream", lambda index: 0)
    monkeypatch.setattr(kv8, "_current_device", lambda: -1)
    monkeypatch.setattr(pages.PagePool, "_on_gpu", lambda self: None)
    good = (ints(3, 2), ints(3), ints(3))
    bad = [(ints(3, 2).long(), ints(3), ints(3)), (ints(2, 3).t(), ints(3), ints(3)), (ints(3, 0), ints(3), ints(3)),
           (ints(3, 2), ints(2), ints(3)), (ints(3, 2), ints(3), ints(2)), (ints(3, 2), ints(3), ints(3).long()),
           (ints(3), ints(3), ints(3))]
    for args in bad:
        with pytest.raises(ValueError):
            pool.trim(*args)
        with pytest.raises(ValueError):
            pool.grow(*args, maps)
    with pytest.raises(ValueError):
        pool.grow(*good, pool.maps(2, 10))
    assert reached == []
    pool.trim(*good)
    pool.grow(*good, maps)
    assert reached == ["trim", "grow"]
