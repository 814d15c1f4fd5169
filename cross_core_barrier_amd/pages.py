"""The pages of a paged cache, handed out and taken back on the GPU: one class
around the ccb_pages_* calls of include/ccb_pages.h.  The page tables that it
keeps are those of Kv8Cache and Kv4Cache.

    pool = PagePool.allocate(pages=4096, page_size=64)
    maps = pool.maps(batch=16, tokens=2048)      # room for a step's new tokens
    pool.trim(cache.page_table, cache.lens, keep)             # ended: keep 0, rejected drafts: fewer, -1: all
    pool.grow(cache.page_table, cache.lens, counts, maps)     # counts[b] new tokens of each sequence
    cache.append(k_new, v_new, maps.slots)       # a Kv4Cache; a Kv8Cache takes maps.granted as its counts

Calls run on the pool's device, whichever is current: on torch's current stream
there, or on `stream` as in Kv8Cache.  They copy nothing to the host, so that a
step that ends in them and begins with them can be captured into a HIP graph.
Calls on one pool, and on one table, follow each other.  Bad lengths, counts
and page numbers are met on the device: they set `pool.err`, which
`pool.check()` reads (and waits for).  That a sequence gets no room because the
pool is empty is no error: maps.granted says so.
"""

from __future__ import annotations

import torch

from . import ccb
from .kv8 import OnDevice, _need

_INT = torch.int32


class SlotMaps:
    """Where a step's new tokens go, packed sequence after sequence (of the
    tokens that the sequences asked for, granted or not):
    slots [tokens] int64, a token's page * page_size + its place there, or -1;
    positions [tokens] int32, its place in its sequence, or -1; sequences
    [tokens] int32, its sequence, or -1 behind the last token; starts [batch +
    1] int32, the first token of each sequence, and their number; granted
    [batch] int32, how many tokens the sequence got room for."""

    def __init__(self, batch: int, tokens: int, device):
        self.slots = torch.full((tokens,), -1, dtype=torch.int64, device=device)
        self.positions, self.sequences = (torch.full((tokens,), -1, dtype=torch.int32, device=device)
                                          for _ in range(2))
        self.starts = torch.zeros(batch + 1, dtype=torch.int32, device=device)
        self.granted = torch.zeros(batch, dtype=torch.int32, device=device)
        self._batch, self._index = batch, self.slots.get_device()
        self._c = ccb.ccbSlotMaps(self.slots.data_ptr(), self.positions.data_ptr(), self.sequences.data_ptr(),
                                  self.starts.data_ptr(), self.granted.data_ptr(), tokens, 0)

    def __setattr__(self, name: str, value) -> None:
        """The kernels get the addresses: contents change, tensors do not."""
        if self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name}: change the tensor in place, or make other maps")
        object.__setattr__(self, name, value)


class PagePool(OnDevice):
    """A pool in the caller's tensors: free [pages] int32, the numbers of the
    free pages as a stack, and count [1] int32, how many of them are in use.
    Both contiguous and on one GPU; they stay the same tensors for the pool's
    life."""

    _what = "page pool"

    def __init__(self, page_size: int, free: torch.Tensor, count: torch.Tensor):
        _need(free.dim() == 1 and free.dtype == torch.int32 and free.is_contiguous()
              and 1 <= free.shape[0] < 2 ** 30, "free: [pages] int32, contiguous")
        _need(tuple(count.shape) == (1,) and count.dtype == torch.int32 and count.device == free.device,
              "count: [1] int32, beside free")
        _need(1 <= page_size <= 32768 and page_size & (page_size - 1) == 0, "page_size: a power of two up to 32768")
        self.page_size, self.free, self.count, self.device = page_size, free, count, free.device
        self._index = free.get_device()  # -1 on the CPU
        self.err = torch.zeros(1, dtype=torch.int32, device=free.device)
        self._state = torch.zeros(ccb.CCB_PAGES_STATE_BYTES // 4, dtype=torch.int32, device=free.device)
        self._err = self.err.data_ptr()
        self._c = ccb.ccbPagePool(free.data_ptr(), count.data_ptr(), self._state.data_ptr(), free.shape[0], page_size)

    @classmethod
    def allocate(cls, pages: int, page_size: int, device="cuda") -> "PagePool":
        """All pages free, the lowest handed out first."""
        free = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)
        return cls(page_size, free, torch.full((1,), pages, dtype=torch.int32, device=device))

    def maps(self, batch: int, tokens: int) -> SlotMaps:
        """Tensors for grow() of `batch` sequences and up to `tokens` new tokens."""
        _need(0 <= batch <= ccb.CCB_PAGES_MAX_BATCH and 0 <= tokens < 2 ** 30,
              f"maps: up to {ccb.CCB_PAGES_MAX_BATCH} sequences, less than 2^30 tokens")
        return SlotMaps(batch, tokens, self.device)

    def _table(self, page_table: torch.Tensor, lens: torch.Tensor, numbers: torch.Tensor, what: str):
        """The table as the library takes it.  The checks are few steps on
        purpose: a call's time on the host is most of a decoding step's."""
        index = self._index
        batch, width = page_table.shape if page_table.dim() == 2 else (-1, 0)
        stride, last = page_table.stride() if batch >= 0 else (0, 0)
        if batch < 0 or width < 1 or last != 1 or page_table.dtype is not _INT or page_table.get_device() != index:
            raise ValueError(f"page_table: [batch, max_pages] int32 on {self.device}, rows contiguous")
        for t in (lens, numbers):
            if t.dtype is not _INT or t.get_device() != index or t.dim() != 1 or t.shape[0] != batch \
                    or not t.is_contiguous():
                raise ValueError(f"{'lens' if t is lens else what}: [{batch}] int32, contiguous, on {self.device}")
        return ccb.ccbPageTable(page_table.data_ptr(), lens.data_ptr(), stride if batch > 1 else width, batch, width)

    def trim(self, page_table: torch.Tensor, lens: torch.Tensor, keep: torch.Tensor, stream=None) -> None:
        """Cut sequence b to its first keep[b] tokens (int32; negative: all stay)
        and take back the pages behind them."""
        if self._index < 0:
            self._on_gpu()
        table = self._table(page_table, lens, keep, "keep")
        s = None if stream is None else self._enter(stream)
        self._call(ccb.ccb_pages_trim, s, self._c, table, keep, self._err)

    def grow(self, page_table: torch.Tensor, lens: torch.Tensor, counts: torch.Tensor, maps: SlotMaps,
             stream=None) -> None:
        """Give sequence b room for counts[b] (int32) more tokens: its pages into
        the table, lens, and where each token goes into maps."""
        if self._index < 0:
            self._on_gpu()
        table = self._table(page_table, lens, counts, "counts")
        if maps._batch != table.batch or maps._index != self._index:
            raise ValueError("maps: for as many sequences, on the pool's device")
        s = None if stream is None else self._enter(stream)
        self._call(ccb.ccb_pages_grow, s, self._c, table, counts, maps._c, self._err)
