"""The 4-bit key/value cache over torch tensors: one class around the
ccb_kv4_* calls of include/ccb_kv4.h.  PyTorch provides memory and streams
only; every step runs in libccb.so's HIP kernels.

    cache = Kv4Cache.allocate(pages=4096, heads=8, page_size=64, head_dim=128, batch=16, max_pages=256)
    pool = PagePool.allocate(4096, 64)           # cross_core_barrier_amd.pages
    maps = pool.maps(batch=16, tokens=16)
    pool.grow(cache.page_table, cache.lens, counts, maps)  # pages and slots of the new tokens
    cache.append(k_new, v_new, maps.slots)       # [tokens, heads, head_dim]
    out, lse = cache.attend(q)                   # q [batch, 1, q_heads, head_dim]

Calls run on the cache's device, whichever is current: on torch's current
stream there, or on `stream` (a torch.cuda.Stream or a raw hipStream_t of that
device) after the work already queued on the current stream, which is then
ordered after them.  They copy nothing to the host and compute no gradients:
rows that ask for one are refused, but under torch.no_grad().  Bad page
numbers, lengths and slots are met on the device: they set `cache.err`, which
`cache.check()` reads (and waits for).
"""

from __future__ import annotations

from typing import Optional

import torch

from . import ccb
from .kv8 import _ROWS, OnDevice, _int32, _need, _no_gradient

GROUP = 32  # dimensions that share a scale
_PACKED = {t: kind for t, kind in _ROWS.items() if kind != ccb.CCB_KV8_FP32}


class Kv4Cache(OnDevice):
    """A cache in the caller's tensors (they are kept, not copied, and stay
    the same tensors with the same storage for the cache's life):
    k, v [pages, heads, page_size, head_dim / 2] uint8, two e2m1 codes to a
    byte, the even dimension in the low half; k_scale, v_scale [pages, heads,
    page_size, head_dim / 32] uint8, e8m0; page_table [batch, max_pages] int32;
    lens [batch] int32.  All contiguous, but for the page table's rows, and on
    one GPU: a cache on the CPU can be made, but every call on it is refused."""

    _what = "4-bit cache"

    def __init__(self, k, v, k_scale, v_scale, page_table, lens):
        _need(k.dim() == 4 and k.dtype == torch.uint8, "k: [pages, heads, page_size, head_dim / 2] uint8")
        pages, heads, page_size, half = k.shape
        _need(v.shape == k.shape and v.dtype == k.dtype, "v: shape and dtype of k")
        _need(half % (GROUP // 2) == 0, "head_dim: a multiple of 32")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(tuple(s.shape) == (pages, heads, page_size, 2 * half // GROUP) and s.dtype == torch.uint8,
                  f"{name}: [pages, heads, page_size, head_dim / 32] uint8")
        _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.shape[1] >= 1 and
              page_table.stride(1) == 1, "page_table: [batch, max_pages] int32")
        batch, max_pages = page_table.shape
        _need(tuple(lens.shape) == (batch,) and lens.dtype == torch.int32, "lens: [batch] int32")
        for t in (k, v, k_scale, v_scale, lens):
            _need(t.is_contiguous(), "cache tensors are contiguous")
        for t in (v, k_scale, v_scale, page_table, lens):
            _need(t.device == k.device, "cache tensors share a device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table, self.lens = page_table, lens
        self.heads, self.head_dim, self.batch, self.device = heads, 2 * half, batch, k.device
        self._index = k.get_device()  # -1 on the CPU
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._err = self.err.data_ptr()
        self._c = ccb.ccbKv4Cache(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
            lens.data_ptr(), page_table.stride(0) if batch > 1 else max_pages, pages, heads, page_size, 2 * half,
            batch, max_pages)

    @classmethod
    def allocate(cls, pages: int, heads: int, page_size: int, head_dim: int, batch: int, max_pages: int,
                 device="cuda") -> "Kv4Cache":
        """Zeroed tensors: no sequence holds a token, every page number is 0."""
        _need(head_dim % GROUP == 0, "head_dim: a multiple of 32")
        k, v = (torch.zeros((pages, heads, page_size, head_dim // 2), dtype=torch.uint8, device=device)
                for _ in range(2))
        ks, vs = (torch.zeros((pages, heads, page_size, head_dim // GROUP), dtype=torch.uint8, device=device)
                  for _ in range(2))
        table = torch.zeros((batch, max_pages), dtype=torch.int32, device=device)
        return cls(k, v, ks, vs, table, torch.zeros(batch, dtype=torch.int32, device=device))

    def _packed(self, t: torch.Tensor, what: str):
        kind = _PACKED.get(t.dtype)
        if kind is not None and t.dim() == 3 and t.get_device() == self._index:
            n, heads, dim = t.shape
            st, sh, sd = t.stride()
            if heads == self.heads and dim == self.head_dim and (sd == 1 or t.numel() == 0):
                # the stride of a dimension with one place is never used
                return ccb.ccbKv8Rows(t.data_ptr(), 0, st if n > 1 else 0, sh if heads > 1 else 0, kind, 0)
        raise ValueError(f"{what}: [tokens, heads {self.heads}, head_dim {self.head_dim}] on {self.device}, "
                         "bfloat16 or float16, the last dimension contiguous")

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """Write tokens k_new, v_new [tokens, heads, head_dim], each to its
        slot (page * page_size + place in the page) of slots [tokens] int64; a
        slot of -1 leaves its token out.  page_table and lens are not looked
        at: PagePool.grow makes all three."""
        if self._index < 0:
            self._on_gpu()
        k, v = self._packed(k_new, "k_new"), self._packed(v_new, "v_new")
        if k_new.requires_grad or v_new.requires_grad:
            _no_gradient("k_new, v_new")
        n = k_new.shape[0]
        if n != v_new.shape[0] or k.type != v.type:
            raise ValueError("v_new: shape and dtype of k_new")
        if n >> 31:
            _int32("tokens", n)
        if slots.dtype is not torch.int64 or slots.dim() != 1 or slots.shape[0] != n \
                or slots.get_device() != self._index or not slots.is_contiguous():
            raise ValueError(f"slots: [{n}] int64, contiguous, on {self.device}")
        s = None if stream is None else self._enter(stream)
        self._call(ccb.ccb_kv4_append, s, self._c, k, v, n, slots, self._err)

    def attend_workspace(self, q_heads: int, queries: int = 1) -> torch.Tensor:
        """A workspace for attend() calls of these sizes that follow each other."""
        if self._index < 0:
            self._on_gpu()
        _int32("attend", q_heads, queries)
        n = ccb.ccb_kv4_attend_workspace_bytes(self._c, q_heads, queries)
        _need(n > 0, "attend: sizes that ccb_kv4_attend refuses")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attend(self, q: torch.Tensor, scale: Optional[float] = None, window: int = 0,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None):
        """Attention of q [batch, queries, q_heads, head_dim], the sequences'
        last tokens; scale None is 1 / sqrt(head_dim).  Returns (out, lse).
        out may be q itself."""
        if self._index < 0:
            self._on_gpu()
        if q.dim() != 4:
            raise ValueError("q: [batch, queries, q_heads, head_dim]")
        if q.requires_grad:
            _no_gradient("q")
        if not 0 <= window < 2 ** 31:  # (the library gets the low 32 bits)
            raise ValueError("window: 0 (none) to 2^31 - 1 tokens")
        shape = q.shape
        queries, q_heads = shape[1], shape[2]
        s = None if stream is None else self._enter(stream)
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=q.device)
            if s is not None:
                out.record_stream(s)
        if lse is None:
            lse = torch.empty(shape[:3], dtype=torch.float32, device=q.device)
            if s is not None:
                lse.record_stream(s)
        qr, outr = self._rows(q, q_heads, "q"), self._rows(out, q_heads, "out")
        if out.shape[1] != queries or outr.type != qr.type:
            raise ValueError("out: shape and dtype of q")
        if lse.shape != shape[:3] or lse.dtype is not torch.float32 or lse.get_device() != self._index \
                or not lse.is_contiguous():
            raise ValueError("lse: [batch, queries, q_heads] float32, contiguous")
        need = 0 if workspace is not None else ccb.ccb_kv4_attend_workspace_bytes(self._c, q_heads, queries)
        ws, size = self._space(workspace, need, s)
        self._call(ccb.ccb_kv4_attend, s, self._c, qr, outr, lse, q_heads, queries,
                   self.head_dim ** -0.5 if scale is None else scale, window, ws, size, self._err)
        return out, lse

    def read(self, count: int, first: Optional[torch.Tensor] = None, dtype=torch.float32, stream=None):
        """The values of `count` tokens of each sequence from first[b] (None: 0)
        as (k, v) [batch, count, heads, head_dim]; zeros where there is none."""
        if self._index < 0:
            self._on_gpu()
        kind = _ROWS.get(dtype)
        if kind is None:
            raise ValueError("dtype: float32, bfloat16 or float16")
        if first is not None:
            self._ints(first, (self.batch,), "first")
        _int32("count", count)
        s = None if stream is None else self._enter(stream)
        both = torch.empty((2, self.batch, count, self.heads, self.head_dim), dtype=dtype, device=self.device)
        if s is not None:
            both.record_stream(s)
        k, v = both.unbind(0)
        row, dim = self.heads * self.head_dim, self.head_dim
        self._call(ccb.ccb_kv4_read, s, self._c, ccb.ccbKv8Rows(k.data_ptr(), count * row, row, dim, kind, 0),
                   ccb.ccbKv8Rows(v.data_ptr(), count * row, row, dim, kind, 0), count, first, self._err)
        return k, v
