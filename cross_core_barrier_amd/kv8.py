"""The 8-bit key/value cache over torch tensors: one class around the
ccb_kv8_* calls of include/ccb_kv8.h.  PyTorch provides memory and streams
only; every step runs in libccb.so's HIP kernels.

    cache = Kv8Cache.allocate(pages=4096, heads=8, page_size=64, head_dim=128,
                              batch=16, max_pages=256, fmt="e4m3", weights=True)
    cache.page_table[...] = ...                # pages from the caller's allocator
    cache.lens += 1                            # one token more for every sequence
    cache.append(k_new, v_new)                 # [batch, 1, heads, head_dim]
    out, lse = cache.attend(q, accumulate=True)  # q [batch, 1, q_heads, head_dim]
    cache.evict(smaller, budget=1024, recent=128, sinks=4, kept=kept)  # kept: which tokens, or None

Calls run on the cache's device, whichever is current: on torch's current
stream there, or on `stream` (a torch.cuda.Stream or a raw hipStream_t of that
device) after the work already queued on the current stream, which is then
ordered after them.  They copy nothing to the host and compute no gradients:
rows that ask for one are refused, but under torch.no_grad().  Bad page
numbers, lengths and counts are met on the device: they set `cache.err`, which
`cache.check()` reads (and waits for).
"""

from __future__ import annotations

from typing import Optional

import torch

from . import ccb
from .workloads import _enter, _leave

_CODES = {torch.int8: ccb.CCB_KV8_INT8, torch.float8_e4m3fn: ccb.CCB_KV8_E4M3}
_FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_current_stream = torch._C._cuda_getCurrentRawStream  # the handle alone: a tenth of the object's cost
_current_device = torch._C._cuda_getDevice
_ROWS = {torch.bfloat16: ccb.CCB_KV8_BF16, torch.float16: ccb.CCB_KV8_FP16, torch.float32: ccb.CCB_KV8_FP32}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _int32(what: str, *numbers: int) -> None:
    """The library's integers have 32 bits: of a larger one it would get the low ones."""
    for n in numbers:
        if not -2 ** 31 <= n < 2 ** 31:
            raise ValueError(f"{what}: {n} is no number of 32 bits")


def _no_gradient(what: str) -> None:
    if torch.is_grad_enabled():
        raise ValueError(f"{what}: no gradient is computed here; detach it, or call under torch.no_grad()")


class OnDevice:
    """What the classes around the paged caches' calls share: tensors of one
    GPU whose addresses the kernels get (device, _index, err; a cache's batch
    and head_dim too), and calls that run there."""

    _what = "paged cache"

    def __setattr__(self, name: str, value) -> None:
        """The kernels get the addresses that the constructor saw: a tensor's
        contents may change (cache.lens += 1, cache.lens[...] = ...), the
        tensor may not."""
        if self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name}: change the tensor in place, or make another {type(self).__name__}")
        object.__setattr__(self, name, value)

    def _on_gpu(self) -> None:
        """Refuses tensors on the CPU, before anything else in every call: what
        follows compares devices with these tensors' only, and the kernels get
        raw addresses."""
        _need(self._index >= 0, f"the {self._what}'s tensors are not on a GPU")

    def _rows(self, t: torch.Tensor, heads: int, what: str):
        kind = _ROWS.get(t.dtype)
        if kind is not None and t.dim() == 4 and t.get_device() == self._index:
            batch, tokens, h, dim = t.shape
            sb, st, sh, sd = t.stride()
            if batch == self.batch and h == heads and dim == self.head_dim and (sd == 1 or t.numel() == 0):
                # the stride of a dimension with one place is never used
                return ccb.ccbKv8Rows(t.data_ptr(), sb if batch > 1 else 0, st if tokens > 1 else 0,
                                      sh if h > 1 else 0, kind, 0)
        raise ValueError(f"{what}: [batch {self.batch}, tokens, heads {heads}, head_dim {self.head_dim}] on "
                         f"{self.device}, bfloat16 or float16, the last dimension contiguous")

    def _ints(self, t: Optional[torch.Tensor], shape: tuple, what: str):
        if t is not None:
            _need(t.shape == shape and t.dtype == torch.int32 and t.is_contiguous()
                  and t.get_device() == self._index, f"{what}: {list(shape)} int32, contiguous")
        return t

    def _space(self, ws: Optional[torch.Tensor], need: int, s):
        """The caller's workspace, or a new one for this call."""
        if ws is None:
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            if s is not None:
                s.wait_stream(torch.cuda.current_stream(self.device))
                ws.record_stream(s)
        _need(ws.is_contiguous() and ws.get_device() == self._index, f"workspace: contiguous, on the {self._what}'s device")
        return ws, ws.nbytes

    def _enter(self, stream):
        """The caller's stream, ordered after torch's."""
        _need(not isinstance(stream, torch.cuda.Stream) or stream.device_index == self._index,
              f"stream: one of the {self._what}'s device")
        return _enter(stream, self.device)

    def _call(self, fn, s, *args) -> None:
        """An entry point with the tensors' device current, on `s` or torch's
        stream there; raises its error and orders torch's stream after `s`."""
        stream = s or _current_stream(self._index)
        if _current_device() == self._index:
            status = fn(*args, stream)
        else:
            with torch.cuda.device(self._index):
                status = fn(*args, stream)
        if status != ccb.CCB_OK:
            raise ccb.CcbError(status, fn.__name__)
        if s is not None:
            _leave(s, self.device)

    def check(self) -> None:
        """Raise if one of this object's calls met bad numbers (pages, lengths,
        counts) since the last check.  Waits for the device."""
        status = int(self.err.item())
        self.err.zero_()
        ccb.check(status, self._what)


class Kv8Cache(OnDevice):
    """A cache in the caller's tensors (they are kept, not copied, and stay
    the same tensors with the same storage for the cache's life):
    k, v [pages, heads, page_size, head_dim] (int8 or float8_e4m3fn); k_scale,
    v_scale [pages, heads] float32; page_table [batch, max_pages] int32; lens
    [batch] int32; weight [batch, heads, at least max_pages * page_size]
    float32 or None.  All contiguous, but for the page table's rows, and on one
    GPU: a cache on the CPU can be made, but every call on it is refused."""

    _what = "8-bit cache"

    def __init__(self, k, v, k_scale, v_scale, page_table, lens, weight=None):
        _need(k.dim() == 4 and k.dtype in _CODES, "k: [pages, heads, page_size, head_dim], int8 or float8_e4m3fn")
        pages, heads, page_size, head_dim = k.shape
        _need(v.shape == k.shape and v.dtype == k.dtype, "v: shape and dtype of k")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(tuple(s.shape) == (pages, heads) and s.dtype == torch.float32, f"{name}: [pages, heads] float32")
        _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.shape[1] >= 1 and
              page_table.stride(1) == 1, "page_table: [batch, max_pages] int32")
        batch, max_pages = page_table.shape
        _need(tuple(lens.shape) == (batch,) and lens.dtype == torch.int32, "lens: [batch] int32")
        if weight is not None:
            _need(weight.dim() == 3 and tuple(weight.shape[:2]) == (batch, heads) and weight.dtype == torch.float32
                  and weight.shape[2] >= max_pages * page_size,
                  "weight: [batch, heads, max_pages * page_size or more] float32")
        for t in (k, v, k_scale, v_scale, lens) + (() if weight is None else (weight,)):
            _need(t.is_contiguous(), "cache tensors are contiguous")
        for t in (v, k_scale, v_scale, page_table, lens) + (() if weight is None else (weight,)):
            _need(t.device == k.device, "cache tensors share a device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table, self.lens, self.weight = page_table, lens, weight
        self.heads, self.head_dim, self.batch, self.device = heads, head_dim, batch, k.device
        self._index = k.get_device()  # -1 on the CPU
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._c = ccb.ccbKv8Cache(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
            lens.data_ptr(), 0 if weight is None else weight.data_ptr(),
            page_table.stride(0) if batch > 1 else max_pages, 0 if weight is None else weight.shape[2],
            _CODES[k.dtype], pages, heads, page_size, head_dim, batch, max_pages, 0)

    @classmethod
    def allocate(cls, pages: int, heads: int, page_size: int, head_dim: int, batch: int, max_pages: int,
                 fmt: str = "e4m3", weights: bool = False, device="cuda") -> "Kv8Cache":
        """Zeroed tensors: no sequence holds a token, every page number is 0."""
        _need(fmt in _FORMATS, "fmt: int8 or e4m3")
        shape = (pages, heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.int8, device=device).view(_FORMATS[fmt]) for _ in range(2))
        ks, vs = (torch.zeros((pages, heads), dtype=torch.float32, device=device) for _ in range(2))
        table = torch.zeros((batch, max_pages), dtype=torch.int32, device=device)
        lens = torch.zeros(batch, dtype=torch.int32, device=device)
        weight = torch.zeros((batch, heads, max_pages * page_size), dtype=torch.float32, device=device) \
            if weights else None
        return cls(k, v, ks, vs, table, lens, weight)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, counts: Optional[torch.Tensor] = None,
               stream=None) -> None:
        """Write each sequence's counts[b] (None: all) new tokens as its last
        ones; lens counts them already.  k_new, v_new [batch, n, heads, head_dim]."""
        if self._index < 0:
            self._on_gpu()
        k, v = self._rows(k_new, self.heads, "k_new"), self._rows(v_new, self.heads, "v_new")
        if k_new.requires_grad or v_new.requires_grad:
            _no_gradient("k_new, v_new")
        n = k_new.shape[1]
        if n >> 31:
            _int32("tokens", n)
        _need(n == v_new.shape[1] and k.type == v.type, "v_new: shape and dtype of k_new")
        self._ints(counts, (self.batch,), "counts")
        s = None if stream is None else self._enter(stream)
        self._call(ccb.ccb_kv8_append, s, self._c, k, v, n, counts, self.err)

    def attend_workspace(self, q_heads: int, queries: int = 1, accumulate: bool = False) -> torch.Tensor:
        """A workspace for attend() calls of these sizes that follow each other.
        With weights it grows with the capacity: 4 bytes for each of the rows
        of a cache head and each token there is room for."""
        if self._index < 0:
            self._on_gpu()
        _int32("attend", q_heads, queries)
        n = ccb.ccb_kv8_attend_workspace_bytes(self._c, q_heads, queries, int(accumulate))
        _need(n > 0, "attend: sizes that ccb_kv8_attend refuses")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attend(self, q: torch.Tensor, scale: Optional[float] = None, window: int = 0, accumulate: bool = False,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None):
        """Attention of q [batch, queries, q_heads, head_dim], the sequences'
        last tokens; scale None is 1 / sqrt(head_dim).  Returns (out, lse).
        out may be q itself, but for weights accumulated over many rows (more
        than 64 a cache head, or 16 in a large cache; refused)."""
        if self._index < 0:
            self._on_gpu()
        _need(q.dim() == 4, "q: [batch, queries, q_heads, head_dim]")
        if q.requires_grad:
            _no_gradient("q")
        if window >> 31:
            _int32("window", window)
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
        _need(out.shape[1] == queries and outr.type == qr.type, "out: shape and dtype of q")
        _need(lse.shape == shape[:3] and lse.dtype == torch.float32 and lse.is_contiguous()
              and lse.get_device() == self._index, "lse: [batch, queries, q_heads] float32, contiguous")
        need = 0 if workspace is not None else \
            ccb.ccb_kv8_attend_workspace_bytes(self._c, q_heads, queries, int(accumulate))
        ws, size = self._space(workspace, need, s)
        self._call(ccb.ccb_kv8_attend, s, self._c, qr, outr, lse, q_heads, queries,
                   self.head_dim ** -0.5 if scale is None else scale, window, int(accumulate), ws, size, self.err)
        return out, lse

    def evict_workspace(self, budget: int) -> torch.Tensor:
        """A workspace for evict() calls with this budget that follow each other."""
        if self._index < 0:
            self._on_gpu()
        _int32("budget", budget)
        n = ccb.ccb_kv8_evict_workspace_bytes(self._c, budget)
        _need(n > 0, "evict: sizes that ccb_kv8_evict refuses")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def evict(self, to: "Kv8Cache", budget: int, recent: int = 0, sinks: int = 0,
              kept: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> Optional[torch.Tensor]:
        """Copy the budget tokens of each sequence and head with the largest
        weight (and its first `sinks` and last `recent`) into the cache `to`.
        kept [batch, heads, budget] int32, where given, gets their numbers; it
        is returned.  Bad pages of either cache are reported by this one's
        check()."""
        if self._index < 0:
            self._on_gpu()
        _need(to._index == self._index, "to: on the cache's device")
        _int32("budget, recent, sinks", budget, recent, sinks)
        self._ints(kept, (self.batch, self.heads, budget), "kept")
        s = None if stream is None else self._enter(stream)
        need = 0 if workspace is not None else ccb.ccb_kv8_evict_workspace_bytes(self._c, budget)
        ws, size = self._space(workspace, need, s)
        self._call(ccb.ccb_kv8_evict, s, self._c, to._c, budget, recent, sinks, kept, ws, size, self.err)
        return kept

    def read(self, count: int, first: Optional[torch.Tensor] = None, dtype=torch.float32, stream=None):
        """The values of `count` tokens of each sequence from first[b] (None: 0)
        as (k, v) [batch, count, heads, head_dim]; zeros where there is none."""
        if self._index < 0:
            self._on_gpu()
        kind = _ROWS.get(dtype)
        _need(kind is not None, "dtype: float32, bfloat16 or float16")
        self._ints(first, (self.batch,), "first")
        _int32("count", count)
        s = None if stream is None else self._enter(stream)
        both = torch.empty((2, self.batch, count, self.heads, self.head_dim), dtype=dtype, device=self.device)
        if s is not None:
            both.record_stream(s)
        k, v = both.unbind(0)
        row = self.heads * self.head_dim
        self._call(ccb.ccb_kv8_read, s, self._c, ccb.ccbKv8Rows(k.data_ptr(), count * row, row, self.head_dim, kind, 0),
                   ccb.ccbKv8Rows(v.data_ptr(), count * row, row, self.head_dim, kind, 0), count, first, self.err)
        return k, v
