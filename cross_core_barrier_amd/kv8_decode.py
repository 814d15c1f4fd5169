"""A decoding session on the 8-bit key/value cache, one attention layer deep:

    python -m cross_core_barrier_amd.kv8_decode --batch 16 --steps 500

Prompts are written on a stream of their own; a CntNotify counter tells the
decoding stream when all of them are there.  A step then appends one token for
every sequence, attends and keeps the attention weights; the step is captured
into a HIP graph once and replayed.  When a sequence is about to pass its limit
the cache is cut to the tokens that drew the most weight, into fresh pages, and
the old pages go back to the pool.  The layer's weights are random; PyTorch does
the projections.
"""

from __future__ import annotations

import argparse
import time

import torch

from . import ccb
from .kv8 import Kv8Cache


class Pages:
    """The numbers of a pool's free pages."""

    def __init__(self, n: int):
        self.free = list(range(n))

    def take(self, n: int) -> list:
        assert n <= len(self.free), "the pool is empty"
        taken, self.free = self.free[:n], self.free[n:]
        return taken

    def give(self, pages: list) -> None:
        self.free += pages


class Session:
    def __init__(self, batch=4, heads=8, q_heads=32, head_dim=128, page_size=64, limit=2048, budget=512, fmt="e4m3",
                 dtype=torch.bfloat16, seed=0):
        if not 1 <= budget < limit:  # a cut has to leave room for the next token
            raise ValueError(f"budget {budget}: at least 1, and less than the limit of {limit} tokens")
        dev = torch.device("cuda")
        self.batch, self.heads, self.q_heads, self.head_dim = batch, heads, q_heads, head_dim
        self.limit, self.budget = limit, budget
        width = -(-limit // page_size)
        self.out_width = -(-budget // page_size)
        # every sequence at its limit, and one cut of the whole batch besides
        self.pages = Pages(batch * (width + self.out_width))
        self.cache = Kv8Cache.allocate(len(self.pages.free), heads, page_size, head_dim, batch, width, fmt,
                                       weights=True)
        # the cut's own table, lengths and weights, over the same pool
        self.cut = Kv8Cache(self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale,
                            torch.zeros((batch, self.out_width), dtype=torch.int32, device=dev),
                            torch.zeros(batch, dtype=torch.int32, device=dev),
                            torch.zeros((batch, heads, self.out_width * page_size), device=dev))
        self.held = [[] for _ in range(batch)]  # pages of each sequence, on the host
        self.lens = [0] * batch
        gen = torch.Generator(device=dev).manual_seed(seed)
        d = q_heads * head_dim
        n = (q_heads + 2 * heads) * head_dim
        self.w_qkv = (torch.randn((d, n), generator=gen, device=dev) / d ** 0.5).to(dtype)
        self.w_out = (torch.randn((d, d), generator=gen, device=dev) / d ** 0.5).to(dtype)
        self.x = torch.zeros((batch, d), dtype=dtype, device=dev)  # a step's input and output
        self.attend_ws = self.cache.attend_workspace(q_heads, 1, accumulate=True)
        self.evict_ws = self.cache.evict_workspace(budget)
        self.graph = None
        self.evictions = 0

    def _reserve(self, lens: list) -> None:
        """Pages for sequences that grow to `lens`."""
        page = self.cache.k.shape[2]
        for b, n in enumerate(lens):
            more = -(-n // page) - len(self.held[b])
            if more > 0:
                first = len(self.held[b])
                self.held[b] += self.pages.take(more)
                self.cache.page_table[b, first:first + more] = torch.tensor(self.held[b][first:], dtype=torch.int32)
        self.lens = list(lens)

    def project(self, x: torch.Tensor):
        """x [batch, tokens, d] as queries, keys and values [batch, tokens, heads, head_dim]."""
        qkv = (x @ self.w_qkv).unflatten(-1, (-1, self.head_dim))
        return qkv.split([self.q_heads, self.heads, self.heads], dim=2)

    def prefill(self, prompts: list) -> None:
        """Write prompts [tokens, d], one for each sequence."""
        lens = [p.shape[0] for p in prompts]
        if len(lens) != self.batch or not all(1 <= n <= self.limit for n in lens):
            raise ValueError(f"prompts: {self.batch} of 1 to {self.limit} tokens each")
        self._reserve(lens)
        rows = torch.nn.utils.rnn.pad_sequence(prompts, batch_first=True)
        counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
        status, done = ccb.ccb_cnt_notify_create()
        ccb.check(status, "ccb_cnt_notify_create")
        writer, here = torch.cuda.Stream(), torch.cuda.current_stream()
        writer.wait_stream(here)
        with torch.cuda.stream(writer):
            self.cache.lens.copy_(counts)
            _, k, v = self.project(rows)
            self.cache.append(k, v, counts)
            ccb.check(ccb.ccb_cnt_notify_record(done, writer, ccb.record_info(ccb.CCB_CNT_RECORD_ADD, 1)), "record")
        there = ccb.wait_info(ccb.CCB_CNT_WAIT_BIGGER_OR_EQUAL, 1, 10, 1)
        ccb.check(ccb.ccb_cnt_notify_wait(done, here, there), "wait")
        here.wait_stream(writer)  # the prompt's tensors are torch's to reuse after this
        here.synchronize()
        ccb.check(ccb.ccb_cnt_notify_destroy(done), "ccb_cnt_notify_destroy")
        for b, p in enumerate(prompts):
            self.x[b] = p[-1]

    def _step(self) -> None:
        q, k, v = self.project(self.x[:, None])
        self.cache.lens.add_(1)
        self.cache.append(k, v)
        out, _ = self.cache.attend(q, accumulate=True, workspace=self.attend_ws)
        y = out.flatten(1) @ self.w_out
        self.x.copy_(y / (y.float().square().mean(-1, keepdim=True) + 1e-6).sqrt().to(y.dtype))

    def _evict(self) -> None:
        """Cut every sequence to the budget, into pages of its own."""
        page = self.cache.k.shape[2]
        stay = [min(n, self.budget) for n in self.lens]
        fresh = [self.pages.take(-(-n // page)) for n in stay]
        for b, pages in enumerate(fresh):
            self.cut.page_table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
        self.cache.evict(self.cut, self.budget, recent=self.budget // 4, sinks=min(4, self.budget // 4),
                         workspace=self.evict_ws)
        self.cache.page_table[:, :self.out_width].copy_(self.cut.page_table)
        self.cache.lens.copy_(self.cut.lens)
        self.cache.weight[:, :, :self.cut.weight.shape[2]].copy_(self.cut.weight)
        for pages in self.held:
            self.pages.give(pages)
        self.held, self.lens = fresh, stay
        self.evictions += 1

    def step(self, graph: bool = True) -> torch.Tensor:
        """One token more for every sequence; returns the layer's output."""
        if max(self.lens) + 1 > self.limit:
            self._evict()
        self._reserve([n + 1 for n in self.lens])
        if not graph:
            self._step()
        else:
            if self.graph is None:
                self._capture()
            self.graph.replay()
        return self.x

    def _capture(self) -> None:
        """Capture the step.  The run outside the capture that this needs is
        made on no tokens: lengths of -1 become 0 and nothing is written."""
        x, lens = self.x.clone(), self.cache.lens.clone()
        self.cache.lens.fill_(-1)
        counts = torch.zeros(self.batch, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q, k, v = self.project(self.x[:, None])
            self.cache.lens.add_(1)
            self.cache.append(k, v, counts)
            self.cache.attend(q, accumulate=True, workspace=self.attend_ws)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(self.graph):
            self._step()
        self.x.copy_(x)
        self.cache.lens.copy_(lens)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--steps", type=int, default=500)
    ap.add_argument("--prompt", type=int, default=1800)
    ap.add_argument("--limit", type=int, default=2048)
    ap.add_argument("--budget", type=int, default=512)
    ap.add_argument("--format", choices=["int8", "e4m3"], default="e4m3")
    ap.add_argument("--eager", action="store_true", help="no HIP graph")
    a = ap.parse_args(argv)
    s = Session(batch=a.batch, limit=a.limit, budget=a.budget, fmt=a.format)
    d = s.x.shape[1]
    # prompts of unlike lengths
    lens = [max(1, a.prompt - 37 * b) for b in range(a.batch)]
    s.prefill([torch.randn((n, d), device="cuda", dtype=s.x.dtype) for n in lens])
    s.step(not a.eager)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps - 1):
        s.step(not a.eager)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    s.cache.check()
    s.cut.check()
    print(f"{a.batch} sequences, {a.steps} steps, {s.evictions} evictions: "
          f"{t / max(1, a.steps - 1) * 1e6:.1f} us a step, {a.batch * (a.steps - 1) / t:.0f} tokens/s; lengths now {min(s.lens)} to {max(s.lens)}")


if __name__ == "__main__":
    main()
