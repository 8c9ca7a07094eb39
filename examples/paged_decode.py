"""Attention blocks of a small decoder over a paged cache, all on the library:
4-bit projections (qmm_gemm), rotary positions with the append
(qmm_rope_append), attention (qmm_paged_attention) and the pages' bookkeeping
(qmm_pages_*).

A prompt is prefilled in chunks, its sequence forked into samples that share
the prompt's full pages, and the samples decode a token each per step, one HIP
graph a step; at the end dropped samples give their pages back and the cache is
closed up.  Run:  python examples/paged_decode.py
"""
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from block_quantized_weight_matmulnbits_amd import qmm  # noqa: E402
from block_quantized_weight_matmulnbits_amd.workloads import make_matmul_case  # noqa: E402

BLOCK, BITS = 128, 4


class Projection:
    """A 4-bit weight [N, K], repacked once."""

    def __init__(self, K, N, seed, dev):
        c = make_matmul_case(1, K, N, BLOCK, BITS, a_dtype="bf16", has_zp=True, seed=seed).to(dev)
        self.K, self.N = K, N
        self.B = qmm.qmm_repack(c.B, c.scales, c.zero_points, K, N, BLOCK, BITS)

    def add_to(self, step, x, y):
        step.add_gemm(x, self.B, None, None, None, y, x.shape[0], self.K, self.N, BLOCK, BITS)

    def __call__(self, x, y):
        qmm.qmm_gemm(x, self.B, None, None, None, y, x.shape[0], self.K, self.N, BLOCK, BITS)


class Decoder:
    """``layers`` attention blocks y = o_proj(attention(rope(qkv_proj(x)))), each
    feeding the next, and the cache that they share the bookkeeping of."""

    def __init__(self, hidden=1024, q_heads=8, kv_heads=2, dim=128, layers=2, slots=8, pages=256,
                 page_size=16, max_len=1024, dev="cuda"):
        self.q_heads, self.kv_heads, self.dim, self.layers = q_heads, kv_heads, dim, layers
        self.hidden, self.slots, self.max_len, self.dev = hidden, slots, max_len, dev
        heads = q_heads + 2 * kv_heads
        self.qkv = [Projection(hidden, heads * dim, 10 + i, dev) for i in range(layers)]
        self.o = [Projection(q_heads * dim, hidden, 50 + i, dev) for i in range(layers)]
        data = torch.zeros(2 * layers, pages, kv_heads, page_size, dim, dtype=torch.bfloat16, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.pool = qmm.PagePool(data, torch.zeros(pages, **i32),
                                 torch.full((slots, -(-max_len // page_size)), -1, **i32),
                                 torch.zeros(slots, **i32), page_size)
        self.kv = [qmm.PagedKV(data[2 * i], data[2 * i + 1]) for i in range(layers)]
        self.inv_freq = 500000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=dev) / dim)
        self.status = torch.zeros(2, **i32)
        self.pages_ws = torch.empty(qmm.qmm_pages_workspace_size(self.pool, slots), dtype=torch.uint8,
                                    device=dev)

    def list(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.dev)

    def batch(self, counts, max_new):
        """The new tokens of every slot (counts, 0 for most) as a batch over the
        pool's own lengths and table, and the buffers that a pass needs."""
        tokens = sum(counts)
        starts = torch.zeros(self.slots + 1, dtype=torch.int32)
        starts[1:] = torch.tensor(counts).cumsum(0)
        b = qmm.PagedBatch(starts.to(self.dev), self.pool.lens, self.pool.table, tokens, max_new,
                           self.max_len)
        def empty(*shape):
            return torch.empty(*shape, dtype=torch.bfloat16, device=self.dev)
        heads = self.q_heads + 2 * self.kv_heads
        b.x = [empty(tokens, self.hidden) for _ in range(self.layers + 1)]
        b.rows = empty(tokens, heads, self.dim)
        b.attended = empty(tokens, self.q_heads, self.dim)
        b.workspace = torch.empty(qmm.qmm_paged_attention_workspace_size(
            b, self.q_heads, self.kv_heads, self.dim), dtype=torch.uint8, device=self.dev)
        return b

    def heads_of(self, b):
        h, k = self.q_heads, self.kv_heads
        return b.rows[:, :h], b.rows[:, h:h + k], b.rows[:, h + k:]

    def forward(self, b):
        """b.x[0] to b.x[-1]; the pages of the new tokens are already reserved."""
        q, k, v = self.heads_of(b)
        for i in range(self.layers):
            self.qkv[i](b.x[i], b.rows.view(len(b.rows), -1))
            qmm.qmm_rope_append(q, k, v, q, self.kv[i], b, self.inv_freq)
            qmm.qmm_paged_attention(q, self.kv[i], b, b.attended, b.workspace)
            self.o[i](b.attended.view(len(b.rows), -1), b.x[i + 1])
        return b.x[-1]

    def prefill(self, slot, x, chunk):
        """The hidden states x [tokens, hidden] of a prompt, ``chunk`` at a time."""
        outs = []
        for at in range(0, len(x), chunk):
            n = min(chunk, len(x) - at)
            counts = [0] * self.slots
            counts[slot] = n
            qmm.qmm_pages_reserve(self.pool, self.list([slot]), self.list([n]), self.status, self.pages_ws)
            b = self.batch(counts, n)
            b.x[0].copy_(x[at:at + n])
            outs.append(self.forward(b).clone())
        return torch.cat(outs)

    def fork(self, parent, children):
        qmm.qmm_pages_fork(self.pool, self.list([parent] * len(children)), self.list(children),
                           self.status, self.pages_ws)

    def free(self, slots):
        qmm.qmm_pages_free(self.pool, self.list(slots))

    def decode_step(self, slots):
        """One token for each of ``slots``, recorded: (step, batch).  Put the
        tokens' hidden states into batch.x[0], launch, read batch.x[-1]."""
        b = self.batch([int(s in slots) for s in range(self.slots)], 1)
        q, k, v = self.heads_of(b)
        step = qmm.Step()
        step.add_pages_reserve(self.pool, self.list(slots), self.list([1] * len(slots)), self.status,
                               self.pages_ws)
        for i in range(self.layers):
            self.qkv[i].add_to(step, b.x[i], b.rows.view(len(b.rows), -1))
            step.add_rope_append(q, k, v, q, self.kv[i], b, self.inv_freq)
            step.add_paged_attention(q, self.kv[i], b, b.attended, b.workspace)
            self.o[i].add_to(step, b.attended.view(len(b.rows), -1), b.x[i + 1])
        return step.finalize(), b

    def compact(self):
        """Closes the cache up; the number of pages in use."""
        p = self.pool
        refs, table = torch.empty_like(p.refs), torch.empty_like(p.table)
        live = torch.zeros(1, dtype=torch.int32, device=self.dev)
        qmm.qmm_pages_compact(p, refs, table, live, self.pages_ws)
        p.refs.copy_(refs)
        p.table.copy_(table)
        return int(live)


def main(prompt=700, samples=6, steps=64):
    d = Decoder()
    g = torch.Generator(device=d.dev).manual_seed(1)
    x = torch.randn(prompt, d.hidden, device=d.dev, generator=g).bfloat16()
    last = d.prefill(0, x, 256)[-1]
    slots = list(range(1, 1 + samples))
    d.fork(0, slots)
    step, b = d.decode_step(slots)
    b.x[0].copy_(last.expand(samples, -1))
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(steps):
        step.launch()
        b.x[0].copy_(b.x[-1])   # a stand-in for sampling and embedding
    torch.cuda.synchronize()
    took = (time.perf_counter() - began) / steps
    used = int((d.pool.refs > 0).sum())
    d.free([0] + slots[1:])
    kept = d.compact()
    print(f"{samples} samples of a {prompt}-token prompt, {d.layers} blocks: {took * 1e6:.0f} us a step; "
          f"{used} pages in use, {kept} after all but one sample were dropped; status {d.status.tolist()}")


if __name__ == "__main__":
    main()
