"""A small decoder from token to token, all on the library: RMS norms that add the
residual stream and write int8 codes (qmm_rms_norm), the projections that read
them (qmm_gemm_compint8_quantized), attention over a paged cache, experts behind a
router (qmm_moe) and sampling (qmm_sample).

A prompt is prefilled and forked into samples; each step of the samples is one
HIP graph, after which the tokens that it drew are embedded for the next one.
Run:  python examples/sampled_decode.py
"""
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for p in (ROOT, os.path.join(ROOT, "examples")):
    if p not in sys.path:
        sys.path.insert(0, p)

import paged_decode  # noqa: E402
from block_quantized_weight_matmulnbits_amd import qmm  # noqa: E402
from block_quantized_weight_matmulnbits_amd.workloads import make_matmul_case  # noqa: E402

BLOCK, BITS = 32, 4


class Int8Projection(paged_decode.Projection):
    """A 4-bit weight [N, K] that reads int8 codes of its inputs."""

    def __init__(self, K, N, seed, dev):
        c = make_matmul_case(1, K, N, BLOCK, BITS, a_dtype="bf16", has_zp=True, seed=seed).to(dev)
        self.K, self.N = K, N
        self.B = qmm.qmm_repack(c.B, c.scales, c.zero_points, K, N, BLOCK, BITS)

    def args(self, codes, scales, y):
        return codes, scales, self.B, None, None, None, y, len(codes), self.K, self.N, BLOCK, BITS


def experts(count, hidden, inter, seed, dev):
    """Random experts of a layer, in the operator's layout."""
    parts = []
    for i, (K, N) in enumerate(((hidden, 2 * inter), (inter, hidden))):
        cs = [make_matmul_case(1, K, N, BLOCK, BITS, a_dtype="bf16", has_zp=True, seed=seed + 2 * e + i) for e in range(count)]
        for t in ("B", "scales", "zero_points"):
            parts.append(torch.stack([getattr(c, t).view(N, -1, BLOCK * BITS // 8) if t == "B" else getattr(c, t).view(N, -1)
                                      for c in cs]).to(dev))
    return qmm.MoeWeights(*parts, hidden, inter, BLOCK, BITS)


class Decoder(paged_decode.Decoder):
    """``layers`` layers of attention and experts, each behind a norm, on a
    residual stream; then a norm, the vocabulary's logits and a token a row."""

    def __init__(self, vocab=8192, count=8, top_k=2, inter=512, **kw):
        super().__init__(**kw)
        heads, L, dev = self.q_heads + 2 * self.kv_heads, self.layers, self.dev
        self.vocab, self.count, self.top_k = vocab, count, top_k
        self.qkv = [Int8Projection(self.hidden, heads * self.dim, 10 + i, dev) for i in range(L)]
        self.router = [paged_decode.Projection(self.hidden, count, 70 + i, dev) for i in range(L)]
        self.experts = [experts(count, self.hidden, inter, 100 + 1000 * i, dev) for i in range(L)]
        self.head = paged_decode.Projection(self.hidden, vocab, 90, dev)
        g = torch.Generator(device=dev).manual_seed(2)
        self.embedding = torch.randn(vocab, self.hidden, generator=g, device=dev).bfloat16()
        self.weights = [(1 + 0.1 * torch.randn(self.hidden, generator=g, device=dev)).bfloat16() for _ in range(2 * L + 1)]

    def batch(self, counts, max_new):
        b = super().batch(counts, max_new)
        T, dev = b.x[0].shape[0], self.dev

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=dev)
        kb = -(-self.hidden // BLOCK)
        b.stream, b.codes, b.scales = empty(T, self.hidden), empty(T, kb * BLOCK, dtype=torch.int8), empty(T, kb, dtype=torch.float32)
        b.normed, b.routed, b.added = empty(T, self.hidden), empty(T, self.count), empty(T, self.hidden)
        b.logits, b.uniform = empty(T, self.vocab), torch.zeros(T, device=dev)
        b.drawn, b.logprobs = empty(T, dtype=torch.int32), empty(T, dtype=torch.float32)
        b.temperature, b.top_p = torch.full((T,), 0.8, device=dev), torch.full((T,), 0.95, device=dev)
        b.moe_ws = empty(qmm.qmm_moe_workspace_size(self.experts[0], T, self.top_k), dtype=torch.uint8)
        b.sample_ws = empty(qmm.qmm_sample_workspace_size(T, self.vocab), dtype=torch.uint8)
        return b

    def calls(self, b):
        """The pass over b.x[0] (embedded tokens) as (name, arguments, options)."""
        q, k, v = self.heads_of(b)
        T = len(b.rows)

        def gemm(p, x, y):
            return "gemm", (x, p.B, None, None, None, y, T, p.K, p.N, paged_decode.BLOCK, paged_decode.BITS), {}
        # h: the residual stream so far; the norms after the first add to it what
        # the layer before them put out.
        h, add = b.x[0], None
        for i in range(self.layers):
            yield "rms_norm", (h, self.weights[2 * i]), dict(residual=add, h=b.stream, codes=b.codes, scales=b.scales, block_size=BLOCK)
            yield "gemm_compint8_quantized", self.qkv[i].args(b.codes, b.scales, b.rows.view(T, -1)), {}
            yield "rope_append", (q, k, v, q, self.kv[i], b, self.inv_freq), {}
            yield "paged_attention", (q, self.kv[i], b, b.attended, b.workspace), {}
            yield gemm(self.o[i], b.attended.view(T, -1), b.added)
            yield "rms_norm", (b.added, self.weights[2 * i + 1]), dict(residual=b.stream, h=b.stream, y=b.normed)
            yield gemm(self.router[i], b.normed, b.routed)
            yield "moe", (b.normed, self.experts[i], b.added, b.moe_ws), dict(logits=b.routed, top_k=self.top_k)
            h, add = b.added, b.stream
        yield "rms_norm", (h, self.weights[-1]), dict(residual=add, y=b.normed)
        yield gemm(self.head, b.normed, b.logits)
        yield "sample", (b.logits, b.uniform, b.drawn, b.sample_ws), dict(
            temperature=b.temperature, top_p=b.top_p, logprobs=b.logprobs)

    def forward(self, b):
        for name, args, kw in self.calls(b):
            getattr(qmm, "qmm_" + name)(*args, **kw)
        return b.drawn

    def embed(self, tokens):
        return self.embedding[tokens.long()]

    def prefill(self, slot, tokens, chunk):
        """The token drawn after every token of a prompt."""
        return super().prefill(slot, self.embed(tokens), chunk)

    def decode_step(self, slots):
        """One token for each of ``slots``, recorded: (step, batch).  Put embedded
        tokens into batch.x[0] and uniforms into batch.uniform, launch, read
        batch.drawn."""
        b = self.batch([int(s in slots) for s in range(self.slots)], 1)
        step = qmm.Step()
        step.add_pages_reserve(self.pool, self.list(slots), self.list([1] * len(slots)), self.status, self.pages_ws)
        for name, args, kw in self.calls(b):
            getattr(step, "add_" + name)(*args, **kw)
        return step.finalize(), b


def main(prompt=200, samples=6, steps=64):
    d = Decoder()
    g = torch.Generator(device=d.dev).manual_seed(1)
    last = d.prefill(0, torch.randint(0, d.vocab, (prompt,), device=d.dev, generator=g), 128)[-1]
    slots = list(range(1, 1 + samples))
    d.fork(0, slots)
    step, b = d.decode_step(slots)
    b.x[0].copy_(d.embed(last.expand(samples)))
    torch.cuda.synchronize()
    began = time.perf_counter()
    drawn = []
    for _ in range(steps):
        b.uniform.uniform_(generator=g)
        step.launch()
        b.x[0].copy_(d.embed(b.drawn))
        drawn.append(b.drawn.clone())
    torch.cuda.synchronize()
    took = (time.perf_counter() - began) / steps
    drawn = torch.stack(drawn)
    print(f"{samples} samples of a {prompt}-token prompt, {d.layers} layers: {took * 1e6:.0f} us a step; "
          f"{len(drawn.unique())} different tokens of {drawn.numel()}; status {d.status.tolist()}")


if __name__ == "__main__":
    main()
