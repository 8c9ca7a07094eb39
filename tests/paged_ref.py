"""The paged-cache operators from their definitions, in 64 bits on the host:
what the GPU tests compare with, and how far rounding may take a result from it."""
from __future__ import annotations

import math

import numpy as np
import torch

# Half a step of each type, relative, and half its smallest subnormal.
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
HALF_TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
F32 = 2.0 ** -24


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make_batch(counts, lens, page, seed=0, extra_pages=2, extra_cols=1):
    """(starts, lens, table, pages) with the pages of the pool in random order."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int64)
    per = -(-lens // page)
    total = int(per.sum()) + extra_pages
    order = rng.permutation(total)
    table = np.full((len(lens), int(per.max(initial=0)) + extra_cols), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(per):
        table[s, :n] = order[at:at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return starts, lens.astype(np.int32), table, total


def rope(q, k, v, k_pages, v_pages, starts, lens, table, inv_freq, interleaved=False, factor=1.0,
         positions=None):
    """(out, k_pages, v_pages, bound of out, bound of k_pages), all float64."""
    q, k, v, kp, vp = (f64(t).copy() for t in (q, k, v, k_pages, v_pages))
    half, page = len(inv_freq), kp.shape[2]
    kb = np.zeros_like(kp)
    out, ob = q.copy(), np.zeros_like(q)
    one = 2 * np.arange(half) if interleaved else np.arange(half)
    two = one + 1 if interleaved else one + half
    for s in range(len(lens)):
        for t in range(starts[s], starts[s + 1]):
            slot = int(lens[s]) - int(starts[s + 1]) + t
            pos = slot if positions is None else int(positions[t])
            angle = np.float64(pos) * inv_freq
            c, si = np.cos(angle) * factor, np.sin(angle) * factor

            def turned(x):
                y, b = x.copy(), np.zeros_like(x)
                a, d = x[:, one], x[:, two]
                y[:, one], y[:, two] = a * c - d * si, d * c + a * si
                # Sine and cosine rounded, two products, their sum: half a
                # step of 32 bits each; and the angle's own 64-bit rounding.
                turn = np.abs(angle) * 2.0 ** -52 * factor
                b[:, one] = (np.abs(a * c) + np.abs(d * si)) * 4 * F32 + (np.abs(a) + np.abs(d)) * turn
                b[:, two] = (np.abs(d * c) + np.abs(a * si)) * 4 * F32 + (np.abs(a) + np.abs(d)) * turn
                return y, b

            out[t], ob[t] = turned(q[t])
            if 0 <= slot < table.shape[1] * page and 0 <= table[s, slot // page] < kp.shape[0]:
                p, at = table[s, slot // page], slot % page
                kp[p, :, at], kb[p, :, at] = turned(k[t])
                vp[p, :, at] = v[t]
    return out, kp, vp, ob, kb


def rounded(y, bound, dtype):
    """The bound of a value rounded once to dtype."""
    return bound + HALF_STEP[dtype] * (np.abs(y) + bound) + HALF_TINY[dtype]


def attention(q, k_pages, v_pages, starts, lens, table, scale, causal=True, window=0, cap=0.0):
    """(out, lse, bound of out, bound of lse) in float64.  A key that is not seen
    takes no part at all, so that what it holds does not matter."""
    dtype = q.dtype
    q, kp, vp = f64(q), f64(k_pages), f64(v_pages)
    T, H, D = q.shape
    KV, page = kp.shape[1], kp.shape[2]
    G = H // KV
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    ob, lb = np.zeros((T, H, D)), np.zeros((T, H))
    for s in range(len(lens)):
        n, length = int(starts[s + 1] - starts[s]), int(lens[s])
        j = np.arange(length)
        ids, at = table[s, j // page], j % page
        for i in range(n):
            t, pos = int(starts[s]) + i, length - n + i
            see = np.ones(length, bool)
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            if not see.any():
                continue
            for h in range(H):
                kk, vv = kp[ids[see], h // G, at[see]], vp[ids[see], h // G, at[see]]
                z = kk @ q[t, h] * scale
                # A dot product of D terms in 32 bits, scaled.
                off = (np.abs(kk) @ np.abs(q[t, h])) * abs(scale) * (D + 8) * F32
                if cap:
                    z = cap * np.tanh(z / cap)
                    off = off + cap * 16 * F32
                with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                    m = z.max()
                    e = np.exp(z - (m if m != -np.inf else 0.0))
                    total = e.sum()
                    p = e / total if total else e
                    out[t, h] = p @ vv
                    lse[t, h] = m + np.log(total) if total else -np.inf
                    # Twice the scores' error (numerator and sum), the sums
                    # over the keys, exp's own steps and its argument's.
                    far = 2 * off.max() + (len(z) + 32) * F32 + 4 * np.abs(z).max() * F32
                    mass = p @ np.abs(vv)
                    # 16-bit probabilities: half a step each, or half the
                    # smallest subnormal (the largest is 1, so the sum >= 1).
                    u = 0.0 if dtype == torch.float32 else HALF_STEP[dtype]
                    tiny = 0.0 if dtype == torch.float32 else HALF_TINY[dtype] * np.abs(vv).sum(0)
                    ob[t, h] = mass * (far + u) * 1.01 + tiny
                    lb[t, h] = far + 8 * F32 * abs(lse[t, h])
    return out, lse, ob, lb


def assert_close(got, want, bound, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= bound))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.size} outside; first at {i}: got "
                             f"{got[i]}, want {want[i]}, bound {bound[i] if np.ndim(bound) else bound}")


class Pool:
    """The pages' bookkeeping in plain Python."""

    def __init__(self, data, refs, table, lens, page):
        self.data, self.refs, self.table, self.lens = (np.array(a) for a in (data, refs, table, lens))
        self.page = page

    def held(self, n):
        return -(-int(n) // self.page)

    def take(self, n):
        free = [p for p in range(len(self.refs)) if self.refs[p] <= 0]
        if len(free) < n:
            return None
        return free[:n]

    def free(self, seqs):
        for s in seqs:
            for c, p in enumerate(self.table[s]):
                if p >= 0:
                    self.refs[p] -= 1
                    self.table[s, c] = -1
            self.lens[s] = 0

    def fork(self, parents, children):
        for a, b in zip(parents, children):
            n = int(self.lens[a])
            full = n // self.page
            row = np.full(self.table.shape[1], -1, np.int32)
            row[:full] = self.table[a, :full]
            for p in row[:full]:
                self.refs[p] += 1
            if n % self.page:
                row[full] = self.take(1)[0]
                self.refs[row[full]] = 1
                self.data[:, row[full]] = self.data[:, self.table[a, full]]
            self.table[b], self.lens[b] = row, n

    def reserve(self, seqs, grow):
        for s, g in zip(seqs, grow):
            a, b = self.held(self.lens[s]), self.held(self.lens[s] + g)
            new = self.take(b - a)
            self.table[s, a:b] = new
            self.refs[new] = 1
            self.lens[s] += g

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        live = len(used)
        to = {p: p for p in used}
        holes = [p for p in range(live) if self.refs[p] <= 0]
        for p, hole in zip([p for p in used if p >= live], holes):
            to[p] = hole
            self.data[:, hole] = self.data[:, p]
        refs = np.zeros_like(self.refs)
        for p, n in to.items():
            refs[n] = self.refs[p]
        table = np.array([[to[p] if p >= 0 else p for p in row] for row in self.table],
                         dtype=np.int32).reshape(self.table.shape)
        self.refs, self.table = refs, table
        return live


def frequencies(half, base=10000.0):
    return base ** (-np.arange(half, dtype=np.float64) / max(half, 1))


def default_scale(dim):
    return 1.0 / math.sqrt(dim)
