"""Plain forms of the operators around a decode step's projections (numpy and
torch on the CPU), written from the formulas in include/qmm.h."""
import math

import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# -- the norm ----------------------------------------------------------------

def norm32(x, weight, residual, eps, offset):
    """(h, y) in 32 bits, as the definition rounds them (the sum in 64)."""
    h = x.float()
    if residual is not None:
        h = h + residual.float()
    i = (1.0 / torch.sqrt(h.double().square().sum(-1, keepdim=True) / h.shape[1] + eps)).float()
    w = torch.ones(h.shape[1]) if weight is None else weight.float()
    return h, h * i * (w + offset)


def int8_of(y, block):
    rows, cols = y.shape
    p = torch.nn.functional.pad(y, (0, -cols % block)).view(rows, -1, block)
    # A maximum that skips NaN.
    top = torch.where(p.isnan(), 0.0, p.abs()).amax(-1, keepdim=True)
    s = top * torch.tensor(1.0 / 127.0)     # the reciprocal rounded to 32 bits
    q = torch.round(p / s).nan_to_num(-127.0, 127.0, -127.0).clamp(-127, 127)
    return torch.where(s != 0, q, 0.0).to(torch.int8).view(rows, -1), s[..., 0]


def fp8_of(v, fmt):
    kind, most = FP8[fmt]
    code = v.clamp(-most, most).to(kind).view(torch.uint8)
    return torch.where(v.isnan(), 0x7F, code.int()).to(torch.uint8)


def mx_of(y, fmt):
    rows, cols = y.shape
    p = torch.nn.functional.pad(y, (0, -cols % 32)).view(rows, -1, 32)
    top = torch.where(p.isnan(), 0.0, p.abs()).amax(-1, keepdim=True)
    e = torch.where(top > 0, top * torch.tensor(1.0 / FP8[fmt][1]), 1.0).view(torch.int32) >> 23
    s = torch.where(e == 255, float("nan"), torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e - 127)).float()
    return fp8_of((p / s).view(rows, -1)[:, :cols], fmt), e[..., 0].to(torch.uint8)


# -- sampling ----------------------------------------------------------------

def sample_row(z, t, k, p, m, u):
    """(token, logprob) of one row of 64-bit logits, by the definition."""
    z = np.where(np.isnan(z), -np.inf, z)
    n = len(z)
    order = np.lexsort((np.arange(n), -z))
    top = z[order[0]]
    if top == -np.inf:
        return -1, -np.inf
    if not t > 0:
        t, k = 1.0, 1
    with np.errstate(invalid="ignore"):
        w = np.where(z == top, 1.0, 0.0 if np.isinf(top) else np.exp((z - top) / t))
    if k <= 0 or k > n:
        k = n
    best = order[:k]
    if p < 1:
        cum = np.cumsum(w[best])
        best = best[:1 + np.searchsorted(cum, max(p, 0.0) * cum[-1], side="left")]
    best = best[w[best] >= min(m, 1.0)] if m > 0 else best
    at = np.sort(best)
    cum = np.cumsum(w[at])
    j = np.searchsorted(cum, u * cum[-1], side="right")
    return int(at[j]), float(np.log(w[at[j]]) - np.log(cum[-1]))


def sample_allowed(z, t, k, p, m, u, vocab):
    """Every (token, logprob) that sums held to the definition's whole units may
    lead to: a unit is 2^-(62 - ceil(log2 vocab)), each weight is off by half of
    one, and the sums of 64 bits here by less than that; so next to a border of u
    or top_p both sides are right."""
    d = vocab * 2.0 ** -(62 - max(0, math.ceil(math.log2(vocab))))
    us = {min(max(u + e, 0.0), 1 - 2.0 ** -53) for e in (-d, 0.0, d)}
    ps = {p} if not p < 1 else {max(p - d, 0.0), p, min(p + d, 1 - 2.0 ** -53)}
    return [sample_row(z, t, k, a, m, b) for a in ps for b in us]


# -- experts -----------------------------------------------------------------

def unpacked(codes, bits):
    """The fields of packed bytes, least significant bits first, along the last
    dimension."""
    if bits == 8:
        return codes.astype(np.int64)
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.int64)


class Experts:
    """Random experts of a layer: packed tensors (torch) and their values (numpy,
    64 bits): code, zero point and scale of every element."""

    def __init__(self, experts, hidden, inter, block, bits, zero_points=True, s_dtype=torch.bfloat16, seed=0):
        self.experts, self.hidden, self.inter, self.block, self.bits = experts, hidden, inter, block, bits
        g = torch.Generator().manual_seed(seed)
        self.parts = []
        for rows, cols in ((2 * inter, hidden), (hidden, inter)):
            kb = -(-cols // block)
            codes = torch.randint(0, 256, (experts, rows, kb, block * bits // 8), dtype=torch.uint8, generator=g)
            scale = (0.4 + 1.2 * torch.rand(experts, rows, kb, generator=g)) / (2 ** bits / 3.5 * math.sqrt(cols))
            zp = None
            if zero_points:
                zp = torch.randint(0, 256, (experts, rows, -(-kb * bits // 8)), dtype=torch.uint8, generator=g)
            self.parts.append((codes, scale.to(s_dtype), zp))

    def tensors(self):
        return [*self.parts[0], *self.parts[1]]

    def values(self, which, e):
        """(codes, zero points, scales) [rows, cols] of an expert's projection."""
        codes, scale, zp = self.parts[which]
        cols = self.inter if which else self.hidden
        c = unpacked(codes[e].reshape(codes.shape[1], -1).numpy(), self.bits)[:, :cols]
        kb, k = scale.shape[2], np.arange(cols) // self.block
        z = np.full((c.shape[0], kb), 1 << (self.bits - 1)) if zp is None else \
            unpacked(zp[e].numpy(), self.bits)[:, :kb]
        return c, z[:, k], scale[e].double().numpy()[:, k]


def route(logits, top_k, normalize):
    """(ids, weights) [tokens, top_k] in 64 bits; -1 and 0 for none."""
    z = logits.double().numpy().copy()
    z[np.isnan(z)] = -np.inf
    T, E = z.shape
    ids, weights = np.full((T, top_k), -1), np.zeros((T, top_k))
    for t in range(T):
        top = z[t].max()
        if top == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            p = np.where(z[t] == top, 1.0, 0.0 if np.isinf(top) else np.exp(z[t] - top))
        best = np.lexsort((np.arange(E), -z[t]))[:top_k]
        w = p[best] / (p[best].sum() if normalize else p.sum())
        ids[t], weights[t] = np.where(w > 0, best, -1), w
    return ids, weights


def moe(x, experts, ids, weights, dtype):
    """(y, bound) [tokens, hidden] in 64 bits.  bound: how far a right layer may be,
    products of x and whole numbers (4-bit codes offset by 16) being summed in 32
    bits: a block's sum and its zero point's part, scaled, then the blocks'."""
    T, H = x.shape
    x64 = x.double().numpy()
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    u = 2.0 ** -23        # a step of 32 bits: sums in matrix cores may be cut, not rounded
    keep = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -16
    field = 16 if experts.bits == 4 and dtype != torch.float32 else 0

    def project(e, which, v, dv):
        c, z, s = experts.values(which, e)
        out = ((c - z) * s) @ v
        terms = min(experts.block, len(v)) + -(-len(v) // experts.block) + 8
        off = terms * u * ((c + z + 2 * field) * np.abs(s)) @ np.abs(v) + np.abs((c - z) * s) @ dv
        return out, off

    for t in range(T):
        for j in range(ids.shape[1]):
            e, w = int(ids[t, j]), float(weights[t, j])
            if e < 0 or e >= experts.experts or w == 0:
                continue
            a, da = project(e, 0, x64[t], np.zeros(H))
            g, up, dg, du = a[:experts.inter], a[experts.inter:], da[:experts.inter], da[experts.inter:]
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            h = silu * up
            # silu's slope is at most 1.1; exp, sum, quotient and product round.
            dh = 1.1 * dg * (np.abs(up) + du) + np.abs(silu) * du + (12 * u + keep) * np.abs(h) + 1e-37
            o, do = project(e, 1, h, dh)
            y[t] += w * o
            bound[t] += abs(w) * do + abs(w) * np.abs(o) * (experts.experts + 16) * u
    return y, bound + HALF_STEP[dtype] * (np.abs(y) + bound) + TINY[dtype]
