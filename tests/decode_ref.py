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
