"""qmm_paged_attention on f32 prompts and wide f32 heads, where many rows meet
long contexts."""
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = 2.0 ** -24


def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def want(x, kp, vp, starts, lens, table):
    """Causal attention a sequence and a head at a time, in 64 bits: (out, lse,
    bound of out, bound of lse), the bounds as in paged_ref.attention."""
    T, H, D = x.shape
    KV, page = kp.shape[1], kp.shape[2]
    scale = 1.0 / math.sqrt(D)
    out, ob = (torch.zeros(T, H, D, dtype=torch.float64, device=DEV) for _ in range(2))
    lse, lb = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV), torch.zeros(T, H, device=DEV).double()
    for s in range(len(lens)):
        t, n, length = int(starts[s]), int(starts[s + 1] - starts[s]), int(lens[s])
        j = np.arange(length)
        ids, at = dev(table[s, j // page].astype(np.int64)), dev(j % page)
        hide = torch.arange(length, device=DEV)[None] > torch.arange(length - n, length, device=DEV)[:, None]
        for h in range(H):
            k, v = (p[ids, h // (H // KV), at].double() for p in (kp, vp))
            q = x[t:t + n, h].double()
            kt = k.T.contiguous()
            z = (q @ kt * scale).masked_fill(hide, -math.inf)
            off = (q.abs() @ kt.abs() * (abs(scale) * (D + 8) * F32)).masked_fill(hide, 0.0).amax(-1)
            big = z.masked_fill(hide, 0.0).abs().amax(-1)
            far = 2 * off + (length + 32) * F32 + 4 * big * F32
            e = torch.logsumexp(z, -1)
            p = torch.exp(z - e[:, None])
            out[t:t + n, h], lse[t:t + n, h] = p @ v, e
            ob[t:t + n, h] = (p @ v.abs()) * far[:, None] * 1.01
            lb[t:t + n, h] = far + 8 * F32 * e.abs()
    return [y.cpu().numpy() for y in (out, lse, ob, lb)]


def check(counts, lens, H, KV, D, page=16, max_len=None, seed=0):
    print(f"[f32] counts={counts[:4]} lens={lens[:4]} H={H} KV={KV} D={D} max_len={max_len}", flush=True)
    q, g = qmm(), torch.Generator(device=DEV).manual_seed(seed)
    starts, lens, table, total = ref.make_batch(counts, lens, page, seed)
    T = int(starts[-1])
    kp, vp = (torch.randn(total, KV, page, D, device=DEV, generator=g) for _ in range(2))
    x = 1.7 * torch.randn(T, H, D, device=DEV, generator=g)
    batch = q.PagedBatch(dev(starts), dev(lens), dev(table), T, max(counts), max_len or int(lens.max()))
    # Room after the workspace that nothing may touch.
    size, guard = q.qmm_paged_attention_workspace_size(batch, H, KV, D), 1 << 20
    ws = torch.full((size + guard,), 0xA5, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty(T, H, D, device=DEV), torch.empty(T, H, device=DEV)
    q.qmm_paged_attention(x, q.PagedKV(kp, vp), batch, out, ws[:size], lse=lse)
    torch.cuda.synchronize()
    assert ws[size:].eq(0xA5).all()
    y, e, yb, eb = want(x, kp, vp, starts, lens, table)
    ref.assert_close(out, y, ref.rounded(y, yb, torch.float32), "out")
    ref.assert_close(lse, e, eb, "lse")


@pytest.mark.parametrize("counts,lens,H,KV", [
    ([2048], [4500], 32, 8),             # 2048 tiles of rows
    ([600], [4500], 32, 8),              # 600
    ([1024, 900], [1024, 4400], 8, 8),   # uneven, a head a group
])
def test_prompts_over_more_than_4096_keys(counts, lens, H, KV):
    check(counts, lens, H, KV, 128)


@pytest.mark.parametrize("seqs", [64, 256])
def test_many_single_tokens_of_wide_heads(seqs):
    lens = [1 + 13 * i % 90 for i in range(seqs - 1)] + [4300]
    check([1] * seqs, lens, 8, 8, 256, max_len=8192)
