"""qmm_paged_attention where one key holds nearly all of a row and the rest,
each too little for 16 bits beside it, make the output."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("place", [0.0, 0.6, 1.0])
@pytest.mark.parametrize("n,length", [(1, 131072), (1, 900), (24, 20000), (40, 3000)])
@pytest.mark.parametrize("below", [9.0, 17.8])
def test_a_sink_over_a_long_context(dtype, place, n, length, below):
    print(f"[sink] {dtype} place={place} n={n} length={length} below={below}", flush=True)
    from block_quantized_weight_matmulnbits_amd import qmm as q
    D, H, page = 64, 2, 16
    g = torch.Generator().manual_seed(n + length)
    starts, lens, table, total = ref.make_batch([n], [length], page)
    kp = (0.3 * torch.randn(total, 1, page, D, generator=g)).to(dtype)
    vp = (1.0 + 0.1 * torch.randn(total, 1, page, D, generator=g)).to(dtype)
    sink = int(place * (length - n))
    kp[table[0, sink // page], 0, sink % page] = below / 8     # its score is `below`, the others' near 0
    vp[table[0, sink // page], 0, sink % page] = 0.0
    x = torch.ones(n, H, D).to(dtype)
    y, e, bound, eb = ref.attention(x, kp, vp, starts, lens, table, 1 / 8)
    if dtype == torch.float16:
        # The oracle allows half of f16's smallest subnormal for each
        # probability, whose largest it takes as 1.  Taken 2^11 larger or more
        # it is 2^-11 of that; a reference up to 1 (log2) above the largest
        # score doubles it.
        j = np.arange(length)
        size = np.abs(ref.f64(vp)[table[0, j // page], 0, j % page])
        loose = ref.HALF_TINY[dtype] * np.cumsum(size, axis=0)[length - n:, None]   # of the keys each token sees
        bound = bound - loose + loose * 2.0 ** -10
        assert (bound < 0.02 * np.abs(y)).all()
    kv = q.PagedKV(kp.to(DEV), vp.to(DEV))
    batch = q.PagedBatch(dev(starts), dev(lens), dev(table), n, n, length)
    out, lse = torch.empty(n, H, D, dtype=dtype, device=DEV), torch.empty(n, H, device=DEV)
    ws = torch.zeros(q.qmm_paged_attention_workspace_size(batch, H, 1, D), dtype=torch.uint8, device=DEV)
    q.qmm_paged_attention(x.to(DEV), kv, batch, out, ws, scale=1 / 8, lse=lse)
    torch.cuda.synchronize()
    ref.assert_close(out, y, ref.rounded(y, bound, dtype), "out")
    ref.assert_close(lse, e, eb, "lse")
