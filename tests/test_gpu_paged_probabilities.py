"""qmm_paged_attention of a few rows in 16 bits: probabilities keep what their
type cannot hold, and a value that is not finite stays what it is."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged_attention import dev, run

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("counts,lens", [([1, 1], [700, 33]), ([3, 2], [61, 300]), ([1], [5000])])
def test_the_output_is_rounded_once(dtype, D, counts, lens):
    """Equal to the definition rounded to the type but for what 32 bits leave
    open: no probability is off by half a step of 16 bits."""
    print(f"[once] {dtype} D={D} counts={counts} lens={lens}", flush=True)
    from block_quantized_weight_matmulnbits_amd import qmm as q
    H, KV, page, g = 4, 2, 16, torch.Generator().manual_seed(D)
    starts, lens, table, total = ref.make_batch(counts, lens, page, D)
    T = int(starts[-1])
    kp, vp = (torch.randn(total, KV, page, D, generator=g).to(dtype) for _ in range(2))
    x = (1.7 * torch.randn(T, H, D, generator=g)).to(dtype)
    y, _, bound, _ = ref.attention(x.float(), kp.float(), vp.float(), starts, lens, table, D ** -0.5)
    # Beside the bound of 32-bit probabilities: what is left after two parts of
    # at least 8 bits each, 2^-16 of |v| weighed by the probabilities.
    weighed = ref.attention(x.float(), kp.float(), vp.float().abs(), starts, lens, table, D ** -0.5)[0]
    bound = bound + 2.0 ** -16 * weighed
    kv = q.PagedKV(kp.to(DEV), vp.to(DEV))
    batch = q.PagedBatch(dev(starts), dev(lens), dev(table), T, max(counts), int(lens.max()))
    out = torch.empty(T, H, D, dtype=dtype, device=DEV)
    ws = torch.zeros(q.qmm_paged_attention_workspace_size(batch, H, KV, D), dtype=torch.uint8, device=DEV)
    q.qmm_paged_attention(x.to(DEV), kv, batch, out, ws)
    torch.cuda.synchronize()
    ref.assert_close(out, y, ref.rounded(y, bound, dtype), "out")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("n,D", [(1, 64), (1, 256), (7, 128), (150, 64)])
def test_a_bad_value_that_every_token_sees(dtype, bad, n, D):
    def spoil(kp, vp, table, lens):
        for j in (5, 40):
            vp[table[0, j // 16], 0, j % 16, 3] = bad
            vp[table[0, j // 16], 1, j % 16, 11] = bad
    run(dtype, [n], [260], 4, 2, D, spoil=spoil)
