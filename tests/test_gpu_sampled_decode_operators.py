"""examples/sampled_decode.py: the projections, the rotary append and the attention
of a pass against 64 bits (its norms, experts and sampling have theirs in
test_gpu_sampled_decode.py)."""
import numpy as np
import pytest
import torch

import oracle
from tests import decode_ref
from tests import paged_ref
from tests.test_gpu_sampled_decode import example, prompt, small  # noqa: F401
from tests.util import TOL, assert_within, f64, u8

pytestmark = pytest.mark.gpu


def weights(example, d):  # noqa: F811
    """The weights of the decoder's projections as they were before the repack, by
    the repacked ones."""
    from block_quantized_weight_matmulnbits_amd.workloads import make_matmul_case
    paged = example.paged_decode
    return {id(p.B): (make_matmul_case(1, p.K, p.N, block, bits, a_dtype="bf16", has_zp=True, seed=seed), p, block, bits)
            for p, seed, block, bits in ((d.qkv[0], 10, example.BLOCK, example.BITS), (d.o[0], 50, paged.BLOCK, paged.BITS),
                                         (d.router[0], 70, paged.BLOCK, paged.BITS), (d.head, 90, paged.BLOCK, paged.BITS))}


def product(x, case, p, block, bits):
    return oracle.matmul_nbits(x, u8(case.B), f64(case.scales), u8(case.zero_points), None, p.N, p.K, block, bits)


def test_every_operator_of_a_pass_is_checked(example):  # noqa: F811
    from block_quantized_weight_matmulnbits_amd import qmm
    d = small(example, layers=1)
    of = weights(example, d)
    d.prefill(3, prompt(30, 3), 30)         # something is cached already
    qmm.qmm_pages_reserve(d.pool, d.list([3]), d.list([21]), d.status, d.pages_ws)
    b = d.batch([0, 0, 0, 21, 0, 0], 21)
    b.x[0].copy_(d.embed(prompt(21, 1)))
    b.uniform.copy_(torch.rand(21, generator=torch.Generator().manual_seed(2)))
    starts, lens, table = (t.cpu().numpy() for t in (b.starts, d.pool.lens, d.pool.table))
    assert lens.tolist() == [0, 0, 0, 51, 0, 0]
    kv, checked = d.kv[0], []
    for name, args, kw in d.calls(b):
        before = [t.cpu() if isinstance(t, torch.Tensor) else t for t in args]
        pages = [kv.k_pages.cpu(), kv.v_pages.cpu()]
        getattr(qmm, "qmm_" + name)(*args, **kw)
        torch.cuda.synchronize()
        if name == "gemm_compint8_quantized":
            case, p, block, bits = of[id(args[2])]
            kb = p.K // block
            a = (before[0].double().view(21, kb, block) * before[1].double()[..., None]).view(21, -1)
            Y, S = product(a.numpy(), case, p, block, bits)
            # A block's term has two roundings (the scales' product, the term), the sum
            # at most kb + 1 more: half a step of 32 bits each; then the output's.
            off = S * (kb + 3) * 2.0 ** -24
            bound = off + decode_ref.HALF_STEP[torch.bfloat16] * (np.abs(Y) + off) + decode_ref.TINY[torch.bfloat16]
            assert np.abs(Y).max() > 0.1        # a product of zeros would pass any bound
            assert (np.abs(f64(args[6]) - Y.reshape(args[6].shape)) <= bound.reshape(args[6].shape)).all()
        elif name == "gemm":
            case, p, block, bits = of[id(args[1])]
            Y, S = product(f64(before[0]), case, p, block, bits)
            assert_within(args[5], Y, S, TOL[torch.bfloat16], f"projection {p.K} -> {p.N}")
        elif name == "rope_append":
            q, k, v = before[:3]
            want = paged_ref.rope(q, k, v, *pages, starts, lens, table, f64(args[6]))
            paged_ref.assert_close(args[3], want[0], paged_ref.rounded(want[0], want[3], torch.bfloat16), "q")
            paged_ref.assert_close(kv.k_pages, want[1],
                                   np.where(want[4] > 0, paged_ref.rounded(want[1], want[4], torch.bfloat16), 0.0), "k")
            paged_ref.assert_close(kv.v_pages, want[2], 0.0, "v")
        elif name == "paged_attention":
            out, _, bound, _ = paged_ref.attention(before[0], *pages, starts, lens, table, paged_ref.default_scale(d.dim))
            paged_ref.assert_close(args[3], out, paged_ref.rounded(out, bound, torch.bfloat16), "attended")
        else:
            assert name in ("rms_norm", "moe", "sample"), name      # in the other file
            continue
        checked.append(name)
    assert checked == ["gemm_compint8_quantized", "rope_append", "paged_attention", "gemm", "gemm", "gemm"]
