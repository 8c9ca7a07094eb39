"""qmm_gemm_compint8_quantized on repacked weights beside qmm_gemm_compint8 on the
activations that the codes were made of."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 17, 40])
@pytest.mark.parametrize("K,N,bs,bits", [(512, 192, 32, 4), (500, 96, 64, 8), (4096, 160, 128, 4), (640, 64, 64, 2),
                                         (1024, 48, 256, 8)])
def test_beside_the_product_that_quantizes(qmm, M, K, N, bs, bits):
    import oracle
    from block_quantized_weight_matmulnbits_amd.workloads import make_matmul_case
    host = make_matmul_case(M, K, N, bs, bits, a_dtype="f32", has_zp=True, has_bias=True, seed=K)
    c = host.to(DEV)
    B = qmm.qmm_repack(c.B, c.scales, c.zero_points, K, N, bs, bits)
    kb = -(-K // bs)
    qa, sa = torch.empty(M, kb * bs, dtype=torch.int8, device=DEV), torch.empty(M, kb, device=DEV)
    qmm.qmm_debug_quantize_a(c.A, M, K, bs, qa, sa)
    ws = torch.empty(qmm.qmm_compint8_workspace_size(M, K, bs), dtype=torch.uint8, device=DEV)
    want, got = (torch.empty(M, N, device=DEV) for _ in range(2))
    qmm.qmm_gemm_compint8(c.A, B, None, None, c.bias, want, M, K, N, bs, bits, ws)
    qmm.qmm_gemm_compint8_quantized(qa, sa, B, None, None, c.bias, got, M, K, N, bs, bits)
    if M > 1:
        # The same kernel on the same codes.
        assert torch.equal(got, want)
    # One token's is another kernel's, which adds the blocks in another order; both
    # are the definition's but for the roundings of 32 bits: two of each block's
    # term, at most kb + 1 of the sum, the bias's.
    a = (qa.cpu().double().view(M, kb, bs) * sa.cpu().double()[..., None]).view(M, -1)[:, :K]
    Y, S = oracle.matmul_nbits(a.numpy(), host.B.numpy(), host.scales.double().numpy(), host.zero_points.numpy(),
                               host.bias.double().numpy(), N, K, bs, bits)
    bound = torch.from_numpy(S) * (kb + 4) * 2.0 ** -24
    for y in (got, want):
        assert ((y.cpu().double() - torch.from_numpy(Y)).abs() <= bound).all()
