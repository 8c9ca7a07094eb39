"""int8 codes of rows that hold a NaN or an infinity: what the norm loses to them
stays to be seen in the scales, and in the product that reads them."""
import pytest
import torch

from tests import decode_ref as ref
from tests.test_gpu_rms_norm import DEV, TYPES, inputs, outputs, qmm  # noqa: F401

pytestmark = pytest.mark.gpu


def wanted(y, block):
    """(codes, scales) of y in 32 bits: a NaN makes its block's scale one, an
    infinite maximum an infinite one, and such blocks have no codes."""
    rows, cols = y.shape
    c, s = ref.int8_of(y, block)
    nan = torch.nn.functional.pad(y, (0, -cols % block)).view(rows, -1, block).isnan().any(-1)
    s = torch.where(nan, float("nan"), s)
    return torch.where(s.isfinite()[..., None], c.view(rows, -1, block), 0).to(torch.int8).view(rows, -1), s


def check(codes, scales, y, block):
    c, s = wanted(y, block)
    scales = scales.cpu()
    assert torch.equal(scales.isnan(), s.isnan())
    assert torch.equal(scales.nan_to_num(-1.0, posinf=-2.0), s.nan_to_num(-1.0, posinf=-2.0))
    assert torch.equal(codes.cpu(), c)
    return s


# A wave a row, one to sixteen waves, several chunks a thread, rows read again;
# blocks inside a wave, of a whole wave, of several.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,block", [(300, 16), (500, 256), (512, 512), (1000, 64), (4096, 128), (4096, 512),
                                        (4096, 1024), (5001, 4096), (9000, 2048), (16384, 32), (20000, 1024),
                                        (33000, 64), (33000, 4096)])
def test_a_row_with_a_nan_or_an_infinity(qmm, cols, block, dtype):  # noqa: F811
    x, r, w = inputs(6, cols, TYPES[dtype], seed=cols)
    x[1, cols // 2] = float("nan")
    x[2, 3] = float("inf")
    r[3, cols - 1] = float("nan")
    r[4, 0] = -float("inf")
    codes, scales, kw = outputs(6, cols, ("int8", "block", block))
    qmm.qmm_rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV), **kw)
    _, y = ref.norm32(x, w, r, 1e-5, 0.0)
    s = check(codes, scales, y, block)
    # A NaN is in every y of its row, an infinity leaves one and zeros.
    assert s[1].isnan().all() and s[3].isnan().all() and s[0].isfinite().all() and s[5].isfinite().all()
    assert s[2].isnan().sum() == 1 and s[4].isnan().sum() == 1


@pytest.mark.parametrize("cols,block", [(300, 32), (4096, 128), (4096, 2048), (33000, 1024)])
def test_a_weight_that_is_nan_and_weights_that_overflow(qmm, cols, block):  # noqa: F811
    x, r, w = inputs(5, cols, torch.float32, seed=cols)
    w[7] = float("nan")
    w[cols - 2] = 3e38
    # 3e38 (h i) overflows where |h i| is 2, and does not where it is a half.
    r[:, cols - 2] = 0
    scale = (x + r).square().mean(-1).sqrt()
    x[:, cols - 2] = scale * torch.tensor([2.0, -2.0, 0.5, 2.0, -0.5])
    codes, scales, kw = outputs(5, cols, ("int8", "block", block))
    qmm.qmm_rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV), **kw)
    _, y = ref.norm32(x, w, r, 1e-5, 0.0)
    s = check(codes, scales, y, block)
    assert s[:, 0].isnan().all()
    if len(s[0]) > 1:
        assert s[:, -1].isinf().tolist() == [True, True, False, True, False] and s[:, 1:].isnan().sum() == 0


@pytest.mark.parametrize("M,K,N,bs,bits", [(4, 512, 96, 32, 4), (4, 512, 96, 128, 8), (4, 256, 64, 32, 3),
                                           (4, 512, 64, 16, 4), (20, 512, 64, 64, 2)])
def test_the_product_of_such_a_row_is_nan(qmm, M, K, N, bs, bits):  # noqa: F811
    """... and the other rows' is what it is without it."""
    from block_quantized_weight_matmulnbits_amd.workloads import make_matmul_case
    c = make_matmul_case(M, K, N, bs, bits, a_dtype="f32", has_zp=True, has_bias=True, seed=K).to(DEV)
    x, r, w = inputs(M, K, torch.float32)
    layouts = [(c.B, c.scales, c.zero_points)]
    if bits != 3 and bs >= 32:
        layouts.append((qmm.qmm_repack(c.B, c.scales, c.zero_points, K, N, bs, bits), None, None))

    def product(x, B, s, z):
        codes, scales, kw = outputs(len(x), K, ("int8", "block", bs))
        qmm.qmm_rms_norm(x.to(DEV), w.to(DEV), residual=r[:len(x)].to(DEV), **kw)
        got = torch.empty(len(x), N, device=DEV)
        qmm.qmm_gemm_compint8_quantized(codes, scales, B, s, z, c.bias, got, len(x), K, N, bs, bits)
        return got
    bad = x.clone()
    bad[1, 40] = float("nan")
    bad[2, 41] = float("inf")
    for b in layouts:
        good, got = product(x, *b), product(bad, *b)
        assert good.isfinite().all()
        assert got[1:3].isnan().all()
        assert torch.equal(got[0], good[0]) and torch.equal(got[3:], good[3:])
        assert product(bad[1:2], *b).isnan().all()      # a token alone
