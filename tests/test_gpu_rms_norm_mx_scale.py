"""MX codes of the norm by the Microscaling formats' scale: codes and scales bit for
bit, what they stand for next to y, and the product that reads them."""
import pytest
import torch

from tests import decode_ref as ref
from tests import mx_ref as mx
from tests.test_gpu_rms_norm import DEV, TYPES, inputs, qmm  # noqa: F401

pytestmark = pytest.mark.gpu


def outputs(rows, cols, fmt):
    c = torch.full((rows, cols), 99, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, -(-cols // 32)), 99, dtype=torch.uint8, device=DEV)
    return c, s, dict(codes=c, scales=s, fmt=fmt, layout="mx_ocp")


def check(codes, scales, y, fmt):
    c, s = mx.ocp_of(y, fmt)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu(), c)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 40), (5, 512), (3, 1000), (64, 4096), (3, 5001), (2, 8192), (2, 20000),
                                       (2, 33000)])
def test_codes_and_what_they_stand_for(qmm, rows, cols, dtype, fmt):  # noqa: F811
    x, r, w = inputs(rows, cols, TYPES[dtype], seed=cols)
    codes, scales, kw = outputs(rows, cols, fmt)
    qmm.qmm_rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV), **kw)
    _, y = ref.norm32(x, w, r, 1e-5, 0.0)
    check(codes, scales, y, fmt)
    got = mx.values(codes.cpu(), scales.cpu(), fmt)
    assert ((got - y.double()).abs() <= mx.bound(y, scales.cpu(), fmt)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_maxima_next_to_powers_of_two_and_extremes(qmm, fmt):  # noqa: F811
    # A row of ones: y is the weight.
    tops = torch.tensor([2.0 ** k * f for k in (-100, -9, 0, 7, 8, 15, 16, 100)
                         for f in (1 - 2.0 ** -24, 1.0, 1 + 2.0 ** -23, 1.75, 1.75 * (1 + 2.0 ** -23))])
    w = torch.zeros(len(tops) + 4, 32)
    w[:len(tops), 5] = tops
    w[:len(tops), 6] = -tops / 3
    w[-4, 3] = float("inf")
    w[-3, 3] = float("nan")
    w[-3, 4] = 1.0
    w[-2, 3] = 2.0 ** -140          # below the least scale
    codes, scales, kw = outputs(1, w.numel(), fmt)
    qmm.qmm_rms_norm(torch.ones(1, w.numel(), device=DEV), w.flatten().to(DEV), eps=0.0, **kw)
    check(codes, scales, w.view(1, -1), fmt)


def test_nan_and_infinities_stay_in_their_row(qmm):  # noqa: F811
    x, r, w = inputs(4, 300, torch.bfloat16)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    codes, scales, kw = outputs(4, 300, "e4m3")
    qmm.qmm_rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV), **kw)
    check(codes, scales, ref.norm32(x, w, r, 1e-5, 0.0)[1], "e4m3")
    assert mx.values(codes.cpu(), scales.cpu(), "e4m3").isnan().sum(1).tolist() == [0, 300, 1, 0]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_the_product_is_near_that_of_y(qmm, fmt):  # noqa: F811
    """Recorded norm and product, replayed, against the product of the unquantized y."""
    M, K, N = 5, 512, 64
    _, r, w = inputs(M, K, torch.bfloat16)
    g = torch.Generator().manual_seed(5)
    b = torch.randint(0, 120, (N, K), generator=g, dtype=torch.uint8)
    bs = torch.randint(118, 126, (N, K // 32), generator=g, dtype=torch.uint8)
    b64 = b.view(torch.float8_e4m3fn).double() * torch.exp2(bs.double() - 127).repeat_interleave(32, 1)
    xd, rd, wd, bd, bsd = torch.empty(M, K, dtype=torch.bfloat16, device=DEV), r.to(DEV), w.to(DEV), b.to(DEV), bs.to(DEV)
    codes, scales, kw = outputs(M, K, fmt)
    out = torch.empty(M, N, device=DEV)
    step = qmm.Step()
    step.add_rms_norm(xd, wd, residual=rd, **kw)
    step.finalize()
    for seed in range(3):
        x, _, _ = inputs(M, K, torch.bfloat16, seed=seed)
        xd.copy_(x)
        step.launch()
        qmm.qmm_lowp_matmul(codes, bd, scales, bsd, None, out, M, N, K, "mx", fmt, "e4m3")
        torch.cuda.synchronize()
        _, y = ref.norm32(x, w, r, 1e-5, 0.0)
        check(codes, scales, y, fmt)
        # The codes' distance from y, and the instruction's own sums: a group of 8
        # products is cut 2^-12 below its largest.
        off = mx.bound(y, scales.cpu(), fmt) @ b64.abs().T
        off += 8 * 2.0 ** -12 * (mx.values(codes.cpu(), scales.cpu(), fmt).abs() @ b64.abs().T) + 1e-30
        assert ((out.cpu().double() - y.double() @ b64.T).abs() <= off).all()
    step.close()
