"""The Microscaling formats' 8-bit codes from their definition, and how far they
may be from what they stand for."""
import torch

from tests import decode_ref as ref

# The exponent of a format's largest value, half a step of its normal values
# (relative) and half a step of its subnormal ones.
EMAX = {"e4m3": 8, "e5m2": 15}
HALF = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}


def ocp_of(y, fmt):
    """(codes, E8M0 scales) of y [rows, cols] in 32 bits: the power of two at or below
    a block's maximum over that of the format's largest value."""
    rows, cols = y.shape
    p = torch.nn.functional.pad(y, (0, -cols % 32)).view(rows, -1, 32)
    top = torch.where(p.isnan(), 0.0, p.abs()).amax(-1, keepdim=True).double()
    # top = m 2^x with m in [1/2, 1)
    e = (torch.frexp(top).exponent - 1 - EMAX[fmt] + 127).clamp(0, 254)
    e = torch.where(top == 0, 127, torch.where(top.isinf(), 255, e))
    s = torch.where(e == 255, float("nan"), torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e - 127)).float()
    return ref.fp8_of((p / s).view(rows, -1)[:, :cols], fmt), e[..., 0].to(torch.uint8)


def values(codes, scales, fmt):
    """What codes and scales stand for, in 64 bits."""
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :codes.shape[1]]
    return codes.view(ref.FP8[fmt][0]).double() * s


def bound(y, scales, fmt):
    """How far a value may be from y: half a step of the format, or, where it is
    clipped, its distance from the largest value, which is at least 7/8 of the next
    power of two, of which a scaled value is below."""
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :y.shape[1]]
    z, (normal, least) = (y.double() / s).abs(), HALF[fmt]
    return s * torch.where(z > ref.FP8[fmt][1], z / 8, (normal * z).clamp(min=least))
