"""Codes of an 8-bit float type and the format that the norm is asked to write."""
import pytest
import torch

from tests.test_decode_host import calls, there


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


@pytest.mark.parametrize("layout", ["mx", "mx_ocp", "tensor"])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e5m2), ("e5m2", torch.float8_e4m3fn)])
def test_codes_of_the_other_format_are_refused(qmm, layout, fmt, dtype):
    c = calls(qmm, lambda n, x: there(x))
    scales = there(torch.ones(1) if layout == "tensor" else torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match=f"codes of {dtype} hold another format than fmt='{fmt}'"):
        c["norm"](layout=layout, fmt=fmt, codes=there(torch.zeros(4, 64).to(dtype)), scales=scales)


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2), ("e4m3", torch.uint8),
                                       ("e5m2", torch.uint8)])
def test_codes_of_the_format_and_bytes_are_taken(qmm, fmt, dtype):
    codes, scales = torch.zeros(4, 64).to(dtype), torch.zeros(4, 2, dtype=torch.uint8)
    assert len(qmm._quant_struct(codes, scales, 4, 64, fmt, "mx", 0)) == 32


def test_formats_of_fewer_bits_are_refused(qmm):
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for fmt in ("e2m3", "e2m1", "int8"):
        with pytest.raises(ValueError, match='fmt must be "e4m3" or "e5m2"'):
            qmm._quant_struct(codes, scales, 4, 64, fmt, "mx", 0)
