"""qmm_rope_append of thousands of tokens, which take four a workgroup and pass
the caches by: every type, pairing, part of the head and width of load."""
import pytest
import torch

from tests.test_gpu_rope import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,half", [(64, 32), (80, 20), (34, 5), (48, 0)])
def test_types_pairings_and_parts(dtype, interleaved, D, half):
    run(dtype, [4100 - 9, 1, 0, 8], [4200, 1, 3, 70], 3, 1, D, half, 16, interleaved, factor=1.25,
        shift=1_000_000, token_major=interleaved, seed=D)


@pytest.mark.parametrize("tokens", [4095, 4096, 4097, 4099])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_counts_around_the_variants_limit(dtype, tokens):
    run(dtype, [tokens - 70, 70], [tokens, 500], 2, 2, 32, 16, 8, alias=True, seed=tokens)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_off_alignment_and_tokens_without_a_page(interleaved):
    def spoil(table, total):
        table[0, 3] = -1
        table[1, 0] = total + 5
    run(torch.bfloat16, [4090, 20], [4090, 20], 2, 1, 64, 32, 16, interleaved, offset=1, spoil=spoil)
