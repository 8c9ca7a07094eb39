"""Experts and sampling where their kernels change course: items of several
rounds, bounds of min_p next to a weight, workspaces that recorded steps share."""
import numpy as np
import pytest
import torch

from tests import decode_ref as ref
from tests.test_gpu_moe import check as check_layer, layer, on_gpu
from tests.test_gpu_sample import check as check_tokens, draw, sample

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, 4), (torch.float16, 8), (torch.float32, 4)])
def test_one_expert_of_many_has_most_tokens(qmm, dtype, bits):
    """More items than workgroups that are resident, and one expert's tokens in
    several tiles after another."""
    ex = ref.Experts(60, 1024, 272, 32, bits, seed=21)
    g = torch.Generator().manual_seed(21)
    x = torch.randn(40, 1024, generator=g).to(dtype)
    ids = torch.randint(0, 60, (40, 3), generator=g, dtype=torch.int32)
    ids[:, 0] = 37
    ids[5] = 37                     # an expert three times
    ids[6] = torch.tensor([-1, 60, 37])
    weights = torch.rand(40, 3, generator=g)
    y = layer(qmm, ex, x, ids=ids, weights=weights)
    check_layer(qmm, ex, x, y, ids.numpy(), weights.double().numpy())


def test_the_same_tokens_alone(qmm):
    """A token's output is the same in a batch of many rounds and by itself."""
    ex = ref.Experts(64, 1024, 272, 64, 4, seed=22)
    w = on_gpu(qmm, ex)
    g = torch.Generator().manual_seed(22)
    x, logits = torch.randn(12, 1024, generator=g).bfloat16(), torch.randn(12, 64, generator=g)
    y = layer(qmm, ex, x, logits, 6, w=w)
    for t in (0, 7, 11):
        assert torch.equal(layer(qmm, ex, x[t:t + 1], logits[t:t + 1], 6, w=w)[0], y[t])


@pytest.mark.parametrize("top", [0.0, 3e4, -3e4])
@pytest.mark.parametrize("temperature", [1e-3, 1.0, 1e3])
def test_min_p_next_to_a_weight(qmm, top, temperature):
    """Logits on either side of top + T log min_p, some of them by one step."""
    m = torch.tensor([1.0, 1 - 2.0 ** -24, 0.5, 0.05, 1e-6, 1e-30, 2.0])
    g = torch.Generator().manual_seed(23)
    rows, vocab = len(m), 6000
    z = torch.full((rows, vocab), top) - temperature * (40 * torch.rand(rows, vocab, generator=g)).abs()
    z[:, 11] = top
    edge = top + temperature * torch.log(m.clamp(max=1).double())
    for i in range(rows):
        # The nearest values of 32 bits that are surely on one side of the edge
        # (the definition's own roundings there are below a thousandth of a step of them).
        e = float(edge[i])
        below = np.nextafter(np.nextafter(np.float32(e), np.float32(-np.inf)), np.float32(-np.inf))
        above = np.nextafter(np.nextafter(np.float32(e), np.float32(np.inf)), np.float32(np.inf))
        z[i, 100:140] = float(below)
        z[i, 3000:3040] = min(float(above), top)
    u = torch.rand(rows, generator=g)
    for _ in range(3):
        check_tokens(qmm, z, u, temperature=temperature, min_p=m)
        check_tokens(qmm, z, u, temperature=temperature, min_p=m, top_p=0.8)
        u = (u + 0.37) % 1


def test_min_p_under_a_temperature_beyond_logits(qmm):
    """T log min_p past 1e30: weights of 1, 0.14 and 0, of which min_p leaves the first."""
    z = torch.full((3, 5000), -2e31)
    z[:, 17] = z[:, 4000] = 0.0
    z[1] = -3e38
    z[1, 40] = 1.0
    u = torch.tensor([0.3, 0.9, 0.7])
    tokens = check_tokens(qmm, z, u, temperature=1e31, min_p=[0.5, 0.5, 0.1])
    assert tokens[:2].tolist() == [17, 40]


def test_recorded_steps_share_workspaces(qmm):
    ex = ref.Experts(6, 128, 96, 32, 4, seed=24)
    w = on_gpu(qmm, ex)
    g = torch.Generator().manual_seed(24)
    ws = torch.zeros(max(qmm.qmm_moe_workspace_size(w, 9, 2), qmm.qmm_sample_workspace_size(9, 20000)), dtype=torch.uint8,
                     device=DEV)
    steps = []
    for n in (9, 2):
        x, logits = torch.randn(n, 128, generator=g).bfloat16(), torch.randn(n, 6, generator=g)
        z, u = draw(n, 20000, torch.bfloat16, seed=25 + n)
        want = layer(qmm, ex, x, logits, 2, w=w), sample(qmm, z, u, top_k=40, top_p=0.9)[0]
        s = qmm.Step()
        y, tokens = torch.empty(n, 128, dtype=torch.bfloat16, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
        kept = [t.to(DEV) for t in (x, logits, z, u)] + [torch.full((n,), 40, dtype=torch.int32, device=DEV),
                                                         torch.full((n,), 0.9, device=DEV)]
        s.add_moe(kept[0], w, y, ws, logits=kept[1], top_k=2)
        s.add_sample(kept[2], kept[3], tokens, ws, top_k=kept[4], top_p=kept[5])
        s.finalize()
        steps.append((s, y, tokens, want, kept))
    for _ in range(4):
        for s, y, tokens, want, _ in steps:
            y.zero_()
            tokens.zero_()
            s.launch()
        torch.cuda.synchronize()
        for s, y, tokens, want, _ in steps:
            assert torch.equal(y.cpu(), want[0]) and torch.equal(tokens.cpu(), want[1])
    for s, *_ in steps:
        s.close()
