"""examples/paged_decode.py: projections, rotary append, attention and the
pages' bookkeeping together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def small(example, **kw):
    return example.Decoder(**{**dict(hidden=256, q_heads=4, kv_heads=2, dim=64, slots=6, pages=64,
                                     page_size=4, max_len=128), **kw})


def hidden(n, width, seed):
    return torch.randn(n, width, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


def test_each_attention_of_a_pass_is_the_definitions(example):
    d = small(example, layers=1)
    d.prefill(2, hidden(37, d.hidden, 0), 16)
    counts = [0, 0, 21, 0, 0, 0]
    from block_quantized_weight_matmulnbits_amd import qmm
    qmm.qmm_pages_reserve(d.pool, d.list([2]), d.list([21]), d.status, d.pages_ws)
    b = d.batch(counts, 21)
    b.x[0].copy_(hidden(21, d.hidden, 1))
    d.forward(b)
    torch.cuda.synchronize()
    q = b.rows[:, :d.q_heads]   # turned in place
    table, lens = d.pool.table.cpu().numpy(), d.pool.lens.cpu().numpy()
    assert lens.tolist() == [0, 0, 58, 0, 0, 0]
    out, _, bound, _ = ref.attention(q, d.kv[0].k_pages, d.kv[0].v_pages, b.starts.cpu().numpy(), lens,
                                     table, ref.default_scale(d.dim))
    ref.assert_close(b.attended, out, ref.rounded(out, bound, torch.bfloat16), "attended")


def test_samples_go_on_as_their_parent_would(example):
    """Forked samples that see the parent's next tokens produce its outputs, bit
    for bit, whether stepped as graphs or by direct calls."""
    d = small(example, layers=2)
    prompt, tail = hidden(43, d.hidden, 2), hidden(6, d.hidden, 3)
    d.prefill(0, prompt, 43)
    d.fork(0, [3, 5])
    d.fork(3, [4])
    step, b = d.decode_step([0, 3, 4, 5])
    for t in tail:
        b.x[0].copy_(t.expand(4, -1))
        step.launch()
        torch.cuda.synchronize()
        y = b.x[-1]
        assert torch.isfinite(y.float()).all()
        for i in range(1, 4):
            assert torch.equal(y[i], y[0])
    assert d.status.tolist() == [0, 0]
    assert d.pool.lens.tolist() == [49, 0, 0, 49, 49, 49]
    # The same tokens by direct calls on a decoder of its own.
    e = small(example, layers=2)
    e.prefill(1, prompt, 43)
    e.fork(1, [0, 2, 4])
    from block_quantized_weight_matmulnbits_amd import qmm
    for t in tail:
        qmm.qmm_pages_reserve(e.pool, e.list([0, 1, 2, 4]), e.list([1] * 4), e.status, e.pages_ws)
        c = e.batch([1, 1, 1, 0, 1, 0], 1)
        c.x[0].copy_(t.expand(4, -1))
        e.forward(c)
    torch.cuda.synchronize()
    assert torch.equal(c.x[-1], y)


def test_a_moved_cache_gives_the_same_outputs(example):
    d = small(example, layers=1)
    d.prefill(0, hidden(30, d.hidden, 4), 30)
    d.prefill(1, hidden(25, d.hidden, 5), 25)
    d.fork(1, [2])
    d.free([0])
    used = int((d.pool.refs > 0).sum())
    before = d.pool.table.clone()
    assert d.compact() == used
    assert not torch.equal(before, d.pool.table) and int(d.pool.table.max()) < used
    step, b = d.decode_step([1, 2])
    b.x[0].copy_(hidden(1, d.hidden, 6).expand(2, -1))
    step.launch()
    torch.cuda.synchronize()
    # The same without the move.
    e = small(example, layers=1)
    e.prefill(0, hidden(30, d.hidden, 4), 30)
    e.prefill(1, hidden(25, d.hidden, 5), 25)
    e.fork(1, [2])
    step2, c = e.decode_step([1, 2])
    c.x[0].copy_(b.x[0])
    step2.launch()
    torch.cuda.synchronize()
    assert torch.equal(b.x[-1], c.x[-1])


def test_main_runs(example, capsys):
    example.main(prompt=100, samples=3, steps=4)
    assert "status [0, 0]" in capsys.readouterr().out
