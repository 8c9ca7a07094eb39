"""examples/sampled_decode.py: norms, projections of int8 codes, attention,
experts and sampling together, recorded and by direct calls."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import decode_ref as ref
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sampled_decode", os.path.join(ROOT, "examples", "sampled_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def small(example, **kw):
    return example.Decoder(**{**dict(vocab=1000, count=6, top_k=2, inter=96, hidden=256, q_heads=4, kv_heads=2, dim=64,
                                     layers=2, slots=6, pages=64, page_size=4, max_len=128), **kw})


def prompt(n, seed):
    return torch.randint(0, 1000, (n,), generator=torch.Generator().manual_seed(seed)).to(DEV)


def test_a_replayed_step_draws_what_direct_calls_draw(example):
    """Graph replays, the program's own work between them, against direct calls on
    a decoder of its own: the same tokens, streams and log-probabilities, bit for
    bit, over steps that feed each other."""
    from block_quantized_weight_matmulnbits_amd import qmm
    d, e = small(example), small(example)
    text = prompt(43, 0)
    first = d.prefill(0, text, 17)[-1]
    assert torch.equal(e.prefill(0, text, 17)[-1], first)
    slots = [1, 2, 4]
    d.fork(0, slots)
    e.fork(0, slots)
    step, b = d.decode_step(slots)
    b.x[0].copy_(d.embed(first.expand(3)))
    x = b.x[0].clone()
    seen = []
    for i in range(6):
        u = torch.rand(3, generator=torch.Generator().manual_seed(i)).to(DEV)
        b.uniform.copy_(u)
        step.launch()
        qmm.qmm_pages_reserve(e.pool, e.list(slots), e.list([1] * 3), e.status, e.pages_ws)
        c = e.batch([0, 1, 1, 0, 1, 0], 1)
        c.x[0].copy_(x)
        c.uniform.copy_(u)
        e.forward(c)
        torch.cuda.synchronize()
        for name in ("stream", "normed", "routed", "added", "logits", "drawn", "logprobs"):
            assert torch.equal(getattr(b, name), getattr(c, name)), (i, name)
        x = d.embed(b.drawn)
        b.x[0].copy_(x)
        seen.append(b.drawn.tolist())
    assert len({t for row in seen for t in row}) > 1 and all(0 <= t < 1000 for row in seen for t in row)
    assert d.status.tolist() == [0, 0] and d.pool.lens.tolist() == [43, 49, 49, 0, 49, 0]


def test_each_operator_of_a_pass_is_the_definitions(example):
    d = small(example, layers=1)
    text = prompt(21, 1)
    from block_quantized_weight_matmulnbits_amd import qmm
    qmm.qmm_pages_reserve(d.pool, d.list([3]), d.list([21]), d.status, d.pages_ws)
    b = d.batch([0, 0, 0, 21, 0, 0], 21)
    b.x[0].copy_(d.embed(text))
    b.uniform.copy_(torch.rand(21, generator=torch.Generator().manual_seed(2)))
    # The inputs of each operator, before the next call writes over them.
    kept = {}
    for at, (name, args, kw) in enumerate(d.calls(b)):
        before = {n: t.cpu() for n, t in kw.items() if isinstance(t, torch.Tensor)}
        inputs = [t.cpu() if isinstance(t, torch.Tensor) else t for t in args]
        getattr(qmm, "qmm_" + name)(*args, **kw)
        torch.cuda.synchronize()
        kept[at, name] = inputs, before, {n: t.cpu() for n, t in kw.items() if isinstance(t, torch.Tensor)}, \
            [t.cpu() if isinstance(t, torch.Tensor) else t for t in args]
    u = 2.0 ** -8
    for (at, name), (args, before, after, outs) in kept.items():
        if name == "rms_norm":
            h, y = ref.norm32(args[0], args[1], before.get("residual"), 1e-5, 0.0)
            if "h" in after:
                assert torch.equal(after["h"], h.bfloat16())
            if "codes" in after:
                q, s = ref.int8_of(y, 32)
                # 1/rms may round the other way where torch's sum of 64 bits does: a
                # step of 32 bits in y and a code at a tie.
                assert ((after["scales"] - s).abs() <= 2.0 ** -22 * s).all()
                assert (after["codes"].int() - q.int()).abs().max() <= 1
                assert (after["codes"] != q).float().mean() < 1e-3
            else:
                assert ((after["y"].double() - y.double()).abs() <= (u + 2.0 ** -22) * y.double().abs()).all()
        elif name == "gemm_compint8_quantized":
            want = torch.empty_like(outs[6]).to(DEV)
            p = d.qkv[0]
            qmm.qmm_gemm_compint8_quantized(args[0].to(DEV), args[1].to(DEV), p.B, None, None, None, want, 21, p.K, p.N, 32, 4)
            assert torch.equal(want.cpu(), outs[6]) and torch.isfinite(outs[6].float()).all()
        elif name == "moe":
            ids, w = ref.route(before["logits"], d.top_k, True)
            ex = ref.Experts(d.count, d.hidden, 96, 32, 4)
            t = {n: None if v is None else v.cpu() for n, v in d.experts[0].tensors.items()}
            ex.parts = [tuple(t[n + s] for s in ("", "_scales", "_zero_points")) for n in ("gate_up", "down")]
            want, bound = ref.moe(args[0], ex, ids, w, torch.bfloat16)
            assert (np.abs(outs[2].double().numpy() - want) <= bound).all()
        elif name == "sample":
            for r in range(21):
                allowed = ref.sample_allowed(args[0][r].double().numpy(), float(before["temperature"][r]), 0,
                                             float(before["top_p"][r]), 0, float(args[1][r]), d.vocab)
                assert int(outs[2][r]) in {t for t, _ in allowed}


def test_main_runs(example, capsys):
    example.main(prompt=100, samples=3, steps=4)
    assert "status [0, 0]" in capsys.readouterr().out
