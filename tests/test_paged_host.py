"""The paged operators without a GPU: the plain forms against worked values,
the entry points' refusals, and the sizes of workspaces."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref

FAKE = 0x10000   # never dereferenced: validation fails before any device work


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


# -- the plain forms ---------------------------------------------------------

def test_a_quarter_turn():
    q = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    kp = torch.zeros(1, 1, 4, 5)
    args = (q, 10 * q, 100 * q, kp, kp, np.array([0, 1]), np.array([2]), np.array([[0]]))
    out, k, v, _, _ = ref.rope(*args, np.array([math.pi / 2, 0.0]))
    np.testing.assert_allclose(out[0, 0], [-3, 2, 1, 4, 5], atol=1e-15)
    np.testing.assert_allclose(k[0, 0, 1], [-30, 20, 10, 40, 50], atol=1e-14)
    np.testing.assert_array_equal(v[0, 0, 1], [100, 200, 300, 400, 500])
    assert not k[0, 0, [0, 2, 3]].any()
    out, _, _, _, _ = ref.rope(*args, np.array([math.pi / 2, 0.0]), interleaved=True, factor=2.0)
    np.testing.assert_allclose(out[0, 0], [-4, 2, 6, 8, 5], atol=1e-15)
    out, _, _, _, _ = ref.rope(*args, np.array([math.pi / 2]), interleaved=True, positions=np.array([3]))
    np.testing.assert_allclose(out[0, 0], [2, -1, 3, 4, 5], atol=1e-15)


def test_attention_worked_values():
    q = torch.tensor([[[math.log(2.0)]], [[math.log(3.0)]]])
    kp = torch.tensor([[[[0.0], [1.0]]], [[[2.0], [float("nan")]]]])
    vp = torch.tensor([[[[1.0], [10.0]]], [[[100.0], [float("nan")]]]])
    args = (q, kp, vp, np.array([0, 2]), np.array([3]), np.array([[0, 1]]), 1.0)
    out, lse, _, _ = ref.attention(*args)
    np.testing.assert_allclose(out[:, 0, 0], [(1 + 20) / 3, (1 + 30 + 900) / 13], rtol=1e-6)
    np.testing.assert_allclose(np.exp(lse[:, 0]), [3, 13], rtol=1e-6)
    out, _, _, _ = ref.attention(*args, window=1)
    np.testing.assert_allclose(out[:, 0, 0], [10, 100])
    out, _, _, _ = ref.attention(*args, causal=False)
    np.testing.assert_allclose(out[0, 0, 0], (1 + 20 + 400) / 7, rtol=1e-6)
    out, lse, _, _ = ref.attention(*args[:4], np.array([1]), *args[5:])   # more tokens than keys
    assert out[0, 0, 0] == 0 and lse[0, 0] == -np.inf and out[1, 0, 0] == 1


def test_pool_worked_values():
    p = ref.Pool(np.arange(6)[None, :, None], [1, 0, 1, 0, 0, 0], [[2, 0, -1], [-1, -1, -1]], [3, 0], 2)
    p.fork([0], [1])
    assert p.table.tolist() == [[2, 0, -1], [2, 1, -1]] and p.refs.tolist() == [1, 1, 2, 0, 0, 0]
    assert p.data[0, 1, 0] == 0 and p.lens.tolist() == [3, 3]
    p.reserve([1], [2])
    assert p.table[1].tolist() == [2, 1, 3] and p.lens[1] == 5
    p.free([0])
    assert p.refs.tolist() == [0, 1, 1, 1, 0, 0]
    assert p.compact() == 3
    assert p.table[1].tolist() == [2, 1, 0] and p.data[0, 0, 0] == 3


# -- refusals at the C boundary ----------------------------------------------

class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int)]


def structs(qmm, **kw):
    a = dict(k=FAKE, v=FAKE, ks=(65536, 2048, 128), vs=(65536, 2048, 128), pages=64, dtype=2, kv=8,
             page=16, dim=128, starts=FAKE, lens=FAKE, table=FAKE, tstride=32, seqs=4, tokens=4,
             width=32, max_new=1, max_len=500, q=FAKE, qt=6144, qh=128, heads=32, out=FAKE,
             oheads=32, kheads=8)
    a.update(kw)
    kv = qmm._PagedKV(a["k"], a["v"], *a["ks"], *a["vs"], a["pages"], a["dtype"], a["kv"], a["page"], a["dim"])
    batch = qmm._PagedBatch(a["starts"], a["lens"], a["table"], a["tstride"], a["seqs"], a["tokens"],
                            a["width"], a["max_new"], a["max_len"])
    q = Heads(a["q"], a["qt"], a["qh"], a["heads"])
    out = Heads(a["out"], 4096, 128, a["oheads"])
    k = Heads(FAKE, 6144, 128, a["kheads"])
    return kv, batch, q, out, k


def attend(qmm, scale=0.1, window=0, cap=0.0, ws=FAKE, ws_bytes=1 << 30, lse=None, **kw):
    kv, batch, q, out, _ = structs(qmm, **kw)
    r = ctypes.byref
    return qmm.lib.qmm_paged_attention(r(q), r(kv), r(batch), r(out), lse, scale, 1, window, cap, ws,
                                       ws_bytes, None)


COMMON = [
    (dict(dtype=7), -1, "not a qmm_dtype"),
    (dict(pages=0), -1, "kv_heads, page_size and head_dim"),
    (dict(page=0), -1, "kv_heads, page_size and head_dim"),
    (dict(k=None), -1, "non-null"),
    (dict(ks=(-1, 2048, 128)), -1, "stride"),
    (dict(q=None), -1, "q must be a non-null"),
    (dict(q=FAKE + 1), -1, "aligned to its element size"),
    (dict(oheads=31), -1, "out has 31 heads"),
    (dict(starts=None), -1, "starts, lens and table"),
    (dict(lens=FAKE + 2), -1, "4-byte aligned"),
    (dict(tokens=-1), -1, "in 0 .. 2^30"),
    (dict(max_len=1 << 31), -1, "in 0 .. 2^30"),
]


@pytest.mark.parametrize("kw,code,needle", COMMON + [
    (dict(heads=30, oheads=30), -1, "do not divide"),
    (dict(dim=100), -2, "multiple of 8"),
    (dict(dim=264), -2, "at most 256"),
    (dict(dim=6, dtype=0), -2, "multiple of 4"),
    (dict(k=FAKE + 8), -1, "16-byte"),
    (dict(vs=(65536, 2048, 124)), -1, "16-byte"),
    (dict(window=-1), -1, "window must be >= 0"),
    (dict(cap=-1.0), -1, "softcap"),
    (dict(scale=float("nan")), -1, "scale must be finite"),
    (dict(lse=FAKE + 2), -1, "lse must be"),
    (dict(ws=None), -3, "workspace"),
    (dict(ws_bytes=100), -3, "workspace"),
    (dict(ws=FAKE + 64), -3, "256-byte aligned"),
    (dict(max_new=1 << 29), -2, "too large for one launch"),
])
def test_attention_rejects(qmm, kw, code, needle):
    assert attend(qmm, **kw) == code
    assert needle in qmm.qmm_last_error(), qmm.qmm_last_error()


def turn(qmm, freq=FAKE, half=64, pos=None, **kw):
    kv, batch, q, out, k = structs(qmm, **kw)
    r = ctypes.byref
    return qmm.lib.qmm_rope_append(r(q), r(k), r(k), r(out), r(kv), r(batch), freq, half, 0, 1.0, pos, None)


@pytest.mark.parametrize("kw,code,needle", COMMON + [
    (dict(kheads=4), -1, "k has 4 heads"),
    (dict(half=65), -1, "do not fit a head"),
    (dict(half=-1), -1, "do not fit a head"),
    (dict(freq=None), -1, "inv_freq"),
    (dict(freq=FAKE + 4), -1, "inv_freq"),
    (dict(pos=FAKE + 2), -1, "positions"),
    (dict(dim=513), -2, "even and at most 512"),
])
def test_rope_rejects(qmm, kw, code, needle):
    assert turn(qmm, **kw) == code
    assert needle in qmm.qmm_last_error(), qmm.qmm_last_error()


def pool_of(qmm, **kw):
    a = dict(data=FAKE, planes=2, pages=64, bytes=256, plane=1 << 14, stride=256, refs=FAKE, table=FAKE,
             lens=FAKE, tstride=8, slots=16, width=8, page=16)
    a.update(kw)
    return qmm._PagePool(a["data"], a["planes"], a["pages"], a["bytes"], a["plane"], a["stride"],
                         a["refs"], a["table"], a["lens"], a["tstride"], a["slots"], a["width"], a["page"])


@pytest.mark.parametrize("kw,code,needle", [
    (dict(pages=0), -1, "pages must be in"),
    (dict(bytes=-1), -1, "planes, page_bytes and strides"),
    (dict(planes=1 << 27), -2, "below 2^32"),
    (dict(data=None), -1, "data must be a non-null"),
    (dict(refs=None), -1, "refs, table and lens"),
    (dict(slots=0), -1, "must be positive"),
    (dict(slots=(1 << 18) + 1), -1, "slots at most"),
    (dict(width=1 << 21), -1, "must be positive"),
    (dict(slots=1 << 18, width=1 << 15), -2, "slots x width"),
    (dict(table=FAKE + 1), -1, "4-byte aligned"),
])
def test_pages_reject_a_bad_pool(qmm, kw, code, needle):
    r = ctypes.byref(pool_of(qmm, **kw))
    assert qmm.lib.qmm_pages_fork(r, FAKE, FAKE, 2, FAKE, FAKE, 1 << 30, None) == code
    assert needle in qmm.qmm_last_error(), qmm.qmm_last_error()
    assert qmm.lib.qmm_pages_compact(r, FAKE + 64, FAKE + 64, FAKE, FAKE, 1 << 30, None) == code


def test_pages_reject_bad_lists_and_workspaces(qmm):
    r, lib = ctypes.byref(pool_of(qmm)), qmm.lib
    size = lib.qmm_pages_workspace_size(r, 2)
    assert size % 256 == 0 and size >= 4 * (2 * 64 + 64 + 4)
    for call, needle in [
            (lambda: lib.qmm_pages_free(r, None, 2, None), "seqs must be"),
            (lambda: lib.qmm_pages_free(r, FAKE, -1, None), "count must be"),
            (lambda: lib.qmm_pages_fork(r, FAKE, FAKE + 2, 2, FAKE, FAKE, size, None), "children must be"),
            (lambda: lib.qmm_pages_reserve(r, FAKE, FAKE, 2, None, FAKE, size, None), "status must be"),
            (lambda: lib.qmm_pages_copy(r, FAKE, None, 2, None), "dst must be"),
            (lambda: lib.qmm_pages_compact(r, FAKE, FAKE + 64, FAKE, FAKE, size, None), "must not be the pool's own"),
            (lambda: lib.qmm_pages_compact(r, None, FAKE + 64, FAKE, FAKE, size, None), "non-null")]:
        assert call() == -1
        assert needle in qmm.qmm_last_error(), qmm.qmm_last_error()
    assert lib.qmm_pages_fork(r, FAKE, FAKE, 2, FAKE, FAKE, size - 256, None) == -3
    assert lib.qmm_pages_reserve(r, FAKE, FAKE, 2, FAKE, None, size, None) == -3
    # Nothing to do is no error.
    assert lib.qmm_pages_free(r, None, 0, None) == 0
    assert lib.qmm_pages_copy(r, None, None, 0, None) == 0


def test_a_batch_without_tokens_is_a_noop(qmm):
    assert attend(qmm, tokens=0, q=None, out=None, ws=None) == 0
    assert turn(qmm, tokens=0, q=None, out=None) == 0


@pytest.mark.parametrize("seqs,max_new,max_len,H,KV,D", [(1, 1, 1, 1, 1, 64), (64, 1, 8192, 32, 8, 128),
                                                         (2, 1, 131072, 32, 8, 128), (1, 4096, 16384, 32, 8, 128),
                                                         (3, 5, 129, 28, 4, 80), (5000, 1, 100, 8, 8, 256)])
def test_attention_workspace_size(qmm, seqs, max_new, max_len, H, KV, D):
    _, batch, _, _, _ = structs(qmm, seqs=seqs, tokens=seqs * max_new, max_new=max_new, max_len=max_len)
    n = qmm.lib.qmm_paged_attention_workspace_size(ctypes.byref(batch), H, KV, D)
    assert n >= 256 and n % 256 == 0 and n < 1 << 30
    assert qmm.lib.qmm_paged_attention_workspace_size(ctypes.byref(batch), H, H + 1, D) == 0


def test_the_binding_packs_the_struct(qmm):
    raw = qmm._pack_heads(FAKE, 6144, 128, 32)
    assert raw == bytes(Heads(FAKE, 6144, 128, 32))


# -- refusals of the binding -------------------------------------------------

def test_the_binding_rejects_what_the_tensors_show(qmm):
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)   # noqa: E731
    kv = qmm.PagedKV(kp, kp.clone())
    batch = qmm.PagedBatch(i32(3), i32(2), i32(2, 4), 5, 3, 64)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    bad = [
        lambda: qmm.PagedKV(kp, kp[:, :, :8]),
        lambda: qmm.PagedKV(kp, kp.float()),
        lambda: qmm.PagedKV(kp.double(), kp.double()),
        lambda: qmm.PagedKV(kp.transpose(2, 3), kp.transpose(2, 3)),
        lambda: qmm.PagedBatch(i32(2), i32(2), i32(2, 4), 5, 3, 64),
        lambda: qmm.PagedBatch(i32(3), i32(2).long(), i32(2, 4), 5, 3, 64),
        lambda: qmm.PagedBatch(i32(3), i32(2), i32(4, 2).t(), 5, 3, 64),
        lambda: qmm.qmm_paged_attention(q[:4], kv, batch, q, ws),
        lambda: qmm.qmm_paged_attention(q.float(), kv, batch, q, ws),
        lambda: qmm.qmm_paged_attention(q, kv, batch, q[:, :2], ws),
        lambda: qmm.qmm_paged_attention(q, kv, batch, q, ws, lse=torch.zeros(5, 5)),
        lambda: qmm.qmm_rope_append(q, q[:, :1], q[:, :2], q, kv, batch, torch.zeros(32).double()),
        lambda: qmm.qmm_rope_append(q, q[:, :2], q[:, :2], q, kv, batch, torch.zeros(32)),
        lambda: qmm.qmm_rope_append(q, q[:, :2], q[:, :2], q, kv, batch, torch.zeros(32).double(),
                                    positions=i32(4)),
        lambda: qmm.PagePool(kp, i32(3), i32(2, 2), i32(2), 16),
        lambda: qmm.PagePool(kp, i32(2), i32(2, 2), i32(3), 16),
        lambda: qmm.PagePool(kp.transpose(2, 3)),
        lambda: qmm.qmm_pages_copy(qmm.PagePool(kp), i32(2), i32(3)),
        lambda: qmm.qmm_pages_free(qmm.PagePool(kp), i32(2).long()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
