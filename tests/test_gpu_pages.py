"""The pages' bookkeeping against plain Python: whole numbers, equal exactly."""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a)).to(DEV, dtype)


class Both:
    """A pool on the device and its plain twin."""

    def __init__(self, pages, page, slots, width, lengths, planes=3, shape=(40,), dtype=torch.int16,
                 seed=0, shared=(), room=64, padded=False):
        rng = np.random.default_rng(seed)
        order = list(rng.permutation(pages))
        table, lens, refs = np.full((slots, width), -1, np.int32), np.zeros(slots, np.int32), np.zeros(pages, np.int32)
        for s, n in lengths.items():
            need = -(-n // page)
            row = [int(order.pop()) for _ in range(need)]
            if s in shared:   # the first page of slot 0
                order.append(row[0])
                row[0] = int(table[0, 0])
            table[s, :need], lens[s] = row, n
            np.add.at(refs, row, 1)
        data = rng.integers(-100, 100, (planes, pages) + shape)
        self.plain = ref.Pool(data, refs, table, lens, page)
        self.data = torch.as_tensor(data).to(dtype).to(DEV)
        if padded:   # pages and planes of a larger buffer, off alignment
            whole = torch.zeros((planes, pages + 2) + (shape[0] + 3,), dtype=dtype, device=DEV)
            view = whole[:, 1:pages + 1, 1:shape[0] + 1]
            view.copy_(self.data)
            self.data = view
        self.refs, self.lens = dev(refs), dev(lens)
        self.table = dev(table)
        q = qmm()
        self.pool = q.PagePool(self.data, self.refs, self.table, self.lens, page)
        self.status = torch.zeros(2, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(q.qmm_pages_workspace_size(self.pool, room), dtype=torch.uint8, device=DEV)
        self.ws.fill_(0xA5)

    def same(self, what=""):
        torch.cuda.synchronize()
        for name in ("refs", "table", "lens", "data"):
            got = getattr(self, name).cpu().numpy()
            np.testing.assert_array_equal(got, getattr(self.plain, name), err_msg=f"{what} {name}")

    def free(self, seqs):
        qmm().qmm_pages_free(self.pool, dev(seqs))
        self.plain.free(seqs)

    def fork(self, parents, children):
        qmm().qmm_pages_fork(self.pool, dev(parents), dev(children), self.status, self.ws)
        self.plain.fork(parents, children)

    def reserve(self, seqs, grow):
        qmm().qmm_pages_reserve(self.pool, dev(seqs), dev(grow), self.status, self.ws)
        self.plain.reserve(seqs, grow)

    def state(self):
        torch.cuda.synchronize()
        return self.status.tolist()


@pytest.mark.parametrize("page", [1, 3, 16])
@pytest.mark.parametrize("shape,dtype", [((8,), torch.int16), ((40,), torch.int16), ((2, 3, 64), torch.int16),
                                         ((5,), torch.int8), ((6,), torch.int32), ((4096,), torch.int16)])
def test_a_turn_of_a_beam_search(page, shape, dtype):
    b = Both(120, page, 12, 40, {0: 17, 1: 16, 2: 1, 3: 31, 4: 5, 5: 9}, planes=2, shape=shape,
             dtype=dtype, seed=page)
    b.free([4, 5, 4, 7])
    b.same("free")
    b.fork([0, 1, 0, 2, 9], [4, 5, 6, 7, 8])
    b.same("fork")
    b.reserve([4, 0, 6, 9], [1, 3, 0, 8])
    b.same("reserve")
    assert b.state() == [0, 0]
    b.free([0, 6, 8])
    b.same("free again")
    b.fork([4], [0])
    b.same("fork again")


def test_many_forks_and_a_large_pool():
    lengths = {s: 3 + 5 * s % 97 for s in range(40)}
    b = Both(5000, 4, 1700, 32, lengths, planes=1, shape=(8,), room=1500)
    rng = np.random.default_rng(1)
    b.fork(rng.integers(0, 40, 1500).tolist(), list(range(100, 1600)))
    b.same("fork")
    b.reserve(list(range(100, 1600)), rng.integers(0, 5, 1500).tolist())
    b.same("reserve")
    assert b.state() == [0, 0]


@pytest.mark.parametrize("what", ["pages", "width", "twice", "range", "full", "parent", "negative"])
def test_a_list_is_served_whole_or_not_at_all(what):
    q = qmm()
    b = Both(14, 4, 8, 6, {0: 17, 1: 6, 2: 8}, shape=(8,))
    seqs, grow, code = [1, 2], [1, 5], 0
    if what == "pages":
        seqs, grow, code = [0, 1, 2, 5], [3, 14, 12, 4], 1
    if what == "width":
        seqs, grow, code = [1, 0], [1, 8], 2
    if what == "twice":
        seqs, grow, code = [1, 2, 1], [1, 1, 1], 3
    if what == "range":
        seqs, grow, code = [1, 8], [1, 1], 3
    if what == "negative":
        seqs, grow, code = [1, 2], [1, -1], 3
    if what == "full":   # a child that is not empty
        q.qmm_pages_fork(b.pool, dev([0, 0]), dev([5, 1]), b.status, b.ws)
        code = 3
    elif what == "parent":
        b.table[0, 2] = 99
        b.plain.table[0, 2] = 99
        q.qmm_pages_fork(b.pool, dev([1, 0]), dev([5, 6]), b.status, b.ws)
        code = 3
    else:
        q.qmm_pages_reserve(b.pool, dev(seqs), dev(grow), b.status, b.ws)
    b.same(what)
    state = b.state()
    assert state[0] == code
    if what == "pages":   # 9 pages are held; 0, 3, 3 and 1 more are needed
        assert state[1] == 2
    # The next call does nothing until the status is cleared.
    q.qmm_pages_fork(b.pool, dev([1]), dev([5]), b.status, b.ws)
    b.same("after")
    b.status.zero_()
    b.fork([1], [5])
    b.same("cleared")


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("pages,lengths", [(37, {0: 9, 1: 30, 3: 16, 4: 1}), (9, {}), (16, {0: 64}),
                                           (1500, {s: 37 for s in range(40)})])
def test_compact(pages, lengths, padded):
    q = qmm()
    b = Both(pages, 4, 45, 18, lengths, shape=(24,), seed=pages, shared=(3, 4), padded=padded)
    refs, table = torch.full_like(b.refs, 7), torch.full_like(b.table, 7)
    live = torch.full((1,), 7, dtype=torch.int32, device=DEV)
    old = b.refs.clone(), b.table.clone()
    q.qmm_pages_compact(b.pool, refs, table, live, b.ws)
    n = b.plain.compact()
    torch.cuda.synchronize()
    assert live.item() == n
    assert torch.equal(b.refs, old[0]) and torch.equal(b.table, old[1])
    np.testing.assert_array_equal(refs.cpu().numpy(), b.plain.refs)
    np.testing.assert_array_equal(table.cpu().numpy(), b.plain.table)
    np.testing.assert_array_equal(b.data.cpu().numpy(), b.plain.data)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("elems", [1, 7, 512, 5000])
def test_copy(elems, padded):
    q = qmm()
    b = Both(50, 4, 2, 2, {}, planes=5, shape=(elems,), padded=padded)
    order = np.random.default_rng(0).permutation(50)
    src, dst = order[:20].tolist(), order[20:40].tolist()
    q.qmm_pages_copy(q.PagePool(b.data), dev(src + [3, -1, 50]), dev(dst + [90, 4, 5]))
    b.plain.data[:, dst] = b.plain.data[:, src]
    b.same("copy")


def test_the_planes_may_be_any_stride_apart():
    """Keys and values of every layer as slices of larger tensors."""
    q = qmm()
    whole = torch.randint(-9, 9, (6, 30, 64), dtype=torch.int16, device=DEV)
    want = whole.clone()
    data = whole[::2]
    q.qmm_pages_copy(q.PagePool(data), dev([1, 2]), dev([11, 12]))
    want[::2, [11, 12]] = want[::2, [1, 2]]
    torch.cuda.synchronize()
    assert torch.equal(whole, want)


def test_reserve_replays_in_a_step():
    q = qmm()
    b = Both(60, 4, 6, 12, {0: 3, 1: 8, 2: 13}, shape=(8,))
    seqs, grow = dev([0, 1, 2]), dev([1, 1, 1])
    step = q.Step()
    step.add_pages_reserve(b.pool, seqs, grow, b.status, b.ws)
    step.finalize()
    for _ in range(6):
        step.launch()
        b.plain.reserve([0, 1, 2], [1, 1, 1])
        b.same("step")
    step.close()


@pytest.mark.parametrize("shape", [(0, 20, 8), (3, 20, 0)])
def test_a_pool_without_contents_keeps_its_tables(shape):
    q = qmm()
    b = Both(20, 4, 6, 5, {0: 9, 1: 4, 3: 16}, shape=(8,))
    b.pool = q.PagePool(torch.empty(shape, dtype=torch.int16, device=DEV), b.refs, b.table, b.lens, 4)
    b.fork([0], [2])
    b.plain.data = b.data.cpu().numpy()
    b.same("fork")
    refs, table = torch.empty_like(b.refs), torch.empty_like(b.table)
    live = torch.zeros(1, dtype=torch.int32, device=DEV)
    q.qmm_pages_compact(b.pool, refs, table, live, b.ws)
    torch.cuda.synchronize()
    assert live.item() == b.plain.compact()
    np.testing.assert_array_equal(refs.cpu().numpy(), b.plain.refs)
    np.testing.assert_array_equal(table.cpu().numpy(), b.plain.table)


def test_pages_past_32_bits_of_bytes():
    q = qmm()
    stride = (1 << 30) + 64                      # bytes between pages
    whole = torch.empty(6 * stride, dtype=torch.uint8, device=DEV)
    data = whole.as_strided((1, 6, 256), (6 * stride, stride, 1))
    data[0, 1] = 7
    data[0, 5] = 9
    q.qmm_pages_copy(q.PagePool(data), dev([5, 1]), dev([0, 4]))
    torch.cuda.synchronize()
    assert data[0, 0].eq(9).all() and data[0, 4].eq(7).all()
