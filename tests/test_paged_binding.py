"""What the binding of the paged operators refuses before the library is called:
tensors that are not on the GPU of the cache, and a pool without tables."""
import pytest
import torch


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_weight_matmulnbits_amd import qmm as q
    return q


class OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU 0 (its memory is never used: every
    call here is refused first)."""

    def get_device(self):
        return 0


def there(t):
    return t.as_subclass(OnGpu)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def rows(heads):
    return torch.zeros(5, heads, 64, dtype=torch.bfloat16)


def arguments(qmm, put):
    """Every tensor of the calls by name, with ``put(name, tensor)`` deciding
    where it is, and the calls."""
    t = {n: put(n, x) for n, x in dict(
        q=rows(4), k=rows(2), v=rows(2), out=rows(4), inv_freq=torch.zeros(32).double(), positions=i32(5),
        lse=torch.zeros(5, 4), workspace=torch.zeros(1 << 16, dtype=torch.uint8), seqs=i32(2), grow=i32(2),
        parents=i32(2), children=i32(2), src=i32(2), dst=i32(2), status=i32(2), refs_out=i32(4),
        table_out=i32(2, 4), live=i32(1)).items()}
    pages = put("cache", torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    kv = qmm.PagedKV(pages, pages)
    batch = qmm.PagedBatch(*(put("batch", x) for x in (i32(3), i32(2), i32(2, 4))), 5, 3, 64)
    pool = qmm.PagePool(put("cache", torch.zeros(2, 4, 64)), *(put("cache", x) for x in (i32(4), i32(2, 4), i32(2))), 16)
    calls = {
        "rope": lambda: qmm.qmm_rope_append(t["q"], t["k"], t["v"], t["out"], kv, batch, t["inv_freq"],
                                             positions=t["positions"]),
        "attention": lambda: qmm.qmm_paged_attention(t["q"], kv, batch, t["out"], t["workspace"], lse=t["lse"]),
        "free": lambda: qmm.qmm_pages_free(pool, t["seqs"]),
        "fork": lambda: qmm.qmm_pages_fork(pool, t["parents"], t["children"], t["status"], t["workspace"]),
        "reserve": lambda: qmm.qmm_pages_reserve(pool, t["seqs"], t["grow"], t["status"], t["workspace"]),
        "copy": lambda: qmm.qmm_pages_copy(pool, t["src"], t["dst"]),
        "compact": lambda: qmm.qmm_pages_compact(pool, t["refs_out"], t["table_out"], t["live"], t["workspace"]),
    }
    return calls


NAMES = [(call, name) for call, names in [
    ("rope", "q k v out batch inv_freq positions"), ("attention", "q batch out workspace lse"), ("free", "seqs"),
    ("fork", "parents children status workspace"), ("reserve", "seqs grow status workspace"), ("copy", "src dst"),
    ("compact", "refs_out table_out live workspace")] for name in names.split()]


@pytest.mark.parametrize("call,name", NAMES)
def test_a_tensor_off_the_caches_gpu_is_refused(qmm, call, name):
    calls = arguments(qmm, lambda n, x: x if n == name else there(x))
    with pytest.raises(ValueError, match=f"{name} is on cpu, the cache on GPU 0"):
        calls[call]()


@pytest.mark.parametrize("call", ["rope", "attention", "free", "fork", "reserve", "copy", "compact"])
def test_a_cache_on_the_host_is_refused(qmm, call):
    calls = arguments(qmm, lambda n, x: x)
    with pytest.raises(ValueError, match="must be on a GPU"):
        calls[call]()


def test_recorded_calls_refuse_the_same(qmm):
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    kv = qmm.PagedKV(there(pages), there(pages))
    batch = qmm.PagedBatch(there(i32(3)), there(i32(2)), there(i32(2, 4)), 5, 3, 64)
    pool = qmm.PagePool(there(torch.zeros(2, 4, 64)), there(i32(4)), there(i32(2, 4)), there(i32(2)), 16)
    ws, freq = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(32).double()
    q, k = there(rows(4)), there(rows(2))
    step = qmm.Step()
    with pytest.raises(ValueError, match="workspace is on cpu"):
        step.add_paged_attention(q, kv, batch, q, ws)
    with pytest.raises(ValueError, match="inv_freq is on cpu"):
        step.add_rope_append(q, k, k, q, kv, batch, freq)
    with pytest.raises(ValueError, match="grow is on cpu"):
        step.add_pages_reserve(pool, there(i32(2)), i32(2), there(i32(2)), there(ws))
    step.close()


def test_compaction_of_a_pool_without_tables_is_refused(qmm):
    pool = qmm.PagePool(there(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)))
    with pytest.raises(qmm.QmmError, match="refs, table and lens must be non-null"):
        qmm.qmm_pages_compact(pool, there(i32(4)), there(i32(2, 4)), there(i32(1)),
                              there(torch.zeros(1 << 16, dtype=torch.uint8)), stream=0)
