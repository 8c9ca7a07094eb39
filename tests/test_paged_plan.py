"""The plan of paged attention without a GPU: the entry points and the plan are
compiled for the host, with launchers that note what they were asked for."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "block_quantized_weight_matmulnbits_amd", "csrc")
FAKE = 1 << 20   # never dereferenced: no launcher here touches memory

STUBS = r"""
#include <string>
#include "paged.h"
#include "qmm_internal.h"
static std::string message;
static int64_t note[6];   // bytes used past the workspace's start, workgroups, threads, parts, joined
static constexpr int64_t BASE = 1 << 20;
namespace qmm {
int set_error(int code, const char* m) { message = m; return code; }
static int width(int d) { return d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : d <= 192 ? 192 : 256; }
static void most(int64_t& x, int64_t y) { if (y > x) x = y; }
static void parts(const AttnArgs& a, int64_t n) {
  const int64_t rows = (int64_t)a.c.tokens * a.q_heads;
  most(note[3], n);
  if (n <= 1) return;
  const int64_t count = (int64_t)a.part_count, stats = (int64_t)a.part_stats, out = (int64_t)a.part_out;
  // The three arrays lie one after another.
  if (count < BASE || count + rows * 4 > stats || stats + rows * n * 8 > out) note[0] = INT64_MAX;
  most(note[0], out + rows * n * width(a.c.dim) * 4 - BASE);
}
static void grid(int64_t groups, int64_t threads) {
  most(note[1], groups);
  most(note[2], groups * threads);
}
hipError_t launch_rope_append(const RopeArgs&) { return hipSuccess; }
static hipError_t rows(const AttnArgs& a, const RowsPlan& p) {
  parts(a, p.splits);
  grid((int64_t)a.c.seqs * p.row_tiles * a.c.kv_heads * p.splits, 256);
  return hipSuccess;
}
static hipError_t tile(const AttnArgs& a, const TilePlan& p, const RowsPlan& few) {
  parts(a, p.splits > few.splits ? p.splits : few.splits);
  grid((int64_t)p.few_groups + (int64_t)p.tiles * a.c.kv_heads, 256 * p.blocks);
  if (p.few_groups != (p.skip_upto > 0 ? (int64_t)a.c.seqs * few.row_tiles * a.c.kv_heads * few.splits : 0))
    note[1] = INT64_MAX;
  return hipSuccess;
}
hipError_t launch_rows_f32(const AttnArgs& a, const RowsPlan& p, int, int) { return rows(a, p); }
hipError_t launch_rows_f16(const AttnArgs& a, const RowsPlan& p, int, int) { return rows(a, p); }
hipError_t launch_rows_bf16(const AttnArgs& a, const RowsPlan& p, int, int) { return rows(a, p); }
hipError_t launch_tile_f16(const AttnArgs& a, const TilePlan& p, const RowsPlan& f) { return tile(a, p, f); }
hipError_t launch_tile_bf16(const AttnArgs& a, const TilePlan& p, const RowsPlan& f) { return tile(a, p, f); }
hipError_t launch_join(const AttnArgs& a, int, int splits) {
  const int64_t rows = (int64_t)a.c.tokens * a.q_heads, lanes = a.c.dim <= 64 ? 16 : a.c.dim <= 128 ? 32 : 64;
  parts(a, splits);
  most(note[2], rows <= 512 ? rows * 1024 : rows <= 4096 ? rows * 256 : (rows * lanes + 255) / 256 * 256);
  note[4] = splits;
  return hipSuccess;
}
size_t pages_workspace_bytes(int64_t, int64_t) { return 0; }
hipError_t launch_pages_free(const PoolArgs&, const int32_t*, int) { return hipSuccess; }
hipError_t launch_pages_fork(const PoolArgs&, const int32_t*, const int32_t*, int, int32_t*) { return hipSuccess; }
hipError_t launch_pages_reserve(const PoolArgs&, const int32_t*, const int32_t*, int, int32_t*) { return hipSuccess; }
hipError_t launch_pages_copy(const PoolArgs&, const int32_t*, const int32_t*, int) { return hipSuccess; }
hipError_t launch_pages_compact(const PoolArgs&, int32_t*, int32_t*, int64_t, int32_t*) { return hipSuccess; }
}
extern "C" const char* hipGetErrorString(hipError_t) { return "an error"; }
extern "C" const char* noted(int64_t* out) {
  for (int i = 0; i < 6; ++i) { out[i] = note[i]; note[i] = 0; }
  return message.c_str();
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from block_quantized_weight_matmulnbits_amd import qmm
    d = tmp_path_factory.mktemp("plan")
    (d / "stubs.cpp").write_text(STUBS)
    lib = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    str(d / "stubs.cpp"), os.path.join(CSRC, "paged_api.cpp"),
                    os.path.join(CSRC, "paged_attn.cpp"), "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    for name in ("qmm_paged_attention", "qmm_paged_attention_workspace_size", "qmm_rope_append",
                 "qmm_pages_free"):
        fn = getattr(so, name)
        fn.argtypes, fn.restype = qmm._SIGS[name]
    so.noted.restype = ctypes.c_char_p
    return Plan(so, qmm)


class Plan:
    def __init__(self, so, qmm):
        self.so, self.qmm = so, qmm

    def structs(self, c):
        m, pad = self.qmm, c["kv"] * 16 * c["dim"]
        kv = m._PagedKV(FAKE, FAKE, pad, 16 * c["dim"], c["dim"], pad, 16 * c["dim"], c["dim"], 64,
                        c["dtype"], c["kv"], 16, c["dim"])
        batch = m._PagedBatch(FAKE, FAKE, FAKE, 1 << 16, c["seqs"], c["tokens"], 1 << 16, c["max_new"],
                              c["max_len"])
        return kv, batch

    def size(self, c):
        batch = self.structs(c)[1]
        return self.so.qmm_paged_attention_workspace_size(ctypes.byref(batch), c["heads"], c["kv"], c["dim"])

    def attend(self, **c):
        """(status, size the library asks for, what the launches were asked for)."""
        c = dict(dict(dtype=0, heads=32, kv=8, dim=128, seqs=1, max_new=1, max_len=1000, window=0, causal=1,
                      scale=0.1, cap=0.0), **c)
        c.setdefault("tokens", c["seqs"] * c["max_new"])
        kv, batch = self.structs(c)
        r = ctypes.byref
        need = self.size(c)
        rows = self.qmm._pack_heads(FAKE, c["heads"] * c["dim"], c["dim"], c["heads"])
        status = self.so.qmm_paged_attention(rows, r(kv), r(batch), rows, None, c["scale"], c["causal"],
                                             c["window"], c["cap"], FAKE, max(need, 1), None)
        out = (ctypes.c_int64 * 6)()
        text = self.so.noted(out).decode()
        return status, need, dict(bytes=out[0], groups=out[1], threads=out[2], parts=out[3], joined=out[4],
                                  message=text)


def fits(plan, **c):
    status, need, did = plan.attend(**c)
    assert status == 0, (c, did)
    assert did["bytes"] <= need, f"{c}: {did['bytes']} bytes are used of {need}"
    assert did["joined"] == (did["parts"] if did["parts"] > 1 else 0), (c, did)


@pytest.mark.parametrize("kw", [dict(max_new=2048, max_len=4097), dict(max_new=2048, max_len=8192),
                                dict(max_new=4096, max_len=8192), dict(max_new=8192, max_len=8192),
                                dict(seqs=4, max_new=1024, max_len=16384),
                                dict(seqs=256, max_len=8192, heads=8, dim=256)])
def test_f32_prompts_keep_to_their_workspace(plan, kw):
    fits(plan, **kw)


def test_every_plan_keeps_to_its_workspace(plan):
    """Types, widths, groups and counts on both sides of every limit of the
    plan, with windows, bounds above the batch and a scale of 0."""
    heads = [(8, 8), (32, 8), (28, 4), (16, 1), (66, 2)]
    for dtype, (h, kv), dim in itertools.product([0, 1, 2], heads, [64, 96, 128, 200]):
        for seqs, new in [(1, 1), (1, 33), (1, 500), (1, 2048), (3, 5), (4, 1024), (63, 1), (64, 4), (257, 1),
                          (2100, 1)]:
            for length in [1, 1500, 2500, 4097, 20000, 131072]:
                for window in (0, 900):
                    fits(plan, dtype=dtype, heads=h, kv=kv, dim=dim, seqs=seqs, max_new=new, max_len=length,
                         window=window)


def test_random_plans_keep_to_their_workspace(plan):
    rng = random.Random(11)

    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    for _ in range(20000):
        kv, group = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 40])
        seqs, new = spread(1, 600), spread(1, 3000)
        tokens = seqs * new if rng.random() < 0.5 else rng.randint(1, seqs * new)
        if tokens * kv * group > 1 << 25:   # past that the join may be too large for a launch
            continue
        fits(plan, dtype=rng.randint(0, 2), heads=kv * group, kv=kv, dim=8 * rng.randint(1, 32), seqs=seqs,
             max_new=new, tokens=tokens, max_len=spread(1, 300000), causal=rng.randint(0, 1),
             window=rng.choice([0, 0, spread(1, 20000)]), scale=rng.choice([0.1, 0.1, 0.0, -0.1]),
             cap=rng.choice([0.0, 30.0]))


def test_a_smaller_workspace_is_refused(plan):
    for c in (dict(max_new=600, max_len=9000), dict(seqs=3, max_len=9000), dict(dtype=2, seqs=3, max_len=9000)):
        c = dict(dict(dtype=0, heads=32, kv=8, dim=128, seqs=1, max_new=1, window=0, causal=1), **c)
        c["tokens"] = c["seqs"] * c["max_new"]
        kv, batch = plan.structs(c)
        rows = plan.qmm._pack_heads(FAKE, 4096, 128, 32)
        need = plan.size(c)
        r = ctypes.byref
        status = plan.so.qmm_paged_attention(rows, r(kv), r(batch), rows, None, 0.1, 1, 0, 0.0, FAKE, need - 1, None)
        assert status == plan.qmm.QMM_ERR_WORKSPACE
        assert plan.so.noted((ctypes.c_int64 * 6)()).decode().find(str(need)) > 0


LAUNCH = 1 << 32   # a launch has fewer threads


@pytest.mark.parametrize("kw", [
    dict(dtype=2, seqs=1 << 20, heads=16, kv=16),                                    # single tokens
    dict(dtype=2, seqs=1 << 23, tokens=(1 << 23) + 63, max_new=64, heads=4, kv=1, max_len=131072),
    dict(dtype=0, seqs=1 << 16, tokens=1 << 20, max_new=1200, heads=8, kv=8),         # bounds above the batch
    dict(dtype=2, seqs=40, tokens=1 << 22, max_new=1 << 21, heads=64, kv=64, dim=256, max_len=1 << 21),
])
def test_a_call_that_is_too_large_for_a_launch_says_so(plan, kw):
    status, _, did = plan.attend(**kw)
    assert status == plan.qmm.QMM_ERR_UNSUPPORTED and "too large for one launch" in did["message"], (status, did)
    assert did["threads"] == 0   # nothing was launched


def test_launches_have_fewer_than_2_to_the_32_threads(plan):
    rng = random.Random(5)
    served = refused = 0
    for _ in range(4000):
        kv, group = rng.choice([1, 8, 32]), rng.choice([1, 4, 16])
        seqs, new = int(2 ** rng.uniform(8, 24)), int(2 ** rng.uniform(0, 9))
        tokens = seqs * new if rng.random() < 0.3 else seqs + rng.randint(0, new)
        if tokens >= 1 << 30:
            continue
        status, _, did = plan.attend(dtype=rng.randint(0, 2), heads=kv * group, kv=kv, dim=rng.choice([64, 128, 256]),
                                     seqs=seqs, tokens=tokens, max_new=new, max_len=int(2 ** rng.uniform(4, 18)))
        assert did["threads"] < LAUNCH and did["groups"] >= 0
        assert status in (0, plan.qmm.QMM_ERR_UNSUPPORTED)
        served, refused = served + (status == 0), refused + (status != 0)
    assert served > 500 and refused > 500


def test_rows_and_lists_that_are_too_long_for_a_launch(plan):
    so, r = plan.so, ctypes.byref
    c = dict(dtype=2, heads=8, kv=8, dim=64, seqs=4, tokens=1 << 26, max_new=1 << 25, max_len=1 << 25)
    kv, batch = plan.structs(c)
    rows = plan.qmm._pack_heads(FAKE, 512, 64, 8)
    out = (ctypes.c_int64 * 6)()
    turn = lambda: so.qmm_rope_append(rows, rows, rows, rows, r(kv), r(batch), FAKE, 32, 0, 1.0, None, None)  # noqa: E731
    assert turn() == plan.qmm.QMM_ERR_UNSUPPORTED
    assert "2^26" in so.noted(out).decode()
    batch.tokens -= 1
    assert turn() == 0
    pool = plan.qmm._PagePool(FAKE, 2, 64, 256, 1 << 14, 256, FAKE, FAKE, FAKE, 8, 16, 8, 16)
    assert so.qmm_pages_free(r(pool), FAKE, 1 << 24, None) == plan.qmm.QMM_ERR_INVALID_ARG
    assert "count must be" in so.noted(out).decode()
    assert so.qmm_pages_free(r(pool), FAKE, (1 << 24) - 1, None) == 0
