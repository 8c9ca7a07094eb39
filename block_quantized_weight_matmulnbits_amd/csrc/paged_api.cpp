// paged_api.cpp -- the extern "C" entry points of the paged cache declared in
// include/qmm.h: arguments are validated on the host (errors say what, why and
// how to fix), then the launchers of rope.hip, paged_attn.cpp and pages.hip
// enqueue the work.  Nothing here allocates device memory or synchronizes.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/qmm.h"
#include "paged.h"
#include "qmm_internal.h"

namespace {

int fail(int code, const char* fmt, ...) {
  char buf[1024];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return qmm::set_error(code, buf);
}

int hip_status(hipError_t e, const char* fn) {
  if (e == hipSuccess) return QMM_OK;
  return fail(QMM_ERR_HIP, "%s: the HIP runtime reported '%s' while enqueueing the kernel. "
              "Why: the launch or an earlier asynchronous operation on this device failed. "
              "How to fix: check the device state and earlier errors on the stream.",
              fn, hipGetErrorString(e));
}

int dtype_size(int dt) { return dt == QMM_F32 ? 4 : dt == QMM_F16 || dt == QMM_BF16 ? 2 : 0; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The largest stride in elements (or bytes), past any allocation.  Kernels
// multiply it in 64 bits by indices that the tensor has, so that a product is an
// offset inside the tensor.
constexpr int64_t MAX_STRIDE = (int64_t)1 << 39;
bool stride_ok(int64_t s) { return s >= 0 && s <= MAX_STRIDE; }

int check_kv(const char* fn, const qmm_paged_kv* kv) {
  if (kv == nullptr) return fail(QMM_ERR_INVALID_ARG, "%s: kv is NULL.", fn);
  if (dtype_size(kv->dtype) == 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: kv.dtype=%d is not a qmm_dtype. How to fix: pass "
                "QMM_F32, QMM_F16 or QMM_BF16.", fn, kv->dtype);
  if (kv->pages <= 0 || kv->pages > INT32_MAX || kv->kv_heads <= 0 || kv->page_size <= 0 ||
      kv->head_dim <= 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: the cache needs pages, kv_heads, page_size and head_dim "
                "> 0 (got %lld, %d, %d, %d). How to fix: pass pages of shape [pages, kv_heads, "
                "page_size, head_dim].", fn, (long long)kv->pages, kv->kv_heads, kv->page_size,
                kv->head_dim);
  if (kv->k_pages == nullptr || kv->v_pages == nullptr)
    return fail(QMM_ERR_INVALID_ARG, "%s: k_pages and v_pages must be non-null device pointers.", fn);
  for (int64_t s : {kv->k_page_stride, kv->k_head_stride, kv->k_token_stride, kv->v_page_stride,
                    kv->v_head_stride, kv->v_token_stride})
    if (!stride_ok(s))
      return fail(QMM_ERR_INVALID_ARG, "%s: a stride of the pages (%lld) is negative or too "
                  "large. How to fix: pass the strides of the pages in elements.", fn, (long long)s);
  const int es = dtype_size(kv->dtype);
  if (!aligned(kv->k_pages, es) || !aligned(kv->v_pages, es))
    return fail(QMM_ERR_INVALID_ARG, "%s: k_pages and v_pages must be aligned to their element "
                "size.", fn);
  return QMM_OK;
}

int check_batch(const char* fn, const qmm_paged_batch* b) {
  if (b == nullptr) return fail(QMM_ERR_INVALID_ARG, "%s: batch is NULL.", fn);
  if (b->seqs < 0 || b->tokens < 0 || b->width < 0 || b->max_new < 0 || b->max_len < 0 ||
      b->seqs > INT32_MAX / 2 || b->tokens > INT32_MAX / 2 || b->width > INT32_MAX / 2 ||
      b->max_new > INT32_MAX / 2 || b->max_len > INT32_MAX / 2 || !stride_ok(b->table_stride))
    return fail(QMM_ERR_INVALID_ARG, "%s: the batch's seqs, tokens, width, table_stride, max_new "
                "and max_len must be in 0 .. 2^30 (got %lld, %lld, %lld, %lld, %lld, %lld).", fn,
                (long long)b->seqs, (long long)b->tokens, (long long)b->width,
                (long long)b->table_stride, (long long)b->max_new, (long long)b->max_len);
  if (b->tokens > 0 && b->seqs > 0 &&
      (b->starts == nullptr || b->lens == nullptr || (b->table == nullptr && b->width > 0)))
    return fail(QMM_ERR_INVALID_ARG, "%s: the batch's starts, lens and table must be non-null "
                "device pointers.", fn);
  if (!aligned(b->starts, 4) || !aligned(b->lens, 4) || !aligned(b->table, 4))
    return fail(QMM_ERR_INVALID_ARG, "%s: starts, lens and table must be 4-byte aligned int32 "
                "arrays.", fn);
  return QMM_OK;
}

int check_heads(const char* fn, const char* name, const qmm_heads* h, int heads, int es,
                int64_t tokens) {
  if (h == nullptr || (h->data == nullptr && tokens > 0))
    return fail(QMM_ERR_INVALID_ARG, "%s: %s must be a non-null device pointer.", fn, name);
  if (h->heads <= 0 || (heads > 0 && h->heads != heads))
    return fail(QMM_ERR_INVALID_ARG, "%s: %s has %d heads, %d are wanted. Why: q and out have the "
                "query heads, k and v the cache's key/value heads.", fn, name, h->heads, heads);
  if (!stride_ok(h->token_stride) || !stride_ok(h->head_stride))
    return fail(QMM_ERR_INVALID_ARG, "%s: %s has a negative or too large stride (%lld, %lld).", fn,
                name, (long long)h->token_stride, (long long)h->head_stride);
  if (!aligned(h->data, es))
    return fail(QMM_ERR_INVALID_ARG, "%s: %s must be aligned to its element size.", fn, name);
  return QMM_OK;
}

qmm::CacheArgs cache_args(const qmm_paged_kv* kv, const qmm_paged_batch* b) {
  qmm::CacheArgs c;
  c.k = (char*)kv->k_pages;
  c.v = (char*)kv->v_pages;
  c.k_page = kv->k_page_stride;
  c.k_head = kv->k_head_stride;
  c.k_token = kv->k_token_stride;
  c.v_page = kv->v_page_stride;
  c.v_head = kv->v_head_stride;
  c.v_token = kv->v_token_stride;
  c.pages = (int)kv->pages;
  c.kv_heads = kv->kv_heads;
  c.page = kv->page_size;
  c.dim = kv->head_dim;
  c.by_page = qmm::fast_div((uint32_t)kv->page_size);
  c.starts = b->starts;
  c.lens = b->lens;
  c.table = b->table;
  c.table_stride = b->table_stride;
  c.seqs = (int)b->seqs;
  c.tokens = (int)b->tokens;
  c.width = (int)b->width;
  c.max_new = (int)b->max_new;
  c.max_len = (int)b->max_len;
  return c;
}

int check_pool(const char* fn, const qmm_page_pool* p, bool tables, bool data) {
  if (p == nullptr) return fail(QMM_ERR_INVALID_ARG, "%s: pool is NULL.", fn);
  if (p->pages <= 0 || p->pages > INT32_MAX / 2)
    return fail(QMM_ERR_INVALID_ARG, "%s: the pool's pages must be in 1 .. 2^30, got %lld.", fn,
                (long long)p->pages);
  if (data) {
    if (p->planes < 0 || p->planes > INT32_MAX / 2 || p->page_bytes < 0 ||
        p->page_bytes > INT32_MAX / 2 || !stride_ok(p->plane_stride) || !stride_ok(p->page_stride))
      return fail(QMM_ERR_INVALID_ARG, "%s: the pool's planes, page_bytes and strides must be >= 0 "
                  "(planes and page_bytes below 2^30; got %lld, %lld, %lld, %lld).", fn,
                  (long long)p->planes, (long long)p->page_bytes, (long long)p->plane_stride,
                  (long long)p->page_stride);
    if (p->planes * p->pages > UINT32_MAX)
      return fail(QMM_ERR_UNSUPPORTED, "%s: planes x pages must be below 2^32, got %lld x %lld.", fn,
                  (long long)p->planes, (long long)p->pages);
    if (p->data == nullptr && p->planes > 0 && p->page_bytes > 0)
      return fail(QMM_ERR_INVALID_ARG, "%s: the pool's data must be a non-null device pointer.", fn);
  }
  if (tables) {
    if (p->refs == nullptr || p->table == nullptr || p->lens == nullptr)
      return fail(QMM_ERR_INVALID_ARG, "%s: the pool's refs, table and lens must be non-null. Why: "
                  "this call reads and changes them. How to fix: make the pool with its reference "
                  "counts, table and lengths.", fn);
    if (p->page_size <= 0 || p->slots <= 0 || p->width <= 0 || p->width > (1 << 20) ||
        p->slots > qmm::POOL_MAX_SLOTS || !stride_ok(p->table_stride))
      return fail(QMM_ERR_INVALID_ARG, "%s: page_size, slots and width must be positive, slots at "
                  "most %lld and width at most %d (got %d, %lld, %lld).", fn,
                  (long long)qmm::POOL_MAX_SLOTS, 1 << 20, p->page_size, (long long)p->slots,
                  (long long)p->width);
    if (p->slots * p->width > UINT32_MAX)
      return fail(QMM_ERR_UNSUPPORTED, "%s: slots x width must be below 2^32, got %lld x %lld.", fn,
                  (long long)p->slots, (long long)p->width);
    if (!aligned(p->refs, 4) || !aligned(p->table, 4) || !aligned(p->lens, 4))
      return fail(QMM_ERR_INVALID_ARG, "%s: refs, table and lens must be 4-byte aligned int32 "
                  "arrays.", fn);
  }
  return QMM_OK;
}

int check_list(const char* fn, const char* name, const int32_t* list, int64_t count) {
  if (count < 0 || count >= (1 << 24))
    return fail(QMM_ERR_INVALID_ARG, "%s: count must be in 0 .. 2^24 - 1, got %lld.", fn,
                (long long)count);
  if (count > 0 && (list == nullptr || !aligned(list, 4)))
    return fail(QMM_ERR_INVALID_ARG, "%s: %s must be a non-null, 4-byte aligned int32 device "
                "array.", fn, name);
  return QMM_OK;
}

int check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need)
    return fail(QMM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, got %zu%s. How to fix: "
                "allocate the size that the workspace_size function of this call gives.", fn, need,
                have, ws == nullptr ? " (NULL)" : "");
  if (!aligned(ws, 256))
    return fail(QMM_ERR_WORKSPACE, "%s: the workspace must be 256-byte aligned.", fn);
  return QMM_OK;
}

qmm::PoolArgs pool_args(const qmm_page_pool* p, void* ws, void* stream) {
  qmm::PoolArgs a;
  a.data = (char*)p->data;
  a.planes = p->planes;
  a.plane_stride = p->plane_stride;
  a.page_stride = p->page_stride;
  a.page_bytes = p->page_bytes;
  a.refs = p->refs;
  a.table = p->table;
  a.lens = p->lens;
  a.table_stride = p->table_stride;
  a.pages = (int)p->pages;
  a.slots = (int)p->slots;
  a.width = (int)p->width;
  a.page = p->page_size;
  a.by_page = qmm::fast_div((uint32_t)(p->page_size > 0 ? p->page_size : 1));
  a.workspace = (char*)ws;
  a.stream = (hipStream_t)stream;
  return a;
}

#define CHECK(call)                    \
  do {                                 \
    const int st_ = (call);            \
    if (st_ != QMM_OK) return st_;     \
  } while (0)

}  // namespace

extern "C" {

int qmm_rope_append(const qmm_heads* q, const qmm_heads* k, const qmm_heads* v,
                    const qmm_heads* out, const qmm_paged_kv* kv, const qmm_paged_batch* batch,
                    const double* inv_freq, int half, int interleaved, double factor,
                    const int32_t* positions, void* stream) {
  const char* fn = "qmm_rope_append";
  CHECK(check_kv(fn, kv));
  CHECK(check_batch(fn, batch));
  const int es = dtype_size(kv->dtype);
  CHECK(check_heads(fn, "q", q, 0, es, batch->tokens));
  CHECK(check_heads(fn, "k", k, kv->kv_heads, es, batch->tokens));
  CHECK(check_heads(fn, "v", v, kv->kv_heads, es, batch->tokens));
  CHECK(check_heads(fn, "out", out, q->heads, es, batch->tokens));
  if (kv->head_dim > 512 || kv->head_dim % 2 != 0)
    return fail(QMM_ERR_UNSUPPORTED, "%s: head_dim must be even and at most 512, got %d.", fn,
                kv->head_dim);
  if (half < 0 || 2 * (int64_t)half > kv->head_dim)
    return fail(QMM_ERR_INVALID_ARG, "%s: half=%d pairs do not fit a head of %d. How to fix: pass "
                "one frequency a pair, at most head_dim / 2.", fn, half, kv->head_dim);
  if (half > 0 && (inv_freq == nullptr || !aligned(inv_freq, 8)))
    return fail(QMM_ERR_INVALID_ARG, "%s: inv_freq must be a non-null, 8-byte aligned float64 "
                "device array.", fn);
  if (!aligned(positions, 4))
    return fail(QMM_ERR_INVALID_ARG, "%s: positions must be a 4-byte aligned int32 array.", fn);
  if ((int64_t)(q->heads + 2 * (int64_t)kv->kv_heads) * kv->head_dim > (1 << 24))
    return fail(QMM_ERR_UNSUPPORTED, "%s: a token's heads pass 2^24 elements.", fn);
  if (batch->tokens >= 1 << 26)
    return fail(QMM_ERR_UNSUPPORTED, "%s: tokens must be below 2^26, got %lld. Why: a launch has fewer "
                "than 2^32 threads. How to fix: split the batch.", fn, (long long)batch->tokens);
  if (batch->tokens == 0) return QMM_OK;
  qmm::RopeArgs a;
  a.c = cache_args(kv, batch);
  a.q = (const char*)q->data;
  a.k = (const char*)k->data;
  a.v = (const char*)v->data;
  a.out = (char*)out->data;
  a.q_token = q->token_stride;
  a.q_head = q->head_stride;
  a.k_token = k->token_stride;
  a.k_head = k->head_stride;
  a.v_token = v->token_stride;
  a.v_head = v->head_stride;
  a.out_token = out->token_stride;
  a.out_head = out->head_stride;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.factor = factor;
  a.q_heads = q->heads;
  a.half = half;
  a.interleaved = interleaved != 0;
  a.dtype = kv->dtype;
  a.stream = (hipStream_t)stream;
  return hip_status(qmm::launch_rope_append(a), fn);
}

size_t qmm_paged_attention_workspace_size(const qmm_paged_batch* batch, int q_heads, int kv_heads,
                                          int head_dim) {
  if (check_batch("qmm_paged_attention_workspace_size", batch) != QMM_OK || kv_heads <= 0 ||
      q_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0 || head_dim > 256)
    return 0;
  return qmm::attn_workspace_bytes((int)batch->seqs, (int)batch->tokens, (int)batch->max_new,
                                   (int)batch->max_len, q_heads, kv_heads, head_dim);
}

int qmm_paged_attention(const qmm_heads* q, const qmm_paged_kv* kv, const qmm_paged_batch* batch,
                        const qmm_heads* out, float* lse, float scale, int causal, int64_t window,
                        float softcap, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "qmm_paged_attention";
  CHECK(check_kv(fn, kv));
  CHECK(check_batch(fn, batch));
  const int es = dtype_size(kv->dtype);
  CHECK(check_heads(fn, "q", q, 0, es, batch->tokens));
  CHECK(check_heads(fn, "out", out, q->heads, es, batch->tokens));
  if (q->heads % kv->kv_heads != 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: %d query heads do not divide into %d key/value heads. "
                "Why: head h reads key/value head h / (heads / kv_heads).", fn, q->heads,
                kv->kv_heads);
  if (kv->head_dim > 256 || kv->head_dim % (16 / es) != 0)
    return fail(QMM_ERR_UNSUPPORTED, "%s: head_dim must be a multiple of %d and at most 256, got "
                "%d. Why: keys and values are read 16 bytes at a time.", fn, 16 / es, kv->head_dim);
  const int v = 16 / es;
  if (!aligned(kv->k_pages, 16) || !aligned(kv->v_pages, 16) || kv->k_page_stride % v != 0 ||
      kv->k_head_stride % v != 0 || kv->k_token_stride % v != 0 || kv->v_page_stride % v != 0 ||
      kv->v_head_stride % v != 0 || kv->v_token_stride % v != 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: k_pages, v_pages and their strides must be 16-byte "
                "aligned. Why: keys and values are read 16 bytes at a time. How to fix: allocate "
                "the pages in one tensor and keep head_dim the dense dimension.", fn);
  if (window < 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: window must be >= 0 (0: none), got %lld.", fn,
                (long long)window);
  if (!isfinite(scale) || !isfinite(softcap) || softcap < 0.f)
    return fail(QMM_ERR_INVALID_ARG, "%s: scale must be finite and softcap finite and >= 0 (0: "
                "none), got %g and %g.", fn, (double)scale, (double)softcap);
  if (!aligned(lse, 4))
    return fail(QMM_ERR_INVALID_ARG, "%s: lse must be a 4-byte aligned float32 array.", fn);
  const int64_t group = q->heads / kv->kv_heads;
  auto too_large = [&] {
    return fail(QMM_ERR_UNSUPPORTED, "%s: seqs x max_new x heads, or with them max_len, is too large "
                "for one launch. How to fix: pass max_new and max_len as the largest counts of new "
                "tokens and of keys, or split the batch.", fn);
  };
  if (batch->max_new * group > (1 << 28) ||
      batch->seqs * kv->kv_heads * (batch->max_new * group / 16 + 1) > (1 << 28))
    return too_large();
  if (batch->tokens == 0 || batch->seqs == 0 || batch->max_new == 0) return QMM_OK;
  CHECK(check_workspace(fn, workspace, workspace_bytes,
                        qmm_paged_attention_workspace_size(batch, q->heads, kv->kv_heads,
                                                           kv->head_dim)));
  qmm::AttnArgs a;
  a.c = cache_args(kv, batch);
  a.q = (const char*)q->data;
  a.out = (char*)out->data;
  a.lse = lse;
  a.q_token = q->token_stride;
  a.q_head = q->head_stride;
  a.out_token = out->token_stride;
  a.out_head = out->head_stride;
  a.lse_token = q->heads;
  a.lse_head = 1;
  a.scale = scale;
  a.softcap = softcap;
  a.q_heads = q->heads;
  a.group = (int)group;
  a.by_group = qmm::fast_div((uint32_t)group);
  a.causal = causal != 0;
  // A window that no sequence fills is none.
  a.window = window >= batch->max_len ? 0 : (int)window;
  a.dtype = kv->dtype;
  a.q_wide = aligned(q->data, 16) && q->token_stride % v == 0 && q->head_stride % v == 0;
  a.out_wide = aligned(out->data, 4 * es) && out->token_stride % 4 == 0 && out->head_stride % 4 == 0;
  a.stream = (hipStream_t)stream;
  const hipError_t e = qmm::launch_paged_attention(a, (char*)workspace, workspace_bytes);
  return e == hipErrorInvalidConfiguration ? too_large() : hip_status(e, fn);
}

size_t qmm_pages_workspace_size(const qmm_page_pool* pool, int64_t count) {
  if (pool == nullptr || pool->pages <= 0 || count < 0) return 0;
  return qmm::pages_workspace_bytes(pool->pages, count);
}

int qmm_pages_free(const qmm_page_pool* pool, const int32_t* seqs, int64_t count, void* stream) {
  const char* fn = "qmm_pages_free";
  CHECK(check_pool(fn, pool, true, false));
  CHECK(check_list(fn, "seqs", seqs, count));
  if (count == 0) return QMM_OK;
  return hip_status(qmm::launch_pages_free(pool_args(pool, nullptr, stream), seqs, (int)count), fn);
}

int qmm_pages_fork(const qmm_page_pool* pool, const int32_t* parents, const int32_t* children,
                   int64_t count, int32_t* status, void* workspace, size_t workspace_bytes,
                   void* stream) {
  const char* fn = "qmm_pages_fork";
  CHECK(check_pool(fn, pool, true, true));
  CHECK(check_list(fn, "parents", parents, count));
  CHECK(check_list(fn, "children", children, count));
  CHECK(check_list(fn, "status", status, 1));
  if (pool->planes * count > UINT32_MAX || count * pool->width > UINT32_MAX)
    return fail(QMM_ERR_UNSUPPORTED, "%s: planes x count and count x width must be below 2^32.", fn);
  if (count == 0) return QMM_OK;
  CHECK(check_workspace(fn, workspace, workspace_bytes, qmm_pages_workspace_size(pool, count)));
  return hip_status(qmm::launch_pages_fork(pool_args(pool, workspace, stream), parents, children,
                                           (int)count, status), fn);
}

int qmm_pages_reserve(const qmm_page_pool* pool, const int32_t* seqs, const int32_t* grow,
                      int64_t count, int32_t* status, void* workspace, size_t workspace_bytes,
                      void* stream) {
  const char* fn = "qmm_pages_reserve";
  CHECK(check_pool(fn, pool, true, false));
  CHECK(check_list(fn, "seqs", seqs, count));
  CHECK(check_list(fn, "grow", grow, count));
  CHECK(check_list(fn, "status", status, 1));
  if (count == 0) return QMM_OK;
  CHECK(check_workspace(fn, workspace, workspace_bytes, qmm_pages_workspace_size(pool, count)));
  return hip_status(qmm::launch_pages_reserve(pool_args(pool, workspace, stream), seqs, grow,
                                              (int)count, status), fn);
}

int qmm_pages_copy(const qmm_page_pool* pool, const int32_t* src, const int32_t* dst,
                   int64_t count, void* stream) {
  const char* fn = "qmm_pages_copy";
  CHECK(check_pool(fn, pool, false, true));
  CHECK(check_list(fn, "src", src, count));
  CHECK(check_list(fn, "dst", dst, count));
  if (pool->planes * count > UINT32_MAX)
    return fail(QMM_ERR_UNSUPPORTED, "%s: planes x count must be below 2^32.", fn);
  if (count == 0 || pool->planes == 0 || pool->page_bytes == 0) return QMM_OK;
  return hip_status(qmm::launch_pages_copy(pool_args(pool, nullptr, stream), src, dst,
                                           (int)count), fn);
}

int qmm_pages_compact(const qmm_page_pool* pool, int32_t* refs_out, int32_t* table_out,
                      int32_t* live, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "qmm_pages_compact";
  CHECK(check_pool(fn, pool, true, true));
  if (refs_out == nullptr || table_out == nullptr || live == nullptr || !aligned(refs_out, 4) ||
      !aligned(table_out, 4) || !aligned(live, 4))
    return fail(QMM_ERR_INVALID_ARG, "%s: refs_out, table_out and live must be non-null, 4-byte "
                "aligned int32 device arrays.", fn);
  if (refs_out == pool->refs || table_out == pool->table)
    return fail(QMM_ERR_INVALID_ARG, "%s: refs_out and table_out must not be the pool's own. Why: "
                "they are written while the old ones are read.", fn);
  CHECK(check_workspace(fn, workspace, workspace_bytes, qmm_pages_workspace_size(pool, 0)));
  return hip_status(qmm::launch_pages_compact(pool_args(pool, workspace, stream), refs_out,
                                              table_out, pool->width, live), fn);
}

}  // extern "C"
