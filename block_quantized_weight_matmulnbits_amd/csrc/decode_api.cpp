// decode_api.cpp -- the extern "C" entry points around a decode step's
// projections declared in include/qmm.h (norm, experts, sampling): arguments are
// validated on the host (errors say what, why and how to fix), then the
// launchers of rms_norm.hip, moe.hip and sample.hip enqueue the work.  Nothing
// here allocates device memory or synchronizes.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/qmm.h"
#include "decode.h"
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

// Past any allocation; kernels multiply it in 64 bits by a row that the tensor has.
constexpr int64_t MAX_STRIDE = (int64_t)1 << 39;

int check_rows(const char* fn, const char* name, const qmm_rows* r, int64_t rows, int64_t cols,
               int es) {
  if (r->data == nullptr || !aligned(r->data, es))
    return fail(QMM_ERR_INVALID_ARG, "%s: %s.data must be a non-null device pointer aligned to its "
                "element size.", fn, name);
  if (r->stride < 0 || r->stride > MAX_STRIDE || (rows > 1 && r->stride < cols))
    return fail(QMM_ERR_INVALID_ARG, "%s: %s.stride=%lld does not hold a row of %lld elements. How "
                "to fix: pass rows that do not overlap, with a dense last dimension.", fn, name,
                (long long)r->stride, (long long)cols);
  return QMM_OK;
}

int check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need)
    return fail(QMM_ERR_WORKSPACE, "%s: the workspace holds %zu bytes at %p, %zu are needed. How to "
                "fix: pass %s_workspace_size bytes of device memory.", fn, bytes, ws, need, fn);
  if (!aligned(ws, 256))
    return fail(QMM_ERR_WORKSPACE, "%s: the workspace must be 256-byte aligned. How to fix: pass "
                "the start of a fresh allocation.", fn);
  return QMM_OK;
}

int check_moe_sizes(const char* fn, const qmm_moe_weights* w) {
  if (w->bits != 4 && w->bits != 8)
    return fail(w->bits == 2 || w->bits == 3 ? QMM_ERR_UNSUPPORTED : QMM_ERR_INVALID_ARG,
                "%s: experts' weights have 4 or 8 bits, got bits=%d. How to fix: export them with "
                "bits=4 or 8.", fn, w->bits);
  if (w->block_size < 16 || (w->block_size & (w->block_size - 1)) || w->block_size > 1 << 20)
    return fail(QMM_ERR_INVALID_ARG, "%s: block_size must be a power of two from 16 to 2^20, got %d.",
                fn, w->block_size);
  if (dtype_size(w->s_dtype) == 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: s_dtype=%d is not a qmm_dtype.", fn, w->s_dtype);
  if (w->hidden <= 0 || w->inter <= 0 || w->experts <= 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: hidden, inter and experts must be positive, got %lld, %lld, "
                "%d.", fn, (long long)w->hidden, (long long)w->inter, w->experts);
  if (w->experts > qmm::MOE_MAX_EXPERTS || w->hidden > 1 << 18 || w->inter > 1 << 18)
    return fail(QMM_ERR_UNSUPPORTED, "%s: at most %d experts, hidden and inter at most 2^18 (got %d, "
                "%lld, %lld).", fn, qmm::MOE_MAX_EXPERTS, w->experts, (long long)w->hidden,
                (long long)w->inter);
  auto bytes = [&](int64_t rows, int64_t cols) {
    return rows * ((cols + w->block_size - 1) / w->block_size) * w->block_size * w->bits / 8;
  };
  if (bytes(2 * w->inter, w->hidden) > INT32_MAX || bytes(w->hidden, w->inter) > INT32_MAX)
    return fail(QMM_ERR_UNSUPPORTED, "%s: the codes of one expert's projection must be below 2^31 "
                "bytes. Why: offsets in it are 32-bit.", fn);
  return QMM_OK;
}

constexpr int64_t SAMPLE_MAX_ROWS = ((int64_t)1 << 21) - 1;

}  // namespace

extern "C" {

int qmm_rms_norm(const qmm_rows* x, const qmm_rows* residual, const qmm_rows* h,
                 const void* weight, int weight_dtype, float offset, double eps, const qmm_rows* y,
                 const qmm_quant* quant, int dtype, int64_t rows, int64_t cols, void* stream) {
  const char* fn = "qmm_rms_norm";
  const int es = dtype_size(dtype);
  if (es == 0 || (weight != nullptr && dtype_size(weight_dtype) == 0))
    return fail(QMM_ERR_INVALID_ARG, "%s: dtype=%d / weight_dtype=%d is not a qmm_dtype. How to fix: "
                "pass QMM_F32, QMM_F16 or QMM_BF16.", fn, dtype, weight_dtype);
  if (rows < 0 || cols <= 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: rows must be >= 0 and cols positive, got rows=%lld "
                "cols=%lld.", fn, (long long)rows, (long long)cols);
  if (rows >= (int64_t)1 << 40 || cols > qmm::NORM_MAX_COLS)
    return fail(QMM_ERR_UNSUPPORTED, "%s: rows must be below 2^40 and cols at most 2^20 (got rows=%lld "
                "cols=%lld). Why: a row is one workgroup's.", fn, (long long)rows, (long long)cols);
  if (!(eps >= 0.0) || isinf(eps) || !isfinite(offset))
    return fail(QMM_ERR_INVALID_ARG, "%s: eps must be finite and not negative, offset finite (got %g, "
                "%g).", fn, eps, (double)offset);
  if (h == nullptr && y == nullptr && quant == nullptr)
    return fail(QMM_ERR_INVALID_ARG, "%s: h, y and quant are all NULL. How to fix: pass an output.", fn);
  if (x == nullptr) return fail(QMM_ERR_INVALID_ARG, "%s: x is NULL.", fn);
  qmm::NormArgs a;
  if (quant != nullptr) {
    const bool ocp = quant->kind == QMM_QUANT_MX_OCP, mx = quant->kind == QMM_QUANT_MX || ocp;
    if (quant->kind != QMM_QUANT_INT8 && !mx && quant->kind != QMM_QUANT_TENSOR)
      return fail(QMM_ERR_INVALID_ARG, "%s: quant.kind=%d is not a qmm_quant_kind.", fn, quant->kind);
    const bool ints = quant->kind == QMM_QUANT_INT8;
    if (ints && (quant->block_size < 16 || quant->block_size > qmm::NORM_MAX_COLS ||
                 (quant->block_size & (quant->block_size - 1))))
      return fail(QMM_ERR_INVALID_ARG, "%s: quant.block_size must be a power of two from 16 to 2^20, "
                  "got %d. How to fix: pass the block_size of the weight that reads the codes.", fn,
                  quant->block_size);
    if (!ints && quant->format != QMM_LOWP_E4M3 && quant->format != QMM_LOWP_E5M2)
      return fail(QMM_ERR_INVALID_ARG, "%s: quant.format=%d must be QMM_LOWP_E4M3 or QMM_LOWP_E5M2. "
                  "Why: the output holds 8 bits an element.", fn, quant->format);
    if (rows > 0 && (quant->codes == nullptr || quant->scales == nullptr ||
                     (!mx && !aligned(quant->scales, 4))))
      return fail(QMM_ERR_INVALID_ARG, "%s: quant.codes and quant.scales must be non-null device "
                  "pointers (float32 scales 4-byte aligned).", fn);
    a.kind = mx ? qmm::QUANT_MX : quant->kind;
    a.format = quant->format;
    if (mx)
      a.top_factor = a.format == QMM_LOWP_E4M3 ? (ocp ? 0x1p-8f : 1.f / 448.f) : (ocp ? 0x1p-15f : 1.f / 57344.f);
    a.block = ints ? quant->block_size : 32;
    a.blocks = (int)((cols + a.block - 1) / a.block);
    a.code_cols = ints ? a.blocks * a.block : (int)cols;
    a.codes = (uint8_t*)quant->codes;
    a.scales = quant->scales;
  }
  if (rows == 0) return QMM_OK;
  const struct { const char* name; const qmm_rows* r; } each[] = {
      {"x", x}, {"residual", residual}, {"h", h}, {"y", y}};
  for (const auto& e : each) {
    if (e.r == nullptr) continue;
    const int st = check_rows(fn, e.name, e.r, rows, cols, es);
    if (st != QMM_OK) return st;
  }
  if (!aligned(weight, weight == nullptr ? 1 : dtype_size(weight_dtype)))
    return fail(QMM_ERR_INVALID_ARG, "%s: weight must be aligned to its element size.", fn);
  if (h != nullptr && y != nullptr && h->data == y->data)
    return fail(QMM_ERR_INVALID_ARG, "%s: h and y are two outputs and cannot be the same rows.", fn);
  for (const qmm_rows* in : {x, residual})
    for (const qmm_rows* out : {h, y})
      if (in != nullptr && out != nullptr && in->data == out->data && in->stride != out->stride && rows > 1)
        return fail(QMM_ERR_INVALID_ARG, "%s: an output begins where an input does, with rows of stride "
                    "%lld over rows of stride %lld. Why: rows would be written before they are read. How "
                    "to fix: pass the input's own rows, or rows apart from it.", fn,
                    (long long)out->stride, (long long)in->stride);
  a.x = (const char*)x->data;
  a.x_stride = x->stride;
  if (residual) a.residual = (const char*)residual->data, a.residual_stride = residual->stride;
  if (h) a.h = (char*)h->data, a.h_stride = h->stride;
  if (y) a.y = (char*)y->data, a.y_stride = y->stride;
  a.weight = (const char*)weight;
  a.weight_dtype = weight_dtype;
  a.offset = offset;
  a.eps = eps;
  a.dtype = dtype;
  a.rows = rows;
  a.cols = (int)cols;
  a.stream = (hipStream_t)stream;
  return hip_status(qmm::launch_rms_norm(a), fn);
}

size_t qmm_sample_workspace_size(int64_t rows, int64_t vocab) {
  if (rows < 0 || rows > SAMPLE_MAX_ROWS || vocab <= 0 || vocab > qmm::SAMPLE_MAX_VOCAB) return 0;
  return qmm::sample_workspace_bytes(rows, vocab);
}

int qmm_sample(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
               const float* temperature, const int32_t* top_k, const float* top_p,
               const float* min_p, const float* uniform, int32_t* tokens, float* logprobs,
               void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "qmm_sample";
  const int es = dtype_size(dtype);
  if (es == 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: dtype=%d is not a qmm_dtype. How to fix: pass QMM_F32, "
                "QMM_F16 or QMM_BF16.", fn, dtype);
  if (rows < 0 || vocab <= 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: rows must be >= 0 and vocab positive, got rows=%lld "
                "vocab=%lld.", fn, (long long)rows, (long long)vocab);
  if (rows > SAMPLE_MAX_ROWS || vocab > qmm::SAMPLE_MAX_VOCAB)
    return fail(QMM_ERR_UNSUPPORTED, "%s: rows must be below 2^21 and vocab at most 2^22 (got "
                "rows=%lld vocab=%lld). How to fix: split the rows.", fn, (long long)rows,
                (long long)vocab);
  if (rows == 0) return QMM_OK;
  if (logits == nullptr || uniform == nullptr || tokens == nullptr)
    return fail(QMM_ERR_INVALID_ARG, "%s: logits, uniform and tokens must be non-null device "
                "pointers.", fn);
  if (!aligned(logits, es) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(uniform, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
    return fail(QMM_ERR_INVALID_ARG, "%s: every array must be aligned to its element size.", fn);
  if (row_stride < 0 || row_stride > MAX_STRIDE || (rows > 1 && row_stride < vocab))
    return fail(QMM_ERR_INVALID_ARG, "%s: row_stride=%lld does not hold a row of %lld logits.", fn,
                (long long)row_stride, (long long)vocab);
  const int st = check_workspace(fn, workspace, workspace_bytes, qmm::sample_workspace_bytes(rows, vocab));
  if (st != QMM_OK) return st;
  qmm::SampleArgs a;
  a.logits = (const char*)logits;
  a.stride = row_stride;
  a.rows = rows;
  a.vocab = (int)vocab;
  a.dtype = dtype;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniform = uniform;
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.stream = (hipStream_t)stream;
  return hip_status(qmm::launch_sample(a, (char*)workspace), fn);
}

size_t qmm_moe_workspace_size(const qmm_moe_weights* w, int64_t tokens, int top_k) {
  if (w == nullptr || tokens < 0 || tokens > qmm::MOE_MAX_TOKENS || top_k < 1 ||
      top_k > qmm::MOE_MAX_TOP_K || check_moe_sizes("qmm_moe_workspace_size", w) != QMM_OK)
    return 0;
  return qmm::moe_workspace_bytes((int)tokens, (int)w->hidden, (int)w->inter, w->experts, top_k);
}

int qmm_moe(const qmm_rows* x, const qmm_moe_weights* w, const qmm_moe_route* route,
            const qmm_rows* y, int dtype, int64_t tokens, void* workspace, size_t workspace_bytes,
            void* stream) {
  const char* fn = "qmm_moe";
  const int es = dtype_size(dtype);
  if (x == nullptr || w == nullptr || route == nullptr || y == nullptr)
    return fail(QMM_ERR_INVALID_ARG, "%s: x, w, route and y must be non-null.", fn);
  if (es == 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: dtype=%d is not a qmm_dtype. How to fix: pass QMM_F32, "
                "QMM_F16 or QMM_BF16.", fn, dtype);
  int st = check_moe_sizes(fn, w);
  if (st != QMM_OK) return st;
  if (tokens < 0)
    return fail(QMM_ERR_INVALID_ARG, "%s: tokens must be >= 0, got %lld.", fn, (long long)tokens);
  if (tokens > qmm::MOE_MAX_TOKENS)
    return fail(QMM_ERR_UNSUPPORTED, "%s: at most %d tokens, got %lld. Why: every expert's tokens are "
                "taken together, for a few of them. How to fix: split the batch, or group the tokens by "
                "expert for qmm_gemm.", fn, qmm::MOE_MAX_TOKENS, (long long)tokens);
  if (route->top_k < 1 || route->top_k > qmm::MOE_MAX_TOP_K ||
      (route->logits != nullptr && route->top_k > w->experts))
    return fail(QMM_ERR_INVALID_ARG, "%s: route.top_k must be from 1 to %d and no more than the "
                "experts (%d), got %d.", fn, qmm::MOE_MAX_TOP_K, w->experts, route->top_k);
  if (tokens == 0) return QMM_OK;
  st = check_rows(fn, "x", x, tokens, w->hidden, es);
  if (st == QMM_OK) st = check_rows(fn, "y", y, tokens, w->hidden, es);
  if (st != QMM_OK) return st;
  if (w->gate_up == nullptr || w->gate_up_scales == nullptr || w->down == nullptr ||
      w->down_scales == nullptr || !aligned(w->gate_up, 16) || !aligned(w->down, 16))
    return fail(QMM_ERR_INVALID_ARG, "%s: the codes must be non-null, 16-byte aligned and the scales "
                "non-null device pointers.", fn);
  const int ss = dtype_size(w->s_dtype);
  if (!aligned(w->gate_up_scales, ss) || !aligned(w->down_scales, ss))
    return fail(QMM_ERR_INVALID_ARG, "%s: scales must be aligned to their element size.", fn);
  if (route->logits != nullptr) {
    const int ls = dtype_size(route->logits_dtype);
    if (ls == 0 || !aligned(route->logits, ls))
      return fail(QMM_ERR_INVALID_ARG, "%s: route.logits must have a qmm_dtype (got %d) and be aligned "
                  "to its element size.", fn, route->logits_dtype);
    if (route->logits_stride < 0 || route->logits_stride > MAX_STRIDE ||
        (tokens > 1 && route->logits_stride < w->experts))
      return fail(QMM_ERR_INVALID_ARG, "%s: route.logits_stride=%lld does not hold a row of %d logits.",
                  fn, (long long)route->logits_stride, w->experts);
  } else if (route->ids == nullptr || route->weights == nullptr || !aligned(route->ids, 4) ||
             !aligned(route->weights, 4)) {
    return fail(QMM_ERR_INVALID_ARG, "%s: route needs logits, or ids and weights (4-byte aligned). How "
                "to fix: pass one of the two.", fn);
  }
  st = check_workspace(fn, workspace, workspace_bytes,
                       qmm::moe_workspace_bytes((int)tokens, (int)w->hidden, (int)w->inter, w->experts,
                                                route->top_k));
  if (st != QMM_OK) return st;
  qmm::MoeArgs a;
  a.x = (const char*)x->data;
  a.y = (char*)y->data;
  a.x_stride = x->stride;
  a.y_stride = y->stride;
  auto proj = [&](const uint8_t* codes, const void* scales, const uint8_t* zp, int64_t rows, int64_t cols) {
    qmm::MoeProj p;
    p.codes = codes;
    p.scales = (const char*)scales;
    p.zp = zp;
    p.rows = (int)rows;
    p.cols = (int)cols;
    p.blocks = (int)((cols + w->block_size - 1) / w->block_size);
    p.row_bytes = (int64_t)p.blocks * w->block_size * w->bits / 8;
    p.zp_row_bytes = ((int64_t)p.blocks * w->bits + 7) / 8;
    return p;
  };
  a.up = proj(w->gate_up, w->gate_up_scales, w->gate_up_zero_points, 2 * w->inter, w->hidden);
  a.down = proj(w->down, w->down_scales, w->down_zero_points, w->hidden, w->inter);
  a.logits = (const char*)route->logits;
  a.ids = route->ids;
  a.weights = route->weights;
  a.logits_stride = route->logits_stride;
  a.logits_dtype = route->logits_dtype;
  a.normalize = route->normalize;
  a.top_k = route->top_k;
  a.tokens = (int)tokens;
  a.hidden = (int)w->hidden;
  a.inter = (int)w->inter;
  a.experts = w->experts;
  a.dtype = dtype;
  a.s_dtype = w->s_dtype;
  a.bits = w->bits;
  a.block = w->block_size;
  a.stream = (hipStream_t)stream;
  return hip_status(qmm::launch_moe(a, (char*)workspace), fn);
}

}  // extern "C"
