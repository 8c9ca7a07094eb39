// step.cpp -- a fixed sequence of calls (for example the projections and the
// attention of one decode step) recorded once and replayed as one HIP graph.
//
// The pages' end-to-end decode measurements put the time lost outside the
// kernels: per-operator fork/join and dispatch, not the matmul itself, made
// decode 2.3x slower than it needed to be, and a persistent pool raised it
// from 6 to 28 tok/s (onnx-runtime-ep-cpu matmul_nbits.rs, module notes on
// the decode step and the persistent decode pool).  On a GPU the same cost is
// the host's work per launch: each qmm_gemv call validates its arguments and
// enqueues one kernel, microseconds that a small projection's kernel does
// not cover.  A step pays it once: qmm_step_finalize validates every
// recorded call and captures their launches into a graph; qmm_step_launch is
// one hipGraphLaunch.  The replayed kernels and their arguments (pointers
// included) are exactly those of the direct calls; callers change inputs in
// place between launches.  The calls contain no memory-set operations.
#include <hip/hip_runtime.h>
#include <stdio.h>

#include <functional>
#include <string>
#include <vector>

#include "../../include/qmm.h"
#include "qmm_internal.h"

struct qmm_step {
  // Each recorded call enqueues itself on the given stream and returns a
  // qmm_status (validation included).
  std::vector<std::function<int(void*)>> calls;
  hipGraph_t graph = nullptr;
  hipGraphExec_t exec = nullptr;
  int device = -1;
};

namespace {

int step_error(int code, const char* fmt, long long v) {
  char msg[512];
  snprintf(msg, sizeof(msg), fmt, v);
  return qmm::set_error(code, msg);
}

int add_call(qmm_step* step, std::function<int(void*)> call) {
  if (step == nullptr) return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step: step is NULL.");
  if (step->exec != nullptr)
    return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_add_*: the step was already "
                          "finalized. How to fix: record every call before qmm_step_finalize.");
  step->calls.push_back(std::move(call));
  return QMM_OK;
}

// A struct that a caller may leave out, kept with the recorded call.
template <typename T> struct Copied {
  bool given = false;
  T value{};
  const T* get() const { return given ? &value : nullptr; }
};
template <typename T> Copied<T> copied(const T* p) { return p ? Copied<T>{true, *p} : Copied<T>{}; }

}  // namespace

extern "C" {

int qmm_step_create(qmm_step** step) {
  if (step == nullptr) return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_create: step is NULL.");
  *step = new qmm_step();
  return QMM_OK;
}

int qmm_step_add_gemv(qmm_step* step, const void* A, int a_dtype, const uint8_t* B,
                      int b_layout, const void* scales, int s_dtype, const uint8_t* zero_points,
                      const int32_t* g_idx, int64_t g_idx_len, const void* bias, void* Y,
                      int64_t K, int64_t N, int block_size, int bits, int accuracy_level) {
  return add_call(step, [=](void* s) {
    return qmm_gemv(A, a_dtype, B, b_layout, scales, s_dtype, zero_points, g_idx, g_idx_len,
                    bias, Y, K, N, block_size, bits, accuracy_level, s);
  });
}

int qmm_step_add_gemm(qmm_step* step, const void* A, int a_dtype, const uint8_t* B,
                      int b_layout, const void* scales, int s_dtype, const uint8_t* zero_points,
                      const int32_t* g_idx, int64_t g_idx_len, const void* bias, void* Y,
                      int64_t M, int64_t K, int64_t N, int block_size, int bits,
                      int accuracy_level) {
  return add_call(step, [=](void* s) {
    return qmm_gemm(A, a_dtype, B, b_layout, scales, s_dtype, zero_points, g_idx, g_idx_len,
                    bias, Y, M, K, N, block_size, bits, accuracy_level, s);
  });
}

int qmm_step_add_gemm_compint8(qmm_step* step, const void* A, int a_dtype, const uint8_t* B,
                               int b_layout, const void* scales, int s_dtype,
                               const uint8_t* zero_points, const int32_t* g_idx,
                               int64_t g_idx_len, const void* bias, void* Y, int64_t M,
                               int64_t K, int64_t N, int block_size, int bits,
                               int accuracy_level, void* workspace, size_t workspace_bytes) {
  return add_call(step, [=](void* s) {
    return qmm_gemm_compint8(A, a_dtype, B, b_layout, scales, s_dtype, zero_points, g_idx,
                             g_idx_len, bias, Y, M, K, N, block_size, bits, accuracy_level,
                             workspace, workspace_bytes, s);
  });
}

// The structs are copied into the recorded call; the arrays are not.
int qmm_step_add_rope_append(qmm_step* step, const qmm_heads* q, const qmm_heads* k,
                             const qmm_heads* v, const qmm_heads* out, const qmm_paged_kv* kv,
                             const qmm_paged_batch* batch, const double* inv_freq, int half,
                             int interleaved, double factor, const int32_t* positions) {
  if (!q || !k || !v || !out || !kv || !batch)
    return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_add_rope_append: q, k, v, out, kv and "
                          "batch must be non-null.");
  const qmm_heads hq = *q, hk = *k, hv = *v, ho = *out;
  const qmm_paged_kv c = *kv;
  const qmm_paged_batch b = *batch;
  return add_call(step, [=](void* s) {
    return qmm_rope_append(&hq, &hk, &hv, &ho, &c, &b, inv_freq, half, interleaved, factor,
                           positions, s);
  });
}

int qmm_step_add_paged_attention(qmm_step* step, const qmm_heads* q, const qmm_paged_kv* kv,
                                 const qmm_paged_batch* batch, const qmm_heads* out, float* lse,
                                 float scale, int causal, int64_t window, float softcap,
                                 void* workspace, size_t workspace_bytes) {
  if (!q || !out || !kv || !batch)
    return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_add_paged_attention: q, kv, batch and out "
                          "must be non-null.");
  const qmm_heads hq = *q, ho = *out;
  const qmm_paged_kv c = *kv;
  const qmm_paged_batch b = *batch;
  return add_call(step, [=](void* s) {
    return qmm_paged_attention(&hq, &c, &b, &ho, lse, scale, causal, window, softcap, workspace,
                               workspace_bytes, s);
  });
}

int qmm_step_add_pages_reserve(qmm_step* step, const qmm_page_pool* pool, const int32_t* seqs,
                               const int32_t* grow, int64_t count, int32_t* status,
                               void* workspace, size_t workspace_bytes) {
  if (!pool)
    return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_add_pages_reserve: pool must be non-null.");
  const qmm_page_pool p = *pool;
  return add_call(step, [=](void* s) {
    return qmm_pages_reserve(&p, seqs, grow, count, status, workspace, workspace_bytes, s);
  });
}

int qmm_step_add_rms_norm(qmm_step* step, const qmm_rows* x, const qmm_rows* residual,
                          const qmm_rows* h, const void* weight, int weight_dtype, float offset,
                          double eps, const qmm_rows* y, const qmm_quant* quant, int dtype,
                          int64_t rows, int64_t cols) {
  const auto rx = copied(x), rr = copied(residual), rh = copied(h), ry = copied(y);
  const auto q = copied(quant);
  return add_call(step, [=](void* s) {
    return qmm_rms_norm(rx.get(), rr.get(), rh.get(), weight, weight_dtype, offset, eps, ry.get(),
                        q.get(), dtype, rows, cols, s);
  });
}

int qmm_step_add_gemm_compint8_quantized(qmm_step* step, const int8_t* qa, const float* sa,
                                         const uint8_t* B, int b_layout, const void* scales,
                                         int s_dtype, const uint8_t* zero_points, const void* bias,
                                         void* Y, int y_dtype, int64_t M, int64_t K, int64_t N,
                                         int block_size, int bits) {
  return add_call(step, [=](void* s) {
    return qmm_gemm_compint8_quantized(qa, sa, B, b_layout, scales, s_dtype, zero_points, bias, Y,
                                       y_dtype, M, K, N, block_size, bits, s);
  });
}

int qmm_step_add_moe(qmm_step* step, const qmm_rows* x, const qmm_moe_weights* w,
                     const qmm_moe_route* route, const qmm_rows* y, int dtype, int64_t tokens,
                     void* workspace, size_t workspace_bytes) {
  const auto rx = copied(x), ry = copied(y);
  const auto cw = copied(w);
  const auto cr = copied(route);
  return add_call(step, [=](void* s) {
    return qmm_moe(rx.get(), cw.get(), cr.get(), ry.get(), dtype, tokens, workspace,
                   workspace_bytes, s);
  });
}

int qmm_step_add_sample(qmm_step* step, const void* logits, int dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const float* temperature, const int32_t* top_k,
                        const float* top_p, const float* min_p, const float* uniform,
                        int32_t* tokens, float* logprobs, void* workspace,
                        size_t workspace_bytes) {
  return add_call(step, [=](void* s) {
    return qmm_sample(logits, dtype, rows, vocab, row_stride, temperature, top_k, top_p, min_p,
                      uniform, tokens, logprobs, workspace, workspace_bytes, s);
  });
}

int qmm_step_finalize(qmm_step* step) {
  if (step == nullptr) return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_finalize: step is NULL.");
  if (step->exec != nullptr) return QMM_OK;
  if (step->calls.empty())
    return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_finalize: no call was recorded.");
  hipError_t e = hipGetDevice(&step->device);
  hipStream_t cs = nullptr;
  if (e == hipSuccess) e = hipStreamCreateWithFlags(&cs, hipStreamNonBlocking);
  if (e == hipSuccess) e = hipStreamBeginCapture(cs, hipStreamCaptureModeRelaxed);
  if (e != hipSuccess) {
    if (cs) (void)hipStreamDestroy(cs);
    return step_error(QMM_ERR_HIP, "qmm_step_finalize: could not start a graph capture (HIP "
                      "error %lld).", (long long)e);
  }
  int st = QMM_OK;
  size_t failed = 0;
  for (size_t i = 0; i < step->calls.size() && st == QMM_OK; ++i) {
    st = step->calls[i](cs);
    failed = i;
  }
  hipGraph_t graph = nullptr;
  const hipError_t ec = hipStreamEndCapture(cs, &graph);
  (void)hipStreamDestroy(cs);
  if (st != QMM_OK) {
    if (graph) (void)hipGraphDestroy(graph);
    // Keep the failing call's message, prefixed with its position.
    std::string msg = "qmm_step_finalize: recorded call " + std::to_string(failed) + " failed: " +
                      qmm_last_error();
    return qmm::set_error(st, msg.c_str());
  }
  if (ec != hipSuccess || graph == nullptr)
    return step_error(QMM_ERR_HIP, "qmm_step_finalize: the graph capture failed (HIP error "
                      "%lld).", (long long)ec);
  hipGraphExec_t exec = nullptr;
  e = hipGraphInstantiate(&exec, graph, nullptr, nullptr, 0);
  if (e != hipSuccess) {
    (void)hipGraphDestroy(graph);
    return step_error(QMM_ERR_HIP, "qmm_step_finalize: hipGraphInstantiate failed (HIP error "
                      "%lld).", (long long)e);
  }
  step->graph = graph;
  step->exec = exec;
  return QMM_OK;
}

int qmm_step_launch(const qmm_step* step, void* stream) {
  if (step == nullptr || step->exec == nullptr)
    return qmm::set_error(QMM_ERR_INVALID_ARG, "qmm_step_launch: the step is NULL or not "
                          "finalized. How to fix: call qmm_step_finalize first.");
  int dev = -1;
  if (hipGetDevice(&dev) == hipSuccess && dev != step->device)
    return step_error(QMM_ERR_INVALID_ARG, "qmm_step_launch: the step was finalized on device "
                      "%lld, another device is current.", (long long)step->device);
  const hipError_t e = hipGraphLaunch(step->exec, (hipStream_t)stream);
  if (e != hipSuccess)
    return step_error(QMM_ERR_HIP, "qmm_step_launch: hipGraphLaunch failed (HIP error %lld).",
                      (long long)e);
  return QMM_OK;
}

int qmm_step_size(const qmm_step* step) {
  return step == nullptr ? 0 : (int)step->calls.size();
}

void qmm_step_destroy(qmm_step* step) {
  if (step == nullptr) return;
  if (step->exec) (void)hipGraphExecDestroy(step->exec);
  if (step->graph) (void)hipGraphDestroy(step->graph);
  delete step;
}

}  // extern "C"
