// decode.h -- host-side interface between the validated entry points around a
// decode step's projections (decode_api.cpp) and their kernel launchers
// (rms_norm.hip, sample.hip, moe.hip).  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace qmm {

enum : int { QUANT_NONE = -1, QUANT_INT8 = 0, QUANT_MX = 1, QUANT_TENSOR = 2 };

struct NormArgs {
  const char *x = nullptr, *residual = nullptr;   // [rows, cols], strides in elements
  char *h = nullptr, *y = nullptr;
  const char* weight = nullptr;                   // [cols] or null
  int64_t x_stride = 0, residual_stride = 0, h_stride = 0, y_stride = 0;
  int64_t rows = 0;
  int cols = 0;
  int dtype = 0, weight_dtype = 0;
  float offset = 0.f;
  double eps = 0.0;
  int kind = QUANT_NONE, format = 0, block = 0;   // block: codes that share a scale
  float top_factor = 0.f;                         // MX: the scale is the exponent of it times the maximum
  uint8_t* codes = nullptr;                       // rows of code_cols bytes
  void* scales = nullptr;
  int code_cols = 0, blocks = 0;                  // of a row
  hipStream_t stream = nullptr;
};
constexpr int64_t NORM_MAX_COLS = 1 << 20;
hipError_t launch_rms_norm(const NormArgs& a);

// One projection of every expert: [experts, rows] rows of `cols` codes.
struct MoeProj {
  const uint8_t* codes = nullptr;
  const char* scales = nullptr;
  const uint8_t* zp = nullptr;        // or null
  int rows = 0, cols = 0, blocks = 0; // blocks of a row
  int64_t row_bytes = 0, zp_row_bytes = 0;
};
struct MoeArgs {
  const char* x = nullptr;            // [tokens, hidden], strides in elements
  char* y = nullptr;
  int64_t x_stride = 0, y_stride = 0;
  MoeProj up, down;                   // up: gate rows, then up rows
  const char* logits = nullptr;       // [tokens, experts], or null and
  const int32_t* ids = nullptr;       // [tokens, top_k]
  const float* weights = nullptr;
  int64_t logits_stride = 0;
  int tokens = 0, hidden = 0, inter = 0, experts = 0, top_k = 0, normalize = 0;
  int dtype = 0, s_dtype = 0, logits_dtype = 0, bits = 0, block = 0;
  hipStream_t stream = nullptr;
};
constexpr int MOE_MAX_TOKENS = 256, MOE_MAX_EXPERTS = 1024, MOE_MAX_TOP_K = 32;
size_t moe_workspace_bytes(int tokens, int hidden, int inter, int experts, int top_k);
hipError_t launch_moe(const MoeArgs& a, char* workspace);

struct SampleArgs {
  const char* logits = nullptr;       // [rows, vocab]
  int64_t stride = 0;                 // in elements
  int64_t rows = 0;
  int vocab = 0, dtype = 0;
  const float* temperature = nullptr; // [rows] each, or null
  const int32_t* top_k = nullptr;
  const float* top_p = nullptr;
  const float* min_p = nullptr;
  const float* uniform = nullptr;     // [rows]
  int32_t* tokens = nullptr;          // [rows]
  float* logprobs = nullptr;          // [rows] or null
  hipStream_t stream = nullptr;
};
constexpr int64_t SAMPLE_MAX_VOCAB = 1 << 22;
size_t sample_workspace_bytes(int64_t rows, int64_t vocab);
hipError_t launch_sample(const SampleArgs& a, char* workspace);

}  // namespace qmm
