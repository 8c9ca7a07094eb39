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
  uint8_t* codes = nullptr;                       // rows of code_cols bytes
  void* scales = nullptr;
  int code_cols = 0, blocks = 0;                  // of a row
  hipStream_t stream = nullptr;
};
constexpr int64_t NORM_MAX_COLS = 1 << 20;
hipError_t launch_rms_norm(const NormArgs& a);

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
