// Row operators around the attention core: norm, 8-bit quantisation, append of projected rows.
#pragma once
#include "mla_internal.cuh"

namespace mla {

struct RowsArgs {
  int act;                // mla_dtype of x, residual, gamma, sum_out, y
  const void* x;
  int64_t x_ld;
  const void* residual;   // or null
  int64_t residual_ld;
  const void* gamma;      // [width] or null
  int n_tok, width;
  float eps;
  void* sum_out;          // or null
  int64_t sum_ld;
  void* y;                // or null
  int64_t y_ld;
  uint8_t* codes;         // or null (then scales is null too)
  int64_t codes_ld;
  float* scales;          // [n_tok, ceil(width / 128)]
  int* err;
};

// y = norm ? rmsnorm(x + residual) * gamma : x, written as act rows and / or as E4M3 blocks.
cudaError_t launch_rows(const RowsArgs& a, bool norm, cudaStream_t st);

cudaError_t launch_append_rows(const mla_dims& d, const void* kv, int64_t kv_ld, int n_tok, const int32_t* seq_idx,
                               const int32_t* pos, const void* gamma, float eps, const float* rcos, const float* rsin,
                               int rope_rows, const CacheView& cv, int* err, cudaStream_t st);

}  // namespace mla
