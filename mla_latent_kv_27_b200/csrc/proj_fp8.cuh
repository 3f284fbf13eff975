// 8-bit projection with block scales.
#pragma once
#include "mla_internal.cuh"

namespace mla {

// out[t, n] = sum_b xs[t, b] ws[n / 128, b] sum_{k in block b} x[t, k] w[n, k]
struct Fp8Args {
  int act;              // mla_dtype of out
  const uint8_t* x;     // [T, K] E4M3, row stride x_ld
  int64_t x_ld;
  const float* xs;      // [T, ceil(K / 128)]
  const uint8_t* w;     // [N, K] E4M3
  const float* ws;      // [ceil(N / 128), ceil(K / 128)]
  int T, N, K;
  void* out;            // [T, N], row stride out_ld
  int64_t out_ld;
  int* err;
};

cudaError_t launch_project_fp8(const Fp8Args& a, cudaStream_t st);

}  // namespace mla
