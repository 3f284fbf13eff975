// 8-bit projection with block scales:
//
//   out[t, n] = sum_b xs[t, b] ws[n / 128, b] sum_{k in block b} x[t, k] w[n, k],
//
// x and w E4M3, one fp32 scale per 128 values of a row of x and per 128 x 128 block of w.  The
// products of one block are summed without scales (exact products, fp32 sums), then the block's
// sum is scaled and added to an fp32 accumulator.
#include "mla_internal.cuh"
#include "proj_fp8.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace p8 {

using namespace sm100;

// ------------------------------------------------------------------ any layout
// fp32 FMA on the CUDA cores: 64 tokens x 64 outputs per CTA, 4 x 4 per thread, 16 values of K at
// a time.  Every width, alignment and leading dimension; the path of what the tensor-core
// kernels do not take.
template <typename T>
__global__ void __launch_bounds__(256) fp8_any_kernel(const Fp8Args a) {
  __shared__ float xs_s[16][64 + 4];
  __shared__ float ws_s[16][64 + 4];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const long t0 = (long)blockIdx.y * 64;
  const int n0 = blockIdx.x * 64;
  const int blocks = (a.K + 127) / 128;
  float acc[4][4] = {};
  for (int b = 0; b < blocks; ++b) {
    float part[4][4] = {};
    const int k_hi = min(a.K, (b + 1) * 128);
    for (int k0 = b * 128; k0 < k_hi; k0 += 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = tid + 256 * i, r = e / 16, k = e % 16;
        const bool in = k0 + k < k_hi;
        xs_s[k][r] = in && t0 + r < a.T ? e4m3_to_f32(a.x[(t0 + r) * a.x_ld + k0 + k]) : 0.f;
        ws_s[k][r] = in && n0 + r < a.N ? e4m3_to_f32(a.w[(long)(n0 + r) * a.K + k0 + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float x[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = xs_s[k][ty + 16 * i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = ws_s[k][tx + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(x[i], w[j], part[i][j]);
      }
      __syncthreads();
    }
    const float ws = a.ws[(long)(n0 / 128) * blocks + b];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long t = t0 + ty + 16 * i;
      const float s = t < a.T ? a.xs[t * blocks + b] * ws : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long t = t0 + ty + 16 * i;
    if (t >= a.T) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n < a.N) static_cast<T*>(a.out)[t * a.out_ld + n] = from_f32<T>(acc[i][j]);
    }
  }
}

}  // namespace p8

// ------------------------------------------------------------------ host side
static cudaError_t launch_fp8_any(const Fp8Args& a, cudaStream_t st) {
  if ((a.T + 63) / 64 > 65535) return kUnsupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + 63) / 64), (unsigned)((a.T + 63) / 64));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cudaError_t e = a.act == MLA_F32 ? cudaLaunchKernelEx(&cfg, p8::fp8_any_kernel<float>, a)
                                   : cudaLaunchKernelEx(&cfg, p8::fp8_any_kernel<__nv_bfloat16>, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_project_fp8(const Fp8Args& a, cudaStream_t st) { return launch_fp8_any(a, st); }

}  // namespace mla
