// Row operators around the attention core (no GEMM):
//
//   norm      r = x + residual;  y = r / sqrt(mean(r^2) + eps) * gamma      (mla_norm_rows)
//   quantise  s = max|y| / 448,  code = e4m3(y / s)  per 128 values        (mla_norm_rows, mla_quantize_rows)
//   append    c' = norm(c) gamma, k' = RoPE_pos(k), into the paged cache   (mla_append_rows)
//
// All three are bound by HBM when there are many rows and by latency when there are few, so each
// reads every input once into registers (16-byte loads, all of a thread's loads in flight before
// the first use), reduces with shuffles, and writes every output once.  Sums and statistics are
// fp32, nothing is rounded before it is stored.
#include "mla_internal.cuh"
#include "rows.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace rows {

using namespace sm100;

// ------------------------------------------------------------------ helpers
// max that keeps a NaN (fmaxf drops it), so a block that holds one gets a NaN scale
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale and its reciprocal of a block whose largest magnitude is amax: amax / 448 and 448 / amax in
// fp32 (the append's decision, so both write the same codes), 1 for an all-zero block.  Below
// 2^-100 the block takes 2^-100's scale: 448 / amax would overflow under about 2^-119.
__device__ __forceinline__ void block_scale(float amax, float& s, float& inv) {
  const float floor_ = 7.888609052210118e-31f;  // 2^-100
  const float a = amax < floor_ ? floor_ : amax;  // (a NaN stays)
  s = amax == 0.f ? 1.f : __fdiv_rn(a, 448.f);
  inv = amax == 0.f ? 1.f : __fdiv_rn(448.f, a);
}

// two E4M3 codes (round to nearest even, saturating; NaN stays NaN), a in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// eight consecutive values in 16-byte accesses
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  uint2 q;
  q.x = e4m3x2(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv)) | (e4m3x2(__fmul_rn(v[2], inv), __fmul_rn(v[3], inv)) << 16);
  q.y = e4m3x2(__fmul_rn(v[4], inv), __fmul_rn(v[5], inv)) | (e4m3x2(__fmul_rn(v[6], inv), __fmul_rn(v[7], inv)) << 16);
  return q;
}
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}
// maximum over the 16 lanes that hold one block of 128 values
__device__ __forceinline__ float amax_block(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Sum over the CTA (whole warps), the same value in every thread; one barrier.
__device__ __forceinline__ float cta_sum(float v, float* part) {
  v = warp_sum(v);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  const int n = blockDim.x / 32, lane = threadIdx.x % 32;
  return warp_sum(lane < n ? part[lane] : 0.f);
}

// ------------------------------------------------------------------ norm / quantise, vector path
// Thread i of a row's CTA holds chunks i, i + blockDim, ... of 8 values, CH of them, so 16
// neighbouring lanes hold one 128-value block.  Without the norm a row is cut into segments
// of blockDim * CH chunks, one CTA each (nothing crosses a block).
template <typename T, int CH, int NT, bool NORM>
__global__ void __launch_bounds__(NT) rows_kernel(const RowsArgs a, int segments) {
  __shared__ float part[32];
  griddep_wait();
  griddep_launch_dependents();
  const long row = NORM ? blockIdx.x : blockIdx.x / segments;
  const int seg = NORM ? 0 : (int)(blockIdx.x % segments);
  const int chunks = a.width / 8;
  const int c0 = seg * blockDim.x * CH + threadIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* res = NORM && a.residual ? static_cast<const T*>(a.residual) + row * a.residual_ld : nullptr;
  const T* gamma = NORM ? static_cast<const T*>(a.gamma) : nullptr;
  float v[CH][8], g[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * blockDim.x;
    if (c < chunks)
      load8(x + 8l * c, v[i]);
    else
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
  }
  if (NORM) {
    if (res) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = c0 + i * blockDim.x;
        if (c < chunks) {
          float r[8];
          load8(res + 8l * c, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] += r[k];
        }
      }
    }
    if (gamma) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = c0 + i * blockDim.x;
        if (c < chunks) load8(gamma + 8l * c, g[i]);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
    const float inv = __frsqrt_rn(cta_sum(ss, part) / (float)a.width + a.eps);
    if (a.sum_out) {
      T* so = static_cast<T*>(a.sum_out) + row * a.sum_ld;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = c0 + i * blockDim.x;
        if (c < chunks) store8(so + 8l * c, v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = gamma ? v[i][k] * inv * g[i][k] : v[i][k] * inv;
    if (a.y) {
      T* y = static_cast<T*>(a.y) + row * a.y_ld;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = c0 + i * blockDim.x;
        if (c < chunks) store8(y + 8l * c, v[i]);
      }
    }
  }
  if (a.codes) {
    uint8_t* q = a.codes + row * a.codes_ld;
    float* sc = a.scales + row * ((a.width + 127) / 128);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = c0 + i * blockDim.x;
      const bool in = c < chunks;
      float s, inv;
      block_scale(amax_block(in ? amax8(v[i]) : 0.f), s, inv);
      if (in) {
        *reinterpret_cast<uint2*>(q + 8l * c) = codes8(v[i], inv);
        if (c % 16 == 0) sc[c / 16] = s;
      }
    }
  }
}

// ------------------------------------------------------------------ norm of many rows
// A CTA walks rows blockIdx, blockIdx + gridDim, ... with a ring of rows in shared memory that bulk
// copies fill ahead of it, so loads are in flight through the barriers, sums and stores of a row (the
// kernel above, a row per CTA, reached 4.1 TB/s on 8191 x 7168 with the residual; this one is noted
// at its launch).  A stage holds a row of x and, after it, the residual's; it is refilled once
// every thread has its values in registers, which the barrier of the row's sum shows.
constexpr int RS_MAX_STAGES = 8;
constexpr int RS_SMEM = 110 * 1024;
constexpr int RS_ROWS = 600;

template <typename T, int CH, int NT>
__global__ void __launch_bounds__(NT) rows_stream_kernel(const RowsArgs a, int stages) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ uint64_t full[RS_MAX_STAGES];
  __shared__ float part[2][32];  // alternating, so one barrier a row is enough
  const uint32_t row_bytes = (uint32_t)a.width * sizeof(T);
  const uint32_t stage_bytes = a.residual ? 2 * row_bytes : row_bytes;
  const long stride = gridDim.x;
  auto fetch = [&](long row, int s) {  // one thread
    mbar_arrive_expect_tx(&full[s], stage_bytes);
    uint8_t* st = ring + (size_t)s * stage_bytes;
    bulk_load(st, static_cast<const T*>(a.x) + row * a.x_ld, row_bytes, &full[s]);
    if (a.residual)
      bulk_load(st + row_bytes, static_cast<const T*>(a.residual) + row * a.residual_ld, row_bytes, &full[s]);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  if (threadIdx.x == 0) {
    griddep_launch_dependents();
    for (int s = 0; s < stages; ++s)
      if (blockIdx.x + s * stride < a.n_tok) fetch(blockIdx.x + s * stride, s);
  }
  const int chunks = a.width / 8;
  const T* gamma = static_cast<const T*>(a.gamma);
  float inv_width = 1.f / (float)a.width;
  int s = 0;
  uint32_t ph = 0, turn = 0;
  for (long row = blockIdx.x; row < a.n_tok; row += stride, turn ^= 1) {
    const bool landed = mbar_wait(&full[s], ph);
    const T* x = reinterpret_cast<const T*>(ring + (size_t)s * stage_bytes);
    float v[CH][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
      if (c < chunks) {
        load8(x + 8 * c, v[i]);
        if (a.residual) {
          float r[8];
          load8(x + a.width + 8 * c, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] += r[k];
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
    }
    ss = warp_sum(ss);
    if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = ss;
    if (!__syncthreads_and(landed ? 1 : 0)) {  // (all threads leave together)
      if (threadIdx.x == 0) {
        record_error(a.err, ERR_TIMEOUT, 70);
        // the loads under way land (bounded) before the CTA's shared memory goes
        for (int k = 0; k < stages && row + k * stride < a.n_tok; ++k)
          mbar_wait(&full[(s + k) % stages], s + k < stages ? ph : ph ^ 1);
      }
      break;
    }
    if (threadIdx.x == 0 && row + stages * stride < a.n_tok) fetch(row + stages * stride, s);
    const int lane = threadIdx.x % 32;
    ss = warp_sum(lane < (int)blockDim.x / 32 ? part[turn][lane] : 0.f);
    const float inv = __frsqrt_rn(ss * inv_width + a.eps);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      const bool in = c < chunks;
      if (in) {
        if (a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_ld + 8 * c, v[i]);
        float g[8];
        if (gamma) load8(gamma + 8 * c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = gamma ? v[i][k] * inv * g[k] : v[i][k] * inv;
        if (a.y) store8(static_cast<T*>(a.y) + row * a.y_ld + 8 * c, v[i]);
      }
      if (a.codes) {
        float sc, iv;
        block_scale(amax_block(in ? amax8(v[i]) : 0.f), sc, iv);
        if (in) {
          *reinterpret_cast<uint2*>(a.codes + row * a.codes_ld + 8 * c) = codes8(v[i], iv);
          if (c % 16 == 0) a.scales[row * ((a.width + 127) / 128) + c / 16] = sc;
        }
      }
    }
    if (++s == stages) {
      s = 0;
      ph ^= 1;
    }
  }
}

// ------------------------------------------------------------------ norm / quantise, any layout
// One CTA per row, element accesses: any width, alignment and leading dimension.  The row is
// read twice (statistics, then outputs); a thread reads an element before it writes any output
// of it, so sum_out and y may be the inputs' own memory.
template <typename T, bool NORM>
__global__ void __launch_bounds__(256) rows_any_kernel(const RowsArgs a) {
  __shared__ float part[32];
  griddep_wait();
  griddep_launch_dependents();
  const long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* res = NORM && a.residual ? static_cast<const T*>(a.residual) + row * a.residual_ld : nullptr;
  const T* gamma = NORM ? static_cast<const T*>(a.gamma) : nullptr;
  float inv = 1.f;
  if (NORM) {
    float ss = 0.f;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
      const float r = to_f32(x[i]) + (res ? to_f32(res[i]) : 0.f);
      ss = fmaf(r, r, ss);
    }
    inv = __frsqrt_rn(cta_sum(ss, part) / (float)a.width + a.eps);
  }
  T* so = NORM && a.sum_out ? static_cast<T*>(a.sum_out) + row * a.sum_ld : nullptr;
  T* y = NORM && a.y ? static_cast<T*>(a.y) + row * a.y_ld : nullptr;
  uint8_t* q = a.codes ? a.codes + row * a.codes_ld : nullptr;
  const int blocks = (a.width + 127) / 128;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int b = warp; b < blocks; b += blockDim.x / 32) {
    float v[4], m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = b * 128 + lane + 32 * i;
      v[i] = 0.f;
      if (k < a.width) {
        const float r = to_f32(x[k]) + (res ? to_f32(res[k]) : 0.f);
        v[i] = NORM ? (gamma ? r * inv * to_f32(gamma[k]) : r * inv) : r;
        if (so) so[k] = from_f32<T>(r);
        if (y) y[k] = from_f32<T>(v[i]);
        m = max_nan(m, fabsf(v[i]));
      }
    }
    if (q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      float s, iv;
      block_scale(m, s, iv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = b * 128 + lane + 32 * i;
        if (k < a.width) q[k] = f32_to_e4m3(__fmul_rn(v[i], iv));
      }
      if (lane == 0) a.scales[row * blocks + b] = s;
    }
  }
}

// ------------------------------------------------------------------ append of projected rows
struct AppendParams {
  const void* kv;
  int64_t kv_ld;
  int T, d_c, d_rope;
  const int32_t* seq_idx;
  const int32_t* pos;
  const void* gamma;
  float eps;
  const float* rcos;
  const float* rsin;
  int rope_rows;
  CacheView cv;
  int* err;
};

// Slot (page * page_size + offset) of token t, or -1 with the error recorded (by one lane).
__device__ __forceinline__ long slot_of(const AppendParams& p, int t, int& ps, bool report) {
  const int seq = p.seq_idx[t];
  ps = p.pos[t];
  if (seq < 0 || seq >= p.cv.num_seqs) {
    if (report) record_error(p.err, ERR_SEQ, seq);
    return -1;
  }
  if (ps < 0 || ps >= p.rope_rows || ps / p.cv.page_size >= p.cv.max_pages) {
    if (report) record_error(p.err, ERR_POS, ps);
    return -1;
  }
  const int pid = p.cv.block_table[(long)seq * p.cv.max_pages + ps / p.cv.page_size];
  if (pid < 0 || pid >= p.cv.num_pages) {
    if (report) record_error(p.err, ERR_PAGE, pid);
    return -1;
  }
  return (long)pid * p.cv.page_size + ps % p.cv.page_size;
}

constexpr int AR_WARPS = 4;

// One warp per token: lane l holds chunks l, l + 32, ... of 8 latent values (CH of them, 16 lanes a
// 128-value block) and, below d_rope / 8 lanes, one chunk of the rotary key.
template <typename T, int CH, bool FP8>
__global__ void __launch_bounds__(AR_WARPS * 32) append_rows_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long t = (long)blockIdx.x * AR_WARPS + threadIdx.x / 32;
  if (t >= p.T) return;
  const T* src = static_cast<const T*>(p.kv) + t * p.kv_ld;
  const T* gamma = static_cast<const T*>(p.gamma);
  const int chunks = p.d_c / 8;
  const bool rot = lane < p.d_rope / 8;
  float v[CH][8], g[CH][8], k[8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + 32 * i;
    if (c < chunks)
      load8(src + 8 * c, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
  }
  if (rot) load8(src + p.d_c + 8 * lane, k);
  if (gamma) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + 32 * i;
      if (c < chunks) load8(gamma + 8 * c, g[i]);
    }
  }
  int ps;
  const long slot = slot_of(p, (int)t, ps, lane == 0);
  if (slot < 0) return;
  if (rot) {
    const long at = (long)ps * (p.d_rope / 2) + 4 * lane;
    const float4 cs = *reinterpret_cast<const float4*>(p.rcos + at);
    const float4 sn = *reinterpret_cast<const float4*>(p.rsin + at);
    const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = k[2 * j], b = k[2 * j + 1];
      k[2 * j] = a * cc[j] - b * ss[j];
      k[2 * j + 1] = a * ss[j] + b * cc[j];
    }
  }
  if (gamma) {
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(v[i][j], v[i][j], sq);
    const float inv = __frsqrt_rn(warp_sum(sq) / (float)p.d_c + p.eps);
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * g[i][j];
  }
  if (FP8) {
    uint8_t* q = static_cast<uint8_t*>(p.cv.rows) + slot * p.d_c;
    float* sc = p.cv.scales + slot * (p.d_c / 128);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + 32 * i;
      const bool in = c < chunks;
      float s, inv;
      block_scale(amax_block(in ? amax8(v[i]) : 0.f), s, inv);
      if (in) {
        *reinterpret_cast<uint2*>(q + 8 * c) = codes8(v[i], inv);
        if (c % 16 == 0) sc[c / 16] = s;
      }
    }
    if (rot) store8(static_cast<__nv_bfloat16*>(p.cv.rope) + slot * p.d_rope + 8 * lane, k);
  } else {
    T* row = static_cast<T*>(p.cv.rows) + slot * (p.d_c + p.d_rope);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + 32 * i;
      if (c < chunks) store8(row + 8 * c, v[i]);
    }
    if (rot) store8(row + p.d_c + 8 * lane, k);
  }
}

// Any d_c, d_rope, alignment and leading dimension: one warp per token, element accesses, the
// latent part read twice when it is normed.
template <typename T, bool FP8>
__global__ void __launch_bounds__(AR_WARPS * 32) append_rows_any_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long t = (long)blockIdx.x * AR_WARPS + threadIdx.x / 32;
  if (t >= p.T) return;
  const T* src = static_cast<const T*>(p.kv) + t * p.kv_ld;
  const T* gamma = static_cast<const T*>(p.gamma);
  int ps;
  const long slot = slot_of(p, (int)t, ps, lane == 0);
  if (slot < 0) return;
  float inv = 1.f;
  if (gamma) {
    float sq = 0.f;
    for (int i = lane; i < p.d_c; i += 32) {
      const float x = to_f32(src[i]);
      sq = fmaf(x, x, sq);
    }
    inv = __frsqrt_rn(warp_sum(sq) / (float)p.d_c + p.eps);
  }
  const int W = p.d_c + p.d_rope;
  T* row = FP8 ? nullptr : static_cast<T*>(p.cv.rows) + slot * W;
  for (int b = 0; b < (p.d_c + 127) / 128; ++b) {
    float v[4], m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = b * 128 + lane + 32 * i;
      v[i] = 0.f;
      if (c < p.d_c) {
        v[i] = to_f32(src[c]);
        if (gamma) v[i] = v[i] * inv * to_f32(gamma[c]);
        if (!FP8) row[c] = from_f32<T>(v[i]);
        m = max_nan(m, fabsf(v[i]));
      }
    }
    if (FP8) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      float s, iv;
      block_scale(m, s, iv);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        static_cast<uint8_t*>(p.cv.rows)[slot * p.d_c + b * 128 + lane + 32 * i] = f32_to_e4m3(__fmul_rn(v[i], iv));
      if (lane == 0) p.cv.scales[slot * (p.d_c / 128) + b] = s;
    }
  }
  const int half = p.d_rope / 2;
  for (int i = lane; i < half; i += 32) {
    const float a = to_f32(src[p.d_c + 2 * i]), b = to_f32(src[p.d_c + 2 * i + 1]);
    const float c = p.rcos[(long)ps * half + i], s = p.rsin[(long)ps * half + i];
    const float r0 = a * c - b * s, r1 = a * s + b * c;
    if (FP8) {
      __nv_bfloat16* kr = static_cast<__nv_bfloat16*>(p.cv.rope) + slot * p.d_rope;
      kr[2 * i] = __float2bfloat16_rn(r0);
      kr[2 * i + 1] = __float2bfloat16_rn(r1);
    } else {
      row[p.d_c + 2 * i] = from_f32<T>(r0);
      row[p.d_c + 2 * i + 1] = from_f32<T>(r1);
    }
  }
}

}  // namespace rows

// ------------------------------------------------------------------ host side
// Launch with programmatic stream serialization (the kernels wait before they read anything).
template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl(void (*kernel)(KArgs...), unsigned grid, unsigned block, cudaStream_t st, int smem, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

static bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <typename T>
static bool rows_vector_ok(const RowsArgs& a, bool norm) {
  const int per16 = 16 / (int)sizeof(T);
  auto ok = [&](const void* p, int64_t ld) { return !p || (aligned(p, 16) && ld % per16 == 0); };
  return a.width % 8 == 0 && (!norm || a.width <= 1024 * 8 * 4) && ok(a.x, a.x_ld) && ok(a.residual, a.residual_ld) &&
         ok(a.gamma, 0) && ok(a.sum_out, a.sum_ld) && ok(a.y, a.y_ld) &&
         (!a.codes || (aligned(a.codes, 8) && a.codes_ld % 8 == 0));
}

template <typename T>
static cudaError_t rows_impl(const RowsArgs& a, bool norm, cudaStream_t st) {
  using namespace rows;
  if (!rows_vector_ok<T>(a, norm)) {
    return norm ? launch_pdl(rows_any_kernel<T, true>, (unsigned)a.n_tok, 256, st, 0, a)
                : launch_pdl(rows_any_kernel<T, false>, (unsigned)a.n_tok, 256, st, 0, a);
  }
  const int chunks = a.width / 8;
  if (!norm) {
    const int nt = chunks >= 256 ? 256 : (chunks + 31) / 32 * 32;
    const long segments = (chunks + nt - 1) / nt;
    if (segments * a.n_tok > 0x7fffffffl) return kUnsupported;
    return launch_pdl(rows_kernel<T, 1, 256, false>, (unsigned)(segments * a.n_tok), nt, st, 0, a, (int)segments);
  }
  // many rows: persistent CTAs, two per SM, rows streamed through shared memory
  const int row_bytes = a.width * (int)sizeof(T) * (a.residual ? 2 : 1);
  const int stages = min(RS_MAX_STAGES, RS_SMEM / row_bytes);
  if (a.n_tok >= RS_ROWS && stages >= 2 && chunks > 256 && chunks <= 1024) {
    auto kernel = rows_stream_kernel<T, 2, 512>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RS_SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, min(a.n_tok, 2 * 148), ((chunks + 1) / 2 + 31) / 32 * 32, st, stages * row_bytes, a, stages);
  }
  auto threads = [&](int ch) { return (unsigned)(((chunks + ch - 1) / ch + 31) / 32 * 32); };
  if (chunks <= 256) return launch_pdl(rows_kernel<T, 1, 256, true>, (unsigned)a.n_tok, threads(1), st, 0, a, 1);
  if (chunks <= 1024) return launch_pdl(rows_kernel<T, 2, 512, true>, (unsigned)a.n_tok, threads(2), st, 0, a, 1);
  return launch_pdl(rows_kernel<T, 4, 1024, true>, (unsigned)a.n_tok, threads(4), st, 0, a, 1);
}

cudaError_t launch_rows(const RowsArgs& a, bool norm, cudaStream_t st) {
  return a.act == MLA_F32 ? rows_impl<float>(a, norm, st) : rows_impl<__nv_bfloat16>(a, norm, st);
}

template <typename T, bool FP8>
static cudaError_t append_rows_impl(const rows::AppendParams& p, cudaStream_t st) {
  using namespace rows;
  const long ctas = ((long)p.T + AR_WARPS - 1) / AR_WARPS;
  const int per16 = 16 / (int)sizeof(T);
  const bool vec = p.d_c % 8 == 0 && p.d_rope % 8 == 0 && p.d_c <= 1024 && p.d_rope <= 256 && p.kv_ld % per16 == 0 &&
                   aligned(p.kv, 16) && aligned(p.gamma, 16) && aligned(p.rcos, 16) && aligned(p.rsin, 16) &&
                   aligned(p.cv.rows, 16) && (!FP8 || aligned(p.cv.rope, 16));
  if (!vec) return launch_pdl(append_rows_any_kernel<T, FP8>, (unsigned)ctas, AR_WARPS * 32, st, 0, p);
  if (p.d_c <= 256) return launch_pdl(append_rows_kernel<T, 1, FP8>, (unsigned)ctas, AR_WARPS * 32, st, 0, p);
  if (p.d_c <= 512) return launch_pdl(append_rows_kernel<T, 2, FP8>, (unsigned)ctas, AR_WARPS * 32, st, 0, p);
  return launch_pdl(append_rows_kernel<T, 4, FP8>, (unsigned)ctas, AR_WARPS * 32, st, 0, p);
}

cudaError_t launch_append_rows(const mla_dims& d, const void* kv, int64_t kv_ld, int n_tok, const int32_t* seq_idx,
                               const int32_t* pos, const void* gamma, float eps, const float* rcos, const float* rsin,
                               int rope_rows, const CacheView& cv, int* err, cudaStream_t st) {
  rows::AppendParams p;
  p.kv = kv;
  p.kv_ld = kv_ld;
  p.T = n_tok;
  p.d_c = d.d_c;
  p.d_rope = d.d_rope;
  p.seq_idx = seq_idx;
  p.pos = pos;
  p.gamma = gamma;
  p.eps = eps;
  p.rcos = rcos;
  p.rsin = rsin;
  p.rope_rows = rope_rows;
  p.cv = cv;
  p.err = err;
  if (d.act_dtype == MLA_F32) return append_rows_impl<float, false>(p, st);
  if (cv.kind == MLA_FP8_E4M3) return append_rows_impl<__nv_bfloat16, true>(p, st);
  return append_rows_impl<__nv_bfloat16, false>(p, st);
}

}  // namespace mla
