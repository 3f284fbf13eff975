// Row operators around the attention core (no GEMM):
//
//   norm      r = x + residual;  y = r / sqrt(mean(r^2) + eps) * gamma      (mla_norm_rows)
//   quantise  s = max|y| / 448,  code = e4m3(y / s)  per 128 values        (mla_norm_rows, mla_quantize_rows)
//   append    c' = norm(c) gamma, k' = RoPE_pos(k), into the paged cache   (mla_append_rows)
//
// All three are bound by HBM when there are many rows and by latency when there are few.  So the vector
// kernels read every input once, with 16-byte loads into registers (all of a thread's loads in flight
// before the first use) or, for many rows, by bulk copies into a ring in shared memory, reduce with
// shuffles, and write every output once.  Of the kernels for other layouts, rows_any_kernel loads single
// elements, once; rows_long_kernel reads x and the residual twice, append_rows_any_kernel a normed latent.  Sums
// and statistics are fp32, nothing is rounded before it is stored.
#include "mla_internal.cuh"
#include "rows.cuh"
#include "sm100_f8.cuh"

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
// fp32, 1 for an all-zero block.  Between 2^-100 and the largest float that is mla_append_cache's decision, so both
// write the same codes.  Below 2^-100 the block takes 2^-100's scale (448 / amax overflows under about 2^-119, as it
// does there), and a NaN amax (max_nan) makes the block NaN, where that call's maximum leaves NaN out.
__device__ __forceinline__ void block_scale(float amax, float& s, float& inv) {
  const float floor_ = 7.888609052210118e-31f;  // 2^-100
  const float a = amax < floor_ ? floor_ : amax;  // (a NaN stays)
  s = amax == 0.f ? 1.f : __fdiv_rn(a, 448.f);
  inv = amax == 0.f ? 1.f : __fdiv_rn(448.f, a);
}

// Eight consecutive values as four packed fp32 pairs: the adds, products and sums of squares then take
// one instruction for two values (these kernels issue for half of their time at full bandwidth).
struct Eight {
  uint64_t p[4];
};

// two E4M3 codes (round to nearest even, saturating; NaN stays NaN), a in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ Eight zero8() { return Eight{{0ull, 0ull, 0ull, 0ull}}; }
// 16-byte accesses
__device__ __forceinline__ Eight load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Eight v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return v;
}
__device__ __forceinline__ Eight load8(const float* p) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0], b = reinterpret_cast<const ulonglong2*>(p)[1];
  return Eight{{a.x, a.y, b.x, b.y}};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Eight& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(v.p[i], lo, hi);
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const Eight& v) {
  reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(v.p[0], v.p[1]);
  reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(v.p[2], v.p[3]);
}
__device__ __forceinline__ Eight add8(const Eight& a, const Eight& b) {
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = add2(a.p[i], b.p[i]);
  return r;
}
__device__ __forceinline__ Eight mul8(const Eight& a, const Eight& b) {
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = mul2(a.p[i], b.p[i]);
  return r;
}
__device__ __forceinline__ Eight scale8(const Eight& a, float f) {
  const uint64_t f2 = pack2(f, f);
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = mul2(a.p[i], f2);
  return r;
}
// running sums of squares (even and odd values apart), and the pair's sum
__device__ __forceinline__ void squares8(uint64_t& ss, const Eight& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) ss = fma2(v.p[i], v.p[i], ss);
}
__device__ __forceinline__ float pair_sum(uint64_t ss) {
  float lo, hi;
  unpack2(ss, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ uint2 codes8(const Eight& v, float inv) {
  const Eight x = scale8(v, inv);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(x.p[i], lo, hi);
    q[i] = e4m3x2(lo, hi);
  }
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}
__device__ __forceinline__ float amax8(const Eight& v) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(v.p[i], lo, hi);
    m = max_nan(m, max_nan(fabsf(lo), fabsf(hi)));
  }
  return m;
}
// maximum over the 16 lanes that hold one block of 128 values
__device__ __forceinline__ float amax_block(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// Scales and reciprocals of CH blocks at once: lane i of each 16 divides for block i and the others get
// its results (a division is some 20 instructions; a thread's CH blocks would take 2 CH of them).
template <int CH>
__device__ __forceinline__ void block_scales(const float (&amax)[CH], float (&s)[CH], float (&inv)[CH]) {
  float mine = amax[0];
#pragma unroll
  for (int i = 1; i < CH; ++i)
    if (threadIdx.x % 16 == i) mine = amax[i];
  float ms, mi;
  block_scale(mine, ms, mi);
  if (CH == 1) {
    s[0] = ms;
    inv[0] = mi;
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      s[i] = __shfl_sync(0xffffffffu, ms, i, 16);
      inv[i] = __shfl_sync(0xffffffffu, mi, i, 16);
    }
  }
}

// Sum over the CTA (whole warps), the same value in every thread; one barrier.
__device__ __forceinline__ float cta_sum(float v, float* part) {
  v = warp_sum(v);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  const int n = blockDim.x / 32, lane = threadIdx.x % 32;
  return warp_sum(lane < n ? part[lane] : 0.f);
}

// ------------------------------------------------------------------ quantise, vector path
// A warp takes 512 values of a row, two chunks of 8 a lane, so 16 neighbouring lanes hold one 128-value
// block.  4096 x 16384 bf16: 36 us, 5.6 TB/s (one chunk a lane 45 us, four 36; a CTA per row 45).
constexpr int RQ_WARPS = 8;

template <typename T>
__global__ void __launch_bounds__(RQ_WARPS * 32) rows_quantize_kernel(const RowsArgs a, int units) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const unsigned unit = blockIdx.x * RQ_WARPS + threadIdx.x / 32;
  const long row = unit / (unsigned)units;
  if (row >= a.n_tok) return;
  const int chunks = a.width / 8, c0 = (int)(unit % (unsigned)units) * 64 + lane;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  Eight v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = c0 + 32 * i < chunks ? load8(x + 8l * (c0 + 32 * i)) : zero8();
  uint8_t* q = a.codes + row * a.codes_ld;
  float* sc = a.scales + row * ((a.width + 127) / 128);
  float m[2], s[2], inv[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) m[i] = amax_block(amax8(v[i]));
  block_scales<2>(m, s, inv);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = c0 + 32 * i;
    if (c < chunks) {
      *reinterpret_cast<uint2*>(q + 8l * c) = codes8(v[i], inv[i]);
      if (c % 16 == 0) sc[c / 16] = s[i];
    }
  }
}

// ------------------------------------------------------------------ norm, vector path
// One CTA per row: thread i holds chunks i, i + blockDim, ... of 8 values, CH of them, so 16
// neighbouring lanes hold one 128-value block.
template <typename T, int CH, int NT>
__global__ void __launch_bounds__(NT) rows_kernel(const RowsArgs a) {
  __shared__ float part[32];
  griddep_wait();
  griddep_launch_dependents();
  const long row = blockIdx.x;
  const int chunks = a.width / 8, c0 = threadIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_ld : nullptr;
  const T* gamma = static_cast<const T*>(a.gamma);
  Eight v[CH], g[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * blockDim.x;
    v[i] = c < chunks ? load8(x + 8l * c) : zero8();
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = c0 + i * blockDim.x;
      if (c < chunks) v[i] = add8(v[i], load8(res + 8l * c));
    }
  }
  if (gamma) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = c0 + i * blockDim.x;
      g[i] = c < chunks ? load8(gamma + 8l * c) : zero8();
    }
  }
  uint64_t sq = 0ull;
#pragma unroll
  for (int i = 0; i < CH; ++i) squares8(sq, v[i]);
  const float inv = __frsqrt_rn(cta_sum(pair_sum(sq), part) / (float)a.width + a.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + i * blockDim.x;
    const bool in = c < chunks;
    if (in && a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_ld + 8l * c, v[i]);
    v[i] = scale8(v[i], inv);
    if (gamma) v[i] = mul8(v[i], g[i]);
    if (in && a.y) store8(static_cast<T*>(a.y) + row * a.y_ld + 8l * c, v[i]);
  }
  if (a.codes) {
    uint8_t* q = a.codes + row * a.codes_ld;
    float* sc = a.scales + row * ((a.width + 127) / 128);
    float m[CH], s[CH], iv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) m[i] = amax_block(amax8(v[i]));
    block_scales<CH>(m, s, iv);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = c0 + i * blockDim.x;
      if (c < chunks) {
        *reinterpret_cast<uint2*>(q + 8l * c) = codes8(v[i], iv[i]);
        if (c % 16 == 0) sc[c / 16] = s[i];
      }
    }
  }
}

// Rows of at most 2048 values: a chunk a thread, and a CTA walks rows blockIdx, blockIdx + gridDim, ...
// with the next row's loads under way (a row per CTA left 16384 x 1536 at 2.7 TB/s: its CTAs come
// and go faster than they are launched).
template <typename T>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}

template <typename T>
__global__ void __launch_bounds__(256) rows_loop_kernel(const RowsArgs a) {
  __shared__ float part[2][32];  // alternating, so one barrier a row is enough
  griddep_wait();
  griddep_launch_dependents();
  const int c = threadIdx.x, lane = threadIdx.x % 32;
  const bool in = c < a.width / 8;
  const T* x = static_cast<const T*>(a.x) + 8 * c;
  const T* res = static_cast<const T*>(a.residual) + 8 * c;
  const Eight g = in && a.gamma ? load8(static_cast<const T*>(a.gamma) + 8 * c) : zero8();
  Raw8<T> nx = {}, nr = {};
  long row = blockIdx.x;
  if (in) {
    nx = raw8(x + row * a.x_ld);
    if (a.residual) nr = raw8(res + row * a.residual_ld);
  }
  for (int turn = 0; row < a.n_tok; row += gridDim.x, turn ^= 1) {
    Eight v = zero8();
    if (in) {
      v = load8(reinterpret_cast<const T*>(&nx));
      if (a.residual) v = add8(v, load8(reinterpret_cast<const T*>(&nr)));
    }
    const long next = row + gridDim.x;
    if (in && next < a.n_tok) {
      nx = raw8(x + next * a.x_ld);
      if (a.residual) nr = raw8(res + next * a.residual_ld);
    }
    uint64_t sq = 0ull;
    squares8(sq, v);
    const float ss = warp_sum(pair_sum(sq));
    if (lane == 0) part[turn][threadIdx.x / 32] = ss;
    __syncthreads();
    const float inv =
        __frsqrt_rn(warp_sum(lane < (int)blockDim.x / 32 ? part[turn][lane] : 0.f) / (float)a.width + a.eps);
    if (in && a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_ld + 8 * c, v);
    v = scale8(v, inv);
    if (a.gamma) v = mul8(v, g);
    if (in && a.y) store8(static_cast<T*>(a.y) + row * a.y_ld + 8 * c, v);
    if (a.codes) {
      float s, iv;
      block_scale(amax_block(amax8(v)), s, iv);
      if (in) {
        *reinterpret_cast<uint2*>(a.codes + row * a.codes_ld + 8 * c) = codes8(v, iv);
        if (c % 16 == 0) a.scales[row * ((a.width + 127) / 128) + c / 16] = s;
      }
    }
  }
}

// ------------------------------------------------------------------ norm of narrow rows
// One warp per row, CH chunks of 8 values a lane, no barrier.
constexpr int RW_WARPS = 4;

template <typename T, int CH>
__global__ void __launch_bounds__(RW_WARPS * 32) rows_warp_kernel(const RowsArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long row = (long)blockIdx.x * RW_WARPS + threadIdx.x / 32;
  if (row >= a.n_tok) return;
  const int chunks = a.width / 8;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_ld : nullptr;
  const T* gamma = static_cast<const T*>(a.gamma);
  Eight v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] = lane + 32 * i < chunks ? load8(x + 8 * (lane + 32 * i)) : zero8();
  uint64_t sq = 0ull;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + 32 * i;
    if (res && c < chunks) v[i] = add8(v[i], load8(res + 8 * c));
    squares8(sq, v[i]);
  }
  const float inv = __frsqrt_rn(warp_sum(pair_sum(sq)) / (float)a.width + a.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + 32 * i;
    const bool in = c < chunks;
    if (in) {
      if (a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_ld + 8 * c, v[i]);
      v[i] = scale8(v[i], inv);
      if (gamma) v[i] = mul8(v[i], load8(gamma + 8 * c));
      if (a.y) store8(static_cast<T*>(a.y) + row * a.y_ld + 8 * c, v[i]);
    }
    if (a.codes) {
      float s, iv;
      block_scale(amax_block(amax8(v[i])), s, iv);
      if (in) {
        *reinterpret_cast<uint2*>(a.codes + row * a.codes_ld + 8 * c) = codes8(v[i], iv);
        if (c % 16 == 0) a.scales[row * ((a.width + 127) / 128) + c / 16] = s;
      }
    }
  }
}

// ------------------------------------------------------------------ norm of many rows
// A CTA walks rows blockIdx, blockIdx + gridDim, ... with a ring of rows in shared memory that bulk
// copies fill ahead of it, so loads are in flight through the barriers, sums and stores of a row (the
// kernel above, a row per CTA, takes 129 us for 8191 x 7168 with the residual, this one 87: 6.1
// TB/s).  A stage holds a row of x and, after it, the residual's; it is refilled once
// every thread has its values in registers, which the barrier of the row's sum shows.
constexpr int RS_MAX_STAGES = 8;
constexpr int RS_SMEM = 220 * 1024;  // of an SM, for its streaming CTAs
constexpr int RS_ROWS = 300;         // per CTA of an SM: about two rows each
constexpr int LOOP_THREADS = 1024;   // threads of an SM's walking CTAs (1536 and 2048: 8 and 2 % slower)

template <typename T, int CH, int NT>
__global__ void __launch_bounds__(NT) rows_stream_kernel(const RowsArgs a, int stages, int gamma_staged) {
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
  const float inv_width = 1.f / (float)a.width;
  // The weight is kept in shared memory (the L1 left beside the ring does not hold it), except where
  // the sum and the normed rows are both written: there, read from L2 for each row, it was the faster
  // (8191 x 7168 with the residual: 87 us against 98; with 8-bit rows and the sum alone 73 against 69).
  const T* gamma = static_cast<const T*>(a.gamma);
  if (gamma_staged) {
    gamma = reinterpret_cast<const T*>(ring + (size_t)stages * stage_bytes);
    for (int c = threadIdx.x; c < chunks; c += blockDim.x)
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k)
        reinterpret_cast<uint4*>(ring + (size_t)stages * stage_bytes)[c * (sizeof(T) / 2) + k] =
            static_cast<const uint4*>(a.gamma)[c * (sizeof(T) / 2) + k];
  }
  int s = 0;
  uint32_t ph = 0, turn = 0;
  for (long row = blockIdx.x; row < a.n_tok; row += stride, turn ^= 1) {
    const bool landed = mbar_wait(&full[s], ph);
    const T* x = reinterpret_cast<const T*>(ring + (size_t)s * stage_bytes);
    Eight v[CH];
    uint64_t sq = 0ull;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      v[i] = zero8();
      if (c < chunks) {
        v[i] = load8(x + 8 * c);
        if (a.residual) v[i] = add8(v[i], load8(x + a.width + 8 * c));
      }
      squares8(sq, v[i]);
    }
    float ss = pair_sum(sq);
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
      if (c < chunks) {
        if (a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_ld + 8 * c, v[i]);
        v[i] = scale8(v[i], inv);
        if (gamma) v[i] = mul8(v[i], load8(gamma + 8 * c));
        if (a.y) store8(static_cast<T*>(a.y) + row * a.y_ld + 8 * c, v[i]);
      }
      if (a.codes) {
        float sc, iv;
        block_scale(amax_block(amax8(v[i])), sc, iv);
        if (c < chunks) {
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
// Element accesses: any width, alignment and leading dimension.  `units` warps share a row, each with J
// blocks of 128 values in registers (lane l holds l, l + 32, l + 64, l + 96 of a block), so all loads
// of a thread are in flight at once and the row is read once.  Where a norm's row takes more than one warp
// they are a CTA; else, and without a norm, the warps are independent.  4000 x 7169 bf16 with the residual
// and every output: 103 us (two passes over the row by 256 threads took 134), one such row 5.0 (15).
// Every value is read before any output of it is written, so sum_out and y may be the inputs' own memory.
template <typename T, bool NORM, int J>
__global__ void __launch_bounds__(1024) rows_any_kernel(const RowsArgs a, int units) {
  __shared__ float part[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const unsigned unit = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const long row = unit / (unsigned)units;
  if (row >= a.n_tok) return;  // (never a part of a row's warps)
  const int b0 = (int)(unit % (unsigned)units), blocks = (a.width + 127) / 128;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  T in[J][4];
  float v[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = (b0 + j * units) * 128 + lane + 32 * i;
      in[j][i] = k < a.width ? x[k] : from_f32<T>(0.f);
    }
  if (NORM && a.residual) {
    const T* res = static_cast<const T*>(a.residual) + row * a.residual_ld;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = (b0 + j * units) * 128 + lane + 32 * i;
        v[j][i] = k < a.width ? to_f32(res[k]) : 0.f;
      }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] += to_f32(in[j][i]);
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = to_f32(in[j][i]);
  }
  const T* gamma = NORM ? static_cast<const T*>(a.gamma) : nullptr;
  if (J <= 2 && gamma) {  // under way during the sum (more blocks leave no registers for it)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = (b0 + j * units) * 128 + lane + 32 * i;
        in[j][i] = k < a.width ? gamma[k] : from_f32<T>(0.f);
      }
  }
  float inv = 1.f;
  if (NORM) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    inv = __frsqrt_rn((units > 1 ? cta_sum(ss, part) : warp_sum(ss)) / (float)a.width + a.eps);
  }
  T* so = NORM && a.sum_out ? static_cast<T*>(a.sum_out) + row * a.sum_ld : nullptr;
  T* y = NORM && a.y ? static_cast<T*>(a.y) + row * a.y_ld : nullptr;
  uint8_t* q = a.codes ? a.codes + row * a.codes_ld : nullptr;
  float m[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    m[j] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = (b0 + j * units) * 128 + lane + 32 * i;
      if (k < a.width) {
        if (so) so[k] = from_f32<T>(v[j][i]);
        if (NORM) v[j][i] = gamma ? v[j][i] * inv * to_f32(J <= 2 ? in[j][i] : gamma[k]) : v[j][i] * inv;
        if (y) y[k] = from_f32<T>(v[j][i]);
        m[j] = max_nan(m[j], fabsf(v[j][i]));
      }
    }
  }
  if (!q) return;
  // maxima of the J blocks, block j's in the lanes with lane % J == j; each lane divides for its block
#pragma unroll
  for (int o = 1; o < J; o *= 2)
#pragma unroll
    for (int j = 0; j < J; j += 2 * o) {
      const bool odd = (lane & o) != 0;
      m[j] = max_nan(odd ? m[j + o] : m[j], __shfl_xor_sync(0xffffffffu, odd ? m[j] : m[j + o], o));
    }
#pragma unroll
  for (int o = J; o < 32; o *= 2) m[0] = max_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
  float ms, mi;
  block_scale(m[0], ms, mi);
  const int mine = b0 + lane * units;
  if (lane < J && mine < blocks) a.scales[row * blocks + mine] = ms;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float iv = __shfl_sync(0xffffffffu, mi, j);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const int k = (b0 + j * units) * 128 + lane + 32 * i;
      const uint32_t c = e4m3x2(__fmul_rn(v[j][i], iv), __fmul_rn(v[j][i + 1], iv));
      if (k < a.width) q[k] = (uint8_t)c;
      if (k + 32 < a.width) q[k + 32] = (uint8_t)(c >> 8);
    }
  }
}

// Norm of rows that neither this nor the vector kernels hold: one CTA per row, read twice (statistics,
// then outputs).  Its loops take as long as the width says, so it does not let the next grid start early (which would
// count its bounded waits from its own start).
template <typename T>
__global__ void __launch_bounds__(1024) rows_long_kernel(const RowsArgs a) {
  __shared__ float part[32];
  griddep_wait();
  const long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_ld : nullptr;
  const T* gamma = static_cast<const T*>(a.gamma);
  float ss = 0.f;
  for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
    const float r = to_f32(x[i]) + (res ? to_f32(res[i]) : 0.f);
    ss = fmaf(r, r, ss);
  }
  const float inv = __frsqrt_rn(cta_sum(ss, part) / (float)a.width + a.eps);
  T* so = a.sum_out ? static_cast<T*>(a.sum_out) + row * a.sum_ld : nullptr;
  T* y = a.y ? static_cast<T*>(a.y) + row * a.y_ld : nullptr;
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
        v[i] = gamma ? r * inv * to_f32(gamma[k]) : r * inv;
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
  int page_shift;  // log2 of page_size, or -1 when it is no power of two (a division is some 30 instructions)
  CacheView cv;
  int* err;
};

__device__ __forceinline__ int page_of(const AppendParams& p, int pos) {
  return p.page_shift >= 0 ? pos >> p.page_shift : pos / p.cv.page_size;
}

// Where a token goes: its page id (or what is wrong with it: PLACE_SEQ, PLACE_POS; an id outside the
// cache stays as it was read) and position.
constexpr int PLACE_SEQ = -0x7fffffff, PLACE_POS = PLACE_SEQ + 1;
struct Place {
  int seq, pos, pid;
  int row;  // of the page
};
__device__ __forceinline__ Place place_of(const AppendParams& p, int seq, int pos) {
  Place r = {seq, pos, PLACE_SEQ, 0};
  if (seq < 0 || seq >= p.cv.num_seqs) return r;
  r.pid = PLACE_POS;
  if (pos < 0 || pos >= p.rope_rows) return r;
  const int page = page_of(p, pos);
  if (page >= p.cv.max_pages) return r;
  r.row = pos - page * p.cv.page_size;
  r.pid = p.cv.block_table[(long)seq * p.cv.max_pages + page];
  return r;
}
// records why a token is skipped
__device__ __forceinline__ void report(const AppendParams& p, const Place& r) {
  if (r.pid == PLACE_SEQ && (r.seq < 0 || r.seq >= p.cv.num_seqs))
    record_error(p.err, ERR_SEQ, r.seq);
  else if (r.pid == PLACE_POS && (r.pos < 0 || r.pos >= p.rope_rows || page_of(p, r.pos) >= p.cv.max_pages))
    record_error(p.err, ERR_POS, r.pos);
  else
    record_error(p.err, ERR_PAGE, r.pid);
}

constexpr int AR_WARPS = 4;

// LANES lanes (16 or 32) per token: lane l holds chunks l, l + LANES, ... of 8 latent values (CH of
// them, 16 lanes a 128-value block) and one chunk of the rotary key below d_rope / 8 lanes.  A group of
// lanes walks tokens w, w + (groups of the grid), ... with the next token's row and its page id (whose
// position came one token earlier still) under way; a token a warp waited for each of these in turn.
// With 16 lanes a warp's instructions serve two tokens, and these kernels issue for half of their time.
// 40007 bf16 tokens of 512 + 64: 18.7 us, 5.5 TB/s (32 lanes 21.2; without the prefetch 25), into the
// 8-bit cache 19.1 (22.8): a fifth fewer bytes in the same time, so instructions bound that form (the maxima over
// 16 lanes, the scales by shuffles, the conversions).
template <typename T, int LANES, int CH, bool FP8>
__global__ void __launch_bounds__(AR_WARPS * 32) append_rows_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int PER_WARP = 32 / LANES;
  const int lane = threadIdx.x % LANES;
  const long stride = (long)gridDim.x * AR_WARPS * PER_WARP;
  const T* gamma = static_cast<const T*>(p.gamma);
  const int chunks = p.d_c / 8;
  const bool rot = lane < p.d_rope / 8;
  Raw8<T> g[CH], nv[CH], nk = {};
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    g[i] = {};
    nv[i] = {};
    if (gamma && lane + LANES * i < chunks) g[i] = raw8(gamma + 8 * (lane + LANES * i));
  }
  // first token of the warp (the same in all lanes), and this group's
  long t0 = ((long)blockIdx.x * AR_WARPS + threadIdx.x / 32) * PER_WARP;
  const int sub = threadIdx.x % 32 / LANES;
  int seq = 0, ps = 0;  // of the token after the current one
  auto where = [&](long t) {
    if (t >= p.T) return;
    seq = p.seq_idx[t];
    ps = p.pos[t];
  };
  Place here = {0, 0, PLACE_SEQ, 0};
  auto fetch = [&](long t) {
    if (t >= p.T) return;
    const T* src = static_cast<const T*>(p.kv) + t * p.kv_ld;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (lane + LANES * i < chunks) nv[i] = raw8(src + 8 * (lane + LANES * i));
    if (rot) nk = raw8(src + p.d_c + 8 * lane);
    here = place_of(p, seq, ps);
  };
  where(t0 + sub);
  fetch(t0 + sub);
  where(t0 + sub + stride);
  for (; t0 < p.T; t0 += stride) {
    const long t = t0 + sub;
    Eight v[CH], k = load8(reinterpret_cast<const T*>(&nk));
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = load8(reinterpret_cast<const T*>(&nv[i]));
    const Place now = here;
    const bool ok = t < p.T && now.pid >= 0 && now.pid < p.cv.num_pages;
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rot && ok) {
      const long at = (long)now.pos * (p.d_rope / 2) + 4 * lane;
      cs = *reinterpret_cast<const float4*>(p.rcos + at);
      sn = *reinterpret_cast<const float4*>(p.rsin + at);
    }
    fetch(t + stride);
    where(t + 2 * stride);
    if (t < p.T && !ok && lane == 0) report(p, now);
    const long slot = (long)now.pid * p.cv.page_size + now.row;  // (used where ok)
    if (gamma) {
      uint64_t sq = 0ull;
#pragma unroll
      for (int i = 0; i < CH; ++i) squares8(sq, v[i]);
      float ss = pair_sum(sq);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = __frsqrt_rn(ss / (float)p.d_c + p.eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) v[i] = mul8(scale8(v[i], inv), load8(reinterpret_cast<const T*>(&g[i])));
    }
    const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      unpack2(k.p[j], a, b);
      k.p[j] = pack2(a * cc[j] - b * ss[j], a * ss[j] + b * cc[j]);
    }
    if (FP8) {
      uint8_t* q = static_cast<uint8_t*>(p.cv.rows) + slot * p.d_c;
      float* sc = p.cv.scales + slot * (p.d_c / 128);
      float m[CH], s[CH], inv[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i) m[i] = amax_block(amax8(v[i]));
      block_scales<CH>(m, s, inv);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = lane + LANES * i;
        if (ok && c < chunks) {
          *reinterpret_cast<uint2*>(q + 8 * c) = codes8(v[i], inv[i]);
          if (c % 16 == 0) sc[c / 16] = s[i];
        }
      }
      if (ok && rot) store8(static_cast<__nv_bfloat16*>(p.cv.rope) + slot * p.d_rope + 8 * lane, k);
    } else {
      T* row = static_cast<T*>(p.cv.rows) + slot * (p.d_c + p.d_rope);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = lane + LANES * i;
        if (ok && c < chunks) store8(row + 8 * c, v[i]);
      }
      if (ok && rot) store8(row + p.d_c + 8 * lane, k);
    }
  }
}

// Any d_c, d_rope, alignment and leading dimension: one warp per token, element accesses, the
// latent part read twice when it is normed.  40007 tokens of 512 + 64 in rows of 577: bf16 31 us, float 41, into the
// 8-bit cache 42 (vector kernel 19, 33, 19): bound by the number of 2- and 1-byte accesses.  (No early start of the
// next grid, as in rows_long_kernel.)
template <typename T, bool FP8>
__global__ void __launch_bounds__(AR_WARPS * 32) append_rows_any_kernel(const AppendParams p) {
  griddep_wait();
  const int lane = threadIdx.x % 32;
  const long t = (long)blockIdx.x * AR_WARPS + threadIdx.x / 32;
  if (t >= p.T) return;
  const T* src = static_cast<const T*>(p.kv) + t * p.kv_ld;
  const T* gamma = static_cast<const T*>(p.gamma);
  const Place at = place_of(p, p.seq_idx[t], p.pos[t]);
  if (at.pid < 0 || at.pid >= p.cv.num_pages) {
    if (lane == 0) report(p, at);
    return;
  }
  const int ps = at.pos;
  const long slot = (long)at.pid * p.cv.page_size + at.row;
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
    // Blocks a warp: two for rows that come few at a time, else four (us on B200, two / four: norm 64 x 7001
    // 5.3 / 6.9, 4000 x 7169 bf16 128 / 103; quantise 64 x 7001 1.8 / 2.0, 3000 x 9001 bf16 32 / 29), but two
    // for the quantisation of floats (3000 x 9001 32 / 38).
    const bool few = a.n_tok <= 592;
    const int blocks = (a.width + 127) / 128;
    if (norm && blocks > 4) {  // a row per CTA
      if (blocks > 128) return launch_pdl(rows_long_kernel<T>, (unsigned)a.n_tok, 1024, st, 0, a);
      const int n = few && blocks <= 64 ? 2 : 4, units = (blocks + n - 1) / n;
      return launch_pdl(n == 2 ? rows_any_kernel<T, true, 2> : rows_any_kernel<T, true, 4>, (unsigned)a.n_tok, units * 32, st,
                        0, a, units);
    }
    const int n = !norm && (few || sizeof(T) == 4) ? 2 : 4, units = (blocks + n - 1) / n;
    const long ctas = ((long)units * a.n_tok + RW_WARPS - 1) / RW_WARPS;
    if (ctas > 0x3fffffffl) return kUnsupported;  // (unit numbers are 32 bits)
    auto kernel = norm ? rows_any_kernel<T, true, 4> : n == 2 ? rows_any_kernel<T, false, 2> : rows_any_kernel<T, false, 4>;
    return launch_pdl(kernel, (unsigned)ctas, RW_WARPS * 32, st, 0, a, units);
  }
  const int chunks = a.width / 8;
  if (!norm) {
    const int units = (chunks + 63) / 64;
    const long ctas = ((long)units * a.n_tok + RQ_WARPS - 1) / RQ_WARPS;
    if (ctas * RQ_WARPS > 0x7fffffffl) return kUnsupported;
    return launch_pdl(rows_quantize_kernel<T>, (unsigned)ctas, RQ_WARPS * 32, st, 0, a, units);
  }
  // Which kernel (us on B200, bf16; its neighbour's time in brackets):
  //   up to 512 values    a warp per row          16384 x 512: 11 [a CTA per row 18]
  //   up to 2048          a CTA per row, then     391 x 1536: 2.2 [walking CTAs 2.9]
  //                       walking CTAs            16384 x 1536 with the residual: 38 [43]
  //   up to 16384         a CTA per row, then     500 x 7168: 8.7 [streaming 9.9]
  //                       streaming CTAs          8191 x 7168: 87 [a CTA per row 129]; 3583 x 16384: 95 [132]
  //   up to 32768         a CTA per row
  // Streaming needs room for two stages.  bf16 rows always have it; float rows with a residual and a staged weight up to
  // 5632 values (two CTAs an SM) and from 8200 to 11264 (one), up to 7040 and 14080 without the weight's copy.  The
  // others stay with a CTA per row: float, residual, sum and 8-bit rows out, 2048 x 11264 53.9 (5.6 TB/s), 2048 x 12288 70.5
  // (4.6), whose kernel also spills (four chunks a thread in 64 registers).
  auto threads = [&](int ch) { return (unsigned)(((chunks + ch - 1) / ch + 31) / 32 * 32); };
  if (chunks <= 64)
    return launch_pdl(rows_warp_kernel<T, 2>, ((unsigned)a.n_tok + RW_WARPS - 1) / RW_WARPS, RW_WARPS * 32, st, 0, a);
  if (chunks <= 256) {
    const int at_once = 148 * (LOOP_THREADS / (int)threads(1));
    if (a.n_tok <= at_once) return launch_pdl(rows_kernel<T, 1, 256>, (unsigned)a.n_tok, threads(1), st, 0, a);
    return launch_pdl(rows_loop_kernel<T>, at_once, threads(1), st, 0, a);
  }
  const int per_sm = chunks <= 1024 ? 2 : 1, room = RS_SMEM / per_sm;
  const int one = a.width * (int)sizeof(T), row_bytes = a.residual ? 2 * one : one;
  const int fixed = a.gamma && !(a.sum_out && a.y) ? one : 0;  // the weight's copy (see the kernel)
  const int stages = min(RS_MAX_STAGES, (room - fixed) / row_bytes);
  if (a.n_tok >= RS_ROWS * per_sm && chunks <= 2048 && stages >= 2) {
    auto kernel = chunks <= 1024 ? rows_stream_kernel<T, 2, 512> : rows_stream_kernel<T, 2, 1024>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, min(a.n_tok, per_sm * 148), threads(2), st, stages * row_bytes + fixed, a, stages,
                      fixed > 0 ? 1 : 0);
  }
  if (chunks <= 1024) return launch_pdl(rows_kernel<T, 1, 1024>, (unsigned)a.n_tok, threads(1), st, 0, a);
  return launch_pdl(rows_kernel<T, 4, 1024>, (unsigned)a.n_tok, threads(4), st, 0, a);
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
  // as many CTAs as run at once
  auto go = [&](auto kernel, int per_warp, int per_sm) {
    const long warps = ((long)p.T + per_warp - 1) / per_warp, ctas = (warps + AR_WARPS - 1) / AR_WARPS;
    return launch_pdl(kernel, (unsigned)(ctas < 148 * per_sm ? ctas : 148 * per_sm), AR_WARPS * 32, st, 0, p);
  };
  if (p.d_c <= 512 && p.d_rope <= 128) {
    // a token a warp while that is shorter: 16-bit rows until the SMs' four CTAs are full (1 row 1.7 us,
    // 592 rows 2.0, against 2.0 and 2.05 with 16 lanes; 4736 rows 3.75 against 3.05), float rows, whose
    // registers leave 16 lanes three CTAs an SM, up to 8192 (4736 rows 5.0 against 6.1; 20000 rows 18.6 against
    // 17.8)
    if (p.T <= (sizeof(T) == 4 ? 8192 : 592)) return go(append_rows_kernel<T, 32, 2, FP8>, 1, 4);
    return go(append_rows_kernel<T, 16, 4, FP8>, 2, sizeof(T) == 4 ? 3 : 4);
  }
  return go(append_rows_kernel<T, 32, 4, FP8>, 1, 3);
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
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (cv.page_size == 1 << s) p.page_shift = s;
  p.cv = cv;
  p.err = err;
  if (d.act_dtype == MLA_F32) return append_rows_impl<float, false>(p, st);
  if (cv.kind == MLA_FP8_E4M3) return append_rows_impl<__nv_bfloat16, true>(p, st);
  return append_rows_impl<__nv_bfloat16, false>(p, st);
}

}  // namespace mla
