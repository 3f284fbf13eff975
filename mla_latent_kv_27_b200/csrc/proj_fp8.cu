// 8-bit projection with block scales:
//
//   out[t, n] = sum_b xs[t, b] ws[n / 128, b] sum_{k in block b} x[t, k] w[n, k],
//
// x and w E4M3, one fp32 scale per 128 values of a row of x and per 128 x 128 block of w.  The
// products of one block are summed without scales (exact products, fp32 sums), then the block's
// sum is scaled and added to an fp32 accumulator.
#include <cuda.h>
#include <cudaTypedefs.h>

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

// ------------------------------------------------------------------ few tokens
// Bound by reading the weights once.  They are the M = 128 operand of the MMA (TMEM lane = output),
// the tokens its N operand (BN columns), and the S CTAs of a cluster each take a range of the
// scale blocks, so that enough loads are in flight on every SM.  One stage is one scale block:
// 128 weight rows and BN token rows of 128 bytes, a single row of the 128-byte swizzle.  Each
// block's products go to a TMEM accumulator of their own (ND of them in turn); the promoting warps
// read it, scale it by xs[t, b] ws[n / 128, b] and add it to fp32 sums in registers.  At the end
// the S partial sums of an output meet in the shared memory of the CTA that owns its row (the
// idle stage ring, over distributed shared memory) and are added in rank order: no workspace, no
// atomics.
constexpr int A_BYTES = 128 * 128;

template <int BN>
struct SkCfg {
  static constexpr int OCC = BN <= 64 ? 2 : 1;                   // CTAs per SM
  static constexpr int NST = BN <= 32 ? 5 : BN == 64 ? 4 : 6;
  static constexpr int STAGE = A_BYTES + BN * 128;
  static constexpr int ND = 4;
  static constexpr uint32_t TCOLS = ND * BN;                     // 64 to 512 columns
  static constexpr int PW = BN <= 64 ? 4 : 8;                    // promoting warps
  static constexpr int CW = BN <= 64 ? BN : 64;                  // columns of one of them
  static constexpr int XC = (PW == 4 ? 256 : 128) / CW;          // scale blocks fetched at a time
  static constexpr int THREADS = 64 + PW * 32;
  static constexpr int XS_OFF = NST * STAGE;                     // per warp: [2][XC][CW] fp32
  static constexpr int BAR_OFF = XS_OFF + PW * 2 * XC * CW * 4;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  static constexpr int RLD = BN + 4;                             // receive row, floats (bank spread)
  static_assert((128 + 8) * RLD * 4 <= NST * STAGE, "the receive buffer aliases the stage ring");
  static_assert(OCC * (SMEM + 1024) <= 233472 && OCC * TCOLS <= 512, "CTAs per SM");
};

template <int BN>
struct SkBars {
  uint64_t full[SkCfg<BN>::NST], empty[SkCfg<BN>::NST], dfull[SkCfg<BN>::ND], dempty[SkCfg<BN>::ND];
  uint32_t tmem_base;
};

struct SkParams {
  const float* xs;
  const float* ws;
  int T, N, blocks, per_cta;  // blocks: scale blocks of K, per_cta of them for each CTA of a cluster
  void* out;
  long out_ld;
  int out_f32;
  int* err;
};

__device__ __forceinline__ void store_out(const SkParams& p, long t, int n, float v) {
  if (p.out_f32)
    static_cast<float*>(p.out)[t * p.out_ld + n] = v;
  else
    static_cast<__nv_bfloat16*>(p.out)[t * p.out_ld + n] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}
// CN (16 or 32) consecutive fp32 columns of this thread's TMEM lane, and the wait for them
template <int CN>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[CN]) {
  if constexpr (CN == 32)
    tmem_ld32(addr, v);
  else
    tmem_ld16(addr, v);
}
template <int CN>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[CN]) {
  if constexpr (CN == 32)
    tmem_wait_ld32(v);
  else
    tmem_wait_ld16(v);
}

template <int BN>
__global__ void __launch_bounds__(SkCfg<BN>::THREADS, SkCfg<BN>::OCC)
    fp8_skinny_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const SkParams p) {
  using C = SkCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  SkBars<BN>* bars = reinterpret_cast<SkBars<BN>*>(smem + C::BAR_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = gridDim.x, rank = blockIdx.x;
  const int n0 = blockIdx.y * 128;
  const int t0 = blockIdx.z * BN;
  const int b0 = rank * p.per_cta;
  const int nb = max(0, min(p.blocks, b0 + p.per_cta) - b0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int d = 0; d < C::ND; ++d) {
      mbar_init(&bars->dfull[d], 1);
      mbar_init(&bars->dempty[d], C::PW);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // sums of this thread's lane (output n0 + 32 quarter + lane) for its CW columns, as pairs
  uint64_t acc[C::CW / 2];
#pragma unroll
  for (int c = 0; c < C::CW / 2; ++c) acc[c] = 0ull;
  const int quarter = warp & 3;
  const int col0 = C::PW == 8 ? ((warp - 2) / 4) * C::CW : 0;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      // The weights' first stages come to L2 while the preceding kernel finishes (a prefetch
      // reads nothing that could be stale); every read follows the wait.
      for (int i = 0; i < min(nb, C::NST); ++i) tma_prefetch_l2_2d(&tm_w, (b0 + i) * 128, n0);
      griddep_wait();
      int issued = 0;
      for (int i = 0; i < nb; ++i) {
        const int s = i % C::NST;
        if (i >= C::NST && !mbar_wait(&bars->empty[s], ((i / C::NST) - 1) & 1)) {
          record_error(p.err, ERR_TIMEOUT, 60);
          break;
        }
        uint8_t* st = smem + s * C::STAGE;
        mbar_arrive_expect_tx(&bars->full[s], C::STAGE);
        tma_load_2d(st, &tm_w, (b0 + i) * 128, n0, &bars->full[s]);
        tma_load_2d(st + A_BYTES, &tm_x, (b0 + i) * 128, t0, &bars->full[s]);
        issued = i + 1;
      }
      // no load of this CTA may still be in flight when the ring is reused or the CTA exits
      for (int i = max(0, issued - C::NST); i < issued; ++i)
        if (!mbar_wait(&bars->full[i % C::NST], (i / C::NST) & 1)) break;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = idesc_e4m3(128, BN);
      for (int i = 0; i < nb; ++i) {
        const int s = i % C::NST, d = i % C::ND;
        if ((i >= C::ND && !mbar_wait(&bars->dempty[d], ((i / C::ND) - 1) & 1)) ||
            !mbar_wait(&bars->full[s], (i / C::NST) & 1)) {
          record_error(p.err, ERR_TIMEOUT, 61);
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_addr(smem + s * C::STAGE), b = a + A_BYTES;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8(tmem + d * BN, umma_desc(a + kk * 32, 16, 1024, UMMA_SW128), umma_desc(b + kk * 32, 16, 1024, UMMA_SW128),
                 idesc, kk > 0 ? 1u : 0u);
        mma_commit(&bars->empty[s]);
        mma_commit(&bars->dfull[d]);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- promoting warps
    griddep_wait();
    if (threadIdx.x == 64) griddep_launch_dependents();
    float* xw = reinterpret_cast<float*>(smem + C::XS_OFF) + (warp - 2) * 2 * C::XC * C::CW;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    // chunk ch of the tokens' scales, XC scale blocks of this warp's CW tokens, zeros past the ends
    auto fetch = [&](int ch) {
      for (int e = lane; e < C::XC * C::CW; e += 32) {
        const int r = e / C::XC, kb = ch * C::XC + e % C::XC, t = t0 + col0 + r;
        const bool in = t < p.T && kb < nb;
        cp_async_4(smem_addr(xw + ((ch & 1) * C::XC + e % C::XC) * C::CW + r),
                   p.xs + (in ? (long)t * p.blocks + b0 + kb : 0), in);
      }
      cp_async_commit();
    };
    const float* wsp = p.ws + (long)blockIdx.y * p.blocks + b0;
    if (nb > 0) fetch(0);
    float wnext = nb > 0 ? wsp[0] : 0.f;
    for (int i = 0; i < nb; ++i) {
      if (i % C::XC == 0) {
        __syncwarp();  // every lane has read the chunk before the last
        fetch(i / C::XC + 1);
        cp_async_wait<1>();
        __syncwarp();
      }
      const float w = wnext;
      if (i + 1 < nb) wnext = wsp[i + 1];
      const uint64_t w2 = pack2(w, w);
      const int d = i % C::ND;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->dfull[d], (i / C::ND) & 1))) {
        if (lane == 0) record_error(p.err, ERR_TIMEOUT, 62);
        break;
      }
      tc_fence_after();
      const ulonglong2* xr = reinterpret_cast<const ulonglong2*>(xw + (((i / C::XC) & 1) * C::XC + i % C::XC) * C::CW);
      constexpr int CN = BN == 16 ? 16 : 32;
#pragma unroll
      for (int c0 = 0; c0 < C::CW; c0 += CN) {
        uint32_t v[CN];
        tmem_ld<CN>(tmem + lane_off + d * BN + col0 + c0, v);
        tmem_wait<CN>(v);
        if (c0 + CN == C::CW) {  // all of it read: the accumulator may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->dempty[d]);
        }
#pragma unroll
        for (int c = 0; c < CN; c += 4) {
          const ulonglong2 x = xr[(c0 + c) / 4];
          uint64_t& a0 = acc[(c0 + c) / 2];
          uint64_t& a1 = acc[(c0 + c) / 2 + 1];
          a0 = fma2(pack2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), mul2(x.x, w2), a0);
          a1 = fma2(pack2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), mul2(x.y, w2), a1);
        }
      }
    }
    cp_async_wait<0>();
  }

  const int m = quarter * 32 + lane;
  if (S == 1) {
    if (warp >= 2 && n0 + m < p.N) {
#pragma unroll
      for (int c = 0; c < C::CW; c += 2) {
        float v0, v1;
        unpack2(acc[c / 2], v0, v1);
        const long t = t0 + col0 + c;
        if (t < p.T) store_out(p, t, n0 + m, v0);
        if (t + 1 < p.T) store_out(p, t + 1, n0 + m, v1);
      }
    }
  } else {
    // Row m of the tile belongs to CTA r = ((m + 1) S - 1) / 128, which owns rows
    // [128 r / S, 128 (r + 1) / S).  Receive buffer: [S][rows of the largest share][RLD].
    float* recv = reinterpret_cast<float*>(smem);
    const int share = (128 + S - 1) / S;
    __syncwarp();
    cluster_arrive();
    cluster_wait();  // every CTA of the cluster has finished with its ring
    if (warp >= 2) {
      const int r = ((m + 1) * S - 1) / 128;
      const uint32_t dst = map_to_rank(recv, r) + (uint32_t)(((rank * share + m - r * 128 / S) * C::RLD + col0) * 4);
#pragma unroll
      for (int c = 0; c < C::CW; c += 4) {
        float v0, v1, v2, v3;
        unpack2(acc[c / 2], v0, v1);
        unpack2(acc[c / 2 + 1], v2, v3);
        st_cluster_v4(dst + c * 4, v0, v1, v2, v3);
      }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    const int lo = rank * 128 / S, rows = (rank + 1) * 128 / S - lo;
    for (int e = threadIdx.x; e < rows * BN; e += C::THREADS) {
      const int mr = e % rows, c = e / rows;
      float v = 0.f;
      for (int s = 0; s < S; ++s) v += recv[(s * share + mr) * C::RLD + c];
      const int n = n0 + lo + mr;
      const long t = t0 + c;
      if (n < p.N && t < p.T) store_out(p, t, n, v);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
}

// ------------------------------------------------------------------ many tokens
// Bound by the tensor pipe.  A pair of CTAs (cta_group::2) computes 256 tokens x 256 outputs: each CTA
// loads 128 token rows and 128 weight rows of a scale block (32 KB a stage, half of what a
// 128 x 256 tile of its own would load), the pair's MMA (M = 256, N = 256, K = 32, four per block)
// leaves 128 tokens x 256 outputs in each CTA's TMEM.  Here the tokens are the lanes, so a thread
// scales its columns by one number per block, xs[t, b] ws[n / 128, b]; eight promoting warps (four
// lane quarters x two column halves, each half one block row of ws) keep 128 fp32 sums a thread,
// while the next block's MMA fills the other half of TMEM.  Persistent over tiles; a finished tile
// goes out through 4 KB of shared memory a warp and TMA stores.
struct WdCfg {
  static constexpr int NST = 5;
  static constexpr int STAGE = 2 * 128 * 128;
  static constexpr int STG_OFF = NST * STAGE;          // 8 warps x 32 rows x 128 bytes
  static constexpr int XS_OFF = STG_OFF + 8 * 4096;    // 8 warps x [2][XC blocks][32 tokens] fp32
  static constexpr int XC = 8;                         // scale blocks fetched at a time
  static constexpr int BAR_OFF = XS_OFF + 8 * 2 * XC * 128;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  // warpgroup 0: TMA, MMA and two idle warps; warpgroups 1 and 2: the promoting warps, which hold 128
  // sums and two 32-column loads a thread.  Registers at launch 384 x 168 = 64512, after the split
  // 128 x 56 + 256 x 224 as many.
  static constexpr int THREADS = 384;
  static constexpr int REGS_FEW = 56, REGS_MANY = 224;
  static_assert(128 * REGS_FEW + 256 * REGS_MANY <= THREADS * 168, "register split");
  static constexpr int GROUP = 8;                      // token tiles walked together (x stays in L2)
  static_assert(SMEM <= 232448, "shared memory of one CTA per SM");
};

struct WdBars {
  uint64_t full[WdCfg::NST], empty[WdCfg::NST], dfull[2], dempty[2];
  uint32_t tmem_base;
};

struct WdParams {
  const float* xs;
  const float* ws;
  int T, N, blocks, tiles_t, tiles_n;
  void* out;
  long out_ld;
  int out_f32, tma_out;
  int* err;
};

// Tile `i` in walking order: groups of GROUP token tiles, within a group the outputs outside and the
// tokens inside, so the tiles under way at one time share both operands in L2.
__device__ __forceinline__ void wd_tile(const WdParams& p, int i, int& t0, int& n0) {
  const int per_group = WdCfg::GROUP * p.tiles_n;
  const int g = i / per_group, r = i % per_group;
  const int in_group = min(WdCfg::GROUP, p.tiles_t - g * WdCfg::GROUP);
  t0 = (g * WdCfg::GROUP + r % in_group) * 256;
  n0 = (r / in_group) * 256;
}

__global__ void __launch_bounds__(WdCfg::THREADS, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ CUtensorMap tm_out, const WdParams p) {
  using C = WdCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  WdBars* bars = reinterpret_cast<WdBars*>(smem + C::BAR_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_ctarank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int tiles = p.tiles_t * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(&bars->dfull[d], 1);
      mbar_init(&bars->dempty[d], 16);  // the promoting warps of both CTAs
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are ready before either signals the other's
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < 4) {
    setmaxnreg_dec<C::REGS_FEW>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ TMA producer (both CTAs)
      griddep_wait();
      int s = 0;             // stage, and the parity of its use
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        int t0, n0;
        wd_tile(p, tile, t0, n0);
        for (int b = 0; b < p.blocks; ++b) {
          if (!mbar_wait(&bars->empty[s], ph ^ 1)) {  // (true at once on a barrier's first use)
            record_error(p.err, ERR_TIMEOUT, 64);
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::STAGE;
          if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * C::STAGE);  // both CTAs' halves
          const uint32_t bar = map_to_rank(&bars->full[s], 0);
          tma_load_2d_pair(st, &tm_x, b * 128, t0 + rank * 128, bar);
          tma_load_2d_pair(st + A_BYTES, &tm_w, b * 128, n0 + rank * 128, bar);
          if (++s == C::NST) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // The loads of both CTAs land before either CTA may exit (the other one waits for this CTA below):
      // the stages' last uses, oldest first (true at once for a stage never used).
      if (rank == 0)
        for (int k = 0; k < C::NST; ++k) {
          if (!mbar_wait(&bars->full[s], ph ^ 1)) break;
          if (++s == C::NST) {
            s = 0;
            ph ^= 1;
          }
        }
    }
    if (warp == 1 && lane == 0 && rank == 0) {
      // ------------------------------------------------------------ MMA issuer (even CTA)
      constexpr uint32_t idesc = idesc_e4m3(256, 256);
      uint32_t it = 0, ph = 0;
      int s = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        for (int b = 0; b < p.blocks; ++b, ++it) {
          const uint32_t d = it & 1;
          if (!mbar_wait(&bars->dempty[d], ((it >> 1) & 1) ^ 1) || !mbar_wait(&bars->full[s], ph)) {
            record_error(p.err, ERR_TIMEOUT, 65);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_addr(smem + s * C::STAGE), w = a + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8_pair(tmem + d * 256, umma_desc(a + kk * 32, 16, 1024, UMMA_SW128),
                        umma_desc(w + kk * 32, 16, 1024, UMMA_SW128), idesc, kk > 0 ? 1u : 0u);
          mma_commit_pair(&bars->empty[s]);
          mma_commit_pair(&bars->dfull[d]);
          if (++s == C::NST) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- promoting warps
    setmaxnreg_inc<C::REGS_MANY>();
    griddep_wait();
    if (threadIdx.x == 128) griddep_launch_dependents();
    const int quarter = warp & 3, half = (warp - 4) / 4;
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
    uint8_t* stg = smem + C::STG_OFF + (warp - 4) * 4096;
    float* xw = reinterpret_cast<float*>(smem + C::XS_OFF) + (warp - 4) * 2 * C::XC * 32;
    const int chunks = (p.blocks + C::XC - 1) / C::XC;
    // The scales of chunk `ch` (XC blocks) of tile `tile`: this lane's token's to shared memory, buffer
    // `buf`, and block ch XC + lane % XC of the outputs' block row in the return value.  Tokens and
    // outputs past the ends take the last one's: what they give is not stored.
    auto fetch = [&](int tile, int ch, int buf) -> float {
      float w = 0.f;
      if (tile < tiles) {
        int t0, n0;
        wd_tile(p, tile, t0, n0);
        const long t = min(t0 + rank * 128 + quarter * 32 + lane, p.T - 1);
        const float* xs = p.xs + t * p.blocks + ch * C::XC;
#pragma unroll
        for (int k = 0; k < C::XC; ++k)
          if (ch * C::XC + k < p.blocks) cp_async_4(smem_addr(xw + (buf * C::XC + k) * 32 + lane), xs + k, true);
        const int wb = min(ch * C::XC + lane % C::XC, p.blocks - 1);
        w = p.ws[(long)(min(n0 + half * 128, p.N - 1) / 128) * p.blocks + wb];
      }
      cp_async_commit();
      return w;
    };
    uint32_t it = 0;
    bool ok = true;
    int buf = 0;
    float wnext = fetch(pair, 0, 0), wcur = 0.f;
    for (int tile = pair; ok && tile < tiles; tile += pairs) {
      int t0, n0;
      wd_tile(p, tile, t0, n0);
      const int row0 = t0 + rank * 128 + quarter * 32;  // this warp's first token
      const int col0 = n0 + half * 128;
      uint64_t acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0ull;
      for (int b = 0; b < p.blocks; ++b, ++it) {
        if (b % C::XC == 0) {
          // the next chunk (of this tile or the next) is on its way while this one is used
          const int ch = b / C::XC + 1;
          wcur = wnext;
          __syncwarp();
          wnext = ch < chunks ? fetch(tile, ch, buf ^ 1) : fetch(tile + pairs, 0, buf ^ 1);
          cp_async_wait<1>();
          buf ^= 1;  // (a lane reads only what it fetched itself)
        }
        const float sc = xw[((buf ^ 1) * C::XC + b % C::XC) * 32 + lane] * __shfl_sync(0xffffffffu, wcur, b % C::XC);
        const uint64_t s2 = pack2(sc, sc);
        const uint32_t d = it & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->dfull[d], (it >> 1) & 1))) {
          if (lane == 0) record_error(p.err, ERR_TIMEOUT, 66);
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[2][32];
        tmem_ld32(taddr + d * 256, v[0]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_wait_ld32(v[q & 1]);
          if (q < 3) {
            tmem_ld32(taddr + d * 256 + (q + 1) * 32, v[(q + 1) & 1]);
          } else {
            // all of it is in registers: the accumulator may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(&bars->dempty[d], 0);
          }
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            uint64_t& a = acc[q * 16 + c / 2];
            a = fma2(pack2(__uint_as_float(v[q & 1][c]), __uint_as_float(v[q & 1][c + 1])), s2, a);
          }
        }
      }
      if (!ok) break;
      // ---- the tile: 32 tokens x 128 outputs of this warp, 128 bytes of each row at a time
      const int per = p.out_f32 ? 32 : 64;  // outputs in 128 bytes
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        if (p.out_f32 || c0 % 64 == 0) {  // the staging rows are free again
          if (p.tma_out) {
            if (lane == 0) bulk_wait_group_read<0>();
          }
          __syncwarp();
        }
        const int chunk0 = p.out_f32 ? 0 : (c0 % 64) / 8;
        if (p.out_f32) {
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            ulonglong2 v = make_ulonglong2(acc[(c0 + c) / 2], acc[(c0 + c) / 2 + 1]);
            *reinterpret_cast<ulonglong2*>(stg + lane * 128 + (((c / 4) ^ (lane & 7)) << 4)) = v;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float lo, hi;
              unpack2(acc[(c0 + c) / 2 + j], lo, hi);
              const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
              w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(stg + lane * 128 + (((chunk0 + c / 8) ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (p.out_f32 || c0 % 64 == 32) {  // 128 bytes of every row are there
          const int cs = col0 + c0 + 32 - per;
          if (p.tma_out) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row0 < p.T && cs < p.N) {
              tma_store_2d(&tm_out, stg, cs, row0);  // rows past T and columns past N are not written
              bulk_commit_group();
            }
          } else {
            __syncwarp();
            const int elt = p.out_f32 ? 4 : 2;
            for (int r = 0; r < 32 && row0 + r < p.T; ++r)
              for (int c = lane; c < per; c += 32) {
                if (cs + c >= p.N) continue;
                const uint8_t* src = stg + r * 128 + ((((c * elt) >> 4) ^ (r & 7)) << 4) + ((c * elt) & 15);
                const long at = (long)(row0 + r) * p.out_ld + cs + c;
                if (p.out_f32)
                  static_cast<float*>(p.out)[at] = *reinterpret_cast<const float*>(src);
                else
                  static_cast<__nv_bfloat16*>(p.out)[at] = *reinterpret_cast<const __nv_bfloat16*>(src);
              }
          }
        }
      }
    }
    cp_async_wait<0>();
    if (p.tma_out && lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no MMA, load or signal of the pair is under way any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace p8

// ------------------------------------------------------------------ host side
static PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// 2-D map over bytes: boxes of 128 bytes x box_rows rows, 128-byte swizzle, zeros outside.
static bool map_bytes(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
static cudaError_t launch_skinny(const Fp8Args& a, cudaStream_t st) {
  using C = p8::SkCfg<BN>;
  CUtensorMap mw, mx;
  if (!map_bytes(&mw, a.w, a.K, a.N, a.K, 128) || !map_bytes(&mx, a.x, a.K, a.T, a.x_ld, BN)) return kUnsupported;
  const int blocks = (a.K + 127) / 128, tiles_n = (a.N + 127) / 128;
  const long tiles_t = (a.T + BN - 1) / BN;
  if (tiles_t > 65535 || tiles_n > 65535) return kUnsupported;
  int S = 1;
  while (S < 8 && tiles_n * tiles_t * (S + 1) <= 148 * C::OCC && (S + 1) * 2 <= blocks) ++S;
  p8::SkParams p;
  p.xs = a.xs;
  p.ws = a.ws;
  p.T = a.T;
  p.N = a.N;
  p.blocks = blocks;
  p.per_cta = (blocks + S - 1) / S;
  p.out = a.out;
  p.out_ld = a.out_ld;
  p.out_f32 = a.act == MLA_F32;
  p.err = a.err;
  cudaError_t e = cudaFuncSetAttribute(p8::fp8_skinny_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S, (unsigned)tiles_n, (unsigned)tiles_t);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, p8::fp8_skinny_kernel<BN>, mw, mx, p);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

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

// Output tiles go out by TMA stores (boxes of 128 bytes x 32 rows) where its alignment rules allow.
static bool map_out(CUtensorMap* m, const Fp8Args& a) {
  auto enc = tmap_encoder();
  const int elt = a.act == MLA_F32 ? 4 : 2;
  if (!enc || (reinterpret_cast<uintptr_t>(a.out) & 15) || (a.out_ld * elt) % 16) return false;
  cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.T};
  cuuint64_t strides[1] = {(cuuint64_t)(a.out_ld * elt)};
  cuuint32_t box[2] = {(cuuint32_t)(128 / elt), 32};
  cuuint32_t es[2] = {1, 1};
  return enc(m, a.act == MLA_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.out, dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static cudaError_t launch_wide(const Fp8Args& a, cudaStream_t st) {
  using C = p8::WdCfg;
  CUtensorMap mw, mx, mo;
  if (!map_bytes(&mw, a.w, a.K, a.N, a.K, 128) || !map_bytes(&mx, a.x, a.K, a.T, a.x_ld, 128)) return kUnsupported;
  p8::WdParams p;
  p.tma_out = map_out(&mo, a);
  if (!p.tma_out) mo = mx;
  p.xs = a.xs;
  p.ws = a.ws;
  p.T = a.T;
  p.N = a.N;
  p.blocks = (a.K + 127) / 128;
  p.tiles_t = (a.T + 255) / 256;
  p.tiles_n = (a.N + 255) / 256;
  p.out = a.out;
  p.out_ld = a.out_ld;
  p.out_f32 = a.act == MLA_F32;
  p.err = a.err;
  const long tiles = (long)p.tiles_t * p.tiles_n;
  if (tiles > (1 << 30)) return kUnsupported;
  cudaError_t e = cudaFuncSetAttribute(p8::fp8_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (tiles < 74 ? tiles : 74)));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, p8::fp8_wide_kernel, mw, mx, mo, p);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// TMA's rules: rows of x and w start on 16-byte boundaries.
static bool tma_layout(const Fp8Args& a) {
  return ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w)) & 15) == 0 && a.K % 16 == 0 &&
         a.x_ld % 16 == 0;
}

cudaError_t launch_project_fp8(const Fp8Args& a, cudaStream_t st) {
  if (!tma_layout(a)) return launch_fp8_any(a, st);
  if (a.T <= 16) return launch_skinny<16>(a, st);
  if (a.T <= 32) return launch_skinny<32>(a, st);
  if (a.T <= 64) return launch_skinny<64>(a, st);
  if (a.T <= 128) return launch_skinny<128>(a, st);
  return launch_wide(a, st);
}

}  // namespace mla
