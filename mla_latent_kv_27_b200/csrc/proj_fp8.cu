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
// Bound by the tensor pipe.  A pair of CTAs (cta_group::2) computes 256 tokens x WN outputs: each CTA
// loads 128 token rows and WN / 2 weight rows of a scale block, and the pair's MMA (M = 256, N = WN,
// K = 32, four per block) leaves 128 tokens x WN outputs in each CTA's TMEM.  Here the tokens are the
// lanes, so a thread scales its columns by one or two numbers per block, xs[t, b] ws[n / 128, b].  Eight
// promoting warps (four lane quarters x two column halves) keep WN / 2 fp32 sums a thread while
// the next block's MMA fills the other accumulator.  Two more warps compute the scales some blocks
// ahead.  Persistent over tiles; a finished tile goes out through 4 KB of shared memory a warp and
// TMA stores.
template <int WN>
struct WdCfg {
  static constexpr int HC = WN / 2;                    // columns of a promoting warp
  static constexpr int NF = HC / 32, TAIL = HC % 32;   // loaded as 32s and a 16
  static constexpr int ND = 512 / WN;                  // accumulators
  static constexpr int NST = 6;
  static constexpr int STAGE = (128 + WN / 2) * 128;
  static constexpr int STG_OFF = NST * STAGE;          // 8 warps x 32 rows x 128 bytes
  static constexpr int SC_OFF = STG_OFF + 8 * 4096;    // scales: [2][XC blocks][2 rows of ws][SLD], 128 tokens
  static constexpr int XC = 8;                         // scale blocks made at a time
  static constexpr int SLD = 130;                      // (bank spread of the writes)
  static constexpr int BAR_OFF = SC_OFF + 2 * XC * 2 * SLD * 4;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  // warpgroup 0: TMA, MMA and two scale warps; warpgroups 1 and 2: the promoting warps, which hold WN / 2
  // sums and as many loaded values a thread.  Registers at launch 384 x 168 = 64512, after the split
  // 128 x 80 + 256 x 208 = 63488.
  static constexpr int THREADS = 384;
  static constexpr int REGS_FEW = 72, REGS_MANY = 216;
  static_assert((TAIL == 0 || TAIL == 16) && STAGE % 1024 == 0 && SMEM <= 232448, "shared memory of one CTA per SM");
  static_assert(128 * REGS_FEW + 256 * REGS_MANY <= THREADS * 168, "register split");
};

template <int WN>
struct WdBars {
  uint64_t full[WdCfg<WN>::NST], empty[WdCfg<WN>::NST], dfull[WdCfg<WN>::ND], dempty[WdCfg<WN>::ND];
  uint64_t sfull[2], sempty[2];
  uint32_t tmem_base;
};

struct WdParams {
  const float* xs;
  const float* ws;
  int T, N, blocks, tiles_t, tiles_n;
  void* out;
  long out_ld;
  int* err;
};

// Tile `i` in walking order: groups of WD_GROUP token tiles, within a group the outputs outside and the
// tokens inside, so the tiles under way at one time share both operands in L2.
constexpr int WD_GROUP = 8;  // token tiles walked together
template <int WN>
__device__ __forceinline__ void wd_tile(const WdParams& p, int i, int& t0, int& n0) {
  const int per_group = WD_GROUP * p.tiles_n;
  const int g = i / per_group, r = i % per_group;
  const int in_group = min(WD_GROUP, p.tiles_t - g * WD_GROUP);
  t0 = (g * WD_GROUP + r % in_group) * 256;
  n0 = (r / in_group) * WN;
}

template <typename T, bool TMA_OUT, int WN>
__global__ void __launch_bounds__(WdCfg<WN>::THREADS, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ CUtensorMap tm_out, const WdParams p) {
  using C = WdCfg<WN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  WdBars<WN>* bars = reinterpret_cast<WdBars<WN>*>(smem + C::BAR_OFF);
  float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_ctarank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int tiles = p.tiles_t * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int d = 0; d < C::ND; ++d) {
      mbar_init(&bars->dfull[d], 1);
      mbar_init(&bars->dempty[d], 16);  // the promoting warps of both CTAs
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(&bars->sfull[d], 2);
      mbar_init(&bars->sempty[d], 8);
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

  // (a wait for the phase before a barrier's first one returns at once)
  if (warp < 4) {
    setmaxnreg_dec<C::REGS_FEW>();
    // The TMA and the MMA warp run their loops with all lanes and issue from an elected one: issued from
    // a one-lane branch, the four MMAs of a block and their waits took 1000 clocks of the thread's
    // time, twice what the tensor pipe needs for them.
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer (both CTAs)
      griddep_wait();
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        int t0, n0;
        wd_tile<WN>(p, tile, t0, n0);
        for (int b = 0; b < p.blocks; ++b) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->empty[s], ph ^ 1));
          if (!ok) {
            if (lane == 0) record_error(p.err, ERR_TIMEOUT, 64);
            break;
          }
          uint8_t* st = smem + s * C::STAGE;
          const uint32_t bar = map_to_rank(&bars->full[s], 0);
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * C::STAGE);  // both CTAs' halves
            tma_load_2d_pair(st, &tm_x, b * 128, t0 + rank * 128, bar);
            tma_load_2d_pair(st + A_BYTES, &tm_w, b * 128, n0 + rank * (WN / 2), bar);
          }
          __syncwarp();
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
          if (!__all_sync(0xffffffffu, mbar_wait(&bars->full[s], ph ^ 1))) break;
          if (++s == C::NST) {
            s = 0;
            ph ^= 1;
          }
        }
    }
    if (warp == 1 && rank == 0) {
      // ------------------------------------------------------------ MMA issuer (even CTA)
      constexpr uint32_t idesc = idesc_e4m3(256, WN);
      const uint64_t a0 = umma_desc(smem_addr(smem), 16, 1024, UMMA_SW128);
      const uint64_t w0 = umma_desc(smem_addr(smem) + A_BYTES, 16, 1024, UMMA_SW128);
      uint32_t ph = 0, dph = 0;  // parities of the current uses of stage s and accumulator d
      int s = 0, d = 0;
      bool ok = true, loaded = false, freed = false;  // asked while the block before is issued
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        for (int b = 0; b < p.blocks; ++b) {
          ok = (loaded || mbar_wait(&bars->full[s], ph)) && (freed || mbar_wait(&bars->dempty[d], dph ^ 1));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            if (lane == 0) record_error(p.err, ERR_TIMEOUT, 65);
            break;
          }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t step = (uint64_t)((s * C::STAGE + kk * 32) >> 4);  // (address fields are in 16 bytes)
              mma_f8_pair(tmem + d * WN, a0 + step, w0 + step, idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit_pair(&bars->dfull[d]);
            mma_commit_pair(&bars->empty[s]);
          }
          __syncwarp();
          if (++s == C::NST) {
            s = 0;
            ph ^= 1;
          }
          if (++d == C::ND) {
            d = 0;
            dph ^= 1;
          }
          loaded = mbar_test(&bars->full[s], ph);
          freed = mbar_test(&bars->dempty[d], dph ^ 1);
        }
      }
    }
    if (warp >= 2) {
      // ------------------------------------------------------------ scales, XC blocks at a time
      // xs[t, b] ws[r, b] for the two block rows r that a tile's outputs can meet.  Eight lanes read the 32 bytes of a
      // token's chunk.  Tokens and outputs past the ends take the last one's: what they give is not
      // stored.
      griddep_wait();
      const int k = lane % C::XC, r0 = (warp - 2) * 64 + lane / C::XC;
      uint32_t cnt = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        int t0, n0;
        wd_tile<WN>(p, tile, t0, n0);
        const float* ws0 = p.ws + (long)(n0 / 128) * p.blocks;
        const float* ws1 = p.ws + (long)min(n0 / 128 + 1, (p.N - 1) / 128) * p.blocks;
        for (int b0 = 0; b0 < p.blocks; b0 += C::XC, ++cnt) {
          const uint32_t slot = cnt & 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&bars->sempty[slot], ((cnt >> 1) & 1) ^ 1))) {
            if (lane == 0) record_error(p.err, ERR_TIMEOUT, 67);
            ok = false;
            break;
          }
          const int b = min(b0 + k, p.blocks - 1);
          const float w0 = ws0[b], w1 = ws1[b];
          float* dst = scales + (slot * C::XC + k) * 2 * C::SLD;
#pragma unroll
          for (int j = 0; j < 64; j += 32) {
            float x[C::XC];
#pragma unroll
            for (int i = 0; i < C::XC; ++i)
              x[i] = p.xs[(long)min(t0 + rank * 128 + r0 + j + i * (32 / C::XC), p.T - 1) * p.blocks + b];
#pragma unroll
            for (int i = 0; i < C::XC; ++i) {
              dst[r0 + j + i * (32 / C::XC)] = x[i] * w0;
              dst[C::SLD + r0 + j + i * (32 / C::XC)] = x[i] * w1;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->sfull[slot]);
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
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::HC;
    uint8_t* stg = smem + C::STG_OFF + (warp - 4) * 4096;
    const float* my_scales = scales + quarter * 32 + lane;
    // all lanes' waits for a barrier
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, mbar_wait_count(bar, parity)); };
    uint32_t cnt = 0, dph = 0;  // chunks of scales used; parity of the current use of accumulator d
    int d = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < tiles; tile += pairs) {
      int t0, n0;
      wd_tile<WN>(p, tile, t0, n0);
      const int row0 = t0 + rank * 128 + quarter * 32;  // this warp's first token
      const int blk0 = n0 % 128 + half * C::HC;  // column c's row of ws is (blk0 + c) / 128 past n0 / 128
      float acc[C::HC];
#pragma unroll
      for (int c = 0; c < C::HC; ++c) acc[c] = 0.f;
      uint32_t v[C::NF][32], vt[16];
      auto load = [&](int j) {  // chunk j of accumulator d
        if (j < C::NF)
          tmem_ld32(taddr + d * WN + j * 32, v[j]);
        else
          tmem_ld16(taddr + d * WN + j * 32, vt);
      };
      auto ready = [&]() -> bool {  // accumulator d is there
        const bool r = wait(&bars->dfull[d], dph);
        tc_fence_after();
        return r;
      };
      constexpr int CH = C::NF + (C::TAIL ? 1 : 0);
      ok = ready();
#pragma unroll
      for (int j = 0; j < CH; ++j) load(j);
      for (int b0 = 0; ok && b0 < p.blocks; b0 += C::XC, ++cnt) {
        const uint32_t slot = cnt & 1;
        ok = wait(&bars->sfull[slot], (cnt >> 1) & 1);
        const float* sp = my_scales + slot * (C::XC * 2 * C::SLD);
        const int n = min(C::XC, p.blocks - b0);
#pragma unroll 1
        for (int k = 0; ok && k < n; ++k, sp += 2 * C::SLD) {
          const float s0 = sp[0], s1 = sp[C::SLD];
          const int freed = d;
          if (++d == C::ND) {
            d = 0;
            dph ^= 1;
          }
          const bool there = mbar_test(&bars->dfull[d], dph);  // (asked now, answered behind the first sums)
#pragma unroll
          for (int j = 0; j < C::NF; ++j) tmem_wait_ld32(v[j]);
          if (C::TAIL) tmem_wait_ld16(vt);
          // all of it is in registers: the accumulator may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(&bars->dempty[freed], 0);
          const bool more = b0 + k + 1 < p.blocks;
#pragma unroll
          for (int j = 0; j < CH; ++j) {
#pragma unroll
            for (int c = 0; c < 32 && j * 32 + c < C::HC; ++c) {
              const float s = blk0 + j * 32 + c / 16 * 16 < 128 ? s0 : s1;  // (rows of ws change at multiples of 16)
              acc[j * 32 + c] = fmaf(__uint_as_float(j < C::NF ? v[j < C::NF ? j : 0][c] : vt[c % 16]), s, acc[j * 32 + c]);
            }
            // the next block's chunk takes the registers at once
            if (more) {
              if (j == 0) {
                if (__all_sync(0xffffffffu, there))
                  tc_fence_after();
                else
                  ok = ready();
              }
              load(j);
            }
          }
        }
        if (lane == 0) mbar_arrive(&bars->sempty[slot]);
      }
      if (!ok && lane == 0) record_error(p.err, ERR_TIMEOUT, 66);
      if (!ok) break;
      // ---- the tile: 32 tokens x WN / 2 outputs of this warp, 16 outputs at a time
      constexpr int ROW = 16 * sizeof(T), NBUF = 4096 / (32 * ROW);  // bytes of a staged row; buffers
#pragma unroll
      for (int j = 0; j < C::HC / 16; ++j) {
        uint8_t* buf = stg + (j % NBUF) * 32 * ROW;
        if (TMA_OUT && lane == 0) bulk_wait_group_read<NBUF - 1>();  // the buffer's last store has read it
        __syncwarp();
#pragma unroll
        for (int q = 0; q < ROW / 16; ++q) {  // 16 bytes, at the place that the 64- or 32-byte swizzle gives them
          uint4 w;
          if constexpr (sizeof(T) == 4) {
            w = make_uint4(__float_as_uint(acc[j * 16 + 4 * q]), __float_as_uint(acc[j * 16 + 4 * q + 1]),
                           __float_as_uint(acc[j * 16 + 4 * q + 2]), __float_as_uint(acc[j * 16 + 4 * q + 3]));
          } else {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(acc[j * 16 + 8 * q + 2 * i], acc[j * 16 + 8 * q + 2 * i + 1]);
              h[i] = *reinterpret_cast<const uint32_t*>(&x);
            }
            w = make_uint4(h[0], h[1], h[2], h[3]);
          }
          *reinterpret_cast<uint4*>(buf + lane * ROW + ((q ^ (sizeof(T) == 4 ? (lane >> 1) & 3 : (lane >> 2) & 1)) << 4)) = w;
        }
        const int cs = n0 + half * C::HC + j * 16;
        if (TMA_OUT) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < p.T && cs < p.N) tma_store_2d(&tm_out, buf, cs, row0);  // clipped to T x N
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          for (int e = lane; e < 32 * 16; e += 32) {
            const int r = e / 16, c = e % 16, at = c * (int)sizeof(T);
            if (row0 + r < p.T && cs + c < p.N)
              static_cast<T*>(p.out)[(long)(row0 + r) * p.out_ld + cs + c] = *reinterpret_cast<const T*>(
                  buf + r * ROW + (((at >> 4) ^ (sizeof(T) == 4 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4) + (at & 15));
          }
        }
      }
    }
    tmem_wait_ld();
    if (TMA_OUT && lane == 0) bulk_wait_group<0>();
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

// Output tiles go out by TMA stores (boxes of 16 outputs x 32 rows) where its alignment rules allow.
static bool map_out(CUtensorMap* m, const Fp8Args& a) {
  auto enc = tmap_encoder();
  const int elt = a.act == MLA_F32 ? 4 : 2;
  if (!enc || (reinterpret_cast<uintptr_t>(a.out) & 15) || (a.out_ld * elt) % 16) return false;
  cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.T};
  cuuint64_t strides[1] = {(cuuint64_t)(a.out_ld * elt)};
  cuuint32_t box[2] = {16, 32};
  cuuint32_t es[2] = {1, 1};
  return enc(m, a.act == MLA_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.out, dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, elt == 4 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int WN>
static cudaError_t launch_wide(const Fp8Args& a, cudaStream_t st) {
  using C = p8::WdCfg<WN>;
  CUtensorMap mw, mx, mo;
  if (!map_bytes(&mw, a.w, a.K, a.N, a.K, WN / 2) || !map_bytes(&mx, a.x, a.K, a.T, a.x_ld, 128)) return kUnsupported;
  p8::WdParams p;
  const bool tma_out = map_out(&mo, a);
  if (!tma_out) mo = mx;
  auto kernel = a.act == MLA_F32 ? (tma_out ? p8::fp8_wide_kernel<float, true, WN> : p8::fp8_wide_kernel<float, false, WN>)
                                 : (tma_out ? p8::fp8_wide_kernel<__nv_bfloat16, true, WN>
                                            : p8::fp8_wide_kernel<__nv_bfloat16, false, WN>);
  p.xs = a.xs;
  p.ws = a.ws;
  p.T = a.T;
  p.N = a.N;
  p.blocks = (a.K + 127) / 128;
  p.tiles_t = (a.T + 255) / 256;
  p.tiles_n = (a.N + WN - 1) / WN;
  p.out = a.out;
  p.out_ld = a.out_ld;
  p.err = a.err;
  const long tiles = (long)p.tiles_t * p.tiles_n;
  if (tiles > (1 << 30)) return kUnsupported;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
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
  e = cudaLaunchKernelEx(&cfg, kernel, mw, mx, mo, p);
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
  return launch_wide<160>(a, st);
}

}  // namespace mla
