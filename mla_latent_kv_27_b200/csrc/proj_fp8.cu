// 8-bit projection with block scales:
//
//   out[t, n] = sum_b xs[t, b] ws[n / 128, b] sum_{k in block b} x[t, k] w[n, k],
//
// x and w E4M3, one fp32 scale per 128 values of a row of x and per 128 x 128 block of w.  The
// products of one block are summed without scales (exact products, fp32 sums), then the block's
// sum is scaled and added to an fp32 accumulator.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "mla_internal.cuh"
#include "proj_fp8.cuh"
#include "sm100_f8.cuh"
#include "store_ring.h"

namespace mla {
namespace p8 {

using namespace sm100;

// ------------------------------------------------------------------ any layout
// fp32 FMA on the CUDA cores: 64 tokens x 64 outputs per CTA, 4 x 4 per thread, 16 values of K at
// a time.  Every width, alignment and leading dimension; the path of what the tensor-core
// kernels do not take (about 22 TFLOP/s; the FMAs, their shared-memory reads and the decoding of the codes
// bound it).
template <typename T>
__global__ void __launch_bounds__(256) fp8_any_kernel(const Fp8Args a) {
  __shared__ float xs_s[16][64 + 4];
  __shared__ float ws_s[16][64 + 4];
  griddep_wait();
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const unsigned tiles_n = (unsigned)(a.N + 63) / 64;
  const long t0 = (long)(blockIdx.x / tiles_n) * 64;
  const int n0 = (int)(blockIdx.x % tiles_n) * 64;
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
  // (not before: the loop takes as long as the width says, and a grid that starts under it would count its bounded
  // waits from its own start)
  griddep_launch_dependents();
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
// block's products go to a TMEM accumulator of their own (ND of them in turn).  One signal a block, the
// commit of its MMAs, tells the loads that the stage is free and the sums that the products are there; with
// a signal for each, and waits that were not asked ahead, the issuing warp bound the kernel (680 clocks a
// block; 64 x 7168 x 16384 28.0 us against 25.8).  The promoting warps
// (four lane quarters x column groups) read it, scale its columns by xs[t, b] ws[n / 128, b] (made by
// a warp of its own, XC blocks at a time) and add it to fp32 sums in registers.  At the end, unless unsplit, each
// CTA lays its sums out in its idle stage ring and sends every other CTA the rows that one owns, one bulk
// copy each into a buffer of the owner's shared memory; the owner adds the S partial sums of its rows
// in rank order and stores them: no workspace, no atomics.
//
// 64 x 7168 x 16384: 25.9 us in a burst, 28.5 in a loop of half a second; 4.5 TB/s of weights (their bytes at copy
// bandwidth: 18.2 us).  56 tiles split in two leave 36 SMs idle (a tile is always 128 outputs high), and the start, the
// exchange and the last sums take some 6 us; 64 x 18944 x 16384, which fills the SMs, reads 5.9 TB/s.
// 64 x 2112 x 7168: 7.7 us (8.4 over 400 MB of operands), 1 x 576 x 2048: 3.1 us, the chain of wait, load, MMA, exchange and
// store.  Tried: 8 promoting warps for 64 columns (42 us against 30 at the time), the exchange by
// asynchronous 16-byte stores from registers (64 x 2112 x 7168 0.4 us longer than by bulk copies), the next
// block's products loaded ahead of the sums (nothing: the issuing warp bound the blocks, not these).
constexpr int A_BYTES = 128 * 128;

template <int BN, int OCC>  // OCC: CTAs per SM
struct SkCfg {
  static constexpr int NST = BN == 128 ? 4 : OCC == 1 ? (BN == 64 ? 7 : 8) : BN == 16 ? 5 : 4;
  static constexpr int STAGE = A_BYTES + BN * 128;
  static constexpr int ND = 4;
  static constexpr uint32_t TCOLS = ND * BN;            // 64 to 512 columns
  static constexpr int PW = BN <= 32 || OCC == 2 ? 8 : 16;  // promoting warps: four lane quarters x column groups
  static constexpr int CW = BN / (PW / 4);              // columns of one of them
  static constexpr int XC = 8;                          // scale blocks made at a time
  static constexpr int SW = BN <= 32 ? 1 : 2;           // warps that make them
  static constexpr int SLD = BN + 4;
  static constexpr int THREADS = 128 + PW * 32;         // warps 0 TMA, 1 MMA, 2 and 3 scales, 4 and up promoting
  static constexpr int SC_OFF = NST * STAGE;            // scales: [2][XC][SLD] fp32
  static constexpr int RLD = BN + 4;                    // floats of a row of partial sums (bank spread)
  static constexpr int RECV_OFF = SC_OFF + 2 * XC * SLD * 4;      // [S][rows of the largest share][RLD]
  static constexpr bool SPLIT = BN != 64 || OCC == 1;   // 64 columns leave no room for RECV beside a second CTA: S = 1
  // (S ceil(128 / S) is at most 135 for S <= 8)
  static constexpr int BAR_OFF = RECV_OFF + (SPLIT ? (128 + 7) * RLD * 4 : 0);
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  static_assert(NST >= ND, "done[] is not signalled again before its block is summed");
  static_assert(128 * RLD * 4 <= NST * STAGE && RECV_OFF % 16 == 0 && BAR_OFF % 8 == 0, "layout");
  static_assert(OCC * (SMEM + 1024) <= 233472 && OCC * TCOLS <= 512, "CTAs per SM");
};

template <int BN, int OCC>
struct SkBars {
  uint64_t full[SkCfg<BN, OCC>::NST], done[SkCfg<BN, OCC>::NST], dempty[SkCfg<BN, OCC>::ND];
  uint64_t sfull[2], sempty[2], received;
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

__device__ __forceinline__ void store_out(const SkParams& p, long at, float v) {
  if (p.out_f32)
    static_cast<float*>(p.out)[at] = v;
  else
    static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}
// (relaxed: the barriers' initialisation is published by its own fence and data by mbarriers; a release would
// wait for every store of the thread, about 1 us here)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// CN (8, 16 or 32) consecutive fp32 columns of this thread's TMEM lane, and the wait for them
template <int CN>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[CN]) {
  if constexpr (CN == 32)
    tmem_ld32(addr, v);
  else if constexpr (CN == 16)
    tmem_ld16(addr, v);
  else
    tmem_ld8(addr, v);
}
template <int CN>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[CN]) {
  if constexpr (CN == 32)
    tmem_wait_ld32(v);
  else if constexpr (CN == 16)
    tmem_wait_ld16(v);
  else
    tmem_wait_ld8(v);
}
// a bounded wait of all lanes of a warp, the same answer in each
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

template <int BN, int OCC>
__global__ void __launch_bounds__(SkCfg<BN, OCC>::THREADS, OCC)
    fp8_skinny_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const SkParams p) {
  using C = SkCfg<BN, OCC>;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a cast of the rounded address: accesses stay shared-memory ones, not generic)
  uint8_t* smem = smem_raw + ((1024u - smem_addr(smem_raw)) & 1023u);
  SkBars<BN, OCC>* bars = reinterpret_cast<SkBars<BN, OCC>*>(smem + C::BAR_OFF);
  float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = C::SPLIT ? gridDim.x : 1, rank = C::SPLIT ? blockIdx.x : 0;
  const int n0 = blockIdx.y * 128;
  const int t0 = blockIdx.z * BN;
  const int b0 = rank * p.per_cta;
  const int nb = max(0, min(p.blocks, b0 + p.per_cta) - b0);
  // CTA r of the cluster owns rows [128 r / S, 128 (r + 1) / S) of the tile
  const int lo = rank * 128 / S, rows = (rank + 1) * 128 / S - lo, share = (128 + S - 1) / S;

  // The weights' first stages come to L2 while the preceding kernel finishes (a prefetch reads nothing
  // that could be stale); every read follows the wait.
  if (warp == 0 && lane < min(nb, C::NST)) tma_prefetch_l2_2d(&tm_w, (b0 + lane) * 128, n0);
  if (warp == 2) {  // a lane a barrier
    if (lane < C::NST) {
      mbar_init(&bars->full[lane], 1);
      mbar_init(&bars->done[lane], 1);
    }
    if (lane < C::ND) {
      mbar_init(&bars->dempty[lane], C::PW);
    }
    if (lane < 2) {
      mbar_init(&bars->sfull[lane], C::SW);
      mbar_init(&bars->sempty[lane], C::PW);
    }
    if (lane == 0) mbar_init(&bars->received, 1);
    fence_mbar_init();
    if (S > 1 && lane == 0) mbar_arrive_expect_tx(&bars->received, (uint32_t)(S * rows * C::RLD * 4));
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S > 1) cluster_arrive();  // peers may send to this CTA after this
  const uint32_t tmem = bars->tmem_base;
  griddep_wait();  // (every warp: none of the bounded waits below is for the grid in front)

  // sums of this thread's lane (output n0 + 32 quarter + lane) for its CW columns, as pairs
  uint64_t acc[C::CW / 2];
#pragma unroll
  for (int c = 0; c < C::CW / 2; ++c) acc[c] = 0ull;
  const int quarter = warp & 3;
  const int col0 = warp >= 4 ? (warp - 4) / 4 * C::CW : 0;

  // (a wait for the phase before a barrier's first one returns at once)
  if (warp == 0) {
    // -------------------------------------------------------------- TMA producer
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nb; ++i) {
      if (!warp_wait(&bars->done[s], ph ^ 1)) {
        if (lane == 0) record_error(p.err, ERR_TIMEOUT, 60);
        break;
      }
      if (elect_one()) {
        uint8_t* st = smem + s * C::STAGE;
        mbar_arrive_expect_tx(&bars->full[s], C::STAGE);
        tma_load_2d(st, &tm_w, (b0 + i) * 128, n0, &bars->full[s]);
        tma_load_2d(st + A_BYTES, &tm_x, (b0 + i) * 128, t0, &bars->full[s]);
      }
      __syncwarp();
      if (++s == C::NST) {
        s = 0;
        ph ^= 1;
      }
    }
    // no load of this CTA may still be in flight when the ring is reused or the CTA exits: the stages'
    // last uses, oldest first (true at once for a stage never used)
    for (int k = 0; k < C::NST; ++k) {
      if (!warp_wait(&bars->full[s], ph ^ 1)) break;
      if (++s == C::NST) {
        s = 0;
        ph ^= 1;
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer (all lanes, an elected one issues)
    constexpr uint32_t idesc = idesc_e4m3(128, BN);
    const uint64_t a0 = umma_desc(smem_addr(smem), 16, 1024, UMMA_SW128);
    const uint64_t x0 = umma_desc(smem_addr(smem) + A_BYTES, 16, 1024, UMMA_SW128);
    int s = 0;
    uint32_t ph = 0;
    bool loaded = false, freed = false;  // asked while the block before is issued
    for (int i = 0; i < nb; ++i) {
      const int d = i % C::ND;
      const bool ok = (loaded || mbar_wait(&bars->full[s], ph)) && (freed || mbar_wait(&bars->dempty[d], ((i / C::ND) & 1) ^ 1));
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) record_error(p.err, ERR_TIMEOUT, 61);
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint64_t at = (uint64_t)((s * C::STAGE) >> 4);  // (address fields are in 16 bytes)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8(tmem + d * BN, a0 + at + 2 * kk, x0 + at + 2 * kk, idesc, kk > 0 ? 1u : 0u);
        mma_commit(&bars->done[s]);
      }
      __syncwarp();
      if (++s == C::NST) {
        s = 0;
        ph ^= 1;
      }
      loaded = mbar_test(&bars->full[s], ph);
      freed = mbar_test(&bars->dempty[(i + 1) % C::ND], (((i + 1) / C::ND) & 1) ^ 1);
    }
  } else if (warp < 2 + C::SW) {
    // -------------------------------------------------------------- scales of the CTA's tokens
    // Eight lanes read the 32 bytes of a token's chunk.  Past the last token: zero.
    const float* ws = p.ws + (long)blockIdx.y * p.blocks;
    for (int c = 0; c * C::XC < nb; ++c) {
      if (!warp_wait(&bars->sempty[c & 1], ((c >> 1) & 1) ^ 1)) {
        if (lane == 0) record_error(p.err, ERR_TIMEOUT, 63);
        break;
      }
      const int k = lane % C::XC, b = min(b0 + c * C::XC + k, p.blocks - 1);
      const float w = ws[b];
      float* dst = scales + ((c & 1) * C::XC + k) * C::SLD;
#pragma unroll 1
      for (int r0 = (warp - 2) * 32; r0 < BN; r0 += C::SW * 32) {
        float x[C::XC];
#pragma unroll
        for (int j = 0; j < C::XC; ++j) {
          const int r = r0 + lane / C::XC + j * (32 / C::XC);
          x[j] = r < BN && t0 + r < p.T ? p.xs[(long)(t0 + r) * p.blocks + b] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < C::XC; ++j) {
          const int r = r0 + lane / C::XC + j * (32 / C::XC);
          if (r < BN) dst[r] = x[j] * w;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->sfull[c & 1]);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- promoting warps
    if (threadIdx.x == 128) griddep_launch_dependents();
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + col0;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nb; ++i) {
      const int c = i / C::XC, d = i % C::ND;
      if ((i % C::XC == 0 && !warp_wait(&bars->sfull[c & 1], (c >> 1) & 1)) ||
          !warp_wait(&bars->done[s], ph)) {
        if (lane == 0) record_error(p.err, ERR_TIMEOUT, 62);
        break;
      }
      tc_fence_after();
      const ulonglong2* xr =
          reinterpret_cast<const ulonglong2*>(scales + ((c & 1) * C::XC + i % C::XC) * C::SLD + col0);
      constexpr int CN = C::CW < 16 ? C::CW : 16;
#pragma unroll
      for (int c0 = 0; c0 < C::CW; c0 += CN) {
        uint32_t v[CN];
        tmem_ld<CN>(taddr + d * BN + c0, v);
        tmem_wait<CN>(v);
        if (c0 + CN == C::CW) {  // all of it read: the accumulator may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->dempty[d]);
        }
#pragma unroll
        for (int q = 0; q < CN; q += 4) {
          const ulonglong2 x = xr[(c0 + q) / 4];
          uint64_t& s0 = acc[(c0 + q) / 2];
          uint64_t& s1 = acc[(c0 + q) / 2 + 1];
          s0 = fma2(pack2(__uint_as_float(v[q]), __uint_as_float(v[q + 1])), x.x, s0);
          s1 = fma2(pack2(__uint_as_float(v[q + 2]), __uint_as_float(v[q + 3])), x.y, s1);
        }
      }
      if (++s == C::NST) {
        s = 0;
        ph ^= 1;
      }
      if (i % C::XC == C::XC - 1) {  // (the CTA's last chunk is not written again)
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->sempty[c & 1]);
      }
    }
  }

  __syncwarp();
  if (S == 1) {
    // ---- unsplit: a warp's lanes are 32 neighbouring outputs of a token, stored from its registers
    const int n = n0 + quarter * 32 + lane;
    const int left = warp >= 4 && n < p.N ? p.T - t0 - col0 : 0;  // tokens of this thread
    long at = (long)(t0 + col0) * p.out_ld + n;
#pragma unroll
    for (int c = 0; c < C::CW; c += 2) {
      float v[2];
      unpack2(acc[c / 2], v[0], v[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i, at += p.out_ld)
        if (c + i < left) store_out(p, at, v[i]);
    }
  } else {
    // ---- partial sums [128 rows][RLD] over this CTA's own ring, idle since its last MMA completed
    float* part = reinterpret_cast<float*>(smem);
    float* recv = reinterpret_cast<float*>(smem + C::RECV_OFF);
    cluster_wait();  // (every CTA of the cluster has begun)
    if (warp >= 4) {
      float* dst = part + (quarter * 32 + lane) * C::RLD + col0;
#pragma unroll
      for (int c = 0; c < C::CW; c += 4)
        *reinterpret_cast<ulonglong2*>(dst + c) = make_ulonglong2(acc[c / 2], acc[c / 2 + 1]);
      fence_proxy_async_smem();
      named_bar_sync(1, C::PW * 32);
      if (warp == 4 && lane < S) {
        const int first = lane * 128 / S, n = (lane + 1) * 128 / S - first;
        bulk_copy_s2cluster(map_to_rank(recv + rank * share * C::RLD, lane), smem_addr(part + first * C::RLD),
                            (uint32_t)(n * C::RLD * 4), map_to_rank(&bars->received, lane));
      }
    }
    const bool ok = warp_wait(&bars->received, 0);
    if (!ok && lane == 0) record_error(p.err, ERR_TIMEOUT, 68);
    cluster_arrive();  // this CTA has all that was sent to it
    // ---- sums of this CTA's rows: a thread takes four tokens of a row, neighbouring lanes neighbouring rows
    const int shift = rows <= 16 ? 4 : rows <= 32 ? 5 : 6;
#pragma unroll 1
    for (int e = threadIdx.x; ok && e < (BN / 4) << shift; e += C::THREADS) {
      const int m = e & ((1 << shift) - 1), c = (e >> shift) * 4;
      if (m >= rows || n0 + lo + m >= p.N || t0 + c >= p.T) continue;
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = r < S ? *reinterpret_cast<const float4*>(recv + (r * share + m) * C::RLD + c) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 1; r < 8; ++r) {  // (in rank order; those past S add zeros)
        v[0].x += v[r].x;
        v[0].y += v[r].y;
        v[0].z += v[r].z;
        v[0].w += v[r].w;
      }
      const float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + c + i < p.T) store_out(p, (long)(t0 + c + i) * p.out_ld + n0 + lo + m, sum[i]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
  __syncwarp();
  if (S > 1) cluster_wait();  // every CTA has received: no copy of this one's sums is under way
}

// ------------------------------------------------------------------ many tokens
// Bound by the fp32 sums between the MMAs: the tensor pipe is active 52 to 55 % of the time.  A pair of CTAs
// (cta_group::2) computes 256 tokens x WN outputs: each CTA
// loads 128 token rows and WN / 2 weight rows of a scale block, and the pair's MMA (M = 256, N = WN,
// K = 32, four per block) leaves 128 tokens x WN outputs in each CTA's TMEM.  Here the tokens are the
// lanes, so a thread scales its columns by one or two numbers per block, xs[t, b] ws[n / 128, b].  Eight
// promoting warps (four lane quarters x two column halves) keep WN / 2 fp32 sums a thread while
// the next blocks' MMAs fill the other accumulators.  Two more warps compute the scales some blocks
// ahead.  Persistent over tiles; a finished tile goes out through 4 KB of shared memory a warp and
// TMA stores.
//
// 2048 x 7168 x 16384: 232 us in a burst, 2.07 PFLOP/s (a long loop of them runs at the power cap, 278 us).  A block of
// 160 outputs takes a pair 0.307 us, of 128 0.26; the MMAs alone need 0.215 for 128 outputs and 0.29 for 256 (an MMA
// of N = 128 runs at two thirds of N = 256's rate).  What it waits for is the sums: 256 outputs leave TMEM room for two
// accumulators only, and the tensor pipe idles while one is read (0.56 us a block); 192 outputs 0.42.  That is some 580
// clocks a block of 160 outputs, of which the packed FMAs of a scheduler's two promoting warps take about 160: the rest is
// their chain of wait, TMEM load, wait and arrival.
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
  // 128 x 72 + 256 x 216 = 64512.
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
  // (an offset, not a cast of the rounded address: accesses stay shared-memory ones, not generic)
  uint8_t* smem = smem_raw + ((1024u - smem_addr(smem_raw)) & 1023u);
  WdBars<WN>* bars = reinterpret_cast<WdBars<WN>*>(smem + C::BAR_OFF);
  float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_ctarank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int tiles = p.tiles_t * p.tiles_n;

  if (warp == 2) {  // a lane a barrier
    if (lane < C::NST) {
      mbar_init(&bars->full[lane], 1);
      mbar_init(&bars->empty[lane], 1);
    }
    if (lane < C::ND) {
      mbar_init(&bars->dfull[lane], 1);
      mbar_init(&bars->dempty[lane], 16);  // the promoting warps of both CTAs
    }
    if (lane < 2) {
      mbar_init(&bars->sfull[lane], 2);
      mbar_init(&bars->sempty[lane], 8);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();  // both CTAs' barriers are ready before either signals the other's
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  griddep_wait();  // (every warp: none of the bounded waits below is for the grid in front)

  // (a wait for the phase before a barrier's first one returns at once)
  if (warp < 4) {
    setmaxnreg_dec<C::REGS_FEW>();
    // The TMA and the MMA warp run their loops with all lanes and issue from an elected one: issued from
    // a one-lane branch, the four MMAs of a block and their waits took 1000 clocks of the thread's
    // time, twice what the tensor pipe needs for them.
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer (both CTAs)
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
    if (threadIdx.x == 128) griddep_launch_dependents();
    const int quarter = warp & 3, half = (warp - 4) / 4;
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::HC;
    uint8_t* stg = smem + C::STG_OFF + (warp - 4) * 4096;
    const float* my_scales = scales + quarter * 32 + lane;
    // all lanes' waits for a barrier
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, mbar_wait_count(bar, parity)); };
    // staged rows of 16 outputs, and buffers of 32 of them
    constexpr int ROW = 16 * (int)sizeof(T), NBUF = 4096 / (32 * ROW);
    StoreRing<NBUF> ring;  // (over all tiles: 160 outputs are 5 stores a tile, no multiple of NBUF)
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
            for (int c = 0; c < 32 && j * 32 + c < C::HC; c += 2) {
              const float sc = blk0 + j * 32 + c / 16 * 16 < 128 ? s0 : s1;  // (rows of ws change at multiples of 16)
              const uint32_t* x = j < C::NF ? &v[j < C::NF ? j : 0][c] : &vt[c % 16];
              float* to = acc + j * 32 + c;
              unpack2(fma2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), pack2(sc, sc), pack2(to[0], to[1])), to[0], to[1]);
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
      // ---- the tile: 32 tokens x WN / 2 outputs of this warp
      auto sixteen_bytes = [&](int c) {  // from sum c on, rounded
        if constexpr (sizeof(T) == 4) {
          return make_uint4(__float_as_uint(acc[c]), __float_as_uint(acc[c + 1]), __float_as_uint(acc[c + 2]),
                            __float_as_uint(acc[c + 3]));
        } else {
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c + 2 * i], acc[c + 2 * i + 1]);
            h[i] = *reinterpret_cast<const uint32_t*>(&x);
          }
          return make_uint4(h[0], h[1], h[2], h[3]);
        }
      };
      constexpr int PER16 = 16 / (int)sizeof(T);
      if constexpr (TMA_OUT) {  // 16 outputs at a time
#pragma unroll
        for (int j = 0; j < C::HC / 16; ++j) {
          uint8_t* buf = stg + ring.take() * 32 * ROW;
          if (lane == 0) bulk_wait_group_read<NBUF - 1>();  // the buffer's last store has read it
          __syncwarp();
#pragma unroll
          for (int q = 0; q < ROW / 16; ++q)  // 16 bytes, at the place that the 64- or 32-byte swizzle gives them
            *reinterpret_cast<uint4*>(buf + lane * ROW + ((q ^ (sizeof(T) == 4 ? (lane >> 1) & 3 : (lane >> 2) & 1)) << 4)) =
                sixteen_bytes(j * 16 + PER16 * q);
          const int cs = n0 + half * C::HC + j * 16;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < p.T && cs < p.N) tma_store_2d(&tm_out, buf, cs, row0);  // clipped to T x N
            bulk_commit_group();
          }
        }
      } else {
        // 128 bytes of each row at a time (what is left of WN / 2 at the end), stored with the lanes along the
        // row: 4 bytes each where every row is 4-byte aligned, else a bf16 value each.  (Rows that straddle
        // sectors cost two writes at each end of a segment: 4011 x 14142 x 176 to floats 88 us,
        // 103 with segments of 16 outputs.)
        const bool words = sizeof(T) == 4 || ((reinterpret_cast<uintptr_t>(p.out) >> 1 | p.out_ld) & 1) == 0;
        auto segment = [&](auto count, int c0) {
          constexpr int N = decltype(count)::value, BYTES = N * (int)sizeof(T);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < BYTES / 16; ++q)
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((q ^ (lane & 7)) << 4)) = sixteen_bytes(c0 + PER16 * q);
          __syncwarp();
          auto staged = [&](int r, int at) { return stg + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15); };
          const int cs = n0 + half * C::HC + c0;
          if (words) {
            constexpr int L = BYTES / 4, RP = 32 / L, V = 4 / (int)sizeof(T);  // lanes a row, rows at once, values a lane
            const int u = lane % L, r0 = lane / L, left = p.T - row0 - r0, here = p.N - cs - u * V;
            T* o = static_cast<T*>(p.out) + (long)(row0 + r0) * p.out_ld + cs + u * V;
#pragma unroll 8
            for (int r = 0; r < 32; r += RP, o += RP * p.out_ld) {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(staged(r0 + r, 4 * u));
              if (r < left && here >= V)
                *reinterpret_cast<uint32_t*>(o) = v;
              else if (r < left && here > 0)  // the first of two
                *reinterpret_cast<uint16_t*>(o) = (uint16_t)v;
            }
          } else if constexpr (sizeof(T) == 2) {
            constexpr int L = N < 32 ? N : 32, RP = 32 / L;
#pragma unroll
            for (int h = 0; h < N; h += L) {
              const int c = h + lane % L, r0 = lane / L, left = p.T - row0 - r0, here = p.N - cs - c;
              T* o = static_cast<T*>(p.out) + (long)(row0 + r0) * p.out_ld + cs + c;
#pragma unroll 8
              for (int r = 0; r < 32; r += RP, o += RP * p.out_ld) {
                const T v = *reinterpret_cast<const T*>(staged(r0 + r, 2 * c));
                if (r < left && here > 0) *o = v;
              }
            }
          }
        };
        constexpr int FULL = 128 / (int)sizeof(T), REST = C::HC % FULL;
#pragma unroll
        for (int c0 = 0; c0 + FULL <= C::HC; c0 += FULL) segment(std::integral_constant<int, FULL>(), c0);
        if constexpr (REST > 0) segment(std::integral_constant<int, REST>(), C::HC - REST);
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

// 2-D map over bytes: boxes of 128 bytes x box_rows rows, 128-byte swizzle, zeros outside.  kUnsupported: not a layout
// that a map takes; anything else that goes wrong is an error of the driver's.
static cudaError_t map_bytes(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows) {
  auto enc = tmap_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t es[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : r == CUDA_ERROR_INVALID_VALUE ? kUnsupported : cudaErrorUnknown;
}

// What is looked up or set once per device: the few-token kernel's shared memory, and how many clusters
// of S of its CTAs the device holds at once (they do not span its GPCs, so it is less than its SMs over S).
template <int BN, int OCC>
static cudaError_t skinny_ready(int dev) {
  using C = p8::SkCfg<BN, OCC>;
  static std::atomic<bool> set[64];
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(p8::fp8_skinny_kernel<BN, OCC>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e == cudaSuccess) set[dev].store(true, std::memory_order_release);
  return e;
}
template <int BN, int OCC>
static int skinny_clusters(int dev, int S) {
  using C = p8::SkCfg<BN, OCC>;
  static std::atomic<int> known[64][9];
  if (dev < 0 || dev >= 64) return 0;
  int n = known[dev][S].load(std::memory_order_relaxed);
  if (n) return n - 1;
  if (skinny_ready<BN, OCC>(dev) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, p8::fp8_skinny_kernel<BN, OCC>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev][S].store(n + 1, std::memory_order_relaxed);
  return n;
}

// CTAs per tile of the few-token kernel: the most that still run all at once, with two scale
// blocks each at least.
template <int BN, int OCC>
static int skinny_split(const Fp8Args& a, int dev) {
  const int blocks = (a.K + 127) / 128;
  const long tiles = (long)((a.N + 127) / 128) * ((a.T + BN - 1) / BN);
  if (p8::SkCfg<BN, OCC>::SPLIT)
    for (int s = min(8, blocks / 2); s >= 2; --s)
      if (tiles * s <= 148 * OCC && tiles <= skinny_clusters<BN, OCC>(dev, s)) return s;
  return 1;
}

template <int BN, int OCC>
static cudaError_t launch_skinny(const Fp8Args& a, int dev, int S, cudaStream_t st) {
  using C = p8::SkCfg<BN, OCC>;
  CUtensorMap mw, mx;
  cudaError_t e = map_bytes(&mw, a.w, a.K, a.N, a.K, 128);
  if (e == cudaSuccess) e = map_bytes(&mx, a.x, a.K, a.T, a.x_ld, BN);
  if (e != cudaSuccess) return e;
  const int blocks = (a.K + 127) / 128, tiles_n = (a.N + 127) / 128;
  const long tiles_t = (a.T + BN - 1) / BN;
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
  e = skinny_ready<BN, OCC>(dev);
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
  e = cudaLaunchKernelEx(&cfg, p8::fp8_skinny_kernel<BN, OCC>, mw, mx, p);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

static cudaError_t launch_fp8_any(const Fp8Args& a, cudaStream_t st) {
  const long tiles = (long)((a.N + 63) / 64) * ((a.T + 63) / 64);
  if (tiles > 0x7fffffffl) return kUnsupported;  // (17 TB of outputs)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles);
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

// Output tiles go out by TMA stores (boxes of 16 outputs x 32 rows) where its alignment rules allow, and where a row's
// outputs end on 16 bytes: with 1087 bf16 outputs in rows of 1088 the clipped box was seen to write the last
// element of the 4 bytes that it shares with an output.
static bool out_aligned(const Fp8Args& a) {
  const int elt = a.act == MLA_F32 ? 4 : 2;
  return (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.out_ld * elt % 16 == 0 && (int64_t)a.N * elt % 16 == 0;
}
static bool map_out(CUtensorMap* m, const Fp8Args& a) {
  auto enc = tmap_encoder();
  const int elt = a.act == MLA_F32 ? 4 : 2;
  if (!enc || !out_aligned(a)) return false;
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
  cudaError_t e = map_bytes(&mw, a.w, a.K, a.N, a.K, WN / 2);
  if (e == cudaSuccess) e = map_bytes(&mx, a.x, a.K, a.T, a.x_ld, 128);
  if (e != cudaSuccess) return e;
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
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
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

// Up to 32 columns the few-token kernel comes with two CTAs per SM or with one and a deeper ring (us at 1 and
// 32 tokens, two / one per SM; a range of K per CTA that is long streams faster from fewer CTAs):
//   7168x16384 (64 blocks per CTA with one per SM)   24.1, 27.1 / 21.9, 23.5
//   4096x7168 (14)                                    7.0, 7.9 / 7.0, 7.7
//   2112x7168 (8)                                     5.4, 6.0 / 5.6, 6.1
//   24576x1536 (12, but two waves)                    8.9, 10.3 / 12.0, 13.5
template <int BN>
static cudaError_t launch_narrow(const Fp8Args& a, int dev, cudaStream_t st) {
  const int blocks = (a.K + 127) / 128, S = skinny_split<BN, 1>(a, dev);
  const long tiles = (long)((a.N + 127) / 128) * ((a.T + BN - 1) / BN);
  if (tiles <= 148 && (blocks + S - 1) / S >= 16) return launch_skinny<BN, 1>(a, dev, S, st);
  return launch_skinny<BN, 2>(a, dev, skinny_split<BN, 2>(a, dev), st);
}

// Which kernel: up to 32 tokens the few-token one (the weights' bytes decide).  Above, the variant with the
// least time by these models of what was measured on B200 (us; a wave is one round of the CTAs or pairs that
// run at once; "+ x if split" is the exchange):
//   few tokens, 32 columns    0.3 blocks per CTA + 2.7, + 0.5 if split, the blocks at 0.6 where SMs hold two CTAs
//                                                          64x576x2048: 3.8 (64 columns: 4.8), 64x2112x7168: 8.4 (7.5)
//   few tokens, 64 columns    waves (0.335 blocks per CTA + 1.8, + 1.4 if split) + 1.5
//                                                          64x7168x16384: 26 (many-token: 43), 64x14336x2048: 8.7
//     with two CTAs per SM, unsplit, for more tiles than SMs: waves (0.53 blocks + 2.2) + 1.5
//                                                          64x24576x1536: 11.2 (one CTA: 16), 64x24576x7168: 33 (49)
//   few tokens, 128 columns   waves (0.39 blocks per CTA + 5.4, + 1.4 if split) + 1.5
//                                                          128x7168x16384: 33 (64 columns: 50)
//   many tokens, 128 outputs  waves (0.26 blocks + 0.75) + 2.8           256x7168x16384: 38 (few-token: 58)
//   many tokens, 160 outputs  waves (0.307 blocks + 2) + 2.8             2048x7168x16384: 233 (128 outputs: 290)
// and 1.5 more a wave of the many-token kernel whose output rows TMA stores do not take (333x1999x2000:
// 11.0, few-token 8.8; 470x5329x256 7.3, few-token 8.3).
template <int BN, int OCC>
static float skinny_us(const Fp8Args& a, int S, float block, float wave, float exchange) {
  const int blocks = (a.K + 127) / 128;
  const long tiles = (long)((a.N + 127) / 128) * ((a.T + BN - 1) / BN);
  const long waves = S > 1 ? 1 : (tiles + 148 * OCC - 1) / (148 * OCC);
  return waves * (block * (tiles * S > 148 ? OCC : 1) * ((blocks + S - 1) / S) + wave + (S > 1 ? exchange : 0.f)) + 1.5f;
}
static float wide_us(const Fp8Args& a, int wn, float block, float wave) {
  const long tiles = (long)((a.N + wn - 1) / wn) * ((a.T + 255) / 256);
  return (tiles + 73) / 74 * (block * ((a.K + 127) / 128) + wave + (out_aligned(a) ? 0.f : 1.5f)) + 2.8f;
}

static cudaError_t launch_tensor_core(const Fp8Args& a, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // the few-token kernels number their tiles of 128 outputs along a grid's y
  const bool few = (a.N + 127) / 128 <= 65535;
  if (a.T <= 16 && few) return launch_narrow<16>(a, dev, st);
  if (a.T <= 32 && few) return launch_narrow<32>(a, dev, st);
  const float w128 = wide_us(a, 128, 0.26f, 0.75f), w160 = wide_us(a, 160, 0.307f, 2.f);
  if (a.T <= 1024 && few) {
    const int S32 = skinny_split<32, 2>(a, dev), S64 = skinny_split<64, 1>(a, dev), S128 = skinny_split<128, 1>(a, dev);
    const float s32 = a.T <= 128 ? skinny_us<32, 2>(a, S32, 0.3f, 1.2f, 0.5f) : 1e30f;
    const float s64 = skinny_us<64, 1>(a, S64, 0.335f, 1.8f, 1.4f);
    const bool many = (long)((a.N + 127) / 128) * ((a.T + 63) / 64) > 148;
    const float s64x2 = many ? skinny_us<64, 2>(a, 1, 0.265f, 2.2f, 0.f) : 1e30f;
    const float s128 = a.T > 64 ? skinny_us<128, 1>(a, S128, 0.39f, 5.4f, 1.4f) : 1e30f;
    const float least = fminf(fminf(s32, s64), fminf(s64x2, s128));
    if (least < fminf(w128, w160))
      return least == s32     ? launch_skinny<32, 2>(a, dev, S32, st)
             : least == s64   ? launch_skinny<64, 1>(a, dev, S64, st)
             : least == s64x2 ? launch_skinny<64, 2>(a, dev, 1, st)
                              : launch_skinny<128, 1>(a, dev, S128, st);
  }
  return w128 < w160 ? launch_wide<128>(a, st) : launch_wide<160>(a, st);
}

cudaError_t launch_project_fp8(const Fp8Args& a, cudaStream_t st) {
  // What no tensor map takes (a row distance of 2^40 bytes, say) goes to the general kernel as well.
  const cudaError_t e = tma_layout(a) ? launch_tensor_core(a, st) : kUnsupported;
  return e == kUnsupported ? launch_fp8_any(a, st) : e;
}

}  // namespace mla
