// Gated feed-forward on FP8 operands: both projections, the activation and
// the product in one kernel, and the backward pass's fused derivative and
// E5M2 cast.
//
//   W = [Wg; Wu] [2F, K],  G = X Wg^T,  U = X Wu^T,  H = act(G) * U
//   dG = (dH * U) * act'(G),  dU = dH * act(G)
//   act: silu, g s with s = 1 / (1 + e^-g), or the exact-erf GELU
//
// Forward: persistent CTAs (one per SM), one 128-token x 128-column tile of H
// at a time.  The B operand of the tile's MMAs is 128 rows of Wg followed by
// the same 128 rows of Wu, so one 128 x 256 accumulator holds G and U of the
// same outputs and an epilogue warp reads both from its own TMEM lanes; H is
// formed from the fp32 accumulators and rounded once.  Training keeps G and U
// as bf16 (the framework's GEMM outputs are bf16), which the backward pass
// reads.
//   warp 0      TMA producer: A (128 tokens) and B (2 x 128 weight rows),
//               128 bytes along K, 128B swizzle, ring of full/empty mbarriers
//   warp 1      TMEM allocator and tcgen05.mma issuer (kind::f8f6f4)
//   warps 2-9   epilogue; warp w reads lanes 32*(w%4)..+31 and columns
//               64*((w-2)/4)..+63 of both halves
// Tensor scaling keeps one accumulator over K; block scaling (1x128 tokens,
// 128x128 weights) promotes every 128-deep partial into fp32 registers.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "pipe.cuh"
#include "ptx.cuh"

namespace fp8lin {
namespace {

using gelu2::dup;
using gelu2::fma2;
using gelu2::mul2;
using gelu2::pk;
using gelu2::upk;

__device__ unsigned g_gated_status;

constexpr int BM = 128, BK = 128, BF = 128;  // tokens, K bytes, columns of H per tile
constexpr int BN = 2 * BF;
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemBudget = 227 * 1024;
constexpr int kMaxStages = 8;

// sigma(g) = 1 / (1 + e^-g), from the hardware's base-2 exponential and
// reciprocal (each within 2 ulp of fp32).  The reciprocal is taken of a quarter
// of the sum: it flushes results below 2^-126, and sigma falls below that at
// g = -87.3 while g sigma(g) is a normal number as far as e^-g is finite (-88.7).
__device__ __forceinline__ float sigmoid_f(float g) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(g, -1.4426950408889634f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(fmaf(e, 0.25f, 0.25f)));
  return __fmul_rn(s, 0.25f);
}
template <int ACT>
__device__ __forceinline__ void act2(float g0, float g1, float &a0, float &a1) {
  if (ACT == FP8_ACT_SILU) {
    a0 = __fmul_rn(g0, sigmoid_f(g0));
    a1 = __fmul_rn(g1, sigmoid_f(g1));
  } else {
    gelu_f2(g0, g1, a0, a1);
  }
}
// GELU and its derivative from one evaluation of the erfc fit (common.cuh):
// Phi(g) is erfc(|g| / sqrt 2) / 2 or one minus it, GELU = g Phi and
// GELU' = Phi + g phi.
__device__ __forceinline__ void gelu_both2(float g0, float g1, float &a0, float &a1, float &d0,
                                           float &d1) {
  uint64_t tq, e64;
  gelu2::parts(g0, g1, tq, e64);
  const uint64_t e = mul2(e64, dup(5.42101086242752217e-20f));  // exp(-g^2 / 2)
  float t0, t1;
  upk(mul2(tq, e), t0, t1);
  const uint64_t g = pk(g0, g1);
  const uint64_t p = pk(g0 >= 0.0f ? __fsub_rn(1.0f, t0) : t0, g1 >= 0.0f ? __fsub_rn(1.0f, t1) : t1);
  upk(mul2(g, p), a0, a1);
  upk(fma2(mul2(g, dup(0.39894228040143268f)), e, p), d0, d1);
}
// act and act' of two values
template <int ACT>
__device__ __forceinline__ void act_grad2(float g0, float g1, float &a0, float &a1, float &d0,
                                          float &d1) {
  if (ACT == FP8_ACT_SILU) {
    const float s0 = sigmoid_f(g0), s1 = sigmoid_f(g1);
    a0 = __fmul_rn(g0, s0);
    a1 = __fmul_rn(g1, s1);
    d0 = __fmul_rn(s0, fmaf(g0, 1.0f - s0, 1.0f));
    d1 = __fmul_rn(s1, fmaf(g1, 1.0f - s1, 1.0f));
  } else {
    gelu_both2(g0, g1, a0, a1, d0, d1);
  }
}

struct GatedCtl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
constexpr int kCtlBytes = (int)((sizeof(GatedCtl) + 127) / 128 * 128);

struct GCfg {
  static constexpr int kEpi = 8;
  static constexpr int kThreads = 32 * (2 + kEpi);
  static constexpr int kStageA = BM * BK, kStageB = BN * BK;
  static constexpr int kStageBytes = kStageA + kStageB;
  static constexpr int kSlabBytes = 32 * 128;  // 32 tokens x 64 bf16 columns
  // One slab buffer per warp, which leaves room for a fourth operand stage
  // (131072 x 2048, K 512, keeping G and U: 302 us; two buffers, three stages 324)
  static constexpr int kOutBytes = kEpi * kSlabBytes;
  static constexpr int kRing = kSmemBudget - 1024 - kOutBytes - kCtlBytes;
  static constexpr int kStages = kRing / kStageBytes;
  static constexpr size_t kSmemBytes =
      1024 + (size_t)kStages * kStageBytes + kOutBytes + kCtlBytes;
  static_assert(kStages >= 2 && kStages <= kMaxStages, "operand ring");
};

struct GatedArgs {
  int64_t N, F;
  int tiles_m, tiles_f, kbs;
  int64_t units;
  const float *x_sinv, *w_sinv;
  int64_t lds;  // row stride (floats) of both block scale arrays
  uint32_t idesc;
  int group_m;  // > 0: units run in groups of group_m token tiles
};

__device__ __forceinline__ void decode_unit(const GatedArgs &g, int64_t u64, int &tm, int &tf) {
  const uint32_t u = (uint32_t)u64, tiles_f = (uint32_t)g.tiles_f;
  if (g.group_m > 0) {
    const uint32_t gmax = (uint32_t)g.group_m, per_group = gmax * tiles_f;
    const uint32_t m0 = u / per_group * gmax, rem = u % per_group;
    const uint32_t gm = min(gmax, (uint32_t)g.tiles_m - m0);
    tm = (int)(m0 + rem % gm);
    tf = (int)(rem / gm);
  } else {
    tm = (int)(u / tiles_f);
    tf = (int)(u % tiles_f);
  }
}

// 32 packed bf16 pairs (64 columns) of one token into a 32 x 64 slab (128-byte
// rows, 128-byte swizzle, as the TMA store expects).
__device__ __forceinline__ void stage64(uint8_t *slab, int row, const uint32_t (&w)[32]) {
  uint8_t *rp = slab + row * 128;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4 *>(rp + ((c ^ (row & 7)) * 16)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

template <int SCALING, int ACT, bool SAVE>
__global__ void __launch_bounds__(GCfg::kThreads, 1)
    gated_fwd_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmU, const GatedArgs g) {
  using C = GCfg;
  constexpr bool kTensor = SCALING == FP8_SCALING_TENSOR;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *out_stage = smem + (size_t)kStages * C::kStageBytes;
  GatedCtl *ctl = reinterpret_cast<GatedCtl *>(out_stage + C::kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&ctl->full[s], 1);
      ptx::mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctl->acc_full[b], 1);
      ptx::mbar_init(&ctl->acc_empty[b], C::kEpi);
    }
    ptx::mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tmX);
    ptx::tma_prefetch_desc(&tmW);
    ptx::tma_prefetch_desc(&tmH);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_wait();  // dependents launch as this grid exits
  const uint32_t tmem = ctl->tmem_base;
  volatile int *abort = &ctl->abort;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return pipe::wait_bar(bar, parity, abort, &g_gated_status);
  };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int last_phase[kStages];
      for (int s = 0; s < kStages; ++s) last_phase[s] = -1;
      bool ok = true;
      for (int64_t u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
        int tm, tf;
        decode_unit(g, u, tm, tf);
        for (int kb = 0; kb < g.kbs; ++kb) {
          if (!wait(&ctl->empty[stage], phase ^ 1)) { ok = false; break; }
          uint8_t *sa = smem + (size_t)stage * C::kStageBytes;
          ptx::mbar_arrive_expect_tx(&ctl->full[stage], C::kStageBytes);
          ptx::tma_load_2d(sa, &tmX, &ctl->full[stage], kb * BK, tm * BM);
          // gate rows, then the up rows of the same columns.  Of a ragged last tile the
          // gate part reads on into Wu and the up part past the weight (zeros): columns
          // that are not stored
          ptx::tma_load_2d(sa + C::kStageA, &tmW, &ctl->full[stage], kb * BK, tf * BF);
          ptx::tma_load_2d(sa + C::kStageA + BF * BK, &tmW, &ctl->full[stage], kb * BK,
                           (int)g.F + tf * BF);
          last_phase[stage] = (int)phase;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok)  // let every issued copy land before the CTA can exit
        for (int s = 0; s < kStages; ++s)
          if (last_phase[s] >= 0)
            pipe::drain_wait(&ctl->full[s], (uint32_t)last_phase[s], &g_gated_status);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, nacc = 0;
      bool ok = true;
      for (int64_t u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
        for (int kb = 0; kb < g.kbs; ++kb) {
          const bool first = !kTensor || kb == 0, last = !kTensor || kb == g.kbs - 1;
          if (!wait(&ctl->full[stage], phase)) { ok = false; break; }
          const uint32_t a_addr = ptx::smem_u32(smem + (size_t)stage * C::kStageBytes);
          const uint64_t adesc = ptx::smem_desc_sw128(a_addr);
          const uint64_t bdesc = ptx::smem_desc_sw128(a_addr + C::kStageA);
          const uint32_t d = tmem + (nacc & 1) * BN;
          // waited for last, and handed over first below: this handover bounds
          // block scaling (2049 tokens, K 4096, F 14336: 224 -> 220 us)
          if (first && !wait(&ctl->acc_empty[nacc & 1], ((nacc >> 1) & 1) ^ 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            ptx::mma_f8f6f4(d, adesc + 2 * k, bdesc + 2 * k, g.idesc, (!first || k > 0) ? 1u : 0u);
          if (last) {
            ptx::mma_commit(&ctl->acc_full[nacc & 1]);
            ++nacc;
          }
          ptx::mma_commit(&ctl->empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      ptx::mma_commit(&ctl->mma_done);
      pipe::drain_wait(&ctl->mma_done, 0, &g_gated_status);
    }
  } else {
    const int ew = warp - 2, q = warp & 3, h = ew >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * 64);
    uint32_t nacc = 0;
    uint8_t *slab = out_stage + (size_t)ew * C::kSlabBytes;
    float s_tensor = 0.0f;
    if (kTensor) s_tensor = __fmul_rn(g.x_sinv[0], g.w_sinv[0]);
    auto release_acc = [&](uint32_t ab) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->acc_empty[ab]);
    };
    auto emit = [&](const CUtensorMap *map, const uint32_t (&w)[32], int col0, int row0) {
      if (lane == 0) ptx::bulk_wait_read<0>();
      __syncwarp();
      stage64(slab, lane, w);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::tma_store_2d(map, slab, col0, row0);
        ptx::bulk_commit();
      }
    };
    for (int64_t u = blockIdx.x; u < g.units; u += gridDim.x) {
      int tm, tf;
      decode_unit(g, u, tm, tf);
      const int row0 = tm * BM + q * 32, col0 = tf * BF + h * 64;
      const bool stored = row0 < g.N && col0 < g.F;  // otherwise the slab is wholly outside
      uint32_t hp[32], gp[SAVE ? 32 : 1], up[SAVE ? 32 : 1];
      // columns 32 half .. +31 of this warp's 64, as G and U
      auto finish = [&](int half, const float (&G)[32], const float (&U)[32]) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float a0, a1;
          act2<ACT>(G[2 * j], G[2 * j + 1], a0, a1);
          hp[16 * half + j] =
              pack_bf16x2(__fmul_rn(a0, U[2 * j]), __fmul_rn(a1, U[2 * j + 1]));
          if constexpr (SAVE) {
            gp[16 * half + j] = pack_bf16x2(G[2 * j], G[2 * j + 1]);
            up[16 * half + j] = pack_bf16x2(U[2 * j], U[2 * j + 1]);
          }
        }
      };
      if constexpr (kTensor) {
        const uint32_t ab = nacc & 1;
        if (!wait(&ctl->acc_full[ab], (nacc >> 1) & 1)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t rg[32], ru[32];
          ptx::tmem_ld32(tl + ab * BN + 32 * half, rg);
          ptx::tmem_ld32(tl + ab * BN + BF + 32 * half, ru);
          ptx::tmem_ld_wait();
          if (half == 1) release_acc(ab);
          float G[32], U[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            G[j] = __fmul_rn(__uint_as_float(rg[j]), s_tensor);
            U[j] = __fmul_rn(__uint_as_float(ru[j]), s_tensor);
          }
          finish(half, G, U);
        }
        ++nacc;
      } else {
        uint64_t acc[64];  // pairs: G columns 0..63, then U columns 0..63
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = 0;
        const int64_t m = (int64_t)row0 + lane;
        const float *xrow = g.x_sinv + (m < g.N ? m : g.N - 1) * g.lds;
        const float *wg = g.w_sinv + (int64_t)tf * g.lds;  // F is a multiple of 128
        const float *wu = wg + (g.F / BF) * g.lds;
        bool ok = true;
        float xs = xrow[0], gs = wg[0], us = wu[0];
        for (int kb = 0; kb < g.kbs; ++kb) {
          const uint32_t ab = nacc & 1;
          const uint64_t sg = dup(__fmul_rn(xs, gs)), su = dup(__fmul_rn(xs, us));
          if (kb + 1 < g.kbs) {
            xs = xrow[kb + 1];
            gs = wg[kb + 1];
            us = wu[kb + 1];
          }
          if (!wait(&ctl->acc_full[ab], (nacc >> 1) & 1)) { ok = false; break; }
          ptx::tc_fence_after();
          // 16 columns at a time, G then U (loads kept in flight across chunks or
          // K blocks measured no faster: 1815 against 1787 us, and slower)
          uint32_t raw[16];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            ptx::tmem_ld16(tl + ab * BN + (c >> 2) * BF + 16 * (c & 3), raw);
            ptx::tmem_ld_wait16(raw);
            if (c == 7) release_acc(ab);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[8 * c + j] = fma2(pk(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1])),
                                    c < 4 ? sg : su, acc[8 * c + j]);
          }
          ++nacc;
        }
        if (!ok) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float G[32], U[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            upk(acc[16 * half + j], G[2 * j], G[2 * j + 1]);
            upk(acc[32 + 16 * half + j], U[2 * j], U[2 * j + 1]);
          }
          finish(half, G, U);
        }
      }
      if (stored) {
        emit(&tmH, hp, col0, row0);
        if constexpr (SAVE) {
          emit(&tmG, gp, col0, row0);
          emit(&tmU, up, col0, row0);
        }
      }
    }
    if (lane == 0) ptx::bulk_wait<0>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- few tokens
// Up to 64 tokens the weight is all the traffic that counts, so the operands
// trade places: 128 weight rows are the M side of the MMAs (gate rows and up
// rows as two accumulators) and NT = 16, 32 or 64 tokens the N side.  One CTA
// streams 256 weight rows of one K range; a cluster of S CTAs shares a tile of
// 128 outputs, splits K, and sums the S partials in rank order over
// distributed shared memory (deterministic, one launch, no workspace).
//
// Tokens that nothing else needs in FP8 (no backward pass follows) can be given
// in bf16: the epilogue warps, idle until the first product, quantize the CTA's
// K blocks into shared memory while the weight's first tiles arrive.  The codes
// and scales are gated_quant_few_kernel's, whose launch is saved (1 token, K
// 4096, F 14336: 23.9 -> 22.5 us; 37 tokens, K 512, F 2048: 8.7 -> 6.8).
constexpr int kSmallEpi = 8;  // epilogue warps: 4 for G, 4 for U
constexpr int kSmallThreads = 32 * (2 + kSmallEpi);  // producer, MMA issuer, epilogue
constexpr int kSmallTokens = 64;  // per CTA
constexpr int kSmallMaxStages = 6;
constexpr int kSmallOwnX = 36 * 1024;  // most of it for tokens that the CTA quantizes itself
constexpr int kSmallOwnItems = 64;     // and most of them, tokens x K blocks
constexpr int kSmallSmem = 200 * 1024;  // one CTA per SM, room for the quantizer's beside it

struct SmallCtl {
  uint64_t full[kSmallMaxStages], empty[kSmallMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done, x_ready;
  uint32_t tmem_base;
  int abort;
  float xmax[kSmallEpi], x_sinv;  // bf16 tokens, tensor scaling
};
constexpr int kSmallCtlBytes = (int)((sizeof(SmallCtl) + 127) / 128 * 128);

struct SmallArgs {
  int64_t N, F;
  int kbs, kbs_cta, split, stages;
  int ring_bytes;
  const float *x_sinv, *w_sinv;
  uint32_t idesc;
  __nv_bfloat16 *H, *G, *U;  // G and U null: not kept
  const uint4 *x;            // bf16 tokens [N, K], or null: FP8 tokens by tmX and x_sinv
  int64_t K;
};
// Shared memory of a CTA's quantized tokens: rows of 128 bytes in groups of 8 per
// K block.  The MMA reads NT rows; those past the tokens' last group are the next
// block's (or the pad's), and only reach accumulator columns that nothing reads.
__host__ __device__ constexpr int x_group_bytes(int tokens) { return (tokens + 7) / 8 * 1024; }
__host__ __device__ constexpr int x_tile_bytes(int kbs_cta, int tokens, int nt) {
  return kbs_cta * x_group_bytes(tokens) + nt * BK - x_group_bytes(tokens);
}

__device__ __forceinline__ float amax8(float m, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) m = amax_acc(amax_acc(m, bf16lo(w[k])), bf16hi(w[k]));
  return m;
}
__device__ __forceinline__ uint2 cast_e4m3(uint4 v, float s) {
  uint2 q;
  q.x = cvt4<FP8_FORMAT_E4M3>(__fmul_rn(bf16lo(v.x), s), __fmul_rn(bf16hi(v.x), s),
                              __fmul_rn(bf16lo(v.y), s), __fmul_rn(bf16hi(v.y), s));
  q.y = cvt4<FP8_FORMAT_E4M3>(__fmul_rn(bf16lo(v.z), s), __fmul_rn(bf16hi(v.z), s),
                              __fmul_rn(bf16lo(v.w), s), __fmul_rn(bf16hi(v.w), s));
  return q;
}

template <int SCALING, int ACT, int NT>
__global__ void __launch_bounds__(kSmallThreads, 1)
    gated_small_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmW, const SmallArgs a) {
  constexpr bool kTensor = SCALING == FP8_SCALING_TENSOR;
  constexpr uint32_t kCols = 4 * NT;  // two buffers of G and U
  const bool own_x = a.x != nullptr;
  const int stage_bytes = 2 * BF * BK + (own_x ? 0 : NT * BK);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  SmallCtl *ctl = reinterpret_cast<SmallCtl *>(ring + a.ring_bytes);
  float *xsc = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(ctl) + kSmallCtlBytes);
  uint8_t *xq = ring + (size_t)a.stages * stage_bytes;  // own_x (inside ring_bytes)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x % a.split, f0 = (int)blockIdx.x / a.split * BF;
  const int n0 = (int)blockIdx.y * NT;                      // first token
  const int tokens = (int)min((int64_t)NT, a.N - n0);       // of this CTA
  // K blocks rank, rank + split, ...: the cluster reads neighbouring 128-byte
  // pieces of the same weight rows at the same time
  const int nkb = (a.kbs - rank + a.split - 1) / a.split;
  auto kx = [&](int i) { return (rank + a.split * i) * BK; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(&ctl->full[s], 1);
      ptx::mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&ctl->acc_full[b], 1);
      ptx::mbar_init(&ctl->acc_empty[b], kSmallEpi);
    }
    ptx::mbar_init(&ctl->mma_done, 1);
    ptx::mbar_init(&ctl->x_ready, kSmallEpi);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_wait();
  const uint32_t tmem = ctl->tmem_base;
  volatile int *abort = &ctl->abort;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return pipe::wait_bar(bar, parity, abort, &g_gated_status);
  };
  float *red = reinterpret_cast<float *>(ring);  // [2][NT][128] partials, once the ring is idle

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int issued = 0;
      for (; issued < nkb; ++issued) {
        if (!wait(&ctl->empty[stage], phase ^ 1)) { ok = false; break; }
        uint8_t *sw = ring + (size_t)stage * stage_bytes;
        ptx::mbar_arrive_expect_tx(&ctl->full[stage], (uint32_t)stage_bytes);
        ptx::tma_load_2d(sw, &tmW, &ctl->full[stage], kx(issued), f0);
        ptx::tma_load_2d(sw + BF * BK, &tmW, &ctl->full[stage], kx(issued), (int)a.F + f0);
        if (!own_x) ptx::tma_load_2d(sw + 2 * BF * BK, &tmX, &ctl->full[stage], kx(issued), n0);
        if (++stage == a.stages) { stage = 0; phase ^= 1; }
      }
      if (!ok)  // the last copies of each stage land before the CTA can exit
        for (int i = max(0, issued - a.stages); i < issued; ++i)
          pipe::drain_wait(&ctl->full[i % a.stages], (uint32_t)((i / a.stages) & 1), &g_gated_status);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, nacc = 0;
      const bool have_x = !own_x || wait(&ctl->x_ready, 0);
      for (int i = 0; have_x && i < nkb; ++i) {
        const bool first = !kTensor || i == 0, last = !kTensor || i == nkb - 1;
        if (first) {
          if (!wait(&ctl->acc_empty[nacc & 1], ((nacc >> 1) & 1) ^ 1)) break;
          ptx::tc_fence_after();
        }
        if (!wait(&ctl->full[stage], phase)) break;
        ptx::tc_fence_after();
        const uint32_t w_addr = ptx::smem_u32(ring + (size_t)stage * stage_bytes);
        const uint64_t gdesc = ptx::smem_desc_sw128(w_addr);
        const uint64_t udesc = ptx::smem_desc_sw128(w_addr + BF * BK);
        const uint64_t xdesc = ptx::smem_desc_sw128(
            own_x ? ptx::smem_u32(xq) + i * x_group_bytes(tokens) : w_addr + 2 * BF * BK);
        const uint32_t d = tmem + (nacc & 1) * 2 * NT;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k) {
          const uint32_t more = (!first || k > 0) ? 1u : 0u;
          ptx::mma_f8f6f4(d, gdesc + 2 * k, xdesc + 2 * k, a.idesc, more);
          ptx::mma_f8f6f4(d + NT, udesc + 2 * k, xdesc + 2 * k, a.idesc, more);
        }
        ptx::mma_commit(&ctl->empty[stage]);
        if (last) {
          ptx::mma_commit(&ctl->acc_full[nacc & 1]);
          ++nacc;
        }
        if (++stage == a.stages) { stage = 0; phase ^= 1; }
      }
      ptx::mma_commit(&ctl->mma_done);
      pipe::drain_wait(&ctl->mma_done, 0, &g_gated_status);
    }
  } else {
    const int q = warp & 3, f = q * 32 + lane, et = (warp - 2) * 32 + lane;
    const int z = (warp - 2) >> 2;  // 0: G, 1: U
    uint64_t acc[NT / 2];           // of this weight row for every token, in pairs
#pragma unroll
    for (int n = 0; n < NT / 2; ++n) acc[n] = 0;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(z * NT);
    if (own_x) {
      float ts = 1.0f;
      const int64_t k8 = a.K / 8;
      if constexpr (kTensor) {  // the whole tensor's maximum, from L2
        float m = 0.0f;
        for (int64_t i = et; i < a.N * k8; i += 32 * kSmallEpi) m = amax8(m, a.x[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) ctl->xmax[warp - 2] = m;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kSmallEpi) : "memory");
#pragma unroll
        for (int k = 0; k < kSmallEpi; ++k) m = fmaxf(m, ctl->xmax[k]);
        float si;
        scale_from_amax(m, kE4M3Max, ts, si);
        if (et == 0) ctl->x_sinv = si;
      }
      // 16 lanes to a token's 128 columns of a K block, all requested at once
      constexpr int kPer = kSmallOwnItems / (2 * kSmallEpi);
      const int hl = lane & 15, items = tokens * nkb;
      uint4 xw[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int it = (et >> 4) + k * 2 * kSmallEpi, c = kx(it % nkb) + 8 * hl;
        xw[k] = it < items && c < a.K ? a.x[(int64_t)(n0 + it / nkb) * k8 + c / 8]
                                      : make_uint4(0, 0, 0, 0);  // past K: zeros
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int it = (et >> 4) + k * 2 * kSmallEpi, n = it / nkb, i = it % nkb;
        float s = ts, si;
        if constexpr (!kTensor) {
          float m = amax8(0.0f, xw[k]);
#pragma unroll
          for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          scale_from_amax(m, kE4M3Max, s, si);
        }
        if (it >= items) continue;
        if (!kTensor && hl == 0) xsc[i * NT + n] = si;
        *reinterpret_cast<uint2 *>(xq + i * x_group_bytes(tokens) + n * 128 +
                                   (((hl >> 1) ^ (n & 7)) * 16) + (hl & 1) * 8) = cast_e4m3(xw[k], s);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->x_ready);
      if (!kTensor) asm volatile("bar.sync 1, %0;" ::"n"(32 * kSmallEpi) : "memory");  // xsc
    } else if constexpr (!kTensor) {
      // token scales of this CTA's K blocks, [K block][token]; absent tokens: 0
      for (int i = et; i < nkb * NT; i += 32 * kSmallEpi) {
        const int n = i / nkb, k = i % nkb;
        xsc[k * NT + n] =
            n < tokens ? a.x_sinv[(int64_t)(n0 + n) * a.kbs + rank + a.split * k] : 0.0f;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kSmallEpi) : "memory");
    }
    const int uses = kTensor ? 1 : nkb;  // split <= kbs: no rank is without a block
    const float *wsc = a.w_sinv + (f0 / BF + z * (a.F / BF)) * a.kbs + rank;
    for (int i = 0; i < uses; ++i) {
      const uint32_t ab = i & 1;
      const uint64_t ws = kTensor ? 0 : dup(wsc[a.split * i]);
      if (!wait(&ctl->acc_full[ab], (i >> 1) & 1)) break;
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        uint32_t raw[16];
        ptx::tmem_ld16(tl + ab * 2 * NT + c, raw);
        ptx::tmem_ld_wait16(raw);
        if (c + 16 == NT) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl->acc_empty[ab]);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const uint64_t v = pk(__uint_as_float(raw[j]), __uint_as_float(raw[j + 1]));
          uint64_t &o = acc[(c + j) / 2];
          o = kTensor ? v : fma2(v, mul2(*reinterpret_cast<const uint64_t *>(xsc + i * NT + c + j), ws), o);
        }
      }
    }
    // the ring is idle: every MMA that read it has completed
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      float v0, v1;
      upk(acc[n / 2], v0, v1);
      red[(z * NT + n) * BF + f] = v0;
      red[(z * NT + n + 1) * BF + f] = v1;
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  if (a.split > 1) ptx::cluster_sync();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, kCols);
  // token rank + split * i of the cluster's tokens, two columns per thread
  const int pairs = BF / 2, sub = (int)threadIdx.x / pairs;  // 5 tokens at a time
  const int f = 2 * ((int)threadIdx.x % pairs);
  float s_tensor = 1.0f;
  if (kTensor) s_tensor = __fmul_rn(own_x ? ctl->x_sinv : a.x_sinv[0], a.w_sinv[0]);
  for (int n = rank + a.split * sub; n < tokens; n += a.split * (kSmallThreads / pairs)) {
    // every rank's partials are requested before the first is added
    float2 x[8], y[8];
    const uint32_t at = ptx::smem_u32(red + n * BF + f), au = at + NT * BF * 4;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      x[r] = y[r] = make_float2(0.0f, 0.0f);
      if (r < a.split) {
        if (a.split > 1) {
          x[r] = ptx::ld_shared_cluster_f2(ptx::mapa_shared(at, r));
          y[r] = ptx::ld_shared_cluster_f2(ptx::mapa_shared(au, r));
        } else {
          x[r] = *reinterpret_cast<float2 *>(red + n * BF + f);
          y[r] = *reinterpret_cast<float2 *>(red + (NT + n) * BF + f);
        }
      }
    }
    float2 g = x[0], u = y[0];
#pragma unroll
    for (int r = 1; r < 8; ++r) {
      g.x += x[r].x;
      g.y += x[r].y;
      u.x += y[r].x;
      u.y += y[r].y;
    }
    if (kTensor) {
      g.x = __fmul_rn(g.x, s_tensor);
      g.y = __fmul_rn(g.y, s_tensor);
      u.x = __fmul_rn(u.x, s_tensor);
      u.y = __fmul_rn(u.y, s_tensor);
    }
    if (f0 + f >= a.F) continue;
    float a0, a1;
    act2<ACT>(g.x, g.y, a0, a1);
    const int64_t o = (int64_t)(n0 + n) * a.F + f0 + f;
    *reinterpret_cast<uint32_t *>(a.H + o) = pack_bf16x2(__fmul_rn(a0, u.x), __fmul_rn(a1, u.y));
    if (a.G) {
      *reinterpret_cast<uint32_t *>(a.G + o) = pack_bf16x2(g.x, g.y);
      *reinterpret_cast<uint32_t *>(a.U + o) = pack_bf16x2(u.x, u.y);
    }
  }
  __syncwarp();
  if (a.split > 1) ptx::cluster_sync();  // no CTA leaves while another reads its partials
}

// Quantizer for few tokens: one CTA per 128 columns holds them for every token
// in registers.  Tensor scaling needs the whole tensor's maximum first, which
// every CTA takes for itself (at most kFewElements, from L2): one launch
// instead of two.
constexpr int kFewThreads = 256;
constexpr int64_t kFewElements = 131072;
constexpr int kFewRows = kSmallTokens / 16;  // tokens per thread

template <bool BLOCK>
__global__ void __launch_bounds__(kFewThreads)
    gated_quant_few_kernel(const uint4 *__restrict__ x, int N, int64_t K, uint8_t *__restrict__ row,
                           uint8_t *__restrict__ col, float *__restrict__ row_scale_inv,
                           float *__restrict__ col_scale, float *__restrict__ col_scale_inv) {
  __shared__ float red[8];
  __shared__ float colmx[16][128];
  __shared__ float colsc[128];
  __shared__ __align__(16) uint8_t tile[128][kSmallTokens + 16];
  pdl_wait_then_release();
  const int t = threadIdx.x, lane = t & 31, cg = t & 15, rr = t >> 4;
  const int64_t c0 = (int64_t)blockIdx.x * 128, k8 = K / 8;
  const int cols_here = (int)min((int64_t)128, K - c0);
  const bool col_ok = 8 * cg < cols_here;
  uint4 xw[kFewRows];  // tokens rr + 16 i, columns 8 cg ..
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) {
    const int n = rr + 16 * i;
    xw[i] = n < N && col_ok ? x[n * k8 + c0 / 8 + cg] : make_uint4(0, 0, 0, 0);
  }
  auto value = [&](int i, int j) {
    const uint32_t w[4] = {xw[i].x, xw[i].y, xw[i].z, xw[i].w};
    return j & 1 ? bf16hi(w[j >> 1]) : bf16lo(w[j >> 1]);
  };
  float ts = 1.0f;
  if (!BLOCK) {
    float m = 0.0f;
    for (int64_t i = t; i < N * k8; i += kFewThreads) m = amax8(m, x[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[t >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = fmaxf(m, red[w]);
    float si;
    scale_from_amax(m, kE4M3Max, ts, si);
    if (blockIdx.x == 0 && t == 0) {
      row_scale_inv[0] = si;
      if (col) {
        col_scale[0] = ts;
        col_scale_inv[0] = si;
      }
    }
  }
  float cm[8] = {};
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) {
    const int n = rr + 16 * i;
    float s = ts, m = 0.0f, v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = value(i, j);
      m = amax_acc(m, v[j]);
      cm[j] = amax_acc(cm[j], v[j]);
    }
    if (BLOCK) {
#pragma unroll
      for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float si;
      scale_from_amax(m, kE4M3Max, s, si);
      if (cg == 0 && n < N) row_scale_inv[(int64_t)n * gridDim.x + blockIdx.x] = si;
    }
    uint2 q;
    q.x = cvt4<FP8_FORMAT_E4M3>(__fmul_rn(v[0], s), __fmul_rn(v[1], s), __fmul_rn(v[2], s),
                                __fmul_rn(v[3], s));
    q.y = cvt4<FP8_FORMAT_E4M3>(__fmul_rn(v[4], s), __fmul_rn(v[5], s), __fmul_rn(v[6], s),
                                __fmul_rn(v[7], s));
    if (n < N && col_ok) *reinterpret_cast<uint2 *>(row + n * K + c0 + 8 * cg) = q;
    if (!BLOCK && col) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        tile[8 * cg + j][n] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
    }
  }
  if (!col) return;
  if (BLOCK) {  // each column's own scale over the tokens (one 1x128 block)
#pragma unroll
    for (int j = 0; j < 8; ++j) colmx[rr][8 * cg + j] = cm[j];
    __syncthreads();
    if (t < 128) {
      float m = 0.0f, s, si;
#pragma unroll
      for (int k = 0; k < 16; ++k) m = fmaxf(m, colmx[k][t]);
      scale_from_amax(m, kE4M3Max, s, si);
      colsc[t] = s;
      if (t < cols_here) {
        col_scale[c0 + t] = s;
        col_scale_inv[c0 + t] = si;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewRows; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t q = cvt2<FP8_FORMAT_E4M3>(__fmul_rn(value(i, j), colsc[8 * cg + j]),
                                                 __fmul_rn(value(i, j + 1), colsc[8 * cg + j + 1]));
        tile[8 * cg + j][rr + 16 * i] = (uint8_t)q;
        tile[8 * cg + j + 1][rr + 16 * i] = (uint8_t)(q >> 8);
      }
  }
  __syncthreads();
  const int Np = (N + 15) / 16 * 16;  // tokens past N: zeros
  for (int i = t; i < cols_here * (Np / 16); i += kFewThreads) {
    const int c = i / (Np / 16), seg = i % (Np / 16);
    *reinterpret_cast<uint4 *>(col + (c0 + c) * Np + 16 * seg) =
        *reinterpret_cast<const uint4 *>(&tile[c][16 * seg]);
  }
}

// ---------------------------------------------------------------- backward
struct GatedBwd {
  const uint4 *dh, *g, *u;  // bf16 [N, F]
  int64_t N, F, ldn;        // ldn: tokens per row of the transposed layout (N rounded up to 16)
  uint8_t *row;             // E5M2 [N, 2F]
  uint8_t *col;             // E5M2 [2F, ldn] (block scaling)
  float *row_scale_inv, *col_scale_inv;  // block scaling; tensor scaling: row_scale_inv (1)
  const float *partials;                 // tensor scaling: maxima of the first pass
  int n_partials;
};

// dG and dU of eight elements.
template <int ACT>
__device__ __forceinline__ void dgu8(uint4 dh, uint4 g, uint4 u, float (&dg)[8], float (&du)[8]) {
  const uint32_t hw[4] = {dh.x, dh.y, dh.z, dh.w}, gw[4] = {g.x, g.y, g.z, g.w},
                 uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a0, a1, d0, d1;
    act_grad2<ACT>(bf16lo(gw[k]), bf16hi(gw[k]), a0, a1, d0, d1);
    const float h0 = bf16lo(hw[k]), h1 = bf16hi(hw[k]);
    dg[2 * k] = __fmul_rn(__fmul_rn(h0, bf16lo(uw[k])), d0);
    dg[2 * k + 1] = __fmul_rn(__fmul_rn(h1, bf16hi(uw[k])), d1);
    du[2 * k] = __fmul_rn(h0, a0);
    du[2 * k + 1] = __fmul_rn(h1, a1);
  }
}

constexpr int kAmaxThreads = 256;
// Tensor scaling, first pass: per-CTA maximum of |dG| and |dU| (NaN ignored).
template <int ACT>
__global__ void __launch_bounds__(kAmaxThreads)
    gated_bwd_amax_kernel(const uint4 *__restrict__ dh, const uint4 *__restrict__ g,
                          const uint4 *__restrict__ u, int64_t n8, float *__restrict__ partials) {
  pdl_wait_then_release();
  float m = 0.0f;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += stride) {
    float dg[8], du[8];
    dgu8<ACT>(dh[i], g[i], u[i], dg, du);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = amax_acc(amax_acc(m, dg[k]), du[k]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  __shared__ float red[kAmaxThreads / 32];
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kAmaxThreads / 32; ++k) m = fmaxf(m, red[k]);
    partials[blockIdx.x] = m;
  }
}

// Eight products, each with its own scale, as E5M2.
__device__ __forceinline__ uint2 cast8(const float (&x)[8], const float (&s)[8]) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) upk(mul2(pk(x[j], x[j + 1]), pk(s[j], s[j + 1])), y[j], y[j + 1]);
  uint2 q;
  q.x = cvt4_finite<FP8_FORMAT_E5M2>(y[0], y[1], y[2], y[3]);
  q.y = cvt4_finite<FP8_FORMAT_E5M2>(y[4], y[5], y[6], y[7]);
  return q;
}

// Tensor scaling, second pass: dG and dU formed again and cast with the one
// scale, rows only; the wgrad GEMM reads them M-major, so no transposed copy is
// made: 8 bytes an output of the forward pass instead of 10, and no shared memory
// between (131072 x 2048: 309 us, 6.9 TB/s; both layouts from 128 x 128 tiles took
// 404).  Last element first, where the first pass ended.  Memory is the bound:
// requesting the next elements before the present ones are formed, 512 threads
// and streaming stores change nothing, five CTAs per SM are slower (378).
constexpr int kCastThreads = 256;
template <int ACT>
__global__ void __launch_bounds__(kCastThreads)
    gated_bwd_cast_rows_kernel(const GatedBwd p) {
  __shared__ float red[kCastThreads / 32];
  __shared__ float scale;
  pdl_wait_then_release();
  const int t = threadIdx.x;
  const int64_t f8 = p.F / 8, n8 = p.N * f8, stride = (int64_t)gridDim.x * kCastThreads;
  int64_t at = n8 - 1 - ((int64_t)blockIdx.x * kCastThreads + t);
  uint4 dh, g, u;
  if (at >= 0) dh = p.dh[at], g = p.g[at], u = p.u[at];
  float m = 0.0f;
  for (int k = t; k < p.n_partials; k += kCastThreads) m = fmaxf(m, p.partials[k]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((t & 31) == 0) red[t >> 5] = m;
  __syncthreads();
  if (t == 0) {
    for (int k = 1; k < kCastThreads / 32; ++k) m = fmaxf(m, red[k]);
    float s, si;
    scale_from_amax(m, kE5M2Max, s, si);
    scale = s;
    if (blockIdx.x == 0) p.row_scale_inv[0] = si;
  }
  __syncthreads();
  float s8[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s8[j] = scale;
  // row and column of element `at`, moved along by whole strides
  int64_t r = at >= 0 ? at / f8 : 0, c = at >= 0 ? at % f8 : 0;
  const int64_t dr = stride / f8, dc = stride % f8;
  while (at >= 0) {
    float dg[8], du[8];
    dgu8<ACT>(dh, g, u, dg, du);
    uint8_t *out = p.row + r * 2 * p.F + 8 * c;
    *reinterpret_cast<uint2 *>(out) = cast8(dg, s8);
    *reinterpret_cast<uint2 *>(out + p.F) = cast8(du, s8);
    r -= dr;
    c -= dc;
    if (c < 0) c += f8, --r;
    at -= stride;
    if (at >= 0) dh = p.dh[at], g = p.g[at], u = p.u[at];
  }
}

constexpr int kBwdThreads = 512;
struct __align__(128) BSmem {
  uint16_t in[3][128 * 128];   // dH, G, U tiles (TMA destinations)
  uint32_t tile[2][128 * 32];  // FP8 bytes of dG and dU for the transposed layout
  float colred[16][2][128];    // per-warp column maxima
  float colsc[2][128];
  float rowsc[2][128];         // row maxima, then row scales
  uint64_t full;
  int abort;
};

__device__ __forceinline__ int swz(int r) { return ((r >> 4) & 7) << 2; }

// Block scaling: one 128-token x 128-column tile of dH, G, U per iteration; dG
// and dU are formed once, in registers, and leave as E5M2 in both layouts, each
// with its own 1x128 blocks.  F is a multiple of 128.
template <int ACT>
__global__ void __launch_bounds__(kBwdThreads, 1)
    gated_bwd_cast_kernel(const __grid_constant__ CUtensorMap tmD,
                          const __grid_constant__ CUtensorMap tmG,
                          const __grid_constant__ CUtensorMap tmU, GatedBwd p) {
  extern __shared__ __align__(1024) uint8_t b_smem_raw[];
  BSmem &S = *reinterpret_cast<BSmem *>(b_smem_raw);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int cg = t & 15, rr = t >> 4;  // 8 columns, rows rr + 32 i
  const int64_t tiles_r = (p.N + 127) / 128, tiles_c = p.F / 128;
  const int64_t ntiles = tiles_r * tiles_c;
  const int64_t F2 = 2 * p.F;
  if (t == 0) {
    ptx::mbar_init(&S.full, 1);
    S.abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tmD);
    ptx::tma_prefetch_desc(&tmG);
    ptx::tma_prefetch_desc(&tmU);
  }
  __syncthreads();
  pdl_wait_then_release();
  auto prefetch = [&](int64_t id) {
    if (t != 0 || id >= ntiles) return;
    const int x = (int)(id % tiles_c) * 128, y = (int)(id / tiles_c) * 128;
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive_expect_tx(&S.full, 3u * 128 * 128 * 2);
    ptx::tma_load_2d(S.in[0], &tmD, &S.full, x, y);
    ptx::tma_load_2d(S.in[1], &tmG, &S.full, x, y);
    ptx::tma_load_2d(S.in[2], &tmU, &S.full, x, y);
  };
  int64_t id = blockIdx.x;
  prefetch(id);
  volatile int *abort = &S.abort;
  for (int k = 0; id < ntiles; ++k, id += gridDim.x) {
    const int64_t tr = id / tiles_c, tc = id % tiles_c;
    const int64_t r0 = tr * 128, c0 = tc * 128;
    const int rows_here = (int)(p.N - r0 < 128 ? p.N - r0 : 128);
    pipe::wait_bar(&S.full, k & 1, abort, &g_gated_status);
    uint4 in[3][4];  // dH, G, U of this thread's 4 rows
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k3 = 0; k3 < 3; ++k3)
        in[k3][i] = *reinterpret_cast<const uint4 *>(&S.in[k3][(rr + 32 * i) * 128 + 8 * cg]);
    // formed before the next tile is requested: the arithmetic is the bound
    // (16384 x 14336: 502 us, after it 519)
    float v[2][4][8];  // [dG, dU][row][column]
#pragma unroll
    for (int i = 0; i < 4; ++i) dgu8<ACT>(in[0][i], in[1][i], in[2][i], v[0][i], v[1][i]);
    __syncthreads();  // the buffers are read, and the last tile's transpose too
    if (*abort) {     // given up (every thread sees it): what was asked for lands before the CTA leaves
      if (t == 0) pipe::drain_wait(&S.full, k & 1, &g_gated_status);
      return;
    }
    prefetch(id + gridDim.x);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      float cm[8] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m = amax_acc(m, v[z][i][j]);
          cm[j] = amax_acc(cm[j], v[z][i][j]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (cg == 0) S.rowsc[z][rr + 32 * i] = m;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) cm[j] = fmaxf(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
      if (lane < 16) {
        float4 *dst = reinterpret_cast<float4 *>(&S.colred[warp][z][8 * cg]);
        dst[0] = make_float4(cm[0], cm[1], cm[2], cm[3]);
        dst[1] = make_float4(cm[4], cm[5], cm[6], cm[7]);
      }
    }
    __syncthreads();
    {  // one scale per thread: rows of dG, rows of dU, columns of dG, columns of dU
      const int z = (t >> 7) & 1, c = t & 127;
      float m, s, si;
      if (t < 256) {
        m = S.rowsc[z][c];
      } else {
        m = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w) m = fmaxf(m, S.colred[w][z][c]);
      }
      scale_from_amax(m, kE5M2Max, s, si);
      if (t < 256) {
        S.rowsc[z][c] = s;
        if (c < rows_here) p.row_scale_inv[(r0 + c) * (2 * tiles_c) + z * tiles_c + tc] = si;
      } else {
        S.colsc[z][c] = s;
        p.col_scale_inv[(z * p.F + c0 + c) * tiles_r + tr] = si;
      }
    }
    __syncthreads();
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      float cs[8], rs[8];
      const float4 *c4 = reinterpret_cast<const float4 *>(&S.colsc[z][8 * cg]);
      const float4 x = c4[0], y = c4[1];
      cs[0] = x.x; cs[1] = x.y; cs[2] = x.z; cs[3] = x.w;
      cs[4] = y.x; cs[5] = y.y; cs[6] = y.z; cs[7] = y.w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = rr + 32 * i;
        const float s = S.rowsc[z][r];
#pragma unroll
        for (int j = 0; j < 8; ++j) rs[j] = s;
        uint2 q = cast8(v[z][i], rs);
        if (r < rows_here)
          *reinterpret_cast<uint2 *>(p.row + (r0 + r) * F2 + z * p.F + c0 + 8 * cg) = q;
        q = cast8(v[z][i], cs);
        *reinterpret_cast<uint2 *>(&S.tile[z][r * 32 + ((2 * cg) ^ swz(r))]) = q;
      }
    }
    __syncthreads();
    {
      // tokens past N are zeros (the TMA load's fill, and dH = 0 gives 0 there)
      const int z = t >> 8, seg = t & 7, w = (t >> 3) & 31;
      if (16 * seg < rows_here) {
        uint32_t a[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = seg * 16 + i;
          a[i] = S.tile[z][r * 32 + (w ^ swz(r))];
        }
        uint32_t o[4][4];
#pragma unroll
        for (int gq = 0; gq < 4; ++gq) {
          const uint32_t t0 = __byte_perm(a[4 * gq + 0], a[4 * gq + 1], 0x5140);
          const uint32_t t1 = __byte_perm(a[4 * gq + 0], a[4 * gq + 1], 0x7362);
          const uint32_t t2 = __byte_perm(a[4 * gq + 2], a[4 * gq + 3], 0x5140);
          const uint32_t t3 = __byte_perm(a[4 * gq + 2], a[4 * gq + 3], 0x7362);
          o[0][gq] = __byte_perm(t0, t2, 0x5410);
          o[1][gq] = __byte_perm(t0, t2, 0x7632);
          o[2][gq] = __byte_perm(t1, t3, 0x5410);
          o[3][gq] = __byte_perm(t1, t3, 0x7632);
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
          *reinterpret_cast<uint4 *>(p.col + (z * p.F + c0 + 4 * w + jj) * p.ldn + r0 + 16 * seg) =
              make_uint4(o[jj][0], o[jj][1], o[jj][2], o[jj][3]);
      }
    }
  }
}

template <typename Kernel>
cudaError_t opt_in_smem(Kernel kernel, size_t bytes, bool *done) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

template <int SCALING, int ACT, bool SAVE>
cudaError_t launch_fwd(const CUtensorMap (&m)[5], const GatedArgs &g, cudaStream_t st) {
  using C = GCfg;
  static bool done[64];
  const cudaError_t e = opt_in_smem(gated_fwd_kernel<SCALING, ACT, SAVE>, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(g.units, num_sms());
  return launch_kernel(gated_fwd_kernel<SCALING, ACT, SAVE>, dim3((unsigned)grid), dim3(C::kThreads),
                       C::kSmemBytes, st, m[0], m[1], m[2], m[3], m[4], g);
}
template <int SCALING, int ACT>
cudaError_t launch_fwd_save(const CUtensorMap (&m)[5], const GatedArgs &g, bool save,
                            cudaStream_t st) {
  return save ? launch_fwd<SCALING, ACT, true>(m, g, st) : launch_fwd<SCALING, ACT, false>(m, g, st);
}

template <int SCALING, int ACT, int NT>
cudaError_t launch_small(const uint8_t *xq, const uint8_t *wq, int64_t K, SmallArgs a,
                         cudaStream_t st) {
  CUtensorMap mx, mw;
  if (!make_u8_map(&mw, wq, 2 * a.F, K, BF)) return cudaErrorInvalidValue;
  if (a.x)
    mx = mw;  // unused
  else if (!make_u8_map(&mx, xq, a.N, K, NT))
    return cudaErrorInvalidValue;
  const int stage_bytes = 2 * BF * BK + (a.x ? 0 : NT * BK);
  const int own = a.x ? x_tile_bytes(a.kbs_cta, (int)a.N, NT) : 0;
  const int scales = SCALING == FP8_SCALING_TENSOR ? 0 : a.kbs_cta * NT * 4;
  const int fixed = 1024 + kSmallCtlBytes + scales;
  a.stages =
      std::max(1, std::min({kSmallMaxStages, a.kbs_cta, (kSmallSmem - fixed - own) / stage_bytes}));
  a.ring_bytes = std::max(a.stages * stage_bytes + own, 2 * NT * BF * 4);
  a.idesc = ptx::idesc_f8f6f4(FP8_FORMAT_E4M3, FP8_FORMAT_E4M3, BM, NT);
  auto kernel = gated_small_kernel<SCALING, ACT, NT>;
  static bool done[64];
  const cudaError_t e = opt_in_smem(kernel, kSmallSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.numAttrs = 1;
  if (pdl_enabled()) {
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  cfg.gridDim = dim3((unsigned)((a.F + BF - 1) / BF * a.split), (unsigned)((a.N + NT - 1) / NT));
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = (size_t)(fixed + a.ring_bytes);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, mx, mw, a);
}
int small_nt(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : 64; }
template <int SCALING, int ACT>
cudaError_t launch_small_nt(const uint8_t *xq, const uint8_t *wq, int64_t K, const SmallArgs &a,
                            cudaStream_t st) {
  switch (small_nt(a.N)) {
    case 16: return launch_small<SCALING, ACT, 16>(xq, wq, K, a, st);
    case 32: return launch_small<SCALING, ACT, 32>(xq, wq, K, a, st);
    default: return launch_small<SCALING, ACT, 64>(xq, wq, K, a, st);
  }
}

template <int ACT>
cudaError_t launch_cast_block(const GatedBwd &p, cudaStream_t st) {
  CUtensorMap m[3];
  if (!make_bf16_tile_map(&m[0], p.dh, p.N, p.F, 128, 128) ||
      !make_bf16_tile_map(&m[1], p.g, p.N, p.F, 128, 128) ||
      !make_bf16_tile_map(&m[2], p.u, p.N, p.F, 128, 128))
    return cudaErrorInvalidValue;
  static bool done[64];
  const cudaError_t e = opt_in_smem(gated_bwd_cast_kernel<ACT>, sizeof(BSmem), done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((p.N + 127) / 128) * (p.F / 128);
  const int64_t grid = std::min<int64_t>(tiles, num_sms());
  LaunchScope ls("gated_bwd_cast_block", st, 10.0 * p.N * p.F, 0.0, p.N, p.F);
  return launch_kernel(gated_bwd_cast_kernel<ACT>, dim3((unsigned)grid), dim3(kBwdThreads),
                       sizeof(BSmem), st, m[0], m[1], m[2], p);
}

// A grid of the kernel's resident CTAs, or as many as n8 vectors fill.
template <typename Kernel>
int64_t vector_grid(Kernel kernel, int threads, int64_t n8, int *bps) {
  const int64_t resident = (int64_t)blocks_per_sm(kernel, threads, bps) * num_sms();
  return std::max<int64_t>(1, std::min<int64_t>((n8 + threads - 1) / threads, resident));
}

template <int ACT>
cudaError_t launch_cast_tensor(GatedBwd p, float *partials, cudaStream_t st) {
  const int64_t n8 = p.N * p.F / 8;
  static int amax_bps[64], cast_bps[64];
  p.n_partials = (int)std::min<int64_t>(
      vector_grid(gated_bwd_amax_kernel<ACT>, kAmaxThreads, n8, amax_bps), kMaxPartials);
  {
    LaunchScope ls("gated_bwd_amax", st, 6.0 * p.N * p.F, 0.0, p.N, p.F);
    const cudaError_t e = launch_kernel(gated_bwd_amax_kernel<ACT>, dim3((unsigned)p.n_partials),
                                        dim3(kAmaxThreads), 0, st, p.dh, p.g, p.u, n8, partials);
    if (e != cudaSuccess) return e;
  }
  p.partials = partials;
  const int64_t grid = vector_grid(gated_bwd_cast_rows_kernel<ACT>, kCastThreads, n8, cast_bps);
  LaunchScope ls("gated_bwd_cast_tensor", st, 8.0 * p.N * p.F, 0.0, p.N, p.F);
  return launch_kernel(gated_bwd_cast_rows_kernel<ACT>, dim3((unsigned)grid), dim3(kCastThreads), 0, st,
                       p);
}

// Whether the few-token kernel takes a call, and its split of K.
// Few tokens; or a deep product whose 128 x 128 tiles would fill less than
// half the SMs: chunks of 64 tokens and the split of K put more of them to
// work, the weight coming from L2 for all chunks but the first (us a pass,
// here / 128-token tiles: 100 tokens, K 4096, F 256: 11.5 / 19.4; 1000, 4096,
// 512: 19.6 / 21.4; in shallower ones the tiles win, 256, 1024, 2048: 12.1 / 10.0)
bool small_plan(int64_t N, int64_t K, int64_t F, SmallArgs &a) {
  const int64_t tiles = (F + BF - 1) / BF;
  if (N > kSmallTokens && ((N + BM - 1) / BM * tiles * 2 > num_sms() || K < 24 * BK)) return false;
  a.N = N;
  a.F = F;
  a.kbs = (int)((K + BK - 1) / BK);
  // the largest split of K that still gives every CTA an SM of its own (a
  // deep ring each; two CTAs per SM with half of it: 10 tokens at K 4096,
  // F 4096 take 11.7 us a pass, here 9.8).  A cluster lies within one GPC, so not
  // every SM can hold a CTA of one: of 152 SMs, clusters of 8 fill 120 and those
  // of 4 144, and one cluster more runs after the others (1 token, K 4096: 15
  // clusters of 8 6.3 us, 16 11.5, as clusters of 4 8.1; 36 of 4 9.3, 37 15.9, as
  // pairs 12.1).  Fixed shares with room for a GPC with fewer SMs: a split that
  // depended on the GPC would change results from one GPU to the next.
  const int64_t ctas = tiles * ((N + kSmallTokens - 1) / kSmallTokens);
  auto fits = [&](int split) {
    const int sixteenths = split == 8 ? 12 : split == 4 ? 15 : 16;
    return split <= a.kbs && ctas * split * 16 <= (int64_t)num_sms() * sixteenths;
  };
  a.split = fits(8) ? 8 : fits(4) ? 4 : fits(2) ? 2 : 1;
  a.kbs_cta = (a.kbs + a.split - 1) / a.split;
  // the token scales of a CTA's K range are kept in shared memory (K up to
  // 8192 at any split, 65536 at the full one; wider ones take the other kernel)
  return a.kbs_cta <= 64 && tiles * a.split < (int64_t(1) << 31);
}

}  // namespace

cudaError_t launch_gated_fwd(const uint8_t *xq, const float *x_sinv, const uint8_t *wq,
                             const float *w_sinv, int64_t N, int64_t K, int64_t F, bool block,
                             int act, void *H, void *G, void *U, cudaStream_t st, const void *x) {
  const bool save = G != nullptr;
  const double bytes = (double)N * K + 2.0 * F * K + (save ? 6.0 : 2.0) * N * F;
  SmallArgs a = {};
  if (small_plan(N, K, F, a)) {
    a.x_sinv = x_sinv;
    a.w_sinv = w_sinv;
    a.H = static_cast<__nv_bfloat16 *>(H);
    a.G = static_cast<__nv_bfloat16 *>(G);
    a.U = static_cast<__nv_bfloat16 *>(U);
    a.x = static_cast<const uint4 *>(x);
    a.K = K;
    LaunchScope ls(block ? "gated_small_block" : "gated_small_tensor", st, bytes + (x ? N * K : 0),
                   4.0 * N * K * F, N, F, K);
    if (block)
      return act == FP8_ACT_SILU
                 ? launch_small_nt<FP8_SCALING_1x128_128x128, FP8_ACT_SILU>(xq, wq, K, a, st)
                 : launch_small_nt<FP8_SCALING_1x128_128x128, FP8_ACT_GELU>(xq, wq, K, a, st);
    return act == FP8_ACT_SILU ? launch_small_nt<FP8_SCALING_TENSOR, FP8_ACT_SILU>(xq, wq, K, a, st)
                               : launch_small_nt<FP8_SCALING_TENSOR, FP8_ACT_GELU>(xq, wq, K, a, st);
  }
  CUtensorMap m[5];
  if (!make_u8_map(&m[0], xq, N, K, BM) || !make_u8_map(&m[1], wq, 2 * F, K, BF) ||
      !make_bf16_slab_map(&m[2], H, N, F))
    return cudaErrorInvalidValue;
  m[3] = m[4] = m[2];
  if (save && (!make_bf16_slab_map(&m[3], G, N, F) || !make_bf16_slab_map(&m[4], U, N, F)))
    return cudaErrorInvalidValue;
  GatedArgs g;
  g.N = N;
  g.F = F;
  g.tiles_m = (int)((N + BM - 1) / BM);
  g.tiles_f = (int)((F + BF - 1) / BF);
  g.kbs = (int)((K + BK - 1) / BK);
  g.units = (int64_t)g.tiles_m * g.tiles_f;
  if (g.units >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  g.x_sinv = x_sinv;
  g.w_sinv = w_sinv;
  g.lds = g.kbs;
  g.idesc = ptx::idesc_f8f6f4(FP8_FORMAT_E4M3, FP8_FORMAT_E4M3, BM, BN);
  // deep K: 16 token tiles share the weight tiles that L2 holds
  g.group_m = g.kbs >= 16 ? std::min(16, g.tiles_m) : 0;
  LaunchScope ls(block ? "gated_fwd_block" : "gated_fwd_tensor", st,
                 bytes, 4.0 * N * K * F, N, F, K);
  if (block)
    return act == FP8_ACT_SILU ? launch_fwd_save<FP8_SCALING_1x128_128x128, FP8_ACT_SILU>(m, g, save, st)
                               : launch_fwd_save<FP8_SCALING_1x128_128x128, FP8_ACT_GELU>(m, g, save, st);
  return act == FP8_ACT_SILU ? launch_fwd_save<FP8_SCALING_TENSOR, FP8_ACT_SILU>(m, g, save, st)
                             : launch_fwd_save<FP8_SCALING_TENSOR, FP8_ACT_GELU>(m, g, save, st);
}

// Up to 64 pieces of 128 columns per CTA, which its threads request at once (us a
// pass, here / through the quantizer: block, 1, 4096, 14336: 22.7 / 23.9; 37, 512,
// 2048: 6.7 / 8.4; 64, 512, 2048: 7.8 / 8.3; more lose, 37, 1024, 4096: 8.8 / 8.6; 8,
// 4096, 14336: 29.3 / 24.6), and while five stages of the weight still fit beside.
bool gated_takes_bf16(int64_t N, int64_t K, int64_t F, bool block) {
  SmallArgs a = {};
  return gated_quantizes_few(N, K, block) && small_plan(N, K, F, a) &&
         N * a.kbs_cta <= kSmallOwnItems &&
         x_tile_bytes(a.kbs_cta, (int)N, small_nt(N)) <= kSmallOwnX;
}

bool gated_quantizes_few(int64_t N, int64_t K, bool block) {
  return N <= kSmallTokens && (block || N * K <= kFewElements);
}

cudaError_t launch_gated_quantize_few(const void *x, int64_t N, int64_t K, bool block, uint8_t *row,
                                      uint8_t *col, float *row_scale_inv, float *col_scale,
                                      float *col_scale_inv, cudaStream_t st) {
  LaunchScope ls(block ? "gated_quant_few_block" : "gated_quant_few_tensor", st,
                 (col ? 4.0 : 3.0) * N * K, 0.0, N, K);
  auto kernel = block ? gated_quant_few_kernel<true> : gated_quant_few_kernel<false>;
  return launch_kernel(kernel, dim3((unsigned)((K + 127) / 128)), dim3(kFewThreads), 0, st,
                       static_cast<const uint4 *>(x), (int)N, K, row, col, row_scale_inv,
                       col_scale, col_scale_inv);
}

cudaError_t launch_gated_bwd_quantize(const void *dH, const void *G, const void *U, int64_t N,
                                      int64_t F, bool block, int act, uint8_t *row, uint8_t *col,
                                      float *row_scale_inv, float *col_scale_inv, float *partials,
                                      cudaStream_t st) {
  const GatedBwd p{static_cast<const uint4 *>(dH), static_cast<const uint4 *>(G),
                   static_cast<const uint4 *>(U), N, F, (N + 15) / 16 * 16, row, col, row_scale_inv,
                   col_scale_inv, nullptr, 0};
  if (block)
    return act == FP8_ACT_SILU ? launch_cast_block<FP8_ACT_SILU>(p, st)
                               : launch_cast_block<FP8_ACT_GELU>(p, st);
  return act == FP8_ACT_SILU ? launch_cast_tensor<FP8_ACT_SILU>(p, partials, st)
                             : launch_cast_tensor<FP8_ACT_GELU>(p, partials, st);
}

cudaError_t gated_read_status(unsigned *status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_gated_status, sizeof(unsigned));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_gated_status, &zero, sizeof(unsigned));
}

}  // namespace fp8lin
