// Products with 4-bit weights for more than 16 tokens, on tcgen05: 128 weight rows
// are the M side of the MMAs, 32 or 64 tokens the N side.
//
// The codes become bf16 integers code - zero (exact) on their way into TMEM, from where
// the MMAs take the weights' side: a lane per weight row.  (Through shared memory their
// four bytes a code, written and read, were the bound: 45 us.)  The tokens arrive in
// shared memory by TMA as they are.  Products are exact, sums within a group are the
// tensor core's in TMEM (four accumulators in turn), and the epilogue adds each group's
// sum times its scale to fp32 sums in registers, again a lane per weight row.  Sums over
// a part of K go to memory and are added by the kernel that follows.
//
// On mma.m16n8k16, which moves every product's operands through the register file, 64
// tokens through [28672, 4096] took 88 us for the 43.1 here (1.4 TB/s of codes; 62 MB).
// What bounds it is the chain of barriers for each 128-deep stage: without any MMA or
// arithmetic on the codes it takes 30.
//
// Every 64 tokens convert the codes again: 2048 tokens take 1409 us, 44 for each 64.
//
// Warps: 0 requests the tokens' tiles, 1 issues the MMAs, 2-5 are the epilogue, 6-13
// turn codes into operands: 32 rows (the TMEM lanes of the warp) by half a stage each.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "pipe.cuh"
#include "ptx.cuh"
#include "w4.cuh"

namespace fp8lin {
namespace {

constexpr int kDepth = 128;              // codes of a row in a stage
constexpr int kStages = 4;               // stages of the weights' operand
constexpr int kStagesB = 6;              // and of the tokens', which come from L2
constexpr int kRing = 8;                 // tiles of codes that a warp has requested
constexpr int kWorkers = 8, kThreads = 32 * (6 + kWorkers);
constexpr int kColsA = kDepth / 2;       // TMEM columns of an operand stage
constexpr int kAcc = 4;                  // accumulators (a power of two)
constexpr int kTmemCols = 512;           // the operand stages, then the accumulators
constexpr int kCodes = 32 * kDepth / 4;  // of one warp and stage: 32 rows of 32 bytes
constexpr int kZeros = 32 * 8;           // its zero points' words
__device__ unsigned g_w4_wide_status;

struct Control {
  uint64_t a_full[kStages], a_empty[kStages], b_full[kStagesB], b_empty[kStagesB];
  uint64_t acc_full[kAcc], acc_empty[kAcc];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

// lists: first token and tiles of tokens before each, and behind the last one.
template <int TN>
constexpr int smem_bytes(int lists) {
  return 1024 + kStagesB * TN * kDepth * 2 + kWorkers * kRing * (kCodes + kZeros) + (int)sizeof(Control) + 8 * (lists + 1);
}

// D[tmem] (+)= A[tmem] B[smem]^T on bf16 operands, issued by one thread.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 32 consecutive 32-bit columns, lane i of the warp to lane (base lane + i).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Instruction descriptor for kind::f16: fp32 accumulator, bf16 A and B, both K-major.
constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Byte j of w, two codes, as bf16 numbers less their zero point: zz = (128 + zero)
// twice.  mask 0x000f000f and bias 0x43004300 come in registers: as constants they took
// an instruction each.
__device__ __forceinline__ uint32_t two_codes(uint32_t w, int j, uint32_t zz, uint32_t mask, uint32_t bias) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(__byte_perm(w, 0u, 0x4440 + j) * 0x1001u), "r"(mask), "r"(bias));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&zz));
  return *reinterpret_cast<const uint32_t *>(&d);
}

// One unit of work: 128 weight rows (gated: 64 of the gate, 64 of the up projection) by
// one part of K, for one tile of a list's tokens.
struct Unit {
  int e, token, count, tile, part, kb0, kbs;  // first token, and the list's tokens from it on
};

template <int TN, int GROUP>
__global__ void __launch_bounds__(kThreads, 1)
    w4_wide_kernel(const __grid_constant__ CUtensorMap tmX, const W4Args a, const int parts, const int per_part) {
  constexpr int kGroups = kDepth / GROUP;  // groups of a row in a stage
  constexpr int kOperandB = TN * kDepth * 2;
  constexpr int kSteps = GROUP / 16;  // MMAs to a group
  constexpr int kHalfGroups = kGroups > 1 ? kGroups / 2 : 1;  // of a row in half a stage
  constexpr int kZeroWords = (kHalfGroups + 6) / 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *opB = smem;
  uint8_t *rings = opB + kStagesB * kOperandB;
  Control *ctl = reinterpret_cast<Control *>(rings + kWorkers * kRing * (kCodes + kZeros));
  const int lists = a.experts ? a.E : 1;
  int *first = reinterpret_cast<int *>(ctl + 1), *before = first + lists + 1;  // of each list, and behind the last
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&ctl->a_full[s], kWorkers);
      ptx::mbar_init(&ctl->a_empty[s], 1);
    }
    for (int s = 0; s < kStagesB; ++s) {
      ptx::mbar_init(&ctl->b_full[s], 1);
      ptx::mbar_init(&ctl->b_empty[s], 1);
    }
    for (int b = 0; b < kAcc; ++b) {
      ptx::mbar_init(&ctl->acc_full[b], 1);
      ptx::mbar_init(&ctl->acc_empty[b], 4);
    }
    ptx::mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    if (!a.experts) {
      first[0] = before[0] = 0;
      first[1] = a.T;
      before[1] = (a.T + TN - 1) / TN;
    }
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl->tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_wait_then_release();
  const uint32_t tmem = ctl->tmem_base, acc0 = tmem + kStages * kColsA;
  volatile int *abort = &ctl->abort;
  const auto wait = [&](uint64_t *bar, uint32_t parity) { return pipe::wait_bar(bar, parity, abort, &g_w4_wide_status); };
  // Warps 0 and 1 wait with one lane, and leave when a wait gives up.  The others wait with
  // all: a lane whose wait gave up is `lost` and goes on with the rest of its warp (numbers
  // that are then wrong, at addresses that are not), since TMEM's loads and stores are
  // instructions of all lanes and another lane may have seen the phase end after all.  A unit
  // later the warp leaves as one.
  const int per = a.gated ? 64 : 128, kbs = (a.K + kDepth - 1) / kDepth;
  // The lists' units, one list's after the other's, are dealt out to the blocks, the tiles of
  // tokens for the same weights in a row (so the codes come from memory once, from L2 then).
  // With as many blocks for every list, 1024 tokens x 2 of 32 experts [2 2048, 4096] and
  // [4096, 2048] took 711 us, and 5278 where two experts had them all; like this 483 and 348.
  const int slices = (a.N + per - 1) / per * parts;
  if (a.experts) {
    for (int l = threadIdx.x; l <= lists; l += kThreads) first[l] = a.offsets[l];
    __syncthreads();
    if (warp == 0) {
      int sum = 0;
      for (int l0 = 0; l0 < lists; l0 += 32) {
        const int l = l0 + lane, n = l < lists ? (first[l + 1] - first[l] + TN - 1) / TN : 0;
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int v = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += v;
        }
        if (l < lists) before[l] = sum + s - n;
        sum += __shfl_sync(0xffffffffu, s, 31);
      }
      if (lane == 0) before[lists] = sum;
    }
    __syncthreads();
  }
  const int units = before[lists] * slices;
  // Unit u < units, for u that only grow; l: its list, 0 at first.
  const auto unit_of = [&](int u, int &l) {
    while (u >= before[l + 1] * slices) ++l;
    const int n = before[l + 1] - before[l], rest = u - before[l] * slices;
    const int slice = n == 1 ? rest : rest / n, tb = (rest - slice * n) * TN;
    const int tile = slice / parts, part = slice - tile * parts;
    return Unit{l, first[l] + tb, first[l + 1] - first[l] - tb, tile, part, part * per_part, min(per_part, kbs - part * per_part)};
  };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int last_phase[kStagesB];
      for (int s = 0; s < kStagesB; ++s) last_phase[s] = -1;
      bool ok = true;
      int l = 0;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit un = unit_of(u, l);
        for (int kb = un.kb0; kb < un.kb0 + un.kbs; ++kb) {
          if (!wait(&ctl->b_empty[stage], phase ^ 1)) {
            ok = false;
            break;
          }
          // (rows past the list's are read too, and not stored)
          ptx::mbar_arrive_expect_tx(&ctl->b_full[stage], kOperandB);
          uint8_t *b = opB + stage * kOperandB;
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int r = 0; r < TN; r += 32)
              ptx::tma_load_2d(b + half * (TN * 128) + r * 128, &tmX, &ctl->b_full[stage], kb * kDepth + 64 * half,
                               un.token + r);
          last_phase[stage] = (int)phase;
          if (++stage == kStagesB) stage = 0, phase ^= 1;
        }
      }
      if (!ok)  // let every issued copy land before the CTA can exit
        for (int s = 0; s < kStagesB; ++s)
          if (last_phase[s] >= 0) pipe::drain_wait(&ctl->b_full[s], (uint32_t)last_phase[s], &g_w4_wide_status);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(128, TN);
      int stage = 0, stage_b = 0;
      uint32_t phase = 0, phase_b = 0, nacc = 0;
      bool ok = true;
      int l = 0;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit un = unit_of(u, l);
        for (int kb = 0; ok && kb < un.kbs; ++kb) {
          if (!wait(&ctl->b_full[stage_b], phase_b) || !wait(&ctl->a_full[stage], phase)) {
            ok = false;
            break;
          }
          const uint32_t ta = tmem + stage * kColsA;
          const uint64_t bd = ptx::smem_desc_sw128(ptx::smem_u32(opB + stage_b * kOperandB));
          for (int g = 0; g < kGroups; ++g) {
            if (!wait(&ctl->acc_empty[nacc % kAcc], (nacc / kAcc & 1) ^ 1)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const int step = g * kSteps + k;  // 16 deep: 32 bytes of a panel of 64
              mma_bf16(acc0 + nacc % kAcc * TN, ta + 8 * step, bd + (step / 4) * (TN * 128 >> 4) + 2 * (step % 4),
                       idesc, k > 0);
            }
            ptx::mma_commit(&ctl->acc_full[nacc % kAcc]);
            ++nacc;
          }
          if (!ok) break;
          ptx::mma_commit(&ctl->a_empty[stage]);
          ptx::mma_commit(&ctl->b_empty[stage_b]);
          if (++stage == kStages) stage = 0, phase ^= 1;
          if (++stage_b == kStagesB) stage_b = 0, phase_b ^= 1;
        }
      }
      ptx::mma_commit(&ctl->mma_done);
      pipe::drain_wait(&ctl->mma_done, 0, &g_w4_wide_status);
    }
  } else if (warp < 6) {
    // lane `row` of the tile: TMEM lanes are a warp's own quarter
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tl = acc0 + ((uint32_t)(quarter * 32) << 16);
    const auto row_of = [&](const Unit &un) {  // this lane's weight row of a unit
      return (a.gated && row >= 64 ? a.N : 0) + min(un.tile * per + (a.gated ? row & 63 : row), a.N - 1);
    };
    const auto first_scale = [&](const Unit &un) {
      return bf16lo(a.scale[((int64_t)un.e * a.rows + row_of(un)) * a.groups + un.kb0 * kGroups]);
    };
    uint32_t nacc = 0;
    bool lost = false;
    int l = 0;
    Unit un = {}, then;
    float ahead = 0.0f;  // the next unit's first scale, a round trip to memory before its use
    if ((int)blockIdx.x < units) ahead = first_scale(un = unit_of(blockIdx.x, l));
    for (int u = blockIdx.x; u < units; u += gridDim.x, un = then) {
      if (__any_sync(0xffffffffu, lost)) break;
      then = u + (int)gridDim.x < units ? unit_of(u + gridDim.x, l) : un;
      const int out = un.tile * per + (a.gated ? row & 63 : row), wrow = row_of(un);
      const uint16_t *scale = a.scale + ((int64_t)un.e * a.rows + wrow) * a.groups;
      float tot[TN] = {};
      float next = ahead;
      ahead = first_scale(then);
      for (int kb = un.kb0; kb < un.kb0 + un.kbs; ++kb)
#pragma unroll 1
        for (int g = kb * kGroups; g < (kb + 1) * kGroups; ++g) {
          const float s = next;
          // (groups past the last one are products with zeros)
          next = bf16lo(scale[min(g + 1, a.groups - 1)]);
          const uint32_t ab = nacc % kAcc;
          lost |= !wait(&ctl->acc_full[ab], nacc / kAcc & 1);
          ptx::tc_fence_after();
#pragma unroll
          for (int i = 0; i < TN; i += 32) {
            uint32_t r[32];
            ptx::tmem_ld32(tl + ab * TN + i, r);
            ptx::tmem_ld_wait();
            if (i + 32 == TN) {
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(&ctl->acc_empty[ab]);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) tot[i + j] = fmaf(__uint_as_float(r[j]), s, tot[i + j]);
          }
          ++nacc;
        }
      if (lost || out >= a.N) continue;
      // a part's sums: token by token, 32 rows at a time
      float *to = static_cast<float *>(a.part) + ((int64_t)un.part * a.P + un.token) * a.rows + wrow;
      const int count = min(TN, un.count);
#pragma unroll
      for (int i = 0; i < TN; ++i)
        if (i < count) to[(int64_t)i * a.rows] = tot[i];
    }
  } else {
    const int quarter = warp & 3, half = (warp - 6) >> 2;  // rows 32 quarter .. of the tile, codes 64 half ..
    uint8_t *ring = rings + (warp - 6) * kRing * (kCodes + kZeros);
    const int row_bytes = a.K / 2;
    // copies: piece `lane & 1` (32 codes) of rows lane / 2 and lane / 2 + 16.  Four rows'
    // 128 bytes hold their pieces at piece 2 (row & 3) + which, moved by row / 4, so that
    // eight rows' same piece touch all banks
    const auto place = [](int row, int which) {
      return (row >> 2) * 128 + ((((row & 3) * 2 + which) ^ (row >> 2 & 1)) << 4);
    };
    const int crow = lane >> 1, cp = lane & 1;
    const int cto = place(crow, cp);  // (16 rows on: 512 bytes)
    const int from0 = place(lane, 0), from1 = place(lane, 1);
    // the first row of a unit's sixteen rows `j` of this warp, within the stack
    const auto first_row = [&](const Unit &un, int j) {
      const int r = (a.gated ? un.tile * 64 + (quarter & 1) * 32 : un.tile * 128 + quarter * 32) + 16 * j;
      return (int64_t)un.e * a.rows + (a.gated ? (quarter >> 1) * a.N : 0) + min(r, a.N - 16);  // past the last: not stored
    };
    // the request that runs kRing - 1 stages ahead: its unit, and where that continues
    int ru = blockIdx.x, rl = 0, rkb = 0, rkbs = 0, into = 0;
    const uint8_t *rsrc0 = nullptr, *rsrc1 = nullptr;  // this lane's next pieces
    int64_t rzero = 0;                                 // this lane's row's zero points
    const auto begin = [&] {
      const Unit un = unit_of(ru, rl);
      rkb = un.kb0;
      rkbs = un.kbs;
      const int64_t r0 = first_row(un, 0), r1 = first_row(un, 1);
      const int at = rkb * (kDepth / 2) + 32 * half + 16 * cp;
      rsrc0 = a.codes + (r0 + crow) * row_bytes + at;
      rsrc1 = a.codes + (r1 + crow) * row_bytes + at;
      rzero = ((lane < 16 ? r0 : r1) + (lane & 15)) * a.groups;
    };
    if (ru < units) begin();
    const auto group_of = [&](int kb) { return kb * kGroups + (kGroups > 1 ? half * kHalfGroups : 0); };
    const auto request = [&] {
      if (ru < units) {
        uint8_t *dst = ring + into * (kCodes + kZeros);
        if (rkb < a.K / kDepth) {
          ptx::cp_async16(dst + cto, rsrc0);
          ptx::cp_async16(dst + cto + 512, rsrc1);
        } else {
          const bool in = rkb * kDepth + 64 * half + 32 * cp < a.K;
          ptx::cp_async16_zfill(dst + cto, in ? rsrc0 : a.codes, in ? 16u : 0u);
          ptx::cp_async16_zfill(dst + cto + 512, in ? rsrc1 : a.codes, in ? 16u : 0u);
        }
        if (a.zero) {
          // the aligned words that hold this lane's row's zero points of this half stage
          const int64_t at = rzero + group_of(rkb);
          const int lead = (int)(at & 3);
#pragma unroll
          for (int i = 0; i < kZeroWords; ++i) {
            const int left = group_of(rkb) < a.groups ? lead + min(kHalfGroups, a.groups - group_of(rkb)) - 4 * i : 0;
            ptx::cp_async4(dst + kCodes + 8 * lane + 4 * i, a.zero + (left > 0 ? at - lead + 4 * i : 0),
                           left > 0 ? (uint32_t)min(left, 4) : 0u);
          }
        }
        ++rkb;
        rsrc0 += kDepth / 2;
        rsrc1 += kDepth / 2;
        if (--rkbs == 0) {
          ru += gridDim.x;
          if (ru < units) begin();
        }
      }
      ptx::cp_async_commit();
      into = into == kRing - 1 ? 0 : into + 1;
    };
    for (int i = 0; i < kRing - 1; ++i) request();
    uint32_t mask, bias;
    asm volatile("mov.b32 %0, 0x000f000f;\n mov.b32 %1, 0x43004300;" : "=r"(mask), "=r"(bias));
    const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + half * (kColsA / 2);
    int stage = 0, held = 0;
    uint32_t phase = 0;
    bool lost = false;
    int l = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      if (__any_sync(0xffffffffu, lost)) break;
      const Unit un = unit_of(u, l);
      const int64_t zero = (first_row(un, lane >> 4) + (lane & 15)) * a.groups;
      for (int kb = un.kb0; kb < un.kb0 + un.kbs; ++kb) {
        cp_async_wait_group<kRing - 2>();
        __syncwarp();
        const uint8_t *src = ring + held * (kCodes + kZeros);
        const uint4 w[2] = {*reinterpret_cast<const uint4 *>(src + from0), *reinterpret_cast<const uint4 *>(src + from1)};
        uint32_t zz[2];  // of each piece's group
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t z = 8u;
          if (a.zero) z = src[kCodes + 8 * lane + (int)((zero + group_of(kb)) & 3) + (GROUP == 32 ? i : 0)] & 15u;
          zz[i] = (0x4300u | z) * 0x10001u;
        }
        __syncwarp();
        request();  // into the tile before this one, which every lane has read
        held = held == kRing - 1 ? 0 : held + 1;
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = w[i >> 2];
          const uint32_t word = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
#pragma unroll
          for (int j = 0; j < 4; ++j) r[4 * i + j] = two_codes(word, j, zz[i >> 2], mask, bias);
        }
        lost |= !wait(&ctl->a_empty[stage], phase ^ 1);
        __syncwarp();
        ptx::tc_fence_after();
        tmem_st32(ta + stage * kColsA, r);
        tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ctl->a_full[stage]);
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
    cp_async_wait_group<0>();
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int TN, int GROUP>
cudaError_t launch_wide(const W4Args &a, const CUtensorMap &tm, const W4Plan &p, int lists, cudaStream_t st) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(w4_wide_kernel<TN, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               smem_bytes<TN>(kMaxExperts));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const int kbs = (a.K + kDepth - 1) / kDepth;
  const int per = a.gated ? 64 : 128;
  // no list has more tiles of tokens than this says, whatever the tokens' choice
  const int64_t units = ((int64_t)a.P / TN + lists) * ((a.N + per - 1) / per) * p.parts;
  if (units > INT32_MAX - (1 << 20)) return cudaErrorInvalidValue;  // units are counted in 32 bits
  return launch_kernel(w4_wide_kernel<TN, GROUP>, dim3((unsigned)std::min<int64_t>(p.blocks, units)), dim3(kThreads),
                       (size_t)smem_bytes<TN>(a.experts ? a.E : 1), st, tm, a, p.parts, (kbs + p.parts - 1) / p.parts);
}
template <int TN>
cudaError_t by_group(const W4Args &a, const CUtensorMap &tm, const W4Plan &p, int lists, cudaStream_t st) {
  if (a.group == 32) return launch_wide<TN, 32>(a, tm, p, lists, st);
  if (a.group == 64) return launch_wide<TN, 64>(a, tm, p, lists, st);
  return launch_wide<TN, 128>(a, tm, p, lists, st);
}

}  // namespace

W4Plan w4_wide_plan(int N, int K, bool gated, int tokens, int lists, int64_t P) {
  W4Plan best = {};
  best.nt = tokens <= 32 ? 4 : 8;
  best.wide = true;
  const int64_t sms = num_sms(), per = gated ? 64 : 128, tiles = (N + per - 1) / per, kbs = (K + kDepth - 1) / kDepth;
  // of tokens, if the lists are of one length
  const int64_t each_list = (P + lists - 1) / lists, token_tiles = lists * ((each_list + 8 * best.nt - 1) / (8 * best.nt));
  best.blocks = (int)sms;
  double least = 0.0;
  for (int64_t parts = 1; parts <= 8 && parts <= kbs; ++parts) {
    const int64_t each = (kbs + parts - 1) / parts, slices = tiles * ((kbs + each - 1) / each);
    const int64_t rounds = (token_tiles * slices + sms - 1) / sms;
    // in times of an SM's share of memory bandwidth for a stage of 8 KB, 0.2 us: a unit's
    // beginning and end cost about 4; the sums' bytes are written and read
    const double cost = (double)(rounds * (each + 4)) +
                        8.0 * (double)P * N * (gated ? 2 : 1) * (double)parts / (8192.0 * (double)sms);
    if (best.parts == 0 || cost < least) {
      least = cost;
      best.parts = (int)((kbs + each - 1) / each);
    }
  }
  best.planes = best.parts;
  return best;
}

cudaError_t launch_w4_wide(const W4Args &a, const W4Plan &p, int lists, cudaStream_t st) {
  CUtensorMap tm;
  if (a.experts && !a.order) return cudaErrorInvalidValue;  // the kernel takes rows in the experts' order
  if (!make_bf16_slab_map(&tm, const_cast<void *>(a.x), a.P, a.K)) return cudaErrorInvalidValue;
  return p.nt == 4 ? by_group<32>(a, tm, p, lists, st) : by_group<64>(a, tm, p, lists, st);
}

cudaError_t w4_wide_read_status(unsigned *status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_w4_wide_status, sizeof(unsigned));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_w4_wide_status, &zero, sizeof(unsigned));
}

}  // namespace fp8lin
