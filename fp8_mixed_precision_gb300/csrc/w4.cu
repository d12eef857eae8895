// Products with 4-bit weights in groups along K, for few tokens:
//
//   W[n, k] = scale[n, k / group] (code[n, k] - zero[n, k / group])
//   linear  y = x W^T;   gated  h = act(x Wg^T) * (x Wu^T) with W = [Wg; Wu]
//
// for one weight, or for a stack of experts each with its own tokens.
//
// Bound by the weights' bytes, if the instructions per byte stay few.  They do with
// fp16 operands on mma.m16n8k16: a 16-bit half with a code in its lowest four or
// next four bits is the fp16 number code 2^-24 or code 2^-20 (subnormal), so a word
// of eight codes becomes four operand registers by four masks and one shift, and
// nothing is ever rounded on the weights' side.  (As bf16 operands, by or-ing codes
// into mantissas and subtracting 128 + zero, it took 15 instructions for these 5 and
// 21.5 us for one token through [28672, 4096]; as E4M3 bytes the instruction is
// emulated on this GPU, 25.9 us.)
//
// The tokens' values are scaled by a power of two, to [2^14, 2^15) for the largest
// of a warp's 256, and become fp16 too: exact for every bf16 value down to 2^-27 of
// that largest one, and below within 2^-34 of it, far less than the rounding of the
// fp32 sums.  Products are exact, sums fp32; zero points enter as zero times the
// group's sum of x; the scale is applied once per group.
//
// A block takes a range of K (256 to a warp) and walks over the weight's rows, 16
// at a time, its tokens' values in registers throughout and the codes on their way
// through a ring of asynchronous copies that every warp has for itself.  Two tiles
// of rows (gated: one of the gate, one of the up projection) end in an exchange of
// the warps' sums.  More ranges of K are the blocks of a cluster, which adds their
// sums over distributed shared memory, or are summed by a second kernel (w4_plan).
// [28672, 4096], groups of 128 without zero points, 62 MB or 8.9 us at the copy rate:
// 13.1 us for one token (ramp and tail; 39.8 for four times the rows, 6.1 TB/s), 21.8 for
// 16, where instructions bound it.  64 tokens through 32 experts [2 2048, 4096] and
// [4096, 2048], groups of 64 with zero points, 440 MB or 65 us: 137.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "w4.cuh"

namespace fp8lin {
namespace {

constexpr int kChunk = 256;              // codes of a row in a tile: 128 bytes
constexpr int kTileBytes = 16 * kChunk / 2;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kW4Cluster = 8;             // parts of K that a cluster sums
constexpr int kTokenStride = 36;         // floats from one token's sums to the next's: no bank conflicts
// Warps of an SM: registers allow 16 with up to 16 tokens to a block, 8 with more.
constexpr int w4_warps(int nt) { return nt <= 2 ? 16 : 8; }

// D += A B on fp16 operands.
__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// What a tile of a warp's ring holds: the codes, and of each row the aligned words
// that hold its scales and zero points, wherever those begin.
template <int GROUP>
struct Tile {
  static constexpr int kGroups = kChunk / GROUP;  // of a row in a tile
  static constexpr int kScaleWords = kGroups / 2 + 1, kZeroWords = (kGroups + 3 + 3) / 4;
  static constexpr int kScale = kTileBytes, kZero = kScale + 16 * kScaleWords * 4;
  static constexpr int kBytes = kZero + 16 * kZeroWords * 4;
};
// Tiles of a warp's ring: what shared memory holds with w4_warps warps to an SM.
constexpr int w4_stages(int nt, int group) { return nt == 2 || (nt == 1 && group == 32) ? 3 : nt == 1 ? 4 : 5; }
// Sums of one token and item that the warps leave before they meet.
constexpr int w4_slots(int nt) { return nt == 1 ? 16 : 8 * nt; }
// A zero point as a number.
__device__ __forceinline__ float number_of(uint8_t z) { return __uint_as_float(0x4b000000u | z) - 8388608.0f; }

// A lane's N neighbouring words of a row.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp16 values divided by 16.
__device__ __forceinline__ uint32_t sixteenth(uint32_t v) {
  const uint32_t by = 0x2c002c00u;
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&by));
  return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float gate_times(float gate, float up, int act) {
  float h;
  if (act == FP8_ACT_SILU) {
    const float t = expf(-fabsf(gate));  // no overflow on either side
    h = gate * __fdiv_rn(gate >= 0.0f ? 1.0f : t, 1.0f + t);
  } else {
    float unused;
    gelu_f2(gate, gate, h, unused);
  }
  return h * up;
}

// The lists' items, one list's after the other's, are cut into pieces of as much work, one
// for a block, which begins within a list and may go on into the next ones.  (A list's
// items cut by themselves, as many pieces of each: 64 tokens through 32 experts 173 us for
// 140.)  What a block takes of list `list`: items item0 .. item0 + mine - 1, perhaps none.
struct Piece {
  int e, first, count, item0, mine, list, last;  // last: nothing follows
};
// Not negative; a 64-bit division takes some 100 instructions.
__device__ __forceinline__ int64_t divided(int64_t a, int b) {
  return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
// All lists' work before a block's.
__device__ __forceinline__ int64_t work_before(const W4Args &a, int64_t work, unsigned block) {
  if (block == gridDim.x) return work;
  return (int64_t)__umul64hi((uint64_t)work, (uint64_t)(block * a.per_block) << 32);
}
__device__ __forceinline__ Piece piece_of(const W4List &at, int next, int items, int l, int64_t from, int64_t to) {
  const int64_t before = at.from * (int64_t)items, after = next * (int64_t)items;
  if (before >= to || before == after) return {0, 0, 0, 0, 0, l, 1};  // (the same: behind the last list)
  const int weight = next - at.from;
  const int item0 = before >= from ? 0 : (int)divided(from - before + weight - 1, weight);
  const int end = after <= to ? items : (int)divided(to - before + weight - 1, weight);
  return {at.e, at.first, at.count, item0, end - item0, l, after >= to};
}

// NT: n-tiles, of 8 tokens each.  GROUP: weights to a scale.  ZERO: zero points.
template <int NT, int GROUP, bool ZERO>
__global__ void __launch_bounds__(32 * w4_warps(NT)) w4_kernel(const W4Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  using R = Tile<GROUP>;
  constexpr int kTokens = 8 * NT, kSlots = w4_slots(NT);
  constexpr int kGroups = R::kGroups, kStages = w4_stages(NT, GROUP);
  constexpr int kSteps = GROUP / 32;  // 32-deep steps to a group
  // A lane takes kSteps neighbouring words of a row's group, lane q those from
  // q kSteps on.  The 16-byte pieces of a row stand at piece ^ f(row), so that
  // these loads touch every bank once.
  constexpr int kRows = 8 / kSteps;
  const int kw = blockDim.x / 32, wk = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  uint8_t *ring = smem + wk * kStages * R::kBytes;
  float *part = reinterpret_cast<float *>(smem + kw * kStages * R::kBytes);  // [2][kw][kSlots][kTokenStride]
  float *sums = part + 2 * kw * kSlots * kTokenStride + wk * kTokens * kGroups;  // [kGroups][kTokens]
  float *joint = sums + (kw - wk) * kTokens * kGroups;  // [2][kSlots][32]: this block's sums for its cluster
  const bool cluster = a.cluster != 0;                  // its blocks are the parts of K
  pdl_wait_then_release();
  const int chunk = blockIdx.y * kw + wk, k0 = chunk * kChunk;
  const int row_bytes = a.K / 2, group0 = chunk * kGroups;
  // Items: `per` output rows, two tiles of 16 weight rows, `second` rows apart.
  const int per = a.gated ? 16 : 32, items = (a.N + per - 1) / per, second = a.gated ? a.N : 16;

  // Codes: of each tile this lane copies piece (lane & 7) of rows lane / 8 + 0, 4, 8, 12,
  // a row's 128 bytes by eight lanes (so that writes touch every bank once, too).
  const int crow = lane >> 3, cpiece = lane & 7;
  const int to0 = crow * 128 + ((cpiece ^ crow % kRows * kSteps) << 4);
  const int to1 = (crow + 4) * 128 + ((cpiece ^ (crow + 4) % kRows * kSteps) << 4);
  const uint32_t in = k0 + 32 * cpiece < a.K ? 16u : 0u;
  const int64_t code_at = (int64_t)crow * row_bytes + (in ? k0 / 2 + 16 * cpiece : 0);
  // Scales and zero points: the words lane, lane + 32, .. of the 16 rows' words,
  // each as far as its row and chunk need it (so nothing behind the arrays is
  // touched).  Weight rows come in sixteens: what is aligned stays so.
  const int need = min(kGroups, a.groups - group0);  // perhaps none
  constexpr int kScaleOps = (16 * R::kScaleWords + 31) / 32, kZeroOps = (16 * R::kZeroWords + 31) / 32;
  int scale_at[kScaleOps], zero_at[kZeroOps];  // bytes from the item's first row's first group
  uint32_t scale_bytes[kScaleOps], zero_bytes[kZeroOps];
  const auto word = [&](int size, int id, int words, int &at, uint32_t &count) {
    const int from = (id / words * a.groups + group0) * size;
    const int lead = from & 3, left = lead + need * size - 4 * (id % words);  // bytes from this word on
    count = need > 0 && left > 0 ? (uint32_t)min(left, 4) : 0u;
    at = count ? from - lead + 4 * (id % words) : 0;
  };
#pragma unroll
  for (int m = 0; m < kScaleOps; ++m) word(2, lane + 32 * m, R::kScaleWords, scale_at[m], scale_bytes[m]);
#pragma unroll
  for (int m = 0; m < kZeroOps; ++m) word(1, lane + 32 * m, R::kZeroWords, zero_at[m], zero_bytes[m]);
  // one tile: codes at `from`, its first row's scales from group `groups` of the stack on
  const auto request = [&](const uint8_t *from, int64_t groups, uint8_t *stage) {
    ptx::cp_async16_zfill(stage + to0, from, in);
    ptx::cp_async16_zfill(stage + to1, from + 4 * row_bytes, in);
    ptx::cp_async16_zfill(stage + to0 + 1024, from + 8 * row_bytes, in);
    ptx::cp_async16_zfill(stage + to1 + 1024, from + 12 * row_bytes, in);
    const uint8_t *sc = reinterpret_cast<const uint8_t *>(a.scale + groups);
#pragma unroll
    for (int m = 0; m < kScaleOps; ++m)
      if (16 * R::kScaleWords % 32 == 0 || lane + 32 * m < 16 * R::kScaleWords)
        ptx::cp_async4(stage + R::kScale + 128 * m + 4 * lane, sc + scale_at[m], scale_bytes[m]);
    if (ZERO) {
#pragma unroll
      for (int m = 0; m < kZeroOps; ++m)
        if (16 * R::kZeroWords % 32 == 0 || lane + 32 * m < 16 * R::kZeroWords)
          ptx::cp_async4(stage + R::kZero + 128 * m + 4 * lane, a.zero + groups + zero_at[m], zero_bytes[m]);
    }
  };
  // where this lane's rows g and g + 8 have their first scale and zero point in a tile
  const int lead2 = (g & a.groups & 1) * 2, lead1 = (g * a.groups + group0) & 3;
  const int scale_lo = R::kScale + g * R::kScaleWords * 4, scale_hi = scale_lo + 8 * R::kScaleWords * 4;
  const int zero_lo = R::kZero + g * R::kZeroWords * 4 + lead1, zero_hi = zero_lo + 8 * R::kZeroWords * 4;

  // One list (one weight, or the expert of one slot of one token): a block takes items
  // blockIdx.x, blockIdx.x + gridDim.x, ..  Lists of tokens, long, short or empty: pieces.
  __shared__ Piece tk;  // (registers are scarce)
  if (a.order) {
    const int most = min(a.E, a.P);
    // (a thread's first entry and the sum come in one round trip to memory)
    int i = threadIdx.x;
    W4List at = a.lists[min(i, most - 1)];
    int next = a.lists[min(i, most - 1) + 1].from;
    const int64_t work = a.lists[most].from * (int64_t)items;
    const int64_t from = work_before(a, work, blockIdx.x), to = work_before(a, work, blockIdx.x + 1);
    if (from >= to) return;
    for (;;) {
      if (i < most && at.from * (int64_t)items <= from && from < next * (int64_t)items)
        tk = piece_of(at, next, items, i, from, to);
      if ((i += blockDim.x) >= most) break;
      at = a.lists[i];
      next = a.lists[i + 1].from;
    }
  } else if (threadIdx.x == 0) {
    const int mine = (items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const int e = a.experts ? a.experts[blockIdx.z] : 0;  // of one token: its slots are the rows
    tk = {e, a.experts ? (int)blockIdx.z : 0, a.T, (int)blockIdx.x, e >= 0 && e < a.E ? mine : 0, 0, 1};
  }
  __syncthreads();
  const int step = a.order ? per : per * (int)gridDim.x;
  for (;;) {
    const int mine = tk.mine, out0 = tk.item0 * per;
    const int64_t row0 = (int64_t)tk.e * a.rows + out0;
    const int side = a.experts ? 1 : gridDim.z, at0 = a.experts ? 0 : blockIdx.z * kTokens;
    for (int tb = at0; mine > 0 && tb < tk.count; tb += side * kTokens) {
      // the item whose tiles are requested next; a second tile past the last row: the
      // first one's rows again, read and not stored
      const uint8_t *from = a.codes + row0 * row_bytes + code_at;
      int64_t groups = row0 * a.groups;
      int ahead = 0, into = 0;
      const auto request_next = [&](int i) {
        if (ahead < mine) {
          const int more = i && (a.gated || out0 + ahead * step + 16 < a.N) ? second : 0;
          request(from + (int64_t)more * row_bytes, groups + (int64_t)more * a.groups, ring + into * R::kBytes);
          if (i) {
            ++ahead;
            from += (int64_t)step * row_bytes;
            groups += (int64_t)step * a.groups;
          }
        }
        ptx::cp_async_commit();
        into = into == kStages - 1 ? 0 : into + 1;
      };
      uint4 two[NT > 1 ? 2 : 1][8];  // the values of one n-tile's tokens, the next one's on their way
      const auto load_tokens = [&](int tb, int j, uint4(&v)[8]) {
        const int n = tb + 8 * j + g, p = tk.first + n;
        const bool some = n < tk.count;
        const int64_t row = !some ? 0 : a.tokens ? (a.order ? a.order[p] : p) / a.k : p;
        const uint16_t *x = static_cast<const uint16_t *>(a.x) + row * a.K + k0 + 8 * kSteps * q;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int k = s / kSteps * GROUP + s % kSteps * 8;
          v[s] = make_uint4(0, 0, 0, 0);
          if (some && k0 + k + 8 * kSteps * q < a.K) v[s] = *reinterpret_cast<const uint4 *>(x + k);
        }
      };
      load_tokens(tb, 0, two[0]);
#pragma unroll
      for (int s = 0; s < kStages - 1; ++s) request_next(s & 1);

      // Column g of n-tile j is token 8 j + g; lane (g, q) has the values that its
      // words' codes meet, those of the codes at bit 4 of a half divided by 16.
      uint32_t b[NT][8][4];
      float unscale[NT][2];                        // of tokens 8 j + 2 q, + 1
      float held_sums[kGroups][2];   // their groups' sums, with one n-tile
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j + 1 < NT) load_tokens(tb, j + 1, two[(j + 1) & 1]);
        const uint4(&v)[8] = two[j & 1];
        uint32_t top = 0u;  // largest |x| as bits, both halves
#pragma unroll
        for (int s = 0; s < 8; ++s)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[s].x & 0x7fff7fffu, v[s].y & 0x7fff7fffu),
                                       __vmaxu2(v[s].z & 0x7fff7fffu, v[s].w & 0x7fff7fffu)));
        top = max(top >> 16, top & 0xffffu);
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        // 2^(14 - exponent), at most 2^126; an infinity or a NaN makes the token's product NaN
        const int up = min(14 + 127 - (int)(top >> 7), 126);
        const bool bad = top >= 0x7f80u;
        const float by = __uint_as_float(bad ? 0x7fc00000u : (uint32_t)(127 + up) << 23);
        // (half of the codes' 2^24 comes back here, half behind the warps' sum: neither
        // overflows nor loses bits before the product itself does)
        const float back = __uint_as_float(bad ? 0x7fc00000u : (uint32_t)(127 + 12 - up) << 23);
        unscale[j][0] = __shfl_sync(kFull, back, 8 * q);
        unscale[j][1] = __shfl_sync(kFull, back, 8 * q + 4);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          b[j][s][0] = f16x2(bf16lo(v[s].x) * by, bf16lo(v[s].z) * by);
          b[j][s][1] = sixteenth(f16x2(bf16hi(v[s].x) * by, bf16hi(v[s].z) * by));
          b[j][s][2] = f16x2(bf16lo(v[s].y) * by, bf16lo(v[s].w) * by);
          b[j][s][3] = sixteenth(f16x2(bf16hi(v[s].y) * by, bf16hi(v[s].w) * by));
        }
        // the groups' sums as they enter the products (times -8 with no zero points):
        // products with codes of one
#pragma unroll
        for (int s = 0; s < kGroups; ++s) {
          float acc[4] = {};
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            const uint32_t *x = b[j][s * kSteps + st];
            mma_add(acc, 0x00010001u, 0u, 0x00100010u, 0u, x[0], x[1]);
            mma_add(acc, 0x00010001u, 0u, 0x00100010u, 0u, x[2], x[3]);
          }
          acc[0] *= ZERO ? -1.0f : -8.0f;
          acc[1] *= ZERO ? -1.0f : -8.0f;
          // (the products' first eight rows are alike)
          if (NT == 1)
            held_sums[s][0] = acc[0], held_sums[s][1] = acc[1];
          else if (g == 0)
            *reinterpret_cast<float2 *>(sums + s * kTokens + 8 * j + 2 * q) = make_float2(acc[0], acc[1]);
        }
      }
      __syncwarp();

      // The warps' sums meet for as many items at once as fit the buffer (all of them,
      // mostly, with one token: a barrier for each item took 3.4 us of 19.4).  Two
      // buffers in turn: a warp writes one again only behind the barrier that follows
      // its last readers.
      const int count = min(kTokens, tk.count - tb);
      const int slots = count <= 1 ? 1 : 1 << (32 - __clz(count - 1)), batch = kSlots / slots;
      int stage = 0, at = 0;
      float *buffer = part;
      // J: n-tiles that have a token
      const auto walk = [&](auto j_tiles) {
        constexpr int J = decltype(j_tiles)::value;
        for (int it = 0; it < mine; ++it) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            cp_async_wait_group<kStages - 2>();
            __syncwarp();
            request_next((kStages - 1 + i) & 1);
            const uint8_t *held = ring + stage * R::kBytes, *base = held + g * 128 + 4 * kSteps * q;
            stage = stage == kStages - 1 ? 0 : stage + 1;
            float tot[J][4] = {};
#pragma unroll
            for (int s = 0; s < kGroups; ++s) {
              uint32_t w[2][kSteps];  // codes of rows g and g + 8
#pragma unroll
              for (int h = 0; h < 2; ++h) load_words<kSteps>(base + 8 * 128 * h + ((s ^ g % kRows) * kSteps << 4), w[h]);
              const float sl = bf16lo(*reinterpret_cast<const uint16_t *>(held + scale_lo + lead2 + 2 * s));
              const float sh = bf16lo(*reinterpret_cast<const uint16_t *>(held + scale_hi + lead2 + 2 * s));
              float acc[J][4];
#pragma unroll
              for (int j = 0; j < J; ++j) {
                const float2 x = NT == 1 ? make_float2(held_sums[s][0], held_sums[s][1])
                                         : *reinterpret_cast<const float2 *>(sums + s * kTokens + 8 * j + 2 * q);
                acc[j][0] = acc[j][2] = x.x;
                acc[j][1] = acc[j][3] = x.y;
              }
              if (ZERO) {
                const float zl = number_of(held[zero_lo + s]), zh = number_of(held[zero_hi + s]);
#pragma unroll
                for (int j = 0; j < J; ++j) acc[j][0] *= zl, acc[j][1] *= zl, acc[j][2] *= zh, acc[j][3] *= zh;
              }
#pragma unroll
              for (int st = 0; st < kSteps; ++st) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t w0 = h ? w[0][st] >> 8 : w[0][st], w1 = h ? w[1][st] >> 8 : w[1][st];
                  const uint32_t a0 = w0 & 0x000f000fu, a1 = w1 & 0x000f000fu, a2 = w0 & 0x00f000f0u, a3 = w1 & 0x00f000f0u;
#pragma unroll
                  for (int j = 0; j < J; ++j)
                    mma_add(acc[j], a0, a1, a2, a3, b[j][s * kSteps + st][2 * h], b[j][s * kSteps + st][2 * h + 1]);
                }
              }
#pragma unroll
              for (int j = 0; j < J; ++j) {
                tot[j][0] = fmaf(sl, acc[j][0], tot[j][0]);
                tot[j][1] = fmaf(sl, acc[j][1], tot[j][1]);
                tot[j][2] = fmaf(sh, acc[j][2], tot[j][2]);
                tot[j][3] = fmaf(sh, acc[j][3], tot[j][3]);
              }
            }
            float *to = buffer + (wk * kSlots + at * slots + 2 * q) * kTokenStride + 16 * i + g;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
              for (int v = 0; v < 2; ++v)
                if (8 * j + 2 * q + v < slots) {
                  to[(8 * j + v) * kTokenStride] = tot[j][v] * unscale[j][v];
                  to[(8 * j + v) * kTokenStride + 8] = tot[j][2 + v] * unscale[j][v];
                }
          }
          if (++at < batch && it + 1 < mine) continue;
          __syncthreads();
          // a lane per row: `id` is one token of one item
          const auto leave = [&](int id, float v) {
            const int t = id & (slots - 1), item = it + 1 - at + id / slots;
            const int out = out0 + item * step + (a.gated ? lane & 15 : lane);
            const int64_t p = tk.first + tb + t;
            if (gridDim.y > 1 && !cluster) {  // one part of K
              if (a.gated || out < a.N)
                static_cast<float *>(a.part)[(blockIdx.y * (int64_t)a.P + p) * a.rows + (lane & 16 && a.gated ? a.N : 0) +
                                             out] = v;
            } else if (a.gated) {
              const float up = __shfl_down_sync(kFull, v, 16);
              if (lane < 16) static_cast<__nv_bfloat16 *>(a.out)[p * a.N + out] = __float2bfloat16_rn(gate_times(v, up, a.act));
            } else if (out < a.N) {
              if (a.out_f32)
                static_cast<float *>(a.out)[p * a.N + out] = v;
              else
                static_cast<__nv_bfloat16 *>(a.out)[p * a.N + out] = __float2bfloat16_rn(v);
            }
          };
          // the warps take them in turn, the next ones each time
          float *result = joint + (buffer == part ? 0 : kSlots * 32) + lane;
          int id = wk + it % kw;
          for (id = id >= kw ? id - kw : id; id < at * slots; id += kw) {
            if ((id & (slots - 1)) >= count) continue;
            float v = 0.0f;
            for (int w = 0; w < kw; ++w) v += buffer[(w * kSlots + id) * kTokenStride + lane];
            v *= 0x1p12f;
            if (cluster)
              result[id * 32] = v;
            else
              leave(id, v);
          }
          if (cluster) {
            // the parts' sums, one block's share each; what is read here is written again
            // behind the next barrier at the earliest
            __syncwarp();
            ptx::cluster_sync();
            const int rank = blockIdx.y, parts = gridDim.y;
            for (id = rank + parts * wk; id < at * slots; id += parts * kw) {
              if ((id & (slots - 1)) >= count) continue;
              const uint32_t at0 = ptx::smem_u32(result + id * 32);
              float v = 0.0f;
              for (int m = 0; m < parts; ++m) v += ptx::ld_shared_cluster_f(ptx::mapa_shared(at0, m));
              leave(id, v);
            }
            __syncwarp();
          }
          at = 0;
          buffer = part + (buffer == part) * kw * kSlots * kTokenStride;
        }
      };
      if constexpr (NT > 1) {
        if (count <= 8)
          walk(std::integral_constant<int, 1>());
        else if (NT > 2 && count <= 16)
          walk(std::integral_constant<int, 2>());
        else
          walk(std::integral_constant<int, NT>());
      } else {
        walk(std::integral_constant<int, 1>());
      }
      cp_async_wait_group<0>();
      if (cluster)
        ptx::cluster_sync();  // no block leaves, or writes again, what another still reads
      else
        __syncthreads();
    }
    if (tk.last) break;
    const int l = tk.list + 1;
    __syncthreads();
    if (threadIdx.x == 0) {
      const int64_t work = a.lists[min(a.E, a.P)].from * (int64_t)items;
      tk = piece_of(a.lists[l], a.lists[l + 1].from, items, l, work_before(a, work, blockIdx.x),
                    work_before(a, work, blockIdx.x + 1));
    }
    __syncthreads();
  }
}

// Sums the parts of K: four outputs a thread.
__global__ void __launch_bounds__(256) w4_finish_kernel(const float *__restrict__ part, int64_t total, int64_t plane,
                                                        int parts, int vecs, int N, int gated, int act,
                                                        void *__restrict__ out) {
  pdl_wait_then_release();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t p = i / vecs;
  const int c = (int)(i - p * vecs) * 4;
  const auto sum = [&](int64_t at) {
    float4 s = *reinterpret_cast<const float4 *>(part + at);
    for (int k = 1; k < parts; ++k) {
      const float4 v = *reinterpret_cast<const float4 *>(part + k * plane + at);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    return s;
  };
  float4 v = sum(p * (gated ? 2 : 1) * N + c);
  if (gated) {
    const float4 u = sum(p * 2 * N + N + c);
    v = make_float4(gate_times(v.x, u.x, act), gate_times(v.y, u.y, act), gate_times(v.z, u.z, act),
                    gate_times(v.w, u.w, act));
  }
  reinterpret_cast<uint2 *>(out)[i] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// y[t] = sum_j w[t, j] z[row of slot t k + j], z fp32 in `parts` planes; the rows of four
// slots on their way at once (one after the other 3 tokens x 8 x 2048 took 9.4 us for 7.4).
__global__ void __launch_bounds__(256) w4_join_kernel(const float *__restrict__ z, const int *__restrict__ experts,
                                                      const int *__restrict__ position,
                                                      const float *__restrict__ weights, int64_t total, int vecs, int k,
                                                      int E, int parts, int64_t plane, void *__restrict__ y) {
  constexpr int kAtOnce = 4;
  pdl_wait_then_release();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t t = i / vecs;
  const int c = (int)(i - t * vecs);
  float4 s = make_float4(0, 0, 0, 0);
  for (int j0 = 0; j0 < k; j0 += kAtOnce) {
    const float4 *from[kAtOnce];
    float w[kAtOnce];
    float4 v[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t slot = t * k + min(j0 + j, k - 1);
      const int e = experts[slot];
      const int64_t row = position ? position[slot] : slot;
      w[j] = weights[slot];
      from[j] = j0 + j < k && e >= 0 && e < E ? reinterpret_cast<const float4 *>(z) + row * vecs + c : nullptr;
      v[j] = make_float4(0, 0, 0, 0);
    }
    for (int m = 0; m < parts; ++m)
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (from[j]) {
          const float4 u = from[j][m * (plane / 4)];
          v[j].x += u.x, v[j].y += u.y, v[j].z += u.z, v[j].w += u.w;
        }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (j0 + j < k) {
        s.x = fmaf(w[j], v[j].x, s.x);
        s.y = fmaf(w[j], v[j].y, s.y);
        s.z = fmaf(w[j], v[j].z, s.z);
        s.w = fmaf(w[j], v[j].w, s.w);
      }
  }
  reinterpret_cast<uint2 *>(y)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// Codes, scales and zero points of bf16 weights, one warp per group:
//   without zero points  scale = bf16(max |w| / 7), code = 8 + round(w / scale) in 0..15
//   with                 scale = bf16((max - min) / 15) over the group and 0,
//                        zero = round(-min / scale) in 0..15, code = zero + round(w / scale) in 0..15
// A group of zeros has scale 1.  Once per weight that is loaded, so not tuned; bound by
// the instructions of a warp's group (two maxima over 32 lanes, four divisions a lane):
// [28672, 4096] in groups of 128 191 us, of 64 with zero points 631, of 32 1253, for
// 44 at the copy rate.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const void *__restrict__ w, int64_t rows, int K, int group,
                                                          int groups, uint8_t *__restrict__ codes,
                                                          uint16_t *__restrict__ scale, uint8_t *__restrict__ zero) {
  pdl_wait_then_release();
  const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (id >= rows * groups) return;
  const int64_t row = id / groups;
  const int k0 = (int)(id - row * groups) * group, len = min(group, K - k0);
  const uint16_t *src = static_cast<const uint16_t *>(w) + row * K + k0;
  float v[4];  // lane's values 4 lane ..
  float hi = 0.0f, lo = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = 4 * lane + i < len ? bf16lo(src[4 * lane + i]) : 0.0f;
    hi = fmaxf(hi, v[i]);
    lo = fminf(lo, v[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
  }
  const float top = fmaxf(hi, -lo);
  float s = zero ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(top, 7.0f);
  if (s == INFINITY) s = __fdiv_rn(0.5f * hi - 0.5f * lo, 7.5f);  // hi - lo past fp32's range, halves are exact
  s = __bfloat162float(__float2bfloat16_rn(s));
  if (s == 0.0f) s = 1.0f;
  float z = 8.0f;
  if (zero) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(v[i], s)) + z, 0.0f), 15.0f);
  if (4 * lane < len)
    *reinterpret_cast<uint16_t *>(codes + (row * K + k0) / 2 + 2 * lane) =
        (uint16_t)(c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12);
  if (lane == 0) {
    scale[id] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    if (zero) zero[id] = (uint8_t)z;
  }
}

// Dynamic shared memory of a block.
template <int NT, int GROUP>
constexpr size_t w4_bytes(int warps) {
  return (size_t)warps * (w4_stages(NT, GROUP) * Tile<GROUP>::kBytes + 2 * w4_slots(NT) * kTokenStride * 4 +
                          8 * NT * (kChunk / GROUP) * 4) +
         2 * w4_slots(NT) * 32 * 4;
}
template <int NT, int GROUP, bool ZERO>
cudaError_t allow_bytes() {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && set[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(w4_kernel<NT, GROUP, ZERO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)w4_bytes<NT, GROUP>(w4_warps(NT)));
  if (e == cudaSuccess && dev >= 0 && dev < 64) set[dev] = true;
  return e;
}
// Clusters of `parts` blocks that the GPU holds at once.  (Its processor clusters are not
// of one size: an eighth of the SMs to each gave 40 clusters of 7 blocks for the 38 that
// fit, and a second wave: 7 tokens through [16384, 14336] took 76 us
// for 41.)
template <int GROUP>
int clusters_of(int warps, int parts) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, (unsigned)parts, 1);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = w4_bytes<1, GROUP>(warps);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.z = 1;
  attr.val.clusterDim.y = (unsigned)parts;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (allow_bytes<1, GROUP, false>() == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&n, w4_kernel<1, GROUP, false>, &cfg) == cudaSuccess && n > 0)
    return n;
  cudaGetLastError();  // no GPU: the plan is not launched
  return std::max(1, num_sms() * (w4_warps(1) / warps) / parts);
}
int64_t max_clusters(int group, int warps, int parts) {
  static std::atomic<int> known[64][3][w4_warps(1) + 1][kW4Cluster + 1];  // 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  std::atomic<int> &n = known[dev][group / 64][warps][parts];
  if (n.load(std::memory_order_relaxed) == 0)
    n.store(group == 32   ? clusters_of<32>(warps, parts)
            : group == 64 ? clusters_of<64>(warps, parts)
                          : clusters_of<128>(warps, parts),
            std::memory_order_relaxed);
  return n.load(std::memory_order_relaxed);
}
template <int NT, int GROUP, bool ZERO>
cudaError_t launch_w4(const W4Args &a, const W4Plan &p, int lists, cudaStream_t st) {
  const cudaError_t e = allow_bytes<NT, GROUP, ZERO>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.blocks, (unsigned)p.parts, a.order ? 1u : (unsigned)lists);
  cfg.blockDim = dim3(32 * p.warps);
  cfg.dynamicSmemBytes = w4_bytes<NT, GROUP>(p.warps);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (a.cluster) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.z = 1;
    attr[0].val.clusterDim.y = (unsigned)p.parts;
    cfg.numAttrs = 1;
  }
  if (pdl_enabled()) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, w4_kernel<NT, GROUP, ZERO>, a);
}
template <int NT, bool ZERO>
cudaError_t by_group(const W4Args &a, const W4Plan &p, int lists, cudaStream_t st) {
  if (a.group == 32) return launch_w4<NT, 32, ZERO>(a, p, lists, st);
  if (a.group == 64) return launch_w4<NT, 64, ZERO>(a, p, lists, st);
  return launch_w4<NT, 128, ZERO>(a, p, lists, st);
}
template <int NT>
cudaError_t by_zero(const W4Args &a, const W4Plan &p, int lists, cudaStream_t st) {
  return a.zero ? by_group<NT, true>(a, p, lists, st) : by_group<NT, false>(a, p, lists, st);
}

}  // namespace

// tcgen05 from 17 tokens and 2^23 weights on, where it saves more than its second launch
// and workspace cost the host (6 us): 32 tokens through [28672, 4096] 44.4 us here and 38.7
// there, 64 tokens 79 and 43; 32 and 64 tokens through [2048, 1024] 4.6 and 6.7, 6.5 and
// 7.8, [2048, 2048] 6.7 and 7.2, 9.1 and 9.7, [4096, 1024] 6.6 and 7.3, 9.7 and 9.4, [4096,
// 2048] 9.0 and 9.1, 10.6 and 10.6; 37 through [2048, 512] 4.8 and 7.0.
// Lists from 32 tokens on in the mean, with or without an expert (us, fp16 operands and
// tcgen05: 32 experts, [2 2048, 4096] and [4096, 2048], mean 24 300 and 332, 32 366 and 336,
// 64 661 and 483, 256 2402 and 1428; 8 experts of [2 14336, 4096] and [4096, 14336], 24 465
// and 549, 32 577 and 551, 64 1074 and 803; shorter lists than the mean, 7 of 8 tokens of
// 512 without an expert, 151 and 328).
bool w4_is_wide(int64_t weights, int K, int64_t tokens, int lists) {
  return tokens >= (lists > 1 ? 32 : 17) && K >= kChunk && weights >= 1 << 23;
}

// As few as let all blocks run within two waves (a warp to 256 of K, 16 to an SM): a
// block with more has longer work, one with fewer reads the codes, which come from L2
// then, once more (37 tokens through [2048, 512] 4.8 us with 8 to a block, 6.5 with 16,
// 9.1 with 32; 12 through [4096, 4096] 6.7 with 8, 7.8 with 16; 16 through [28672, 4096]
// 23.6 with 8, 21.9 with 16).
int w4_block_tokens(int N, int K, bool gated, int64_t T) {
  const int64_t per = gated ? 16 : 32, work = (N + per - 1) / per * ((K + kChunk - 1) / kChunk);
  const int64_t two_waves = 2 * (int64_t)num_sms() * w4_warps(1);
  int tokens = 8;
  while (tokens < 32 && tokens < T && work * ((T + tokens - 1) / tokens) > two_waves) tokens *= 2;
  return tokens;
}

W4Plan w4_plan(int N, int K, int group, bool gated, int tokens, int lists, int side, int64_t P, bool joined) {
  W4Plan best = {};
  best.nt = tokens <= 8 ? 1 : tokens <= 16 ? 2 : 4;
  const int64_t sms = num_sms(), chunks = (K + kChunk - 1) / kChunk, per = gated ? 16 : 32;
  // (a list's items follow those of the list before it)
  const int64_t items = (N + per - 1) / per * lists;
  const int most = w4_warps(best.nt);
  const int64_t fewest = (chunks + most - 1) / most;
  // A cluster's exchange is worth its barriers where it saves a second kernel and the
  // sums are few (4096 x 14336, 7 tokens: 11.2 us against 11.6 and 7 us less of the
  // host; 2 x 57344 x 4096, 32 tokens: 209 us against 161).
  const bool cluster = best.nt == 1 && !joined && fewest <= kW4Cluster;
  const int64_t limit = cluster ? kW4Cluster : std::max<int64_t>(16, fewest);
  double least = 0.0;
  for (int64_t parts = fewest; parts <= limit && parts <= chunks; ++parts) {
    const int64_t warps = (chunks + parts - 1) / parts, resident = most / warps;
    const int64_t slots =
        cluster && parts > 1 ? max_clusters(group, (int)warps, (int)parts) : sms * resident / parts;
    const int64_t blocks = std::max<int64_t>(1, std::min(items, slots / side));
    const int64_t rounds = (items + blocks - 1) / blocks, together = (blocks * parts * side + sms - 1) / sms;
    // in times of an SM's share of memory bandwidth for 4 KB (a warp's two tiles),
    // about 0.1 us; an exchange costs about 2 of them, one through a cluster 6, the
    // second kernel 15, and the sums' bytes, written and read
    const double bytes = 8.0 * (double)P * N * (gated ? 2 : 1) * (double)parts;
    const double cost = (double)rounds * (double)(warps * together + (parts > 1 && cluster ? 6 : 2)) +
                        (cluster || (parts == 1 && !joined) ? 0.0 : (joined ? 0.0 : 15.0) + bytes / (4096.0 * (double)sms));
    if (best.warps == 0 || cost < least) {
      least = cost;
      best.warps = (int)warps;
      best.parts = (int)((chunks + warps - 1) / warps);
      best.blocks = (int)blocks;
    }
  }
  best.planes = cluster ? 1 : best.parts;
  return best;
}

cudaError_t launch_w4_product(W4Args a, const W4Plan &p, int lists, cudaStream_t st) {
  a.groups = (a.K + a.group - 1) / a.group;
  a.per_block = (unsigned)((1ull << 32) / (unsigned)p.blocks - (p.blocks == 1));
  a.cluster = !p.wide && p.parts > 1 && p.planes == 1;
  {
    const double weights = (double)a.rows * a.K * (a.experts ? std::min(a.E, lists) : 1);
    LaunchScope ls(a.gated ? "w4_gated" : "w4_linear", st, weights * (0.5 + (a.zero ? 3.0 : 2.0) / a.group),
                   2.0 * a.rows * a.K * a.P, a.P, a.N, a.K);
    const cudaError_t e = p.wide      ? launch_w4_wide(a, p, lists, st)
                          : p.nt == 1 ? by_zero<1>(a, p, lists, st)
                          : p.nt == 2 ? by_zero<2>(a, p, lists, st)
                                      : by_zero<4>(a, p, lists, st);
    if (e != cudaSuccess || (p.planes == 1 && !p.wide) || a.out_f32) return e;
  }
  const int vecs = a.N / 4;
  const int64_t total = (int64_t)a.P * vecs;
  LaunchScope ls("w4_finish", st, 4.0 * p.parts * a.P * a.rows + 2.0 * a.P * a.N, (double)p.parts * a.P * a.rows, a.P,
                 a.N, p.parts);
  return launch_kernel(w4_finish_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st,
                       (const float *)a.part, total, (int64_t)a.P * a.rows, p.parts, vecs, a.N, a.gated, a.act, a.out);
}

cudaError_t launch_w4_join(const float *z, const int *experts, const int *position, const float *weights, int64_t T,
                           int64_t N, int k, int E, int parts, void *y, cudaStream_t st) {
  const int vecs = (int)(N / 4);
  LaunchScope ls("w4_join", st, 4.0 * T * N * k * parts + 2.0 * T * N, 2.0 * T * N * k, T, N, k);
  return launch_kernel(w4_join_kernel, dim3((unsigned)((T * vecs + 255) / 256)), dim3(256), 0, st, z, experts, position,
                       weights, T * vecs, vecs, k, E, parts, T * k * N, y);
}

cudaError_t launch_w4_quantize(const void *w, int64_t rows, int64_t K, int group, uint8_t *codes, void *scale,
                               uint8_t *zero, cudaStream_t st) {
  const int groups = (int)((K + group - 1) / group);
  LaunchScope ls("w4_quantize", st, rows * K * (2.5 + 2.0 / group), 0.0, rows, K);
  return launch_kernel(w4_quantize_kernel, dim3((unsigned)((rows * groups + 7) / 8)), dim3(256), 0, st, w, rows, (int)K,
                       group, groups, codes, static_cast<uint16_t *>(scale), zero);
}

}  // namespace fp8lin
