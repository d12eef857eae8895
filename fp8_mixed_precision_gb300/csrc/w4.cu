// Products with 4-bit weights in groups along K, for few tokens:
//
//   W[n, k] = scale[n, k / group] (code[n, k] - zero[n, k / group])
//   linear  y = x W^T;   gated  h = act(x Wg^T) * (x Wu^T) with W = [Wg; Wu]
//
// for one weight, or for a stack of experts each with its own tokens.
//
// Bound by the weights' bytes: each is read once, by asynchronous copies into a
// ring that every warp has for itself.  A warp holds tiles of 16 weight rows
// against 8 NT tokens on mma.m16n8k16: code - zero is an integer of at most 15
// in magnitude, exact in bf16, so the products within a group are exact and
// their sum (fp32) is scaled once per group; no weight is ever rounded.  The
// codes of a 32-bit word are k .. k + 7; one and + or turns nibbles i and i + 4
// into the bf16 pair (128 + code), one packed subtraction takes 128 + zero off,
// and the tokens' values are paired to match (x_i, x_{i+4}).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8lin {
namespace {

constexpr int kW4Warps = 8, kW4Threads = 32 * kW4Warps;
constexpr int kStages = 3;
constexpr int kChunk = 256;              // codes of a row in a stage: 128 bytes
constexpr int kTileBytes = 16 * kChunk / 2;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kColStride = 20;           // floats from one token's partial sums to the next's

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes i and i + 4 of a word, as bf16, less zz = (128 + zero, 128 + zero).
__device__ __forceinline__ uint32_t codes_at(uint32_t w, int i, uint32_t zz) {
  const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&zz));
  return *reinterpret_cast<const uint32_t *>(&d);
}
__device__ __forceinline__ uint32_t lds32(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The tokens of block row y: expert, first row in the experts' order and count.
struct Tokens {
  int e, first, count;
};
__device__ __forceinline__ Tokens tokens_of(const W4Args &a, int y) {
  if (!a.experts) return {0, 0, a.T};
  const auto valid = [&](int e) { return e >= 0 && e < a.E; };
  if (!a.order) {  // one token: its slots are the rows
    const int e = a.experts[y];
    return valid(e) ? Tokens{e, y, 1} : Tokens{0, 0, 0};
  }
  int e = y;
  if (a.by_row) {  // fewer rows than experts: the first row of an expert stands for it
    if (y >= a.offsets[a.E]) return {0, 0, 0};
    e = a.experts[a.order[y]];
    if (a.offsets[e] != y) return {0, 0, 0};
  }
  return {e, a.offsets[e], a.counts[e]};
}

// TILES: tiles of 16 weight rows to a warp (gated: one of the gate, one of the
// up projection).  GROUP: weights to a scale.
template <int TILES, int NT, int GROUP>
__global__ void __launch_bounds__(kW4Threads) w4_kernel(const W4Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStage = TILES * kTileBytes;
  constexpr int kGroups = kChunk / GROUP;      // groups of a row in a chunk
  constexpr int kHeld = kGroups / 2;           // of a tile's 2 kGroups scales, those that a lane loads
  constexpr int kSteps = GROUP / 32;           // 32-deep steps to a group
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int kw = a.warps_k, wk = warp % kw, wr = warp / kw;
  uint8_t *ring = smem + warp * kStages * kStage;
  pdl_wait_then_release();
  const Tokens tk = tokens_of(a, blockIdx.y);
  if (tk.count == 0) return;
  const int tile = blockIdx.x * (kW4Warps / kw) + wr;  // of 16 TILES output rows (gated: 16)
  const int rows_out = a.gated ? 16 : 16 * TILES;
  const int n0 = tile * rows_out;
  const int64_t row_bytes = a.K / 2;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const bool live = n0 < a.N;
  // first weight row of each tile within the stack
  int64_t first[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    int r = a.gated ? i * a.N + n0 : n0 + 16 * i;
    if (r > a.rows - 16) r = a.rows - 16;  // a second tile past the last row: not stored
    first[i] = (int64_t)tk.e * a.rows + (live ? r : 0);
  }

  const auto request = [&](int c, int stage) {
    if (live && c < chunks) {
#pragma unroll
      for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (lane >> 3) + 4 * j, p = lane & 7;
          const bool in = c * kChunk + p * 32 < a.K;
          const uint8_t *src = a.codes + (first[i] + r) * row_bytes + (in ? c * (kChunk / 2) + p * 16 : 0);
          ptx::cp_async16_zfill(ring + stage * kStage + i * kTileBytes + r * 128 + ((p ^ (r & 7)) << 4), src,
                                in ? 16u : 0u);
        }
    }
    ptx::cp_async_commit();
  };
  // Of the scales of rows g and g + 8 (half h, group s of the chunk: number
  // h kGroups + s), lane q of a row's four holds those of number q modulo 4:
  // the scale in the upper, 128 + zero (bf16) in the lower 16 bits.
  const auto scales = [&](int c, uint32_t (&sz)[TILES][kHeld]) {
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int m = 0; m < kHeld; ++m) {
        const int id = q + 4 * m, h = id / kGroups, s = id % kGroups;
        const int at = min(c * kGroups + s, a.groups - 1);
        sz[i][m] = 0u;
        if (live && c < chunks) {
          const int64_t o = (first[i] + g + 8 * h) * a.groups + at;
          sz[i][m] = (uint32_t)a.scale[o] << 16 | 0x4300u | (a.zero ? a.zero[o] & 15u : 8u);
        }
      }
  };

  for (int tb = 0; tb < tk.count; tb += 8 * NT) {
    const uint16_t *xp[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int p = tk.first + tb + 8 * n + g;
      xp[n] = nullptr;
      if (tb + 8 * n + g < tk.count) {
        const int64_t row = a.tokens ? (a.order ? a.order[p] : p) / a.k : p;
        xp[n] = static_cast<const uint16_t *>(a.x) + row * a.K + 8 * q;
      }
    }
    float tot[TILES][NT][4] = {};
    uint32_t sz[TILES][kHeld];
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) request(wk + s * kw, s);
    scales(wk, sz);
    int stage = 0;
    for (int c = wk; c < chunks; c += kw) {
      cp_async_wait_group<kStages - 2>();
      __syncwarp();
      request(c + (kStages - 1) * kw, stage == 0 ? kStages - 1 : stage - 1);
      uint32_t next[TILES][kHeld];
      scales(c + kw, next);
      const uint8_t *base = ring + stage * kStage;
      if (live) {
#pragma unroll
        for (int s = 0; s < kGroups; ++s) {
          uint32_t lo[TILES], hi[TILES];  // rows g, g + 8: scale and zero of this group
#pragma unroll
          for (int i = 0; i < TILES; ++i) {
            lo[i] = __shfl_sync(kFull, sz[i][s / 4], s % 4, 4);
            hi[i] = __shfl_sync(kFull, sz[i][(kGroups + s) / 4], (kGroups + s) % 4, 4);
          }
          float acc[TILES][NT][4] = {};
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            const int step = s * kSteps + st;
            uint32_t b[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint4 v = make_uint4(0, 0, 0, 0);
              const int kk = c * kChunk + 32 * step;
              if (xp[n] && kk < a.K) v = *reinterpret_cast<const uint4 *>(xp[n] + kk);
              b[n][0] = __byte_perm(v.x, v.z, 0x5410);
              b[n][1] = __byte_perm(v.x, v.z, 0x7632);
              b[n][2] = __byte_perm(v.y, v.w, 0x5410);
              b[n][3] = __byte_perm(v.y, v.w, 0x7632);
            }
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
              const uint8_t *p = base + i * kTileBytes + g * 128 + ((step ^ g) << 4) + 4 * q;
              const uint32_t w0 = lds32(p), w1 = lds32(p + 8 * 128);
              const uint32_t z0 = __byte_perm(lo[i], 0, 0x1010), z1 = __byte_perm(hi[i], 0, 0x1010);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a0 = codes_at(w0, 2 * h, z0), a1 = codes_at(w1, 2 * h, z1);
                const uint32_t a2 = codes_at(w0, 2 * h + 1, z0), a3 = codes_at(w1, 2 * h + 1, z1);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16(acc[i][n], a0, a1, a2, a3, b[n][2 * h], b[n][2 * h + 1]);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < TILES; ++i) {
            const float s0 = bf16hi(lo[i]), s1 = bf16hi(hi[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              tot[i][n][0] = fmaf(acc[i][n][0], s0, tot[i][n][0]);
              tot[i][n][1] = fmaf(acc[i][n][1], s0, tot[i][n][1]);
              tot[i][n][2] = fmaf(acc[i][n][2], s1, tot[i][n][2]);
              tot[i][n][3] = fmaf(acc[i][n][3], s1, tot[i][n][3]);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int m = 0; m < kHeld; ++m) sz[i][m] = next[i][m];
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    cp_async_wait_group<0>();
    __syncwarp();
    // partial sums over K, [tile][token][row], in the warp's own ring
    float *mine = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          mine[(i * 8 * NT + 8 * n + 2 * q + (v & 1)) * kColStride + g + (v >> 1) * 8] = tot[i][n][v];
    __syncthreads();
    const int per = a.gated ? 16 : 16 * TILES;  // output rows of a tile
    for (int id = threadIdx.x; id < kW4Warps / kw * per * 8 * NT; id += kW4Threads) {
      const int r = id % per, n = id / per % (8 * NT), w0 = id / (per * 8 * NT) * kw;
      const int out = (blockIdx.x * (kW4Warps / kw) + id / (per * 8 * NT)) * per + r;
      if (tb + n >= tk.count || out >= a.N) continue;
      const float *from = reinterpret_cast<const float *>(smem + w0 * kStages * kStage);
      constexpr int kWarpFloats = kStages * kStage / 4;
      const auto sum = [&](int i) {
        float s = 0.0f;
        for (int w = 0; w < kw; ++w) s += from[w * kWarpFloats + (i * 8 * NT + n) * kColStride + (r & 15)];
        return s;
      };
      const int64_t o = (int64_t)(tk.first + tb + n) * a.N + out;
      if (a.gated) {
        const float gate = sum(0), up = sum(TILES - 1);
        float h;
        if (a.act == FP8_ACT_SILU) {
          const float t = expf(-fabsf(gate));  // no overflow on either side
          h = gate * __fdiv_rn(gate >= 0.0f ? 1.0f : t, 1.0f + t);
        } else {
          float unused;
          gelu_f2(gate, gate, h, unused);
        }
        static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(h * up);
      } else if (a.out_f32) {
        static_cast<float *>(a.out)[o] = sum(r >> 4);
      } else {
        static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(sum(r >> 4));
      }
    }
    __syncthreads();
  }
}

// y[t] = sum_j w[t, j] z[row of slot t k + j], z fp32.
__global__ void __launch_bounds__(256) w4_join_kernel(const float *__restrict__ z, const int *__restrict__ experts,
                                                      const int *__restrict__ position,
                                                      const float *__restrict__ weights, int64_t total, int vecs, int k,
                                                      int E, void *__restrict__ y) {
  pdl_wait_then_release();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t t = i / vecs;
  const int c = (int)(i - t * vecs);
  float4 s = make_float4(0, 0, 0, 0);
  for (int j = 0; j < k; ++j) {
    const int64_t slot = t * k + j;
    const int e = experts[slot];
    const float w = weights[slot];
    float4 v = make_float4(0, 0, 0, 0);
    if (e >= 0 && e < E) v = reinterpret_cast<const float4 *>(z)[(position ? position[slot] : slot) * vecs + c];
    s.x = fmaf(w, v.x, s.x);
    s.y = fmaf(w, v.y, s.y);
    s.z = fmaf(w, v.z, s.z);
    s.w = fmaf(w, v.w, s.w);
  }
  reinterpret_cast<uint2 *>(y)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// Codes, scales and zero points of bf16 weights, one warp per group:
//   without zero points  scale = bf16(max |w| / 7), code = 8 + round(w / scale) in 0..15
//   with                 scale = bf16((max - min) / 15) over the group and 0,
//                        zero = round(-min / scale) in 0..15, code = zero + round(w / scale) in 0..15
// A group of zeros has scale 1.
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
  if (!(fabsf(s) < INFINITY)) s = 3.0e38f;  // hi - lo past fp32's range
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

template <int TILES, int NT, int GROUP>
cudaError_t launch_w4(const W4Args &a, dim3 grid, cudaStream_t st) {
  constexpr size_t smem = (size_t)kW4Warps * kStages * TILES * kTileBytes;
  static_assert(TILES * 8 * NT * kColStride * 4 <= kStages * TILES * kTileBytes, "partial sums fit a warp's ring");
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(w4_kernel<TILES, NT, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  return launch_kernel(w4_kernel<TILES, NT, GROUP>, grid, dim3(kW4Threads), smem, st, a);
}
template <int TILES, int NT>
cudaError_t by_group(const W4Args &a, dim3 grid, cudaStream_t st) {
  if (a.group == 32) return launch_w4<TILES, NT, 32>(a, grid, st);
  if (a.group == 64) return launch_w4<TILES, NT, 64>(a, grid, st);
  return launch_w4<TILES, NT, 128>(a, grid, st);
}

}  // namespace

cudaError_t launch_w4_product(W4Args a, int lists, int likely, cudaStream_t st) {
  a.groups = (a.K + a.group - 1) / a.group;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  for (a.warps_k = kW4Warps; a.warps_k > chunks; a.warps_k /= 2) {
  }
  const int tiles = a.gated ? (a.N + 15) / 16 : (a.N + 31) / 32;
  const dim3 grid((unsigned)((tiles + kW4Warps / a.warps_k - 1) / (kW4Warps / a.warps_k)), (unsigned)lists);
  const double weights = (double)a.rows * a.K * (a.experts ? std::min(a.E, lists) : 1);
  LaunchScope ls(a.gated ? "w4_gated" : "w4_linear", st, weights * (0.5 + (a.zero ? 3.0 : 2.0) / a.group),
                 2.0 * a.rows * a.K * a.T, a.T, a.N, a.K);
  if (likely <= 8) return by_group<2, 1>(a, grid, st);
  if (likely <= 16) return by_group<2, 2>(a, grid, st);
  return by_group<2, 4>(a, grid, st);
}

cudaError_t launch_w4_join(const float *z, const int *experts, const int *position, const float *weights, int64_t T,
                           int64_t N, int k, int E, void *y, cudaStream_t st) {
  const int vecs = (int)(N / 4);
  LaunchScope ls("w4_join", st, 4.0 * T * N * k + 2.0 * T * N, 2.0 * T * N * k, T, N, k);
  return launch_kernel(w4_join_kernel, dim3((unsigned)((T * vecs + 255) / 256)), dim3(256), 0, st, z, experts, position,
                       weights, T * vecs, vecs, k, E, y);
}

cudaError_t launch_w4_quantize(const void *w, int64_t rows, int64_t K, int group, uint8_t *codes, void *scale,
                               uint8_t *zero, cudaStream_t st) {
  const int groups = (int)((K + group - 1) / group);
  LaunchScope ls("w4_quantize", st, rows * K * (2.5 + 2.0 / group), 0.0, rows, K);
  return launch_kernel(w4_quantize_kernel, dim3((unsigned)((rows * groups + 7) / 8)), dim3(256), 0, st, w, rows, (int)K,
                       group, groups, codes, static_cast<uint16_t *>(scale), zero);
}

}  // namespace fp8lin
