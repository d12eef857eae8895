// Root-mean-square norm of the residual stream, with the residual's addition
// and an E4M3 output in 1x128 blocks, and its backward pass.
//
//   r = bf16(x + residual)          (no residual: r = x)
//   rstd = 1 / sqrt(mean(r^2) + eps)
//   y = (r * rstd) * w              fp32, quantized without another rounding
//   backward, with g = dy * w and c = mean(g * r) over a row's C columns:
//     dx = dr + rstd * g - r * (rstd^3 * c)      (x and the residual share it)
//     dw = sum over rows of (dy * r) * rstd
//
// All arithmetic and sums are fp32; r and dx are rounded to bf16 once, as the
// framework keeps activations and gradients.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "pipe.cuh"
#include "ptx.cuh"

namespace fp8lin {
namespace {

__device__ unsigned g_norm_status;
constexpr int kNormThreads = 256;

// Norm weight: bf16 or fp32, eight consecutive values.
struct NormW {
  const void *w;
  int f32;
};
__device__ __forceinline__ void load_w8(const NormW &w, int64_t c, float (&v)[8]) {
  if (w.f32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w.w) + c);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w.w) + c));
    v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
    v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
  }
}
__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
  v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
// rstd is kept as a pair hi + lo (lo: what fp32 cannot hold of it), and
// y = r * (hi + lo) * w is rounded once: t + e is r * rstd to about 2^-45, and
// the last fma adds e * w to t * w exactly.  With rstd within 2^-43 (the sum of
// squares keeps its errors) both layouts quantize the correctly rounded fp32 y,
// all but about one in 2^18, so their scales and codes are those of the exact
// norm (none of 3 x 10^8 codes differs) and do not depend on the summation
// order.  Squares summed in fp32 four at a time left rstd at 2^-24: one scale
// in 15 and one code in 10^7 differed, in the same time.
__device__ __forceinline__ void norm8(uint4 r, float hi, float lo, const float (&w)[8],
                                      float (&y)[8]) {
  using namespace gelu2;
  float v[8];
  unpack8(r, v);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint64_t x = pk(v[k], v[k + 1]), ww = pk(w[k], w[k + 1]);
    const uint64_t t = mul2(x, dup(hi));
    const uint64_t e = fma2(x, dup(lo), fma2(x, dup(hi), mul2(t, dup(-1.0f))));
    upk(fma2(t, ww, mul2(e, ww)), y[k], y[k + 1]);
  }
}
// (a + b) as the rounded sum and its error.
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}
// 1 / sqrt((hi + lo) / C + eps) as a pair, from the hardware's approximate
// reciprocal square root (relative error below 2^-22) and one Newton step with
// its residual in full: what is left is below 2^-43.  inv_c: 1 / C as a pair.
// A sum that is not finite gives the root's own value and lo = 0.
__device__ __forceinline__ void rstd_pair(float hi, float lo, float C, float2 inv_c, float eps,
                                          float &r, float &rlo) {
  const float q = __fmul_rn(hi, inv_c.x);
  const float qlo = fmaf(__fadd_rn(fmaf(-q, C, hi), lo), inv_c.x, 0.0f);
  float m, mlo;
  two_sum(q, eps, m, mlo);
  mlo = __fadd_rn(mlo, qlo);
  const float r0 = rsqrtf(m);
  const float t = __fmul_rn(r0, r0), tlo = fmaf(r0, r0, -t);
  const float e = fmaf(-mlo, t, fmaf(-m, tlo, fmaf(-m, t, 1.0f)));
  // 1/sqrt(1 - e) = 1 + e/2 + 3/8 e^2 + ...
  const float d = __fmul_rn(r0, __fmul_rn(e, fmaf(0.375f, e, 0.5f)));
  r = __fadd_rn(r0, d);
  rlo = __fadd_rn(__fsub_rn(r0, r), d);
  if (!isfinite(rlo)) {
    r = r0;
    rlo = 0.0f;
  }
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Eight values -> eight E4M3 bytes (the hardware's conversion maps every NaN to
// 0x7F, the library's NaN byte, and infinities to the largest magnitude).
__device__ __forceinline__ uint2 cast8(const float (&v)[8]) {
  return make_uint2(cvt4_finite<FP8_FORMAT_E4M3>(v[0], v[1], v[2], v[3]),
                    cvt4_finite<FP8_FORMAT_E4M3>(v[4], v[5], v[6], v[7]));
}
// v * s, two products per instruction
__device__ __forceinline__ void scale8(const float (&v)[8], float s, float (&q)[8]) {
  using namespace gelu2;
#pragma unroll
  for (int k = 0; k < 8; k += 2) upk(mul2(pk(v[k], v[k + 1]), dup(s)), q[k], q[k + 1]);
}

struct NormFwd {
  const uint4 *x, *res;  // bf16 [R, C]; res may be null
  NormW w;
  int64_t R, C;
  float eps;
  float2 inv_c;  // 1 / C as a pair
  uint4 *r;      // bf16 [R, C]; written when res is given
  float *rstd, *rstd_lo;  // [R] or null
  uint4 *y;      // bf16 [R, C] or null
  uint8_t *row;  // E4M3 [R, C] or null
  float *row_scale, *row_scale_inv;
};

// Larger magnitude of each half of two bf16 pairs.
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) {
  const __nv_bfloat162 v = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&m),
                                   __habs2(*reinterpret_cast<__nv_bfloat162 *>(&w)));
  return *reinterpret_cast<const uint32_t *>(&v);
}
// bf16(x + res): the exact sum rounded once.
__device__ __forceinline__ uint4 add8(uint4 x, uint4 res) {
  auto add = [](uint32_t a, uint32_t b) {
    const __nv_bfloat162 s = __hadd2(*reinterpret_cast<__nv_bfloat162 *>(&a),
                                     *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&s);
  };
  return make_uint4(add(x.x, res.x), add(x.y, res.y), add(x.z, res.z), add(x.w, res.w));
}

// Rows: a group of WPR warps, or of LANES = 16 lanes of one, holds one row in
// registers (VPT vectors of 8 elements per thread), so x and the residual are
// read once and everything that the row alone determines is written from
// there; many small CTAs per SM hide the latency of the row sum.  Half a warp
// takes the rows of up to 512 columns: what is done once per row (joining the
// sum, the root, the scales' divisions) is then spread over twice the elements.
template <int VPT, int WPR, int LANES = 32>
__global__ void __launch_bounds__(WPR > 8 ? 32 * WPR : kNormThreads)
    rmsnorm_rows_kernel(NormFwd a) {
  static_assert(LANES == 32 || (LANES == 16 && WPR == 1), "half a warp per row");
  constexpr int kWarps = WPR > 8 ? WPR : kNormThreads / 32;
  constexpr int kRows = kWarps * 32 / (WPR * LANES);  // rows per CTA
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lir = lane % LANES;
  const int wir = warp % WPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / (WPR * LANES);
  const bool live = row < a.R;
  const int nv = (int)(a.C / 8);
  const int64_t base = row * nv;
  // vectors that hold columns of the row, whole groups at a time
  const int vecs = min(VPT, (nv - wir * LANES + WPR * LANES - 1) / (WPR * LANES));
  auto vec = [&](int j) { return (j * WPR + wir) * LANES + lir; };
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 rv[VPT], sv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const bool in = live && vec(j) < nv;
    rv[j] = in ? a.x[base + vec(j)] : zero;
    sv[j] = in && a.res ? a.res[base + vec(j)] : zero;
  }
  uint32_t most = 0;  // largest magnitude, bf16 pair
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (a.res) {
      rv[j] = add8(rv[j], sv[j]);
      if (live && vec(j) < nv) a.r[base + vec(j)] = rv[j];
    }
    most = absmax2(absmax2(absmax2(absmax2(most, rv[j].x), rv[j].y), rv[j].z), rv[j].w);
  }
  // Sums of the even and the odd columns, and their errors.  They start from the
  // largest square of the thread, so that each addition has the larger operand
  // in front: the part of a square that the sum takes up, and so the rest, is then
  // exact (the fma forms the 16 bits of the square without rounding).
  using namespace gelu2;
  const float top = fmaxf(bf16lo(most), bf16hi(most));
  const float start = top < 1e17f ? __fmul_rn(top, top) : 0.0f;  // not finite: as it comes
  uint64_t s2 = dup(start), l2 = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const uint32_t w4[4] = {rv[j].x, rv[j].y, rv[j].z, rv[j].w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint64_t x = pk(bf16lo(w4[h]), bf16hi(w4[h]));
      const uint64_t t = fma2(x, x, s2);
      l2 = fma2(fma2(x, x, fma2(t, dup(-1.0f), s2)), dup(1.0f), l2);
      s2 = t;
    }
  }
  float ss, lo;
  {
    float even, odd, le, lod, e0, e1, e2;
    upk(s2, even, odd);
    upk(l2, le, lod);
    two_sum(even, -start, even, e0);
    two_sum(odd, -start, odd, e1);
    two_sum(even, odd, ss, e2);
    lo = __fadd_rn(__fadd_rn(__fadd_rn(le, e0), __fadd_rn(lod, e1)), e2);
  }
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) {
    float e;
    const float other_lo = __shfl_xor_sync(0xffffffffu, lo, o);
    two_sum(ss, __shfl_xor_sync(0xffffffffu, ss, o), ss, e);
    lo = __fadd_rn(__fadd_rn(lo, other_lo), e);
  }
  if constexpr (WPR > 1) {
    __shared__ float2 red[kWarps];
    if (lane == 0) red[warp] = make_float2(ss, lo);
    __syncthreads();
    ss = lo = 0.0f;
#pragma unroll
    for (int k = 0; k < WPR; ++k) {
      const float2 v = red[warp / WPR * WPR + k];
      float e;
      two_sum(ss, v.x, ss, e);
      lo = __fadd_rn(__fadd_rn(lo, v.y), e);
    }
  }
  if (__all_sync(0xffffffffu, !live)) return;
  float rstd, rstd_lo;
  rstd_pair(ss, lo, (float)a.C, a.inv_c, a.eps, rstd, rstd_lo);
  if (live && wir == 0 && lir == 0) {
    if (a.rstd) a.rstd[row] = rstd;
    if (a.rstd_lo) a.rstd_lo[row] = rstd_lo;
  }
  const int64_t nb = (a.C + 127) / 128;
  float y[VPT][8], mx[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (j >= vecs) break;
    float w8[8] = {};
    if (vec(j) < nv) load_w8(a.w, (int64_t)vec(j) * 8, w8);
    norm8(rv[j], rstd, rstd_lo, w8, y[j]);
    if (a.y && live && vec(j) < nv) a.y[base + vec(j)] = pack8(y[j]);
    mx[j] = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx[j] = amax_acc(mx[j], y[j][k]);
  }
  if (!a.row) return;
  // the block scales of the thread's vectors: lane j of each half warp divides
  // for vector j, and the others take the result from it
  float m = 0.0f, s, si;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (j >= vecs) break;
#pragma unroll
    for (int o = 8; o; o >>= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
    if ((lane & 15) == j) m = mx[j];
  }
  scale_from_amax(m, kE4M3Max, s, si);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (j >= vecs) break;
    const int v = vec(j);
    const float sj = __shfl_sync(0xffffffffu, s, (lane & 16) + j);
    if (live && v < nv) {
      float q8[8];
      scale8(y[j], sj, q8);
      *reinterpret_cast<uint2 *>(a.row + row * a.C + (int64_t)v * 8) = cast8(q8);
    }
    if (live && (lane & 15) == j && v - j < nv) {  // v - j: the block's first vector
      a.row_scale[row * nb + v / 16] = s;
      a.row_scale_inv[row * nb + v / 16] = si;
    }
  }
}

struct NormCols {
  NormW w;
  int64_t R, C, ldr;  // ldr: tokens per row of the transposed layout (R rounded up to 16)
  const float *rstd, *rstd_lo;
  uint8_t *col;  // E4M3 [C, ldr]
  float *col_scale, *col_scale_inv;
};

// Tile of the transposing pass: 128 tokens x 64 columns per CTA of 4 warps.
constexpr int kColThreads = 128, kColTile = 64;
struct __align__(128) CSmem {
  uint16_t in[2][128 * kColTile];
  uint32_t tile[128 * kColTile / 4 + 32];  // FP8 bytes, 4 words of padding per 16 rows
  float colred[4][kColTile];
  float colsc[kColTile];
  float2 rs[128];
  uint64_t full[2];
  int abort;
};

// Word w (4 columns) of tile row r.  The padding puts the transpose's lanes (8
// groups of 16 rows, 4 words) on 32 different banks.
__device__ __forceinline__ int tile_word(int r, int w) {
  return r * (kColTile / 4) + (r >> 4) * 4 + w;
}

// Transposed copy: 128 tokens x 64 columns per iteration.  r comes back by
// TMA, y is formed again from r, rstd and w, each column's maximum over its
// 128 tokens gives its scale, and the bytes go through a padded tile so that
// 16 tokens leave in one store.  Tokens past R are zeros.  Tiles run last to
// first: the end of r is what L2 still holds after the row pass.  What bounds
// it is the instructions between a tile's barriers, so CTAs are small (4 warps,
// four CTAs per SM).
__global__ void __launch_bounds__(kColThreads, 4)
    rmsnorm_cols_kernel(const __grid_constant__ CUtensorMap tmr, NormCols p) {
  extern __shared__ __align__(1024) uint8_t n_smem_raw[];
  CSmem &S = *reinterpret_cast<CSmem *>(n_smem_raw);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int cg = t & 7, rr = t >> 3;  // 8 columns, rows rr + 16 i
  const int64_t tiles_r = (p.R + 127) / 128, tiles_c = (p.C + kColTile - 1) / kColTile;
  const int64_t ntiles = tiles_r * tiles_c;
  if (t == 0) {
    ptx::mbar_init(&S.full[0], 1);
    ptx::mbar_init(&S.full[1], 1);
    S.abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tmr);
  }
  __syncthreads();
  pdl_wait_then_release();
  auto prefetch = [&](int64_t id, int b) {
    if (t != 0 || id >= ntiles) return;
    const int64_t tr = (ntiles - 1 - id) / tiles_c, tc = (ntiles - 1 - id) % tiles_c;
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive_expect_tx(&S.full[b], 128u * kColTile * 2);
    ptx::tma_load_2d(S.in[b], &tmr, &S.full[b], (int)(tc * kColTile), (int)(tr * 128));
  };
  int64_t id = blockIdx.x;
  volatile int *abort = &S.abort;
  prefetch(id, 0);
  prefetch(id + gridDim.x, 1);
  for (int k = 0; id < ntiles; ++k, id += gridDim.x) {
    const int b = k & 1;
    const int64_t tr = (ntiles - 1 - id) / tiles_c, tc = (ntiles - 1 - id) % tiles_c;
    const int64_t r0 = tr * 128, c0 = tc * kColTile;
    const int rows_here = (int)(p.R - r0 < 128 ? p.R - r0 : 128);
    const int cols_here = (int)(p.C - c0 < kColTile ? p.C - c0 : kColTile);
    float w8[8] = {};
    if (8 * cg < cols_here) load_w8(p.w, c0 + 8 * cg, w8);
    S.rs[t] = t < rows_here ? make_float2(p.rstd[r0 + t], p.rstd_lo[r0 + t]) : make_float2(0.0f, 0.0f);
    pipe::wait_bar(&S.full[b], (k >> 1) & 1, abort, &g_norm_status);
    __syncthreads();
    const bool gave_up = *abort;  // the same for every thread
    float y[8][8];  // rows rr + 16 i; tokens past R: zeros
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rr + 16 * i;
      const float2 rs = S.rs[r];
      norm8(*reinterpret_cast<const uint4 *>(&S.in[b][r * kColTile + 8 * cg]), rs.x, rs.y, w8, y[i]);
      if (r >= rows_here)
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = 0.0f;
    }
    float cm[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) cm[j] = amax_acc(cm[j], y[i][j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cm[j] = fmaxf(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 8));
      cm[j] = fmaxf(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
    }
    if (lane < 8) {
      float4 *dst = reinterpret_cast<float4 *>(&S.colred[warp][8 * cg]);
      dst[0] = make_float4(cm[0], cm[1], cm[2], cm[3]);
      dst[1] = make_float4(cm[4], cm[5], cm[6], cm[7]);
    }
    __syncthreads();
    if (gave_up) {  // what was asked for lands before the CTA leaves
      if (t == 0) {
        pipe::drain_wait(&S.full[b], (k >> 1) & 1, &g_norm_status);
        if (id + gridDim.x < ntiles)
          pipe::drain_wait(&S.full[b ^ 1], ((k + 1) >> 1) & 1, &g_norm_status);
      }
      return;
    }
    prefetch(id + 2 * (int64_t)gridDim.x, b);  // every thread holds its elements
    if (t < kColTile) {
      const float m = fmaxf(fmaxf(S.colred[0][t], S.colred[1][t]),
                            fmaxf(S.colred[2][t], S.colred[3][t]));
      float s, si;
      scale_from_amax(m, kE4M3Max, s, si);
      S.colsc[t] = s;
      if (t < cols_here) {
        p.col_scale[(c0 + t) * tiles_r + tr] = s;
        p.col_scale_inv[(c0 + t) * tiles_r + tr] = si;
      }
    }
    __syncthreads();
    float cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = S.colsc[8 * cg + j];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      using namespace gelu2;
      float q8[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        upk(mul2(pk(y[i][j], y[i][j + 1]), pk(cs[j], cs[j + 1])), q8[j], q8[j + 1]);
      *reinterpret_cast<uint2 *>(&S.tile[tile_word(rr + 16 * i, 2 * cg)]) = cast8(q8);
    }
    __syncthreads();
    const int seg = t & 7, w = t >> 3;  // rows seg*16..+15, columns 4w..4w+3
    if (4 * w < cols_here && 16 * seg < rows_here) {
      uint32_t a[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i] = S.tile[tile_word(seg * 16 + i, w)];
      uint32_t o[4][4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t t0 = __byte_perm(a[4 * g + 0], a[4 * g + 1], 0x5140);
        const uint32_t t1 = __byte_perm(a[4 * g + 0], a[4 * g + 1], 0x7362);
        const uint32_t t2 = __byte_perm(a[4 * g + 2], a[4 * g + 3], 0x5140);
        const uint32_t t3 = __byte_perm(a[4 * g + 2], a[4 * g + 3], 0x7362);
        o[0][g] = __byte_perm(t0, t2, 0x5410);
        o[1][g] = __byte_perm(t0, t2, 0x7632);
        o[2][g] = __byte_perm(t1, t3, 0x5410);
        o[3][g] = __byte_perm(t1, t3, 0x7632);
      }
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
        *reinterpret_cast<uint4 *>(p.col + (c0 + 4 * w + jj) * p.ldr + r0 + 16 * seg) =
            make_uint4(o[jj][0], o[jj][1], o[jj][2], o[jj][3]);
    }
  }
}

struct NormBwd {
  const uint4 *dy, *dr, *r;  // bf16 [R, C]; dr may be null
  const float *rstd;
  NormW w;
  int64_t R, C;
  uint4 *dx;        // bf16 [R, C]
  float *partials;  // [gridDim.x, C] sums of this CTA's rows
};

// One producer thread per CTA streams whole groups of rows (contiguous in
// memory) of the three inputs into a shared-memory ring with bulk copies, so
// the bytes in flight do not depend on how far the warps have come.
constexpr int kRingStages = 8;
struct RingCtl {
  uint64_t full[kRingStages], empty[kRingStages];
  int abort;
};
constexpr int kRingCtlBytes = (int)((sizeof(RingCtl) + 127) / 128 * 128);

// Warps per CTA that work on rows, for WPR warps per row; the producer is one more.
constexpr int ring_warps(int wpr) { return wpr > 8 ? wpr : 8; }

// The producer's loop: stages of `group` rows (row_bytes each) of the tensors
// in[0 .. NIN - 1] (null ones are skipped).
template <int NIN>
__device__ __forceinline__ void ring_produce(RingCtl *ctl, uint8_t *ring, int stages, int group,
                                             int64_t R, int64_t row_bytes,
                                             const void *const (&in)[NIN]) {
  volatile int *abort = &ctl->abort;
  int issued = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * group; row0 < R; row0 += (int64_t)gridDim.x * group) {
    const int s = issued % stages;
    if (!pipe::wait_bar(&ctl->empty[s], ((issued / stages) & 1) ^ 1, abort, &g_norm_status)) break;
    const int64_t rows = R - row0 < group ? R - row0 : group;
    const uint32_t bytes = (uint32_t)(rows * row_bytes);
    uint32_t all = 0;
#pragma unroll
    for (int k = 0; k < NIN; ++k) all += in[k] ? bytes : 0;
    ptx::mbar_arrive_expect_tx(&ctl->full[s], all);
    uint8_t *dst = ring + (int64_t)s * NIN * group * row_bytes;
#pragma unroll
    for (int k = 0; k < NIN; ++k)
      if (in[k])
        ptx::bulk_load(dst + k * group * row_bytes,
                       static_cast<const uint8_t *>(in[k]) + row0 * row_bytes, bytes, &ctl->full[s]);
    ++issued;
  }
  // the last copies land before the CTA can exit, also if the warps gave up on one
  for (int i = max(0, issued - stages); i < issued; ++i)
    pipe::drain_wait(&ctl->full[i % stages], (uint32_t)((i / stages) & 1), &g_norm_status);
}
__device__ __forceinline__ void ring_init(RingCtl *ctl, int stages, int warps) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&ctl->full[s], 1);
      ptx::mbar_init(&ctl->empty[s], warps);
    }
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
}
// Joins the WPR warps of group grp (whole CTA rows: barrier 1 + grp).
template <int WPR>
__device__ __forceinline__ void group_sync(int grp) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * WPR) : "memory");
}

// Backward: a group of WPR warps per row, fed by the ring; each thread keeps
// the dw sums of its own columns over all rows of its group.  A row is read
// from shared memory twice (for c, then for dx) instead of being held.
template <int VPT, int WPR>
__global__ void __launch_bounds__(32 * (ring_warps(WPR) + 1), WPR > 8 ? 1 : 3)
    rmsnorm_bwd_kernel(NormBwd a, int stages) {
  constexpr int kWarps = ring_warps(WPR), kGroup = kWarps / WPR;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  RingCtl *ctl = reinterpret_cast<RingCtl *>(ring_smem);
  uint8_t *ring = ring_smem + kRingCtlBytes;
  __shared__ float red[2][kWarps];
  ring_init(ctl, stages, kWarps);
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row_bytes = a.C * 2;
  const int wir = warp % WPR, grp = warp / WPR;
  const int nv = (int)(a.C / 8);
  float dw[VPT][8] = {};
  if (warp == kWarps) {
    const void *const in[3] = {a.dy, a.r, a.dr};
    if (lane == 0) ring_produce<3>(ctl, ring, stages, kGroup, a.R, row_bytes, in);
  } else {
    const float inv_c = __fdiv_rn(1.0f, (float)a.C);
    int it = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * kGroup; row0 < a.R;
         row0 += (int64_t)gridDim.x * kGroup, ++it) {
      const int s = it % stages;
      const int64_t row = row0 + grp;
      const bool live = row < a.R;
      const float rstd = live ? a.rstd[row] : 0.0f;
      pipe::wait_bar(&ctl->full[s], (it / stages) & 1, &ctl->abort, &g_norm_status);
      const uint4 *pd = reinterpret_cast<const uint4 *>(ring + (int64_t)s * 3 * kGroup * row_bytes +
                                                        grp * row_bytes);
      const uint4 *pr = pd + kGroup * nv, *pe = pr + kGroup * nv;
      float c = 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = (j * WPR + wir) * 32 + lane;
        if (live && v < nv) {
          float w8[8], d[8], r[8];
          load_w8(a.w, (int64_t)v * 8, w8);
          unpack8(pd[v], d);
          unpack8(pr[v], r);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float dr = d[k] * r[k];
            c = fmaf(dr, w8[k], c);
            dw[j][k] = fmaf(dr, rstd, dw[j][k]);
          }
        }
      }
      c = warp_sum(c);
      if constexpr (WPR > 1) {
        if (lane == 0) red[it & 1][warp] = c;
        group_sync<WPR>(grp);
        c = 0.0f;
#pragma unroll
        for (int k = 0; k < WPR; ++k) c += red[it & 1][grp * WPR + k];
      }
      const float c3 = c * inv_c * rstd * rstd * rstd;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = (j * WPR + wir) * 32 + lane;
        if (live && v < nv) {
          float w8[8], d[8], r[8], e[8] = {};
          load_w8(a.w, (int64_t)v * 8, w8);
          unpack8(pd[v], d);
          unpack8(pr[v], r);
          if (a.dr) unpack8(pe[v], e);
#pragma unroll
          for (int k = 0; k < 8; ++k) e[k] = fmaf(-r[k], c3, fmaf(d[k] * w8[k], rstd, e[k]));
          a.dx[row * nv + v] = pack8(e);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl->empty[s]);
    }
  }
  // this CTA's column sums: the groups in order, through the idle ring
  float *sums = reinterpret_cast<float *>(ring);  // [kGroup - 1][C]
  __syncthreads();
  if (kGroup > 1 && warp < kWarps && grp > 0)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = (j * WPR + wir) * 32 + lane;
      if (v < nv)
#pragma unroll
        for (int k = 0; k < 8; ++k) sums[(int64_t)(grp - 1) * a.C + v * 8 + k] = dw[j][k];
    }
  __syncthreads();
  if (grp == 0)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = (j * WPR + wir) * 32 + lane;
      if (v < nv) {
        for (int g = 1; g < kGroup; ++g)
#pragma unroll
          for (int k = 0; k < 8; ++k) dw[j][k] += sums[(int64_t)(g - 1) * a.C + v * 8 + k];
        float4 *dst = reinterpret_cast<float4 *>(a.partials + (int64_t)blockIdx.x * a.C + v * 8);
        dst[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        dst[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
      }
    }
}

// dw[c] = sum of the CTAs' partials in a fixed order: 16 columns (4 lanes of
// four) x 128 parts of the CTAs per block, the parts joined in order.
__global__ void __launch_bounds__(512) rmsnorm_dw_kernel(const float *__restrict__ partials, int n,
                                                         int64_t C, float *__restrict__ dw) {
  pdl_wait_then_release();
  __shared__ float4 part[128][4];
  const int quad = threadIdx.x & 3, k0 = threadIdx.x >> 2;
  const int64_t c = (int64_t)blockIdx.x * 16 + quad * 4;  // C is a multiple of 16
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [](float4 &s, float4 v) {
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  };
#pragma unroll 5
  for (int k = k0; k < n; k += 128)
    add(s, *reinterpret_cast<const float4 *>(partials + (int64_t)k * C + c));
  part[k0][quad] = s;
  __syncthreads();
#pragma unroll
  for (int d = 64; d; d >>= 1) {  // pairwise, in a fixed order
    if (k0 < d) {
      add(s, part[k0 + d][quad]);
      part[k0][quad] = s;
    }
    __syncthreads();
  }
  if (k0 == 0) *reinterpret_cast<float4 *>(dw + c) = s;
}

// Warps per row at VPT vectors per thread: a power of two that covers C.
int bwd_vpt(int64_t C) { return C > 8192 ? 4 : 2; }
int row_warps(int64_t C, int vpt) {
  int wpr = 1;
  while ((int64_t)wpr * 256 * vpt < C) wpr *= 2;
  return wpr;
}

template <typename Kernel>
cudaError_t opt_in_smem(Kernel kernel, size_t bytes, std::atomic<bool> *done) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}
// Shared memory of a ring kernel's CTA: three CTAs per SM, one with 16 warps a row.
template <int WPR>
constexpr int kRingSmem = WPR > 8 ? 208 * 1024 : 72 * 1024;
// Stages that fit, for groups of `group` rows of `tensors` tensors.
int ring_stages(int smem, int group, int64_t C, int tensors) {
  return (int)std::min<int64_t>(kRingStages, (smem - kRingCtlBytes) / (group * C * 2 * tensors));
}

template <int VPT, int WPR, int LANES = 32>
cudaError_t launch_rows(const NormFwd &a, cudaStream_t st) {
  constexpr int kThreads = WPR > 8 ? 32 * WPR : kNormThreads;
  constexpr int kRows = kThreads / (WPR * LANES);
  return launch_kernel(rmsnorm_rows_kernel<VPT, WPR, LANES>,
                       dim3((unsigned)((a.R + kRows - 1) / kRows)), dim3(kThreads), 0, st, a);
}

template <int VPT, int WPR>
cudaError_t launch_bwd(NormBwd a, int grid, cudaStream_t st) {
  constexpr int kWarps = ring_warps(WPR);
  static std::atomic<bool> done[64];
  const cudaError_t e = opt_in_smem(rmsnorm_bwd_kernel<VPT, WPR>, kRingSmem<WPR>, done);
  if (e != cudaSuccess) return e;
  const int stages = ring_stages(kRingSmem<WPR>, kWarps / WPR, a.C, 3);
  return launch_kernel(rmsnorm_bwd_kernel<VPT, WPR>, dim3((unsigned)grid), dim3(32 * (kWarps + 1)),
                       kRingSmem<WPR>, st, a, stages);
}

}  // namespace

// CTAs of the backward pass (one wave): a function of the shape alone, so that
// the order of the dw sums is too.
int norm_bwd_ctas(int64_t rows, int64_t cols) {
  const int wpr = row_warps(cols, bwd_vpt(cols));
  const int64_t group = ring_warps(wpr) / wpr, most = wpr > 8 ? 152 : 456;
  return (int)std::max<int64_t>(1, std::min<int64_t>((rows + group - 1) / group, most));
}

cudaError_t launch_rmsnorm_rows(const void *x, const void *res, const void *w, int w_f32,
                                int64_t rows, int64_t cols, float eps, void *r, float *rstd,
                                float *rstd_lo, void *y, uint8_t *row, float *row_scale,
                                float *row_scale_inv, cudaStream_t st) {
  const float inv = (float)(1.0 / (double)cols);
  NormFwd a{static_cast<const uint4 *>(x), static_cast<const uint4 *>(res), {w, w_f32}, rows, cols,
            eps, make_float2(inv, (float)(1.0 / (double)cols - (double)inv)),
            static_cast<uint4 *>(r), rstd, rstd_lo, static_cast<uint4 *>(y), row, row_scale,
            row_scale_inv};
  const double n = (double)rows * cols;
  LaunchScope ls("rmsnorm_rows", st,
                 n * (2 + (res ? 4 : 0) + (y ? 2 : 0) + (row ? 1 : 0)) +
                     rows * 8.0 * ((cols + 127) / 128),
                 4 * n, rows, cols);
  if (cols <= 256) return launch_rows<2, 1, 16>(a, st);
  if (cols <= 512) return launch_rows<4, 1, 16>(a, st);
  switch (row_warps(cols, 4)) {  // up to kMaxNormCols
    case 1: return launch_rows<4, 1>(a, st);
    case 2: return launch_rows<4, 2>(a, st);
    case 4: return launch_rows<4, 4>(a, st);
    case 8: return launch_rows<4, 8>(a, st);
    default: return launch_rows<4, 16>(a, st);
  }
}

cudaError_t launch_rmsnorm_cols(const void *r, const float *rstd, const float *rstd_lo,
                                const void *w, int w_f32, int64_t rows, int64_t cols, uint8_t *col, float *col_scale,
                                float *col_scale_inv, cudaStream_t st) {
  CUtensorMap tm;
  if (!make_bf16_tile_map(&tm, r, rows, cols, 128, kColTile)) return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        rmsnorm_cols_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(CSmem));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  NormCols p{{w, w_f32}, rows, cols, (rows + 15) / 16 * 16, rstd, rstd_lo, col, col_scale, col_scale_inv};
  const int64_t tiles = ((rows + 127) / 128) * ((cols + kColTile - 1) / kColTile);
  const int64_t grid = std::min<int64_t>(tiles, (int64_t)num_sms() * 4);
  LaunchScope ls("rmsnorm_cols", st,
                 3.0 * rows * cols + 4.0 * rows + 8.0 * cols * ((rows + 127) / 128),
                 2.0 * rows * cols, rows, cols);
  return launch_kernel(rmsnorm_cols_kernel, dim3((unsigned)grid), dim3(kColThreads),
                       sizeof(CSmem), st, tm, p);
}

cudaError_t launch_rmsnorm_bwd(const void *dy, const void *dr, const void *r, const float *rstd,
                               const void *w, int w_f32, int64_t rows, int64_t cols, void *dx,
                               float *dw, float *partials, cudaStream_t st) {
  NormBwd a{static_cast<const uint4 *>(dy), static_cast<const uint4 *>(dr),
            static_cast<const uint4 *>(r), rstd, {w, w_f32}, rows, cols, static_cast<uint4 *>(dx),
            partials};
  const int grid = norm_bwd_ctas(rows, cols);
  {
    LaunchScope ls("rmsnorm_bwd", st, (dr ? 8.0 : 6.0) * rows * cols + 4.0 * rows,
                   8.0 * rows * cols, rows, cols);
    cudaError_t e;
    const int wpr = row_warps(cols, bwd_vpt(cols));
    if (bwd_vpt(cols) == 4) e = launch_bwd<4, 16>(a, grid, st);
    else if (wpr == 1) e = launch_bwd<2, 1>(a, grid, st);
    else if (wpr == 2) e = launch_bwd<2, 2>(a, grid, st);
    else if (wpr == 4) e = launch_bwd<2, 4>(a, grid, st);
    else if (wpr == 8) e = launch_bwd<2, 8>(a, grid, st);
    else e = launch_bwd<2, 16>(a, grid, st);
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls("rmsnorm_dw", st, 4.0 * grid * cols + 4.0 * cols, (double)grid * cols, grid, cols);
  // a plain launch: overlapped with the pass before it, a forward and backward
  // at 16379 x 4096 took 237 us instead of 220
  return launch_kernel_as(false, rmsnorm_dw_kernel, dim3((unsigned)(cols / 16)), dim3(512), 0, st,
                       (const float *)partials, grid, cols, dw);
}

cudaError_t norm_read_status(unsigned *status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_norm_status, sizeof(unsigned));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_norm_status, &zero, sizeof(unsigned));
}

}  // namespace fp8lin
