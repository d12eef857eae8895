// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over all tensors of g^2)
//   coef = min(1, max_norm / (norm + 1e-6)), or 1 when the norm is not finite
//   out  = g * coef
//
// The tensors are cut into chunks of at most `chunk` elements; a table of
// chunks in device memory (pointer, pointer, count, type) lets one launch
// cover tensors of any number and size.  Bound by memory: the first pass reads
// every gradient once, the second reads it again (from L2 where it still is)
// and writes it once; a set of few chunks takes one kernel that does both.  Sums
// are fp32 within a thread's part of a chunk, pairs of fp32 over its chunks, fp32
// within a CTA and pairs over the CTAs, in an order that depends on the table and
// the GPU alone.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace fp8lin {
namespace {

constexpr int kClipThreads = 512;

__device__ __forceinline__ bool vec_ok(const ClipChunk &c) {
  return ((reinterpret_cast<uintptr_t>(c.src) | reinterpret_cast<uintptr_t>(c.dst)) & 15) == 0;
}
__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
  v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}
__device__ __forceinline__ float load1(const ClipChunk &c, int i) {
  return c.f32 ? static_cast<const float *>(c.src)[i]
               : bf16lo(static_cast<const uint16_t *>(c.src)[i]);
}

// Squares of a vector's elements, into four sums.
__device__ __forceinline__ void add_squares(uint4 w, int f32, float (&a)[4]) {
  if (f32) {
    const float x = __uint_as_float(w.x), y = __uint_as_float(w.y);
    const float z = __uint_as_float(w.z), q = __uint_as_float(w.w);
    a[0] = fmaf(x, x, a[0]);
    a[1] = fmaf(y, y, a[1]);
    a[2] = fmaf(z, z, a[2]);
    a[3] = fmaf(q, q, a[3]);
  } else {
    float v[8];
    unpack8(w, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k & 3] = fmaf(v[k], v[k], a[k & 3]);
  }
}
// A vector's elements times coef.
__device__ __forceinline__ uint4 scaled(uint4 w, int f32, float coef) {
  if (coef == 1.0f) return w;
  if (f32)
    return make_uint4(__float_as_uint(__fmul_rn(__uint_as_float(w.x), coef)),
                      __float_as_uint(__fmul_rn(__uint_as_float(w.y), coef)),
                      __float_as_uint(__fmul_rn(__uint_as_float(w.z), coef)),
                      __float_as_uint(__fmul_rn(__uint_as_float(w.w), coef)));
  float v[8];
  unpack8(w, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], coef);
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// One element of a chunk times coef.
__device__ __forceinline__ void store1(const ClipChunk &c, int i, float coef) {
  float v = load1(c, i);
  if (coef != 1.0f) v = __fmul_rn(v, coef);
  if (c.f32)
    static_cast<float *>(c.dst)[i] = v;
  else
    static_cast<__nv_bfloat16 *>(c.dst)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ float clip_coef(float norm, float max_norm) {
  return isfinite(norm) ? fminf(1.0f, __fdiv_rn(max_norm, norm + 1e-6f)) : 1.0f;
}

// A sum as an unevaluated pair of fp32 (about 48 bits): this GPU's fp64 rate is
// so low that forming the norm in it took 1.2 us longer.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const float s = __fadd_rn(a.hi, b.hi);
  const float z = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, z)), __fsub_rn(b.hi, z));
  // an infinite sum stays one (its error term would be a NaN)
  return {s, isfinite(s) ? __fadd_rn(e, __fadd_rn(a.lo, b.lo)) : 0.0f};
}

// Sum over the CTA's 512 threads, in a fixed order; thread 0 has the result.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float red[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  if (threadIdx.x == 0)
    for (int k = 0; k < kClipThreads / 32; ++k) v += red[k];
  return v;
}

// The first kAhead vectors per thread of a chunk, requested before they are
// needed (a chunk off the 16-byte grid has none).
constexpr int kAhead = 8;
__device__ __forceinline__ int vectors_of(const ClipChunk &c) {
  return vec_ok(c) ? c.n / (c.f32 ? 4 : 8) : 0;
}
__device__ __forceinline__ void request(const ClipChunk &c, int nv, uint4 (&w)[kAhead],
                                        int from = 0) {
  const uint4 *p = static_cast<const uint4 *>(c.src);
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = from + threadIdx.x + k * kClipThreads;
    w[k] = i < nv ? p[i] : make_uint4(0, 0, 0, 0);
  }
}

__global__ void __launch_bounds__(kClipThreads, 2) clip_norm_kernel(const ClipChunk *__restrict__ table,
                                                                    int64_t chunks,
                                                                    float *__restrict__ partials) {
  pdl_wait_then_release();
  Pair sum = {0.0f, 0.0f};
  int64_t id = blockIdx.x;
  ClipChunk c = {};
  if (id < chunks) c = table[id];
  while (id < chunks) {
    const int nv = vectors_of(c);
    float a[4] = {};
    uint4 w[kAhead];
    request(c, nv, w);
    const ClipChunk now = c;
    id += gridDim.x;
    if (id < chunks) c = table[id];  // arrives while this chunk is worked on
#pragma unroll
    for (int k = 0; k < kAhead; ++k) add_squares(w[k], now.f32, a);
    for (int from = kAhead * kClipThreads; from < nv; from += kAhead * kClipThreads) {
      request(now, nv, w, from);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) add_squares(w[k], now.f32, a);
    }
    for (int e = nv * (now.f32 ? 4 : 8) + threadIdx.x; e < now.n; e += kClipThreads) {
      const float v = load1(now, e);
      a[0] = fmaf(v, v, a[0]);
    }
    // closed here, so that no chain is longer than a chunk's, however large the set
    // (2^31 equal values, one chain: the norm 430 units of roundoff off)
    sum = add(sum, Pair{(a[0] + a[1]) + (a[2] + a[3]), 0.0f});
  }
  const float s = block_sum(__fadd_rn(sum.hi, sum.lo));
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// Every warp forms the norm from the partials, in the same order.
__device__ __forceinline__ float norm_of(const float *partials, int n) {
  __shared__ Pair red[kClipThreads / 32];
  const int lane = threadIdx.x & 31;
  auto across = [](Pair s, int from) {
    for (int o = from; o; o >>= 1)
      s = add(s, Pair{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    return s;
  };
  Pair s = {0.0f, 0.0f};
  for (int k = threadIdx.x; k < n; k += kClipThreads) s = add(s, Pair{partials[k], 0.0f});
  s = across(s, 16);
  if (lane == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = across(red[lane & (kClipThreads / 32 - 1)], kClipThreads / 64);
  return __fsqrt_rn(__fadd_rn(s.hi, s.lo));
}

__global__ void __launch_bounds__(kClipThreads, 2) clip_scale_kernel(const ClipChunk *__restrict__ table,
                                                                  int64_t chunks,
                                                                  const float *__restrict__ partials,
                                                                  int n_partials, float max_norm,
                                                                  float *__restrict__ norm_out) {
  pdl_wait_then_release();
  // last chunk first: what the first pass read last may still be in L2; the
  // first vectors are on their way while the norm is formed
  int64_t id = blockIdx.x;
  ClipChunk c = {};
  uint4 w[kAhead];
  if (id < chunks) c = table[chunks - 1 - id];
  request(c, vectors_of(c), w);
  const float norm = norm_of(partials, n_partials);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float coef = clip_coef(norm, max_norm);
  while (id < chunks) {
    const int nv = vectors_of(c);
    const ClipChunk now = c;
    id += gridDim.x;
    if (id < chunks) c = table[chunks - 1 - id];
    if (now.dst != now.src || coef != 1.0f) {  // in place, a factor of 1 changes nothing
      uint4 *q = static_cast<uint4 *>(now.dst);
      for (int from = 0; from < nv; from += kAhead * kClipThreads) {
        if (from) request(now, nv, w, from);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = from + threadIdx.x + k * kClipThreads;
          if (i < nv) q[i] = scaled(w[k], now.f32, coef);
        }
      }
      for (int e = nv * (now.f32 ? 4 : 8) + threadIdx.x; e < now.n; e += kClipThreads)
        store1(now, e, coef);
    }
    if (id < chunks) request(c, vectors_of(c), w);
  }
}

// Few chunks (kClipFewChunks of kClipFewElements at most): one CTA does both
// passes in one launch, 64 threads to a chunk, the gradients staying in registers
// in between.  Bound by the launch and the round trips to memory: 9 vectors of
// 515 floats take 3.6 us a library call (2.7 in a graph), as the two kernels 5.2
// (4.0); 16 full chunks 4.6 (4.4) against 5.2 (4.0).  A cluster of eight CTAs joined over
// distributed shared memory: 5.5.
constexpr int kFewThreads = 1024, kFewGroup = kFewThreads / kClipFewChunks;
static_assert(kClipFewElements / 4 == kAhead * kFewGroup, "a chunk's vectors fit its threads' registers");
static_assert(kFewThreads == 32 * 32, "one lane per warp's sum");

__global__ void __launch_bounds__(kFewThreads) clip_few_kernel(const ClipChunk *__restrict__ table,
                                                               int chunks, int write, float max_norm,
                                                               float *__restrict__ norm_out) {
  __shared__ float red[kFewThreads / 32];
  pdl_wait_then_release();
  const int t = threadIdx.x, g = t / kFewGroup, l = t % kFewGroup;
  ClipChunk c = {};
  if (g < chunks) c = table[g];
  const int nv = vectors_of(c), e0 = nv * (c.f32 ? 4 : 8) + l;
  uint4 w[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = l + k * kFewGroup;
    w[k] = i < nv ? static_cast<const uint4 *>(c.src)[i] : make_uint4(0, 0, 0, 0);
  }
  float a[4] = {};
  for (int e = e0; e < c.n; e += kFewGroup) {
    const float v = load1(c, e);
    a[0] = fmaf(v, v, a[0]);
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) add_squares(w[k], c.f32, a);
  float s = (a[0] + a[1]) + (a[2] + a[3]);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((t & 31) == 0) red[t >> 5] = s;
  __syncthreads();
  s = red[t & 31];  // every warp forms the same sum
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float norm = __fsqrt_rn(s);
  if (t == 0) *norm_out = norm;
  const float coef = clip_coef(norm, max_norm);
  if (!write || (c.dst == c.src && coef == 1.0f)) return;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = l + k * kFewGroup;
    if (i < nv) static_cast<uint4 *>(c.dst)[i] = scaled(w[k], c.f32, coef);
  }
  for (int e = e0; e < c.n; e += kFewGroup) store1(c, e, coef);
}

}  // namespace

int clip_ctas(int64_t chunks) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (int64_t)num_sms() * 2));
}

cudaError_t launch_clip(const ClipChunk *table, int64_t chunks, bool few, double in_bytes, double elements,
                        bool write, float max_norm, float *norm, float *partials, cudaStream_t st) {
  if (few) {
    LaunchScope ls("clip_few", st, (write ? 2.0 : 1.0) * in_bytes, 3.0 * elements, (int64_t)elements);
    return launch_kernel(clip_few_kernel, dim3(1), dim3(kFewThreads), 0, st, table, (int)chunks,
                         (int)write, max_norm, norm);
  }
  const int grid = clip_ctas(chunks);
  {
    LaunchScope ls("clip_norm", st, in_bytes, 2.0 * elements, (int64_t)elements);
    const cudaError_t e = launch_kernel(clip_norm_kernel, dim3((unsigned)grid), dim3(kClipThreads),
                                        0, st, table, chunks, partials);
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls("clip_scale", st, write ? 2.0 * in_bytes : 0.0, elements, (int64_t)elements);
  return launch_kernel(clip_scale_kernel, dim3(write ? (unsigned)grid : 1u), dim3(kClipThreads), 0,
                       st, table, write ? chunks : (int64_t)0, (const float *)partials, grid,
                       max_norm, norm);
}

}  // namespace fp8lin
