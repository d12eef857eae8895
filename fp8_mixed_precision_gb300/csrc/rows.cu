// Rows in the experts' order: a stable counting sort of the T k slots (slot
// t k + j: token t's choice j) by expert, token rows gathered in that order,
// and the experts' output rows weighted and summed per token.
//
//   offsets[e]     first row of expert e, a multiple of `align`; offsets[E]: rows in use
//   counts[e]      its rows
//   position[slot] the slot's row, -1 where it has no expert
//   order[row]     the row's slot, -1 for a row between an expert's last and the
//                  next one's first
//
// Every row movement runs over tokens: a token's row is read once and written
// to (or formed from) its k places, so each byte crosses memory once, and each
// sum has one order.  Bound by memory: with 6785 GB/s as a plain copy's rate, 131072
// rows of 512 to 2 of 16 experts are gathered in 59 us (6.9 TB/s), 16379 of 4096 to 4 of
// 64 in 101 (6.7); their order takes 9 and 10.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "w4.cuh"

namespace fp8lin {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kOrderThreads = 256, kOrderWarps = kOrderThreads / 32;
constexpr int kOrderChunk = 2048;  // slots of a block

__device__ __forceinline__ int expert_of(const int *experts, int64_t slot, int E) {
  const int e = experts[slot];
  return e >= 0 && e < E ? e : -1;
}

// hist[e][b]: slots of expert e in chunk b.
__global__ void __launch_bounds__(kOrderThreads) order_count_kernel(const int *__restrict__ experts, int64_t n, int E,
                                                                    int *__restrict__ hist) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kOrderThreads) count[e] = 0;
  pdl_wait_then_release();
  __syncthreads();
  const int64_t from = (int64_t)blockIdx.x * kOrderChunk;
#pragma unroll
  for (int i = 0; i < kOrderChunk / kOrderThreads; ++i) {
    const int64_t s = from + i * kOrderThreads + threadIdx.x;
    const int e = s < n ? expert_of(experts, s, E) : -1;
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kOrderThreads) hist[(int64_t)e * gridDim.x + blockIdx.x] = count[e];
}

// One warp per expert: exclusive sums of hist[e] over the chunks, in place, and
// the total.
__global__ void __launch_bounds__(kOrderThreads) order_scan_kernel(int *__restrict__ hist, int E, int chunks,
                                                                   int *__restrict__ counts) {
  pdl_wait_then_release();
  const int e = blockIdx.x * kOrderWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
  if (e >= E) return;
  int *h = hist + (int64_t)e * chunks;
  int total = 0;
  for (int b = 0; b < chunks; b += 32) {
    const int v = b + lane < chunks ? h[b + lane] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += u;
    }
    if (b + lane < chunks) h[b + lane] = total + s - v;
    total += __shfl_sync(kFull, s, 31);
  }
  if (lane == 0) counts[e] = total;
}

// Places a chunk's slots.  hist null: the one chunk of a small problem, which
// counts for itself.  Each warp ranks its part of the chunk in order; warps'
// counts and the chunks' are summed before.
__global__ void __launch_bounds__(kOrderThreads) order_place_kernel(const int *__restrict__ experts, int64_t n, int E,
                                                                    int align, const int *__restrict__ hist,
                                                                    int *__restrict__ counts, int *__restrict__ offsets,
                                                                    int *__restrict__ position,
                                                                    int *__restrict__ order, W4List *__restrict__ lists,
                                                                    int most, int tile) {
  extern __shared__ int smem[];
  int *mine = smem;                    // [kOrderWarps][E]: rows before this warp's next slot of e
  int *start = smem + kOrderWarps * E;  // [E + 1]
  __shared__ int part[kOrderWarps];
  __shared__ int64_t part64[kOrderWarps];
  pdl_wait_then_release();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kOrderWarps * E; i += kOrderThreads) mine[i] = 0;
  __syncthreads();
  constexpr int kBatches = kOrderChunk / kOrderThreads;
  const int64_t from = (int64_t)blockIdx.x * kOrderChunk + warp * (kOrderChunk / kOrderWarps);
  int e[kBatches];
#pragma unroll
  for (int i = 0; i < kBatches; ++i) {
    const int64_t s = from + 32 * i + lane;
    e[i] = s < n ? expert_of(experts, s, E) : -1;
    if (e[i] >= 0) atomicAdd(&mine[warp * E + e[i]], 1);
  }
  __syncthreads();
  // per expert: the warps' counts become what lies before each of them
  for (int x = threadIdx.x; x < E; x += kOrderThreads) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < kOrderWarps; ++w) {
      const int c = mine[w * E + x];
      mine[w * E + x] = before;
      before += c;
    }
    if (!hist) counts[x] = before;
    start[x] = hist ? counts[x] : before;
  }
  __syncthreads();
  // exclusive sums of the aligned counts, 256 experts at a time (and for the products of
  // the experts' tokens those of the lists and their work)
  int total = 0;
  int64_t listed = 0;  // lists << 32 | work
  for (int b = 0; b < E; b += kOrderThreads) {
    const int x = b + threadIdx.x;
    const int v = x < E ? (start[x] + align - 1) / align * align : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    int before = total;
    for (int w = 0; w < warp; ++w) before += part[w];
    const int first = before + s - v;
    if (x < E) {
      // rows between this expert's last and the next one's first
      if (blockIdx.x == 0) offsets[x] = first;
      if (x % gridDim.x == blockIdx.x)
        for (int r = start[x]; r < v; ++r) order[first + r] = -1;
    }
    for (int w = 0; w < kOrderWarps; ++w) total += part[w];
    __syncthreads();
    if (lists && blockIdx.x == 0) {
      const int n = x < E ? start[x] : 0;
      const int64_t own = n ? (int64_t(1) << 32) + list_work(n, tile) : 0;
      int64_t sum = own;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int64_t u = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += u;
      }
      if (lane == 31) part64[warp] = sum;
      __syncthreads();
      for (int w = 0; w < warp; ++w) sum += part64[w];
      const int64_t at = listed + sum - own;
      if (n) lists[at >> 32] = W4List{x, first, n, (int)at};
      for (int w = 0; w < kOrderWarps; ++w) listed += part64[w];
      __syncthreads();
    }
    if (x < E) {
      const int base = first + (hist ? hist[(int64_t)x * gridDim.x + blockIdx.x] : 0);
#pragma unroll
      for (int w = 0; w < kOrderWarps; ++w) mine[w * E + x] += base;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = total;
  if (lists && blockIdx.x == 0)
    for (int l = (int)(listed >> 32) + threadIdx.x; l <= most; l += kOrderThreads)
      lists[l] = W4List{0, 0, 0, (int)listed};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBatches; ++i) {
    const int64_t s = from + 32 * i + lane;
    const unsigned same = __match_any_sync(kFull, e[i]);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int row = -1;
    if (e[i] >= 0) row = mine[warp * E + e[i]] + rank;
    __syncwarp();
    if (e[i] >= 0 && rank == 0) mine[warp * E + e[i]] += __popc(same);
    __syncwarp();
    if (s < n) {
      position[s] = row;
      if (row >= 0) order[row] = (int)s;
    }
  }
}

constexpr int kRowThreads = 256;

__device__ __forceinline__ uint4 load16(const void *p, int64_t i) { return static_cast<const uint4 *>(p)[i]; }
__device__ __forceinline__ void add8(uint4 v, float w, float (&a)[8]) {
  a[0] = fmaf(bf16lo(v.x), w, a[0]); a[1] = fmaf(bf16hi(v.x), w, a[1]);
  a[2] = fmaf(bf16lo(v.y), w, a[2]); a[3] = fmaf(bf16hi(v.y), w, a[3]);
  a[4] = fmaf(bf16lo(v.z), w, a[4]); a[5] = fmaf(bf16hi(v.z), w, a[5]);
  a[6] = fmaf(bf16lo(v.w), w, a[6]); a[7] = fmaf(bf16hi(v.w), w, a[7]);
}
__device__ __forceinline__ uint4 pack8(const float (&a)[8]) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
}
// Piece i of rows of `vecs` pieces: (row, piece).  A 64-bit division takes some 100
// instructions.
__device__ __forceinline__ int64_t row_of(int64_t i, int vecs, int &c) {
  if (i >> 32) {
    const int64_t t = i / vecs;
    c = (int)(i - t * vecs);
    return t;
  }
  const uint32_t t = (uint32_t)i / (uint32_t)vecs;
  c = (int)((uint32_t)i - t * (uint32_t)vecs);
  return t;
}
// The rows behind an expert's last, up to the next one's first: zeros, so that
// products over whole aligned groups of rows take nothing from them.
__device__ __forceinline__ void zero_gap(void *rows, int vecs, int e, const int *counts, const int *offsets) {
  const int64_t first = (int64_t)(offsets[e] + counts[e]) * vecs, last = (int64_t)offsets[e + 1] * vecs;
  for (int64_t i = first + threadIdx.x; i < last; i += kRowThreads)
    static_cast<uint4 *>(rows)[i] = make_uint4(0, 0, 0, 0);
}

// One thread per 16 bytes of a token's row; the blocks from `blocks` on zero
// the gaps, one expert each.
__global__ void __launch_bounds__(kRowThreads) rows_gather_kernel(const void *__restrict__ x,
                                                                  const int *__restrict__ position, int64_t total,
                                                                  int vecs, int k, unsigned blocks,
                                                                  const int *__restrict__ counts,
                                                                  const int *__restrict__ offsets, void *__restrict__ xs) {
  pdl_wait_then_release();
  if (blockIdx.x >= blocks) return zero_gap(xs, vecs, blockIdx.x - blocks, counts, offsets);
  const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (i >= total) return;
  const uint4 v = load16(x, i);
  int c;
  const int64_t t = row_of(i, vecs, c);
  for (int j = 0; j < k; ++j) {
    const int p = position[t * k + j];
    if (p >= 0) static_cast<uint4 *>(xs)[(int64_t)p * vecs + c] = v;
  }
}

// weights null: the sum of the rows.  A slot without an expert counts as its
// weight times zero, so that a weight that is NaN shows.  One 16-byte piece to a
// thread, the rows of four slots on the way at once: 131072 x 2 x 512 takes 69 us (59 at
// the copy rate), 131072 x 8 x 512 174 (178); two pieces to a thread 81 and 227.
__global__ void __launch_bounds__(kRowThreads) rows_combine_kernel(const void *__restrict__ z,
                                                                   const int *__restrict__ position,
                                                                   const float *__restrict__ weights, int64_t total,
                                                                   int vecs, int k, void *__restrict__ y) {
  constexpr int kAtOnce = 4;
  pdl_wait_then_release();
  const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (i >= total) return;
  int c;
  const int64_t slot = row_of(i, vecs, c) * k;
  float a[8] = {};
  for (int j0 = 0; j0 < k; j0 += kAtOnce) {
    int p[kAtOnce];
    float w[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const bool in = j0 + j < k;
      p[j] = in ? position[slot + j0 + j] : -1;
      w[j] = !in ? 0.0f : weights ? weights[slot + j0 + j] : 1.0f;
    }
    uint4 v[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      v[j] = p[j] >= 0 ? load16(z, (int64_t)p[j] * vecs + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) add8(v[j], w[j], a);
  }
  static_cast<uint4 *>(y)[i] = pack8(a);
}

// dz[row] = w dy[t] and dweights[slot] = <dy[t], z[row]>: TPT threads per token,
// AT choices at a time, so that dy is read once for as many.  131072 x 2 x 512 takes
// 101 us (6.6 TB/s), 16379 x 4 x 4096 175 (6.9).
template <int TPT, int AT>
__global__ void __launch_bounds__(kRowThreads) rows_combine_bwd_kernel(
    const void *__restrict__ dy, const void *__restrict__ z, const int *__restrict__ position,
    const float *__restrict__ weights, int64_t T, int vecs, int k, unsigned blocks, const int *__restrict__ counts,
    const int *__restrict__ offsets, void *__restrict__ dz, float *__restrict__ dweights) {
  constexpr int kTokens = kRowThreads / TPT, kWarps = TPT / 32;
  __shared__ float red[kTokens][kWarps][AT];
  pdl_wait_then_release();
  if (blockIdx.x >= blocks) return zero_gap(dz, vecs, blockIdx.x - blocks, counts, offsets);
  const int slot = threadIdx.x / TPT, at = threadIdx.x % TPT;
  const int64_t t = (int64_t)blockIdx.x * kTokens + slot;
  for (int j0 = 0; j0 < k; j0 += AT) {
    int p[AT];
    float w[AT], dot[AT] = {};
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      const bool in = t < T && j0 + j < k;
      p[j] = in ? position[t * k + j0 + j] : -1;
      w[j] = in ? weights[t * k + j0 + j] : 0.0f;
    }
    if (t < T)
      for (int c = at; c < vecs; c += TPT) {
        const uint4 d = load16(dy, t * vecs + c);
        uint4 v[AT];
#pragma unroll
        for (int j = 0; j < AT; ++j) v[j] = p[j] >= 0 ? load16(z, (int64_t)p[j] * vecs + c) : make_uint4(0, 0, 0, 0);
        const float f[8] = {bf16lo(d.x), bf16hi(d.x), bf16lo(d.y), bf16hi(d.y),
                            bf16lo(d.z), bf16hi(d.z), bf16lo(d.w), bf16hi(d.w)};
#pragma unroll
        for (int j = 0; j < AT; ++j) {
          if (p[j] < 0) continue;
          float s = dot[j];
          s = fmaf(f[0], bf16lo(v[j].x), s); s = fmaf(f[1], bf16hi(v[j].x), s);
          s = fmaf(f[2], bf16lo(v[j].y), s); s = fmaf(f[3], bf16hi(v[j].y), s);
          s = fmaf(f[4], bf16lo(v[j].z), s); s = fmaf(f[5], bf16hi(v[j].z), s);
          s = fmaf(f[6], bf16lo(v[j].w), s); s = fmaf(f[7], bf16hi(v[j].w), s);
          dot[j] = s;
          float g[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) g[q] = f[q] * w[j];
          static_cast<uint4 *>(dz)[(int64_t)p[j] * vecs + c] = pack8(g);
        }
      }
#pragma unroll
    for (int j = 0; j < AT; ++j)
#pragma unroll
      for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(kFull, dot[j], o);
    if (kWarps > 1) {
      if ((at & 31) == 0)
#pragma unroll
        for (int j = 0; j < AT; ++j) red[slot][at / 32][j] = dot[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < AT; ++j) {
        dot[j] = 0.0f;
#pragma unroll
        for (int w2 = 0; w2 < kWarps; ++w2) dot[j] += red[slot][w2][j];
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < AT; ++j)
      if (t < T && at == j && j0 + j < k) dweights[t * k + j0 + j] = dot[j];
  }
}

}  // namespace

int order_chunks(int64_t slots) { return (int)((slots + kOrderChunk - 1) / kOrderChunk); }

cudaError_t launch_expert_order(const int *experts, int64_t slots, int E, int align, int *counts, int *offsets,
                                int *position, int *order, int *hist, cudaStream_t st, W4List *lists, int most,
                                int tile) {
  const int chunks = order_chunks(slots);
  const size_t smem = (size_t)(kOrderWarps * E + E + 1) * 4;
  if (chunks > 1) {
    {
      LaunchScope ls("order_count", st, 4.0 * slots, 0.0, slots, E);
      const cudaError_t e = launch_kernel(order_count_kernel, dim3((unsigned)chunks), dim3(kOrderThreads), 0, st,
                                          experts, slots, E, hist);
      if (e != cudaSuccess) return e;
    }
    LaunchScope ls("order_scan", st, 8.0 * E * chunks, 0.0, slots, E);
    const cudaError_t e = launch_kernel(order_scan_kernel, dim3((unsigned)((E + kOrderWarps - 1) / kOrderWarps)),
                                        dim3(kOrderThreads), 0, st, hist, E, chunks, counts);
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls("order_place", st, 12.0 * slots, 0.0, slots, E);
  return launch_kernel(order_place_kernel, dim3((unsigned)chunks), dim3(kOrderThreads), smem, st, experts, slots, E,
                       align, chunks > 1 ? (const int *)hist : (const int *)nullptr, counts, offsets, position, order, lists, most,
                       tile);
}

cudaError_t launch_rows_gather(const void *x, int64_t T, int64_t C, int k, int E, int align, const int *counts,
                               const int *offsets, const int *position, void *xs, cudaStream_t st) {
  const int vecs = (int)(C / 8);
  const unsigned blocks = (unsigned)((T * vecs + kRowThreads - 1) / kRowThreads);
  LaunchScope ls("rows_gather", st, 2.0 * T * C * (1 + k), 0.0, T, C, k);
  return launch_kernel(rows_gather_kernel, dim3(blocks + (align > 1 ? E : 0)), dim3(kRowThreads), 0, st, x, position,
                       T * vecs, vecs, k, blocks, counts, offsets, xs);
}

cudaError_t launch_rows_combine(const void *z, const int *position, const float *weights, int64_t T, int64_t C, int k,
                                void *y, cudaStream_t st) {
  const int vecs = (int)(C / 8);
  LaunchScope ls("rows_combine", st, 2.0 * T * C * (1 + k), 2.0 * T * C * k, T, C, k);
  return launch_kernel(rows_combine_kernel, dim3((unsigned)((T * vecs + kRowThreads - 1) / kRowThreads)),
                       dim3(kRowThreads), 0, st, z, position, weights, T * vecs, vecs, k, y);
}

cudaError_t launch_rows_combine_bwd(const void *dy, const void *z, const int *position, const float *weights, int64_t T,
                                    int64_t C, int k, int E, int align, const int *counts, const int *offsets, void *dz,
                                    float *dweights, cudaStream_t st) {
  const int vecs = (int)(C / 8);
  LaunchScope ls("rows_combine_bwd", st, 2.0 * T * C * (1 + 2 * k), 4.0 * T * C * k, T, C, k);
  auto go = [&](auto kernel, int tpt) {
    const unsigned blocks = (unsigned)((T + kRowThreads / tpt - 1) / (kRowThreads / tpt));
    return launch_kernel(kernel, dim3(blocks + (align > 1 ? E : 0)), dim3(kRowThreads), 0, st, dy, z, position, weights,
                         T, vecs, k, blocks, counts, offsets, dz, dweights);
  };
  // One or two choices: room in registers for more tokens at once (131072 x 2 x 512 114 us
  // with four, 101 with two).  Threads to a token: a warp walks 16-byte pieces best where
  // tokens are many (32768 x 2 x 2048 115 us with 256, 101 with 128, 100 with 32), a block
  // where rows are long or few (16379 x 4 x 4096 175 and 182, 37 x 4 x 4096 3.2 and 9.8).
  const auto by_row = [&](auto at) {
    constexpr int AT = decltype(at)::value;
    if (vecs > 256) return go(rows_combine_bwd_kernel<256, AT>, 256);
    return vecs > 128 ? go(rows_combine_bwd_kernel<128, AT>, 128) : go(rows_combine_bwd_kernel<32, AT>, 32);
  };
  return k <= 2 ? by_row(std::integral_constant<int, 2>()) : by_row(std::integral_constant<int, 4>());
}

}  // namespace fp8lin
