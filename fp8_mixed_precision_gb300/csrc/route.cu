// Routing of tokens to experts.
//
//   s = softmax(l) or sigmoid(l) over a token's E logits
//   c = s + bias                                    (selection only)
//   group score = sum of the group's best 1 or 2 c; the best groups stay
//   experts = the k largest c left, descending, ties to the lowest index
//   w_j = scale s_j / (sum of the chosen s), or scale s_j
//
// An expert with logit or bias -inf is never chosen; slots left over get expert
// -1 and weight 0.  Renormalised weights are the softmax of log s over the
// chosen ones, which no underflow of s can make 0 / 0.
//
// The choice is that of the exact scores.  Where c is monotone in the logits
// (no bias, and at most one score to a group) the logits are compared
// themselves.  Elsewhere c is formed in fp32; where two scores that decide
// something are closer than fp32's error, fp64 decides: between the experts in
// question, or, where groups are, for the whole row.
//
// LANES threads hold one token's logits in registers, four consecutive ones
// each, CHUNKS times.  Bound by instructions (a row of 128 logits is 256 bytes, its
// eight rounds of finding the largest some 150 instructions of a warp): bf16
// logits that choose by themselves are packed with their index into one word, sorted
// within each lane, and each round is one warp-wide maximum.  131072 tokens, 8 of 128
// experts: 29 us, 19 backward (33.5 MB of logits read, and as much written: 10 us);
// 16379 tokens, 6 of 256 with a bias and groups: 26 and 6.6.  One token: 1.5.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace fp8lin {
namespace {

constexpr int kRouteThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

// Order-preserving map of fp32 onto unsigned; 0 stands for "not a candidate"
// (below every number's image but that of a NaN with the sign set).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 ties with +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

template <int LANES>
__device__ __forceinline__ float sum_over(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float max_over(float v) {
  if constexpr (LANES == 32) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}
template <int LANES>
__device__ __forceinline__ uint32_t max_over(uint32_t v) {
  if constexpr (LANES == 32) {
    return __reduce_max_sync(kFull, v);
  } else {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}
// Largest key of the token's lanes and the lowest index that has it.
template <int LANES>
__device__ __forceinline__ void best_over(uint32_t &key, int &at) {
  if constexpr (LANES == 32) {
    const uint32_t m = __reduce_max_sync(kFull, key);
    at = (int)__reduce_min_sync(kFull, key == m ? (unsigned)at : 0xffffffffu);
    key = m;
  } else {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) {
      const uint32_t k2 = __shfl_xor_sync(kFull, key, o);
      const int a2 = __shfl_xor_sync(kFull, at, o);
      if (k2 > key || (k2 == key && a2 < at)) key = k2, at = a2;
    }
  }
}

__device__ __forceinline__ float load_logit(const void *l, int f32, int64_t i) {
  return f32 ? static_cast<const float *>(l)[i] : bf16lo(static_cast<const uint16_t *>(l)[i]);
}

// The four logits from e on of a row (those from E on: -inf).  vec: rows begin
// on the vector's boundary, E a multiple of 4.
__device__ __forceinline__ void load4(const void *l, int f32, bool vec, int64_t row, int e, int E,
                                      float (&v)[4]) {
  const int64_t i = row * E + e;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = -INFINITY;
  if (vec) {
    if (e >= E) return;
    if (f32) {
      const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(l) + i);
      v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(l) + i);
      v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (e + q < E) v[q] = load_logit(l, f32, i + q);
}

// Order-preserving map of fp64 onto unsigned (-0 and +0 alike), and back.
__device__ __forceinline__ unsigned long long key_of(double v) {
  const unsigned long long b = __double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double of_key(unsigned long long k) {
  return __longlong_as_double(k >> 63 ? k & ~(1ull << 63) : ~k);
}

// A row's maximum and sum of exponentials in fp64 (softmax; sigmoid: 0 and 1), by the
// LANES lanes of its token (`mask`).
template <int LANES>
__device__ __forceinline__ void softmax64(unsigned mask, const RouteArgs &a, int64_t t, double &m, double &z) {
  const int lane = threadIdx.x & (LANES - 1);
  m = 0.0;
  z = 1.0;
  if (a.sigmoid) return;
  float top = -INFINITY;
  for (int e = lane; e < a.E; e += LANES) top = fmaxf(top, load_logit(a.logits, a.f32, t * a.E + e));
  for (int o = LANES / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
  m = top;
  z = 0.0;
  for (int e = lane; e < a.E; e += LANES) z += exp((double)load_logit(a.logits, a.f32, t * a.E + e) - m);
  for (int o = LANES / 2; o; o >>= 1) z += __shfl_xor_sync(mask, z, o);
}
// The key of expert e's score, 0 where it is no candidate.
__device__ __forceinline__ unsigned long long score64(const RouteArgs &a, int64_t t, int e, double m, double z) {
  const double l = load_logit(a.logits, a.f32, t * a.E + e);
  if (!(l > -INFINITY)) return 0ull;
  const double c = (a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / z) + (a.bias ? (double)a.bias[e] : 0.0);
  return c > -INFINITY ? key_of(c) : 0ull;
}

// The kept groups of one row (bit g), decided in fp64; c: E keys of shared memory.
template <int LANES>
__device__ __noinline__ unsigned groups64(unsigned mask, const RouteArgs &a, int64_t t, unsigned long long *c) {
  const int lane = threadIdx.x & (LANES - 1);
  double m, z;
  softmax64<LANES>(mask, a, t, m, z);
  __syncwarp(mask);
  for (int e = lane; e < a.E; e += LANES) c[e] = score64(a, t, e, m, z);
  __syncwarp(mask);
  const int share = LANES / a.groups_pow2, g = lane / share;
  unsigned long long two0 = 0ull, two1 = 0ull;
  if (g < a.groups)
    for (int i = lane % share; i < a.per; i += share) {
      const unsigned long long v = c[g * a.per + i];
      two1 = max(two1, min(two0, v));
      two0 = max(two0, v);
    }
  for (int o = share / 2; o; o >>= 1) {
    const unsigned long long b0 = __shfl_xor_sync(mask, two0, o), b1 = __shfl_xor_sync(mask, two1, o);
    two1 = max(min(two0, b0), max(two1, b1));
    two0 = max(two0, b0);
  }
  unsigned long long score = 0ull;
  if (g < a.groups && lane % share == 0 && two0)
    score = a.top == 2 && two1 ? key_of(of_key(two0) + of_key(two1)) : two0;
  unsigned kept = 0u;
  for (int n = 0; n < a.kept; ++n) {
    unsigned long long best = score;
    int at = g;
    for (int o = LANES / 2; o; o >>= 1) {
      const unsigned long long b2 = __shfl_xor_sync(mask, best, o);
      const int a2 = __shfl_xor_sync(mask, at, o);
      if (b2 > best || (b2 == best && a2 < at)) best = b2, at = a2;
    }
    if (best == 0ull) break;
    kept |= 1u << at;
    if (at == g) score = 0ull;
  }
  return kept;
}

// The choice among the kept groups' experts in fp64; lane j of the token returns
// expert j.  c: E keys of shared memory.
template <int LANES>
__device__ __noinline__ int choose64(unsigned mask, const RouteArgs &a, int64_t t, unsigned kept, unsigned long long *c) {
  const int lane = threadIdx.x & (LANES - 1);
  double m, z;
  softmax64<LANES>(mask, a, t, m, z);
  __syncwarp(mask);
  for (int e = lane; e < a.E; e += LANES)
    c[e] = a.groups == 1 || kept >> (e / a.per) & 1u ? score64(a, t, e, m, z) : 0ull;
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = 0ull;
    int at = 0x7fffffff;
    for (int e = lane; e < a.E; e += LANES)
      if (c[e] > best) best = c[e], at = e;
    for (int o = LANES / 2; o; o >>= 1) {
      const unsigned long long b2 = __shfl_xor_sync(mask, best, o);
      const int a2 = __shfl_xor_sync(mask, at, o);
      if (b2 > best || (b2 == best && a2 < at)) best = b2, at = a2;
    }
    if (best == 0ull) break;
    if (j == lane) mine = at;
    if (at % LANES == lane) c[at] = 0ull;  // read by this lane alone
  }
  return mine;
}

// As choose64, between n <= LANES experts alone: lane i's candidate `e`.  The others
// are known to be below the k best of these.
template <int LANES>
__device__ __noinline__ int choose64_of(unsigned mask, const RouteArgs &a, int64_t t, int e, int n, int *list) {
  const int lane = threadIdx.x & (LANES - 1);
  double m, z;
  softmax64<LANES>(mask, a, t, m, z);
  const unsigned long long key = lane < n ? score64(a, t, e, m, z) : 0ull;
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned long long k2 = __shfl_sync(mask, key, i, LANES);
    const int e2 = __shfl_sync(mask, e, i, LANES);
    rank += k2 > key || (k2 == key && e2 < e);
  }
  __syncwarp(mask);
  if (lane < n && rank < a.k) list[rank] = e;
  __syncwarp(mask);
  return lane < min(n, a.k) ? list[lane] : -1;
}

// sigmoid(l), its smallest values included
__device__ __forceinline__ float sigmoid(float l) {
  const float t = expf(-fabsf(l));
  return __fdiv_rn(l >= 0.0f ? 1.0f : t, 1.0f + t);
}
// log(sigmoid(l))
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }

enum RouteMode {
  kPacked,  // bf16 logits choose by themselves
  kLogits,  // logits choose by themselves
  kSums,    // logits choose experts, sums of two scores groups
  kBiased,  // scores with a bias choose
};

// Sorts N keys, largest first: runs of `half` in order are merged, the second one
// taken backwards.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&k)[N]) {
  const auto exchange = [&](int i, int j) {
    const uint32_t hi = max(k[i], k[j]), lo = min(k[i], k[j]);
    k[i] = hi;
    k[j] = lo;
  };
#pragma unroll
  for (int half = 1; half < N; half *= 2) {
#pragma unroll
    for (int i = 0; i < N; i += 2 * half) {
#pragma unroll
      for (int j = 0; j < half; ++j) exchange(i + j, i + 2 * half - 1 - j);
    }
#pragma unroll
    for (int d = half / 2; d; d /= 2) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(i & d)) exchange(i, i + d);
    }
  }
}

template <int LANES, int CHUNKS, RouteMode MODE>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteArgs a, float *__restrict__ weights,
                                                              int *__restrict__ experts) {
  constexpr bool GENERAL = MODE == kSums || MODE == kBiased;  // scores are formed
  constexpr int kOwn = 4 * CHUNKS;                            // logits of a lane
  constexpr int kTokens = kRouteThreads / LANES;
  // a row of c: fp32 for the groups' scores, fp64 for the choice made anew
  __shared__ double rows[MODE == kPacked ? 1 : kTokens][GENERAL ? 4 * LANES * CHUNKS : 2 * LANES * CHUNKS];
  pdl_wait_then_release();
  const int lane = threadIdx.x & (LANES - 1), slot = MODE == kPacked ? 0 : threadIdx.x / LANES;
  const int64_t row = (int64_t)blockIdx.x * kTokens + threadIdx.x / LANES;
  const int64_t t = row < a.T ? row : a.T - 1;  // spare lanes repeat the last token and write nothing
  const unsigned mask = LANES == 32 ? kFull : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));

  float l[CHUNKS][4];
  bool bad = false;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    load4(a.logits, a.f32, a.vec, t, 4 * LANES * c + 4 * lane, a.E, l[c]);
#pragma unroll
    for (int q = 0; q < 4; ++q) bad |= !(l[c][q] < INFINITY) && (!a.sigmoid || isnan(l[c][q]));
  }
  int mine = -1;  // the expert in slot `lane`
  float x = 0.0f;  // its logit
  float m = -INFINITY, z = 1.0f;
  const auto maximum = [&] {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) m = fmaxf(m, l[c][q]);
    m = max_over<LANES>(m);
  };
  const auto total = [&] {
    z = 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // within 2 + 1.2 (m - l) ulp: of a term that is e^-(m - l) of the largest one
        const float p = GENERAL ? expf(l[c][q] - m) : __expf(l[c][q] - m);
        z += l[c][q] > -INFINITY ? p : 0.0f;
      }
    z = sum_over<LANES>(z);
  };

  if constexpr (MODE == kPacked) {
    uint32_t key[4 * CHUNKS];  // the ordered bf16, and below it the index from the end
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        key[4 * c + q] = l[c][q] > -INFINITY
                             ? (key_of(l[c][q]) & 0xffff0000u) | (uint32_t)(0xffff - (4 * LANES * c + 4 * lane + q))
                             : 0u;
    sort_down(key);
    uint32_t got = 0u;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const uint32_t best = max_over<LANES>(key[0]);
      if (lane == j) got = best;
      if (key[0] == best) {
#pragma unroll
        for (int i = 0; i + 1 < 4 * CHUNKS; ++i) key[i] = key[i + 1];
        key[4 * CHUNKS - 1] = 0u;
      }
    }
    if (got) {
      mine = 0xffff - (int)(got & 0xffffu);
      x = of_key(got & 0x80000000u ? got & 0xffff0000u : got | 0xffffu);
    }
    if (!a.sigmoid && !a.renorm) {
      m = __shfl_sync(kFull, got ? x : -INFINITY, 0, LANES);
      total();
    }
  } else {
    if (!a.sigmoid && (GENERAL || !a.renorm)) {
      maximum();
      total();
    }
    uint32_t key[CHUNKS][4];
    float *line = reinterpret_cast<float *>(rows[slot]);
    float tol = 0.0f, top_score = 0.0f;
    {
      float smax = 0.0f, cmax = 0.0f;
      const float rz = GENERAL ? __fdiv_rn(1.0f, z) : 1.0f;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 4 * LANES * c + 4 * lane + q;
          const float y = l[c][q];
          float v = y, g = y;  // what chooses experts, and groups
          if (GENERAL) {
            // (2 ulp off at most: the choice allows for it)
            const float s = a.sigmoid ? __fdividef(1.0f, 1.0f + expf(-y)) : expf(y - m) * rz;
            const float b = MODE == kBiased && e < a.E ? a.bias[e] : 0.0f;
            const float score = s + b;
            if (y > -INFINITY) {
              bad |= isnan(score);
              smax = fmaxf(smax, s);
              if (fabsf(score) < INFINITY) cmax = fmaxf(cmax, fabsf(score));
            }
            if (MODE == kBiased) v = score;
            g = a.top == 2 ? score : v;
          }
          const bool some = y > -INFINITY && v > -INFINITY;
          key[c][q] = some ? key_of(v) : 0u;
          if (a.groups > 1) line[e] = some ? g : -INFINITY;
        }
      // twice the fp32 error of a score, in units of roundoff: of s, 8 (sigmoid:
      // exponential, sum, quotient) or 8 and half the terms of a lane's and the lanes'
      // sum; of the addition, 1.  Scores below the smallest normal number, 2^-126, may have
      // become 0 (a row whose sigmoids all underflow, with a bias of zeros: all alike here)
      if (GENERAL) {
        tol = (a.sigmoid ? 16.0f : 16.0f + kOwn + 6) * 0x1p-24f * max_over<LANES>(smax) +
              0x1p-23f * (cmax = max_over<LANES>(cmax)) + 0x1p-125f;
        top_score = cmax;
      }
    }
    unsigned kept = 0u;  // groups
    if (a.groups > 1) {
      __syncwarp();
      // a group's scores are shared out over `share` lanes
      const int share = LANES / a.groups_pow2, g = lane / share;
      float two0 = -INFINITY, two1 = -INFINITY;
      if (g < a.groups)
        for (int i = lane % share; i < a.per; i += share) {
          const float v = line[g * a.per + i];
          two1 = fmaxf(two1, fminf(two0, v));
          two0 = fmaxf(two0, v);
        }
      for (int o = share / 2; o; o >>= 1) {
        const float b0 = __shfl_xor_sync(kFull, two0, o), b1 = __shfl_xor_sync(kFull, two1, o);
        two1 = fmaxf(fminf(two0, b0), fmaxf(two1, b1));
        two0 = fmaxf(two0, b0);
      }
      const float score = a.top == 2 && two1 > -INFINITY ? two0 + two1 : two0;
      uint32_t gkey = g < a.groups && lane % share == 0 && two0 > -INFINITY ? key_of(score) : 0u;
      float last = 0.0f;
      for (int n = 0; n < a.kept; ++n) {
        uint32_t k1 = gkey;
        int at = g;
        best_over<LANES>(k1, at);
        if (k1 == 0) continue;
        kept |= 1u << at;
        last = of_key(k1);
        if (at == g) gkey = 0u;
      }
      if (GENERAL) {  // (a sum of two rounds once more)
        const bool close = kept && gkey && !(of_key(gkey) <= last - 2.0f * tol - 0x1p-22f * fabsf(last));
        if (__ballot_sync(kFull, close) & mask)
          kept = groups64<LANES>(mask, a, t, reinterpret_cast<unsigned long long *>(rows[slot]));
        __syncwarp();
      }
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 4 * LANES * c + 4 * lane + q;
          if (!(kept >> ((unsigned)e * a.per_magic >> 20 & 31u) & 1u)) key[c][q] = 0u;
        }
    }
    tol += kOwn * 0x1p-22f * top_score;  // what a lane's numbers take of the keys
    uint32_t mine_key = 0u, last_key = 0u;
    uint32_t kept_keys[kOwn];  // kBiased: a lane's keys in order, their lowest bits the number within the lane
    if constexpr (MODE == kBiased) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        kept_keys[i] = key[i / 4][i % 4] ? (key[i / 4][i % 4] & ~(uint32_t)(kOwn - 1)) | (uint32_t)(kOwn - 1 - i) : 0u;
      sort_down(kept_keys);
      for (int j = 0; j < a.k; ++j) {
        const int i = kOwn - 1 - (int)(kept_keys[0] & (kOwn - 1));
        int at = 4 * LANES * (i / 4) + 4 * lane + i % 4;
        // equal but for the numbers within the lanes: one of those below says so
        uint32_t best = kept_keys[0] | (kOwn - 1);
        const int own_at = at;
        best_over<LANES>(best, at);
        if (kept_keys[0] && own_at == at) {
#pragma unroll
          for (int n = 0; n + 1 < kOwn; ++n) kept_keys[n] = kept_keys[n + 1];
          kept_keys[kOwn - 1] = 0u;
        }
        if (best > (uint32_t)(kOwn - 1)) {
          if (lane == j) mine = at, mine_key = best;
          last_key = best;
        }
      }
    } else {
      // each lane's best; the lane that had the best of all looks for its next one
      uint32_t own = 0u;
      int own_at = 0x7fffffff;
      const auto own_best = [&] {
        own = 0u;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (key[c][q] > own) own = key[c][q], own_at = 4 * LANES * c + 4 * lane + q;
      };
      own_best();
      for (int j = 0; j < a.k; ++j) {
        uint32_t best = own;
        int at = own_at;
        best_over<LANES>(best, at);
        if (best) {
          if (lane == j) mine = at;
          if (own == best && own_at == at) {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (at == 4 * LANES * c + 4 * lane + q) key[c][q] = 0u;
            own_best();
          }
        }
      }
    }
    x = mine >= 0 ? load_logit(a.logits, a.f32, t * a.E + mine) : 0.0f;
    bool close = false;  // experts in question
    float edge = 0.0f;
    const auto index_of = [&](uint32_t k) {  // of a key of this lane
      const int i = kOwn - 1 - (int)(k & (kOwn - 1));
      return 4 * LANES * (i / 4) + 4 * lane + i % 4;
    };
    const auto near = [&](uint32_t k) { return k && !(of_key(k | (kOwn - 1)) <= edge); };
    if constexpr (MODE == kBiased) {
      // neighbours in the order closer than the error, and those left that come as
      // close to the last one chosen (an exact tie is no question: equal logits and
      // biases, told by the index)
      const float b = mine >= 0 ? a.bias[mine] : 0.0f;
      const float x2 = __shfl_down_sync(kFull, x, 1, LANES), b2 = __shfl_down_sync(kFull, b, 1, LANES);
      const uint32_t k2 = __shfl_down_sync(kFull, mine_key, 1, LANES);
      if (lane + 1 < a.k && k2 && !(of_key(k2) <= of_key(mine_key) - tol)) close = x != x2 || b != b2;
      const float xl = __shfl_sync(kFull, x, a.k - 1, LANES), bl = __shfl_sync(kFull, b, a.k - 1, LANES);
      edge = of_key(last_key) - tol;
      if (near(kept_keys[0])) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
          if (near(kept_keys[i])) {
            const int e = index_of(kept_keys[i]);
            close |= load_logit(a.logits, a.f32, t * a.E + e) != xl || a.bias[e] != bl;
          }
      }
    }
    bad = __any_sync(kFull, bad) && (__ballot_sync(kFull, bad) & mask);
    if (GENERAL) {
      close = (__ballot_sync(kFull, close) & mask) && !bad;
      if constexpr (MODE == kBiased) {
        if (close) {
          int *list = reinterpret_cast<int *>(rows[slot]);
          __syncwarp(mask);
          int n = __popc(__ballot_sync(mask, mine >= 0) & mask);
          if (mine >= 0) list[lane] = mine;
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            const bool one = near(kept_keys[i]);
            const unsigned who = __ballot_sync(mask, one) & mask;
            const int at = n + __popc(who & ((1u << (threadIdx.x & 31)) - 1u));
            if (one && at < LANES) list[at] = index_of(kept_keys[i]);
            n += __popc(who);
          }
          __syncwarp(mask);
          if (n <= LANES)
            mine = choose64_of<LANES>(mask, a, t, lane < n ? list[lane] : 0, n, list);
          else
            mine = choose64<LANES>(mask, a, t, kept, reinterpret_cast<unsigned long long *>(rows[slot]));
          x = mine >= 0 ? load_logit(a.logits, a.f32, t * a.E + mine) : 0.0f;
        }
      }
      __syncwarp();
    }
  }
  if (!GENERAL) bad = __any_sync(kFull, bad) && (__ballot_sync(kFull, bad) & mask);
  const bool some = mine >= 0;
  float w = 0.0f;
  if (a.renorm) {
    const float g = some ? (a.sigmoid ? log_sigmoid(x) : x) : -INFINITY;
    const float top = max_over<LANES>(g);
    const float u = some ? expf(g - top) : 0.0f;
    const float all = sum_over<LANES>(u);
    if (some) w = __fdiv_rn(u, all) * a.scale;
  } else if (some) {
    w = (a.sigmoid ? sigmoid(x) : __fdiv_rn(expf(x - m), z)) * a.scale;
  }
  if (row < a.T && lane < a.k) {
    weights[t * a.k + lane] = bad ? __int_as_float(0x7fc00000) : w;
    experts[t * a.k + lane] = bad ? -1 : mine;
  }
}

// dL/dlog s_j = w_j g_j, or w_j (g_j - sum_i g_i w_i / scale) with renormalised
// weights; softmax: dl_e = that of e - s_e times their sum (0 when
// renormalised); sigmoid: times 1 - s_e.
template <int LANES, int CHUNKS>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_kernel(const RouteArgs a, const float *__restrict__ dweights,
                                                                  const float *__restrict__ weights,
                                                                  const int *__restrict__ experts,
                                                                  void *__restrict__ dlogits) {
  constexpr int kTokens = kRouteThreads / LANES;
  pdl_wait_then_release();
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t row = (int64_t)blockIdx.x * kTokens + threadIdx.x / LANES;
  const int64_t t = row < a.T ? row : a.T - 1;
  int e = -1;
  float w = 0.0f, g = 0.0f;
  if (lane < a.k) {
    e = experts[t * a.k + lane];
    w = weights[t * a.k + lane];
    g = dweights[t * a.k + lane];
  }
  const bool some = e >= 0 && e < a.E;
  float d = some ? w * g : 0.0f;
  if (a.renorm) {
    const float total = sum_over<LANES>(d);
    if (some) d = w * (g - __fdiv_rn(total, a.scale));
  }
  if (a.sigmoid && some) d *= sigmoid(-load_logit(a.logits, a.f32, t * a.E + e));
  float v[CHUNKS][4];
  if (!a.sigmoid && !a.renorm) {
    float m = -INFINITY, z = 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      load4(a.logits, a.f32, a.vec, t, 4 * LANES * c + 4 * lane, a.E, v[c]);
#pragma unroll
      for (int q = 0; q < 4; ++q) m = fmaxf(m, v[c][q]);
    }
    m = max_over<LANES>(m);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[c][q] = v[c][q] > -INFINITY ? __expf(v[c][q] - m) : 0.0f;
        z += v[c][q];
      }
    z = sum_over<LANES>(z);
    const float total = sum_over<LANES>(d);
    const float f = z > 0.0f ? -__fdiv_rn(total, z) : 0.0f;  // a row without a candidate: zeros
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[c][q] = f == 0.0f ? 0.0f : v[c][q] * f;  // (v is NaN at a logit of +inf)
  } else {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[c][q] = 0.0f;
  }
  // The chosen experts' part meets the row in shared memory (k rounds of comparing
  // every lane's indices took 45.7 us for 131072 x 128 with k = 8).  An expert
  // named twice in a row, which the forward pass does not do, takes those rounds.
  __shared__ float4 rows[kTokens][LANES * CHUNKS];
  float4 *line = rows[threadIdx.x / LANES];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) line[LANES * c + lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncwarp();
  if (some) reinterpret_cast<int *>(line)[e] = lane;
  __syncwarp();
  const bool twice = some && reinterpret_cast<int *>(line)[e] != lane;  // another lane wrote there too
  if (__any_sync(kFull, twice)) {
    for (int j = 0; j < a.k; ++j) {
      const int ej = __shfl_sync(kFull, some ? e : -1, j, LANES);
      const float dj = __shfl_sync(kFull, d, j, LANES);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (ej == 4 * LANES * c + 4 * lane + q) v[c][q] += dj;
    }
  } else {
    if (some) reinterpret_cast<float *>(line)[e] = d;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const float4 w4 = line[LANES * c + lane];
      v[c][0] += w4.x, v[c][1] += w4.y, v[c][2] += w4.z, v[c][3] += w4.w;
    }
  }
  if (row >= a.T) return;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int e0 = 4 * LANES * c + 4 * lane;
    const int64_t i = t * a.E + e0;
    if (a.vec) {
      if (e0 >= a.E) continue;
      if (a.f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(dlogits) + i) = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
      else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(dlogits) + i) =
            make_uint2(pack_bf16x2(v[c][0], v[c][1]), pack_bf16x2(v[c][2], v[c][3]));
      continue;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e0 + q < a.E) {
        if (a.f32)
          static_cast<float *>(dlogits)[i + q] = v[c][q];
        else
          static_cast<__nv_bfloat16 *>(dlogits)[i + q] = __float2bfloat16_rn(v[c][q]);
      }
  }
}

// Calls f with LANES and CHUNKS that hold E experts, k choices and the groups.  With
// many tokens as few lanes to a token as `chunks` allows: what is done once per lane,
// and the rounds across lanes, then serve several tokens (131072 x 128 with k = 8,
// forward + backward: 32 lanes 78 us, 8 lanes 45).  With few, all 32: the shortest way
// to one token's result.
template <int MOST, typename F>
cudaError_t with_shape(const RouteArgs &a, F f) {
  using std::integral_constant;
  const int lanes = std::max(a.k, a.groups);
  const auto chunks = [&](int l) { return (a.E + 4 * l - 1) / (4 * l); };
  if (a.T >= (int64_t)num_sms() * 32) {
    if (lanes <= 8 && chunks(8) <= 1) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (lanes <= 8 && chunks(8) <= 2) return f(integral_constant<int, 8>(), integral_constant<int, 2>());
    if constexpr (MOST >= 4)
      if (lanes <= 8 && chunks(8) <= 4) return f(integral_constant<int, 8>(), integral_constant<int, 4>());
    if (lanes <= 16 && chunks(16) <= 2) return f(integral_constant<int, 16>(), integral_constant<int, 2>());
    if constexpr (MOST >= 4)
      if (lanes <= 16 && chunks(16) <= 4) return f(integral_constant<int, 16>(), integral_constant<int, 4>());
  }
  if (chunks(32) <= 1) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
  if (chunks(32) <= 2) return f(integral_constant<int, 32>(), integral_constant<int, 2>());
  if (chunks(32) <= 4) return f(integral_constant<int, 32>(), integral_constant<int, 4>());
  return f(integral_constant<int, 32>(), integral_constant<int, 8>());
}

}  // namespace

cudaError_t launch_route_fwd(RouteArgs a, float *weights, int *experts, cudaStream_t st) {
  a.per = a.E / a.groups;
  a.per_magic = (1u << 20) / (unsigned)a.per + 1u;
  for (a.groups_pow2 = 1; a.groups_pow2 < a.groups;) a.groups_pow2 *= 2;
  LaunchScope ls("route_fwd", st, (double)a.T * (a.E * (a.f32 ? 4.0 : 2.0) + 8.0 * a.k), 4.0 * a.T * a.E, a.T, a.E,
                 a.k);
  const auto go = [&](auto kernel, int l) {
    return launch_kernel(kernel, dim3((unsigned)((a.T + kRouteThreads / l - 1) / (kRouteThreads / l))),
                         dim3(kRouteThreads), 0, st, a, weights, experts);
  };
  // (with a bias 16 logits to a lane take more of the keys than they save: 16379 x 256
  // 40 us against 33)
  if (a.bias)
    return with_shape<2>(a, [&](auto l, auto c) { return go(route_kernel<l(), c(), kBiased>, l()); });
  if (a.groups > 1 && a.top == 2)
    return with_shape<4>(a, [&](auto l, auto c) { return go(route_kernel<l(), c(), kSums>, l()); });
  return with_shape<4>(a, [&](auto l, auto c) {
    if constexpr (c() <= 4)  // (more than 16 keys are more than a lane can keep in order)
      if (!a.f32 && a.groups == 1) return go(route_kernel<l(), c(), kPacked>, l());
    return go(route_kernel<l(), c(), kLogits>, l());
  });
}

cudaError_t launch_route_bwd(RouteArgs a, const float *dweights, const float *weights, const int *experts,
                             void *dlogits, cudaStream_t st) {
  LaunchScope ls("route_bwd", st, (double)a.T * (a.E * (a.f32 ? 4.0 : 2.0) + 12.0 * a.k), 2.0 * a.T * a.E, a.T, a.E,
                 a.k);
  return with_shape<4>(a, [&](auto lanes, auto chunks) {
    constexpr int L = decltype(lanes)::value, C = decltype(chunks)::value;
    const dim3 grid((unsigned)((a.T + kRouteThreads / L - 1) / (kRouteThreads / L)));
    return launch_kernel(route_bwd_kernel<L, C>, grid, dim3(kRouteThreads), 0, st, a, dweights, weights, experts,
                         dlogits);
  });
}

}  // namespace fp8lin
