// What the kernels of 4-bit weights share.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace fp8lin {

// The tokens of list y: expert, first row in the experts' order and count.
struct Tokens {
  int e, first, count;
};
__device__ __forceinline__ Tokens tokens_of(const W4Args &a, int y) {
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

}  // namespace fp8lin
