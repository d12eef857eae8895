// What the kernels of 4-bit weights share.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace fp8lin {

// A list's work for one item of the weight's rows, as kernels of `tile` tokens (8, 16 or
// 32) at a time take them: what a block does for the codes is worth as much as for eight
// tokens' products.
__host__ __device__ __forceinline__ int list_work(int count, int tile) {
  const int rest = (count % tile + 7) / 8;
  return count / tile * (1 + tile / 8) + (rest == 0 ? 0 : rest == 3 ? 5 : 1 + rest);
}

}  // namespace fp8lin
