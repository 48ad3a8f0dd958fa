// Position -> slot arithmetic of paged KV caches, shared by the attention and
// the compaction kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8blk {

// Division of n < 2^31 by a fixed d in [1, 2^30]: with 2^s >= d the smallest
// such power and m = ceil(2^(31+s) / d) < 2^32, floor(n m / 2^(31+s)) =
// floor(n / d), since m d exceeds 2^(31+s) by less than d <= 2^s and n < 2^31.
struct FastDiv {
  uint32_t m, s, d;
};

inline FastDiv make_fastdiv(int64_t d) {
  uint32_t s = 0;
  while ((int64_t(1) << s) < d) ++s;
  const uint64_t p = uint64_t(1) << (31 + s);
  return FastDiv{(uint32_t)((p + (uint64_t)d - 1) / (uint64_t)d), 31 + s, (uint32_t)d};
}

__device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv f) { return (uint32_t)(((uint64_t)n * f.m) >> f.s); }

// Slot of position j under a sequence's row of the block table, or -1 where
// it is outside the pool of num_slots < 2^31 slots.
__device__ __forceinline__ int slot_of(const int64_t* __restrict__ row, uint32_t j, FastDiv f, int num_slots) {
  const uint32_t b = div_by(j, f);
  const int64_t e = row[b];
  if ((uint64_t)e > (uint32_t)num_slots) return -1;
  const int64_t s = e * (int64_t)f.d + (j - b * f.d);
  return s < num_slots ? (int)s : -1;
}

}  // namespace fp8blk
