// What the few-row kernels (a key per tensor-memory lane, a row per column) share.
#pragma once

#include "fa_paged.cuh"

namespace fa {

constexpr int kDecCluster = 8;      // CTAs of the largest cluster that shares a unit
constexpr float kNoMax = -3.0e38f;  // reference max of a row that has seen no key

inline int padded_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// Reduce v[0 .. 16) over the 32 lanes; afterwards lane l holds column l / 2 in v[0]. A halving exchange: 16
// shuffles instead of 80.
template <typename F>
__device__ __forceinline__ void columns_reduce(float (&v)[16], int lane, F f) {
#pragma unroll
  for (int half = 8; half > 0; half >>= 1) {
    const bool up = lane & (2 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, 2 * half));
    }
  }
  v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

__device__ __forceinline__ bool vote_any(bool x, int id) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

}  // namespace fa
