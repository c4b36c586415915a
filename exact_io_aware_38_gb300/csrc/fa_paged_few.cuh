// What the few-row kernels (a key per tensor-memory lane, a row per column) share.
#pragma once

#include "fa_paged.cuh"

namespace fa {

constexpr int kDecCluster = 8;      // CTAs of the largest cluster that shares a unit
constexpr float kNoMax = -3.0e38f;  // reference max of a row that has seen no key

inline int padded_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// Reduce the N columns v over the 32 lanes; afterwards lane l holds column l N / 32 in v[0]. A halving exchange: 16
// shuffles for 16 columns instead of 80.
template <int N, typename F>
__device__ __forceinline__ void columns_reduce(float (&v)[N], int lane, F f) {
  constexpr int kLanes = 32 / N;  // of a column in the end
#pragma unroll
  for (int half = N / 2; half > 0; half >>= 1) {
    const bool up = lane & (kLanes * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, kLanes * half));
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
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
