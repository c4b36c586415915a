// The online-softmax step of the 128-row query tiles (forward kernels): one key tile's scores in
// tensor memory become P, and the running row max and row sum follow.
#pragma once

#include <type_traits>

#include "sm103_ptx.cuh"

namespace fa {
namespace tc {

// O is rescaled only when a row max grows by more than kRescale in log2 units (lazy; exact since
// l and O share the stale max). The e4m3 P is 2^8 exp2(s - m): with m at most 0.8 below the
// true max it stays <= 2^8.8 < 448, the largest e4m3 value, so it never saturates (measured:
// the e4m3 forward 4% faster than with an exact running max).
template <bool F8>
constexpr float kRescale = F8 ? 0.8f : 8.0f;
template <bool F8>
constexpr float kPExp = F8 ? 8.0f : 0.0f;  // P is computed as 2^kPExp exp2(s - m)

// One key tile of the online softmax for the query row this thread owns (its tensor-memory
// lane): S is read at tS, O (at tO) is rescaled when the row max grows by more than a factor 2^kRescale,
// P is written over the first columns of S and m, l are updated. With `masked`, the keys at
// columns >= lim are excluded. first: the row's first key tile. Called by whole warps.
// LD_BATCH: chunks of 32 columns of S loaded from tensor memory per wait.
template <int D, bool F8, int LD_BATCH, typename PreWrite>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, uint32_t tP, bool masked, int lim, float sl2,
                                             bool first, float& m, float& l, PreWrite&& pre_write) {
  // Columns [32c, 32c + 32) of the row of S: the loads of kLdBatch chunks share one wait.
  uint32_t sr[LD_BATCH * 32];
  auto chunk = [&](int c, uint32_t(&rr)[32]) {
    constexpr int NB = LD_BATCH;
    if (c % NB == 0) {
#pragma unroll
      for (int j = 0; j < NB; ++j) tmem_ld32(tS + (c + j) * 32, *reinterpret_cast<uint32_t(*)[32]>(sr + j * 32));
      tmem_ld_wait();
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) rr[i] = sr[(c % NB) * 32 + i];
  };
  // Pass 1: row max of the (masked) scores, 32 columns at a time.
  auto row_max = [&](auto mask_tag) -> float {
    constexpr bool MASK = decltype(mask_tag)::value;
    float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t rr[32];
      chunk(c, rr);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float v0 = __uint_as_float(rr[i]), v1 = __uint_as_float(rr[i + 1]);
        if constexpr (MASK) {
          v0 = (c * 32 + i < lim) ? v0 : -INFINITY;
          v1 = (c * 32 + i + 1 < lim) ? v1 : -INFINITY;
        }
        pm[(i >> 1) & 3] = fmax3(pm[(i >> 1) & 3], v0, v1);
      }
    }
    return fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
  };
  const float mx = masked ? row_max(std::true_type{}) : row_max(std::false_type{});
  const float mc = mx * sl2;
  pre_write();  // O and P may be written once the previous P V has completed
  if (first) {
    m = mc;
  } else if (__any_sync(0xffffffffu, mc > m + kRescale<F8>)) {
    const float mn = fmaxf(m, mc);
    const float alpha = (mn == -INFINITY) ? 1.f : ex2_approx(m - mn);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t rr[32];
      tmem_ld32(tO + c * 32, rr);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
      tmem_st32(tO + c * 32, rr);
    }
    l *= alpha;
    m = mn;
  }
  const float mu = (m == -INFINITY) ? 0.f : m;
  // Pass 2: P = exp2(c log2(e) s - m) over the first columns of S (bf16: 64 columns; e4m3,
  // as 2^8 P: 32 columns; each chunk is written only over columns already read), and the
  // row sum of P.
  auto exp_pass = [&](auto mask_tag) -> float {
    constexpr bool MASK = decltype(mask_tag)::value;
    const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(kPExp<F8> - mu, kPExp<F8> - mu);
    float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t rr[32];
      chunk(c, rr);
      uint32_t pk[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 x = fma2(make_float2(__uint_as_float(rr[2 * i]), __uint_as_float(rr[2 * i + 1])), sc2, nm2);
        float p0 = ex2_approx(x.x);
        float p1 = ex2_approx(x.y);
        if constexpr (MASK) {
          p0 = (c * 32 + 2 * i < lim) ? p0 : 0.f;
          p1 = (c * 32 + 2 * i + 1 < lim) ? p1 : 0.f;
        }
        ps[i & 1] = add2(ps[i & 1], make_float2(p0, p1));
        if constexpr (F8) {  // four e4m3 values per column, key 4w + j in byte j of column w
          const uint32_t pair = pack_e4m3x2(p0, p1);
          pk[i >> 1] = (i & 1) ? (pk[i >> 1] | (pair << 16)) : pair;
        } else {
          pk[i] = pack_bf16x2(p0, p1);
        }
      }
      if constexpr (F8) {
        tmem_st8(tP + c * 8, *reinterpret_cast<const uint32_t(*)[8]>(pk));
      } else {
        tmem_st16(tP + c * 16, pk);
      }
    }
    return (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
  };
  const float sum = masked ? exp_pass(std::true_type{}) : exp_pass(std::false_type{});
  tmem_st_wait();
  l += sum;
}

}  // namespace tc
}  // namespace fa
