// The paged cache's own operators: append of new keys and values, and eviction by weight. Both move
// rows and compute next to nothing, so they are bound by memory and, on small calls, by latency.
#include "fa_paged.cuh"

namespace fa {
namespace {

// Append: one warp per new token and tensor (K, V), 16 bytes a lane.
__global__ void __launch_bounds__(256) paged_append_kernel(const FaPagedArgs a) {
  grid_dependency_wait();
  const PagedShape& s = a.s;
  const int lane = threadIdx.x & 31, chunks = s.d / 8;  // 16-byte chunks of a head's row
  const size_t items = (size_t)s.B * s.Nq * 2;
  const size_t step = ((size_t)gridDim.x * blockDim.x) >> 5;
  for (size_t w = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < items; w += step) {
    const bool is_v = w & 1;
    const int i = (int)((w >> 1) % s.Nq), b = (int)((w >> 1) / s.Nq);
    const SeqInfo seq = paged_seq(s, b);
    if (i >= seq.Lq) continue;
    const long long j = (long long)__ldg(s.seqlens + b) - seq.Lq + i;  // the unclamped length places the token
    if (j < 0 || (j >> s.page_shift) >= s.max_pages) {
      if (lane == 0) report_status(a.status, FA_ERR_BOUNDS);
      continue;
    }
    const int page = paged_page(s, b, (int)(j >> s.page_shift), a.status);
    if (page < 0) continue;
    const int slot = (int)(j & ((1 << s.page_shift) - 1));
    const FaStrides& ts = is_v ? a.sv_new : a.sk_new;
    const FaStrides& td = is_v ? a.sv : a.sk;
    const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(is_v ? a.v_new : a.k_new);
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v : a.k);
    for (int c = lane; c < s.Hkv * chunks; c += 32) {
      const int h = c / chunks, e = c % chunks * 8;
      *reinterpret_cast<uint4*>(dst + paged_offset(td, page, slot, h) + e) =
          *reinterpret_cast<const uint4*>(src + elem_offset(ts, seq.bb, seq.q0 + i, h) + e);
    }
    if (!is_v && a.weights != nullptr)
      for (int h = lane; h < s.Hkv; h += 32) a.weights[weight_offset(s, page, h, slot)] = 0.f;
  }
}

// ----------------------------------------------------------------------------- eviction

constexpr int kSelThreads = 1024;

// The order of weights as unsigned integers: larger weight, larger number; -0 equals 0, NaN is 0.
__device__ __forceinline__ uint32_t weight_rank(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block of one number per thread, and the total.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int base = 0;
  total = 0;
  for (int i = 0; i < kSelThreads / 32; ++i) {
    if (i < warp) base += warp_sums[i];
    total += warp_sums[i];
  }
  __syncthreads();
  return base + inc - x;
}

// One CTA per (sequence, K/V head): the rank of the last kept weight is found digit by digit from the
// top (8 bits a pass), then one pass in key order writes the kept indices: every larger weight and, of
// the equal ones, the first few.
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const FaPagedArgs a) {
  grid_dependency_wait();
  __shared__ int hist[256];
  __shared__ int warp_sums[kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const PagedShape& s = a.s;
  const int hk = blockIdx.x % s.Hkv, b = blockIdx.x / s.Hkv;
  const int L = paged_seq(s, b).Lk;
  int32_t* kept = a.kept + ((size_t)b * s.Hkv + hk) * a.keep;
  if (hk == 0 && threadIdx.x == 0) a.seqlens_out[b] = min(L, a.keep);
  if (L <= a.keep) {
    for (int t = threadIdx.x; t < a.keep; t += kSelThreads) kept[t] = t < L ? t : -1;
    return;
  }
  const int old = L - a.recent, take = a.keep - a.recent;  // candidates, and how many of them stay
  auto rank_of = [&](int j) -> uint32_t {
    const int page = paged_page(s, b, j >> s.page_shift, a.status);
    return page < 0 ? 0u : weight_rank(a.weights[weight_offset(s, page, hk, j & ((1 << s.page_shift) - 1))]);
  };
  if (threadIdx.x == 0) {
    s_prefix = 0u;
    s_need = take;
  }
  if (take > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (threadIdx.x < 256) hist[threadIdx.x] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix, above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int j = threadIdx.x; j < old; j += kSelThreads) {
        const uint32_t r = rank_of(j);
        if ((r & above) == prefix) atomicAdd(&hist[(r >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        int need = s_need, digit = 255;
        while (hist[digit] < need) need -= hist[digit--];
        s_prefix = prefix | ((uint32_t)digit << shift);
        s_need = need;
      }
      __syncthreads();
    }
  }
  __syncthreads();
  const uint32_t last = s_prefix;  // rank of the last kept weight
  int equal_left = s_need;         // how many weights of that rank stay
  int written = 0;
  if (take > 0)
    for (int j0 = 0; j0 < old; j0 += kSelThreads) {
      const int j = j0 + threadIdx.x;
      const uint32_t r = j < old ? rank_of(j) : 0u;
      const bool eq = j < old && r == last;
      int equals, stays;
      const int eq_before = block_scan(eq, warp_sums, equals);
      const bool stay = j < old && (r > last || (eq && eq_before < equal_left));
      const int at = block_scan(stay, warp_sums, stays);
      if (stay) kept[written + at] = j;
      written += stays;
      equal_left -= min(equals, equal_left);
    }
  for (int t = threadIdx.x; t < a.recent; t += kSelThreads) kept[take + t] = old + t;
}

// One CTA per (sequence, K/V head, K or V): the kept rows move down in blocks. Since kept[t] >= t, a
// block's destinations hold no row that a later block still has to read; within a block every row is
// read before any is written.
constexpr int kMoveRows = 64, kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const FaPagedArgs a) {
  grid_dependency_wait();
  const PagedShape& s = a.s;
  const bool is_v = blockIdx.x & 1;
  const int hk = (blockIdx.x >> 1) % s.Hkv, b = (blockIdx.x >> 1) / s.Hkv;
  if (paged_seq(s, b).Lk <= a.keep) return;
  const int32_t* kept = a.kept + ((size_t)b * s.Hkv + hk) * a.keep;
  const FaStrides& ts = is_v ? a.sv : a.sk;
  __nv_bfloat16* base = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v : a.k);
  const int chunks = s.d / 8, mask = (1 << s.page_shift) - 1;
  constexpr int kPer = kMoveRows * 16 / kMoveThreads;
  for (int t0 = 0; t0 < a.keep; t0 += kMoveRows) {
    uint4 x[kPer];
    float w = 0.f;
    auto row_of = [&](int j) -> __nv_bfloat16* {
      const int page = paged_page(s, b, j >> s.page_shift, a.status);
      return page < 0 ? nullptr : base + paged_offset(ts, page, j & mask, hk);
    };
    auto weight_of = [&](int j) -> float* {
      const int page = paged_page(s, b, j >> s.page_shift, a.status);
      return page < 0 ? nullptr : a.weights + weight_offset(s, page, hk, j & mask);
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = threadIdx.x + i * kMoveThreads, t = t0 + c / chunks;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c < kMoveRows * chunks && t < a.keep)
        if (const __nv_bfloat16* p = row_of(kept[t])) x[i] = *reinterpret_cast<const uint4*>(p + c % chunks * 8);
    }
    const int tw = t0 + threadIdx.x;
    const bool has_w = !is_v && threadIdx.x < kMoveRows && tw < a.keep;
    if (has_w)
      if (const float* p = weight_of(kept[tw])) w = *p;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = threadIdx.x + i * kMoveThreads, t = t0 + c / chunks;
      if (c < kMoveRows * chunks && t < a.keep)
        if (__nv_bfloat16* p = row_of(t)) *reinterpret_cast<uint4*>(p + c % chunks * 8) = x[i];
    }
    if (has_w)
      if (float* p = weight_of(tw)) *p = w;
    __syncthreads();
  }
}

}  // namespace
}  // namespace fa

cudaError_t fa_launch_paged_append(const FaPagedArgs& a, cudaStream_t st) {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const size_t ctas = ((size_t)a.s.B * a.s.Nq * 2 + 7) / 8;
  const unsigned grid = (unsigned)(ctas < (size_t)sms * 8 ? ctas : (size_t)sms * 8);
  return launch_dependent(fa::paged_append_kernel, dim3(grid), dim3(256), 0, st, a);
}

cudaError_t fa_launch_paged_evict(const FaPagedArgs& a, cudaStream_t st) {
  const unsigned heads = (unsigned)(a.s.B * a.s.Hkv);
  const cudaError_t e = launch_dependent(fa::paged_select_kernel, dim3(heads), dim3(fa::kSelThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa::paged_move_kernel, dim3(heads * 2), dim3(fa::kMoveThreads), 0, st, a);
}
