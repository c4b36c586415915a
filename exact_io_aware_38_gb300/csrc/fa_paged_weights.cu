// Attention of new tokens over a paged K/V cache, and the attention weight each cached key receives.
//
// First form, one warp per query row (or per key): the row max and row sum run along (online softmax),
// so nothing of the size keys x rows is stored. Bound by instructions, not by memory.
#include "fa_paged.cuh"

namespace fa {
namespace {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
__device__ __forceinline__ void load_row(const void* base, size_t off, int lane, float (&x)[D / 32]) {
  const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(base) + off + lane * (D / 32);
#pragma unroll
  for (int e = 0; e < D / 32; ++e) x[e] = __bfloat162float(p[e]);
}

// One warp per (sequence, K/V head, key): the rows that see the key, in order.
template <int D>
__global__ void __launch_bounds__(256) paged_keys_kernel(const FaPagedArgs a) {
  grid_dependency_wait();
  constexpr int PER = D / 32;
  const PagedShape& s = a.s;
  const int lane = threadIdx.x & 31, G = s.H / s.Hkv;
  const size_t keys = (size_t)s.B * s.Hkv * s.max_k;
  const size_t step = ((size_t)gridDim.x * blockDim.x) >> 5;
  for (size_t w = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < keys; w += step) {
    const int j = (int)(w % s.max_k), hk = (int)(w / s.max_k % s.Hkv), b = (int)(w / s.max_k / s.Hkv);
    const SeqInfo seq = paged_seq(s, b);
    if (j >= seq.Lk) continue;
    const int page = paged_page(s, b, j >> s.page_shift, a.status);
    if (page < 0) continue;
    const int slot = j & ((1 << s.page_shift) - 1);
    float k[PER], q[PER];
    load_row<D>(a.k, paged_offset(a.sk, page, slot, hk), lane, k);
    float sum = 0.f;
    for (int i = s.causal ? max(0, j - seq.off) : 0; i < seq.Lq; ++i)
      for (int h = hk * G; h < hk * G + G; ++h) {
        load_row<D>(a.q, elem_offset(a.sq, seq.bb, seq.q0 + i, h), lane, q);
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) x += q[e] * k[e];
        x = warp_sum(x) * a.scale;
        const float lse = a.lse[paged_row(s, seq, b, h, i)];
        if (lse != -INFINITY) sum += expf(x - lse);
      }
    if (lane == 0) a.weights[weight_offset(s, page, hk, slot)] += sum;
  }
}

int grid_for(size_t warps) {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const size_t ctas = (warps + 7) / 8;
  return (int)(ctas < (size_t)sms * 8 ? ctas : (size_t)sms * 8);
}

}  // namespace
}  // namespace fa

cudaError_t fa_launch_paged_key_weights(const FaPagedArgs& a, cudaStream_t st) {
  auto k = a.s.d == 64 ? fa::paged_keys_kernel<64> : fa::paged_keys_kernel<128>;
  return launch_dependent(k, dim3(fa::grid_for((size_t)a.s.B * a.s.Hkv * a.s.max_k)), dim3(256), 0, st, a);
}
