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
constexpr int kSelRegs = 16;                           // weights a thread keeps in registers
constexpr int kSelSpan = kSelThreads * kSelRegs;       // weights a CTA keeps in registers

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A store into the shared memory of CTA `cta` of the cluster, at the address that `p` has there.
__device__ __forceinline__ void store_peer(int* p, uint32_t cta, int x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(cta));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

// The order of weights as unsigned integers: larger weight, larger number; -0 equals 0, NaN is 0.
__device__ __forceinline__ uint32_t weight_rank(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int warp_add(int x) { return __reduce_add_sync(0xffffffffu, x); }

// One cluster per (sequence, K/V head), of the size that keeps all candidates' weights in registers
// (16 384 a CTA; beyond eight CTAs the rest is read again in each step). The rank of the last kept
// weight is found bit by bit from the top, by counting: 32 counts over registers need no histogram
// and so no atomics, whose conflicts the few exponents of attention weights would provoke. Then a
// key's place is the number of larger weights before it plus that of equal ones, as far as those
// stay; both come from ballots and one scan, in key order.
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const FaPagedArgs a) {
  grid_dependency_wait();
  __shared__ int warp_cnt[2][32];
  __shared__ int cta_cnt[2][8];                  // the cluster's counts, per parity of the step
  __shared__ int before_gt[32], before_eq[32];   // per warp of a row of 1024 keys
  __shared__ int cta_gt[8], cta_eq[8];
  const PagedShape& s = a.s;
  const uint32_t cta = cluster_rank(), ctas = cluster_size();
  const int head = blockIdx.x / ctas, hk = head % s.Hkv, b = head / s.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = paged_seq(s, b).Lk;
  int32_t* kept = a.kept + (size_t)head * a.keep;
  if (hk == 0 && cta == 0 && threadIdx.x == 0) a.seqlens_out[b] = min(L, a.keep);
  if (L <= a.keep) {  // (the whole cluster)
    for (int t = cta * kSelThreads + threadIdx.x; t < a.keep; t += ctas * kSelThreads) kept[t] = t < L ? t : -1;
    return;
  }
  const int old = L - a.recent, take = a.keep - a.recent;  // candidates, and how many of them stay
  for (int t = cta * kSelThreads + threadIdx.x; t < a.recent; t += ctas * kSelThreads) kept[take + t] = old + t;
  if (take == 0) return;
  const int rows = ((old + (int)ctas - 1) / (int)ctas + kSelThreads - 1) / kSelThreads;  // of 1024 keys, per CTA
  const int j0 = (int)cta * rows * kSelThreads + threadIdx.x;
  auto rank_of = [&](int j) -> uint32_t {
    if (j >= old) return 0u;
    const int page = paged_page(s, b, j >> s.page_shift, a.status);
    return page < 0 ? 0u : weight_rank(a.weights[weight_offset(s, page, hk, j & ((1 << s.page_shift) - 1))]);
  };
  uint32_t r[kSelRegs];
#pragma unroll
  for (int k = 0; k < kSelRegs; ++k) r[k] = k < rows ? rank_of(j0 + k * kSelThreads) : 0u;
  uint32_t last = 0u;  // the largest rank that `take` candidates reach
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = last | (1u << bit);
    int cnt = 0;
#pragma unroll
    for (int k = 0; k < kSelRegs; ++k)
      if (k < rows) cnt += r[k] >= c;
    for (int k = kSelRegs; k < rows; ++k) cnt += rank_of(j0 + k * kSelThreads) >= c;
    cnt = warp_add(cnt);
    if (lane == 0) warp_cnt[bit & 1][warp] = cnt;
    __syncthreads();
    cnt = warp_add(warp_cnt[bit & 1][lane]);
    if (ctas > 1) {
      if (threadIdx.x < ctas) store_peer(&cta_cnt[bit & 1][cta], threadIdx.x, cnt);
      cluster_sync();
      cnt = warp_add(lane < (int)ctas ? cta_cnt[bit & 1][lane] : 0);
    }
    if (cnt >= take) last = c;
  }
  // Per CTA the larger and equal weights, then the places.
  auto larger = [&](int j, uint32_t x) { return j < old && x > last; };
  auto equal = [&](int j, uint32_t x) { return j < old && x == last; };
  int gt = 0, eq = 0;
#pragma unroll
  for (int k = 0; k < kSelRegs; ++k)
    if (k < rows) {
      gt += larger(j0 + k * kSelThreads, r[k]);
      eq += equal(j0 + k * kSelThreads, r[k]);
    }
  for (int k = kSelRegs; k < rows; ++k) {
    const uint32_t x = rank_of(j0 + k * kSelThreads);
    gt += larger(j0 + k * kSelThreads, x);
    eq += equal(j0 + k * kSelThreads, x);
  }
  gt = warp_add(gt);
  eq = warp_add(eq);
  __syncthreads();  // the last step's counts are read
  if (lane == 0) {
    warp_cnt[0][warp] = gt;
    warp_cnt[1][warp] = eq;
  }
  __syncthreads();
  gt = warp_add(warp_cnt[0][lane]);
  eq = warp_add(warp_cnt[1][lane]);
  if (threadIdx.x < ctas) {
    store_peer(&cta_gt[cta], threadIdx.x, gt);
    store_peer(&cta_eq[cta], threadIdx.x, eq);
  }
  cluster_sync();
  int all_gt = 0, gt_before = 0, eq_before = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    all_gt += cta_gt[c];
    if (c < cta) {
      gt_before += cta_gt[c];
      eq_before += cta_eq[c];
    }
  }
  const int equal_stay = take - all_gt;
  const uint32_t below = (1u << lane) - 1u;
  auto place = [&](int k, uint32_t x) {
    const int j = j0 + k * kSelThreads;
    const bool g = larger(j, x), e = equal(j, x);
    const uint32_t mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
    if (lane == 0) {
      before_gt[warp] = __popc(mg);
      before_eq[warp] = __popc(me);
    }
    __syncthreads();
    const int wg = before_gt[lane], we = before_eq[lane];
    const int pg = gt_before + warp_add(lane < warp ? wg : 0) + __popc(mg & below);
    const int pe = eq_before + warp_add(lane < warp ? we : 0) + __popc(me & below);
    if (g || (e && pe < equal_stay)) kept[pg + min(pe, equal_stay)] = j;
    gt_before += warp_add(wg);
    eq_before += warp_add(we);
    __syncthreads();
  };
#pragma unroll
  for (int k = 0; k < kSelRegs; ++k)
    if (k < rows) place(k, r[k]);
  for (int k = kSelRegs; k < rows; ++k) place(k, rank_of(j0 + k * kSelThreads));
}

// One cluster per (sequence, K/V head, K or V). The kept rows move down in blocks of the cluster's
// shared memory: every row of a block is read before any is written, and since kept[t] >= t a block's
// destinations hold no row that a later block still has to read. A row that keeps its place is not
// moved. Bound by memory, with the latency of index, page and row once per block.
constexpr int kMoveThreads = 256, kMoveCtas = 8;

__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const FaPagedArgs a, int per) {  // per: rows a CTA takes of a block
  grid_dependency_wait();
  extern __shared__ __align__(16) uint8_t rows_smem[];
  __shared__ int from[256];
  const PagedShape& s = a.s;
  const int cta = (int)cluster_rank(), unit = blockIdx.x / kMoveCtas;
  const bool is_v = unit & 1;
  const int head = unit >> 1, hk = head % s.Hkv, b = head / s.Hkv;
  if (paged_seq(s, b).Lk <= a.keep) return;  // (the whole cluster)
  const int32_t* kept = a.kept + (size_t)head * a.keep;
  const FaStrides& ts = is_v ? a.sv : a.sk;
  __nv_bfloat16* base = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v : a.k);
  const int chunks = s.d / 8, mask = (1 << s.page_shift) - 1;  // 16-byte chunks of a row
  auto row_of = [&](int j) -> __nv_bfloat16* {
    const int page = paged_page(s, b, j >> s.page_shift, a.status);
    return page < 0 ? nullptr : base + paged_offset(ts, page, j & mask, hk);
  };
  auto weight_of = [&](int j) -> float* {
    const int page = paged_page(s, b, j >> s.page_shift, a.status);
    return page < 0 ? nullptr : a.weights + weight_offset(s, page, hk, j & mask);
  };
  for (int t0 = cta * per; t0 - cta * per < a.keep; t0 += kMoveCtas * per) {
    const int n = min(per, a.keep - t0);  // this CTA's rows of the block (none or fewer at the end)
    float w = 0.f;
    __syncthreads();  // the last block's rows are written
    if ((int)threadIdx.x < n) {
      const int j = kept[t0 + threadIdx.x];
      from[threadIdx.x] = j == t0 + (int)threadIdx.x ? -1 : j;
      if (!is_v && j != t0 + (int)threadIdx.x)
        if (const float* p = weight_of(j)) w = *p;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n * chunks; c += kMoveThreads) {
      const int j = from[c / chunks];
      if (j < 0) continue;
      if (const __nv_bfloat16* p = row_of(j))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(rows_smem + c * 16)),
                     "l"(p + c % chunks * 8)
                     : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    cluster_sync();
    for (int c = threadIdx.x; c < n * chunks; c += kMoveThreads) {
      const int t = t0 + c / chunks;
      if (from[c / chunks] < 0) continue;
      if (__nv_bfloat16* p = row_of(t))
        *reinterpret_cast<uint4*>(p + c % chunks * 8) = *reinterpret_cast<const uint4*>(rows_smem + c * 16);
    }
    if (!is_v && (int)threadIdx.x < n && from[threadIdx.x] >= 0)
      if (float* p = weight_of(t0 + threadIdx.x)) *p = w;
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
  const long long heads = (long long)a.s.B * a.s.Hkv;
  // The smallest cluster whose registers hold the candidates of the longest sequence.
  unsigned ctas = 1;
  while (ctas < 8 && (long long)ctas * fa::kSelSpan < a.s.max_k) ctas *= 2;
  cudaError_t e = launch_dependent_cluster(fa::paged_select_kernel, dim3((unsigned)(heads * ctas)),
                                           dim3(fa::kSelThreads), 0, ctas, st, a);
  if (e != cudaSuccess) return e;
  // A block of 8 CTAs' rows: all of `keep` where it fits (the latency is then paid once), at most 256 a CTA.
  const int share = (a.keep + fa::kMoveCtas - 1) / fa::kMoveCtas;
  const int per = share < 16 ? 16 : share > 256 ? 256 : share;
  const size_t smem = (size_t)per * a.s.d * 2;
  e = cudaFuncSetAttribute(fa::paged_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 256 * 128 * 2);
  if (e != cudaSuccess) return e;
  return launch_dependent_cluster(fa::paged_move_kernel, dim3((unsigned)(heads * 2 * fa::kMoveCtas)),
                                  dim3(fa::kMoveThreads), smem, fa::kMoveCtas, st, a, per);
}
