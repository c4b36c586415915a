// The paged cache's own operators: append of new keys and values, and eviction by weight. Both move
// rows and compute next to nothing, so they are bound by memory and, on small calls, by latency.
#include "fa_paged.cuh"

namespace fa {
namespace {

// Append: one warp per new token and tensor (K, V), 16 bytes a lane and up to four of them in flight.
// Bound by memory: the rows are read and written once (134 MB of 16384 tokens in 23 us, 5.8 TB/s; a thread
// per 16 bytes took 32 us). 64 tokens take 2.3 us, the latency of a launch and three loads in a row. Packed
// batches take a warp per row, not per sequence and longest length, which a batch of one prompt and many
// single tokens would leave idle.
__global__ void __launch_bounds__(256) paged_append_kernel(const FaPagedArgs a) {
  let_dependent_start();
  grid_dependency_wait();
  const PagedShape& s = a.s;
  const int lane = threadIdx.x & 31, shift = s.d == 128 ? 4 : 3;  // 16-byte chunks of a head's row
  const uint32_t w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, row = w >> 1;
  const bool is_v = w & 1;
  int b, i = 0;
  if (s.cu_q != nullptr) {
    if (row >= (uint32_t)s.rows_q) return;
    b = sequence_of(s, (int)row);
  } else {
    b = (int)(row / (uint32_t)s.Nq);
    i = (int)(row % (uint32_t)s.Nq);
  }
  if (b >= s.B) return;
  const SeqInfo seq = paged_seq(s, b);
  if (s.cu_q != nullptr) i = (int)row - seq.q0;
  if (i < 0 || i >= seq.Lq) return;
  const long long j = (long long)s.seqlens[b] - seq.Lq + i;  // the unclamped length places the token
  if (j < 0 || (j >> s.page_shift) >= s.max_pages) {
    if (lane == 0) report_status(a.status, FA_ERR_BOUNDS);
    return;
  }
  const FaStrides& ts = is_v ? a.sv_new : a.sk_new;
  const FaStrides& td = is_v ? a.sv : a.sk;
  const __nv_bfloat16* src =
      reinterpret_cast<const __nv_bfloat16*>(is_v ? a.v_new : a.k_new) + elem_offset(ts, seq.bb, seq.q0 + i, 0);
  const int chunks = s.Hkv << shift;
  uint4 x[4];
  auto load = [&](int c0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * 32 + lane;
      if (c < chunks)
        x[k] = *reinterpret_cast<const uint4*>(src + (size_t)(c >> shift) * ts.head + (c & ((1 << shift) - 1)) * 8);
    }
  };
  load(0);  // on its way while the page is looked up
  const int page = paged_page(s, b, (int)(j >> s.page_shift), a.status);
  if (page < 0) return;
  const int slot = (int)(j & ((1 << s.page_shift) - 1));
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v : a.k) + paged_offset(td, page, slot, 0);
  for (int c0 = 0; c0 < chunks; c0 += 128) {
    if (c0 > 0) load(c0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * 32 + lane;
      if (c < chunks)
        *reinterpret_cast<uint4*>(dst + (size_t)(c >> shift) * td.head + (c & ((1 << shift) - 1)) * 8) = x[k];
    }
  }
  if (!is_v && a.weights != nullptr)
    for (int h = lane; h < s.Hkv; h += 32) a.weights[weight_offset(s, page, h, slot)] = 0.f;
}

// ----------------------------------------------------------------------------- eviction

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32, kSelRow = 4 * kSelThreads;

// The order of weights as unsigned integers: larger weight, larger number; -0 equals 0, NaN is 0.
__device__ __forceinline__ uint32_t weight_rank(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sums over the threads of the CTA before this one, and over all (exclusive scan).
__device__ __forceinline__ int cta_scan(int x, int* warp_tot, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // the last scan's totals are read
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  int before = inc - x;
  total = 0;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) {
    if (i < warp) before += warp_tot[i];
    total += warp_tot[i];
  }
  return before;
}

// A cluster (or one CTA) selects the keys of a (sequence, K/V head) into `kept`. A row is 1024 consecutive
// keys, four to a thread (a page holds them together, so one table entry and one 16-byte load fetch them); a
// thread keeps R rows' weights as ranks in registers and reads those of further rows again in each pass. The rank of
// the last kept weight is found 8 bits at a time from the top, in four passes of a histogram in shared memory
// (summed over the cluster) of which each thread scans a bin (three passes of 11 bits: the same time in one CTA,
// twice as long in a cluster of 8). Then a key's place is the number of larger weights before it plus that of equal
// ones, as far as those stay, by a scan over threads and rows in key order.
// Bound by latency: 4.5 us for 8 heads of 1030 keys, 11 for 12 x 8 of up to 8192; counting against bounds instead, 16
// steps of 2 bits, took 13 us for the former.
template <int R>
__device__ __forceinline__ void select_keys(const FaPagedArgs& a, int b, int hk, int L, uint32_t cta, uint32_t ctas,
                                            int32_t* kept) {
  __shared__ int hist[2][256];
  __shared__ int warp_tot[kSelWarps];
  __shared__ int s_digit, s_need;
  __shared__ int cta_tot;  // this CTA's larger and equal weights, packed below
  __shared__ int cta_eq;
  const PagedShape& s = a.s;
  const int tid = threadIdx.x;
  const int old = L - a.recent, take = a.keep - a.recent;  // candidates, and how many of them stay
  for (int t = cta * kSelThreads + tid; t < a.recent; t += ctas * kSelThreads) kept[take + t] = old + t;
  if (take == 0) return;
  const int rows = ((old + (int)ctas - 1) / (int)ctas + kSelRow - 1) / kSelRow;  // per CTA
  const int j0 = (int)cta * rows * kSelRow + 4 * tid;                           // first key of row 0
  hist[0][tid] = 0;
  // Ranks of the thread's four keys of a row; 0 past the end and on a page that is none of the cache's.
  // No branch: such a place reads page 0, and the loads of all rows are in flight together.
  bool bad = false;
  auto page_at = [&](int k) {
    return s.table[(size_t)b * s.max_pages + (min(j0 + k * kSelRow, old - 1) >> s.page_shift)];
  };
  auto ranks_at = [&](int k, int page) -> uint4 {
    const int j = j0 + k * kSelRow, left = k < rows ? old - j : 0;  // keys of the four that are candidates
    const bool ok = (unsigned)page < (unsigned)s.num_pages;
    bad |= !ok && left > 0;
    const float4 w = *reinterpret_cast<const float4*>(
        a.weights + weight_offset(s, ok ? page : 0, hk, j & ((1 << s.page_shift) - 1)));
    const int n = ok ? left : 0;
    return make_uint4(n > 0 ? weight_rank(w.x) : 0u, n > 1 ? weight_rank(w.y) : 0u, n > 2 ? weight_rank(w.z) : 0u,
                      n > 3 ? weight_rank(w.w) : 0u);
  };
  uint4 r[R];
  {
    int page[R];
#pragma unroll
    for (int k = 0; k < R; ++k) page[k] = page_at(k);
#pragma unroll
    for (int k = 0; k < R; ++k) r[k] = ranks_at(k, page[k]);
    if (bad) report_status(a.status, FA_ERR_BOUNDS);
  }
  // Places past the end count as weights of rank 0, which changes no choice above it.
  uint32_t last = 0u;  // the digits found so far of the rank of the last kept weight
  int need = take;     // of the weights with those digits, how many stay
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass, buf = pass & 1;
    const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
    auto count = [&](uint32_t x) {
      if ((x & above) == last) atomicAdd(&hist[buf][(x >> shift) & 255], 1);
    };
    __syncthreads();  // the bins are 0
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (k < rows) {
        count(r[k].x);
        count(r[k].y);
        count(r[k].z);
        count(r[k].w);
      }
    for (int k = R; k < rows; ++k) {
      const uint4 x = ranks_at(k, page_at(k));
      count(x.x);
      count(x.y);
      count(x.z);
      count(x.w);
    }
    hist[buf ^ 1][tid] = 0;
    int bin = 255 - tid, mine;  // thread 0 has the largest digit
    if (ctas > 1) {
      cluster_sync();
      mine = 0;
      for (uint32_t c = 0; c < ctas; ++c) mine += load_peer(&hist[buf][bin], c);
      cluster_sync();  // every CTA has read these bins before they are cleared
    } else {
      __syncthreads();
      mine = hist[buf][bin];
    }
    int total;
    const int larger = cta_scan(mine, warp_tot, total);
    if (larger < need && larger + mine >= need) {
      s_digit = bin;
      s_need = need - larger;
    }
    __syncthreads();
    last |= (uint32_t)s_digit << shift;
    need = s_need;
  }
  // Places: larger and equal weights of the thread per row (packed: gt | eq << 16).
  auto count4 = [&](uint4 x, int k) -> uint32_t {
    const int left = k < rows ? old - (j0 + k * kSelRow) : 0;
    uint32_t n = 0;
    n += (left > 0 && x.x > last) + (left > 1 && x.y > last) + (left > 2 && x.z > last) + (left > 3 && x.w > last);
    n += ((uint32_t)((left > 0 && x.x == last) + (left > 1 && x.y == last) + (left > 2 && x.z == last) +
                     (left > 3 && x.w == last)))
         << 16;
    return n;
  };
  int gt_before = 0, eq_before = 0;  // in the CTAs before this one, then also in the rows before
  if (ctas > 1) {
    int gt = 0, eq = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const uint32_t n = count4(r[k], k);
      gt += n & 0xffff;
      eq += n >> 16;
    }
    for (int k = R; k < rows; ++k) {
      const uint32_t n = count4(ranks_at(k, page_at(k)), k);
      gt += n & 0xffff;
      eq += n >> 16;
    }
    int all_gt, all_eq;
    cta_scan(gt, warp_tot, all_gt);
    cta_scan(eq, warp_tot, all_eq);
    if (tid == 0) {
      cta_tot = all_gt;
      cta_eq = all_eq;
    }
    cluster_sync();
    for (uint32_t c = 0; c < cta; ++c) {
      gt_before += load_peer(&cta_tot, c);
      eq_before += load_peer(&cta_eq, c);
    }
    cluster_sync();  // no CTA leaves while its totals are read
  }
  auto place = [&](uint4 x, int k) {
    const uint32_t n = count4(x, k);
    int total;
    const uint32_t before = (uint32_t)cta_scan((int)n, warp_tot, total);
    int g = gt_before + (int)(before & 0xffff), e = eq_before + (int)(before >> 16);
    const int j = j0 + k * kSelRow, left = k < rows ? old - j : 0;
    auto put = [&](uint32_t y, int i) {
      if (i >= left || y < last) return;
      if (y > last) {
        kept[g + min(e, need)] = j + i;
        ++g;
      } else {
        if (e < need) kept[g + e] = j + i;
        ++e;
      }
    };
    put(x.x, 0);
    put(x.y, 1);
    put(x.z, 2);
    put(x.w, 3);
    gt_before += total & 0xffff;
    eq_before += (uint32_t)total >> 16;
  };
#pragma unroll
  for (int k = 0; k < R; ++k)
    if (k < rows) place(r[k], k);
  for (int k = R; k < rows; ++k) place(ranks_at(k, page_at(k)), k);
}

// The end of a selection that needs none: the lengths, and all keys of a sequence within the budget. True then.
__device__ __forceinline__ bool keeps_all(const FaPagedArgs& a, int b, int hk, int L, uint32_t cta, uint32_t ctas,
                                          int32_t* kept) {
  if (hk == 0 && cta == 0 && threadIdx.x == 0) a.seqlens_out[b] = min(L, a.keep);
  if (L > a.keep) return false;
  for (int t = cta * kSelThreads + threadIdx.x; t < a.keep; t += ctas * kSelThreads) kept[t] = t < L ? t : -1;
  return true;
}

template <int R>
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const FaPagedArgs a) {
  let_dependent_start();
  grid_dependency_wait();
  const PagedShape& s = a.s;
  const uint32_t cta = cluster_rank(), ctas = cluster_size();
  const int head = blockIdx.x / ctas, hk = head % s.Hkv, b = head / s.Hkv, L = paged_seq(s, b).Lk;
  int32_t* kept = a.kept + (size_t)head * a.keep;
  if (!keeps_all(a, b, hk, L, cta, ctas, kept)) select_keys<R>(a, b, hk, L, cta, ctas, kept);  // (the whole cluster)
}

// The kept rows of T tensors (K, V, or both; the weights go with K) move down in blocks of a cluster's shared
// memory: every row of a block is read before any is written, and since kept[t] >= t a block's destinations hold no
// row that a later block still has to read. A row that keeps its place is not moved. Bound by memory, with the
// latency of index, page and row once per block: 12 x 8 heads of up to 8192 keys down to 2050, 211 MB in 35 us, 6.0
// TB/s (blocks of 128 rows a CTA: 39, of 64: 44).
constexpr int kMoveThreads = 256, kMoveCtas = 8, kMoveRows = 256;

template <int T>
__device__ __forceinline__ void move_rows(const FaPagedArgs& a, int b, int hk, int tensor, int cta, int per,
                                          const int32_t* kept, uint8_t* rows_smem) {  // per: rows a CTA takes of a block
  __shared__ const __nv_bfloat16* from[kMoveRows];  // of a row of the block (T = 2: K's, then V's); null: it stays
  __shared__ __nv_bfloat16* to[kMoveRows];
  const PagedShape& s = a.s;
  const int shift = s.d == 128 ? 4 : 3, mask = (1 << s.page_shift) - 1;  // 16-byte chunks of a row
  for (int t0 = cta * per; t0 - cta * per < a.keep; t0 += kMoveCtas * per) {
    const int n = max(0, min(per, a.keep - t0));  // this CTA's rows of the block (none or fewer at the end)
    float w = 0.f, *wt = nullptr;
    __syncthreads();  // the last block's rows are written
    if ((int)threadIdx.x < T * per) {
      const int is_v = T == 1 ? tensor : (int)threadIdx.x >= per, i = threadIdx.x - (T == 1 ? 0 : is_v * per);
      from[threadIdx.x] = nullptr;
      if (i < n) {
        const FaStrides& ts = is_v ? a.sv : a.sk;
        __nv_bfloat16* base = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v : a.k);
        const int t = t0 + i, j = kept[t];
        const int pt = paged_page(s, b, t >> s.page_shift, a.status);
        const int pj = paged_page(s, b, j >> s.page_shift, a.status);
        const bool moves = j != t && pt >= 0 && pj >= 0;
        if (moves) from[threadIdx.x] = base + paged_offset(ts, pj, j & mask, hk);
        to[threadIdx.x] = base + paged_offset(ts, max(pt, 0), t & mask, hk);
        if (!is_v && moves) {
          w = a.weights[weight_offset(s, pj, hk, j & mask)];
          wt = a.weights + weight_offset(s, pt, hk, t & mask);
        }
      }
    }
    __syncthreads();
    const int chunks = (T == 1 ? n : T * per) << shift;
#pragma unroll 4
    for (int c = threadIdx.x; c < chunks; c += kMoveThreads) {
      const __nv_bfloat16* p = from[c >> shift];
      if (p != nullptr)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(rows_smem + c * 16)),
                     "l"(p + (c & ((1 << shift) - 1)) * 8)
                     : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    cluster_sync();
#pragma unroll 4
    for (int c = threadIdx.x; c < chunks; c += kMoveThreads)
      if (from[c >> shift] != nullptr)
        *reinterpret_cast<uint4*>(to[c >> shift] + (c & ((1 << shift) - 1)) * 8) =
            *reinterpret_cast<const uint4*>(rows_smem + c * 16);
    if (wt != nullptr) *wt = w;
  }
}

// An eviction's dependents start after its new lengths are written, since the forwards over contiguous tensors read their
// lengths as data that nothing writes while they live.

// One cluster per (sequence, K/V head, K or V).
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const FaPagedArgs a, int per) {
  grid_dependency_wait();  // the selection, which writes the lengths, is complete
  let_dependent_start();
  extern __shared__ __align__(16) uint8_t rows_smem[];
  const PagedShape& s = a.s;
  const int unit = blockIdx.x / kMoveCtas, head = unit >> 1, hk = head % s.Hkv, b = head / s.Hkv;
  if (paged_seq(s, b).Lk <= a.keep) return;  // (the whole cluster)
  move_rows<1>(a, b, hk, unit & 1, (int)cluster_rank(), per, a.kept + (size_t)head * a.keep, rows_smem);
}

// Both in one launch, for short sequences: one cluster per (sequence, K/V head), of which each CTA selects all keys by
// itself (into its shared memory, without a cluster barrier) and moves its rows of K and V. The weights that the
// others still read are written after the move's barrier only.
constexpr int kEvictRows = 2;  // rows of 1024 candidates at most

__global__ void __launch_bounds__(kMoveThreads) paged_evict_kernel(const FaPagedArgs a, int per) {
  grid_dependency_wait();
  extern __shared__ __align__(16) uint8_t rows_smem[];
  const PagedShape& s = a.s;
  const int cta = (int)cluster_rank(), head = blockIdx.x / kMoveCtas, hk = head % s.Hkv, b = head / s.Hkv;
  const int L = paged_seq(s, b).Lk;
  int32_t* kept = a.kept + (size_t)head * a.keep;
  if (keeps_all(a, b, hk, L, cta, kMoveCtas, kept)) return;  // (the whole cluster)
  int32_t* mine = reinterpret_cast<int32_t*>(rows_smem + (size_t)2 * per * s.d * 2);
  if (hk == 0 && cta == 0 && threadIdx.x == 0) __threadfence();  // the length that this thread wrote
  select_keys<kEvictRows>(a, b, hk, L, 0, 1, mine);
  __syncthreads();
  let_dependent_start();
  for (int t = cta * kMoveThreads + threadIdx.x; t < a.keep; t += kMoveCtas * kMoveThreads) kept[t] = mine[t];
  move_rows<2>(a, b, hk, 0, cta, per, mine, rows_smem);
}

// One launch for a few heads of short sequences, where every CTA has an SM to itself and repeats the selection for
// nothing (16 heads have 128 CTAs): 8 heads of 1030 keys 6.8 us for 7.4 (and a launch less on the host, 22 us for 25), of
// 2000 keys 8.0 for 8.4. From 16 to 32 heads neither form is far ahead: of 1030 keys 7.8 for 8.0 and 8.1 for 8.8, of 2000
// keys 9.6 for 8.9 and 10.0 for 10.3 (13.6 for 13.1 in another set-up); 128 heads 36 for 27.
bool evict_at_once(const PagedShape& s) {
  return s.max_k <= kEvictRows * kSelRow && (long long)s.B * s.Hkv <= 16;
}

template <int R>
cudaError_t launch_select(const FaPagedArgs& a, unsigned ctas, cudaStream_t st) {
  return launch_dependent_cluster(paged_select_kernel<R>, dim3((unsigned)(a.s.B * a.s.Hkv) * ctas), dim3(kSelThreads), 0,
                                  ctas, st, a);
}

}  // namespace
}  // namespace fa

cudaError_t fa_launch_paged_append(const FaPagedArgs& a, cudaStream_t st) {
  const long long rows = a.s.cu_q != nullptr ? a.s.rows_q : (long long)a.s.B * a.s.Nq;
  const long long ctas = (rows * 2 + 7) / 8;  // (threads below 2^32: rows times d are below 2^31)
  return launch_dependent(fa::paged_append_kernel, dim3((unsigned)ctas), dim3(256), 0, st, a);
}

cudaError_t fa_launch_paged_evict(const FaPagedArgs& a, cudaStream_t st) {
  const long long heads = (long long)a.s.B * a.s.Hkv;
  const int share = (a.keep + fa::kMoveCtas - 1) / fa::kMoveCtas;  // rows of a CTA
  auto even = [share](int most) {  // in blocks of equal size, of at most `most` rows
    const int blocks = (share + most - 1) / most, n = (share + blocks - 1) / blocks;
    return n < 16 ? 16 : n;
  };
  cudaError_t e;
  if (fa::evict_at_once(a.s)) {
    // (with a.keep >= max_k nothing is selected, and no more than max_k kept keys are ever in shared memory)
    const int per = even(fa::kMoveRows / 2);
    const size_t smem = (size_t)2 * per * a.s.d * 2 + (size_t)(a.keep < a.s.max_k ? a.keep : a.s.max_k) * sizeof(int32_t);
    e = cudaFuncSetAttribute(fa::paged_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             256 * 128 * 2 + fa::kEvictRows * fa::kSelRow * 4);
    if (e != cudaSuccess) return e;
    return launch_dependent_cluster(fa::paged_evict_kernel, dim3((unsigned)(heads * fa::kMoveCtas)),
                                    dim3(fa::kMoveThreads), smem, fa::kMoveCtas, st, a, per);
  }
  // Registers for the candidates of the longest sequence: up to 8 rows a thread, then CTAs, then 16 rows. CTAs
  // that need not be there cost cluster barriers (1030 keys: 4.5 us with one, 7.7 with two; 12 x 8 heads of 8192
  // keys: 11, 15, 17 and 29 with 1, 2, 4 and 8), rows past the registers are read five times (8 heads of 16384
  // keys: 24, 14, 12 and 12; of 65536: 123, 90, 41 and 16).
  const long long rows = ((long long)a.s.max_k + fa::kSelRow - 1) / fa::kSelRow;
  const unsigned ctas = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
  e = rows <= 2    ? fa::launch_select<2>(a, ctas, st)
                  : rows <= 64 ? fa::launch_select<8>(a, ctas, st)
                               : fa::launch_select<16>(a, ctas, st);
  if (e != cudaSuccess) return e;
  const int per = even(fa::kMoveRows);
  const size_t smem = (size_t)per * a.s.d * 2;
  e = cudaFuncSetAttribute(fa::paged_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 256 * 128 * 2);
  if (e != cudaSuccess) return e;
  return launch_dependent_cluster(fa::paged_move_kernel, dim3((unsigned)(heads * 2 * fa::kMoveCtas)),
                                  dim3(fa::kMoveThreads), smem, fa::kMoveCtas, st, a, per);
}
