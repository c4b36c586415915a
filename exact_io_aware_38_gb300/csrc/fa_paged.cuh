// Shared definitions of the paged-cache operators (attention over a cache in pages, append, key
// weights, eviction); the readings are stated in include/fa.h.
#pragma once

#include "fa_common.cuh"
#include "fa_tmap.h"

namespace fa {

struct PagedShape {
  int B, H, Hkv, d;
  int Nq;                 // fixed length: new tokens per sequence; packed: their maximum
  int max_k;              // bound on the key count: min(the caller's, capacity)
  const int32_t* cu_q;    // [B + 1] or null, as in AttnShape
  int rows_q;
  int causal;
  int page_shift;         // log2(slots per page)
  int num_pages, max_pages;
  const int32_t* table;    // [B][max_pages]
  const int32_t* seqlens;  // [B]
  int min_q, max_q;        // to paged_part, sequences with fewer or more new tokens are without any: another kernel has them
};

// The kernels of this family are programmatic dependents of one another. Each lets its own dependent be
// scheduled as soon as all its CTAs run, sets up what is not in global memory, and then waits for the kernel
// before it; the dependent does the same, so one kernel's set-up lies under the other's end. The order of
// memory stays that of the stream: nothing is read or written before the wait, and a kernel that the
// predecessor waited for is complete when the predecessor is. Lengths, offsets and page tables are read by ordinary
// loads for this reason: a kernel may be resident while one before it still writes them (an eviction its lengths), and
// the read-only path (__ldg) holds only for data that nothing writes while the kernel lives.
__device__ __forceinline__ void let_dependent_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// One sequence of the batch: its new rows, its keys and the causal offset (key j visible to row i iff
// j <= i + off). Everything is clamped to the tensors' extents, so no array in device memory can make
// a kernel index outside them.
__device__ __forceinline__ SeqInfo paged_seq(const PagedShape& s, int b) {
  SeqInfo r;
  if (s.cu_q != nullptr) {
    r.q0 = clampi(s.cu_q[b], 0, s.rows_q);
    r.Lq = clampi(s.cu_q[b + 1] - r.q0, 0, min(s.Nq, s.rows_q - r.q0));
    r.bb = 0;
  } else {
    r.q0 = 0;
    r.Lq = s.Nq;
    r.bb = b;
  }
  r.Lk = clampi(s.seqlens[b], 0, s.max_k);
  r.k0 = 0;
  r.off = r.Lk - r.Lq;
  r.krows = r.Lk;
  return r;
}
// The same for the kernels that may share the sequences of a batch by their new tokens. (Not for all: an append of 64 tokens takes
// 2.1 us without the look at the limits and 2.2 with it.)
__device__ __forceinline__ SeqInfo paged_part(const PagedShape& s, int b) {
  SeqInfo r = paged_seq(s, b);
  if (r.Lq < s.min_q || r.Lq > s.max_q) {
    r.Lq = 0;
    r.off = r.Lk;
  }
  return r;
}

// Index of row (token i of the sequence, head h) in the LSE's order: [B][H][Nq], packed [H][rows_q].
__device__ __forceinline__ size_t paged_row(const PagedShape& s, const SeqInfo& q, int b, int h, int i) {
  return s.cu_q != nullptr ? (size_t)h * s.rows_q + q.q0 + i : ((size_t)b * s.H + h) * s.Nq + i;
}

// The page of the table entry `e` of sequence b, or -1 (reported) when it is none of the cache's.
__device__ __forceinline__ int paged_page(const PagedShape& s, int b, int e, int* status) {
  const int page = s.table[(size_t)b * s.max_pages + e];
  if ((unsigned)page < (unsigned)s.num_pages) return page;
  report_status(status, FA_ERR_BOUNDS);
  return -1;
}

// The sequence of packed row `row`: the number of sequences that end at or before it. A whole warp looks, 32
// ends at a time, so 32 sequences take one load and 1000 take two.
__device__ __forceinline__ int sequence_of(const PagedShape& s, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = s.B;  // the answer is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) >> 5, at = (lane + 1) * step;  // the lane's probe: sequence lo + at - 1
    const int cnt = __popc(__ballot_sync(0xffffffffu, at <= n && s.cu_q[lo + min(at, n)] <= row));
    lo += cnt * step;
    n = min(n - cnt * step, step - 1);
  }
  return lo;
}

// Element offset of (page, slot, head) in a cache.
__device__ __forceinline__ size_t paged_offset(const FaStrides& t, int page, int slot, int h) {
  return (size_t)page * t.batch + (size_t)slot * t.row + (size_t)h * t.head;
}

// Offset of (page, head, slot) in the weights, [num_pages][Hkv][page_size].
__device__ __forceinline__ size_t weight_offset(const PagedShape& s, int page, int hk, int slot) {
  return (((size_t)page * s.Hkv + hk) << s.page_shift) + slot;
}

// A cache's tensor map, boxes of a page's slots (128 at most). At d = 64 a head's row is 128 bytes and the next 128 are
// often another head's, which misses of 256 bytes would fetch for nothing and lose before its turn: 128 sequences of
// 2048 keys, 12 heads, took 182 us that way and 128 to 138 on two cards this way (4.4 and 5.8 to 6.3 TB/s; 48 of 1024 keys
// 33 and 31); with a head's slots next to one another in the page 128 either way.
inline bool paged_tmap(CUtensorMap* m, const void* cache, const PagedShape& s, const FaStrides& t) {
  const int P = 1 << s.page_shift;
  return fa_make_tmap_bf16(m, cache, s.d, P, s.Hkv, s.num_pages, t.row, t.head, t.batch, P < 128 ? P : 128, 1, s.d > 64);
}

// The two copying warps of the chunk and key-weight kernels: at d = 128 each copies 64 columns of every page, at d = 64
// every other page (a lane per page either way), and the first warp Q.
template <int D>
struct CopyShare {
  int who;  // 0 or 1
  __device__ int column() const { return D == 128 ? who : 0; }  // in units of 64
  __device__ bool lane(int l, int pages) const { return l < pages && (D == 128 || (l & 1) == who); }
  __device__ int bytes(int pages, int rows) const {
    return (D == 128 ? pages : (pages + 1 - who) >> 1) * rows * 128;
  }
  __device__ bool copies_q() const { return who < D / 64; }
};

// How query rows lie in tiles: gs heads side by side for each of tpt tokens; Hv such groups of heads,
// per_kv of them per K/V head.
struct FastDiv {  // division of 0 <= n < 2^31 by a constant of the launch: n ceil(2^(31 + k) / d) >> (31 + k), 2^k >= d
  uint32_t mul, shift;
  __device__ int div(int n) const { return (int)(((unsigned long long)(uint32_t)n * mul) >> shift); }
};
inline FastDiv fast_div(int d) {
  uint32_t k = 0;
  while ((1 << k) < d) ++k;
  return {(uint32_t)(((1ull << (31 + k)) + d - 1) / d), 31 + k};
}
struct PagedRows {
  int gs, Hv, per_kv, tpt;
  FastDiv by_per_kv, by_tpt;
};
inline PagedRows paged_rows(int gs, int Hv, int per_kv, int tpt) {
  return {gs, Hv, per_kv, tpt, fast_div(per_kv), fast_div(tpt)};
}

// 128-row tiles: the divisor of the heads per K/V head that fills the rows best, the largest of equals
// (a K/V tile then serves more heads). It does not look at how many tokens there are: a few of a group that does not
// divide 128 take more tiles than they could (10 tokens of 7 heads: seven of one head each, where one would hold all).
inline PagedRows paged_rows_for(const PagedShape& s) {
  const int G = s.H / s.Hkv;
  int best = 1;
  for (int g = 1; g <= G && g <= 128; ++g)
    if (G % g == 0 && 128 / g * g >= 128 / best * best) best = g;
  return paged_rows(best, s.H / best, G / best, 128 / best);
}

// Up to 64 rows (tokens x heads of one K/V head) fit the few-row kernels: one tile of 16, 32 or 64
// columns per K/V head. Both sides at 64 rows, 8 K/V heads, d = 128: 16 sequences of 8192 keys 111 us in
// few-row tiles and 122 in 128-row tiles, 64 of 1000 keys 76 and 100 (d = 64: 78 and 106, 59 and 80); the key
// weights 50 and 87, 31 and 48. Four rows: 87 and 119, 51 and 99.
inline bool paged_few_rows(const PagedShape& s) { return (long long)s.Nq * (s.H / s.Hkv) <= 64; }

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
// A load from the shared memory of CTA `cta` of the cluster, at the address that `p` has there.
__device__ __forceinline__ int load_peer(const int* p, uint32_t cta) {
  uint32_t at;
  int x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(cta));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ float load_peer(const float* p, uint32_t cta) {
  return __int_as_float(load_peer(reinterpret_cast<const int*>(p), cta));
}
__device__ __forceinline__ float4 load_peer4(const float* p, uint32_t cta) {
  uint32_t at;
  float4 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(cta));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(at)
               : "memory");
  return x;
}

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// sum of floor((a i + b) / m) for 0 <= i < n, by Euclid's steps on (a, m), or without a division where both are powers
// of two (head counts that divide 128). The arguments and a n + b are positions of keys, tokens or tiles and fit
// 31 bits, so the divisions are 32-bit ones.
__device__ inline long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  if ((a & (a - 1)) == 0 && (m & (m - 1)) == 0) {
    const int x = 31 - __clz(m), y = 31 - __clz(a);
    const long long pairs = (long long)n * (n - 1) / 2;
    if (y >= x) return (pairs << (y - x)) + (long long)n * (b >> x);
    const int r = x - y;  // floor((a i + b) / m) = (i + b / a) >> r
    auto below = [r](long long e) {  // sum of j >> r for j < e
      const long long k = e >> r;
      return (k * (k - 1) / 2 << r) + k * (e - (k << r));
    };
    return below((long long)(b >> y) + n) - below(b >> y);
  }
  long long sum = 0;
  while (n > 0) {
    sum += (long long)n * (n - 1) / 2 * (a / m) + (long long)n * (b / m);
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    n = top / m;
    b = top % m;
    const uint32_t x = a;
    a = m;
    m = x;
    if (m == 0) break;
  }
  return sum;
}

// a / b of numbers >= 0: 64-bit divisions take a few hundred cycles, and those here mostly fit 32 bits.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int div_pos(int a, int b) { return (int)((uint32_t)a / (uint32_t)b); }

// A CTA's share of the work. Units (of key tiles, or of query tiles) stand in one line, ordered by
// sequence, head and unit; each is kOpen positions, which stand for the time a unit takes besides its
// tiles, and then a position per tile. Of `total` positions CTA c of n takes total / n, the first total % n
// CTAs one more. A share that begins inside a unit's first kOpen positions begins with its first tile; one
// that ends there has none of them. Pos counts positions: int where a caller has shown that they fit.
template <typename Pos>
struct ShareOf {
  int b, head, unit, tile;   // where the CTA begins
  Pos todo;                  // its positions, from there
  int first_cta, first_slot; // of the unit in which it begins: the CTA with its first tile, the slot of that piece
};
using Share = ShareOf<long long>;

template <typename Pos>
struct Division {
  Pos each, more;  // positions of a CTA; CTAs with one more
  __device__ Division(Pos total, Pos n) : each(div_pos(total, n)), more(total - each * n) {}
  __device__ Pos begin(Pos c) const { return each * c + min(c, more); }
  __device__ Pos cta(Pos at) const {
    const Pos wide = more * (each + 1);
    return at < wide ? div_pos(at, each + 1) : more + div_pos(at - wide, each);
  }
};

// Finds the share of CTA `cta` of `ctas`; all threads of the CTA take part, and `sh`, `scan` (an entry per
// warp) and `at` are in shared memory; `at` becomes the units of sequence sh.b where the share is not
// empty. Units, made by make(b): heads, count, before(u) (positions before unit u, one head's), tiles(u), and open,
// the positions of a unit before its first tile. Every kernel begins with this and can load nothing before it knows its
// share, so it counts in full: each sequence is looked at once, and few divisions are left. In 32 bits its loops are not
// unrolled (the 8-bit cache's kernel waits for its instructions); in 64 bits that is the compiler's choice (0: no pragma), which is ahead
// of four steps at a time: a mixed batch 124.4 us and 125.7, key weights of its chunks 51.7 and 52.2.
template <int kThreads, int kScan, typename Units, typename Make, typename Pos>
__device__ void find_share(int B, Make&& make, ShareOf<Pos>& sh, Pos (&scan)[kScan], Units& at, int cta = blockIdx.x,
                           int ctas = gridDim.x) {
  static_assert(kScan >= kThreads / 32 && kScan >= 2, "scan has an entry per warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = B <= kThreads ? 1 : (B + kThreads - 1) / kThreads, first = threadIdx.x * per, last = min(B, first + per);
  Units x;
  Pos size = 0, mine = 0;  // of the thread's first sequence (one head's), and of all of its
  if (first < last) {
    x = make(first);
    size = x.before(x.count);
    mine = size * x.heads;
    for (int b = first + 1; b < last; ++b) {
      const Units y = make(b);
      mine += y.before(y.count) * y.heads;
    }
  }
  const int warps = min(kThreads / 32, per == 1 ? (B + 31) >> 5 : kThreads / 32);  // that have sequences
  Pos inc = mine;
  if (warp < warps) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Pos y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) scan[warp] = inc;
  }
  if (threadIdx.x == 0) sh.todo = 0;
  __syncthreads();
  Pos base = inc - mine, total = 0;
#pragma unroll (sizeof(Pos) == 4 ? 1 : 0)
  for (int i = 0; i < warps; ++i) {
    if (i < warp) base += scan[i];
    total += scan[i];
  }
  __syncthreads();  // scan is read
  if (total == 0) return;
  const Pos n = min(total, (Pos)ctas), c = cta;  // no CTA before the last busy one is idle
  if (c >= n) return;
  const Division<Pos> cut(total, n);
  const Pos lo = cut.begin(c);
  if (lo >= base && lo < base + mine) {  // the sequence, and the line's position where it begins
    int b = first;
    while (lo >= base + size * x.heads) {
      base += size * x.heads;
      x = make(++b);
      size = x.before(x.count);
    }
    sh.b = b;
    at = x;
    scan[0] = base;
    scan[1] = size;
  }
  __syncthreads();
  const Pos from = scan[0];
  size = scan[1];
  const int head = (int)div_pos(lo - from, size);
  const Pos line = from + head * size;  // where the head's units begin
  const int count = at.count, open = at.open;
#pragma unroll (sizeof(Pos) == 4 ? 1 : 0)
  for (int u = threadIdx.x; u < count; u += kThreads) {
    const Pos start = line + at.before(u);
    if (start > lo || lo >= start + at.tiles(u) + open) continue;
    sh.head = head;
    sh.unit = u;
    sh.tile = (int)(lo - start);
    sh.todo = cut.begin(c + 1) - lo;
    const Pos c0 = cut.cta(start + open);
    sh.first_cta = (int)c0;
    sh.first_slot = 2 * (int)c0 + (cut.begin(c0) >= start ? 0 : 1);
  }
  __syncthreads();
}

}  // namespace fa

struct FaPagedArgs {
  fa::PagedShape s;
  const void* q;
  void *k, *v;  // the caches
  void* o;
  float* lse;
  FaStrides sq, sk, sv, so;
  const void *k_new, *v_new;  // append
  void *k_out, *v_out;        // reading back
  FaStrides sk_new, sv_new;   // of either
  uint8_t* codes;             // of an 8-bit cache, [num_pages][Hkv][page_size][2]
  float* weights;
  float scale;
  int* status;
  int num_sms;      // CTAs the attention's work is divided among
  void* workspace;
  int keep, recent;  // evict
  int32_t *kept, *seqlens_out;
};

// Attention of few rows (paged_few_rows) and of more, with the workspace each needs.
size_t fa_paged_decode_workspace(const fa::PagedShape& s, int num_sms);
cudaError_t fa_launch_paged_decode(const FaPagedArgs& a, cudaStream_t st);
size_t fa_paged_chunk_workspace(const fa::PagedShape& s, int num_sms);
cudaError_t fa_launch_paged_chunk(const FaPagedArgs& a, cudaStream_t st);
namespace fa {

// Joins the partials (normalised O and LSE in log2 units, in slots of ROWS rows) that CTAs c0 .. c1 left of
// one row, for its elements [e, e + 4): M = max LSE, w = 2^(LSE - M), O = sum w O / sum w, LSE = M + log2
// sum w. CTA c0's lie in slot0, those of a later CTA c in slot 2 c. Eight pieces are in flight at a time.
template <int D, int ROWS>
__device__ __forceinline__ void join_pieces(const FaPagedArgs& a, const float* part_o, const float* part_lse, int c0,
                                            int c1, int slot0, int row, int e, const SeqInfo& seq, int b, int i,
                                            int h) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, sum = 0.f;
  for (int c = c0; c <= c1; c += 8) {
    float l[8];
    float4 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const size_t at = (size_t)(c + k == c0 ? slot0 : 2 * (c + k)) * ROWS + row;
      const bool there = c + k <= c1;
      l[k] = there ? part_lse[at] : -INFINITY;
      o[k] = there ? *reinterpret_cast<const float4*>(part_o + at * D + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = M;
    bool any = false;  // a piece with a visible key, or with NaN (which no maximum shows)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      top = fmaxf(top, l[k]);
      any |= l[k] != -INFINITY;
    }
    if (!any) continue;
    const float alpha = exp2f(M - top);
    acc = make_float4(acc.x * alpha, acc.y * alpha, acc.z * alpha, acc.w * alpha);
    sum *= alpha;
    M = top;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = exp2f(l[k] - M);
      sum += w;
      acc.x += w * o[k].x;
      acc.y += w * o[k].y;
      acc.z += w * o[k].z;
      acc.w += w * o[k].w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.o) + elem_offset(a.so, seq.bb, seq.q0 + i, h) + e) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (e == 0) a.lse[paged_row(a.s, seq, b, h, i)] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

}  // namespace fa

cudaError_t fa_launch_paged_append(const FaPagedArgs& a, cudaStream_t st);
size_t fa_paged_weights_workspace(const fa::PagedShape& s, int num_sms);
cudaError_t fa_launch_paged_key_weights(const FaPagedArgs& a, cudaStream_t st);
cudaError_t fa_launch_paged_evict(const FaPagedArgs& a, cudaStream_t st);
// The cache held in 8 bits: append, reading rows back, and the attention with its workspace.
cudaError_t fa_launch_paged_append_fp8(const FaPagedArgs& a, cudaStream_t st);
cudaError_t fa_launch_paged_read_fp8(const FaPagedArgs& a, cudaStream_t st);
// Attention by the kernel that reads the bytes as they lie, in units of `tokens` new tokens (tokens x grouped heads up to
// 64): the tokens of a unit for which it takes the whole batch, or 0 where there are too many rows.
int fa_paged_few8_tokens(const fa::PagedShape& s);
size_t fa_paged_few8_workspace(const fa::PagedShape& s, int tokens, int num_sms);
cudaError_t fa_launch_paged_few8(const FaPagedArgs& a, int tokens, cudaStream_t st);
size_t fa_paged_fp8_workspace(const fa::PagedShape& s, int num_sms);
cudaError_t fa_launch_paged_fp8(const FaPagedArgs& a, cudaStream_t st);
