// The paged cache held in 8 bits: rows written as e4m3 numbers with an exponent each, rows read back in bf16, and the
// attention of many rows by way of read-back keys and values.
//
// A row x of d values becomes y = rn_e4m3(x 2^(127 - code)) with code = floor(log2 max|x|) - 7 + 127: the largest number lies in
// [128, 256], well inside e4m3's 448, and those 2^-13 below it are still normal. A power of two costs e4m3 nothing (its
// precision is relative) and keeps y 2^(code - 127) a bf16 number, so reading back is exact and the cache stands for one set
// of bf16 rows whoever reads it.
#include <cuda_fp16.h>

#include "fa_paged.cuh"

namespace fa {
namespace {

// The code of a row whose largest magnitude has these bf16 bits.
__device__ __forceinline__ uint32_t row_code(uint32_t top) {
  return top == 0 ? 0u : top >= 0x7f80u ? 255u : (top >> 7) < 54 ? 47u : (top >> 7) - 7u;
}

// Eight values (16 bytes of bf16) times `by` as eight e4m3 bytes; bytes 0 where by is 0.
__device__ __forceinline__ uint2 quantised8(uint4 x, float by) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(y)
        : "f"(__uint_as_float(w[i] & 0xffff0000u) * by), "f"(__uint_as_float(w[i] << 16) * by));
    r[i] = by == 0.f ? 0u : y;
  }
  return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}

// Eight e4m3 bytes times 2^(code - 127) as eight bf16 values, each exact: f16 holds every e4m3 number.
__device__ __forceinline__ uint4 read8(uint2 y, uint32_t code) {
  const float by = code == 255 ? NAN : __uint_as_float(code << 23);
  const uint32_t w[2] = {y.x, y.y};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i >> 1] >> ((i & 1) * 16))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    r[i] = pack_bf16x2(f.x * by, f.y * by);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

constexpr int kRowThreads = 64;  // (of a block, appending 64 tokens: 2.3 us; 128: 2.4, 256: 2.7)

// Both ways move kRows rows per warp, keys and values: one, all of 8 heads at d = 128 in flight at once, or as many of fewer
// heads (400000 rows of one head, d = 64, written and read: 29 and 29 us, one per warp 203 and 202). Where the rows are a warp
// each, or a few, one is less to look up: 4096 packed ones of one head, each a sequence, take 5 us, 4 or 8 a warp 6.
int rows_per_warp(const PagedShape& s, long long rows) {
  const int most = 1024 / (s.Hkv * s.d);
  return rows < (s.cu_q != nullptr ? 8192 : 2048) || most < 2 ? 1 : most < 4 ? 2 : most < 8 ? 4 : 8;
}

// Which key of which sequence this lane's row is, of the warp's rows from `first` on (packed or fixed), by the whole warp:
// false where it has no place (reported where it should).
struct Place {
  int b, key;
  int row, batch;  // in the tensors of new tokens
};
template <int kRows>
__device__ __forceinline__ bool find_place(const PagedShape& s, uint32_t first, int* status, Place& at) {
  const uint32_t own = (threadIdx.x & 31) / (32 / kRows), row = first + own;
  int b, i = 0;
  if (s.cu_q != nullptr) {
    if (first >= (uint32_t)s.rows_q) return false;
    b = sequence_of(s, (int)first);
    if (kRows > 1 && (b >= s.B || s.cu_q[b + 1] < (int)first + kRows)) {
#pragma unroll 1
      for (int n = 1; n < kRows; ++n) {
        const int of = sequence_of(s, (int)first + n);
        if (n == own) b = of;
      }
    }
    if (row >= (uint32_t)s.rows_q) return false;
  } else {
    b = (int)(row / (uint32_t)s.Nq);
    i = (int)(row % (uint32_t)s.Nq);
  }
  if (b >= s.B) return false;
  const SeqInfo seq = paged_seq(s, b);
  if (s.cu_q != nullptr) i = (int)row - seq.q0;
  if (i < 0 || i >= seq.Lq) return false;
  const long long j = (long long)s.seqlens[b] - seq.Lq + i;  // the unclamped length places the token
  if (j < 0 || (j >> s.page_shift) >= s.max_pages) {
    report_status(status, FA_ERR_BOUNDS);
    return false;
  }
  at = Place{b, (int)j, seq.q0 + i, seq.bb};
  return true;
}

// Append: bound by memory, 6 bytes a value (a row of 8 heads is read and written by one warp). 16 values a lane here: a row's
// largest takes one exchange less (64 tokens of 8 heads, d = 128, 2.4 us, with 8 values 3.0; 16388 tokens 18.7 and 20.8).
template <int D, int kRows>
__global__ void __launch_bounds__(kRowThreads) paged_append_fp8_kernel(const FaPagedArgs a) {
  let_dependent_start();
  grid_dependency_wait();
  constexpr int kLanes = D / 16, kWide = 32 / kRows;  // lanes of a head's row, of a row
  const PagedShape& s = a.s;
  const int lane = threadIdx.x % kWide, chunks = s.Hkv * kLanes;
  Place at{};
  const bool placed = find_place<kRows>(s, ((blockIdx.x * blockDim.x + threadIdx.x) >> 5) * kRows, a.status, at);
  if (kRows == 1 && !placed) return;
  const __nv_bfloat16* src[2] = {
      static_cast<const __nv_bfloat16*>(a.k_new) + elem_offset(a.sk_new, at.batch, at.row, 0) + lane % kLanes * 16,
      static_cast<const __nv_bfloat16*>(a.v_new) + elem_offset(a.sv_new, at.batch, at.row, 0) + lane % kLanes * 16};
  const long long from[2] = {a.sk_new.head, a.sv_new.head}, to[2] = {a.sk.head, a.sv.head};
  uint4 x[2][2][2];  // [tensor][step][half]
  auto load = [&](int c0) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint4* p = reinterpret_cast<const uint4*>(src[t] + (c0 + kWide * k) / kLanes * from[t]);
        x[t][k][0] = x[t][k][1] = make_uint4(0, 0, 0, 0);
        if ((kRows == 1 || placed) && c0 + kWide * k < chunks) {
          x[t][k][0] = p[0];
          x[t][k][1] = p[1];
        }
      }
  };
  load(lane);  // on its way while the page is looked up
  const int page = kRows == 1 || placed ? paged_page(s, at.b, at.key >> s.page_shift, a.status) : -1;
  const int slot = at.key & ((1 << s.page_shift) - 1);
  if (kRows == 1 && page < 0) return;
  uint8_t* dst[2] = {static_cast<uint8_t*>(a.k) + paged_offset(a.sk, page, slot, 0) + lane % kLanes * 16,
                     static_cast<uint8_t*>(a.v) + paged_offset(a.sv, page, slot, 0) + lane % kLanes * 16};
  for (int c0 = lane; c0 < chunks + lane; c0 += 2 * kWide) {
    if (c0 > lane) load(c0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = c0 + kWide * k, h = c / kLanes;
      const bool mine = c < chunks && page >= 0;
      if (c - lane >= chunks) break;  // (by whole warps)
      uint32_t code[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint4 p = x[t][k][0], q = x[t][k][1];
        uint32_t m = 0;  // magnitudes of two values in each word: bf16 bits without the sign are ordered as integers
        for (uint32_t w : {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}) m = __vmaxu2(m, w & 0x7fff7fffu);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        code[t] = row_code(max(m & 0xffffu, m >> 16));
        const float by = code[t] == 0 || code[t] == 255 ? 0.f : __uint_as_float((254 - code[t]) << 23);
        const uint2 lo = quantised8(p, by), hi = quantised8(q, by);
        if (mine) *reinterpret_cast<uint4*>(dst[t] + h * to[t]) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
      if (mine && c % kLanes == 0)
        *reinterpret_cast<uint16_t*>(a.codes + 2 * weight_offset(s, page, h, slot)) = (uint16_t)(code[0] | code[1] << 8);
    }
  }
}

// One key and value of the cache as rows of bf16, by a warp or kWide lanes of it, 8 values a lane: every store of the warp is then whole lines
// (57345 rows of 8 heads 36.5 us, 6.2 TB/s; with 16 values 44.4). kJoint: for the attention, where a value of NaN would reach rows
// that do not see it (0 times NaN): its key becomes NaN, which only rows that see it look at, and the value 0.
template <int D, int kWide, bool kJoint>
__device__ __forceinline__ void read_row(const FaPagedArgs& a, int page, int slot, __nv_bfloat16* k, long long k_head,
                                         __nv_bfloat16* v, long long v_head) {
  constexpr int kLanes = D / 8, kSteps = 4;  // steps in flight
  const PagedShape& s = a.s;
  const int lane = threadIdx.x % kWide, chunks = s.Hkv * kLanes;
  const uint8_t* src[2] = {static_cast<const uint8_t*>(a.k) + paged_offset(a.sk, page, slot, 0),
                           static_cast<const uint8_t*>(a.v) + paged_offset(a.sv, page, slot, 0)};
  const uint8_t* codes = a.codes + 2 * weight_offset(s, page, 0, slot);
  const long long from[2] = {a.sk.head, a.sv.head}, to[2] = {k_head, v_head};
  __nv_bfloat16* dst[2] = {k, v};
  for (int c0 = lane; c0 < chunks; c0 += kWide * kSteps) {
    uint2 y[2][kSteps];
    uint32_t both[kSteps];
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      const int h = (c0 + kWide * n) / kLanes, at = (kWide % kLanes ? c0 + kWide * n : lane) % kLanes * 8;
      if (c0 + kWide * n >= chunks) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) y[t][n] = *reinterpret_cast<const uint2*>(src[t] + h * from[t] + at);
      both[n] = *reinterpret_cast<const uint16_t*>(codes + ((size_t)h << s.page_shift) * 2);
    }
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      const int h = (c0 + kWide * n) / kLanes, at = (kWide % kLanes ? c0 + kWide * n : lane) % kLanes * 8;
      if (c0 + kWide * n >= chunks) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t code = (both[n] >> (8 * t)) & 255u;
        if (kJoint) code = t == 0 && (both[n] >> 8) == 255u ? 255u : t == 1 && code == 255u ? 0u : code;
        *reinterpret_cast<uint4*>(dst[t] + h * to[t] + at) = read8(y[t][n], code);
      }
    }
  }
}

// Reading the last L_q keys of each sequence.
template <int D, int kRows>
__global__ void __launch_bounds__(kRowThreads) paged_read_fp8_kernel(const FaPagedArgs a) {
  let_dependent_start();
  grid_dependency_wait();
  Place at;
  if (!find_place<kRows>(a.s, ((blockIdx.x * blockDim.x + threadIdx.x) >> 5) * kRows, a.status, at)) return;
  const int page = paged_page(a.s, at.b, at.key >> a.s.page_shift, a.status);
  if (page < 0) return;
  read_row<D, 32 / kRows, false>(a, page, at.key & ((1 << a.s.page_shift) - 1),
                     static_cast<__nv_bfloat16*>(a.k_out) + elem_offset(a.sk_new, at.batch, at.row, 0), a.sk_new.head,
                     static_cast<__nv_bfloat16*>(a.v_out) + elem_offset(a.sv_new, at.batch, at.row, 0), a.sv_new.head);
}

// Reading all keys of every sequence into a cache of its own, in pages of 128 keys [page][head][slot][d], `tiles` of them
// a sequence, and that cache's page table. A warp per key, or per kRows keys of few heads, counted on over the sequences;
// looking at the sequences one by one, 2048 of 256 keys of one head, d = 64, took 1190 us with the attention, 32 at a time 278,
// with eight keys a warp 166.
struct Staged {
  __nv_bfloat16 *k, *v;
  int32_t* table;
  int tiles;
};

template <int D, int kRows>
__global__ void __launch_bounds__(256) paged_stage_fp8_kernel(const FaPagedArgs a, const Staged to) {
  let_dependent_start();
  grid_dependency_wait();
  const PagedShape& s = a.s;
  const int at = blockIdx.x * blockDim.x + threadIdx.x, threads = gridDim.x * blockDim.x;
  for (int i = at; i < s.B * to.tiles; i += threads) to.table[i] = i;
  const int lane = threadIdx.x & 31;
  auto keys_of = [&](int b) {
    if (b >= s.B) return 0;
    const SeqInfo seq = paged_part(s, b);
    return seq.Lq > 0 ? seq.Lk : 0;
  };
  // A lane's keys (all the warp's, or one of its kRows), counted from the first sequence of the 32 (or 256) that the warp looks
  // at: a lane has one each (or eight, whose loads are in flight together, where none of the 256 may concern the warp).
  const int step = (threads >> 5) * kRows;
  for (int b0 = 0, j = at / (32 / kRows); b0 < s.B; b0 += 32) {
    if (s.B - b0 > 64 && b0 % 256 == 0) {
      int sum = 0;
#pragma unroll
      for (int n = 0; n < 8; ++n) sum += keys_of(b0 + 32 * n + lane);
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (__all_sync(0xffffffffu, j >= sum)) {
        j -= sum;
        b0 += 256 - 32;
        continue;
      }
    }
    int end = keys_of(b0 + lane);  // (the sum of all lengths fits an int)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += up;
    }
    const int total = __shfl_sync(0xffffffffu, end, 31);
    while (__any_sync(0xffffffffu, j < total)) {
      int of = 0;  // sequences that end at or before j
      if (kRows == 1) {
        of = __popc(__ballot_sync(0xffffffffu, end <= j));
      } else {
#pragma unroll
        for (int n = 16; n > 0; n >>= 1)
          if (__shfl_sync(0xffffffffu, end, of + n - 1) <= j) of += n;
      }
      const int before = __shfl_sync(0xffffffffu, end, max(of - 1, 0));
      if (j >= total) continue;
      const int b = b0 + of, key = of == 0 ? j : j - before;
      j += step;
      const int page = paged_page(s, b, key >> s.page_shift, a.status);
      if (page < 0) continue;
      const size_t row = ((size_t)(b * to.tiles + (key >> 7)) * s.Hkv * 128 + (key & 127)) * D;
      read_row<D, 32 / kRows, true>(a, page, key & ((1 << s.page_shift) - 1), to.k + row, 128 * D, to.v + row, 128 * D);
    }
    j -= total;
  }
}

// Sequences whose keys and values are read back at a time: as many as fit 1 GiB, at least one. More sequences take
// several rounds through the same workspace.
constexpr size_t kStageBytes = (size_t)1 << 30;

struct StagePlan {
  int group, tiles;
  size_t attend, table, tensor;  // bytes of the attention's workspace, of the page table, and of K or V
  size_t bytes() const { return attend + table + 2 * tensor; }
};

PagedShape staged_shape(const PagedShape& s, int group, int tiles) {
  PagedShape t = s;
  t.B = group;
  t.page_shift = 7;
  t.num_pages = group * tiles;
  t.max_pages = tiles;
  return t;
}

StagePlan stage_plan(const PagedShape& s, int num_sms) {
  StagePlan p;
  p.tiles = (s.max_k + 127) >> 7;
  const size_t one = (size_t)p.tiles * 128 * s.Hkv * s.d * sizeof(__nv_bfloat16);
  const size_t fit = kStageBytes / (2 * one);
  p.group = fit < 1 ? 1 : fit < (size_t)s.B ? (int)fit : s.B;
  p.table = up256((size_t)p.group * p.tiles * sizeof(int32_t));
  p.tensor = up256(p.group * one);
  const PagedShape t = staged_shape(s, p.group, p.tiles);
  p.attend = up256(fa_paged_chunk_workspace(t, num_sms));
  return p;
}

// A packed batch whose sequences are of different lengths may hold prompts beside single tokens, and a token's keys are not
// read back for it alone: sequences of up to four units of 16 rows (of more than 64 heads of a K/V head: as many as go this
// way alone) go to the few-row kernel. What the host knows is the sum of the new tokens' lengths, and bounds. The further launches
// take 15 to 20 us, which few or short sequences do not give back: 6 sequences up to 6001 keys, two of them of one token,
// 163 us apart and 156 together, 12 up to 4000 of 12 heads, d = 64, 131 and 132; 33 up to 8000 606 and 679.
struct Apart {
  int unit, most;  // tokens of a unit, and of a sequence that goes this way: 0 where all sequences go one way
};

Apart apart_tokens(const PagedShape& s) {
  const int G = s.H / s.Hkv;
  if (s.cu_q == nullptr || G > 256 || s.rows_q * 4ll > 3ll * s.B * s.Nq) return {};
  if ((double)s.B * s.max_k * s.Hkv * s.d < (double)(1 << 26)) return {};
  if (G > 64) return {1, 4 / ((G + 63) / 64)};
  const int unit = G <= 16 ? 16 / G : 1;
  return {unit, 4 * unit};
}

// Appending (16 values a lane) or reading, a warp per kRows rows.
template <int D, int kRows, bool kAppend>
cudaError_t launch_rows(const FaPagedArgs& a, cudaStream_t st) {
  const long long rows = a.s.cu_q != nullptr ? a.s.rows_q : (long long)a.s.B * a.s.Nq, warps = (rows + kRows - 1) / kRows;
  const dim3 grid((unsigned)((warps * 32 + kRowThreads - 1) / kRowThreads)), block(kRowThreads);
  if constexpr (kAppend) return launch_dependent(paged_append_fp8_kernel<D, kRows>, grid, block, 0, st, a);
  else return launch_dependent(paged_read_fp8_kernel<D, kRows>, grid, block, 0, st, a);
}

template <int D, bool kAppend>
cudaError_t launch_rows(const FaPagedArgs& a, cudaStream_t st) {
  const long long rows = a.s.cu_q != nullptr ? a.s.rows_q : (long long)a.s.B * a.s.Nq;
  switch (rows_per_warp(a.s, rows)) {
    case 8:
      if constexpr (!kAppend || D == 64) return launch_rows<D, 8, kAppend>(a, st);  // (two lanes have no row of 128 to append)
    case 4: return launch_rows<D, 4, kAppend>(a, st);
    case 2: return launch_rows<D, 2, kAppend>(a, st);
    default: return launch_rows<D, 1, kAppend>(a, st);
  }
}

template <int D>
cudaError_t launch_stage(const FaPagedArgs& a, const Staged& to, cudaStream_t st) {
  const dim3 grid(a.num_sms * 8), block(256);
  switch (rows_per_warp(a.s, (long long)a.s.B * a.s.max_k)) {
    case 8: return launch_dependent(paged_stage_fp8_kernel<D, 8>, grid, block, 0, st, a, to);
    case 4: return launch_dependent(paged_stage_fp8_kernel<D, 4>, grid, block, 0, st, a, to);
    case 2: return launch_dependent(paged_stage_fp8_kernel<D, 2>, grid, block, 0, st, a, to);
    default: return launch_dependent(paged_stage_fp8_kernel<D, 1>, grid, block, 0, st, a, to);
  }
}

}  // namespace
}  // namespace fa

cudaError_t fa_launch_paged_append_fp8(const FaPagedArgs& a, cudaStream_t st) {
  return a.s.d == 64 ? fa::launch_rows<64, true>(a, st) : fa::launch_rows<128, true>(a, st);
}

cudaError_t fa_launch_paged_read_fp8(const FaPagedArgs& a, cudaStream_t st) {
  return a.s.d == 64 ? fa::launch_rows<64, false>(a, st) : fa::launch_rows<128, false>(a, st);
}

size_t fa_paged_fp8_workspace(const fa::PagedShape& s, int num_sms) {
  if (const int tokens = fa_paged_few8_tokens(s)) return fa_paged_few8_workspace(s, tokens, num_sms);
  const fa::Apart apart = fa::apart_tokens(s);
  const size_t few = apart.most > 0 ? fa_paged_few8_workspace(s, apart.unit, num_sms) : 0, staged = fa::stage_plan(s, num_sms).bytes();
  return few > staged ? few : staged;
}

cudaError_t fa_launch_paged_fp8(const FaPagedArgs& a, cudaStream_t st) {
  if (const int tokens = fa_paged_few8_tokens(a.s)) return fa_launch_paged_few8(a, tokens, st);
  fa::PagedShape s = a.s;
  if (const fa::Apart apart = fa::apart_tokens(s); apart.most > 0) {
    FaPagedArgs x = a;
    x.s.max_q = apart.most;
    const cudaError_t e = fa_launch_paged_few8(x, apart.unit, st);
    if (e != cudaSuccess) return e;
    s.min_q = apart.most + 1;
  }
  const fa::StagePlan plan = fa::stage_plan(s, a.num_sms);
  char* ws = static_cast<char*>(a.workspace);
  fa::Staged to;
  to.table = reinterpret_cast<int32_t*>(ws + plan.attend);
  to.k = reinterpret_cast<__nv_bfloat16*>(ws + plan.attend + plan.table);
  to.v = reinterpret_cast<__nv_bfloat16*>(ws + plan.attend + plan.table + plan.tensor);
  to.tiles = plan.tiles;
  for (int b = 0; b < s.B; b += plan.group) {
    const int group = s.B - b < plan.group ? s.B - b : plan.group;
    FaPagedArgs x = a;  // the sequences [b, b + group)
    x.s = s;
    x.s.B = group;
    x.s.table += (size_t)b * s.max_pages;
    x.s.seqlens += b;
    if (s.cu_q != nullptr) {
      x.s.cu_q += b;
    } else {
      x.q = static_cast<const __nv_bfloat16*>(a.q) + (size_t)b * a.sq.batch;
      x.o = static_cast<__nv_bfloat16*>(a.o) + (size_t)b * a.so.batch;
      x.lse += (size_t)b * s.H * s.Nq;
    }
    cudaError_t e = s.d == 64 ? fa::launch_stage<64>(x, to, st) : fa::launch_stage<128>(x, to, st);
    if (e != cudaSuccess) return e;
    x.s = fa::staged_shape(x.s, group, plan.tiles);
    x.s.table = to.table;
    x.k = to.k;
    x.v = to.v;
    x.sk.row = s.d;
    x.sk.head = 128ll * s.d;
    x.sk.batch = 128ll * s.d * s.Hkv;
    x.sv = x.sk;
    e = fa_launch_paged_chunk(x, st);  // (what comes this way has more than 64 rows)
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
