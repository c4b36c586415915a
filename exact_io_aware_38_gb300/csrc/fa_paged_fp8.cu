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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

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

// Append: one warp per new token, its keys and values both; 16 values a lane and two such chunks of each in flight.
template <int D>
__global__ void __launch_bounds__(128) paged_append_fp8_kernel(const FaPagedArgs a) {
  let_dependent_start();
  grid_dependency_wait();
  constexpr int kLanes = D / 16;  // that share a head's row
  const PagedShape& s = a.s;
  const int lane = threadIdx.x & 31;
  const uint32_t row = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
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
  const uint8_t* src[2] = {
      reinterpret_cast<const uint8_t*>(a.k_new) + 2 * elem_offset(a.sk_new, seq.bb, seq.q0 + i, 0),
      reinterpret_cast<const uint8_t*>(a.v_new) + 2 * elem_offset(a.sv_new, seq.bb, seq.q0 + i, 0)};
  const long long head[2] = {2 * a.sk_new.head, 2 * a.sv_new.head};
  const int chunks = s.Hkv * kLanes;
  uint4 x[2][2][2];  // [tensor][chunk][half]
  auto load = [&](int c0) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = c0 + k * 32 + lane;
        if (c < chunks) {
          const uint4* at = reinterpret_cast<const uint4*>(src[t] + (c / kLanes) * head[t]) + (c % kLanes) * 2;
          x[t][k][0] = at[0];
          x[t][k][1] = at[1];
        } else {
          x[t][k][0] = x[t][k][1] = make_uint4(0, 0, 0, 0);
        }
      }
  };
  load(0);  // on its way while the page is looked up
  const int page = paged_page(s, b, (int)(j >> s.page_shift), a.status);
  if (page < 0) return;
  const int slot = (int)(j & ((1 << s.page_shift) - 1));
  uint8_t* dst[2] = {static_cast<uint8_t*>(a.k) + paged_offset(a.sk, page, slot, 0),
                     static_cast<uint8_t*>(a.v) + paged_offset(a.sv, page, slot, 0)};
  const long long to[2] = {a.sk.head, a.sv.head};
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    if (c0 > 0) load(c0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = c0 + k * 32 + lane;
      uint32_t code[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint4 p = x[t][k][0], q = x[t][k][1];
        uint32_t m = 0;  // magnitudes of two values in each word: bf16 bits without the sign are ordered as integers
        for (uint32_t w : {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}) m = max_u16x2(m, w & 0x7fff7fffu);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
        code[t] = row_code(max(m & 0xffffu, m >> 16));
        const float by = code[t] == 0 || code[t] == 255 ? 0.f : __uint_as_float((254 - code[t]) << 23);
        const uint2 lo = quantised8(p, by), hi = quantised8(q, by);
        if (c < chunks)
          *reinterpret_cast<uint4*>(dst[t] + (c / kLanes) * to[t] + (c % kLanes) * 16) =
              make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
      if (c < chunks && c % kLanes == 0)
        *reinterpret_cast<uint16_t*>(a.codes + 2 * weight_offset(s, page, c / kLanes, slot)) =
            (uint16_t)(code[0] | code[1] << 8);
    }
  }
}

// 16 e4m3 bytes times 2^(code - 127) as 16 bf16 values, each exact: f16 holds every e4m3 number.
__device__ __forceinline__ void read16(uint4 y, uint32_t code, uint4 (&out)[2]) {
  const float by = code == 255 ? NAN : __uint_as_float(code << 23);
  const uint32_t w[4] = {y.x, y.y, y.z, y.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t two = (uint16_t)(w[i >> 1] >> ((i & 1) * 16));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    r[i] = pack_bf16x2(f.x * by, f.y * by);
  }
  out[0] = make_uint4(r[0], r[1], r[2], r[3]);
  out[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// One key and value of the cache as rows of bf16, by a warp: 16 values a lane. kJoint: for the attention, where a value of
// NaN would reach rows that do not see it (0 times NaN): its key becomes NaN, which only rows that see it look at, and the value 0.
template <int D, bool kJoint>
__device__ __forceinline__ void read_row(const FaPagedArgs& a, int page, int slot, __nv_bfloat16* k, long long k_head,
                                         __nv_bfloat16* v, long long v_head) {
  constexpr int kLanes = D / 16;
  const PagedShape& s = a.s;
  const int lane = threadIdx.x & 31, chunks = s.Hkv * kLanes;
  const uint8_t* src[2] = {static_cast<const uint8_t*>(a.k) + paged_offset(a.sk, page, slot, 0),
                           static_cast<const uint8_t*>(a.v) + paged_offset(a.sv, page, slot, 0)};
  const long long from[2] = {a.sk.head, a.sv.head}, to[2] = {k_head, v_head};
  __nv_bfloat16* dst[2] = {k, v};
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    uint4 y[2][2];
    uint32_t codes[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int c = c0 + n * 32 + lane;
      if (c >= chunks) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        y[t][n] = *reinterpret_cast<const uint4*>(src[t] + (c / kLanes) * from[t] + (c % kLanes) * 16);
      codes[n] = *reinterpret_cast<const uint16_t*>(a.codes + 2 * weight_offset(s, page, c / kLanes, slot));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int c = c0 + n * 32 + lane;
      if (c >= chunks) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint4 out[2];
        uint32_t code = (codes[n] >> (8 * t)) & 255u;
        if (kJoint) code = t == 0 && (codes[n] >> 8) == 255u ? 255u : t == 1 && code == 255u ? 0u : code;
        read16(y[t][n], code, out);
        uint4* at = reinterpret_cast<uint4*>(dst[t] + (c / kLanes) * to[t] + (c % kLanes) * 16);
        at[0] = out[0];
        at[1] = out[1];
      }
    }
  }
}

// Reading the last L_q keys of each sequence: one warp per row.
template <int D>
__global__ void __launch_bounds__(128) paged_read_fp8_kernel(const FaPagedArgs a) {
  let_dependent_start();
  grid_dependency_wait();
  const PagedShape& s = a.s;
  const int lane = threadIdx.x & 31;
  const uint32_t row = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
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
  const long long j = (long long)s.seqlens[b] - seq.Lq + i;
  if (j < 0 || (j >> s.page_shift) >= s.max_pages) {
    if (lane == 0) report_status(a.status, FA_ERR_BOUNDS);
    return;
  }
  const int page = paged_page(s, b, (int)(j >> s.page_shift), a.status);
  if (page < 0) return;
  read_row<D, false>(a, page, (int)(j & ((1 << s.page_shift) - 1)),
              static_cast<__nv_bfloat16*>(a.k_out) + elem_offset(a.sk_new, seq.bb, seq.q0 + i, 0), a.sk_new.head,
              static_cast<__nv_bfloat16*>(a.v_out) + elem_offset(a.sv_new, seq.bb, seq.q0 + i, 0), a.sv_new.head);
}

// Reading all keys of every sequence into a cache of its own, in pages of 128 keys [page][head][slot][d], `tiles` of them
// a sequence, and that cache's page table.
struct Staged {
  __nv_bfloat16 *k, *v;
  int32_t* table;
  int tiles;
};

template <int D>
__global__ void __launch_bounds__(256) paged_stage_fp8_kernel(const FaPagedArgs a, const Staged to) {
  let_dependent_start();
  grid_dependency_wait();
  const PagedShape& s = a.s;
  const int at = blockIdx.x * blockDim.x + threadIdx.x, threads = gridDim.x * blockDim.x;
  for (int i = at; i < s.B * to.tiles; i += threads) to.table[i] = i;
  const int warps = threads >> 5;
  for (int b = 0; b < s.B; ++b) {
    const SeqInfo seq = paged_seq(s, b);
    if (seq.Lq == 0) continue;
    for (int j = at >> 5; j < seq.Lk; j += warps) {
      const int page = paged_page(s, b, j >> s.page_shift, a.status);
      if (page < 0) continue;
      const size_t row = ((size_t)(b * to.tiles + (j >> 7)) * s.Hkv * 128 + (j & 127)) * D;
      read_row<D, true>(a, page, j & ((1 << s.page_shift) - 1), to.k + row, 128 * D, to.v + row, 128 * D);
    }
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
  p.attend = up256(paged_few_rows(t) ? fa_paged_decode_workspace(t, num_sms) : fa_paged_chunk_workspace(t, num_sms));
  return p;
}

unsigned row_blocks(const PagedShape& s) {  // a warp per row, four to a block
  const long long rows = s.cu_q != nullptr ? s.rows_q : (long long)s.B * s.Nq;
  return (unsigned)((rows + 3) / 4);
}

}  // namespace
}  // namespace fa

cudaError_t fa_launch_paged_append_fp8(const FaPagedArgs& a, cudaStream_t st) {
  const dim3 grid(fa::row_blocks(a.s)), block(128);
  return a.s.d == 64 ? launch_dependent(fa::paged_append_fp8_kernel<64>, grid, block, 0, st, a)
                     : launch_dependent(fa::paged_append_fp8_kernel<128>, grid, block, 0, st, a);
}

cudaError_t fa_launch_paged_read_fp8(const FaPagedArgs& a, cudaStream_t st) {
  const dim3 grid(fa::row_blocks(a.s)), block(128);
  return a.s.d == 64 ? launch_dependent(fa::paged_read_fp8_kernel<64>, grid, block, 0, st, a)
                     : launch_dependent(fa::paged_read_fp8_kernel<128>, grid, block, 0, st, a);
}

size_t fa_paged_fp8_workspace(const fa::PagedShape& s, int num_sms) {
  return fa_paged_few8(s) ? fa_paged_few8_workspace(s, num_sms) : fa::stage_plan(s, num_sms).bytes();
}

cudaError_t fa_launch_paged_fp8(const FaPagedArgs& a, cudaStream_t st) {
  const fa::PagedShape& s = a.s;
  if (fa_paged_few8(s)) return fa_launch_paged_few8(a, st);
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
    const dim3 grid(a.num_sms * 8), block(256);
    cudaError_t e = s.d == 64 ? launch_dependent(fa::paged_stage_fp8_kernel<64>, grid, block, 0, st, x, to)
                              : launch_dependent(fa::paged_stage_fp8_kernel<128>, grid, block, 0, st, x, to);
    if (e != cudaSuccess) return e;
    x.s = fa::staged_shape(x.s, group, plan.tiles);
    x.s.table = to.table;
    x.k = to.k;
    x.v = to.v;
    x.sk.row = s.d;
    x.sk.head = 128ll * s.d;
    x.sk.batch = 128ll * s.d * s.Hkv;
    x.sv = x.sk;
    e = fa::paged_few_rows(x.s) ? fa_launch_paged_decode(x, st) : fa_launch_paged_chunk(x, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
