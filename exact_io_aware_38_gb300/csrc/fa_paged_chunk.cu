// Attention of chunks of new tokens over a paged cache: more rows per K/V head than the few-row
// kernel takes, so the pass is bound by the tensor cores (and by the exponentials beside them).
//
// What it computes: two 128-row query tiles share every 128-key tile; S = Q K^T, the online softmax
// and O += P V as in the forward kernel over contiguous tensors, with P in tensor memory (rounded to bf16, the type of V
// beside it in the product: off by 2^-8 of each probability at most; the row sums take it unrounded). A row of a
// tile is a (token, head) pair: the gs query heads of a group lie side by side for each of tpt = 128 /
// gs tokens, so a K/V tile serves all of them and a chunk of 32 tokens with 4 heads fills a tile.
//
// Division of the work: units (sequence, head group, pair of query tiles) of as many key tiles as
// their last row sees stand in one line that the CTAs (one per SM, persistent) divide evenly; a unit
// cut by a border leaves fp32 partials (two slots per CTA) that the merge kernel joins. A grid of one
// CTA per unit instead runs in whole waves: 2048 tokens x 32 heads are 256 units on 152 SMs, 1.7
// waves that take the time of 2.
//
// Roles: warp 0 and the last warp read the page table and copy (a warp issues a copy per ~100 cycles, and small
// pages need many: 2048 tokens over 16384 keys in pages of 16 take 372 us, with one warp 561; d = 64 322 and 411), warp 1 issues the MMAs, warps 2-5 and 6-9 are the softmax of tile 0 and tile 1. Copies run ahead
// across units. Stage t of the ring holds V of key tile t and K of key tile t + 1.
//
// Measured: 2048 tokens over 16384 keys, 32 heads over 8 of d = 128: 368 us, 1400 TFLOP/s, the tensor pipe 61% busy: a
// pair of query tiles takes 3214 cycles a key tile, of which its products are 2048; the softmax step is the
// length, as in the forward over contiguous tensors. Six sequences of 1 to 509 tokens over up to 6001 keys: 123 us, 945
// TFLOP/s (shares of 55 key tiles; 13000 cycles each until the first scores, and 13 us of joining).
//
// Tensor memory: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D); P over S.
#include "fa_paged.cuh"
#include "fa_softmax.cuh"
#include "fa_tmap.h"

namespace fa {
namespace {

using namespace tc;

template <int D>
struct ChCfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kThreads = 352;
  static constexpr int kStaging = 8 * 4096;  // the epilogue's, 32 rows of 128 bytes per warp
  static constexpr int kSmem = 2 * kTileBytes + 2 * kStages * kTileBytes + kStaging + 1024;
  static constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
  static constexpr uint32_t kIdPV = idesc_bf16(128, D, false, true);
};

// A unit's copies of Q and its epilogue take the time of about four key tiles (weighed as 1, 2, 3, 4, 6: a mixed batch
// 127, 125, 134, 125 and 125 us, 2048 tokens over 16384 keys 374, 370, 370, 369 and 370).
constexpr int kChOpen = 4;

// The units of one sequence, for one head group: unit u has tokens [u U, u U + U).
struct Units {
  int heads, count, open, U, causal, none;
  SeqInfo q;
  Units() = default;
  __device__ Units(const PagedShape& s, const PagedRows& c, int b)
      : heads(c.Hv), count(0), open(kChOpen), U(2 * c.tpt), causal(s.causal), none(0), q(paged_seq(s, b)) {
    count = c.by_tpt.div(q.Lq + U - 1) >> 1;
    // With more tokens than keys the first units see no key: one empty tile each.
    if (q.off < 0) none = c.by_tpt.div(-q.off) >> 1;
  }
  // Key tiles that token `last` of the sequence, and so any row before it, may see.
  __device__ int tiles_to(int last) const {
    const int keys = causal ? min(q.Lk, last + q.off + 1) : q.Lk;
    return keys <= 0 ? 0 : (keys + 127) >> 7;
  }
  __device__ int tiles(int u) const { return max(1, tiles_to(min(q.Lq, (u + 1) * U) - 1)); }
  __device__ long long before(int u) const {
    long long sum = (long long)u * open;
    if (!causal) return sum + (long long)u * max(1, tiles_to(q.Lq - 1));
    int n = u;
    if (u == count && u > 0) {
      --n;
      sum += tiles(n);
    }
    const int empty = min(n, none);
    return sum + empty + floor_sum(n - empty, 128, U, q.off + (empty + 1) * U + 127);
  }
};

template <int D>
struct ChCtl {
  uint64_t q_full, q_empty, k0_full, k0_empty;
  uint64_t full[4], empty[4];
  uint64_t s_full[2], o_done[2], o_free[2];
  uint64_t p_ready, tail, drain;  // p_ready: of tile 1
  uint32_t tmem_base;
  int abort_flag;
  long long scan[ChCfg<D>::kThreads / 32];  // an entry per warp
  Share share;
  Units units;  // of the sequence where the share begins
  int issued_q[2], issued_k0[2], issued_t[2], issued_tail[2];  // copies issued, by producer (abort-path drain)
  int needs_p0[4];   // by stage buffer: tile 0's softmax arrives on its last stage
  int p0_last[128];  // by row of tile 0: the last stage its thread arrived on
};

struct JoinDesc {
  int b, hv, u, first_cta, first_slot;
  int Lq, q0, bb;  // of the sequence
};

struct ChWork {
  float* part_o;    // [2 CTAs][256][D]
  float* part_lse;  // [2 CTAs][256], log2 units
  JoinDesc* desc;   // [CTAs]; b = -1: no unit ends here in pieces
};

// The pieces of a CTA's share: key tiles [kt, end) of the n that unit u sees.
struct ChPieces {
  const PagedShape& s;
  const PagedRows& c;
  int b, hv, u, kt, n, end, nu;
  long long todo;  // positions from the piece on
  bool finished;
  SeqInfo seq;
  __device__ ChPieces(const PagedShape& s_, const PagedRows& c_, const Share& sh)
      : s(s_), c(c_), b(sh.b), hv(sh.head), u(sh.unit), kt(0), n(0), end(0), nu(0), todo(sh.todo), finished(false) {
    if (todo == 0) return;
    sequence(Units(s, c, b));
    open(sh.tile);
  }
  __device__ void sequence(const Units& x) {
    seq = x.q;
    nu = x.count;
  }
  __device__ int tiles_to(int last) const {  // key tiles that token `last` sees
    const int keys = s.causal ? min(seq.Lk, last + seq.off + 1) : seq.Lk;
    return keys <= 0 ? 0 : (keys + 127) >> 7;
  }
  __device__ void open(int at) {  // at: position within the unit
    n = max(1, tiles_to(min(seq.Lq, 2 * (u + 1) * c.tpt) - 1));
    kt = max(0, at - kChOpen);
    const long long stop = at + todo - kChOpen;
    end = stop < n ? (int)stop : n;
    todo -= min((long long)(n + kChOpen - at), todo);
    if (end <= kt) finished = true;  // the share ends before the unit's first tile
  }
  __device__ bool done() const { return finished || nu == 0; }
  __device__ bool whole() const { return kt == 0 && end == n; }
  __device__ void next() {
    if (todo == 0) {
      finished = true;
      return;
    }
    if (++u == nu) {
      u = 0;
      if (++hv == c.Hv) {
        hv = 0;
        do {  // todo > 0: a later sequence has units
          ++b;
          sequence(Units(s, c, b));
        } while (nu == 0);
      }
    }
    open(0);
  }
  // Key tiles query tile x sees, and whether it exists.
  __device__ int tiles(int x) const {
    const int first = (2 * u + x) * c.tpt, last = min(seq.Lq, first + c.tpt) - 1;
    if (first >= seq.Lq) return 0;
    return tiles_to(last);
  }
};

template <int D>
__global__ void __launch_bounds__(ChCfg<D>::kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const FaPagedArgs a, const PagedRows rows,
                       const ChWork wk) {
  using C = ChCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ChCtl<D> ctl;
  const uint32_t sQ = (smem_u32(smem_raw) + 1023u) & ~1023u;  // two tiles
  const uint32_t sKV = sQ + 2 * C::kTileBytes;                // stage i: V then K
  const uint32_t sO = sKV + 2 * C::kStages * C::kTileBytes;
  volatile int* abort_flag = &ctl.abort_flag;
  const PagedShape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto sV = [&](int i) { return sKV + 2 * i * C::kTileBytes; };
  auto sK = [&](int i) { return sKV + (2 * i + 1) * C::kTileBytes; };
  auto bar = [&](uint64_t& x) { return smem_u32(&x); };

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int i = 0; i < 2; ++i) ctl.issued_q[i] = ctl.issued_k0[i] = ctl.issued_t[i] = ctl.issued_tail[i] = 0;
    mbar_init(bar(ctl.q_full), D / 64);
    mbar_init(bar(ctl.q_empty), 1);
    mbar_init(bar(ctl.k0_full), 2);
    mbar_init(bar(ctl.k0_empty), 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bar(ctl.full[i]), 2 + 128);  // the copies, and P of tile 0 (or its stand-in)
      mbar_init(bar(ctl.empty[i]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(ctl.s_full[x]), 1);
      mbar_init(bar(ctl.o_done[x]), 1);
      mbar_init(bar(ctl.o_free[x]), 128);
    }
    mbar_init(bar(ctl.p_ready), 128);
    mbar_init(bar(ctl.tail), 2);
    mbar_init(bar(ctl.drain), 1);
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem_base), 512);
    tmem_relinquish();
  }
  // Rows of the query tiles that no copy fills are zero.
  const int used = rows.gs * rows.tpt;
  for (int i = threadIdx.x; i < 2 * (D / 64) * (128 - used) * 8; i += C::kThreads) {
    const int r = used + i / 8 % (128 - used), part = i / 8 / (128 - used);
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(sQ + (part * 128 + r) * 128 + (i & 7) * 16), "r"(0)
                 : "memory");
  }
  fence_proxy_async_smem();
  __syncthreads();
  let_dependent_start();  // (this CTA has its tensor memory: a dependent that takes some cannot be in its way)
  grid_dependency_wait();
  find_share<C::kThreads>(s.B, [&](int b) { return Units(s, rows, b); }, ctl.share, ctl.scan, ctl.units);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  ChPieces w(s, rows, ctl.share);  // (looks again: carrying ctl.units here spilled registers, 384 us for 376)
  if (threadIdx.x == 0) {
    JoinDesc d{};
    d.b = !w.done() && w.kt > 0 && w.end == w.n ? w.b : -1;
    d.hv = w.hv;
    d.u = w.u;
    d.first_cta = ctl.share.first_cta;
    d.first_slot = ctl.share.first_slot;
    d.Lq = w.seq.Lq;
    d.q0 = w.seq.q0;
    d.bb = w.seq.bb;
    wk.desc[blockIdx.x] = d;
  }

  if (warp == 0 || warp == C::kThreads / 32 - 1) {
    // ------------------------------------------------------------------ copies
    const int who = warp != 0;
    const CopyShare<D> my{who};
    const int P = 1 << s.page_shift, prows = min(P, 128), shift = min(s.page_shift, 7), per = 128 >> shift;
    bool run = true;
    auto page_of = [&](const ChPieces& x, int kt) -> int {
      const int key = (kt << 7) + (lane << shift);
      return lane < per && key < x.seq.Lk ? paged_page(s, x.b, key >> s.page_shift, a.status) : 0;
    };
    auto pages_in = [&](const ChPieces& x, int kt) -> int {
      const int left = x.seq.Lk - (kt << 7);
      return left <= 0 ? 0 : min(per, (left + prows - 1) >> shift);
    };
    auto copy = [&](uint32_t dst, const CUtensorMap* tm, const ChPieces& x, int kt, int page, uint32_t on) {
      if (my.lane(lane, pages_in(x, kt)))
        tma_load_4d(dst + my.column() * 16384 + lane * prows * 128, tm, my.column() * 64, (kt << 7) & (P - 1), x.hv / rows.per_kv,
                    page, on);
    };
    auto copy_q = [&](const ChPieces& x, int piece) {
      if (!my.copies_q()) return;
      if (run && piece > 0) run = mbar_wait(bar(ctl.q_empty), (piece - 1) & 1, abort_flag, a.status);
      run = __all_sync(0xffffffffu, run) && !*abort_flag;
      if (!run || lane > 0) return;
      const int tiles = (2 * x.u + 1) * rows.tpt < x.seq.Lq ? 2 : 1;
      mbar_expect_tx(bar(ctl.q_full), tiles * used * 128);
      for (int y = 0; y < tiles; ++y)
        tma_load_4d(sQ + y * C::kTileBytes + who * 16384, &tmQ, who * 64, x.hv * rows.gs,
                    x.seq.q0 + (2 * x.u + y) * rows.tpt, x.seq.bb, bar(ctl.q_full));
      ctl.issued_q[who] = piece + 1;
    };
    if (!w.done()) {
      ChPieces v = w;  // the piece of the next K
      int vkt = v.kt, vpiece = 0;
      int page = page_of(w, w.kt);
      copy_q(w, 0);
      if (lane == 0) {
        mbar_expect_tx(bar(ctl.k0_full), my.bytes(pages_in(w, w.kt), prows));
        ctl.issued_k0[who] = 1;
      }
      __syncwarp();
      copy(sK(C::kStages - 1), &tmK, w, w.kt, page, bar(ctl.k0_full));
      int t = 0, tails = 0;
      for (; !w.done(); w.next()) {
        for (int kt = w.kt; kt < w.end; ++kt, ++t) {
          const int st = t % C::kStages;
          if (++vkt == v.end) {
            v.next();
            vkt = 0;
            ++vpiece;
          }
          const bool more = !v.done();
          const int next = more ? page_of(v, vkt) : 0;
          if (run && t == C::kStages - 1) run = mbar_wait(bar(ctl.k0_empty), 0, abort_flag, a.status);
          if (run && t >= C::kStages)
            run = mbar_wait(bar(ctl.empty[st]), (t / C::kStages - 1) & 1, abort_flag, a.status);
          run = __all_sync(0xffffffffu, run) && !*abort_flag;
#ifdef FA_TEST_WITHHOLD_KV  // a test-only build: every wait for a stage must run out cleanly
          run = false;
#endif
          if (!run) continue;
          const int valid = w.seq.Lk - (kt << 7);
          const int vbytes = my.bytes(pages_in(w, kt), prows), kbytes = more ? my.bytes(pages_in(v, vkt), prows) : 0;
          if (lane == 0 && who == 0) {
            const bool p0 = kt < w.tiles(0);
            if (!p0) mbar_arrive_cnt(bar(ctl.full[st]), 128);  // tile 0 has no P for this key tile
            ctl.needs_p0[st] = p0;
          }
          if (valid >= 128) {
            if (lane == 0) {
              mbar_expect_tx(bar(ctl.full[st]), vbytes + kbytes);
              ctl.issued_t[who] = t + 1;
            }
            __syncwarp();
            copy(sV(st), &tmV, w, kt, page, bar(ctl.full[st]));
            if (more) copy(sK(st), &tmK, v, vkt, next, bar(ctl.full[st]));
          } else {
            // The last tile: value rows past the last key may hold anything, and 0 times NaN is NaN.
            // They become 0 here, between the copy of V (on a barrier of its own) and the stage.
            if (lane == 0) {
              mbar_add_tx(bar(ctl.full[st]), kbytes);
              mbar_expect_tx(bar(ctl.tail), vbytes);
              ctl.issued_t[who] = t + 1;
              ctl.issued_tail[who] = tails + 1;
            }
            __syncwarp();
            copy(sV(st), &tmV, w, kt, page, bar(ctl.tail));
            if (more) copy(sK(st), &tmK, v, vkt, next, bar(ctl.full[st]));
            run = mbar_wait(bar(ctl.tail), tails & 1, abort_flag, a.status);
            run = __all_sync(0xffffffffu, run);
            ++tails;
            if (run)
              for (int i = max(valid, 0) * 8 + lane + (D == 128 ? 0 : 32 * who); i < 128 * 8; i += D == 128 ? 32 : 64)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(sV(st) + my.column() * 16384 + i * 16), "r"(0)
                             : "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ctl.full[st]));  // after a failed wait too: K may be in flight
          }
          if (more && vkt == 0) copy_q(v, vpiece);
          page = next;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0 && !w.done()) {
      // The pipe idles while this thread does anything but issue, so the tiles inside a unit that both query
      // tiles see (all but its ends) run in a loop of two waits, four products and three commits.
      bool run = true;
      uint32_t p1phase = 0, seen0 = 0, seen1 = 0;  // parity of tile 1's P; pieces with tiles, per query tile
      ChPieces v = w;
      int vkt = v.kt, vpiece = 0;
      int vn0 = v.tiles(0), vn1 = v.tiles(1);  // key tiles each query tile sees, in the piece of the next S
      const uint64_t dq0 = desc_kmajor_sw128(sQ), dk0 = desc_kmajor_sw128(sK(0)), dv0 = desc_mnmajor_sw128(sV(0), 16384);
      auto issue_s = [&](int x, int st) {
        const uint64_t dq = desc_add(dq0, x * C::kTileBytes), dk = desc_add(dk0, st * 2 * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_ss(tmem + x * 128, desc_add(dq, off), desc_add(dk, off), C::kIdS, kk > 0);
        }
        mma_commit(bar(ctl.s_full[x]));
      };
      auto issue_pv = [&](int x, int st, bool first) {
        const uint64_t dv = desc_add(dv0, st * 2 * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + x * D, tmem + x * 128 + kk * 8, desc_add(dv, kk * 2048), C::kIdPV,
                 (first && kk == 0) ? 0u : 1u);
      };
      auto wait_p1 = [&]() {
        run = mbar_wait_spin(bar(ctl.p_ready), p1phase, abort_flag, a.status);
        p1phase ^= 1;
        fence_after_sync();
      };
      run = mbar_wait_spin(bar(ctl.q_full), 0, abort_flag, a.status);
      if (run) run = mbar_wait_spin(bar(ctl.k0_full), 0, abort_flag, a.status);
      fence_after_sync();
      if (run) {
        if (vkt < vn0) issue_s(0, C::kStages - 1);
        if (vkt < vn1) issue_s(1, C::kStages - 1);
        mma_commit(bar(ctl.k0_empty));
        if (vkt + 1 == v.end) mma_commit(bar(ctl.q_empty));
      }
      int st = 0;
      uint32_t phase = 0;
      auto wait_stage = [&]() {  // V of this tile, K of the next, and P of tile 0
        run = mbar_wait_spin(bar(ctl.full[st]), phase, abort_flag, a.status);
        fence_after_sync();
      };
      auto next_stage = [&]() {
        mma_commit(bar(ctl.empty[st]));
        if (++st == C::kStages) {
          st = 0;
          phase ^= 1;
        }
      };
      for (; !w.done() && run; w.next()) {
        const int wn0 = vn0, wn1 = vn1, last0 = min(w.end, wn0) - 1, last1 = min(w.end, wn1) - 1;
        const int steady = min(last0, last1);  // key tiles (w.kt, steady) are inside the unit for both
        for (int kt = w.kt; kt < w.end && run; ++kt) {
          for (; kt > w.kt && kt < steady; ++kt) {
            wait_stage();
            if (!run) break;
            issue_pv(0, st, false);
            issue_s(0, st);
            wait_p1();
            if (!run) break;
            issue_pv(1, st, false);
            issue_s(1, st);
            if (kt + 2 == w.end) mma_commit(bar(ctl.q_empty));
            next_stage();
          }
          if (!run) break;
          const bool crosses = kt + 1 == w.end;  // the next S belongs to the next piece
          if (crosses) {
            v.next();
            ++vpiece;
            if (!v.done()) {
              vn0 = v.tiles(0);
              vn1 = v.tiles(1);
            }
          }
          vkt = crosses ? 0 : kt + 1;
          const bool more = !v.done();
          wait_stage();
          if (run && kt <= last0) {
            if (kt == w.kt && seen0++ > 0)  // O still holds the last piece's until its epilogue has read it
              run = mbar_wait_spin(bar(ctl.o_free[0]), seen0 & 1, abort_flag, a.status);
            fence_after_sync();
            if (!run) break;
            issue_pv(0, st, kt == w.kt);
            if (kt == last0) mma_commit(bar(ctl.o_done[0]));
          }
          if (run && !crosses && vkt < vn0) issue_s(0, st);
          if (run && kt <= last1) {
            if (kt == w.kt && seen1++ > 0) run = mbar_wait_spin(bar(ctl.o_free[1]), seen1 & 1, abort_flag, a.status);
            if (run) wait_p1();
            if (!run) break;
            issue_pv(1, st, kt == w.kt);
            if (kt == last1) mma_commit(bar(ctl.o_done[1]));
          }
          if (run && !crosses && vkt < vn1) issue_s(1, st);
          if (!run) break;
          if (crosses && more) {
            run = mbar_wait_spin(bar(ctl.q_full), vpiece & 1, abort_flag, a.status);
            fence_after_sync();
            if (!run) break;
            if (vkt < vn0) issue_s(0, st);
            if (vkt < vn1) issue_s(1, st);
          }
          if (more && vkt + 1 == v.end) mma_commit(bar(ctl.q_empty));
          next_stage();
        }
      }
      mma_commit(bar(ctl.drain));
      mbar_wait_drain(bar(ctl.drain), 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax, epilogue
    const int x = (warp - 2) >> 2;
    const int quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + x * 128, tO = tmem + lane_off + 256 + x * D;
    const float sl2 = a.scale * kLog2e;
    const int ti = r / rows.gs, g = r - ti * rows.gs;  // token within the tile, head within the group
    bool run = true;
    uint32_t cnt = 0, pieces = 0;
    int t0 = 0;  // position of the piece's first tile in the ring
    if (x == 0) ctl.p0_last[r] = -1;
    for (int piece = 0; !w.done(); ++piece, t0 += w.end - w.kt, w.next()) {
      const SeqInfo& seq = w.seq;
      const int first = (2 * w.u + x) * rows.tpt;  // the tile's first token
      if (first >= seq.Lq) continue;
      const int i = first + ti;
      const bool live = r < used && i < seq.Lq;
      const int end = min(w.end, w.tiles(x));
      float m = -INFINITY, l = 0.f;
      for (int kt = w.kt; kt < end; ++kt, ++cnt) {
        if (run) run = mbar_wait(bar(ctl.s_full[x]), cnt & 1, abort_flag, a.status);
        fence_after_sync();
        const int k0 = kt << 7;
        const bool masked = (s.causal && k0 + 127 > first + seq.off) || k0 + 128 > seq.Lk;
        const int lim = min(seq.Lk - k0, s.causal ? i + seq.off - k0 + 1 : 128);  // keys [k0, k0 + lim) visible
        softmax_tile<D, false, 1>(tS, tO, tS, masked, lim, sl2, kt == w.kt, m, l, [] {});
        fence_before_sync();
        if (run) {
          const int t = t0 + kt - w.kt;
          mbar_arrive(x == 0 ? bar(ctl.full[t % C::kStages]) : bar(ctl.p_ready));
          if (x == 0) ctl.p0_last[r] = t;
        }
      }
      const bool any = w.kt < end;
      if (any) {
        if (run) run = mbar_wait(bar(ctl.o_done[x]), pieces & 1, abort_flag, a.status);
        ++pieces;
        fence_after_sync();
      }
      const float inv = l == 0.f ? 0.f : 1.f / l, lse2 = l == 0.f ? -INFINITY : m + log2f(l);  // (a NaN stays one)
      const bool whole = w.whole();
      const size_t slot = (size_t)(2 * blockIdx.x + (piece == 0 ? 0 : 1)) * 256 + x * 128 + r;
      const int h = w.hv * rows.gs + g;
      // A thread has a row of O; written as it lies, every store would touch 32 lines (5000 to 11000 cycles a
      // piece). So 128 bytes of each of the warp's rows at a time cross through shared memory (chunks of 16
      // bytes in an order that keeps the banks apart) and leave as whole lines.
      const uint32_t stage = sO + (warp - 2) * 4096;
      const long long at = live ? (long long)elem_offset(a.so, seq.bb, seq.q0 + i, h) : -1;
      float* part = wk.part_o + (slot - lane) * D;  // (a row that does not exist leaves something there, which is not read)
      auto write_lines = [&](const uint32_t (&y)[32], auto&& store) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(stage + lane * 128 + ((k ^ (lane & 7)) << 4)),
                       "r"(y[4 * k]), "r"(y[4 * k + 1]), "r"(y[4 * k + 2]), "r"(y[4 * k + 3])
                       : "memory");
        __syncwarp();
#pragma unroll 2  // (all 8 spill registers: 376 us for 371)
        for (int k = 0; k < 8; ++k) {
          const int row = 4 * k + (lane >> 3);
          uint4 z;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(z.x), "=r"(z.y), "=r"(z.z), "=r"(z.w)
                       : "r"(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4))
                       : "memory");
          store(row, z);
        }
        __syncwarp();
      };
      auto load_o = [&](int c, uint32_t(&o)[32]) {  // columns [32 c, 32 c + 32) of the row, normalised
        if (any) {
          tmem_ld32(tO + c * 32, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = any ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
      };
      if (whole) {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t y[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t o[32];
            load_o(2 * c + half, o);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              y[half * 16 + k] = pack_bf16x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
          }
          write_lines(y, [&](int row, uint4 z) {
            const long long to = __shfl_sync(0xffffffffu, at, row);
            if (to >= 0) *reinterpret_cast<uint4*>(out + to + c * 64 + (lane & 7) * 8) = z;
          });
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          load_o(c, o);
          write_lines(o, [&](int row, uint4 z) {
            *reinterpret_cast<uint4*>(part + row * D + c * 32 + (lane & 7) * 4) = z;
          });
        }
      }
      if (any) {
        fence_before_sync();
        if (run) mbar_arrive(bar(ctl.o_free[x]));
      }
      if (live) {
        if (whole)
          a.lse[paged_row(s, seq, w.b, h, i)] = lse2 * kLn2;
        else
          wk.part_lse[slot] = lse2;
      }
    }
  }

  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) {
    // Copies still in flight land before the CTA exits: the last ones issued on each barrier. A producer that
    // stopped before the other did has its arrival made here.
    auto drain = [&](uint64_t& full, int parity, const int (&issued)[2], int i, int producers = 2) {
      for (int p = 0; p < producers; ++p)
        if (issued[p] <= i) mbar_arrive(bar(full));
      mbar_wait_drain(bar(full), parity);
    };
    const int nq = max(ctl.issued_q[0], ctl.issued_q[1]), nt = max(ctl.issued_t[0], ctl.issued_t[1]);
    const int ntail = max(ctl.issued_tail[0], ctl.issued_tail[1]);
    if (nq > 0) drain(ctl.q_full, (nq - 1) & 1, ctl.issued_q, nq - 1, D / 64);
    if (ctl.issued_k0[0] + ctl.issued_k0[1] > 0) drain(ctl.k0_full, 0, ctl.issued_k0, 0);
    if (ntail > 0) drain(ctl.tail, (ntail - 1) & 1, ctl.issued_tail, ntail - 1);
    for (int t = max(0, nt - C::kStages); t < nt; ++t) {
      // The arrivals of tile 0's softmax that never came, or of its stand-in, are made here: a thread that stopped
      // earlier arrived on no later stage.
      const int st = t % C::kStages;
      if (mbar_test(bar(ctl.full[st]), (t / C::kStages) & 1)) continue;
      if (ctl.issued_t[0] <= t || ctl.needs_p0[st]) {
        int arrived = 0;
        for (int i = 0; i < 128; ++i) arrived += ctl.p0_last[i] >= t;
        if (arrived < 128) mbar_arrive_cnt(bar(ctl.full[st]), 128 - arrived);
      }
      drain(ctl.full[st], (t / C::kStages) & 1, ctl.issued_t, t);
    }
  }
}

// Joins the pieces of each divided unit by their log-sum-exp: M = max LSE, w = 2^(LSE - M),
// O = sum w O / sum w, LSE = M + log2 sum w. Block (c, y) takes kJoinRows rows of the unit that ends in CTA c's first
// piece, if it began before; a thread takes four elements of two rows, whose loads from two pieces are in flight
// together (four rows and a piece at a time: a mixed batch 125 us for 123, 2048 tokens over 16384 keys 370 for 368;
// letting its own dependent start early: 125). It and the kernel border before it are 13 us of those.
constexpr int kJoinRows = 16;
template <int D>
__global__ void __launch_bounds__(256, 5) paged_chunk_join_kernel(const FaPagedArgs a, const PagedRows rows,
                                                                  const ChWork wk) {
  grid_dependency_wait();
  const JoinDesc d = wk.desc[blockIdx.x];
  if (d.b < 0) return;
  constexpr int kPer = kJoinRows * (D / 4) / 256, kStep = 256 / (D / 4);  // rows of a thread, and between them
  const PagedShape& s = a.s;
  const int r0 = blockIdx.y * kJoinRows + threadIdx.x / (D / 4), e = threadIdx.x % (D / 4) * 4, c1 = blockIdx.x;
  float4 acc[kPer];
  float M[kPer], sum[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    M[k] = -INFINITY;
    sum[k] = 0.f;
  }
  for (int c = d.first_cta; c <= c1; c += 2) {
    float l[2][kPer];
    float4 o[2][kPer];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const size_t slot = (size_t)(c + p == d.first_cta ? d.first_slot : 2 * min(c + p, c1)) * 256 + r0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {  // (rows that do not exist hold anything; they are not written)
        l[p][k] = wk.part_lse[slot + k * kStep];
        o[p][k] = *reinterpret_cast<const float4*>(wk.part_o + (slot + k * kStep) * D + e);
      }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (c + p > c1 || l[p][k] == -INFINITY) continue;
        const float top = fmaxf(M[k], l[p][k]), old = exp2f(M[k] - top), w = exp2f(l[p][k] - top);
        M[k] = top;
        sum[k] = sum[k] * old + w;
        acc[k] = make_float4(acc[k].x * old + w * o[p][k].x, acc[k].y * old + w * o[p][k].y,
                             acc[k].z * old + w * o[p][k].z, acc[k].w * old + w * o[p][k].w);
      }
  }
  SeqInfo seq{};
  seq.Lq = d.Lq;
  seq.q0 = d.q0;
  seq.bb = d.bb;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = r0 + k * kStep, rr = r & 127;
    const int ti = rr / rows.gs, i = (2 * d.u + (r >> 7)) * rows.tpt + ti, h = d.hv * rows.gs + rr - ti * rows.gs;
    if (rr >= rows.gs * rows.tpt || i >= seq.Lq) continue;
    const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.o) + elem_offset(a.so, seq.bb, seq.q0 + i, h) + e) =
        make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    if (e == 0)
      a.lse[paged_row(s, seq, d.b, h, i)] = sum[k] == 0.f ? -INFINITY : (M[k] + log2f(sum[k])) * kLn2;
  }
}

template <int D>
cudaError_t launch_chunk(const FaPagedArgs& a, cudaStream_t st) {
  using C = ChCfg<D>;
  const PagedShape& s = a.s;
  const bool packed = s.cu_q != nullptr;
  const PagedRows rows = paged_rows_for(s);
  CUtensorMap tq, tk, tv;
  if (!fa_make_tmap_bf16(&tq, a.q, D, s.H, packed ? s.rows_q : s.Nq, packed ? 1 : s.B, a.sq.head, a.sq.row, a.sq.batch,
                         rows.gs, rows.tpt) ||
      !paged_tmap(&tk, a.k, s, a.sk) || !paged_tmap(&tv, a.v, s, a.sv))
    return cudaErrorInvalidValue;
  ChWork wk;
  char* ws = static_cast<char*>(a.workspace);
  wk.desc = reinterpret_cast<JoinDesc*>(ws);
  ws += up256((size_t)a.num_sms * sizeof(JoinDesc));
  wk.part_lse = reinterpret_cast<float*>(ws);
  ws += up256((size_t)a.num_sms * 512 * sizeof(float));
  wk.part_o = reinterpret_cast<float*>(ws);
  auto kern = paged_chunk_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kern, dim3(a.num_sms), dim3(C::kThreads), C::kSmem, st, tq, tk, tv, a, rows, wk);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_chunk_join_kernel<D>, dim3(a.num_sms, 256 / kJoinRows), dim3(256), 0, st, a, rows, wk);
}

}  // namespace
}  // namespace fa

size_t fa_paged_chunk_workspace(const fa::PagedShape& s, int num_sms) {
  const size_t rows = (size_t)num_sms * 512;
  return fa::up256((size_t)num_sms * sizeof(fa::JoinDesc)) + fa::up256(rows * sizeof(float)) +
         rows * s.d * sizeof(float);
}

cudaError_t fa_launch_paged_chunk(const FaPagedArgs& a, cudaStream_t st) {
  return a.s.d == 64 ? fa::launch_chunk<64>(a, st) : fa::launch_chunk<128>(a, st);
}
