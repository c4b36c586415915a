// The attention weight that new tokens pay every cached key: W[j] += sum over the rows i that see key
// j of exp(c q_i k_j - LSE_i), with the LSE known from the attention itself.
//
// S^T = K Q^T puts a key on each tensor-memory lane and a row on each column, so a key's sum over the
// rows stays within one thread: no value crosses threads, no atomics, and K is read once. With few
// rows (one query tile) the pass streams K and is bound by memory; with many it is bound by the
// exponentials, one per (row, key) pair.
//
// Division of the work: units (sequence, K/V head, key tile) of as many query tiles as see the key
// tile stand in one line that the CTAs (one per SM, persistent) divide evenly. A unit cut by a border
// leaves 128 partial sums per piece (two slots per CTA), which the join kernel adds in the pieces'
// order; with one query tile per unit nothing is cut.
//
// Roles: warp 0 and the last warp read the page table and copy (a warp issues a copy per ~100 cycles, and small
// pages need many: 16 x 8192 keys in pages of 16 take 50 us, with one warp 56; d = 64 37 and 41); one warp issues the MMAs, or with many rows two, a
// query tile each in turn: an MMA takes its thread about 70 cycles whatever its width, so a tile's eight and
// the waits around them fill 1200 cycles of one thread, twice what the tensor pipe needs. Groups of four
// warps (three, with many rows four) take the query tiles in turn; with many rows a last group adds their
// sums of a finished unit to the weights, so that no exponential waits for that read and write.
// Tensor memory: four score buffers of NP columns.
//
// Measured: 16 sequences of up to 8192 keys, one token, 32 heads over 8 of d = 128: 216 MB in 41 us, 5.3 TB/s (79% of
// the copy rate; 4 us until the first keys arrive). 700 tokens over 8192 keys: 51 us, 870 TFLOP/s, the tensor and the
// exponential pipe busy 39% each: 900 cycles a tile of 128 x 128, of which either needs 512.
#include "fa_paged.cuh"
#include "fa_tmap.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace tc;

// NP: rows of a query tile (columns of S^T); FEW: one query tile holds all rows of a K/V head (NP <=
// 64), stays in shared memory for all key tiles of the head and the ring holds K; else the ring
// that matters holds query tiles.
template <int D, int NP>
struct WCfg {
  static constexpr bool kFew = NP <= 64;
  static constexpr int kKBytes = 128 * D * 2, kQBytes = NP * D * 2;
  // With two issuers a tile may be done before the one in front of it, so each score buffer needs a group of
  // its own, which sees the buffer's every phase.
  static constexpr int kGroups = kFew ? 3 : 4;
  static constexpr int kIssuers = kFew ? 1 : 2;
  static constexpr int kIssuer2 = 2 + 4 * kGroups + 4;  // the second issuer's warp, behind the sums' group
  static constexpr int kThreads = 64 + 128 * kGroups + (kFew ? 0 : 128 + 32) + 32;
  static constexpr int kKBufs = (kFew ? (NP == 64 ? 5 : 6) : 2) * (128 / D);
  static constexpr int kQBufs = kFew ? 2 : 4 * (128 / D);  // (even: a buffer has one issuer, which sees its every phase)
  // A unit's sums and hand-over, in query tiles (weighed as 1, 2, 3, 4: 51.3, 51.6, 52.1 and 53.4 us).
  static constexpr int kOpen = kFew ? 0 : 1;
  static constexpr int kSmem = kKBufs * kKBytes + kQBufs * kQBytes + 1024;
  static constexpr uint32_t kTmemCols = NP == 16 ? 64 : NP == 32 ? 128 : NP == 64 ? 256 : 512;
  static constexpr uint32_t kId = idesc_bf16(128, NP, false, false);
};

// One sequence's units, per K/V head: key tile kt is seen by the token tiles from first(kt) on, each
// of per_kv groups.
struct WUnits {
  SeqInfo q;
  int heads, count, open, ntt, tpt, per_kv, causal;
  FastDiv by_tpt;
  WUnits() = default;
  __device__ WUnits(const PagedShape& s, const PagedRows& c, int b, int open_)
      : q(paged_seq(s, b)),
        heads(s.Hkv),
        count(0),
        open(open_),
        ntt(c.by_tpt.div(q.Lq + c.tpt - 1)),
        tpt(c.tpt),
        per_kv(c.per_kv),
        causal(s.causal),
        by_tpt(c.by_tpt) {
    if (q.Lq > 0) count = (q.Lk + 127) >> 7;
  }
  __device__ int first(int kt) const { return causal ? by_tpt.div(max(0, (kt << 7) - q.off)) : 0; }
  __device__ int tiles(int kt) const { return per_kv * (ntt - first(kt)); }
  __device__ long long before(int kt) const {
    long long sum = (long long)kt * ntt;
    if (causal) {
      const int none = min(kt, max(0, (q.off + 127) >> 7));  // key tiles that every token sees whole
      sum -= floor_sum(kt - none, tpt, 128, (none << 7) - q.off);
    }
    return sum * per_kv + (long long)kt * open;
  }
};

template <int D, int NP>
struct WCtl {
  uint64_t k_full[12], k_empty[12], q_full[8], q_empty[8], s_full[4], s_free[4], sum_ready[2], sum_free[2], drain;
  uint32_t tmem_base;
  int abort_flag;
  long long scan[WCfg<D, NP>::kThreads / 32];  // an entry per warp
  Share share;
  WUnits units;                         // of the sequence where the share begins
  int issued_k[2], issued_q[2];         // copies issued, by producer (abort-path drain)
  alignas(16) float nlse[4][2][NP];  // -LSE (log2 units) of the rows, per group and parity; -inf: no weight
  alignas(16) int seen[4][2][NP];    // last key the row sees
  float sums[2][4][NP == 128 ? 128 : 1];  // many rows: the groups' sums of a piece, per parity
};

struct WJoin {
  int b, hk, kt, first_cta, first_slot, pad[3];
};

struct WWork {
  float* part;   // [2 CTAs][128]
  WJoin* desc;   // [CTAs]; b = -1: no unit ends here in pieces
};

// The pieces of a CTA's share: query tiles [it, end) of the n that see key tile kt.
template <bool FEW>
struct WPieces {
  const PagedShape& s;
  const PagedRows& c;
  int b, hk, kt, it, end;
  long long todo;  // positions from the piece on
  bool head;       // first piece of its (sequence, K/V head) in this CTA
  bool finished;
  int n, tt0;
  WUnits x;
  __device__ WPieces(const PagedShape& s_, const PagedRows& c_, const Share& sh, const WUnits& first)
      : s(s_), c(c_), b(sh.b), hk(sh.head), kt(sh.unit), it(0), end(0), todo(sh.todo), head(true),
        finished(sh.todo == 0), n(0), tt0(0), x(first) {
    if (todo > 0) unit(sh.tile);
  }
  __device__ void unit(int at) {  // opens unit kt at position `at` of it
    if (FEW) {  // one tile and no opening
      n = end = 1;
      --todo;
      return;
    }
    tt0 = x.first(kt);
    n = x.per_kv * (x.ntt - tt0);
    it = max(0, at - x.open);
    const long long stop = at + todo - x.open;
    end = stop < n ? (int)stop : n;
    todo -= min((long long)(n + x.open - at), todo);
    finished = end <= it;  // the share ends before the unit's first tile
  }
  __device__ bool done() const { return finished; }
  __device__ bool whole() const { return it == 0 && end == n; }
  __device__ void next() {
    if (todo == 0) {
      finished = true;
      return;
    }
    head = ++kt == x.count;
    if (head) {
      kt = 0;
      if (++hk == s.Hkv) {
        hk = 0;
        do x = WUnits(s, c, ++b, x.open);
        while (x.count == 0);  // todo > 0: a later sequence has units
      }
    }
    unit(0);
  }
  __device__ void skip_to(const WPieces& o) {
    b = o.b;
    hk = o.hk;
    kt = o.kt;
    it = o.it;
    end = o.end;
    todo = o.todo;
    head = o.head;
    finished = o.finished;
    n = o.n;
    tt0 = o.tt0;
    x = o.x;
  }
  // A query tile of the unit: its first token, and the first head of its group.
  struct Cursor {
    int tt, g;  // token tile, group
    __device__ Cursor(const WPieces& w, int i) : tt(w.c.by_per_kv.div(i)), g(i - tt * w.c.per_kv) { tt += w.tt0; }
    __device__ void advance(const WPieces& w, int by) {
      for (g += by; g >= w.c.per_kv; g -= w.c.per_kv) ++tt;
    }
    __device__ int token(const WPieces& w) const { return tt * w.c.tpt; }
    __device__ int head0(const WPieces& w) const { return (w.hk * w.c.per_kv + g) * w.c.gs; }
  };
};

// One query tile's part of a key's sum: 2^(c log2(e) s - LSE) over the columns (rows) of this thread's
// lane, the first `cols` of them rounded up to a chunk (the others carry no weight).
template <int NP, bool MASK>
__device__ __forceinline__ float tile_sum(uint32_t tS, const float* nls, const int* sees, int key, int cols,
                                          float sl2) {
  constexpr int W = 16;  // columns per load; the next ones are on their way while these are worked on
  float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  uint32_t x[2][W];
  tmem_ld16(tS, x[0]);
#pragma unroll
  for (int c = 0; c < NP; c += W) {
    if (c >= cols) break;
    const uint32_t(&y)[W] = x[(c / W) & 1];
    tmem_ld_wait();
    if (c + W < NP) tmem_ld16(tS + c + W, x[(c / W + 1) & 1]);
#pragma unroll
    for (int k = 0; k < W; k += 4) {
      const float4 n4 = *reinterpret_cast<const float4*>(nls + c + k);
      const float2 sc = make_float2(sl2, sl2);
      const float2 y0 = fma2(make_float2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), sc, make_float2(n4.x, n4.y));
      const float2 y1 =
          fma2(make_float2(__uint_as_float(y[k + 2]), __uint_as_float(y[k + 3])), sc, make_float2(n4.z, n4.w));
      float p0 = ex2_approx(y0.x), p1 = ex2_approx(y0.y), p2 = ex2_approx(y1.x), p3 = ex2_approx(y1.y);
      if constexpr (MASK) {
        const int4 see = *reinterpret_cast<const int4*>(sees + c + k);
        p0 = key <= see.x ? p0 : 0.f;
        p1 = key <= see.y ? p1 : 0.f;
        p2 = key <= see.z ? p2 : 0.f;
        p3 = key <= see.w ? p3 : 0.f;
      }
      part[0] = add2(part[0], make_float2(p0, p1));
      part[1] = add2(part[1], make_float2(p2, p3));
    }
  }
  tmem_ld_wait();  // (a load past the last columns may be under way)
  return (part[0].x + part[0].y) + (part[1].x + part[1].y);
}

template <int D, int NP>
__global__ void __launch_bounds__(WCfg<D, NP>::kThreads, 1)
    paged_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const FaPagedArgs a, const PagedRows rows, const WWork wk) {
  using C = WCfg<D, NP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ WCtl<D, NP> ctl;
  const uint32_t sK = (smem_u32(smem_raw) + 1023u) & ~1023u, sQ = sK + C::kKBufs * C::kKBytes;
  volatile int* abort_flag = &ctl.abort_flag;
  const PagedShape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](uint64_t& x) { return smem_u32(&x); };

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int i = 0; i < 2; ++i) ctl.issued_k[i] = ctl.issued_q[i] = 0;
    for (int i = 0; i < C::kKBufs; ++i) {
      mbar_init(bar(ctl.k_full[i]), 2);
      mbar_init(bar(ctl.k_empty[i]), C::kIssuers);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(bar(ctl.q_full[i]), D / 64);
      mbar_init(bar(ctl.q_empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(ctl.s_full[i]), 1);
      mbar_init(bar(ctl.s_free[i]), 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(ctl.sum_ready[i]), 128 * C::kGroups);
      mbar_init(bar(ctl.sum_free[i]), 128);
    }
    mbar_init(bar(ctl.drain), C::kIssuers);
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  // Rows of the query tiles that no copy fills are zero.
  const int used = rows.gs * rows.tpt;
  for (int i = threadIdx.x; i < C::kQBufs * (D / 64) * (NP - used) * 8; i += C::kThreads) {
    const int r = used + i / 8 % (NP - used), part = i / 8 / (NP - used);
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(sQ + (part * NP + r) * 128 + (i & 7) * 16), "r"(0)
                 : "memory");
  }
  fence_proxy_async_smem();
  __syncthreads();
  let_dependent_start();  // (this CTA has its tensor memory: a dependent that takes some cannot be in its way)
  grid_dependency_wait();
  find_share<C::kThreads>(s.B, [&](int b) { return WUnits(s, rows, b, C::kOpen); }, ctl.share, ctl.scan, ctl.units);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  WPieces<C::kFew> w(s, rows, ctl.share, ctl.units);
  if (!C::kFew && threadIdx.x == 0) {
    WJoin d{};
    d.b = !w.done() && w.it > 0 && w.end == w.n ? w.b : -1;
    d.hk = w.hk;
    d.kt = w.kt;
    d.first_cta = ctl.share.first_cta;
    d.first_slot = ctl.share.first_slot;
    wk.desc[blockIdx.x] = d;
  }

  if (warp == 0 || warp == C::kThreads / 32 - 1) {
    // ------------------------------------------------------------------ copies
    const int who = warp != 0;
    const CopyShare<D> my{who};
    const int P = 1 << s.page_shift, prows = min(P, 128), shift = min(s.page_shift, 7), per = 128 >> shift;
    bool run = true;
    int kn = 0, qn = 0;  // key tiles and query tiles copied
    auto page_of = [&](const WPieces<C::kFew>& x) -> int {
      const int key = (x.kt << 7) + (lane << shift);
      return lane < per && key < x.x.q.Lk ? paged_page(s, x.b, key >> s.page_shift, a.status) : 0;
    };
    auto go = [&]() {
      run = __all_sync(0xffffffffu, run) && !*abort_flag;
      return run;
    };
    auto copy_q = [&](int token, int head0) {
      if (!my.copies_q()) return;
      const int st = qn % C::kQBufs, u = qn / C::kQBufs;
      if (run && u > 0) run = mbar_wait(bar(ctl.q_empty[st]), (u - 1) & 1, abort_flag, a.status);
      if (go() && lane == 0) {
        mbar_expect_tx(bar(ctl.q_full[st]), used * 128);
        tma_load_4d(sQ + st * C::kQBytes + who * NP * 128, &tmQ, who * 64, head0, w.x.q.q0 + token, w.x.q.bb,
                    bar(ctl.q_full[st]));
        ctl.issued_q[who] = qn + 1;
      }
      ++qn;
    };
    int page = w.done() ? 0 : page_of(w);
    while (!w.done()) {
      if (C::kFew && w.head) copy_q(0, w.hk * rows.gs);
      const int st = kn % C::kKBufs, u = kn / C::kKBufs;
      if (run && u > 0) run = mbar_wait(bar(ctl.k_empty[st]), (u - 1) & 1, abort_flag, a.status);
#ifdef FA_TEST_WITHHOLD_KV  // a test-only build: every wait for a key tile must run out cleanly
      run = false;
#endif
      if (go()) {
        const int pages = min(per, (w.x.q.Lk - (w.kt << 7) + prows - 1) >> shift);
        if (lane == 0) {
          mbar_expect_tx(bar(ctl.k_full[st]), my.bytes(pages, prows));
          ctl.issued_k[who] = kn + 1;
        }
        __syncwarp();
        if (my.lane(lane, pages))
          tma_load_4d(sK + st * C::kKBytes + my.column() * 16384 + lane * prows * 128, &tmK, my.column() * 64,
                      (w.kt << 7) & (P - 1), w.hk, page, bar(ctl.k_full[st]));
      }
      ++kn;
      if (!C::kFew) {
        typename WPieces<C::kFew>::Cursor at(w, w.it);
        for (int i = w.it; i < w.end; ++i, at.advance(w, 1)) copy_q(at.token(w), at.head0(w));
      }
      w.next();
      page = w.done() ? 0 : page_of(w);
    }
  } else if (warp == 1 || (C::kIssuers == 2 && warp == C::kIssuer2)) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      // Positions in the rings are counters and the group that sees the scores releases the query tile:
      // every instruction between a thread's products is time the pipe may idle.
      const int me = warp == 1 ? 0 : 1;
      bool run = true;
      int t = 0, ks = 0, qs = 0, sb = 0, qn = 0;
      uint32_t kphase = 0, qphase = 0, sphase = 1;  // parity awaited on the ring's current buffer
      while (!w.done() && run) {
        if (C::kFew && w.head) {
          qs = qn % C::kQBufs;
          run = mbar_wait_spin(bar(ctl.q_full[qs]), (qn / C::kQBufs) & 1, abort_flag, a.status);
          ++qn;
        }
        if (run) run = mbar_wait_spin(bar(ctl.k_full[ks]), kphase, abort_flag, a.status);
        const uint64_t dk = desc_kmajor_sw128(sK + ks * C::kKBytes);
        for (int i = w.it; i < w.end && run; ++i, ++t) {
          if (C::kIssuers == 1 || (t & 1) == me) {
            if (!C::kFew) run = mbar_wait_spin(bar(ctl.q_full[qs]), qphase, abort_flag, a.status);
            if (run && t >= 4) run = mbar_wait_spin(bar(ctl.s_free[sb]), sphase, abort_flag, a.status);
            fence_after_sync();
            if (!run) break;
            const uint64_t dq = desc_kmajor_sw128(sQ + qs * C::kQBytes);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + sb * NP, desc_add(dk, (kk >> 2) * 16384 + (kk & 3) * 32),
                     desc_add(dq, (kk >> 2) * NP * 128 + (kk & 3) * 32), C::kId, kk > 0);
            mma_commit(bar(ctl.s_full[sb]));
          }
          if (++sb == 4) {
            sb = 0;
            sphase ^= 1;
          }
          if (!C::kFew && ++qs == C::kQBufs) {
            qs = 0;
            qphase ^= 1;
          }
        }
        if (!run) break;
        mma_commit(bar(ctl.k_empty[ks]));
        if (++ks == C::kKBufs) {
          ks = 0;
          kphase ^= 1;
        }
        w.next();
        if (C::kFew && !w.done() && w.head) mma_commit(bar(ctl.q_empty[qs]));
      }
      mma_commit(bar(ctl.drain));
      mbar_wait_drain(bar(ctl.drain), 0);
    }
  } else if (warp < 2 + 4 * C::kGroups) {
    // ------------------------------------------------------------------ exponentials and sums
    const int gr = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane;  // group; key (and row, for the LSE)
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float sl2 = a.scale * kLog2e;
    const int ti = r / rows.gs, g = r - ti * rows.gs;
    bool run = true, hidden = false;
    int t = 0, flip = 0;
    bool fresh = true;  // few rows: the head changed since this group's last tile
    // The LSE of row r of a query tile (-inf: no such row); used one tile later, so that no thread
    // waits for the load.
    auto load_lse = [&](int token, int head0) -> float {
      const int i = token + ti;
      return r < used && i < w.x.q.Lq ? a.lse[paged_row(s, w.x.q, w.b, head0 + g, i)] : -INFINITY;
    };
    // Puts it where the group reads it; `hidden`: some column's scores must not enter the sum as they
    // are (a copied row of another sequence, or one without weight).
    auto stage_lse = [&](int token, float lse) {
      const bool dead = lse == -INFINITY;
      flip ^= 1;
      if (r < NP) {
        ctl.nlse[gr][flip][r] = dead ? -INFINITY : -lse * kLog2e;
        ctl.seen[gr][flip][r] = dead ? -1 : (s.causal ? token + ti + w.x.q.off : 0x7fffffff);
      }
      __syncwarp();
      uint32_t any;
      asm volatile(
          "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, 128, p; selp.u32 %0, 1, 0, q; }"
          : "=r"(any)
          : "r"((uint32_t)(dead && r < used)), "r"(1 + gr)
          : "memory");
      hidden = any != 0;
    };
    auto tile = [&](int token) -> float {
      const bool masked = hidden || (s.causal && (w.kt << 7) + 127 > token + w.x.q.off);
      const int cols = min(used, (w.x.q.Lq - token) * rows.gs), key = (w.kt << 7) + r;
      const int sb = t & 3;
      if (run) run = mbar_wait(bar(ctl.s_full[sb]), (t >> 2) & 1, abort_flag, a.status);
      if (!C::kFew && run && r == 0) mbar_arrive(bar(ctl.q_empty[t % C::kQBufs]));  // the product has read it
      __syncwarp();
      fence_after_sync();
      const float* nls = ctl.nlse[gr][flip];
      const int* sees = ctl.seen[gr][flip];
      const uint32_t tS = tmem + lane_off + sb * NP;
      const float sum = masked ? tile_sum<NP, true>(tS, nls, sees, key, cols, sl2)
                               : tile_sum<NP, false>(tS, nls, sees, key, cols, sl2);
      fence_before_sync();
      if (run) mbar_arrive(bar(ctl.s_free[sb]));
      return sum;
    };
    if constexpr (C::kFew) {
      // One tile per key tile: its group also adds to the weights, which it reads a turn ahead (the page a
      // tile earlier than the weight it leads to).
      auto page_of = [&](const WPieces<C::kFew>& y) -> int {
        const int key = (y.kt << 7) + r;
        return key < y.x.q.Lk ? s.table[(size_t)y.b * s.max_pages + (key >> s.page_shift)] : 0;
      };
      auto weight_at = [&](const WPieces<C::kFew>& y, int page) -> float* {
        const int key = (y.kt << 7) + r;
        if (key >= y.x.q.Lk) return nullptr;
        if ((unsigned)page >= (unsigned)s.num_pages) {
          report_status(a.status, FA_ERR_BOUNDS);
          return nullptr;
        }
        return a.weights + weight_offset(s, page, y.hk, key & ((1 << s.page_shift) - 1));
      };
      for (; t < gr && !w.done(); ++t) w.next();
      float* at = w.done() ? nullptr : weight_at(w, page_of(w));
      float old = at != nullptr ? *at : 0.f;
      while (!w.done()) {
        WPieces<C::kFew> ahead = w;
        bool turns = false;  // the head changes before this group's next tile
        for (int i = 0; i < C::kGroups && !ahead.done(); ++i) {
          ahead.next();
          turns |= ahead.head;
        }
        const int page = ahead.done() ? 0 : page_of(ahead);
        if (fresh) stage_lse(0, load_lse(0, w.hk * rows.gs));
        fresh = turns;
        const float sum = tile(0);
        float* then = ahead.done() ? nullptr : weight_at(ahead, page);
        const float before = then != nullptr ? *then : 0.f;
        if (at != nullptr) *at = old + sum;
        at = then;
        old = before;
        w.skip_to(ahead);
        t += C::kGroups;
        __syncwarp();
      }
    } else {
      // The LSE of a piece's first tile is on its way while the sums of the piece before are handed over.
      typename WPieces<C::kFew>::Cursor at(w, 0);
      float lse = 0.f;
      int i = 0;
      auto first_tile = [&]() {
        i = w.it + (gr + C::kGroups - t % C::kGroups) % C::kGroups;  // this group's first tile of the piece
        at = typename WPieces<C::kFew>::Cursor(w, i);
        if (i < w.end) lse = load_lse(at.token(w), at.head0(w));
      };
      if (!w.done()) first_tile();
      for (int piece = 0; !w.done(); ++piece) {
        const int t0 = t - w.it;
        float sum = 0.f;
        for (; i < w.end; i += C::kGroups) {
          t = t0 + i;
          const int token = at.token(w);
          stage_lse(token, lse);
          at.advance(w, C::kGroups);
          if (i + C::kGroups < w.end) lse = load_lse(at.token(w), at.head0(w));
          sum += tile(token);
        }
        t = t0 + w.end;
        w.next();
        if (!w.done()) first_tile();
        const int pp = piece & 1;
        if (run && piece >= 2) run = mbar_wait(bar(ctl.sum_free[pp]), ((piece >> 1) - 1) & 1, abort_flag, a.status);
        ctl.sums[pp][gr][r] = sum;
        if (run) mbar_arrive(bar(ctl.sum_ready[pp]));
        __syncwarp();
      }
    }
  } else if constexpr (!C::kFew) {
    // ------------------------------------------------------------------ sums to weights
    const int r = threadIdx.x - (64 + 128 * C::kGroups);
    bool run = true;
    for (int piece = 0; !w.done(); ++piece, w.next()) {
      const int key = (w.kt << 7) + r, pp = piece & 1;
      float* at = nullptr;
      float old = 0.f;
      if (w.whole() && key < w.x.q.Lk) {
        const int page = paged_page(s, w.b, key >> s.page_shift, a.status);
        if (page >= 0) {
          at = a.weights + weight_offset(s, page, w.hk, key & ((1 << s.page_shift) - 1));
          old = *at;
        }
      } else if (!w.whole()) {
        at = wk.part + (size_t)(2 * blockIdx.x + (piece == 0 ? 0 : 1)) * 128 + r;
      }
      if (run) run = mbar_wait(bar(ctl.sum_ready[pp]), (piece >> 1) & 1, abort_flag, a.status);
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < C::kGroups; ++g) sum += ctl.sums[pp][g][r];
      if (run) mbar_arrive(bar(ctl.sum_free[pp]));
      if (at != nullptr) *at = old + sum;
      __syncwarp();
    }
  }

  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) {
    // Copies still in flight land before the CTA exits: the last one issued into each buffer. A producer that stopped
    // before the other did has its arrival made here.
    auto drain = [&](uint64_t& full, int parity, const int (&issued)[2], int i, int producers = 2) {
      for (int p = 0; p < producers; ++p)
        if (issued[p] <= i) mbar_arrive(bar(full));
      mbar_wait_drain(bar(full), parity);
    };
    const int nq = max(ctl.issued_q[0], ctl.issued_q[1]), nk = max(ctl.issued_k[0], ctl.issued_k[1]);
    for (int i = max(0, nq - C::kQBufs); i < nq; ++i)
      drain(ctl.q_full[i % C::kQBufs], (i / C::kQBufs) & 1, ctl.issued_q, i, D / 64);
    for (int i = max(0, nk - C::kKBufs); i < nk; ++i)
      drain(ctl.k_full[i % C::kKBufs], (i / C::kKBufs) & 1, ctl.issued_k, i);
  }
}

// Adds the pieces of each divided unit, in their order: block c the one that ends in CTA c's first piece.
__global__ void __launch_bounds__(128) paged_weights_join_kernel(const FaPagedArgs a, const WWork wk) {
  let_dependent_start();
  grid_dependency_wait();
  const WJoin d = wk.desc[blockIdx.x];
  if (d.b < 0) return;
  const PagedShape& s = a.s;
  const int key = (d.kt << 7) + threadIdx.x;
  if (key >= paged_seq(s, d.b).Lk) return;
  float sum = wk.part[(size_t)d.first_slot * 128 + threadIdx.x];
  for (int c = d.first_cta + 1; c <= (int)blockIdx.x; ++c) sum += wk.part[(size_t)c * 256 + threadIdx.x];
  const int page = paged_page(s, d.b, key >> s.page_shift, a.status);
  if (page >= 0) a.weights[weight_offset(s, page, d.hk, key & ((1 << s.page_shift) - 1))] += sum;
}

template <int D, int NP>
cudaError_t launch_weights(const FaPagedArgs& a, const PagedRows& rows, cudaStream_t st) {
  using C = WCfg<D, NP>;
  static_assert(C::kSmem + sizeof(WCtl<D, NP>) <= 227 * 1024, "with the control block");
  const PagedShape& s = a.s;
  const bool packed = s.cu_q != nullptr;
  CUtensorMap tq, tk;
  if (!fa_make_tmap_bf16(&tq, a.q, D, s.H, packed ? s.rows_q : s.Nq, packed ? 1 : s.B, a.sq.head, a.sq.row, a.sq.batch,
                         rows.gs, rows.tpt) ||
      !paged_tmap(&tk, a.k, s, a.sk))
    return cudaErrorInvalidValue;
  WWork wk{};
  if (!C::kFew) {
    wk.desc = static_cast<WJoin*>(a.workspace);
    wk.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + (size_t)a.num_sms * sizeof(WJoin));
  }
  auto kern = paged_weights_kernel<D, NP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kern, dim3(a.num_sms), dim3(C::kThreads), C::kSmem, st, tq, tk, a, rows, wk);
  if (e != cudaSuccess || C::kFew) return e;
  return launch_dependent(paged_weights_join_kernel, dim3(a.num_sms), dim3(128), 0, st, a, wk);
}

template <int D>
cudaError_t launch_weights_d(const FaPagedArgs& a, cudaStream_t st) {
  const int G = a.s.H / a.s.Hkv;
  if (!paged_few_rows(a.s)) return launch_weights<D, 128>(a, paged_rows_for(a.s), st);
  const PagedRows few = paged_rows(G, a.s.Hkv, 1, a.s.Nq);  // all rows of a K/V head in one tile
  const int n = a.s.Nq * G;
  return n <= 16 ? launch_weights<D, 16>(a, few, st)
         : n <= 32 ? launch_weights<D, 32>(a, few, st)
                   : launch_weights<D, 64>(a, few, st);
}

}  // namespace
}  // namespace fa

size_t fa_paged_weights_workspace(const fa::PagedShape& s, int num_sms) {
  if (fa::paged_few_rows(s)) return 0;  // a key tile is one query tile's work
  return (size_t)num_sms * (sizeof(fa::WJoin) + 2 * 128 * sizeof(float));
}

cudaError_t fa_launch_paged_key_weights(const FaPagedArgs& a, cudaStream_t st) {
  return a.s.d == 64 ? fa::launch_weights_d<64>(a, st) : fa::launch_weights_d<128>(a, st);
}
