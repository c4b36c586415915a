// Attention of a few new tokens per sequence over a paged cache (decode, drafted tokens): at most 64
// rows (tokens x query heads of one K/V head), so the pass is bound by reading K and V once.
//
// What it computes: for the R = L_q G rows of a (sequence, K/V head), key tiles of 128 stream through
// shared memory; S^T = K Q^T puts a key on each tensor-memory lane and a row on each column, so the
// products cost N = 16, 32 or 64 columns instead of a 128-row tile that would be nearly empty, and a
// softmax thread handles 16 numbers per tile instead of 128. P^T goes back through shared memory
// (bf16, keys x rows) and O^T += V^T P^T accumulates in tensor memory, a head dimension per lane.
// Measured: 32 sequences of up to 8192 keys, 32 heads over 8 of d = 128, one token: 824 MB in 132 us, 6.2 TB/s (94% of the
// copy rate); 48 of up to 1024 keys, 12 heads of d = 64: 116 MB in 31 us (a share has 13 tiles and 2.6 units' borders);
// one sequence of 777 keys: 8.4 us, latency.
// The exponentials are taken against a reference max per row, set by the row's first tile and raised
// (O and the row sums rescaled) only when a score exceeds it by more than 2^8: exact, since fp32 and bf16
// keep their relative precision over that range (a wider one would leave values near the top of bf16
// less room in O), and one vote per tile replaces a max over 128 keys.
//
// Division of the work: all sequences' key tiles form one line, ordered (sequence, head, tile), which
// the CTAs (one or two per SM, persistent) divide evenly, whatever the lengths are. A CTA's share
// begins and ends inside a (sequence, head) at most twice; those pieces leave normalised fp32
// partials (two slots per CTA) that the merge kernel joins by their log-sum-exp; whole ones are
// written directly. Few (sequence, head) units of not too many tiles are shared by a cluster each instead, whose
// CTAs join their parts through shared memory: one launch, no workspace and no search for the share.
//
// Roles: warp 0 and at d = 128 the last warp read the page table and copy (TMA, a lane per page; 64 columns
// each, since a warp issues a copy per ~100 cycles and small pages need many: 16 x 8192 keys in pages of 16 in
// 93 us, with one warp 100, in pages of 8 107 and 155, of 32 and more 89 both ways),
// warp 1 issues the MMAs, groups of four warps are the softmax and the epilogue, of 16 rows each. Copies run ahead across pieces, so memory never waits for an
// epilogue.
#include "fa_paged.cuh"
#include "fa_tmap.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace tc;

constexpr int kDecCluster = 8;       // CTAs of the largest cluster that shares a unit
constexpr float kNoMax = -3.0e38f;   // reference max of a row that has seen no key
constexpr float kRaise = 8.f;       // log2 units a score may exceed the reference by

// CTAs per SM.
constexpr int dec_ctas(int d, int np) { return d == 64 && np < 64 ? 2 : 1; }

template <int D, int NP>
struct DecCfg {
  static constexpr int kTileBytes = 128 * D * 2;
  // d = 128: one CTA per SM, 192 KB of K and V in flight. d = 64: tiles are half as large and the
  // latencies of a tile (scores, exponentials, P, product) would show, so two CTAs share an SM, with
  // 80 KB each in flight. 64-row tiles take the registers of a whole SM: one CTA, 128 KB.
  static constexpr int kCtas = dec_ctas(D, NP);
  // Groups of four softmax warps, 16 rows (columns of S^T, which are independent) each: one group for all
  // leaves a scheduler one warp and its chain of dependent steps (64 sequences of 1000 keys, 8 K/V heads, d = 128:
  // 64 rows 112 us with one group, 87 with two, 76 with four; 32 rows 64 and 61; d = 64: 99, 69 and 59; 54 and 41).
  static constexpr int kGroups = NP / 16, kThreads = 64 + 128 * kGroups + 32 * (D / 64 - 1);
  static constexpr int kKStages = NP == 64 ? 256 / D : 3, kVStages = NP == 64 ? 256 / D : D == 64 ? 2 : 3;
  static constexpr int kQBytes = NP * D * 2;
  static constexpr int kQBufs = 2;
  // P has two buffers: 128 keys, a 128-byte row each, of which a tile's P takes 2 NP bytes. With up to 32
  // rows they lie side by side, else one behind the other.
  static constexpr int kPBytes = (NP == 64 ? 2 : 1) * 128 * 128;
  static constexpr int kPStep = NP == 64 ? 128 * 128 : NP * 2;
  static constexpr int kSmem = kQBufs * kQBytes + (kKStages + kVStages) * kTileBytes + kPBytes + 1024;
  static_assert(kCtas * (kSmem + 576 + 32 * NP + 1024) <= 228 * 1024, "with the control block");
  static constexpr uint32_t kTmemCols = NP == 16 ? 64 : NP == 32 ? 128 : 256;  // S x 2, O x 2
  static constexpr uint32_t kIdS = idesc_bf16(128, NP, false, false);
  // O^T = V^T P^T has D rows; at D = 64 the upper 64 lanes multiply whatever follows V in shared
  // memory and are never read (a lane's result depends on its own row alone).
  static constexpr uint32_t kIdPV = idesc_bf16(128, NP, true, true);
};

// A unit (sequence, K/V head) without keys still has a tile, which writes its zeros. Its epilogue takes
// the time of about one tile (weighed as 1, 2 or 3: 48 sequences of 1024 keys, 12 heads of d = 64, in 34.4, 34.9
// and 35.1 us).
constexpr int kDecOpen = 1;

struct DecUnits {
  int heads, count, open;
  SeqInfo q;
  DecUnits() = default;
  __device__ DecUnits(const PagedShape& s, int b) : heads(s.Hkv), count(0), open(kDecOpen), q(paged_seq(s, b)) {
    count = q.Lq > 0;
  }
  __device__ int tiles(int = 0) const { return max(1, (q.Lk + 127) >> 7); }
  __device__ long long before(int u) const { return u * (tiles() + open); }
};

template <int D, int NP>
struct DecCtl {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2];
  uint64_t p_ready[2], pv_done[2];  // per buffer of P
  uint64_t o_free[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  long long scan[DecCfg<D, NP>::kThreads / 32];  // an entry per warp
  Share share;
  DecUnits units;  // of the sequence where the share begins
  int issued_q[2], issued_t[2];                   // copies issued, by producer (abort-path drain)
  alignas(16) float m[NP];
  alignas(16) float alpha[NP];
  float wmax[4][NP];
  float part_lse[NP];  // log2 units, of this CTA's part of a unit that a cluster shares
  int lim[NP];
};

// The pieces of a CTA's share: key tiles [kt, end) of the n of (b, hk), walked in order by every role.
struct Pieces {
  const PagedShape& s;
  int b, hk, kt, n, end;
  long long todo;  // positions from the piece on
  bool finished;
  SeqInfo seq;
  __device__ Pieces(const PagedShape& s_, const Share& sh, const DecUnits& first)
      : s(s_), b(sh.b), hk(sh.head), kt(0), n(0), end(0), todo(sh.todo), finished(false) {
    if (todo == 0) return;
    sequence(first);
    open(sh.tile);
  }
  __device__ void sequence(const DecUnits& x) {
    seq = x.q;
    n = x.count ? x.tiles() : 0;
  }
  __device__ void open(int at) {  // at: position within the unit
    kt = max(0, at - kDecOpen);
    const long long stop = at + todo - kDecOpen;
    end = stop < n ? (int)stop : n;
    todo -= min((long long)(n + kDecOpen - at), todo);
    if (end <= kt) finished = true;  // the share ends before the unit's first tile
  }
  __device__ bool done() const { return finished || n == 0; }
  __device__ bool whole() const { return kt == 0 && end == n; }
  __device__ void next() {
    if (todo == 0) {
      finished = true;
      return;
    }
    if (++hk == s.Hkv) {
      hk = 0;
      do {  // todo > 0: a later sequence has new tokens
        ++b;
        sequence(DecUnits(s, b));
      } while (n == 0);
    }
    open(0);
  }
};

// Reduce v[0 .. 16) over the 32 lanes; afterwards lane l holds column l / 2 in v[0]. A halving exchange: 16
// shuffles instead of 80.
template <typename F>
__device__ __forceinline__ void columns_reduce(float (&v)[16], int lane, F f) {
#pragma unroll
  for (int half = 8; half > 0; half >>= 1) {
    const bool up = lane & (2 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, 2 * half));
    }
  }
  v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

__device__ __forceinline__ bool vote_any(bool x, int id) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

struct DecWork {
  float* part_o;    // [2 CTAs][NP][D]
  float* part_lse;  // [2 CTAs][NP], log2 units
  int4* desc;       // [CTAs][2]: {b, hk, first CTA, its slot}, {L_q, q0, bb, 0} of the sequence; b = -1: no (sequence,
                    // head) ends here in pieces. Null: every (sequence, head) has a CTA or a cluster of its own
};

template <int D, int NP>
__global__ void __launch_bounds__(DecCfg<D, NP>::kThreads, DecCfg<D, NP>::kCtas)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const FaPagedArgs a, const DecWork wk) {
  using C = DecCfg<D, NP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) DecCtl<D, NP> ctl;
  const uint32_t sK0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sV0 = sK0 + C::kKStages * C::kTileBytes, sP = sV0 + C::kVStages * C::kTileBytes;
  const uint32_t sQ = sP + C::kPBytes;
  float* my_part = reinterpret_cast<float*>(smem_raw + (sK0 - smem_u32(smem_raw)));
  volatile int* abort_flag = &ctl.abort_flag;
  const PagedShape& s = a.s;
  const int G = s.H / s.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto sK = [&](int i) { return sK0 + i * C::kTileBytes; };
  auto sV = [&](int i) { return sV0 + i * C::kTileBytes; };
  auto bar = [&](uint64_t& x) { return smem_u32(&x); };

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      ctl.issued_q[i] = ctl.issued_t[i] = 0;
      mbar_init(bar(ctl.q_full[i]), D / 64);
      mbar_init(bar(ctl.q_empty[i]), 1);
      mbar_init(bar(ctl.s_full[i]), 1);
      mbar_init(bar(ctl.o_free[i]), 128 * C::kGroups);
      mbar_init(bar(ctl.p_ready[i]), 128 * C::kGroups);
      mbar_init(bar(ctl.pv_done[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(ctl.k_full[i]), D / 64);
      mbar_init(bar(ctl.k_empty[i]), 1);
      mbar_init(bar(ctl.v_full[i]), D / 64);
      mbar_init(bar(ctl.v_empty[i]), 1);
    }
    mbar_init(bar(ctl.drain), 1);
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (threadIdx.x < NP) ctl.part_lse[threadIdx.x] = -INFINITY;
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  // Rows of Q that no copy fills (the box has Nq G rows) are zero.
  const int box = s.Nq * G;
  for (int i = threadIdx.x; i < C::kQBufs * (D / 64) * (NP - box) * 8; i += C::kThreads) {
    const int r = box + i / 8 % (NP - box), part = i / 8 / (NP - box);  // part: buffer and column half
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(sQ + (part * NP + r) * 128 + (i & 7) * 16), "r"(0)
                 : "memory");
  }
  fence_proxy_async_smem();
  __syncthreads();
  let_dependent_start();  // (this CTA has its tensor memory: a dependent that takes some cannot be in its way)
  grid_dependency_wait();
  const int ctas = wk.desc != nullptr ? 1 : (int)cluster_size();  // that share a unit
  if (wk.desc != nullptr) {
    find_share<C::kThreads>(s.B, [&](int b) { return DecUnits(s, b); }, ctl.share, ctl.scan, ctl.units);
  } else if (threadIdx.x == 0) {  // tiles [n rank / ctas, n (rank + 1) / ctas) of the cluster's unit
    const int unit = blockIdx.x / ctas, rank = blockIdx.x - unit * ctas, b = unit / s.Hkv;
    const DecUnits x(s, b);
    const int n = x.count ? x.tiles() : 0, lo = n * rank / ctas, hi = n * (rank + 1) / ctas;
    ctl.share = Share{b, unit - b * s.Hkv, 0, kDecOpen + lo, hi - lo, 0, 0};
    ctl.units = x;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  Pieces w(s, ctl.share, ctl.units);
  if (wk.desc != nullptr && threadIdx.x == 0) {
    const bool joins = !w.done() && w.kt > 0 && w.end == w.n;
    wk.desc[2 * blockIdx.x] = make_int4(joins ? w.b : -1, w.hk, ctl.share.first_cta, ctl.share.first_slot);
    wk.desc[2 * blockIdx.x + 1] = make_int4(w.seq.Lq, w.seq.q0, w.seq.bb, 0);
  }

  if (warp == 0 || (D > 64 && warp == C::kThreads / 32 - 1)) {
    // ------------------------------------------------------------------ copies
    const int half = warp != 0;  // the 64 columns that this warp copies, of Q, K and V
    const int P = 1 << s.page_shift, rows = min(P, 128), shift = min(s.page_shift, 7), per = 128 >> shift;
    bool run = true;
    int t = 0;
    // Page of tile kt that this lane copies (-1, reported: none of the cache's, reads as zero).
    auto page_of = [&](const Pieces& x, int kt) -> int {
      const int key = (kt << 7) + (lane << shift);
      return lane < per && key < x.seq.Lk ? paged_page(s, x.b, key >> s.page_shift, a.status) : 0;
    };
    for (int piece = 0; !w.done(); ++piece) {
      const int qb = piece % C::kQBufs, qu = piece / C::kQBufs;
      int page = page_of(w, w.kt);
      if (run && qu > 0) run = mbar_wait(bar(ctl.q_empty[qb]), (qu - 1) & 1, abort_flag, a.status);
      run = __all_sync(0xffffffffu, run) && !*abort_flag;
      if (run && lane == 0) {
        mbar_expect_tx(bar(ctl.q_full[qb]), box * 128);
        tma_load_4d(sQ + (qb * (D / 64) + half) * NP * 128, &tmQ, half * 64, w.hk * G, w.seq.q0, w.seq.bb,
                    bar(ctl.q_full[qb]));
        ctl.issued_q[half] = piece + 1;
      }
      for (int kt = w.kt; kt < w.end; ++kt, ++t) {
        const int left = w.seq.Lk - (kt << 7), pages = left <= 0 ? 0 : min(per, (left + rows - 1) >> shift);
        const int slot = (kt << 7) & (P - 1);
        const int next = kt + 1 < w.end ? page_of(w, kt + 1) : 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int stages = x ? C::kVStages : C::kKStages, st = t % stages, u = t / stages;
          const uint32_t full = x ? bar(ctl.v_full[st]) : bar(ctl.k_full[st]);
          if (run && u > 0)
            run = mbar_wait(x ? bar(ctl.v_empty[st]) : bar(ctl.k_empty[st]), (u - 1) & 1, abort_flag, a.status);
          run = __all_sync(0xffffffffu, run) && !*abort_flag;
#ifdef FA_TEST_WITHHOLD_KV  // a test-only build: every wait for keys and values must run out cleanly
          run = false;
#endif
          if (!run) continue;
          if (lane == 0) {
            mbar_expect_tx(full, pages * rows * 128);
            ctl.issued_t[half] = 2 * t + x + 1;
          }
          __syncwarp();
          if (lane < pages)
            tma_load_4d((x ? sV(st) : sK(st)) + half * 16384 + lane * rows * 128, x ? &tmV : &tmK, half * 64, slot, w.hk,
                        page, full);
        }
        page = next;
      }
      w.next();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      // An MMA takes this thread about 70 cycles and everything between MMAs adds to a tile's time, so the
      // positions in the rings are counters and descriptors are built once.
      bool run = true;
      Pieces v = w;  // the piece of the next S
      int left = v.end - v.kt, ks = 0, vpiece = 0;  // its key tiles without S; ring position
      uint32_t kphase = 0, sb = 0;
      bool opens = true;
      const uint64_t dk0 = desc_kmajor_sw128(sK(0)), dq0 = desc_kmajor_sw128(sQ), dv0 = desc_mnmajor_sw128(sV(0), 16384);
      const uint64_t dp0 = desc_mnmajor_sw128(sP, 16384);
      auto issue_s = [&]() {
        const int qb = vpiece & 1;
        if (run && opens) run = mbar_wait_spin(bar(ctl.q_full[qb]), (vpiece >> 1) & 1, abort_flag, a.status);
        if (run) run = mbar_wait_spin(bar(ctl.k_full[ks]), kphase, abort_flag, a.status);
        fence_after_sync();
        if (run) {
          const uint64_t dk = desc_add(dk0, ks * C::kTileBytes), dq = desc_add(dq0, qb * C::kQBytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + sb * NP, desc_add(dk, (kk >> 2) * 16384 + (kk & 3) * 32),
                   desc_add(dq, (kk >> 2) * NP * 128 + (kk & 3) * 32), C::kIdS, kk > 0);
          mma_commit(bar(ctl.s_full[sb]));
          mma_commit(bar(ctl.k_empty[ks]));
          if (left == 1) mma_commit(bar(ctl.q_empty[qb]));
        }
        sb ^= 1;
        if (++ks == C::kKStages) {
          ks = 0;
          kphase ^= 1;
        }
        opens = --left == 0;
        if (opens) {
          v.next();
          left = v.end - v.kt;
          ++vpiece;
        }
      };
      if (!w.done()) issue_s();
      int vs = 0;
      uint32_t vphase = 0, pb = 0, pphase = 0;
      for (int piece = 0; !w.done(); ++piece) {
        const uint32_t tO = tmem + (2 + (piece & 1)) * NP;
        for (int kt = w.kt; kt < w.end; ++kt) {
          if (!v.done()) issue_s();
          if (run) run = mbar_wait_spin(bar(ctl.p_ready[pb]), pphase, abort_flag, a.status);
          if (run) run = mbar_wait_spin(bar(ctl.v_full[vs]), vphase, abort_flag, a.status);
          if (run && kt == w.kt && piece >= 2)
            run = mbar_wait_spin(bar(ctl.o_free[piece & 1]), ((piece >> 1) - 1) & 1, abort_flag, a.status);
          fence_after_sync();
          if (run) {
            const uint64_t dv = desc_add(dv0, vs * C::kTileBytes), dp = desc_add(dp0, pb * C::kPStep);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ss(tO, desc_add(dv, kk * 2048), desc_add(dp, kk * 2048), C::kIdPV, kk > 0 || kt > w.kt);
            mma_commit(bar(ctl.v_empty[vs]));
            mma_commit(bar(ctl.pv_done[pb]));
          }
          pphase ^= pb;
          pb ^= 1;
          if (++vs == C::kVStages) {
            vs = 0;
            vphase ^= 1;
          }
        }
        w.next();
      }
      mma_commit(bar(ctl.drain));
      mbar_wait_drain(bar(ctl.drain), 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax, epilogue
    const int quad = warp & 3, r = quad * 32 + lane;  // key within the tile; head dimension of O^T
    constexpr int NC = 16;
    const int gr = C::kGroups == 1 ? 0 : (warp - 2) >> 2, n0 = gr * NC, on = 1 + gr;  // group, first column, barrier
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float sl2 = a.scale * kLog2e;
    bool run = true;
    int t = 0;
    auto wait_pv = [&](int j) -> bool {  // P V of tile j has completed
      return mbar_wait(bar(ctl.pv_done[j & 1]), (j >> 1) & 1, abort_flag, a.status);
    };
    for (int piece = 0; !w.done(); ++piece) {
      const SeqInfo& seq = w.seq;
      const int live = seq.Lq * G;  // rows that exist
      const uint32_t tO = tmem + lane_off + (2 + (piece & 1)) * NP + n0;
      if (r < NC) ctl.lim[n0 + r] = s.causal ? min(seq.Lk, (n0 + r) / G + seq.off + 1) : seq.Lk;  // keys [0, lim) visible
      const int least = s.causal ? min(seq.Lk, seq.off + 1) : seq.Lk;
      float l[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) l[n] = 0.f;
      for (int kt = w.kt; kt < w.end; ++kt, ++t) {
        if (run) run = mbar_wait(bar(ctl.s_full[t & 1]), (t >> 1) & 1, abort_flag, a.status);
        fence_after_sync();
        float x[NC];
        {
          tmem_ld16(tmem + lane_off + (t & 1) * NP + n0, reinterpret_cast<uint32_t(&)[NC]>(x));
          tmem_ld_wait();
        }
        const int key = (kt << 7) + r;
        const bool opens = kt == w.kt;
        if (opens) named_bar_sync(on, 128);  // ctl.lim is written; the last piece's ctl.m is no longer read
        if ((kt << 7) + 128 > least) {
#pragma unroll
          for (int n = 0; n < NC; ++n) x[n] = key < ctl.lim[n0 + n] ? x[n] : -INFINITY;
        }
        bool raise = opens;
        if (!opens) {
          bool big = false;
#pragma unroll
          for (int n = 0; n < NC; n += 4) {
            const float4 m = *reinterpret_cast<const float4*>(ctl.m + n0 + n);
            big |= fmaxf(fmax3(fmaf(x[n], sl2, -m.x), fmaf(x[n + 1], sl2, -m.y), fmaf(x[n + 2], sl2, -m.z)),
                         fmaf(x[n + 3], sl2, -m.w)) > kRaise;
          }
          raise = vote_any(big, on);
        }
        if (raise) {
          float y[NC];
#pragma unroll
          for (int n = 0; n < NC; ++n) y[n] = x[n] * sl2;
          columns_reduce(y, lane, [](float p, float q) { return fmaxf(p, q); });
          ctl.wmax[quad][n0 + (lane >> 1)] = y[0];
          named_bar_sync(on, 128);
          if (r < NC) {
            const int n = n0 + r;
            const float old = opens ? kNoMax : ctl.m[n];
            const float now = fmaxf(fmaxf(fmaxf(ctl.wmax[0][n], ctl.wmax[1][n]), fmaxf(ctl.wmax[2][n], ctl.wmax[3][n])),
                                    old);
            ctl.alpha[n] = ex2_approx(old - now);
            ctl.m[n] = now;
          }
          __syncwarp();
          named_bar_sync(on, 128);
          if (!opens) {
            if (run) run = wait_pv(t - 1);
            fence_after_sync();
            uint32_t o[NC];
            tmem_ld16(tO, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < NC; ++i) {
              const float alpha = ctl.alpha[n0 + i];
              o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              l[i] *= alpha;
            }
            tmem_st16(tO, o);
            tmem_st_wait();
          }
        }
        // P is rounded to bf16, the type of V beside it in the product (off by 2^-8 of each probability at most); the sum
        // that O is divided by takes it unrounded.
        uint32_t pk[NC / 2];
#pragma unroll
        for (int n = 0; n < NC; n += 4) {
          const float4 m = *reinterpret_cast<const float4*>(ctl.m + n0 + n);
          const float p0 = ex2_approx(fmaf(x[n], sl2, -m.x)), p1 = ex2_approx(fmaf(x[n + 1], sl2, -m.y));
          const float p2 = ex2_approx(fmaf(x[n + 2], sl2, -m.z)), p3 = ex2_approx(fmaf(x[n + 3], sl2, -m.w));
          l[n] += p0;
          l[n + 1] += p1;
          l[n + 2] += p2;
          l[n + 3] += p3;
          pk[n / 2] = pack_bf16x2(p0, p1);
          pk[n / 2 + 1] = pack_bf16x2(p2, p3);
        }
        // P's buffer is free: the P V that read it, of tile t - 2, was issued before S of tile t, which has
        // completed.
        const uint32_t sPt = sP + (NP == 64 ? (t & 1) * C::kPStep : 0);
        const int c0 = n0 / 8 + (NP == 64 ? 0 : (t & 1) * (C::kPStep / 16));  // first 16-byte chunk of the row
#pragma unroll
        for (int c = 0; c < NC / 8; ++c)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(sPt + r * 128 + (((c + c0) ^ (r & 7)) << 4)),
                       "r"(pk[4 * c]), "r"(pk[4 * c + 1]), "r"(pk[4 * c + 2]), "r"(pk[4 * c + 3])
                       : "memory");
        // Value rows past the last key may hold anything, and 0 times NaN is NaN: they become 0.
        const int valid = seq.Lk - (kt << 7);
        if (valid < 128) {
          const int st = t % C::kVStages;
          if (run) run = mbar_wait(bar(ctl.v_full[st]), (t / C::kVStages) & 1, abort_flag, a.status);
          if (run && r >= valid)
#pragma unroll
            for (int c = gr * (D / 8 / C::kGroups); c < (gr + 1) * (D / 8 / C::kGroups); ++c)
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(sV(st) + (c >> 3) * 16384 + r * 128 +
                                                                          (c & 7) * 16),
                           "r"(0)
                           : "memory");
          __syncwarp();
        }
        fence_proxy_async_smem();
        fence_before_sync();
        if (run) mbar_arrive(bar(ctl.p_ready[t & 1]));
      }
      // ---------------------------------------------------------------- end of the piece
      columns_reduce(l, lane, [](float p, float q) { return p + q; });
      ctl.wmax[quad][n0 + (lane >> 1)] = l[0];
      named_bar_sync(on, 128);
      const bool whole = w.whole() && ctas == 1;
      const int slot = 2 * blockIdx.x + (piece == 0 ? 0 : 1);
      if (r < NC) {
        const int n = n0 + r;
        const float sum = (ctl.wmax[0][n] + ctl.wmax[1][n]) + (ctl.wmax[2][n] + ctl.wmax[3][n]);
        ctl.alpha[n] = sum == 0.f ? 0.f : 1.f / sum;  // (0: no visible key; a NaN stays one)
        const float lse2 = sum == 0.f ? -INFINITY : ctl.m[n] + log2f(sum);
        if (whole) {
          if (n < live) a.lse[paged_row(s, seq, w.b, w.hk * G + n % G, n / G)] = lse2 * kLn2;
        } else {
          (ctas > 1 ? ctl.part_lse : wk.part_lse + (size_t)slot * NP)[n] = lse2;
        }
      }
      __syncwarp();
      named_bar_sync(on, 128);
      if (run) run = wait_pv(t - 1);
      fence_after_sync();
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + elem_offset(a.so, seq.bb, seq.q0, w.hk * G) + r;
      // (the cluster's parts lie over the ring: with the last P V done nothing reads it or is on its way there)
      float* part = (ctas > 1 ? my_part : wk.part_o + (size_t)slot * NP * D) + r;
      int i = n0 / G, g = n0 % G;  // token and head of the group of column n
      uint32_t o[NC];
      tmem_ld16(tO, o);
      tmem_ld_wait();
      if (r < D) {
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          const int n = n0 + k;
          if (n < live) {
            const float val = __uint_as_float(o[k]) * ctl.alpha[n];
            if (whole)
              out[(size_t)i * a.so.row + (size_t)g * a.so.head] = __float2bfloat16(val);
            else
              part[n * D] = val;
          }
          if (++g == G) {
            g = 0;
            ++i;
          }
        }
      }
      fence_before_sync();
      if (run) mbar_arrive(bar(ctl.o_free[piece & 1]));
      w.next();
    }
  }

  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (ctas > 1) {
    // The cluster's CTAs join their parts, each some of the elements: M = max LSE, w = 2^(LSE - M), O = sum w O / sum w.
    cluster_sync();
    const SeqInfo& seq = ctl.units.q;
    const int unit = blockIdx.x / ctas, rank = blockIdx.x - unit * ctas, b = unit / s.Hkv, hk = unit - b * s.Hkv;
    for (int x = rank * C::kThreads + threadIdx.x; x < seq.Lq * G * (D / 4); x += ctas * C::kThreads) {
      const int n = x / (D / 4), e = x % (D / 4) * 4, i = n / G, h = hk * G + n - i * G;
      float l[kDecCluster], M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int c = 0; c < kDecCluster; ++c) {
        l[c] = c < ctas ? load_peer(ctl.part_lse + n, c) : -INFINITY;
        M = fmaxf(M, l[c]);
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kDecCluster; ++c)
        if (l[c] != -INFINITY) {
          const float wt = exp2f(l[c] - M);
          const float4 o = load_peer4(my_part + n * D + e, c);
          sum += wt;
          acc = make_float4(acc.x + wt * o.x, acc.y + wt * o.y, acc.z + wt * o.z, acc.w + wt * o.w);
        }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.o) + elem_offset(a.so, seq.bb, seq.q0 + i, h) + e) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (e == 0) a.lse[paged_row(s, seq, b, h, i)] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
    cluster_sync();  // no CTA leaves while its part is read
  }
  if (threadIdx.x == 0 && *abort_flag) {
    // Copies still in flight land before the CTA exits: the last one issued into each buffer. A producer that stopped
    // before the other did has its arrival made here.
    const int nq = max(ctl.issued_q[0], ctl.issued_q[1]), nt = max(ctl.issued_t[0], ctl.issued_t[1]);
    auto drain = [&](uint64_t& full, int parity, const int (&issued)[2], int i) {
      for (int p = 0; p < D / 64; ++p)
        if (issued[p] <= i) mbar_arrive(bar(full));
      mbar_wait_drain(bar(full), parity);
    };
    for (int i = max(0, nq - C::kQBufs); i < nq; ++i)
      drain(ctl.q_full[i % C::kQBufs], (i / C::kQBufs) & 1, ctl.issued_q, i);
    for (int i = max(0, nt - 8); i < nt; ++i) {
      const int t = i >> 1, stages = (i & 1) ? C::kVStages : C::kKStages;
      if (t + stages <= (nt - 1 - (i & 1)) >> 1) continue;  // a later copy used the buffer
      drain((i & 1) ? ctl.v_full[t % stages] : ctl.k_full[t % stages], (t / stages) & 1, ctl.issued_t, i);
    }
  }
}

// Joins the pieces of each divided (sequence, head). Block (c, y) takes 16 rows of the one that ends in CTA c's
// first piece, if it began before; a thread has four elements of a row.
template <int D, int NP>
__global__ void __launch_bounds__(4 * D) paged_join_kernel(const FaPagedArgs a, const DecWork wk) {
  let_dependent_start();
  grid_dependency_wait();
  const int4 d = wk.desc[2 * blockIdx.x], of = wk.desc[2 * blockIdx.x + 1];
  const PagedShape& s = a.s;
  const int G = s.H / s.Hkv, n = blockIdx.y * 16 + threadIdx.x / (D / 4), e = threadIdx.x % (D / 4) * 4;
  if (d.x < 0 || n >= of.x * G) return;
  SeqInfo seq{};
  seq.Lq = of.x;
  seq.q0 = of.y;
  seq.bb = of.z;
  join_pieces<D, NP>(a, wk.part_o, wk.part_lse, d.z, blockIdx.x, d.w, n, e, seq, d.x, n / G, d.y * G + n % G);
}

int padded_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// CTAs that share a (sequence, head) unit where nothing is divided by the lengths, or 0. Alone up to two tiles (one
// sequence of 8 K/V heads, d = 128, 250 keys: 6.8 us with 1 CTA a unit, 7.1 with 2, 7.6 with 8, 8.4 divided), else the
// largest cluster that does not outnumber the tiles twice and of which all run at once (16 clusters of 8 do not, 15.9
// us for 8.5): a cluster lies within a part of the chip, and 152 SMs hold 15 clusters of 8, 36 of 4 and 76 of 2 at a CTA
// per SM (by cudaOccupancyMaxActiveClusters). The rule takes 8 up to 2/3 of the CTAs and 4 up to 7/8 (12 and 33 clusters),
// which leaves some where other work has SMs of such a part. At most four tiles a CTA of a cluster (777 keys: 8.5 us with
// 8, 8.9 with 4, 9.6 divided; 4096 keys: 11.1 with 8, 11.6 divided; 8192 keys: 15.4 and 13.6) or eight of one alone (16
// sequences of 8 heads, 1024 keys: 13.9 and 17.2; of 12 heads of d = 64: 13.8 and 15.8, of 2048 keys 26 and 24).
int unit_ctas(const PagedShape& s, int num_sms) {
  const long long units = (long long)s.B * s.Hkv, room = (long long)num_sms * dec_ctas(s.d, padded_rows(s.Nq * (s.H / s.Hkv)));
  const int tiles = (s.max_k + 127) >> 7;
  int ctas = 1;
  if (tiles > 2) {
    if (tiles > 4 && units * 8 * 3 <= room * 2)
      ctas = 8;
    else if (units * 4 * 8 <= room * 7)
      ctas = 4;
    else if (units * 2 <= room)
      ctas = 2;
  }
  return units * ctas <= room && tiles <= (ctas == 1 ? 8 : 4 * ctas) ? ctas : 0;
}

template <int D, int NP>
cudaError_t launch_decode(const FaPagedArgs& a, cudaStream_t st) {
  using C = DecCfg<D, NP>;
  const PagedShape& s = a.s;
  const bool packed = s.cu_q != nullptr;
  const int G = s.H / s.Hkv;
  CUtensorMap tq, tk, tv;
  // Q by tokens and heads: a box holds the G heads of a K/V head for Nq tokens, in row order token G + head.
  if (!fa_make_tmap_bf16(&tq, a.q, D, s.H, packed ? s.rows_q : s.Nq, packed ? 1 : s.B, a.sq.head, a.sq.row, a.sq.batch,
                         G, s.Nq) ||
      !paged_tmap(&tk, a.k, s, a.sk) || !paged_tmap(&tv, a.v, s, a.sv))
    return cudaErrorInvalidValue;
  const int shared = unit_ctas(s, a.num_sms), ctas = shared > 0 ? s.B * s.Hkv * shared : a.num_sms * C::kCtas;
  DecWork wk{};
  if (shared == 0) {
    char* ws = static_cast<char*>(a.workspace);
    wk.desc = reinterpret_cast<int4*>(ws);
    ws += up256((size_t)ctas * 2 * sizeof(int4));
    wk.part_lse = reinterpret_cast<float*>(ws);
    ws += up256((size_t)ctas * 2 * NP * sizeof(float));
    wk.part_o = reinterpret_cast<float*>(ws);
  }
  auto kern = paged_decode_kernel<D, NP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if (C::kCtas > 1) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  if (shared > 0)
    return launch_dependent_cluster(kern, dim3(ctas), dim3(C::kThreads), C::kSmem, shared, st, tq, tk, tv, a, wk);
  e = launch_dependent(kern, dim3(ctas), dim3(C::kThreads), C::kSmem, st, tq, tk, tv, a, wk);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_join_kernel<D, NP>, dim3(ctas, NP / 16), dim3(4 * D), 0, st, a, wk);
}

}  // namespace
}  // namespace fa

size_t fa_paged_decode_workspace(const fa::PagedShape& s, int num_sms) {
  if (fa::unit_ctas(s, num_sms) > 0) return 0;
  const int np = fa::padded_rows(s.Nq * (s.H / s.Hkv));
  const size_t ctas = (size_t)num_sms * fa::dec_ctas(s.d, np), rows = ctas * 2 * np;
  return fa::up256(ctas * 2 * sizeof(int4)) + fa::up256(rows * sizeof(float)) + rows * s.d * sizeof(float);
}

cudaError_t fa_launch_paged_decode(const FaPagedArgs& a, cudaStream_t st) {
  const int np = fa::padded_rows(a.s.Nq * (a.s.H / a.s.Hkv));
  if (a.s.d == 64)
    return np == 16   ? fa::launch_decode<64, 16>(a, st)
           : np == 32 ? fa::launch_decode<64, 32>(a, st)
                      : fa::launch_decode<64, 64>(a, st);
  return np == 16   ? fa::launch_decode<128, 16>(a, st)
         : np == 32 ? fa::launch_decode<128, 32>(a, st)
                    : fa::launch_decode<128, 64>(a, st);
}
