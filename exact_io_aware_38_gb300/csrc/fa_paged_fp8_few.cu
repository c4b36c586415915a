// Attention of a few new tokens per sequence over a paged cache held in 8 bits (decode, drafted tokens, short chunks): bound by
// reading K and V once, half the bytes of the bf16 cache.
//
// What it computes: as fa_paged_decode.cu, S^T = K Q^T with a key on each tensor-memory lane and a row on each column, and
// O^T += V^T P^T, but the products take the e4m3 bytes as they lie in the cache (kind::f8f6f4), so nothing is converted on
// its way and a 128-key tile is half as many bytes and products. The other operands are split into parts of 8 bits:
//   Q  a row is scaled by a power of two to a largest element in [128, 256) and split into hi + lo / 32, both e4m3: a bf16
//      number has 8 bits, hi takes 4 and the signed rest 4, so the sum is exact for elements from the largest's binade to 2^-14 of it;
//      smaller ones are off by at most 2^-22 of the largest.
//   P  = hi + mid / 8 + lo / 64, three e5m2 numbers cut from its fp16 rounding: off by 2^-11 (fp16) and 2^-9 (lo) of its binade,
//      together by 1.1 x 2^-9 of a probability at most (bf16 2^-8), or by 1.25 x 2^-23 where that is more; the row's largest is
//      2^7 at least. The factors lift mid and lo out of e5m2's last bits (2^-16): without them 2^18 equal keys of one piece beside a key
//      of about their weight were off by up to 2.3%, 2^20 by 11%; with them by no more than O's rounding (2^-8).
// The parts lie side by side as columns of one product (N = 2 rows for S, 3 rows for O), and are added up in fp32 when they
// are read: at few rows the columns cost nothing beside the 128 lanes.
//
// The exponents of a key and its value are a lane's: the key's scales the scores of its lane, and the value's goes into the
// exponent of P, y = c s 2^k log2 e + v, P = 2^(y - ref). So P V needs no further factor, and the reference follows the
// products P |V|: a key with much weight but a tiny value (or none) does not push the others out of e5m2's range. The row sum
// takes P 2^-v, which must not be lost where P is too small for fp32: the exponential is taken without v where v < 0 and P is a lane's
// constant times it; where v > 0 the sum's FMA has the constant (else keys of values of zeros beside 2^60 are missing from the sums; the
// multiplication costs 1%: 4096 x 128 keys of 12 heads, d = 64, 362 -> 365 us, 48 x 1024, 20 rows, 38.3 -> 38.9).
//
// The exponentials are taken against a reference per row that starts 2^7 below the first tile's largest and is raised
// (O and the row sums rescaled) only when a score exceeds it by more than 2^15.
//
// Rows: up to 64 (tokens x heads of a K/V head) are one unit of 8, 16, 32 or 64 columns; more are up to four units that each
// read the keys, mostly from L2: of more tokens, or of a token's heads where there are more than 64 (64 x 4096 keys of one head,
// d = 128, with 128 heads on it: 54 us, 84 read back to bf16; 65 heads 51 and 1539). Division of the work, pieces,
// clusters and joins as in fa_paged_decode.cu.
//
// Roles: warp 0 copies keys and codes (TMA, a lane per page; the codes by 8-byte asynchronous copies, four keys a lane), warp 1
// issues S, groups of four warps are the softmax and the epilogue, of 16 rows each, the warp before the last issues P V, and
// the last copies values and splits Q, a piece ahead. Each of these takes 600 to 1300 cycles a tile: one thread that issued both
// products took 2000, and issuers that also copied more, since whatever follows an MMA waits for its dispatch.
#include <cuda_fp16.h>

#include "fa_paged_few.cuh"
#include "fa_tmap.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace tc;

constexpr float kFirst = 7.f;    // log2 units that the reference starts below the first tile's largest
constexpr float kRaise8 = 15.f;  // and that a score may exceed it by: 2^15 is near the top of e5m2 and fp16
constexpr float kLoScale = 32.f;
constexpr float kMidScale = 8.f;  // of P's second part; the third's is its square
constexpr int kZeroRow = -80;    // exponent that stands for a value row of zeros: only its place in the row sum counts

constexpr int few8_ctas(int np) { return np <= 16 ? 2 : 1; }  // per SM

template <int D, int NP>
struct F8Cfg {
  static constexpr int kTileBytes = 128 * D;
  static constexpr int kCtas = few8_ctas(NP);
  // Rows of a group of four softmax warps, and groups: eight of 8 rows, a shorter chain of steps with twice the warps, else 16. Of 17 to 32
  // rows at d = 128 groups of 16 are ahead (16 x 4099 keys, 20 rows: 30.5 us, of 8 31.7; 64 x 8192 keys, 24 rows 151 and 159), at d = 64
  // mostly groups of 8 (512 x 500 keys of 12 heads, 24 rows 266 and 218, 48 x 1024 39.8 and 38.9, 64 x 4096 116 and 126). Of 16 rows, twice
  // on an SM, groups of 16 (16 x 4099 keys 26.7 and, of 8, 26.8; 48 x 1024 keys of 12 heads, d = 64, 24.4 and 25.4).
  static constexpr int kCols = NP == 8 || (NP == 32 && D == 64) ? 8 : 16, kGroups = NP / kCols;
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kKStages = NP <= 16 ? (D == 128 ? 3 : 5) : NP == 32 ? (D == 128 ? 5 : 8) : D == 128 ? 4 : 6;
  static constexpr int kVStages = NP <= 16 ? (D == 128 ? 2 : 5) : NP == 32 ? (D == 128 ? 5 : 8) : D == 128 ? 3 : 6;
  static constexpr int kQBytes = 2 * NP * D, kQBufs = 2;
  // Columns of P V: three parts of every row (at 8 rows a fourth, unused, since N is a multiple of 16).
  static constexpr int kParts = NP == 8 ? 32 : 3 * NP;
  // P: 128 keys, a row of kParts bytes each, cut into blocks of 128. Two buffers: up to 16 rows side by side in a row, else
  // one behind the other.
  static constexpr int kPBlocks = (kParts + 127) / 128;
  static constexpr int kPStep = NP <= 16 ? 64 : kPBlocks * 16384;
  static constexpr int kPBytes = NP <= 16 ? 16384 : 2 * kPStep;
  static constexpr int kSmem = kQBufs * kQBytes + (kKStages + kVStages) * kTileBytes + kPBytes + 1024;
  static constexpr bool kSoftSplit = NP > 16;  // the softmax warps split Q
  // Tensor memory: S x 2, then O. One O is enough: the first P of a piece follows the last one's epilogue.
  static constexpr uint32_t kO = 4 * NP;
  static constexpr uint32_t kTmemCols = NP == 8 ? 64 : NP == 16 ? 128 : NP == 32 ? 256 : 512;
  static_assert(kO + kParts <= kTmemCols);
  static constexpr uint32_t kIdS = idesc_e4m3(128, 2 * NP);
  // O^T has D rows; at D = 64 the upper 64 lanes multiply whatever follows V in shared memory and are never read.
  static constexpr uint32_t kIdPV = idesc_e4m3_e5m2_mn(128, kParts);
};

// Codes wait in a ring of their own, longer than the keys' (whose copies they go with): a copy of keys t follows S of t - kKStages,
// which follows P V of two tiles before that, so the codes of t - 16 are read.
constexpr int kCodeStages = 16;

// Positions of a unit before its first tile, for its epilogue and the first tile of the next (weighed as 1 and 3: 16 x 2048 keys of 32
// heads 39.3 and 38.7 us; 64 x 8192 keys 123.0 and 123.1, 64 x 4096 of 12 heads at d = 64 56.9 and 57.0).
constexpr int kF8Open = 3;
// Positions fit an int: a sequence with new tokens has at most 4 units a head of max_k / 128 + 4 positions each, sequences times
// heads are fewer than 2^26 and times keys fewer than 2^31 (checked by the caller). In 64 bits the search for a CTA's share
// is longer code, each line of which is waited for at the start (48 x 1024 keys of 12 heads, d = 64: 23.4 us, so 22.6).

// How the work is cut. The K/V heads of a sequence are `turns` turns of `side` neighbours each: CTA c takes head c % side of every
// turn, and the line of units that the CTAs of one residue divide has a turn where it would have a head. So `side` CTAs walk
// over the same keys of neighbouring heads at about the same time, and what lies next to one another in memory is
// fetched at about the same time.
// A unit has `tokens` tokens of all heads of a K/V head, or, of more than 64 heads, one token of one of `parts` parts of them
// (a kernel of its own: these divisions alone cost the others 1 to 10%).
struct F8Cut {
  int tokens;               // of a unit
  int heads, group, parts;  // of a K/V head, of a unit; units of a token
  int side, turns;
};

template <bool kParts>  // more than one unit of a token
struct F8Units {
  int heads, count, open;
  SeqInfo q;
  F8Units() = default;
  __device__ F8Units(const PagedShape& s, const F8Cut& c, int b) : heads(c.turns), open(kF8Open), q(paged_part(s, b)) {
    count = q.Lq <= c.tokens ? q.Lq > 0 : (q.Lq + c.tokens - 1) / c.tokens;
    if (kParts) count *= c.parts;
  }
  __device__ int tiles(int = 0) const { return max(1, (q.Lk + 127) >> 7); }
  __device__ int before(int u) const { return u * (tiles() + open); }
};

template <int D, int NP, bool kParts>
struct F8Ctl {
  uint64_t q_raw[2], q_full[2], q_empty[2];
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];  // (k_full: codes too; v_empty: also that P V has completed)
  uint64_t s_full[2];
  uint64_t p_ready[2];  // per buffer of P
  uint64_t drain[2];    // per issuer
  uint32_t tmem_base;
  int abort_flag;
  int scan[F8Cfg<D, NP>::kThreads / 32];  // an entry per warp
  ShareOf<int> share;
  F8Units<kParts> units;     // of the sequence where the share begins
  int issued_k, issued_v;    // copies issued (abort-path drain)
  alignas(16) uint8_t codes[kCodeStages][256];  // key and value of each slot
  alignas(16) float qmul[2][NP];      // by buffer of Q: c log2 e times the row's power of two
  alignas(16) float ref[NP];
  alignas(16) float alpha[NP], root[NP];  // a raise's factor, and its square root
  float wmax[4][NP];
  float part_lse[NP];  // log2 units, of this CTA's part of a unit that a cluster shares
  int lim[NP];
};

// The pieces of a CTA's share: key tiles [kt, end) of the n of (b, hk, u), walked in order by every role.
template <bool kParts>
struct F8Pieces {
  const PagedShape& s;
  const F8Cut& cut;
  int b, hk, u, kt, n, end, count;
  int todo;  // positions from the piece on
  bool finished;
  SeqInfo seq;
  __device__ F8Pieces(const PagedShape& s_, const F8Cut& cut_, const ShareOf<int>& sh, const F8Units<kParts>& first, int beside)
      : s(s_), cut(cut_), b(sh.b), hk(sh.head * cut.side + beside), u(sh.unit), kt(0), n(0), end(0), count(0), todo(sh.todo),
        finished(false) {
    if (todo == 0) return;
    sequence(first);
    open(sh.tile);
  }
  __device__ void sequence(const F8Units<kParts>& x) {
    seq = x.q;
    count = x.count;
    n = count ? x.tiles() : 0;
  }
  __device__ void open(int at) {  // at: position within the unit
    kt = max(0, at - kF8Open);
    end = min(at + todo - kF8Open, n);
    todo -= min(n + kF8Open - at, todo);
    if (end <= kt) finished = true;  // the share ends before the unit's first tile
  }
  __device__ bool done() const { return finished || n == 0; }
  __device__ bool whole() const { return kt == 0 && end == n; }
  __device__ bool more() const { return todo > kF8Open; }  // another piece follows
  // The unit's first token and head, and its rows.
  __device__ int token() const { return kParts ? u / cut.parts : u * cut.tokens; }
  __device__ int head() const { return kParts ? hk * cut.heads + u % cut.parts * cut.group : hk * cut.group; }
  __device__ int rows() const {
    return kParts ? min(cut.group, (hk + 1) * cut.heads - head()) : min(cut.tokens, seq.Lq - token()) * cut.group;
  }
  __device__ void next() {
    if (todo == 0) {
      finished = true;
      return;
    }
    if (++u == count) {
      u = 0;
      hk += cut.side;
      if (hk >= s.Hkv) {
        hk -= s.Hkv;
        do {  // todo > 0: a later sequence has new tokens
          ++b;
          sequence(F8Units<kParts>(s, cut, b));
        } while (n == 0);
      }
    }
    open(0);
  }
};

struct F8Work {
  float* part_o;    // [2 CTAs][NP][D]
  float* part_lse;  // [2 CTAs][NP], log2 units
  int4* desc;       // [CTAs][2]: {b, first head, first CTA, its slot}, {rows, q0, bb, first token} of the unit; b = -1: none
                    // ends here in pieces. Null: every unit has a CTA or a cluster of its own
  F8Cut cut;
  FastDiv by_group;  // rows to tokens
};

// What the kernel needs of FaPagedArgs: a role's first look at a line of its arguments is a miss.
struct F8Args {
  PagedShape s;
  const void* q;
  const uint8_t* codes;
  void* o;
  float* lse;
  FaStrides sq, so;
  float scale;
  int* status;
};

// A wait that is mostly over when it is asked for: what else it takes is a call, out of the way of the code around it, since the
// kernel waits for its instructions (512 x 500 keys of 12 heads, d = 64, 16 rows: 218 us inline and 140). Not for the issuers of MMAs
// (16 x 4099 keys, 16 rows: 26 and 29.5).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return mbar_wait(bar, parity, abort_flag, status);
}
__device__ __forceinline__ bool wait_near(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (__builtin_expect(mbar_try(bar, parity), 1)) return true;
  return wait_on(bar, parity, abort_flag, status);
}

// Two probabilities' parts: hi and mid by cutting their fp16 after two fraction bits (a byte), lo by rounding the rest; mid is held 8 and
// lo 64 times larger. All of it but the fp16 and lo's rounding is exact, also among fp16's subnormals: P is at most 2^15, what is left
// of it after hi less than 2^12, after mid less than 2^9.
__device__ __forceinline__ void split_p(float p0, float p1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  __half2 h = __floats2half2_rn(p0, p1);
  hi = *reinterpret_cast<uint32_t*>(&h) & 0xff00ff00u;
  const __half2 eight = __float2half2_rn(kMidScale);
  __half2 r = __hmul2(__hsub2(h, *reinterpret_cast<__half2*>(&hi)), eight);
  mid = *reinterpret_cast<uint32_t*>(&r) & 0xff00ff00u;
  r = __hmul2(__hsub2(r, *reinterpret_cast<__half2*>(&mid)), eight);
  uint16_t y;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(y) : "r"(*reinterpret_cast<uint32_t*>(&r)));
  lo = y;
}

__device__ __forceinline__ void load_cols(uint32_t at, uint32_t (&r)[16]) { tmem_ld16(at, r); }
__device__ __forceinline__ void load_cols(uint32_t at, uint32_t (&r)[8]) { tmem_ld8(at, r); }
__device__ __forceinline__ void store_cols(uint32_t at, const uint32_t (&r)[16]) { tmem_st16(at, r); }
__device__ __forceinline__ void store_cols(uint32_t at, const uint32_t (&r)[8]) { tmem_st8(at, r); }

__device__ __forceinline__ void store16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Where 16 bytes of row n of Q lie as they arrive: the row's first half in hi's place, its second in lo's.
template <int D, int NP>
__device__ __forceinline__ uint32_t raw_q(uint32_t q, int n, int part) {
  return q + (part / (D / 16) * NP + n) * D + part % (D / 16) * 16;
}

// Splits kTimes x 256 / D rows from `first` on in place, by a warp: D / 8 lanes a row. store: false where the buffer may still be
// in use (after a wait that ran out).
template <int D, int NP, int kTimes>
__device__ __forceinline__ void split_rows(uint32_t q, float* qmul, int first, float sl2, bool store) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;
  const int lane = threadIdx.x & 31, r0 = lane / kLanes, part = lane % kLanes;
#pragma unroll
  for (int k = 0; k < kTimes; ++k) {
    const int n = first + k * kPer + r0;
    uint32_t v[4];
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(raw_q<D, NP>(q, n, part))
                 : "memory");
    uint32_t m = 0;  // magnitudes of two elements in each word: bf16 bits without the sign are ordered as integers
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, v[i] & 0x7fff7fffu);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t top = max(m & 0xffffu, m >> 16);
    const bool bad = top >= 0x7f80u;
    const uint32_t code = (top >> 7) > 8 ? (top >> 7) - 7 : 1;
    const float by = bad ? 0.f : __uint_as_float((254 - code) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f0 = __uint_as_float(v[i] << 16) * by, f1 = __uint_as_float(v[i] & 0xffff0000u) * by;
      hi[i] = pack_e4m3x2(f0, f1);
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)hi[i]));
      const float2 g = __half22float2(*reinterpret_cast<__half2*>(&h));
      lo[i] = pack_e4m3x2((f0 - g.x) * kLoScale, (f1 - g.y) * kLoScale);
      if (bad) hi[i] = lo[i] = 0;
    }
    if (!store) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // (the row's lanes have all read: they have exchanged their maxima)
      const int row = half * NP + n;
      const uint32_t* z = half ? lo : hi;
      const uint32_t chunk = D == 128 ? ((part >> 1) ^ (row & 7)) : ((part >> 1) ^ ((row >> 1) & 3));
      asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(q + row * D + (chunk << 4) + (part & 1) * 8),
                   "r"(z[0] | z[1] << 16), "r"(z[2] | z[3] << 16)
                   : "memory");
    }
    if (part == 0) qmul[n] = bad ? NAN : sl2 * __uint_as_float(code << 23);
  }
}

template <int D, int NP, bool kParts>
__global__ void __launch_bounds__(F8Cfg<D, NP>::kThreads, F8Cfg<D, NP>::kCtas)
    paged_few8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const F8Args a, const F8Work wk) {
  using C = F8Cfg<D, NP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) F8Ctl<D, NP, kParts> ctl;
  const uint32_t sK0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sV0 = sK0 + C::kKStages * C::kTileBytes, sP = sV0 + C::kVStages * C::kTileBytes;
  const uint32_t sQ = sP + C::kPBytes;
  float* my_part = reinterpret_cast<float*>(smem_raw + (sK0 - smem_u32(smem_raw)));
  volatile int* abort_flag = &ctl.abort_flag;
  const PagedShape& s = a.s;
  const int G = wk.cut.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto sV = [&](int i) { return sV0 + i * C::kTileBytes; };
  auto bar = [&](uint64_t& x) { return smem_u32(&x); };

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    ctl.issued_k = ctl.issued_v = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(ctl.q_raw[i]), 32);
      mbar_init(bar(ctl.q_full[i]), C::kSoftSplit ? 4 * C::kGroups : 1);
      mbar_init(bar(ctl.q_empty[i]), 1 + 4 * C::kGroups);
      mbar_init(bar(ctl.s_full[i]), 2);
      mbar_init(bar(ctl.p_ready[i]), 4 * C::kGroups);
      mbar_init(bar(ctl.drain[i]), 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(bar(ctl.k_full[i]), 1 + 32);
      mbar_init(bar(ctl.k_empty[i]), 1);
      mbar_init(bar(ctl.v_full[i]), 1);
      mbar_init(bar(ctl.v_empty[i]), 1);
    }
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (threadIdx.x < NP) ctl.part_lse[threadIdx.x] = -INFINITY;
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  let_dependent_start();  // (this CTA has its tensor memory: a dependent that takes some cannot be in its way)
  grid_dependency_wait();
  const int ctas = wk.desc != nullptr ? 1 : (int)cluster_size();  // that share a unit
  // The CTA among those that divide the work, and its number: those of one residue follow one another.
  const int beside = blockIdx.x % wk.cut.side, group = blockIdx.x / wk.cut.side, groups = gridDim.x / wk.cut.side;
  const int me = beside * groups + group;
  if (wk.desc != nullptr) {
    find_share<C::kThreads>(s.B, [&](int b) { return F8Units<kParts>(s, wk.cut, b); }, ctl.share, ctl.scan, ctl.units, group,
                            groups);
  } else if (threadIdx.x == 0) {  // tiles [n rank / ctas, n (rank + 1) / ctas) of the cluster's unit
    const int unit = blockIdx.x / ctas, rank = blockIdx.x - unit * ctas, b = unit / s.Hkv;
    const F8Units<kParts> x(s, wk.cut, b);
    const int n = x.count ? x.tiles() : 0, lo = n * rank / ctas, hi = n * (rank + 1) / ctas;
    ctl.share = ShareOf<int>{b, unit - b * s.Hkv, 0, kF8Open + lo, hi - lo, 0, 0};
    ctl.units = x;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  F8Pieces<kParts> w(s, wk.cut, ctl.share, ctl.units, beside);
  if (wk.desc != nullptr && threadIdx.x == 0) {
    const bool joins = !w.done() && w.kt > 0 && w.end == w.n;
    wk.desc[2 * me] = make_int4(joins ? w.b : -1, w.head(), ctl.share.first_cta + me - group,
                                ctl.share.first_slot + 2 * (me - group));
    wk.desc[2 * me + 1] = make_int4(joins ? w.rows() : 0, w.seq.q0, w.seq.bb, w.token());
  }

  constexpr int kLast = C::kThreads / 32 - 1;
  if (warp == 0 || warp == kLast) {
    // ------------------------------------------------------------------ copies of K and codes; of V, and Q split
    const bool values = warp != 0;
    const int P = 1 << s.page_shift, rows = min(P, 128), shift = min(s.page_shift, 7), per = 128 >> shift;
    const int stages = values ? C::kVStages : C::kKStages;
    const uint32_t full0 = values ? bar(ctl.v_full[0]) : bar(ctl.k_full[0]);
    const uint32_t empty0 = values ? bar(ctl.v_empty[0]) : bar(ctl.k_empty[0]);
    const uint32_t tile0 = values ? sV0 : sK0;
    const CUtensorMap* tm = values ? &tmV : &tmK;
    bool run = true;
    F8Pieces<kParts> x = w;  // of the next copy
    int xkt = x.kt, xt = 0, xst = 0;
    uint32_t xphase = 1;
    // The page of the next copy that is this lane's, as the table has it: it is looked at when the copy is made, so that
    // nothing waits for the load.
    auto look_up = [&]() -> int {
      const int key = (xkt << 7) + (lane << shift);
      return lane < per && key < x.seq.Lk ? s.table[(size_t)x.b * s.max_pages + (key >> s.page_shift)] : 0;
    };
    int listed = x.done() ? 0 : look_up();
    const uint64_t once = l2_evict_first();
    auto copy = [&]() {  // the next tile
      const int left = x.seq.Lk - (xkt << 7), pages = left <= 0 ? 0 : min(per, (left + rows - 1) >> shift);
      const uint32_t full = full0 + xst * 8;
      if (run && xt >= stages) run = wait_near(empty0 + xst * 8, xphase, abort_flag, a.status);
      run = __all_sync(0xffffffffu, run) && !*abort_flag;
#ifdef FA_TEST_WITHHOLD_KV  // a test-only build: every wait for keys and values must run out cleanly
      run = false;
#endif
      if (run) {
        const bool ours = (unsigned)listed < (unsigned)s.num_pages;
        if (!ours) report_status(a.status, FA_ERR_BOUNDS);
        const int page = ours ? listed : -1;  // (-1 reads as zero)
        if (lane == 0) {
          mbar_expect_tx(full, pages * rows * D);
          (values ? ctl.issued_v : ctl.issued_k) = xt + 1;
        }
        __syncwarp();
        if (lane < pages)
          tma_load_4d_policy(tile0 + xst * C::kTileBytes + lane * rows * D, tm, 0, (xkt << 7) & (P - 1), x.hk, page, full,
                             once);
        if (!values) {
          const int at = __shfl_sync(0xffffffffu, page, (4 * lane) >> shift), key = (xkt << 7) + 4 * lane;
          const int to = xt % kCodeStages;
          if (key < x.seq.Lk && at >= 0)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(ctl.codes[to] + 8 * lane)),
                         "l"(a.codes + 2 * weight_offset(s, at, x.hk, key & (P - 1)))
                         : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
        }
      }
      ++xt;
      if (++xst == stages) {
        xst = 0;
        xphase ^= 1;
      }
      if (++xkt == x.end) {
        x.next();
        xkt = x.kt;
      }
      if (!x.done()) listed = look_up();
    };
    // Q of a piece is asked for while the one before it runs, once the buffer's last piece is sure to be over (or, in a short
    // piece, behind its last copy). Its rows arrive where their parts will lie, all at once, and up to 16 are split here, a few
    // behind each copy, more by the softmax warps: 32 rows in this loop take 8000 cycles.
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows at a time
    const int r0 = lane / kLanes, part = lane % kLanes;
    F8Pieces<kParts> y = w;
    int piece = 0, at = -1;  // of y; the next row, -1: none has been asked for
    auto step_q = [&]() {
      const int qb = piece & 1;
      const uint32_t to = sQ + qb * C::kQBytes;
      if (at < 0) {
        if (run && piece >= 2) run = wait_near(bar(ctl.q_empty[qb]), ((piece >> 1) - 1) & 1, abort_flag, a.status);
        run = __all_sync(0xffffffffu, run) && !*abort_flag;
        const int live = y.rows();
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                 elem_offset(a.sq, y.seq.bb, y.seq.q0 + y.token(), y.head()) + part * 8;
        if (run)
#pragma unroll 2
          for (int n = r0; n < NP; n += kPer) {  // (rows that do not exist become zeros)
            const int i = n < live ? wk.by_group.div(n) : 0, g = n < live ? n - i * G : 0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(raw_q<D, NP>(to, n, part)),
                         "l"(q + (size_t)i * a.sq.row + (size_t)g * a.sq.head), "r"(n < live ? 16 : 0)
                         : "memory");
          }
        at = 0;
        if constexpr (!C::kSoftSplit) return;
        if (run)
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(ctl.q_raw[qb])) : "memory");
      } else {
        if (at == 0) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
        }
        split_rows<D, NP, D / 64>(to, ctl.qmul[qb], at, a.scale * kLog2e, run);
        at += D / 64 * kPer;  // (4 rows for either d; others tried: 8 at d = 64, 512 x 500 keys of 12 heads, 16 rows 140 us and with 4 135; 2 at d = 128: 5% more)
        if (at < NP) return;
        fence_proxy_async_smem();
        __syncwarp();
        if (run && lane == 0) mbar_arrive(bar(ctl.q_full[qb]));
      }
      at = -1;
      ++piece;
      y.next();
    };
    // (One loop for both warps, and one place for a step: what they share is fetched once.)
    bool ended = true;
    int of = -1, copied = 0, due = -1, more = 1;  // the piece of the copies, its tiles so far; the last whose Q has to be there
    for (;;) {
      if (values)
#pragma unroll 1
        while (!y.done() && (piece <= due || (piece == of + 1 && more-- > 0))) step_q();
      if (x.done()) break;
      if (ended) {
        ++of;
        copied = 0;
      }
      copy();
      ++copied;
      ended = x.done() || xkt == x.kt;
      due = ended ? of + 1 : of;
      more = copied > C::kVStages;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1 || warp == kLast - 1) {
    // ------------------------------------------------------------------ MMAs: S; P V
    // (Their waits suspend: polling takes issue slots from the softmax, 39.4 us for 37.4 with 16 x 4099 keys and 20 rows.)
    const bool scores = warp == 1;
    bool run = true;
    int t = 0, st = 0;
    uint32_t phase = 0;
    if (scores) {
      const uint64_t dk0 = D == 128 ? desc_kmajor_sw128(sK0) : desc_kmajor_sw64(sK0);
      const uint64_t dq0 = D == 128 ? desc_kmajor_sw128(sQ) : desc_kmajor_sw64(sQ);
      for (int piece = 0; !w.done(); ++piece, w.next()) {
        const int qb = piece & 1;
        if (run) run = mbar_wait(bar(ctl.q_full[qb]), (piece >> 1) & 1, abort_flag, a.status);
        for (int kt = w.kt; kt < w.end; ++kt, ++t) {
          // With P V of tile t - 2 done, its scores are read and its P's buffer is free for tile t.
          if (run && t >= 2)
            run = mbar_wait(bar(ctl.v_empty[(t - 2) % C::kVStages]), ((t - 2) / C::kVStages) & 1, abort_flag, a.status);
          if (run) run = mbar_wait(bar(ctl.k_full[st]), phase, abort_flag, a.status);
          run = __all_sync(0xffffffffu, run);
          fence_after_sync();
          if (run && lane == 0) {
            mbar_arrive(bar(ctl.s_full[t & 1]));  // (the codes are there: what this thread has seen, the softmax will)
            const uint64_t dk = desc_add(dk0, st * C::kTileBytes), dq = desc_add(dq0, qb * C::kQBytes);
            const uint32_t to = tmem + (t & 1) * 2 * NP;
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_ss_f8(to, desc_add(dk, kk * 32), desc_add(dq, kk * 32), C::kIdS, kk > 0);
            mma_commit(bar(ctl.s_full[t & 1]));
            mma_commit(bar(ctl.k_empty[st]));
            if (kt + 1 == w.end) mma_commit(bar(ctl.q_empty[qb]));
          }
          __syncwarp();
          if (++st == C::kKStages) {
            st = 0;
            phase ^= 1;
          }
        }
      }
    } else {
      const uint64_t dv0 = D == 128 ? desc_mnmajor_sw128(sV0, 16384) : desc_mnmajor_sw64(sV0, C::kTileBytes);
      const uint64_t dp0 = desc_mnmajor_sw128(sP, 16384);
      const uint32_t tO = tmem + C::kO;
      for (; !w.done(); w.next()) {
        for (int kt = w.kt; kt < w.end; ++kt, ++t) {
          if (run) run = mbar_wait(bar(ctl.v_full[st]), phase, abort_flag, a.status);
          if (run) run = mbar_wait(bar(ctl.p_ready[t & 1]), (t >> 1) & 1, abort_flag, a.status);
          run = __all_sync(0xffffffffu, run);
          fence_after_sync();
          if (run && lane == 0) {
            const uint64_t dv = desc_add(dv0, st * C::kTileBytes), dp = desc_add(dp0, (t & 1) * C::kPStep);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss_f8(tO, desc_add(dv, kk * 32 * D), desc_add(dp, kk * 4096), C::kIdPV, kk > 0 || kt > w.kt);
            mma_commit(bar(ctl.v_empty[st]));
          }
          __syncwarp();
          if (++st == C::kVStages) {
            st = 0;
            phase ^= 1;
          }
        }
      }
    }
    if (lane == 0) {
      mma_commit(bar(ctl.drain[scores ? 0 : 1]));
      mbar_wait_drain(bar(ctl.drain[scores ? 0 : 1]), 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax, epilogue
    const int quad = warp & 3, r = quad * 32 + lane;  // key within the tile; head dimension of O^T
    constexpr int NC = C::kCols;
    const int gr = C::kGroups == 1 ? 0 : (warp - 2) >> 2, n0 = gr * NC, on = 1 + gr;  // group, first column, barrier
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::kO + n0;
    bool run = true;
    int t = 0, vs = 0;
    uint32_t vphase = 0;
    auto wait_pv = [&](int j) -> bool {  // P V of tile j has completed
      return wait_near(bar(ctl.v_empty[j % C::kVStages]), (j / C::kVStages) & 1, abort_flag, a.status);
    };
    auto split_q = [&](int piece) {  // four rows a warp of the piece's Q
      const int qb = piece & 1;
      if (run) run = wait_near(bar(ctl.q_raw[qb]), (piece >> 1) & 1, abort_flag, a.status);
      run = __all_sync(0xffffffffu, run);
      if (4 * quad < NC) split_rows<D, NP, D / 64>(sQ + qb * C::kQBytes, ctl.qmul[qb], n0 + 4 * quad, a.scale * kLog2e, run);
      fence_proxy_async_smem();
      __syncwarp();
      if (run && lane == 0) mbar_arrive(bar(ctl.q_full[qb]));
    };
    int split = 0;  // pieces whose Q is
    for (int piece = 0; !w.done(); ++piece) {
      const SeqInfo& seq = w.seq;
      const int live = w.rows(), tok = w.token(), head = w.head(), qb = piece & 1;
      if (r < NC) ctl.lim[n0 + r] = s.causal ? min(seq.Lk, tok + wk.by_group.div(n0 + r) + seq.off + 1) : seq.Lk;  // keys [0, lim) visible
      const int least = s.causal ? min(seq.Lk, tok + seq.off + 1) : seq.Lk;
      float l[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) l[n] = 0.f;
      for (int kt = w.kt; kt < w.end; ++kt, ++t) {
        if constexpr (C::kSoftSplit) {  // Q of this piece, if it is the first, and before the last tile that of the next
          const int due = kt + 1 == w.end && w.more() ? piece + 1 : piece;
#pragma unroll 1
          for (; split <= due; ++split) split_q(split);
        }
        if (run && kt == w.kt) run = wait_near(bar(ctl.q_full[qb]), (piece >> 1) & 1, abort_flag, a.status);
        if (run) run = wait_near(bar(ctl.s_full[t & 1]), (t >> 1) & 1, abort_flag, a.status);
        fence_after_sync();
        uint32_t shi[NC], slo[NC];
        load_cols(tmem + lane_off + (t & 1) * 2 * NP + n0, shi);
        load_cols(tmem + lane_off + (t & 1) * 2 * NP + NP + n0, slo);
        const uint32_t code = *reinterpret_cast<const uint16_t*>(ctl.codes[t % kCodeStages] + 2 * r);
        const uint32_t kc = code & 255u, vc = code >> 8;
        const float kmul = kc == 255u ? NAN : __uint_as_float(kc << 23);
        const int ve = vc == 0u ? kZeroRow : (int)vc - 127;
        const float up = vc == 255u ? NAN : (float)max(ve, 0), down = (float)min(ve, 0);
        const float small = __uint_as_float((uint32_t)(127 + min(ve, 0)) << 23);  // 2^down
        const float back = __uint_as_float((uint32_t)(127 - min(max(ve, 0), 126)) << 23);  // 2^-up
        tmem_ld_wait();
        float y[NC];  // the exponents of P 2^-down, and (below) their distance from the reference
        {
          const float2 part = make_float2(1.f / kLoScale, 1.f / kLoScale), km = make_float2(kmul, kmul);
          const float2 u2 = make_float2(up, up);
#pragma unroll
          for (int n = 0; n < NC; n += 4) {
            const float4 q = *reinterpret_cast<const float4*>(ctl.qmul[qb] + n0 + n);
            const float2 x0 = fma2(make_float2(__uint_as_float(slo[n]), __uint_as_float(slo[n + 1])), part,
                                   make_float2(__uint_as_float(shi[n]), __uint_as_float(shi[n + 1])));
            const float2 x1 = fma2(make_float2(__uint_as_float(slo[n + 2]), __uint_as_float(slo[n + 3])), part,
                                   make_float2(__uint_as_float(shi[n + 2]), __uint_as_float(shi[n + 3])));
            const float2 z0 = fma2(x0, mul2(km, make_float2(q.x, q.y)), u2);
            const float2 z1 = fma2(x1, mul2(km, make_float2(q.z, q.w)), u2);
            y[n] = z0.x;
            y[n + 1] = z0.y;
            y[n + 2] = z1.x;
            y[n + 3] = z1.y;
          }
        }
        const int key = (kt << 7) + r;
        const bool opens = kt == w.kt;
        if (opens) named_bar_sync(on, 128);  // ctl.lim is written; the last piece's ctl.ref is no longer read
        if ((kt << 7) + 128 > least) {
#pragma unroll
          for (int n = 0; n < NC; ++n) y[n] = key < ctl.lim[n0 + n] ? y[n] : -INFINITY;
        }
        auto from_ref = [&](const float (&x)[NC], float (&d)[NC]) {
#pragma unroll
          for (int n = 0; n < NC; n += 4) {
            const float4 m = *reinterpret_cast<const float4*>(ctl.ref + n0 + n);
            d[n] = x[n] - m.x;
            d[n + 1] = x[n + 1] - m.y;
            d[n + 2] = x[n + 2] - m.z;
            d[n + 3] = x[n + 3] - m.w;
          }
        };
        bool raise = opens;
        float d[NC];
        if (!opens) {
          from_ref(y, d);
          float big = d[0];
#pragma unroll
          for (int n = 1; n < NC - 1; n += 2) big = fmax3(big, d[n], d[n + 1]);
          raise = vote_any(fmaxf(big, d[NC - 1]) > kRaise8 - down, on);
        }
        if (raise) {
          float z[NC];
#pragma unroll
          for (int n = 0; n < NC; ++n) z[n] = y[n] + down;
          columns_reduce(z, lane, [](float p, float q) { return fmaxf(p, q); });
          ctl.wmax[quad][n0 + lane * NC / 32] = z[0];
          named_bar_sync(on, 128);
          if (r < NC) {
            const int n = n0 + r;
            const float old = opens ? kNoMax : ctl.ref[n];
            const float now = fmaxf(
                fmaxf(fmaxf(ctl.wmax[0][n], ctl.wmax[1][n]), fmaxf(ctl.wmax[2][n], ctl.wmax[3][n])) - kFirst, old);
            ctl.alpha[n] = ex2_approx(old - now);
            ctl.root[n] = ex2_approx(0.5f * (old - now));
            ctl.ref[n] = now;
          }
          __syncwarp();
          named_bar_sync(on, 128);
          if (!opens) {
            if (run) run = wait_pv(t - 1);
            fence_after_sync();
// (512 x 500 keys of 12 heads, d = 64, 16 rows: 182 us unrolled and 148; of 8 rows, 4096 x 128 keys, 365 and 376)
#pragma unroll (NP == 8 ? 3 : 1)
            for (int part = 0; part < 3; ++part) {
              uint32_t o[NC];
              load_cols(tO + part * NP, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < NC; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * ctl.alpha[n0 + i]);
              store_cols(tO + part * NP, o);
            }
            tmem_st_wait();
#pragma unroll
            for (int i = 0; i < NC; ++i) l[i] = l[i] * ctl.root[n0 + i] * ctl.root[n0 + i];
          }
          from_ref(y, d);
        }
        uint32_t hi[NC / 4], mid[NC / 4], lo[NC / 4];
#pragma unroll
        for (int n = 0; n < NC; n += 4) {
          const float p0 = ex2_approx(d[n]), p1 = ex2_approx(d[n + 1]), p2 = ex2_approx(d[n + 2]), p3 = ex2_approx(d[n + 3]);
          const float2 l0 = fma2(make_float2(p0, p1), make_float2(back, back), make_float2(l[n], l[n + 1]));
          const float2 l1 = fma2(make_float2(p2, p3), make_float2(back, back), make_float2(l[n + 2], l[n + 3]));
          l[n] = l0.x;
          l[n + 1] = l0.y;
          l[n + 2] = l1.x;
          l[n + 3] = l1.y;
          uint32_t ha, hb, ma, mb, la, lb;
          const float2 s0 = mul2(make_float2(p0, p1), make_float2(small, small));
          const float2 s1 = mul2(make_float2(p2, p3), make_float2(small, small));
          split_p(s0.x, s0.y, ha, ma, la);
          split_p(s1.x, s1.y, hb, mb, lb);
          hi[n / 4] = __byte_perm(ha, hb, 0x7531);
          mid[n / 4] = __byte_perm(ma, mb, 0x7531);
          lo[n / 4] = la | lb << 16;
        }
        // P's buffer is free: S of tile t, which has completed, was issued when the P V that read it had.
        const uint32_t sPt = sP + (NP <= 16 ? 0 : (t & 1) * C::kPStep) + r * 128;
        auto put = [&](int c, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {  // c: 16-byte chunk of the row
          store16(sPt + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4), x0, x1, x2, x3);
        };
        const int c0 = n0 / 16 + (NP <= 16 ? (t & 1) * 4 : 0);
        if constexpr (NP == 8) {
          put(c0, hi[0], hi[1], mid[0], mid[1]);
          put(c0 + 1, lo[0], lo[1], 0, 0);
        } else if constexpr (NC == 8) {
          auto put8 = [&](int c, const uint32_t (&x)[2]) {
            asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(sPt + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4) + (n0 & 8)),
                         "r"(x[0]), "r"(x[1])
                         : "memory");
          };
          put8(c0, hi);
          put8(c0 + NP / 16, mid);
          put8(c0 + 2 * (NP / 16), lo);
        } else {
          put(c0, hi[0], hi[1], hi[2], hi[3]);
          put(c0 + NP / 16, mid[0], mid[1], mid[2], mid[3]);
          put(c0 + 2 * (NP / 16), lo[0], lo[1], lo[2], lo[3]);
        }
        // Value rows past the last key may hold anything, and 0 times NaN is NaN: they become 0.
        const int valid = seq.Lk - (kt << 7);
        if (valid < 128) {
          if (run) run = wait_near(bar(ctl.v_full[vs]), vphase, abort_flag, a.status);
          if (run && r >= valid)
#pragma unroll
            for (int c = gr * (D / 16 / C::kGroups); c < (gr + 1) * (D / 16 / C::kGroups); ++c)
              store16(sV(vs) + r * D + c * 16, 0, 0, 0, 0);
          __syncwarp();
        }
        fence_proxy_async_smem();
        fence_before_sync();
        __syncwarp();
        if (run && lane == 0) mbar_arrive(bar(ctl.p_ready[t & 1]));
        if (++vs == C::kVStages) {
          vs = 0;
          vphase ^= 1;
        }
      }
      // ---------------------------------------------------------------- end of the piece
      __syncwarp();
      if (run && lane == 0) mbar_arrive(bar(ctl.q_empty[qb]));  // (its scales are read)
      columns_reduce(l, lane, [](float p, float q) { return p + q; });
      ctl.wmax[quad][n0 + lane * NC / 32] = l[0];
      named_bar_sync(on, 128);
      const bool whole = w.whole() && ctas == 1;
      const int slot = 2 * me + (piece == 0 ? 0 : 1);
      auto total = [&](int n) { return (ctl.wmax[0][n] + ctl.wmax[1][n]) + (ctl.wmax[2][n] + ctl.wmax[3][n]); };
      if (r < NC) {
        const float sum = total(n0 + r);
        ctl.alpha[n0 + r] = sum == 0.f ? 0.f : 1.f / sum;  // (0: no visible key; a NaN stays one)
      }
      __syncwarp();
      named_bar_sync(on, 128);
      if (quad == 3 && lane < NC) {  // (a warp that at d = 64 has nothing to store)
        const int n = n0 + lane;
        const float sum = total(n), lse2 = sum == 0.f ? -INFINITY : ctl.ref[n] + log2f(sum);
        if (whole) {
          const int i = wk.by_group.div(n);
          if (n < live) a.lse[paged_row(s, seq, w.b, head + n - i * G, tok + i)] = lse2 * kLn2;
        } else {
          (ctas > 1 ? ctl.part_lse : wk.part_lse + (size_t)slot * NP)[n] = lse2;
        }
      }
      if (run) run = wait_pv(t - 1);
      fence_after_sync();
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + elem_offset(a.so, seq.bb, seq.q0 + tok, head) + r;
      // (the cluster's parts lie over the ring: with the last P V done nothing reads it or is on its way there)
      float* part = (ctas > 1 ? my_part : wk.part_o + (size_t)slot * NP * D) + r;
      int i = wk.by_group.div(n0), g = n0 - i * G;  // token and head of the group of column n
      float o[NC];
      {
        uint32_t x[NC], z[NC];
        load_cols(tO, reinterpret_cast<uint32_t(&)[NC]>(o));
        load_cols(tO + NP, x);
        load_cols(tO + 2 * NP, z);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < NC; ++k)
          o[k] += (__uint_as_float(x[k]) + __uint_as_float(z[k]) * (1.f / kMidScale)) * (1.f / kMidScale);
      }
      if (r < D) {
        // The strides are looked at once: their lines of the arguments miss (48 x 1024 keys of 12 heads, d = 64, 64 rows: 75 us and
        // 66, 16 rows 34.8 and 29.4). Not with 16 rows at d = 128, whose loop needs the registers (16 x 4099 keys: 27.4 and 26.4).
        constexpr bool kStep = NP != 16 || D == 64;
        const long long step = a.so.head, wrap = a.so.row - (long long)G * a.so.head;
        __nv_bfloat16* to = out + (size_t)i * a.so.row + (size_t)g * a.so.head;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          const int n = n0 + k;
          if (n >= live) break;
          const float val = o[k] * ctl.alpha[n];
          if (!whole)
            part[n * D] = val;
          else if constexpr (kStep)
            *to = __float2bfloat16(val);
          else
            out[(size_t)i * a.so.row + (size_t)g * a.so.head] = __float2bfloat16(val);
          to += step;
          if (++g == G) {
            g = 0;
            ++i;
            to += wrap;
          }
        }
      }
      w.next();  // (the arrival on the next tile's P orders the reads of O before the product that overwrites it)
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
  if (threadIdx.x == 0 && *abort_flag) {  // copies still in flight land before the CTA exits: the last one into each buffer
    for (int i = max(0, ctl.issued_k - C::kKStages); i < ctl.issued_k; ++i)
      mbar_wait_drain(bar(ctl.k_full[i % C::kKStages]), (i / C::kKStages) & 1);
    for (int i = max(0, ctl.issued_v - C::kVStages); i < ctl.issued_v; ++i)
      mbar_wait_drain(bar(ctl.v_full[i % C::kVStages]), (i / C::kVStages) & 1);
  }
}

// Joins the pieces of each divided unit. Block (c, y) takes 16 rows of the one that ends in CTA c's first piece, if it
// began before; a thread has four elements of a row.
template <int D, int NP>
__global__ void __launch_bounds__(4 * D) paged_few8_join_kernel(const FaPagedArgs a, const F8Work wk) {
  let_dependent_start();
  grid_dependency_wait();
  const int4 d = wk.desc[2 * blockIdx.x], of = wk.desc[2 * blockIdx.x + 1];
  const PagedShape& s = a.s;
  const int G = wk.cut.group, n = blockIdx.y * 16 + threadIdx.x / (D / 4), e = threadIdx.x % (D / 4) * 4;
  if (d.x < 0 || n >= of.x) return;
  SeqInfo seq{};
  seq.q0 = of.y;
  seq.bb = of.z;
  join_pieces<D, NP>(a, wk.part_o, wk.part_lse, d.z, blockIdx.x, d.w, n, e, seq, d.x, of.w + n / G, d.y + n % G);
}

// Units of a token, 1 unless a K/V head has more than 64 heads: then parts of them as equal as may be, of 33 heads or more.
int token_units(const PagedShape& s) { return (s.H / s.Hkv + 63) / 64; }
int unit_heads(const PagedShape& s) { return (s.H / s.Hkv + token_units(s) - 1) / token_units(s); }

int unit_rows(const PagedShape& s, int tokens) {
  const int rows = tokens * unit_heads(s);
  return rows <= 8 ? 8 : padded_rows(rows);
}

// Heads side by side: the most that leave no more than 3% of the CTAs without work.
F8Cut cut_of(const PagedShape& s, int tokens, int ctas) {
  int side = s.Hkv;
  while (side > 1 && (s.Hkv % side != 0 || ctas / side * side * 100ll < 97ll * ctas)) --side;
  return {tokens, s.H / s.Hkv, unit_heads(s), token_units(s), side, s.Hkv / side};
}

// CTAs that share a (sequence, head) unit where nothing is divided by the lengths, or 0: the rule of fa_paged_decode.cu with
// limits of its own, since a tile is half as many bytes. Eight tiles a CTA of a cluster (8 sequences of 8 heads, 4000 keys:
// 13.9 us, divided 14.3; one of 777 8.4 and 9.5, of 8000 12.5 and 12.7; 4 of 4000 12.8 and 11.9, which clusters of 8 would do in 10.9; with
// 16 tiles 8 of 8000 21.5 and 19.5) or 16 of one alone (24 of 12 heads, d = 64, 2000 keys: 16.1 and 18.1). Nearly two units a place, of up
// to 8 tiles, mostly gain undivided (48 of 12 heads, d = 64, 1024 keys in pages of 64: 19.5 and 20.3, with 16 rows 24.4 and 28.2; 64 of 8
// heads, d = 128, 500 keys 17.9 and 19.3; 128 keys 13.5 and 13.2), and are one launch without a workspace. Not a few more than the
// places (40 of 8 heads, 1000 keys: 20.9 and 19.0), nor 16 tiles (64 of 8 heads, 2000 keys: 40.2 and 37.8).
int unit_ctas(const PagedShape& s, int tokens, int num_sms) {
  if (tokens < s.Nq || token_units(s) > 1) return 0;
  const long long units = (long long)s.B * s.Hkv, room = (long long)num_sms * few8_ctas(unit_rows(s, tokens));
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
  if (2 * units >= 3 * room && units <= 2 * room && tiles <= 8) return 1;
  return units * ctas <= room && tiles <= (ctas == 1 ? 16 : 8 * ctas) ? ctas : 0;
}

template <int D, int NP, bool kParts = false>
cudaError_t launch_few8(const FaPagedArgs& a, int tokens, cudaStream_t st) {
  using C = F8Cfg<D, NP>;
  const PagedShape& s = a.s;
  const int P = 1 << s.page_shift, box = P < 128 ? P : 128;
  // A miss fetches 128 bytes, at d = 64 two heads' rows (64, 128 and 256: within 1% while neighbours walk together; 147, - and 190 us
  // of 64 x 8192 keys before they did).
  constexpr bool kWideL2 = false;
  CUtensorMap tk, tv;
  if (!fa_make_tmap_u8(&tk, a.k, D, P, s.Hkv, s.num_pages, a.sk.row, a.sk.head, a.sk.batch, D, box, kWideL2) ||
      !fa_make_tmap_u8(&tv, a.v, D, P, s.Hkv, s.num_pages, a.sv.row, a.sv.head, a.sv.batch, D, box, kWideL2))
    return cudaErrorInvalidValue;
  const int shared = unit_ctas(s, tokens, a.num_sms);
  int ctas = shared > 0 ? s.B * s.Hkv * shared : a.num_sms * C::kCtas;
  F8Work wk{};
  wk.cut = {tokens, s.H / s.Hkv, unit_heads(s), token_units(s), 1, s.Hkv};
  wk.by_group = fast_div(unit_heads(s));
  if (shared == 0) {
    wk.cut = cut_of(s, tokens, ctas);
    ctas = ctas / wk.cut.side * wk.cut.side;
    char* ws = static_cast<char*>(a.workspace);
    wk.desc = reinterpret_cast<int4*>(ws);
    ws += up256((size_t)ctas * 2 * sizeof(int4));
    wk.part_lse = reinterpret_cast<float*>(ws);
    ws += up256((size_t)ctas * 2 * NP * sizeof(float));
    wk.part_o = reinterpret_cast<float*>(ws);
  }
  const F8Args x{s, a.q, a.codes, a.o, a.lse, a.sq, a.so, a.scale, a.status};
  auto kern = paged_few8_kernel<D, NP, kParts>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if (C::kCtas > 1) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  if (shared > 0) return launch_dependent_cluster(kern, dim3(ctas), dim3(C::kThreads), C::kSmem, shared, st, tk, tv, x, wk);
  e = launch_dependent(kern, dim3(ctas), dim3(C::kThreads), C::kSmem, st, tk, tv, x, wk);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_few8_join_kernel<D, NP>, dim3(ctas, (NP + 15) / 16), dim3(4 * D), 0, st, a, wk);
}

}  // namespace
}  // namespace fa

// Up to four units of 64 rows; more go by way of the chunk kernel. Where a number of heads that divides 128 fills its tiles,
// it is ahead from three units on at d = 64 (128 sequences of 1000 keys, 12 heads: 100 rows 256 us and 290, 130 rows 375 and 346), and
// from four at d = 128 (16 x 4000 keys, 32 / 8 heads: 132 rows 121 and 155, 240 rows 157 and 157; 300 x 500 674 and 430).
int fa_paged_few8_tokens(const fa::PagedShape& s) {
  const int G = s.H / s.Hkv;
  if (G > 64) return (long long)s.Nq * fa::token_units(s) <= 4 ? 1 : 0;
  const int most = 128 % G != 0 ? 4 : s.d == 128 ? 3 : 2;
  if (s.Nq > most * (64 / G)) return 0;
  return (long long)s.Nq * G <= 64 ? s.Nq : 64 / G;
}

size_t fa_paged_few8_workspace(const fa::PagedShape& s, int tokens, int num_sms) {
  if (fa::unit_ctas(s, tokens, num_sms) > 0) return 0;
  const int np = fa::unit_rows(s, tokens);
  const size_t ctas = (size_t)num_sms * fa::few8_ctas(np), rows = ctas * 2 * np;
  return fa::up256(ctas * 2 * sizeof(int4)) + fa::up256(rows * sizeof(float)) + rows * s.d * sizeof(float);
}

namespace fa {
namespace {
template <int D>
cudaError_t launch_rows(const FaPagedArgs& a, int tokens, cudaStream_t st) {
  switch (unit_rows(a.s, tokens)) {
    case 8: return launch_few8<D, 8>(a, tokens, st);
    case 16: return launch_few8<D, 16>(a, tokens, st);
    case 32: return launch_few8<D, 32>(a, tokens, st);
    default: return token_units(a.s) > 1 ? launch_few8<D, 64, true>(a, tokens, st) : launch_few8<D, 64>(a, tokens, st);
  }
}
}  // namespace
}  // namespace fa

cudaError_t fa_launch_paged_few8(const FaPagedArgs& a, int tokens, cudaStream_t st) {
  return a.s.d == 64 ? fa::launch_rows<64>(a, tokens, st) : fa::launch_rows<128>(a, tokens, st);
}
