// k_packed_attn.cu - attention of single tokens and chunks of up to kPackedRows rows over the 8-bit paged
// cache.  Rows, masks and results as in k_paged_attn.cu; K_j = 2^ek_j k_j and V_j = 2^ev_j v_j with e4m3
// codes k_j, v_j.
//
// Codes go to the 5th-generation tensor cores as they lie: no value of the cache is converted.  The
// other operands are sums of e4m3 numbers, which have 4 significant bits each, as more columns of the
// product:
//   q = 2^eq (q1 + q2/16 [+ q3/256])     two are exact for bf16's 8 bits, three for fp16's 11
//   w = w1 + w2/16 + w3/256              fp16's 11 bits; w is at most 256, so 2^-26 of that is its floor
// Keys are the rows of both products, a thread of the softmax owns a key of each tile:
//   S[j][r]  = k_j . q_r                 M = 128 keys, N = parts x R rows, K = D
//   w[j][r]  = 2^(s_jr - m_r + 8 + ev_j - E_r),   s_jr = S c 2^(ek_j + eq_r)
//   O[d][r]  = sum_j v_jd w_jr           M = D dims, N = 3 x R rows, K = 128 keys a tile
// A step is four tiles of 2 or 4 rows, two of 8, one of more: a thread has 8 to 32 scores a step, and what a
// step costs beside them (barriers, maxima, the epilogue) is paid for several tiles.  (A tile at a time, few
// rows took as long as 32: 313 us on the 64-session tick; tiles of 8 rows for one: 261 us.)
// m_r is the step's own maximum and E_r the whole number from max_j (s_jr - m_r + ev_j) on, or up to kSlack
// above it: a row keeps the precision of what weighs in it, whatever else it sees.  A step depends on nothing
// before it.  The epilogue adds the steps up in fp32, in order: acc = acc 2^(M - M') + O 2^(m - 8 + E_r - M').
//
// A work unit is (sequence, key head, split of its keys, row tile of up to R rows).  Each CTA takes a run
// of consecutive units with about as many tiles as the others'; a sequence's splits depend on its own
// lengths, the head counts and max_q only.  A unit that is not its rows' only one leaves (m, l, O) in
// scratch and k_packed_join adds the splits up in split order.
//
//   warp 0       the units and their tiles' pages, up to 32 tiles ahead.  (With lookups in the warps that
//                load, a tile took 1150 clocks and a unit's start 3600.)
//   warp 1       one thread issues the MMAs of S
//   warps 2, 16  K tiles with both scales, two at a time; V tiles
//   warp 3       one thread issues the MMAs of O.  (One thread for both took 1900 clocks a tile.)
//   warps 4-7, 8-11   softmax of every second step
//   warps 12-15  epilogue: a thread owns one dim
//   warps 17-18  the units' queries, as parts.  (One warp took 13000 clocks for 32 rows.)
//
// Measured (in a graph, with the join): 64 sequences, one token, up to 3000 entries, 32 heads of 128 dims, bf16:
// 157 us, 4.9 TB/s; 8 sequences of up to 5 tokens over up to 65000 entries, 32 heads on 8, pages of 16, fp16:
// 161 us, 2.9 TB/s; one token over 3000 entries, 32 heads: 18 us.  Bound, with a row to a key head, by units'
// ends and the SMs' unequal runs; with 20 rows by the softmax's instructions (4850 of a warp a tile, at half
// the issue rate); alone by latencies.
//
// What no row of a unit sees must not reach the second product, where a weight of zero times a NaN
// would be one: those rows of V are zeroed in shared memory.  An entry that only some rows see and
// that holds a NaN code is zeroed too, and its scale taken for NaN, which only its seers' weights get.
#include <type_traits>

#include "pp_paged.cuh"
#include "pp_tcgen05.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kThreads = 608;
constexpr int kReaders = 16;         // of the units: both issuers, eight of softmax, epilogue, queries
constexpr int kSlots = 32;           // tiles that are planned, and those whose scales are held
constexpr int kParts = 3;            // of a weight
constexpr float kTop = 8.f;          // a step's largest weight is 2^8 (e4m3 holds up to 448)
// Where the V exponents of a warp's keys are no further apart than this, its largest one stands for the largest
// weighted one and nothing has to be looked for: weights are held to 2^-20 of the step's largest then, to 2^-25
// otherwise.  (Looked for in every step, 8 long caches took 173 us in place of 161.)
constexpr int kSlack = 6;
// Buffers of a softmax group's maxima.  A warp writes a step's while another of its group may still read those
// of the group's step before; past its own meeting it comes only when that one has read them and arrived there too.
constexpr int kMaxima = 2;

// Few rows: a thread has 8 or 16 scores a step all the same.
__host__ __device__ constexpr int step_tiles(int R) { return R < 8 ? 4 : R == 8 ? 2 : 1; }

template <typename T, int D, int R>
struct Cfg {
  static constexpr int QP = sizeof(T) == 2 && Num<T>::kShift == 0.f ? 2 : 3;   // parts of a query
  static constexpr int NQ = (QP * R + 15) / 16 * 16;                 // columns of S
  static constexpr int NP = (kParts * R + 15) / 16 * 16;             // columns of O
  static constexpr int KT = step_tiles(R);                           // tiles of a step
  static constexpr int W = R < 8 ? R : 8;                            // rows at a time
  static constexpr int SB = KT * NQ <= 64 ? 4 : 2;                   // buffers of S in tensor memory
  static constexpr int kTileBytes = kTile * D;
  // Stages of K, which a product frees at once, and of V, which waits for the softmax.
  static constexpr int KS = D == 128 ? 4 : 8;
  static constexpr int VS = D == 128 ? (R < 32 ? 7 : QP == 2 ? 6 : 5) : 8;
  static constexpr int kQBytes = NQ * 128;
  static constexpr int kPBytes = NP / 16 * 2048;
  static constexpr int kVOff = KS * kTileBytes;
  static constexpr int kQOff = (KS + VS) * kTileBytes;
  static constexpr int kPOff = kQOff + 2 * kQBytes;
  static constexpr int kScaleOff = kPOff + 2 * KT * kPBytes;         // K's, then V's: 128 bytes a tile
  static constexpr int kCtlOff = kScaleOff + 2 * kSlots * kTile;
};

// A tile as its loads need it: the pages of its groups of 16 entries (n_pages: none) and the groups that miss
// one; key head (-1: no more tiles), first entry's row; tiles that its step lacks (-1: more of it follow).
struct alignas(16) Tile {
  int page[8];
  int h, row, lack;
  uint32_t bad;
};

struct Ctl {
  UnitRing ring;
  Tile tile[kSlots];
  uint64_t tfull[kSlots], tempty[kSlots], kfull[8], kempty[8], vempty[8], qfull[2], qempty[2];
  uint64_t sfull[4], sempty[4], vfull[8], pfull[2], ofull[2], oempty[2], meet[2], done;
  uint32_t bad[kSlots];
  int any_bad;                         // a tile of this CTA had a page that is missing
  uint32_t tmem;
  int abort;
  // of the two units in flight: each row's factor of its scores (to powers of two) and its entry
  alignas(16) float row_c[2][32];
  int row_at[2][32];
  // of the groups' steps, by warps: maxima of rows, and E for that maximum
  float warp_max[2][kMaxima][4][32];
  float warp_e[2][kMaxima][4][32];
  // each warp's copy of the references (negative), and of -E
  alignas(16) float ref[2][4][32];
  alignas(16) float fit[2][4][32];
  float m[2][32], l[2][4][32];
  uint32_t e[2][32];
  alignas(16) float keep[4][32];       // epilogue warps: factors of acc and of O
  alignas(16) float add[4][32];
};

// What a Unit of the ring holds here: `row` and `first` of its first row (token's row, its entry), nt =
// the last row's entry, tag = rows | head of the first row << 8, ns = the first row's token within
// its chunk, split = split | splits << 8.
constexpr int kHeadShift = 8;

// ---- units -----------------------------------------------------------------------------------
// Tokens that R consecutive rows (heads within tokens) touch, at most.
__host__ __device__ __forceinline__ int row_span(int R, int G) { return (R - 1) / G + 2; }
// Key tiles that a row tile can touch, at most.
__host__ __device__ __forceinline__ int64_t most_tiles(int64_t entries, int window, int span) {
  const int64_t all = (entries + kTile - 1) / kTile;
  const int64_t seen = ((int64_t)window + span - 2) / kTile + 2;
  return window && seen < all ? seen : all;
}
// Tiles of one split, at most: `share` splits of each key head fill the SMs when a sequence is alone.  Twelve (a
// unit's ends cost 4000 clocks, as much as six tiles: with four to eight, the 64-session tick took 201 us) to 24
// (runs of units come out even), and at most 128 splits.  Splits are counted upwards and made even, so that
// units can have little more than half of it: 13 tiles are two of 6 and 7.
constexpr int kLeast = 12, kMost = 24;
__host__ __device__ __forceinline__ int64_t split_tiles(int64_t tiles, int share) {
  int64_t st = (tiles + share - 1) / share;
  st = st < kLeast ? kLeast : st > kMost ? kMost : st;
  const int64_t even = (tiles + 127) / 128;
  return st > even ? st : even;
}
__host__ __device__ __forceinline__ int n_splits(int64_t tiles, int share) {
  const int64_t st = split_tiles(tiles, share);
  return tiles <= st ? 1 : (int)((tiles + st - 1) / st);
}

struct Shape {       // of a sequence's units
  int rt, ns, cost;
  // A chunk longer than the caller said is not split: scratch has no room for its parts.
  __device__ __forceinline__ Shape(const Args& a, const Seq& s, int R, int max_q, int share) {
    const int mt = (int)most_tiles(s.len, a.window, row_span(R, a.G));
    rt = (int)(((int64_t)s.n * a.G + R - 1) / R);
    ns = s.n > max_q ? 1 : n_splits(mt, share);
    // Of a unit, in about 250 clocks: its tiles (by rows), steps and ends.  (Counted by tiles and steps alone,
    // the SMs' times went from 108 to 201 us on the 64-session tick.)
    const int per = step_tiles(R), st = (mt + ns - 1) / ns, chunks = (min(s.n * a.G, R) + 7) / 8;
    cost = R < 8 ? 2 * st + 4 * ((st + per - 1) / per) + 12 : st * (per == 2 ? 4 : 3 + 2 * chunks) + 12;
  }
};

struct Walk {
  const Args& a;
  const int R, max_q, share;
  int64_t at, end;
  int b, h, i;
  Seq s;
  int rt, ns, cost;

  // (the prefix sums are looked at here only)
  __device__ __forceinline__ Walk(const Args& a_, const int64_t* pre, int R_, int max_q_, int share_)
      : a(a_), R(R_), max_q(max_q_), share(share_) {
    const int64_t total = pre[a.n_seqs];
    at = total * blockIdx.x / gridDim.x;
    end = total * (blockIdx.x + 1) / gridDim.x;
    if (at >= end) return;
    b = find_seq(pre, a.n_seqs, at);
    sequence();
    const int64_t k = (at - pre[b] + cost - 1) / cost;   // the first unit that starts in the run
    h = (int)(k / (rt * ns));
    i = (int)(k - (int64_t)h * (rt * ns));
    at = pre[b] + k * cost;
    if (h == a.Hk) next_sequence();
  }
  __device__ __forceinline__ bool done() const { return at >= end; }
  __device__ __forceinline__ void sequence() {
    s = seq_of(a, b);
    const Shape x(a, s, R, max_q, share);
    rt = x.rt;
    ns = x.ns;
    cost = x.cost;
  }
  __device__ __forceinline__ void next_sequence() {
    h = i = 0;
    do {
      ++b;
      s = b < a.n_seqs ? seq_of(a, b) : Seq{};
    } while (b < a.n_seqs && s.n == 0);
    if (b < a.n_seqs) sequence();
  }
  __device__ __forceinline__ void next() {
    at += cost;
    if (++i == rt * ns) {
      i = 0;
      if (++h == a.Hk) next_sequence();
    }
  }
  // Row tiles of a split follow each other: its keys are in L2 for the second.
  __device__ __forceinline__ Unit unit() const {
    Unit x;
    const int split = i / rt, r0 = (i - split * rt) * R, rows = min(R, s.n * a.G - r0);
    const int t0 = r0 / a.G, g0 = r0 - t0 * a.G;
    x.b = b;
    x.h = h;
    x.row = s.row0 + t0;
    x.first = s.total - s.n + t0;
    x.nt = x.first + (g0 + rows - 1) / a.G;
    x.tag = rows | g0 << kHeadShift;
    x.ns = t0;
    x.stop = min(max(x.nt + 1, 0), s.len);
    x.low = a.window ? min(max(x.first - a.window + 1, 0), x.stop) : 0;
    const int ta = x.low / kTile, tb = (x.stop + kTile - 1) / kTile;
    x.tile0 = ta + (int)((int64_t)(tb - ta) * split / ns);       // even splits
    x.tile1 = ta + (int)((int64_t)(tb - ta) * (split + 1) / ns);
    x.split = split | ns << 8;
    return x;
  }
};

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// ---- loads -----------------------------------------------------------------------------------
// Scales go by asynchronous copies of 16 bytes, a lane to each: a bulk copy for every page was slower with
// pages of 16, and through registers a tile waits for memory's latency.
constexpr int kScaleLanes = kTile / 16;
// Table entries come to the planner's registers 32 at a time, a lane to each (those of 4 to 64 tiles), ahead
// of their turn.
struct Ahead {
  int first, raw;        // the first entry; this lane's, as it lies
};
__device__ __forceinline__ Ahead find(const Args& a, int b, int first, int end, int lane) {
  const bool in = first + lane <= (end - 1) >> a.lps;
  return Ahead{first, in ? a.table[(int64_t)b * a.table_ld + first + lane] : 0};
}
// Codes of a tile by its groups' lanes (0 to 7); pages that are missing arrive as zeros.
template <int D>
__device__ __forceinline__ void load_codes(const Args& a, const CUtensorMap* map, const Tile& x, uint32_t dst,
                                           uint32_t bar, int l) {
  // (copies may land before their bytes are expected: the phase waits for this arrival)
  if (l == 0) mbar_expect_tx(bar, (uint32_t)(kTile * D));
  const int groups = 1 << (min(a.lps, 7) - 4);             // of a page
  if (l < kTile / 16 && (l & (groups - 1)) == 0)
    tma_load_4d(dst + l * 16 * D, map, 0, (x.row + l * 16) & ((1 << a.lps) - 1), x.h, x.page[l], bar);
}
// Its scales: K's by lanes 0 to 7, V's by lanes 8 to 15.  Nothing is read of a page that is missing.
__device__ __forceinline__ void load_scales(const Args& a, const Packed& kv, const Tile& x, uint32_t k_dst,
                                            uint32_t v_dst, uint32_t bar, int l) {
  const int i = l & (kScaleLanes - 1), page = x.page[i];
  const bool have = page < a.n_pages;
  const uint8_t* src = l < kScaleLanes ? kv.k_scale : kv.v_scale;
  if (have)
    src += page * kv.scale_stride + ((int64_t)x.h << a.lps) + ((x.row + i * 16) & ((1 << a.lps) - 1));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((l < kScaleLanes ? k_dst : v_dst) + i * 16),
               "l"(src), "r"(have ? 16 : 0)
               : "memory");
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- products --------------------------------------------------------------------------------
// Matrix descriptors: the lower word has the address and the leading offset (bytes), the upper one the stride
// and the layout (2: 128-byte swizzle, 4: 64-byte, 0: none) and does not change.
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride, uint32_t layout) {
  return (stride >> 4) | 1u << 14 | layout << 29;
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return (addr >> 4 & 0x3fffu) | (lead >> 4) << 16;
}
// D = A B (`acc` false) or D += A B.  (The issuing thread is alone: every instruction between two counts.)
template <uint32_t kAHi, uint32_t kBHi>
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %4};\n"
      " mov.b64 b, {%2, %5};\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kAHi), "n"(kBHi), "r"((uint32_t)acc));
}

constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kTile >> 4) << 24);   // fp32 of e4m3, M = 128

// ---- numbers ---------------------------------------------------------------------------------
// Two values as fp16 (nearest; the first one in the lower half)
__device__ __forceinline__ uint32_t to_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four fp16 numbers of at most 2^8 as `P` words of four codes: each part is what the ones before left,
// sixteen times, which fp16 holds exactly.
template <int P>
__device__ __forceinline__ void split4(uint32_t x, uint32_t y, uint32_t (&w)[P]) {
  const __half2 up = __float2half2_rn(16.f), down = __float2half2_rn(-16.f);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(x));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(y));
    w[p] = a | (uint32_t)b << 16;
    if (p + 1 == P) break;
    auto left = [&](uint32_t z, uint16_t code) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(code));
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&h), down,
                                __hmul2(*reinterpret_cast<const __half2*>(&z), up));
      return *reinterpret_cast<const uint32_t*>(&r);
    };
    x = left(x, a);
    y = left(y, b);
  }
}
// 2^(byte - 127), NaN for 255
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
}
// W consecutive columns of this thread's tensor-memory lane (no wait)
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t* r) {
  if constexpr (W == 8)
    tmem_ld8(t, r);
  else if constexpr (W == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(t));
  else
    tmem_ld2(t, r);
}
template <int W>
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t* r) {
  if constexpr (W == 8)
    tmem_st8(t, r);
  else if constexpr (W == 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(t), "r"(r[0]), "r"(r[1])
                 : "memory");
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
    k_packed_attn(const __grid_constant__ Args a, const int max_q, const int share, const int ns_cap,
                  const __grid_constant__ AttnOut o, const __grid_constant__ Packed kv,
                  const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                  const T* q, const int64_t q_stride) {
  using C = Cfg<T, D, R>;
  constexpr int KS = C::KS, VS = C::VS;
  constexpr uint32_t kRowLayout = D == 128 ? 2 : 4;   // of the tiles, rows of D bytes: swizzled by them
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler then knows that it is shared memory)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kCtlOff);
  int64_t* pre = reinterpret_cast<int64_t*>(smem);       // until the first tile is planned
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (by lanes: one thread for all of them took 4 us)
  if (warp == 0) {
    auto init = [&](uint64_t* bars, int n, uint32_t count) {
      if (lane < n) mbar_init(smem_u32(bars + lane), count);
    };
    init(ctl->kfull, KS, 1 + 2 * kScaleLanes);
    init(ctl->kempty, KS, 1);
    init(ctl->vempty, VS, 1);                            // epilogue
    // V by steps, as many of them as there are stages at most
    init(ctl->vfull, 8, C::KT + (lane == 0 ? a.withhold : 0));
    init(ctl->tfull, kSlots, 1);
    init(ctl->tempty, kSlots, 2);                        // K, V
    init(ctl->sfull, C::SB, 2);                          // the product, and its issuer, who has seen the scales
    init(ctl->sempty, C::SB, 4);                         // softmax
    init(ctl->qfull, 2, 2);
    init(ctl->qempty, 2, 8);                             // softmax
    init(ctl->pfull, 2, 4);
    init(ctl->ofull, 2, 1);
    init(ctl->oempty, 2, 4);
    init(ctl->meet, 2, 4);
    init(&ctl->done, 1, 2);
    init(ctl->ring.full, kUnits, 1);
    init(ctl->ring.empty, kUnits, kReaders);
    if (lane == 0) ctl->abort = ctl->any_bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctl->tmem)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  pdl_wait_and_trigger();
  pdl_trigger();
  prefix_units(a, pre, [&](int b) -> int64_t {
    const Seq s = seq_of(a, b);
    if (s.n == 0) return 0;
    check_len(a, s);
    const Shape x(a, s, R, max_q, share);
    return (int64_t)a.Hk * x.rt * x.ns * x.cost;
  });
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (tiles come to the same memory)
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  // S in SB buffers of a step each, then O in two
  const uint32_t tmem = ctl->tmem;
  // (waits that go on are calls: with their loops in place the roles' code is larger than the
  // instruction cache)
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_phase<true>(a, bar, parity, abort_flag); };
  // The tiles of K, with both scales, or of V, as the planner has them: two at a time, half a warp to each.
  // (One at a time took 1000 clocks a tile, nearly all of it latencies.)
  auto load_tiles = [&](auto kind, const CUtensorMap& map, uint64_t* empty) {
    constexpr bool kV = decltype(kind)::value;
    constexpr uint32_t S = kV ? VS : KS;
    const int half = lane >> 4, l = lane & 15;
    uint32_t n = 0, step = 0;                            // of tiles and steps before this round
    bool live = true;
#pragma unroll 1
    while (live) {
      const uint32_t m = n + half, i = m % S, slot = m % kSlots;
      wait(&ctl->tfull[slot], (m / kSlots) & 1);
      const Tile& x = ctl->tile[slot];
      const int lack = x.lack;
      live = x.h >= 0;
      if (live && m >= S) wait(&empty[i], (m / S - 1) & 1);
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
      const int ends = __shfl_sync(0xffffffffu, lack >= 0, 0);   // the first tile ends a step
      if (live) {
        const uint32_t full = smem_u32(kV ? &ctl->vfull[(step + (half ? ends : 0)) % 8] : &ctl->kfull[i]);
        if (!kV) {
          const uint32_t scale = smem_u32(smem + C::kScaleOff + slot * kTile);
          load_scales(a, kv, x, scale, scale + kSlots * kTile, full, l);
          if (l == 0) {
            ctl->bad[slot] = x.bad;
            if (x.bad) ctl->any_bad = 1;
          }
        }
        load_codes<D>(a, &map, x, smem_u32(smem + (kV ? C::kVOff : 0) + i * C::kTileBytes), full, l);
        // V is waited for by steps: the tiles that a step lacks count as there
        if (kV && lack > 0 && l == 0) mbar_arrive_n(full, lack);
      }
      __syncwarp();                                      // (the half warp has read the tile before it is given back)
      if (live && l == 0) mbar_arrive(smem_u32(&ctl->tempty[slot]));
      const uint32_t both = __ballot_sync(0xffffffffu, live);
      n += (both & 1u) + (both >> 16 & 1u);
      step += (both & 1u ? ends : 0) + __shfl_sync(0xffffffffu, live && lack >= 0 ? 1 : 0, 16);
      live = both == 0xffffffffu;
    }
    // every copy lands before the CTA may exit (bounded waits)
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) {
      if (kV) {
#pragma unroll 1
        for (uint32_t i = step > 8 ? step - 8 : 0; i < step; ++i)
          drain_phase(a, &ctl->vfull[i % 8], (i / 8) & 1);
      } else {
#pragma unroll 1
        for (uint32_t i = n > S ? n - S : 0; i < n; ++i) drain_phase(a, &ctl->kfull[i % S], (i / S) & 1);
      }
    }
    __syncwarp();
  };

  if (warp == 0) {
    // ---- planner: units, and their tiles' pages -------------------------------------------
    uint32_t n = 0, bad = 0;
    Walk walk(a, pre, R, max_q, share);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    bool more = !walk.done();
    Unit x{}, y{};
    Ahead now, next{};                                   // next: the next block of this unit, or the next unit's
    if (more) {
      x = walk.unit();
      next = find(a, x.b, x.tile0 * kTile >> a.lps, x.stop, lane);
    }
    uint32_t nu = 0;
#pragma unroll 1
    for (; more && !*abort_flag; x = y) {
      put_unit<true>(a, ctl->ring, nu++, x, lane, abort_flag);
      // the next unit's first entries are on their way while this one's tiles are handed on
      const int end = min(x.stop, x.tile1 * kTile);
      now = next;
      Ahead then = find(a, x.b, now.first + 32, end, lane);
      walk.next();
      more = !walk.done();
      if (more) {
        y = walk.unit();
        next = find(a, y.b, y.tile0 * kTile >> a.lps, y.stop, lane);
      }
      const bool past = x.nt >= x.stop;
#pragma unroll 1
      for (int t = x.tile0; t < x.tile1; ++t, ++n) {
        const int slot = n % kSlots, j0 = t * kTile, j = j0 + (lane & 7) * 16;
        if ((j0 >> a.lps) - now.first >= 32) {
          now = then;
          then = find(a, x.b, now.first + 32, end, lane);
        }
        const int raw = __shfl_sync(0xffffffffu, now.raw, (j >> a.lps) - now.first);
        const bool in = j < x.stop, have = in && (unsigned)raw < (unsigned)a.n_pages;
        const uint32_t missing = __ballot_sync(0xffffffffu, lane < 8 && !have && (in || past));
        if (n >= kSlots) wait(&ctl->tempty[slot], (n / kSlots - 1) & 1);
        if (*abort_flag) break;
        if (lane < 8) ctl->tile[slot].page[lane] = have ? raw : a.n_pages;
        if (lane == 0) {
          const int k = (t - x.tile0) % C::KT;
          ctl->tile[slot].h = x.h;
          ctl->tile[slot].row = j0 & ((1 << a.lps) - 1);
          ctl->tile[slot].lack = k == C::KT - 1 || t + 1 == x.tile1 ? C::KT - 1 - k : -1;
          ctl->tile[slot].bad = missing;
        }
        bad |= missing;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->tfull[slot]));
      }
    }
    Unit last{};
    last.b = -1;
    put_unit<true>(a, ctl->ring, nu, last, lane, abort_flag);
#pragma unroll 1
    for (int i = 0; i < 2; ++i, ++n) {                   // (two: tiles are loaded in pairs)
      const int slot = n % kSlots;
      if (n >= kSlots) wait(&ctl->tempty[slot], (n / kSlots - 1) & 1);
      if (lane == 0 && !*abort_flag) {
        ctl->tile[slot].h = -1;
        mbar_arrive(smem_u32(&ctl->tfull[slot]));
      }
    }
    if (bad && lane == 0) raise(a, PP_S_INDEX);
    __syncwarp();
  } else if (warp == 2) {
    load_tiles(std::false_type(), mapK, ctl->kempty);
  } else if (warp == 16) {
    load_tiles(std::true_type(), mapV, ctl->vempty);
  } else if (warp == 1) {
    // ---- MMA issuer of S ------------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t id = kIdesc | ((uint32_t)(C::NQ >> 3) << 17);
      const uint32_t k0 = desc_lo(smem_u32(smem), 0), q0 = desc_lo(smem_u32(smem + C::kQOff), 0);
      uint32_t n = 0, step = 0, nq = 0;
      Unit x;
#pragma unroll 1
      for (uint32_t nu = 0; get_unit<true>(a, ctl->ring, nu, x, lane, true, abort_flag); ++nu) {
        if (x.tile0 == x.tile1) continue;
        wait(&ctl->qfull[nq & 1], (nq >> 1) & 1);
#pragma unroll 1
        for (int t = x.tile0; t < x.tile1; t += C::KT, ++step) {
          const uint32_t sb = step % C::SB;
          if (step >= C::SB) wait(&ctl->sempty[sb], (step / C::SB - 1) & 1);
          const int tiles = min(C::KT, x.tile1 - t);
#pragma unroll 1
          for (int k = 0; k < tiles; ++k, ++n) {
            const uint32_t i = n % KS;
            wait(&ctl->kfull[i], (n / KS) & 1);
            if (*abort_flag) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t kt = k0 + i * (C::kTileBytes >> 4), qt = q0 + (nq & 1) * (C::kQBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_e4m3<desc_hi(8 * D, kRowLayout), desc_hi(1024, 2)>(
                  tmem + sb * (256 / C::SB) + k * C::NQ, kt + kk * 2, qt + kk * 2, id, kk > 0);
            umma_commit(smem_u32(&ctl->kempty[i]));
          }
          if (*abort_flag) break;
          mbar_arrive(smem_u32(&ctl->sfull[sb]));
          umma_commit(smem_u32(&ctl->sfull[sb]));
        }
        ++nq;
      }
      // every MMA is done before tensor memory is given back (bounded waits)
      umma_commit(smem_u32(&ctl->done));
      drain_phase(a, &ctl->done, 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---- MMA issuer of O ------------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t id = kIdesc | ((uint32_t)(C::NP >> 3) << 17) | (1u << 15) | (1u << 16);
      // V: dims contiguous, 8 keys to an atom of 8 D bytes (with 64 dims rows 64-127 of the product are
      // the keys 8 further on, and nobody reads them).  Weights: 16 columns of 8 keys to 128 bytes, keys
      // following each other, the next columns 2048 bytes on.
      const uint32_t v0 = desc_lo(smem_u32(smem + C::kVOff), 512), w0 = desc_lo(smem_u32(smem + C::kPOff), 128);
      uint32_t n = 0, step = 0;
      Unit x;
#pragma unroll 1
      for (uint32_t nu = 0; get_unit<true>(a, ctl->ring, nu, x, lane, true, abort_flag); ++nu) {
#pragma unroll 1
        for (int t = x.tile0; t < x.tile1; t += C::KT, ++step) {
          const uint32_t g = step & 1;
          wait(&ctl->vfull[step % 8], (step / 8) & 1);
          wait(&ctl->pfull[g], (step >> 1) & 1);        // (whose arrivals have waited for the last O of this buffer)
          if (*abort_flag) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const int tiles = min(C::KT, x.tile1 - t);
#pragma unroll 1
          for (int k = 0; k < tiles; ++k, ++n) {
            const uint32_t vt = v0 + n % VS * (C::kTileBytes >> 4);
            const uint32_t wt = w0 + (g * C::KT + k) * (C::kPBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < kTile / 32; ++kk)
              umma_e4m3<desc_hi(8 * D, kRowLayout), desc_hi(2048, 0)>(
                  tmem + 256 + g * 128, vt + kk * (32 * D >> 4), wt + kk * (512 >> 4), id, k + kk > 0);
          }
          umma_commit(smem_u32(&ctl->ofull[g]));
        }
      }
      umma_commit(smem_u32(&ctl->done));
      drain_phase(a, &ctl->done, 0);
    }
    __syncwarp();
  } else if (warp >= 17) {
    // ---- queries: L lanes to a row, four dims to a lane -----------------------------------
    constexpr int L = D / 4, kSide = 2 * 32 / L;           // rows side by side, of two warps
    constexpr int kAhead = R <= kSide ? 1 : R / kSide < 4 ? R / kSide : 4;   // passes loaded at once
    const int l = lane % L, side = (threadIdx.x - 544) / L;
    const uint32_t per_head = (65536u + a.G - 1) / a.G;    // f / G for f G < 2^16
    uint32_t nq = 0;
    Unit x;
#pragma unroll 1
    for (uint32_t nu = 0; get_unit<true>(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
      if (x.tile0 == x.tile1) continue;
      const uint32_t qb = nq & 1;
      if (nq >= 2) wait(&ctl->qempty[qb], ((nq >> 1) - 1) & 1);
      if (*abort_flag) break;
      const int rows = x.tag & 0xff, g0 = x.tag >> kHeadShift;
      const T* base = q + (int64_t)x.row * q_stride + (int64_t)x.h * a.G * D + l * 4;
      uint8_t* to = smem + C::kQOff + qb * C::kQBytes;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += kSide * kAhead) {
        uint2 raw[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int r = r0 + k * kSide + side;
          const uint32_t f = g0 + r, t = f * per_head >> 16;
          raw[k] = make_uint2(0u, 0u);
          if (r < rows)
            raw[k] = *reinterpret_cast<const uint2*>(base + t * q_stride + (int)(f - t * a.G) * D);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int r = r0 + k * kSide + side;
          float y[4] = {Num<T>::to_float(raw[k].x & 0xffffu), Num<T>::to_float(raw[k].x >> 16),
                        Num<T>::to_float(raw[k].y & 0xffffu), Num<T>::to_float(raw[k].y >> 16)};
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
#pragma unroll
          for (int w = L / 2; w > 0; w >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, w));
          // the row's power of two, as a cache entry's; a row that is not finite has NaN scores
          const bool wild = top >= 0x7f800000u;
          const int byte = max((int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
          const float f = wild ? 0.f : __uint_as_float((254u - (uint32_t)byte) << 23);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = wild ? 0.f : y[e] * f;
          uint32_t w[C::QP];
          split4<C::QP>(to_half(y[0], y[1]), to_half(y[2], y[3]), w);
          if (r >= R) continue;                          // (fewer rows than lie side by side)
#pragma unroll
          for (int p = 0; p < C::QP; ++p) {
            const int n = p * R + r;
            *reinterpret_cast<uint32_t*>(to + n * 128 + (((l >> 2) ^ (n & 7)) << 4) + (l & 3) * 4) =
                w[p];
          }
          if (l == 0) {
            ctl->row_c[qb][r] = wild ? __uint_as_float(0x7fc00000u) : a.c * scale_of((uint32_t)byte);
            ctl->row_at[qb][r] = x.first + (int)((g0 + r) * per_head >> 16);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->qfull[qb]));
      ++nq;
    }
  } else if (warp < 12) {
    // ---- softmax: thread k of a group owns key k of the group's tiles ---------------------
    const uint32_t g = warp >= 8;
    constexpr int W = C::W;
    const int wq = warp & 3, key = wq * 32 + lane;
    uint8_t* const weights = smem + C::kPOff + g * C::KT * C::kPBytes + key * 16;
    uint32_t n = 0, step = 0, nq = 0, meets = 0;
    Unit x;
#pragma unroll 1
    for (uint32_t nu = 0; get_unit<true>(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
      if (x.tile0 == x.tile1) continue;
      const uint32_t qb = nq & 1;
      const int rows = x.tag & 0xff;
      const bool mixed = x.first != x.nt;                // rows of several tokens
      wait(&ctl->qfull[qb], (nq >> 1) & 1);
#pragma unroll 1
      for (int t = x.tile0; t < x.tile1; t += C::KT, ++step) {
        const int tiles = min(C::KT, x.tile1 - t);
        n += tiles;
        if ((step & 1) != g) continue;
        if (*abort_flag) break;
        const uint32_t n0 = n - tiles;                   // the step's first tile
        auto k_scale = [&](int k) { return scale_of(smem[C::kScaleOff + (n0 + k) % kSlots * kTile + key]); };
        auto v_scale = [&](int k) -> uint32_t {
          return smem[C::kScaleOff + (kSlots + (n0 + k) % kSlots) * kTile + key];
        };
        const uint32_t sb = step % C::SB;
        const uint32_t scores = tmem + ((uint32_t)(wq * 32) << 16) + sb * (256 / C::SB);
        wait(&ctl->sfull[sb], (step / C::SB) & 1);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const bool bad = *reinterpret_cast<volatile int*>(&ctl->any_bad) != 0;
        // does every row see every key of the step?
        const int j0 = t * kTile + key;
        const bool partly = (t + tiles) * kTile - 1 > min(x.first, x.stop - 1) ||
                            (a.window && t * kTile <= x.nt - a.window);
        const bool edge = bad || partly;
        uint32_t see = ~0u;                              // bit k R + r: row r sees this thread's key of tile k
        uint32_t live = ~0u;                             // bit k: some row does
        if (edge) {
          see = live = 0u;
#pragma unroll 1
          for (int k = 0; k < tiles; ++k) {
            const int j = j0 + k * kTile;
            if (j >= x.stop || j < x.low || (ctl->bad[(n0 + k) % kSlots] >> (key >> 4) & 1u)) continue;
            live |= 1u << k;
            if (!mixed) {
              see |= (R == 32 ? ~0u : (1u << (R & 31)) - 1u) << (k * R);
              continue;
            }
#pragma unroll 1
            for (int r = 0; r < rows; ++r) {
              const int at = ctl->row_at[qb][r];
              see |= (j <= at && !(a.window && j <= at - a.window) ? 1u : 0u) << (k * R + r);
            }
          }
        }
        // ---- scores, as powers of two, -infinity where a row does not see the key, and the step's
        // maxima: lane r has row r's.  The scores wait in tensor memory, over S.
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < rows; c += W) {
          float most[W], f[W];
#pragma unroll
          for (int e = 0; e < W; ++e) {
            most[e] = -INFINITY;
            f[e] = ctl->row_c[qb][c + e];
          }
#pragma unroll 1
          for (int k = 0; k < tiles; ++k) {
            const uint32_t at = scores + k * C::NQ + c;
            uint32_t s[R < 8 ? 16 : C::QP * 8];          // parts side by side, R (8) columns apart
            if constexpr (R < 8) {
              tmem_ld16(at, s);
            } else {
#pragma unroll
              for (int p = 0; p < C::QP; ++p) tmem_ld8(at + p * R, s + p * 8);
            }
            const float kf = k_scale(k);
            const uint64_t kf2 = f32x2(kf, kf);
            float v[W];
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < W; e += 2) {
              uint64_t y = f32x2(after_wait(s[(C::QP - 1) * W + e]), after_wait(s[(C::QP - 1) * W + e + 1]));
#pragma unroll
              for (int p = C::QP - 2; p >= 0; --p)
                y = fma2(y, f32x2(0.0625f, 0.0625f),
                         f32x2(after_wait(s[p * W + e]), after_wait(s[p * W + e + 1])));
              y = mul2(y, mul2(kf2, f32x2(f[e], f[e + 1])));
              v[e] = lo_of(y);
              v[e + 1] = hi_of(y);
            }
            if (edge) {
              const uint32_t seen = see >> (k * R + c);
#pragma unroll
              for (int e = 0; e < W; ++e) v[e] = seen & (1u << e) ? v[e] : -INFINITY;
            }
            tmem_st<W>(at, reinterpret_cast<const uint32_t*>(v));
#pragma unroll
            for (int e = 0; e < W; ++e) most[e] = fmaxf(most[e], v[e]);
          }
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float y = warp_max(most[e]);
            if (lane - c == e) top = y;
          }
        }
        tmem_wait_st();
        // ---- V's scales (they came with K's): bit k of nan_value: the value of tile k reads as NaN
        uint32_t nan_value = 0, high = 0, low = 255;
#pragma unroll 1
        for (int k = 0; k < tiles; ++k) {
          const uint32_t ev = v_scale(k);
          if (ev == 255u) {
            nan_value |= 1u << k;
          } else if (live >> k & 1u) {
            high = max(high, ev);
            low = min(low, ev);
          }
        }
        high = __reduce_max_sync(0xffffffffu, high);
        low = __reduce_min_sync(0xffffffffu, low);
        float E = (float)high;
        if ((int)(high - low) > kSlack || (mixed && partly)) {
          // by the scores, and by what each row sees itself: lane r has row r's
          E = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < rows; c += W) {
            float most[W], f[W];
#pragma unroll
            for (int e = 0; e < W; ++e) {
              most[e] = -INFINITY;
              f[e] = -__shfl_sync(0xffffffffu, top, c + e);
            }
#pragma unroll 1
            for (int k = 0; k < tiles; ++k) {
              uint32_t s[W];
              tmem_ld<W>(scores + k * C::NQ + c, s);
              const uint32_t ev = v_scale(k);
              const float vf = ev == 255u ? 0.f : (float)ev;
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < W; ++e)                // (where there is no maximum: a NaN, which passes by)
                most[e] = fmaxf(most[e], after_wait(s[e]) + f[e] + vf);
            }
#pragma unroll
            for (int e = 0; e < W; ++e) {
              const float y = warp_max(most[e]);
              if (lane - c == e) E = y;
            }
          }
        }
        const uint32_t mb = (step >> 1) % kMaxima;
        if (lane < R) {
          ctl->warp_max[g][mb][wq][lane] = top;
          ctl->warp_e[g][mb][wq][lane] = E;
        }
        sync_warps<true>(a, &ctl->meet[g], meets, lane, abort_flag);
        // lane r works row r's reference out for its warp
        if (lane < R) {
#pragma unroll
          for (int w = 0; w < 4; ++w) top = fmaxf(top, ctl->warp_max[g][mb][w][lane]);
          E = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w)
            E = fmaxf(E, ctl->warp_e[g][mb][w][lane] + (ctl->warp_max[g][mb][w][lane] - top));
          E = ceilf(E);
          if (top != top) top = -INFINITY;               // (a row of NaN: its weights are NaN all the same)
          ctl->ref[g][wq][lane] = top == -INFINITY ? 0.f : kTop - top;
          ctl->fit[g][wq][lane] = -E;
        }
        // the last step's weights and sums of this buffer have been used
        if (step >= 2) wait(&ctl->oempty[g], ((step >> 1) - 1) & 1);
        // rows of V that must not be multiplied.  (Only such steps look at V here: its phases of eight steps
        // ago have been waited for by the product that this wait tells of.)
        if (edge) {
          wait(&ctl->vfull[step % 8], (step / 8) & 1);
#pragma unroll 1
          for (int k = 0; k < tiles; ++k) {
            const int j = j0 + k * kTile;
            uint4* row = reinterpret_cast<uint4*>(smem + C::kVOff + (n0 + k) % VS * C::kTileBytes + key * D);
            bool clear = !(live >> k & 1u);
            if (!clear && !(j <= x.first && (!a.window || j > x.nt - a.window))) {
              // some rows do not see it: its NaN codes must not meet their weights of zero
              uint32_t z = 0;
#pragma unroll 1
              for (int y = 0; y < D / 16; ++y) {
                const uint4 w = row[y];
                z |= ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                     ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
              }
              clear = (z & 0x80808080u) != 0;
              if (clear) nan_value |= 1u << k;
            }
            if (clear) {
#pragma unroll 1
              for (int y = 0; y < D / 16; ++y) row[y] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        if (wq == 0 && lane < R) {
          ctl->m[g][lane] = top;
          ctl->e[g][lane] = (uint32_t)E;
        }
        __syncwarp();
        // ---- weights, with an exponential of their own: p 2^(ev - E) would be 0 or not finite where p is below
        // fp32's range, or that power above it
#pragma unroll 1
        for (int c = 0; c < rows; c += W) {
          float f[W], u[W], sum[W];
#pragma unroll
          for (int e = 0; e < W; ++e) {
            f[e] = ctl->ref[g][wq][c + e];
            u[e] = ctl->fit[g][wq][c + e];
            sum[e] = 0.f;
          }
#pragma unroll 1
          for (int k = 0; k < tiles; ++k) {
            uint32_t s[W], y[W / 2];
            tmem_ld<W>(scores + k * C::NQ + c, s);
            const float vf = nan_value >> k & 1u ? __uint_as_float(0x7fc00000u) : (float)v_scale(k);
            const uint64_t vf2 = f32x2(vf, vf);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < W; e += 2) {
              const float v0 = after_wait(s[e]), v1 = after_wait(s[e + 1]);
              const uint64_t x2 = add2(f32x2(v0, v1), f32x2(f[e], f[e + 1]));
              const float p0 = exp2_approx(lo_of(x2)), p1 = exp2_approx(hi_of(x2));
              const uint64_t w2 = add2(x2, add2(vf2, f32x2(u[e], u[e + 1])));
              float w0 = exp2_approx(lo_of(w2)), w1 = exp2_approx(hi_of(w2));
              if (edge) {                                // (not a NaN of a value that a row does not see)
                if (v0 == -INFINITY) w0 = 0.f;
                if (v1 == -INFINITY) w1 = 0.f;
              }
              y[e / 2] = to_half(w0, w1);
              sum[e] += p0;
              sum[e + 1] += p1;
            }
            uint8_t* to = weights + k * C::kPBytes;
            uint32_t w[2][kParts];
            if constexpr (W == 2) {                      // columns: two rows' first parts, then their second, ..
              split4<kParts>(y[0], y[0], w[0]);
              *reinterpret_cast<uint2*>(to) =
                  make_uint2(__byte_perm(w[0][0], w[0][1], 0x5410), w[0][2] & 0xffffu);
            } else if constexpr (W == 4) {
              split4<kParts>(y[0], y[1], w[0]);
              *reinterpret_cast<uint2*>(to) = make_uint2(w[0][0], w[0][1]);
              *reinterpret_cast<uint32_t*>(to + 8) = w[0][2];
            } else {
              split4<kParts>(y[0], y[1], w[0]);
              split4<kParts>(y[2], y[3], w[1]);
#pragma unroll
              for (int p = 0; p < kParts; ++p) {
                const int col = p * R + c;
                *reinterpret_cast<uint2*>(to + (col >> 4) * 2048 + (col & 15)) = make_uint2(w[0][p], w[1][p]);
              }
            }
          }
          // sums of the rows over the warp's keys: lanes halve the rows while there are several
          int row = c;
#pragma unroll
          for (int d = 16, k = W / 2; d > 0; d >>= 1, k >>= 1) {
            if (k > 0) {
              const bool up = lane & d;
              row += up ? k : 0;
#pragma unroll
              for (int e = 0; e < k; ++e) {
                const float give = up ? sum[e] : sum[e + k];
                sum[e] = (up ? sum[e + k] : sum[e]) + __shfl_xor_sync(0xffffffffu, give, d);
              }
            } else {
              sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], d);
            }
          }
          if ((lane & (32 / W - 1)) == 0) ctl->l[g][wq][row] = sum[0];
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctl->pfull[g]));
          mbar_arrive(smem_u32(&ctl->sempty[sb]));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->qempty[qb]));
      ++nq;
    }
  } else {
    // ---- epilogue: thread d owns dim d; lane r of each warp keeps row r's maximum and sum ---
    constexpr int W = C::W;
    const int wq = warp & 3, d = wq * 32 + lane, H = a.Hk * a.G;
    const uint32_t lane_at = tmem + ((uint32_t)(wq * 32) << 16) + 256;
    uint32_t n = 0, step = 0;
    Unit x;
#pragma unroll 1
    for (uint32_t nu = 0; get_unit<true>(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
      const int rows = x.tag & 0xff;
      float acc[R], M = -INFINITY, Lsum = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = 0.f;
#pragma unroll 1
      for (int t = x.tile0; t < x.tile1; t += C::KT, ++step) {
        const uint32_t g = step & 1, ph = (step >> 1) & 1;
        wait(&ctl->pfull[g], ph);                        // sums and maxima
        if (lane < R) {
          const float m = ctl->m[g][lane];
          const float l = (ctl->l[g][0][lane] + ctl->l[g][1][lane]) +
                          (ctl->l[g][2][lane] + ctl->l[g][3][lane]);
          const float top = fmaxf(M, m);
          // (a side without a reference has nothing, or NaN, which passes)
          const float keep = M == -INFINITY ? 0.f : exp2_approx(M - top);
          const float add = m == -INFINITY ? 0.f : exp2_approx(m - top);
          constexpr float down = 1.f / 256.f;            // 2^-kTop
          Lsum = Lsum * keep + l * (add * down);
          M = top;
          ctl->keep[wq][lane] = keep;
          ctl->add[wq][lane] = add * scale_of(ctl->e[g][lane]) * down;
        }
        __syncwarp();
        wait(&ctl->ofull[g], ph);
        if (*abort_flag) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int c = 0; c < R; c += W) {
          if (c >= rows) break;
          uint32_t y[R < 8 ? 16 : kParts * 8];           // parts side by side, R (8) columns apart
          if constexpr (R < 8) {
            tmem_ld16(lane_at + g * 128, y);
          } else {
#pragma unroll
            for (int p = 0; p < kParts; ++p) tmem_ld8(lane_at + g * 128 + p * R + c, y + p * 8);
          }
          float keep[W], add[W];
#pragma unroll
          for (int e = 0; e < W; ++e) {
            keep[e] = ctl->keep[wq][c + e];
            add[e] = ctl->add[wq][c + e];
          }
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float z = fmaf(fmaf(after_wait(y[2 * W + e]), 0.0625f, after_wait(y[W + e])), 0.0625f,
                                 after_wait(y[e]));
            acc[c + e] = fmaf(acc[c + e], keep[e], z * add[e]);
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->oempty[g]));
        const int tiles = min(C::KT, x.tile1 - t);
        if (wq == 0 && lane < tiles) mbar_arrive(smem_u32(&ctl->vempty[(n + lane) % VS]));
        n += tiles;
      }
      if (*abort_flag) break;
      // lane r: where row r goes
      const int f = (x.tag >> kHeadShift) + min(lane, rows - 1), tk = f / a.G;
      const int hd = x.h * a.G + f - tk * a.G;
      const bool whole = x.split >> 8 == 1;
      const int64_t row = (int64_t)(x.row + tk) * H + hd;
      const int64_t rec =
          (((int64_t)x.b * max_q + x.ns + tk) * H + hd) * ns_cap + (x.split & 0xff);
      const float inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
      if (wq == 0 && lane < rows) {
        if (!whole)
          o.part_ml[rec] = make_float2(M, Lsum);
        else if (o.lse)
          o.lse[row] = Lsum == 0.f ? -INFINITY : (M + log2f(Lsum)) * kLn2;
      }
      const int64_t place = whole ? row : rec;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const int64_t to = __shfl_sync(0xffffffffu, place, r) * D + d;
        const float scale = __shfl_sync(0xffffffffu, inv, r);
        if (d >= D) continue;
        if (!whole)
          o.part[to] = acc[r];
        else
          reinterpret_cast<uint16_t*>(o.out)[to] = (uint16_t)Num<T>::pack(acc[r] * scale, 0.f);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// Join the splits of each row, in split order: one warp to a (token, head).
template <typename T, int D>
__global__ void __launch_bounds__(128)
    k_packed_join(const __grid_constant__ Args a, const int R, const int max_q, const int share,
                  const int ns_cap, const __grid_constant__ AttnOut o) {
  pdl_wait_and_trigger();
  pdl_trigger();
  const int lane = threadIdx.x & 31, H = a.Hk * a.G;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);   // (sequence, token, head)
  const int64_t rest = id / H;
  const int hd = (int)(id - rest * H), b = (int)(rest / max_q), tk = (int)(rest - (int64_t)b * max_q);
  if (b >= a.n_seqs) return;
  const Seq s = seq_of(a, b);
  if (s.n > max_q || tk >= s.n) return;
  const int ns = n_splits(most_tiles(s.len, a.window, row_span(R, a.G)), share);
  if (ns == 1) return;
  const int64_t row = (int64_t)(s.row0 + tk) * H + hd;
  join_row<T, D>(o.part, o.part_ml, id * ns_cap, ns, reinterpret_cast<T*>(o.out) + row * D,
                 o.lse ? o.lse + row : nullptr, lane);
}

template <typename T, int D, int R>
cudaError_t run(const Args& a, const PackedPlan& p, const Maps& maps, const AttnOut& o, const Packed& kv,
                const void* q, int64_t q_stride, cudaStream_t s) {
  using C = Cfg<T, D, R>;
  static_assert(C::KS + C::SB * C::KT <= kSlots && C::VS <= 8, "scales outlive the steps that are under way");
  static_assert(C::kQBytes % 1024 == 0 && C::kPBytes % 1024 == 0 && C::KT * C::NQ <= 128 && C::NP <= 128,
                "operands start on 1024 bytes, products fit their columns");
  constexpr size_t smem = C::kCtlOff + sizeof(Ctl) + 1024, most_smem = smem;
  static_assert((kMaxSeqs + 1) * sizeof(int64_t) <= C::kVOff, "prefix sums lie where the K tiles come to");
  static_assert(most_smem <= 227 * 1024, "attention shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(k_packed_attn<T, D, R>), most_smem, done);
  if (err != cudaSuccess) return err;
  // no more CTAs than units there can be
  const int64_t row_tiles = (int64_t)a.T * a.G / R + a.n_seqs;
  const int64_t most = row_tiles * a.Hk * p.ns_cap;
  const int nsm = sm_count();
  err = launch(k_packed_attn<T, D, R>, dim3((unsigned)(most < nsm ? most : nsm)), kThreads, smem, s, a,
               p.max_q, p.share, p.ns_cap, o, kv, maps.k, maps.v, reinterpret_cast<const T*>(q), q_stride);
  if (err != cudaSuccess || p.ns_cap == 1) return err;
  const int64_t rows = (int64_t)a.n_seqs * p.max_q * a.Hk * a.G;
  return launch(k_packed_join<T, D>, dim3((unsigned)((rows + 3) / 4)), 128, 0, s, a, R, p.max_q, p.share,
                p.ns_cap, o);
}

template <typename T, int D>
cudaError_t pick(const Args& a, const PackedPlan& p, const Maps& maps, const AttnOut& o,
                 const Packed& kv, const void* q, int64_t q_stride, cudaStream_t s) {
  return p.R == 2    ? run<T, D, 2>(a, p, maps, o, kv, q, q_stride, s)
         : p.R == 4  ? run<T, D, 4>(a, p, maps, o, kv, q, q_stride, s)
         : p.R == 8  ? run<T, D, 8>(a, p, maps, o, kv, q, q_stride, s)
         : p.R == 16 ? run<T, D, 16>(a, p, maps, o, kv, q, q_stride, s)
                     : run<T, D, 32>(a, p, maps, o, kv, q, q_stride, s);
}

}  // namespace

PackedPlan packed_plan(const Args& a, int max_q) {
  PackedPlan p{};
  const int rows = max_q * a.G;
  p.R = 2;
  while (p.R < rows && p.R < 32) p.R *= 2;
  p.max_q = max_q;
  const int heads = a.Hk * ((rows + p.R - 1) / p.R);
  p.share = kSms / heads < 1 ? 1 : kSms / heads;
  const int64_t tiles = most_tiles((int64_t)a.table_ld << a.lps, a.window, row_span(p.R, a.G));
  // shorter sequences have `share` splits at most or one for every kMost tiles, and one for every kLeast at most
  int64_t most = (tiles + kLeast - 1) / kLeast;
  const int64_t by_share = p.share > (tiles + kMost - 1) / kMost ? p.share : (tiles + kMost - 1) / kMost;
  if (by_share < most) most = by_share;
  p.ns_cap = (int)(most < 1 ? 1 : most < 128 ? most : 128);
  const size_t recs = (size_t)a.n_seqs * max_q * a.Hk * a.G * p.ns_cap;
  p.rec_bytes = p.ns_cap == 1 ? 0 : (recs * a.D * sizeof(float) + 255) & ~(size_t)255;
  p.ml_bytes = p.ns_cap == 1 ? 0 : (recs * sizeof(float2) + 255) & ~(size_t)255;
  return p;
}

cudaError_t launch_packed_attn(const Args& a, int type, const PackedPlan& plan, const Maps& maps,
                               const AttnOut& o, const Packed& kv, const void* q, int64_t q_stride,
                               cudaStream_t s) {
  if (type == PP_BF16)
    return a.D == 128 ? pick<__nv_bfloat16, 128>(a, plan, maps, o, kv, q, q_stride, s)
                      : pick<__nv_bfloat16, 64>(a, plan, maps, o, kv, q, q_stride, s);
  return a.D == 128 ? pick<__half, 128>(a, plan, maps, o, kv, q, q_stride, s)
                    : pick<__half, 64>(a, plan, maps, o, kv, q, q_stride, s);
}

}  // namespace paged
}  // namespace pp
