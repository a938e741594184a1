// k_paged_attn.cu - attention of a chunk of new tokens over the paged cache: single tokens and
// short chunks (k_paged_attn_tc.cu has the long ones).
//
// For row (t, g) of a sequence (new token t of n, query head g of a key head's G), with L
// cache entries, the new ones included and last:
//   p(t) = L - n + t;  keys j in (p - window, p] (or [0, p]) that the table's row has room for;
//   out = sum_j exp(s_j - lse) V_j,  s_j = scale q . K_j,  lse = log sum_j exp(s_j).
// One pass over the keys with a running reference m and sum l, in powers of two.
//
// Bound by reading K and V once.  A work unit is (sequence, row tile, key head, split of its
// keys): up to 16 * WR rows (whole tokens with all their G heads, so a key is read once for all
// of them) against a run of 128-key tiles.  Each CTA takes a run of consecutive units with about
// the same number of tiles as the others; a sequence's splits depend on its own lengths and the
// head counts only, so its bits do not depend on the rest of the batch.
//
//   warp 0      the units, their query rows and K tiles by TMA, one box to a lane;
//   warp 1      the V tiles (with pages of 16 a tile is 16 boxes: one warp for both was 328 us on
//               the 64-session tick);
//   warps 4-11  in two teams of four.  Up to 16 rows: a team to every second tile of a unit; up to 32:
//               a team to 16 rows, both to every tile.  A warp takes 32 keys of a tile: S and P V
//               as 16 x 8 x 16 matrix products, P handed from one to the other in registers,
//               with the warp's own m, l and O (16 rows x D in fp32 registers).
//               (All 32 rows in one warp, a team to every second tile, measured 295 us on 8
//               sequences of up to 5 tokens x 4 heads over up to 65000 entries.)
//
// The warps meet only at a unit's end, where the eight (m, l, O) are joined through shared
// memory.  (A tile shared by all warps, with the maxima and P exchanged under two barriers a
// tile, measured 350 us on the 64-session tick: its tile took 4500 clocks, of which the products
// were a third.)  A unit that is not its rows' only one leaves (m, l, O) in fp32 in scratch and
// k_paged_join adds the splits up in split order.
//
// Keys that some row of a tile may not see need care in the second product, where a
// weight of zero times a stored infinity would be NaN: on such tiles every non-finite
// value of V is taken out of the product and, at the unit's end, added to the rows that see
// the key.
//
// Measured (128 dims, in a graph): 64 sequences of 1 token and up to 3000 entries, 32 heads on 32
// key heads, pages of 64, bf16: 269 us, 5.7 TB/s (0.84 of the measured copy rate; 1.01 with equal
// lengths: what is left are the ends of the many short units, about 4500 clocks each).  8
// sequences of up to 5 tokens and 65000 entries, 32 heads on 8, pages of 16, fp16: 212 us, 4.4
// TB/s, bound by the products of up to 20 rows with mma.sync.  One token over 3000 entries, 32
// heads: 14 us, half of it launches, the first tiles' way and the join.
#include "pp_paged.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 128 + kWarps * 32;
// registers a thread: launched with 168; warps 4-11 take what warps 0-3 give up
// (56 + 2 x 224 = 3 x 168)
constexpr int kRegsFew = 56, kRegsMany = 224;
constexpr int kQBufs = 2;
constexpr int kJoinRows = 4;         // rows joined at a time at a unit's end
constexpr float kLag = 8.f;          // a row's maximum may exceed its reference by this (log2)

template <int D, int WR>
struct Cfg {
  static constexpr int R = 16 * WR;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int KS = D == 128 ? 3 : 6;
  static constexpr int VS = D == 128 ? (WR == 1 ? 3 : 2) : (WR == 1 ? 6 : 5);
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kVOff = KS * kTileBytes;
  static constexpr int kQOff = kVOff + VS * kTileBytes;
  static constexpr int kJoinOff = kQOff + kQBufs * kQBytes;       // [8 warps][4 rows][D] floats
  static constexpr int kMlOff = kJoinOff + kWarps * kJoinRows * D * 4;   // [8 warps][16] (m, l)
  static constexpr int kCtlOff = kMlOff + kWarps * 16 * 8;
};

struct Ctl {
  UnitRing ring;
  uint64_t kfull[6], kempty[6], vfull[6], vempty[6], qfull[kQBufs], qempty[kQBufs];
  uint64_t meet;         // of the eight warps
  uint32_t bad[6];
  int wild;              // 1 + place of the unit in which a non-finite V was taken out
  int abort;
};

// Key tiles that a row tile of up to tp tokens can touch, at most.
__device__ __forceinline__ int max_tiles(const Args& a, int len, int tp) {
  const int all = (len + kTile - 1) / kTile;
  return a.window ? min(all, (int)(((int64_t)a.window + tp - 2) / kTile) + 2) : all;
}
// Tiles of one split.  Only chunks of a single row tile are split (the host's plan expects no
// others).  `share` splits of each key head fill the SMs when a sequence is alone (its bits do
// not depend on whether it is).  A split has at least four tiles: its end costs 4500 clocks,
// which four tiles' loads (2900 clocks each at an SM's share of the bandwidth) hide and two do
// not.  It has at most eight, so that runs of units come out even, and a sequence at most 128
// splits.
__host__ __device__ __forceinline__ int split_tiles(int tiles, int share) {
  int st = (tiles + share - 1) / share;
  st = st < 4 ? 4 : st > 8 ? 8 : st;
  const int even = (tiles + 127) / 128;
  return st > even ? st : even;
}
__host__ __device__ __forceinline__ int n_splits(int tiles, int share) {
  const int st = split_tiles(tiles, share);
  return tiles <= st ? 1 : (tiles + st - 1) / st;
}

// A walk over this CTA's units, in order.
struct Walk {
  const Args& a;
  const int* pre;
  const int tp, share;
  int at, end;           // cost before this unit, cost where the run ends (half tiles)
  int b, h, i;           // sequence, key head, unit of the head
  Seq s;
  int rt, st, ns, per;   // row tiles, tiles of a split, splits, units of a head
  int cost;              // of a unit
  int t0, nt;            // first token of the row tile, its tokens
  int first;             // entry index of that token
  int tile0, tile1;      // key tiles of the split
  int stop;              // entries that the last row sees end here (or the table's row does)

  __device__ __forceinline__ Walk(const Args& a_, const int* pre_, int tp_, int share_)
      : a(a_), pre(pre_), tp(tp_), share(share_) {
    const int64_t total = pre[a.n_seqs];
    at = (int)(total * blockIdx.x / gridDim.x);
    end = (int)(total * (blockIdx.x + 1) / gridDim.x);
    if (at >= end) return;
    b = find_seq(pre, a.n_seqs, at);
    sequence();
    const int k = (at - pre[b] + cost - 1) / cost;   // the first unit that starts in the run
    h = k / per;
    i = k - h * per;
    at = pre[b] + k * cost;
    if (h == a.Hk) next_sequence();
    unit();
  }
  __device__ __forceinline__ bool done() const { return at >= end; }
  // Units of one head: its splits, or (several row tiles) one for each.  A unit costs its
  // tiles' loads or, if they are few, their products and its end.
  static __device__ __forceinline__ int head_units(const Args& a, const Seq& s, int tp, int share,
                                                   int& rt, int& st, int& ns, int& cost) {
    rt = (s.n + tp - 1) / tp;
    const int mt = max_tiles(a, s.len, tp), few = min(split_tiles(mt, share), max(mt, 1));
    st = split_tiles(mt, share);
    ns = rt > 1 ? 1 : n_splits(mt, share);
    cost = rt > 1 ? 1 : max(2 * few, few + 3);
    return rt > 1 ? rt : ns;
  }
  __device__ __forceinline__ void sequence() {
    s = seq_of(a, b);
    per = head_units(a, s, tp, share, rt, st, ns, cost);
  }
  __device__ __forceinline__ void next_sequence() {
    h = i = 0;
    do {
      ++b;
    } while (b < a.n_seqs && pre[b + 1] == pre[b]);
    if (b < a.n_seqs) sequence();
  }
  __device__ __forceinline__ void next() {
    at += cost;
    if (++i == per) {
      i = 0;
      if (++h == a.Hk) next_sequence();
    }
    unit();
  }
  __device__ __forceinline__ void unit() {
    if (done()) return;
    t0 = rt > 1 ? i * tp : 0;
    nt = min(tp, s.n - t0);
    first = s.total - s.n + t0;
    stop = min(max(first + nt, 0), s.len);
    const int lo = a.window ? max(first - a.window + 1, 0) : 0;
    const int ta = min(lo, stop) / kTile, tb = (stop + kTile - 1) / kTile;
    tile0 = rt > 1 ? ta : min(ta + i * st, tb);
    tile1 = rt > 1 ? tb : min(tile0 + st, tb);
  }
};

// Row half i of the accumulators (rows 8i .. 8i + 7) times f.
template <int D>
__device__ __forceinline__ void scale_rows(float (&acc)[D / 8][4], int i, float f) {
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    acc[n][i * 2] *= f;
    acc[n][i * 2 + 1] *= f;
  }
}

template <typename T, int D, int WR>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attn(const __grid_constant__ Args a, const int tp, const int share, const int ns_cap, const __grid_constant__ AttnOut o,
                 const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                 const __grid_constant__ CUtensorMap mapQ, const void* v_pages) {
  using C = Cfg<D, WR>;
  using N = Num<T>;
  constexpr int R = C::R;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler then knows that it is shared memory)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kCtlOff);
  int* pre = reinterpret_cast<int*>(ctl + 1);
  volatile int* abort_flag = &ctl->abort;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KS; ++i) {
      mbar_init(smem_u32(&ctl->kfull[i]), 1);
      mbar_init(smem_u32(&ctl->kempty[i]), kWarps);
    }
    for (int i = 0; i < C::VS; ++i) {
      mbar_init(smem_u32(&ctl->vfull[i]), i == 0 ? 1 + a.withhold : 1);
      mbar_init(smem_u32(&ctl->vempty[i]), kWarps);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(smem_u32(&ctl->qfull[i]), 1);
      mbar_init(smem_u32(&ctl->qempty[i]), kWarps);
    }
    ring_init(ctl->ring, kWarps + 1);   // the V producer too
    mbar_init(smem_u32(&ctl->meet), kWarps);
    ctl->wild = 0;
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait_and_trigger();
  pdl_trigger();
  prefix_units(a, pre, [&](int b) {
    const Seq s = seq_of(a, b);
    if (s.n == 0) return 0;
    check_len(a, s);
    int rt, st, ns, cost;
    return a.Hk * Walk::head_units(a, s, tp, share, rt, st, ns, cost) * cost;
  });
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_phase(a, bar, parity, abort_flag); };

  if (threadIdx.x < 128) {
    // ---- producer -------------------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (threadIdx.x < 32) {
      uint32_t nq = 0, nk = 0, nu = 0, seen_bad = 0;
      Walk x(a, pre, tp, share);
#pragma unroll 1
      for (; !x.done() && !*abort_flag; x.next()) {
        put_unit(a, ctl->ring, nu++,
                 Unit{x.b, x.h, x.s.row0 + x.t0, x.nt, x.first, x.tile0, x.tile1,
                      a.window ? max(x.first - a.window + 1, 0) : 0, x.stop, x.i, x.ns, x.at + 1},
                 lane, abort_flag);
        if (x.tile0 == x.tile1) continue;
        const bool past = x.first + x.nt > x.stop;
        TilePages next = find_pages(a, x.b, x.tile0 * kTile, x.stop, past, lane);
        const int qb = nq % kQBufs;
        if (nq >= kQBufs) wait(&ctl->qempty[qb], (nq / kQBufs - 1) & 1);
        if (*abort_flag) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&ctl->qfull[qb]);
          const uint32_t dst = smem_u32(smem + C::kQOff + qb * C::kQBytes);
          // rows past the row tile's tokens may be another sequence's: their results go nowhere
          mbar_expect_tx(bar, (uint32_t)(tp * a.G * D * 2));
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_4d(dst + bx * (R * 128), &mapQ, bx * 64, x.h * a.G, x.s.row0 + x.t0, 0, bar);
        }
        ++nq;
#pragma unroll 1
        for (int t = x.tile0; t < x.tile1; ++t, ++nk) {
          const int ks = nk % C::KS;
          const TilePages now = next;
          if (t + 1 < x.tile1) next = find_pages(a, x.b, (t + 1) * kTile, x.stop, past, lane);
          if (nk >= C::KS) wait(&ctl->kempty[ks], (nk / C::KS - 1) & 1);
          if (*abort_flag) break;
          load_key_tile(a, &mapK, smem_u32(smem + ks * C::kTileBytes), smem_u32(&ctl->kfull[ks]),
                        now, x.h, t * kTile, lane, nullptr);
          seen_bad |= now.bad;
        }
      }
      Unit last{};
      last.b = -1;
      put_unit(a, ctl->ring, nu, last, lane, abort_flag);
      if (seen_bad && lane == 0) raise(a, PP_S_INDEX);
      // every copy lands before the CTA may exit (bounded waits)
      if (lane == 0) {
#pragma unroll 1
        for (uint32_t i = nq > kQBufs ? nq - kQBufs : 0; i < nq; ++i)
          drain_phase(a, &ctl->qfull[i % kQBufs], (i / kQBufs) & 1);
#pragma unroll 1
        for (uint32_t i = nk > C::KS ? nk - C::KS : 0; i < nk; ++i)
          drain_phase(a, &ctl->kfull[i % C::KS], (i / C::KS) & 1);
      }
    } else if (threadIdx.x < 64) {
      uint32_t nv = 0;
      Unit x;
#pragma unroll 1
      for (uint32_t nu = 0; get_unit(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
        if (x.tile0 == x.tile1) continue;
        const bool past = x.first + x.nt > x.stop;
        TilePages next = find_pages(a, x.b, x.tile0 * kTile, x.stop, past, lane);
#pragma unroll 1
        for (int t = x.tile0; t < x.tile1; ++t, ++nv) {
          const int vs = nv % C::VS;
          const TilePages now = next;
          if (t + 1 < x.tile1) next = find_pages(a, x.b, (t + 1) * kTile, x.stop, past, lane);
          if (nv >= C::VS) wait(&ctl->vempty[vs], (nv / C::VS - 1) & 1);
          if (*abort_flag) break;
          load_key_tile(a, &mapV, smem_u32(smem + C::kVOff + vs * C::kTileBytes),
                        smem_u32(&ctl->vfull[vs]), now, x.h, t * kTile, lane, &ctl->bad[vs]);
        }
      }
      if (lane == 0) {
#pragma unroll 1
        for (uint32_t i = nv > C::VS ? nv - C::VS : 0; i < nv; ++i)
          drain_phase(a, &ctl->vfull[i % C::VS], (i / C::VS) & 1);
      }
    }
    return;
  }

  // ---- consumers ----------------------------------------------------------------------------
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
  const int tid = threadIdx.x - 128, warp = tid >> 5;
  const int lm = lane >> 3, lr = lane & 7;      // ldmatrix: matrix and row of this lane
  const int fr = lane >> 2, fc = (lane & 3) * 2;   // fragment row and column pair
  float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff);
  float* join = reinterpret_cast<float*>(smem + C::kJoinOff);
  const int team = warp >> 2, part = warp & 3;   // which of a tile's keys
  constexpr bool kRowTeams = WR == 2;
  const int row0 = kRowTeams ? team * 16 : 0;    // this warp's first row
  int tok[2];                                    // this thread's rows: their token of the row tile
#pragma unroll
  for (int i = 0; i < 2; ++i) tok[i] = (row0 + i * 8 + fr) / a.G;
  uint32_t nq = 0, n = 0, meets = 0;            // n: tiles of this CTA
  Unit x;
#pragma unroll 1
  for (uint32_t nu = 0; get_unit(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
    const int rows = x.nt * a.G;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[D / 8][4];
#pragma unroll
    for (int y = 0; y < D / 8; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[y][e] = 0.f;

    const int qb = nq % kQBufs;
    const uint32_t qbuf = smem_u32(smem + C::kQOff + qb * C::kQBytes);
    if (x.tile0 < x.tile1) wait(&ctl->qfull[qb], (nq / kQBufs) & 1);
    uint32_t aq[D / 16][4];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      ldsm4(tile_addr(qbuf, R * 128, row0 + (lm & 1) * 8 + lr, kk * 2 + (lm >> 1)), aq[kk]);
#pragma unroll 1
    for (int t = x.tile0; t < x.tile1; ++t, ++n) {
      const int ks = n % C::KS, vs = n % C::VS;
      wait(&ctl->kfull[ks], (n / C::KS) & 1);
      // (counted within the unit: which warp sums a tile must not depend on this CTA's past units)
      if (!kRowTeams && ((t - x.tile0) & 1) != team) {
        // the other team's tile: every warp sees every phase of every stage all the same (a
        // phase that passed unseen could not be told from the one before it)
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->kempty[ks]));
        wait(&ctl->vfull[vs], (n / C::VS) & 1);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->vempty[vs]));
        continue;
      }
      const int j1 = t * kTile + part * 32;     // this warp's first key
      // ---- S = Q K^T: this warp's 32 keys, every row
      const uint32_t kbuf = smem_u32(smem + ks * C::kTileBytes);
      float s[4][4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[y][e] = 0.f;
      constexpr int kAhead = 4;                 // steps whose loads go out together
#pragma unroll
      for (int k0 = 0; k0 < D / 16; k0 += kAhead) {
        uint32_t bk[kAhead][2][4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            ldsm4(tile_addr(kbuf, kTile * 128, part * 32 + y * 16 + (lm >> 1) * 8 + lr,
                            (k0 + k) * 2 + (lm & 1)), bk[k][y]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            N::mma(s[y], aq[k0 + k], bk[k][y >> 1][(y & 1) * 2], bk[k][y >> 1][(y & 1) * 2 + 1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->kempty[ks]));
      // which parts of the tile have no page comes with its V tile
      const uint32_t vbuf = smem_u32(smem + C::kVOff + vs * C::kTileBytes);
      wait(&ctl->vfull[vs], (n / C::VS) & 1);
      const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&ctl->bad[vs]);
      // does every row see every key of the tile?
      const bool edge = bad != 0 || (t + 1) * kTile - 1 > x.first ||
                        (a.window && t * kTile <= x.first + x.nt - 1 - a.window);
      if (edge) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // the row sees keys (lo, hi], counted from this thread's first
          const int hi = x.first + min(tok[i], x.nt - 1) - j1 - fc;
          const int lo = a.window ? hi - a.window : -1;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const bool none = (bad >> (part * 2 + (y >> 1))) & 1u;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (none || y * 8 + e > hi || y * 8 + e <= lo)
                s[y][i * 2 + e] = -INFINITY;
          }
        }
      }
      uint32_t ap[2][4];                        // P as the second product's operand
      float grow[2];
      bool grown = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float p[4][2];
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) p[y][e] = s[y][i * 2 + e];
        float top = fmaxf(fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[1][0], p[1][1])),
                          fmaxf(fmaxf(p[2][0], p[2][1]), fmaxf(p[3][0], p[3][1])));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = fmaf(top, a.c, -N::kShift);
        // the reference follows the maximum only when it falls behind by kLag (or is none yet)
        const float mn = top > m[i] + kLag || m[i] == -INFINITY ? fmaxf(m[i], top) : m[i];
        grow[i] = mn == m[i] ? 1.f : exp2_approx(m[i] - mn);
        grown = grown || mn != m[i];
        m[i] = mn;
        const float ref = mn == -INFINITY ? 0.f : -mn;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) p[y][e] = exp2_approx(fmaf(p[y][e], a.c, ref));
        l[i] = fmaf(l[i], grow[i], ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1])) +
                                       ((p[2][0] + p[2][1]) + (p[3][0] + p[3][1])));
#pragma unroll
        for (int y = 0; y < 4; ++y)
          ap[y >> 1][(y & 1) * 2 + i] = N::pack(p[y][0], p[y][1]);
      }
      // ---- O = diag(grow) O + P V
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) scale_rows<D>(acc, i, grow[i]);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {             // 16 keys
        constexpr int B = D / 16;               // 16-dim blocks: their loads go out together
        uint32_t bv[B][4];
#pragma unroll
        for (int k = 0; k < B; ++k)
          ldsm4_t(tile_addr(vbuf, kTile * 128, part * 32 + y * 16 + (lm & 1) * 8 + lr,
                            k * 2 + (lm >> 1)), bv[k]);
        if (edge) {
          uint32_t z = 0;
#pragma unroll
          for (int k = 0; k < B; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) N::probe(z, bv[k][e]);
          if (z & 0x7fff7fffu) {              // rare: a non-finite value
#pragma unroll
            for (int k = 0; k < B; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = j1 + y * 16 + (e & 1) * 8 + fc;
                uint32_t& w = bv[k][e];
                if ((w & N::kExp) == N::kExp) {
                  w &= 0xffff0000u;
                  if (j >= x.low && j < x.stop) ctl->wild = x.tag;
                }
                if (((w >> 16) & N::kExp) == N::kExp) {
                  w &= 0xffffu;
                  if (j + 1 >= x.low && j + 1 < x.stop) ctl->wild = x.tag;
                }
              }
          }
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
          N::mma(acc[k * 2], ap[y], bv[k][0], bv[k][1]);
          N::mma(acc[k * 2 + 1], ap[y], bv[k][2], bv[k][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->vempty[vs]));
    }
    if (x.tile0 < x.tile1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->qempty[qb]));
      ++nq;
    }

    // ---- join the warps that share rows: everyone's (m, l) first, then O, four rows at a time
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) ml[warp * 16 + i * 8 + fr] = make_float2(m[i], l[i]);
    }
    sync_warps(a, &ctl->meet, meets, lane, abort_flag);
    const bool wild = *reinterpret_cast<volatile int*>(&ctl->wild) == x.tag;
    constexpr int kShare = kRowTeams ? kWarps / 2 : kWarps;   // warps that share rows
    const int w0 = kRowTeams ? team * kShare : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY;
#pragma unroll 4
      for (int w = w0; w < w0 + kShare; ++w) top = fmaxf(top, ml[w * 16 + i * 8 + fr].x);
      // (a warp without a reference has nothing, or NaN: either passes unscaled)
      scale_rows<D>(acc, i, m[i] == -INFINITY ? 1.f : exp2_approx(m[i] - top));
    }
    auto join_rows = [&](int i, int half) {
      if (fr / kJoinRows == half) {
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
          *reinterpret_cast<float2*>(join + (warp * kJoinRows + (fr & 3)) * D +
                                     ((y * 8 + fc) ^ ((fr & 3) << 3))) =
              make_float2(acc[y][i * 2], acc[y][i * 2 + 1]);
      }
      sync_warps(a, &ctl->meet, meets, lane, abort_flag);
      const int id = tid - w0 * 32, d = id % (D / 2) * 2;
#pragma unroll 1
      for (int jr = id / (D / 2); jr < kJoinRows; jr += kShare * 32 / (D / 2)) {
        const int rl = i * 8 + half * kJoinRows + jr, r = row0 + rl;
        if (r >= rows) break;
        float M = -INFINITY, L = 0.f, sum[2] = {0.f, 0.f};
#pragma unroll 4
        for (int w = w0; w < w0 + kShare; ++w) M = fmaxf(M, ml[w * 16 + rl].x);
#pragma unroll 2
        for (int w = w0; w < w0 + kShare; ++w) {
          const float2 y = ml[w * 16 + rl];
          L += (y.x == -INFINITY ? 1.f : exp2_approx(y.x - M)) * y.y;
          const float2 z =
              *reinterpret_cast<const float2*>(join + (w * kJoinRows + jr) * D + (d ^ (jr << 3)));
          sum[0] += z.x;
          sum[1] += z.y;
        }
        const int tk = r / a.G, hd = x.h * a.G + r - tk * a.G;
        if (wild)
          add_lost<N, 2>(a, v_pages, x.b, x.h, x.tile0, x.tile1, x.stop, x.first, x.first + x.nt - 1,
                         x.first + tk, d, sum);
        if (x.ns == 1) {
          const int64_t row = (int64_t)(x.row + tk) * (a.Hk * a.G) + hd;
          const float inv = L == 0.f ? 0.f : 1.f / L;
          *reinterpret_cast<uint32_t*>(reinterpret_cast<T*>(o.out) + row * D + d) =
              N::pack(sum[0] * inv, sum[1] * inv);
          if (o.lse && d == 0) o.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        } else {
          const int64_t rec = (((int64_t)x.b * tp + tk) * (a.Hk * a.G) + hd) * ns_cap + x.split;
          *reinterpret_cast<float2*>(o.part + rec * D + d) = make_float2(sum[0], sum[1]);
          if (d == 0) o.part_ml[rec] = make_float2(M, L);
        }
      }
      // the buffer, and after the last rows (m, l), may change
      sync_warps(a, &ctl->meet, meets, lane, abort_flag);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll 1
      for (int half = 0; half < 2 && i * 8 + half * kJoinRows < rows; ++half) join_rows(i, half);
    }
  }
}

// Join the splits of each row, in split order: one warp to a (token, head).
template <typename T, int D>
__global__ void __launch_bounds__(128)
    k_paged_join(const __grid_constant__ Args a, const int tp, const int share, const int ns_cap, const __grid_constant__ AttnOut o) {
  pdl_wait_and_trigger();
  pdl_trigger();
  const int lane = threadIdx.x & 31, H = a.Hk * a.G;
  const uint32_t id = blockIdx.x * 4 + (threadIdx.x >> 5);   // (sequence, token, head)
  const uint32_t rest = id / (uint32_t)H;
  const int hd = (int)(id - rest * H), b = (int)(rest / (uint32_t)tp), tk = (int)(rest - b * tp);
  if (b >= a.n_seqs) return;
  const Seq s = seq_of(a, b);
  if (s.n > tp || tk >= s.n) return;
  const int ns = n_splits(max_tiles(a, s.len, tp), share);
  if (ns == 1) return;
  const int64_t row = (int64_t)(s.row0 + tk) * H + hd;
  join_row<T, D>(o.part, o.part_ml, (((int64_t)b * tp + tk) * H + hd) * ns_cap, ns,
                 reinterpret_cast<T*>(o.out) + row * D, o.lse ? o.lse + row : nullptr, lane);
}

template <typename T, int D, int WR>
cudaError_t run(const Args& a, const AttnPlan& p, const Maps& maps, const AttnOut& o,
                const void* v_pages, cudaStream_t s) {
  const size_t smem =
      Cfg<D, WR>::kCtlOff + sizeof(Ctl) + (size_t)(a.n_seqs + 1) * sizeof(int) + 1024;
  constexpr size_t most_smem =
      Cfg<D, WR>::kCtlOff + sizeof(Ctl) + (kMaxSeqs + 1) * sizeof(int) + 1024;
  static_assert(most_smem <= 227 * 1024, "attention shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(k_paged_attn<T, D, WR>), most_smem, done);
  if (err != cudaSuccess) return err;
  // no more CTAs than units there can be
  const int64_t row_tiles = (int64_t)a.T / p.tp + a.n_seqs;
  const int64_t most = row_tiles * a.Hk * p.ns_cap;
  const int nsm = sm_count();
  err = launch(k_paged_attn<T, D, WR>, dim3((unsigned)(most < nsm ? most : nsm)), kThreads, smem, s,
               a, p.tp, p.share, p.ns_cap, o, maps.k, maps.v, maps.q, v_pages);
  if (err != cudaSuccess || p.ns_cap == 1) return err;
  const int64_t rows = (int64_t)a.n_seqs * p.tp * a.Hk * a.G;
  return launch(k_paged_join<T, D>, dim3((unsigned)((rows + 3) / 4)), 128, 0, s, a, p.tp, p.share,
                p.ns_cap, o);
}

template <typename T, int D>
cudaError_t pick(const Args& a, const AttnPlan& p, const Maps& maps, const AttnOut& o,
                 const void* v_pages, cudaStream_t s) {
  return p.wr == 1 ? run<T, D, 1>(a, p, maps, o, v_pages, s)
                   : run<T, D, 2>(a, p, maps, o, v_pages, s);
}

}  // namespace

AttnPlan attn_plan(const Args& a, int max_q) {
  AttnPlan p{};
  const int64_t rows = (int64_t)max_q * a.G;
  p.wr = rows <= 16 ? 1 : 2;
  p.tp = 16 * p.wr / a.G;
  if (max_q < p.tp) p.tp = max_q;
  p.share = kSms / a.Hk < 1 ? 1 : kSms / a.Hk;
  const int64_t entries = (int64_t)a.table_ld << a.lps;
  int64_t tiles = (entries + kTile - 1) / kTile;
  if (a.window) {
    const int64_t seen = ((int64_t)a.window + p.tp - 2) / kTile + 2;
    if (seen < tiles) tiles = seen;
  }
  // at four tiles each or more, at most `share` splits or one for every eight tiles, 128 in all
  int64_t most = (tiles + 3) / 4;
  const int64_t by_share = p.share > (tiles + 7) / 8 ? p.share : (tiles + 7) / 8;
  if (by_share < most) most = by_share;
  p.ns_cap = (int)(most < 1 ? 1 : most < 128 ? most : 128);
  const size_t recs = (size_t)a.n_seqs * p.tp * a.Hk * a.G * p.ns_cap;
  p.rec_bytes = p.ns_cap == 1 ? 0 : (recs * a.D * sizeof(float) + 255) & ~(size_t)255;
  p.ml_bytes = p.ns_cap == 1 ? 0 : (recs * sizeof(float2) + 255) & ~(size_t)255;
  return p;
}

cudaError_t launch_paged_attn(const Args& a, int type, const AttnPlan& plan, const Maps& maps,
                              const AttnOut& o, const void* v_pages, cudaStream_t s) {
  if (type == PP_BF16)
    return a.D == 128 ? pick<__nv_bfloat16, 128>(a, plan, maps, o, v_pages, s)
                      : pick<__nv_bfloat16, 64>(a, plan, maps, o, v_pages, s);
  return a.D == 128 ? pick<__half, 128>(a, plan, maps, o, v_pages, s)
                    : pick<__half, 64>(a, plan, maps, o, v_pages, s);
}

}  // namespace paged
}  // namespace pp
