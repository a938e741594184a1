// k_paged_attn_tc.cu - attention of long chunks over the paged cache, on the 5th-generation
// tensor cores.  Rows, masks and results as in k_paged_attn.cu.
//
// A unit is (sequence, pair of row tiles, key head); a row tile is 128 rows, floor(128 / G)
// tokens with all G heads of the key head.  The two tiles of a pair take turns: while the tensor
// cores multiply for one, the other's softmax runs.  Units go to the SMs in waves; those of a last,
// partial wave are split over their keys and joined by k_paged_join_units (628 -> 580 us on the
// case below, whose 512 units are 3.4 waves).
//
// Measured: 4096 tokens, 32 query heads on 8 of 128 dims, over 12000 entries, bf16: 565 us, 1180
// TFLOP/s, 0.62 of the measured cuBLAS rate.  Bound by the two tiles' alternation: for each 128
// keys of both tiles the products take 2048 clocks, a softmax about 1500 from its S to its P.
//
//   S_t = Q_t K^T   M = 128 rows, N = 128 keys, operands in shared memory, S in tensor memory
//   P_t = 2^(S c - m), in the cache's type over S's own tensor-memory columns
//   O_t += P_t V    A = P from tensor memory, B = V as it lies (keys x dims, dims contiguous)
//
// Tensor memory: S0, S1 (128 columns each), O0, O1 (D columns each).
//   warp 0       producer: queries of the pair, then K and V tiles in turn, by TMA
//   warp 1       one thread issues every MMA.  Order for each tile of keys: O0 += P0 V,
//                S0 = Q0 K', O1 += P1 V, S1 = Q1 K' (K' the next keys).  A thread's MMAs run in
//                issue order, so S_t may overwrite P_t right after the product that reads it.
//                (An issuer for each tile measured 689 us against 605: the two softmaxes then
//                fall into step, and neither hides behind the other's MMAs.)
//   warps 4-7, 8-11  softmax of tile 0, 1: one thread to a row.  A row's reference m follows
//                its maximum only when it would fall behind by more than 2^8, so the sums of
//                O in tensor memory are rarely rescaled; p stays below 2^8 (2^15 in fp16),
//                and m cancels in the end.
//
// Where some row does not see some key of a tile, non-finite values of V are taken out of
// shared memory before the product (zero times infinity would be NaN) and added to the rows
// that do see the key at the end.
#include <type_traits>

#include "pp_paged.cuh"
#include "pp_tcgen05.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kThreads = 384;
constexpr int kRowsT = 128;          // rows of a row tile
constexpr int kMaxParts = 304;       // split units of a call, at most: two to an SM
constexpr int kMostParts = 16;       // parts of one unit
constexpr int kUnitRows = 2 * kRowsT;
constexpr float kLag = 8.f;          // a row's maximum may exceed its reference by this (log2)
// registers a thread: launched with 168; the softmax warps take what the others give up
// (80 + 2 x 208 = 496 <= 3 x 168 for each three threads)
constexpr int kRegsFew = 80, kRegsMany = 208;

template <int D>
struct Cfg {
  static constexpr int kSlots = D == 128 ? 4 : 8;   // K and V tiles
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQBytes = kRowsT * D * 2;    // one row tile
  static constexpr int kQOff = kSlots * kTileBytes;
  static constexpr int kCtlOff = kQOff + 2 * kQBytes;
};

struct Ctl {
  UnitRing ring;
  uint64_t full[8], empty[8];
  uint64_t qfull, qempty, sfull[2], pfull[2], ofull[2], done;
  uint64_t clean[2][2];   // [group][edge tile & 1]: the group's half of V is clean
  uint32_t bad[8];
  uint32_t tmem;
  // tag of the unit in which a softmax group took a non-finite value out of V.  The ring keeps a
  // group at most kUnits units ahead of the other.
  int wild[2][2 * kUnits];
  int abort;
};

// Units before any split: (pair of row tiles, key head).
__device__ __forceinline__ int seq_units(const Args& a, int b, int tp) {
  const Seq s = seq_of(a, b);
  if (s.n > 0) check_len(a, s);
  return a.Hk * ((s.n + 2 * tp - 1) / (2 * tp));
}

// The units run in waves of one to an SM.  Those of the last wave, if it is not full, are split
// over their keys, each in `parts`, so that its end comes sooner: of `units`, the first `whole`
// stay in one piece.  `room` parts have a place in scratch: never too few, unless row offsets
// that fall make more units than T rows can have.
struct Waves {
  int units, whole, parts;
};
__device__ __forceinline__ Waves waves_of(int units, int most_parts, int room) {
  Waves w;
  w.units = units;
  const int rest = units % (int)gridDim.x;
  w.whole = units - rest;
  // time of the last wave in 1/64 of a unit's, 4 of them for each part's start and join: a lane to
  // each number of parts (a loop over them took 1.8 us), the fewest of the fastest win
  const int p = (int)(threadIdx.x & 31) + 1, grid = (int)gridDim.x;
  const bool may = p > 1 && p <= most_parts && rest > 0 && rest * p <= room;
  const int time = may ? (rest * p + grid - 1) / grid * (64 / p + 4) : p == 1 ? 64 : 1 << 20;
  w.parts = (int)(__reduce_min_sync(0xffffffffu, (unsigned)(time * 64 + p)) & 63u);
  if (w.parts == 1) w.whole = units;
  return w;
}

// A split has at least four tiles of keys: the last ones of a short sequence may have none.
__device__ __forceinline__ Unit unit_of(const Args& a, const int* pre, const Waves& w, int u,
                                        int tp) {
  Unit x;
  x.tag = u + 1;
  int slot = 0, part = 0;
  x.ns = 1;
  if (u >= w.whole) {
    slot = (u - w.whole) / w.parts;
    part = u - w.whole - slot * w.parts;
    x.ns = w.parts;
    u = w.whole + slot;
  }
  x.split = slot * kMostParts + part;
  x.b = find_seq(pre, a.n_seqs, u);
  const Seq s = seq_of(a, x.b);
  u -= pre[x.b];
  // the last pairs, whose rows see most, come first; heads vary fastest
  const int p = (s.n + 2 * tp - 1) / (2 * tp) - 1 - u / a.Hk;
  x.h = u % a.Hk;
  const int t0 = p * 2 * tp;
  x.row = s.row0 + t0;
  x.nt = min(2 * tp, s.n - t0);
  x.first = s.total - s.n + t0;
  x.stop = min(max(x.first + x.nt, 0), s.len);
  x.low = a.window ? min(max(x.first - a.window + 1, 0), x.stop) : 0;
  const int ta = x.low / kTile, tb = (x.stop + kTile - 1) / kTile;
  const int st = max((tb - ta + x.ns - 1) / x.ns, x.ns > 1 ? 4 : 0);
  x.tile0 = min(ta + part * st, tb);
  x.tile1 = min(x.tile0 + st, tb);
  return x;
}

// One MMA.  Descriptors come as lower words: the issuing thread is alone on its scheduler slot
// and every instruction between two MMAs counts.  `acc` false: D = A B, else D += A B.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                        bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %4};\n"
      " mov.b64 b, {%2, %4};\n tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"((uint32_t)acc));
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                        bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"((uint32_t)acc));
}

// 32 columns of this thread's tensor-memory lane
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Zeroes the non-finite halves of w; true if there were any.
template <typename N>
__device__ __forceinline__ bool finite_only(uint32_t& w) {
  uint32_t keep = 0xffffffffu;
  if ((w & N::kExp) == N::kExp) keep &= 0xffff0000u;
  if (((w >> 16) & N::kExp) == N::kExp) keep &= 0xffffu;
  w &= keep;
  return keep != 0xffffffffu;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attn_tc(const __grid_constant__ Args a, const int tp, const int most_parts,
                    const int room,
                    const __grid_constant__ AttnOut o,
                    const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapV,
                    const __grid_constant__ CUtensorMap mapQ, const void* v_pages) {
  using C = Cfg<D>;
  using N = Num<T>;
  constexpr int kSlots = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler then knows that it is shared memory)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kCtlOff);
  int* pre = reinterpret_cast<int*>(ctl + 1);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), i == 1 ? 1 + a.withhold : 1);   // (1: the first V)
      mbar_init(smem_u32(&ctl->empty[i]), 1);
    }
    mbar_init(smem_u32(&ctl->qfull), 1);
    mbar_init(smem_u32(&ctl->qempty), 1);
    mbar_init(smem_u32(&ctl->done), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&ctl->sfull[t]), 1);
      mbar_init(smem_u32(&ctl->pfull[t]), 4);
      mbar_init(smem_u32(&ctl->ofull[t]), 1);
      for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ctl->clean[t][i]), 4);
      for (int i = 0; i < 2 * kUnits; ++i) ctl->wild[t][i] = 0;
    }
    ring_init(ctl->ring, 9);            // the MMA issuer, eight softmax warps
    ctl->abort = 0;
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
  prefix_units(a, pre, [&](int b) { return seq_units(a, b, tp); });
  const Waves waves = waves_of(pre[a.n_seqs], most_parts, room);
  // what the join needs to find its rows: the waves and the sequences' units
  if (blockIdx.x == 0 && most_parts > 1) {
    if (threadIdx.x == 0) {
      o.plan[0] = waves.units;
      o.plan[1] = waves.whole;
      o.plan[2] = waves.parts;
    }
    for (int b = threadIdx.x; b <= a.n_seqs; b += kThreads) o.plan[4 + b] = pre[b];
  }
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = ctl->tmem;
  const int units = waves.whole + (waves.units - waves.whole) * waves.parts;
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_phase(a, bar, parity, abort_flag); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      // ---- producer -----------------------------------------------------------------------
      uint32_t nq = 0, nl = 0, nu = 0, seen_bad = 0;
#pragma unroll 1
      for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x) {
        const Unit x = unit_of(a, pre, waves, u, tp);
        put_unit(a, ctl->ring, nu++, x, lane, abort_flag);
        if (x.tile0 == x.tile1) continue;
        const int tiles = x.nt > tp ? 2 : 1;
        if (nq > 0) wait(&ctl->qempty, (nq - 1) & 1);
        if (*abort_flag) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&ctl->qfull);
          mbar_expect_tx(bar, (uint32_t)(tiles * tp * a.G * D * 2));
          for (int t = 0; t < tiles; ++t)
            for (int bx = 0; bx < D / 64; ++bx)
              tma_load_4d(smem_u32(smem + C::kQOff + t * C::kQBytes + bx * kRowsT * 128), &mapQ,
                          bx * 64, x.h * a.G, x.row + t * tp, 0, bar);
        }
        ++nq;
        const bool past = x.first + x.nt > x.stop;
        TilePages now{}, next = find_pages(a, x.b, x.tile0 * kTile, x.stop, past, lane);
#pragma unroll 1
        for (int i = 0; i < 2 * (x.tile1 - x.tile0); ++i) {
          const int slot = nl % kSlots, t = x.tile0 + (i >> 1);
          if ((i & 1) == 0) {
            now = next;
            if (t + 1 < x.tile1) next = find_pages(a, x.b, (t + 1) * kTile, x.stop, past, lane);
            seen_bad |= now.bad;
          }
          if (nl >= kSlots) wait(&ctl->empty[slot], (nl / kSlots - 1) & 1);
          if (*abort_flag) break;
          load_key_tile(a, (i & 1) ? &mapV : &mapK, smem_u32(smem + slot * C::kTileBytes),
                        smem_u32(&ctl->full[slot]), now, x.h, t * kTile, lane, &ctl->bad[slot]);
          ++nl;
        }
      }
      Unit none{};
      none.b = -1;
      put_unit(a, ctl->ring, nu, none, lane, abort_flag);
      if (seen_bad && lane == 0) raise(a, PP_S_INDEX);
      // every copy lands before the CTA may exit (bounded waits)
      if (lane == 0) {
        if (nq > 0) drain_phase(a, &ctl->qfull, (nq - 1) & 1);
#pragma unroll 1
        for (uint32_t i = nl > kSlots ? nl - kSlots : 0; i < nl; ++i)
          drain_phase(a, &ctl->full[i % kSlots], (i / kSlots) & 1);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---- MMA issuer ---------------------------------------------------------------------
      // The tensor pipe takes little ahead of time, so a wait between two MMAs leaves it idle, a
      // completed one too (about 100 clocks).  So the next barrier is tested while two MMAs are
      // still to be issued, and V is waited for by the softmax threads, before they hand over P.
      // (Handing P over in two halves, for an earlier start, cost more in waits than it gave:
      // 644 us against 605.)
      if (lane == 0) {
        constexpr uint32_t id = (1u << 4) | N::kMmaTypes | ((uint32_t)(kRowsT >> 4) << 24);
        constexpr uint32_t id_s = id | ((uint32_t)(kTile >> 3) << 17);
        constexpr uint32_t id_o = id | ((uint32_t)(D >> 3) << 17) | (1u << 16);   // B = V by keys
        // lower descriptor words: the tiles' addresses in units of 16 bytes (below 2^14), and
        // for V the distance of its 64-dim boxes
        const uint32_t t_lo = smem_u32(smem) >> 4, q_lo = smem_u32(smem + C::kQOff) >> 4;
        const uint32_t v_lo = t_lo | ((uint32_t)(kTile * 128 >> 4) << 16);
        uint32_t nq = 0, nl = 0, np[2] = {0, 0};
        constexpr int kS = D / 16, kP = kTile / 16;   // MMAs of one S, of one P V
        auto scores = [&](int t, uint32_t slot, int from, int to) {
          const uint32_t q = q_lo + t * (C::kQBytes >> 4), k = t_lo + slot * (C::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kS; ++kk) {
            if (kk < from || kk >= to) continue;
            const uint32_t off = ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
            umma_ss(tmem + t * kTile, q + off, k + off, id_s, kk > 0);
          }
        };
        auto values = [&](int t, uint32_t slot, int from, int to, bool acc) {
          const uint32_t v = v_lo + slot * (C::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kP; ++kk) {
            if (kk < from || kk >= to) continue;
            umma_ts(tmem + 2 * kTile + t * D, tmem + t * kTile + kk * 8, v + kk * (2048 >> 4), id_o,
                    acc || kk > 0);
          }
        };
        Unit x;
#pragma unroll 1
        for (uint32_t nu = 0; get_unit(a, ctl->ring, nu, x, lane, true, abort_flag); ++nu) {
          const int nt = x.tile1 - x.tile0;
          if (nt == 0) continue;
          const int tiles = x.nt > tp ? 2 : 1;
          wait(&ctl->qfull, nq & 1);
          ++nq;
          wait(&ctl->full[nl % kSlots], (nl / kSlots) & 1);
          if (*abort_flag) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          for (int t = 0; t < tiles; ++t) {
            scores(t, nl % kSlots, 0, kS);
            umma_commit(smem_u32(&ctl->sfull[t]));
          }
          umma_commit(smem_u32(&ctl->empty[nl % kSlots]));
          if (nt == 1) umma_commit(smem_u32(&ctl->qempty));
          ++nl;
          bool ready = false;                          // the next P has been seen
#pragma unroll 1
          for (int j = 0; j < nt; ++j) {
            const uint32_t sv = nl % kSlots, sk = (nl + 1) % kSlots, kp = ((nl + 1) / kSlots) & 1;
            const bool more = j + 1 < nt;
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
              if (!ready) wait(&ctl->pfull[t], np[t] & 1);
              ++np[t];
              const int next = t + 1 < tiles ? t + 1 : 0;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              if (more) {
                values(t, sv, 0, kP - 2, j > 0);
                const bool k_in = t > 0 || mbar_test(smem_u32(&ctl->full[sk]), kp);
                values(t, sv, kP - 2, kP, true);
                if (!k_in) wait(&ctl->full[sk], kp);
                scores(t, sk, 0, kS - 2);
                ready = mbar_test(smem_u32(&ctl->pfull[next]), np[next] & 1);
                scores(t, sk, kS - 2, kS);
                umma_commit(smem_u32(&ctl->sfull[t]));
              } else {
                values(t, sv, 0, kP - 2, j > 0);
                ready = next != 0 && mbar_test(smem_u32(&ctl->pfull[next]), np[next] & 1);
                values(t, sv, kP - 2, kP, true);
                umma_commit(smem_u32(&ctl->ofull[t]));
              }
            }
            if (*abort_flag) break;
            umma_commit(smem_u32(&ctl->empty[sv]));
            if (more) {
              umma_commit(smem_u32(&ctl->empty[sk]));
              if (j + 2 == nt) umma_commit(smem_u32(&ctl->qempty));
              nl += 2;
            } else {
              nl += 1;
            }
          }
        }
        // every MMA is done before tensor memory is given back (bounded wait)
        umma_commit(smem_u32(&ctl->done));
        drain_phase(a, &ctl->done, 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    // ---- softmax: thread r of the group owns row r of its tile -------------------------------
    const int t = (warp - 4) >> 2;
    const int r = threadIdx.x - 128 - t * 128;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_base + t * kTile, o_at = lane_base + 2 * kTile + t * D;
    const uint64_t c2 = f32x2(a.c, a.c);
    uint32_t ns_ = 0, no = 0, nl = 0, ne = 0, nu = 0;
    Unit x;
#pragma unroll 1
    for (; get_unit(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
      const int nt = x.tile1 - x.tile0;
      const int tiles = x.nt > tp ? 2 : 1;
      if (t >= tiles) {        // a pair of one tile: nothing to do here but count
        nl += 2 * nt;
        continue;
      }
      const int first = x.first;
      const int tokens = min(tp, x.nt - t * tp);
      const int tk = min(r / a.G, tokens - 1);
      const int pos = first + t * tp + tk;
      const bool live = r < tokens * a.G;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        const int j0 = (x.tile0 + j) * kTile;
        // does some row of the pair not see some key?
        const int last = first + x.nt - 1;
        const uint32_t vslot = (nl + 2 * j + 1) % kSlots;
        // S first: it comes after everything that earlier units loaded, so the phase of V's slot
        // can then be no earlier one, although this group may have passed over whole units
        wait(&ctl->sfull[t], ns_ & 1);
        ++ns_;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        wait(&ctl->full[vslot], ((nl + 2 * j + 1) / kSlots) & 1);
        const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&ctl->bad[vslot]);
        const bool edge = bad || j0 + kTile - 1 > first || (a.window && j0 <= last - a.window);
        if (edge) {
          // take non-finite values out of V (this group's rows of the tile)
          const int share = kTile / tiles;
          uint8_t* vt = smem + vslot * C::kTileBytes;
          bool found = false, any = false;
          auto chunk = [&](int i) {       // 16 bytes of the tile
            const int row = t * share + i / (D / 8), ch = i % (D / 8);
            return reinterpret_cast<uint4*>(vt + (ch >> 3) * (kTile * 128) + row * 128 +
                                            (((ch & 7) ^ (row & 7)) << 4));
          };
          // four at a time, as the share is a multiple of them; looked at closer only if need be
#pragma unroll 1
          for (int i0 = r; i0 < share * (D / 8); i0 += 4 * 128) {
            uint4 w[4];
            uint32_t z = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = *chunk(i0 + k * 128);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              N::probe(z, w[k].x);
              N::probe(z, w[k].y);
              N::probe(z, w[k].z);
              N::probe(z, w[k].w);
            }
            if ((z & 0x7fff7fffu) == 0) continue;
            any = true;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              const int i = i0 + k * 128, row = t * share + i / (D / 8);
              uint4 y = *chunk(i);
              const bool hit = finite_only<N>(y.x) | finite_only<N>(y.y) | finite_only<N>(y.z) |
                               finite_only<N>(y.w);
              if (hit) {
                *chunk(i) = y;
                found = found || (j0 + row >= x.low && j0 + row < x.stop);
              }
            }
          }
          if (found) ctl->wild[t][nu % (2 * kUnits)] = x.tag;
          if (any) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          if (tiles == 2) {    // both halves, before either product
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->clean[t][ne & 1]));
            wait(&ctl->clean[t ^ 1][ne & 1], (ne >> 1) & 1);
            ++ne;
          }
        }
        auto weights = [&](auto masked) {
          uint32_t s[kTile];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_at + i * 32, s + i * 32);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kTile; ++i) asm volatile("" : "+r"(s[i]));
          if constexpr (decltype(masked)::value) {
            // keys (pos - window, pos], as places in this tile; 32 at a time, for few of which
            // some row of the warp does not see all
            const int hi = pos - j0, lo = a.window ? hi - a.window : -1;
#pragma unroll
            for (int c = 0; c < kTile / 32; ++c) {
              const int h = hi - c * 32, b = lo - c * 32;
              uint32_t see = h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1u;
              if (b >= 0) see &= b >= 31 ? 0u : ~((2u << b) - 1u);
              if ((bad >> (2 * c)) & 1u) see &= 0xffff0000u;
              if ((bad >> (2 * c + 1)) & 1u) see &= 0xffffu;
              if (__any_sync(0xffffffffu, see != ~0u)) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!((see >> i) & 1u)) s[c * 32 + i] = 0xff800000u;
              }
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kTile; i += 2)
            m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], __uint_as_float(s[i]),
                                    __uint_as_float(s[i + 1]));
          const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
          const float want = mx * a.c - N::kShift;
          if (j == 0) {
            m = mx == -INFINITY ? -INFINITY : want;
          } else if (__any_sync(0xffffffffu, want > m + kLag)) {
            // O = O 2^(old - new), row by row; the product that O holds is done, since S was
            // issued after it
            const float mn = want > m + kLag ? want : m;
            const float f = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
            l *= f;
            m = mn;
#pragma unroll 1
            for (int i = 0; i < D / 8; ++i) {
              uint32_t w[8];
              tmem_ld8(o_at + i * 8, w);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(after_wait(w[e]) * f);
              tmem_st8(o_at + i * 8, w);
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t r2 = f32x2(-ref, -ref);
          uint64_t sum2[2] = {f32x2(l, 0.f), 0};
          uint32_t p[kTile / 2];
#pragma unroll
          for (int i = 0; i < kTile; i += 2) {
            const uint64_t z = fma2((uint64_t)s[i] | ((uint64_t)s[i + 1] << 32), c2, r2);
            const float p0 = exp2_approx(lo_of(z)), p1 = exp2_approx(hi_of(z));
            sum2[(i >> 1) & 1] = add2(sum2[(i >> 1) & 1], f32x2(p0, p1));
            p[i >> 1] = N::pack(p0, p1);
          }
          tmem_st32(s_at, p);
          tmem_st32(s_at + 32, p + 32);
          tmem_wait_st();
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->pfull[t]));
          const uint64_t both = add2(sum2[0], sum2[1]);
          l = lo_of(both) + hi_of(both);
        };
        if (edge)
          weights(std::true_type());
        else
          weights(std::false_type());
      }
      nl += 2 * nt;

      // ---- the rows' results, or the split's partials --------------------------------------
      const int H = a.Hk * a.G;
      const int token = x.row + t * tp + tk, hd = x.h * a.G + r - tk * a.G;
      const int64_t row = (int64_t)token * H + hd;
      const int slot = x.split / kMostParts, part = x.split % kMostParts;
      const int64_t rec = ((int64_t)slot * kUnitRows + t * kRowsT + r) * x.ns + part;
      const bool whole = x.ns == 1;
      bool wild = false;
      if (nt > 0) {
        wait(&ctl->ofull[t], no & 1);
        ++no;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        wild = *reinterpret_cast<volatile int*>(&ctl->wild[0][nu % (2 * kUnits)]) == x.tag ||
               *reinterpret_cast<volatile int*>(&ctl->wild[1][nu % (2 * kUnits)]) == x.tag;
      }
      const float f = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t w[32];
        if (nt > 0) {
          tmem_ld32(o_at + i * 32, w);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) asm volatile("" : "+r"(w[e]));
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = 0;
        }
        if (wild && live) {
          // rare (their weights are positive)
          float add[32] = {};
          add_lost<N, 32>(a, v_pages, x.b, x.h, x.tile0, x.tile1, x.stop, first, first + x.nt - 1,
                          pos, i * 32, add);
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) + add[e]);
        }
        if (live) {
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(o.out) + row * D + i * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[k] = N::pack(__uint_as_float(w[e * 8 + k * 2]) * f,
                               __uint_as_float(w[e * 8 + k * 2 + 1]) * f);
              dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (nt > 0) {
            uint4* dst = reinterpret_cast<uint4*>(o.part + rec * D + i * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_uint4(w[e * 4], w[e * 4 + 1], w[e * 4 + 2], w[e * 4 + 3]);
          }
        }
      }
      if (live) {
        if (!whole)
          o.part_ml[rec] = make_float2(m, l);
        else if (o.lse)
          o.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      // the next unit's products into O come after this group's next P
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// Join the parts of each split unit's rows: one warp to a row.
template <typename T, int D>
__global__ void __launch_bounds__(128)
    k_paged_join_units(const __grid_constant__ Args a, const int tp,
                       const __grid_constant__ AttnOut o) {
  pdl_wait_and_trigger();
  pdl_trigger();
  const int lane = threadIdx.x & 31, H = a.Hk * a.G;
  const int id = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int slot = id / kUnitRows, at = id - slot * kUnitRows;   // unit, row of its two tiles
  const int t = at / kRowsT, r = at - t * kRowsT;
  const int whole = o.plan[1], u = whole + slot, ns = o.plan[2];
  if (u >= o.plan[0] || r >= tp * a.G) return;
  const int* pre = o.plan + 4;
  const int b = find_seq(pre, a.n_seqs, u);
  const Seq s = seq_of(a, b);
  const int k = u - pre[b];
  const int p = (s.n + 2 * tp - 1) / (2 * tp) - 1 - k / a.Hk;
  const int tk = r / a.G, token = p * 2 * tp + t * tp + tk;
  if (token >= s.n) return;
  const int64_t row = (int64_t)(s.row0 + token) * H + k % a.Hk * a.G + r - tk * a.G;
  join_row<T, D>(o.part, o.part_ml, (int64_t)id * ns, ns, reinterpret_cast<T*>(o.out) + row * D,
                 o.lse ? o.lse + row : nullptr, lane);
}

template <typename T, int D>
cudaError_t run(const Args& a, const LongPlan& p, const Maps& maps, const AttnOut& o,
                const void* v_pages, cudaStream_t s) {
  const size_t smem = Cfg<D>::kCtlOff + sizeof(Ctl) + (size_t)(a.n_seqs + 1) * sizeof(int) + 1024;
  constexpr size_t most_smem = Cfg<D>::kCtlOff + sizeof(Ctl) + (kMaxSeqs + 1) * sizeof(int) + 1024;
  static_assert(most_smem <= 227 * 1024, "long-chunk attention shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(k_paged_attn_tc<T, D>), most_smem, done);
  if (err != cudaSuccess) return err;
  const int64_t most = p.units * p.parts;
  const int nsm = sm_count();
  err = launch(k_paged_attn_tc<T, D>, dim3((unsigned)(most < nsm ? most : nsm)), kThreads, smem, s,
               a, p.tp, p.parts, p.room, o, maps.k, maps.v, maps.q, v_pages);
  if (err != cudaSuccess || p.parts == 1) return err;
  const int64_t split = p.units < nsm ? p.units : nsm;   // units of the last wave, at most
  return launch(k_paged_join_units<T, D>, dim3((unsigned)(split * kUnitRows / 4)), 128, 0, s, a,
                p.tp, o);
}

}  // namespace

LongPlan long_plan(const Args& a, int T) {
  LongPlan p{};
  p.tp = kRowsT / a.G;
  p.units = ((int64_t)T / (2 * p.tp) + a.n_seqs) * a.Hk;
  const int64_t parts = (((int64_t)a.table_ld << a.lps) + 4 * kTile - 1) / (4 * kTile);
  p.parts = parts < 1 ? 1 : parts > kMostParts ? kMostParts : (int)parts;
  p.room = p.units * p.parts < kMaxParts ? (int)(p.units * p.parts) : kMaxParts;
  const size_t recs = p.parts == 1 ? 0 : (size_t)p.room * kUnitRows;
  p.rec_bytes = recs * a.D * sizeof(float);
  p.ml_bytes = recs * sizeof(float2);
  p.plan_bytes = (size_t)(a.n_seqs + 5) * sizeof(int);
  return p;
}

cudaError_t launch_paged_attn_tc(const Args& a, int type, const LongPlan& plan, const Maps& maps,
                                 const AttnOut& o, const void* v_pages, cudaStream_t s) {
  if (type == PP_BF16)
    return a.D == 128 ? run<__nv_bfloat16, 128>(a, plan, maps, o, v_pages, s)
                      : run<__nv_bfloat16, 64>(a, plan, maps, o, v_pages, s);
  return a.D == 128 ? run<__half, 128>(a, plan, maps, o, v_pages, s)
                    : run<__half, 64>(a, plan, maps, o, v_pages, s);
}

}  // namespace paged
}  // namespace pp
