// k_paged_attn.cu - attention of a chunk of new tokens over the paged cache.
//
// For row (t, g) of a sequence (new token t of n, query head g of a key head's G), with L
// cache entries, the new ones included and last:
//   p(t) = L - n + t;  keys j in (p - window, p] (or [0, p]);
//   out = sum_j exp(s_j - lse) V_j,  s_j = scale q . K_j,  lse = log sum_j exp(s_j).
// One pass over the keys with a running maximum m and sum l, in powers of two.
//
// A work unit is (sequence, row tile, key head, split of its keys): up to 16 * WR rows (whole
// tokens with all their G heads, so a key is read once for all of them) against a run of
// 128-key tiles.  CTAs walk the units with one stride; a sequence's splits depend on its own
// lengths only, so its bits do not depend on the rest of the batch.
//
//   warp 8      producer: query rows, K and V tiles by TMA, one box to a lane;
//   warps 0-7   S: warp w takes keys 16w .. 16w+15 of the tile and every row; row maxima
//               meet in shared memory; P = 2^(s - m) goes to shared memory in the cache's
//               type; O: warp w takes D/8 of the dims, all keys, all rows - so no output is
//               ever added up across warps.
//
// A unit that is not its rows' only one leaves (m, l, O) in fp32 in scratch and
// k_paged_join adds the splits up in split order.
//
// Keys that some row of a tile may not see need care in the second product, where a
// weight of zero times a stored infinity would be NaN: on such tiles every non-finite
// value of V is taken out of the product and its infinities and NaNs are added to just
// the rows that see the key.
#include "pp_paged.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32 + 32;
constexpr int kQBufs = 2;

template <int D, int WR>
struct Cfg {
  static constexpr int R = 16 * WR;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int KS = D == 128 ? 3 : 5;
  static constexpr int VS = D == 128 ? (WR == 4 ? 2 : 3) : 5;
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kPBytes = R * kTile * 2;
  static constexpr int kVOff = KS * kTileBytes;
  static constexpr int kQOff = kVOff + VS * kTileBytes;
  static constexpr int kPOff = kQOff + kQBufs * kQBytes;
  static constexpr int kRedOff = kPOff + kPBytes;           // [R][8] floats
  static constexpr int kSumOff = kRedOff + R * 8 * 4;        // [R][8] floats
  static constexpr int kCtlOff = kSumOff + R * 8 * 4;
};

struct Ctl {
  uint64_t kfull[8], kempty[8], vfull[8], vempty[8], qfull[kQBufs], qempty[kQBufs];
  uint32_t bad[8];
  int abort;
};

struct Unit {
  int b, h, split, ns;
  int row0, n, len;      // of the sequence
  int t0, nt;            // first token of the row tile, its tokens
  int tile0, tile1;      // key tiles of the split
  int end;               // entries the last row sees end here
};

// Key tiles that a row tile of up to tp tokens can touch, at most.
__device__ __forceinline__ int max_tiles(const Args& a, int len, int tp) {
  const int all = (len + kTile - 1) / kTile;
  return a.window ? min(all, (int)(((int64_t)a.window + tp - 2) / kTile) + 2) : all;
}
// Tiles of one split.  Only chunks of a single row tile are split: longer ones have work
// for many CTAs already.  At most 128 splits; a split is long enough that writing its
// partial (rows x D floats) stays small beside reading its keys.
__host__ __device__ __forceinline__ int split_tiles(int tiles, int wr) {
  const int least = 2 * wr, even = (tiles + 127) / 128;
  return least > even ? least : even;
}
__host__ __device__ __forceinline__ int n_splits(int tiles, int wr) {
  const int st = split_tiles(tiles, wr);
  return tiles <= st ? 1 : (tiles + st - 1) / st;
}

template <int WR>
__device__ __forceinline__ int seq_units(const Args& a, int b, int tp) {
  const Seq s = seq_of(a, b);
  if (s.n == 0) return 0;
  const int rt = (s.n + tp - 1) / tp;
  return a.Hk * (rt > 1 ? rt : n_splits(max_tiles(a, s.len, tp), WR));
}

template <int WR>
__device__ __forceinline__ Unit unit_of(const Args& a, const int* pre, int u, int tp) {
  Unit x;
  x.b = find_seq(pre, a.n_seqs, u);
  const Seq s = seq_of(a, x.b);
  u -= pre[x.b];
  const int rt = (s.n + tp - 1) / tp;
  const int mt = max_tiles(a, s.len, tp);
  x.ns = rt > 1 ? 1 : n_splits(mt, WR);
  const int per = rt > 1 ? rt : x.ns;   // units of one key head
  x.h = u / per;
  const int i = u - x.h * per;
  x.split = rt > 1 ? 0 : i;
  x.t0 = rt > 1 ? i * tp : 0;
  x.nt = min(tp, s.n - x.t0);
  x.row0 = s.row0;
  x.n = s.n;
  x.len = s.len;
  const int first = s.len - s.n + x.t0;            // index of the tile's first token
  x.end = max(first + x.nt, 0);
  const int lo = a.window ? max(first - a.window + 1, 0) : 0;
  const int ta = min(lo, x.end) / kTile, tb = (x.end + kTile - 1) / kTile;
  const int st = rt > 1 ? tb - ta : split_tiles(mt, WR);
  x.tile0 = min(ta + x.split * st, tb);
  x.tile1 = min(x.tile0 + st, tb);
  return x;
}

template <typename T, int D, int WR>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attn(const Args a, const int tp, const int ns_cap, const AttnOut o,
                 const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                 const __grid_constant__ CUtensorMap mapQ) {
  using C = Cfg<D, WR>;
  using N = Num<T>;
  constexpr int R = C::R, DC = D / 8;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kCtlOff);
  int* pre = reinterpret_cast<int*>(ctl + 1);
  float* red = reinterpret_cast<float*>(smem + C::kRedOff);
  float* sums = reinterpret_cast<float*>(smem + C::kSumOff);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&ctl->kfull[i]), 1);
      mbar_init(smem_u32(&ctl->kempty[i]), kWarps);
      mbar_init(smem_u32(&ctl->vfull[i]), 1);
      mbar_init(smem_u32(&ctl->vempty[i]), kWarps);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(smem_u32(&ctl->qfull[i]), 1);
      mbar_init(smem_u32(&ctl->qempty[i]), kWarps);
    }
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait_and_trigger();
  pdl_trigger();
  prefix_units(pre, a.n_seqs, [&](int b) { return seq_units<WR>(a, b, tp); });
  const int units = pre[a.n_seqs];
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_phase(a, bar, parity, abort_flag); };

  if (warp == kWarps) {
    // ---- producer -------------------------------------------------------------------------
    uint32_t nq = 0, nk = 0, nv = 0;
    uint32_t seen_bad = 0;
    for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x) {
      const Unit x = unit_of<WR>(a, pre, u, tp);
      if (x.tile0 == x.tile1) continue;
      const int qb = nq % kQBufs;
      if (nq >= kQBufs) wait(&ctl->qempty[qb], (nq / kQBufs - 1) & 1);
      if (*abort_flag) break;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&ctl->qfull[qb]);
        const uint32_t dst = smem_u32(smem + C::kQOff + qb * C::kQBytes);
        // rows past the row tile's tokens may be another sequence's: their results go nowhere
        mbar_expect_tx(bar, (uint32_t)(tp * a.G * D * 2));
        for (int bx = 0; bx < D / 64; ++bx)
          tma_load_4d(dst + bx * (R * 128), &mapQ, bx * 64, x.h * a.G, x.row0 + x.t0, 0, bar);
      }
      ++nq;
      for (int t = x.tile0; t < x.tile1; ++t) {
        const int ks = nk % C::KS, vs = nv % C::VS;
        if (nk >= C::KS) wait(&ctl->kempty[ks], (nk / C::KS - 1) & 1);
        if (*abort_flag) break;
        const uint32_t bad =
            load_key_tile(a, &mapK, smem_u32(smem + ks * C::kTileBytes),
                          smem_u32(&ctl->kfull[ks]), x.b, x.h, t * kTile, x.end, lane, nullptr);
        seen_bad |= bad;
        ++nk;
        if (nv >= C::VS) wait(&ctl->vempty[vs], (nv / C::VS - 1) & 1);
        if (*abort_flag) break;
        load_key_tile(a, &mapV, smem_u32(smem + C::kVOff + vs * C::kTileBytes),
                      smem_u32(&ctl->vfull[vs]), x.b, x.h, t * kTile, x.end, lane, &ctl->bad[vs]);
        ++nv;
      }
    }
    if (seen_bad && lane == 0) raise(a, PP_S_INDEX);
    // every copy lands before the CTA may exit (bounded waits)
    if (lane == 0) {
      for (uint32_t i = nq > kQBufs ? nq - kQBufs : 0; i < nq; ++i)
        mbar_wait(smem_u32(&ctl->qfull[i % kQBufs]), (i / kQBufs) & 1);
      for (uint32_t i = nk > C::KS ? nk - C::KS : 0; i < nk; ++i)
        mbar_wait(smem_u32(&ctl->kfull[i % C::KS]), (i / C::KS) & 1);
      for (uint32_t i = nv > C::VS ? nv - C::VS : 0; i < nv; ++i)
        mbar_wait(smem_u32(&ctl->vfull[i % C::VS]), (i / C::VS) & 1);
    }
    return;
  }

  // ---- consumers ----------------------------------------------------------------------------
  const int lm = lane >> 3, lr = lane & 7;      // ldmatrix: matrix and row of this lane
  const int fr = lane >> 2, fc = (lane & 3) * 2;   // fragment row and column pair
  const uint32_t pbuf = smem_u32(smem + C::kPOff);
  uint32_t nq = 0, nk = 0, nv = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit x = unit_of<WR>(a, pre, u, tp);
    const int first = x.len - x.n + x.t0;
    const int rows = x.nt * a.G;
    int pos[2 * WR];
#pragma unroll
    for (int i = 0; i < 2 * WR; ++i)
      pos[i] = first + min((i * 8 + fr) / a.G, x.nt - 1);
    float m[2 * WR], l[2 * WR], acc[WR][D / 64][4];
#pragma unroll
    for (int i = 0; i < 2 * WR; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < WR; ++i)
#pragma unroll
      for (int n = 0; n < D / 64; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;

    const int qb = nq % kQBufs;
    const uint32_t qbuf = smem_u32(smem + C::kQOff + qb * C::kQBytes);
    if (x.tile0 < x.tile1) wait(&ctl->qfull[qb], (nq / kQBufs) & 1);
    for (int t = x.tile0; t < x.tile1; ++t) {
      const int j0 = t * kTile;
      // ---- S = Q K^T: this warp's 16 keys, every row
      const int ks = nk % C::KS;
      const uint32_t kbuf = smem_u32(smem + ks * C::kTileBytes);
      wait(&ctl->kfull[ks], (nk / C::KS) & 1);
      float s[WR][2][4];
#pragma unroll
      for (int i = 0; i < WR; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t bk[4];
        ldsm4(tile_addr(kbuf, kTile * 128, warp * 16 + (lm >> 1) * 8 + lr, kk * 2 + (lm & 1)), bk);
#pragma unroll
        for (int i = 0; i < WR; ++i) {
          uint32_t aq[4];
          ldsm4(tile_addr(qbuf, R * 128, i * 16 + (lm & 1) * 8 + lr, kk * 2 + (lm >> 1)), aq);
          N::mma(s[i][0], aq, bk[0], bk[1]);
          N::mma(s[i][1], aq, bk[2], bk[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->kempty[ks]));
      ++nk;
      // which parts of the tile have no page comes with its V tile
      const int vs = nv % C::VS;
      const uint32_t vbuf = smem_u32(smem + C::kVOff + vs * C::kTileBytes);
      wait(&ctl->vfull[vs], (nv / C::VS) & 1);
      const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&ctl->bad[vs]);
      // does every row see every key of the tile?
      const bool edge = bad != 0 || j0 + kTile - 1 > first ||
                        (a.window && j0 <= first + x.nt - 1 - a.window);
      auto sees = [&](int p, int j) {
        return j <= p && (!a.window || j > p - a.window) &&
               !((bad >> ((j - j0) >> 4)) & 1u);
      };
#pragma unroll
      for (int i = 0; i < 2 * WR; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = s[i >> 1][n][(i & 1) * 2 + e] * a.c;
            if (edge && !sees(pos[i], j0 + warp * 16 + n * 8 + fc + e)) v = -INFINITY;
            s[i >> 1][n][(i & 1) * 2 + e] = v;
            mx = fmaxf(mx, v);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if ((lane & 3) == 0) red[(i * 8 + fr) * 8 + warp] = mx;
      }
      named_sync(1, kWarps * 32);
      // ---- P = 2^(s - m)
      float grow[2 * WR];
#pragma unroll
      for (int i = 0; i < 2 * WR; ++i) {
        const float4 r0 = *reinterpret_cast<const float4*>(red + (i * 8 + fr) * 8);
        const float4 r1 = *reinterpret_cast<const float4*>(red + (i * 8 + fr) * 8 + 4);
        const float top = fmaxf(fmaxf(fmaxf(r0.x, r0.y), fmaxf(r0.z, r0.w)),
                                fmaxf(fmaxf(r1.x, r1.y), fmaxf(r1.z, r1.w))) - N::kShift;
        const float mn = fmaxf(m[i], top);
        const float ref = mn == -INFINITY ? 0.f : mn;
        grow[i] = exp2f(m[i] - ref);
        m[i] = mn;
        l[i] *= grow[i];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = exp2_approx(s[i >> 1][n][(i & 1) * 2] - ref);
          const float p1 = exp2_approx(s[i >> 1][n][(i & 1) * 2 + 1] - ref);
          l[i] += p0 + p1;
          const uint32_t at = tile_addr(pbuf, R * 128, i * 8 + fr, warp * 2 + n) + fc * 2;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(N::pack(p0, p1)) : "memory");
        }
      }
      named_sync(1, kWarps * 32);
      // ---- O = diag(grow) O + P V: this warp's D/8 dims, every key and row
#pragma unroll
      for (int i = 0; i < WR; ++i)
#pragma unroll
        for (int n = 0; n < D / 64; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][n][e] *= grow[i * 2 + (e >> 1)];
#pragma unroll
      for (int kk = 0; kk < kTile / 32; ++kk) {
        // 32 keys x 8 dims, or twice 16 keys x 16 dims
        uint32_t bv[D / 64][4];
        if constexpr (D == 64) {
          ldsm4_t(tile_addr(vbuf, kTile * 128, kk * 32 + lm * 8 + lr, warp), bv[0]);
        } else {
#pragma unroll
          for (int y = 0; y < 2; ++y)
            ldsm4_t(tile_addr(vbuf, kTile * 128, kk * 32 + y * 16 + (lm & 1) * 8 + lr,
                              warp * 2 + (lm >> 1)), bv[y]);
        }
        uint32_t wild = 0;   // non-finite halves of V
        uint32_t lost[D / 64][4];
        if (edge) {
#pragma unroll
          for (int y = 0; y < D / 64; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = bv[y][e];
              uint32_t mask = 0;
              if ((w & N::kExp) == N::kExp) mask |= 0xffffu;
              if (((w >> 16) & N::kExp) == N::kExp) mask |= 0xffff0000u;
              lost[y][e] = w & mask;
              bv[y][e] = w & ~mask;
              wild |= mask;
            }
          wild = __ballot_sync(0xffffffffu, wild != 0);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t ap[WR][4];
#pragma unroll
          for (int i = 0; i < WR; ++i) {
            ldsm4(tile_addr(pbuf, R * 128, i * 16 + (lm & 1) * 8 + lr, kk * 4 + y * 2 + (lm >> 1)),
                  ap[i]);
            if constexpr (D == 64) {
              N::mma(acc[i][0], ap[i], bv[0][y * 2], bv[0][y * 2 + 1]);
            } else {
              N::mma(acc[i][0], ap[i], bv[y][0], bv[y][1]);
              N::mma(acc[i][1], ap[i], bv[y][2], bv[y][3]);
            }
          }
          if (wild) {
            // rare: count, per row and dim, the +inf, -inf and NaN entries that the row sees
#pragma unroll
            for (int i = 0; i < WR; ++i) {
              uint32_t av[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = j0 + kk * 32 + y * 16 + (e >> 1) * 8 + fc;
                const int p = pos[i * 2 + (e & 1)];
                av[e] = (sees(p, j) ? N::kOne : 0u) |
                        (sees(p, j + 1) ? N::kOne << 16 : 0u);
              }
#pragma unroll
              for (int n = 0; n < D / 64; ++n) {
                float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kind = 0; kind < 3; ++kind) {
                  uint32_t ind[2];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const uint32_t w = D == 64 ? lost[0][y * 2 + e] : lost[y][n * 2 + e];
                    auto is = [&](uint32_t hw) -> uint32_t {
                      if ((hw & N::kExp) != N::kExp) return 0u;
                      const int k2 = (hw & 0x7fffu) != N::kExp ? 2 : (int)(hw >> 15);
                      return k2 == kind ? N::kOne : 0u;
                    };
                    ind[e] = is(w & 0xffffu) | (is(w >> 16) << 16);
                  }
                  float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                  N::mma(cnt, av, ind[0], ind[1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (cnt[e] > 0.f)
                      add[e] += kind == 0 ? INFINITY : kind == 1 ? -INFINITY : NAN;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][n][e] += add[e];
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->vempty[vs]));
      ++nv;
    }
    if (x.tile0 < x.tile1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->qempty[qb]));
      ++nq;
    }

    // ---- row sums over the warps, then the result or the split's partial
    if (x.tile0 == x.tile1) named_sync(1, kWarps * 32);   // the last unit's sums are read
#pragma unroll
    for (int i = 0; i < 2 * WR; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) sums[(i * 8 + fr) * 8 + warp] = l[i];
    }
    named_sync(1, kWarps * 32);
#pragma unroll
    for (int i = 0; i < 2 * WR; ++i) {
      const int r = i * 8 + fr;
      if (r >= rows) continue;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += sums[r * 8 + w];
      const int tk = x.t0 + r / a.G, hd = x.h * a.G + r % a.G;
      const int d0 = warp * DC + fc;
      if (x.ns == 1) {
        const int64_t row = (int64_t)(x.row0 + tk) * (a.Hk * a.G) + hd;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int n = 0; n < D / 64; ++n)
          *reinterpret_cast<uint32_t*>(reinterpret_cast<T*>(o.out) + row * D + d0 + n * 8) =
              N::pack(acc[i >> 1][n][(i & 1) * 2] * inv, acc[i >> 1][n][(i & 1) * 2 + 1] * inv);
        if (o.lse && warp == 0 && (lane & 3) == 0)
          o.lse[row] = sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * kLn2;
      } else {
        const int64_t rec = (((int64_t)x.b * tp + tk) * (a.Hk * a.G) + hd) * ns_cap + x.split;
#pragma unroll
        for (int n = 0; n < D / 64; ++n)
          *reinterpret_cast<float2*>(o.part + rec * D + d0 + n * 8) =
              make_float2(acc[i >> 1][n][(i & 1) * 2], acc[i >> 1][n][(i & 1) * 2 + 1]);
        if (warp == 0 && (lane & 3) == 0) o.part_ml[rec] = make_float2(m[i], sum);
      }
    }
  }
}

// Join the splits of each row, in split order: one warp to a (token, head).
template <typename T, int D, int WR>
__global__ void __launch_bounds__(128)
    k_paged_join(const Args a, const int tp, const int ns_cap, const AttnOut o) {
  pdl_wait_and_trigger();
  pdl_trigger();
  const int lane = threadIdx.x & 31, H = a.Hk * a.G;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int hd = (int)(id % H), tk = (int)(id / H % tp), b = (int)(id / H / tp);
  if (b >= a.n_seqs) return;
  const Seq s = seq_of(a, b);
  if (s.n > tp || tk >= s.n) return;
  const int ns = n_splits(max_tiles(a, s.len, tp), WR);
  if (ns == 1) return;
  const int64_t row = (int64_t)(s.row0 + tk) * H + hd;
  join_row<T, D>(o.part, o.part_ml, (((int64_t)b * tp + tk) * H + hd) * ns_cap, ns,
                 reinterpret_cast<T*>(o.out) + row * D, o.lse ? o.lse + row : nullptr, lane);
}

template <typename T, int D, int WR>
cudaError_t run(const Args& a, const AttnPlan& p, const Maps& maps, const AttnOut& o,
                cudaStream_t s) {
  const size_t smem =
      Cfg<D, WR>::kCtlOff + sizeof(Ctl) + (size_t)(a.n_seqs + 1) * sizeof(int) + 1024;
  cudaError_t err = cudaFuncSetAttribute(k_paged_attn<T, D, WR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  // no more CTAs than units there can be
  const int64_t row_tiles = (int64_t)a.T / p.tp + a.n_seqs;
  const int64_t most = row_tiles * a.Hk * p.ns_cap;
  const int nsm = sm_count();
  err = launch(k_paged_attn<T, D, WR>, dim3((unsigned)(most < nsm ? most : nsm)), kThreads, smem, s,
               a, p.tp, p.ns_cap, o, maps.k, maps.v, maps.q);
  if (err != cudaSuccess || p.ns_cap == 1) return err;
  const int64_t rows = (int64_t)a.n_seqs * p.tp * a.Hk * a.G;
  return launch(k_paged_join<T, D, WR>, dim3((unsigned)((rows + 3) / 4)), 128, 0, s, a, p.tp,
                p.ns_cap, o);
}

template <typename T, int D>
cudaError_t pick(const Args& a, const AttnPlan& p, const Maps& maps, const AttnOut& o,
                 cudaStream_t s) {
  switch (p.wr) {
    case 1: return run<T, D, 1>(a, p, maps, o, s);
    case 2: return run<T, D, 2>(a, p, maps, o, s);
    default: return run<T, D, 4>(a, p, maps, o, s);
  }
}

}  // namespace

AttnPlan attn_plan(const Args& a, int max_q) {
  AttnPlan p{};
  static_cast<RowTile&>(p) = row_tile(a.G, max_q);
  const int64_t entries = (int64_t)a.table_ld << a.lps;
  int64_t tiles = (entries + kTile - 1) / kTile;
  if (a.window) {
    const int64_t seen = ((int64_t)a.window + p.tp - 2) / kTile + 2;
    if (seen < tiles) tiles = seen;
  }
  // the count of splits does not fall as a sequence grows past 128 * least tiles
  const int64_t least = 2 * p.wr;
  const int64_t most = (tiles + least - 1) / least;
  p.ns_cap = (int)(most < 1 ? 1 : most < 128 ? most : 128);
  const size_t recs = (size_t)a.n_seqs * p.tp * a.Hk * a.G * p.ns_cap;
  p.rec_bytes = p.ns_cap == 1 ? 0 : (recs * a.D * sizeof(float) + 255) & ~(size_t)255;
  p.ml_bytes = p.ns_cap == 1 ? 0 : (recs * sizeof(float2) + 255) & ~(size_t)255;
  return p;
}

cudaError_t launch_paged_attn(const Args& a, int type, const AttnPlan& plan, const Maps& maps,
                              const AttnOut& o, cudaStream_t s) {
  if (type == PP_BF16)
    return a.D == 128 ? pick<__nv_bfloat16, 128>(a, plan, maps, o, s)
                      : pick<__nv_bfloat16, 64>(a, plan, maps, o, s);
  return a.D == 128 ? pick<__half, 128>(a, plan, maps, o, s) : pick<__half, 64>(a, plan, maps, o, s);
}

}  // namespace paged
}  // namespace pp
