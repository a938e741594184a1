// k_paged_mass.cu - the attention weight that each cache entry receives.
//
//   mass_j = decay mass_j + sum over rows (t, g) of the chunk that see j of exp(s_j - lse)
// with the rows and scores of k_paged_attn.cu and the row sums that it returned.  A unit is
// (sequence, key head, 128-key tile): the rows that see the tile go past it, and each key's
// sum is added up by one warp in row order, so nothing is added atomically and the bits are
// the same in every run.
//   warp 8      producer: the key tile, then the row tiles, by TMA;
//   warps 0-7   16 keys each, held as matrix fragments while the rows pass.
#include "pp_paged.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32 + 32;
constexpr int kKS = 3, kQS = 3;

template <int D, int WR>
struct Cfg {
  static constexpr int R = 16 * WR;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kQOff = kKS * kTileBytes;
  static constexpr int kCtlOff = kQOff + kQS * kQBytes;
};

struct Ctl {
  uint64_t kfull[kKS], kempty[kKS], qfull[kQS], qempty[kQS];
  int abort;
};

struct Unit {
  int b, h, j0;
  int row0, n, len;
  int t0, t1;        // tokens that see some key of the tile
};

__device__ __forceinline__ Unit unit_of(const Args& a, const int* pre, int u) {
  Unit x;
  x.b = find_seq(pre, a.n_seqs, u);
  const Seq s = seq_of(a, x.b);
  u -= pre[x.b];
  const int tiles = (s.len + kTile - 1) / kTile;
  x.h = u / tiles;
  x.j0 = (u - x.h * tiles) * kTile;
  x.row0 = s.row0;
  x.n = s.n;
  x.len = s.len;
  const int first = s.len - s.n;
  x.t0 = max(0, x.j0 - first);
  x.t1 = s.n;
  if (a.window)
    x.t1 = (int)min((int64_t)s.n, (int64_t)min(x.j0 + kTile, s.len) - 1 + a.window - first);
  if (x.t1 < x.t0) x.t1 = x.t0;
  return x;
}

template <typename T, int D, int WR>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_mass(const Args a, const int tp, const float* lse, float* mass, const float decay,
                 const __grid_constant__ CUtensorMap mapK,
                 const __grid_constant__ CUtensorMap mapQ) {
  using C = Cfg<D, WR>;
  using N = Num<T>;
  constexpr int R = C::R;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kCtlOff);
  int* pre = reinterpret_cast<int*>(ctl + 1);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKS; ++i) {
      mbar_init(smem_u32(&ctl->kfull[i]), 1);
      mbar_init(smem_u32(&ctl->kempty[i]), kWarps);
    }
    for (int i = 0; i < kQS; ++i) {
      mbar_init(smem_u32(&ctl->qfull[i]), 1);
      mbar_init(smem_u32(&ctl->qempty[i]), kWarps);
    }
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait_and_trigger();
  pdl_trigger();
  prefix_units(pre, a.n_seqs, [&](int b) { return a.Hk * ((seq_len(a, b) + kTile - 1) / kTile); });
  const int units = pre[a.n_seqs];
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*abort_flag) return;
    if (!mbar_wait(smem_u32(bar), parity)) {
      *abort_flag = 1;
      raise(a, PP_S_TIMEOUT);
    }
  };

  if (warp == kWarps) {
    uint32_t nk = 0, nq = 0, seen_bad = 0;
    for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x) {
      const Unit x = unit_of(a, pre, u);
      if (x.t0 == x.t1) continue;
      const int ks = nk % kKS;
      if (nk >= kKS) wait(&ctl->kempty[ks], (nk / kKS - 1) & 1);
      if (*abort_flag) break;
      const uint32_t bad = load_key_tile(a, &mapK, smem_u32(smem + ks * C::kTileBytes),
                                         smem_u32(&ctl->kfull[ks]), x.b, x.h, x.j0, x.len, lane,
                                         nullptr);
      seen_bad |= bad;
      ++nk;
      for (int t = x.t0; t < x.t1; t += tp) {
        const int qs = nq % kQS;
        if (nq >= kQS) wait(&ctl->qempty[qs], (nq / kQS - 1) & 1);
        if (*abort_flag) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&ctl->qfull[qs]);
          const uint32_t dst = smem_u32(smem + C::kQOff + qs * C::kQBytes);
          mbar_expect_tx(bar, (uint32_t)(tp * a.G * D * 2));
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_4d(dst + bx * (R * 128), &mapQ, bx * 64, x.h * a.G, x.row0 + t, 0, bar);
        }
        ++nq;
      }
    }
    if (seen_bad && lane == 0) raise(a, PP_S_INDEX);
    if (lane == 0) {
      for (uint32_t i = nk > kKS ? nk - kKS : 0; i < nk; ++i)
        mbar_wait(smem_u32(&ctl->kfull[i % kKS]), (i / kKS) & 1);
      for (uint32_t i = nq > kQS ? nq - kQS : 0; i < nq; ++i)
        mbar_wait(smem_u32(&ctl->qfull[i % kQS]), (i / kQS) & 1);
    }
    return;
  }

  const int lm = lane >> 3, lr = lane & 7;
  const int fr = lane >> 2, fc = (lane & 3) * 2;
  const int H = a.Hk * a.G;
  uint32_t nk = 0, nq = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit x = unit_of(a, pre, u);
    const int first = x.len - x.n;
    const int key0 = x.j0 + warp * 16 + fc;
    // this warp's four key columns: where their sums go (entries of no page have none)
    float* dst[4];
    float old[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = key0 + (k >> 1) * 8 + (k & 1);
      const int p = j < x.len ? page_of(a, x.b, j) : -1;
      dst[k] = p < 0 ? nullptr
                     : mass + ((((int64_t)p * a.Hk + x.h) << a.lps) + (j & ((1 << a.lps) - 1)));
      old[k] = dst[k] && decay != 0.f && fr == 0 ? *dst[k] * decay : 0.f;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (x.t0 < x.t1) {
      const int ks = nk % kKS;
      const uint32_t kbuf = smem_u32(smem + ks * C::kTileBytes);
      wait(&ctl->kfull[ks], (nk / kKS) & 1);
      uint32_t bk[D / 16][4];
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        ldsm4(tile_addr(kbuf, kTile * 128, warp * 16 + (lm >> 1) * 8 + lr, kk * 2 + (lm & 1)),
              bk[kk]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->kempty[ks]));
      ++nk;
      for (int t = x.t0; t < x.t1; t += tp) {
        const int nt = min(tp, x.t1 - t), rows = nt * a.G;
        // rows past the tile's tokens give nothing: their sum counts as infinite
        float ref[2 * WR];
        int pos[2 * WR];
#pragma unroll
        for (int i = 0; i < 2 * WR; ++i) {
          const int r = i * 8 + fr, tk = r / a.G;
          const bool in = r < rows;
          const float z =
              in ? lse[(int64_t)(x.row0 + t + tk) * H + x.h * a.G + (r - tk * a.G)] : -INFINITY;
          ref[i] = z == -INFINITY ? INFINITY : z * kLog2e;
          pos[i] = in ? first + t + tk : -1;
        }
        const int qs = nq % kQS;
        const uint32_t qbuf = smem_u32(smem + C::kQOff + qs * C::kQBytes);
        wait(&ctl->qfull[qs], (nq / kQS) & 1);
        float s[WR][2][4];
#pragma unroll
        for (int i = 0; i < WR; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int i = 0; i < WR; ++i) {
            uint32_t aq[4];
            ldsm4(tile_addr(qbuf, R * 128, i * 16 + (lm & 1) * 8 + lr, kk * 2 + (lm >> 1)), aq);
            N::mma(s[i][0], aq, bk[kk][0], bk[kk][1]);
            N::mma(s[i][1], aq, bk[kk][2], bk[kk][3]);
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->qempty[qs]));
        ++nq;
#pragma unroll
        for (int i = 0; i < 2 * WR; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = key0 + (k >> 1) * 8 + (k & 1);
            const bool see = j <= pos[i] && (!a.window || j > pos[i] - a.window) &&
                             ref[i] != INFINITY;
            const float v = fmaf(s[i >> 1][k >> 1][(i & 1) * 2 + (k & 1)], a.c, -ref[i]);
            sum[k] += see ? exp2_approx(v) : 0.f;
          }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
      if (fr == 0 && dst[k]) *dst[k] = old[k] + sum[k];
    }
  }
}

template <typename T, int D, int WR>
cudaError_t run(const Args& a, const Maps& maps, int tp, const float* lse, float* mass, float decay,
                cudaStream_t s) {
  const size_t smem = Cfg<D, WR>::kCtlOff + sizeof(Ctl) + (size_t)(a.n_seqs + 1) * sizeof(int) + 1024;
  cudaError_t err = cudaFuncSetAttribute(k_paged_mass<T, D, WR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const int nsm = sm_count();
  const int64_t tiles = (((int64_t)a.table_ld << a.lps) + kTile - 1) / kTile;
  const int64_t most = (int64_t)a.n_seqs * a.Hk * tiles;
  return launch(k_paged_mass<T, D, WR>, dim3((unsigned)(most < nsm ? most : nsm)), kThreads, smem,
                s, a, tp, lse, mass, decay, maps.k, maps.q);
}

template <typename T, int D>
cudaError_t pick(const Args& a, const Maps& maps, int wr, int tp, const float* lse, float* mass,
                 float decay, cudaStream_t s) {
  switch (wr) {
    case 1: return run<T, D, 1>(a, maps, tp, lse, mass, decay, s);
    case 2: return run<T, D, 2>(a, maps, tp, lse, mass, decay, s);
    default: return run<T, D, 4>(a, maps, tp, lse, mass, decay, s);
  }
}

}  // namespace

cudaError_t launch_paged_mass(const Args& a, int type, const RowTile& r, const Maps& maps,
                              const float* lse, float* mass, float decay, cudaStream_t s) {
  if (type == PP_BF16)
    return a.D == 128 ? pick<__nv_bfloat16, 128>(a, maps, r.wr, r.tp, lse, mass, decay, s)
                      : pick<__nv_bfloat16, 64>(a, maps, r.wr, r.tp, lse, mass, decay, s);
  return a.D == 128 ? pick<__half, 128>(a, maps, r.wr, r.tp, lse, mass, decay, s)
                    : pick<__half, 64>(a, maps, r.wr, r.tp, lse, mass, decay, s);
}

}  // namespace paged
}  // namespace pp
