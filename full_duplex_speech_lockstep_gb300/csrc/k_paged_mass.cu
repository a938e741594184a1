// k_paged_mass.cu - the attention weight that each cache entry receives.
//
//   mass_j = decay mass_j + sum over rows (t, g) of the chunk that see j of exp(s_j - lse)
// with the rows and scores of k_paged_attn.cu and the row sums that it returned.  A unit is
// (sequence, key head, 128-key tile); the rows that see the tile go past it in steps of up to
// 128 rows:
//   S' = K Q^T   M = 128 keys, N = the step's rows, on the 5th-generation tensor cores
// so that a thread owns a key (a tensor-memory lane) and adds up its weights in row order:
// no sum crosses threads but one (two groups take alternate columns), nothing is added
// atomically, and the bits are the same in every run.
//
//   warp 0        producer: the key tile, then the steps' rows, by TMA
//   warp 1        one thread issues the MMAs, up to four steps ahead of the sums
//   warps 2-3     what the sums need from memory, ahead of them: each row's lse (with the
//                 rows that do not count set to infinity), each key's old mass and page
//   warps 4-7, 8-11   the sums: columns 0-15, 32-47, ... and 16-31, 48-63, ...
#include "pp_paged.cuh"
#include "pp_tcgen05.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kThreads = 384;
constexpr int kBufs = 4;             // S buffers of 128 columns: all of tensor memory
constexpr int kAux = 8;              // steps and units that the memory warps may be ahead
constexpr int kMaxStages = 8;
constexpr int kQStages = 3;

struct Ctl {
  uint64_t kfull[kMaxStages], kempty[kMaxStages], qfull[kQStages], qempty[kQStages];
  uint64_t sfull[kBufs], sfree[kBufs];
  uint64_t lfull[kAux], lempty[kAux], ufull[kAux], uempty[kAux];
  uint64_t done;
  uint32_t tmem;
  int abort;
  float ref[kAux][kTile];            // lse * log2(e) of a step's rows
  float old[kAux][kTile];            // decayed mass of a unit's keys
  int page[kAux][8];                 // pages of its 16-key groups, -1 for none
  float half[2][kTile];              // the second group's sums
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

// 16 columns of this thread's tensor-memory lane
__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_mass(const Args a, const int tp, const int N_, const int KS, const float* lse,
                 float* mass, const float decay, const __grid_constant__ CUtensorMap mapK,
                 const __grid_constant__ CUtensorMap mapQ) {
  constexpr int kTileBytes = kTile * D * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int q_bytes = N_ * D * 2;                       // a stage of rows
  uint8_t* q_smem = smem + KS * kTileBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(q_smem + kQStages * q_bytes);
  int* pre = reinterpret_cast<int*>(ctl + 1);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = N_ > 16 ? 2 : 1;                   // groups that sum
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(smem_u32(&ctl->kfull[i]), 1);
      mbar_init(smem_u32(&ctl->kempty[i]), 1);
    }
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(smem_u32(&ctl->qfull[i]), 1);
      mbar_init(smem_u32(&ctl->qempty[i]), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_u32(&ctl->sfull[i]), 1);
      mbar_init(smem_u32(&ctl->sfree[i]), 4 * groups);
    }
    for (int i = 0; i < kAux; ++i) {
      mbar_init(smem_u32(&ctl->lfull[i]), 2);
      mbar_init(smem_u32(&ctl->lempty[i]), 4 * groups);
      mbar_init(smem_u32(&ctl->ufull[i]), 2);
      mbar_init(smem_u32(&ctl->uempty[i]), 4);
    }
    mbar_init(smem_u32(&ctl->done), 1);
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
  prefix_units(pre, a.n_seqs, [&](int b) { return a.Hk * ((seq_len(a, b) + kTile - 1) / kTile); });
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = ctl->tmem;
  const int units = pre[a.n_seqs];
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*abort_flag) return;
    if (!mbar_wait(smem_u32(bar), parity)) {
      *abort_flag = 1;
      raise(a, PP_S_TIMEOUT);
    }
  };
  // A unit that no row sees has nothing to add; without decay it is left out.
  auto skip = [&](const Unit& x) { return x.t0 == x.t1 && decay == 1.f; };

  if (warp == 0) {
    // ---- producer -------------------------------------------------------------------------
    uint32_t nk = 0, nq = 0, seen_bad = 0;
    for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x) {
      const Unit x = unit_of(a, pre, u);
      if (x.t0 == x.t1) continue;
      const int ks = nk % KS;
      if (nk >= KS) wait(&ctl->kempty[ks], (nk / KS - 1) & 1);
      if (*abort_flag) break;
      seen_bad |= load_key_tile(a, &mapK, smem_u32(smem + ks * kTileBytes),
                                smem_u32(&ctl->kfull[ks]), x.b, x.h, x.j0, x.len, lane, nullptr);
      ++nk;
      for (int t = x.t0; t < x.t1; t += tp) {
        const int qs = nq % kQStages;
        if (nq >= kQStages) wait(&ctl->qempty[qs], (nq / kQStages - 1) & 1);
        if (*abort_flag) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&ctl->qfull[qs]);
          mbar_expect_tx(bar, (uint32_t)(tp * a.G * D * 2));
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_4d(smem_u32(q_smem + qs * q_bytes + bx * N_ * 128), &mapQ, bx * 64, x.h * a.G,
                        x.row0 + t, 0, bar);
        }
        ++nq;
      }
    }
    if (seen_bad && lane == 0) raise(a, PP_S_INDEX);
    if (lane == 0) {   // every copy lands before the CTA may exit (bounded waits)
      for (uint32_t i = nk > KS ? nk - KS : 0; i < nk; ++i)
        mbar_wait(smem_u32(&ctl->kfull[i % KS]), (i / KS) & 1);
      for (uint32_t i = nq > kQStages ? nq - kQStages : 0; i < nq; ++i)
        mbar_wait(smem_u32(&ctl->qfull[i % kQStages]), (i / kQStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer -----------------------------------------------------------------------
    if (lane == 0) {
      const uint32_t id = (1u << 4) | Num<T>::kMmaTypes | ((uint32_t)(kTile >> 4) << 24) |
                          ((uint32_t)(N_ >> 3) << 17);
      uint32_t nk = 0, nq = 0;
      for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x) {
        const Unit x = unit_of(a, pre, u);
        if (x.t0 == x.t1) continue;
        const int ks = nk % KS;
        wait(&ctl->kfull[ks], (nk / KS) & 1);
        ++nk;
        const uint32_t kb = smem_u32(smem + ks * kTileBytes);
        for (int t = x.t0; t < x.t1; t += tp) {
          const int qs = nq % kQStages, bb = nq % kBufs;
          wait(&ctl->qfull[qs], (nq / kQStages) & 1);
          if (nq >= kBufs) wait(&ctl->sfree[bb], (nq / kBufs - 1) & 1);
          if (*abort_flag) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t qb = smem_u32(q_smem + qs * q_bytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tmem + bb * kTile,
                      smem_desc(kb + (kk >> 2) * (kTile * 128) + (kk & 3) * 32),
                      smem_desc(qb + (kk >> 2) * (N_ * 128) + (kk & 3) * 32), id, kk > 0);
          umma_commit(smem_u32(&ctl->sfull[bb]));
          umma_commit(smem_u32(&ctl->qempty[qs]));
          ++nq;
        }
        umma_commit(smem_u32(&ctl->kempty[ks]));
      }
      // every MMA is done before tensor memory is given back (bounded wait)
      umma_commit(smem_u32(&ctl->done));
      mbar_wait(smem_u32(&ctl->done), 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---- memory warps: two values to a thread ---------------------------------------------
    const int i = threadIdx.x - 64;
    const int H = a.Hk * a.G;
    uint32_t nl = 0, nu = 0;
    for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x) {
      const Unit x = unit_of(a, pre, u);
      if (skip(x)) continue;
      const int us = nu % kAux;
      if (nu >= kAux) wait(&ctl->uempty[us], (nu / kAux - 1) & 1);
      if (*abort_flag) break;
      if (i < 8) {
        const int j = x.j0 + i * 16;
        ctl->page[us][i] = j < x.len ? page_of(a, x.b, j) : -1;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int j = x.j0 + i + k * 64;
        float old = 0.f;
        if (decay != 0.f && j < x.len) {
          const int p = page_of(a, x.b, j);
          if (p >= 0)
            old = decay *
                  mass[(((int64_t)p * a.Hk + x.h) << a.lps) + (j & ((1 << a.lps) - 1))];
        }
        ctl->old[us][i + k * 64] = old;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->ufull[us]));
      ++nu;
      for (int t = x.t0; t < x.t1; t += tp) {
        const int ls = nl % kAux;
        const int rows = min(tp, x.t1 - t) * a.G;
        if (nl >= kAux) wait(&ctl->lempty[ls], (nl / kAux - 1) & 1);
        if (*abort_flag) break;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = i + k * 64, tk = r / a.G;
          // rows that are not there, or that saw nothing, give nothing
          float z = r < rows
                        ? lse[(int64_t)(x.row0 + t + tk) * H + x.h * a.G + (r - tk * a.G)] * kLog2e
                        : INFINITY;
          ctl->ref[ls][r] = z == -INFINITY ? INFINITY : z;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->lfull[ls]));
        ++nl;
      }
    }
  } else if (warp < 4 + 4 * groups) {
    // ---- sums: a thread to a key --------------------------------------------------------------
    const int g = (warp - 4) >> 2, key = threadIdx.x - 128 - g * 128;
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t c2 = f32x2(a.c, a.c);
    uint32_t nl = 0, nu = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Unit x = unit_of(a, pre, u);
      if (skip(x)) continue;
      const int first = x.len - x.n, j = x.j0 + key;
      float sum = 0.f;
      for (int t = x.t0; t < x.t1; t += tp) {
        const int bb = nl % kBufs, ls = nl % kAux;
        const int nt = min(tp, x.t1 - t);
        // the rows of the step that see this key: columns [lo, hi)
        int lo = 0, hi = nt * a.G;
        const bool edge = hi < N_ || x.j0 + kTile - 1 > first + t ||
                          (a.window && x.j0 <= first + t + nt - 1 - a.window);
        if (edge) {
          lo = max(0, j - first - t) * a.G;
          if (a.window) hi = (int)min((int64_t)hi, ((int64_t)j + a.window - first - t) * a.G);
        }
        wait(&ctl->lfull[ls], (nl / kAux) & 1);
        wait(&ctl->sfull[bb], (nl / kBufs) & 1);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int c0 = g * 16; c0 < N_; c0 += 16 * groups) {
          uint32_t s[16];
          tmem_ld16(at + bb * kTile + c0, s);
          tmem_wait_ld();
          const float4* rp = reinterpret_cast<const float4*>(&ctl->ref[ls][c0]);
          uint64_t part = 0;   // (0, 0)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 z = rp[i / 4];
            const uint64_t e0 = fma2(f32x2(after_wait(s[i]), after_wait(s[i + 1])), c2,
                                     f32x2(-z.x, -z.y));
            const uint64_t e1 = fma2(f32x2(after_wait(s[i + 2]), after_wait(s[i + 3])), c2,
                                     f32x2(-z.z, -z.w));
            float p[4] = {exp2_approx(lo_of(e0)), exp2_approx(hi_of(e0)), exp2_approx(lo_of(e1)),
                          exp2_approx(hi_of(e1))};
            if (edge) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c0 + i + k < lo || c0 + i + k >= hi) p[k] = 0.f;
            }
            part = add2(part, add2(f32x2(p[0], p[1]), f32x2(p[2], p[3])));
          }
          sum += lo_of(part) + hi_of(part);
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctl->sfree[bb]));
          mbar_arrive(smem_u32(&ctl->lempty[ls]));
        }
        ++nl;
      }
      if (groups == 2) {
        // the second group's sums come through shared memory, two units deep
        if (g == 1) ctl->half[nu & 1][key] = sum;
        named_sync(1, 256);
        if (g == 0) sum += ctl->half[nu & 1][key];
      }
      if (g == 0) {
        const int us = nu % kAux;
        wait(&ctl->ufull[us], (nu / kAux) & 1);
        const int p = ctl->page[us][key >> 4];
        sum += ctl->old[us][key];
        if (p >= 0 && j < x.len)
          mass[(((int64_t)p * a.Hk + x.h) << a.lps) + (j & ((1 << a.lps) - 1))] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->uempty[us]));
      }
      ++nu;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

template <typename T, int D>
cudaError_t run(const Args& a, const Maps& maps, int tp, const float* lse, float* mass, float decay,
                cudaStream_t s) {
  const int n = (tp * a.G + 15) / 16 * 16;
  const int q_bytes = n * D * 2, tile = kTile * D * 2;
  // key tiles fill what the rows and the control block leave of 227 KB
  const int fixed = (int)(sizeof(Ctl) + (a.n_seqs + 1) * sizeof(int)) + 1024 + kQStages * q_bytes;
  int ks = (227 * 1024 - fixed) / tile;
  if (ks > kMaxStages) ks = kMaxStages;
  const size_t smem = (size_t)fixed + (size_t)ks * tile;
  cudaError_t err = cudaFuncSetAttribute(k_paged_mass<T, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const int nsm = sm_count();
  const int64_t tiles = (((int64_t)a.table_ld << a.lps) + kTile - 1) / kTile;
  const int64_t most = (int64_t)a.n_seqs * a.Hk * tiles;
  return launch(k_paged_mass<T, D>, dim3((unsigned)(most < nsm ? most : nsm)), kThreads, smem, s, a,
                tp, n, ks, lse, mass, decay, maps.k, maps.q);
}

}  // namespace

int mass_tokens(int G, int max_q) {
  const int tp = kTile / G;
  return max_q < tp ? max_q : tp;
}

cudaError_t launch_paged_mass(const Args& a, int type, const Maps& maps, const float* lse,
                              float* mass, float decay, int tp, cudaStream_t s) {
  if (type == PP_BF16)
    return a.D == 128 ? run<__nv_bfloat16, 128>(a, maps, tp, lse, mass, decay, s)
                      : run<__nv_bfloat16, 64>(a, maps, tp, lse, mass, decay, s);
  return a.D == 128 ? run<__half, 128>(a, maps, tp, lse, mass, decay, s)
                    : run<__half, 64>(a, maps, tp, lse, mass, decay, s);
}

}  // namespace paged
}  // namespace pp
