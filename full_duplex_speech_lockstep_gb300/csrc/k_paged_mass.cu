// k_paged_mass.cu - the attention weight that each cache entry receives.
//
//   mass_j = decay mass_j + sum over rows (t, g) of the chunk that see j of exp(s_j - lse)
// with the rows and scores of k_paged_attn.cu and the row sums that it returned.  A unit is
// (sequence, key head, pair of 128-key tiles); the rows that see the pair go past it in steps of
// up to 128 rows:
//   S' = K Q^T   M = 128 keys, N = the step's rows, on the 5th-generation tensor cores
// so that a thread owns a key (a tensor-memory lane) and adds up its weights in row order:
// no sum crosses threads, nothing is added atomically, and the bits are the same in every run.
// (With one tile to a unit each step's 32 KB of rows served 128 keys only, and reading them
// from L2 bounded the kernel: 114 us for the 4 x 300 tokens below.)
//
// Measured (bf16, 128 dims, in a graph): 64 sequences of 1 token and up to 3000 entries, 32 heads on
// 32 key heads: 130 us, 6.0 TB/s, bound by reading K once and by the units' starts, two tiles to
// a unit.  4 sequences of up to 300 tokens and 16000 entries, 32 heads on 8: 95 us, 805 TFLOP/s,
// 2500 clocks a step of two tiles, whose products take 1024 and whose exponentials as many; what
// takes the rest is not known (16 warps of sums instead of 8: the same).
//
// A CTA takes a run of consecutive units of about the same number of steps as the others (pairs of
// tiles that no row sees, below a window, only decay and count as little; without a decay they are no
// units: 4096 tokens under a window of 1000 over 65000 entries, 32 heads on 8: 613 -> 62 us):
//   warp 0        producer: the units and their key tiles, by TMA
//   warp 1        one thread issues the MMAs, up to four steps ahead of the sums
//   warp 2        each key's old mass and page, a unit ahead
//   warp 3        the steps' rows by TMA; each row's lse, a step ahead; rows that do not count:
//                 minus infinity
//   warps 4-7, 8-11   the sums of the pair's first and second tile
#include <type_traits>

#include "pp_paged.cuh"
#include "pp_tcgen05.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kThreads = 384;
constexpr int kBufs = 4;             // S buffers of 128 columns: all of tensor memory
constexpr int kAux = 8;              // steps and units that the memory warps may be ahead
constexpr int kMaxStages = 8;
constexpr int kQStages = 2;

struct Ctl {
  UnitRing ring;
  uint64_t kfull[kMaxStages], kempty[kMaxStages], qfull[kQStages], qempty[kQStages];
  uint64_t sfull[kBufs], sfree[kBufs];
  uint64_t lfull[kAux], lempty[kAux], ufull[kAux], uempty[kAux];
  uint64_t done;
  uint32_t tmem;
  int abort;
  alignas(16) float ref[kAux][kTile];   // -lse * log2(e) of a step's rows
  alignas(16) float old[kAux][2 * kTile];   // decayed mass of a unit's keys
  int page[kAux][16];                // pages of its 16-key groups, -1 for none
};

// A head's units: pairs [from, seen) of tiles of which no row sees a key, which only decay and cost 1
// (none without a decay), and pairs [seen, pairs), which cost the steps of all rows.
struct Head {
  int from, seen, pairs, steps;
  __device__ __forceinline__ Head() {}
  __device__ __forceinline__ Head(const Args& a, const Seq& s, int tp, bool decays) {
    const int first = s.total - s.n;                 // the first row's entry
    const int low = s.n == 0 ? s.len : a.window ? min(max(first - a.window + 1, 0), s.len) : 0;
    pairs = (s.len + 2 * kTile - 1) / (2 * kTile);
    seen = low < s.len ? low / (2 * kTile) : pairs;
    from = decays ? 0 : seen;
    steps = (s.n + tp - 1) / tp;
  }
  __device__ __forceinline__ int64_t cost() const {
    return seen - from + (int64_t)(pairs - seen) * steps;
  }
};

// A walk over this CTA's units, in order.
struct Walk {
  const Args& a;
  const int64_t* pre;
  const int tp;
  const bool decays;
  int64_t at, end;      // cost before this unit, cost where the run ends
  int b, h, pair;
  Head head;            // of the sequence
  Seq s;
  int j0, t0, t1;       // the unit's first key; the tokens that see some key of it

  __device__ __forceinline__ Walk(const Args& a_, const int64_t* pre_, int tp_, bool decays_)
      : a(a_), pre(pre_), tp(tp_), decays(decays_) {
    const int64_t total = pre[a.n_seqs];
    at = total * blockIdx.x / gridDim.x;
    end = total * (blockIdx.x + 1) / gridDim.x;
    if (at >= end) return;
    b = find_seq(pre, a.n_seqs, at);
    sequence();
    // the first unit that starts in the run
    const int64_t cost = head.cost(), dim = head.seen - head.from;
    h = (int)((at - pre[b]) / cost);
    const int64_t in = at - pre[b] - h * cost;
    const int64_t i = in <= dim ? in : dim + (in - dim + head.steps - 1) / head.steps;
    pair = head.from + (int)i;
    at = pre[b] + h * cost + (i <= dim ? i : dim + (i - dim) * head.steps);
    if (pair == head.pairs) next_head();
    unit();
  }
  __device__ __forceinline__ bool done() const { return at >= end; }
  __device__ __forceinline__ void sequence() {
    s = seq_of(a, b);
    head = Head(a, s, tp, decays);
  }
  __device__ __forceinline__ void next_head() {
    if (++h == a.Hk) {
      h = 0;
      do {
        ++b;
      } while (b < a.n_seqs && pre[b + 1] == pre[b]);
      if (b < a.n_seqs) sequence();
    }
    pair = head.from;
  }
  __device__ __forceinline__ void next() {
    at += pair < head.seen ? 1 : head.steps;
    if (++pair == head.pairs) next_head();
    unit();
  }
  __device__ __forceinline__ void unit() {
    if (done()) return;
    j0 = pair * 2 * kTile;
    const int first = s.total - s.n;
    t0 = max(0, j0 - first);
    t1 = s.n;
    if (a.window)
      t1 = (int)min((int64_t)s.n, (int64_t)min(j0 + 2 * kTile, s.len) - 1 + a.window - first);
    if (t1 < t0) t1 = t0;
  }
};

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

// Sum of 2^(s c + ref) over the columns [0, cols) of a lane, those outside [lo, hi) left out
// (`masked`); cols is a multiple of W otherwise.  Rows of no sum have a ref of -infinity and give 0
// unless their s is a NaN or +infinity: then the sum is NaN, but for masked steps of few rows, which
// leave them out.  The next W columns are on their way from tensor memory while these are summed.
template <int W, typename M>
__device__ __forceinline__ float weigh(uint32_t at, const float* ref, uint64_t c2, int cols, int lo,
                                       int hi, M) {
  uint64_t part[2] = {0, 0};   // two sums of two
  uint32_t s[2][W];
  auto load = [&](uint32_t (&r)[W], int c0) {
#pragma unroll
    for (int i = 0; i < W / 16; ++i) tmem_ld16(at + c0 + 16 * i, r + 16 * i);
  };
  auto sum = [&](uint32_t (&r)[W], int c0) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const float4 z = reinterpret_cast<const float4*>(ref + c0)[i];
      const uint64_t e0 = fma2((uint64_t)r[4 * i] | ((uint64_t)r[4 * i + 1] << 32), c2,
                               f32x2(z.x, z.y));
      const uint64_t e1 = fma2((uint64_t)r[4 * i + 2] | ((uint64_t)r[4 * i + 3] << 32), c2,
                               f32x2(z.z, z.w));
      float p[4] = {exp2_approx(lo_of(e0)), exp2_approx(hi_of(e0)), exp2_approx(lo_of(e1)),
                    exp2_approx(hi_of(e1))};
      if constexpr (M::value) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float zk = k == 0 ? z.x : k == 1 ? z.y : k == 2 ? z.z : z.w;
          if (c0 + 4 * i + k < lo || c0 + 4 * i + k >= hi || (W == 16 && zk == -INFINITY)) p[k] = 0.f;
        }
      }
      part[0] = add2(part[0], f32x2(p[0], p[1]));
      part[1] = add2(part[1], f32x2(p[2], p[3]));
    }
  };
  auto landed = [&](uint32_t (&r)[W]) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < W; ++i) asm volatile("" : "+r"(r[i]));
  };
  load(s[0], 0);
  landed(s[0]);
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += 2 * W) {
    if (c0 + W < cols) load(s[1], c0 + W);
    sum(s[0], c0);
    if (c0 + W >= cols) break;
    landed(s[1]);
    if (c0 + 2 * W < cols) load(s[0], c0 + 2 * W);
    sum(s[1], c0 + W);
    if (c0 + 2 * W < cols) landed(s[0]);
  }
  const uint64_t both = add2(part[0], part[1]);
  return lo_of(both) + hi_of(both);
}

// The same sum, bit for bit, that leaves out rows of no sum (a ref of -infinity) whatever s they
// hold: minus infinity plus a NaN or an infinity is a NaN.  Rare, so short rather than fast.
__device__ __forceinline__ float weigh_live(uint32_t at, const float* ref, uint64_t c2, int cols,
                                            int lo, int hi) {
  uint64_t part[2] = {0, 0};
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += 16) {
    uint32_t s[16];
    tmem_ld16(at + c0, s);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(s[i]));
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float z[2] = {ref[c0 + i], ref[c0 + i + 1]};
      const uint64_t e = fma2((uint64_t)s[i] | ((uint64_t)s[i + 1] << 32), c2, f32x2(z[0], z[1]));
      float p[2] = {exp2_approx(lo_of(e)), exp2_approx(hi_of(e))};
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (c0 + i + k < lo || c0 + i + k >= hi || z[k] == -INFINITY) p[k] = 0.f;
      part[(i >> 1) & 1] = add2(part[(i >> 1) & 1], f32x2(p[0], p[1]));
    }
  }
  const uint64_t both = add2(part[0], part[1]);
  return lo_of(both) + hi_of(both);
}

template <typename T, int D, int W>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_mass(const __grid_constant__ Args a, const int tp, const int N_, const int KS, const float* lse,
                 float* mass, const float decay, const __grid_constant__ CUtensorMap mapK,
                 const __grid_constant__ CUtensorMap mapQ) {
  constexpr int kTileBytes = kTile * D * 2;
  // Steps of few rows pass through many units, and with every wait's loop in place the roles' code is
  // larger than the instruction cache: there the loop is a function (137 us instead of 180 for the
  // tick).  Steps of many rows wait more than they fetch code (106 us instead of 104.5).
  constexpr bool kCall = W == 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler then knows that it is shared memory)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int q_bytes = N_ * D * 2;                       // a stage of rows
  uint8_t* q_smem = smem + KS * kTileBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(q_smem + kQStages * q_bytes);
  int64_t* pre = reinterpret_cast<int64_t*>(ctl + 1);
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(smem_u32(&ctl->kfull[i]), i == 0 ? 1 + a.withhold : 1);
      mbar_init(smem_u32(&ctl->kempty[i]), 1);
    }
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(smem_u32(&ctl->qfull[i]), 1);
      mbar_init(smem_u32(&ctl->qempty[i]), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_u32(&ctl->sfull[i]), 1);
      mbar_init(smem_u32(&ctl->sfree[i]), 4);
    }
    for (int i = 0; i < kAux; ++i) {
      mbar_init(smem_u32(&ctl->lfull[i]), 1);
      mbar_init(smem_u32(&ctl->lempty[i]), 8);
      mbar_init(smem_u32(&ctl->ufull[i]), 1);
      mbar_init(smem_u32(&ctl->uempty[i]), 8);
    }
    mbar_init(smem_u32(&ctl->done), 1);
    ring_init(ctl->ring, 11);            // MMA issuer, two memory warps, eight of sums
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
  // (a sequence without new rows only decays, and not even that at 1)
  prefix_units(a, pre, [&](int b) -> int64_t {
    const Seq s = seq_of(a, b);
    if (s.n == 0 && decay == 1.f) return 0;
    check_len(a, s);
    return a.Hk * Head(a, s, tp, decay != 1.f).cost();
  });
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = ctl->tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_phase<kCall>(a, bar, parity, abort_flag); };
  if (warp == 0) {
    // ---- producer -------------------------------------------------------------------------
    uint32_t nk = 0, nu = 0, seen_bad = 0;
    Walk x(a, pre, tp, decay != 1.f);
    TilePages next[2];
    auto find = [&] {
      if (x.done()) return;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        next[i] = find_pages(a, x.b, x.j0 + i * kTile, x.s.len, false, lane);
    };
    find();
#pragma unroll 1
    while (!x.done() && !*abort_flag) {
      // this unit, and the next one's pages on their way
      const Unit u{x.b, x.h, x.s.row0 + x.t0, x.t1 - x.t0, x.s.total - x.s.n + x.t0, 2 * x.pair,
                   min(2 * x.pair + 2, (x.s.len + kTile - 1) / kTile), 0, x.s.len, 0, 1, 0};
      const TilePages now[2] = {next[0], next[1]};
      x.next();
      find();
      put_unit<kCall>(a, ctl->ring, nu++, u, lane, abort_flag);
      if (u.nt == 0) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (u.tile0 + i >= u.tile1) break;
        const int ks = nk % KS;
        if (nk >= KS) wait(&ctl->kempty[ks], (nk / KS - 1) & 1);
        if (*abort_flag) break;
        load_key_tile(a, &mapK, smem_u32(smem + ks * kTileBytes), smem_u32(&ctl->kfull[ks]), now[i],
                      u.h, (u.tile0 + i) * kTile, lane, nullptr);
        seen_bad |= now[i].bad;
        ++nk;
      }
    }
    Unit last{};
    last.b = -1;
    put_unit<kCall>(a, ctl->ring, nu, last, lane, abort_flag);
    if (seen_bad && lane == 0) raise(a, PP_S_INDEX);
    if (lane == 0) {   // every copy lands before the CTA may exit (bounded waits)
#pragma unroll 1
      for (uint32_t i = nk > KS ? nk - KS : 0; i < nk; ++i)
        drain_phase(a, &ctl->kfull[i % KS], (i / KS) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer -----------------------------------------------------------------------
    if (lane == 0) {
      const uint32_t id = (1u << 4) | Num<T>::kMmaTypes | ((uint32_t)(kTile >> 4) << 24) |
                          ((uint32_t)(N_ >> 3) << 17);
      uint32_t nk = 0, nq = 0, n2 = 0;   // n2: steps of units with two tiles
      Unit x;
      auto scores = [&](uint32_t buf, int ks, uint32_t qb) {
        const uint32_t kb = smem_u32(smem + ks * kTileBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_bf16(tmem + buf * kTile, smem_desc(kb + (kk >> 2) * (kTile * 128) + (kk & 3) * 32),
                    smem_desc(qb + (kk >> 2) * (N_ * 128) + (kk & 3) * 32), id, kk > 0);
        umma_commit(smem_u32(&ctl->sfull[buf]));
      };
#pragma unroll 1
      for (uint32_t nu = 0; get_unit<kCall>(a, ctl->ring, nu, x, lane, true, abort_flag); ++nu) {
        if (x.nt == 0) continue;
        const bool two = x.tile1 - x.tile0 == 2;
        const int k0 = nk % KS, k1 = (nk + 1) % KS;
        wait(&ctl->kfull[k0], (nk / KS) & 1);
        if (two) wait(&ctl->kfull[k1], ((nk + 1) / KS) & 1);
        nk += two ? 2 : 1;
#pragma unroll 1
        for (int t = 0; t < x.nt; t += tp) {
          const int qs = nq % kQStages;
          const uint32_t b0 = (nq & 1) * 2, b1 = (n2 & 1) * 2 + 1;
          wait(&ctl->qfull[qs], (nq / kQStages) & 1);
          if (nq >= 2) wait(&ctl->sfree[b0], ((nq >> 1) - 1) & 1);
          if (*abort_flag) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t qb = smem_u32(q_smem + qs * q_bytes);
          scores(b0, k0, qb);
          if (two) {
            if (n2 >= 2) wait(&ctl->sfree[b1], ((n2 >> 1) - 1) & 1);
            if (*abort_flag) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            scores(b1, k1, qb);
            ++n2;
          }
          umma_commit(smem_u32(&ctl->qempty[qs]));
          ++nq;
        }
        umma_commit(smem_u32(&ctl->kempty[k0]));
        if (two) umma_commit(smem_u32(&ctl->kempty[k1]));
      }
      // every MMA is done before tensor memory is given back (bounded wait)
      umma_commit(smem_u32(&ctl->done));
      drain_phase(a, &ctl->done, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- old mass and pages: eight keys to a lane; a unit's loads are issued before the last
    // unit's values are handed on
    Unit x;
    float old[8] = {};
    int page = -1;
    bool have = false;
#pragma unroll 1
    for (uint32_t nu = 0;; ++nu) {
      float next[8] = {};
      int next_page = -1;
      const bool more = get_unit<kCall>(a, ctl->ring, nu, x, lane, false, abort_flag);
      if (more) {
        const int j = x.tile0 * kTile + lane * 8;        // one page: 8 divides the page size
        next_page = j < x.stop ? page_of(a, x.b, j) : -1;
        if (next_page >= 0 && decay != 0.f) {
          const float* src =
              mass + ((((int64_t)next_page * a.Hk + x.h) << a.lps) + (j & ((1 << a.lps) - 1)));
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (j + k < x.stop) next[k] = src[k];
        }
      }
      if (have) {
        const uint32_t n = nu - 1, us = n % kAux;
        if (n >= kAux) wait(&ctl->uempty[us], (n / kAux - 1) & 1);
        float4* to = reinterpret_cast<float4*>(&ctl->old[us][lane * 8]);
        to[0] = make_float4(old[0] * decay, old[1] * decay, old[2] * decay, old[3] * decay);
        to[1] = make_float4(old[4] * decay, old[5] * decay, old[6] * decay, old[7] * decay);
        if ((lane & 1) == 0) ctl->page[us][lane >> 1] = page;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->ufull[us]));
      }
      if (!more) break;
      have = true;
      page = next_page;
#pragma unroll
      for (int k = 0; k < 8; ++k) old[k] = next[k];
    }
  } else if (warp == 3) {
    // ---- the steps' rows by TMA, and lse: four rows to a lane; a step's loads are issued before
    // the last step's values are handed on
    const int H = a.Hk * a.G;
    int tk[4], gh[4];                                   // a lane's rows: token and head of a step
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      tk[k] = (lane + k * 32) / a.G;
      gh[k] = lane + k * 32 - tk[k] * a.G;
    }
    Unit x;
    float z[4] = {};
    uint32_t nl = 0;
    bool have = false;
    auto hand_on = [&](uint32_t n) {
      const int ls = n % kAux;
      if (n >= kAux) wait(&ctl->lempty[ls], (n / kAux - 1) & 1);
      // rows that are not there, or that saw nothing, give nothing
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ctl->ref[ls][lane + k * 32] = z[k] == -INFINITY ? -INFINITY : z[k] * -kLog2e;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->lfull[ls]));
    };
#pragma unroll 1
    for (uint32_t nu = 0; get_unit<kCall>(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
#pragma unroll 1
      for (int t = 0; t < x.nt && !*abort_flag; t += tp, ++nl) {
        const int nt = min(tp, x.nt - t), qs = nl % kQStages;
        if (nl >= kQStages) wait(&ctl->qempty[qs], (nl / kQStages - 1) & 1);
        if (*abort_flag) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&ctl->qfull[qs]);
          mbar_expect_tx(bar, (uint32_t)(tp * a.G * D * 2));
          for (int bx = 0; bx < D / 64; ++bx)
            tma_load_4d(smem_u32(q_smem + qs * q_bytes + bx * N_ * 128), &mapQ, bx * 64, x.h * a.G,
                        x.row + t, 0, bar);
        }
        float next[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          next[k] = tk[k] < nt ? lse[(int64_t)(x.row + t + tk[k]) * H + x.h * a.G + gh[k]]
                               : -INFINITY;
        if (have) hand_on(nl - 1);
        have = true;
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = next[k];
      }
      // the last step of a unit is handed on at once: the next unit may be far off
      if (have) hand_on(nl - 1);
      have = false;
    }
    if (lane == 0) {   // every copy lands before the CTA may exit (bounded waits)
#pragma unroll 1
      for (uint32_t i = nl > kQStages ? nl - kQStages : 0; i < nl; ++i)
        drain_phase(a, &ctl->qfull[i % kQStages], (i / kQStages) & 1);
    }
    __syncwarp();
  } else {
    // ---- sums: a thread to a key, a group to a tile -----------------------------------------
    const int g = (warp - 4) >> 2, key = threadIdx.x - 128;
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t c2 = f32x2(a.c, a.c);
    uint32_t nl = 0, ns = 0;           // steps; this group's
    Unit x;
#pragma unroll 1
    for (uint32_t nu = 0; get_unit<kCall>(a, ctl->ring, nu, x, lane, false, abort_flag); ++nu) {
      const int j0 = (x.tile0 + g) * kTile, j = x.tile0 * kTile + key;
      const bool mine = x.tile0 + g < x.tile1;
      float sum = 0.f;
#pragma unroll 1
      for (int t = 0; t < x.nt; t += tp, ++nl) {
        const int ls = nl % kAux;
        wait(&ctl->lfull[ls], (nl / kAux) & 1);
        if (mine) {
          const uint32_t buf = (ns & 1) * 2 + g;
          const int nt = min(tp, x.nt - t), cols = nt * a.G, first = x.first + t;
          // the rows of the step that see this key: columns [lo, hi)
          int lo = 0, hi = cols;
          const bool edge = (cols % W) || j0 + kTile - 1 > first ||
                            (a.window && j0 <= first + nt - 1 - a.window);
          if (edge) {
            lo = (int)min((int64_t)cols, (int64_t)max(0, j - first) * a.G);
            if (a.window) {
              const int64_t end = ((int64_t)j + a.window - first) * a.G;
              hi = (int)max((int64_t)0, min((int64_t)hi, end));
            }
          }
          wait(&ctl->sfull[buf], (ns >> 1) & 1);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t s_at = at + buf * kTile;
          float w = 0.f;
          // a NaN may come from a row of no sum: once more without them.  (Steps of 32 columns and more
          // do that apart: comparing refs in all their masked sums took 107 us against 104 on the 4 x
          // 300 rows.)
          if constexpr (W == 16) {
            if (!edge) w = weigh<W>(s_at, ctl->ref[ls], c2, cols, lo, hi, std::false_type());
            if (edge || __any_sync(0xffffffffu, w != w))
              w = weigh<W>(s_at, ctl->ref[ls], c2, cols, lo, hi, std::true_type());
          } else {
            if (edge)
              w = weigh<W>(s_at, ctl->ref[ls], c2, cols, lo, hi, std::true_type());
            else
              w = weigh<W>(s_at, ctl->ref[ls], c2, cols, lo, hi, std::false_type());
            if (__any_sync(0xffffffffu, w != w))
              w = weigh_live(s_at, ctl->ref[ls], c2, cols, lo, hi);
          }
          sum += w;
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->sfree[buf]));
          ++ns;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->lempty[ls]));
      }
      const int us = nu % kAux;
      wait(&ctl->ufull[us], (nu / kAux) & 1);
      const int p = ctl->page[us][key >> 4];
      sum += ctl->old[us][key];
      if (p >= 0 && j < x.stop)
        mass[(((int64_t)p * a.Hk + x.h) << a.lps) + (j & ((1 << a.lps) - 1))] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->uempty[us]));
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
  const int fixed = (int)(sizeof(Ctl) + (a.n_seqs + 1) * sizeof(int64_t)) + 1024 + kQStages * q_bytes;
  constexpr int most_smem = 227 * 1024;
  int ks = (most_smem - fixed) / tile;
  if (ks > kMaxStages) ks = kMaxStages;
  const size_t smem = (size_t)fixed + (size_t)ks * tile;
  // a few rows go 16 columns at a time (the others may not be there at all), many 32
  const auto kernel = n <= 16 ? k_paged_mass<T, D, 16> : k_paged_mass<T, D, 32>;
  static std::atomic<uint64_t> done[2] = {};
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), most_smem, done[n <= 16]);
  if (err != cudaSuccess) return err;
  const int nsm = sm_count();
  const int64_t tiles = (((int64_t)a.table_ld << a.lps) + kTile - 1) / kTile;
  const int64_t most = (int64_t)a.n_seqs * a.Hk * tiles;
  return launch(kernel, dim3((unsigned)(most < nsm ? most : nsm)), kThreads, smem, s, a, tp, n, ks,
                lse, mass, decay, maps.k, maps.q);
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
