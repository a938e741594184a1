// k_paged_cache.cu - what goes into the paged cache and what leaves it.
//
// k_paged_append: for each head of a new token's queries and keys
//   y = x / sqrt(mean(x^2) + eps) * alpha   (left out without alpha), then each pair
//   (y_a, y_b) of the first `rot` dims turned by position * base^(-2i/rot);
// queries to a plain array, keys and values into the token's cache entry.  One rounding, at
// the end.  The angle's turns are a 64-bit product modulo 2^64, that is modulo a whole
// turn, so far positions lose nothing to a float's mantissa.
//
// k_paged_select / k_paged_move: the entries that stay - the newest `recent` and of the
// others the heaviest, lower index first among equals - in their old order into the
// destination's pages.  The threshold weight is found a few bits at a time (radix selection
// over order-preserving integers), so no sort is needed.
#include <cooperative_groups.h>

#include "pp_paged.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 4;        // heads of a token whose loads a thread has in flight

// 8 consecutive values (16-byte loads), and as floats
template <typename I>
struct Raw {
  uint4 w[sizeof(I) / 2];
  __device__ __forceinline__ void load(const I* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(I) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void values(float x[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(I) == 4)
        x[i] = __uint_as_float(u[i]);
      else
        x[i] = Num<I>::to_float(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xffffu);
    }
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, const float x[8]) {
  uint4 a;
  a.x = Num<T>::pack(x[0], x[1]);
  a.y = Num<T>::pack(x[2], x[3]);
  a.z = Num<T>::pack(x[4], x[5]);
  a.w = Num<T>::pack(x[6], x[7]);
  *reinterpret_cast<uint4*>(p) = a;
}

// One CTA to a token, D/8 lanes to a head.  Bound by reading and writing the rows once: the
// first heads' loads go out before the token's place in the cache is known, whose chain of
// lookups (row offsets, length, page) they hide.
// Measured (in a graph): 4 sequences of up to 6000 tokens, 6021 in all, 32 + 2 x 8 heads of 128
// dims, bf16: 43 us, 3.5 TB/s (39 without the norm, 50 with halves); fp32 in: 53 us, 4.2 TB/s; 64
// tokens of 32 + 2 x 32 heads, fp32 in: 6 us.  Bound by a CTA's chain (loads, lookups, angles, norm,
// stores), of which four to an SM overlap: 64 registers a thread (at 114, two CTAs, 65 us; at 48,
// five, they spill).  Halves through shared
// memory took 75 us.  (Ten tokens to a CTA with the next one's loads ahead: no faster, and slower
// for few tokens.)
template <typename I, typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, sizeof(I) == 2 ? 4 : 3)
    k_paged_append(const __grid_constant__ Args a, const __grid_constant__ AppendArgs x,
                   const __grid_constant__ Turns turns) {
  constexpr int L = D / 8;                       // lanes of one head
  constexpr int kHeads = kAppendThreads / L;     // heads side by side
  __shared__ float2 cs[D / 2];
  __shared__ float row[kHeads][D + 4];
  __shared__ int found, entry;          // the token's sequence and cache entry
  pdl_wait_and_trigger();
  pdl_trigger();
  const int t = blockIdx.x, H = a.Hk * a.G, rows = H + 2 * a.Hk;
  const int group = threadIdx.x / L, l = threadIdx.x % L;
  Raw<I> raw[kAppendRows];
  auto load = [&](int r0) {                      // queries, then keys, then values
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
      const int r = r0 + i * kHeads + group;
      if (r >= rows) break;
      const I* src = r < H ? reinterpret_cast<const I*>(x.q) + t * x.q_stride + r * D
                     : r < H + a.Hk
                         ? reinterpret_cast<const I*>(x.k) + t * x.k_stride + (r - H) * D
                         : reinterpret_cast<const I*>(x.v) + t * x.v_stride + (r - H - a.Hk) * D;
      raw[i].load(src + l * 8);
    }
  };
  load(0);
  // the token's sequence: a thread to each
  const int given = x.positions ? x.positions[t] : 0;
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < a.n_seqs; b += kAppendThreads) {
    const Seq s = seq_of(a, b);
    if (t >= s.row0 && t < s.row0 + s.n) {
      found = b;
      entry = s.total - s.n + (t - s.row0);
    }
  }
  __syncthreads();
  const int b = found, j = entry;
  if (b < 0) return;                             // a row of no sequence
  const int page = j >= 0 && j < table_entries(a) ? page_of(a, b, j) : -1;
  const int in_page = j & ((1 << a.lps) - 1);
  if (j >= 0 && page < 0 && threadIdx.x == 0) raise(a, PP_S_INDEX);
  const int pos = x.positions ? given : j;
  // partners half a rotation apart: in one lane's same place if that is a multiple of 8 dims (then
  // cs lies by places, for lanes to read neighbouring words)
  const int half = x.rot / 2;
  const bool by_lane = x.halves && (half & 7) == 0;
  for (int i = threadIdx.x; i < half; i += kAppendThreads) {
    const uint64_t angle = (uint64_t)(int64_t)pos * turns.f[i];
    float sn, cn;
    sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &sn, &cn);
    cs[by_lane ? (i & 7) * (D / 16) + (i >> 3) : i] = make_float2(cn, sn);
  }
  __syncthreads();
  float2 turn[4];                                // of this thread's neighbouring pairs
#pragma unroll
  for (int e = 0; e < 4; ++e) turn[e] = !x.halves && l * 8 + 2 * e < x.rot ? cs[l * 4 + e] : float2{};
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += kAppendRows * kHeads) {
    if (r0 > 0) load(r0);
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
      // (a warp's heads are consecutive: past the last row together, but for the lanes that
      // share its shuffles)
      const int r = r0 + i * kHeads + group;
      if (r - (int)(threadIdx.x % 32) / L >= rows) break;
      const bool live = r < rows;
      const int kind = r < H ? 0 : r < H + a.Hk ? 1 : 2;   // query, key, value
      const int h = kind == 0 ? r : kind == 1 ? r - H : r - H - a.Hk;
      float y[8] = {};
      if (live) raw[i].values(y);
      const float* alpha = kind == 0 ? x.q_alpha : kind == 1 ? x.k_alpha : nullptr;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (live && alpha) {
        const float inv = rsqrtf(ss * (1.f / D) + x.eps);   // off by 2^-22 at most
        const float4 a0 = reinterpret_cast<const float4*>(alpha + l * 8)[0];
        const float4 a1 = reinterpret_cast<const float4*>(alpha + l * 8)[1];
        const float al[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * al[e];
      }
      if (by_lane) {
        const int hl = half / 8, lane = threadIdx.x & 31;
        const bool lo = l < hl, in = l < 2 * hl;
        const int from = !in ? lane : lo ? lane + hl : lane - hl, place = lo ? l : l - hl;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = __shfl_sync(0xffffffffu, y[e], from);
          if (!in || kind == 2) continue;
          const float2 w = cs[e * (D / 16) + place];
          y[e] = lo ? y[e] * w.x - o * w.y : o * w.y + y[e] * w.x;
        }
      } else if (x.halves) {
        // any distance: through shared memory
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) row[group][l * 8 + e] = y[e];
        __syncwarp();
        if (kind != 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int d = l * 8 + e;
            if (d >= x.rot) continue;
            const bool lo = d < half;
            const float2 w = cs[lo ? d : d - half];
            const float o = row[group][lo ? d + half : d - half];
            y[e] = lo ? y[e] * w.x - o * w.y : o * w.y + y[e] * w.x;
          }
        }
      } else if (kind != 2) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int d = l * 8 + e;
          if (d >= x.rot) continue;
          const float2 w = turn[e / 2];
          const float p = y[e], o = y[e + 1];
          y[e] = p * w.x - o * w.y;
          y[e + 1] = p * w.y + o * w.x;
        }
      }
      if (!live) continue;
      if (kind == 0) {
        store8(reinterpret_cast<T*>(x.q_out) + ((int64_t)t * H + h) * D + l * 8, y);
      } else if (page >= 0) {
        T* pool = reinterpret_cast<T*>(kind == 1 ? x.k_pages : x.v_pages);
        store8(pool + page * a.page_stride + (((int64_t)h << a.lps) + in_page) * D + l * 8, y);
        if (kind == 1 && x.mass && l == 0)
          x.mass[(((int64_t)page * a.Hk + h) << a.lps) + in_page] = 0.f;
      }
    }
  }
}

// ---- eviction --------------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 44 * 1024;   // weights that a CTA holds on chip; longer slices are read again
constexpr int kBins = 4096;           // of the first 12 bits; then twice 1024 of 10 bits

// Order-preserving integer of a weight: larger weight, larger integer; NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One cluster of CTAs to a (sequence, key head), a slice of the older entries to a CTA.  Each
// round counts the next bits of the keys that still match, adds the CTAs' counts up through
// distributed shared memory and finds, in every CTA alike, the digit of the last key to stay.
// With the copy below: 16 sequences x 32 heads of 128 dims, up to 3000 entries down to 1500: 109
// us, 5.3 TB/s; 2 x 8, 40000 entries down to 5001, pages of 16: 36 us (one CTA to a pair: 100).
// Few pairs are bound by the rounds' latency (three, each with three cluster barriers), many by
// the copy.
__global__ void __launch_bounds__(kSelThreads)
    k_paged_select(const __grid_constant__ Args a, const __grid_constant__ EvictArgs x,
                   const int cluster_size) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t sums[kBins], share_sum;
  __shared__ uint32_t scan[kSelWarps], pick[2];       // digit, wanted among its keys
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps], total[2];   // larger keys, equal ones
  const cg::cluster_group cluster = cg::this_cluster();
  pdl_wait_and_trigger();
  pdl_trigger();
  const int pair = blockIdx.x / cluster_size, rank = blockIdx.x % cluster_size;
  const int b = pair / a.Hk, h = pair - b * a.Hk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = seq_len(a, b);
  const int m = min(len, x.budget);
  const int safe = min(x.recent, len);
  const int old = len - safe;                       // entries that compete
  const uint32_t want = (uint32_t)(m - safe);       // of which this many stay
  int32_t* kept = x.kept + (int64_t)pair * x.budget;
  const int step = cluster_size * kSelThreads, first = rank * kSelThreads + tid;
  if (h == 0 && first == 0) {
    x.to_len[b] = m;
    if (a.len[b] > len) raise(a, PP_S_INDEX);
  }
  for (int i = m + first; i < x.budget; i += step) kept[i] = -1;
  if (m == len) {
    for (int i = first; i < m; i += step) kept[i] = i;
    return;
  }
  for (int i = first; i < safe; i += step) kept[m - safe + i] = old + i;
  if (want == 0) return;
  // this CTA's slice; entries of pages outside the pool count as the lowest
  const int j0 = (int)((int64_t)old * rank / cluster_size);
  const int n = (int)((int64_t)old * (rank + 1) / cluster_size) - j0;
  auto weight = [&](int i) {
    const int j = j0 + i, p = page_of(a, b, j);
    return p < 0 ? 0u
                 : weight_key(x.mass[(((int64_t)p * a.Hk + h) << a.lps) + (j & ((1 << a.lps) - 1))]);
  };
  const bool on_chip = n <= kSelKeys;
  if (on_chip) {
#pragma unroll 4
    for (int i = tid; i < n; i += kSelThreads) keys[i] = weight(i);
  }
  auto key = [&](int i) { return on_chip ? keys[i] : weight(i); };

  // ---- the want-th largest key
  uint32_t prefix = 0, left = want;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = 20 - 10 * round, bits = round == 0 ? 12 : 10, bins = 1 << bits;
    for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = key(i);
      if (round == 0 || (k >> (shift + bits)) == prefix)
        atomicAdd(&hist[(k >> shift) & (uint32_t)(bins - 1)], 1u);
    }
    cluster.sync();
    // a CTA adds up its share of the bins over all CTAs (each thread neighbouring words, as
    // distributed shared memory likes them) ...
    const int share = bins / cluster_size;
    uint32_t sum = 0;
    for (int i = tid; i < share; i += kSelThreads) {
      uint32_t c = 0;
      for (int r = 0; r < cluster_size; ++r) c += cluster.map_shared_rank(hist, r)[rank * share + i];
      sums[i] = c;
      sum += c;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) scan[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const uint32_t c = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? scan[lane] : 0u);
      if (lane == 0) share_sum = c;
    }
    cluster.sync();
    // ... then all of them find the share, and in it the bin, of the left-th key from the top
    uint32_t above = 0;
    int at = cluster_size - 1;
    for (;; --at) {
      const uint32_t c = *cluster.map_shared_rank(&share_sum, at);
      if (at == 0 || above + c >= left) break;
      above += c;
    }
    const uint32_t* counts = cluster.map_shared_rank(sums, at);
    const int run = (share + kSelThreads - 1) / kSelThreads;   // 8, 4, 2 or 1 bins to a thread
    const int top = share - 1 - tid * run;            // this thread's highest bin
    uint32_t c[kBins / kSelThreads];
    sum = 0;
#pragma unroll
    for (int e = 0; e < kBins / kSelThreads; ++e) {
      c[e] = e < run && top - e >= 0 ? counts[top - e] : 0u;
      sum += c[e];
    }
    uint32_t over = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, over, o);
      if (lane >= o) over += y;
    }
    if (lane == 31) scan[warp] = over;
    __syncthreads();
    above += over - sum;
    above += __reduce_add_sync(0xffffffffu, lane < warp ? scan[lane] : 0u);
    if (above < left && left <= above + sum) {
#pragma unroll
      for (int e = 0; e < kBins / kSelThreads; ++e) {
        if (above < left && left <= above + c[e]) {
          pick[0] = (uint32_t)(at * share + top - e);
          pick[1] = left - above;
        }
        above += c[e];
      }
    }
    cluster.sync();                                   // also: every CTA has read every count
    prefix = (prefix << bits) | pick[0];
    left = pick[1];
  }

  // ---- larger keys stay, and of the equal ones the first `left`, in index order
  const int part = (n + kSelWarps - 1) / kSelWarps;   // a run of the slice to each warp
  const int i0 = min(warp * part, n), i1 = min(i0 + part, n);
  int gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = key(i);
    gt += k > prefix;
    eq += k == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const int g = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? warp_gt[lane] : 0);
    const int e = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? warp_eq[lane] : 0);
    if (lane == 0) {
      total[0] = g;
      total[1] = e;
    }
  }
  cluster.sync();
  // equal keys, and entries that stay, before this warp's run
  int ties = 0, at = 0;
  auto pass = [&](int g, int e) {
    at += g + min(max((int)left - ties, 0), e);
    ties += e;
  };
  for (int r = 0; r < rank; ++r) {
    const int* remote = cluster.map_shared_rank(total, r);
    pass(remote[0], remote[1]);
  }
  for (int w = 0; w < warp; ++w) pass(warp_gt[w], warp_eq[w]);
  const unsigned below = (1u << lane) - 1u;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0u;
    const bool tie = i + lane < i1 && k == prefix;
    const unsigned eqs = __ballot_sync(0xffffffffu, tie);
    const bool stay = i + lane < i1 &&
                      (k > prefix || (tie && ties + __popc(eqs & below) < (int)left));
    const unsigned stays = __ballot_sync(0xffffffffu, stay);
    if (stay) kept[at + __popc(stays & below)] = j0 + i + lane;
    ties += __popc(eqs);
    at += __popc(stays);
  }
  cluster.sync();                                     // no CTA leaves while its totals are read
}

// Copy the entries that stay: a group of D/8 lanes to an entry and 16 bytes to a lane.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;        // destination entries of one CTA

template <int D>
__global__ void __launch_bounds__(kMoveThreads)
    k_paged_move(const __grid_constant__ Args a, const __grid_constant__ EvictArgs x, const int blocks) {
  constexpr int L = D / 8;
  pdl_wait_and_trigger();
  pdl_trigger();
  const int bh = blockIdx.x / blocks, block = blockIdx.x - bh * blocks, b = bh / a.Hk, h = bh % a.Hk;
  const int m = min(seq_len(a, b), x.budget);
  const int32_t* kept = x.kept + (int64_t)bh * x.budget;
  const int l = threadIdx.x % L;
  const int end = min(m, (block + 1) * kMoveRows);
  for (int i = block * kMoveRows + threadIdx.x / L; i < end; i += kMoveThreads / L) {
    const int j = kept[i];
    const int p = page_of(a, b, j);
    const int q = x.to_table[(int64_t)b * x.to_table_ld + (i >> x.to_lps)];
    if (p < 0 || (unsigned)q >= (unsigned)x.to_n_pages) {
      if (l == 0) raise(a, PP_S_INDEX);
      continue;
    }
    const int64_t from = p * a.page_stride +
                         (((int64_t)h << a.lps) + (j & ((1 << a.lps) - 1))) * D + l * 8;
    const int64_t to = q * x.to_page_stride +
                       (((int64_t)h << x.to_lps) + (i & ((1 << x.to_lps) - 1))) * D + l * 8;
    const uint4 kk = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x.k) + from);
    const uint4 vv = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x.v) + from);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(x.to_k) + to) = kk;
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(x.to_v) + to) = vv;
    if (l == 0 && x.to_mass)
      x.to_mass[(((int64_t)q * a.Hk + h) << x.to_lps) + (i & ((1 << x.to_lps) - 1))] =
          x.mass[(((int64_t)p * a.Hk + h) << a.lps) + (j & ((1 << a.lps) - 1))];
  }
}

template <typename I, typename T>
cudaError_t append(const Args& a, const AppendArgs& x, const Turns& turns, cudaStream_t s) {
  if (a.D == 128)
    return launch(k_paged_append<I, T, 128>, dim3((unsigned)a.T), kAppendThreads, 0, s, a, x, turns);
  return launch(k_paged_append<I, T, 64>, dim3((unsigned)a.T), kAppendThreads, 0, s, a, x, turns);
}

}  // namespace

cudaError_t launch_paged_append(const Args& a, const AppendArgs& x, const Turns& turns, int in_type,
                                int type, cudaStream_t s) {
  if (type == PP_BF16)
    return in_type == PP_F32 ? append<float, __nv_bfloat16>(a, x, turns, s)
                             : append<__nv_bfloat16, __nv_bfloat16>(a, x, turns, s);
  return in_type == PP_F32 ? append<float, __half>(a, x, turns, s)
                           : append<__half, __half>(a, x, turns, s);
}

cudaError_t launch_paged_evict(const Args& a, const EvictArgs& x, cudaStream_t s) {
  const int pairs = a.n_seqs * a.Hk;
  const int64_t entries = (int64_t)a.table_ld << a.lps;
  // CTAs to a pair: enough for two on every SM, while a slice keeps two entries to a thread
  int cluster = 1;
  while (cluster < 8 && pairs * cluster * 2 <= 2 * kSms &&
         entries >= (int64_t)cluster * 2 * 2 * kSelThreads)
    cluster *= 2;
  const int64_t slice = (entries + cluster - 1) / cluster;
  const size_t smem = (size_t)(slice < kSelKeys ? slice : kSelKeys) * sizeof(uint32_t);
  static std::atomic<uint64_t> done{0};
  cudaError_t err = allow_smem(reinterpret_cast<const void*>(k_paged_select),
                               kSelKeys * (int)sizeof(uint32_t), done);
  if (err != cudaSuccess) return err;
  err = launch_cluster(cluster, k_paged_select, dim3((unsigned)(pairs * cluster)), kSelThreads, smem,
                       s, a, x, cluster);
  const int64_t most = entries < x.budget ? entries : x.budget;
  if (err != cudaSuccess || most == 0) return err;
  const int blocks = (int)((most + kMoveRows - 1) / kMoveRows);
  const dim3 grid((unsigned)((int64_t)blocks * pairs));
  return a.D == 128 ? launch(k_paged_move<128>, grid, kMoveThreads, 0, s, a, x, blocks)
                    : launch(k_paged_move<64>, grid, kMoveThreads, 0, s, a, x, blocks);
}

}  // namespace paged
}  // namespace pp
