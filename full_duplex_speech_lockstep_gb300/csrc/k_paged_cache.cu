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
// destination's pages.  The threshold weight is found byte by byte (radix selection over
// order-preserving integers), so no sort is needed.
#include "pp_paged.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kAppendThreads = 128;

// 8 consecutive values as floats (16-byte loads)
__device__ __forceinline__ void load8(const float* p, float x[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float x[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = Num<T>::to_float(w[i] & 0xffffu);
    x[2 * i + 1] = Num<T>::to_float(w[i] >> 16);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float x[8]) {
  uint4 a;
  a.x = Num<T>::pack(x[0], x[1]);
  a.y = Num<T>::pack(x[2], x[3]);
  a.z = Num<T>::pack(x[4], x[5]);
  a.w = Num<T>::pack(x[6], x[7]);
  *reinterpret_cast<uint4*>(p) = a;
}

// One CTA to a token; D/8 lanes to a head.
template <typename I, typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
    k_paged_append(const __grid_constant__ Args a, const __grid_constant__ AppendArgs x, const __grid_constant__ Turns turns) {
  constexpr int L = D / 8;                       // lanes of one head
  __shared__ float2 cs[D / 2];
  __shared__ float row[kAppendThreads / L][D + 4];
  pdl_wait_and_trigger();
  pdl_trigger();
  const int t = blockIdx.x;
  // the token's sequence: how many end at or before it
  int before = 0;
  for (int b0 = 0; b0 < a.n_seqs; b0 += kAppendThreads) {
    const int b = b0 + threadIdx.x;
    before += __syncthreads_count(b < a.n_seqs && a.cu[b + 1] <= t);
  }
  if (before >= a.n_seqs || t < a.cu[before]) return;   // a row of no sequence
  const Seq s = seq_of(a, before);
  if (t < s.row0 || t >= s.row0 + s.n) return;
  const int j = s.len - s.n + (t - s.row0);             // the token's cache entry
  const int page = j >= 0 ? page_of(a, before, j) : -1;
  const int in_page = j & ((1 << a.lps) - 1);
  if (j >= 0 && page < 0 && threadIdx.x == 0) raise(a, PP_S_INDEX);
  const int pos = x.positions ? x.positions[t] : j;
  for (int i = threadIdx.x; i < x.rot / 2; i += kAppendThreads) {
    const uint64_t turn = (uint64_t)(int64_t)pos * turns.f[i];
    float sn, cn;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
  __syncthreads();
  const int H = a.Hk * a.G, group = threadIdx.x / L, l = threadIdx.x % L;
  const int half = x.rot / 2;
  for (int r0 = 0; r0 < H + 2 * a.Hk; r0 += kAppendThreads / L) {
    const int r = r0 + group;
    const bool live = r < H + 2 * a.Hk;
    const int kind = r < H ? 0 : r < H + a.Hk ? 1 : 2;   // query, key, value
    const int h = kind == 0 ? r : kind == 1 ? r - H : r - H - a.Hk;
    float y[8] = {};
    if (live) {
      const I* src = kind == 0 ? reinterpret_cast<const I*>(x.q) + t * x.q_stride
                   : kind == 1 ? reinterpret_cast<const I*>(x.k) + t * x.k_stride
                               : reinterpret_cast<const I*>(x.v) + t * x.v_stride;
      load8(src + h * D + l * 8, y);
    }
    const float* alpha = kind == 0 ? x.q_alpha : kind == 1 ? x.k_alpha : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (live && alpha) {
      const float inv = 1.f / sqrtf(ss * (1.f / D) + x.eps);
      float al[8];
      load8(alpha + l * 8, al);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * al[e];
    }
    if (x.halves) {
      // partners lie half a rotation apart, in another lane
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
        const float2 w = cs[d / 2];
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

// ---- eviction --------------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelKeys = 48 * 1024;   // weights held on chip; longer rows are read again

// Order-preserving integer of a weight: larger weight, larger integer; NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) k_paged_select(const __grid_constant__ Args a, const __grid_constant__ EvictArgs x) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[3];          // prefix, still wanted, spare
  __shared__ int warp_sum[33];
  pdl_wait_and_trigger();
  pdl_trigger();
  const int b = blockIdx.x / a.Hk, h = blockIdx.x % a.Hk, tid = threadIdx.x;
  const int len = seq_len(a, b);
  const int m = min(len, x.budget);
  const int safe = min(x.recent, len);
  const int old = len - safe;                       // entries that compete
  const uint32_t want = (uint32_t)(m - safe);       // of which this many stay
  int32_t* kept = x.kept + (int64_t)blockIdx.x * x.budget;
  if (h == 0 && tid == 0) x.to_len[b] = m;
  for (int i = m + tid; i < x.budget; i += kSelThreads) kept[i] = -1;
  if (m == len) {
    for (int i = tid; i < m; i += kSelThreads) kept[i] = i;
    return;
  }
  // weights of pages outside the pool count as the lowest
  auto weight = [&](int j) {
    const int p = page_of(a, b, j);
    return p < 0 ? 0u
                 : weight_key(x.mass[(((int64_t)p * a.Hk + h) << a.lps) + (j & ((1 << a.lps) - 1))]);
  };
  const bool on_chip = old <= kSelKeys;
  if (on_chip)
    for (int j = tid; j < old; j += kSelThreads) keys[j] = weight(j);
  auto key = [&](int j) { return on_chip ? keys[j] : weight(j); };
  // the want-th largest key, a byte at a time from the top
  uint32_t prefix = 0, left = want;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < old; j += kSelThreads) {
      const uint32_t k = key(j);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t sum = 0;
      int d = 255;
      while (d > 0 && sum + hist[d] < left) sum += hist[d--];
      pick[0] = (prefix << 8) | (uint32_t)d;
      pick[1] = left - sum;
    }
    __syncthreads();
    prefix = pick[0];
    left = pick[1];
  }
  // larger keys stay, and of the equal ones the first `left` (none when want is 0)
  if (want == 0) left = 0;
  int done = 0, ties = 0;
  for (int j0 = 0; j0 < len; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t k = j < old ? key(j) : 0u;
    const bool tie = j < old && k == prefix;
    bool stay = j < len && (j >= old || k > prefix);
    // ranks of the ties, then of those that stay, in index order
    for (int pass = 0; pass < 2; ++pass) {
      const bool f = pass == 0 ? tie : stay;
      const unsigned bal = __ballot_sync(0xffffffffu, f);
      if ((tid & 31) == 0) warp_sum[tid >> 5] = __popc(bal);
      __syncthreads();
      if (tid < 32) {
        int v = warp_sum[tid], s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, s, o);
          if (tid >= o) s += y;
        }
        warp_sum[tid] = s - v;
        if (tid == 31) warp_sum[32] = s;
      }
      __syncthreads();
      const int rank = warp_sum[tid >> 5] + __popc(bal & ((1u << (tid & 31)) - 1u));
      const int total = warp_sum[32];
      if (pass == 0) {
        if (tie && ties + rank < (int)left) stay = true;
        ties += total;
      } else {
        if (stay) kept[done + rank] = j;
        done += total;
      }
      __syncthreads();
    }
  }
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
  const size_t smem = (size_t)(entries < kSelKeys ? entries : kSelKeys) * sizeof(uint32_t);
  cudaError_t err = cudaFuncSetAttribute(k_paged_select,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  err = launch(k_paged_select, dim3((unsigned)pairs), kSelThreads, smem, s, a, x);
  const int64_t most = entries < x.budget ? entries : x.budget;
  if (err != cudaSuccess || most == 0) return err;
  const int blocks = (int)((most + kMoveRows - 1) / kMoveRows);
  const dim3 grid((unsigned)((int64_t)blocks * pairs));
  return a.D == 128 ? launch(k_paged_move<128>, grid, kMoveThreads, 0, s, a, x, blocks)
                    : launch(k_paged_move<64>, grid, kMoveThreads, 0, s, a, x, blocks);
}

}  // namespace paged
}  // namespace pp
