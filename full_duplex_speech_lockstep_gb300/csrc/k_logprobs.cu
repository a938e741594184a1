// k_logprobs.cu - log probabilities of given tokens, entropy and the likeliest alternatives.
//
// For a row of logits x (those that are finite), with m = max x, l = sum exp(x_i - m) and
// t = sum exp(x_i - m) (x_i - m):
//   log p_i = x_i - m - log l,   entropy = -sum p_i log p_i = log l - t / l.
// A thread's values lie in registers: their maximum first, then the sums; a longer row's threads take
// several blocks of them and rescale (m, l, t) when the maximum grows.
//
// The `top` largest: the maximum of each of 64 groups of threads is one of the row's values, so the
// top-th largest of the maxima bounds the row's top-th largest value from below.  What reaches the bound
// (a few more than `top`) is listed and put in order by counting.  Values and places make one 64-bit key,
// so that equal values go by their place and no two keys are equal.  Where too many reach the bound (long
// runs of equal values) the exact top-th key is found bit by bit.
//
// Bound by reading the logits once; an exponential a value costs nearly as much.  A row that a CTA's
// registers hold (up to 512 threads of eight 16-byte vectors) is one CTA's; longer rows are cut into
// slices, one to a CTA of a cluster of up to eight; rows of up to 1024 values are a warp's.
//
// Measured: 3001 rows of 32000 bf16 values with 20 alternatives and entropy 71 us (2.7 TB/s), 1024 rows of
// 2048 fp32 values with 4 alternatives 6.7 us, one row of 32000 fp32 values 6.3 us, 60896 rows of 14 fp32
// values with 5 alternatives 23 us.  Of the 71 us the loads and the sums (about 17 instructions a value) are
// half; the rest are a row's barriers and the listing and ordering of its alternatives, which only the SM's
// other CTA hides.
#include <cooperative_groups.h>

#include <type_traits>

#include "pp_paged.cuh"

namespace pp {
namespace logprobs {
namespace {

namespace cg = cooperative_groups;
using paged::Num;
using paged::exp2_approx;
using paged::kLog2e;

constexpr int kGroups = 64;           // of threads, for the bound
constexpr int kMost = 64;             // alternatives at most
static_assert(kMost <= kGroups, "the bound is one of the groups' maxima");
constexpr int kList = 1024;           // keys that may reach the bound before it is made exact
constexpr int kCluster = 8;
constexpr float kFar = -1e4f;         // a distance below the maximum that weighs nothing

struct Call {
  const void* x;
  int64_t ld, inner_ld, token_ld, rows;
  int inner, n, top, slice;
  const int32_t* tokens;
  float *logprob, *entropy;
  int32_t* top_tokens;
  float* top_logprobs;
  uint32_t* status;
};

struct Stat {
  float m, l, t;
};
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  // (without a finite value a side has no weight: -infinity less -infinity is a NaN, which fmaxf drops)
  const float da = fmaxf(a.m - m, kFar), db = fmaxf(b.m - m, kFar);
  const float fa = exp2_approx(da * kLog2e), fb = exp2_approx(db * kLog2e);
  return Stat{m, a.l * fa + b.l * fb, fa * fmaf(a.l, da, a.t) + fb * fmaf(b.l, db, b.t)};
}

// Of all lanes, the same bits in each of them; `most`: the maximum of groups of kGroup lanes
template <int kGroup, bool kEntropy>
__device__ __forceinline__ Stat warp_join(Stat s, float& most) {
  float m = s.m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o == kGroup) most = m;
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (kGroup == 32) most = m;
  const float d = fmaxf(s.m - m, kFar), f = exp2_approx(d * kLog2e);
  s.t = f * fmaf(s.l, d, s.t);
  s.l *= f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    s.l += __shfl_xor_sync(0xffffffffu, s.l, o);
    if (kEntropy) s.t += __shfl_xor_sync(0xffffffffu, s.t, o);
  }
  s.m = m;
  return s;
}

// Order of values as unsigned integers (0: below all); -0 counts as 0.
__device__ __forceinline__ uint32_t order(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ uint64_t key_of(float v, int place) {
  return (uint64_t)order(v) << 32 | (uint32_t)~place;
}

template <typename T>
__device__ __forceinline__ float load_value(const T* p) {
  if constexpr (sizeof(T) == 4)
    return *p;
  else
    return Num<T>::to_float(*reinterpret_cast<const uint16_t*>(p));
}
// Two values of a word (16 bits each), or the word itself
template <typename T>
__device__ __forceinline__ float value_at(uint32_t w, int e) {
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(w);
  else
    return Num<T>::to_float(e ? w >> 16 : w & 0xffffu);
}
// The larger of two words' values, half by half (a NaN loses)
template <typename T>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  } else {
    uint32_t r;
    if constexpr (Num<T>::kShift == 0.f)
      asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
      asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
}
// z += 0 w: stays zero while every value is finite
template <typename T>
__device__ __forceinline__ void probe(uint32_t& z, uint32_t w) {
  if constexpr (sizeof(T) == 4)
    z = __float_as_uint(fmaf(__uint_as_float(w), 0.f, __uint_as_float(z)));
  else
    Num<T>::probe(z, w);
}
// The word with -infinity for each value that is not finite; `bad` if one is a NaN or +infinity
template <typename T>
__device__ __forceinline__ uint32_t finite_word(uint32_t w, bool& bad) {
  if constexpr (sizeof(T) == 4) {
    const float v = __uint_as_float(w);
    bad |= !(v < INFINITY);
    return fabsf(v) < INFINITY ? w : 0xff800000u;
  } else {
    constexpr uint32_t exp = Num<T>::kExp, last = exp & (~exp + 1), none = (0x8000u | exp) * 0x10001u;
    // (one more on an exponent of ones carries into the sign's place)
    const uint32_t ones = ((w & exp * 0x10001u) + last * 0x10001u) >> 15 & 0x10001u, all = ones * 0xffffu;
    bad |= ((w ^ none) & all) != 0;
    w = (w & ~all) | (none & all);
    return w;
  }
}

// A thread's part of its CTA's slice [s0, s1) of a row: whole vectors from p0 on, and up to V - 1 values on
// either side of them, one to a thread.
template <typename T, int kThreads, int kVectors>
struct Slice {
  static constexpr int N = 4 / sizeof(T);                // values of a word
  static constexpr int V = 4 * N;                        // values of a vector
  static constexpr int kWords = kVectors * 4;
  uint32_t w[kWords];
  const uint4* body;
  int p0, nv;                                            // first place, vectors
  int tid, side;                                         // place of this thread's single value, or -1
  float single;

  __device__ __forceinline__ Slice(const T* x, int s0, int s1, int tid_) : tid(tid_) {
    const int skew = (int)((16 - (reinterpret_cast<uintptr_t>(x + s0) & 15)) & 15) / (int)sizeof(T);
    p0 = min(s0 + skew, s1);
    nv = (s1 - p0) / V;
    const int p1 = p0 + nv * V;
    side = tid < p0 - s0 ? s0 + tid : tid >= V && tid - V < s1 - p1 ? p1 + tid - V : -1;
    body = reinterpret_cast<const uint4*>(x + p0);
  }
  __device__ __forceinline__ bool whole() const { return nv <= kVectors * kThreads; }
  // A block of vectors; -infinity where there are none
  __device__ __forceinline__ void load(int v0) {
    constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : (0x8000u | Num16::kExp) * 0x10001u;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int v = v0 + u * kThreads + tid;
      const uint4 x = v < nv ? body[v] : make_uint4(none, none, none, none);
      w[4 * u] = x.x;
      w[4 * u + 1] = x.y;
      w[4 * u + 2] = x.z;
      w[4 * u + 3] = x.w;
    }
  }
  // The block's values that are not finite become -infinity.
  __device__ __forceinline__ void clean(int v0, bool& bad) {
    uint32_t z = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if (v0 + i / 4 * kThreads + tid < nv) probe<T>(z, w[i]);
    if ((z & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) == 0) return;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = finite_word<T>(w[i], bad);
  }
  __device__ __forceinline__ float largest() const {
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < kWords; ++i) m = max_word<T>(m, w[i]);
    return N == 1 ? value_at<T>(m, 0) : fmaxf(value_at<T>(m, 0), value_at<T>(m, 1));
  }
  // The block's share of (l, t) for the maximum m
  template <bool kEntropy>
  __device__ __forceinline__ void sums(Stat& s) const {
    const float ref = s.m == -INFINITY ? 0.f : -s.m;
    const uint64_t ref2 = paged::f32x2(ref, ref), log2e = paged::f32x2(kLog2e, kLog2e);
    uint64_t l2 = 0, t2 = 0;
#pragma unroll
    for (int i = 0; i < kWords; i += 2 / N) {
      uint64_t d = paged::add2(paged::f32x2(value_at<T>(w[i], 0), value_at<T>(w[N == 1 ? i + 1 : i], 1)), ref2);
      if constexpr (kEntropy)                            // (0 times minus infinity would be a NaN)
        d = paged::f32x2(fmaxf(paged::lo_of(d), kFar), fmaxf(paged::hi_of(d), kFar));
      const uint64_t e = paged::mul2(d, log2e);
      const uint64_t p = paged::f32x2(exp2_approx(paged::lo_of(e)), exp2_approx(paged::hi_of(e)));
      l2 = paged::add2(l2, p);
      if constexpr (kEntropy) t2 = paged::fma2(p, d, t2);
    }
    s.l += paged::lo_of(l2) + paged::hi_of(l2);
    if constexpr (kEntropy) s.t += paged::lo_of(t2) + paged::hi_of(t2);
  }
  // f(key) for each finite value from `least` on: its order above the complement of its place
  template <typename F>
  __device__ __forceinline__ void each(float least, F& f) {
    if (side >= 0 && fabsf(single) < INFINITY && single >= least) f(key_of(single, side));
#pragma unroll 1
    for (int v0 = 0; v0 < nv; v0 += kVectors * kThreads) {
      if (!whole()) load(v0);
      uint32_t hits = 0;                                 // vectors that reach it: hardly any
#pragma unroll
      for (int u = 0; u < kVectors; ++u) {
        const uint32_t m =
            max_word<T>(max_word<T>(w[4 * u], w[4 * u + 1]), max_word<T>(w[4 * u + 2], w[4 * u + 3]));
        const float most = N == 1 ? value_at<T>(m, 0) : fmaxf(value_at<T>(m, 0), value_at<T>(m, 1));
        if (most >= least && most > -INFINITY) hits |= 1u << u;
      }
#pragma unroll 1
      for (; hits; hits &= hits - 1) {
        const int u = __ffs(hits) - 1, place = p0 + (v0 + u * kThreads + tid) * V;
        uint32_t own[4];
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i == 0 || u == i) own[j] = w[4 * i + j];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float v = value_at<T>(own[i / N], i % N);
          if (fabsf(v) < INFINITY && v >= least) f(key_of(v, place + i));
        }
      }
    }
  }

 private:
  using Num16 = Num<typename std::conditional<sizeof(T) == 4, __half, T>::type>;
};
struct Keys {                         // from `least` on: counted, and listed if there is a list
  uint64_t least;
  uint64_t* list;
  int* count;
  int mine;
  __device__ __forceinline__ void operator()(uint64_t key) {
    if (key < least) return;
    if (!list) {
      ++mine;
      return;
    }
    const int at = atomicAdd(count, 1);
    if (at < kList) list[at] = key;
  }
};

template <int kThreads>
struct Shared {
  Stat stat[kThreads / 32];           // of the warps, then [0]: of the CTA
  __align__(16) float most[kGroups];  // the groups' maxima
  float bound;
  float chosen;                       // rank 0: the given token's value
  int token;
  int count;
  uint64_t list[kList];
  uint64_t best[kMost];               // this CTA's largest, in order; 0: none
  uint64_t all[kCluster * kMost];     // rank 0: everyone's
};

// The `top` largest of the `c` keys of `list`, in order (0: none).  By the whole CTA.
template <int kThreads>
__device__ __forceinline__ void put_in_order(const uint64_t* list, int c, uint64_t* out, int top) {
#pragma unroll 1
  for (int i = threadIdx.x; i < c; i += kThreads) {
    const uint64_t key = list[i];
    int above = 0;
#pragma unroll 4
    for (int k = 0; k < c; ++k) {
      const uint64_t other = list[k];
      above += other > key || (other == key && k < i);  // (only keys of 0 are equal)
    }
    if (above < top) out[above] = key;
  }
#pragma unroll 1
  for (int i = c + threadIdx.x; i < top; i += kThreads) out[i] = 0;
  __syncthreads();
}

template <typename T, int kThreads, int kVectors, bool kEntropy>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    k_logprobs(const __grid_constant__ Call a) {
  using S = Slice<T, kThreads, kVectors>;
  __shared__ Shared<kThreads> sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int size = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s0 = min(rank * a.slice, a.n), s1 = min(s0 + a.slice, a.n);
  const uint32_t row = blockIdx.x / (uint32_t)size, group_of = row / (uint32_t)a.inner;
  const int64_t r = row, group = group_of, in = row - group_of * (uint32_t)a.inner;
  const T* x = reinterpret_cast<const T*>(a.x) + group * a.ld + in * a.inner_ld;
  pdl_wait_and_trigger();
  pdl_trigger();
  S part(x, s0, s1, tid);
  part.load(0);
  part.single = part.side >= 0 ? load_value(x + part.side) : -INFINITY;
  if (tid == 0) sh.count = 0;

  bool bad = !(part.single < INFINITY);
  if (!(fabsf(part.single) < INFINITY)) part.single = -INFINITY;
  Stat s{part.single, part.single == -INFINITY ? 0.f : 1.f, 0.f};
#pragma unroll 1
  for (int v0 = 0; v0 < part.nv; v0 += kVectors * kThreads) {
    if (v0 > 0) part.load(v0);
    part.clean(v0, bad);
    const float m = part.largest();
    if (m > s.m) {
      const float d = fmaxf(s.m - m, kFar), f = exp2_approx(d * kLog2e);
      s.t = f * fmaf(s.l, d, s.t);
      s.l *= f;
      s.m = m;
    }
    part.template sums<kEntropy>(s);
  }
  if (bad && a.status) atomicOr(a.status, PP_S_NAN);
  float most;                                       // of this thread's group of kThreads / kGroups lanes
  s = warp_join<kThreads / kGroups, kEntropy>(s, most);
  if (lane == 0) sh.stat[warp] = s;
  if (a.top > 0 && tid % (kThreads / kGroups) == 0) sh.most[tid / (kThreads / kGroups)] = most;
  __syncthreads();
  if (warp == kThreads / 32 - 1) {                  // (the last warp: the first ones rank the maxima)
    float unused;
    const Stat y = warp_join<32, kEntropy>(
        lane < kThreads / 32 ? sh.stat[lane] : Stat{-INFINITY, 0.f, 0.f}, unused);
    __syncwarp();
    if (lane == 0) sh.stat[0] = y;
  }
  if (tid == kThreads - 64 && rank == 0 && a.logprob) {
    const int32_t token = a.tokens[group * a.token_ld + in];
    sh.token = token;
    if (token >= 0 && token < a.n) sh.chosen = load_value(x + token);
  }
  if (a.top > 0) {
    if (tid < kGroups) {
      const float mine = sh.most[tid];
      int above = 0;
#pragma unroll 4
      for (int i = 0; i < kGroups; i += 4) {
        const float4 y = *reinterpret_cast<const float4*>(&sh.most[i]);
        above += y.x > mine || (y.x == mine && i < tid);
        above += y.y > mine || (y.y == mine && i + 1 < tid);
        above += y.z > mine || (y.z == mine && i + 2 < tid);
        above += y.w > mine || (y.w == mine && i + 3 < tid);
      }
      if (above == a.top - 1) sh.bound = mine;
    }
    __syncthreads();
    const float bound = sh.bound;
    // Listed at once; or, where too many reach the bound, counted from keys that are made bit by bit, up
    // to the top-th largest, and listed from there.
    const uint64_t known = (uint64_t)order(bound) << 32;
    uint64_t least = 0;
    int c, bit = 64;
    Keys keys{0, sh.list, &sh.count, 0};
#pragma unroll 1
    for (;;) {
      part.each(bound, keys);
      if (keys.mine) atomicAdd(&sh.count, keys.mine);
      __syncthreads();
      c = sh.count;
      if (keys.list && c <= kList) break;
      if (!keys.list && c >= a.top) least = keys.least;
      __syncthreads();
      if (tid == 0) sh.count = 0;
      uint64_t at = least;
#pragma unroll 1
      while (--bit >= 0) {
        at = least | (uint64_t)1 << bit;
        if (at > known) break;                      // (at least `top` keys reach the bound)
        least = at;
      }
      keys = Keys{at, bit < 0 ? sh.list : nullptr, &sh.count, 0};
      __syncthreads();
    }
    put_in_order<kThreads>(sh.list, c, sh.best, a.top);
  } else {
    __syncthreads();
  }
  if (size > 1) {
    cluster.sync();
    if (rank == 0) {
      if (tid == 0) {
        Stat y = sh.stat[0];
#pragma unroll 1
        for (int i = 1; i < size; ++i) y = join(y, cluster.map_shared_rank(&sh, i)->stat[0]);
        sh.stat[0] = y;
      }
#pragma unroll 1
      for (int i = tid; i < size * a.top; i += kThreads)
        sh.all[i] = cluster.map_shared_rank(&sh, i / a.top)->best[i % a.top];
    }
    cluster.sync();                                 // the others' memory has been read
    if (rank > 0) return;
    if (a.top > 0) put_in_order<kThreads>(sh.all, size * a.top, sh.best, a.top);
  }
  const Stat y = sh.stat[0];
  const float log_l = logf(y.l);
  if (tid == 0) {
    if (a.logprob) {
      const int32_t token = sh.token;
      float lp = 0.f;
      if (token >= a.n) {
        if (a.status) atomicOr(a.status, PP_S_INDEX);
      } else if (token >= 0) {
        const float v = sh.chosen;
        lp = fabsf(v) < INFINITY ? (v - y.m) - log_l : -INFINITY;
      }
      a.logprob[r] = lp;
    }
    if (kEntropy) a.entropy[r] = y.l > 0.f ? fmaxf(log_l - y.t / y.l, 0.f) : 0.f;
  }
#pragma unroll 1
  for (int i = tid; i < a.top; i += kThreads) {
    const uint64_t key = sh.best[i];
    if (a.top_tokens) a.top_tokens[r * a.top + i] = key ? (int32_t)~(uint32_t)key : -1;
    if (a.top_logprobs)
      a.top_logprobs[r * a.top + i] =
          key ? (value_of((uint32_t)(key >> 32)) - y.m) - log_l : -INFINITY;
  }
}

// Rows of up to 32 V values: a warp to a row, lane l has places l, l + 32, ..; the alternatives one by one.
constexpr int kWarps = 8;
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps) k_logprobs_few(const __grid_constant__ Call a) {
  pdl_wait_and_trigger();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const uint32_t row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const uint32_t group = row / (uint32_t)a.inner, in = row - group * (uint32_t)a.inner;
  const T* x = reinterpret_cast<const T*>(a.x) + group * a.ld + in * a.inner_ld;
  const int32_t token = a.logprob ? a.tokens[group * a.token_ld + in] : -1;
  float v[V], m = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = i * 32 + lane < a.n ? load_value(x + i * 32 + lane) : -INFINITY;
  const float chosen = token >= 0 && token < a.n ? load_value(x + token) : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= !(v[i] < INFINITY);
    if (!(fabsf(v[i]) < INFINITY)) v[i] = -INFINITY;
    m = fmaxf(m, v[i]);
  }
  if (bad && a.status) atomicOr(a.status, PP_S_NAN);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, t = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float d = fmaxf(v[i] - m, kFar), p = exp2_approx(d * kLog2e);   // (without a finite value: 0)
    l += p;
    t = fmaf(p, d, t);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  const float log_l = logf(l);
  if (lane == 0) {
    if (a.logprob) {
      float lp = 0.f;
      if (token >= a.n) {
        if (a.status) atomicOr(a.status, PP_S_INDEX);
      } else if (token >= 0) {
        lp = fabsf(chosen) < INFINITY ? (chosen - m) - log_l : -INFINITY;
      }
      a.logprob[row] = lp;
    }
    if (a.entropy) a.entropy[row] = l > 0.f ? fmaxf(log_l - t / l, 0.f) : 0.f;
  }
  if (a.top == 0) return;
  uint32_t o[V], best[2] = {0, 0}, place[2] = {0, 0};   // the lane's values; alternatives lane and 32 + lane
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = v[i] == -INFINITY ? 0u : order(v[i]);
#pragma unroll 1
  for (int k = 0; k < a.top; ++k) {
    uint32_t most = 0, at = ~0u;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (o[i] >= most) {
        most = o[i];
        at = i * 32 + lane;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, most);
    if (top == 0) break;
    at = __reduce_min_sync(0xffffffffu, most == top ? at : ~0u);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at == i * 32 + lane) o[i] = 0;
    if (lane == (k & 31)) {
      best[k >> 5 & 1] = top;
      place[k >> 5 & 1] = at;
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int k = 32 * j + lane;
    if (k >= a.top) continue;
    if (a.top_tokens) a.top_tokens[(int64_t)row * a.top + k] = best[j] ? (int32_t)place[j] : -1;
    if (a.top_logprobs)
      a.top_logprobs[(int64_t)row * a.top + k] = best[j] ? (value_of(best[j]) - m) - log_l : -INFINITY;
  }
}

template <typename T, int kThreads, int kVectors>
cudaError_t run(Call a, cudaStream_t s) {
  constexpr int kBlock = kThreads * kVectors * 16 / (int)sizeof(T);
  int size = 1;
  while (size < kCluster && (int64_t)size * kBlock < a.n) size *= 2;
  a.slice = ((a.n + size - 1) / size + 7) / 8 * 8;  // (whole vectors, where the row is aligned)
  auto kern = a.entropy ? k_logprobs<T, kThreads, kVectors, true> : k_logprobs<T, kThreads, kVectors, false>;
  return paged::launch_cluster(size, kern, dim3((unsigned)(a.rows * size)), kThreads, 0, s, a);
}
template <typename T, int V>
cudaError_t run_few(const Call& a, cudaStream_t s) {
  return paged::launch(k_logprobs_few<T, V>, dim3((unsigned)((a.rows + kWarps - 1) / kWarps)), 32 * kWarps, 0,
                       s, a);
}
// By the row's length alone, so that a row's bits do not depend on the others.  20000 rows with 5 alternatives:
// of 1024 fp32 values by warps 47 us, by CTAs of 128 threads 76; of 2048 96 and 76; of 2049 by CTAs of 256
// threads 156, of 512 304.
template <typename T>
cudaError_t pick(const Call& a, cudaStream_t s) {
  constexpr int kVector = 16 / (int)sizeof(T);
  if (a.n <= 64) return run_few<T, 2>(a, s);
  if (a.n <= 256) return run_few<T, 8>(a, s);
  if (a.n <= 512) return run_few<T, 16>(a, s);
  if (a.n <= 1024) return run_few<T, 32>(a, s);
  if (a.n <= 128 * 4 * kVector) return run<T, 128, 4>(a, s);
  if (a.n <= 256 * 8 * kVector) return run<T, 256, 8>(a, s);
  return run<T, 512, 8>(a, s);
}

}  // namespace
}  // namespace logprobs
}  // namespace pp

using namespace pp;
using namespace pp::logprobs;

extern "C" int pp_token_logprobs(const void* logits, int type, int64_t ld, int rows, int inner,
                                 int64_t inner_ld, int n, const int32_t* tokens, int64_t token_ld,
                                 int top, float* logprob, float* entropy, int32_t* top_tokens,
                                 float* top_logprobs, uint32_t* status, void* stream) {
  if (type != PP_F32 && type != PP_BF16 && type != PP_F16) return PP_EINVAL;
  if (rows < 0 || inner < 1 || n < 1 || n > 1 << 24 || top < 0 || top > kMost) return PP_EINVAL;
  if ((int64_t)rows * inner >= (int64_t)1 << 28 || ld < 0 || inner_ld < 0 || token_ld < 0 ||
      ld >= (int64_t)1 << 38 || inner_ld >= (int64_t)1 << 38 || token_ld >= (int64_t)1 << 38)
    return PP_EINVAL;
  if (rows == 0) return PP_OK;
  const uintptr_t bytes = type == PP_F32 ? 4 : 2;
  auto off = [](const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; };
  if (!logits || off(logits, bytes) || off(tokens, 4) || off(logprob, 4) || off(entropy, 4) ||
      off(top_tokens, 4) || off(top_logprobs, 4) || (logprob && !tokens))
    return PP_EINVAL;
  // (without a place for them no alternative is looked for)
  Call a{logits, ld, inner_ld, token_ld, (int64_t)rows * inner, inner, n,
         top_tokens || top_logprobs ? top : 0, 0, tokens, logprob, entropy, top_tokens, top_logprobs, status};
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t err = type == PP_F32    ? pick<float>(a, s)
                          : type == PP_BF16 ? pick<__nv_bfloat16>(a, s)
                                            : pick<__half>(a, s);
  return err == cudaSuccess ? PP_OK : PP_E_CUDA;
}
