// k_logprobs.cu - log probabilities of given tokens, entropy and the likeliest alternatives.
//
// For a row of logits x (those that are finite), with m = max x, l = sum exp(x_i - m) and
// t = sum exp(x_i - m) (x_i - m):
//   log p_i = x_i - m - log l,   entropy = -sum p_i log p_i = log l - t / l.
// One pass: a thread keeps its own (m, l, t) and rescales them when its maximum grows.
//
// The `top` largest: every thread's maximum is one of the row's values, so the top-th largest of the
// maxima bounds the row's top-th largest value from below.  What reaches the bound (a few more than
// `top`) is listed and put in order by counting.  Values and places make one 64-bit key, so that
// equal values go by their place and no two keys are equal.  Where too many reach the bound (long runs
// of equal values) the exact top-th key is found bit by bit.
//
// Bound by reading the logits once: a row is cut into slices, one to a CTA of a cluster, of 8192
// values, or of an eighth of the row where that is more; a slice of 8192 stays in registers for its
// second look.
#include <cooperative_groups.h>

#include "pp_paged.cuh"

namespace pp {
namespace logprobs {
namespace {

namespace cg = cooperative_groups;
using paged::Num;
using paged::exp2_approx;
using paged::kLog2e;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 8192;          // values that a CTA's registers hold
constexpr int kMost = 64;             // alternatives at most
constexpr int kList = 1024;           // keys that may reach the bound before it is made exact
constexpr int kCluster = 8;
constexpr float kFar = -1e4f;         // a distance below the maximum that weighs nothing

struct Call {
  const void* x;
  int64_t ld, inner_ld, token_ld;
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

// N more values
template <int N>
__device__ __forceinline__ void take(const float (&y)[N], Stat& s, bool& bad) {
  float v[N], top = s.m;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    bad |= !(y[e] < INFINITY);
    v[e] = fabsf(y[e]) < INFINITY ? y[e] : -INFINITY;
    top = fmaxf(top, v[e]);
  }
  if (top > s.m) {
    const float d = fmaxf(s.m - top, kFar), f = exp2_approx(d * kLog2e);
    s.t = f * fmaf(s.l, d, s.t);
    s.l *= f;
    s.m = top;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float d = fmaxf(v[e] - s.m, kFar);        // (a NaN, minus infinity less itself, goes too)
    const float p = exp2_approx(d * kLog2e);
    s.l += p;
    s.t = fmaf(p, d, s.t);
  }
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
// Value e of a 16-byte vector
template <typename T>
__device__ __forceinline__ float value_at(const uint4& w, int e) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(u[e]);
  else
    return Num<T>::to_float(e & 1 ? u[e >> 1] >> 16 : u[e >> 1] & 0xffffu);
}

// A thread's part of its CTA's slice [s0, s1) of a row: whole vectors in [p0, ..), and up to V - 1 values
// on either side of them, one to a thread.
template <typename T>
struct Slice {
  static constexpr int V = 16 / sizeof(T);               // values of a vector
  static constexpr int U = kBlock / (kThreads * V);      // vectors of a thread, held in registers
  uint4 w[U];
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
  __device__ __forceinline__ void load(int v0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + u * kThreads + tid;
      if (v < nv) w[u] = body[v];
    }
  }
  // f(key) for each finite value: its order above the complement of its place
  template <typename F>
  __device__ __forceinline__ void each(F f) {
    if (side >= 0 && fabsf(single) < INFINITY) f(key_of(single, side));
#pragma unroll 1
    for (int v0 = 0; v0 < nv; v0 += U * kThreads) {
      if (nv > U * kThreads) load(v0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * kThreads + tid;
        if (v >= nv) break;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float y = value_at<T>(w[u], e);
          if (fabsf(y) < INFINITY) f(key_of(y, p0 + v * V + e));
        }
      }
    }
  }
};
struct ListFrom {                     // keys from `least` on into a list
  uint64_t least;
  int* count;
  uint64_t* list;
  __device__ __forceinline__ void operator()(uint64_t key) const {
    if (key < least) return;
    const int at = atomicAdd(count, 1);
    if (at < kList) list[at] = key;
  }
};
struct CountFrom {
  uint64_t least;
  int* count;
  __device__ __forceinline__ void operator()(uint64_t key) const { *count += key >= least; }
};

struct Shared {
  Stat stat[kWarps];                  // of the warps, then [0]: of the CTA
  uint64_t list[kList];
  uint64_t best[kMost];               // this CTA's largest, in order; 0: none
  uint64_t all[kCluster * kMost];     // rank 0: everyone's
  int count, found;
};

// Ranks the `c` keys of `list` and writes the first `top` in order (0: none).  By the whole CTA.
__device__ __forceinline__ void put_in_order(const uint64_t* list, int c, uint64_t* out, int top) {
  for (int i = threadIdx.x; i < top; i += kThreads) out[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < c; i += kThreads) {
    const uint64_t key = list[i];
    int above = 0;
    for (int k = 0; k < c; ++k) above += list[k] > key;
    if (key != 0 && above < top) out[above] = key;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_logprobs(const __grid_constant__ Call a) {
  constexpr int V = Slice<T>::V, U = Slice<T>::U;
  __shared__ Shared sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int size = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t r = blockIdx.x / size;              // the row
  const int64_t group = r / a.inner, in = r - group * a.inner;
  const T* x = reinterpret_cast<const T*>(a.x) + group * a.ld + in * a.inner_ld;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait_and_trigger();
  pdl_trigger();
  Slice<T> in_slice(x, min(rank * a.slice, a.n), min(rank * a.slice + a.slice, a.n), tid);
  uint4 (&w)[U] = in_slice.w;
  const int nv = in_slice.nv, side = in_slice.side;
  in_slice.load(0);
  const float single = in_slice.single = side >= 0 ? load_value(x + side) : -INFINITY;

  Stat s{-INFINITY, 0.f, 0.f};
  bool bad = false;
  if (side >= 0) {
    const float y[1] = {single};
    take<1>(y, s, bad);
  }
  for (int v0 = 0; v0 < nv; v0 += U * kThreads) {
    if (v0 > 0) in_slice.load(v0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (v0 + u * kThreads + tid >= nv) break;
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = value_at<T>(w[u], e);
      take<V>(y, s, bad);
    }
  }
  const float mine = s.m;                           // this thread's largest value
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat y{__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.l, o),
                 __shfl_xor_sync(0xffffffffu, s.t, o)};
    // the lower lane's side first, in both lanes
    s = (lane & o) ? join(y, s) : join(s, y);
  }
  if (lane == 0) sh.stat[warp] = s;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  if (tid == 0) {
    Stat y = sh.stat[0];
    for (int i = 1; i < kWarps; ++i) y = join(y, sh.stat[i]);
    sh.stat[0] = y;
  }
  if (bad && a.status) atomicOr(a.status, PP_S_NAN);

  if (a.top > 0) {
    const uint32_t most = mine == -INFINITY ? 0u : order(mine);
    // the top-th largest of the threads' maxima, by bits from the highest; 16 of them are enough for
    // a bound
    uint32_t bound = 0;
#pragma unroll 1
    for (int b = 31; b >= 16; --b) {
      const uint32_t at = bound | 1u << b;
      if (__syncthreads_count(most >= at) >= a.top) bound = at;
    }
    if (most >= bound) in_slice.each(ListFrom{(uint64_t)bound << 32, &sh.count, sh.list});
    __syncthreads();
    int c = sh.count;
    if (c > kList) {
      // the top-th largest key itself, bit by bit: at least `top` keys reach the bound
      uint64_t least = 0;
#pragma unroll 1
      for (int b = 63; b >= 0; --b) {
        const uint64_t at = least | (uint64_t)1 << b;
        if (at <= (uint64_t)bound << 32) {
          least = at;
          continue;
        }
        if (tid == 0) sh.found = 0;
        __syncthreads();
        int k = 0;
        in_slice.each(CountFrom{at, &k});
        if (k) atomicAdd(&sh.found, k);
        __syncthreads();
        if (sh.found >= a.top) least = at;
        __syncthreads();
      }
      if (tid == 0) sh.count = 0;
      __syncthreads();
      in_slice.each(ListFrom{least, &sh.count, sh.list});
      __syncthreads();
      c = sh.count;
    }
    put_in_order(sh.list, c, sh.best, a.top);
  } else {
    __syncthreads();
  }
  if (size > 1) {
    cluster.sync();
    if (rank == 0) {
      if (tid == 0) {
        Stat y = sh.stat[0];
        for (int i = 1; i < size; ++i) y = join(y, cluster.map_shared_rank(&sh, i)->stat[0]);
        sh.stat[0] = y;
      }
      for (int i = tid; i < size * a.top; i += kThreads)
        sh.all[i] = cluster.map_shared_rank(&sh, i / a.top)->best[i % a.top];
    }
    cluster.sync();                                 // the others' memory has been read
    if (rank > 0) return;
    if (a.top > 0) put_in_order(sh.all, size * a.top, sh.best, a.top);
  }
  __syncthreads();
  const Stat y = sh.stat[0];
  const float log_l = logf(y.l);
  if (tid == 0) {
    if (a.logprob) {
      const int32_t token = a.tokens[group * a.token_ld + in];
      float lp = 0.f;
      if (token >= a.n) {
        if (a.status) atomicOr(a.status, PP_S_INDEX);
      } else if (token >= 0) {
        const float v = load_value(x + token);
        lp = fabsf(v) < INFINITY ? (v - y.m) - log_l : -INFINITY;
      }
      a.logprob[r] = lp;
    }
    if (a.entropy) a.entropy[r] = y.l > 0.f ? fmaxf(log_l - y.t / y.l, 0.f) : 0.f;
  }
  for (int i = tid; i < a.top; i += kThreads) {
    const uint64_t key = sh.best[i];
    if (a.top_tokens) a.top_tokens[r * a.top + i] = key ? (int32_t)~(uint32_t)key : -1;
    if (a.top_logprobs)
      a.top_logprobs[r * a.top + i] =
          key ? (value_of((uint32_t)(key >> 32)) - y.m) - log_l : -INFINITY;
  }
}

template <typename T>
cudaError_t run(const Call& a, int64_t rows, int size, cudaStream_t s) {
  return paged::launch_cluster(size, k_logprobs<T>, dim3((unsigned)(rows * size)), kThreads, 0, s, a);
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
  Call a{logits, ld, inner_ld, token_ld, inner, n, top_tokens || top_logprobs ? top : 0, 0, tokens,
         logprob, entropy, top_tokens, top_logprobs, status};
  int size = 1;
  while (size < kCluster && (int64_t)size * kBlock < n) size *= 2;
  a.slice = ((n + size - 1) / size + 7) / 8 * 8;    // (whole vectors, where the row is aligned)
  const int64_t all = (int64_t)rows * inner;
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t err = type == PP_F32    ? run<float>(a, all, size, s)
                          : type == PP_BF16 ? run<__nv_bfloat16>(a, all, size, s)
                                            : run<__half>(a, all, size, s);
  return err == cudaSuccess ? PP_OK : PP_E_CUDA;
}
