// pp_paged.cuh - the paged cache as its kernels see it: sequences, rows, key tiles, page
// lookups, and the tile loads, matrix fragments and masks that they share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "pp_async.cuh"
#include "pp_internal.cuh"

namespace pp {
namespace paged {

constexpr int kTile = 128;       // cache entries of one key tile
constexpr int kSms = 152;        // that a split is made for: a number of the GPU, not asked of the device,
                                 // so that neither bits nor scratch sizes depend on which one is current
constexpr int kMaxSeqs = 2048;   // sequences of one call (their prefix sums sit in shared memory)
constexpr int kMaxGroup = 64;    // query heads to a key head
constexpr int kMaxLen = 1 << 30; // larger kv_len count as this: four times the longest table row, and
                                 // differences of places and windows stay within 32 bits
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One call's cache and batch.  Lengths come from the device and are clamped to what the
// host has checked, so no length or offset can carry an access out of the arrays.
struct Args {
  const int32_t* table;
  const int32_t* len;      // cache entries of each sequence
  const int32_t* cu;       // first row of each sequence, and the end of the last
  int64_t page_stride;     // elements
  int n_pages, lps;        // pages of the pool; log2(page size)
  int Hk, G, D;            // key heads, query heads to each, head dim
  int n_seqs, table_ld, T;
  int window;              // 0: none
  float c;                 // scale * log2(e): scores in powers of two
  uint32_t* status;
  uint32_t wait_limit;     // polls before a wait gives up
  int withhold;            // 1 in a failure-detection test: the barrier of a CTA's first tile waits for
                           // an arrival that never comes
};

struct Seq {
  int row0, n;             // first row, new tokens
  int total, len;          // kv_len (new tokens included), and the entries that have a place
};

// Lengths and tables are read with plain loads: an earlier kernel of the same stream may
// have written them while this one was already on its SM (programmatic launch), which the
// non-coherent path does not allow.
__device__ __forceinline__ int table_entries(const Args& a) { return a.table_ld << a.lps; }
__device__ __forceinline__ int seq_len(const Args& a, int b) {
  return min(max(a.len[b], 0), table_entries(a));
}

__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  Seq s;
  s.row0 = min(max(a.cu[b], 0), a.T);
  s.n = min(max(a.cu[b + 1], s.row0), a.T) - s.row0;
  s.total = min(max(a.len[b], 0), kMaxLen);
  s.len = min(s.total, table_entries(a));
  return s;
}

// Page of entries [j, j + 1) of sequence b, or -1 when the table holds no page of the pool.
__device__ __forceinline__ int page_of(const Args& a, int b, int j) {
  const int p = a.table[(int64_t)b * a.table_ld + (j >> a.lps)];
  return (unsigned)p < (unsigned)a.n_pages ? p : -1;
}

__device__ __forceinline__ void raise(const Args& a, uint32_t bits) {
  if (a.status) atomicOr(a.status, bits);
}

// New tokens sit where kv_len says, so rows and entries are counted from it; entries past the
// table's row have no place and take no part.  One CTA of a call reports a length that has such.
__device__ __forceinline__ void check_len(const Args& a, const Seq& s) {
  if (s.total > s.len && blockIdx.x == 0) raise(a, PP_S_INDEX);
}

// Bounded wait for a barrier's phase.  A phase that has completed costs one test; only a wait
// that goes on looks at the CTA's abort flag, and one that runs out sets it and reports.
// (`kCall`: what goes on is a function call, so that the wait's code is short.  Not for kernels that
// split registers between warps: a call's are those of the whole kernel.)
__device__ __forceinline__ void poll_phase(uint32_t* status, uint32_t limit, uint32_t at,
                                           uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1     // (unrolled, the many waits of a kernel outgrow the instruction cache)
  for (uint32_t i = 0; i < limit; ++i) {
    if (*abort_flag) return;
    if (mbar_try_wait(at, parity)) return;
  }
  *abort_flag = 1;
  if (status) atomicOr(status, PP_S_TIMEOUT);
}
[[maybe_unused]] static __device__ __noinline__ void poll_phase_call(uint32_t* status, uint32_t limit,
                                                                     uint32_t at, uint32_t parity,
                                                                     volatile int* abort_flag) {
  poll_phase(status, limit, at, parity, abort_flag);
}
template <bool kCall = false>
__device__ __forceinline__ void wait_phase(const Args& a, uint64_t* bar, uint32_t parity,
                                           volatile int* abort_flag) {
  const uint32_t at = smem_u32(bar);
  if (mbar_try_wait(at, parity)) return;
  if constexpr (kCall)
    poll_phase_call(a.status, a.wait_limit, at, parity, abort_flag);
  else
    poll_phase(a.status, a.wait_limit, at, parity, abort_flag);
}

// The same for a thread that has nothing to report: copies in flight, the last MMAs.  Both come in
// microseconds, so a test's short limit does not cut them off.
__device__ __forceinline__ void drain_phase(const Args& a, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
#pragma unroll 1
  for (uint32_t i = 0; i < max(a.wait_limit, 1u << 16); ++i)
    if (mbar_try_wait(at, parity)) return;
}

// Prefix sums of count(b) over the sequences into pre[0..n], by one CTA; ends with a
// barrier.  Only row offsets that fall, so that sequences share rows, can make more units than a
// 32-bit sum holds: then there are none, and PP_S_INDEX tells.
template <typename I, typename F>
__device__ __forceinline__ void prefix_units(const Args& a, I* pre, F count) {
  const int n = a.n_seqs;
#pragma unroll 1
  for (int b = threadIdx.x; b < n; b += blockDim.x) pre[b + 1] = count(b);
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    I base = 0;
    float all = 0.f;
#pragma unroll 1
    for (int b0 = 0; b0 < n; b0 += 32) {
      const int b = b0 + threadIdx.x;
      I x = b < n ? pre[b + 1] : 0;
      all += (float)x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const I y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)threadIdx.x >= o) x += y;
      }
      if (b < n) pre[b + 1] = base + x;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if constexpr (sizeof(I) == 4) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      if (all > 2.1e9f) {
#pragma unroll 1
        for (int b = threadIdx.x; b < n; b += 32) pre[b + 1] = 0;
        if (threadIdx.x == 0) raise(a, PP_S_INDEX);
      }
    }
  }
  __syncthreads();
}

// The sequence whose units hold u: pre[b] <= u < pre[b + 1].
template <typename I>
__device__ __forceinline__ int find_seq(const I* pre, int n, I u) {
  int lo = 0, hi = n;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// ---- units ----------------------------------------------------------------------------------
// The producer warp works out a CTA's units and tells the other roles through a ring in shared
// memory: the others spend no instructions (and no instruction cache) on it.
struct alignas(16) Unit {
  int b, h;              // sequence (-1: no more units), key head
  int row, nt;           // first row of the unit's tokens, how many
  int first;             // entry index of that token (of the sequence's first one: k_paged_mass)
  int tile0, tile1;      // key tiles
  int low, stop;         // entries that some row sees lie in [low, stop); stop < first + nt where
                         // the table's row ends before the last token
  int split, ns;         // split of the keys, of how many
  int tag;               // 1 + the unit's place in this CTA's run
};
static_assert(sizeof(Unit) == 48, "three 16-byte words");
constexpr int kUnits = 8;
struct UnitRing {
  Unit unit[kUnits];
  uint64_t full[kUnits], empty[kUnits];
};

__device__ __forceinline__ void ring_init(UnitRing& r, int readers) {
  for (int i = 0; i < kUnits; ++i) {
    mbar_init(smem_u32(&r.full[i]), 1);
    mbar_init(smem_u32(&r.empty[i]), readers);
  }
}
// By the producer warp: the k-th unit.
template <bool kCall = false>
__device__ __forceinline__ void put_unit(const Args& a, UnitRing& r, uint32_t k, const Unit& x,
                                         int lane, volatile int* abort_flag) {
  const int i = k % kUnits;
  if (k >= kUnits) wait_phase<kCall>(a, &r.empty[i], (k / kUnits - 1) & 1, abort_flag);
  if (lane == 0) {
    r.unit[i] = x;
    mbar_arrive(smem_u32(&r.full[i]));
  }
}
// By each reader (a warp, or one thread of it with `alone`): the k-th unit, false after the
// last one or when the CTA gives up.
template <bool kCall = false>
__device__ __forceinline__ bool get_unit(const Args& a, UnitRing& r, uint32_t k, Unit& x, int lane,
                                         bool alone, volatile int* abort_flag) {
  const int i = k % kUnits;
  wait_phase<kCall>(a, &r.full[i], (k / kUnits) & 1, abort_flag);
  x = r.unit[i];
  if (!alone) __syncwarp();
  if (alone || lane == 0) mbar_arrive(smem_u32(&r.empty[i]));
  return x.b >= 0 && !*abort_flag;
}

// Bounded barrier of `count` warps on an mbarrier initialised with that count.
template <bool kCall = false>
__device__ __forceinline__ void sync_warps(const Args& a, uint64_t* bar, uint32_t& phase, int lane,
                                           volatile int* abort_flag) {
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(bar));
  wait_phase<kCall>(a, bar, phase & 1, abort_flag);
  ++phase;
}

// ---- shared-memory tiles -----------------------------------------------------------------
// A tile of R rows of D 16-bit values is D/64 boxes of R rows x 128 bytes, each in the
// 128-byte swizzle: 16-byte chunk c of row r sits at chunk c ^ (r & 7).

__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int box_bytes, int row, int chunk) {
  return base + (chunk >> 3) * box_bytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// Loading a key tile (entries [j0, j0 + 128) of head h) by one warp, a lane for each (page, 64-dim
// box).  Its lane's page comes first, so that the lookup can be on its way ahead of time.  Pages at
// or past `end` and pages outside the pool arrive as zeros.  `past`: the table's row ends at `end`,
// and rows beyond it would see zeros there as keys, so these groups are marked too.
struct TilePages {
  int page;              // of this lane's box; past the last page: zeros
  uint32_t bad;          // in every lane: the tile's 16-key groups without a page of the pool
};
__device__ __forceinline__ TilePages find_pages(const Args& a, int b, int j0, int end, bool past,
                                                int lane) {
  const int per = min(1 << a.lps, kTile);          // rows of one box
  const int pages = kTile / per;
  const int j = j0 + (lane % pages) * per;
  TilePages x{a.n_pages, 0u};
  bool bad = past && j >= end;
  if (lane < pages * (a.D >> 6) && j < end) {      // at most 16 loads
    const int p = page_of(a, b, j);
    bad = p < 0;
    if (!bad) x.page = p;
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, bad && lane < pages);
  if (mask) {                                      // rare: from pages to groups
#pragma unroll 1
    for (int g = 0; g < 8; ++g) x.bad |= ((mask >> (g * 16 / per)) & 1u) << g;
  }
  return x;
}
// With `bad_out` the mask is stored before the copy's barrier is armed: whoever has waited for
// the tile may read it.
__device__ __forceinline__ void load_key_tile(const Args& a, const CUtensorMap* map, uint32_t dst,
                                              uint32_t bar, const TilePages& x, int h, int j0,
                                              int lane, uint32_t* bad_out) {
  const int per = min(1 << a.lps, kTile), pages = kTile / per;
  const int pg = lane % pages, bx = lane / pages;
  if (lane == 0) {
    if (bad_out) *reinterpret_cast<volatile uint32_t*>(bad_out) = x.bad;
    mbar_expect_tx(bar, (uint32_t)(kTile * a.D * 2));
  }
  __syncwarp();
  if (bx < (a.D >> 6))
    tma_load_4d(dst + bx * (kTile * 128) + pg * per * 128, map, bx * 64,
                (j0 + pg * per) & ((1 << a.lps) - 1), h, x.page, bar);
}

// The non-finite values of V that a row at entry `pos` sees in the tiles where they were taken
// out of the product (those with a key that some row from `first` to `last` does not see):
// their sum for dims [d, d + W) is added to acc.  Rare, so slow but small.
template <typename N, int W>
__device__ __noinline__ void add_lost(const Args& a, const void* v_pages, int b, int h,
                                         int tile0, int tile1, int end, int first, int last,
                                         int pos, int d, float* acc) {
#pragma unroll 1
  for (int t = tile0; t < tile1; ++t) {
    const int j0 = t * kTile, j1 = min(j0 + kTile, end);
    bool edge = j0 + kTile - 1 > min(first, end - 1) || (a.window && j0 <= last - a.window);
#pragma unroll 1
    for (int j = j0; j < j1; j += 1 << a.lps) edge |= page_of(a, b, j) < 0;
    if (!edge) continue;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const int p = page_of(a, b, j);
      if (j > pos || (a.window && j <= pos - a.window) || p < 0) continue;
      const uint16_t* v = reinterpret_cast<const uint16_t*>(v_pages) + p * a.page_stride +
                          (((int64_t)h << a.lps) + (j & ((1 << a.lps) - 1))) * a.D + d;
#pragma unroll
      for (int e = 0; e < W; ++e)
        if ((v[e] & N::kExp) == N::kExp) acc[e] += N::to_float(v[e]);
    }
  }
}

// ---- matrix fragments ----------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The two 16-bit types: their product, their packed rounding, their non-finite values, and
// the power of two that softmax weights carry so that small ones stay normal numbers
// (fp16 has no exponents below 2^-14; bf16 has fp32's).  The weights are rounded before the second
// product, by at most 2^-8 (bf16) or 2^-11 (fp16) of each, which its operands' common type asks for;
// what that adds to the output's error (0.0015 in bf16) is less than the output's own rounding
// (0.0017).  Weights as hi + lo would double that product.
template <typename T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static constexpr float kShift = 0.f;
  static constexpr uint32_t kExp = 0x7f80u;
  static constexpr uint32_t kMmaTypes = (1u << 7) | (1u << 10);   // A and B in an MMA descriptor
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float to_float(uint32_t h) { return __uint_as_float(h << 16); }
  // z += 0 * w: stays zero while every w is finite
  static __device__ __forceinline__ void probe(uint32_t& z, uint32_t w) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(w), "r"(0));
  }
  static __device__ __forceinline__ void mma(float d[4], const uint32_t a[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Num<__half> {
  static constexpr float kShift = 7.f;
  static constexpr uint32_t kExp = 0x7c00u;
  static constexpr uint32_t kMmaTypes = 0u;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void probe(uint32_t& z, uint32_t w) {
    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(w), "r"(0));
  }
  static __device__ __forceinline__ float to_float(uint32_t h) {
    return __half2float(__ushort_as_half((unsigned short)h));
  }
  static __device__ __forceinline__ void mma(float d[4], const uint32_t a[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float lo_of(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi_of(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

// Split partials of one row joined by one warp, in split order: rec is the row's first record
// and ns <= 128 their count.
template <typename T, int D>
__device__ __forceinline__ void join_row(const float* part, const float2* part_ml, int64_t rec,
                                         int ns, T* out, float* lse, int lane) {
  float2 ml[4];                        // four records to a lane
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = i * 32 + lane;
    ml[i] = k < ns ? __ldcg(part_ml + rec + k) : make_float2(-INFINITY, 0.f);
    top = fmaxf(top, ml[i].x);
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
  const float ref = top == -INFINITY ? 0.f : top;
  // (a split without a reference has no keys that this row sees: -1, nothing to add; or scores of NaN
  // alone, which its sum tells)
  float f[4], sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = ml[i].x == -INFINITY ? -1.f : exp2_approx(ml[i].x - ref);
    sum += ml[i].x == -INFINITY ? ml[i].y : f[i] * ml[i].y;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  constexpr int DL = D / 32;
  float acc[DL] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int cnt = min(32, ns - i * 32);
#pragma unroll 4
    for (int k = 0; k < cnt; ++k) {
      const float w = __shfl_sync(0xffffffffu, f[i], k);
      const float* src = part + (rec + i * 32 + k) * D + lane * DL;
      if (w < 0.f) continue;           // (a weight of 0 counts: 0 times a NaN is one)
#pragma unroll
      for (int e = 0; e < DL; e += 2) {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(src + e));
        acc[e] = fmaf(w, y.x, acc[e]);
        acc[e + 1] = fmaf(w, y.y, acc[e + 1]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < DL; e += 2)
    *reinterpret_cast<uint32_t*>(out + lane * DL + e) = Num<T>::pack(acc[e] * inv, acc[e + 1] * inv);
  if (lse && lane == 0) *lse = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 1;
  return n;
}

// ---- launches ------------------------------------------------------------------------------
// A kernel's limit on dynamic shared memory belongs to the process and the device, and calls from
// several threads share it: it is set once to the most that any call asks for, never to one call's
// own size, which another call might lower between this one's setting and its launch.  `done` (one
// for each kernel) has a bit for each device.
inline cudaError_t allow_smem(const void* kern, int most, std::atomic<uint64_t>& done) {
  int dev = 0;
  const cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;   // from 64 on it is set at every call
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t set =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (set == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return set;
}

// Programmatic dependent launch: every kernel of this family waits for its predecessor
// (griddepcontrol.wait) before it reads anything, so it may be scheduled early.
template <typename... KArgs, typename... Args_>
cudaError_t launch_cluster(int cluster, void (*kern)(KArgs...), dim3 grid, int threads, size_t smem,
                           cudaStream_t s, Args_... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}
template <typename... KArgs, typename... Args_>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                   Args_... args) {
  return launch_cluster(1, kern, grid, threads, smem, s, args...);
}

struct Maps {
  CUtensorMap k, v, q;
};

// Split of the rows and keys of a call of short chunks (k_paged_attn.cu).
struct AttnPlan {
  int wr;          // 16-row fragments of a row tile: 1 or 2
  int tp;          // tokens of a row tile
  int share;       // SMs for each (sequence, key head), at least 1
  int ns_cap;      // splits of the longest sequence that the table can hold
  size_t rec_bytes, ml_bytes;
};
AttnPlan attn_plan(const Args& a, int max_q);

// Chunks of more than kShortRows rows (tokens x heads of a key head) run on the 5th-generation
// tensor cores (k_paged_attn_tc.cu): row tiles of 128 rows, taken in pairs.
constexpr int kShortRows = 32;
struct LongPlan {
  int tp;          // tokens of a row tile
  int64_t units;   // pairs of row tiles x key heads, at most
  int parts;       // splits of a unit's keys, at most
  int room;        // split units that scratch holds
  size_t rec_bytes, ml_bytes, plan_bytes;
};
LongPlan long_plan(const Args& a, int T);

struct AttnOut {
  void* out;
  float* lse;      // may be null
  float* part;     // split partials: [row][split][D] and [row][split] (reference, sum)
  float2* part_ml;
  int* plan;       // long chunks: units, whole units, parts, -, units before each sequence
};

cudaError_t launch_paged_attn(const Args& a, int type, const AttnPlan& plan, const Maps& maps,
                              const AttnOut& o, const void* v_pages, cudaStream_t s);
cudaError_t launch_paged_attn_tc(const Args& a, int type, const LongPlan& plan, const Maps& maps,
                                 const AttnOut& o, const void* v_pages, cudaStream_t s);
// Tokens of one step of rows (k_paged_mass.cu).
int mass_tokens(int G, int max_q);
cudaError_t launch_paged_mass(const Args& a, int type, const Maps& maps, const float* lse,
                              float* mass, float decay, int tp, cudaStream_t s);

struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *q_alpha, *k_alpha;
  float eps;
  int rot, halves;
  const int32_t* positions;
  void *q_out, *k_pages, *v_pages;
  float* mass;
  uint8_t *k_scale, *v_scale;   // of a cache in 8 bits, else null
  int64_t scale_stride;
};
struct Turns {
  uint64_t f[64];   // turns of each pair per position, as a fraction of 2^64
};
cudaError_t launch_paged_append(const Args& a, const AppendArgs& x, const Turns& turns, int in_type,
                                int type, cudaStream_t s);

struct EvictArgs {
  const void *k, *v;
  const float* mass;
  void *to_k, *to_v;
  float* to_mass;
  const int32_t* to_table;
  int64_t to_page_stride;
  int to_n_pages, to_lps, to_table_ld;
  int budget, recent;
  int32_t *to_len, *kept;
};
cudaError_t launch_paged_evict(const Args& a, const EvictArgs& x, cudaStream_t s);

// ---- the cache in 8 bits ---------------------------------------------------------------------
// (Args::page_stride counts its bytes)
struct Packed {
  const uint8_t *k, *v, *k_scale, *v_scale;
  int64_t scale_stride;
};

// Entries as 16-bit values into another cache's pages (k_packed_read.cu).
struct ReadArgs {
  Packed from;
  void *to_k, *to_v;
  float* to_mass;            // may be null
  int32_t* to_table;
  int64_t to_page_stride;    // elements
  int to_n_pages, to_lps, to_table_ld;
  int mirror;                // 1: `to` is a copy for an attention call: entries that its rows see, at
                             // page b * table_ld + i for page i of sequence b, which to_table is told
};
cudaError_t launch_packed_read(const Args& a, int type, const ReadArgs& x, cudaStream_t s);

// Chunks of up to kPackedRows rows (tokens x heads of a key head) run on the codes themselves
// (k_packed_attn.cu); longer ones on a 16-bit copy of what they see.  8 sequences of 20000 entries, 8 key
// heads: 64 rows 262 us on the codes, 321 on a copy; 128 rows 488 and 322.
constexpr int kPackedRows = 64;
struct PackedPlan {
  int R;           // rows of a row tile: 2, 4, 8, 16 or 32
  int max_q;
  int share;       // SMs for each (sequence, key head, row tile), at least 1
  int ns_cap;      // splits of the longest sequence that the table can hold
  size_t rec_bytes, ml_bytes;
};
PackedPlan packed_plan(const Args& a, int max_q);
cudaError_t launch_packed_attn(const Args& a, int type, const PackedPlan& plan, const Maps& maps,
                               const AttnOut& o, const Packed& kv, const void* q, int64_t q_stride,
                               cudaStream_t s);

}  // namespace paged
}  // namespace pp
