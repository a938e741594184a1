// k_packed_read.cu - entries of the 8-bit paged cache as 16-bit values into the pages of another cache.
//
//   value = code 2^e: the code as fp16 (exact), times a power of two (exact in fp32), rounded to the
//   cache's type (bf16 holds it exactly; fp16 what is within its range).
//
// Bound by reading 1 + 1/D bytes and writing two for each value.  A unit is 64 entries of a key head, K and
// V; a thread has 16 codes of several entries on their way at once and stores 32 bytes for each.
// Measured (in a graph): 16 sequences of up to 3000 entries, 32 heads of 128 dims, bf16: 108 us, 5.2 TB/s.
#include "pp_paged.cuh"

namespace pp {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kEntries = 64;         // of a unit: 64 divides a key tile
constexpr int kCtas = 4;             // to an SM

__device__ __forceinline__ uint32_t two_codes(uint32_t codes) {   // two e4m3 codes as fp16
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return h;
}
template <typename T>
__device__ __forceinline__ uint32_t two_values(uint32_t codes, float scale) {
  const uint32_t h = two_codes(codes);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return Num<T>::pack(f.x * scale, f.y * scale);
}
// 2^(byte - 127), NaN for 255
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Entries [from, to) that a sequence's unit range covers: all of them, or what an attention's rows see.
__device__ __forceinline__ int2 range_of(const Args& a, int b, bool seen) {
  if (!seen) return make_int2(0, seq_len(a, b));
  const Seq s = seq_of(a, b);
  if (s.n == 0) return make_int2(0, 0);
  const int low = a.window ? max(s.total - s.n - a.window + 1, 0) : 0;
  return make_int2(min(low, s.len) / kTile * kTile, s.len);   // whole key tiles
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_packed_read(const __grid_constant__ Args a, const __grid_constant__ ReadArgs x) {
  extern __shared__ int pre[];
  constexpr int L = D / 16;                       // threads of one entry
  constexpr int kRows = kThreads / L;             // entries side by side
  constexpr int kSteps = (kEntries + kRows - 1) / kRows;
  pdl_wait_and_trigger();
  pdl_trigger();
  prefix_units(a, pre, [&](int b) {
    const int2 r = range_of(a, b, x.mirror);
    return (r.y - r.x + kEntries - 1) / kEntries * a.Hk;
  });
  const int units = pre[a.n_seqs], l = threadIdx.x % L, row = threadIdx.x / L;
  const int in_page = (1 << a.lps) - 1, to_in_page = (1 << x.to_lps) - 1;
  bool lost = false;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int b = find_seq(pre, a.n_seqs, u);
    const int2 r = range_of(a, b, x.mirror);
    const int i = u - pre[b], h = i % a.Hk, j0 = r.x + i / a.Hk * kEntries;
    if (i == 0 && threadIdx.x == 0) lost |= a.len[b] > table_entries(a);
    uint4 codes[2][kSteps];
    uint32_t scale[2][kSteps];
    int page[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int j = j0 + s * kRows + row;
      page[s] = j < min(r.y, j0 + kEntries) ? page_of(a, b, j) : -2;
      if (page[s] < 0) continue;
      const int64_t at = ((int64_t)h << a.lps) + (j & in_page);
      const int64_t byte = page[s] * a.page_stride + at * D + l * 16;
      codes[0][s] = *reinterpret_cast<const uint4*>(x.from.k + byte);
      codes[1][s] = *reinterpret_cast<const uint4*>(x.from.v + byte);
      scale[0][s] = x.from.k_scale[page[s] * x.from.scale_stride + at];
      scale[1][s] = x.from.v_scale[page[s] * x.from.scale_stride + at];
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int j = j0 + s * kRows + row;
      if (page[s] == -2) continue;
      int to;
      if (x.mirror) {
        const int64_t slot = (int64_t)b * a.table_ld + (j >> a.lps);
        to = page[s] < 0 ? -1 : (int)slot;
        // (each page's first entry tells, and a range's first)
        if (h == 0 && l == 0 && ((j & in_page) == 0 || j == r.x)) x.to_table[slot] = to;
      } else {
        to = j < x.to_table_ld << x.to_lps ? x.to_table[(int64_t)b * x.to_table_ld + (j >> x.to_lps)] : -1;
        if ((unsigned)to >= (unsigned)x.to_n_pages) to = -1;
        lost |= to < 0 || page[s] < 0;
      }
      if (to < 0 || page[s] < 0) continue;
      const int64_t at = ((int64_t)h << x.to_lps) + (j & to_in_page);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t w[4] = {codes[kv][s].x, codes[kv][s].y, codes[kv][s].z, codes[kv][s].w};
        const float f = scale_of(scale[kv][s]);
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(kv ? x.to_v : x.to_k) +
                                              to * x.to_page_stride + at * D + l * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          dst[e] = make_uint4(two_values<T>(w[2 * e], f), two_values<T>(w[2 * e] >> 16, f),
                              two_values<T>(w[2 * e + 1], f), two_values<T>(w[2 * e + 1] >> 16, f));
      }
      if (x.to_mass && l == 0) x.to_mass[(((int64_t)to * a.Hk + h) << x.to_lps) + (j & to_in_page)] = 0.f;
    }
  }
  if (lost) raise(a, PP_S_INDEX);
}

template <typename T>
cudaError_t run(const Args& a, const ReadArgs& x, cudaStream_t s) {
  const int64_t entries = (int64_t)a.table_ld << a.lps;
  const int64_t most = (int64_t)a.n_seqs * a.Hk * ((entries + kEntries - 1) / kEntries);
  const int64_t ctas = (int64_t)sm_count() * kCtas;
  const dim3 grid((unsigned)(most < ctas ? most : ctas));
  const size_t smem = (size_t)(a.n_seqs + 1) * sizeof(int);
  return a.D == 128 ? launch(k_packed_read<T, 128>, grid, kThreads, smem, s, a, x)
                    : launch(k_packed_read<T, 64>, grid, kThreads, smem, s, a, x);
}

}  // namespace

cudaError_t launch_packed_read(const Args& a, int type, const ReadArgs& x, cudaStream_t s) {
  return type == PP_BF16 ? run<__nv_bfloat16>(a, x, s) : run<__half>(a, x, s);
}

}  // namespace paged
}  // namespace pp
