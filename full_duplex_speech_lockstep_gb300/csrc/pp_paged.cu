// pp_paged.cu - the C entry points of the paged-cache operators: argument checks, tensor
// maps and launches.
#include <math.h>

#include "pp_paged.cuh"

using namespace pp;
using namespace pp::paged;

namespace {

// pp_test_paged_faults: of this host thread's calls
thread_local int test_wait_polls = 0, test_withhold = 0;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The cache's own description: sizes, alignments, and offsets that stay within 64 bits.
bool cache_ok(const pp_paged_kv* kv) {
  if (!kv || !kv->k || !kv->v || !kv->table) return false;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->mass, 4) || !aligned(kv->table, 4))
    return false;
  if (kv->type != PP_BF16 && kv->type != PP_F16) return false;
  if (kv->head_dim != 64 && kv->head_dim != 128) return false;
  if (kv->page_size < 16 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1)))
    return false;
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024 || kv->n_pages < 1) return false;
  if (kv->n_seqs < 1 || kv->n_seqs > kMaxSeqs || kv->table_ld < 1) return false;
  if ((int64_t)kv->table_ld * kv->page_size > (int64_t)1 << 28) return false;
  // units, tiles and blocks of a call are counted in 32 bits
  if ((int64_t)kv->n_seqs * kv->n_kv_heads *
          (((int64_t)kv->table_ld * kv->page_size + kTile - 1) / kTile) >= (int64_t)1 << 28)
    return false;
  const int64_t page = (int64_t)kv->n_kv_heads * kv->page_size * kv->head_dim;
  if (kv->page_stride < page || (kv->page_stride & 7) || kv->page_stride >= (int64_t)1 << 38)
    return false;
  return true;
}

Args base_args(const pp_paged_kv* kv, const int32_t* kv_len, uint32_t* status) {
  Args a{};
  a.table = kv->table;
  a.len = kv_len;
  a.page_stride = kv->page_stride;
  a.n_pages = kv->n_pages;
  while ((1 << a.lps) < kv->page_size) ++a.lps;
  a.Hk = kv->n_kv_heads;
  a.G = 1;
  a.D = kv->head_dim;
  a.n_seqs = kv->n_seqs;
  a.table_ld = kv->table_ld;
  a.status = status;
  a.wait_limit = test_wait_polls ? (uint32_t)test_wait_polls : kWaitLimit;
  a.withhold = test_withhold;
  return a;
}

// The new rows of a call: cu, T and the query heads.
bool rows_ok(const pp_paged_kv* kv, const int32_t* cu, const int32_t* kv_len, int T, int n_heads) {
  if (!cu || !kv_len || !aligned(cu, 4) || !aligned(kv_len, 4)) return false;
  if (T < 0 || n_heads < 1 || n_heads % kv->n_kv_heads != 0) return false;
  const int G = n_heads / kv->n_kv_heads;
  return G <= kMaxGroup && T <= 1 << 28 && (int64_t)T * n_heads < (int64_t)1 << 31;
}

// A window that no row outgrows is none.
int effective_window(int window) { return window >= kMaxLen ? 0 : window; }

bool scores_ok(float scale, int window, int max_q) {
  return scale > 0.f && scale <= 1e30f && window >= 0 && max_q >= 1;
}

// Pages as [page][head][row][dim], box 64 dims x one page or one key tile, and queries as
// [token][head][dim], box 64 dims x the G heads of a key head x the tokens of a row tile.  PP_E_CUDA
// where there is no driver to encode them.
int encode(CUtensorMap* m, int type, const void* base, const cuuint64_t dim[4],
           const cuuint64_t stride[3], const cuuint32_t box[4]) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return PP_E_CUDA;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = fn(
      m, type == PP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
      const_cast<void*>(base), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PP_OK : PP_EINVAL;
}
int page_map(CUtensorMap* m, const pp_paged_kv* kv, const void* base) {
  const cuuint64_t D = kv->head_dim, P = kv->page_size;
  const cuuint64_t dim[4] = {D, P, (cuuint64_t)kv->n_kv_heads, (cuuint64_t)kv->n_pages};
  const cuuint64_t stride[3] = {D * 2, P * D * 2, (cuuint64_t)kv->page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)(P < kTile ? P : kTile), 1, 1};
  return encode(m, kv->type, base, dim, stride, box);
}
int query_map(CUtensorMap* m, const Args& a, int type, const void* q, int64_t stride_q, int tp) {
  const cuuint64_t D = a.D, H = (cuuint64_t)a.Hk * a.G;
  const cuuint64_t dim[4] = {D, H, (cuuint64_t)a.T, 1};
  const cuuint64_t stride[3] = {D * 2, (cuuint64_t)stride_q * 2, (cuuint64_t)stride_q * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)a.G, (cuuint32_t)tp, 1};
  return encode(m, type, q, dim, stride, box);
}

// Do T rows of `len` bytes, `stride` >= len bytes apart, meet the `n` bytes from `at`?
bool rows_meet(const void* rows, int64_t stride, int64_t len, int T, const void* at, int64_t n) {
  const int64_t d = reinterpret_cast<intptr_t>(at) - reinterpret_cast<intptr_t>(rows);
  const int64_t t = d < len ? 0 : (d - len) / stride + 1;   // the first row that ends past `at`
  return t < T && t * stride < d + n;
}

bool is_long(const Args& a, int max_q) { return (int64_t)max_q * a.G > kShortRows; }

int rc(cudaError_t err) { return err == cudaSuccess ? PP_OK : PP_E_CUDA; }

}  // namespace

extern "C" {

int pp_paged_append(const pp_paged_kv* kv, const void* q, int64_t q_stride, const void* k,
                    int64_t k_stride, const void* v, int64_t v_stride, int in_type,
                    const float* q_alpha, const float* k_alpha, float eps, float rope_base,
                    int rot_dim, int halves, const int32_t* positions, const int32_t* cu,
                    const int32_t* kv_len, int T, int n_heads, void* q_out, uint32_t* status,
                    void* stream) {
  if (!cache_ok(kv) || !rows_ok(kv, cu, kv_len, T, n_heads)) return PP_EINVAL;
  if (in_type != PP_F32 && in_type != kv->type) return PP_EINVAL;
  if (rot_dim < 0 || rot_dim > kv->head_dim || (rot_dim & 1)) return PP_EINVAL;
  if (!(rope_base >= 1.f) || !(eps >= 0.f) || isinf(rope_base) || isinf(eps)) return PP_EINVAL;
  if (T == 0) return PP_OK;
  const int64_t D = kv->head_dim;
  if (!q || !k || !v || !q_out || q_stride < n_heads * D || k_stride < kv->n_kv_heads * D ||
      v_stride < kv->n_kv_heads * D)
    return PP_EINVAL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(q_alpha, 16) || !aligned(k_alpha, 16) || !aligned(positions, 4) ||
      ((q_stride | k_stride | v_stride) & 7))
    return PP_EINVAL;
  Args a = base_args(kv, kv_len, status);
  a.cu = cu;
  a.T = T;
  a.G = n_heads / kv->n_kv_heads;
  AppendArgs x{};
  x.q = q;
  x.k = k;
  x.v = v;
  x.q_stride = q_stride;
  x.k_stride = k_stride;
  x.v_stride = v_stride;
  x.q_alpha = q_alpha;
  x.k_alpha = k_alpha;
  x.eps = eps;
  x.rot = rot_dim;
  x.halves = halves != 0;
  x.positions = positions;
  x.q_out = q_out;
  x.k_pages = kv->k;
  x.v_pages = kv->v;
  x.mass = kv->mass;
  // turns of pair i per position: base^(-2i/rot) / 2 pi, below a sixth, in units of 2^-64
  Turns turns{};
  const double step = rot_dim ? pow((double)rope_base, -2.0 / rot_dim) : 1.0;
  double f = 18446744073709551616.0 / 6.283185307179586476925;
  for (int i = 0; i < rot_dim / 2; ++i, f *= step) turns.f[i] = (uint64_t)f;
  return rc(launch_paged_append(a, x, turns, in_type, kv->type, (cudaStream_t)stream));
}

int pp_test_paged_faults(int32_t wait_polls, int32_t withhold) {
  if (wait_polls < 0 || (withhold != 0 && withhold != 1)) return PP_EINVAL;
  test_wait_polls = wait_polls;
  test_withhold = withhold;
  return PP_OK;
}

size_t pp_paged_attention_scratch_bytes(const pp_paged_kv* kv, int n_heads, int T, int max_q,
                                        int window) {
  const int32_t any = 0;
  if (!cache_ok(kv) || !rows_ok(kv, &any, &any, T, n_heads) || !scores_ok(1.f, window, max_q))
    return 0;
  Args a = base_args(kv, nullptr, nullptr);
  a.G = n_heads / kv->n_kv_heads;
  a.window = effective_window(window);
  if (is_long(a, max_q)) {
    const LongPlan p = long_plan(a, T);
    return p.rec_bytes + p.ml_bytes + p.plan_bytes + 256;
  }
  const AttnPlan p = attn_plan(a, max_q);
  return p.rec_bytes + p.ml_bytes + 256;
}

int pp_paged_attention(const pp_paged_kv* kv, const void* q, int64_t q_stride, const int32_t* cu,
                       const int32_t* kv_len, int T, int max_q, int n_heads, float scale,
                       int window, void* out, float* lse, uint32_t* status, void* scratch,
                       size_t scratch_bytes, void* stream) {
  if (!cache_ok(kv) || !rows_ok(kv, cu, kv_len, T, n_heads) || !scores_ok(scale, window, max_q))
    return PP_EINVAL;
  if (T == 0) return PP_OK;
  const int64_t D = kv->head_dim;
  if (!q || !out || !scratch || q_stride < n_heads * D || (q_stride & 7) ||
      q_stride >= (int64_t)1 << 38)
    return PP_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(scratch, 256))
    return PP_EINVAL;
  if (scratch_bytes < pp_paged_attention_scratch_bytes(kv, n_heads, T, max_q, window))
    return PP_E_NOSPACE;
  // a CTA's queries are read while others' outputs are written
  if (rows_meet(q, q_stride * 2, n_heads * D * 2, T, out, T * n_heads * D * 2)) return PP_EINVAL;
  Args a = base_args(kv, kv_len, status);
  a.cu = cu;
  a.T = T;
  a.G = n_heads / kv->n_kv_heads;
  a.window = effective_window(window);
  a.c = scale * kLog2e;
  AttnOut o{};
  o.out = out;
  o.lse = lse;
  o.part = reinterpret_cast<float*>(scratch);
  Maps maps;
  int bad = page_map(&maps.k, kv, kv->k);
  if (bad || (bad = page_map(&maps.v, kv, kv->v))) return bad;
  if (is_long(a, max_q)) {
    const LongPlan p = long_plan(a, T);
    if ((bad = query_map(&maps.q, a, kv->type, q, q_stride, p.tp))) return bad;
    o.part_ml = reinterpret_cast<float2*>(reinterpret_cast<char*>(scratch) + p.rec_bytes);
    o.plan = reinterpret_cast<int*>(reinterpret_cast<char*>(scratch) + p.rec_bytes + p.ml_bytes);
    return rc(launch_paged_attn_tc(a, kv->type, p, maps, o, kv->v, (cudaStream_t)stream));
  }
  const AttnPlan p = attn_plan(a, max_q);
  if ((bad = query_map(&maps.q, a, kv->type, q, q_stride, p.tp))) return bad;
  o.part_ml = reinterpret_cast<float2*>(reinterpret_cast<char*>(scratch) + p.rec_bytes);
  return rc(launch_paged_attn(a, kv->type, p, maps, o, kv->v, (cudaStream_t)stream));
}

int pp_paged_mass(const pp_paged_kv* kv, const void* q, int64_t q_stride, const float* lse,
                  const int32_t* cu, const int32_t* kv_len, int T, int max_q, int n_heads,
                  float scale, int window, float decay, uint32_t* status, void* stream) {
  if (!cache_ok(kv) || !kv->mass || !rows_ok(kv, cu, kv_len, T, n_heads) ||
      !scores_ok(scale, window, max_q))
    return PP_EINVAL;
  if (!(decay >= 0.f && decay <= 1.f)) return PP_EINVAL;
  const int64_t D = kv->head_dim;
  Args a = base_args(kv, kv_len, status);
  a.cu = cu;
  a.T = T;
  a.G = n_heads / kv->n_kv_heads;
  a.window = effective_window(window);
  a.c = scale * kLog2e;
  if (T > 0 && (!q || !lse || q_stride < n_heads * D || (q_stride & 7) ||
                q_stride >= (int64_t)1 << 38 || !aligned(q, 16) || !aligned(lse, 4)))
    return PP_EINVAL;
  const int tp = mass_tokens(a.G, max_q);
  Maps maps;
  // without a row the query map is never used: any valid one will do
  Args qa = a;
  if (T == 0) qa.T = 1;
  int bad = page_map(&maps.k, kv, kv->k);
  if (bad || (bad = query_map(&maps.q, qa, kv->type, T ? q : kv->k, T ? q_stride : n_heads * D, tp)))
    return bad;
  return rc(launch_paged_mass(a, kv->type, maps, lse, kv->mass, decay, tp, (cudaStream_t)stream));
}

int pp_paged_evict(const pp_paged_kv* kv, const int32_t* kv_len, int budget, int recent,
                   const pp_paged_kv* to, int32_t* to_len, int32_t* kept, uint32_t* status,
                   void* stream) {
  if (!cache_ok(kv) || !cache_ok(to) || !kv->mass || !kv_len || !to_len || !kept) return PP_EINVAL;
  if (!aligned(kv_len, 4) || !aligned(to_len, 4) || !aligned(kept, 4)) return PP_EINVAL;
  if (budget < 1 || budget > 1 << 28 || recent < 0 || recent > budget) return PP_EINVAL;
  if (to->type != kv->type || to->head_dim != kv->head_dim || to->n_kv_heads != kv->n_kv_heads ||
      to->n_seqs != kv->n_seqs)
    return PP_EINVAL;
  // the destination's table holds the longest row that can stay
  const int64_t entries = (int64_t)kv->table_ld * kv->page_size;
  const int64_t most = entries < budget ? entries : budget;
  if ((int64_t)to->table_ld * to->page_size < most) return PP_E_RANGE;
  // its own pages: entries would be written over before they are read
  if (to->k == kv->k && to->table == kv->table) return PP_EINVAL;
  Args a = base_args(kv, kv_len, status);
  EvictArgs x{};
  x.k = kv->k;
  x.v = kv->v;
  x.mass = kv->mass;
  x.to_k = to->k;
  x.to_v = to->v;
  x.to_mass = to->mass;
  x.to_table = to->table;
  x.to_page_stride = to->page_stride;
  x.to_n_pages = to->n_pages;
  while ((1 << x.to_lps) < to->page_size) ++x.to_lps;
  x.to_table_ld = to->table_ld;
  x.budget = budget;
  x.recent = recent;
  x.to_len = to_len;
  x.kept = kept;
  return rc(launch_paged_evict(a, x, (cudaStream_t)stream));
}

}  // extern "C"
