// C ABI of the 16-bit paged serving calls: argument checks on the host, then kernel launches.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/gqa_attn.h"
#include "kernels.h"

namespace {

using gqa::PagedKv;
using gqa::RowsArg;

constexpr int64_t kMaxStride = int64_t(1) << 38;   // elements: a tensor map holds 2^40 bytes
constexpr int kMost = 0x7fffffff - 1024;           // positions, rows, sequences: a tile past them fits an int

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool type_ok(int type) { return type == ATTN_TYPE_FP16 || type == ATTN_TYPE_BF16; }

bool heads_ok(int H, int Hkv, int D) {
  return H >= 1 && Hkv >= 1 && H % Hkv == 0 && H / Hkv <= 128 && D >= 16 && D <= 128 && D % 8 == 0;
}

bool decode_sizes_ok(int H, int Hkv, int D, int B, int max_len) {
  return heads_ok(H, Hkv, D) && B >= 1 && static_cast<int64_t>(B) * H <= 1 << 24 && max_len >= 0 &&
         max_len <= kMost;
}

// Rows [T, heads, D]: strides of at least D (in whole 16-byte steps) along the axes that have more
// than one element; `apart` (outputs): no two rows share memory, in either order of the axes.
int rows_of(const attn_rows* r, int T, int heads, int D, bool apart, RowsArg* out) {
  if (!r || !r->p) return ATTN_ERR_NULL;
  if (!aligned16(r->p)) return ATTN_ERR_ALIGN;
  const int64_t head = heads > 1 ? r->head_stride : D;
  const int64_t token = T > 1 ? r->token_stride : D;
  if (token % 8 || head % 8) return ATTN_ERR_ALIGN;
  if (token < D || head < D || token > kMaxStride || head > kMaxStride) return ATTN_ERR_SHAPE;
  if (apart && token < (heads - 1) * head + D && head < (T - 1) * token + D) return ATTN_ERR_PARAM;
  out->p = r->p;
  out->token = token;
  out->head = head;
  return ATTN_OK;
}

int cache_of(const attn_paged_kv* c, int Hkv, int D, PagedKv* out) {
  if (!c || !c->k || !c->v) return ATTN_ERR_NULL;
  if (!aligned16(c->k) || !aligned16(c->v)) return ATTN_ERR_ALIGN;
  int shift = 4;
  while (shift < 10 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size || c->pages < 1) return ATTN_ERR_SHAPE;
  const int64_t least = (static_cast<int64_t>(Hkv) * D) << shift;
  const int64_t stride = c->pages > 1 ? c->page_stride : least;
  if (stride % 8) return ATTN_ERR_ALIGN;
  if (stride < least || stride > kMaxStride) return ATTN_ERR_SHAPE;
  *out = PagedKv{c->k, c->v, stride, c->pages, shift};
  return ATTN_OK;
}

float scale_of(float scale, int D) { return scale > 0.f ? scale : 1.0f / sqrtf((float)D); }

// The opt-in non-finite check: 16-bit rows and pages, and fp32 norm weights.
int finite_gate(gqa::Finite16Job* j, const float* w0, const float* w1, int D, int32_t* status,
                cudaStream_t s, const int32_t** skip) {
  *skip = nullptr;
  if (!gqa::check_finite_enabled()) return ATTN_OK;
  if (!status) return ATTN_ERR_NULL;
  *skip = status;
  j->status = status;
  if (const int rc = gqa::record_cuda_error(gqa::launch_finite16_check(*j, s))) return rc;
  gqa::FiniteJob f{};
  for (const float* w : {w0, w1}) {
    if (!w) continue;
    gqa::FiniteRegion& r = f.r[f.n++];
    r.p = w; r.B = 1; r.NH = 1; r.R = 1; r.C = D; r.ld = D; r.mode = gqa::kFiniteAll;
  }
  f.status = status;
  return f.n ? gqa::record_cuda_error(gqa::launch_finite_check(f, s)) : ATTN_OK;
}

bool rope_ok(const attn_rope_params* rp, int D) {
  return attn_rope_table_bytes(rp, D) != 0;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of a shared-prefix call: the prefix's partial outputs and their weights, then the
// decode's. `parts` 0: the prefix is read with each row's own positions, which costs
// less than a kernel more where all rows together read at most kRereadBytes of it, mostly
// from L2. What a call's own layout takes moves both ways as rows come and go (parts go down where
// another pair of tiles is begun); `total` is a bound on it that no smaller B, prefix_len or max_len
// passes, so that the workspace of the largest batch serves every other.
constexpr double kRereadBytes = 64 << 20;
struct SharedLayout {
  size_t ml, decode, total;
  int parts;
};
SharedLayout shared_layout(int B, int H, int Hkv, int D, int prefix_len, int max_len) {
  SharedLayout y{};
  y.total = gqa::decode_paged_bytes(B, H, Hkv, D, max_len, 0, prefix_len);
  if (4.0 * B * prefix_len * Hkv * D <= kRereadBytes) return y;
  y.parts = gqa::shared_prefix_plan(B, H, Hkv, prefix_len).parts();
  const size_t rows = static_cast<size_t>(B) * H;
  y.ml = align256(rows * y.parts * D * sizeof(float));
  y.decode = y.ml + align256(rows * y.parts * 2 * sizeof(float));
  const size_t most = gqa::shared_prefix_rows(B, H, Hkv, prefix_len);
  y.total = std::max(y.total, align256(most * D * sizeof(float)) + align256(most * 2 * sizeof(float)) +
                                  gqa::decode_paged_bytes(B, H, Hkv, D, max_len, 0, 0));
  return y;
}

struct DecodeCall {
  int type;
  const attn_rows *q, *out;
  const attn_paged_kv* cache;
  const int32_t* block_table;
  int table_width;
  const int32_t* cache_len;
  int32_t max_cache_len;
  int B, H, Hkv, D, window;
  float softcap, scale;
};

// What both decode calls check; fills the job but for its workspace.
int decode_checks(const DecodeCall& c, gqa::DecodePagedJob* j) {
  if (!type_ok(c.type) || !heads_ok(c.H, c.Hkv, c.D) || c.B < 0 || c.window < 0 ||
      c.max_cache_len < 0 || c.max_cache_len > kMost || c.table_width < 1 ||
      static_cast<int64_t>(c.B) * c.H > (1 << 24))
    return ATTN_ERR_SHAPE;
  if (!isfinite(c.softcap) || !isfinite(c.scale)) return ATTN_ERR_PARAM;
  if (c.B == 0) return ATTN_OK;
  if (!c.block_table || !c.cache_len) return ATTN_ERR_NULL;
  if (int rc = rows_of(c.q, c.B, c.H, c.D, false, &j->q)) return rc;
  if (int rc = rows_of(c.out, c.B, c.H, c.D, true, &j->out)) return rc;
  if (int rc = cache_of(c.cache, c.Hkv, c.D, &j->cache)) return rc;
  if (c.max_cache_len > (static_cast<int64_t>(c.table_width) << j->cache.page_shift))
    return ATTN_ERR_CAPACITY;
  j->bf16 = c.type == ATTN_TYPE_BF16;
  j->block_table = c.block_table;
  j->width = c.table_width;
  j->cache_len = c.cache_len;
  j->max_len = c.max_cache_len;
  j->B = c.B; j->H = c.H; j->Hkv = c.Hkv; j->D = c.D;
  j->window = c.window;
  j->softcap = c.softcap;
  j->scale = scale_of(c.scale, c.D);
  return ATTN_OK;
}

gqa::Finite16Job finite_job(const gqa::DecodePagedJob& j) {
  gqa::Finite16Job f{};
  f.bf16 = j.bf16;
  f.D = j.D; f.Hkv = j.Hkv; f.T = j.B; f.B = j.B;
  f.rows[0] = j.q;
  f.heads[0] = j.H;
  f.cache = j.cache;
  gqa::Finite16Pages& p = f.pages[0];
  p.table = j.block_table; p.len = j.cache_len; p.width = j.width; p.B = j.B;
  p.max_len = j.max_len; p.window = j.window;
  return f;
}

}  // namespace

extern "C" {

int kv_cache_append_paged(int type, const attn_rows* q, const attn_rows* q_out, const attn_rows* k,
                          const attn_rows* k_out, const attn_rows* v, int T, int B, int H, int Hkv,
                          int D, const int32_t* cu_seqlens, const int32_t* start, int32_t max_pos,
                          const attn_rope_params* rp, const float* table, const float* q_norm_w,
                          const float* k_norm_w, float norm_eps, const attn_paged_kv* cache,
                          const int32_t* block_table, int table_width, int32_t* status,
                          void* stream) {
  if (!type_ok(type) || !heads_ok(H, Hkv, D) || T < 0 || B < 0 || B > kMost || table_width < 1 ||
      static_cast<int64_t>(T) * (H + 2 * static_cast<int64_t>(Hkv)) > 0x7fffffff ||
      (!cu_seqlens && T != B))
    return ATTN_ERR_SHAPE;
  if (T == 0 || B == 0) return ATTN_OK;
  gqa::AppendPagedJob j{};
  const bool with_q = q && q->p;
  if (!start || !block_table) return ATTN_ERR_NULL;
  if (with_q != (q_out && q_out->p)) return ATTN_ERR_NULL;
  if (with_q) {
    if (int rc = rows_of(q, T, H, D, false, &j.q)) return rc;
    if (int rc = rows_of(q_out, T, H, D, true, &j.q_out)) return rc;
  }
  if (int rc = rows_of(k, T, Hkv, D, false, &j.k)) return rc;
  if (int rc = rows_of(v, T, Hkv, D, false, &j.v)) return rc;
  if (k_out && k_out->p)
    if (int rc = rows_of(k_out, T, Hkv, D, true, &j.k_out)) return rc;
  if (int rc = cache_of(cache, Hkv, D, &j.cache)) return rc;
  if (rp ? !table : (table || q_norm_w || k_norm_w)) return rp ? ATTN_ERR_NULL : ATTN_ERR_PARAM;
  if ((rp && !rope_ok(rp, D)) || !(norm_eps >= 0.f) || (q_norm_w && !with_q)) return ATTN_ERR_PARAM;
  if ((table && !aligned16(table)) || (q_norm_w && !aligned16(q_norm_w)) ||
      (k_norm_w && !aligned16(k_norm_w)))
    return ATTN_ERR_ALIGN;
  if (max_pos < 0) return ATTN_ERR_POSITION;
  if (rp && max_pos >= (rp->max_positions > 0 ? rp->max_positions : 8192)) return ATTN_ERR_POSITION;
  if (max_pos >= (static_cast<int64_t>(table_width) << j.cache.page_shift)) return ATTN_ERR_CAPACITY;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  j.bf16 = type == ATTN_TYPE_BF16;
  j.T = T; j.B = B; j.H = H; j.Hkv = Hkv; j.D = D;
  j.R = rp ? (rp->rope_dim > 0 ? rp->rope_dim : D) : 0;
  j.cu = cu_seqlens; j.start = start; j.max_pos = max_pos;
  j.table = reinterpret_cast<const float2*>(table);
  j.q_norm_w = q_norm_w; j.k_norm_w = k_norm_w; j.norm_eps = norm_eps;
  j.block_table = block_table; j.width = table_width; j.status = status;
  gqa::Finite16Job f{};
  f.bf16 = j.bf16;
  f.D = D; f.Hkv = Hkv; f.T = T; f.B = B; f.cu = cu_seqlens;
  f.rows[0] = j.q; f.rows[1] = j.k; f.rows[2] = j.v;
  f.heads[0] = H; f.heads[1] = Hkv; f.heads[2] = Hkv;
  if (int rc = finite_gate(&f, q_norm_w, k_norm_w, D, status, s, &j.skip)) return rc;
  return gqa::record_cuda_error(gqa::launch_append_paged(j, s));
}

size_t gqa_attn_decode_paged_workspace_size(int B, int H, int Hkv, int D, int32_t max_cache_len,
                                            int window) {
  if (!decode_sizes_ok(H, Hkv, D, B, max_cache_len) || window < 0) return 0;
  return gqa::decode_paged_bytes(B, H, Hkv, D, max_cache_len, window, 0);
}

int gqa_attn_decode_paged(int type, const attn_rows* q, const attn_paged_kv* cache,
                          const int32_t* block_table, int table_width, const int32_t* cache_len,
                          int32_t max_cache_len, const attn_rows* out, int B, int H, int Hkv, int D,
                          int window, float softcap, float scale, void* workspace,
                          size_t workspace_bytes, int32_t* status, void* stream) {
  gqa::DecodePagedJob j{};
  const DecodeCall c{type, q, out, cache, block_table, table_width, cache_len, max_cache_len,
                     B, H, Hkv, D, window, softcap, scale};
  if (int rc = decode_checks(c, &j)) return rc;
  if (B == 0) return ATTN_OK;
  const size_t need = gqa::decode_paged_bytes(B, H, Hkv, D, max_cache_len, window, 0);
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (need && !aligned16(workspace)) return ATTN_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  j.partial = static_cast<float*>(workspace);
  j.status = status;
  gqa::Finite16Job f = finite_job(j);
  if (int rc = finite_gate(&f, nullptr, nullptr, D, status, s, &j.skip)) return rc;
  return gqa::record_cuda_error(gqa::launch_decode_paged(j, s));
}

size_t gqa_attn_decode_shared_workspace_size(int B, int H, int Hkv, int D, int32_t prefix_len,
                                             int32_t max_cache_len) {
  if (!decode_sizes_ok(H, Hkv, D, B, max_cache_len) || prefix_len < 1 || prefix_len > kMost) return 0;
  return shared_layout(B, H, Hkv, D, prefix_len, max_cache_len).total;
}

int gqa_attn_decode_shared(int type, const attn_rows* q, const attn_paged_kv* cache,
                           const int32_t* prefix_table, int prefix_width, int32_t prefix_len,
                           const int32_t* block_table, int table_width, const int32_t* cache_len,
                           int32_t max_cache_len, const attn_rows* out, int B, int H, int Hkv,
                           int D, float softcap, float scale, void* workspace,
                           size_t workspace_bytes, int32_t* status, void* stream) {
  gqa::DecodePagedJob j{};
  const DecodeCall c{type, q, out, cache, block_table, table_width, cache_len, max_cache_len,
                     B, H, Hkv, D, 0, softcap, scale};
  if (prefix_len < 1 || prefix_len > kMost || prefix_width < 1) return ATTN_ERR_SHAPE;
  if (int rc = decode_checks(c, &j)) return rc;
  if (B == 0) return ATTN_OK;
  if (!prefix_table) return ATTN_ERR_NULL;
  if (prefix_len > (static_cast<int64_t>(prefix_width) << j.cache.page_shift))
    return ATTN_ERR_CAPACITY;
  const SharedLayout y = shared_layout(B, H, Hkv, D, prefix_len, max_cache_len);
  if (y.total && (!workspace || workspace_bytes < y.total)) return ATTN_ERR_WORKSPACE;
  if (y.total && !aligned16(workspace)) return ATTN_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  gqa::Finite16Job f = finite_job(j);
  gqa::Finite16Pages& p = f.pages[1];
  p.table = prefix_table; p.width = prefix_width; p.B = 1; p.fixed_len = p.max_len = prefix_len;
  if (int rc = finite_gate(&f, nullptr, nullptr, D, status, s, &j.skip)) return rc;
  j.status = status;
  if (y.parts == 0) {
    j.prefix_table = prefix_table;
    j.prefix_len = prefix_len;
    j.partial = reinterpret_cast<float*>(w);
    return gqa::record_cuda_error(gqa::launch_decode_paged(j, s));
  }
  gqa::Attn16Job a{};
  a.bf16 = j.bf16;
  a.q = j.q;
  a.cache = j.cache;
  a.prefix_table = prefix_table; a.prefix_len = prefix_len;
  a.T = B; a.B = B; a.H = H; a.Hkv = Hkv; a.D = D;
  a.softcap = softcap; a.scale = j.scale;
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + y.ml);
  a.status = status; a.skip = j.skip;
  if (int rc = gqa::record_cuda_error(a.bf16 ? gqa::launch_attn16_bf16(a, s)
                                             : gqa::launch_attn16_fp16(a, s)))
    return rc;
  j.prefix.o = a.part_o;
  j.prefix.ml = a.part_ml;
  j.prefix.nsplit = y.parts;
  j.partial = reinterpret_cast<float*>(w + y.decode);
  return gqa::record_cuda_error(gqa::launch_decode_paged(j, s));
}

int gqa_attn_prefill_packed(int type, const attn_rows* q, const attn_rows* k, const attn_rows* v,
                            const int32_t* cu_seqlens, int32_t max_len, const attn_rows* out, int T,
                            int B, int H, int Hkv, int D, int window, float softcap, float scale,
                            int32_t* status, void* stream) {
  if (!type_ok(type) || !heads_ok(H, Hkv, D) || T < 0 || B < 0 || max_len < 0 || window < 0 ||
      T > kMost || static_cast<int64_t>(T) * H > 0x7fffffff ||
      (static_cast<int64_t>(T) + B) * Hkv > kMost)
    return ATTN_ERR_SHAPE;
  if (!isfinite(softcap) || !isfinite(scale)) return ATTN_ERR_PARAM;
  if (T == 0 || B == 0) return ATTN_OK;
  if (!cu_seqlens) return ATTN_ERR_NULL;
  gqa::Attn16Job a{};
  if (int rc = rows_of(q, T, H, D, false, &a.q)) return rc;
  if (int rc = rows_of(k, T, Hkv, D, false, &a.k)) return rc;
  if (int rc = rows_of(v, T, Hkv, D, false, &a.v)) return rc;
  if (int rc = rows_of(out, T, H, D, true, &a.out)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.bf16 = type == ATTN_TYPE_BF16;
  a.cu = cu_seqlens; a.T = T; a.B = B; a.max_len = max_len;
  a.H = H; a.Hkv = Hkv; a.D = D;
  a.window = window; a.softcap = softcap; a.scale = scale_of(scale, D);
  a.status = status;
  gqa::Finite16Job f{};
  f.bf16 = a.bf16;
  f.D = D; f.Hkv = Hkv; f.T = T; f.B = B; f.cu = cu_seqlens;
  f.rows[0] = a.q; f.rows[1] = a.k; f.rows[2] = a.v;
  f.heads[0] = H; f.heads[1] = Hkv; f.heads[2] = Hkv;
  if (int rc = finite_gate(&f, nullptr, nullptr, D, status, s, &a.skip)) return rc;
  return gqa::record_cuda_error(a.bf16 ? gqa::launch_attn16_bf16(a, s)
                                       : gqa::launch_attn16_fp16(a, s));
}

}  // extern "C"
