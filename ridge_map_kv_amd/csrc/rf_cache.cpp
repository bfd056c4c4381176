// C entry points of the cache calls (rotary positions, head norms, append, read, attention,
// attention weight, eviction): argument checks and the host side of the rotation's frequencies.
// Device work is in rf_rope.hip, rf_norm.hip, rf_attend.hip, rf_weight.hip and rf_evict.hip.
#include "rf_cache.h"

#include <cmath>

#include "rf_error.h"

namespace {

using rf::fail;
using rf::hip_fail;
using rf::ok;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Bounds that keep every grid below 2^32 threads.
constexpr int64_t kMaxRows = 1 << 23;         // of a rotation or an append: up to a workgroup of 256 each
constexpr int64_t kMaxQueries = 1 << 26;      // batch * query heads * max_q
constexpr int64_t kMaxWeights = 1 << 29;      // batch * max_len of the attention weight

constexpr double kTwoPi = 6.283185307179586476925286766559;

// The rotation's angle per position of every pair, in turns; head_dim bounds rotary_dim.
rf_status make_freq(const rf_rope* r, int head_dim, rf::RopeFreq& f) {
  const int rot = r->rotary_dim ? r->rotary_dim : head_dim;
  if (rot < 16 || rot % 16 || rot > head_dim)
    return fail(RF_E_SHAPE, "rotary_dim = %d must be 0 or a multiple of 16 up to head_dim = %d",
                r->rotary_dim, head_dim);
  if (r->layout != RF_ROPE_HALF && r->layout != RF_ROPE_INTERLEAVED)
    return fail(RF_E_INVALID, "rope.layout = %d", r->layout);
  if (r->scaling < RF_ROPE_PLAIN || r->scaling > RF_ROPE_YARN)
    return fail(RF_E_INVALID, "rope.scaling = %d", r->scaling);
  if (!(r->theta > 1.0) || !std::isfinite(r->theta))
    return fail(RF_E_INVALID, "rope.theta must be finite and > 1");
  if (!(r->mscale >= 0.0) || !std::isfinite(r->mscale))
    return fail(RF_E_INVALID, "rope.mscale must be finite and >= 0");
  const bool scaled = r->scaling != RF_ROPE_PLAIN;
  if (scaled && (!(r->factor >= 1.0) || !std::isfinite(r->factor)))
    return fail(RF_E_INVALID, "rope.factor must be finite and >= 1");
  const bool ramp = r->scaling == RF_ROPE_BANDS || r->scaling == RF_ROPE_YARN;
  if (ramp && (r->orig_len < 1 || !(r->low > 0.0) || !(r->high > r->low) || !std::isfinite(r->high)))
    return fail(RF_E_INVALID, "rope: orig_len >= 1 and 0 < low < high are needed");
  const double s = scaled ? r->factor : 1.0, L = r->orig_len;
  const double theta = r->scaling == RF_ROPE_NTK ? r->theta * std::pow(s, rot / (rot - 2.0)) : r->theta;
  double p = 0.0, q = 1.0;
  if (r->scaling == RF_ROPE_YARN) {
    const auto pair_at = [&](double n) { return rot * std::log(L / (kTwoPi * n)) / (2.0 * std::log(r->theta)); };
    p = std::fmax(std::floor(pair_at(r->high)), 0.0);
    q = std::fmin(std::ceil(pair_at(r->low)), rot - 1.0);
  }
  for (int j = 0; j < rot / 2; ++j) {
    double w = std::pow(theta, -2.0 * j / rot);
    double t = 1.0;                                  // share that is divided by the factor
    if (r->scaling == RF_ROPE_BANDS)
      t = 1.0 - (L * w / kTwoPi - r->low) / (r->high - r->low);
    else if (r->scaling == RF_ROPE_YARN)
      t = (j - p) / std::fmax(q - p, 1e-3);
    else if (r->scaling != RF_ROPE_LINEAR)
      t = 0.0;
    t = std::fmin(std::fmax(t, 0.0), 1.0);
    f.turns[j] = (t * w / s + (1.0 - t) * w) / kTwoPi;
  }
  f.m = (float)(r->mscale > 0.0 ? r->mscale : r->scaling == RF_ROPE_YARN ? 0.1 * std::log(s) + 1.0 : 1.0);
  f.rot = rot;
  f.layout = r->layout;
  return RF_OK;
}

// The batch descriptor; `append`: head sizes up to 256, lengths not needed.
rf_status check_batch(const rf_paged_batch* kv, bool append, rf::Batch& b) {
  if (!kv) return fail(RF_E_INVALID, "kv is NULL");
  if (kv->batch < 1 || kv->batch > 65535) return fail(RF_E_SHAPE, "batch = %d must be in 1..65535", kv->batch);
  if (kv->max_len < 1 || kv->page_size < 1 || kv->num_pages < 1)
    return fail(RF_E_SHAPE, "max_len, page_size and num_pages must be >= 1");
  if (kv->max_len > (1 << 30) || (int64_t)kv->batch * kv->max_len > (int64_t)1 << 36)
    return fail(RF_E_SHAPE, "max_len = %d must be at most 2^30, batch * max_len at most 2^36", kv->max_len);
  if (kv->table_stride < ((int64_t)kv->max_len + kv->page_size - 1) / kv->page_size)
    return fail(RF_E_SHAPE, "table_stride = %lld holds fewer than max_len = %d rows",
                (long long)kv->table_stride, kv->max_len);
  if ((int64_t)kv->num_pages * kv->page_size > INT32_MAX)
    return fail(RF_E_SHAPE, "num_pages * page_size must be below 2^31");
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 256)
    return fail(RF_E_SHAPE, "n_kv_heads = %d must be in 1..256", kv->n_kv_heads);
  if (append ? (kv->head_dim < 16 || kv->head_dim > 256 || kv->head_dim % 16)
             : (kv->head_dim != 64 && kv->head_dim != 128))
    return fail(RF_E_SHAPE, append ? "head_dim = %d must be a multiple of 16 up to 256"
                                   : "head_dim = %d must be 64 or 128", kv->head_dim);
  b = {kv->block_tables, kv->lengths, kv->table_stride, kv->batch, kv->max_len,
       kv->page_size, kv->num_pages, kv->n_kv_heads, kv->head_dim};
  return RF_OK;
}

// Its device pointers, and a workspace of at least `need` bytes.
rf_status check_memory(const rf::Batch& b, const void* ws, size_t ws_bytes, size_t need) {
  if (!b.tables || !b.lengths) return fail(RF_E_INVALID, "kv: block_tables or lengths is NULL");
  if (!aligned(b.tables, 4) || !aligned(b.lengths, 4))
    return fail(RF_E_SHAPE, "block_tables and lengths need 4-byte alignment");
  if (!ws) return fail(RF_E_INVALID, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(RF_E_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return fail(RF_E_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
  return RF_OK;
}

rf_status check_heads(const rf::Batch& b, int n_q_heads, int max_q) {
  if (n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % b.n_kv)
    return fail(RF_E_SHAPE, "n_q_heads = %d must be a multiple of n_kv_heads = %d, at most 4096",
                n_q_heads, b.n_kv);
  if (max_q < 1 || max_q > 64) return fail(RF_E_SHAPE, "max_q = %d must be in 1..64", max_q);
  if ((int64_t)b.batch * n_q_heads * max_q > kMaxQueries)
    return fail(RF_E_SHAPE, "batch * n_q_heads * max_q must be at most 2^26");
  return RF_OK;
}

rf_status check_weights(const rf::Batch& b) {
  if ((int64_t)b.batch * b.max_len > kMaxWeights)
    return fail(RF_E_SHAPE, "batch * max_len must be at most 2^29 for the attention weight");
  return RF_OK;
}

rf_status check_queries(const rf::Batch& b, const uint16_t* q, int n_q_heads, int64_t q_stride,
                        const int32_t* q_start, int64_t n_q, int max_q, const uint64_t* mask,
                        float scale) {
  rf_status s = check_heads(b, n_q_heads, max_q);
  if (s != RF_OK) return s;
  if (n_q < 0 || n_q > INT32_MAX) return fail(RF_E_SHAPE, "n_q = %lld out of range", (long long)n_q);
  if (!std::isfinite(scale)) return fail(RF_E_INVALID, "scale must be finite");
  if (!q_start || (n_q > 0 && !q)) return fail(RF_E_INVALID, "q or q_start is NULL");
  if (q_stride < (int64_t)n_q_heads * b.hd || q_stride % 8 || !aligned(q, 16) ||
      !aligned(q_start, 4) || !aligned(mask, 8))
    return fail(RF_E_SHAPE, "q: 16-byte alignment, a stride >= n_q_heads * head_dim that is a "
                "multiple of 8; q_start 4-byte, tree_mask 8-byte alignment");
  return RF_OK;
}

// The arguments of an append, and the rotation's frequencies.
rf_status check_append(const rf_rope* rope, const rf::Batch& b, const uint16_t* q, int32_t n_q_heads, int64_t q_stride,
                       const uint16_t* q_out, int64_t q_out_stride, const uint16_t* k, int64_t k_stride,
                       const uint16_t* v, int64_t v_stride, int64_t n_rows, const int32_t* seq, const int32_t* rows,
                       const int32_t* positions, const void* k_pages, const void* v_pages, const uint32_t* status,
                       rf::RopeFreq& f) {
  if (!status || !aligned(status, 4))
    return fail(RF_E_INVALID, "status must be a 4-byte aligned device pointer");
  if (n_rows < 0 || n_rows > kMaxRows)
    return fail(RF_E_SHAPE, "n_rows = %lld must be in 0..2^23", (long long)n_rows);
  f = {};
  f.layout = RF_ROPE_HALF;
  if (rope) {
    const rf_status s = make_freq(rope, b.hd, f);
    if (s != RF_OK) return s;
  }
  if (n_q_heads < 0 || n_q_heads > 4096) return fail(RF_E_SHAPE, "n_q_heads = %d must be in 0..4096", n_q_heads);
  if ((n_q_heads > 0) != (q != nullptr || q_out != nullptr) || (q != nullptr) != (q_out != nullptr)) {
    if (n_rows > 0 || n_q_heads == 0)
      return fail(RF_E_INVALID, "q and q_out go together, and with n_q_heads > 0");
  }
  const int64_t kw = (int64_t)b.n_kv * b.hd, qw = (int64_t)n_q_heads * b.hd;
  if (k_stride < kw || v_stride < kw || k_stride % 8 || v_stride % 8)
    return fail(RF_E_SHAPE, "k_stride and v_stride must be >= n_kv_heads * head_dim and multiples of 8");
  if (n_q_heads && (q_stride < qw || q_out_stride < qw || q_stride % 8 || q_out_stride % 8))
    return fail(RF_E_SHAPE, "q_stride and q_out_stride must be >= n_q_heads * head_dim and multiples of 8");
  if (n_q_heads && q == q_out && q_stride != q_out_stride)
    return fail(RF_E_INVALID, "rotating q in place needs equal strides");
  if (n_rows == 0) return RF_OK;
  if (!k || !v || !rows || !k_pages || !v_pages || !b.tables)
    return fail(RF_E_INVALID, "null pointer among k, v, rows, k_pages, v_pages, block_tables");
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(rows, 4) || !aligned(seq, 4) ||
      !aligned(positions, 4) || !aligned(b.tables, 4))
    return fail(RF_E_SHAPE, "q, q_out, k, v and the pages need 16-byte, the index lists 4-byte alignment");
  return RF_OK;
}

// A tensor of heads and what is made of it; strides in elements of `step` to 16 bytes.
rf_status check_heads_of(const char* name, const void* x, int heads, int hd, int64_t stride, int step) {
  if (stride < (int64_t)heads * hd || stride % step)
    return fail(RF_E_SHAPE, "%s: the stride must be >= heads * head_dim and a multiple of %d", name, step);
  if (!aligned(x, 16)) return fail(RF_E_SHAPE, "%s needs 16-byte alignment", name);
  return RF_OK;
}

rf_status check_norm(const rf_head_norm* norm) {
  if (!norm) return RF_OK;
  if (norm->reserved != 0) return fail(RF_E_INVALID, "norm.reserved must be 0");
  if (!(norm->eps >= 0.f) || !std::isfinite(norm->eps)) return fail(RF_E_INVALID, "norm.eps must be finite and >= 0");
  if (!aligned(norm->q_w, 16) || !aligned(norm->k_w, 16))
    return fail(RF_E_SHAPE, "the norms' weights need 16-byte alignment");
  return RF_OK;
}

// What the norm's forward and backward calls share.
rf_status check_norm_call(const rf_rope* rope, const rf_head_norm* norm, int32_t type, int64_t n, int hd, int n_q,
                          int n_k, rf::RopeFreq& f) {
  if (type != RF_TYPE_BF16 && type != RF_TYPE_F32) return fail(RF_E_INVALID, "type = %d", type);
  if (hd < 16 || hd > 256 || hd % 16) return fail(RF_E_SHAPE, "head_dim = %d must be a multiple of 16 up to 256", hd);
  if (n_q < 0 || n_q > 4096 || n_k < 0 || n_k > 4096 || n_q + n_k == 0)
    return fail(RF_E_SHAPE, "n_q_heads = %d and n_k_heads = %d must be in 0..4096, not both 0", n_q, n_k);
  if (n < 0 || n > kMaxRows) return fail(RF_E_SHAPE, "n_rows = %lld must be in 0..2^23", (long long)n);
  f = {};
  f.layout = RF_ROPE_HALF;
  const rf_status s = check_norm(norm);
  return s != RF_OK || !rope ? s : make_freq(rope, hd, f);
}

// One layer's pools.
rf_status check_pools(const rf_cache* cache, const rf::Batch& b, rf::Pools& p) {
  if (!cache) return fail(RF_E_INVALID, "cache is NULL");
  if (cache->type != RF_CACHE_BF16 && cache->type != RF_CACHE_FP8 && cache->type != RF_CACHE_INT8)
    return fail(RF_E_INVALID, "cache.type = %d", cache->type);
  if (cache->reserved != 0) return fail(RF_E_INVALID, "cache.reserved must be 0");
  const bool held = cache->type != RF_CACHE_BF16;
  if (held && b.hd % 32) return fail(RF_E_SHAPE, "head_dim = %d must be a multiple of 32 for 8 bits", b.hd);
  if (held != (cache->k_scales != nullptr) || (held && cache->v_pages && !cache->v_scales) || (!held && cache->v_scales))
    return fail(RF_E_INVALID, "caches of 8 bits have k_scales and v_scales, others have none");
  if (!cache->k_pages) return fail(RF_E_INVALID, "cache.k_pages is NULL");
  if (!aligned(cache->k_pages, 16) || !aligned(cache->v_pages, 16) || !aligned(cache->k_scales, 16) ||
      !aligned(cache->v_scales, 16))
    return fail(RF_E_SHAPE, "the cache's pools need 16-byte alignment");
  p = {cache->type, cache->k_pages, cache->v_pages, cache->k_scales, cache->v_scales};
  return RF_OK;
}

constexpr int64_t kMaxSharedQueries = 1 << 25;   // batch * query heads * max_q of a call with prefixes

// The prefixes of a batch, and that its queries fit a call with them.
rf_status check_prefix(const rf_prefix* pre, const rf::Batch& b, int n_q_heads, int max_q, rf::PrefixCall& p) {
  if (pre->groups < 1 || pre->groups > 65535 || (int64_t)pre->groups * b.n_kv > 1 << 22)
    return fail(RF_E_SHAPE, "prefix.groups = %d must be in 1..65535, times n_kv_heads at most 2^22", pre->groups);
  if (pre->max_len < 1 || pre->max_len > 1 << 30)
    return fail(RF_E_SHAPE, "prefix.max_len = %d must be in 1..2^30", pre->max_len);
  if (pre->table_stride < ((int64_t)pre->max_len + b.page_size - 1) / b.page_size)
    return fail(RF_E_SHAPE, "prefix.table_stride = %lld holds fewer than max_len = %d rows",
                (long long)pre->table_stride, pre->max_len);
  if ((int64_t)b.batch * n_q_heads * max_q > kMaxSharedQueries)
    return fail(RF_E_SHAPE, "batch * n_q_heads * max_q must be at most 2^25 with a prefix");
  p = {pre->block_tables, pre->lengths, pre->group_start, pre->table_stride, pre->groups, pre->max_len};
  return RF_OK;
}

}  // namespace

extern "C" {

rf_status ridgefill_rope(const rf_rope* rope, const void* x, int32_t x_type, int64_t n_rows,
                         int32_t n_heads, int32_t head_dim, int64_t x_stride,
                         const int32_t* positions, void* out, int64_t out_stride,
                         int32_t transpose, void* stream) {
  if (!rope) return fail(RF_E_INVALID, "rope is NULL");
  if (x_type != RF_TYPE_BF16 && x_type != RF_TYPE_F32) return fail(RF_E_INVALID, "x_type = %d", x_type);
  if (head_dim < 16 || head_dim > 256 || head_dim % 16)
    return fail(RF_E_SHAPE, "head_dim = %d must be a multiple of 16 up to 256", head_dim);
  if (n_heads < 1 || n_heads > 4096) return fail(RF_E_SHAPE, "n_heads = %d must be in 1..4096", n_heads);
  if (n_rows < 0 || n_rows > kMaxRows)
    return fail(RF_E_SHAPE, "n_rows = %lld must be in 0..2^23", (long long)n_rows);
  if (transpose != 0 && transpose != 1) return fail(RF_E_INVALID, "transpose must be 0 or 1");
  rf::RopeFreq f;
  rf_status s = make_freq(rope, head_dim, f);
  if (s != RF_OK) return s;
  const int64_t width = (int64_t)n_heads * head_dim;
  const int step = x_type == RF_TYPE_F32 ? 4 : 8;
  if (x_stride < width || out_stride < width || x_stride % step || out_stride % step)
    return fail(RF_E_SHAPE, "strides must be >= n_heads * head_dim and multiples of %d", step);
  if (n_rows == 0) return ok();
  if (!x || !positions || !out) return fail(RF_E_INVALID, "null pointer among x, positions, out");
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4))
    return fail(RF_E_SHAPE, "x and out need 16-byte, positions 4-byte alignment");
  if (x == out && x_stride != out_stride)
    return fail(RF_E_INVALID, "rotating in place needs equal strides");
  const rf::RopeCall c = {x, out, positions, n_rows, x_stride, out_stride, n_heads, head_dim, transpose};
  hipError_t e = rf::launch_rope(f, c, x_type == RF_TYPE_F32, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "rope launch");
  return ok();
}

rf_status ridgefill_append_rows(const rf_rope* rope, const rf_paged_batch* kv, const uint16_t* q,
                                int32_t n_q_heads, int64_t q_stride, uint16_t* q_out,
                                int64_t q_out_stride, const uint16_t* k, int64_t k_stride,
                                const uint16_t* v, int64_t v_stride, int64_t n_rows,
                                const int32_t* seq, const int32_t* rows, const int32_t* positions,
                                uint16_t* k_pages, uint16_t* v_pages, uint32_t* status,
                                void* stream) {
  rf::Batch b;
  rf_status s = check_batch(kv, true, b);
  if (s != RF_OK) return s;
  rf::RopeFreq f;
  s = check_append(rope, b, q, n_q_heads, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, n_rows, seq, rows,
                   positions, k_pages, v_pages, status, f);
  if (s != RF_OK) return s;
  if (n_rows == 0) {
    hipError_t e = rf::launch_clear_status(status, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "status clear");
  }
  const rf::AppendCall c = {q, q_out, k, v, k_pages, v_pages, seq, rows, positions, status,
                            n_rows, q_stride, q_out_stride, k_stride, v_stride, n_q_heads};
  hipError_t e = rf::launch_append(f, b, c, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "append launch");
  return ok();
}

size_t ridgefill_tree_attention_workspace_bytes(const rf_paged_batch* kv, int32_t n_q_heads,
                                                int32_t max_q) {
  rf::Batch b;
  if (check_batch(kv, false, b) != RF_OK || check_heads(b, n_q_heads, max_q) != RF_OK) return 0;
  return rf::attend_workspace(b, n_q_heads, max_q);
}

rf_status ridgefill_tree_attention(const rf_paged_batch* kv, const uint16_t* k_pages,
                                   const uint16_t* v_pages, const uint16_t* q, int32_t n_q_heads,
                                   int64_t q_stride, const int32_t* q_start, int64_t n_q,
                                   int32_t max_q, const uint64_t* tree_mask, float scale,
                                   uint16_t* out, int64_t out_stride, float* lse, void* ws,
                                   size_t ws_bytes, void* stream) {
  rf::Batch b;
  rf_status s = check_batch(kv, false, b);
  if (s == RF_OK)
    s = check_queries(b, q, n_q_heads, q_stride, q_start, n_q, max_q, tree_mask, scale);
  if (s == RF_OK) s = check_memory(b, ws, ws_bytes, rf::attend_workspace(b, n_q_heads, max_q));
  if (s != RF_OK) return s;
  if (!k_pages || (!out && !lse && n_q > 0) || (out && !v_pages))
    return fail(RF_E_INVALID, "k_pages, one of out and lse, and with out v_pages are required");
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return fail(RF_E_SHAPE, "the pages and out need 16-byte, lse 4-byte alignment");
  if (out && (out_stride < (int64_t)n_q_heads * b.hd || out_stride % 8))
    return fail(RF_E_SHAPE, "out_stride must be >= n_q_heads * head_dim and a multiple of 8");
  const rf::Queries Q = {q, q_start, tree_mask, q_stride, n_q, n_q_heads, max_q, scale};
  hipError_t e = rf::launch_attend(b, k_pages, v_pages, Q, out, out_stride, lse, ws,
                                   static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "attention launch");
  return ok();
}

size_t ridgefill_attention_weight_workspace_bytes(const rf_paged_batch* kv, int32_t n_q_heads,
                                                  int32_t max_q) {
  rf::Batch b;
  if (check_batch(kv, false, b) != RF_OK || check_heads(b, n_q_heads, max_q) != RF_OK ||
      check_weights(b) != RF_OK)
    return 0;
  return rf::weight_workspace(b, n_q_heads, max_q);
}

rf_status ridgefill_attention_weight(const rf_paged_batch* kv, const uint16_t* k_pages,
                                     const uint16_t* q, int32_t n_q_heads, int64_t q_stride,
                                     const int32_t* q_start, int64_t n_q, int32_t max_q,
                                     const uint64_t* tree_mask, float scale, const float* lse,
                                     float decay, const float* acc, float* acc_out,
                                     int64_t acc_stride, void* ws, size_t ws_bytes, void* stream) {
  rf::Batch b;
  rf_status s = check_batch(kv, false, b);
  if (s == RF_OK)
    s = check_queries(b, q, n_q_heads, q_stride, q_start, n_q, max_q, tree_mask, scale);
  if (s == RF_OK) s = check_weights(b);
  if (s == RF_OK) s = check_memory(b, ws, ws_bytes, rf::weight_workspace(b, n_q_heads, max_q));
  if (s != RF_OK) return s;
  if (!k_pages || !acc_out || (n_q > 0 && !lse))
    return fail(RF_E_INVALID, "null pointer among k_pages, lse, acc_out");
  if (!std::isfinite(decay)) return fail(RF_E_INVALID, "decay must be finite");
  if (acc_stride < b.max_len) return fail(RF_E_SHAPE, "acc_stride must be >= max_len");
  if (!aligned(k_pages, 16) || !aligned(lse, 4) || !aligned(acc, 4) || !aligned(acc_out, 4))
    return fail(RF_E_SHAPE, "the pages need 16-byte, lse, acc and acc_out 4-byte alignment");
  const rf::Queries Q = {q, q_start, tree_mask, q_stride, n_q, n_q_heads, max_q, scale};
  hipError_t e = rf::launch_weight(b, k_pages, Q, lse, decay, acc, acc_out, acc_stride, ws,
                                   static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "attention-weight launch");
  return ok();
}

size_t ridgefill_evict_workspace_bytes(const rf_paged_batch* kv, int32_t n_keep) {
  rf::Batch b;
  if (check_batch(kv, true, b) != RF_OK || n_keep < 0) return 0;
  return rf::evict_workspace(b, n_keep);
}

rf_status ridgefill_evict_rows(const rf_paged_batch* kv, const rf_layer* layers, int32_t n_layers,
                               const float* acc, const int32_t* positions, int64_t stride,
                               int32_t n_keep, int32_t n_sink, int32_t n_recent, float* acc_out,
                               int32_t* positions_out, int32_t* lengths_out, void* ws,
                               size_t ws_bytes, void* stream) {
  rf::Batch b;
  rf_status s = check_batch(kv, true, b);
  if (s != RF_OK) return s;
  if (n_keep < 0 || n_sink < 0 || n_recent < 0)
    return fail(RF_E_INVALID, "n_keep, n_sink and n_recent must be >= 0");
  if (n_layers < 0 || n_layers > 1024) return fail(RF_E_SHAPE, "n_layers = %d must be in 0..1024", n_layers);
  s = check_memory(b, ws, ws_bytes, rf::evict_workspace(b, n_keep));
  if (s != RF_OK) return s;
  if (!acc || !positions || !acc_out || !positions_out || !lengths_out || (n_layers > 0 && !layers))
    return fail(RF_E_INVALID, "null pointer among layers, acc, positions, acc_out, positions_out, lengths_out");
  if (stride < b.max_len) return fail(RF_E_SHAPE, "stride must be >= max_len");
  if (!aligned(acc, 4) || !aligned(positions, 4) || !aligned(acc_out, 4) ||
      !aligned(positions_out, 4) || !aligned(lengths_out, 4))
    return fail(RF_E_SHAPE, "acc, positions and lengths need 4-byte alignment");
  uint16_t* pools[2 * 1024];
  for (int i = 0; i < n_layers; ++i) {
    if (!layers[i].k_pages || !layers[i].v_pages) return fail(RF_E_INVALID, "layer %d has a null page pool", i);
    if (!aligned(layers[i].k_pages, 16) || !aligned(layers[i].v_pages, 16))
      return fail(RF_E_SHAPE, "layer %d: the pages need 16-byte alignment", i);
    pools[2 * i] = layers[i].k_pages;
    pools[2 * i + 1] = layers[i].v_pages;
  }
  const rf::EvictCall c = {acc, positions, acc_out, positions_out, lengths_out, stride,
                           n_keep, n_sink, n_recent};
  hipError_t e = rf::launch_evict(b, c, pools, 2 * n_layers, ws, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "eviction launch");
  return ok();
}

rf_status ridgefill_norm_rope(const rf_rope* rope, const rf_head_norm* norm, int32_t type,
                              int64_t n_rows, int32_t head_dim, const int32_t* positions,
                              const void* q, int32_t n_q_heads, int64_t q_stride, void* q_out,
                              int64_t q_out_stride, const void* k, int32_t n_k_heads,
                              int64_t k_stride, void* k_out, int64_t k_out_stride, void* stream) {
  rf::RopeFreq f;
  rf_status s = check_norm_call(rope, norm, type, n_rows, head_dim, n_q_heads, n_k_heads, f);
  if (s != RF_OK) return s;
  const int step = type == RF_TYPE_F32 ? 4 : 8;
  const rf::NormTensor t[2] = {
      {q, norm ? norm->q_w : nullptr, nullptr, q_out, nullptr, q_stride, 0, q_out_stride, n_q_heads},
      {k, norm ? norm->k_w : nullptr, nullptr, k_out, nullptr, k_stride, 0, k_out_stride, n_k_heads}};
  for (int i = 0; i < 2; ++i) {
    const char* name = i ? "k" : "q";
    if ((t[i].x || t[i].out) && !t[i].heads) return fail(RF_E_INVALID, "%s without heads", name);
    if (!t[i].heads) continue;
    s = check_heads_of(name, t[i].x, t[i].heads, head_dim, t[i].x_stride, step);
    if (s == RF_OK) s = check_heads_of(i ? "k_out" : "q_out", t[i].out, t[i].heads, head_dim, t[i].out_stride, step);
    if (s != RF_OK) return s;
    if (n_rows > 0 && (!t[i].x || !t[i].out)) return fail(RF_E_INVALID, "%s or its output is NULL", name);
    if (t[i].x && t[i].x == t[i].out && t[i].x_stride != t[i].out_stride)
      return fail(RF_E_INVALID, "%s in place needs equal strides", name);
  }
  if (n_rows == 0) return ok();
  if (rope && !positions) return fail(RF_E_INVALID, "positions is NULL");
  if (!aligned(positions, 4)) return fail(RF_E_SHAPE, "positions needs 4-byte alignment");
  const rf::NormCall c = {{t[0], t[1]}, positions, n_rows, norm ? norm->eps : 0.f, head_dim};
  hipError_t e = rf::launch_norm_rope(f, c, type == RF_TYPE_F32, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "norm launch");
}

size_t ridgefill_norm_rope_grad_workspace_bytes(int64_t n_rows, int32_t n_q_heads,
                                                int32_t n_k_heads, int32_t head_dim) {
  rf::RopeFreq f;
  if (check_norm_call(nullptr, nullptr, RF_TYPE_BF16, n_rows, head_dim, n_q_heads, n_k_heads, f) != RF_OK) return 0;
  return rf::norm_grad_workspace(n_rows, head_dim);
}

rf_status ridgefill_norm_rope_grad(const rf_rope* rope, const rf_head_norm* norm, int32_t type,
                                   int64_t n_rows, int32_t head_dim, const int32_t* positions,
                                   const void* q, int32_t n_q_heads, int64_t q_stride,
                                   const void* gq, int64_t gq_stride, void* q_grad,
                                   int64_t q_grad_stride, float* qw_grad, const void* k,
                                   int32_t n_k_heads, int64_t k_stride, const void* gk,
                                   int64_t gk_stride, void* k_grad, int64_t k_grad_stride,
                                   float* kw_grad, void* ws, size_t ws_bytes, void* stream) {
  rf::RopeFreq f;
  rf_status s = check_norm_call(rope, norm, type, n_rows, head_dim, n_q_heads, n_k_heads, f);
  if (s != RF_OK) return s;
  const int step = type == RF_TYPE_F32 ? 4 : 8;
  const rf::NormTensor t[2] = {
      {q, norm ? norm->q_w : nullptr, gq, q_grad, qw_grad, q_stride, gq_stride, q_grad_stride, n_q_heads},
      {k, norm ? norm->k_w : nullptr, gk, k_grad, kw_grad, k_stride, gk_stride, k_grad_stride, n_k_heads}};
  for (int i = 0; i < 2; ++i) {
    const char* name = i ? "k" : "q";
    if ((t[i].x || t[i].g || t[i].out || t[i].dw) && !t[i].heads) return fail(RF_E_INVALID, "%s without heads", name);
    if (!t[i].heads) continue;
    if (t[i].w) s = check_heads_of(name, t[i].x, t[i].heads, head_dim, t[i].x_stride, step);
    if (s == RF_OK) s = check_heads_of(i ? "gk" : "gq", t[i].g, t[i].heads, head_dim, t[i].g_stride, step);
    if (s == RF_OK) s = check_heads_of(i ? "k_grad" : "q_grad", t[i].out, t[i].heads, head_dim, t[i].out_stride, step);
    if (s != RF_OK) return s;
    if (!aligned(t[i].dw, 4)) return fail(RF_E_SHAPE, "%sw_grad needs 4-byte alignment", name);
    if (n_rows > 0 && (!t[i].g || !t[i].out || (t[i].w && !t[i].x)))
      return fail(RF_E_INVALID, "%s, g%s or %s_grad is NULL", name, name, name);
    if (t[i].g && t[i].g == t[i].out && t[i].g_stride != t[i].out_stride)
      return fail(RF_E_INVALID, "%s_grad in place of g%s needs equal strides", name, name);
  }
  if (qw_grad && qw_grad == kw_grad) return fail(RF_E_INVALID, "qw_grad and kw_grad are the same memory");
  if (n_rows > 0 && rope && !positions) return fail(RF_E_INVALID, "positions is NULL");
  if (!aligned(positions, 4)) return fail(RF_E_SHAPE, "positions needs 4-byte alignment");
  if (!ws) return fail(RF_E_INVALID, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(RF_E_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t need = rf::norm_grad_workspace(n_rows, head_dim);
  if (ws_bytes < need) return fail(RF_E_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
  const rf::NormCall c = {{t[0], t[1]}, positions, n_rows, norm ? norm->eps : 0.f, head_dim};
  hipError_t e = rf::launch_norm_grad(f, c, type == RF_TYPE_F32, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "norm gradient launch");
}

rf_status ridgefill_append_cache(const rf_rope* rope, const rf_head_norm* norm,
                                 const rf_paged_batch* kv, const rf_cache* cache,
                                 const uint16_t* q, int32_t n_q_heads, int64_t q_stride,
                                 uint16_t* q_out, int64_t q_out_stride, const uint16_t* k,
                                 int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                 int64_t n_rows, const int32_t* seq, const int32_t* rows,
                                 const int32_t* positions, uint32_t* status, void* stream) {
  rf::Batch b;
  rf::RopeFreq f;
  rf::HoldCall c = {};
  rf_status s = check_batch(kv, true, b);
  if (s == RF_OK) s = check_pools(cache, b, c.pools);
  if (s == RF_OK) s = check_norm(norm);
  if (s == RF_OK)
    s = check_append(rope, b, q, n_q_heads, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, n_rows, seq, rows,
                     positions, c.pools.k, c.pools.v, status, f);
  if (s != RF_OK) return s;
  if (n_rows == 0) {
    hipError_t e = rf::launch_clear_status(status, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "status clear");
  }
  c.a = {q, q_out, k, v, nullptr, nullptr, seq, rows, positions, status,
         n_rows, q_stride, q_out_stride, k_stride, v_stride, n_q_heads};
  c.q_w = norm ? static_cast<const uint16_t*>(norm->q_w) : nullptr;
  c.k_w = norm ? static_cast<const uint16_t*>(norm->k_w) : nullptr;
  c.eps = norm ? norm->eps : 0.f;
  hipError_t e = rf::launch_hold(f, b, c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "append launch");
}

rf_status ridgefill_read_rows(const rf_paged_batch* kv, const rf_cache* cache, int64_t n_rows,
                              const int32_t* seq, const int32_t* rows, int32_t type, void* k_out,
                              int64_t k_out_stride, void* v_out, int64_t v_out_stride,
                              uint32_t* status, void* stream) {
  rf::Batch b;
  rf::ReadCall c = {};
  rf_status s = check_batch(kv, true, b);
  if (s == RF_OK) s = check_pools(cache, b, c.pools);
  if (s != RF_OK) return s;
  if (type != RF_TYPE_BF16 && type != RF_TYPE_F32) return fail(RF_E_INVALID, "type = %d", type);
  if (!status || !aligned(status, 4))
    return fail(RF_E_INVALID, "status must be a 4-byte aligned device pointer");
  if (n_rows < 0 || n_rows > kMaxRows || n_rows * b.n_kv * b.hd > (int64_t)1 << 34)
    return fail(RF_E_SHAPE, "n_rows = %lld must be in 0..2^23, n_rows * n_kv_heads * head_dim at most 2^34", (long long)n_rows);
  const int step = type == RF_TYPE_F32 ? 4 : 8;
  if (k_out) s = check_heads_of("k_out", k_out, b.n_kv, b.hd, k_out_stride, step);
  if (s == RF_OK && v_out) s = check_heads_of("v_out", v_out, b.n_kv, b.hd, v_out_stride, step);
  if (s != RF_OK) return s;
  if (n_rows == 0) {
    hipError_t e = rf::launch_clear_status(status, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, "status clear");
  }
  if (!rows || !b.tables || (!k_out && !v_out) || (v_out && !c.pools.v))
    return fail(RF_E_INVALID, "null pointer among rows, block_tables, v_pages, or no output");
  if (!aligned(rows, 4) || !aligned(seq, 4) || !aligned(b.tables, 4))
    return fail(RF_E_SHAPE, "the index lists need 4-byte alignment");
  c.k_out = k_out;
  c.v_out = v_out;
  c.seq = seq;
  c.rows = rows;
  c.status = status;
  c.n = n_rows;
  c.k_stride = k_out_stride;
  c.v_stride = v_out_stride;
  hipError_t e = rf::launch_read(b, c, type == RF_TYPE_F32, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "read launch");
}

size_t ridgefill_cache_attention_workspace_bytes(const rf_paged_batch* kv, const rf_prefix* prefix,
                                                 int32_t n_q_heads, int32_t max_q, int64_t n_q) {
  rf::Batch b;
  rf::PrefixCall p;
  if (check_batch(kv, false, b) != RF_OK || check_heads(b, n_q_heads, max_q) != RF_OK || n_q < 0 || n_q > INT32_MAX ||
      (prefix && check_prefix(prefix, b, n_q_heads, max_q, p) != RF_OK))
    return 0;
  return rf::cache_attend_workspace(b, prefix ? &p : nullptr, n_q_heads, max_q, n_q);
}

rf_status ridgefill_cache_attention(const rf_paged_batch* kv, const rf_prefix* prefix,
                                    const rf_cache* cache, const uint16_t* q, int32_t n_q_heads,
                                    int64_t q_stride, const int32_t* q_start, int64_t n_q,
                                    int32_t max_q, const uint64_t* tree_mask, float scale,
                                    uint16_t* out, int64_t out_stride, float* lse, void* ws,
                                    size_t ws_bytes, void* stream) {
  rf::Batch b;
  rf::Pools pools;
  rf::PrefixCall p = {};
  rf_status s = check_batch(kv, false, b);
  if (s == RF_OK) s = check_pools(cache, b, pools);
  if (s == RF_OK)
    s = check_queries(b, q, n_q_heads, q_stride, q_start, n_q, max_q, tree_mask, scale);
  if (s == RF_OK && prefix) s = check_prefix(prefix, b, n_q_heads, max_q, p);
  if (s == RF_OK)
    s = check_memory(b, ws, ws_bytes, rf::cache_attend_workspace(b, prefix ? &p : nullptr, n_q_heads, max_q, n_q));
  if (s != RF_OK) return s;
  if (prefix) {
    if (!p.tables || !p.lengths || !p.starts)
      return fail(RF_E_INVALID, "prefix: block_tables, lengths or group_start is NULL");
    if (!aligned(p.tables, 4) || !aligned(p.lengths, 4) || !aligned(p.starts, 4))
      return fail(RF_E_SHAPE, "prefix: block_tables, lengths and group_start need 4-byte alignment");
  }
  if ((!out && !lse && n_q > 0) || (out && !pools.v))
    return fail(RF_E_INVALID, "one of out and lse, and with out cache.v_pages are required");
  if (!aligned(out, 16) || !aligned(lse, 4)) return fail(RF_E_SHAPE, "out needs 16-byte, lse 4-byte alignment");
  if (out && (out_stride < (int64_t)n_q_heads * b.hd || out_stride % 8))
    return fail(RF_E_SHAPE, "out_stride must be >= n_q_heads * head_dim and a multiple of 8");
  const rf::Queries Q = {q, q_start, tree_mask, q_stride, n_q, n_q_heads, max_q, scale};
  hipError_t e = rf::launch_cache_attend(b, prefix ? &p : nullptr, pools, Q, out, out_stride, lse, ws,
                                         static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "attention launch");
}

}  // extern "C"
