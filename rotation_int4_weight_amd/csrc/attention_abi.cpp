// attention_abi.cpp - C-ABI of the attention and key-value cache entry
// points: argument validation, workspace layout and launch-error mapping.
// Declarations and the contract of every entry point are in include/paro.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "abi.hpp"
#include "attention.hpp"
#include "paro.h"

namespace {

using paro::act_dtype;
using paro::align_up;
using paro::aligned;
using paro::fail;
using paro::hip_fail;
using paro::kCounterBytes;
using paro::ok;
using paro::overlap;

constexpr int64_t kMaxRows = int64_t(1) << 21;
constexpr int kMaxHeads = 256;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxTokenStride = int64_t(1) << 24;  // a tile of 64 keys is loaded with 32-bit offsets
constexpr int64_t kMaxPool = int64_t(1) << 22;
constexpr int64_t kMaxTable = int64_t(1) << 20;
constexpr int64_t kMaxLength = int64_t(1) << 30;
constexpr int kMaxLayers = 1024;
static_assert((size_t)paro::kDecodeCounters * 4 <= paro::kCounterBytes, "the join's counters fit the counter area");

int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

int check_head_dim(int d) {
  if (d != 64 && d != 128) return fail(PARO_ERR_UNSUPPORTED, "head_dim=%d: the GPU path supports 64 and 128", d);
  return PARO_OK;
}

int32_t *kv_work(void *workspace) { return (int32_t *)((char *)workspace + kCounterBytes); }

int64_t page_elements(const paro_kv_cache *c) { return (int64_t)c->kv_heads * c->page_size * c->head_dim; }
size_t pool_bytes(const paro_kv_cache *c) { return (size_t)c->layers * c->num_pages * page_elements(c) * 2; }

// Sizes and tables; `data`: K and V are needed too.
int check_cache(const paro_kv_cache *c, bool data) {
  if (!c) return fail(PARO_ERR_NULL, "cache is NULL");
  int rc = check_head_dim(c->head_dim);
  if (rc) return rc;
  if (page_shift(c->page_size) < 0)
    return fail(PARO_ERR_UNSUPPORTED, "page_size=%d must be 16, 32, 64, 128 or 256", c->page_size);
  if (c->layers < 1 || c->layers > kMaxLayers)
    return fail(PARO_ERR_SHAPE, "layers=%d must be in 1..%d", c->layers, kMaxLayers);
  if (c->kv_heads < 1 || c->kv_heads > kMaxHeads)
    return fail(PARO_ERR_SHAPE, "kv_heads=%d must be in 1..%d", c->kv_heads, kMaxHeads);
  if (c->num_pages < 1 || c->num_pages > kMaxPool)
    return fail(PARO_ERR_SHAPE, "num_pages=%lld must be in 1..%lld", (long long)c->num_pages, (long long)kMaxPool);
  if (c->slots < 1 || c->slots > paro::kMaxSlots)
    return fail(PARO_ERR_SHAPE, "slots=%d must be in 1..%d", c->slots, paro::kMaxSlots);
  if (c->max_pages < 1 || c->max_pages > kMaxTable || (int64_t)c->max_pages * c->page_size > kMaxLength)
    return fail(PARO_ERR_SHAPE, "max_pages=%d must be in 1..%lld and max_pages * page_size at most %lld", c->max_pages,
                (long long)kMaxTable, (long long)kMaxLength);
  if (!act_dtype(c->dt)) return fail(PARO_ERR_DTYPE, "cache dtype %d must be F16 or BF16", (int)c->dt);
  if (!c->refs || !c->table || !c->lengths) return fail(PARO_ERR_NULL, "refs, table and lengths are required");
  if (!aligned(c->refs, 4) || !aligned(c->table, 4) || !aligned(c->lengths, 4))
    return fail(PARO_ERR_ALIGN, "refs, table and lengths must be 4-byte aligned");
  const size_t rb = (size_t)c->num_pages * 4, tb = (size_t)c->slots * c->max_pages * 4, lb = (size_t)c->slots * 4;
  if (overlap(c->refs, rb, c->table, tb) || overlap(c->refs, rb, c->lengths, lb) ||
      overlap(c->table, tb, c->lengths, lb))
    return fail(PARO_ERR_SHAPE, "refs, table and lengths must not overlap");
  if (data) {
    if (!c->k || !c->v) return fail(PARO_ERR_NULL, "the cache's k and v are required");
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
      return fail(PARO_ERR_ALIGN, "the cache's k and v must be 16-byte aligned");
    const size_t pb = pool_bytes(c);
    if (overlap(c->k, pb, c->v, pb)) return fail(PARO_ERR_SHAPE, "the cache's k and v overlap");
  }
  return PARO_OK;
}

int check_layer(const paro_kv_cache *c, int layer) {
  if (layer < 0 || layer >= c->layers) return fail(PARO_ERR_SHAPE, "layer=%d must be in 0..%d", layer, c->layers - 1);
  return PARO_OK;
}

paro::KvLayer kv_layer(const paro_kv_cache *c, int layer) {
  paro::KvLayer kv;
  const int64_t at = (int64_t)layer * c->num_pages * page_elements(c);
  kv.k = (uint16_t *)c->k + at;
  kv.v = (uint16_t *)c->v + at;
  kv.table = c->table;
  kv.lengths = c->lengths;
  kv.page_stride = page_elements(c);
  kv.num_pages = (int)c->num_pages;
  kv.max_pages = c->max_pages;
  kv.slots = c->slots;
  kv.page_shift = page_shift(c->page_size);
  return kv;
}

int check_heads(const paro_attention_shape *s) {
  if (!s) return fail(PARO_ERR_NULL, "shape is NULL");
  int rc = check_head_dim(s->head_dim);
  if (rc) return rc;
  if (s->kv_heads < 1 || s->q_heads < 1 || s->q_heads > kMaxHeads || s->q_heads % s->kv_heads)
    return fail(PARO_ERR_SHAPE, "q_heads=%d must be a multiple of kv_heads=%d in 1..%d", s->q_heads, s->kv_heads,
                kMaxHeads);
  // the kernels work in base 2: an infinite scale * log2(e) would make NaN of a score of 0
  if (!(std::fabs(s->scale) <= 0x1p127f)) return fail(PARO_ERR_SHAPE, "scale must be finite and at most 2^127 in size");
  return PARO_OK;
}

int check_stride(int64_t s, const char *what) {
  if (s < 0 || s >= kMaxStride || s % 8)
    return fail(PARO_ERR_SHAPE, "%s=%lld must be a multiple of 8 elements in 0..2^40", what, (long long)s);
  return PARO_OK;
}

// Bytes from the first to past the last element of a strided tensor.
size_t extent(int64_t rows, int heads, int dim, int64_t token, int64_t head) {
  return rows <= 0 ? 0 : (size_t)((rows - 1) * token + (heads - 1) * head + dim) * 2;
}

// y's rows and heads lie apart from each other.
int check_output_strides(const paro_attention_shape *s, int64_t rows) {
  const int64_t d = s->head_dim;
  const bool heads_inside = (s->q_heads == 1 || s->y_head >= d) &&
                            (rows <= 1 || s->y_token >= (s->q_heads - 1) * s->y_head + d);
  const bool rows_inside = (rows <= 1 || s->y_token >= d) &&
                           (s->q_heads == 1 || s->y_head >= (rows - 1) * s->y_token + d);
  if (!heads_inside && !rows_inside)
    return fail(PARO_ERR_SHAPE, "y strides (token %lld, head %lld) make rows or heads overlap", (long long)s->y_token,
                (long long)s->y_head);
  return PARO_OK;
}

int check_qy(const paro_attention_shape *s, const void *q, const void *y, int64_t rows) {
  int rc = check_stride(s->q_token, "q_token");
  if (!rc) rc = check_stride(s->q_head, "q_head");
  if (!rc) rc = check_stride(s->y_token, "y_token");
  if (!rc) rc = check_stride(s->y_head, "y_head");
  if (!rc) rc = check_output_strides(s, rows);
  if (rc) return rc;
  if (!q || !y) return fail(PARO_ERR_NULL, "q and y are required");
  if (!aligned(q, 16) || !aligned(y, 16)) return fail(PARO_ERR_ALIGN, "q and y must be 16-byte aligned");
  if (overlap(q, extent(rows, s->q_heads, s->head_dim, s->q_token, s->q_head), y,
              extent(rows, s->q_heads, s->head_dim, s->y_token, s->y_head)))
    return fail(PARO_ERR_SHAPE, "y overlaps q");
  return PARO_OK;
}

int check_cache_and_shape(const paro_kv_cache *c, int layer, const paro_attention_shape *s) {
  int rc = check_cache(c, true);
  if (!rc) rc = check_layer(c, layer);
  if (!rc) rc = check_heads(s);
  if (rc) return rc;
  if (s->kv_heads != c->kv_heads || s->head_dim != c->head_dim)
    return fail(PARO_ERR_SHAPE, "shape has %d kv heads of %d channels, the cache %d of %d", s->kv_heads, s->head_dim,
                c->kv_heads, c->head_dim);
  return PARO_OK;
}

// (k and v: where the call has them)
bool overlaps_cache(const paro_kv_cache *c, const void *p, size_t bytes) {
  return (c->k && overlap(p, bytes, c->k, pool_bytes(c))) || (c->v && overlap(p, bytes, c->v, pool_bytes(c))) ||
         overlap(p, bytes, c->table, (size_t)c->slots * c->max_pages * 4) ||
         overlap(p, bytes, c->lengths, (size_t)c->slots * 4) || overlap(p, bytes, c->refs, (size_t)c->num_pages * 4);
}

int check_apart_from_cache(const paro_kv_cache *c, const paro_attention_shape *s, const void *y, int64_t rows) {
  if (overlaps_cache(c, y, extent(rows, s->q_heads, s->head_dim, s->y_token, s->y_head)))
    return fail(PARO_ERR_SHAPE, "y overlaps the cache");
  return PARO_OK;
}

paro::AttentionArgs attention_args(const paro_attention_shape *s, const void *q, void *y, paro_dtype dt) {
  paro::AttentionArgs a = {};
  a.q = (const uint16_t *)q;
  a.y = (uint16_t *)y;
  a.q_token = s->q_token;
  a.q_head = s->q_head;
  a.k_token = s->k_token;
  a.k_head = s->k_head;
  a.v_token = s->v_token;
  a.v_head = s->v_head;
  a.y_token = s->y_token;
  a.y_head = s->y_head;
  a.q_heads = s->q_heads;
  a.kv_heads = s->kv_heads;
  a.group = s->q_heads / s->kv_heads;
  a.head_dim = s->head_dim;
  a.dt = (int)dt;
  a.causal = s->causal != 0;
  a.scale = s->scale;
  return a;
}

int check_rows(int64_t n, const char *what, int64_t most) {
  if (n < 0) return fail(PARO_ERR_SHAPE, "%s=%lld is negative", what, (long long)n);
  if (n > most) return fail(PARO_ERR_UNSUPPORTED, "%s=%lld exceeds %lld", what, (long long)n, (long long)most);
  return PARO_OK;
}

// n entries of the bookkeeping calls
int check_entries(int64_t n) {
  if (n < 0 || n > paro::kMaxSlots)
    return fail(PARO_ERR_SHAPE, "n=%lld must be in 0..%d", (long long)n, paro::kMaxSlots);
  return PARO_OK;
}

int check_kv_workspace(const paro_kv_cache *c, const void *workspace, size_t bytes) {
  const size_t need = paro_kv_workspace_bytes(c);
  if (!workspace || bytes < need)
    return fail(PARO_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace ? bytes : 0, need);
  if (!aligned(workspace, 16)) return fail(PARO_ERR_ALIGN, "workspace must be 16-byte aligned");
  if (overlaps_cache(c, workspace, need))
    return fail(PARO_ERR_SHAPE, "the workspace overlaps the cache");
  return PARO_OK;
}

// An int32 list of the caller's that a bookkeeping call reads or writes.
int check_list(const paro_kv_cache *c, const void *p, int64_t n, const void *workspace, const char *what) {
  if (!p) return fail(PARO_ERR_NULL, "%s is required", what);
  if (!aligned(p, 4)) return fail(PARO_ERR_ALIGN, "%s must be 4-byte aligned", what);
  const size_t b = (size_t)n * 4;
  if (overlaps_cache(c, p, b) || (workspace && overlap(p, b, workspace, paro_kv_workspace_bytes(c))))
    return fail(PARO_ERR_SHAPE, "%s overlaps the cache or the workspace", what);
  return PARO_OK;
}

}  // namespace

extern "C" {

int paro_attention_prompt(const paro_attention_shape *s, const void *q, const void *k, const void *v, paro_dtype dt,
                          const int64_t *cu_q, const int64_t *cu_k, int64_t sequences, int64_t q_tokens,
                          int64_t k_tokens, void *y, void *stream) {
  int rc = check_heads(s);
  if (!rc) rc = check_rows(q_tokens, "q_tokens", kMaxRows);
  if (!rc) rc = check_rows(k_tokens, "k_tokens", kMaxRows);
  if (!rc) rc = check_rows(sequences, "sequences", paro::kMaxSequences);
  if (rc) return rc;
  if (!act_dtype(dt)) return fail(PARO_ERR_DTYPE, "dtype %d must be F16 or BF16", (int)dt);
  if (q_tokens == 0 || sequences == 0) return ok();
  if ((rc = check_qy(s, q, y, q_tokens))) return rc;
  if ((rc = check_stride(s->k_token, "k_token")) || (rc = check_stride(s->k_head, "k_head")) ||
      (rc = check_stride(s->v_token, "v_token")) || (rc = check_stride(s->v_head, "v_head")))
    return rc;
  if (s->k_token > kMaxTokenStride || s->v_token > kMaxTokenStride)
    return fail(PARO_ERR_UNSUPPORTED, "k_token=%lld, v_token=%lld: at most %lld", (long long)s->k_token,
                (long long)s->v_token, (long long)kMaxTokenStride);
  if (!cu_q || !cu_k) return fail(PARO_ERR_NULL, "cu_q and cu_k are required");
  if (!aligned(cu_q, 8) || !aligned(cu_k, 8)) return fail(PARO_ERR_ALIGN, "cu_q and cu_k must be 8-byte aligned");
  if (k_tokens > 0 && (!k || !v)) return fail(PARO_ERR_NULL, "k and v are required");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(PARO_ERR_ALIGN, "k and v must be 16-byte aligned");
  const size_t yb = extent(q_tokens, s->q_heads, s->head_dim, s->y_token, s->y_head);
  if (overlap(y, yb, k, extent(k_tokens, s->kv_heads, s->head_dim, s->k_token, s->k_head)) ||
      overlap(y, yb, v, extent(k_tokens, s->kv_heads, s->head_dim, s->v_token, s->v_head)))
    return fail(PARO_ERR_SHAPE, "y overlaps k or v");
  if (overlap(y, yb, cu_q, (size_t)(sequences + 1) * 8) || overlap(y, yb, cu_k, (size_t)(sequences + 1) * 8))
    return fail(PARO_ERR_SHAPE, "y overlaps cu_q or cu_k");
  paro::AttentionArgs a = attention_args(s, q, y, dt);
  a.k = (const uint16_t *)k;
  a.v = (const uint16_t *)v;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.sequences = (int)sequences;
  a.q_tokens = q_tokens;
  a.k_tokens = k_tokens;
  hipError_t e = paro::launch_attention_prompt(a, false, 1, nullptr, nullptr, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "prompt attention launch");
  return ok();
}

size_t paro_attention_prompt_cached_workspace_bytes(const paro_kv_cache *c, int64_t sequences, int64_t q_tokens,
                                                    int q_heads) {
  if (check_cache(c, false) || sequences <= 0 || sequences > paro::kMaxSequences || q_tokens <= 0 ||
      q_tokens > kMaxRows || q_heads < 1 || q_heads > kMaxHeads || q_heads % c->kv_heads)
    return 0;
  const int splits = paro::attention_prompt_splits(q_tokens, sequences, q_heads, c->kv_heads,
                                                   (int64_t)c->max_pages * c->page_size);
  if (splits == 1) return 0;
  return kCounterBytes +
         paro::attention_prompt_partial_bytes(splits, q_tokens, sequences, q_heads, c->kv_heads, c->head_dim);
}

int paro_attention_prompt_cached(const paro_kv_cache *c, int layer, const paro_attention_shape *s, const void *q,
                                 const int32_t *slots, const int64_t *cu_q, int64_t sequences, int64_t q_tokens,
                                 void *y, void *workspace, size_t workspace_bytes, void *stream) {
  int rc = check_cache_and_shape(c, layer, s);
  if (!rc) rc = check_rows(q_tokens, "q_tokens", kMaxRows);
  if (!rc) rc = check_rows(sequences, "sequences", paro::kMaxSequences);
  if (rc) return rc;
  if (q_tokens == 0 || sequences == 0) return ok();
  if ((rc = check_qy(s, q, y, q_tokens)) || (rc = check_apart_from_cache(c, s, y, q_tokens))) return rc;
  if (!slots || !cu_q) return fail(PARO_ERR_NULL, "slots and cu_q are required");
  if (!aligned(slots, 4) || !aligned(cu_q, 8))
    return fail(PARO_ERR_ALIGN, "slots must be 4-byte aligned, cu_q 8-byte aligned");
  const size_t yb = extent(q_tokens, s->q_heads, s->head_dim, s->y_token, s->y_head);
  if (overlap(y, yb, cu_q, (size_t)(sequences + 1) * 8) || overlap(y, yb, slots, (size_t)sequences * 4))
    return fail(PARO_ERR_SHAPE, "y overlaps cu_q or slots");
  const size_t need = paro_attention_prompt_cached_workspace_bytes(c, sequences, q_tokens, s->q_heads);
  const bool split = workspace && need > 0;
  if (split) {
    if (workspace_bytes < need)
      return fail(PARO_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
    if (!aligned(workspace, 16)) return fail(PARO_ERR_ALIGN, "workspace must be 16-byte aligned");
    if (overlap(workspace, need, y, yb) ||
        overlap(workspace, need, q, extent(q_tokens, s->q_heads, s->head_dim, s->q_token, s->q_head)) ||
        overlap(workspace, need, cu_q, (size_t)(sequences + 1) * 8) ||
        overlap(workspace, need, slots, (size_t)sequences * 4) || overlaps_cache(c, workspace, need))
      return fail(PARO_ERR_SHAPE, "the workspace overlaps q, y, cu_q, slots or the cache");
  }
  paro::AttentionArgs a = attention_args(s, q, y, c->dt);
  a.cu_q = cu_q;
  a.slots = slots;
  a.sequences = (int)sequences;
  a.q_tokens = q_tokens;
  a.kv = kv_layer(c, layer);
  hipError_t e = paro::launch_attention_prompt(
      a, true,
      split ? paro::attention_prompt_splits(q_tokens, sequences, s->q_heads, c->kv_heads,
                                            (int64_t)c->max_pages * c->page_size)
            : 1,
      split ? (uint32_t *)workspace : nullptr, split ? (float *)((char *)workspace + kCounterBytes) : nullptr,
      (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "cached prompt attention launch");
  return ok();
}

size_t paro_attention_decode_workspace_bytes(const paro_kv_cache *c, int64_t rows, int q_heads) {
  if (check_cache(c, false) || rows <= 0 || rows > paro::kMaxDecodeRows || q_heads < 1 || q_heads > kMaxHeads ||
      q_heads % c->kv_heads)
    return 0;
  const paro::DecodeAttentionPlan p =
      paro::plan_attention_decode(rows, q_heads, c->kv_heads, (int64_t)c->max_pages * c->page_size);
  return kCounterBytes + paro::attention_decode_partial_bytes(p, rows, c->kv_heads, c->head_dim);
}

int paro_attention_decode(const paro_kv_cache *c, int layer, const paro_attention_shape *s, const void *q,
                          const int32_t *slots, int64_t rows, void *y, void *workspace, size_t workspace_bytes,
                          void *stream) {
  int rc = check_cache_and_shape(c, layer, s);
  if (!rc) rc = check_rows(rows, "rows", paro::kMaxDecodeRows);
  if (rc) return rc;
  if (rows == 0) return ok();
  if ((rc = check_qy(s, q, y, rows)) || (rc = check_apart_from_cache(c, s, y, rows))) return rc;
  if (!slots) return fail(PARO_ERR_NULL, "slots is required");
  if (!aligned(slots, 4)) return fail(PARO_ERR_ALIGN, "slots must be 4-byte aligned");
  const size_t yb = extent(rows, s->q_heads, s->head_dim, s->y_token, s->y_head);
  if (overlap(y, yb, slots, (size_t)rows * 4)) return fail(PARO_ERR_SHAPE, "y overlaps slots");
  const size_t need = paro_attention_decode_workspace_bytes(c, rows, s->q_heads);
  if (!workspace || workspace_bytes < need)
    return fail(PARO_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace ? workspace_bytes : 0, need);
  if (!aligned(workspace, 16)) return fail(PARO_ERR_ALIGN, "workspace must be 16-byte aligned");
  if (overlap(workspace, need, y, yb) ||
      overlap(workspace, need, q, extent(rows, s->q_heads, s->head_dim, s->q_token, s->q_head)) ||
      overlap(workspace, need, slots, (size_t)rows * 4) || overlaps_cache(c, workspace, need))
    return fail(PARO_ERR_SHAPE, "the workspace overlaps q, y, slots or the cache");
  paro::AttentionArgs a = attention_args(s, q, y, c->dt);
  a.slots = slots;
  a.sequences = (int)rows;
  a.q_tokens = rows;
  a.kv = kv_layer(c, layer);
  const paro::DecodeAttentionPlan p =
      paro::plan_attention_decode(rows, s->q_heads, c->kv_heads, (int64_t)c->max_pages * c->page_size);
  hipError_t e = paro::launch_attention_decode(a, p, (uint32_t *)workspace,
                                               (float *)((char *)workspace + kCounterBytes),
                                               (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "decode attention launch");
  return ok();
}

int paro_kv_append(const paro_kv_cache *c, int layer, const void *k, int64_t k_token, int64_t k_head, const void *v,
                   int64_t v_token, int64_t v_head, const int32_t *slots, const int64_t *cu, const int32_t *granted,
                   int64_t n, int64_t tokens, void *stream) {
  int rc = check_cache(c, true);
  if (!rc) rc = check_layer(c, layer);
  if (!rc) rc = check_rows(n, "n", paro::kMaxSequences);
  if (!rc) rc = check_rows(tokens, "tokens", kMaxRows);
  if (rc) return rc;
  if (!cu && tokens != n)
    return fail(PARO_ERR_SHAPE, "without cu there is one row per entry: tokens=%lld, n=%lld", (long long)tokens,
                (long long)n);
  if (tokens == 0 || n == 0) return ok();
  if ((rc = check_stride(k_token, "k_token")) || (rc = check_stride(k_head, "k_head")) ||
      (rc = check_stride(v_token, "v_token")) || (rc = check_stride(v_head, "v_head")))
    return rc;
  if (!k || !v || !slots) return fail(PARO_ERR_NULL, "k, v and slots are required");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(PARO_ERR_ALIGN, "k and v must be 16-byte aligned");
  if (!aligned(slots, 4) || !aligned(cu, 8) || !aligned(granted, 4))
    return fail(PARO_ERR_ALIGN, "slots and granted must be 4-byte aligned, cu 8-byte aligned");
  const size_t pb = pool_bytes(c), kb = extent(tokens, c->kv_heads, c->head_dim, k_token, k_head),
               vb = extent(tokens, c->kv_heads, c->head_dim, v_token, v_head);
  if (overlap(k, kb, c->k, pb) || overlap(k, kb, c->v, pb) || overlap(v, vb, c->k, pb) || overlap(v, vb, c->v, pb))
    return fail(PARO_ERR_SHAPE, "k or v overlaps the cache");
  if (overlaps_cache(c, slots, (size_t)n * 4) || (cu && overlaps_cache(c, cu, (size_t)(n + 1) * 8)) ||
      (granted && overlaps_cache(c, granted, (size_t)n * 4)))
    return fail(PARO_ERR_SHAPE, "slots, cu or granted overlaps the cache");
  hipError_t e = paro::launch_kv_append(kv_layer(c, layer), c->kv_heads, c->head_dim, (const uint16_t *)k, k_token,
                                        k_head, (const uint16_t *)v, v_token, v_head, slots, cu, granted,
                                        (int)n, tokens,
                                        (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv append launch");
  return ok();
}

size_t paro_kv_workspace_bytes(const paro_kv_cache *c) {
  if (check_cache(c, false)) return 0;
  return kCounterBytes + paro::kv_work_ints(*c) * 4;
}

int paro_kv_reserve(const paro_kv_cache *c, const int32_t *slots, const int32_t *grow, int64_t n, int32_t *granted,
                    void *workspace, size_t workspace_bytes, void *stream) {
  int rc = check_cache(c, true);
  if (!rc) rc = check_entries(n);
  if (rc) return rc;
  if (n == 0) return ok();
  if ((rc = check_kv_workspace(c, workspace, workspace_bytes)) ||
      (rc = check_list(c, slots, n, workspace, "slots")) || (rc = check_list(c, grow, n, workspace, "grow")) ||
      (rc = check_list(c, granted, n, workspace, "granted")))
    return rc;
  if (overlap(granted, (size_t)n * 4, slots, (size_t)n * 4) || overlap(granted, (size_t)n * 4, grow, (size_t)n * 4))
    return fail(PARO_ERR_SHAPE, "granted overlaps slots or grow");
  hipError_t e = paro::launch_kv_reserve(*c, slots, grow, (int)n, granted, kv_work(workspace), (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv reserve launch");
  return ok();
}

int paro_kv_fork(const paro_kv_cache *c, const int32_t *parents, const int32_t *children, int64_t n, int32_t *granted,
                 void *workspace, size_t workspace_bytes, void *stream) {
  int rc = check_cache(c, false);
  if (!rc) rc = check_entries(n);
  if (rc) return rc;
  if (n == 0) return ok();
  if ((rc = check_kv_workspace(c, workspace, workspace_bytes)) ||
      (rc = check_list(c, parents, n, workspace, "parents")) ||
      (rc = check_list(c, children, n, workspace, "children")) ||
      (rc = check_list(c, granted, n, workspace, "granted")))
    return rc;
  if (overlap(granted, (size_t)n * 4, parents, (size_t)n * 4) ||
      overlap(granted, (size_t)n * 4, children, (size_t)n * 4))
    return fail(PARO_ERR_SHAPE, "granted overlaps parents or children");
  hipError_t e =
      paro::launch_kv_fork(*c, parents, children, (int)n, granted, kv_work(workspace), (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv fork launch");
  return ok();
}

int paro_kv_free(const paro_kv_cache *c, const int32_t *slots, int64_t n, void *stream) {
  int rc = check_cache(c, false);
  if (!rc) rc = check_entries(n);
  if (rc) return rc;
  if (n == 0) return ok();
  if ((rc = check_list(c, slots, n, nullptr, "slots"))) return rc;
  hipError_t e = paro::launch_kv_free(*c, slots, (int)n, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv free launch");
  return ok();
}

int paro_kv_compact(const paro_kv_cache *c, int32_t *used, void *workspace, size_t workspace_bytes, void *stream) {
  int rc = check_cache(c, true);
  if (rc) return rc;
  if ((rc = check_kv_workspace(c, workspace, workspace_bytes)) || (rc = check_list(c, used, 1, workspace, "used")))
    return rc;
  hipError_t e = paro::launch_kv_compact(*c, used, kv_work(workspace), (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv compact launch");
  return ok();
}

}  // extern "C"
