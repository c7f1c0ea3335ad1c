// The C-ABI of the key/value cache: argument checks, the split of attention
// over workgroups, launches.  No allocation, no state.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "nc_kv.h"

using namespace nc;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool valid_dim(int32_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// fmt, dim and page, then sizes: slots and tiles are numbered in 31 bits.
nc_status check_cache(const nc_kv_cache* c, bool data) {
  if (c == nullptr) return NC_E_ARG;
  if ((c->fmt != NC_E2M1 && c->fmt != NC_E4M3) || !valid_dim(c->dim)) return NC_E_UNSUPPORTED;
  if (c->page <= 0 || c->page % kKvTokens != 0) return NC_E_SHAPE;
  if (c->pages < 0 || c->heads < 1) return NC_E_ARG;
  const int64_t most = INT32_MAX;
  if (c->heads > 65536 || c->pages > most / c->page || c->pages * (c->page / kKvTokens) > most / c->heads) return NC_E_ARG;
  if (!data || c->pages == 0) return NC_OK;
  if (c->data == nullptr) return NC_E_ARG;
  return aligned16(c->data) ? NC_OK : NC_E_ALIGN;
}

// 16-byte pieces of rows: pointer and strides.
nc_status check_rows(const void* p, int64_t ts, int64_t hs, nc_dtype dt) {
  const int64_t unit = dt == NC_BF16 ? 8 : 4;
  if (p == nullptr || ts < 0 || hs < 0) return NC_E_ARG;
  return aligned16(p) && ts % unit == 0 && hs % unit == 0 ? NC_OK : NC_E_ALIGN;
}

KvCache cache_of(const nc_kv_cache* c) { 
  return KvCache{c->data, c->pages * c->page, c->page, c->heads, kv_div((uint32_t)(c->page / kKvTokens)), kv_div((uint32_t)c->heads)};
}
nc_status hip_status(hipError_t e) { return e == hipSuccess ? NC_OK : NC_E_HIP; }

nc_status check_tokens(const nc_kv_cache* c, const nc_kv_rows* k, const nc_kv_rows* v, int64_t tokens, nc_dtype dtype,
                       const int64_t* slots) {
  nc_status s = check_cache(c, true);
  if (s != NC_OK) return s;
  if (dtype != NC_F32 && dtype != NC_BF16) return NC_E_UNSUPPORTED;
  // one lane per eight elements, numbered in 32 bits
  if (tokens < 0 || tokens > ((int64_t)1 << 31) || (tokens + 16) * c->heads > ((int64_t)1 << 32) / (c->dim / 8) - 256)
    return NC_E_ARG;
  if (tokens == 0) return NC_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return NC_E_ARG;
  if (((uintptr_t)slots & 7u) != 0) return NC_E_ALIGN;
  if ((s = check_rows(k->data, k->token_stride, k->head_stride, dtype)) != NC_OK) return s;
  return check_rows(v->data, v->token_stride, v->head_stride, dtype);
}

// The split of a call.  span: tiles of 16 keys that a row group may reach.  It
// goes by max_q, as if every sequence had so many queries: a prompt among single
// tokens takes the single tokens to the prompt's kernel (one sequence of 512
// queries among 31 single tokens, 8192 tokens each, 8 heads of 128 x 4, E2M1: 267
// us, and 172 as two calls).
//
// The many-row kernel does 1.6 times the work of the few-row kernel in the same
// time once it has a workgroup for every compute unit (4096 queries over 16384
// keys, 32 heads of 128: 0.93 ms against 1.49), and loses below that (100 over
// 600, 5 x 32 heads, 125 workgroups: 43 us against 25; 312 workgroups: 70
// against 67).
//
// Shares cost a second kernel, about 7 us; without them a workgroup runs through
// all of its keys.  128 tiles take 8 waves 8 steps, about as long.  Where the row
// groups of 16 take most of the compute units, and no more than all, shares gain
// less and 256 tiles are run through (E2M1, heads of 128: a row group each of 32
// sequences of 4000 tokens, 8 heads, 34 us with shares, 26 without; of 16
// sequences of 4090 20 against 23).  Two row groups and more of 16 would be one
// and more of 32 with shares: half of the units do there (16 sequences of 4000,
// 4 heads, 32 rows: 30 against 25).
//
// Without shares and with a compute unit for each row group of 16, groups of 16
// rows and 8 waves take less time than half as many of 32 and 4 waves (5 queries
// of 16 sequences over 1029 keys, 4 heads of 8 query heads: 11 us against 16);
// with more than that the waves get in each other's way (200 over 200, 5 x 15
// heads: 24 against 14).
//
// Shares number all tiles of all row groups in 31 bits, and joining them takes 256 threads for each row; a call
// that may have more goes without them.
constexpr int64_t kDirectTiles = 128;
constexpr int64_t kMostThreads = UINT32_MAX;   // of a launch
int32_t shares_of(int32_t dim, nc_dtype dtype, int64_t groups, int32_t rows, int64_t span) {
  const int64_t all = std::max<int64_t>(1, groups) * span;
  return (int32_t)std::min<int64_t>(kv_few_slots(dtype, dim, rows), (all + kKvShareLeast - 1) / kKvShareLeast);
}

KvPlan plan_of(int32_t dim, nc_dtype dtype, int64_t batch, int64_t heads, int64_t rows_all, int64_t span) {
  KvPlan p = {};
  const int64_t groups = batch * heads * ((rows_all + 15) / 16);
  const bool most = groups >= (rows_all > 16 ? kKvUnits / 2 : kKvUnits * 3 / 4) && groups <= kKvUnits;
  const bool direct = span <= (most ? 2 * kDirectTiles : kDirectTiles);
  if (batch * heads * ((rows_all + kKvManyRows - 1) / kKvManyRows) >= kKvUnits && rows_all > kKvManyRows / 2)
    p.rows = kKvManyRows;
  else
    p.rows = rows_all <= 16 || (direct && groups <= kKvUnits) ? 16 : kv_few_rows(dtype, dim);
  p.row_groups = (int32_t)((rows_all + p.rows - 1) / p.rows);
  const int64_t segments = batch * heads;
  if (p.rows != kKvManyRows && !direct && segments * p.row_groups <= INT32_MAX / (span + 1) &&
      segments * rows_all <= kMostThreads / 256)
    p.shares = shares_of(dim, dtype, segments * p.row_groups, p.rows, span);
  return p;
}

int64_t span_of(int64_t max_kv, int64_t max_q, int64_t window) {
  const int64_t keys = window > 0 ? std::min<int64_t>(max_kv, window + max_q) : max_kv;
  return (keys + kKvTokens - 1) / kKvTokens + (window > 0 ? 1 : 0);
}

nc_status check_sizes(const nc_kv_cache* c, int32_t q_heads, int32_t batch, int32_t max_q, int32_t max_kv) {
  if (batch < 0 || max_q < 0 || max_kv < 0 || q_heads < 1) return NC_E_ARG;
  if (q_heads % c->heads != 0) return NC_E_SHAPE;
  // rows of a sequence and head, and of all, are numbered in 31 bits
  if ((int64_t)max_q * (q_heads / c->heads) > INT32_MAX / 2) return NC_E_ARG;
  if ((int64_t)batch * c->heads > INT32_MAX / std::max<int64_t>(1, (int64_t)max_q * (q_heads / c->heads))) return NC_E_ARG;
  return NC_OK;
}

}  // namespace

extern "C" {

size_t nc_kv_cache_bytes(int64_t pages, int32_t page, int32_t heads, int32_t dim, int32_t fmt) {
  const nc_kv_cache c = {nullptr, pages, page, heads, dim, fmt};
  if (check_cache(&c, false) != NC_OK) return 0;
  return (size_t)(pages * (page / kKvTokens) * heads * kv_tile_bytes(fmt, dim));
}

nc_status nc_kv_write(const nc_kv_cache* c, const nc_kv_rows* k, const nc_kv_rows* v, int64_t tokens, nc_dtype dtype,
                      const int64_t* slots, nc_mx_rule rule, void* stream) {
  if (rule != NC_MX_OCP && rule != NC_MX_PLUS1 && rule != NC_MX_CEIL) return NC_E_UNSUPPORTED;
  const nc_status s = check_tokens(c, k, v, tokens, dtype, slots);
  if (s != NC_OK || tokens == 0) return s;
  return hip_status(launch_kv_write(cache_of(c), c->fmt, c->dim, {k->data, k->token_stride, k->head_stride},
                                    {v->data, v->token_stride, v->head_stride}, dtype, slots, tokens, rule,
                                    (hipStream_t)stream));
}

nc_status nc_kv_read(const nc_kv_cache* c, const nc_kv_rows* k, const nc_kv_rows* v, int64_t tokens, nc_dtype dtype,
                     const int64_t* slots, void* stream) {
  const nc_status s = check_tokens(c, k, v, tokens, dtype, slots);
  if (s != NC_OK || tokens == 0) return s;
  return hip_status(launch_kv_read(cache_of(c), c->fmt, c->dim, {k->data, k->token_stride, k->head_stride},
                                   {v->data, v->token_stride, v->head_stride}, dtype, slots, tokens, (hipStream_t)stream));
}

size_t nc_kv_workspace_bytes(const nc_kv_cache* c, nc_dtype dtype, int32_t q_heads, int32_t batch, int32_t max_q,
                             int32_t max_kv) {
  if (check_cache(c, false) != NC_OK || (dtype != NC_F32 && dtype != NC_BF16)) return 0;
  if (check_sizes(c, q_heads, batch, max_q, max_kv) != NC_OK || batch == 0 || max_q == 0) return 0;
  const int64_t rows = (int64_t)max_q * (q_heads / c->heads), span = span_of(max_kv, max_q, 0) + 1;
  // Enough for every plan of these and of smaller sizes, whether this plan has
  // shares or not: a window, and anything that shrinks, makes fewer tiles.
  if (span <= kDirectTiles) return 0;
  size_t most = 0;
  for (int32_t r = 16; r <= kv_few_rows(dtype, c->dim); r += 16) {
    KvPlan p = {};
    p.rows = r;
    p.shares = shares_of(c->dim, dtype, (int64_t)batch * c->heads * ((rows + r - 1) / r), r, span);
    most = std::max(most, kv_part_bytes(p, c->dim));
    if (rows <= 16) break;
  }
  return most;
}

nc_status nc_kv_attention(const nc_kv_cache* c, const nc_kv_attn* a, nc_dtype dtype, void* ws, size_t ws_bytes,
                          void* stream) {
  nc_status s = check_cache(c, true);
  if (s != NC_OK) return s;
  if (dtype != NC_F32 && dtype != NC_BF16) return NC_E_UNSUPPORTED;
  if (a == nullptr) return NC_E_ARG;
  if ((s = check_sizes(c, a->q_heads, a->batch, a->max_q, a->max_kv)) != NC_OK) return s;
  const float scale2 = a->scale * 1.4426950408889634f;
  if (a->total_q < 0 || a->table_pages < 0 || a->window < 0 || !std::isfinite(scale2)) return NC_E_ARG;
  if (a->batch == 0 || a->max_q == 0 || a->total_q == 0) return NC_OK;
  if (a->q_start == nullptr || a->kv_len == nullptr || (a->table == nullptr && a->table_pages > 0)) return NC_E_ARG;
  if ((s = check_rows(a->q, a->q_token_stride, a->q_head_stride, dtype)) != NC_OK) return s;
  if ((s = check_rows(a->out, a->out_token_stride, a->out_head_stride, dtype)) != NC_OK) return s;
  if (a->lse_token_stride < 0) return NC_E_ARG;
  if ((((uintptr_t)a->q_start | (uintptr_t)a->kv_len | (uintptr_t)a->table | (uintptr_t)a->lse) & 3u) != 0) return NC_E_ALIGN;

  KvAttn k = {};
  k.cache = cache_of(c);
  k.q = {a->q, a->q_token_stride, a->q_head_stride};
  k.out = {a->out, a->out_token_stride, a->out_head_stride};
  k.lse = a->lse;
  k.lse_ts = a->lse_token_stride;
  k.q_start = a->q_start;
  k.kv_len = a->kv_len;
  k.table = a->table;
  k.table_w = c->pages > 0 ? a->table_pages : 0;
  k.batch = a->batch;
  k.total_q = a->total_q;
  k.max_q = a->max_q;
  k.max_kv = std::min(a->max_kv, INT32_MAX - 15);   // a cache's most; the end of its last tile is 2^31 - 16
  k.group = a->q_heads / c->heads;
  k.by_group = kv_div((uint32_t)k.group);
  k.causal = a->causal != 0;
  k.window = a->window;
  // at least the smallest normal number, so that a masked score of -inf stays that; a scale of 0 gives
  // equal weights all the same
  k.scale2 = std::copysign(std::max(std::fabs(scale2), FLT_MIN), a->scale);
  const int64_t rows = (int64_t)a->max_q * k.group;
  const int64_t span = span_of(a->max_kv, a->max_q, a->window);
  const KvPlan p = plan_of(c->dim, dtype, a->batch, c->heads, rows, span);
  k.row_groups = p.row_groups;
  k.by_row_groups = kv_div((uint32_t)p.row_groups);
  k.by_segments = kv_div((uint32_t)(c->heads * p.row_groups));
  k.shares = p.shares;
  k.part = (float*)ws;
  if ((int64_t)a->batch * c->heads * p.row_groups > kMostThreads / 512) return NC_E_ARG;   // 256 or 512 threads each
  if (p.shares > 0 && (ws == nullptr || !aligned16(ws) || ws_bytes < kv_part_bytes(p, c->dim))) return NC_E_WORKSPACE;
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e;
  const bool b16 = dtype == NC_BF16;
  if (p.rows == kKvManyRows) {
    if (c->fmt == NC_E2M1) e = b16 ? kv_many_e2m1_bf16(k, c->dim, st) : kv_many_e2m1_f32(k, c->dim, st);
    else e = b16 ? kv_many_e4m3_bf16(k, c->dim, st) : kv_many_e4m3_f32(k, c->dim, st);
  } else {
    if (c->fmt == NC_E2M1) e = b16 ? kv_few_e2m1_bf16(k, c->dim, p, st) : kv_few_e2m1_f32(k, c->dim, p, st);
    else e = b16 ? kv_few_e4m3_bf16(k, c->dim, p, st) : kv_few_e4m3_f32(k, c->dim, p, st);
  }
  if (e == hipSuccess && p.shares > 0) e = launch_kv_join(k, c->dim, dtype, p, st);
  return hip_status(e);
}

}  // extern "C"
