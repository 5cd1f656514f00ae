// C entry points of the operators around a paged cache (include/mattn.h): argument
// checks, TMA views, workspace layout and launches.  Nothing here allocates device
// memory but the device's error word on its first use (mattn_decode_paged,
// mattn_attention_packed); mattn_cache_write and mattn_cache_read need none.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "kernel_params.h"
#include "launch_prep.h"
#include "mattn.h"
#include "op_checks.h"
#include "paged_ops.h"
#include "plan_rules.h"

namespace mattn {
namespace {

// Test hook: the copies that the next launches leave out (DecodePagedParams, PackedParams).
std::atomic<int> g_wait_selftest{0};

bool cache_dtype(int t) { return t == MATTN_BF16 || t == MATTN_E4M3; }

// Whether x[..] of three dimensions with these strides (in elements, rows of d last)
// lies in rows that do not overlap: sorted by stride, each dimension steps over the
// whole of those below it.
bool rows_apart(const int64_t (&stride)[3], const int64_t (&size)[3], int64_t row) {
  int o[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[o[j]] > stride[o[j + 1]]) {
        const int x = o[j];
        o[j] = o[j + 1];
        o[j + 1] = x;
      }
  int64_t end = row;
  for (int i = 0; i < 3; ++i) {
    if (size[o[i]] == 1) continue;
    if (stride[o[i]] < end) return false;
    end += stride[o[i]] * (size[o[i]] - 1);
  }
  return true;
}

// Rows in memory: rows of `row` bytes at base + sum i_j stride_j, 0 <= i_j < size_j (in bytes;
// the rows of one do not overlap: rows_apart).
struct RowSet {
  const void* base;
  int64_t stride[3], size[3], row;
  Extent extent() const {
    uint64_t end = row;
    for (int j = 0; j < 3; ++j) end += (uint64_t)(size[j] - 1) * stride[j];
    return extent_of(base, size[0] ? end : 0);
  }
};

// Whether -lb < at + sum n_j stride_j < la for some |n_j| < size_j, j from i on: the largest
// stride left takes the sum to within itself of 0, as those below it span less, or it does not.
bool rows_meet(int64_t at, const int64_t* stride, const int64_t* size, int i, int n, int64_t la, int64_t lb) {
  if (i == n) return at > -lb && at < la;
  const int64_t s = stride[i], f = -(at >= 0 ? (at + s - 1) / s : -(-at / s));  // floor(-at / s)
  for (int64_t x = f; x <= f + 1; ++x)
    if (x > -size[i] && x < size[i] && rows_meet(at + x * s, stride, size, i + 1, n, la, lb)) return true;
  return false;
}

// Whether two sets share no byte.  Sets whose extents meet may be interleaved (k and v of one
// pool, codes beside their exponents): with the same strides, or page by page with the same
// stride from one page to the next.  Other ways are not told apart from an overlap.
bool apart(const RowSet& a, const RowSet& b) {
  if (!a.extent().meets(b.extent())) return true;
  const int64_t at = (int64_t)(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
  int64_t stride[3], size[3];
  int n = 0;
  bool same = true;
  for (int j = 0; j < 3; ++j) {
    same = same && a.size[j] == b.size[j] && (a.size[j] == 1 || a.stride[j] == b.stride[j]);
    if (a.size[j] == 1) continue;
    int i = n++;  // (largest stride first)
    for (; i > 0 && stride[i - 1] < a.stride[j]; --i) {
      stride[i] = stride[i - 1];
      size[i] = size[i - 1];
    }
    stride[i] = a.stride[j];
    size[i] = a.size[j];
  }
  if (same) return !rows_meet(at, stride, size, 0, n, a.row, b.row);
  const int64_t page = a.stride[0];
  if (a.size[0] == 1 || a.size[0] != b.size[0] || page != b.stride[0]) return false;
  auto span = [](const RowSet& x) { return (x.size[1] - 1) * x.stride[1] + (x.size[2] - 1) * x.stride[2] + x.row; };
  const int64_t r = (at % page + page) % page;
  return r >= span(a) && r + span(b) <= page;
}

// The same of the rows of k and v (or of their exponents), whose pages of one number must be
// apart.  A page of one number may be another's of the other tensor, in one pool from whose
// numbers the table gives each sequence its own (k in the even ones, v a page behind): sets a
// whole number of pages apart.
bool pages_apart(const RowSet& a, const RowSet& b) {
  RowSet x = a, y = b;
  x.size[0] = y.size[0] = 1;
  const int64_t at = (int64_t)(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
  return apart(x, y) && ((a.stride[0] == b.stride[0] && at % a.stride[0] == 0) || apart(a, b));
}

int check_cache(const char* what, const mattn_paged_cache* c, int B, int H_kv, int d) {
  if (!c) return report_error(MATTN_ERR_INVALID_ARG, "%s: the cache is NULL", what);
  if (B < 1 || H_kv < 1) return report_error(MATTN_ERR_INVALID_ARG, "%s: B and H_kv must be >= 1", what);
  if (d != 64 && d != 128 && d != 256)
    return report_error(MATTN_ERR_UNSUPPORTED, "%s: head dim %d (64, 128, 256)", what, d);
  if (!cache_dtype(c->dtype)) return report_error(MATTN_ERR_UNSUPPORTED, "%s: a cache is bf16 or e4m3", what);
  const bool e8 = c->dtype == MATTN_E4M3;
  if (!c->k || !c->v || !c->page_table)
    return report_error(MATTN_ERR_INVALID_ARG, "%s: the pages and the page table must be non-NULL", what);
  if (e8 ? !c->k_exponents || !c->v_exponents : c->k_exponents || c->v_exponents)
    return report_error(MATTN_ERR_INVALID_ARG, "%s: exponents come with e4m3 pages, and only with them", what);
  if (c->page < 16 || c->page % 16)
    return report_error(MATTN_ERR_UNSUPPORTED, "%s: page size %d is not a multiple of 16", what, c->page);
  if (c->table_pages < 1 || c->n_pages < 1)
    return report_error(MATTN_ERR_INVALID_ARG, "%s: table_pages and n_pages must be >= 1", what);
  if ((int64_t)c->table_pages * c->page > kMaxRows)
    return report_error(MATTN_ERR_UNSUPPORTED, "%s: table_pages * page exceeds 2^30", what);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4))
    return report_error(MATTN_ERR_UNSUPPORTED, "%s: pages must be 16-byte and the page table 4-byte aligned", what);
  const int es = e8 ? 1 : 2;
  const int64_t size[3] = {c->n_pages, H_kv, c->page};
  for (int i = 0; i < 2; ++i) {
    const int64_t s[3] = {c->page_stride[i], c->head_stride[i], c->row_stride[i]};
    const int64_t e[3] = {c->exp_page_stride[i], c->exp_head_stride[i], c->exp_row_stride[i]};
    for (int j = 0; j < 3; ++j) {
      if (s[j] <= 0 || (s[j] * es) % 16)
        return report_error(MATTN_ERR_UNSUPPORTED, "%s: strides of the pages must be positive multiples of 16 bytes", what);
      if (s[j] >= (int64_t(1) << 40) / es)
        return report_error(MATTN_ERR_UNSUPPORTED, "%s: a stride of the pages exceeds 2^40 bytes", what);
      if (e8 && e[j] <= 0) return report_error(MATTN_ERR_UNSUPPORTED, "%s: strides of the exponents must be positive", what);
    }
    if (!rows_apart(s, size, d) || (e8 && !rows_apart(e, size, 1)))
      return report_error(MATTN_ERR_INVALID_ARG, "%s: rows of the cache overlap", what);
  }
  return MATTN_OK;
}

// The rows of k's (0) and v's (1) pages, and of their exponents (2, 3; none in bf16).
RowSet cache_rows(const mattn_paged_cache* c, int i, int H_kv, int d) {
  const int64_t es = i > 1 || c->dtype == MATTN_E4M3 ? 1 : 2;
  const int t = i & 1;
  if (i > 1 && c->dtype != MATTN_E4M3) return {nullptr, {0, 0, 0}, {0, 0, 0}, 0};
  if (i > 1)
    return {t ? c->v_exponents : c->k_exponents, {c->exp_page_stride[t], c->exp_head_stride[t], c->exp_row_stride[t]},
            {c->n_pages, H_kv, c->page}, 1};
  return {t ? c->v : c->k, {c->page_stride[t] * es, c->head_stride[t] * es, c->row_stride[t] * es}, {c->n_pages, H_kv, c->page},
          d * es};
}

int fill_rows(const char* what, const void* k, const void* v, const int64_t* token_stride, const int64_t* head_stride,
              const mattn_paged_cache* c, const int32_t* cu, const int32_t* starts, int B, int T, int H_kv, int d,
              int dtype, bool reads, CacheRowsParams* p) {
  int rc = check_cache(what, c, B, H_kv, d);
  if (rc) return rc;
  if (dtype != MATTN_BF16) return report_error(MATTN_ERR_UNSUPPORTED, "%s takes bf16 rows", what);
  if ((T != 0 && (!k || !v)) || !token_stride || !head_stride)
    return report_error(MATTN_ERR_INVALID_ARG, "%s: k, v and their strides must be non-NULL", what);
  if (T < 0) return report_error(MATTN_ERR_INVALID_ARG, "%s: T must be >= 0", what);
  if (!cu && T != B) return report_error(MATTN_ERR_INVALID_ARG, "%s: without cu_seqlens there is one token for each sequence", what);
  if ((int64_t)T * H_kv > INT32_MAX) return report_error(MATTN_ERR_UNSUPPORTED, "%s: T * H_kv exceeds 2^31 - 1", what);
  if (!aligned(k, 16) || !aligned(v, 16)) return report_error(MATTN_ERR_UNSUPPORTED, "%s: k and v must be 16-byte aligned", what);
  if (!aligned(cu, 4) || !aligned(starts, 4))
    return report_error(MATTN_ERR_INVALID_ARG, "%s: cu_seqlens and starts must be 4-byte aligned", what);
  memset(p, 0, sizeof(*p));
  const void* rows[2] = {k, v};
  void* pages[2] = {c->k, c->v};
  void* exps[2] = {c->k_exponents, c->v_exponents};
  Extent at[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t ts = token_stride[i], hs = head_stride[i];
    if (ts % 8 || hs % 8) return report_error(MATTN_ERR_UNSUPPORTED, "%s: rows must start on 16-byte boundaries", what);
    if (ts < 0 || hs < 0) return report_error(MATTN_ERR_INVALID_ARG, "%s: strides must be >= 0", what);
    const int64_t s[3] = {ts, hs, 0}, size[3] = {T, H_kv, 1};
    if (reads && T > 0 && !rows_apart(s, size, d))
      return report_error(MATTN_ERR_INVALID_ARG, "%s: rows of an output overlap", what);
    at[i].lo = reinterpret_cast<uintptr_t>(rows[i]);
    at[i].hi = at[i].lo + (T > 0 ? ((uint64_t)(T - 1) * ts + (uint64_t)(H_kv - 1) * hs + d) * 2 : 0);
    p->rows[i] = const_cast<void*>(rows[i]);
    p->row_token[i] = ts;
    p->row_head[i] = hs;
    p->pages[i] = pages[i];
    p->page_stride[i] = c->page_stride[i];
    p->head_stride[i] = c->head_stride[i];
    p->row_stride[i] = c->row_stride[i];
    p->exps[i] = static_cast<uint8_t*>(exps[i]);
    p->exp_page[i] = c->exp_page_stride[i];
    p->exp_head[i] = c->exp_head_stride[i];
    p->exp_row[i] = c->exp_row_stride[i];
  }
  // rows are read and written in no order.  (Interleaved views, as k and v of one
  // projection or of one pool, share an extent without sharing a byte: the
  // tensors of a side may; whole sides may not.)
  const Extent small[3] = {extent_of(c->page_table, (uint64_t)B * c->table_pages * 4), extent_of(cu, ((uint64_t)B + 1) * 4),
                           extent_of(starts, (uint64_t)B * 4)};
  RowSet of[4], to[2];
  for (int j = 0; j < 4; ++j) of[j] = cache_rows(c, j, H_kv, d);
  for (int i = 0; i < 2; ++i) to[i] = {rows[i], {token_stride[i] * 2, head_stride[i] * 2, 0}, {T, H_kv, 1}, d * 2};
  for (int i = 0; i < 2 && T > 0; ++i)
    for (int j = 0; j < 4; ++j)
      if (at[i].meets(of[j].extent())) return report_error(MATTN_ERR_INVALID_ARG, "%s: the rows overlap the cache", what);
  for (const Extent& x : small) {
    for (int i = 0; i < 4 && T > 0; ++i)
      if (reads ? i < 2 && at[i].meets(x) : of[i].extent().meets(x))
        return report_error(MATTN_ERR_INVALID_ARG, "%s: an output overlaps the page table, cu_seqlens or starts", what);
  }
  if (reads && T > 0 && !apart(to[0], to[1]))
    return report_error(MATTN_ERR_INVALID_ARG, "%s: k and v overlap", what);
  for (int i = 0; i < (c->dtype == MATTN_E4M3 ? 4 : 2) && !reads && T > 0; ++i)
    for (int j = 0; j < i; ++j)
      if (i - j == 1 && i % 2 ? !pages_apart(of[j], of[i]) : !apart(of[j], of[i]))
        return report_error(MATTN_ERR_INVALID_ARG, "%s: two of the cache's tensors overlap", what);
  p->table = c->page_table;
  p->cu = cu;
  p->starts = starts;
  p->B = B; p->T = T; p->H_kv = H_kv; p->d = d;
  p->page = c->page;
  p->table_pages = c->table_pages;
  p->n_pages = c->n_pages;
  return check_device();
}

// CTAs of a group's cluster for lists of `tiles` tiles at most, or 0: equal shares of all
// lists.  A cluster saves the states, their merge and a launch (about 3 us), and costs the
// rounds of a tile for every warp by which its CTAs take longer than all SMs would: up to
// two and a half, or five of bf16's half as many keys, it is the faster (32 / 8 heads of 128, lengths
// between L / 2 and L, clusters and shares, us: in e4m3 16 sequences of L = 1,024 10.5 and 16.3, of
// 4,096 28.3 and 33.9, of 16,384 89.6 and 73.9, one of 8,192 11.0 and 14.2, of 32,768 28.0 and 25.0;
// in bf16 16 of 1,024 14.3 and 17.0, of 4,096 38.2 and 42.5, one of 32,768 33.2 and 31.0).  Eight
// CTAs only where eight clusters of them do: sixteen do not find their places at once
// (two sequences of 8,192: 16.6 and 13.7).
int paged_cluster(int64_t groups, int64_t tiles, int d, bool e4m3) {
  if (groups > kPlanSms) return 0;
  const int warps = decode_rows_warps(d);
  int64_t cluster = 1;
  while (cluster < (groups <= 8 ? 8 : 4) && groups * cluster * 2 <= kPlanSms && cluster * warps < tiles) cluster *= 2;
  const int64_t rounds = (tiles + cluster * warps - 1) / (cluster * warps);
  // (in 152 * warps-ths of a round)
  const int64_t over = rounds * kPlanSms * warps - groups * tiles;
  return over * 2 <= (e4m3 ? 5 : 10) * kPlanSms * warps ? (int)cluster : 0;
}

// Tiles of a list at most: the window's (which may begin and end inside one) and the
// first tokens', or all.
int64_t list_tiles_at_most(int64_t L, int window, int first, int d, bool e4m3, int group) {
  const int tk = paged_tile(d, e4m3, group);
  const int64_t all = (L + tk - 1) / tk;
  if (!window) return all;
  const int64_t seen = ((int64_t)window + tk - 1) / tk + 1 + (first + tk - 1) / tk;
  return all < seen ? all : seen;
}

// The tiles of all lists at most, and the warps of a CTA that share them.
int check_paged(int B, int H, int H_kv, int table_pages, int page, int d, int dtype, int64_t* tiles) {
  const int rc = check_heads("decode_paged", B, H, H_kv, d, MATTN_BF16);
  if (rc) return rc;
  if (!cache_dtype(dtype)) return report_error(MATTN_ERR_UNSUPPORTED, "decode_paged: a cache is bf16 or e4m3");
  if (table_pages < 1 || page < 1)
    return report_error(MATTN_ERR_INVALID_ARG, "decode_paged: table_pages and page must be >= 1");
  const int64_t L = (int64_t)table_pages * page;
  if (L > kMaxRows) return report_error(MATTN_ERR_UNSUPPORTED, "decode_paged: table_pages * page exceeds 2^30");
  const int tk = paged_tile(d, dtype == MATTN_E4M3, H / H_kv);
  *tiles = (int64_t)B * H_kv * ((L + tk - 1) / tk + 1);  // (a window's first tile and the first tokens' last one are parts)
  if (*tiles > INT32_MAX) return report_error(MATTN_ERR_UNSUPPORTED, "decode_paged: more than 2^31 - 1 tiles of keys");
  return MATTN_OK;
}

// The plan, then the links of marked items.
size_t packed_plan_bytes(int64_t T, int64_t B) {
  return round256(sizeof(PackedPlan) + (size_t)packed_pairs(T, B) * sizeof(PackedPair));
}
// (heads of 256: two items a pair and head)
size_t packed_bytes(int64_t T, int64_t B, int64_t H) { return packed_plan_bytes(T, B) + (size_t)(packed_pairs(T, B) * H) * 8; }

// Whether each CTA finds its items itself, without the plan kernel: where it has few, in up to
// kDirectSequences sequences, which it then looks through, 32 at a time, before its first one (64
// rows of four sequences, with empty ones behind them, us so and with the plan: 4 in all 8.2 and 11.5,
// 128 8.9 and 11.5, 384 11.3 and 11.5, 512 12.6 and 11.5, 4,096 47.5 and 15.6).
constexpr int kDirectSequences = 384;
bool packed_direct(int64_t T, int64_t B, int64_t H, int d) {
  return d != 256 && B <= kDirectSequences && packed_pairs(T, B) * H <= kPackedDirect * kPlanSms;
}

int check_packed(int B, int T, int H) {
  if (B < 1 || H < 1 || T < 0) return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: B, H must be >= 1 and T >= 0");
  if (T > kMaxRows) return report_error(MATTN_ERR_UNSUPPORTED, "attention_packed: T exceeds 2^30");
  // the items are numbered in 32 bits
  if ((int64_t)H * (T / 256 + (int64_t)B) > INT32_MAX)
    return report_error(MATTN_ERR_UNSUPPORTED, "attention_packed: H * (T / 256 + B) exceeds 2^31 - 1");
  return MATTN_OK;
}

}  // namespace
}  // namespace mattn

using namespace mattn;

extern "C" {

int mattn_cache_write(const void* k, const void* v, const int64_t token_stride[2], const int64_t head_stride[2],
                      const mattn_paged_cache* cache, const int32_t* cu_seqlens, const int32_t* starts, int B, int T,
                      int H_kv, int d, int dtype, void* stream) {
  CacheRowsParams p;
  const int rc = fill_rows("cache_write", k, v, token_stride, head_stride, cache, cu_seqlens, starts, B, T, H_kv, d, dtype,
                           false, &p);
  if (rc || T == 0) return rc;
  return launched(launch_cache_write(p, cache->dtype == MATTN_E4M3, static_cast<cudaStream_t>(stream)), "cache_write launch");
}

int mattn_cache_read(void* k, void* v, const int64_t token_stride[2], const int64_t head_stride[2],
                     const mattn_paged_cache* cache, const int32_t* cu_seqlens, const int32_t* starts, int B, int T,
                     int H_kv, int d, int dtype, void* stream) {
  CacheRowsParams p;
  const int rc = fill_rows("cache_read", k, v, token_stride, head_stride, cache, cu_seqlens, starts, B, T, H_kv, d, dtype,
                           true, &p);
  if (rc || T == 0) return rc;
  return launched(launch_cache_read(p, cache->dtype == MATTN_E4M3, static_cast<cudaStream_t>(stream)), "cache_read launch");
}

int mattn_decode_paged_workspace(int B, int H, int H_kv, int table_pages, int page, int d, int cache_dtype,
                                 size_t* bytes_out) {
  if (!bytes_out) return report_error(MATTN_ERR_INVALID_ARG, "decode_paged: bytes_out is NULL");
  int64_t tiles = 0;
  const int rc = check_paged(B, H, H_kv, table_pages, page, d, cache_dtype, &tiles);
  if (rc) return rc;
  *bytes_out = rows_layout((int64_t)B * H_kv, H / H_kv, kPlanSms * decode_share_warps(tiles, d), d).all();
  return MATTN_OK;
}

int mattn_decode_paged(const void* q, const mattn_paged_cache* cache, void* o, float* lse, const int32_t* seq_lens,
                       int B, int H, int H_kv, int d, int dtype, int window, int sink_tokens, const float* sink,
                       float softmax_scale, void* workspace, size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int rc = check_heads("decode_paged", B, H, H_kv, d, dtype);
  if (rc) return rc;
  if ((rc = check_cache("decode_paged", cache, B, H_kv, d))) return rc;
  int64_t tiles = 0;
  if ((rc = check_paged(B, H, H_kv, cache->table_pages, cache->page, d, cache->dtype, &tiles))) return rc;
  if (!q || !o) return report_error(MATTN_ERR_INVALID_ARG, "decode_paged: q and o must be non-NULL");
  if (!aligned(q, 16) || !aligned(o, 16))
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_paged: q and o must be 16-byte aligned");
  if (window < 0 || sink_tokens < 0 || (!window && sink_tokens))
    return report_error(MATTN_ERR_INVALID_ARG, "decode_paged: window and sink_tokens must be >= 0, sink_tokens 0 without a window");
  if ((rc = check_small("decode_paged", lse, seq_lens, sink))) return rc;
  if ((rc = check_scale("decode_paged", softmax_scale))) return rc;
  const bool e8 = cache->dtype == MATTN_E4M3;
  const int warps = decode_share_warps(tiles, d);
  const RowsLayout lay = rows_layout((int64_t)B * H_kv, H / H_kv, kPlanSms * warps, d);
  if ((rc = check_workspace("decode_paged", workspace, workspace_bytes, lay.all()))) return rc;
  const Extent ins[] = {extent_of(q, (uint64_t)B * H * d * 2), cache_rows(cache, 0, H_kv, d).extent(),
                        cache_rows(cache, 1, H_kv, d).extent(), cache_rows(cache, 2, H_kv, d).extent(),
                        cache_rows(cache, 3, H_kv, d).extent(), extent_of(cache->page_table, (uint64_t)B * cache->table_pages * 4),
                        extent_of(seq_lens, (uint64_t)B * 4), extent_of(sink, (uint64_t)H * 4)};
  const Extent outs[] = {extent_of(o, (uint64_t)B * H * d * 2), extent_of(lse, (uint64_t)B * H * 4),
                         extent_of(workspace, lay.all())};
  if (any_meet(ins, outs))
    return report_error(MATTN_ERR_INVALID_ARG, "decode_paged: an output or the workspace overlaps an input or another output");
  uint32_t* err = nullptr;
  if ((rc = device_error_word(stream, &err))) return rc;
  DecodePagedParams p;
  memset(&p, 0, sizeof(p));
  void* pages[2] = {cache->k, cache->v};
  void* exps[2] = {cache->k_exponents, cache->v_exponents};
  for (int i = 0; i < 2; ++i) {
    if ((rc = make_pages_map(i ? &p.tv : &p.tk, pages[i], e8, d, cache->page, H_kv, cache->n_pages, cache->row_stride[i],
                             cache->head_stride[i], cache->page_stride[i])))
      return rc;
    p.exps[i] = static_cast<const uint8_t*>(exps[i]);
    p.exp_page[i] = cache->exp_page_stride[i];
    p.exp_head[i] = cache->exp_head_stride[i];
    p.exp_row[i] = cache->exp_row_stride[i];
  }
  p.q = q;
  p.table = cache->page_table;
  p.seq_lens = seq_lens;
  DecodeRowsParams at;
  place_rows(&at, lay, static_cast<char*>(workspace));
  p.part_o = at.part_o;
  p.part_ml = at.part_ml;
  p.group_start = at.group_start;
  p.err = err;
  p.timeout_ns = device_wait_timeout_ns();
  p.B = B; p.H = H; p.H_kv = H_kv;
  p.page = cache->page;
  p.table_pages = cache->table_pages;
  p.n_pages = cache->n_pages;
  p.L = cache->table_pages * cache->page;
  p.window = window;
  p.first = sink_tokens < p.L ? sink_tokens : p.L;
  p.ctas = kPlanSms;
  p.warps = warps;
  p.selftest = g_wait_selftest.load();
  p.scale_log2 = scale_log2(softmax_scale, d);
  p.sink = sink;
  p.o = o;
  p.lse = lse;
  p.cluster = paged_cluster((int64_t)B * H_kv, list_tiles_at_most(p.L, window, p.first, d, e8, H / H_kv), d, e8);
  if ((rc = launched(launch_decode_paged(p, d, e8, stream), "paged launch")) || p.cluster) return rc;
  MergeParams m;
  memset(&m, 0, sizeof(m));
  m.b_o = p.part_o;
  m.b_ml = p.part_ml;
  m.group_start = p.group_start;
  m.warps = lay.warps;
  m.seq_lens = seq_lens;
  m.L = p.L;
  m.tile_shift = paged_shift(d, e8, H / H_kv);
  m.window = p.window;
  m.first = p.first;
  m.sink = sink;
  m.o = o;
  m.lse = lse;
  m.B = B; m.H = H; m.H_kv = H_kv;
  m.states = 1 + (int)(lay.warps / ((int64_t)B * H_kv));
  // (us with four in flight and with sixteen, e4m3, warm: 229 states a row, 131,071 keys of 256 57.6 and
  // 54.5, of 128 54.9 and 51.3; 115, two sequences of 65,536 of 128 53.6 and 51.8; 58, four 91.1 and 90.5,
  // eight of 32,768 52.1 and 51.2; 29, 51.4 and 51.2; 13, the same; 7, 103.9 and 105.2)
  m.many = m.states >= 32 ? 1 : 0;
  return launched(launch_decode_merge(m, d, stream), "merge launch");
}

int mattn_attention_packed_workspace(int B, int T, int H, size_t* bytes_out) {
  if (!bytes_out) return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: bytes_out is NULL");
  const int rc = check_packed(B, T, H);
  if (rc) return rc;
  *bytes_out = packed_bytes(T, B, H);
  return MATTN_OK;
}

int mattn_attention_packed(const void* q, const void* k, const void* v, const int64_t token_stride[3],
                           const int64_t head_stride[3], void* o, float* lse, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, int B, int T, int T_k, int H, int H_kv, int d, int dtype,
                           int causal, int window, const float* sink, float softmax_scale, void* workspace,
                           size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int rc = check_packed(B, T, H);
  if (rc) return rc;
  if (H_kv < 1 || H % H_kv)
    return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: H = %d is not a multiple of H_kv = %d", H, H_kv);
  if (d != 64 && d != 80 && d != 96 && d != 128 && d != 256)
    return report_error(MATTN_ERR_UNSUPPORTED, "attention_packed: head dim %d (64, 80, 96, 128, 256)", d);
  if (d == 256 && 2 * (int64_t)H * (T / 256 + (int64_t)B) > INT32_MAX)  // (an item is a query tile there, not a pair)
    return report_error(MATTN_ERR_UNSUPPORTED, "attention_packed: H * (T / 256 + B) exceeds 2^30 - 1 at d = 256");
  if (dtype != MATTN_BF16) return report_error(MATTN_ERR_UNSUPPORTED, "attention_packed takes bf16");
  if (T_k < 0) return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: T_k must be >= 0");
  if (T_k > kMaxRows) return report_error(MATTN_ERR_UNSUPPORTED, "attention_packed: T_k exceeds 2^30");
  if (!cu_seqlens_q || (T > 0 && (!q || !o)) || (T_k > 0 && (!k || !v)) || !token_stride || !head_stride)
    return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: q, k, v, o, their strides and cu_seqlens_q must be non-NULL");
  if (!cu_seqlens_k && T_k != T)
    return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: other keys than queries need cu_seqlens_k");
  if (window < 0 || (window && !causal))
    return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: window must be >= 0, and 0 without causal");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return report_error(MATTN_ERR_UNSUPPORTED, "attention_packed: q, k, v and o must be 16-byte aligned");
  if (!aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
    return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: cu_seqlens must be 4-byte aligned");
  if ((rc = check_small("attention_packed", lse, nullptr, sink))) return rc;
  if ((rc = check_scale("attention_packed", softmax_scale))) return rc;
  int64_t ts[3], hs[3];
  for (int i = 0; i < 3; ++i) {
    // (the stride of a dimension of one entry says nothing)
    ts[i] = (i ? T_k : T) > 1 ? token_stride[i] : d;
    hs[i] = (i ? H_kv : H) > 1 ? head_stride[i] : d;
    if (ts[i] <= 0 || hs[i] <= 0 || ts[i] % 8 || hs[i] % 8 || ts[i] >= int64_t(1) << 39 || hs[i] >= int64_t(1) << 39)
      return report_error(MATTN_ERR_UNSUPPORTED,
                          "attention_packed: strides must be positive multiples of 16 bytes below 2^40");
  }
  // (items are read and written in no order, some twice)
  if ((rc = check_workspace("attention_packed", workspace, workspace_bytes, packed_bytes(T, B, H)))) return rc;
  auto rows_of = [&](const void* x, int64_t rows, int heads, int i) {
    return extent_of(x, rows > 0 ? ((uint64_t)(rows - 1) * ts[i] + (uint64_t)(heads - 1) * hs[i] + d) * 2 : 0);
  };
  const Extent ins[] = {rows_of(q, T, H, 0), rows_of(k, T_k, H_kv, 1), rows_of(v, T_k, H_kv, 2),
                        extent_of(cu_seqlens_q, ((uint64_t)B + 1) * 4), extent_of(cu_seqlens_k, ((uint64_t)B + 1) * 4),
                        extent_of(sink, (uint64_t)H * 4)};
  const Extent outs[] = {extent_of(o, (uint64_t)T * H * d * 2), extent_of(lse, (uint64_t)T * H * 4),
                         extent_of(workspace, packed_bytes(T, B, H))};
  if (any_meet(ins, outs))
    return report_error(MATTN_ERR_INVALID_ARG, "attention_packed: an output or the workspace overlaps an input or another output");
  uint32_t* err = nullptr;
  if ((rc = device_error_word(stream, &err))) return rc;
  if (T == 0) return MATTN_OK;
  PackedParams p;
  memset(&p, 0, sizeof(p));
  const int rem = d % 64, vw = d % 64 == 0 ? 64 : (d % 32 == 0 ? 32 : 16);
  auto maps = [&](CUtensorMap* m, const void* x, int64_t rows, int heads, int i) {  // 64-column chunks and the rest
    const int e = make_packed_map(&m[0], x, d, 64, kTile, rows, heads, ts[i], hs[i]);
    if (e || !rem) return e;
    return make_packed_map(&m[1], static_cast<const char*>(x) + (d - rem) * 2, rem, rem, kTile, rows, heads, ts[i], hs[i]);
  };
  if ((rc = maps(p.tq, q, T, H, 0))) return rc;
  if (T_k > 0) {  // (else no tile is loaded)
    if ((rc = maps(p.tk, k, T_k, H_kv, 1))) return rc;
    if ((rc = make_packed_map(&p.tv, v, d, vw, d == 256 ? kPackedValues256 : kTile, T_k, H_kv, ts[2], hs[2]))) return rc;
  }
  p.o = o;
  p.lse = lse;
  p.sink = sink;
  p.v = v;
  p.v_token = ts[2];
  p.v_head = hs[2];
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k ? cu_seqlens_k : cu_seqlens_q;
  p.plan = static_cast<PackedPlan*>(workspace);
  p.marked = reinterpret_cast<int*>(static_cast<char*>(workspace) + packed_plan_bytes(T, B));
  p.err = err;
  p.timeout_ns = device_wait_timeout_ns();
  p.B = B; p.T = T; p.T_k = T_k; p.H = H; p.H_kv = H_kv;
  p.group = H / H_kv;
  p.causal = causal ? 1 : 0;
  p.wide = aligned(o, 32) ? 1 : 0;
  p.window = window < kMaxRows ? window : (int)kMaxRows;
  p.max_pairs = (int)packed_pairs(T, B);
  while (((2 * ((int64_t)T_k / 128 + 1)) >> p.work_shift) >= 1024) ++p.work_shift;
  p.direct = packed_direct(T, B, H, d) ? 1 : 0;
  p.scale_log2 = scale_log2(softmax_scale, d);
  p.selftest = g_wait_selftest.load();
  return launched(launch_attention_packed(p, d, stream), "attention_packed launch");
}

// Test hook (not in the public header), host only: how decode_paged reads its lists:
// {CTAs of a group's cluster or 0 for equal shares, warps of a CTA then, keys of a tile}.
int mattn_internal_paged_plan(int B, int H, int H_kv, int table_pages, int page, int d, int dtype, int window,
                              int sink_tokens, int* out) {
  int64_t tiles = 0;
  const int rc = check_paged(B, H, H_kv, table_pages, page, d, dtype, &tiles);
  if (rc) return rc;
  const bool e8 = dtype == MATTN_E4M3;
  out[0] = paged_cluster((int64_t)B * H_kv, list_tiles_at_most((int64_t)table_pages * page, window, sink_tokens, d, e8, H / H_kv),
                         d, e8);
  out[1] = decode_share_warps(tiles, d);
  out[2] = paged_tile(d, e8, H / H_kv);
  return MATTN_OK;
}

// Test hook (not in the public header), host only: whether attention_packed goes without its plan.
int mattn_internal_packed_direct(int B, int T, int H, int d) { return packed_direct(T, B, H, d) ? 1 : 0; }

// Test hook (not in the public header): the launches of decode_paged and
// attention_packed until the next call leave out the first keys' copies (1), so that the
// bounded waits and the error word can be exercised without a hang; 0: nothing.
int mattn_internal_paged_wait_selftest(int what) {
  if (what < 0 || what > 1) return report_error(MATTN_ERR_INVALID_ARG, "what must be 0 or 1");
  g_wait_selftest.store(what);
  return MATTN_OK;
}

}  // extern "C"
