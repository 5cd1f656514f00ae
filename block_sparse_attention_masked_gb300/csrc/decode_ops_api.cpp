// C entry points of the decode step's operators (include/mattn.h): argument
// checks, TMA views, workspace layout and launches.  Nothing here allocates
// device memory but the device's error word on its first use: the caller
// passes the workspace, so that calls on different streams and captured
// graphs never share one unless the caller makes them.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "decode_ops.h"
#include "kernel_params.h"
#include "launch_prep.h"
#include "mattn.h"

namespace mattn {
namespace {

// Test hook: the copies that the next launches leave out (DecodeRowsParams, SharedParams).
std::atomic<int> g_wait_selftest{0};

constexpr int64_t kMaxRows = 1 << 30;
constexpr int kMaxGroup = 16;  // query heads per key/value head

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

int check_heads(const char* what, int B, int H, int H_kv, int d, int dtype) {
  if (B < 1 || H < 1 || H_kv < 1) return report_error(MATTN_ERR_INVALID_ARG, "%s: B, H, H_kv must be >= 1", what);
  if (H % H_kv) return report_error(MATTN_ERR_INVALID_ARG, "%s: H = %d is not a multiple of H_kv = %d", what, H, H_kv);
  if (H / H_kv > kMaxGroup)
    return report_error(MATTN_ERR_UNSUPPORTED, "%s: up to %d query heads per key/value head", what, kMaxGroup);
  if (d != 64 && d != 128 && d != 256)
    return report_error(MATTN_ERR_UNSUPPORTED, "%s: head dim %d (64, 128, 256)", what, d);
  if (dtype != MATTN_BF16) return report_error(MATTN_ERR_UNSUPPORTED, "%s takes bf16", what);
  if ((int64_t)B * H > kMaxRows) return report_error(MATTN_ERR_UNSUPPORTED, "%s: B * H too large", what);
  // the (sequence, key/value head) pairs are the second grid dimension
  if ((int64_t)B * H_kv > 65535)
    return report_error(MATTN_ERR_UNSUPPORTED, "%s: B * H_kv = %lld exceeds 65535", what, (long long)B * H_kv);
  return MATTN_OK;
}

int check_scale(const char* what, float scale) {
  if (!(scale >= 0.f) || std::isinf(scale))
    return report_error(MATTN_ERR_INVALID_ARG, "%s: softmax_scale must be finite and >= 0", what);
  return MATTN_OK;
}

int check_small(const char* what, const void* lse, const void* lens, const void* sink) {
  if (!aligned(lse, 4) || !aligned(lens, 4) || !aligned(sink, 4))
    return report_error(MATTN_ERR_INVALID_ARG, "%s: lse, seq_lens and sink must be 4-byte aligned", what);
  return MATTN_OK;
}

int check_workspace(const char* what, const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return report_error(MATTN_ERR_CAPACITY, "%s: the workspace holds %zu bytes, %zu are needed", what, ws ? have : 0,
                        need);
  if (!aligned(ws, 256)) return report_error(MATTN_ERR_INVALID_ARG, "%s: the workspace must be 256-byte aligned", what);
  return MATTN_OK;
}

int launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return report_error(MATTN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return MATTN_OK;
}

float scale_log2(float scale, int d) {
  return (scale > 0.f ? scale : 1.0f / std::sqrt((float)d)) * 1.4426950408889634f;
}

// States of `rows` query rows in n splits: O, then (reference, sum).
size_t state_bytes(int64_t rows, int n, int d) {
  return round256((size_t)rows * n * d * 4) + round256((size_t)rows * n * 8);
}

// States of the own lists: a slot for each (warp, group) piece, then the
// lists' starts (DecodeRowsParams).
struct RowsLayout {
  int warps;
  size_t o_bytes, ml_bytes, start_bytes;
  size_t all() const { return o_bytes + ml_bytes + start_bytes; }
};

RowsLayout rows_layout(int64_t groups, int G, int warps, int d) {
  RowsLayout r;
  r.warps = warps;
  r.o_bytes = round256((size_t)(warps + groups) * G * d * 4);
  r.ml_bytes = round256((size_t)(warps + groups) * G * 8);
  r.start_bytes = round256((size_t)(groups + 1) * 4);
  return r;
}

void place_rows(DecodeRowsParams* p, const RowsLayout& r, char* ws) {
  p->part_o = reinterpret_cast<float*>(ws);
  p->part_ml = reinterpret_cast<float*>(ws + r.o_bytes);
  p->group_start = reinterpret_cast<int*>(ws + r.o_bytes + r.ml_bytes);
}

int list_tiles(int top_k, int block, int d) {
  const int tk = decode_rows_tile(d);
  return (int)(((int64_t)top_k * block + tk - 1) / tk);
}

struct SharedLayout {
  SharedPlan prefix;
  int own_warps;  // of a CTA of the own keys
  RowsLayout own;
  size_t prefix_bytes, own_bytes;
};

SharedLayout shared_layout(int B, int H, int H_kv, int P, int L, int d) {
  SharedLayout s;
  s.prefix = shared_plan(B, H, H_kv, P, L, d);
  s.prefix_bytes = P > 0 ? state_bytes((int64_t)B * H, s.prefix.n_split, d) : 0;
  const int64_t groups = (int64_t)B * H_kv;
  s.own_warps = P > 0 ? shared_row_warps(d, s.prefix.sub) : decode_share_warps(groups * list_tiles(L, 1, d), d);
  s.own = rows_layout(groups, H / H_kv, s.prefix.own_ctas * s.own_warps, d);
  s.own_bytes = L > 0 ? s.own.all() : 0;
  return s;
}

int check_shared(int B, int H, int H_kv, int P, int L, int d, int dtype) {
  int rc = check_heads("decode_shared", B, H, H_kv, d, dtype);
  if (rc) return rc;
  if (P < 0 || L < 0) return report_error(MATTN_ERR_INVALID_ARG, "decode_shared: P and L must be >= 0");
  if (P > kMaxRows || L > kMaxRows) return report_error(MATTN_ERR_UNSUPPORTED, "decode_shared: P or L exceeds 2^30");
  // (numbered in 32 bits)
  if ((int64_t)B * H_kv * list_tiles(L, 1, d) > INT32_MAX)
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_shared: more than 2^31 - 1 tiles of own keys");
  return MATTN_OK;
}

int check_blocks(int B, int H, int H_kv, int top_k, int block, int d, int dtype) {
  int rc = check_heads("decode_blocks", B, H, H_kv, d, dtype);
  if (rc) return rc;
  if (block < 16 || block % 16)
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_blocks: block size %d is not a multiple of 16", block);
  if (block > (1 << 20)) return report_error(MATTN_ERR_UNSUPPORTED, "decode_blocks: block size %d exceeds 2^20", block);
  if (top_k < 1) return report_error(MATTN_ERR_INVALID_ARG, "decode_blocks: top_k must be >= 1");
  if ((int64_t)top_k * block > kMaxRows)
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_blocks: top_k * block exceeds 2^30");
  // the tiles of all lists are numbered in 32 bits
  if ((int64_t)B * H_kv * list_tiles(top_k, block, d) > INT32_MAX)
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_blocks: more than 2^31 - 1 key tiles in all lists");
  return MATTN_OK;
}

int check_select(int B, int H, int H_kv, int n_blocks, int d, int dtype) {
  int rc = check_heads("decode_select", B, H, H_kv, d, dtype);
  if (rc) return rc;
  if (n_blocks < 1) return report_error(MATTN_ERR_INVALID_ARG, "decode_select: n_blocks must be >= 1");
  if (n_blocks > kSelectMaxBlocks)
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_select: n_blocks = %d exceeds %d", n_blocks, kSelectMaxBlocks);
  return MATTN_OK;
}

// A buffer's bytes [lo, hi); hi wraps for no buffer that can exist.
struct Extent {
  uintptr_t lo, hi;
  bool meets(const Extent& x) const { return lo < x.hi && x.lo < hi; }
};

size_t select_bytes(int B, int H_kv, int n_blocks) { return 2 * round256((size_t)B * H_kv * n_blocks * 8); }

}  // namespace
}  // namespace mattn

using namespace mattn;

extern "C" {

int mattn_qk_rope(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* v_out,
                  const int32_t* positions, const int32_t* starts, const int32_t* lens, int B, int H, int H_kv, int N,
                  int L, int d, int dtype, const mattn_rope_desc* desc, void* stream) {
  if (!desc) return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: the descriptor is NULL");
  if (!q || !k || !q_out || !k_out)
    return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: q, k and their outputs must be non-NULL");
  if (!v != !v_out) return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: v and v_out come together");
  if (B < 1 || H < 1 || H_kv < 1 || N < 1 || L < 1)
    return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: B, H, H_kv, N, L must be >= 1");
  if (d != 32 && d != 64 && d != 80 && d != 96 && d != 128 && d != 256)
    return report_error(MATTN_ERR_UNSUPPORTED, "qk_rope: head dim %d (32, 64, 80, 96, 128, 256)", d);
  if (dtype != MATTN_BF16 && dtype != MATTN_F32)
    return report_error(MATTN_ERR_UNSUPPORTED, "qk_rope: dtype %d not supported", dtype);
  if ((int64_t)B * N > kMaxRows || H > 65536 || H_kv > 65536)
    return report_error(MATTN_ERR_UNSUPPORTED, "qk_rope: more than 2^30 tokens or 65536 heads");
  if (desc->n_axes < 1 || desc->n_axes > 3)
    return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: 1 to 3 position axes (got %d)", desc->n_axes);
  RopeParams p;
  memset(&p, 0, sizeof(p));
  int64_t rot = 0;
  for (int a = 0; a < 3; ++a) {
    if (a < desc->n_axes) {
      if (desc->sections[a] < 0) return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: sections must be >= 0");
      rot += desc->sections[a];
    }
    if (rot > d / 2)
      return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: the sections hold more than d / 2 = %d pairs", d / 2);
    p.axis_end[a] = (int)rot;
  }
  if (rot % 8) return report_error(MATTN_ERR_UNSUPPORTED, "qk_rope: %d rotated pairs (a multiple of 8)", (int)rot);
  if (rot && !desc->inv_freq) return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: inv_freq is NULL");
  if (!aligned(desc->inv_freq, 4) || !aligned(desc->q_weight, 4) || !aligned(desc->k_weight, 4) ||
      !aligned(positions, 4) || !aligned(starts, 4) || !aligned(lens, 4))
    return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: 32-bit arrays must be 4-byte aligned");
  if (!(desc->eps >= 0.f) || std::isinf(desc->eps))
    return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: eps must be finite and >= 0");
  const void* in[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  const int es = dtype == MATTN_F32 ? 4 : 2, n_tensors = v ? 3 : 2;
  Extent read[3], written[3];
  p.wide = true;
  for (int t = 0; t < n_tensors; ++t) {
    const int64_t ts = desc->token_stride[t], bs = desc->batch_stride[t];
    if (!aligned(in[t], 16) || !aligned(out[t], 16) || (ts * es) % 16 || (bs * es) % 16)
      return report_error(MATTN_ERR_UNSUPPORTED, "qk_rope: rows must start on 16-byte boundaries");
    if (ts < 0 || bs < 0) return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: strides must be >= 0");
    p.wide = p.wide && aligned(in[t], 32) && aligned(out[t], 32) && (ts * es) % 32 == 0 && (bs * es) % 32 == 0;
    const int64_t heads = t ? H_kv : H, rows = t ? L : N;
    read[t].lo = reinterpret_cast<uintptr_t>(in[t]);
    read[t].hi = read[t].lo + ((uint64_t)(B - 1) * bs + (uint64_t)(N - 1) * ts + heads * d) * es;
    written[t].lo = reinterpret_cast<uintptr_t>(out[t]);
    written[t].hi = written[t].lo + (uint64_t)B * heads * rows * d * es;
    p.src[t] = in[t];
    p.dst[t] = out[t];
    p.token_stride[t] = ts;
    p.batch_stride[t] = bs;
  }
  // warps read and write rows in no order
  for (int t = 0; t < n_tensors; ++t)
    for (int u = 0; u < n_tensors; ++u)
      if (written[t].meets(read[u]) || (t < u && written[t].meets(written[u])))
        return report_error(MATTN_ERR_INVALID_ARG, "qk_rope: an output overlaps an input or another output");
  const int rc = check_device();
  if (rc) return rc;
  p.positions = positions;
  p.starts = starts;
  p.lens = lens;
  p.inv_freq = desc->inv_freq;
  p.weight[0] = desc->q_weight;
  p.weight[1] = desc->k_weight;
  p.B = B; p.H = H; p.H_kv = H_kv; p.N = N; p.L = L; p.d = d;
  p.rot = (int)rot;
  p.interleaved = desc->interleaved ? 1 : 0;
  p.eps = desc->eps;
  // Few tokens: several warps share one token's rows, so that the machine
  // holds about sixteen warps per SM (64 tokens of 48 rows of 128).
  const int rpw = 32 / (d / 16);
  const int64_t its = (H + rpw - 1) / rpw + (int64_t)(v ? 2 : 1) * ((H_kv + rpw - 1) / rpw);
  int64_t segs = ((int64_t)kPlanSms * 16 + (int64_t)B * N - 1) / ((int64_t)B * N);
  p.segs = (int)(segs < 1 ? 1 : (segs > its ? its : segs));
  return launched(launch_qk_rope(p, dtype == MATTN_F32, static_cast<cudaStream_t>(stream)), "qk_rope launch");
}

int mattn_decode_shared_workspace(int B, int H, int H_kv, int P, int L, int d, size_t* bytes_out) {
  if (!bytes_out) return report_error(MATTN_ERR_INVALID_ARG, "decode_shared: bytes_out is NULL");
  const int rc = check_shared(B, H, H_kv, P, L, d, MATTN_BF16);
  if (rc) return rc;
  const SharedLayout s = shared_layout(B, H, H_kv, P, L, d);
  *bytes_out = s.prefix_bytes + s.own_bytes;
  return MATTN_OK;
}

int mattn_decode_shared(const void* q, const void* k_prefix, const void* v_prefix, const void* k, const void* v,
                        void* o, float* lse, const int32_t* seq_lens, int B, int H, int H_kv, int P, int P_cap, int L,
                        int d, int dtype, const float* sink, float softmax_scale, void* workspace,
                        size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int rc = check_shared(B, H, H_kv, P, L, d, dtype);
  if (rc) return rc;
  if (!q || !o) return report_error(MATTN_ERR_INVALID_ARG, "decode_shared: q and o must be non-NULL");
  if (P > P_cap) return report_error(MATTN_ERR_INVALID_ARG, "decode_shared: P = %d exceeds P_cap = %d", P, P_cap);
  if ((P > 0 && (!k_prefix || !v_prefix)) || (L > 0 && (!k || !v)))
    return report_error(MATTN_ERR_INVALID_ARG, "decode_shared: a key or value buffer is NULL");
  if (!aligned(q, 16) || !aligned(o, 16) || (P > 0 && (!aligned(k_prefix, 16) || !aligned(v_prefix, 16))) ||
      (L > 0 && (!aligned(k, 16) || !aligned(v, 16))))
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_shared: buffers must be 16-byte aligned");
  if ((rc = check_small("decode_shared", lse, seq_lens, sink))) return rc;
  if ((rc = check_scale("decode_shared", softmax_scale))) return rc;
  const SharedLayout s = shared_layout(B, H, H_kv, P, L, d);
  if ((rc = check_workspace("decode_shared", workspace, workspace_bytes, s.prefix_bytes + s.own_bytes))) return rc;
  uint32_t* err = nullptr;
  if ((rc = device_error_word(stream, &err))) return rc;
  const int64_t rows = (int64_t)B * H;
  char* ws = static_cast<char*>(workspace);
  MergeParams m;
  memset(&m, 0, sizeof(m));
  SharedParams sp;
  DecodeRowsParams rp;
  if (P > 0) {
    memset(&sp, 0, sizeof(sp));
    if ((rc = make_rows_map(&sp.tk, k_prefix, d, P, P_cap, H_kv, shared_key_tile(d)))) return rc;
    if ((rc = make_rows_map(&sp.tv, v_prefix, d, P, P_cap, H_kv, shared_key_tile(d)))) return rc;
    if ((rc = make_box_map(&sp.tq, q, d, H, H, B, H / H_kv, s.prefix.seqs))) return rc;
    sp.part_o = reinterpret_cast<float*>(ws);
    sp.part_ml = reinterpret_cast<float*>(ws + round256((size_t)rows * s.prefix.n_split * d * 4));
    if ((rc = make_state_map(&sp.to, sp.part_o, d, s.prefix.n_split, rows / H_kv, H_kv))) return rc;
    sp.err = err;
    sp.timeout_ns = device_wait_timeout_ns();
    sp.B = B; sp.H = H; sp.H_kv = H_kv; sp.P = P;
    sp.rows = (int)(rows / H_kv);
    sp.plan = s.prefix;
    sp.selftest = g_wait_selftest.load();
    sp.scale_log2 = scale_log2(softmax_scale, d);
    m.a_o = sp.part_o;
    m.a_ml = sp.part_ml;
    m.na = s.prefix.n_split;
  }
  if (L > 0) {
    memset(&rp, 0, sizeof(rp));
    if ((rc = make_rows_map(&rp.tk, k, d, L, L, (int64_t)B * H_kv, 16))) return rc;
    if ((rc = make_rows_map(&rp.tv, v, d, L, L, (int64_t)B * H_kv, 16))) return rc;
    rp.q = q;
    rp.seq_lens = seq_lens;
    place_rows(&rp, s.own, ws + s.prefix_bytes);
    rp.err = err;
    rp.timeout_ns = device_wait_timeout_ns();
    rp.B = B; rp.H = H; rp.H_kv = H_kv; rp.L = L;
    rp.block = 16;
    rp.box16 = 1;
    rp.ctas = s.prefix.own_ctas;
    rp.warps = s.own_warps;
    rp.selftest = g_wait_selftest.load();
    rp.scale_log2 = scale_log2(softmax_scale, d);
    m.b_o = rp.part_o;
    m.b_ml = rp.part_ml;
    m.group_start = rp.group_start;
    m.warps = s.own.warps;
    m.seq_lens = seq_lens;
    m.L = L;
  }
  m.sink = sink;
  m.o = o;
  m.lse = lse;
  m.B = B; m.H = H; m.H_kv = H_kv;
  m.states = m.na + (L > 0 ? 1 + (int)(s.own.warps / ((int64_t)B * H_kv)) : 0);
  if (P > 0) {
    if (L > 0) sp.own = rp;
    rc = launched(launch_decode_shared(sp, d, stream), "prefix launch");
  } else if (L > 0) {
    rc = launched(launch_decode_rows(rp, d, stream), "own-key launch");
  }
  if (rc) return rc;
  return launched(launch_decode_merge(m, d, stream), "merge launch");
}

int mattn_block_means(const void* k, void* means, const int32_t* seq_lens, const int32_t* first, int B, int H_kv,
                      int L, int d, int dtype, int block, int max_new, void* stream) {
  int rc = check_heads("block_means", B, H_kv, H_kv, d, dtype);
  if (rc) return rc;
  if (!k || !means) return report_error(MATTN_ERR_INVALID_ARG, "block_means: k and means must be non-NULL");
  if (L < 1 || L > kMaxRows) return report_error(MATTN_ERR_INVALID_ARG, "block_means: L must be in 1..2^30");
  if (block < 16 || block % 16)
    return report_error(MATTN_ERR_UNSUPPORTED, "block_means: block size %d is not a multiple of 16", block);
  if (max_new < 1) return report_error(MATTN_ERR_INVALID_ARG, "block_means: max_new must be >= 1");
  if (!aligned(k, 16) || !aligned(means, 16))
    return report_error(MATTN_ERR_UNSUPPORTED, "block_means: buffers must be 16-byte aligned");
  if ((rc = check_small("block_means", nullptr, seq_lens, first))) return rc;
  if ((rc = check_device())) return rc;
  BlockMeansParams p;
  p.k = k;
  p.means = means;
  p.seq_lens = seq_lens;
  p.first = first;
  p.B = B; p.H_kv = H_kv; p.L = L;
  p.block = block;
  p.n_blocks = (L - 1) / block + 1;
  p.max_new = max_new;
  // new keys that start anywhere in a block reach into one block more
  const int64_t span = ((int64_t)max_new - 1) / block + 2;
  p.span = (int)(span < p.n_blocks ? span : p.n_blocks);
  if ((int64_t)B * H_kv * p.span > (int64_t)1 << 31)
    return report_error(MATTN_ERR_UNSUPPORTED, "block_means: more than 2^31 blocks");
  return launched(launch_block_means(p, d, static_cast<cudaStream_t>(stream)), "block_means launch");
}

int mattn_decode_select_workspace(int B, int H, int H_kv, int n_blocks, int d, size_t* bytes_out) {
  if (!bytes_out) return report_error(MATTN_ERR_INVALID_ARG, "decode_select: bytes_out is NULL");
  const int rc = check_select(B, H, H_kv, n_blocks, d, MATTN_BF16);
  if (rc) return rc;
  *bytes_out = select_bytes(B, H_kv, n_blocks);
  return MATTN_OK;
}

int mattn_decode_select(const void* q, const void* means, const int32_t* seq_lens, int32_t* block_ids, int B, int H,
                        int H_kv, int n_blocks, int d, int dtype, int block, int top_k, int keep_first,
                        int keep_recent, void* workspace, size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int rc = check_select(B, H, H_kv, n_blocks, d, dtype);
  if (rc) return rc;
  if (!q || !means || !block_ids)
    return report_error(MATTN_ERR_INVALID_ARG, "decode_select: q, means and block_ids must be non-NULL");
  if (block < 1) return report_error(MATTN_ERR_INVALID_ARG, "decode_select: the block size must be >= 1");
  if (top_k < 1 || keep_first < 0 || keep_recent < 0 || (int64_t)keep_first + keep_recent > top_k)
    return report_error(MATTN_ERR_INVALID_ARG,
                        "decode_select: top_k >= 1 and keep_first + keep_recent <= top_k (got %d, %d, %d)", top_k,
                        keep_first, keep_recent);
  if ((int64_t)B * H_kv * top_k > kMaxRows) return report_error(MATTN_ERR_UNSUPPORTED, "decode_select: top_k too large");
  if (!aligned(q, 16) || !aligned(means, 32))
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_select: q must be 16-byte and means 32-byte aligned");
  if ((rc = check_small("decode_select", block_ids, seq_lens, nullptr))) return rc;
  const size_t need = select_bytes(B, H_kv, n_blocks);
  if ((rc = check_workspace("decode_select", workspace, workspace_bytes, need))) return rc;
  if ((rc = check_device())) return rc;
  DecodeSelectParams p;
  p.q = q;
  p.means = means;
  p.seq_lens = seq_lens;
  p.scores = static_cast<Score*>(workspace);
  p.again = reinterpret_cast<double*>(static_cast<char*>(workspace) + need / 2);
  p.ids = block_ids;
  p.B = B; p.H = H; p.H_kv = H_kv;
  p.n_blocks = n_blocks;
  p.block = block;
  p.top_k = top_k;
  p.keep_first = keep_first;
  p.keep_recent = keep_recent;
  return launched(launch_decode_select(p, d, stream), "decode_select launch");
}

int mattn_decode_blocks_workspace(int B, int H, int H_kv, int top_k, int block, int d, size_t* bytes_out) {
  if (!bytes_out) return report_error(MATTN_ERR_INVALID_ARG, "decode_blocks: bytes_out is NULL");
  const int rc = check_blocks(B, H, H_kv, top_k, block, d, MATTN_BF16);
  if (rc) return rc;
  const ListPlan plan = decode_list_plan((int64_t)B * H_kv, top_k, list_tiles(top_k, block, d), d);
  *bytes_out = plan.cluster ? 0 : rows_layout((int64_t)B * H_kv, H / H_kv, kPlanSms * plan.warps, d).all();
  return MATTN_OK;
}

int mattn_decode_blocks(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* seq_lens,
                        const int32_t* block_ids, int B, int H, int H_kv, int L, int d, int dtype, int block,
                        int top_k, const float* sink, float softmax_scale, void* workspace, size_t workspace_bytes,
                        void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int rc = check_blocks(B, H, H_kv, top_k, block, d, dtype);
  if (rc) return rc;
  if (!q || !k || !v || !o || !block_ids)
    return report_error(MATTN_ERR_INVALID_ARG, "decode_blocks: q, k, v, o and block_ids must be non-NULL");
  if (L < 1 || L > kMaxRows) return report_error(MATTN_ERR_INVALID_ARG, "decode_blocks: L must be in 1..2^30");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return report_error(MATTN_ERR_UNSUPPORTED, "decode_blocks: buffers must be 16-byte aligned");
  if ((rc = check_small("decode_blocks", lse, seq_lens, sink))) return rc;
  if (!aligned(block_ids, 4)) return report_error(MATTN_ERR_INVALID_ARG, "decode_blocks: block_ids must be 4-byte aligned");
  if ((rc = check_scale("decode_blocks", softmax_scale))) return rc;
  const int tiles = list_tiles(top_k, block, d);
  const ListPlan plan = decode_list_plan((int64_t)B * H_kv, top_k, tiles, d);
  const RowsLayout lay = rows_layout((int64_t)B * H_kv, H / H_kv, kPlanSms * plan.warps, d);
  if ((rc = check_workspace("decode_blocks", workspace, workspace_bytes, plan.cluster ? 0 : lay.all()))) return rc;
  uint32_t* err = nullptr;
  if ((rc = device_error_word(stream, &err))) return rc;
  DecodeRowsParams p;
  memset(&p, 0, sizeof(p));
  if ((rc = make_rows_map(&p.tk, k, d, L, L, (int64_t)B * H_kv, 16))) return rc;
  if ((rc = make_rows_map(&p.tv, v, d, L, L, (int64_t)B * H_kv, 16))) return rc;
  p.q = q;
  p.seq_lens = seq_lens;
  p.ids = block_ids;
  p.err = err;
  p.timeout_ns = device_wait_timeout_ns();
  p.B = B; p.H = H; p.H_kv = H_kv; p.L = L;
  p.top_k = top_k;
  p.block = block;
  p.box16 = block / 16;
  p.list_tiles = tiles;
  p.ctas = kPlanSms;
  p.warps = plan.warps;
  p.selftest = g_wait_selftest.load();
  p.scale_log2 = scale_log2(softmax_scale, d);
  if (plan.cluster) {
    p.cluster = plan.cluster;
    p.sink = sink;
    p.o = o;
    p.lse = lse;
    return launched(launch_decode_lists(p, d, stream), "list launch");
  }
  place_rows(&p, lay, static_cast<char*>(workspace));
  if ((rc = launched(launch_decode_rows(p, d, stream), "block launch"))) return rc;
  MergeParams m;
  memset(&m, 0, sizeof(m));
  m.b_o = p.part_o;
  m.b_ml = p.part_ml;
  m.group_start = p.group_start;
  m.warps = lay.warps;
  m.seq_lens = seq_lens;
  m.L = L;
  m.list_tiles = p.list_tiles;
  m.sink = sink;
  m.o = o;
  m.lse = lse;
  m.B = B; m.H = H; m.H_kv = H_kv;
  m.states = 1 + (int)(lay.warps / ((int64_t)B * H_kv));
  return launched(launch_decode_merge(m, d, stream), "merge launch");
}

// Test hook (not in the public header), host only: where the merge looks for
// the states of a list whose first tile the table gives as `start`.
void mattn_internal_list_pieces(int start, int tiles, int per, int warps, int* w0, int* n) {
  const ListPieces own = list_pieces(start, tiles, per, warps);
  *w0 = own.w0;
  *n = own.n;
}

// Test hook (not in the public header): the launches of decode_shared and
// decode_blocks until the next call leave out copies that their kernels wait for,
// so that the bounded waits and the error word can be exercised without a hang:
// 1 the row workers' first keys, 2 the prefix's queries, 0 none.
int mattn_internal_decode_wait_selftest(int what) {
  if (what < 0 || what > 2) return report_error(MATTN_ERR_INVALID_ARG, "what must be 0, 1 or 2");
  g_wait_selftest.store(what);
  return MATTN_OK;
}

// Test hook (not in the public header), host only: the plan of a decode_shared
// call: {sub, seqs, row_tiles, n_split, tiles, per_split, own_ctas}.
int mattn_internal_shared_plan(int B, int H, int H_kv, int P, int L, int d, int* out) {
  const int rc = check_shared(B, H, H_kv, P, L, d, MATTN_BF16);
  if (rc) return rc;
  const SharedPlan s = shared_plan(B, H, H_kv, P, L, d);
  const int v[7] = {s.sub, s.seqs, s.row_tiles, s.n_split, s.tiles, s.per_split, s.own_ctas};
  memcpy(out, v, sizeof(v));
  return MATTN_OK;
}

// Test hook (not in the public header), host only: how decode_blocks reads its
// lists: {CTAs of a group's cluster or 0 for equal shares, warps of a CTA}.
int mattn_internal_list_plan(int B, int H, int H_kv, int top_k, int block, int d, int* out) {
  const int rc = check_blocks(B, H, H_kv, top_k, block, d, MATTN_BF16);
  if (rc) return rc;
  const ListPlan s = decode_list_plan((int64_t)B * H_kv, top_k, list_tiles(top_k, block, d), d);
  out[0] = s.cluster;
  out[1] = s.warps;
  return MATTN_OK;
}

}  // extern "C"
