// Checks and layouts that the C entry points of the operators share
// (decode_ops_api.cpp, paged_ops_api.cpp).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "decode_ops.h"
#include "launch_prep.h"
#include "mattn.h"

namespace mattn {

constexpr int64_t kMaxRows = 1 << 30;
constexpr int kMaxGroup = 16;  // query heads per key/value head

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

inline int check_heads(const char* what, int B, int H, int H_kv, int d, int dtype) {
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

inline int check_scale(const char* what, float scale) {
  if (!(scale >= 0.f) || std::isinf(scale))
    return report_error(MATTN_ERR_INVALID_ARG, "%s: softmax_scale must be finite and >= 0", what);
  return MATTN_OK;
}

inline int check_small(const char* what, const void* lse, const void* lens, const void* sink) {
  if (!aligned(lse, 4) || !aligned(lens, 4) || !aligned(sink, 4))
    return report_error(MATTN_ERR_INVALID_ARG, "%s: lse, seq_lens and sink must be 4-byte aligned", what);
  return MATTN_OK;
}

inline int check_workspace(const char* what, const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return report_error(MATTN_ERR_CAPACITY, "%s: the workspace holds %zu bytes, %zu are needed", what, ws ? have : 0,
                        need);
  if (!aligned(ws, 256)) return report_error(MATTN_ERR_INVALID_ARG, "%s: the workspace must be 256-byte aligned", what);
  return MATTN_OK;
}

inline int launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return report_error(MATTN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return MATTN_OK;
}

inline float scale_log2(float scale, int d) {
  return (scale > 0.f ? scale : 1.0f / std::sqrt((float)d)) * 1.4426950408889634f;
}

// States of `rows` query rows in n splits: O, then (reference, sum).
inline size_t state_bytes(int64_t rows, int n, int d) {
  return round256((size_t)rows * n * d * 4) + round256((size_t)rows * n * 8);
}

// States of the own lists: a slot for each (warp, group) piece, then the
// lists' starts (DecodeRowsParams).
struct RowsLayout {
  int warps;
  size_t o_bytes, ml_bytes, start_bytes;
  size_t all() const { return o_bytes + ml_bytes + start_bytes; }
};

inline RowsLayout rows_layout(int64_t groups, int G, int warps, int d) {
  RowsLayout r;
  r.warps = warps;
  r.o_bytes = round256((size_t)(warps + groups) * G * d * 4);
  r.ml_bytes = round256((size_t)(warps + groups) * G * 8);
  r.start_bytes = round256((size_t)(groups + 1) * 4);
  return r;
}

inline void place_rows(DecodeRowsParams* p, const RowsLayout& r, char* ws) {
  p->part_o = reinterpret_cast<float*>(ws);
  p->part_ml = reinterpret_cast<float*>(ws + r.o_bytes);
  p->group_start = reinterpret_cast<int*>(ws + r.o_bytes + r.ml_bytes);
}

// A buffer's bytes [lo, hi); hi wraps for no buffer that can exist.
struct Extent {
  uintptr_t lo, hi;
  bool meets(const Extent& x) const { return lo < x.hi && x.lo < hi && lo < hi && x.lo < x.hi; }
};
inline Extent extent_of(const void* p, uint64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (p ? bytes : 0)};
}
// Whether one of `outs` meets one of `ins` or another of `outs`.
template <int N, int M>
bool any_meet(const Extent (&ins)[N], const Extent (&outs)[M]) {
  for (int i = 0; i < M; ++i) {
    for (const Extent& x : ins)
      if (outs[i].meets(x)) return true;
    for (int j = 0; j < i; ++j)
      if (outs[i].meets(outs[j])) return true;
  }
  return false;
}

}  // namespace mattn
