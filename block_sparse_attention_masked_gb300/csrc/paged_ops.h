// Launch parameters and host-side plans of the operators around a paged cache:
// rows written into it and read back (paged_cache.cu), decode attention over
// it (decode_paged.cu) and attention over packed prompts (attention_packed.cu).
// Their C entry points are in paged_ops_api.cpp.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_ops.h"

namespace mattn {

// ------------------------------------------------------------ paged_cache.cu
struct CacheRowsParams {
  void* rows[2];             // k and v rows: (t, h, c) at t * row_token + h * row_head + c (bf16)
  int64_t row_token[2], row_head[2];
  void* pages[2];            // (page, h, r, c) at page * page_stride + h * head_stride + r * row_stride + c
  int64_t page_stride[2], head_stride[2], row_stride[2];  // in elements
  uint8_t* exps[2];          // e4m3: (page, h, r) at ..
  int64_t exp_page[2], exp_head[2], exp_row[2];
  const int32_t* table;      // [B][table_pages]
  const int32_t* cu;         // [B + 1], or null: token t is sequence t's
  const int32_t* starts;     // [B] position of a sequence's first row, or null: 0
  int B, T, H_kv, d;
  int page, table_pages, n_pages;
  int heads, segs;           // of a lane group; segs of them are a token (set by the launch)
};
cudaError_t launch_cache_write(const CacheRowsParams& p, bool e4m3, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheRowsParams& p, bool e4m3, cudaStream_t stream);

// ------------------------------------------------------------ decode_paged.cu
// Keys per tile: as the row workers' of decode_rows.cuh in bf16; in eight bits 32, 64 at
// d = 64 (8 KB of K and V; half of it took 64 sequences of 6,144 keys 101 us, so 86), 16 for
// more than eight query heads of 256, whose states leave few registers (16 sequences:
// 82 us with 32, 55 so).
constexpr int paged_tile(int d, bool e4m3, int group) {
  return !e4m3 ? decode_rows_tile(d) : (d == 64 ? 64 : (d == 256 && group > 8 ? 16 : 32));
}
constexpr int paged_shift(int d, bool e4m3, int group) {
  return paged_tile(d, e4m3, group) == 64 ? 6 : (paged_tile(d, e4m3, group) == 32 ? 5 : 4);
}

struct DecodePagedParams {
  CUtensorMap tk, tv;        // [n_pages][H_kv][page][d] views, boxes of 16 keys x 128 bytes (or a row of 64)
  const void* q;             // [B][H][d] bf16
  const int32_t* table;      // [B][table_pages]
  const int32_t* seq_lens;   // [B] or null: table_pages * page
  const uint8_t* exps[2];    // e4m3
  int64_t exp_page[2], exp_head[2], exp_row[2];
  float* part_o;             // states and the lists' starts as DecodeRowsParams has them
  float* part_ml;
  int* group_start;
  uint32_t* err;
  unsigned long long timeout_ns;
  int B, H, H_kv;
  int page, table_pages, n_pages, L;  // L = table_pages * page
  int window, first;         // keys [len - window, len) and [0, first); window 0: all
  int ctas, warps;
  int cluster;               // CTAs of a group (decode_paged_cluster_kernel writes o itself), or 0: equal shares and states
  const float* sink;
  void* o;                   // [B][H][d] bf16
  float* lse;                // [B][H] or null
  float scale_log2;
  int selftest;              // 1: every worker's first copies are left out, so that its wait runs out
};
cudaError_t launch_decode_paged(const DecodePagedParams& p, int d, bool e4m3, cudaStream_t stream);

// ------------------------------------------------------------ attention_packed.cu
// A pair of query tiles of one sequence, as the plan kernel lists them (most key tiles
// first): rows q_row .. q_row + rows - 1 of the packed queries, the sequence's keys
// k_row .. k_row + keys - 1, the first row's position among them (negative: none).
struct __align__(16) PackedPair {
  int q_row, rows, k_row, keys, pos0, pad[3];
};
constexpr int kPackedDirect = 4;
struct PackedPlan {        // in the workspace
  int next;                // the next item that no CTA has
  int pairs;
  int pad[14];
  PackedPair pair[1];
};
// Pairs of T rows in B sequences at most (256 rows each, a shorter one behind).
inline int64_t packed_pairs(int64_t T, int64_t B) { return T / 256 + (B < T ? B : T); }

struct PackedParams {
  CUtensorMap tq[2], tk[2], tv;  // [T][heads][d] views: boxes of 128 rows of one head (tile_mma.cuh; d = 256, v: 32)
  void* o;                       // [T][H][d] bf16
  float* lse;                    // [H][T] or null
  const float* sink;             // [H] or null
  const void* v;                 // the values once more, for keys that are not finite (attention_packed.cu)
  int64_t v_token, v_head;
  const int32_t *cu_q, *cu_k;    // [B + 1]
  PackedPlan* plan;
  int* marked;                   // [2 max_pairs * H] of a CTA's marked items, the one marked before it
  uint32_t* err;
  unsigned long long timeout_ns;
  int B, T, T_k, H, H_kv, group;
  int causal, window;            // window 0: none
  int wide;                      // o is 32-byte aligned
  int max_pairs, work_shift;
  int direct;                    // no plan: at most kPackedDirect items a CTA, in the sequences' order (packed_direct)
  float scale_log2;
  int selftest;                  // 1: the first K tile is left out, so that the wait for it runs out
};
cudaError_t launch_attention_packed(const PackedParams& p, int d, cudaStream_t stream);
// Behind the plan, for heads of 256 (attention_packed_256.cu), whose boxes of v are of
// this many rows.
constexpr int kPackedValues256 = 32;
cudaError_t launch_attention_packed_256(const PackedParams& p, cudaStream_t stream);

}  // namespace mattn
