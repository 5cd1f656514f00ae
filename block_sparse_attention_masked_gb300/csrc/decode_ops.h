// Launch parameters and host-side plans of the decode step's operators: the
// head norms with the position rotation (qk_rope.cu), attention over a
// shared prefix (decode_shared.cu), attention over a sequence's own keys or
// its selected blocks (decode_rows.cu), block means and block selection
// (block_select.cu).  Their C entry points are in decode_ops_api.cpp.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace mattn {

// Every plan below is a function of the sizes alone, so that the workspace
// queries need no device: this is the SM count of the one target (GB300).
constexpr int kPlanSms = 152;

// Raises a kernel's dynamic shared-memory limit, once per kernel and device
// (the attribute call costs as much as a tenth of a launch).  `done`: the
// kernel's own bit set, one bit per device; devices past 64 ask every time.
template <class Kernel>
cudaError_t allow_shared(Kernel kern, size_t bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit && (done->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches a kernel as a programmatic dependent of the stream's previous grid:
// its CTAs are set up while that one ends, and each of these kernels begins with
// after_previous() (its first access to memory comes after the previous grid has
// completed), so that a chain of short calls does not pay a launch between each
// two (one token's rows for 64 requests: 6.1 us a call in a chain, 3.5 so).
template <class Kernel, class Params>
cudaError_t launch_chained(Kernel kern, unsigned grid_x, unsigned grid_y, int threads, size_t smem, int cluster,
                           const Params& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

#ifdef __CUDACC__
// Waits until the previous grid has completed and its results are visible, then
// lets the next one's CTAs be set up.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

// Two softmax weights as pairs of bf16 values, hi + lo, 2^-16 of a weight off at
// most.  Of a positive weight both are positive (its last bit is taken as set), so
// that an infinite value stays infinite in both products: a part that is 0 or
// negative would make it NaN.
__device__ __forceinline__ void two_bf16(float a, float b, uint32_t* hi, uint32_t* lo) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  *hi = __byte_perm(ua, ub, 0x7632);
  const float x = __uint_as_float(ua | 1u) - __uint_as_float(ua & 0xffff0000u);
  const float y = __uint_as_float(ub | 1u) - __uint_as_float(ub & 0xffff0000u);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(*lo) : "f"(y), "f"(x));
}
#endif

// ------------------------------------------------------------ qk_rope.cu
struct RopeParams {
  const void* src[3];       // q, k, v rows: element (b, n, head, c) at b * batch_stride + n * token_stride + head * d + c
  void* dst[3];             // q: [B][H][N][d]; k, v: [B][H_kv][L][d] (v may be null)
  int64_t batch_stride[3];  // in elements
  int64_t token_stride[3];
  const int32_t* positions; // [axes][B][N] or null: start + n on every axis
  const int32_t* starts;    // [B] cache row of token 0, or null: 0
  const int32_t* lens;      // [B] tokens of each sequence, or null: N
  const float* inv_freq;    // [rot]
  const float* weight[2];   // [d] norm weights of q and k, or null: no norm
  int B, H, H_kv, N, L, d;
  int axis_end[3];          // pairs [axis_end[a - 1], axis_end[a]) turn with axis a
  int rot;                  // rotated pairs
  int interleaved;          // pairs (2p, 2p + 1) instead of (p, p + rot)
  bool wide;                // fp32: every row starts on a 32-byte boundary
  int segs;                 // warps that share one token's rows
  float eps;
};
cudaError_t launch_qk_rope(const RopeParams& p, bool f32, cudaStream_t stream);

// ------------------------------------------------------------ decode_rows.cu
// Keys per tile (8 KB of K and V, 16 KB at d = 256) and warps of a CTA at most, each
// with two tiles in flight: 192 KB per SM.
constexpr int decode_rows_tile(int d) { return d == 64 ? 32 : 16; }
constexpr int decode_rows_warps(int d) { return d == 256 ? 6 : 12; }

struct DecodeRowsParams {
  CUtensorMap tk, tv;       // [B*H_kv][L][d] bf16 views, boxes of 64 columns x 16 keys (128-byte swizzle)
  const void* q;            // [B][H][d] bf16
  const int32_t* seq_lens;  // [B] or null: L
  const int32_t* ids;       // [B*H_kv][top_k] selected blocks, or null: every key in order
  float* part_o;            // [warps + B*H_kv][G][d] states, unnormalised (decode_rows.cuh)
  float* part_ml;           // [warps + B*H_kv][G][2]
  int* group_start;         // [B*H_kv] number of each list's first tile, then the tiles of a warp's share
  uint32_t* err;
  unsigned long long timeout_ns;
  int B, H, H_kv, L;
  int top_k, block, box16;  // block = 16 box16 keys
  int list_tiles;           // tiles of a list of top_k blocks (0: by the sequence's length)
  int ctas;                 // of the grid
  int warps;                // of a CTA
  int cluster;              // decode_lists_kernel: CTAs per group
  const float* sink;        // decode_lists_kernel writes o itself: [H] or null
  void* o;                  // [B][H][d] bf16
  float* lse;               // [B][H] or null
  float scale_log2;
  int selftest;             // 1: every worker's first copies are left out, so that its wait runs out
};
cudaError_t launch_decode_rows(const DecodeRowsParams& p, int d, cudaStream_t stream);

cudaError_t launch_decode_lists(const DecodeRowsParams& p, int d, cudaStream_t stream);

int decode_share_warps(int64_t tiles, int d);
struct ListPlan {
  int cluster;  // CTAs per group of decode_lists_kernel, or 0: decode_rows_kernel
  int warps;    // of a CTA
};
ListPlan decode_list_plan(int64_t groups, int top_k, int list_tiles, int d);

// ------------------------------------------------------------ decode_shared.cu
struct SharedPlan {
  int sub;      // query tiles per CTA (1 or 2)
  int seqs;     // sequences of a query tile, 128 / G: seqs * G of its 128 rows are used
  int row_tiles;
  int n_split;  // key splits
  int tiles;    // key tiles of the prefix
  int per_split;
  int own_ctas; // CTAs of the own keys, behind the prefix's
};
constexpr int shared_key_tile(int d) { return d == 256 ? 64 : 128; }
// Tiles in flight of a CTA (32 KB; 16 KB at d = 64).  More than the latency asks for
// cost bandwidth: 6 against 4 at 128 rows of 128 take 107.1 and 102.8 us for 640 MB,
// 12 against 6 at 256 rows of 64 110.9 and 107.5 for 320.
constexpr int shared_slots(int d, int sub) { return d == 64 ? 6 : (d == 256 || sub == 2 ? 5 : 4); }
// Row workers of a CTA among the prefix's (decode_share_warps where there is no prefix).
constexpr int shared_row_warps(int d, int sub) { return d == 256 ? 6 : (sub == 2 ? 12 : 8); }
SharedPlan shared_plan(int B, int H, int H_kv, int P, int L, int d);

struct SharedParams {
  CUtensorMap tk, tv;       // [H_kv][P][d] bf16 views, boxes of 64 columns x shared_key_tile(d) keys
  CUtensorMap tq;           // [B][H][d] bf16 view, boxes of 64 columns x G heads x plan.seqs sequences
  DecodeRowsParams own;     // the sequences' own keys (L = 0: none)
  CUtensorMap to;           // part_o as [H_kv][B * G][n_split][d]: boxes of 32 columns (128 bytes) x 32 rows
  float* part_o;            // [H_kv * B * G][n_split][d]
  float* part_ml;           // [H_kv * B * G][n_split][2]
  uint32_t* err;
  unsigned long long timeout_ns;
  int B, H, H_kv, P;
  int rows;                 // B * G
  SharedPlan plan;
  float scale_log2;
  int selftest;             // 2: the queries' copies are left out, so that the wait for them runs out
};
cudaError_t launch_decode_shared(const SharedParams& p, int d, cudaStream_t stream);

// The pieces of a group's own list: the row workers w0 .. w0 + n - 1 of `warps`,
// from the list's first tile, its tiles and the tiles of a worker's share.  A
// worker that gave up a wait leaves the rest of its share's entries unwritten, so
// the table may hold anything: n = 0 where it names no place among the workers.
struct ListPieces {
  int w0, n;
};
#ifdef __CUDACC__
__host__ __device__
#endif
inline ListPieces list_pieces(int start, int tiles, int per, int warps) {
  if (start < 0 || tiles < 1 || per < 1) return {0, 0};
  const uint32_t first = (uint32_t)start / (uint32_t)per;
  const uint32_t last = ((uint32_t)start + (uint32_t)(tiles - 1)) / (uint32_t)per;  // (below 2^32)
  if (last >= (uint32_t)warps) return {0, 0};
  return {(int)first, (int)(last - first) + 1};
}

// One merge for all: row (b, h)'s states of the prefix and of its own list,
// with the sink logit, into o and the log-sum-exp.
struct MergeParams {
  const float *a_o, *a_ml;   // prefix states [H_kv * B * G][na][..]
  const float *b_o, *b_ml;   // own states (DecodeRowsParams)
  const int* group_start;    // DecodeRowsParams'; null: no own lists
  const int32_t* seq_lens;
  int na;
  int warps;                 // row workers of the own lists
  int states;                // of a row, about
  int L, list_tiles;
  const float* sink;
  void* o;
  float* lse;
  int B, H, H_kv;
};
cudaError_t launch_decode_merge(const MergeParams& p, int d, cudaStream_t stream);

// ------------------------------------------------------------ block_select.cu
struct BlockMeansParams {
  const void* k;            // [B*H_kv][L][d] bf16
  void* means;              // [B*H_kv][n_blocks][d] bf16
  const int32_t* seq_lens;  // [B] or null: L
  const int32_t* first;     // [B] or null: 0
  int B, H_kv, L, n_blocks, block;
  int max_new, span;        // new keys of a sequence at most, and the blocks they can lie in
};
cudaError_t launch_block_means(const BlockMeansParams& p, int d, cudaStream_t stream);

constexpr int kSelectMaxBlocks = 32768;

// A block's score as an ordered key, and a bound of its error.
struct __align__(8) Score {
  uint32_t key;
  float err;
};

struct DecodeSelectParams {
  const void* q;            // [B][H][d] bf16
  const void* means;        // [B*H_kv][n_blocks][d] bf16
  const int32_t* seq_lens;  // [B] or null: n_blocks * block
  Score* scores;            // [B*H_kv][n_blocks]
  double* again;            // [B*H_kv][n_blocks] scores formed again in 64 bits
  int32_t* ids;             // out [B*H_kv][top_k]
  int B, H, H_kv, n_blocks, block, top_k, keep_first, keep_recent;
  int ctas;                 // of a (sequence, key/value head)'s cluster (set by the launch)
};
cudaError_t launch_decode_select(const DecodeSelectParams& p, int d, cudaStream_t stream);

}  // namespace mattn
