// Attention over packed sequences (mattn_attention_packed), for sm_103a: sequence b has
// queries cu_q[b] .. cu_q[b + 1] - 1 and keys cu_k[b] .. cu_k[b + 1] - 1 of the packed
// rows, and query i of n sees, of its sequence's m keys, all, or (causal) those up to
// m - n + i, of them the last `window`:
//   O_i = sum_j p_ij v_j / (sum_j p_ij + exp(sink)),  p_ij = exp(scale q_i . k_j).
// 4 d FLOPs a visible (head, pair): bound by the tensor cores and the exponentials, as
// the persistent forward (attention_persist.cu), whose schedule this one has: a CTA per
// SM takes pairs of 128-row query tiles of one (sequence, head), runs each tile's
//     S = Q K^T, P = exp2(S scale log2e - m), O += P V
// over its key tiles (tcgen05, P from tensor memory) with the two tiles sharing the
// staged K and V, and begins the next pair's products while the last one is written.
//
// What differs: the work is known to the device alone.  packed_plan_kernel, one CTA,
// lists the pairs with most key tiles first; item i of the grid is pair i / H, head i % H
// (the heads of one pair run side by side and share K and V in L2), and a CTA takes the
// next item that none has (a counter) when the K tiles of its current one run out: long
// prompts first, short ones fill the end.
//
// What a row does not see.  Tiles begin at any packed row and reach into the next sequence
// (past the last row TMA fills zeros): query rows past the end are not written, keys past
// it are masked.  A hidden key's weight is 0, but 0 times an infinity or NaN among its
// values is NaN, so a row whose output is not finite and that saw a tile in part marks its
// item, and a CTA does its marked items again after its others: with those tiles' values
// looked over in shared memory before the product, rows past the end and values that are
// not finite taken out, and the latter added to the output of each row that sees them.
// (Looking over every such tile the first time, beside the pipeline, cost 5% of the 16,384
// tokens of eight prompts and 16% of a window of 576.)
//
// Roles (384 threads) and tensor memory: as attention_persist.cu; every wait is bounded
// in time (those for an item: in time without a key tile's progress) and gives up by
// raising a CTA-wide abort flag and a device error bit.
//
// Measured (TFLOP/s of visible pairs): one causal sequence of 16,384, 8 heads of 128, 349-357 us =
// 1,540-1,576 (attention_fwd.cu's paired schedule 367), eight prompts of 1 to 3,352 tokens, 32 heads,
// 306-323 us = 1,175-1,240, the same tokens as 64 prompts of 256 91 us = 380, 12 images of 1 to 3,038 patches, 16 heads of 80,
// 186 us = 929.  Long lists run at the forward's own rate; an item costs 2.5 to 5 us beside its
// tiles (its first S, its last P V and its output, which only the other query tile's work hides).
// Tried without gain: the output staged in shared memory (d = 80 and 64 2% slower), O read from tensor memory 32 or
// 64 columns at a time, a warp for K tiles alone, the scheduler's next pair fetched ahead.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention_packed.cuh"
#include "attention_tiles.cuh"
#include "kernel_params.h"
#include "paged_ops.h"
#include "plan_rules.h"
#include "ptx.cuh"
#include "tile_mma.cuh"

namespace mattn {
namespace {

// ------------------------------------------------------------ the plan
constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;

__device__ __forceinline__ int pair_work(const PackedParams& p, const PackedPair& x) {
  int w = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    int lo, hi;
    seen_tiles<7>(p, x.pos0 + 128 * s, min(x.rows - 128 * s, 128), x.keys, &lo, &hi);
    w += hi - lo + 1;
  }
  return w;
}

// Lists the pairs by the number of key tiles they multiply, most first (a counting sort;
// the order inside a bin is any: an item's result does not depend on it).
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const __grid_constant__ PackedParams p) {
  __shared__ int before[kPlanThreads + 1];  // pairs of the chunk's sequences before each
  __shared__ int bins[kBins];
  __shared__ int sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  after_previous();
  // exclusive sums of x over the CTA; the whole sum in `total`
  auto scan = [&](int x, int* total) {
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    const int mine = sums[lane];
    int all = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, all, off);
      if (lane >= off) all += y;
    }
    *total = __shfl_sync(0xffffffffu, all, 31);
    const int base = __shfl_sync(0xffffffffu, all - mine, warp);
    __syncthreads();
    return base + incl - x;
  };
  auto chunk = [&](int b0) {  // pairs of sequences b0 .. b0 + kPlanThreads - 1 into `before`; how many
    int n = 0, total;
    if (b0 + tid < p.B) n = (sequence(p, b0 + tid).nq + 255) / 256;
    before[tid] = scan(n, &total);
    if (tid == 0) before[kPlanThreads] = total;
    __syncthreads();
    return total;
  };
  auto pair_at = [&](int b0, int j) {  // pair j of the chunk
    int lo = 0, hi = kPlanThreads;     // before[lo] <= j < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= j) lo = mid;
      else hi = mid;
    }
    const Sequence s = sequence(p, b0 + lo);
    const int i = (j - before[lo]) * 256;
    PackedPair x;
    x.q_row = s.q0 + i;
    x.rows = s.nq - i;
    x.k_row = s.k0;
    x.keys = s.nk;
    x.pos0 = s.nk - s.nq + i;
    return x;
  };
  auto bin_of = [&](const PackedPair& x) {
    const int w = pair_work(p, x) >> p.work_shift;
    return kBins - 1 - min(w, kBins - 1);
  };
  bins[tid] = 0;
  __syncthreads();
  const bool one = p.B <= kPlanThreads;
  int n = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    n = chunk(b0);
    for (int j = tid; j < n; j += kPlanThreads) atomicAdd(&bins[bin_of(pair_at(b0, j))], 1);
    __syncthreads();
  }
  int total;
  bins[tid] = scan(bins[tid], &total);
  if (tid == 0) {
    p.plan->next = 0;
    p.plan->pairs = min(total, p.max_pairs);
  }
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    if (!one) n = chunk(b0);
    for (int j = tid; j < n; j += kPlanThreads) {
      const PackedPair x = pair_at(b0, j);
      const int at = atomicAdd(&bins[bin_of(x)], 1);
      // (sequences that overlap could have more pairs than there is room for)
      if (at >= 0 && at < p.max_pairs) p.plan->pair[at] = x;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ the attention
constexpr int kThreads = 384;
constexpr uint32_t kRegsControl = 56, kRegsSoftmax = 224;
static_assert(kRegsControl + 2 * kRegsSoftmax == 3 * 168, "register split must match the launch budget");
constexpr int kItems = 4;   // of the ring
constexpr int kQSlots = 3;
constexpr int kReaders = 11;  // of an item: the V producer, two issuers, eight softmax warps

// An item as every role reads it, or (h < 0) the word to finish what is under way, after
// which there is nothing more (kEnd) or may be (kDrain).
constexpr int kDrain = -2, kEnd = -1;
struct Item {
  int q_row, rows, k_row, keys, pos0, h, id;
  int lo, n;                    // its key tiles lo .. lo + n - 1
  int lo0, hi0, lo1, hi1;       // those of each query tile (hi < lo: none)
  int marked;                   // some row of its output is not finite
  int again;                    // the second time
  __device__ __forceinline__ void set(const PackedParams& p, const PackedPair& pair, int item) {
    const int4 a = *reinterpret_cast<const int4*>(&pair);
    q_row = a.x; rows = a.y; k_row = a.z; keys = a.w;
    pos0 = pair.pos0;
    // (a pair that the plan left unwritten, as for sequences that overlap, may hold anything: no rows then)
    if (!in_bounds(p, pair)) rows = 0;
    h = item % p.H;
    id = item;
    seen_tiles<7>(p, pos0, min(rows, 128), keys, &lo0, &hi0);
    seen_tiles<7>(p, pos0 + 128, min(rows - 128, 128), keys, &lo1, &hi1);
    lo = hi0 < lo0 ? lo1 : (hi1 < lo1 ? lo0 : min(lo0, lo1));
    const int end = max(hi0, hi1);
    n = end < lo ? 0 : end - lo + 1;
  }
  __device__ __forceinline__ bool uses(int s, int kt) const { return s ? kt >= lo1 && kt <= hi1 : kt >= lo0 && kt <= hi0; }
  __device__ __forceinline__ int first(int s) const { return s ? (hi1 < lo1 ? -1 : lo1) : (hi0 < lo0 ? -1 : lo0); }
  __device__ __forceinline__ int last(int s) const { return s ? hi1 : hi0; }
  // the key tiles [lo, hi] that every row of query tile s sees whole
  __device__ __forceinline__ void whole(const PackedParams& p, int s, int* lo, int* hi) const {
    const int pos = pos0 + 128 * s;
    *hi = ((p.causal ? min(keys, pos + 1) : keys) >> 7) - 1;
    *lo = p.window ? (max(0, pos + min(rows - 128 * s, 128) - p.window) + 127) >> 7 : 0;
  }
  // whether some row of a query tile that multiplies key tile kt does not see all of it
  __device__ __forceinline__ bool partial(const PackedParams& p, int kt) const {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      int whole_lo, whole_hi;
      whole(p, s, &whole_lo, &whole_hi);
      if (uses(s, kt) && (kt < whole_lo || kt > whole_hi)) return true;
    }
    return false;
  }
};

// The item marked before `id` in its CTA, or -1.
__device__ __forceinline__ int next_marked(const PackedParams& p, int id) {
  const int x = p.marked[id];
  return x < p.max_pairs * p.H ? x : -1;
}

struct Bar {
  uint64_t q_full[kQSlots], q_empty[kQSlots];
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t v_land;
  uint64_t s_full[2], p_full[2], o_full[2], drain[2];
  uint64_t item_full[kItems], item_empty[kItems];
  uint32_t tmem_base;
  int abort_flag;
  uint32_t mma_turn;
  uint32_t tiles;          // K tiles whose copies are under way, of all items
  int marked;              // the CTA's last marked item, from which PackedParams::marked leads to the others; -1: none
  Item items[kItems];
  PackedPair direct[kPackedDirect];  // the CTA's items' pairs, where there is no plan
  int direct_total;                  // items of the grid
  __device__ __forceinline__ const PackedPair& pair(const PackedParams& p, int item) const {
    return p.direct ? direct[item / (int)gridDim.x] : p.plan->pair[item / p.H];
  }
};

// Without a plan, a CTA's k-th item: there and back through the CTAs, so that those with
// the first, longest ones of a sequence get the last ones too.
__device__ __forceinline__ int direct_item(int k) {
  return k * (int)gridDim.x + ((k & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
}
// The pairs of this CTA's items (one warp), in the sequences' order: few items need no
// order by length, and the plan kernel takes 3 us (8 prompts of 700 tokens 13.8 us with
// it, 10.7 so; 9 of 64 with 32 heads 16.0 and 12.3; 4 of 500 23.2 and 22.3).
__device__ __forceinline__ void plan_direct(const PackedParams& p, Bar* bar) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    Sequence s = {0, 0, 0, 0};
    if (b0 + lane < p.B) s = sequence(p, b0 + lane);
    const int n = (s.nq + 255) / 256;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
#pragma unroll
    for (int k = 0; k < kPackedDirect; ++k) {
      // (a sequence's last rows, which see most keys, first)
      const int i = before + incl - 1 - direct_item(k) / p.H;
      if (i >= 0 && i < n) bar->direct[k] = {s.q0 + i * 256, s.nq - i * 256, s.k0, s.nk, s.nk - s.nq + i * 256, {0, 0, 0}};
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) bar->direct_total = min(before, p.max_pairs) * p.H;
  __syncwarp();
}

__device__ __forceinline__ void fail(const PackedParams& p, Bar* bar, uint32_t bit) {
  *reinterpret_cast<volatile int*>(&bar->abort_flag) = 1;
  atomicOr(p.err, bit);
}
// 128 rows of one head from packed row `row` on, laid out as tile_mma.cuh has them.
template <int D>
__device__ __forceinline__ void load_rows(const CUtensorMap* maps, uint8_t* dst, uint64_t* bar, int h, int row,
                                          uint64_t policy) {
  using G = Geo<D>;
#pragma unroll
  for (int c = 0; c < G::kChunks; ++c)
    ptx::tma_load_3d_hint(dst + c * G::kChunkBytes, &maps[0], bar, c * 64, h, row, policy);
  if (G::kRem) ptx::tma_load_3d_hint(dst + G::kChunks * G::kChunkBytes, &maps[1], bar, 0, h, row, policy);
}

// The scheduler and the Q and K streams (one thread).  Three cursors over the CTA's
// items, none of which blocks another: the item to publish, the Q tile to load, the K
// tile to load.
template <int D, int KS>
__device__ __forceinline__ void produce_items(const PackedParams& p, Bar* bar, uint8_t* sq, uint8_t* sk,
                                              volatile int* abort_flag) {
  using G = Geo<D>;
  const uint64_t keep = ptx::l2_policy_evict_last(), once = ptx::l2_policy_evict_first();
  const int total = p.direct ? bar->direct_total : p.plan->pairs * p.H;
  int id = blockIdx.x;
  int pub = 0;        // items published
  bool done = false;  // the last of them is the end
  bool again = false; // the marked items' turn has come
  int drain = -1;     // the item whose end it waits for
  int qi = 0, qs = 0, t = 0;
  int ki = 0, kj = 0, e = 0;
  uint64_t t_idle = 0;
  uint32_t idle = 0;
  while (!(done && qi == pub - 1 && ki == pub - 1)) {
    bool moved = false;
    // the next item, once the K tiles of the current one run out
    if (!done && (pub == ki || (pub == ki + 1 && bar->items[ki % kItems].n - kj <= 4)) && pub < qi + kItems &&
        ptx::mbar_test_wait(&bar->item_empty[pub % kItems], ((pub / kItems) & 1) ^ 1) &&
        (drain < 0 || ptx::mbar_test_wait(&bar->item_empty[drain % kItems], (drain / kItems) & 1))) {
      if (drain >= 0) {  // every item so far is written
        drain = -1;
        again = true;
        id = *reinterpret_cast<volatile int*>(&bar->marked);
      }
      Item& it = bar->items[pub % kItems];
      if (again ? id >= 0 : id < total) {
        it.set(p, bar->pair(p, id), id);
        it.marked = 0;
        it.again = again ? 1 : 0;
        id = again ? next_marked(p, id) : (p.direct ? direct_item(id / (int)gridDim.x + 1) : gridDim.x + atomicAdd(&p.plan->next, 1));
      } else {
        it.h = again ? kEnd : kDrain;
        it.n = 0;
        it.lo0 = it.lo1 = 0;
        it.hi0 = it.hi1 = -1;
        done = again;
        if (!again) drain = pub;
      }
      ptx::mbar_arrive(&bar->item_full[pub % kItems]);
      ++pub;
      moved = true;
    }
    if (ki < pub - (done ? 1 : 0)) {
      const Item& it = bar->items[ki % kItems];
      if (kj == it.n) {
        ++ki;
        kj = 0;
        moved = true;
      } else if (ptx::mbar_test_wait(&bar->k_empty[e % KS], ((e / KS) & 1) ^ 1)) {
        const int slot = e % KS;
        const int row = it.k_row + (it.lo + kj) * kTile;
        if (!debug_check(p.err, row >= 0 && row < p.T_k && it.h < p.H, kSiteLoad)) {
          *abort_flag = 1;
          break;
        }
        ptx::mbar_arrive_expect_tx(&bar->k_full[slot], G::kTileBytes);
        if (!(p.selftest == 1 && e == 0))
          load_rows<D>(p.tk, sk + slot * G::kTileBytes, &bar->k_full[slot], it.h / p.group, row, keep);
        ++e;
        ++kj;
        moved = true;
        *reinterpret_cast<volatile uint32_t*>(&bar->tiles) = (uint32_t)e;
      }
    }
    if (qi < pub - (done ? 1 : 0)) {
      const Item& it = bar->items[qi % kItems];
      if (it.first(qs) < 0) {  // nothing to multiply: no Q tile
        qi += qs;
        qs ^= 1;
        moved = true;
      } else if (ptx::mbar_test_wait(&bar->q_empty[t % kQSlots], ((t / kQSlots) & 1) ^ 1)) {
        const int slot = t % kQSlots, row = it.q_row + 128 * qs;
        if (!debug_check(p.err, row >= 0 && row < p.T, kSiteLoad)) {
          *abort_flag = 1;
          break;
        }
        ptx::mbar_arrive_expect_tx(&bar->q_full[slot], G::kTileBytes);
        load_rows<D>(p.tq, sq + slot * G::kTileBytes, &bar->q_full[slot], it.h, row, once);
        ++t;
        qi += qs;
        qs ^= 1;
        moved = true;
      }
    }
    if (moved) {
      idle = 0;
    } else if ((++idle & 63u) == 0) {
      // bounded like every wait: gives up after timeout_ns without progress
      if (*abort_flag) break;
      const uint64_t now = ptx::globaltimer_ns();
      if (idle == 64) {
        t_idle = now;
      } else if (now - t_idle > p.timeout_ns) {
        fail(p, bar, kErrProducer);
        break;
      }
    }
  }
  let_copies_land(abort_flag);
}

// A landed V tile: rows from `rows` on and values that are not finite become zeros.  One
// warp; the layout does not matter, as a row's columns lie in rows of every chunk.
template <int D>
__device__ __forceinline__ void clean_tile(uint8_t* tile, int rows) {
  using G = Geo<D>;
  constexpr int kRow = G::kVW * 2;
  const int lane = threadIdx.x & 31, n = rows * kRow / 16;  // 16-byte pieces of a chunk
  for (int c = 0; c < G::kVChunks; ++c) {
    uint4* x = reinterpret_cast<uint4*>(tile + c * G::kVChunkBytes);
    for (int i = lane; i < kTile * kRow / 16; i += 32) {
      const uint4 v = x[i];
      x[i] = i < n ? make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w)) : make_uint4(0, 0, 0, 0);
    }
  }
  ptx::fence_proxy_async_shared();
  __syncwarp();
}

// A marked item's output, written the second time without the values that are not finite
// and that some row of their tile does not see: they are added to the rows that see them
// (with a positive weight each).  A thread a row.
template <int D>
__device__ __forceinline__ void add_odd_values(const PackedParams& p, const Item& it, int row) {
  const int s = row >> 7;
  int lo = 0, hi = it.keys - 1;
  if (p.causal) {
    hi = min(hi, it.pos0 + row);
    if (p.window) lo = max(0, it.pos0 + row - p.window + 1);
  }
  if (row >= it.rows || it.first(s) < 0) return;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.o) + (((int64_t)it.q_row + row) * p.H + it.h) * D;
  for (int kt = it.lo; kt < it.lo + it.n; ++kt) {
    if (!it.partial(p, kt)) continue;
    for (int j = max(lo, kt * kTile); j <= min(hi, kt * kTile + kTile - 1); ++j) {
      const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.v) + (it.k_row + (int64_t)j) * p.v_token +
                               (it.h / p.group) * p.v_head;
#pragma unroll 4
      for (int c = 0; c < D; c += 2) {
        const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(v + c)), odd = x ^ clean(x);
        if (!odd) continue;
        __nv_bfloat162* to = reinterpret_cast<__nv_bfloat162*>(o + c);
        const float2 y = __bfloat1622float2(*to);
        *to = __floats2bfloat162_rn(y.x + __uint_as_float(odd << 16), y.y + __uint_as_float(odd & 0xffff0000u));
      }
    }
  }
}

// Waits for the CTA's item i; null if the wait gave up.
__device__ __forceinline__ const Item* take_item(const PackedParams& p, Bar* bar, int i, volatile int* abort_flag) {
  // (the softmax of a query tile without rows is here while the other's keys pass)
  const bool got = item_wait(&bar->tiles, abort_flag, [&] {
    return ptx::mbar_wait(&bar->item_full[i % kItems], (i / kItems) & 1, p.timeout_ns, abort_flag);
  });
  return __all_sync(0xffffffffu, got) ? &bar->items[i % kItems] : nullptr;
}
__device__ __forceinline__ void drop_item(Bar* bar, int i) {  // (one warp, after its last read)
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bar->item_empty[i % kItems]);
}

// This thread's row of a tile that it sees in part: the scores of columns outside [lo, hi]
// (none inside where lo > hi) become -inf where they lie, in tensor memory.  In the pass
// over the scores itself the same selects slow every tile, masked or not, as its code is
// fetched and its registers are held (one sequence of 16,384, 8 heads of 128: 369 us, so 359, and
// 348 with the bounds of the tiles seen whole kept in registers).
__device__ __forceinline__ void mask_scores(uint32_t s_tmem, int lo, int hi) {
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    const uint32_t vis = range_bits(g, lo, hi);
    if (__all_sync(0xffffffffu, vis == 0xffffffffu)) continue;
    float x[32];
    ptx::tmem_ld32(s_tmem + 32 * g, x);
    ptx::tmem_wait_ld();
    uint32_t u[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) u[j] = (vis >> j) & 1u ? __float_as_uint(x[j]) : 0xff800000u;
    ptx::tmem_st32(s_tmem + 32 * g, u);
  }
  ptx::tmem_wait_st();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_packed_kernel(const __grid_constant__ PackedParams p) {
  using G = Geo<D>;
  constexpr int KS = G::kStages, VS = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = base;
  uint8_t* sk = sq + kQSlots * G::kTileBytes;
  uint8_t* sv = sk + KS * G::kTileBytes;
  Bar* bar = reinterpret_cast<Bar*>(sv + VS * G::kTileBytes);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&p.tq[0]);
    ptx::prefetch_tmap(&p.tk[0]);
    ptx::prefetch_tmap(&p.tv);
    for (int i = 0; i < kQSlots; ++i) {
      ptx::mbar_init(&bar->q_full[i], 1);
      ptx::mbar_init(&bar->q_empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      ptx::mbar_init(&bar->k_full[i], 1);
      ptx::mbar_init(&bar->k_empty[i], 2);  // one commit from each issuer
      ptx::mbar_init(&bar->v_full[i], 1);
      ptx::mbar_init(&bar->v_empty[i], 2);
    }
    ptx::mbar_init(&bar->v_land, 1);
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bar->s_full[s], 1);
      ptx::mbar_init(&bar->p_full[s], kTile);
      ptx::mbar_init(&bar->o_full[s], 1);
      ptx::mbar_init(&bar->drain[s], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      ptx::mbar_init(&bar->item_full[i], 1);
      ptx::mbar_init(&bar->item_empty[i], kReaders);
    }
    bar->abort_flag = 0;
    bar->mma_turn = 0;
    bar->tiles = 0;
    bar->marked = -1;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&bar->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  after_previous();  // the plan, and whatever the inputs come from
  if (p.direct) {
    if (warp == 0) plan_direct(p, bar);
    __syncthreads();
  }

  if (warp == 0) {
    ptx::setmaxnreg_dec<kRegsControl>();
    if (lane == 0) produce_items<D, KS>(p, bar, sq, sk, abort_flag);
  } else if (warp == 3) {
    // ------------------------------------------------------------ V producer
    ptx::setmaxnreg_dec<kRegsControl>();
    const uint64_t keep = ptx::l2_policy_evict_last();
    int e = 0;
    uint32_t lands = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Item* it = take_item(p, bar, i, abort_flag);
      if (!it) {
        ok = false;
        break;
      }
      if (it->h == kEnd) break;
      const int n = it->n, lo = it->lo, keys = it->keys, k_row = it->k_row, h = it->h / p.group;  // (kDrain: n = 0)
      for (int j = 0; j < n; ++j, ++e) {
        const int slot = e % VS, kt = lo + j;
        uint8_t* tile = sv + slot * G::kTileBytes;
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->v_empty[slot], ((e / VS) & 1) ^ 1, p.timeout_ns, abort_flag))) {
          ok = false;
          break;
        }
        const bool look = it->again && it->partial(p, kt);
        uint64_t* landing = look ? &bar->v_land : &bar->v_full[slot];
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(landing, G::kTileBytes);
#pragma unroll
          for (int c = 0; c < G::kVChunks; ++c)
            ptx::tma_load_3d_hint(tile + c * G::kVChunkBytes, &p.tv, landing, c * G::kVW, h, k_row + kt * kTile, keep);
        }
        __syncwarp();
        if (look) {
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->v_land, lands & 1, p.timeout_ns, abort_flag))) {
            ok = false;
            break;
          }
          ++lands;
          clean_tile<D>(tile, min(keys - kt * kTile, kTile));
          if (lane == 0) ptx::mbar_arrive(&bar->v_full[slot]);
        }
      }
      if (ok) drop_item(bar, i);
    }
    if (!ok && lane == 0) fail(p, bar, kErrProducer);
    __syncwarp();
    let_copies_land(abort_flag);
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------ MMA issuers
    // As attention_persist.cu's: both walk every entry e of the CTA's stream and, in
    // ticket order 2 e + s, issue P V (e - 1) and S (e).
    ptx::setmaxnreg_dec<kRegsControl>();
    const int s = warp - 1;
    auto wait_all = [&](uint64_t* b, uint32_t parity) {
      return __all_sync(0xffffffffu, ptx::mbar_wait(b, parity, p.timeout_ns, abort_flag));
    };
    constexpr uint32_t tile4 = G::kTileBytes >> 4;  // descriptor start-address units
    const uint32_t q4 = ptx::smem_addr(sq) >> 4;
    const uint32_t k4 = ptx::smem_addr(sk) >> 4;
    const uint32_t v4 = ptx::smem_addr(sv) >> 4;
    const uint32_t s_tm = tmem + s * 128;
    const uint32_t o_tm = tmem + 256 + s * 128;
    bool ok = true, issued_any = false;
    bool pend = false, pend_first = false, pend_last = false;
    bool open = false;    // entry e - 1's V is not released yet
    uint32_t pcount = 0;  // P tiles consumed
    int e = 0;
    int t = 0;  // Q tiles of both query tiles so far
    // the last entry so far: its V slot and this query tile's pending P V
    auto finish = [&]() {
      if (!open) return true;
      const int ve = e - 1;
      if (!wait_all(&bar->v_full[ve % VS], (ve / VS) & 1)) return false;
      if (pend) {
        if (!wait_all(&bar->p_full[s], pcount & 1)) return false;
        ++pcount;
        ptx::tc_fence_after();
        if (ptx::elect_one()) issue_pv<D>(o_tm, s_tm, v4 + (ve % VS) * tile4, !pend_first);
        __syncwarp();
        ptx::mma_commit_elect(&bar->o_full[s]);
      }
      ptx::mma_commit_elect(&bar->v_empty[ve % VS]);
      pend = open = false;
      return true;
    };
    for (int i = 0; ok; ++i) {
      const Item* it = take_item(p, bar, i, abort_flag);
      if (!it) {
        ok = false;
        break;
      }
      const int what = it->h;
      if (what < 0) {
        drop_item(bar, i);
        ok = finish();
        if (what == kEnd) break;
        continue;
      }
      const int n = it->n, lo = it->lo;
      const int first_use = it->first(s), last_use = it->last(s);
      const int has0 = it->first(0) >= 0, has1 = it->first(1) >= 0;
      drop_item(bar, i);
      if (n == 0) {
        // (no entry carries the last P V along, and the ring's slots wait for its output)
        ok = finish();
        continue;
      }
      const int tq = t + (s ? has0 : 0);  // this query tile's Q
      t += has0 + has1;
      const int qslot = tq % kQSlots;
      const uint32_t qpar = (tq / kQSlots) & 1;
      for (int j = 0; j < n; ++j, ++e) {
        const int kt = lo + j;
        const bool use = first_use >= 0 && kt >= first_use && kt <= last_use;
        const int ks = e % KS;
        const bool rel_v = open;
        const int ve = e - 1;
        if (rel_v && !wait_all(&bar->v_full[ve % VS], (ve / VS) & 1)) { ok = false; break; }
        if (!wait_all(&bar->k_full[ks], (e / KS) & 1)) { ok = false; break; }
        if (pend) {
          if (!wait_all(&bar->p_full[s], pcount & 1)) { ok = false; break; }
          ++pcount;
          ptx::tc_fence_after();
        }
        if (use && kt == first_use && !wait_all(&bar->q_full[qslot], qpar)) { ok = false; break; }
        const uint32_t ticket = (uint32_t)(2 * e + s);
        if (!__all_sync(0xffffffffu, mma_turn_wait(bar, ticket, p.timeout_ns, abort_flag))) { ok = false; break; }
        if (ptx::elect_one()) {
          if (pend) issue_pv<D>(o_tm, s_tm, v4 + (ve % VS) * tile4, !pend_first);
          if (use) issue_qk<D>(s_tm, q4 + qslot * tile4, k4 + ks * tile4);
        }
        __syncwarp();
        if (lane == 0) mma_turn_pass(bar, ticket);
        if (use) {
          ptx::mma_commit_elect(&bar->s_full[s]);
          issued_any = true;
        }
        if (rel_v) ptx::mma_commit_elect(&bar->v_empty[ve % VS]);
        ptx::mma_commit_elect(&bar->k_empty[ks]);
        if (pend && pend_last) ptx::mma_commit_elect(&bar->o_full[s]);
        if (use && kt == last_use) ptx::mma_commit_elect(&bar->q_empty[qslot]);
        open = true;
        pend = use;
        pend_first = use && kt == first_use;
        pend_last = use && kt == last_use;
      }
    }
    if (!ok) {
      if (lane == 0) fail(p, bar, kErrMma);
      if (issued_any) {
        // wait (bounded) for the MMAs already issued before tensor memory is freed
        ptx::mma_commit_elect(&bar->drain[s]);
        ptx::mbar_wait_time_only(&bar->drain[s], 0, p.timeout_ns);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    ptx::setmaxnreg_inc<kRegsSoftmax>();
    const int s = (warp - 4) >> 2;
    const int quarter = warp & 3;  // tensor-memory lane quarter this warp may access
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tmem = tmem + lane_off + s * 128;
    const uint32_t o_tmem = tmem + lane_off + 256 + s * 128;
    const float sl2 = p.scale_log2;
    uint32_t count = 0;  // S tiles of this query tile so far (all items)
    int o_items = 0;     // items whose O_s has been read
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Item* it = take_item(p, bar, i, abort_flag);
      if (!it) {
        ok = false;
        if (lane == 0) fail(p, bar, kErrSoftmax);
        break;
      }
      if (it->h == kEnd) break;
      if (it->h == kDrain) {
        drop_item(bar, i);
        continue;
      }
      const int keys = it->keys, h = it->h;
      const bool valid = row < it->rows - 128 * s;
      const int pos = it->pos0 + 128 * s + row;
      int lo = 0, hi = keys - 1;  // keys this row sees
      if (p.causal) {
        hi = min(hi, pos);
        if (p.window) lo = max(0, pos - p.window + 1);
      }
      if (!valid) hi = -1;
      const int first = it->first(s), last = it->last(s);
      int whole_lo, whole_hi;
      it->whole(p, s, &whole_lo, &whole_hi);
      float m = -INFINITY;  // running (stale) max of scaled scores, log2 domain
      float l = 0.f;        // running sum of exp2(x - m)
      float lr = 0.f;       // of these as P V takes them, where there are few
      const bool some_few = few_keys(p, p.causal ? min(keys - 1, pos - row) : keys - 1);  // (the first row sees least)
      for (int kt = first < 0 ? last + 1 : first; kt <= last; ++kt) {
        const bool got = ptx::mbar_wait(&bar->s_full[s], count & 1, p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) fail(p, bar, kErrSoftmax);
          ok = false;
          break;
        }
        ++count;
        ptx::tc_fence_after();
        bool sees = valid;  // this row sees a key of the tile
        if (kt < whole_lo || kt > whole_hi) {
          const int c_lo = max(lo - kt * kTile, 0), c_hi = min(hi - kt * kTile, 127);
          mask_scores(s_tmem, c_lo, c_hi);
          sees = c_lo <= c_hi;
        }
        float x[128];
        ptx::tmem_ld32(s_tmem + 0, *reinterpret_cast<float(*)[32]>(&x[0]));
        ptx::tmem_ld32(s_tmem + 32, *reinterpret_cast<float(*)[32]>(&x[32]));
        ptx::tmem_ld32(s_tmem + 64, *reinterpret_cast<float(*)[32]>(&x[64]));
        ptx::tmem_ld32(s_tmem + 96, *reinterpret_cast<float(*)[32]>(&x[96]));
        ptx::tmem_wait_ld();
        // P = exp2(s * scale * log2e - m) into tensor memory, by the stale-max rule of
        // attention_fwd.cu; rows past the sequence's end (another's, or nothing) take
        // no part in it
        const bool fresh = m == -INFINITY;
        float ts = exp_to_tmem(x, sl2, fresh ? 0.f : m, s_tmem);
        const bool redo = valid && (!(ts <= kMaxTileSum) || (fresh && sees && !(ts >= kMinTileSum)));
        if (fresh && sees && !redo) m = 0.f;  // the row's reference from here on
        if (__any_sync(0xffffffffu, redo)) {
          ptx::tmem_wait_st();  // let these stores land before they are overwritten
          // the warp's other rows keep their reference, and with it every bit
          const float m_new = redo ? fmaxf(m, row_max(x) * sl2) : m;
          const bool need_rescale = !fresh && m_new > m;
          if (fresh) m = m_new;
          if (__any_sync(0xffffffffu, need_rescale)) {
            const float alpha = need_rescale ? ptx::ex2(m - m_new) : 1.f;
            rescale_o<D>(o_tmem, alpha);
            if (need_rescale) {
              l *= alpha;
              lr *= alpha;
              m = m_new;
            }
          }
          ts = exp_to_tmem(x, sl2, (m == -INFINITY) ? 0.f : m, s_tmem);
        }
        l += ts;
        ptx::tmem_wait_st();
        if (some_few) lr += rounded_sum<64>(s_tmem);
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar->p_full[s]);
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue
      const bool has_o = first >= 0;
      const float b2 = p.sink ? __ldg(p.sink + h) * kLog2e : -INFINITY;
      const float M = fmaxf(m, b2);
      const float ref = M == -INFINITY ? 0.f : M;  // (no key and no sink: l = 0; scores that are NaN: l is)
      const float em = m == -INFINITY ? 1.f : ptx::ex2(m - ref);
      const float zs = b2 == -INFINITY ? 0.f : ptx::ex2(b2 - ref), z = l * em + zs;
      const float o_scale = z == 0.f ? 0.f : em / (few_keys(p, hi) ? lr * em + zs : z);
      const int64_t q_row = (int64_t)it->q_row + 128 * s + row;
      if (valid && p.lse) p.lse[(int64_t)h * p.T + q_row] = z == 0.f ? -INFINITY : (ref + ptx::lg2(z)) * kLn2;
      if (has_o) {
        const bool got = ptx::mbar_wait(&bar->o_full[s], o_items & 1, p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) fail(p, bar, kErrEpilogue);
          ok = false;
          break;
        }
        ++o_items;
        ptx::tc_fence_after();
      }
      // a row's output that is not finite may be a hidden key's values' doing (see above)
      const bool part = has_o && (first < whole_lo || last > whole_hi) && !it->again;
      float2 sum = make_float2(0.f, 0.f);
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + (q_row * p.H + h) * D;
      const uint64_t o_policy = ptx::l2_policy_evict_first();
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 16) {
        float ov[16];
        if (has_o) {
          ptx::tmem_ld16(o_tmem + c0, ov);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) ov[k] *= o_scale;
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) ov[k] = 0.f;
        }
        if (part) {  // (a sum is finite only if its terms are)
#pragma unroll
          for (int k = 0; k < 16; k += 2) sum = ptx::fadd2(sum, make_float2(ov[k], ov[k + 1]));
        }
        if (valid) {
          uint32_t pk[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) pk[k] = ptx::pack_bf16x2(ov[2 * k], ov[2 * k + 1]);
          if (p.wide) {
            st_global_32(dst + c0, pk, o_policy);
          } else {
            uint4* to = reinterpret_cast<uint4*>(dst + c0);
            ptx::st_global_v4_hint(to, make_uint4(pk[0], pk[1], pk[2], pk[3]), o_policy);
            ptx::st_global_v4_hint(to + 1, make_uint4(pk[4], pk[5], pk[6], pk[7]), o_policy);
          }
        }
      }
      if (__any_sync(0xffffffffu, part && valid && !(fabsf(sum.x + sum.y) < INFINITY)) && lane == 0 &&
          atomicExch(&const_cast<Item*>(it)->marked, 1) == 0)
        p.marked[it->id] = atomicExch(&bar->marked, it->id);
      drop_item(bar, i);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x < 256 && !*abort_flag) {
    for (int id = bar->marked; id >= 0; id = next_marked(p, id)) {
      Item it;
      it.set(p, bar->pair(p, id), id);
      add_odd_values<D>(p, it, threadIdx.x);
    }
  }
}

cudaError_t launch_plan(const PackedParams& p, cudaStream_t stream) {
  return launch_chained(packed_plan_kernel, 1, 1, kPlanThreads, 0, 1, p, stream);
}

template <int D>
cudaError_t launch_d(const PackedParams& p, cudaStream_t stream) {
  using G = Geo<D>;
  constexpr size_t need = (size_t)(kQSlots + 2 * G::kStages) * G::kTileBytes + sizeof(Bar) + 1024;
  // (at least half of an SM's shared memory: one CTA owns the SM and its tensor memory)
  constexpr size_t smem = need < 120 * 1024 ? 120 * 1024 : need;
  static_assert(smem <= 227 * 1024, "shared memory");
  auto kern = attention_packed_kernel<D>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kern, smem, &done);
  if (e != cudaSuccess) return e;
  if (!p.direct && (e = launch_plan(p, stream)) != cudaSuccess) return e;
  const int64_t items = (int64_t)p.max_pairs * p.H;
  return launch_chained(kern, (unsigned)(items < kPlanSms ? items : kPlanSms), 1, kThreads, smem, 1, p, stream);
}

}  // namespace

cudaError_t launch_attention_packed(const PackedParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_d<64>(p, stream);
    case 80: return launch_d<80>(p, stream);
    case 96: return launch_d<96>(p, stream);
    case 128: return launch_d<128>(p, stream);
    case 256: {
      const cudaError_t e = launch_plan(p, stream);
      return e == cudaSuccess ? launch_attention_packed_256(p, stream) : e;
    }
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mattn
