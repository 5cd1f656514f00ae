// attention_packed.cu's attention for heads of 256, for sm_103a, where two query tiles'
// accumulators would take all of tensor memory: one 128-row query tile at a time against
// key tiles of 128, S double-buffered,
//   S_g = Q K_g^T     M128 N128 K256, into S buffer g % 2
//   P_g = exp2(S_g scale log2e - m)    two threads a row, 64 keys each, P over its S
//   O  += P_g V_g     M128 N256 K128
//   issue order  S_0, S_1, [P_0] PV_0, S_2, [P_1] PV_1, S_3, ...
// 4 d FLOPs a visible (head, pair): bound by the tensor cores.  Tensor memory: S [0, 256),
// O [256, 512).  Shared memory: Q (64 KB) and rings of 16 KB pieces, five of K (64 columns
// of a tile) and five of V (32 rows of it), as two whole tiles of each do not fit.
//
// A CTA per SM takes items, the query tiles of packed_plan_kernel's pairs head by head,
// longest first, from a counter; copies run ahead into the next item, and its first scores are
// made while the last output is read.  What a row does not
// see is treated as there: items whose output hidden values may have spoilt are marked,
// and done again after the others.
//
// Roles (384 threads): warp 0 Q and K; warp 1 tensor memory and the products; warp 2 V;
// warp 3 the items; warps 4..11 softmax and output: warps w and w + 4 the same 32 rows, half
// of a tile's keys and of the output's columns each.  Every wait is bounded in time (the
// scheduler's: in time without a tile's progress) and gives up by raising a CTA-wide abort
// flag and a device error bit; the two warps of a pair, which meet at barriers, give up
// together.
//
// Measured (TFLOP/s of visible pairs): one causal sequence of 16,384, 8 heads, 700-725 us = 1,517-1,571,
// eight prompts of 1 to 3,352 tokens, 32 heads, 595-607 us = 1,251-1,277, 16 of 1,024 not causal
// 398-405 us = 1,357-1,381, 64 of 256 150-155 us = 444-459.  Key tiles of 64, as in attention_sp.cu, took 882 us for the
// first: a product of 64 columns takes as long as one of 128.  Items that begin when the last
// one is written took 677, 617, 444 and 191.  The next item's first scores before the last P V
// of this one gained nothing: they wait for its Q.
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

namespace mattn {
namespace {

constexpr int kD = 256;
constexpr int kThreads = 384;
constexpr int kItems = 3, kReaders = 11;  // of the ring; of an item: the warps but the scheduler's
constexpr int kPieces = 4, kRing = 5;  // pieces of a K or V tile; in each ring
constexpr int kQChunk = kTile * 128, kQBytes = kD / 64 * kQChunk;  // chunks of 64 columns, 128-byte swizzle
constexpr int kPiece = kQChunk;                                    // of K: such a chunk
constexpr int kVRows = kPackedValues256, kVChunk = kVRows * 128;   // of V: four chunks of 32 rows
static_assert(kVRows * kPieces == kTile && kVChunk * (kD / 64) == kPiece, "pieces");

// An item: a query tile of a pair, and its key tiles lo .. lo + n - 1; or (h < 0) the word to
// finish what is under way, after which there is nothing more (kEnd) or may be (kDrain).
constexpr int kDrain = -2, kEnd = -1;
struct Item {
  int q_row, rows, k_row, keys, pos, h, id;
  int lo, n;
  int whole_lo, whole_hi;  // the key tiles that every row sees whole
  int marked;              // some row of its output is not finite
  int again;               // the second time
  __device__ __forceinline__ void set(const PackedParams& p, int item) {
    const int pair = item / (2 * p.H), i = item - pair * 2 * p.H;
    const int s = i < p.H ? 1 : 0;  // (the second query tile, which sees most keys, first)
    const PackedPair& x = p.plan->pair[pair];
    q_row = x.q_row + 128 * s;
    rows = in_bounds(p, x) ? min(x.rows - 128 * s, 128) : 0;
    k_row = x.k_row;
    keys = x.keys;
    pos = x.pos0 + 128 * s;
    h = i < p.H ? i : i - p.H;
    id = item;
    int hi;
    seen_tiles<7>(p, pos, rows, keys, &lo, &hi);
    n = hi < lo ? 0 : hi - lo + 1;
    whole_hi = ((p.causal ? min(keys, pos + 1) : keys) >> 7) - 1;
    whole_lo = p.window ? (max(0, pos + rows - p.window) + 127) >> 7 : 0;
    marked = 0;
  }
  __device__ __forceinline__ void say(int what) {
    h = what;
    n = 0;
  }
  __device__ __forceinline__ bool partial(int kt) const { return kt < whole_lo || kt > whole_hi; }
};

struct Bar {
  uint64_t q_full, q_empty;
  uint64_t k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing];
  uint64_t v_land;
  uint64_t s_full[2], p_full[2];
  uint64_t pv_done;          // one phase per P V product
  uint64_t o_full, o_empty;  // one per item with keys: after its last product, once its output is read
  uint64_t drain;
  uint64_t item_full[kItems], item_empty[kItems];
  uint32_t tmem_base;
  int abort_flag;
  int marked;                // the CTA's last marked item, from which PackedParams::marked leads to the others; -1: none
  uint32_t tiles;            // K tiles whose copies are under way, of all items
  Item items[kItems];
  uint32_t redo[2][4];       // rows of each half and 32 rows whose tile is done again
  float half[2][kTile];      // a row's maximum over half a tile, at last half its sum
};

__device__ __forceinline__ uint64_t dsc(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

__device__ __forceinline__ void fail(const PackedParams& p, Bar* bar, uint32_t bit) {
  *reinterpret_cast<volatile int*>(&bar->abort_flag) = 1;
  atomicOr(p.err, bit);
}

// The scheduler's wait for a ring slot.
__device__ __forceinline__ bool slot_wait(const PackedParams& p, Bar* bar, uint64_t* b, uint32_t parity,
                                          volatile int* abort_flag) {
  return item_wait(&bar->tiles, abort_flag,
                   [&] { return ptx::mbar_wait_backoff(b, parity, p.timeout_ns, abort_flag, 200); });
}

// The items, in order (one thread).
__device__ __forceinline__ void schedule(const PackedParams& p, Bar* bar, volatile int* abort_flag) {
  const int total = p.plan->pairs * 2 * p.H;
  int id = blockIdx.x;
  for (int i = 0, again = 0;; ++i) {
    const int slot = i % kItems;
    const uint32_t phase = (i / kItems) & 1;
    if (!slot_wait(p, bar, &bar->item_empty[slot], phase ^ 1, abort_flag)) break;
    Item& it = bar->items[slot];
    if (!again) {
      for (; id < total; id = (int)gridDim.x + atomicAdd(&p.plan->next, 1)) {
        it.set(p, id);
        if (it.rows > 0) break;
      }
      it.again = 0;
      if (id < total) {
        ptx::mbar_arrive(&bar->item_full[slot]);
        id = (int)gridDim.x + atomicAdd(&p.plan->next, 1);
        continue;
      }
      // every item so far written: then the marked ones
      it.say(kDrain);
      ptx::mbar_arrive(&bar->item_full[slot]);
      if (!slot_wait(p, bar, &bar->item_empty[slot], phase, abort_flag)) break;
      again = 1;
      id = *reinterpret_cast<volatile int*>(&bar->marked);
      continue;
    }
    if (id < 0 || id >= p.max_pairs * 2 * p.H) {
      it.say(kEnd);
      ptx::mbar_arrive(&bar->item_full[slot]);
      return;
    }
    it.set(p, id);
    it.again = 1;
    ptx::mbar_arrive(&bar->item_full[slot]);
    id = p.marked[id];
  }
  fail(p, bar, kErrProducer);
}

// Waits for the CTA's item i (a warp); null if the wait gave up.
__device__ __forceinline__ const Item* take_item(const PackedParams& p, Bar* bar, int i, volatile int* abort_flag) {
  const bool got = ptx::mbar_wait(&bar->item_full[i % kItems], (i / kItems) & 1, p.timeout_ns, abort_flag);
  return __all_sync(0xffffffffu, got) ? &bar->items[i % kItems] : nullptr;
}
__device__ __forceinline__ void drop_item(Bar* bar, int i) {  // (one warp, after its last read)
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&bar->item_empty[i % kItems]);
}

// A landed piece of V: rows from `rows` on and values that are not finite become zeros (one warp).
__device__ __forceinline__ void clean_piece(uint8_t* piece, int rows) {
  const int lane = threadIdx.x & 31;
  for (int c = 0; c < kD / 64; ++c) {
    uint4* x = reinterpret_cast<uint4*>(piece + c * kVChunk);
    for (int i = lane; i < kVChunk / 16; i += 32) {
      const uint4 v = x[i];
      x[i] = i < rows * 8 ? make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w)) : make_uint4(0, 0, 0, 0);
    }
  }
  ptx::fence_proxy_async_shared();
  __syncwarp();
}

// A barrier of the two warps of 32 rows; whether x holds in any of their threads.
__device__ __forceinline__ bool pair_any(int quarter, bool x) {
  int r;
  asm volatile(
      "{\n.reg .pred a, b;\nsetp.ne.s32 a, %1, 0;\nbarrier.cta.red.or.pred b, %2, 64, a;\nselp.s32 %0, 1, 0, b;\n}"
      : "=r"(r)
      : "r"((int)x), "r"(1 + quarter)
      : "memory");
  return r;
}

// The values that clean_piece took out, added to the output of the row (a thread's, half of
// the columns from `col` on) that sees them.
__device__ __forceinline__ void add_odd_values(const PackedParams& p, const Item& it, int row, int col, int lo, int hi) {
  if (row >= it.rows) return;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.o) + (((int64_t)it.q_row + row) * p.H + it.h) * kD;
  for (int kt = it.lo; kt < it.lo + it.n; ++kt) {
    if (!it.partial(kt)) continue;
    for (int j = max(lo, kt * kTile); j <= min(hi, kt * kTile + kTile - 1); ++j) {
      const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.v) + (it.k_row + (int64_t)j) * p.v_token +
                               (it.h / p.group) * p.v_head;
#pragma unroll 4
      for (int c = col; c < col + kD / 2; c += 2) {
        const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(v + c)), odd = x ^ clean(x);
        if (!odd) continue;
        __nv_bfloat162* to = reinterpret_cast<__nv_bfloat162*>(o + c);
        const float2 y = __bfloat1622float2(*to);
        *to = __floats2bfloat162_rn(y.x + __uint_as_float(odd << 16), y.y + __uint_as_float(odd & 0xffff0000u));
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) attention_packed_256_kernel(const __grid_constant__ PackedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = base;
  uint8_t* sk = sq + kQBytes;
  uint8_t* sv = sk + kRing * kPiece;
  Bar* bar = reinterpret_cast<Bar*>(sv + kRing * kPiece);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&p.tq[0]);
    ptx::prefetch_tmap(&p.tk[0]);
    ptx::prefetch_tmap(&p.tv);
    ptx::mbar_init(&bar->q_full, 1);
    ptx::mbar_init(&bar->q_empty, 1);
    for (int i = 0; i < kRing; ++i) {
      ptx::mbar_init(&bar->k_full[i], 1);
      ptx::mbar_init(&bar->k_empty[i], 1);
      ptx::mbar_init(&bar->v_full[i], 1);
      ptx::mbar_init(&bar->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bar->s_full[i], 1);
      ptx::mbar_init(&bar->p_full[i], 2 * kTile);
    }
    ptx::mbar_init(&bar->pv_done, 1);
    ptx::mbar_init(&bar->v_land, 1);
    ptx::mbar_init(&bar->o_full, 1);
    ptx::mbar_init(&bar->o_empty, 8);
    for (int i = 0; i < kItems; ++i) {
      ptx::mbar_init(&bar->item_full[i], 1);
      ptx::mbar_init(&bar->item_empty[i], kReaders);
    }
    ptx::mbar_init(&bar->drain, 1);
    bar->abort_flag = 0;
    bar->marked = -1;
    bar->tiles = 0;
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

  if (warp == 3) {
    if (lane == 0) schedule(p, bar, abort_flag);
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------ Q and K
    const uint64_t keep = ptx::l2_policy_evict_last(), once = ptx::l2_policy_evict_first();
    auto wait_all = [&](uint64_t* b, uint32_t parity) {
      return __all_sync(0xffffffffu, ptx::mbar_wait(b, parity, p.timeout_ns, abort_flag));
    };
    bool ok = true;
    uint32_t g = 0, tiles = 0;  // pieces of K, Q tiles
    for (int i = 0; ok; ++i) {
      const Item* it = take_item(p, bar, i, abort_flag);
      if (!it) {
        ok = false;
        break;
      }
      const int n = it->n, h = it->h, q_row = it->q_row, k_row = it->k_row + it->lo * kTile;
      drop_item(bar, i);
      if (h == kEnd) break;
      if (n == 0) continue;  // (kDrain too)
      const int h_kv = h / p.group;
      ok = debug_check(p.err, q_row >= 0 && q_row < p.T && h < p.H, kSiteLoad) && wait_all(&bar->q_empty, (tiles & 1) ^ 1);
      ++tiles;
      if (ok && lane == 0) {
        ptx::mbar_arrive_expect_tx(&bar->q_full, kQBytes);
#pragma unroll
        for (int c = 0; c < kD / 64; ++c)
          ptx::tma_load_3d_hint(sq + c * kQChunk, &p.tq[0], &bar->q_full, c * 64, h, q_row, once);
      }
      __syncwarp();
      for (int t = 0; ok && t < n; ++t) {
        const int row = k_row + t * kTile;
        ok = debug_check(p.err, row >= 0 && row < p.T_k, kSiteLoad);
        for (int c = 0; ok && c < kPieces; ++c, ++g) {
          const uint32_t slot = g % kRing;
          if (!wait_all(&bar->k_empty[slot], ((g / kRing) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (c == 0) *reinterpret_cast<volatile uint32_t*>(&bar->tiles) = g / kPieces + 1;
            ptx::mbar_arrive_expect_tx(&bar->k_full[slot], kPiece);
            if (!(p.selftest == 1 && g == 0))
              ptx::tma_load_3d_hint(sk + slot * kPiece, &p.tk[0], &bar->k_full[slot], c * 64, h_kv, row, keep);
          }
          __syncwarp();
        }
      }
    }
    if (!ok && lane == 0) fail(p, bar, kErrProducer);
    __syncwarp();
    let_copies_land(abort_flag);
  } else if (warp == 2) {
    // ------------------------------------------------------------ V
    const uint64_t keep = ptx::l2_policy_evict_last();
    bool ok = true;
    uint32_t g = 0, lands = 0;  // pieces, those looked over
    for (int i = 0; ok; ++i) {
      const Item* ring = take_item(p, bar, i, abort_flag);
      if (!ring) {
        ok = false;
        break;
      }
      const Item it = *ring;
      drop_item(bar, i);
      if (it.h == kEnd) break;
      const int h_kv = it.h / p.group;
      for (int t = 0; ok && t < it.n; ++t) {
        const int kt = it.lo + t, row = it.k_row + kt * kTile;
        ok = debug_check(p.err, row >= 0 && row < p.T_k, kSiteLoad);
        const bool look = it.again && it.partial(kt);
        for (int c = 0; ok && c < kPieces; ++c, ++g) {
          const uint32_t slot = g % kRing;
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->v_empty[slot], ((g / kRing) & 1) ^ 1, p.timeout_ns, abort_flag))) {
            ok = false;
            break;
          }
          uint8_t* piece = sv + slot * kPiece;
          uint64_t* landing = look ? &bar->v_land : &bar->v_full[slot];
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(landing, kPiece);
#pragma unroll
            for (int j = 0; j < kD / 64; ++j)
              ptx::tma_load_3d_hint(piece + j * kVChunk, &p.tv, landing, j * 64, h_kv, row + c * kVRows, keep);
          }
          __syncwarp();
          if (look) {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->v_land, lands & 1, p.timeout_ns, abort_flag))) {
              ok = false;
              break;
            }
            ++lands;
            clean_piece(piece, max(min(it.keys - kt * kTile - c * kVRows, kVRows), 0));
            if (lane == 0) ptx::mbar_arrive(&bar->v_full[slot]);
          }
        }
      }
    }
    if (!ok && lane == 0) fail(p, bar, kErrProducer);
    __syncwarp();
    let_copies_land(abort_flag);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    auto wait_all = [&](uint64_t* b, uint32_t parity) {
      return __all_sync(0xffffffffu, ptx::mbar_wait(b, parity, p.timeout_ns, abort_flag));
    };
    const uint32_t q4 = ptx::smem_addr(sq) >> 4;
    const uint32_t k4 = ptx::smem_addr(sk) >> 4;
    const uint32_t v4 = ptx::smem_addr(sv) >> 4;
    constexpr uint32_t hi128 = ptx::smem_desc_hi(1024, ptx::kSw128);
    constexpr uint32_t lbo_k = 1u << 16;  // unused for swizzled K-major operands
    constexpr uint32_t lbo_v = (uint32_t)(kVChunk >> 4) << 16;  // V's atoms of 64 columns lie a chunk apart
    constexpr uint32_t idesc_qk = ptx::idesc_bf16(128, kTile, 0);
    constexpr uint32_t idesc_pv = ptx::idesc_bf16(128, kD, 1);
    bool ok = true, issued = false;
    uint32_t e = 0, passes = 0;  // tiles, items with keys before the current one
    auto issue_s = [&](uint32_t g) {  // S = Q K^T, piece after piece as they land
      for (int c = 0; c < kPieces; ++c) {
        const uint32_t piece = g * kPieces + c, slot = piece % kRing;
        if (!wait_all(&bar->k_full[slot], (piece / kRing) & 1)) return false;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t qo = (uint32_t)((c * kQChunk + k * 32) >> 4) + lbo_k;
            const uint32_t ko = (uint32_t)((slot * kPiece + k * 32) >> 4) + lbo_k;
            ptx::mma_ss(tmem + (g & 1) * kTile, dsc(q4 + qo, hi128), dsc(k4 + ko, hi128), idesc_qk, (c > 0 || k > 0) ? 1u : 0u);
          }
        }
        __syncwarp();
        ptx::mma_commit_elect(&bar->k_empty[slot]);
        issued = true;
      }
      ptx::mma_commit_elect(&bar->s_full[g & 1]);
      return true;
    };
    for (int i = 0; ok; ++i) {
      const Item* it = take_item(p, bar, i, abort_flag);
      if (!it) {
        ok = false;
        break;
      }
      const int h = it->h, n = it->n;
      drop_item(bar, i);
      if (h == kEnd) break;
      if (n == 0) continue;  // (kDrain too)
      ok = wait_all(&bar->q_full, passes & 1);
      for (int t = 0; ok && t < 2 && t < n; ++t) ok = issue_s(e + t);
      if (ok && n <= 2) ptx::mma_commit_elect(&bar->q_empty);
      // the last item's output read: O may be overwritten
      ok = ok && wait_all(&bar->o_empty, (passes & 1) ^ 1);
      for (int t = 0; ok && t < n; ++t, ++e) {
        // P there: O += P V, piece after piece, then the next scores over P
        const int sb = e & 1;
        ok = wait_all(&bar->p_full[sb], (e >> 1) & 1);
        for (int c = 0; ok && c < kPieces; ++c) {
          const uint32_t g = e * kPieces + c, slot = g % kRing;
          if (!wait_all(&bar->v_full[slot], (g / kRing) & 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
#pragma unroll
            for (int k = 0; k < kVRows / 16; ++k) {
              // 16 keys: 8 tensor-memory columns of P, those of a half 64 on, 16 rows (2 KB) of V
              const int step = c * (kVRows / 16) + k;
              const uint32_t vo = (uint32_t)((slot * kPiece + k * 16 * 128) >> 4) + lbo_v;
              ptx::mma_ts(tmem + 256, tmem + sb * kTile + (step >> 2) * 64 + (step & 3) * 8, dsc(v4 + vo, hi128), idesc_pv,
                          (t > 0 || step > 0) ? 1u : 0u);
            }
          }
          __syncwarp();
          ptx::mma_commit_elect(&bar->v_empty[slot]);
        }
        if (!ok) break;
        ptx::mma_commit_elect(&bar->pv_done);
        if (t + 2 < n) {
          ok = issue_s(e + 2);
          if (ok && t + 3 == n) ptx::mma_commit_elect(&bar->q_empty);  // the item's last
        }
      }
      if (ok) ptx::mma_commit_elect(&bar->o_full);
      ++passes;
    }
    if (!ok) {
      if (lane == 0) fail(p, bar, kErrMma);
      if (issued) {
        // wait (bounded) for the MMAs already issued before tensor memory is freed
        ptx::mma_commit_elect(&bar->drain);
        ptx::mbar_wait_time_only(&bar->drain, 0, p.timeout_ns);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    const int half = (warp - 4) >> 2;
    const int quarter = warp & 3;  // tensor-memory lane quarter this warp may access
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + 256;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int e = 0;            // tiles before the item's
    uint32_t passes = 0;  // items with keys before it
    for (int i = 0;; ++i) {
      const Item* ring = take_item(p, bar, i, abort_flag);
      if (pair_any(quarter, !ring)) {
        ok = false;
        break;
      }
      const Item it = *ring;
      if (it.h < 0) {
        drop_item(bar, i);
        if (it.h == kEnd) break;
        continue;
      }
      const int n = it.n;
      const bool again = it.again;
      const bool valid = row < it.rows;
      int lo = 0, hi = it.keys - 1;  // keys this row sees
      if (p.causal) {
        hi = min(hi, it.pos + row);
        if (p.window) lo = max(0, it.pos + row - p.window + 1);
      }
      if (!valid) hi = -1;
      float m = -INFINITY;  // running (stale) max of scaled scores, log2 domain; both halves have the same
      float l = 0.f;        // running sum of exp2(x - m) of this half's keys
      float lr = 0.f;       // of these as P V takes them, where there are few
      const bool some_few = few_keys(p, p.causal ? min(it.keys - 1, it.pos) : it.keys - 1);  // (the first row sees least)
      for (int t = 0; t < n; ++t) {
        const int g = e + t, sb = g & 1, kt = it.lo + t;
        const uint32_t s_tmem = tmem + lane_off + sb * kTile + half * 64;
        const bool got = ptx::mbar_wait(&bar->s_full[sb], (g >> 1) & 1, p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, got)) ok = false;  // (and on to the barrier that the other warp may be at)
        ptx::tc_fence_after();
        float x[64];
        bool sees = valid, sees_half = valid;  // this row sees a key of the tile, of this half
        float ts = 0.f;
        if (ok) {
          ptx::tmem_ld32(s_tmem, *reinterpret_cast<float(*)[32]>(&x[0]));
          ptx::tmem_ld32(s_tmem + 32, *reinterpret_cast<float(*)[32]>(&x[32]));
          ptx::tmem_wait_ld();
          if (it.partial(kt)) {
            const int c_lo = max(lo - kt * kTile, 0), c_hi = min(hi - kt * kTile, kTile - 1);
            sees = c_lo <= c_hi;
            sees_half = max(c_lo, 64 * half) <= min(c_hi, 64 * half + 63);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t vis = range_bits(2 * half + j, c_lo, c_hi);
#pragma unroll
              for (int k = 0; k < 32; ++k) x[32 * j + k] = ((vis >> k) & 1u) ? x[32 * j + k] : -INFINITY;
            }
          }
          ts = exp_to_tmem(x, sl2, m == -INFINITY ? 0.f : m, s_tmem);
        }
        // (the stale-max rule, for half a tile each, and rows that keep their reference while
        // another's is redone, as in attention_packed.cu)
        const bool fresh = m == -INFINITY;
        const bool mine = valid && (!(ts <= kMaxTileSum) || (fresh && sees_half && !(ts >= kMinTileSum)));
        const bool slow = pair_any(quarter, mine || !ok);
        if (!slow) {
          if (fresh && sees) m = 0.f;  // the row's reference from here on
        } else {
          if (ok) ptx::tmem_wait_st();  // let these stores land before they are overwritten
          const uint32_t rows = __ballot_sync(0xffffffffu, mine);
          bar->half[half][row] = ok ? row_max(x) : 0.f;
          if (lane == 0) bar->redo[half][quarter] = rows;
          if (pair_any(quarter, !ok)) {
            ok = false;
            break;
          }
          const bool redo = ((rows | bar->redo[half ^ 1][quarter]) >> lane) & 1u;
          const float m_new = redo ? fmaxf(m, fmaxf(bar->half[0][row], bar->half[1][row]) * sl2) : (fresh && sees ? 0.f : m);
          const bool need_rescale = !fresh && m_new > m;
          if (fresh) m = m_new;
          if (__any_sync(0xffffffffu, need_rescale)) {
            // the last product adds into O: wait for it (S_t there means that the one before
            // it is done, so the barrier is one phase behind at most)
            const bool pv = ptx::mbar_wait(&bar->pv_done, (g - 1) & 1, p.timeout_ns, abort_flag);
            ok = __all_sync(0xffffffffu, pv);
            ptx::tc_fence_after();
            if (ok) rescale_o<kD>(o_tmem, need_rescale ? ptx::ex2(m - m_new) : 1.f, half * (kD / 2), (half + 1) * (kD / 2));
            if (need_rescale) {
              l *= ptx::ex2(m - m_new);
              lr *= ptx::ex2(m - m_new);
              m = m_new;
            }
          }
          if (ok) ts = exp_to_tmem(x, sl2, (m == -INFINITY) ? 0.f : m, s_tmem);
          if (pair_any(quarter, !ok)) {  // (and the maxima are read)
            ok = false;
            break;
          }
        }
        l += ts;
        ptx::tmem_wait_st();
        if (some_few) lr += rounded_sum<32>(s_tmem);
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar->p_full[sb]);
      }
      if (!ok) break;
      if (n > 0) {
        const bool got = ptx::mbar_wait(&bar->o_full, passes & 1, p.timeout_ns, abort_flag);
        ok = __all_sync(0xffffffffu, got);
        ++passes;
        ptx::tc_fence_after();
        bar->half[half][row] = l;
        if (pair_any(quarter, !ok)) {
          ok = false;
          break;
        }
        l = bar->half[0][row] + bar->half[1][row];
        if (some_few) {
          pair_any(quarter, false);  // (l is read)
          bar->half[half][row] = lr;
          pair_any(quarter, false);
          lr = bar->half[0][row] + bar->half[1][row];
        }
      }
      e += n;
      const float b2 = p.sink ? __ldg(p.sink + it.h) * kLog2e : -INFINITY;
      const float M = fmaxf(m, b2);
      const float ref = M == -INFINITY ? 0.f : M;  // (no key and no sink: l = 0; scores that are NaN: l is)
      const float em = m == -INFINITY ? 1.f : ptx::ex2(m - ref);
      const float zs = b2 == -INFINITY ? 0.f : ptx::ex2(b2 - ref), z = l * em + zs;
      const float o_scale = z == 0.f ? 0.f : em / (few_keys(p, hi) ? lr * em + zs : z);
      const int64_t q_row = (int64_t)it.q_row + row;
      if (valid && p.lse && half == 0) p.lse[(int64_t)it.h * p.T + q_row] = z == 0.f ? -INFINITY : (ref + ptx::lg2(z)) * kLn2;
      // a row's output that is not finite may be a hidden key's values' doing
      const bool part = n > 0 && (it.partial(it.lo) || it.partial(it.lo + n - 1)) && !again;
      float2 sum = make_float2(0.f, 0.f);
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + (q_row * p.H + it.h) * kD;
      const uint64_t o_policy = ptx::l2_policy_evict_first();
#pragma unroll 1
      for (int c0 = half * (kD / 2); c0 < (half + 1) * (kD / 2); c0 += 16) {
        float ov[16];
        if (n > 0) {
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
      if (n > 0) {  // O is read: the next item's first product may overwrite it
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar->o_empty);
      }
      if (__any_sync(0xffffffffu, part && valid && !(fabsf(sum.x + sum.y) < INFINITY)) && lane == 0 &&
          atomicExch(&const_cast<Item*>(ring)->marked, 1) == 0)
        p.marked[it.id] = atomicExch(&bar->marked, it.id);
      if (again) add_odd_values(p, it, row, half * (kD / 2), lo, hi);
      drop_item(bar, i);
    }
    if (!ok && lane == 0) fail(p, bar, kErrSoftmax);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_attention_packed_256(const PackedParams& p, cudaStream_t stream) {
  constexpr size_t smem = 1024 + kQBytes + 2 * kRing * kPiece + sizeof(Bar);
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(attention_packed_256_kernel, smem, &done);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.max_pairs * 2 * p.H;
  return launch_chained(attention_packed_256_kernel, (unsigned)(items < kPlanSms ? items : kPlanSms), 1, kThreads, smem, 1, p,
                        stream);
}

}  // namespace mattn
