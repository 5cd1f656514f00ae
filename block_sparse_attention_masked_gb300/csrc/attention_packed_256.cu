// attention_packed.cu's attention for heads of 256, for sm_103a, where two query tiles'
// accumulators would take all of tensor memory: one 128-row query tile at a time against
// key tiles of 64, S double-buffered, as attention_sp.cu has it:
//   S_t = Q K_t^T     M128 N64 K256, into S buffer t % 2
//   P_t = exp2(S_t scale log2e - m)    one row a thread, P over its S
//   O  += P_t V_t     M128 N256 K64
//   issue order  S_0, S_1, [P_0] PV_0, S_2, [P_1] PV_1, S_3, ...
// 4 d FLOPs a visible (head, pair): bound by the tensor cores.  Tensor memory: S_0 [0, 64),
// S_1 [64, 128), O [256, 512).  Shared memory: Q (64 KB), rings of two K and two V tiles
// (32 KB each).
//
// A CTA per SM takes items, the query tiles of packed_plan_kernel's pairs head by head,
// longest first, from a counter, one after another: an item begins when the last one is
// written.  What a row does not see is treated as there, but that an item whose output
// may have been spoilt by hidden values is done again at once.
//
// Roles (256 threads): warp 0 the items and the TMA copies; warp 1 tensor memory and the
// products; warps 4..7 softmax and output.  Every wait is bounded in time and gives up by
// raising a CTA-wide abort flag and a device error bit.
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

constexpr int kD = 256, kKT = kPackedKeys256;
static_assert(kKT == 64, "a key tile's scores are two groups of 32 columns");
constexpr int kThreads = 256, kStages = 2;
constexpr int kQChunk = kTile * 128, kQBytes = kD / 64 * kQChunk;  // chunks of 64 columns, 128-byte swizzle
constexpr int kKVChunk = kKT * 128, kKVBytes = kD / 64 * kKVChunk;

// An item: a query tile of a pair, and its key tiles lo .. lo + n - 1.
struct Item {
  int q_row, rows, k_row, keys, pos, h;  // h < 0: there are no more
  int lo, n;
  int whole_lo, whole_hi;  // the key tiles that every row sees whole
  __device__ __forceinline__ void set(const PackedParams& p, const PackedPair& x, int s, int head) {
    q_row = x.q_row + 128 * s;
    rows = in_bounds(p, x) ? min(x.rows - 128 * s, 128) : 0;
    k_row = x.k_row;
    keys = x.keys;
    pos = x.pos0 + 128 * s;
    h = head;
    int hi;
    seen_tiles<6>(p, pos, rows, keys, &lo, &hi);
    n = hi < lo ? 0 : hi - lo + 1;
    whole_hi = ((p.causal ? min(keys, pos + 1) : keys) >> 6) - 1;
    whole_lo = p.window ? (max(0, pos + rows - p.window) + 63) >> 6 : 0;
  }
  __device__ __forceinline__ bool partial(int kt) const { return kt < whole_lo || kt > whole_hi; }
};

struct Bar {
  uint64_t q_full;
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t v_land;
  uint64_t s_full[2], p_full[2];
  uint64_t pv_done;  // one phase per P V product
  uint64_t o_full;   // one per item with keys, after its last
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int marked[3];     // of item i in [i % 3]: some row of its output is not finite
  Item items[2];
};

__device__ __forceinline__ uint64_t dsc(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

__device__ __forceinline__ void fail(const PackedParams& p, Bar* bar, uint32_t bit) {
  *reinterpret_cast<volatile int*>(&bar->abort_flag) = 1;
  atomicOr(p.err, bit);
}

// The next item from number `id` on that has rows (one thread).  The heads of a pair run
// side by side, its second query tile, which sees most keys, first.
__device__ __forceinline__ void next_item(const PackedParams& p, int64_t total, int64_t id, Item* it) {
  for (;; id = (int64_t)gridDim.x + atomicAdd(&p.plan->next, 1)) {
    if (id >= total) {
      it->h = -1;
      return;
    }
    const int pair = (int)(id / (2 * p.H)), i = (int)(id - (int64_t)pair * 2 * p.H);
    it->set(p, p.plan->pair[pair], i < p.H ? 1 : 0, i < p.H ? i : i - p.H);
    if (it->rows > 0) return;
  }
}

// A landed V tile: rows from `rows` on and values that are not finite become zeros (one warp).
__device__ __forceinline__ void clean_tile(uint8_t* tile, int rows) {
  const int lane = threadIdx.x & 31;
  for (int c = 0; c < kD / 64; ++c) {
    uint4* x = reinterpret_cast<uint4*>(tile + c * kKVChunk);
    for (int i = lane; i < kKVChunk / 16; i += 32) {
      const uint4 v = x[i];
      x[i] = i < rows * 8 ? make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w)) : make_uint4(0, 0, 0, 0);
    }
  }
  ptx::fence_proxy_async_shared();
  __syncwarp();
}

// The values that clean_tile took out, added to the output of the row (a thread's) that
// sees them.
__device__ __forceinline__ void add_odd_values(const PackedParams& p, const Item& it, int row, int lo, int hi) {
  if (row >= it.rows) return;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.o) + (((int64_t)it.q_row + row) * p.H + it.h) * kD;
  for (int kt = it.lo; kt < it.lo + it.n; ++kt) {
    if (!it.partial(kt)) continue;
    for (int j = max(lo, kt * kKT); j <= min(hi, kt * kKT + kKT - 1); ++j) {
      const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.v) + (it.k_row + (int64_t)j) * p.v_token +
                               (it.h / p.group) * p.v_head;
#pragma unroll 4
      for (int c = 0; c < kD; c += 2) {
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
  uint8_t* sv = sk + kStages * kKVBytes;
  Bar* bar = reinterpret_cast<Bar*>(sv + kStages * kKVBytes);
  volatile int* abort_flag = &bar->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&p.tq[0]);
    ptx::prefetch_tmap(&p.tk[0]);
    ptx::prefetch_tmap(&p.tv);
    ptx::mbar_init(&bar->q_full, 1);
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&bar->k_full[i], 1);
      ptx::mbar_init(&bar->k_empty[i], 1);
      ptx::mbar_init(&bar->v_full[i], 1);
      ptx::mbar_init(&bar->v_empty[i], 1);
      ptx::mbar_init(&bar->s_full[i], 1);
      ptx::mbar_init(&bar->p_full[i], kTile);
    }
    ptx::mbar_init(&bar->v_land, 1);
    ptx::mbar_init(&bar->pv_done, 1);
    ptx::mbar_init(&bar->o_full, 1);
    ptx::mbar_init(&bar->drain, 1);
    bar->abort_flag = 0;
    bar->marked[0] = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&bar->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  after_previous();  // the plan, and whatever the inputs come from
  int64_t total = 0;
  if (threadIdx.x == 0) {
    total = (int64_t)p.plan->pairs * 2 * p.H;
    next_item(p, total, blockIdx.x, &bar->items[0]);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bar->tmem_base;

  int e = 0;           // key tiles before the current item's
  int passes = 0;      // Q tiles and outputs, likewise
  uint32_t lands = 0;  // V tiles looked over
  for (int i = 0, again = 0;;) {
    const Item it = bar->items[i & 1];
    if (it.h < 0) break;
    const int n = it.n;
    if (warp == 0) {
      // ---------------------------------------------------------- items and copies
      const uint64_t keep = ptx::l2_policy_evict_last(), once = ptx::l2_policy_evict_first();
      const int h_kv = it.h / p.group;
      bool ok = true;
      if (n > 0 && lane == 0) {
        ptx::mbar_arrive_expect_tx(&bar->q_full, kQBytes);
        if (debug_check(p.err, it.q_row >= 0 && it.q_row < p.T && it.h < p.H, kSiteLoad)) {
#pragma unroll
          for (int c = 0; c < kD / 64; ++c)
            ptx::tma_load_3d_hint(sq + c * kQChunk, &p.tq[0], &bar->q_full, c * 64, it.h, it.q_row, once);
        }
      }
      for (int t = 0; t < n; ++t) {
        const int slot = (e + t) % kStages, kt = it.lo + t, row = it.k_row + kt * kKT;
        const uint32_t par = (((e + t) / kStages) & 1) ^ 1;
        if (!debug_check(p.err, row >= 0 && row < p.T_k, kSiteLoad) ||
            !__all_sync(0xffffffffu, ptx::mbar_wait(&bar->k_empty[slot], par, p.timeout_ns, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&bar->k_full[slot], kKVBytes);
          if (!(p.selftest == 1 && e + t == 0)) {
#pragma unroll
            for (int c = 0; c < kD / 64; ++c)
              ptx::tma_load_3d_hint(sk + slot * kKVBytes + c * kKVChunk, &p.tk[0], &bar->k_full[slot], c * 64, h_kv, row, keep);
          }
        }
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->v_empty[slot], par, p.timeout_ns, abort_flag))) {
          ok = false;
          break;
        }
        const bool look = again && it.partial(kt);
        uint8_t* tile = sv + slot * kKVBytes;
        uint64_t* landing = look ? &bar->v_land : &bar->v_full[slot];
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(landing, kKVBytes);
#pragma unroll
          for (int c = 0; c < kD / 64; ++c)
            ptx::tma_load_3d_hint(tile + c * kKVChunk, &p.tv, landing, c * 64, h_kv, row, keep);
        }
        __syncwarp();
        if (look) {
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bar->v_land, lands & 1, p.timeout_ns, abort_flag))) {
            ok = false;
            break;
          }
          ++lands;
          clean_tile(tile, min(it.keys - kt * kKT, kKT));
          if (lane == 0) ptx::mbar_arrive(&bar->v_full[slot]);
        }
      }
      if (!ok && lane == 0) fail(p, bar, kErrProducer);
      if (lane == 0 && !again) {
        next_item(p, total, (int64_t)gridDim.x + atomicAdd(&p.plan->next, 1), &bar->items[(i + 1) & 1]);
        bar->marked[(i + 1) % 3] = 0;
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- products
      auto wait_all = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(0xffffffffu, ptx::mbar_wait(b, parity, p.timeout_ns, abort_flag));
      };
      const uint32_t q4 = ptx::smem_addr(sq) >> 4;
      const uint32_t k4 = ptx::smem_addr(sk) >> 4;
      const uint32_t v4 = ptx::smem_addr(sv) >> 4;
      constexpr uint32_t hi128 = ptx::smem_desc_hi(1024, ptx::kSw128);
      constexpr uint32_t lbo_k = 1u << 16;  // unused for swizzled K-major operands
      constexpr uint32_t lbo_v = (uint32_t)(kKVChunk >> 4) << 16;  // V's atoms of 64 columns lie a chunk apart
      constexpr uint32_t idesc_qk = ptx::idesc_bf16(128, kKT, 0);
      constexpr uint32_t idesc_pv = ptx::idesc_bf16(128, kD, 1);
      bool ok = true, issued = false;
      auto issue_s = [&](int t) {  // K_t landed: S = Q K_t^T
        const int slot = (e + t) % kStages;
        if (!wait_all(&bar->k_full[slot], ((e + t) / kStages) & 1)) return false;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          uint32_t acc = 0;
#pragma unroll 1
          for (int step = 0; step < kD / 16; ++step) {
            const uint32_t qo = (uint32_t)(((step >> 2) * kQChunk + (step & 3) * 32) >> 4) + lbo_k;
            const uint32_t ko = (uint32_t)((slot * kKVBytes + (step >> 2) * kKVChunk + (step & 3) * 32) >> 4) + lbo_k;
            ptx::mma_ss(tmem + slot * kKT, dsc(q4 + qo, hi128), dsc(k4 + ko, hi128), idesc_qk, acc);
            acc = 1;
          }
        }
        __syncwarp();
        ptx::mma_commit_elect(&bar->s_full[slot]);
        ptx::mma_commit_elect(&bar->k_empty[slot]);
        issued = true;
        return true;
      };
      if (n > 0) ok = wait_all(&bar->q_full, passes & 1);
      for (int t = 0; ok && t < 2 && t < n; ++t) ok = issue_s(t);
      for (int t = 0; ok && t < n; ++t) {
        // P_t and V_t there: O += P_t V_t, then the next scores over P_t
        const int slot = (e + t) % kStages;
        if (!wait_all(&bar->p_full[slot], ((e + t) / kStages) & 1) ||
            !wait_all(&bar->v_full[slot], ((e + t) / kStages) & 1)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
#pragma unroll 1
          for (int k = 0; k < kKT / 16; ++k) {
            // 16 keys: 8 tensor-memory columns of P, 16 rows (2 KB) of V
            const uint32_t vo = (uint32_t)((slot * kKVBytes + k * 16 * 128) >> 4) + lbo_v;
            ptx::mma_ts(tmem + 256, tmem + slot * kKT + k * 8, dsc(v4 + vo, hi128), idesc_pv, (t > 0 || k > 0) ? 1u : 0u);
          }
        }
        __syncwarp();
        ptx::mma_commit_elect(&bar->pv_done);
        ptx::mma_commit_elect(&bar->v_empty[slot]);
        if (t + 2 < n) ok = issue_s(t + 2);
      }
      if (ok && n > 0) ptx::mma_commit_elect(&bar->o_full);
      if (!ok) {
        if (lane == 0) fail(p, bar, kErrMma);
        if (issued) {
          // wait (bounded) for the MMAs already issued before tensor memory is freed
          ptx::mma_commit_elect(&bar->drain);
          ptx::mbar_wait_time_only(&bar->drain, 0, p.timeout_ns);
        }
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- softmax and output
      const int quarter = warp & 3;  // tensor-memory lane quarter this warp may access
      const int row = quarter * 32 + lane;
      const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
      const uint32_t o_tmem = tmem + lane_off + 256;
      const float sl2 = p.scale_log2;
      const bool valid = row < it.rows;
      int lo = 0, hi = it.keys - 1;  // keys this row sees
      if (p.causal) {
        hi = min(hi, it.pos + row);
        if (p.window) lo = max(0, it.pos + row - p.window + 1);
      }
      if (!valid) hi = -1;
      bool ok = true;
      float m = -INFINITY;  // running (stale) max of scaled scores, log2 domain
      float l = 0.f;        // running sum of exp2(x - m)
      for (int t = 0; t < n; ++t) {
        const int slot = (e + t) % kStages, kt = it.lo + t;
        const uint32_t s_tmem = tmem + lane_off + slot * kKT;
        const bool got = ptx::mbar_wait(&bar->s_full[slot], ((e + t) / kStages) & 1, p.timeout_ns, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        float x[kKT];
        ptx::tmem_ld32(s_tmem, *reinterpret_cast<float(*)[32]>(&x[0]));
        ptx::tmem_ld32(s_tmem + 32, *reinterpret_cast<float(*)[32]>(&x[32]));
        ptx::tmem_wait_ld();
        bool sees = valid;  // this row sees a key of the tile
        if (it.partial(kt)) {
          const int c_lo = max(lo - kt * kKT, 0), c_hi = min(hi - kt * kKT, kKT - 1);
          sees = c_lo <= c_hi;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint32_t vis = range_bits(g, c_lo, c_hi);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[32 * g + j] = ((vis >> j) & 1u) ? x[32 * g + j] : -INFINITY;
          }
        }
        // (the stale-max rule, and rows that keep their reference while another's is redone,
        // as in attention_packed.cu)
        const bool fresh = m == -INFINITY;
        float ts = exp_to_tmem(x, sl2, fresh ? 0.f : m, s_tmem);
        const bool redo = valid && (!(ts <= kMaxTileSum) || (fresh && sees && !(ts >= kMinTileSum)));
        if (fresh && sees && !redo) m = 0.f;  // the row's reference from here on
        if (__any_sync(0xffffffffu, redo)) {
          ptx::tmem_wait_st();  // let these stores land before they are overwritten
          const float m_new = redo ? fmaxf(m, row_max(x) * sl2) : m;
          const bool need_rescale = !fresh && m_new > m;
          if (fresh) m = m_new;
          if (__any_sync(0xffffffffu, need_rescale)) {
            // the last product adds into O: wait for it (S_t there means that the one before
            // it is done, so the barrier is one phase behind at most)
            const bool pv = ptx::mbar_wait(&bar->pv_done, (e + t - 1) & 1, p.timeout_ns, abort_flag);
            if (!__all_sync(0xffffffffu, pv)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const float alpha = need_rescale ? ptx::ex2(m - m_new) : 1.f;
            rescale_o<kD>(o_tmem, alpha);
            if (need_rescale) {
              l *= alpha;
              m = m_new;
            }
          }
          ts = exp_to_tmem(x, sl2, (m == -INFINITY) ? 0.f : m, s_tmem);
        }
        l += ts;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bar->p_full[slot]);
      }
      if (ok && n > 0) {
        const bool got = ptx::mbar_wait(&bar->o_full, passes & 1, p.timeout_ns, abort_flag);
        ok = __all_sync(0xffffffffu, got);
        ptx::tc_fence_after();
      }
      if (!ok) {
        if (lane == 0) fail(p, bar, kErrSoftmax);
      } else {
        const float b2 = p.sink ? __ldg(p.sink + it.h) * kLog2e : -INFINITY;
        const float M = fmaxf(m, b2);
        const float ref = M == -INFINITY ? 0.f : M;  // (no key and no sink: l = 0; scores that are NaN: l is)
        const float em = m == -INFINITY ? 1.f : ptx::ex2(m - ref);
        const float z = l * em + (b2 == -INFINITY ? 0.f : ptx::ex2(b2 - ref));
        const float o_scale = z == 0.f ? 0.f : em / z;
        const int64_t q_row = (int64_t)it.q_row + row;
        if (valid && p.lse) p.lse[(int64_t)it.h * p.T + q_row] = z == 0.f ? -INFINITY : (ref + ptx::lg2(z)) * kLn2;
        // a row's output that is not finite may be a hidden key's values' doing
        const bool part = n > 0 && (it.partial(it.lo) || it.partial(it.lo + n - 1)) && !again;
        float2 sum = make_float2(0.f, 0.f);
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + (q_row * p.H + it.h) * kD;
        const uint64_t o_policy = ptx::l2_policy_evict_first();
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += 16) {
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
        if (part && valid && !(fabsf(sum.x + sum.y) < INFINITY)) *reinterpret_cast<volatile int*>(&bar->marked[i % 3]) = 1;
        if (again) add_odd_values(p, it, row, lo, hi);
        ptx::tc_fence_before();  // (O is read: the next item's first product may overwrite it)
      }
    }
    const int stop = __syncthreads_or(*abort_flag);
    ptx::tc_fence_after();
    if (stop) break;
    e += n;
    passes += n > 0 ? 1 : 0;
    if (!again && bar->marked[i % 3]) {
      again = 1;
    } else {
      again = 0;
      ++i;
    }
  }
  if (threadIdx.x == 0) let_copies_land(abort_flag);
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_attention_packed_256(const PackedParams& p, cudaStream_t stream) {
  constexpr size_t smem = 1024 + kQBytes + 2 * kStages * kKVBytes + sizeof(Bar);
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(attention_packed_256_kernel, smem, &done);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.max_pairs * 2 * p.H;
  return launch_chained(attention_packed_256_kernel, (unsigned)(items < kPlanSms ? items : kPlanSms), 1, kThreads, smem, 1, p,
                        stream);
}

}  // namespace mattn
