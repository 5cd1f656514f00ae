// Decode attention over a prefix that every sequence of the batch shares,
// for sm_103a: the states (reference m, sum l, unnormalised O) of all
// B * G query rows of a key/value head against the P prefix keys, so that the
// prefix is read once per key/value head and not once per sequence.  The
// sequences' own keys are the row worker's (decode_rows.cuh), in further CTAs of
// the same grid, and decode_merge_kernel joins the states with the sink logit:
//   o = (sum_s 2^(m_s - M) O_s) / (sum_s 2^(m_s - M) l_s + exp(sink)).
//
// B * G rows against P keys is a matrix product of 4 d B G P FLOPs over 4 d P
// bytes: tensor-core work from a few rows on.  With KT keys per key tile
// (128; 64 at d = 256) and 128 query rows per tile:
//   S = Q K^T    M128 N=KT K=D   (shared memory x shared memory -> TMEM)
//   P = exp2(S * scale*log2e - m)  (one row per softmax thread)
//   O += P V     M128 N=D  K=KT  (P from TMEM)
// Step u of a CTA uses S buffer u & 1.  One query tile (SUB = 1): steps are its
// key tiles, and S_u+1 is formed while the softmax works on S_u.  Two query
// tiles (SUB = 2, head dims 64 and 128, when there are more than 128 rows):
// step 2 t + s is key tile t for query tile s, so each key tile read from
// memory is used twice and the tensor cores run one query tile's products
// during the other's softmax.
//
// Up to 128 rows a key tile costs ~1,000 tensor-core cycles against ~2,800 of
// an SM's share of HBM, so the prefix streams at memory speed (16 sequences of
// 4 heads of 256 a key/value head over 128K: 94 us with the merge, 6.1 TB/s);
// from 256 rows on the tensor cores and the exponentials bound it (1.63 us for
// 256 rows x 128 keys of 128 on an SM, 10.3 TFLOP/s; 1.9 beside own keys), and the
// states' way to memory and back (64 sequences over 32K: 48.2 us, of which the
// products end after 38).
//
// K and V tiles share one ring of slots in the order the products take them;
// the split of the keys over CTAs (shared_plan) fills the SMs, and every wait
// is bounded in time.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_ops.h"
#include "decode_rows.cuh"
#include "kernel_params.h"
#include "ptx.cuh"

namespace mattn {
namespace {

// A tile whose row sum passes 2^40 against the running reference, or a first
// tile whose sum against 0 stays below 2^-64, is redone against its own maximum
// (the forward kernels' rule): the common tile needs no maximum at all.
constexpr float kMaxTileSumS = 1099511627776.0f;
constexpr float kMinTileSumS = 5.421010862427522e-20f;

template <int D, int SUB>
struct ShGeo {
  static constexpr int KT = shared_key_tile(D);
  static constexpr int kQChunk = 128 * 128;                  // 128 rows x 64 columns
  static constexpr int kQTile = (D / 64) * kQChunk;
  static constexpr int kKVChunk = KT * 128;
  static constexpr int kSlot = (D / 64) * kKVChunk;          // one K or V tile: 32 KB (16 KB at d = 64)
  static constexpr int kSlots = shared_slots(D, SUB);
  static constexpr int kThreads = 128 + 128 * SUB;
  static constexpr int kOcol = 2 * KT > 256 ? 2 * KT : 256;  // first tensor-memory column of O
  static_assert(kOcol + SUB * D <= 512, "tensor memory");
  static_assert(kSlots <= 6, "barriers");
  static_assert(SUB * 128 * D * 4 <= SUB * kQTile + kSlots * kSlot, "the staged O must fit");
  // of the prefix's CTAs, and of the own keys'
  static constexpr size_t kPrefix = (size_t)SUB * kQTile + (size_t)kSlots * kSlot;
  static constexpr size_t kRows = (size_t)shared_row_warps(D, SUB) * (rows::Geo<D>::kRing + rows::Geo<D>::NS * 8) + 16;
};

struct ShBar {
  uint64_t full[6], empty[6];  // of each slot
  uint64_t q_full;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_final;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

__device__ __forceinline__ void fail_sh(const SharedParams& p, ShBar* bar, uint32_t bit) {
  *reinterpret_cast<volatile int*>(&bar->abort_flag) = 1;
  atomicOr(p.err, bit);
}

// NT: groups of eight query heads of the row workers in the grid's last CTAs,
// 0 = none.  TWO: one row tile.  The tensor cores idle for half of the time then,
// and P goes to them as the sum of two bf16 values (the lower parts in the other half of
// S's columns): outputs are as near to 64 bits as from 32-bit weights.  With more
// row tiles P is rounded to one bf16, as in the forward kernels, half a step (2^-8) off at
// most: the error against 64 bits is then 0.0023 of the output where its own rounding
// makes 0.0017, and two parts would cost (32K prefix, 8 key/value heads of 128) 256 rows
// each 40.3 -> 56.1 us, 512 67.6 -> 105.9; 512 of 64 34.0 -> 44.9; 256 of 256 45.6 -> 50.6.
template <int D, int SUB, int NT, bool TWO>
__global__ void __launch_bounds__(ShGeo<D, SUB>::kThreads, 1)
    decode_shared_kernel(const __grid_constant__ SharedParams p) {
  using Geo = ShGeo<D, SUB>;
  constexpr int KT = Geo::KT, NSL = Geo::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sq = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if constexpr (NT > 0) {
    const int first = p.plan.row_tiles * p.plan.n_split * p.H_kv;
    if ((int)blockIdx.x >= first) {
      // ------------------------------------------------------ the sequences' own keys
      using Rows = rows::Geo<D>;
      constexpr int kWarps = shared_row_warps(D, SUB);
      uint64_t* full = reinterpret_cast<uint64_t*>(sq + kWarps * Rows::kRing);
      volatile int* stop = reinterpret_cast<volatile int*>(full + kWarps * Rows::NS);
      if (threadIdx.x < kWarps * Rows::NS) ptx::mbar_init(full + threadIdx.x, 1);
      if (threadIdx.x == 0) *stop = 0;
      ptx::fence_barrier_init();
      __syncthreads();
      after_previous();
      const int w = threadIdx.x >> 5, ctas = gridDim.x - first;
      if (w < kWarps)
        rows::work<D, NT>(p.own, w * ctas + (int)blockIdx.x - first, ctas * kWarps, sq + w * Rows::kRing,
                          full + w * Rows::NS, stop);
      return;
    }
  }
  uint8_t* ring = sq + SUB * Geo::kQTile;
  ShBar* bar = reinterpret_cast<ShBar*>(ring + NSL * Geo::kSlot);
  volatile int* abort_flag = &bar->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // neighbouring CTAs: the row tiles of one key split, which share its keys in L2
  const int rt = blockIdx.x % p.plan.row_tiles;
  const int split = (blockIdx.x / p.plan.row_tiles) % p.plan.n_split;
  const int kvh = blockIdx.x / (p.plan.row_tiles * p.plan.n_split);
  const int G = p.H / p.H_kv;
  const int t_lo = split * p.plan.per_split;
  const int t_hi = t_lo + p.plan.per_split < p.plan.tiles ? t_lo + p.plan.per_split : p.plan.tiles;
  const int nt = t_hi - t_lo;       // key tiles of this CTA (>= 1: shared_plan)
  const int n_steps = nt * SUB;

  // Load order = the order the products take the tiles.  SUB 1: K0 K1 V0 K2 V1
  // ... ; SUB 2: K0 V0 K1 V1 ...  Load i of 2 nt: its tile and whether it is V.
  auto load_tile_of = [&](int i, int* t) -> bool {
    if (SUB == 2 || nt == 1) {
      *t = i >> 1;
      return i & 1;
    }
    if (i == 0) {
      *t = 0;
      return false;
    }
    if (i == 2 * nt - 1) {
      *t = nt - 1;
      return true;
    }
    *t = (i & 1) ? (i + 1) / 2 : i / 2 - 1;
    return !(i & 1);
  };
  auto issue_load = [&](int i) {
    int t;
    const bool v = load_tile_of(i, &t);
    const int slot = i % NSL;
    const int k0 = (t_lo + t) * KT;
    ptx::mbar_arrive_expect_tx(&bar->full[slot], Geo::kSlot);
    if (!debug_check(p.err, k0 >= 0 && k0 < p.P && kvh < p.H_kv, kSiteLoad)) {
      *abort_flag = 1;
      return;
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      ptx::tma_load_3d(ring + slot * Geo::kSlot + c * Geo::kKVChunk, v ? &p.tv : &p.tk, &bar->full[slot], c * 64, k0,
                       kvh);
  };
  // Set-up, side by side: warp 0 makes the barriers and starts the copies of the
  // queries and the first keys, warp 1 takes the tensor memory.  Queries: row r
  // of a query tile is head r % G of the tile's sequence r / G, whole sequences
  // only, so that a tile is one box of q as [B][H][d]; the rows left over
  // (128 mod G) are zeros.
  constexpr int kAhead = SUB == 2 ? 1 : 2;  // tiles started before the CTA's first barrier
  if (warp == 0) {
    if (lane < NSL) {
      ptx::mbar_init(&bar->full[lane], 1);
      ptx::mbar_init(&bar->empty[lane], 1);
    }
    if (lane < 2) {
      ptx::mbar_init(&bar->s_full[lane], 1);
      ptx::mbar_init(&bar->p_full[lane], 128);
      ptx::mbar_init(&bar->pv_done[lane], 1);
    }
    if (lane == 31) {
      ptx::mbar_init(&bar->q_full, 1);
      ptx::mbar_init(&bar->o_final, 1);
      ptx::mbar_init(&bar->drain, 1);
      bar->abort_flag = 0;
    }
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_shared();
    __syncwarp();
    after_previous();
    if (lane == 0) {
      if (p.selftest != 2) {
        ptx::mbar_arrive_expect_tx(&bar->q_full, (uint32_t)(SUB * (D / 64) * p.plan.seqs * G * 128));
#pragma unroll
        for (int x = 0; x < SUB; ++x)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            ptx::tma_load_3d(sq + x * Geo::kQTile + c * Geo::kQChunk, &p.tq, &bar->q_full, c * 64, kvh * G,
                             (rt * SUB + x) * p.plan.seqs);
      }
      for (int i = 0; i < kAhead && i < 2 * nt; ++i) issue_load(i);
    }
  } else if (warp == 1) {
    ptx::tmem_alloc(&bar->tmem_base, 512);
    ptx::tmem_relinquish();
  } else if (p.plan.seqs * G < 128) {
    const int used = p.plan.seqs * G;
    for (int i = threadIdx.x - 64; i < SUB * (D / 64) * (128 - used) * 8; i += Geo::kThreads - 64) {
      const int r = used + (i >> 3) % (128 - used), xc = (i >> 3) / (128 - used);  // xc: query tile and chunk
      *reinterpret_cast<uint4*>(sq + xc * Geo::kQChunk + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    ptx::fence_proxy_async_shared();
  }
  if (warp > 0) after_previous();  // (the states are written over what the previous grid may read)
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bar->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      for (int i = kAhead; i < 2 * nt; ++i) {
        if (i >= NSL && !ptx::mbar_wait(&bar->empty[i % NSL], ((i / NSL) & 1) ^ 1, p.timeout_ns, abort_flag)) {
          fail_sh(p, bar, kErrProducer);
          break;
        }
        issue_load(i);
        if (kDebugChecks && *abort_flag) break;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    auto wait_all = [&](uint64_t* b, uint32_t parity) {
      return __all_sync(0xffffffffu, ptx::mbar_wait(b, parity, p.timeout_ns, abort_flag));
    };
    const uint32_t q4 = ptx::smem_addr(sq) >> 4, r4 = ptx::smem_addr(ring) >> 4;
    constexpr uint32_t hi128 = ptx::smem_desc_hi(1024, ptx::kSw128);
    constexpr uint32_t lbo_k = 1u << 16;  // unused for swizzled K-major operands
    constexpr uint32_t idesc_qk = ptx::idesc_bf16(128, KT, 0);
    constexpr uint32_t idesc_pv = ptx::idesc_bf16(128, D, 1);
    constexpr uint32_t lbo_v = (uint32_t)(Geo::kKVChunk >> 4) << 16;  // 64-column atoms of V lie a chunk apart
    auto k_load = [&](int t) { return SUB == 2 || nt == 1 ? 2 * t : (t == 0 ? 0 : 2 * t - 1); };
    auto v_load = [&](int t) { return SUB == 2 || nt == 1 ? 2 * t + 1 : (t == nt - 1 ? 2 * nt - 1 : 2 * t + 2); };
    auto issue_s = [&](int u) -> bool {  // S_{u & 1} = Q K_t^T
      const int t = u / SUB, sub = u % SUB, ld = k_load(t), slot = ld % NSL;
      if (!wait_all(&bar->full[slot], (ld / NSL) & 1)) return false;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t qo = (uint32_t)((sub * Geo::kQTile + (k >> 2) * Geo::kQChunk + (k & 3) * 32) >> 4) + lbo_k;
          const uint32_t ko = (uint32_t)((slot * Geo::kSlot + (k >> 2) * Geo::kKVChunk + (k & 3) * 32) >> 4) + lbo_k;
          ptx::mma_ss(tmem + (u & 1) * KT, desc64(q4 + qo, hi128), desc64(r4 + ko, hi128), idesc_qk, k > 0);
        }
      }
      __syncwarp();
      ptx::mma_commit_elect(&bar->s_full[u & 1]);
      if (sub == SUB - 1) ptx::mma_commit_elect(&bar->empty[slot]);
      return true;
    };
    bool ok = wait_all(&bar->q_full, 0), issued = false;
    for (int u = 0; ok && u < 2 && u < n_steps; ++u) {
      ok = issue_s(u);
      issued = issued || ok;
    }
    for (int u = 0; ok && u < n_steps; ++u) {
      // P_u written, V landed: O_sub += P V
      const int t = u / SUB, sub = u % SUB, ld = v_load(t), slot = ld % NSL;
      if (!wait_all(&bar->p_full[u & 1], (u >> 1) & 1) || !wait_all(&bar->full[slot], (ld / NSL) & 1)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint32_t p_tm = tmem + (u & 1) * KT, o_tm = tmem + Geo::kOcol + sub * D;
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          // 16 keys: 8 tensor-memory columns of P, 16 rows (2 KB) of V
          const uint32_t vo = (uint32_t)((slot * Geo::kSlot + k * 16 * 128) >> 4) + lbo_v;
          ptx::mma_ts(o_tm, p_tm + k * 8, desc64(r4 + vo, hi128), idesc_pv, t > 0 || k > 0);
        }
        if constexpr (TWO) {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k) {
            const uint32_t vo = (uint32_t)((slot * Geo::kSlot + k * 16 * 128) >> 4) + lbo_v;
            ptx::mma_ts(o_tm, p_tm + KT / 2 + k * 8, desc64(r4 + vo, hi128), idesc_pv, 1);
          }
        }
      }
      __syncwarp();
      ptx::mma_commit_elect(&bar->pv_done[sub]);
      if (sub == SUB - 1) ptx::mma_commit_elect(&bar->empty[slot]);
      if (u + 2 < n_steps) ok = issue_s(u + 2);
    }
    if (ok) {
      ptx::mma_commit_elect(&bar->o_final);
    } else {
      if (lane == 0) fail_sh(p, bar, kErrMma);
      if (issued) {
        ptx::mma_commit_elect(&bar->drain);
        ptx::mbar_wait_time_only(&bar->drain, 0, p.timeout_ns);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax + state output
    const int sub = (warp - 4) >> 2;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int local = (warp & 3) * 32 + lane, used = p.plan.seqs * G;
    const int row = (rt * SUB + sub) * used + local;  // of the key/value head's B * G rows
    const uint32_t o_tmem = tmem + lane_off + Geo::kOcol + sub * D;
    const float sl2 = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
      const int u = t * SUB + sub;
      const uint32_t s_tmem = tmem + lane_off + (u & 1) * KT;
      const bool got = ptx::mbar_wait(&bar->s_full[u & 1], (u >> 1) & 1, p.timeout_ns, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      float x[KT];
#pragma unroll
      for (int c0 = 0; c0 < KT; c0 += 32) ptx::tmem_ld32(s_tmem + c0, *reinterpret_cast<float(*)[32]>(&x[c0]));
      ptx::tmem_wait_ld();
      const int left = p.P - (t_lo + t) * KT;  // keys of this tile that exist
      if (left < KT) {
#pragma unroll
        for (int c = 0; c < KT; ++c) x[c] = c < left ? x[c] : -INFINITY;
      }
      auto exp_pass = [&](float mref, float& sum) {
        const float2 sl2v = make_float2(sl2, sl2), negm = make_float2(-mref, -mref);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c0 = 0; c0 < KT; c0 += 64) {
          uint32_t pk[32], lo[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 tt = ptx::ffma2(make_float2(x[c0 + 2 * i], x[c0 + 2 * i + 1]), sl2v, negm);
            const float2 pp = make_float2(ptx::ex2(tt.x), ptx::ex2(tt.y));
            if constexpr (TWO) two_bf16(pp.x, pp.y, &pk[i], &lo[i]);
            else pk[i] = ptx::pack_bf16x2(pp.x, pp.y);
            acc[i & 1] = ptx::fadd2(acc[i & 1], pp);
          }
          ptx::tmem_st32(s_tmem + c0 / 2, pk);
          if constexpr (TWO) ptx::tmem_st32(s_tmem + KT / 2 + c0 / 2, lo);
        }
        const float2 a = ptx::fadd2(acc[0], acc[1]);
        sum = a.x + a.y;
      };
      float ts = 0.f;
      const bool first = m == -INFINITY;
      exp_pass(first ? 0.f : m, ts);
      const bool slow = __any_sync(0xffffffffu, !(ts <= kMaxTileSumS) || (first && !(ts >= kMinTileSumS)));
      if (!slow) {
        if (first) m = 0.f;  // the row's reference from here on
      } else {
        ptx::tmem_wait_st();
        float mx = x[0];
#pragma unroll
        for (int c = 1; c < KT; ++c) mx = fmaxf(mx, x[c]);
        const float m_new = fmaxf(m, mx * sl2);
        const bool rescale = m != -INFINITY && m_new > m;
        if (m == -INFINITY) m = m_new;
        if (__any_sync(0xffffffffu, rescale)) {
          // the previous product of this query tile adds into O: wait for it.
          // One product of this tile completes one phase, and the next one
          // starts only after this step's P is written, so phase t - 1 is the
          // last one completed or under way.
          const bool pv = t == 0 || ptx::mbar_wait(&bar->pv_done[sub], (t - 1) & 1, p.timeout_ns, abort_flag);
          if (!__all_sync(0xffffffffu, pv)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const float alpha = rescale ? ptx::ex2(m - m_new) : 1.f;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float ov[32];
            ptx::tmem_ld32(o_tmem + c0, ov);
            ptx::tmem_wait_ld();
            uint32_t ou[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) ou[i] = __float_as_uint(ov[i] * alpha);
            ptx::tmem_st32(o_tmem + c0, ou);
          }
          if (rescale) {
            l *= alpha;
            m = m_new;
          }
        }
        exp_pass(m == -INFINITY ? 0.f : m, ts);
      }
      l += ts;
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bar->p_full[u & 1]);
    }
    if (ok) {
      const bool got = ptx::mbar_wait(&bar->o_final, 0, p.timeout_ns, abort_flag);
      ok = __all_sync(0xffffffffu, got);
      ptx::tc_fence_after();
    }
    if (!ok) {
      if (lane == 0) fail_sh(p, bar, kErrSoftmax);
    } else {
      // O leaves through shared memory (the queries and the ring are idle by
      // now: every tile was consumed), as boxes of 32 rows x 32 columns in the 128-byte swizzle,
      // whose rows the threads write without bank conflicts.  (16-byte stores
      // from the registers touch 32 rows each, and a copy per row costs the
      // copy engine 8 ns: 2 us for 256 rows.)
      const bool valid = local < used && row < p.rows;
      const int64_t at = ((int64_t)kvh * p.rows + (valid ? row : 0)) * p.plan.n_split + split;
      uint8_t* stage = sq + (warp - 4) * (32 * D * 4);
#pragma unroll 2
      for (int c0 = 0; c0 < D; c0 += 32) {
        float ov[32];
        ptx::tmem_ld32(o_tmem + c0, ov);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(stage + c0 * 128 + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
      }
      ptx::fence_proxy_async_shared();
      __syncwarp();
      const int first = row - lane;  // the warp's first row; a box ends at the head's last row by itself
      if (((warp & 3) + 1) * 32 <= used) {
        if (lane == 0 && first < p.rows)
          for (int c = 0; c < D / 32; ++c)
            ptx::tma_store_4d(&p.to, stage + c * 4096, c * 64, split, first, kvh);
      } else if (valid) {
        // rows past the tile's last sequence belong to the next tile: row by row
        for (int c = 0; c < D / 4; ++c)
          *reinterpret_cast<float4*>(p.part_o + at * D + c * 4) = *reinterpret_cast<const float4*>(
              stage + (c >> 3) * 4096 + lane * 128 + (((c & 7) ^ (lane & 7)) << 4));
      }
      if (valid) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
      ptx::bulk_commit_group();
      ptx::bulk_wait_all();
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  // Whoever gave up did so before the barrier, perhaps long after the last load was
  // started: copies still in flight land before the shared memory goes away.
  if (threadIdx.x == 0 && *abort_flag) {
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t it = 0; it < 0x10000000u && ptx::globaltimer_ns() - t0 < 2000000ull; ++it) { }
  }
}

template <int D, int SUB, int NT, bool TWO>
cudaError_t launch_nt(const SharedParams& p, cudaStream_t stream) {
  using Geo = ShGeo<D, SUB>;
  constexpr size_t prefix = Geo::kPrefix + sizeof(ShBar), own = NT ? Geo::kRows : 0;
  constexpr size_t smem = 1024 + (prefix > own ? prefix : own);
  static_assert(smem <= 227 * 1024, "shared memory");
  // A CTA takes all of an SM's tensor memory before it waits for the previous grid.
  // If a second one could lie beside it, a CTA of that grid might find the tensor memory
  // taken by one that waits for it, and neither would end: no SM holds two.
  static_assert(2 * (smem + 1024) > 228 * 1024, "one CTA per SM, by its shared memory");
  auto kern = decode_shared_kernel<D, SUB, NT, TWO>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kern, smem, &done);
  if (e != cudaSuccess) return e;
  const int grid = p.plan.row_tiles * p.plan.n_split * p.H_kv + (NT ? p.plan.own_ctas : 0);
  return launch_chained(kern, (unsigned)grid, 1, Geo::kThreads, smem, 1, p, stream);
}

template <int D, int SUB, bool TWO>
cudaError_t launch_sub(const SharedParams& p, cudaStream_t stream) {
  if (p.own.L == 0) return launch_nt<D, SUB, 0, TWO>(p, stream);
  return p.H / p.H_kv <= 8 ? launch_nt<D, SUB, 1, TWO>(p, stream) : launch_nt<D, SUB, 2, TWO>(p, stream);
}

}  // namespace

cudaError_t launch_decode_shared(const SharedParams& p, int d, cudaStream_t stream) {
  switch (d * 4 + p.plan.sub) {  // (d <= 128: two query tiles a CTA from the second row tile on)
    case 64 * 4 + 1: return launch_sub<64, 1, true>(p, stream);
    case 64 * 4 + 2: return launch_sub<64, 2, false>(p, stream);
    case 128 * 4 + 1: return launch_sub<128, 1, true>(p, stream);
    case 128 * 4 + 2: return launch_sub<128, 2, false>(p, stream);
    case 256 * 4 + 1: return p.plan.row_tiles == 1 ? launch_sub<256, 1, true>(p, stream) : launch_sub<256, 1, false>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

// The prefix's split over `sms` SMs: a CTA holds its SM, so the launch runs in
// waves; of the splits that fill one to four waves (and of none) the one whose
// waves cost least, a wave costing its key tiles and a start-up and state output
// of about six steps, and each split 0.02 for its states' merge.  Returns the steps.
static double split_over(SharedPlan* s, int H_kv, int sms) {
  const int64_t units = (int64_t)s->row_tiles * H_kv;
  double best = 1e300;
  for (int64_t w = 0; w <= 4; ++w) {
    int64_t ns = w * sms / units;
    ns = ns < 1 ? 1 : (ns > s->tiles ? s->tiles : ns);
    const int64_t per = (s->tiles + ns - 1) / ns;
    ns = (s->tiles + per - 1) / per;  // no split without tiles
    const int64_t waves = (units * ns + sms - 1) / sms;
    const double cost = (double)waves * ((double)per * s->sub + 6.0) + 0.02 * (double)ns;
    if (cost < best - 1e-9) {
      best = cost;
      s->n_split = (int)ns;
      s->per_split = (int)per;
    }
  }
  return best;
}

// The own keys' CTAs run beside the prefix's on SMs of their own, as many as make
// both end together if the sequences hold half of their capacity: the prefix is
// bound by the tensor cores or the memory, the own keys by the memory's latency,
// and one after the other (a CTA for every SM, which wait for free ones) they take
// their sum at most.  Measured beside each other: own keys 60 GB/s an SM and 6 us of
// start-up, a prefix step (128 rows x a key tile) 0.95 us, at most 6.5 TB/s; own
// keys on all SMs 4.5 TB/s and 8 us.  (64 sequences, 32 / 8 heads of 128, 32K
// prefix, 256 own keys on average: 55.0 us one after the other, 53.1, 48.4 and
// 52.8 with 16, 32 and 48 SMs for the own keys; 128 over 8K: 58.3 one after the
// other, 42.5 and 34.1 with 32 and 56.  The plan takes 32 and 56.)  Of each split
// the SMs that it leaves free are priced, and the own keys get those alone only
// where that is the lower price: their shares are dealt out once, and no SM that
// ends the prefix takes any of them over (64 sequences of 16,384 own keys behind
// 2,048 and 2,304 shared ones: 1,729 and 5,096 us with the 24 and 8 SMs left free,
// 745 and 735 with a CTA on every SM; the bytes at the copy rate take 644).
SharedPlan shared_plan(int B, int H, int H_kv, int P, int L, int d) {
  SharedPlan s = {};
  s.seqs = 128 / (H / H_kv);
  s.sub = B > s.seqs && d <= 128 ? 2 : 1;
  s.row_tiles = (B + s.seqs * s.sub - 1) / (s.seqs * s.sub);
  const int kt = shared_key_tile(d);
  s.tiles = (P + kt - 1) / kt;
  s.n_split = 1;
  s.per_split = s.tiles;
  s.own_ctas = kPlanSms;
  if (s.tiles == 0) return s;
  const double own_bytes = 2.0 * d * H_kv * (double)B * L;
  const double stream_us = 4.0 * d * H_kv * (double)P / 6.5e6;
  double best = 1e300;
  SharedPlan chosen = s;
  for (int r = 0; r <= kPlanSms / 2; r += 8) {
    SharedPlan t = s;
    const double steps = split_over(&t, H_kv, kPlanSms - r);
    const double prefix = steps * 0.95 > stream_us ? steps * 0.95 : stream_us;
    double cost = prefix + (L > 0 ? 8.0 + own_bytes / 4.5e6 : 0.0);
    const int64_t free = kPlanSms - (int64_t)t.row_tiles * t.n_split * H_kv;
    if (L > 0 && free >= 8) {
      const double own = 6.0 + own_bytes / ((double)free * 60e3), beside = prefix > own ? prefix : own;
      if (beside < cost) {
        cost = beside;
        t.own_ctas = (int)free;
      }
    }
    if (cost < best - 1e-9) {
      best = cost;
      chosen = t;
    }
    if (L <= 0) break;
  }
  return chosen;
}

}  // namespace mattn
