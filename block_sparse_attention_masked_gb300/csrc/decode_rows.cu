// Decode attention over a sequence's own keys or over its selected blocks,
// for sm_103a: one query token per sequence, the G query heads of a
// key/value head together.
//
//   o_h = sum_j p_hj v_j / (sum_j p_hj + exp(sink_h)),  p_hj = exp(scale q_h . k_j)
//
// over the sequence's list of keys: every cached key in order, or those of
// the listed blocks.  4 d bytes per key against 4 d G FLOPs: HBM-bound, and on
// the CUDA cores the issue slots would be the bound at G = 8 (decode.cu), so
// the products run on warp-level matrix instructions with the keys as the
// tall operand (no row of a 16 x 8 x 16 product is padding at G = 8):
//   S^T = K Q^T   16 keys x 8 heads,  K rows by ldmatrix, Q^T kept in registers
//   O^T += V^T P^T   16 dims x 8 heads,  V by transposing ldmatrix; P^T is S^T's
//                 register layout turned by movmatrix
// so that a head's scores, running maximum and O columns sit in the same
// lanes.  A tcgen05 product would spend a 128-row tile on these 8 rows.
//
// Each warp runs its own ring of key tiles (decode_rows_tile keys of K and V,
// 128-byte-swizzled TMA boxes): the warp that consumes a stage refills it, so
// the only waits are for landed copies.  Warps of a CTA take the tiles of its
// split in turn and merge in shared memory; the CTA writes the split's state,
// or o itself where there is one split.
//
// Rows of a tile that hold no key of the list (past the sequence's end, an
// unused list entry) may hold anything: their scores are replaced by -inf and
// their value rows by zeros before the product, so that what a cache holds
// there never reaches a result.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_ops.h"
#include "kernel_params.h"
#include "ptx.cuh"

namespace mattn {
namespace {

constexpr float kLog2eR = 1.4426950408889634f;
constexpr float kLn2R = 0.6931471805599453f;
constexpr int kRowWarps = 4;

template <int D>
struct RowGeo {
  static constexpr int TK = decode_rows_tile(D);
  static constexpr int kChunks = D / 64;             // 64-column boxes of a row
  static constexpr int kChunk = TK * 128;            // bytes of one box column
  static constexpr int kTensor = kChunks * kChunk;   // K or V of a tile
  static constexpr int kStage = 2 * kTensor;
  static constexpr int NS = D == 64 ? 6 : 3;         // stages per warp (192 KB per CTA)
  static constexpr int kRing = kRowWarps * NS * kStage;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c += a b, 16 x 8 x 16, bf16 inputs and fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct RowBar {
  uint64_t full[kRowWarps][8];
  int abort_flag;
};

// NT: groups of eight query heads.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kRowWarps, 1) decode_rows_kernel(const __grid_constant__ DecodeRowsParams p,
                                                                       int after) {
  using Geo = RowGeo<D>;
  constexpr int TK = Geo::TK, NS = Geo::NS, MT = TK / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  RowBar* bar = reinterpret_cast<RowBar*>(ring + Geo::kRing);
  float* wml = reinterpret_cast<float*>(bar + 1);       // [kRowWarps][8 NT][2]
  float* wo = reinterpret_cast<float*>(ring);           // [kRowWarps][8 NT][D], after the loop
  volatile int* abort_flag = &bar->abort_flag;

  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x;
  const int bkv = blockIdx.y, b = bkv / p.H_kv, kvh = bkv % p.H_kv;
  const int G = p.H / p.H_kv;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kRowWarps; ++w)
      for (int s = 0; s < NS; ++s) ptx::mbar_init(&bar->full[w][s], 1);
    bar->abort_flag = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();

  int len = p.seq_lens ? p.seq_lens[b] : p.L;
  len = len < 0 ? 0 : (len > p.L ? p.L : len);
  const int32_t* ids = p.ids ? p.ids + (int64_t)bkv * p.top_k : nullptr;
  // entries of the key list: the sequence's keys, or the listed blocks up to
  // the last entry that names a block with cached keys
  int keys = len;
  if (ids) {
    int last = -1;
    for (int i = lane; i < p.top_k; i += 32) {
      const int id = ids[i];
      if (id >= 0 && (int64_t)id * p.block < len) last = i;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    keys = (last + 1) * p.block;  // the host keeps top_k * block below 2^30
  }
  const int n_tiles = (keys + TK - 1) / TK;
  const int per = (n_tiles + p.n_split - 1) / p.n_split;
  const int t_lo = split * per;
  const int t_hi = t_lo + per < n_tiles ? t_lo + per : n_tiles;

  const int64_t bh0 = (int64_t)b * p.H + kvh * G;
  const int hc = (lane & 3) * 2;  // this lane's head columns hc, hc + 1 (of each group of eight)
  float m[NT][2], l[NT][2];
  float o[NT][D / 16][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
  }

  // Row r of tile t: whether it holds a key of the list; lane r's answer for
  // its row goes into the tile's mask.
  auto row_key = [&](int t, int r) -> int {  // key position, or -1
    const int i = t * TK + r;
    if (i >= keys) return -1;
    if (!ids) return i;
    const int j = i / p.block;
    const int id = ids[j];
    const int64_t pos = (int64_t)id * p.block + (i - j * p.block);
    return id >= 0 && pos < len ? (int)pos : -1;
  };
  auto tile_mask = [&](int t) -> uint32_t {
    return __ballot_sync(0xffffffffu, lane < TK && row_key(t, lane < TK ? lane : 0) >= 0);
  };
  uint8_t* wring = ring + warp * NS * Geo::kStage;
  // The tile's boxes: box_rows keys x 64 columns each; a box whose first row
  // holds no key is not loaded (its rows hold none: boxes never straddle
  // blocks).
  auto issue = [&](int t, int stage, uint32_t mask) {
    const int nb = TK / p.box_rows;
    uint32_t boxes = 0;
    for (int x = 0; x < nb; ++x) boxes += (mask >> (x * p.box_rows)) & 1u;
    uint64_t* full = &bar->full[warp][stage];
    if (lane == 0) ptx::mbar_arrive_expect_tx(full, boxes * (uint32_t)(2 * Geo::kChunks * p.box_rows * 128));
    __syncwarp();
    if (lane < nb * Geo::kChunks * 2) {
      const int x = lane / (Geo::kChunks * 2), c = (lane / 2) % Geo::kChunks, tensor = lane & 1;
      if ((mask >> (x * p.box_rows)) & 1u) {
        const int pos = row_key(t, x * p.box_rows);
        if (debug_check(p.err, pos >= 0 && pos < p.L && bkv < p.B * p.H_kv && stage < NS, kSiteLoad))
          ptx::tma_load_3d(wring + stage * Geo::kStage + tensor * Geo::kTensor + c * Geo::kChunk + x * p.box_rows * 128,
                           tensor ? &p.tv : &p.tk, full, c * 64, pos, bkv);
      }
    }
  };

  // queries of the group as B operands: k = dims, n = heads
  uint32_t qf[NT][D / 16][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int g = nt * 8 + (lane >> 2);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                            (bh0 + (g < G ? g : 0)) * D) + (lane & 3);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      qf[nt][i][0] = g < G ? __ldg(src + i * 8) : 0u;
      qf[nt][i][1] = g < G ? __ldg(src + i * 8 + 4) : 0u;
    }
  }

  // this warp's tiles, t_lo + warp + n kRowWarps; stage n % NS, phase n / NS
  const int mine = t_hi - t_lo > warp ? (t_hi - t_lo - warp + kRowWarps - 1) / kRowWarps : 0;
  auto tile_at = [&](int n) { return t_lo + warp + n * kRowWarps; };
  for (int n = 0; n < NS && n < mine; ++n) issue(tile_at(n), n, tile_mask(tile_at(n)));
  const uint32_t ring_s = ptx::smem_addr(wring);
  bool ok = true;
  for (int n = 0; n < mine; ++n) {
    const int stage = n % NS;
    const uint32_t mask = tile_mask(tile_at(n));
    const bool got = ptx::mbar_wait(&bar->full[warp][stage], (n / NS) & 1, p.timeout_ns, abort_flag);
    if (!__all_sync(0xffffffffu, got)) {
      ok = false;
      break;
    }
    const uint32_t ks = ring_s + stage * Geo::kStage, vs = ks + Geo::kTensor;
    constexpr uint32_t kAll = TK == 32 ? 0xffffffffu : ((1u << TK) - 1u);
    if (mask != kAll) {
      // value rows without a key: zeros (their weights are 0, and 0 x NaN is NaN)
      for (int r = 0; r < TK; ++r) {
        if ((mask >> r) & 1u) continue;
        for (int i = lane; i < Geo::kChunks * 8; i += 32)
          *reinterpret_cast<uint4*>(wring + stage * Geo::kStage + Geo::kTensor + (i >> 3) * Geo::kChunk + r * 128 +
                                    (i & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    // S^T: two accumulators per tile so that neighbouring products do not wait on each other
    float s[NT][MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float acc[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nt][a][j] = 0.f;
      const int key = mt * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int u = 2 * i + (lane >> 4);  // 16-byte piece of the row
        uint32_t a[4];
        ldsm4(a, ks + (u >> 3) * Geo::kChunk + key * 128 + (((u & 7) ^ (key & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][i & 1], a, qf[nt][i][0], qf[nt][i][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][mt][j] = (acc[nt][0][j] + acc[nt][1][j]) * p.scale_log2;
    }
    if (mask != kAll) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const bool v0 = (mask >> (mt * 16 + (lane >> 2))) & 1u, v1 = (mask >> (mt * 16 + 8 + (lane >> 2))) & 1u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (!v0) s[nt][mt][0] = s[nt][mt][1] = -INFINITY;
          if (!v1) s[nt][mt][2] = s[nt][mt][3] = -INFINITY;
        }
      }
    }
    // online softmax per head column (log2 domain)
    float alpha[NT][2];
    uint32_t pf[NT][MT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(s[nt][mt][e], s[nt][mt][e + 2]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float m_new = fmaxf(m[nt][e], mx);
        alpha[nt][e] = m[nt][e] == m_new ? 1.f : ptx::ex2(m[nt][e] - m_new);
        m[nt][e] = m_new;
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        float sum = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          s[nt][mt][e] = ptx::ex2(s[nt][mt][e] - ref);
          s[nt][mt][e + 2] = ptx::ex2(s[nt][mt][e + 2] - ref);
          sum += s[nt][mt][e] + s[nt][mt][e + 2];
        }
        l[nt][e] = l[nt][e] * alpha[nt][e] + sum;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        // P^T as B operand (k = keys, n = heads): the weights as bf16, whose
        // half step of 2^-9 stays below the output's own rounding; the sums
        // above are of the unrounded weights
        pf[nt][mt][0] = movm_t(ptx::pack_bf16x2(s[nt][mt][0], s[nt][mt][1]));
        pf[nt][mt][1] = movm_t(ptx::pack_bf16x2(s[nt][mt][2], s[nt][mt][3]));
      }
    }
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) moved = moved || alpha[nt][0] != 1.f || alpha[nt][1] != 1.f;
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[nt][i][0] *= alpha[nt][0];
          o[nt][i][1] *= alpha[nt][1];
          o[nt][i][2] *= alpha[nt][0];
          o[nt][i][3] *= alpha[nt][1];
        }
    }
    // O^T += V^T P^T
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int key = mt * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int u = 2 * i + ((lane >> 3) & 1);
        uint32_t a[4];
        ldsm4_t(a, vs + (u >> 3) * Geo::kChunk + key * 128 + (((u & 7) ^ (key & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a, pf[nt][mt][0], pf[nt][mt][1]);
      }
    }
    __syncwarp();
    if (n + NS < mine) {
      if (mask != kAll) ptx::fence_proxy_async_shared();  // the zeros above before the copy that overwrites them
      __syncwarp();
      issue(tile_at(n + NS), stage, tile_mask(tile_at(n + NS)));
    }
  }
  if (!ok) {
    if (lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, kErrProducer);
    }
    // let copies already in flight land before the shared memory goes away
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t it = 0; it < 0x10000000u && ptx::globaltimer_ns() - t0 < 2000000ull; ++it) { }
  }

  // merge the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
  __syncthreads();  // every copy of every ring has landed and been read
  constexpr int HP = 8 * NT;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (lane < 4) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        wml[(warp * HP + nt * 8 + hc + e) * 2 + 0] = m[nt][e];
        wml[(warp * HP + nt * 8 + hc + e) * 2 + 1] = l[nt][e];
      }
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        wo[(warp * HP + nt * 8 + hc + (j & 1)) * D + i * 16 + (lane >> 2) + (j >> 1) * 8] = o[nt][i][j];
  }
  __syncthreads();
  if (*abort_flag) return;
  for (int t = threadIdx.x; t < G * D; t += 32 * kRowWarps) {
    const int g = t / D, c = t % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, wml[(w * HP + g) * 2]);
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      const float mw = wml[(w * HP + g) * 2];
      // a warp without a key adds nothing; one whose scores are all -inf or
      // NaN carries its sums (0 or NaN) along
      const float e = mw == M ? 1.f : ptx::ex2(mw - M);
      L = fmaf(wml[(w * HP + g) * 2 + 1], e, L);
      O = fmaf(wo[(w * HP + g) * D + c], e, O);
    }
    const int64_t row = bh0 + g;
    if (p.part_o) {
      p.part_o[(row * p.n_split + split) * D + c] = O;
      if (c == 0) {
        p.part_ml[(row * p.n_split + split) * 2 + 0] = M;
        p.part_ml[(row * p.n_split + split) * 2 + 1] = L;
      }
    } else {
      const float b2 = p.sink ? p.sink[kvh * G + g] * kLog2eR : -INFINITY;
      const float Mt = fmaxf(M, b2);
      const float e = Mt == M ? 1.f : ptx::ex2(M - Mt);
      const float z = L * e + (b2 == -INFINITY ? 0.f : ptx::ex2(b2 - Mt));
      const float out = z == 0.f ? 0.f : O * e / z;
      reinterpret_cast<__nv_bfloat16*>(p.o)[row * D + c] = __float2bfloat16_rn(out);
      if (c == 0 && p.lse) p.lse[row] = z == 0.f ? -INFINITY : (Mt + __log2f(z)) * kLn2R;
    }
  }
  // launched beside the previous grid: complete only after it, so that a
  // grid that waits for this one finds both results
  if (after) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, int NT>
cudaError_t launch_nt(const DecodeRowsParams& p, bool after, cudaStream_t stream) {
  using Geo = RowGeo<D>;
  static_assert(kRowWarps * 8 * NT * D * 4 <= Geo::kRing, "the warps' O must fit in the ring");
  const size_t smem = 1024 + Geo::kRing + sizeof(RowBar) + kRowWarps * 8 * NT * 2 * sizeof(float);
  auto kern = decode_rows_kernel<D, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kern, smem, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_split, p.B * p.H_kv);
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, after ? 1 : 0);
}

// One row (b, h) per CTA of four warps: the warps take the states in turn,
// lanes hold D / 32 values each.
template <int D>
__global__ void __launch_bounds__(128) decode_merge_kernel(const MergeParams p) {
  constexpr int V = D / 32;
  __shared__ float sl[4], so[4][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t bh = blockIdx.x;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H), G = p.H / p.H_kv;
  const int64_t ra = ((int64_t)(h / G) * p.B + b) * G + h % G;
  float M = -INFINITY, L = 0.f, O[V];
#pragma unroll
  for (int i = 0; i < V; ++i) O[i] = 0.f;
  // the largest reference first: every weight is then formed once
  for (int s = lane; s < p.na + p.nb; s += 32)
    M = fmaxf(M, s < p.na ? p.a_ml[(ra * p.na + s) * 2] : p.b_ml[(bh * p.nb + s - p.na) * 2]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll 4
  for (int s = warp; s < p.na + p.nb; s += 4) {
    const bool a = s < p.na;
    const int64_t at = a ? ra * p.na + s : bh * p.nb + s - p.na;
    const float2 ml = *reinterpret_cast<const float2*>((a ? p.a_ml : p.b_ml) + at * 2);
    const float* src = (a ? p.a_o : p.b_o) + at * D + lane * V;
    float v[V];
    if constexpr (V == 2) {
      const float2 x = *reinterpret_cast<const float2*>(src);
      v[0] = x.x; v[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(src + i);
        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
      }
    }
    const float e = ml.x == M ? 1.f : ptx::ex2(ml.x - M);
    L = fmaf(ml.y, e, L);
#pragma unroll
    for (int i = 0; i < V; ++i) O[i] = fmaf(v[i], e, O[i]);
  }
  if (lane == 0) sl[warp] = L;
#pragma unroll
  for (int i = 0; i < V; ++i) so[warp][lane * V + i] = O[i];
  __syncthreads();
  const float b2 = p.sink ? p.sink[h] * kLog2eR : -INFINITY;
  const float Mt = fmaxf(M, b2);
  const float e = Mt == M ? 1.f : ptx::ex2(M - Mt);
  const float z = (sl[0] + sl[1] + sl[2] + sl[3]) * e + (b2 == -INFINITY ? 0.f : ptx::ex2(b2 - Mt));
  for (int c = threadIdx.x; c < D; c += 128) {
    const float x = (so[0][c] + so[1][c] + so[2][c] + so[3][c]) * e;
    reinterpret_cast<__nv_bfloat16*>(p.o)[bh * D + c] = __float2bfloat16_rn(z == 0.f ? 0.f : x / z);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[bh] = z == 0.f ? -INFINITY : (Mt + __log2f(z)) * kLn2R;
}

template <int D>
cudaError_t launch_merge_d(const MergeParams& p, bool after, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * p.H);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, decode_merge_kernel<D>, p);
}

}  // namespace

cudaError_t launch_decode_rows(const DecodeRowsParams& p, int d, bool after, cudaStream_t stream) {
  const int nt = (p.H / p.H_kv + 7) / 8;
  switch (d * 4 + nt) {
    case 64 * 4 + 1: return launch_nt<64, 1>(p, after, stream);
    case 64 * 4 + 2: return launch_nt<64, 2>(p, after, stream);
    case 128 * 4 + 1: return launch_nt<128, 1>(p, after, stream);
    case 128 * 4 + 2: return launch_nt<128, 2>(p, after, stream);
    case 256 * 4 + 1: return launch_nt<256, 1>(p, after, stream);
    case 256 * 4 + 2: return launch_nt<256, 2>(p, after, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_merge(const MergeParams& p, int d, bool after, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_merge_d<64>(p, after, stream);
    case 128: return launch_merge_d<128>(p, after, stream);
    case 256: return launch_merge_d<256>(p, after, stream);
    default: return cudaErrorInvalidValue;
  }
}

// Splits: the CTAs hold their SM (the rings fill its shared memory), so the
// launch runs in waves; the count is the one whose waves cost least, a wave
// costing its share of tiles and a start-up of about eight tiles.
int decode_rows_splits(int64_t groups, int64_t keys, int d) {
  const int64_t tk = decode_rows_tile(d) * kRowWarps;  // a CTA's tiles in step
  const int64_t steps = (keys + tk - 1) / tk;
  if (steps <= 1) return 1;
  int best = 1;
  double best_cost = 1e300;
  for (int64_t ns = 1; ns <= steps && ns <= 256; ++ns) {
    const int64_t waves = (groups * ns + kPlanSms - 1) / kPlanSms;
    const double cost = (double)waves * ((double)((steps + ns - 1) / ns) + 2.0) + (ns > 1 ? 2.0 : 0.0);
    if (cost < best_cost - 1e-9) {
      best_cost = cost;
      best = (int)ns;
    }
  }
  return best;
}

}  // namespace mattn
