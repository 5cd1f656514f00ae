// The row worker: one warp's share of decode attention over the sequences' own
// keys or their selected blocks, for sm_103a.  It runs on every warp of
// decode_rows_kernel (decode_rows.cu) and of the own keys' CTAs of
// decode_shared_kernel; decode_lists_kernel takes its tiles and its state, and
// shares the work its own way.
//
//   o_h = sum_j p_hj v_j / (sum_j p_hj + exp(sink_h)),  p_hj = exp(scale q_h . k_j)
//
// over a sequence's list of keys, the G query heads of a key/value head
// together: 4 d bytes per key against 4 d G FLOPs, so HBM-bound, and on the
// CUDA cores issue-bound from G = 4 on (decode.cu).  The products run on
// warp-level matrix instructions with the keys as the tall operand, so that
// no row of a 16 x 8 x 16 product is padding at G = 8 (a tcgen05 product would
// spend a 128-row tile on these rows):
//   S^T = K Q^T   16 keys x 8 heads,  K rows by ldmatrix, Q^T kept in registers
//   O^T += V^T P^T   16 dims x 8 heads,  V by transposing ldmatrix; P^T is S^T's
//                 register layout turned by movmatrix
// so that a head's scores, running maximum and O columns sit in the same
// lanes.
//
// Work: the lists of all (sequence, key/value head) groups g, laid end to end
// in tiles of decode_rows_tile keys, are cut into equal shares, warp w taking
// tiles [w * per, (w + 1) * per): every SM streams the same amount whatever
// the lengths are.  A share crosses group borders; each piece of a group that
// a warp has worked through becomes one state (reference m, sum l, O
// unnormalised) in slot w + g, which no other piece has, as w or g (or both)
// grows from one piece to the next.  The group's first tile's number goes to
// group_start[g], from which decode_merge_kernel finds its pieces.
//
// Loads: each warp has its own ring of tiles (128-byte-swizzled TMA boxes of
// 16 keys x 64 columns) and refills a stage itself after reading it, across
// group borders: the only waits are for landed copies.
//
// Rows of a tile that hold no key of the list (past the sequence's end, an
// unused list entry) may hold anything: their scores are replaced by -inf and
// their value rows by zeros before the product, so that what a cache holds
// there never reaches a result.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_ops.h"
#include "kernel_params.h"
#include "ptx.cuh"

namespace mattn {
namespace rows {

template <int D>
struct Geo {
  static constexpr int TK = decode_rows_tile(D), MT = TK / 16;
  static constexpr int kChunks = D / 64;             // 64-column boxes of a row
  static constexpr int kChunk = TK * 128;            // bytes of one box column
  static constexpr int kTensor = kChunks * kChunk;   // K or V of a tile
  static constexpr int kStage = 2 * kTensor;         // 8 KB; 16 KB at d = 256
  static constexpr int NS = 2;                       // stages per warp
  static constexpr uint32_t kAll = TK == 32 ? 0xffffffffu : ((1u << (TK & 31)) - 1u);
  static constexpr int kRing = NS * kStage;          // bytes per warp
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
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// A word of a CTA of this cluster, at this CTA's address p.
__device__ __forceinline__ float cluster_ld(const float* p, uint32_t rank) {
  uint32_t a;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
  return x;
}

__device__ __forceinline__ int cached_keys(const DecodeRowsParams& p, int b) {
  const int len = p.seq_lens ? __ldg(p.seq_lens + b) : p.L;
  return len < 0 ? 0 : (len > p.L ? p.L : len);
}
// Tiles of each of sequence b's lists.
template <int D>
__device__ __forceinline__ int list_tiles(const DecodeRowsParams& p, int len) {
  constexpr int TK = Geo<D>::TK;
  return p.ids ? p.list_tiles : (len + TK - 1) / TK;
}

// One warp's running state of one (sequence, key/value head)'s query heads.
template <int D, int NT>
struct State {
  using S = Geo<D>;
  static constexpr int TK = S::TK, MT = S::MT;
  float m[NT][2], l[NT][2], o[NT][D / 16][4];
  uint32_t qf[NT][D / 16][2];  // queries as B operands: k = dims, n = heads

  // Head columns 2 (lane % 4) + e of each group of eight are this lane's.
  __device__ __forceinline__ void begin(const void* q, int64_t bh0, int G) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + (lane >> 2);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(reinterpret_cast<const __nv_bfloat16*>(q) +
                                                              (bh0 + (g < G ? g : 0)) * D) + (lane & 3);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        qf[nt][i][0] = g < G ? __ldg(src + i * 8) : 0u;
        qf[nt][i][1] = g < G ? __ldg(src + i * 8 + 4) : 0u;
      }
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
    }
  }

  // The sums over a tile's keys end up spread over the lanes of a head column:
  // the whole sums, on all of them.
  __device__ __forceinline__ float sum(int nt, int e) const {
    float s = l[nt][e];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
  }

  // Adds a landed tile: ks, vs are the lane's addresses of its K and V rows (see
  // lane_k, lane_v), v_rows the V tile, mask (not 0) the rows that hold a key.
  __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, uint8_t* v_rows, uint32_t mask, float scale_log2) {
    const int lane = threadIdx.x & 31;
    if (mask != S::kAll) {
      // value rows without a key: zeros (their weights are 0, and 0 x NaN is NaN)
      for (int r = 0; r < TK; ++r) {
        if ((mask >> r) & 1u) continue;
        for (int i = lane; i < S::kChunks * 8; i += 32)
          *reinterpret_cast<uint4*>(v_rows + (i >> 3) * S::kChunk + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    // S^T: four accumulators per tile so that neighbouring products do not wait on each other
    float s[NT][MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float acc[NT][4][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nt][a][j] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4];
        ldsm4(a, (ks ^ ((2 * i & 7) << 4)) + (i >> 2) * S::kChunk + mt * 2048);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ptx::mma16816(acc[nt][i & 3], a, qf[nt][i][0], qf[nt][i][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][mt][j] = (acc[nt][0][j] + acc[nt][1][j]) + (acc[nt][2][j] + acc[nt][3][j]);
    }
    if (mask != S::kAll) {
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
    // online softmax per head column: the reference m in the log2 domain
    float mx[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(s[nt][0][e], s[nt][0][e + 2]);
        if (MT == 2) x = fmaxf(x, fmaxf(s[nt][MT - 1][e], s[nt][MT - 1][e + 2]));
        mx[nt][e] = x;
      }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[nt][e] = fmaxf(m[nt][e], mx[nt][e] * scale_log2);
        moved = moved || mx[nt][e] != m[nt][e];
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          alpha[e] = m[nt][e] == mx[nt][e] ? 1.f : ptx::ex2(m[nt][e] - mx[nt][e]);
          m[nt][e] = mx[nt][e];
          l[nt][e] *= alpha[e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[nt][i][0] *= alpha[0];
          o[nt][i][1] *= alpha[1];
          o[nt][i][2] *= alpha[0];
          o[nt][i][3] *= alpha[1];
        }
      }
    }
    uint32_t pf[NT][MT][2], pg[NT][MT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
        float sum = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          s[nt][mt][e] = ptx::ex2(fmaf(s[nt][mt][e], scale_log2, -ref));
          s[nt][mt][e + 2] = ptx::ex2(fmaf(s[nt][mt][e + 2], scale_log2, -ref));
          sum += s[nt][mt][e] + s[nt][mt][e + 2];
        }
        l[nt][e] += sum;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        // P^T as B operand (k = keys, n = heads), each weight in two parts: one
        // alone would add an error as large as the output's own rounding, and the
        // tensor cores idle here
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t hi, lo;
          two_bf16(s[nt][mt][2 * r], s[nt][mt][2 * r + 1], &hi, &lo);
          pf[nt][mt][r] = movm_t(hi);
          pg[nt][mt][r] = movm_t(lo);
        }
      }
    }
    // O^T += V^T P^T, four pieces' first parts before their second ones, which
    // add into the same sums
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i0 = 0; i0 < D / 16; i0 += 4) {
        uint32_t a[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ldsm4_t(a[i], (vs ^ ((2 * (i0 + i) & 7) << 4)) + ((i0 + i) >> 2) * S::kChunk + mt * 2048);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ptx::mma16816(o[nt][i0 + i], a[i], pf[nt][mt][0], pf[nt][mt][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) ptx::mma16816(o[nt][i0 + i], a[i], pg[nt][mt][0], pg[nt][mt][1]);
        }
      }
    }
  }
};

// 16-byte piece u = 2 i + e of row r lies at piece (u & 7) ^ (r & 7) of the
// row's 128 bytes in chunk u >> 3: the lane's row and e make one address, from
// which i's is an exclusive or and a constant away.
__device__ __forceinline__ uint32_t lane_k(uint32_t tile) {
  const int lane = threadIdx.x & 31;
  return tile + ((lane & 7) + ((lane >> 3) & 1) * 8) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
}
__device__ __forceinline__ uint32_t lane_v(uint32_t tile) {
  const int lane = threadIdx.x & 31;
  return tile + ((lane & 7) + (lane >> 4) * 8) * 128 + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
}

// Loads a tile of (sequence, key/value head) bkv into `stage` of a warp's ring, a
// lane per copy: boxes x < MT start at key pos[x] and cnt[x] of their rows hold
// keys (a box without any is not loaded); returns the rows that do.
template <int D>
__device__ __forceinline__ uint32_t issue_tile(const DecodeRowsParams& p, uint8_t* ring, uint64_t* full, int stage,
                                               int bkv, const int (&pos)[Geo<D>::MT], const int (&cnt)[Geo<D>::MT]) {
  using S = Geo<D>;
  constexpr int MT = S::MT, kPer = S::kChunks * 2;  // copies per box
  const int lane = threadIdx.x & 31;
  uint32_t mask = 0, bytes = 0;
#pragma unroll
  for (int x = 0; x < MT; ++x) {
    mask |= ((1u << cnt[x]) - 1u) << (16 * x);
    bytes += cnt[x] > 0 ? kPer * 2048u : 0u;
  }
  if (lane == 0) ptx::mbar_arrive_expect_tx(full + stage, bytes);
  __syncwarp();
  const int x = lane / kPer, ch = (lane >> 1) % S::kChunks, tensor = lane & 1;
  const int n = MT == 2 && x ? cnt[MT - 1] : cnt[0], at = MT == 2 && x ? pos[MT - 1] : pos[0];
  if (x < MT && n > 0 &&
      debug_check(p.err, at >= 0 && at < p.L && bkv >= 0 && bkv < p.B * p.H_kv && stage < S::NS, kSiteLoad))
    ptx::tma_load_3d(ring + stage * S::kStage + tensor * S::kTensor + ch * S::kChunk + x * 2048, tensor ? &p.tv : &p.tk,
                     full + stage, ch * 64, at, bkv);
  return mask;
}

// Waits for a warp's stage; false if the wait gave up (the abort flag is then
// raised, and copies already in flight have landed before the shared memory goes).
__device__ __forceinline__ bool await(const DecodeRowsParams& p, uint64_t* bar, uint32_t parity,
                                      volatile int* abort_flag) {
  const bool got = ptx::mbar_wait(bar, parity, p.timeout_ns, abort_flag);
  if (__all_sync(0xffffffffu, got)) return true;
  if ((threadIdx.x & 31) == 0) {
    *abort_flag = 1;
    atomicOr(p.err, kErrProducer);
  }
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 0; it < 0x10000000u && ptx::globaltimer_ns() - t0 < 2000000ull; ++it) { }
  return false;
}

// Where a tile lies: sequence b, key/value head h, tile t of its list.
struct Cursor {
  int b, h, t, tiles, len;
};
// The same for the tile to load, with its place in a block list: entry j, box
// r of its box16, the entry's block and the next one's (loaded ahead).
struct Feed : Cursor {
  int j, r, id, next, blocks;  // blocks: the sequence's blocks that hold cached keys
};

// One warp's share.  ring: Geo<D>::kRing bytes, 1024-byte aligned; full: its
// NS barriers (one arrival each), initialised and visible; w of W warps.
// Returns false if a wait gave up (the abort flag is then raised).
// NT: groups of eight query heads.
template <int D, int NT>
__device__ __forceinline__ bool work(const DecodeRowsParams& p, int w, int W, uint8_t* ring, uint64_t* full,
                                     volatile int* abort_flag) {
  using G_ = Geo<D>;
  constexpr int MT = G_::MT, NS = G_::NS;
  static_assert(NS == 2, "the masks of the stages are two registers");
  const int lane = threadIdx.x & 31;
  const int G = p.H / p.H_kv;

  // this warp's share of all lists' tiles
  int total;
  if (p.ids || !p.seq_lens) {
    total = p.B * p.H_kv * list_tiles<D>(p, p.L);
  } else {
    int sum = 0;
#pragma unroll 4
    for (int b = lane; b < p.B; b += 32) sum += list_tiles<D>(p, cached_keys(p, b));
    total = __reduce_add_sync(0xffffffffu, sum) * p.H_kv;
  }
  const int per = total ? (total - 1) / W + 1 : 1;  // (total: to 2^31 - 1)
  if (w == 0 && lane == 0) p.group_start[p.B * p.H_kv] = per;
  const int64_t first = (int64_t)w * per;
  if (first >= total) return true;
  const int x0 = (int)first, n_mine = total - x0 < per ? total - x0 : per;

  Cursor c;
  if (p.ids || !p.seq_lens) {
    c.tiles = list_tiles<D>(p, p.L);
    const int g = x0 / c.tiles;
    c.t = x0 - g * c.tiles;
    c.b = g / p.H_kv;
    c.h = g - c.b * p.H_kv;
    c.len = cached_keys(p, c.b);
  } else {
    // the sequence that holds tile x0: running sums of 32 sequences at a time
    int before = 0, b0 = 0, mine, incl;
    uint32_t past;
    for (;; b0 += 32) {
      mine = b0 + lane < p.B ? list_tiles<D>(p, cached_keys(p, b0 + lane)) * p.H_kv : 0;
      incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      past = __ballot_sync(0xffffffffu, before + incl > x0);
      if (past || b0 + 32 >= p.B) break;  // (x0 < total: some sequence is past it)
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int at = __ffs(past) - 1;
    const int start = before + __shfl_sync(0xffffffffu, incl - mine, at);
    c.b = b0 + at;
    c.len = cached_keys(p, c.b);
    c.tiles = list_tiles<D>(p, c.len);
    c.h = (x0 - start) / c.tiles;
    c.t = x0 - start - c.h * c.tiles;
  }
  auto advance = [&](Cursor& k) -> bool {  // true: to another list
    if (++k.t < k.tiles) return false;
    k.t = 0;
    if (++k.h < p.H_kv) return true;
    k.h = 0;
    do {
      ++k.b;
      k.len = k.b < p.B ? cached_keys(p, k.b) : 0;
      k.tiles = list_tiles<D>(p, k.len);
    } while (k.b < p.B && k.tiles == 0);
    return true;
  };
  auto entry = [&](const Feed& f, int j) {
    return j < p.top_k ? __ldg(p.ids + (int64_t)(f.b * p.H_kv + f.h) * p.top_k + j) : -1;
  };
  auto enter_list = [&](Feed& f) {  // at tile f.t
    if (!p.ids) return;
    f.j = f.t * MT / p.box16;
    f.r = f.t * MT - f.j * p.box16;
    f.id = entry(f, f.j);  // (loaded beside the sequence's length)
    f.next = entry(f, f.j + 1);
    f.blocks = (f.len + p.block - 1) / p.block;
  };
  auto feed_on = [&](Feed& f) {
    if (advance(f)) {
      enter_list(f);
    } else if (p.ids) {
      for (f.r += MT; f.r >= p.box16; f.r -= p.box16) {
        ++f.j;
        f.id = f.next;
        f.next = entry(f, f.j + 1);
      }
    }
  };
  // Box x of the feed's tile (16 keys): the position of its first key; *cnt of
  // its rows hold keys (the first ones: a box lies inside one block).
  auto box_at = [&](const Feed& f, int x, int* cnt) -> int {
    int pos = (f.t * MT + x) << 4;
    if (p.ids) {
      const bool over = f.r + x >= p.box16;  // (x < MT <= 2: into the next entry at most)
      const int id = over ? f.next : f.id, r = over ? f.r + x - p.box16 : f.r + x;
      pos = (uint32_t)id < (uint32_t)f.blocks ? id * p.block + (r << 4) : f.len;
    }
    const int left = f.len - pos;
    *cnt = left < 0 ? 0 : (left < 16 ? left : 16);
    return pos;
  };
  auto issue = [&](const Feed& f, int stage) -> uint32_t {
    int pos[MT], cnt[MT];
#pragma unroll
    for (int x = 0; x < MT; ++x) pos[x] = box_at(f, x, &cnt[x]);
    const int bkv = f.b * p.H_kv + f.h;
    // the list's queries into L1, for the state that begins two tiles later
    if (f.t == 0 && lane * 64 < G * D)
      ptx::prefetch_l1(reinterpret_cast<const __nv_bfloat16*>(p.q) + (int64_t)bkv * G * D + lane * 64);
    return issue_tile<D>(p, ring, full, stage, bkv, pos, cnt);
  };

  State<D, NT> st;
  auto end_group = [&](int g) {  // the piece's state
    const int64_t slot = (int64_t)w + g;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float s = st.sum(nt, e);
        const int head = nt * 8 + (lane & 3) * 2 + e;
        if (head < G) {
          if (lane < 4) *reinterpret_cast<float2*>(p.part_ml + (slot * G + head) * 2) = make_float2(st.m[nt][e], s);
          float* dst = p.part_o + (slot * G + head) * D + (lane >> 2);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            dst[i * 16] = st.o[nt][i][e];
            dst[i * 16 + 8] = st.o[nt][i][e + 2];
          }
        }
      }
  };

  Feed f;  // the last tile loaded
  static_cast<Cursor&>(f) = c;
  f.j = f.r = f.id = f.next = f.blocks = 0;
  enter_list(f);
  uint32_t masks[2] = {0, 0};
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (n < n_mine) {
      if (n) feed_on(f);
      if (n || p.selftest != 1) masks[n] = issue(f, n);
    }
  const uint32_t at_k = lane_k(ptx::smem_addr(ring)), at_v = lane_v(ptx::smem_addr(ring) + G_::kTensor);
  for (int n = 0; n < n_mine; ++n) {
    if (n == 0 || c.t == 0) {
      if (c.t == 0 && lane == 0) p.group_start[c.b * p.H_kv + c.h] = x0 + n;
      st.begin(p.q, (int64_t)c.b * p.H + c.h * G, G);
    }
    const int stage = n & 1;
    const uint32_t mask = stage ? masks[1] : masks[0];
    if (!await(p, full + stage, (n >> 1) & 1, abort_flag)) return false;
    if (mask)  // warp-uniform
      st.step(at_k + stage * G_::kStage, at_v + stage * G_::kStage, ring + stage * G_::kStage + G_::kTensor, mask,
              p.scale_log2);
    __syncwarp();
    if (n + NS < n_mine) {
      if (mask != G_::kAll) ptx::fence_proxy_async_shared();  // the zeros above before the copy that overwrites them
      __syncwarp();
      feed_on(f);
      const uint32_t x = issue(f, stage);
      if (stage) masks[1] = x;
      else masks[0] = x;
    }
    const int g = c.b * p.H_kv + c.h;
    const bool last = n + 1 == n_mine;
    if (last || c.t + 1 == c.tiles) end_group(g);
    if (!last) advance(c);
  }
  return true;
}

}  // namespace rows
}  // namespace mattn
