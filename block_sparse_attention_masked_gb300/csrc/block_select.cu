// Block means of a key cache and the choice of the blocks a decode query
// attends, for sm_103a.
//
//   mean_n  = (1 / |n|) sum of the cached keys of block n, rounded to bf16
//   score_n = max over the G query heads of the key/value head of q_g . mean_n
//
// and of the sequence's blocks the first and the newest ones (as many as the
// caller keeps) and then those of highest score, lowest index first on equal
// scores, top_k in all, in ascending order.
//
// block_means_kernel: 16 bytes per lane, 32-bit sums; it reads every key of a
// block that holds new ones once and is HBM-bound.  A warp per block where there
// are blocks for all SMs (8 caches of 32K keys, 403 MB: 64 us, 81 with four
// warps per block and their meeting), four where there are few: a quarter of a
// 64-key block is one batch of loads, so that a decode step's update waits for
// the memory once and not four times (64 requests: 4.2 us, 5.2 with one).
//
// Selection.  The choice is that of exact arithmetic on the bf16 means and
// queries, so that it does not depend on how a product was summed:
//   1. Scores by matrix instructions with fp32 sums, and e_n, a bound of each
//      one's error: |sum of d rounded products - exact| <= u d' sum |q_c k_c| <=
//      u d' |q| |k_n|; with d / 16 <= 16 sums of 16 products each, u d' <= 2^-17
//      even if each of them loses 2^-21 of its terms' magnitudes, and 2^-15 is
//      used.  Lanes load 16 bytes of a mean's row straight into operand
//      registers: the order of the dims inside a product is free as long as the
//      queries use the same one, so the means pass through no shared memory.
//      One pass over the means: HBM-bound.
//   2. The k-th largest score T: the scores' range is cut into 512 even bins,
//      counted, and the bin that holds T ranked by one warp (or cut again, where
//      it holds more than 32).  Every set of k scores bounds the exact k-th score
//      from below by the least of its members' score - e, and every set of
//      n - k + 1 from above by the most of score + e; applied to {score >= T} and
//      {score <= T} this gives lo <= exact k-th <= hi.  A block is in if
//      score - e > hi, out if score + e < lo; the few between are formed again in
//      64 bits (products of two bf16 are exact there) and ranked.
// One launch: a cluster of up to eight CTAs scores one (sequence, key/value
// head)'s blocks, and its first CTA, after the cluster's barrier, selects with
// the scores in shared memory (up to 6,144 blocks; more are read from L2).  The
// selection's stages are short and end in a sum over the threads, so that its
// time is what each warp issues once: eight of the sixteen warps go on to it.
// (128 groups of 2,048 blocks of 128, 50 MB: 21.2 us, the means read after 6 to
// 15: of the 256 CTAs 48 have an SM to themselves and the others share one in pairs.  The scores as a grid of small CTAs
// before the selection: 23.3.  The scores straight to the first CTA's shared memory:
// 21.5.  Prefetching a warp's later steps to L2: 1.2 us later.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_ops.h"
#include "ptx.cuh"

namespace mattn {
namespace {

__device__ __forceinline__ float bfl(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bfh(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// ------------------------------------------------------------ block means
constexpr int kMeanWarps = 4;

// PARTS: warps per block.
template <int D, int PARTS>
__global__ void __launch_bounds__(32 * kMeanWarps) block_means_kernel(const __grid_constant__ BlockMeansParams p) {
  constexpr int LPR = D / 8;          // lanes of a key row
  constexpr int RPI = 32 / LPR;       // keys per warp load
  constexpr int U = 8;                // loads in flight per lane
  constexpr int kMeanBlocks = kMeanWarps / PARTS;
  static_assert(kMeanBlocks * PARTS == kMeanWarps, "whole blocks in a CTA");
  __shared__ float sums[PARTS > 1 ? kMeanWarps : 1][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = warp / PARTS, part = warp % PARTS;
  const int64_t w = (int64_t)blockIdx.x * kMeanBlocks + slot;
  const int64_t row = w / p.span;     // (sequence, key/value head)
  int n = 0;                          // cached keys of the block, 0: not one to form
  after_previous();
  int64_t blk = 0;
  if (row < (int64_t)p.B * p.H_kv) {
    const int b = (int)(row / p.H_kv);
    int len = p.seq_lens ? p.seq_lens[b] : p.L;
    len = len < 0 ? 0 : (len > p.L ? p.L : len);
    int first = p.first ? p.first[b] : 0;
    first = first < 0 ? 0 : first;
    const int64_t end64 = (int64_t)first + p.max_new;
    const int end = end64 < len ? (int)end64 : len;  // new keys: [first, end)
    blk = first / p.block + w % p.span;
    const int64_t k0 = blk * p.block;
    if (first < end && k0 < end && blk < p.n_blocks) n = len - k0 < p.block ? (int)(len - k0) : p.block;
  }
  const int sub = lane % LPR, r0 = lane / LPR;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  const int share = p.block / PARTS, lo = part * share, hi = lo + share < n ? lo + share : n;
  if (lo < hi) {
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.k) +
                                                      (row * p.L + blk * p.block) * D) + sub;
    for (int r = lo + r0; r < hi; r += RPI * U) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] = r + u * RPI < hi ? __ldg(src + (int64_t)(r + u * RPI) * LPR) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        acc[0] += bfl(x[u].x); acc[1] += bfh(x[u].x);
        acc[2] += bfl(x[u].y); acc[3] += bfh(x[u].y);
        acc[4] += bfl(x[u].z); acc[5] += bfh(x[u].z);
        acc[6] += bfl(x[u].w); acc[7] += bfh(x[u].w);
      }
    }
  }
#pragma unroll
  for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
  const float c = (float)n;
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.means) + (row * p.n_blocks + blk) * D;
  if constexpr (PARTS == 1) {
    if (lane < LPR && n > 0)
      reinterpret_cast<uint4*>(dst)[sub] =
          make_uint4(ptx::pack_bf16x2(acc[0] / c, acc[1] / c), ptx::pack_bf16x2(acc[2] / c, acc[3] / c),
                     ptx::pack_bf16x2(acc[4] / c, acc[5] / c), ptx::pack_bf16x2(acc[6] / c, acc[7] / c));
    return;
  }
  if (lane < LPR) {
    *reinterpret_cast<float4*>(&sums[warp][sub * 8]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    *reinterpret_cast<float4*>(&sums[warp][sub * 8 + 4]) = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  __syncthreads();
  // the block's dims over its warps, two values per lane
  if (n > 0)
    for (int d = (part * 32 + lane) * 2; d < D; d += PARTS * 64) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        x += sums[slot * PARTS + k][d];
        y += sums[slot * PARTS + k][d + 1];
      }
      reinterpret_cast<uint32_t*>(dst)[d / 2] = ptx::pack_bf16x2(x / c, y / c);
    }
}

// ------------------------------------------------------------ selection
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kPick = 256;       // threads that select
constexpr int kPickWarps = kPick / 32;
constexpr int kSelKept = 6144;   // scores kept in shared memory
constexpr int kBatch = 8;        // scores a thread works on at once
constexpr int kCutBins = 2 * kPick;
constexpr int kCuts = 8;         // at most: what is left then goes to the 64-bit scores
constexpr int kDigit = 11;
constexpr int kBins = 1 << kDigit;
constexpr int kSmallBand = 256;  // candidates ranked in shared memory; more go through the digits again
constexpr float kScoreErr = 3.0517578125e-05f;  // 2^-15 (see above)

// 32 bytes of a mean's row (a whole 128-byte line by four lanes).
__device__ __forceinline__ void ld32(const uint4* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ float sq2(uint32_t x, float s) { return fmaf(bfl(x), bfl(x), fmaf(bfh(x), bfh(x), s)); }
__device__ __forceinline__ float sq8(const uint4& x, float s) {
  return sq2(x.x, sq2(x.y, sq2(x.z, sq2(x.w, s))));
}

// Keys that order like the floats; NaN is taken as -inf.
__device__ __forceinline__ uint32_t key32(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unkey32(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ unsigned long long key64(double x) {
  if (x != x) x = -INFINITY;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ int blocks_of(const DecodeSelectParams& p, int b) {
  if (!p.seq_lens) return p.n_blocks;
  const int len = p.seq_lens[b];
  const int64_t n = len <= 0 ? 0 : ((int64_t)len + p.block - 1) / p.block;
  return n < p.n_blocks ? (int)n : p.n_blocks;
}

static_assert(kSmallBand * 16 * sizeof(double) <= kSelKept * sizeof(uint2), "the products of a band take the scores' place");
constexpr uint32_t kKeyMin = 0x00800000u, kKeyMax = 0xff7fffffu;  // keys of the least and largest finite float

struct SelShared {
  uint4 q[2][8][32];                       // the group's queries as operands: [group of 8 heads][32 dims][lane]
  uint32_t hist[kBins];
  uint32_t member[kSelectMaxBlocks / 32];  // blocks chosen
  uint32_t band[kSelectMaxBlocks / 32];    // blocks between lo and hi
  double val[kSmallBand];
  int idx[kSmallBand];
  uint32_t wsum[kPickWarps];
  uint2 bound[kPickWarps];
  uint4 range[kPickWarps];
  uint32_t list[32];
  int n_list;
  uint32_t digit, above;
  int n_in, n_band;
  uint2 kept[kSelKept];                    // Score
};

// Barrier of the threads that select.
__device__ __forceinline__ void pick_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kPick) : "memory"); }

// Exclusive prefix sum over the selecting threads; *total gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* wsum, uint32_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  pick_sync();
  if (lane == 31) wsum[warp] = x;
  pick_sync();
  const uint32_t w = lane < kPickWarps ? wsum[lane] : 0u;
  *total = __reduce_add_sync(0xffffffffu, w);
  return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u) + x - v;
}

// The bin of the histogram's BINS, from the top, at which the count from above
// reaches `want` (1-based): sh->digit = the bin, sh->above = entries in higher ones.
template <int BINS>
__device__ __forceinline__ void pick_digit(SelShared* sh, uint32_t want) {
  constexpr int PER = BINS / kPick;
  // thread t holds the bins of descending order t * PER ...
  uint32_t c[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = sh->hist[BINS - 1 - (threadIdx.x * PER + i)];
    sum += c[i];
  }
  uint32_t total;
  uint32_t before = block_scan(sum, sh->wsum, &total);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (before < want && before + c[i] >= want) {
      sh->digit = BINS - 1 - (threadIdx.x * PER + i);
      sh->above = before;
    }
    before += c[i];
  }
  pick_sync();
}

// Scores of the blocks [0, n) of one group, shared by the `ctas` CTAs of a
// cluster: a warp takes 16 blocks at a time, block rows the tall operand, the
// group's heads (NT groups of eight) the other.
template <int D, int NT>
__device__ __forceinline__ void score_blocks(const DecodeSelectParams& p, SelShared* sh, int b, int kvh, int rank,
                                             int ctas) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.H / p.H_kv;
  const int r = lane >> 2, j = lane & 3;
  const int64_t row = (int64_t)b * p.H_kv + kvh;
  // operand i, lane j of a row: 16-byte pieces 8 (i / 2) + 2 j + i % 2
  const uint4* mean = reinterpret_cast<const uint4*>(p.means) + row * p.n_blocks * (D / 8) + 2 * j;
  uint4 x[D / 32], y[D / 32];
  auto load = [&](int t, int n) {
    const int r0 = t * 16 + r, r1 = r0 + 8;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = y[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) {
      if (r0 < n) ld32(mean + (int64_t)r0 * (D / 8) + i * 4, x[i], x[i + 1]);
      if (r1 < n) ld32(mean + (int64_t)r1 * (D / 8) + i * 4, y[i], y[i + 1]);
    }
  };
  int t = rank * kSelWarps + warp;
  load(t, p.n_blocks);  // in flight while the sequence's length and the queries arrive
  for (int k = threadIdx.x; k < NT * (D / 32) * 32; k += kSelThreads) {
    const int l = k & 31, i = (k >> 5) % (D / 32), nt = (k >> 5) / (D / 32), g = nt * 8 + (l >> 2);
    sh->q[nt][i][l] = g < G ? __ldg(reinterpret_cast<const uint4*>(p.q) + ((int64_t)b * p.H + kvh * G + g) * (D / 8) +
                                    (i >> 1) * 8 + (l & 3) * 2 + (i & 1))
                            : make_uint4(0, 0, 0, 0);
  }
  const int n = blocks_of(p, b);
  __syncthreads();
  float qq = 0.f;  // the longest query's squared length
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = sq8(sh->q[nt][i][lane], s);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    qq = fmaxf(qq, s);
  }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) qq = fmaxf(qq, __shfl_xor_sync(0xffffffffu, qq, off));
  const float err = kScoreErr * sqrtf(qq + 1e-40f);
  for (; t * 16 < n; t += ctas * kSelWarps, load(t, n)) {
    const int r0 = t * 16 + r, r1 = r0 + 8;
    float acc[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[nt][a][k] = 0.f;
    float sx = 0.f, sy = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 q = sh->q[nt][i][lane];
        ptx::mma16816(acc[nt][0], {x[i].x, y[i].x, x[i].y, y[i].y}, q.x, q.y);
        ptx::mma16816(acc[nt][1], {x[i].z, y[i].z, x[i].w, y[i].w}, q.z, q.w);
      }
      sx = sq8(x[i], sx);
      sy = sq8(y[i], sy);
    }
    // heads of this lane: 2 j, 2 j + 1 (of each eight); rows r0 and r1
    const float nan = __int_as_float(0x7fffffff);
    float s0 = -INFINITY, s1 = -INFINITY;
    bool nan0 = false, nan1 = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (nt * 8 + 2 * j + e < G) {
          const float u = acc[nt][0][e] + acc[nt][1][e], v = acc[nt][0][e + 2] + acc[nt][1][e + 2];
          nan0 = nan0 || u != u;
          nan1 = nan1 || v != v;
          s0 = fmaxf(s0, u);
          s1 = fmaxf(s1, v);
        }
    if (nan0) s0 = nan;
    if (nan1) s1 = nan;
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, s0, off), v = __shfl_xor_sync(0xffffffffu, s1, off);
      s0 = u != u || s0 != s0 ? nan : fmaxf(s0, u);
      s1 = v != v || s1 != s1 ? nan : fmaxf(s1, v);
      sx += __shfl_xor_sync(0xffffffffu, sx, off);
      sy += __shfl_xor_sync(0xffffffffu, sy, off);
    }
    if (j == 0) {
      // (the small terms cover squares and products that underflow)
      Score* dst = p.scores + row * p.n_blocks;
      if (r0 < n) dst[r0] = Score{key32(s0), fmaf(err, sqrtf(sx + 1e-40f), 1e-36f)};
      if (r1 < n) dst[r1] = Score{key32(s1), fmaf(err, sqrtf(sy + 1e-40f), 1e-36f)};
    }
  }
}

// A cluster per (sequence, key/value head).
template <int D, int NT>
__global__ void __launch_bounds__(kSelThreads, D == 256 || NT == 2 ? 1 : 2)
    decode_select_kernel(const __grid_constant__ DecodeSelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelShared* sh = reinterpret_cast<SelShared*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % p.ctas, bkv = blockIdx.x / p.ctas;
  const int b = bkv / p.H_kv, kvh = bkv % p.H_kv, G = p.H / p.H_kv;
  after_previous();
  // (before the length is known: where every block fits, the scores go unread)
  if (p.n_blocks > p.top_k) score_blocks<D, NT>(p, sh, b, kvh, rank, p.ctas);
  const int n = blocks_of(p, b);
  const int words = (n + 31) / 32;
  // blocks kept whatever their score: [0, f0) and [f1, n)
  const int f0 = p.keep_first < n ? p.keep_first : n;
  const int f1 = n - p.keep_recent > f0 ? n - p.keep_recent : f0;
  const int rest = f1 - f0;                          // blocks that compete
  const int want = p.top_k - f0 - (n - f1);          // places left for them (>= 0: checked on the host)
  const bool choose = want > 0 && rest > want;       // the same in all CTAs of the cluster
  if (rank == 0) {
    for (int w = tid; w < words; w += kSelThreads) {
      // the kept blocks' bits; all of them when every block fits
      uint32_t bits = 0;
      if (rest <= want) {
        bits = n - w * 32 >= 32 ? 0xffffffffu : (1u << (n - w * 32)) - 1u;
      } else {
        for (int i = w * 32; i < f0 && i < w * 32 + 32; ++i) bits |= 1u << (i & 31);
        for (int i = f1 > w * 32 ? f1 : w * 32; i < n && i < w * 32 + 32; ++i) bits |= 1u << (i & 31);
      }
      sh->member[w] = bits;
      sh->band[w] = 0;
    }
    if (tid == 0) sh->n_in = sh->n_band = 0;
  }
  if (choose && p.ctas > 1) {
    // every CTA's scores before the first one's selection
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (rank || tid >= kPick) return;
  if (choose) {
    const uint2* far = reinterpret_cast<const uint2*>(p.scores + (int64_t)bkv * p.n_blocks + f0);
    const bool kept = rest <= kSelKept;
    // fn(place, its score, whether there is one) over this thread's places, eight
    // loaded at once: fn has no branch that its lanes take apart, so that the
    // eight overlap
    auto each = [&](bool near, auto&& fn) {
#pragma unroll 1
      for (int base = tid; base < rest; base += kPick * kBatch) {
        uint2 u[kBatch];
        if (near) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int i = base + j * kPick;
            u[j] = sh->kept[i < rest ? i : 0];
          }
        } else {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int i = base + j * kPick;
            u[j] = __ldcg(far + (i < rest ? i : 0));
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) fn(base + j * kPick, u[j].x, __uint_as_float(u[j].y), base + j * kPick < rest);
      }
    };
    // the interval of the want-th largest score: keys [from, to]
    uint32_t from = 0, to = 0xffffffffu, above = 0;  // above: scores past `to`
    int left = rest;
    float emax = 0.f;  // the largest bound of an error
    float bin_width = 0.f;
    bool unknown = false;  // some score or error is not finite
#pragma unroll 1
    for (int cut = 0; cut < kCuts && left > 1; ++cut) {
      // the finite scores' range inside the interval (and the scores to shared memory)
      const uint32_t first = from > kKeyMin ? from : kKeyMin, span = (to < kKeyMax ? to : kKeyMax) - first;
      const bool some = to >= kKeyMin && from <= kKeyMax;
      uint32_t kmin = 0xffffffffu, kmax = 0;
      each(kept && cut > 0, [&](int i, uint32_t k, float err, bool there) {
        if (kept && cut == 0 && there) sh->kept[i] = make_uint2(k, __float_as_uint(err));
        const bool in = some && there && k - first <= span;
        kmin = min(kmin, in ? k : 0xffffffffu);
        kmax = max(kmax, in ? k : 0u);
        const bool fine = k - kKeyMin <= kKeyMax - kKeyMin && err < INFINITY;
        emax = fmaxf(emax, there && fine ? err : 0.f);
        unknown = unknown || (there && !fine);
      });
      kmin = __reduce_min_sync(0xffffffffu, kmin);
      kmax = __reduce_max_sync(0xffffffffu, kmax);
      const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(emax));  // (>= 0: ordered as it is)
      const uint32_t u = __any_sync(0xffffffffu, unknown);
      if (lane == 0) sh->range[warp] = make_uint4(kmin, kmax, e, u);
      sh->hist[tid] = sh->hist[tid + kPick] = 0;
      if (tid == 0) sh->n_list = 0;
      pick_sync();
      const uint4 range = lane < kPickWarps ? sh->range[lane] : make_uint4(0xffffffffu, 0u, 0u, 0u);
      kmin = __reduce_min_sync(0xffffffffu, range.x);
      kmax = __reduce_max_sync(0xffffffffu, range.y);
      emax = __uint_as_float(__reduce_max_sync(0xffffffffu, range.z));
      unknown = __any_sync(0xffffffffu, range.w != 0u);
      if (kmin >= kmax) break;  // equal scores, or none finite
      const float s0 = unkey32(kmin), width = unkey32(kmax) - s0, per = __fdividef((float)(kCutBins - 2), width);
      if (!(width < INFINITY) || !(per < INFINITY) || !(per > 0.f)) break;
      bin_width = width / (float)(kCutBins - 2);
      // a bin of each score, growing with it (infinities at the ends)
      auto bin_of = [&](uint32_t k) {
        return (int)fminf(fmaxf((unkey32(k) - s0) * per, -1.f), (float)(kCutBins - 2)) + 1;
      };
      each(kept, [&](int, uint32_t k, float, bool there) {
        const int bin = bin_of(k);
        if (there && k - from <= to - from) atomicAdd(&sh->hist[bin], 1u);
      });
      pick_sync();
      pick_digit<kCutBins>(sh, (uint32_t)want - above);
      const int bin = (int)sh->digit;
      above += sh->above;
      left = (int)sh->hist[bin];
      // the bin's keys: listed and ranked where they are few, else an interval again
      if (left <= 32) {
        each(kept, [&](int, uint32_t k, float, bool there) {
          if (there && k - from <= to - from && bin_of(k) == bin) sh->list[atomicAdd(&sh->n_list, 1)] = k;
        });
        pick_sync();
        // every warp: the key that fewer than want - above and, with its equals, at least that many pass
        const uint32_t k = lane < left ? sh->list[lane] : 0u;  // (0 is no score's key)
        int more = 0, same = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint32_t o = __shfl_sync(0xffffffffu, k, j);
          more += o > k;
          same += o == k;
        }
        const int rank_ = want - (int)above;
        const uint32_t hit = __ballot_sync(0xffffffffu, lane < left && more < rank_ && more + same >= rank_);
        from = to = __shfl_sync(0xffffffffu, k, __ffs(hit) - 1);
        break;
      }
      uint32_t f = 0xffffffffu, t = 0;
      each(kept, [&](int, uint32_t k, float, bool there) {
        const bool in = there && k - from <= to - from && bin_of(k) == bin;
        f = min(f, in ? k : 0xffffffffu);
        t = max(t, in ? k : 0u);
      });
      f = __reduce_min_sync(0xffffffffu, f);
      t = __reduce_max_sync(0xffffffffu, t);
      if (lane == 0) sh->bound[warp] = make_uint2(f, t);
      pick_sync();
      const uint2 now = lane < kPickWarps ? sh->bound[lane] : make_uint2(0xffffffffu, 0u);
      from = __reduce_min_sync(0xffffffffu, now.x);
      to = __reduce_max_sync(0xffffffffu, now.y);
      pick_sync();  // (the next cut writes the same words)
    }
    // Bounds of the exact want-th score.  One border score (from == to) and errors
    // well below the scores' spacing: itself, give or take the largest error.  Else
    // from the scores' own errors (of a score that is not finite nothing is known).
    float lo, hi;
    const float border = unkey32(from);
    if (from == to && emax <= bin_width && !unknown) {
      lo = border - emax;
      hi = border + emax;
    } else {
      uint32_t klo = 0xffffffffu, khi = 0;
      each(kept, [&](int, uint32_t k, float err, bool there) {
        const float s = unkey32(k);
        const bool fine = fabsf(s) < INFINITY && err < INFINITY;
        const uint32_t down = key32(fine ? s - err : -INFINITY), up = key32(fine ? s + err : INFINITY);
        klo = min(klo, there && k >= from ? down : 0xffffffffu);
        khi = max(khi, there && k <= to ? up : 0u);
      });
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      pick_sync();
      if (lane == 0) sh->bound[warp] = make_uint2(klo, khi);
      pick_sync();
      const uint2 bound = lane < kPickWarps ? sh->bound[lane] : make_uint2(0xffffffffu, 0u);
      lo = unkey32(__reduce_min_sync(0xffffffffu, bound.x));
      hi = unkey32(__reduce_max_sync(0xffffffffu, bound.y));
    }
    int in = 0;
    each(kept, [&](int i, uint32_t k, float err, bool there) {
      const float s = unkey32(k);
      const bool fine = fabsf(s) < INFINITY && err < INFINITY;
      const bool sure = there && fine && s - err > hi, maybe = there && !sure && (!fine || s + err >= lo);
      in += sure;
      if (sure || maybe) {
        const int x = f0 + i;
        atomicOr(sure ? &sh->member[x >> 5] : &sh->band[x >> 5], 1u << (x & 31));
        if (maybe) {
          const int at = atomicAdd(&sh->n_band, 1);
          if (at < kSmallBand) sh->idx[at] = x;
        }
      }
    });
    in = __reduce_add_sync(0xffffffffu, in);
    if (lane == 0 && in) atomicAdd(&sh->n_in, in);
    pick_sync();
    const int band = sh->n_band, need = want - sh->n_in;  // 0 < need <= band
    double* again = p.again + (int64_t)bkv * p.n_blocks;
    // one warp: block i's product with head g in 64 bits; a lane takes D / 32
    // dims, the queries' from the operands in shared memory
    constexpr int VPL = D / 32;
    const int piece = lane * VPL / 8, at = lane * VPL % 8;
    auto dot64 = [&](int i, int g) -> double {
      const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(p.means) +
                                 ((int64_t)bkv * p.n_blocks + i) * D + lane * VPL;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(
                              &sh->q[g >> 3][(piece >> 3) * 2 + (piece & 1)][(g & 7) * 4 + ((piece & 7) >> 1)]) + at / 2;
      double s = 0.0;
#pragma unroll
      for (int c = 0; c < VPL; c += 2) {
        const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(row + c)), v = q[c / 2];
        // (the products are exact in 64 bits; in 32 they could overflow)
        s = fma((double)bfl(v), (double)bfl(u), s);
        s = fma((double)bfh(v), (double)bfh(u), s);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      return s;
    };
    // the greatest of a block's products; NaN ranks below everything
    auto greatest = [&](const double* s) -> double {
      double best = -INFINITY;
      for (int g = 0; g < G; ++g) {
        if (s[g] != s[g]) return -INFINITY;
        best = s[g] > best ? s[g] : best;
      }
      return best;
    };
    if (need >= band) {
      for (int w = tid; w < words; w += kPick) sh->member[w] |= sh->band[w];
    } else if (band <= kSmallBand) {
      // a warp per (block, head): 64-bit arithmetic is slow here (two products a
      // clock and SM), and mostly two or three blocks are left to tell apart
      double* dots = reinterpret_cast<double*>(sh->kept);  // (the scores there are done with)
      pick_sync();
      for (int x = warp; x < band * G; x += kPickWarps) {
        const double s = dot64(sh->idx[x / G], x % G);
        if (lane == 0) dots[x] = s;
      }
      pick_sync();
      for (int x = tid; x < band; x += kPick) sh->val[x] = greatest(dots + x * G);
      pick_sync();
      for (int x = tid; x < band; x += kPick) {
        const double s = sh->val[x];
        const int i = sh->idx[x];
        int rank = 0;
        for (int y = 0; y < band; ++y) rank += sh->val[y] > s || (sh->val[y] == s && sh->idx[y] < i);
        if (rank < need) atomicOr(&sh->member[i >> 5], 1u << (i & 31));
      }
    } else {
      // many near-equal scores: the digits of the 64-bit scores, then the
      // lowest indices among those equal to the last one in
      for (int i = f0 + warp; i < f1; i += kPickWarps)
        if ((sh->band[i >> 5] >> (i & 31)) & 1u) {
          double best = -INFINITY;
          bool bad = false;
          for (int g = 0; g < G; ++g) {
            const double s = dot64(i, g);
            bad = bad || s != s;
            best = s > best ? s : best;
          }
          if (lane == 0) again[i] = bad ? -INFINITY : best;
        }
      __threadfence_block();
      unsigned long long pre = 0;
      uint32_t todo = (uint32_t)need;
      for (int shift = 55; ; shift -= kDigit) {
        const int sft = shift > 0 ? shift : 0;
        const int bits = shift >= 0 ? kDigit : kDigit + shift;  // the last digit is what is left
        pick_sync();
        for (int i = tid; i < kBins; i += kPick) sh->hist[i] = 0;
        pick_sync();
        for (int i = f0 + tid; i < f1; i += kPick)
          if ((sh->band[i >> 5] >> (i & 31)) & 1u) {
            const unsigned long long k = key64(again[i]);
            // (a shift by 64 or more is undefined: the first digit has no prefix)
            if (sft + bits >= 64 || (k >> (sft + bits)) == pre)
              atomicAdd(&sh->hist[(uint32_t)(k >> sft) & ((1u << bits) - 1u)], 1u);
          }
        pick_sync();
        pick_digit<kBins>(sh, todo);
        pre = (pre << bits) | sh->digit;
        todo -= sh->above;
        if (sft == 0) break;
      }
      // pre: the last score in; todo of those equal to it belong
      const int per = (rest + kPick - 1) / kPick;
      const int i0 = f0 + tid * per, i1 = i0 + per < f1 ? i0 + per : f1;
      uint32_t equal = 0;
      for (int i = i0; i < i1; ++i)
        if ((sh->band[i >> 5] >> (i & 31)) & 1u) {
          const unsigned long long k = key64(again[i]);
          if (k > pre) atomicOr(&sh->member[i >> 5], 1u << (i & 31));
          equal += k == pre;
        }
      uint32_t total;
      uint32_t before = block_scan(equal, sh->wsum, &total);
      for (int i = i0; i < i1; ++i)
        if (((sh->band[i >> 5] >> (i & 31)) & 1u) && key64(again[i]) == pre) {
          if (before < todo) atomicOr(&sh->member[i >> 5], 1u << (i & 31));
          ++before;
        }
    }
  }
  pick_sync();
  // the chosen blocks in ascending order, -1 behind them: a share of the words per
  // warp, whose place is the number of bits in the words before
  int32_t* out = p.ids + (int64_t)bkv * p.top_k;
  const int wper = (words + kPickWarps - 1) / kPickWarps;
  const int w0 = warp * wper, w1 = w0 + wper < words ? w0 + wper : words;
  int before = 0, all = 0;
  for (int w = lane; w < words; w += 32) {
    const int c = __popc(sh->member[w]);
    before += w < w0 ? c : 0;
    all += c;
  }
  int at = __reduce_add_sync(0xffffffffu, before);
  const int total = __reduce_add_sync(0xffffffffu, all);
#pragma unroll 4
  for (int w = w0; w < w1; ++w) {
    const uint32_t u = sh->member[w];
    const int i = at + __popc(u & ((1u << lane) - 1u));
    if ((u >> lane & 1u) && i < p.top_k) out[i] = w * 32 + lane;
    at += __popc(u);
  }
  for (int i = total + tid; i < p.top_k; i += kPick) out[i] = -1;
}

template <int D, int NT>
cudaError_t launch_select_nt(const DecodeSelectParams& p0, cudaStream_t stream) {
  DecodeSelectParams p = p0;
  // CTAs per cluster: enough to fill the SMs (two CTAs each; one where the
  // registers allow no more), each warp with at least one step of 16 blocks
  const int rows = p.B * p.H_kv, slots = kPlanSms * (D == 256 || NT == 2 ? 1 : 2);
  const int steps = (p.n_blocks + 16 * kSelWarps - 1) / (16 * kSelWarps);
  p.ctas = 1;
  while (p.ctas < 8 && rows * p.ctas * 2 <= slots && p.ctas * 2 <= steps) p.ctas *= 2;
  static_assert(2 * (sizeof(SelShared) + 1024) <= 228 * 1024, "two CTAs per SM");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(decode_select_kernel<D, NT>, sizeof(SelShared), &done);
  if (e != cudaSuccess) return e;
  return launch_chained(decode_select_kernel<D, NT>, (unsigned)(rows * p.ctas), 1, kSelThreads, sizeof(SelShared), p.ctas,
                        p, stream);
}

template <int D>
cudaError_t launch_select_d(const DecodeSelectParams& p, cudaStream_t stream) {
  return (p.H / p.H_kv) <= 8 ? launch_select_nt<D, 1>(p, stream) : launch_select_nt<D, 2>(p, stream);
}

template <int D, int PARTS>
cudaError_t launch_means_parts(const BlockMeansParams& p, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.B * p.H_kv * p.span * PARTS;
  return launch_chained(block_means_kernel<D, PARTS>, (unsigned)((warps + kMeanWarps - 1) / kMeanWarps), 1,
                        32 * kMeanWarps, 0, 1, p, stream);
}

template <int D>
cudaError_t launch_means_d(const BlockMeansParams& p, cudaStream_t stream) {
  // four warps per block while those fill no more than the SMs' 64 warps
  return (int64_t)p.B * p.H_kv * p.span <= kPlanSms * 16 ? launch_means_parts<D, 4>(p, stream)
                                                         : launch_means_parts<D, 1>(p, stream);
}

}  // namespace

cudaError_t launch_block_means(const BlockMeansParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_means_d<64>(p, stream);
    case 128: return launch_means_d<128>(p, stream);
    case 256: return launch_means_d<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_select(const DecodeSelectParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_select_d<64>(p, stream);
    case 128: return launch_select_d<128>(p, stream);
    case 256: return launch_select_d<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mattn
