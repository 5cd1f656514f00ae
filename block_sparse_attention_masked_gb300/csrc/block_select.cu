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
// block_means_kernel: one warp per block, 16 bytes per lane, 32-bit sums: it
// reads every new key once and is HBM-bound.
//
// Selection.  The choice is that of exact arithmetic on the bf16 means and
// queries, so that it does not depend on how a product was summed:
//   1. decode_scores_kernel: score_n by matrix instructions with fp32 sums, and
//      e_n, a bound of its error: |sum of d rounded products - exact| <= u d'
//      sum |q_c k_c| <= u d' |q| |k_n|; with d / 16 <= 16 sums of 16 products
//      each, u d' <= 2^-17 even if each of them loses 2^-21 of its terms'
//      magnitudes, and 2^-15 is used.  Lanes load 16 bytes of a mean's row
//      straight into operand registers: the order of the dims inside a product
//      is free as long as the queries use the same one, so no shared memory.
//      One pass over the means: HBM-bound.
//   2. decode_select_kernel, one CTA per (sequence, key/value head): the k-th
//      largest score by digits (22 bits: T lies in [t0, t1)).  Every set of k
//      scores bounds the exact k-th score from below by the least of its
//      members' score - e, and every set of n - k + 1 from above by the most of
//      score + e; applied to {score >= t0} and {score < t1} this gives
//      lo <= exact k-th <= hi.  A block is in if score - e > hi, out if
//      score + e < lo; the few between are formed again in 64 bits (products of
//      two bf16 are exact there) and ranked.
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
constexpr int kMeanWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMeanWarps) block_means_kernel(const __grid_constant__ BlockMeansParams p) {
  constexpr int LPR = D / 8;          // lanes of a key row
  constexpr int RPI = 32 / LPR;       // keys per warp load
  constexpr int U = 8;                // loads in flight per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kMeanWarps + warp;
  const int64_t row = w / p.span;     // (sequence, key/value head)
  if (row >= (int64_t)p.B * p.H_kv) return;
  const int b = (int)(row / p.H_kv);
  int len = p.seq_lens ? p.seq_lens[b] : p.L;
  len = len < 0 ? 0 : (len > p.L ? p.L : len);
  int first = p.first ? p.first[b] : 0;
  first = first < 0 ? 0 : first;
  const int64_t end64 = (int64_t)first + p.max_new;
  const int end = end64 < len ? (int)end64 : len;  // new keys: [first, end)
  const int64_t blk = first / p.block + w % p.span;
  const int64_t k0 = blk * p.block;
  if (first >= end || k0 >= end || blk >= p.n_blocks) return;
  const int n = len - k0 < p.block ? (int)(len - k0) : p.block;
  const int sub = lane % LPR, r0 = lane / LPR;
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.k) +
                                                    (row * p.L + k0) * D) + sub;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int r = r0; r < n; r += RPI * U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      x[u] = r + u * RPI < n ? __ldg(src + (int64_t)(r + u * RPI) * LPR) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      acc[0] += bfl(x[u].x); acc[1] += bfh(x[u].x);
      acc[2] += bfl(x[u].y); acc[3] += bfh(x[u].y);
      acc[4] += bfl(x[u].z); acc[5] += bfh(x[u].z);
      acc[6] += bfl(x[u].w); acc[7] += bfh(x[u].w);
    }
  }
#pragma unroll
  for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
  if (lane < LPR) {
    const float c = (float)n;
    uint4 y;
    y.x = ptx::pack_bf16x2(acc[0] / c, acc[1] / c);
    y.y = ptx::pack_bf16x2(acc[2] / c, acc[3] / c);
    y.z = ptx::pack_bf16x2(acc[4] / c, acc[5] / c);
    y.w = ptx::pack_bf16x2(acc[6] / c, acc[7] / c);
    reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.means) + (row * p.n_blocks + blk) * D)[sub] = y;
  }
}

// ------------------------------------------------------------ scores
constexpr int kScoreWarps = 4;
constexpr float kScoreErr = 3.0517578125e-05f;  // 2^-15 (see above)

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float sq2(uint32_t x, float s) { return fmaf(bfl(x), bfl(x), fmaf(bfh(x), bfh(x), s)); }
__device__ __forceinline__ float sq8(const uint4& x, float s) {
  return sq2(x.x, sq2(x.y, sq2(x.z, sq2(x.w, s))));
}

__device__ __forceinline__ int blocks_of(const DecodeSelectParams& p, int b) {
  if (!p.seq_lens) return p.n_blocks;
  const int len = p.seq_lens[b];
  const int64_t n = len <= 0 ? 0 : ((int64_t)len + p.block - 1) / p.block;
  return n < p.n_blocks ? (int)n : p.n_blocks;
}

// A warp scores 16 blocks at a time: block rows are the tall operand, the
// group's heads (NT groups of eight) the other.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kScoreWarps) decode_scores_kernel(const __grid_constant__ DecodeSelectParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bkv = blockIdx.y, b = bkv / p.H_kv, kvh = bkv % p.H_kv, G = p.H / p.H_kv;
  const int n = blocks_of(p, b);
  const int r = lane >> 2, j = lane & 3;
  const uint4* mean = reinterpret_cast<const uint4*>(p.means) + (int64_t)bkv * p.n_blocks * (D / 8) + j;
  uint4 q[NT][D / 32];
  float qq = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int g = nt * 8 + r;
    const uint4* src = reinterpret_cast<const uint4*>(p.q) + ((int64_t)b * p.H + kvh * G + (g < G ? g : 0)) * (D / 8) + j;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      q[nt][i] = g < G ? __ldg(src + i * 4) : make_uint4(0, 0, 0, 0);
      s = sq8(q[nt][i], s);
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    qq = fmaxf(qq, s);
  }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) qq = fmaxf(qq, __shfl_xor_sync(0xffffffffu, qq, off));
  const float err = kScoreErr * sqrtf(qq + 1e-40f);
  for (int t = blockIdx.x * kScoreWarps + warp; t * 16 < n; t += gridDim.x * kScoreWarps) {
    const int r0 = t * 16 + r, r1 = r0 + 8;
    uint4 x[D / 32], y[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      x[i] = r0 < n ? __ldg(mean + (int64_t)r0 * (D / 8) + i * 4) : make_uint4(0, 0, 0, 0);
      y[i] = r1 < n ? __ldg(mean + (int64_t)r1 * (D / 8) + i * 4) : make_uint4(0, 0, 0, 0);
    }
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
        mma_bf16(acc[nt][0], x[i].x, y[i].x, x[i].y, y[i].y, q[nt][i].x, q[nt][i].y);
        mma_bf16(acc[nt][1], x[i].z, y[i].z, x[i].w, y[i].w, q[nt][i].z, q[nt][i].w);
      }
      sx = sq8(x[i], sx);
      sy = sq8(y[i], sy);
    }
    // heads of this lane: 2 j, 2 j + 1 (of each eight); rows r0 and r1
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
    if (nan0) s0 = __int_as_float(0x7fffffff);
    if (nan1) s1 = __int_as_float(0x7fffffff);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, s0, off), v = __shfl_xor_sync(0xffffffffu, s1, off);
      s0 = u != u || s0 != s0 ? __int_as_float(0x7fffffff) : fmaxf(s0, u);
      s1 = v != v || s1 != s1 ? __int_as_float(0x7fffffff) : fmaxf(s1, v);
      sx += __shfl_xor_sync(0xffffffffu, sx, off);
      sy += __shfl_xor_sync(0xffffffffu, sy, off);
    }
    if (j == 0) {
      // (the small terms cover squares and products that underflow)
      float2* dst = p.scores + (int64_t)bkv * p.n_blocks;
      if (r0 < n) dst[r0] = make_float2(s0, fmaf(err, sqrtf(sx + 1e-40f), 1e-36f));
      if (r1 < n) dst[r1] = make_float2(s1, fmaf(err, sqrtf(sy + 1e-40f), 1e-36f));
    }
  }
}

// ------------------------------------------------------------ selection
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kDigit = 11;
constexpr int kBins = 1 << kDigit;
constexpr int kSmallBand = 256;  // candidates ranked in shared memory; more go through the digits again

// Keys that order like the floats; NaN is taken as -inf.
__device__ __forceinline__ uint32_t key32(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long key64(double x) {
  if (x != x) x = -INFINITY;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

struct SelShared {
  uint32_t hist[kBins];
  uint32_t member[kSelectMaxBlocks / 32];  // blocks chosen
  uint32_t band[kSelectMaxBlocks / 32];    // blocks between lo and hi
  double val[kSmallBand];
  int idx[kSmallBand];
  uint32_t wsum[kSelWarps];
  float wlo[kSelWarps], whi[kSelWarps];
  uint32_t digit, above;
  int n_in, n_band;
};

// Exclusive prefix sum over the CTA's threads; *total gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* wsum, uint32_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint32_t s = wsum[w];
    before += w < warp ? s : 0u;
    all += s;
  }
  *total = all;
  return before + x - v;
}

// The digit d of the histogram, from the top, at which the count from above
// reaches `want` (1-based): sh->digit = d, sh->above = entries in digits > d.
__device__ __forceinline__ void pick_digit(SelShared* sh, uint32_t want) {
  constexpr int PER = kBins / kSelThreads;
  // thread t holds the bins of descending order t * PER ...
  uint32_t c[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = sh->hist[kBins - 1 - (threadIdx.x * PER + i)];
    sum += c[i];
  }
  uint32_t total;
  uint32_t before = block_scan(sum, sh->wsum, &total);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (before < want && before + c[i] >= want) {
      sh->digit = kBins - 1 - (threadIdx.x * PER + i);
      sh->above = before;
    }
    before += c[i];
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) decode_select_kernel(const __grid_constant__ DecodeSelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelShared* sh = reinterpret_cast<SelShared*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bkv = blockIdx.x, b = bkv / p.H_kv, kvh = bkv % p.H_kv, G = p.H / p.H_kv;
  const int n = blocks_of(p, b);
  const int words = (n + 31) / 32;
  // blocks kept whatever their score: [0, f0) and [f1, n)
  const int f0 = p.keep_first < n ? p.keep_first : n;
  const int f1 = n - p.keep_recent > f0 ? n - p.keep_recent : f0;
  const int rest = f1 - f0;                          // blocks that compete
  const int want = p.top_k - f0 - (n - f1);          // places left for them (>= 0: checked on the host)
  for (int w = tid; w < words; w += kSelThreads) {
    // the kept blocks' bits; all of them when every block fits
    uint32_t bits = 0;
    for (int i = 0; i < 32; ++i) {
      const int x = w * 32 + i;
      if (x < n && (x < f0 || x >= f1 || rest <= want)) bits |= 1u << i;
    }
    sh->member[w] = bits;
    sh->band[w] = 0;
  }
  for (int i = tid; i < kBins; i += kSelThreads) sh->hist[i] = 0;
  if (tid == 0) sh->n_in = sh->n_band = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  const float2* sc = p.scores + (int64_t)bkv * p.n_blocks;
  if (want > 0 && rest > want) {
    // T: two digits of 11 bits of the want-th largest score
    for (int i = f0 + tid; i < f1; i += kSelThreads) atomicAdd(&sh->hist[key32(sc[i].x) >> 21], 1u);
    __syncthreads();
    pick_digit(sh, (uint32_t)want);
    const uint32_t d1 = sh->digit, left = (uint32_t)want - sh->above;
    __syncthreads();
    for (int i = tid; i < kBins; i += kSelThreads) sh->hist[i] = 0;
    __syncthreads();
    for (int i = f0 + tid; i < f1; i += kSelThreads) {
      const uint32_t k = key32(sc[i].x);
      if ((k >> 21) == d1) atomicAdd(&sh->hist[(k >> 10) & (kBins - 1)], 1u);
    }
    __syncthreads();
    pick_digit(sh, left);
    const uint32_t prefix = (d1 << 11) | sh->digit;  // the want-th largest score's top 22 bits
    // bounds of the exact want-th score
    float lo = INFINITY, hi = -INFINITY;
    for (int i = f0 + tid; i < f1; i += kSelThreads) {
      const float2 s = sc[i];
      const uint32_t k = key32(s.x) >> 10;
      const bool fine = fabsf(s.x) < INFINITY && s.y < INFINITY;  // else nothing is known of it
      if (k >= prefix) lo = fminf(lo, fine ? s.x - s.y : -INFINITY);
      if (k <= prefix) hi = fmaxf(hi, fine ? s.x + s.y : INFINITY);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    if (lane == 0) {
      sh->wlo[warp] = lo;
      sh->whi[warp] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      lo = fminf(lo, sh->wlo[w]);
      hi = fmaxf(hi, sh->whi[w]);
    }
    int in = 0;
    for (int i = f0 + tid; i < f1; i += kSelThreads) {
      const float2 s = sc[i];
      const bool fine = fabsf(s.x) < INFINITY && s.y < INFINITY;
      if (fine && s.x - s.y > hi) {
        atomicOr(&sh->member[i >> 5], 1u << (i & 31));
        ++in;
      } else if (!fine || s.x + s.y >= lo) {
        atomicOr(&sh->band[i >> 5], 1u << (i & 31));
        const int at = atomicAdd(&sh->n_band, 1);
        if (at < kSmallBand) sh->idx[at] = i;
      }
    }
    if (in) atomicAdd(&sh->n_in, in);
    __syncthreads();
    const int band = sh->n_band, need = want - sh->n_in;  // 0 < need <= band
    double* again = p.again + (int64_t)bkv * p.n_blocks;
    const __nv_bfloat16* q0 = reinterpret_cast<const __nv_bfloat16*>(p.q) + ((int64_t)b * p.H + kvh * G) * D;
    const __nv_bfloat16* m0 = reinterpret_cast<const __nv_bfloat16*>(p.means) + (int64_t)bkv * p.n_blocks * D;
    // one warp: the score of block i in 64 bits (NaN ranks below everything)
    auto score64 = [&](int i) -> double {
      double best = -INFINITY;
      for (int g = 0; g < G; ++g) {
        double s = 0.0;
#pragma unroll
        for (int c = lane; c < D; c += 32)
          s = fma((double)__bfloat162float(q0[g * D + c]), (double)__bfloat162float(m0[(int64_t)i * D + c]), s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (s != s) return -INFINITY;
        best = s > best ? s : best;
      }
      return best;
    };
    if (need >= band) {
      for (int w = tid; w < words; w += kSelThreads) sh->member[w] |= sh->band[w];
    } else if (band <= kSmallBand) {
      for (int x = warp; x < band; x += kSelWarps) {
        const double s = score64(sh->idx[x]);
        if (lane == 0) sh->val[x] = s;
      }
      __syncthreads();
      for (int x = tid; x < band; x += kSelThreads) {
        const double s = sh->val[x];
        const int i = sh->idx[x];
        int rank = 0;
        for (int y = 0; y < band; ++y) rank += sh->val[y] > s || (sh->val[y] == s && sh->idx[y] < i);
        if (rank < need) atomicOr(&sh->member[i >> 5], 1u << (i & 31));
      }
    } else {
      // many near-equal scores: the digits of the 64-bit scores, then the
      // lowest indices among those equal to the last one in
      for (int i = f0 + warp; i < f1; i += kSelWarps)
        if ((sh->band[i >> 5] >> (i & 31)) & 1u) {
          const double s = score64(i);
          if (lane == 0) again[i] = s;
        }
      __threadfence_block();
      unsigned long long pre = 0;
      uint32_t todo = (uint32_t)need;
      for (int shift = 55; ; shift -= kDigit) {
        const int sft = shift > 0 ? shift : 0;
        const int bits = shift >= 0 ? kDigit : kDigit + shift;  // the last digit is what is left
        __syncthreads();
        for (int i = tid; i < kBins; i += kSelThreads) sh->hist[i] = 0;
        __syncthreads();
        for (int i = f0 + tid; i < f1; i += kSelThreads)
          if ((sh->band[i >> 5] >> (i & 31)) & 1u) {
            const unsigned long long k = key64(again[i]);
            // (a shift by 64 or more is undefined: the first digit has no prefix)
            if (sft + bits >= 64 || (k >> (sft + bits)) == pre)
              atomicAdd(&sh->hist[(uint32_t)(k >> sft) & ((1u << bits) - 1u)], 1u);
          }
        __syncthreads();
        pick_digit(sh, todo);
        pre = (pre << bits) | sh->digit;
        todo -= sh->above;
        if (sft == 0) break;
      }
      // pre: the last score in; todo of those equal to it belong
      const int per = (rest + kSelThreads - 1) / kSelThreads;
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
  __syncthreads();
  // the chosen blocks in ascending order, -1 behind them
  int32_t* out = p.ids + (int64_t)bkv * p.top_k;
  const int wper = (words + kSelThreads - 1) / kSelThreads;
  uint32_t cnt = 0;
  for (int w = tid * wper; w < words && w < (tid + 1) * wper; ++w) cnt += __popc(sh->member[w]);
  uint32_t total;
  uint32_t at = block_scan(cnt, sh->wsum, &total);
  for (int w = tid * wper; w < words && w < (tid + 1) * wper; ++w)
    for (uint32_t u = sh->member[w]; u; u &= u - 1) {
      if (at < (uint32_t)p.top_k) out[at] = w * 32 + __ffs(u) - 1;
      ++at;
    }
  for (int i = (int)total + tid; i < p.top_k; i += kSelThreads) out[i] = -1;
}

template <int D, int NT>
cudaError_t launch_select_nt(const DecodeSelectParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.B * p.H_kv;
  const int tiles = (p.n_blocks + 15) / 16;  // 16 blocks per warp step
  // enough CTAs for about eight per SM, each warp at least one step
  int64_t gx = (8 * kPlanSms + rows - 1) / rows;
  const int64_t most = (tiles + kScoreWarps - 1) / kScoreWarps;
  gx = gx < 1 ? 1 : (gx > most ? most : gx);
  decode_scores_kernel<D, NT><<<dim3((unsigned)gx, (unsigned)rows), 32 * kScoreWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_select_d(const DecodeSelectParams& p, cudaStream_t stream) {
  cudaError_t e = (p.H / p.H_kv) <= 8 ? launch_select_nt<D, 1>(p, stream) : launch_select_nt<D, 2>(p, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * p.H_kv);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = sizeof(SelShared);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static_assert(sizeof(SelShared) <= 48 * 1024, "static shared-memory limit");
  return cudaLaunchKernelEx(&cfg, decode_select_kernel<D>, p);
}

template <int D>
cudaError_t launch_means_d(const BlockMeansParams& p, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.B * p.H_kv * p.span;
  block_means_kernel<D><<<(unsigned)((warps + kMeanWarps - 1) / kMeanWarps), 32 * kMeanWarps, 0, stream>>>(p);
  return cudaGetLastError();
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
