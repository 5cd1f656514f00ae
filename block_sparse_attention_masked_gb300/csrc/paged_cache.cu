// Rows into the pages of a cache and back (mattn_cache_write, mattn_cache_read),
// for sm_103a.
//
// Row (t, h) of packed sequences, d bf16 values, is position starts_b + t - cu_b of
// its sequence b; its place is row pos % page of page table[b][pos / page], as bf16 or
// as e4m3 codes with a power of two (e4m3.cuh).  Each row is read once and written once,
// k and v together, since they share the place: HBM-bound (2 d + d + 1 bytes a row and
// tensor in eight bits, 4 d in bf16).
//
// d / 16 lanes take a row, two 16-byte pieces each, half a row apart, so that every
// load and store of a warp covers whole 32-byte sectors.  Measured: 32,768 rows of 8 heads
// of 128 written in e4m3 in 36.6 us = 202 MB at 5.5 TB/s, read back in 35.3; in bf16 43.8 and 44.4
// us = 268 MB at 6.1; 64 single tokens 4.1 (a launch and three trips to memory: the sequence,
// its page, the rows).  A place looked up per row and head took 39.5 and 38.2 (27 against 16 million
// instructions); CTAs of 128 threads, one or four heads' loads together and finer shares of a token's
// heads gave 35 to 37.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "e4m3.cuh"
#include "paged_ops.h"
#include "ptx.cuh"

namespace mattn {
namespace {

constexpr int kCacheThreads = 256;

// Where row (t, h) lies in the cache: false where it is no sequence's (padding).
// page < 0: the position has no page.
struct Place {
  int64_t page;
  int row;
};

// The sequence that token t is in, from b on (b: at or before it).
__device__ __forceinline__ bool locate(const CacheRowsParams& p, int t, int& b, Place& at) {
  int first = t;
  if (p.cu) {
    while (b + 1 < p.B && t >= __ldg(p.cu + b + 1)) ++b;
    first = __ldg(p.cu + b);
    if (t < first || t >= __ldg(p.cu + b + 1)) return false;
  } else {
    b = t;
    if (t >= p.B) return false;
  }
  const int64_t pos = (p.starts ? (int64_t)__ldg(p.starts + b) : 0) + ((int64_t)t - first);
  at.page = -1;
  at.row = 0;
  if (pos >= 0 && pos < (int64_t)p.table_pages * p.page) {
    const uint32_t j = (uint32_t)pos / (uint32_t)p.page;
    const int id = __ldg(p.table + (int64_t)b * p.table_pages + j);
    if (id >= 0 && id < p.n_pages) at.page = id;
    at.row = (int)((uint32_t)pos - j * (uint32_t)p.page);
  }
  return true;
}

// The last b with cu[b] <= t, or 0 (bisection: 2^(-k) of the sequences are left after k steps).
__device__ __forceinline__ int sequence_of(const CacheRowsParams& p, int t) {
  if (!p.cu) return 0;
  int lo = 0, hi = p.B;  // cu[lo] <= t or lo = 0; cu[hi] > t or hi = B
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint4 ld16(const void* p) {  // read once
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t x) { return __vmaxu2(m, x & 0x7fff7fffu); }

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Eight values times f as eight codes.
__device__ __forceinline__ uint2 codes8(uint4 x, float f) {
  uint2 r;
  r.x = e4m3::pack2(bf_lo(x.x) * f, bf_hi(x.x) * f) | e4m3::pack2(bf_lo(x.y) * f, bf_hi(x.y) * f) << 16;
  r.y = e4m3::pack2(bf_lo(x.z) * f, bf_hi(x.z) * f) | e4m3::pack2(bf_lo(x.w) * f, bf_hi(x.w) * f) << 16;
  return r;
}
__device__ __forceinline__ uint32_t values2(uint32_t half2, float f) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&half2));
  return ptx::pack_bf16x2(v.x * f, v.y * f);
}
// Eight codes times f as eight bf16 values.
__device__ __forceinline__ uint4 values8(uint2 c, float f) {
  return make_uint4(values2(e4m3::to_half2(c.x), f), values2(e4m3::to_half2_hi(c.x), f), values2(e4m3::to_half2(c.y), f),
                    values2(e4m3::to_half2_hi(c.y), f));
}

// A lane group takes a token, `heads` of its heads and k and v of each: one look-up of the
// place, pointers moved from head to head, U heads' loads together.
template <int D, bool E8, bool READ>
__global__ void __launch_bounds__(kCacheThreads) cache_rows_kernel(const __grid_constant__ CacheRowsParams p) {
  constexpr int LPR = D / 16, GW = 32 / LPR, U = 2;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t warp = (int64_t)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  // (segments of a token's heads are neighbours, then tokens: GW tokens a warp and segment)
  const int64_t block = warp / p.segs;
  const int seg = (int)(warp - block * p.segs), t = (int)(block * GW) + sub;
  const int h0 = seg * p.heads, h1 = min(h0 + p.heads, p.H_kv);
  after_previous();
  if (block * GW >= p.T) return;  // (whole warps)
  int b = t < p.T ? sequence_of(p, t) : 0;
  Place at;
  at.page = -1;
  const bool row = t < p.T && locate(p, t, b, at);  // (a row of some sequence)
  const bool there = row && at.page >= 0;
  // this lane's piece of the head's row and of its place, for k and v
  const char* src[2];
  char* dst[2];
  int64_t src_step[2], dst_step[2], exp_step[2];
  uint8_t* ex[2];
  constexpr int kCell = E8 ? 1 : 2;  // bytes of a cached value
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    char* r = static_cast<char*>(p.rows[i]) + 2 * (t * p.row_token[i] + h0 * p.row_head[i] + l * 8);
    char* c = static_cast<char*>(p.pages[i]) +
              kCell * ((there ? at.page * p.page_stride[i] + at.row * p.row_stride[i] : 0) + h0 * p.head_stride[i] + l * 8);
    src[i] = READ ? c : r;
    dst[i] = READ ? r : c;
    src_step[i] = READ ? kCell * p.head_stride[i] : 2 * p.row_head[i];
    dst_step[i] = READ ? 2 * p.row_head[i] : kCell * p.head_stride[i];
    if (E8) {
      ex[i] = p.exps[i] + (there ? at.page * p.exp_page[i] + at.row * p.exp_row[i] : 0) + h0 * p.exp_head[i];
      exp_step[i] = p.exp_head[i];
    }
  }
  for (int h = h0; h < h1; h += U) {
    uint4 x[U][2][2];  // [..][tensor][half of the row]
    uint32_t e[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[u][i][0] = x[u][i][1] = make_uint4(0, 0, 0, 0);
        e[u][i] = 0;
        if (there && h + u < h1) {
          if (READ && E8) {
            const uint2 a = ld8(src[i]), c = ld8(src[i] + D / 2);
            x[u][i][0] = make_uint4(a.x, a.y, c.x, c.y);
            e[u][i] = __ldg(ex[i]);
          } else {
            x[u][i][0] = ld16(src[i]);
            x[u][i][1] = ld16(src[i] + D);
          }
        }
        src[i] += src_step[i];
        if (READ && E8) ex[i] += exp_step[i];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (READ) {
          uint4 lo = x[u][i][0], hi = x[u][i][1];
          if (E8) {
            const float f = e4m3::power((int)e[u][i]);
            hi = values8(make_uint2(lo.z, lo.w), f);
            lo = values8(make_uint2(lo.x, lo.y), f);
          }
          if (row && h + u < h1) {
            *reinterpret_cast<uint4*>(dst[i]) = lo;
            *reinterpret_cast<uint4*>(dst[i] + D) = hi;
          }
        } else if (E8) {
          const uint4 a = x[u][i][0], c = x[u][i][1];
          uint32_t m = max_abs(max_abs(max_abs(max_abs(0, a.x), a.y), a.z), a.w);
          m = max_abs(max_abs(max_abs(max_abs(m, c.x), c.y), c.z), c.w);
#pragma unroll
          for (int off = 1; off < LPR; off <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
          m = max(m >> 16, m & 0xffffu);
          const int power = e4m3::row_exponent(m);
          const float f = e4m3::inverse(power);
          if (there && h + u < h1) {
            *reinterpret_cast<uint2*>(dst[i]) = codes8(a, f);
            *reinterpret_cast<uint2*>(dst[i] + D / 2) = codes8(c, f);
            if (l == 0) *ex[i] = (uint8_t)power;
          }
          ex[i] += exp_step[i];
        } else if (there && h + u < h1) {
          *reinterpret_cast<uint4*>(dst[i]) = x[u][i][0];
          *reinterpret_cast<uint4*>(dst[i] + D) = x[u][i][1];
        }
        dst[i] += dst_step[i];
      }
  }
}

template <int D, bool E8, bool READ>
cudaError_t launch_d(const CacheRowsParams& p0, cudaStream_t stream) {
  CacheRowsParams p = p0;
  constexpr int GW = 32 / (D / 16);
  // Heads of a lane group: all of a token's, fewer where that leaves the machine without
  // its 32 warps an SM.
  const int64_t blocks = ((int64_t)p.T + GW - 1) / GW;
  int64_t segs = (kPlanSms * 32 + blocks - 1) / blocks;
  const int64_t most = (p.H_kv + 1) / 2;
  segs = segs < 1 ? 1 : (segs > most ? most : segs);
  p.heads = (int)((p.H_kv + segs - 1) / segs);
  p.heads += p.heads & 1;
  p.segs = (p.H_kv + p.heads - 1) / p.heads;
  const int64_t warps = blocks * p.segs, ctas = (warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  return launch_chained(cache_rows_kernel<D, E8, READ>, (unsigned)ctas, 1, kCacheThreads, 0, 1, p, stream);
}

template <bool READ>
cudaError_t launch_rows(const CacheRowsParams& p, bool e4m3, cudaStream_t stream) {
  switch (p.d * 2 + (e4m3 ? 1 : 0)) {
    case 128: return launch_d<64, false, READ>(p, stream);
    case 129: return launch_d<64, true, READ>(p, stream);
    case 256: return launch_d<128, false, READ>(p, stream);
    case 257: return launch_d<128, true, READ>(p, stream);
    case 512: return launch_d<256, false, READ>(p, stream);
    case 513: return launch_d<256, true, READ>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsParams& p, bool e4m3, cudaStream_t stream) {
  return launch_rows<false>(p, e4m3, stream);
}
cudaError_t launch_cache_read(const CacheRowsParams& p, bool e4m3, cudaStream_t stream) {
  return launch_rows<true>(p, e4m3, stream);
}

}  // namespace mattn
