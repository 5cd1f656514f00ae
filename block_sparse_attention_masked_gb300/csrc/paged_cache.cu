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
// load and store of a warp covers whole 32-byte sectors; rows go to warps in memory
// order of the packed side, U groups' loads together.
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
  const int64_t pos = (p.starts ? (int64_t)__ldg(p.starts + b) : 0) + (t - first);
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

template <int D, bool E8, bool READ>
__global__ void __launch_bounds__(kCacheThreads) cache_rows_kernel(const __grid_constant__ CacheRowsParams p) {
  constexpr int LPR = D / 16, RW = 32 / LPR, U = 2;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t warp = (int64_t)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  const int64_t rows = (int64_t)p.T * p.H_kv;
  int64_t r = warp * p.per_warp * RW + sub;  // this lane's first row
  after_previous();
  if (r - sub >= rows) return;  // (whole warps)
  int t = (int)(r / p.H_kv), h = (int)(r - (int64_t)t * p.H_kv);
  int b = sequence_of(p, t);
  for (int g = 0; g < p.per_warp; g += U) {
    uint4 x[U][2][2];  // [..][tensor][half of the row]
    Place at[U];
    int ts[U], hs[U];
    bool live[U];
    uint32_t ex[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      live[u] = r < rows && g + u < p.per_warp && locate(p, t, b, at[u]);
      ts[u] = t;
      hs[u] = h;
      if (!READ) live[u] = live[u] && at[u].page >= 0;
      const bool has = live[u] && at[u].page >= 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[u][i][0] = x[u][i][1] = make_uint4(0, 0, 0, 0);
        ex[u][i] = 0;
        if (!has) continue;
        if (READ && E8) {
          const uint8_t* src = static_cast<const uint8_t*>(p.pages[i]) + at[u].page * p.page_stride[i] +
                               h * p.head_stride[i] + at[u].row * p.row_stride[i] + l * 8;
          const uint2 a = ld8(src), c = ld8(src + D / 2);
          x[u][i][0] = make_uint4(a.x, a.y, c.x, c.y);
          ex[u][i] = __ldg(p.exps[i] + at[u].page * p.exp_page[i] + h * p.exp_head[i] + at[u].row * p.exp_row[i]);
        } else {
          const __nv_bfloat16* src =
              READ ? static_cast<const __nv_bfloat16*>(p.pages[i]) + at[u].page * p.page_stride[i] +
                         h * p.head_stride[i] + at[u].row * p.row_stride[i]
                   : static_cast<const __nv_bfloat16*>(p.rows[i]) + t * p.row_token[i] + h * p.row_head[i];
          x[u][i][0] = ld16(src + l * 8);
          x[u][i][1] = ld16(src + D / 2 + l * 8);
        }
      }
      r += RW;
      h += RW;
      while (h >= p.H_kv) {
        h -= p.H_kv;
        ++t;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (READ) {
          if (!live[u]) continue;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.rows[i]) + ts[u] * p.row_token[i] + hs[u] * p.row_head[i] + l * 8;
          uint4 lo = x[u][i][0], hi = x[u][i][1];
          if (E8) {
            const float f = e4m3::power((int)ex[u][i]);
            hi = values8(make_uint2(lo.z, lo.w), f);
            lo = values8(make_uint2(lo.x, lo.y), f);
          }
          *reinterpret_cast<uint4*>(dst) = lo;
          *reinterpret_cast<uint4*>(dst + D / 2) = hi;
          continue;
        }
        int e = 0;
        if (E8) {  // (all lanes: rows of one warp end together)
          const uint4 a = x[u][i][0], c = x[u][i][1];
          uint32_t m = max_abs(max_abs(max_abs(max_abs(0, a.x), a.y), a.z), a.w);
          m = max_abs(max_abs(max_abs(max_abs(m, c.x), c.y), c.z), c.w);
#pragma unroll
          for (int off = 1; off < LPR; off <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
          m = max(m >> 16, m & 0xffffu);
          e = e4m3::row_exponent(m);
        }
        if (!live[u]) continue;
        const int64_t to = at[u].page * p.page_stride[i] + hs[u] * p.head_stride[i] + at[u].row * p.row_stride[i] + l * 8;
        if (E8) {
          uint8_t* dst = static_cast<uint8_t*>(p.pages[i]) + to;
          const float f = e4m3::inverse(e);
          *reinterpret_cast<uint2*>(dst) = codes8(x[u][i][0], f);
          *reinterpret_cast<uint2*>(dst + D / 2) = codes8(x[u][i][1], f);
          if (l == 0)
            p.exps[i][at[u].page * p.exp_page[i] + hs[u] * p.exp_head[i] + at[u].row * p.exp_row[i]] = (uint8_t)e;
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.pages[i]) + to;
          *reinterpret_cast<uint4*>(dst) = x[u][i][0];
          *reinterpret_cast<uint4*>(dst + D / 2) = x[u][i][1];
        }
      }
    }
    if (__all_sync(0xffffffffu, r >= rows)) break;
  }
}

template <int D, bool E8, bool READ>
cudaError_t launch_d(const CacheRowsParams& p0, cudaStream_t stream) {
  CacheRowsParams p = p0;
  constexpr int RW = 32 / (D / 16);
  const int64_t groups = ((int64_t)p.T * p.H_kv + RW - 1) / RW;
  // groups of a warp: more than one only where the machine has eight warps a
  // scheduler without
  const int64_t most = groups / (kPlanSms * 32);
  p.per_warp = (int)(most < 2 ? (most < 1 ? 1 : 2) : (most > 8 ? 8 : (most & ~int64_t(1))));
  const int64_t warps = (groups + p.per_warp - 1) / p.per_warp, ctas = (warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
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
