// Norms of queries and keys per head with the position rotation in the same
// pass, from the projection's layout into the attention's layouts, for sm_103a.
//
// A row x (one head of one token, d values) becomes
//   y = x * rsqrt(mean(x^2) + eps) * w            (when weights are given)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t) for each of the `rot`
//             pairs of its first 2 rot values, t = position * inv_freq,
// in 32 bits with one rounding at the store; queries go to [B][H][N][d],
// keys and (unchanged) values to row start + n of their caches.  Each value
// is read once and written once, so the pass is HBM-bound: a warp takes one
// token's rows (d / 16 lanes per row, each two pieces of 8 values that hold whole
// pairs, so no lane needs another's values but for the row's mean square) and
// forms the token's cosines and sines once for all its heads.  What counts is
// loads in flight: with the angles and weights in shared memory and two rows a
// lane group at a time the kernel keeps 64 registers and 32 warps an SM (28 and
// 72 in fp32), in small CTAs, whose warps wait for no more than three others (805 MB
// in bf16: 131 us, 6.1 TB/s; 136 with eight warps a CTA, 143 with sixteen; 156
// with angles and weights in registers, four rows and 16 warps an SM).  fp32 rows
// move 32 bytes an access (503 MB: 77.7 us, 6.5 TB/s; 80.5 with 32 warps an SM; 100
// with 16 bytes).  Two values an instruction (f32x2) change nothing.  Where
// tokens are few, warps share a token's rows.
//
// Angles: inv_freq / 2 pi is held as a 64-bit fraction of a turn: the constant
// and the product round in 64 bits (2^-52 of the turns together), and the fraction is cut
// to 2^-64 of a turn.  Position times it modulo a whole turn is one wrapping
// 64-bit product, so nothing else is lost at far positions, where a 32-bit product is
// off by 0.06 rad at position 2^20.  The nearest quarter turn is taken off in
// whole numbers, and the rest, an eighth of a turn at most, is rounded to 32 bits:
// relative to itself, so that cosines and sines are right to 2^-22 of their own values
// next to their zeros too.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_ops.h"

namespace mattn {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeMaxPairs = 128;
constexpr int kRopeBatch = 2;  // rows in flight per lane group

// 8 values of a row: 16 bytes of bf16, or 32 of fp32 (`wide`: as one access,
// where every row starts on a 32-byte boundary).
template <bool F32>
struct Piece;
template <>
struct Piece<false> {
  uint4 u;
  __device__ __forceinline__ void load(const void* base, int64_t e, bool) {
    u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + e));
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(void* base, int64_t e, bool) const {
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + e) = u;
  }
};
template <>
struct Piece<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t e, bool wide) {
    const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + e);
    if (wide) {
      asm volatile("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w), "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                   : "l"(s));
    } else {
      a = __ldg(s);
      b = __ldg(s + 1);
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void store(void* base, int64_t e, bool wide) const {
    float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + e);
    if (wide) {
      asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(d), "f"(a.x), "f"(a.y), "f"(a.z),
                   "f"(a.w), "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w)
                   : "memory");
    } else {
      d[0] = a;
      d[1] = b;
    }
  }
};

__device__ __forceinline__ void get8(float (&x)[8], const float* s) {
  const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Sum over the GL lanes of a row's group, the same order on every lane.
template <int GL>
__device__ __forceinline__ float group_sum(float v, int lane0) {
  if constexpr ((GL & (GL - 1)) == 0) {
#pragma unroll
    for (int off = 1; off < GL; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  } else {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < GL; ++i) s += __shfl_sync(0xffffffffu, v, lane0 + i);
    return s;
  }
}

template <int D, bool F32, bool INTER>
__global__ void __launch_bounds__(32 * kRopeWarps, F32 ? 7 : 8) qk_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int GL = D / 16;       // lanes of a row
  constexpr int RPW = 32 / GL;     // rows of a warp
  __shared__ unsigned long long turn[kRopeMaxPairs];          // inv_freq / 2 pi as a 2^-64 fraction of a turn
  __shared__ __align__(16) float trig[kRopeWarps][2][kRopeMaxPairs];  // cosines, sines of the warp's token
  __shared__ __align__(16) float weights[2][D];               // of the norms of q and k
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int64_t token = gw / p.segs;
  const int seg = (int)(gw % p.segs);
  const bool live = token < (int64_t)p.B * p.N;
  const int b = live ? (int)(token / p.N) : 0, n = live ? (int)(token % p.N) : 0;

  const int grp = lane / GL, sub = lane - grp * GL;
  const bool idle = grp >= RPW;  // lanes past the last whole row (d = 80, 96)
  const int lane0 = grp * GL;
  const int r8 = p.rot / 8;      // lanes of a row that hold rotated pairs
  // the lane's two pieces of the row, of 8 values each
  int ca, cb;
  if (INTER) {
    ca = 2 * sub;
    cb = ca + 1;
  } else if (sub < r8) {
    ca = sub;
    cb = sub + r8;
  } else {
    ca = 2 * r8 + 2 * (sub - r8);
    cb = ca + 1;
  }
  const bool rotated = !idle && sub < r8;

  // the token's rows in steps of RPW heads: its of q, then of k, then of v;
  // this warp's are [i_lo, i_hi)
  const int its_q = (p.H + RPW - 1) / RPW, its_k = (p.H_kv + RPW - 1) / RPW, its_v = p.dst[2] ? its_k : 0;
  const int total = its_q + its_k + its_v;
  const int i_lo = (int)((int64_t)total * seg / p.segs), i_hi = (int)((int64_t)total * (seg + 1) / p.segs);
  Piece<F32> a[kRopeBatch], c[kRopeBatch];
  // steps it .. of tensor t, at src0
  auto load = [&](const void* src, int64_t src0, int heads, int it, int hi) {
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) {
      const int head = (it + u) * RPW + grp;
      if (!idle && it + u < hi && head < heads) {
        a[u].load(src, src0 + (int64_t)head * D + ca * 8, p.wide);
        c[u].load(src, src0 + (int64_t)head * D + cb * 8, p.wide);
      } else {
        a[u].zero();
        c[u].zero();
      }
    }
  };
  after_previous();
  // (the first rows, the length and the position are on their way while the
  // frequencies are turned into fractions)
  if (live) {
    const int t = i_lo < its_q ? 0 : (i_lo < its_q + its_k ? 1 : 2);
    const int base = t == 0 ? 0 : (t == 1 ? its_q : its_q + its_k);
    load(p.src[t], (int64_t)b * p.batch_stride[t] + (int64_t)n * p.token_stride[t], t == 0 ? p.H : p.H_kv, i_lo - base,
         min(i_hi - base, t == 0 ? its_q : its_k));
  }
  const int len = live && p.lens ? p.lens[b] : p.N;
  const int start = live && p.starts ? p.starts[b] : 0;
  for (int i = threadIdx.x; i < p.rot; i += blockDim.x) {
    const double t = (double)p.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    // (of a negative frequency the fraction's negative: 1 less it would round to 2^-54)
    const unsigned long long f = __double2ull_rz((fabs(t) - floor(fabs(t))) * 18446744073709551616.0);
    turn[i] = t < 0.0 ? 0ull - f : f;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
    if (p.weight[t])
      for (int i = threadIdx.x; i < D; i += blockDim.x) weights[t][i] = __ldg(p.weight[t] + i);
  __syncthreads();
  if (!live || n >= len) return;  // the batch's padding
  for (int i = lane; i < p.rot; i += 32) {
    const int axis = i < p.axis_end[0] ? 0 : (i < p.axis_end[1] ? 1 : 2);
    const int64_t pos = p.positions ? p.positions[((int64_t)axis * p.B + b) * p.N + n] : (int64_t)start + n;
    // whole quarter turns, and what is left in half turns of [-1/4, 1/4)
    const unsigned long long f = (unsigned long long)pos * turn[i];
    const unsigned quarter = (unsigned)((f + (1ull << 61)) >> 62);
    const float x = __ll2float_rn((long long)(f - ((unsigned long long)quarter << 62))) * 1.0842021724855044e-19f;  // 2^-63
    float s, co;
    sincospif(x, &s, &co);
    if (quarter & 1u) {
      const float t = co;
      co = -s;
      s = t;
    }
    if (quarter & 2u) {
      co = -co;
      s = -s;
    }
    trig[warp][0][i] = co;
    trig[warp][1][i] = s;
  }
  __syncwarp();

  bool loaded = true;  // the first rows
  int base = 0;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    const int its = t == 0 ? its_q : (t == 1 ? its_k : its_v);
    const int lo = max(i_lo, base) - base, hi = min(i_hi, base + its) - base;
    base += its;
    if (lo >= hi) continue;
    const int heads = t == 0 ? p.H : p.H_kv;
    const int64_t to = t == 0 ? (int64_t)n : (int64_t)start + n, rows = t == 0 ? p.N : p.L;
    const bool there = to >= 0 && to < rows;  // rows outside the cache are not written
    const void* src = p.src[t];
    const int64_t src0 = (int64_t)b * p.batch_stride[t] + (int64_t)n * p.token_stride[t];
    const int64_t dst0 = ((int64_t)b * heads * rows + to) * D;
    const bool norm = t < 2 && p.weight[t < 2 ? t : 0];
    for (int it = lo; it < hi; it += kRopeBatch) {
      if (!loaded) load(src, src0, heads, it, hi);
      loaded = false;
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        if (it + u >= hi) break;  // warp-uniform
        const int head = (it + u) * RPW + grp;
        if (t < 2) {
          float x[8], y[8];
          a[u].get(x);
          c[u].get(y);
          if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
            ss = group_sum<GL>(ss, lane0);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
            float w[8];
            get8(w, &weights[t < 2 ? t : 0][(idle ? 0 : ca) * 8]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
            get8(w, &weights[t < 2 ? t : 0][(idle ? 0 : cb) * 8]);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= r * w[i];
          }
          if (rotated) {
            float cs[8], sn[8];
            get8(cs, &trig[warp][0][sub * 8]);
            get8(sn, &trig[warp][1][sub * 8]);
            if (INTER) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
                x[2 * i] = x0 * cs[i] - x1 * sn[i];
                x[2 * i + 1] = x1 * cs[i] + x0 * sn[i];
                y[2 * i] = y0 * cs[4 + i] - y1 * sn[4 + i];
                y[2 * i + 1] = y1 * cs[4 + i] + y0 * sn[4 + i];
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float x0 = x[i], y0 = y[i];
                x[i] = x0 * cs[i] - y0 * sn[i];
                y[i] = y0 * cs[i] + x0 * sn[i];
              }
            }
          }
          a[u].set(x);
          c[u].set(y);
        }
        if (there && !idle && head < heads) {
          a[u].store(p.dst[t], dst0 + (int64_t)head * rows * D + ca * 8, p.wide);
          c[u].store(p.dst[t], dst0 + (int64_t)head * rows * D + cb * 8, p.wide);
        }
      }
    }
  }
}

template <int D, bool F32>
cudaError_t launch_d(const RopeParams& p, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.B * p.N * p.segs;
  const unsigned grid = (unsigned)((warps + kRopeWarps - 1) / kRopeWarps);
  return launch_chained(p.interleaved ? qk_rope_kernel<D, F32, true> : qk_rope_kernel<D, F32, false>, grid, 1,
                        32 * kRopeWarps, 0, 1, p, stream);
}

template <bool F32>
cudaError_t launch_t(const RopeParams& p, cudaStream_t stream) {
  switch (p.d) {
    case 32: return launch_d<32, F32>(p, stream);
    case 64: return launch_d<64, F32>(p, stream);
    case 80: return launch_d<80, F32>(p, stream);
    case 96: return launch_d<96, F32>(p, stream);
    case 128: return launch_d<128, F32>(p, stream);
    case 256: return launch_d<256, F32>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_qk_rope(const RopeParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_t<true>(p, stream) : launch_t<false>(p, stream);
}

}  // namespace mattn
