// Decode attention over a paged cache (mattn_decode_paged), for sm_103a: one query per
// sequence,
//
//   o_h = sum_j p_hj v_j / (sum_j p_hj + exp(sink_h)),  p_hj = exp(scale q_h . k_j)
//
// over the sequence's cached keys [0, len), or those of a window and the first tokens,
// key j in row j % page of page table[b][j / page], in bf16 or as e4m3 codes with a
// power of two a row (e4m3.cuh).  4 d bytes a key, or 2 (d + 1), against 4 d G FLOPs:
// HBM-bound.
//
// The work is shared out as the row workers' of decode_rows.cuh: the lists of all
// (sequence, key/value head) groups laid end to end in tiles, equal shares of them to
// all warps of the machine, each warp with its own ring of TMA boxes; a state per piece,
// merged by decode_merge_kernel.  bf16 tiles take that file's step; this one has the
// step in eight bits.
//
// Eight bits.  Codes become f16 exactly (cvt, two a lane and instruction; bf16 would take
// four) and meet on f16 matrix instructions, keys and dims as the tall operand:
//   S^T = K Q^T: the query row times a power of two that puts its largest value in
//     [2^14, 2^15): 11 bits of each value, 2^-39 of the largest one off at most where it
//     is smaller; the scores get that power and the key's own back in fp32.
//   O^T += V^T W^T: a weight carries its value row's power, w_j = 2^(x_j + e_j - M),
//     x_j the score in the log2 domain, M a running maximum of x_j + e_j beside the
//     softmax's own m: w <= 1 whatever the powers are.  Times 2^14 and rounded to f16: off
//     by 2^-11 of itself at most (an eighth of the output's own rounding) down to 2^-28 of
//     the largest weight, and by 2^-39 of the largest below.
// Any order of the 16 keys of a product and of the dims does, as long as both operands
// have the same one, so codes are read from shared memory 16 a lane and load: a lane's
// key rows are r(g), its dims 16 r(..) .., r the rotation of three bits by one, which
// puts the eight lanes of a load's phase into eight different 16-byte columns of the
// swizzled tile.
//
// Measured: 64 sequences of 4K to 8K keys, 32 / 8 heads of 128 in e4m3 133-138 us = 850 MB at 6.2-6.4
// TB/s (HBM; loads without products take 133.6), 16 of 16K to 32K in bf16 245-255 us = 1.64 GB
// at 6.4-6.7, one of 131,071, heads of 256, 54.5-54.9 us = 270 MB at 4.9 (8 to 10 us of it are the two
// launches, the first loads and the states).  With more than eight query heads a key/value
// head the e4m3 step bounds it (64 sequences, 32 / 2 heads 63 us against 30 by the bytes): the
// products of 16 heads and two exponentials a score on three warps a scheduler, with registers
// that do not suffice (60 bytes a thread spill at d = 64, 116 at 128, 152 at 256).  Tried without
// gain: 64 keys a tile and six warps at d = 128 (160 us for 134), pages looked up for 32 boxes at
// a time, a tile's boxes as one copy, exponent bytes as words, states of a CTA's warps joined in shared
// memory where there are many (138 for 134).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_rows.cuh"
#include "e4m3.cuh"
#include "kernel_params.h"
#include "paged_ops.h"
#include "ptx.cuh"

namespace mattn {
namespace {

// c += a b on one warp, 16 x 8 x 16, f16 inputs and fp32 sums.
__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Tiles of a warp's ring.
template <int D, int NT, bool E8>
struct Tile {
  static constexpr int kHeads = 8 * NT;  // rows of a state
  static constexpr int TK = paged_tile(D, E8, 8 * NT), MT = TK / 16, kShift = paged_shift(D, E8, 8 * NT);
  static constexpr int kLanes = TK < 32 ? TK : 32, kRows = TK / kLanes;  // rows lane, lane + 32 of a tile are a lane's
  static constexpr int kRow = E8 && D == 64 ? 64 : 128;    // bytes of a box's row
  static constexpr int kCols = D * (E8 ? 1 : 2) / kRow;    // box columns of a tile
  static constexpr int kBox = 16 * kRow;                   // bytes of a box
  static constexpr int kChunk = TK * kRow;                 // of a box column
  static constexpr int kTensor = kCols * kChunk;           // K or V of a tile
  static constexpr int kStage = 2 * kTensor;
  static constexpr int NS = 2;
  static constexpr int kRing = NS * kStage;
  using Mask = typename std::conditional<TK == 64, uint64_t, uint32_t>::type;  // of a tile's rows
  static constexpr Mask kAll = TK == 16 ? Mask(0xffff) : ~Mask(0);
};

// One warp's running state of one group's query heads over e4m3 tiles.
template <int D, int NT>
struct State8 {
  using T = Tile<D, NT, true>;
  float m[NT][2], l[NT][2], mo[NT][2], o[NT][D / 16][4];  // m: of the scores; mo: of score + value power
  uint32_t qf[NT][D / 16][2];
  float qs[NT][2];  // takes a product to the score in the log2 domain, without the key's power

  // Three bits rotated by one (heads of 64: as they are): see above.
  static __device__ __forceinline__ int rot(int x) { return D == 64 ? x : (x >> 1) | ((x & 1) << 2); }

  __device__ __forceinline__ void begin(const void* q, int64_t bh0, int G, float scale_log2) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + (lane >> 2);
      const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(q) + (bh0 + (g < G ? g : 0)) * D;
      uint2 x[D / 16];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        // product i's dims of this lane: four from here on (State8::step's order)
        const int c = D == 64 ? 16 * t + 4 * i : (i >> 3) * 128 + ((i >> 2) & 1) * 64 + 16 * t + 4 * (i & 3);
        x[i] = g < G ? __ldg(reinterpret_cast<const uint2*>(row + c)) : make_uint2(0, 0);
        top = __vmaxu2(__vmaxu2(top, x[i].x & 0x7fff7fffu), x[i].y & 0x7fff7fffu);
      }
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = max(top >> 16, top & 0xffffu);
      // the row's power: 2^(14 - exponent), within 2^-113 .. 2^120 (rows of 0, infinities and NaN are as good with any)
      int e = 14 - ((int)(top >> 7) - 127);
      e = e > 120 ? 120 : e;
      const float f = __uint_as_float((uint32_t)(e + 127) << 23);
      const float back = scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        qf[nt][i][0] = half2_of(__uint_as_float(x[i].x << 16) * f, __uint_as_float(x[i].x & 0xffff0000u) * f);
        qf[nt][i][1] = half2_of(__uint_as_float(x[i].y << 16) * f, __uint_as_float(x[i].y & 0xffff0000u) * f);
      }
      qs[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      qs[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
      m[nt][0] = m[nt][1] = mo[nt][0] = mo[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
    }
  }

  __device__ __forceinline__ float sum(int nt, int e) const {
    float s = l[nt][e];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
  }

  // Adds a landed tile at `tile` (K, then V); mask (not 0): its rows that hold a key;
  // kx, vx: the exponent bytes of the lane's rows.
  __device__ __forceinline__ void step(uint8_t* tile, typename T::Mask mask, const uint32_t (&kx)[T::kRows],
                                       const uint32_t (&vx)[T::kRows]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int MT = T::MT;
    if (mask != T::kAll) {
      // value rows without a key: zeros (their weights are 0, and 0 x NaN is NaN)
      for (int r = 0; r < T::TK; ++r) {
        if ((mask >> r) & 1u) continue;
        for (int i = lane; i < T::kCols * (T::kRow / 16); i += 32)
          *reinterpret_cast<uint4*>(tile + T::kTensor + (i / (T::kRow / 16)) * T::kChunk + r * T::kRow +
                                    (i % (T::kRow / 16)) * 16) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    const uint32_t ks = ptx::smem_addr(tile), vs = ks + T::kTensor;
    const int kr = rot(g);  // this lane's first key row of each 16
    float s[NT][MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      constexpr int A = NT == 2 && D >= 128 ? 2 : 4;  // sums that do not wait on each other, by the registers left
      float acc[NT][A][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int a = 0; a < A; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nt][a][j] = 0.f;
#pragma unroll
      for (int i0 = 0; i0 < D / 16; i0 += 4) {  // 16 bytes of two rows: four products
        uint32_t at;
        if (D == 64) at = ks + (mt * 16 + kr) * 64 + ((t ^ ((kr >> 1) & 3)) << 4);
        else at = ks + (i0 >> 3) * T::kChunk + (mt * 16 + kr) * 128 + (((((i0 >> 2) & 1) * 4 + t) ^ kr) << 4);
        const uint4 a = lds16(at), b = lds16(at + 8 * T::kRow);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t f[4] = {e4m3::to_half2(wa[w]), e4m3::to_half2(wb[w]), e4m3::to_half2_hi(wa[w]),
                                 e4m3::to_half2_hi(wb[w])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816_f16(acc[nt][w % A], f, qf[nt][i0 + w][0], qf[nt][i0 + w][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[nt][mt][j] = A == 4 ? (acc[nt][0][j] + acc[nt][1][j]) + (acc[nt][A - 2][j] + acc[nt][A - 1][j])
                                : acc[nt][0][j] + acc[nt][1][j];
    }
    // the rows' powers, from the lane that loaded them
    float kp[T::kRows], vp[T::kRows];
#pragma unroll
    for (int i = 0; i < T::kRows; ++i) {
      kp[i] = e4m3::power((int)kx[i]);
      vp[i] = vx[i] == 255u ? __uint_as_float(0x7fffffffu) : (float)((int)vx[i] - 127);
    }
    float ve[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = mt * 16 + r * 8 + kr;
        const float k2 = __shfl_sync(0xffffffffu, kp[mt / 2 % T::kRows], row & 31);
        ve[mt][r] = __shfl_sync(0xffffffffu, vp[mt / 2 % T::kRows], row & 31);
        const bool there = (mask >> row) & 1u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)  // (the powers first: either alone may take a product out of fp32's range)
            s[nt][mt][2 * r + e] = there ? s[nt][mt][2 * r + e] * (qs[nt][e] * k2) : -INFINITY;
        ve[mt][r] = there ? ve[mt][r] : 0.f;
      }
    float mx[NT][2], my[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[nt][e] = my[nt][e] = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mx[nt][e] = fmaxf(mx[nt][e], s[nt][mt][2 * r + e]);
            my[nt][e] = fmaxf(my[nt][e], s[nt][mt][2 * r + e] + ve[mt][r]);
          }
      }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
          my[nt][e] = fmaxf(my[nt][e], __shfl_xor_sync(0xffffffffu, my[nt][e], off));
        }
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[nt][e] = fmaxf(m[nt][e], mx[nt][e]);
        my[nt][e] = fmaxf(mo[nt][e], my[nt][e]);
        moved = moved || mx[nt][e] != m[nt][e] || my[nt][e] != mo[nt][e];
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[nt][e] *= m[nt][e] == mx[nt][e] ? 1.f : ptx::ex2(m[nt][e] - mx[nt][e]);
          alpha[e] = mo[nt][e] == my[nt][e] ? 1.f : ptx::ex2(mo[nt][e] - my[nt][e]);
          m[nt][e] = mx[nt][e];
          mo[nt][e] = my[nt][e];
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
    uint32_t wf[NT][MT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float ref[2], refo[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ref[e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
        refo[e] = (mo[nt][e] == -INFINITY ? 0.f : mo[nt][e]) - 14.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = s[nt][mt][2 * r + e];
            l[nt][e] += ptx::ex2(x - ref[e]);
            w[e] = ptx::ex2((x - refo[e]) + ve[mt][r]);
          }
          wf[nt][mt][r] = rows::movm_t(half2_of(w[0], w[1]));
        }
    }
    // O^T += V^T W^T: k index 2 t, 2 t + 1 (+ 8) is key row rot(2 t), rot(2 t + 1) (+ 8)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int ra = mt * 16 + rot(2 * t), rb = mt * 16 + rot(2 * t + 1);
      if (D == 64) {  // dims 8 g .. 8 g + 7
        const uint32_t col = (g & 1) * 8, c = g >> 1;
        const uint2 a = lds8(vs + ra * 64 + ((c ^ ((ra >> 1) & 3)) << 4) + col);
        const uint2 b = lds8(vs + rb * 64 + ((c ^ ((rb >> 1) & 3)) << 4) + col);
        const uint2 cc = lds8(vs + (ra + 8) * 64 + ((c ^ ((ra >> 1) & 3)) << 4) + col);
        const uint2 d = lds8(vs + (rb + 8) * 64 + ((c ^ ((rb >> 1) & 3)) << 4) + col);
        add_values(0, a.x, b.x, cc.x, d.x, wf, mt);
        add_values(2, a.y, b.y, cc.y, d.y, wf, mt);
      } else {  // dims 16 rot(g) .. + 15 of each box column
#pragma unroll
        for (int ch = 0; ch < T::kCols; ++ch) {
          const uint32_t at = vs + ch * T::kChunk;
          const uint4 a = lds16(at + ra * 128 + ((kr ^ (ra & 7)) << 4)), b = lds16(at + rb * 128 + ((kr ^ (rb & 7)) << 4));
          const uint4 c = lds16(at + (ra + 8) * 128 + ((kr ^ (ra & 7)) << 4)),
                      d = lds16(at + (rb + 8) * 128 + ((kr ^ (rb & 7)) << 4));
          add_values(ch * 8, a.x, b.x, c.x, d.x, wf, mt);
          add_values(ch * 8 + 2, a.y, b.y, c.y, d.y, wf, mt);
          add_values(ch * 8 + 4, a.z, b.z, c.z, d.z, wf, mt);
          add_values(ch * 8 + 6, a.w, b.w, c.w, d.w, wf, mt);
        }
      }
    }
  }

  // Products i and i + 1: four dims of the key rows a, b (k = 2 t, 2 t + 1) and c, d (+ 8).
  __device__ __forceinline__ void add_values(int i, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                             const uint32_t (&wf)[NT][T::MT][2], int mt) {
    const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
    const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
    const uint32_t f0[4] = {e4m3::to_half2(ab0), e4m3::to_half2_hi(ab0), e4m3::to_half2(cd0), e4m3::to_half2_hi(cd0)};
    const uint32_t f1[4] = {e4m3::to_half2(ab1), e4m3::to_half2_hi(ab1), e4m3::to_half2(cd1), e4m3::to_half2_hi(cd1)};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma16816_f16(o[nt][i], f0, wf[nt][mt][0], wf[nt][mt][1]);
      mma16816_f16(o[nt][i + 1], f1, wf[nt][mt][0], wf[nt][mt][1]);
    }
  }

  // The state: O [G][D] against the softmax's reference m, and (m, sum) [G][2].
  __device__ __forceinline__ void store(float* to_o, float* to_ml, int G) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float z = sum(nt, e);
        const int head = nt * 8 + (lane & 3) * 2 + e;
        if (head >= G) continue;
        if (lane < 4) *reinterpret_cast<float2*>(to_ml + head * 2) = make_float2(m[nt][e], z);
        // times 2^(mo - 14 - m), its root twice: mo - m lies in [-127, 127], and ex2 gives zeros below 2^-126
        const float f = m[nt][e] == -INFINITY ? 1.f : ptx::ex2(0.5f * (mo[nt][e] - 14.f - m[nt][e]));
        float* dst = to_o + head * D + rot(lane >> 2) * (D == 64 ? 8 : 16);
#pragma unroll
        for (int i = 0; i < D / 16; i += 2) {
          float* to = dst + (D == 64 ? 2 * i : (i >> 3) * 128 + 2 * (i & 7));
          *reinterpret_cast<float4*>(to) = make_float4(o[nt][i][e] * f * f, o[nt][i][e + 2] * f * f,
                                                       o[nt][i + 1][e] * f * f, o[nt][i + 1][e + 2] * f * f);
        }
      }
  }
};

// The same of a bf16 state.
template <int D, int NT>
__device__ __forceinline__ void store(const rows::State<D, NT>& st, float* to_o, float* to_ml, int G) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float s = st.sum(nt, e);
      const int head = nt * 8 + (lane & 3) * 2 + e;
      if (head >= G) continue;
      if (lane < 4) *reinterpret_cast<float2*>(to_ml + head * 2) = make_float2(st.m[nt][e], s);
      float* dst = to_o + head * D + (lane >> 2);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        dst[i * 16] = st.o[nt][i][e];
        dst[i * 16 + 8] = st.o[nt][i][e + 2];
      }
    }
}
template <int D, int NT>
__device__ __forceinline__ void store(State8<D, NT>& st, float* to_o, float* to_ml, int G) {
  st.store(to_o, to_ml, G);
}

template <int D, int NT, bool E8>
using StateOf = typename std::conditional<E8, State8<D, NT>, rows::State<D, NT>>::type;

// Begins a group's state, with its queries.
template <int D, int NT>
__device__ __forceinline__ void begin(State8<D, NT>& st, const DecodePagedParams& p, int64_t bh0, int G) {
  st.begin(p.q, bh0, G, p.scale_log2);
}
template <int D, int NT>
__device__ __forceinline__ void begin(rows::State<D, NT>& st, const DecodePagedParams& p, int64_t bh0, int G) {
  st.begin(p.q, bh0, G);
}
// Adds a landed tile (mask: not 0).
template <int D, int NT, class T = Tile<D, NT, true>>
__device__ __forceinline__ void add_tile(State8<D, NT>& st, const DecodePagedParams& p, uint8_t* tile,
                                         typename T::Mask mask, const uint32_t (&kx)[T::kRows],
                                         const uint32_t (&vx)[T::kRows]) {
  st.step(tile, mask, kx, vx);
}
template <int D, int NT, class T = Tile<D, NT, false>>
__device__ __forceinline__ void add_tile(rows::State<D, NT>& st, const DecodePagedParams& p, uint8_t* tile, uint32_t mask,
                                         const uint32_t (&)[T::kRows], const uint32_t (&)[T::kRows]) {
  st.step(rows::lane_k(ptx::smem_addr(tile)), rows::lane_v(ptx::smem_addr(tile) + T::kTensor), tile + T::kTensor, mask,
          p.scale_log2);
}

__device__ __forceinline__ int cached_keys(const DecodePagedParams& p, int b) {
  const int len = p.seq_lens ? __ldg(p.seq_lens + b) : p.L;
  return len < 0 ? 0 : (len > p.L ? p.L : len);
}

// Where a tile lies: sequence b, key/value head h, tile t of its list.
struct Cursor {
  int b, h, t;
  KeySpan s;
};

// Loads the cursor's tile into `stage` of a warp's ring, a lane per copy; returns its rows
// that hold a visible key, and (eight bits) the exponent bytes of rows lane, lane + 32.
template <int D, int NT, bool E8, class T = Tile<D, NT, E8>>
__device__ __forceinline__ typename T::Mask issue_tile(const DecodePagedParams& p, uint8_t* ring, uint64_t* full,
                                                       const Cursor& f, int stage, uint32_t (&kx)[T::kRows],
                                                       uint32_t (&vx)[T::kRows]) {
  constexpr int MT = T::MT, NS = T::NS;
  const int lane = threadIdx.x & 31, G = p.H / p.H_kv;
  const int at = (f.t < f.s.head ? f.t : f.s.t0 + f.t - f.s.head) << T::kShift;  // position of its first key
  uint32_t half[2] = {0, 0};
  int id[T::kRows], r[T::kRows];
#pragma unroll
  for (int i = 0; i < T::kRows; ++i) {
    const int pos = at + lane + 32 * i;
    bool seen = lane < T::kLanes && pos < f.s.len && (pos >= f.s.w0 || pos < p.first);
    const int j = (uint32_t)pos / (uint32_t)p.page;
    r[i] = pos - j * p.page;
    id[i] = seen ? __ldg(p.table + (int64_t)f.b * p.table_pages + j) : -1;
    seen = seen && (uint32_t)id[i] < (uint32_t)p.n_pages;
    half[i] = __ballot_sync(0xffffffffu, seen);
    if (E8) {
      kx[i] = vx[i] = 0;
      if (seen) {
        kx[i] = __ldg(p.exps[0] + id[i] * p.exp_page[0] + f.h * p.exp_head[0] + r[i] * p.exp_row[0]);
        vx[i] = __ldg(p.exps[1] + id[i] * p.exp_page[1] + f.h * p.exp_head[1] + r[i] * p.exp_row[1]);
      }
    }
  }
  // a list's queries into L1, for the state that begins two tiles later
  if (f.t == 0 && lane * 64 < G * D)
    ptx::prefetch_l1(reinterpret_cast<const __nv_bfloat16*>(p.q) + (int64_t)(f.b * p.H_kv + f.h) * G * D + lane * 64);
  constexpr int kPer = T::kCols * 2;  // copies per box of 16 keys (of one page)
  const int x = lane / kPer, col = (lane >> 1) % T::kCols, tensor = lane & 1;
  uint32_t bytes = 0;
#pragma unroll
  for (int y = 0; y < MT; ++y) bytes += (half[y >> 1] >> (16 * (y & 1))) & 0xffffu ? kPer * (uint32_t)T::kBox : 0u;
  if (lane == 0) ptx::mbar_arrive_expect_tx(full + stage, bytes);
  __syncwarp();
  // the box's page and row from the lane of a visible key of it
  const uint32_t box = x < MT ? (half[MT > 2 ? x >> 1 : 0] >> (16 * (x & 1))) & 0xffffu : 0u;
  const int from = 16 * (x & 1) + (box ? __ffs(box) - 1 : 0);
  int page = __shfl_sync(0xffffffffu, id[0], from), row = __shfl_sync(0xffffffffu, r[0], from);
  if (T::kRows == 2) {
    const int id1 = __shfl_sync(0xffffffffu, id[T::kRows - 1], from), r1 = __shfl_sync(0xffffffffu, r[T::kRows - 1], from);
    if (x >= 2) page = id1, row = r1;
  }
  row &= ~15;
  if (box && debug_check(p.err, page >= 0 && page < p.n_pages && row >= 0 && row < p.page && f.h < p.H_kv && stage < NS,
                         kSiteLoad))
    ptx::tma_load_4d(ring + stage * T::kStage + tensor * T::kTensor + col * T::kChunk + x * T::kBox,
                     tensor ? &p.tv : &p.tk, full + stage, col * (E8 ? 128 : 64), row, f.h, page);
  if constexpr (T::TK == 64) return (uint64_t)half[1] << 32 | half[0];
  else return half[0];
}

// After a wait that gave up: the abort flag, the error word, and time for the copies in
// flight to land before the shared memory goes.
__device__ __forceinline__ void give_up(const DecodePagedParams& p, volatile int* abort_flag) {
  if ((threadIdx.x & 31) == 0) {
    *abort_flag = 1;
    atomicOr(p.err, kErrProducer);
  }
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 0; it < 0x10000000u && ptx::globaltimer_ns() - t0 < 2000000ull; ++it) { }
}

template <int D, int NT, bool E8>
__device__ __forceinline__ void paged_work(const DecodePagedParams& p, int w, int W, uint8_t* ring, uint64_t* full,
                                           volatile int* abort_flag) {
  using T = Tile<D, NT, E8>;
  constexpr int NS = T::NS;
  static_assert(NS == 2, "the masks of the stages are two registers");
  const int lane = threadIdx.x & 31;
  const int G = p.H / p.H_kv;
  auto span = [&](int b) { return key_span(b < p.B ? cached_keys(p, b) : 0, p.window, p.first, T::kShift); };

  // this warp's share of all lists' tiles
  int sum = 0;
  for (int b = lane; b < p.B; b += 32) sum += span(b).tiles;
  const int total = __reduce_add_sync(0xffffffffu, sum) * p.H_kv;
  const int per = total ? (total - 1) / W + 1 : 1;
  if (w == 0 && lane == 0) p.group_start[p.B * p.H_kv] = per;
  const int64_t first = (int64_t)w * per;
  if (first >= total) return;
  const int x0 = (int)first, n_mine = total - x0 < per ? total - x0 : per;

  // the sequence that holds tile x0: running sums of 32 sequences at a time
  Cursor c;
  {
    int before = 0, b0 = 0, mine, incl;
    uint32_t past;
    for (;; b0 += 32) {
      mine = span(b0 + lane).tiles * p.H_kv;
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
    c.s = span(c.b);
    c.h = (x0 - start) / c.s.tiles;
    c.t = x0 - start - c.h * c.s.tiles;
  }
  auto advance = [&](Cursor& k) {
    if (++k.t < k.s.tiles) return;
    k.t = 0;
    if (++k.h < p.H_kv) return;
    k.h = 0;
    do k.s = span(++k.b);
    while (k.b < p.B && k.s.tiles == 0);
  };
  StateOf<D, NT, E8> st;
  Cursor f = c;  // the last tile loaded
  typename T::Mask masks[2] = {0, 0};
  uint32_t kx[2][T::kRows] = {}, vx[2][T::kRows] = {};
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (n < n_mine) {
      if (n) advance(f);
      if (n || p.selftest != 1) masks[n] = issue_tile<D, NT, E8>(p, ring, full, f, n, kx[n], vx[n]);
    }
  for (int n = 0; n < n_mine; ++n) {
    if (n == 0 || c.t == 0) {
      if (c.t == 0 && lane == 0) p.group_start[c.b * p.H_kv + c.h] = x0 + n;
      begin(st, p, (int64_t)c.b * p.H + c.h * G, G);
    }
    const int stage = n & 1;
    const typename T::Mask mask = stage ? masks[1] : masks[0];
    const bool got = ptx::mbar_wait(full + stage, (n >> 1) & 1, p.timeout_ns, abort_flag);
    if (!__all_sync(0xffffffffu, got)) return give_up(p, abort_flag);
    if (mask) {  // warp-uniform
      uint32_t k[T::kRows], v[T::kRows];
#pragma unroll
      for (int i = 0; i < T::kRows; ++i) {
        k[i] = stage ? kx[1][i] : kx[0][i];
        v[i] = stage ? vx[1][i] : vx[0][i];
      }
      add_tile(st, p, ring + stage * T::kStage, mask, k, v);
    }
    __syncwarp();
    if (n + NS < n_mine) {
      if (mask != T::kAll) ptx::fence_proxy_async_shared();  // the zeros of step before the copy that overwrites them
      __syncwarp();
      advance(f);
      uint32_t k[T::kRows], v[T::kRows];
      const typename T::Mask x = issue_tile<D, NT, E8>(p, ring, full, f, stage, k, v);
      masks[0] = stage ? masks[0] : x;
      masks[1] = stage ? x : masks[1];
#pragma unroll
      for (int i = 0; i < T::kRows && E8; ++i) {
        kx[0][i] = stage ? kx[0][i] : k[i];
        kx[1][i] = stage ? k[i] : kx[1][i];
        vx[0][i] = stage ? vx[0][i] : v[i];
        vx[1][i] = stage ? v[i] : vx[1][i];
      }
    }
    const int g = c.b * p.H_kv + c.h;
    const bool last = n + 1 == n_mine;
    if (last || c.t + 1 == c.s.tiles) {
      const int64_t at = ((int64_t)w + g) * G;
      store(st, p.part_o + at * D, p.part_ml + at * 2, G);
    }
    if (!last) advance(c);
  }
}

template <class T>
constexpr size_t paged_smem(int warps) {
  return 1024 + (size_t)warps * (T::kRing + T::NS * 8) + 16;
}

// One CTA per SM, of p.warps warps; warp w of the grid is warp w / grid of CTA w % grid,
// so that few shares spread over the SMs.
template <int D, int NT, bool E8>
__global__ void __launch_bounds__(32 * decode_rows_warps(D), 1)
    decode_paged_kernel(const __grid_constant__ DecodePagedParams p) {
  using T = Tile<D, NT, E8>;
  const int warps = blockDim.x >> 5;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + warps * T::kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + warps * T::NS);
  if (threadIdx.x < warps * T::NS) ptx::mbar_init(full + threadIdx.x, 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  ptx::fence_barrier_init();
  __syncthreads();
  after_previous();
  const int warp = threadIdx.x >> 5;
  paged_work<D, NT, E8>(p, warp * gridDim.x + blockIdx.x, gridDim.x * warps, ring + warp * T::kRing, full + warp * T::NS,
                        abort_flag);
}

// Few groups with short lists: a cluster of CTAs a group, warps in turn with a tile each, no
// states in memory and no second launch.  The warps of a CTA meet in its shared memory, the
// CTAs of the cluster in each other's, each CTA finishing a share of the G x D outputs.
template <class T, int D>
struct ClusterSmem {
  static constexpr int kWarps = decode_rows_warps(D), kUnits = kWarps + 1;  // the warps' states and the CTA's
  static constexpr size_t kRing = (size_t)kWarps * T::kRing, kStates = (size_t)kUnits * T::kHeads * (D + 2) * 4;
  static constexpr size_t kBytes = 1024 + (kRing > kStates ? kRing : kStates) + kWarps * T::NS * 8 + 16;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D, int NT, bool E8>
__global__ void __launch_bounds__(32 * decode_rows_warps(D), 1)
    decode_paged_cluster_kernel(const __grid_constant__ DecodePagedParams p) {
  using T = Tile<D, NT, E8>;
  using Mem = ClusterSmem<T, D>;
  constexpr int W = Mem::kWarps, HP = T::kHeads, NS = T::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + Mem::kBytes - 1024 - W * NS * 8 - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + W * NS);
  const int warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, bkv = blockIdx.x / p.cluster, G = p.H / p.H_kv;
  const int64_t bh0 = (int64_t)bkv * G;
  if (threadIdx.x < W * NS) ptx::mbar_init(bars + threadIdx.x, 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  ptx::fence_barrier_init();
  __syncthreads();
  after_previous();

  uint8_t* ring = base + warp * T::kRing;
  uint64_t* full = bars + warp * NS;
  Cursor c;
  c.b = bkv / p.H_kv;
  c.h = bkv - c.b * p.H_kv;
  c.s = key_span(cached_keys(p, c.b), p.window, p.first, T::kShift);
  const int first = rank + warp * p.cluster, step = p.cluster * W;  // this warp's tiles: first, first + step, ..
  const int mine = first < c.s.tiles ? (c.s.tiles - first + step - 1) / step : 0;
  typename T::Mask mask = 0, mask1 = 0;  // of the tile at hand and the one behind it
  uint32_t kx[T::kRows] = {}, vx[T::kRows] = {}, kx1[T::kRows] = {}, vx1[T::kRows] = {};
  c.t = first;
  if (mine > 0 && p.selftest != 1) mask = issue_tile<D, NT, E8>(p, ring, full, c, 0, kx, vx);
  c.t += step;
  if (mine > 1) mask1 = issue_tile<D, NT, E8>(p, ring, full, c, 1, kx1, vx1);
  StateOf<D, NT, E8> st;
  begin(st, p, bh0, G);
  for (int n = 0; n < mine; ++n) {
    const int stage = n & 1;
    const bool got = ptx::mbar_wait(full + stage, (n >> 1) & 1, p.timeout_ns, abort_flag);
    if (!__all_sync(0xffffffffu, got)) {
      give_up(p, abort_flag);
      break;
    }
    if (mask) add_tile(st, p, ring + stage * T::kStage, mask, kx, vx);  // warp-uniform
    __syncwarp();
    if (mask != T::kAll) ptx::fence_proxy_async_shared();  // the zeros of a step before the copy that overwrites them
    __syncwarp();
    mask = mask1;
#pragma unroll
    for (int i = 0; i < T::kRows; ++i) kx[i] = kx1[i], vx[i] = vx1[i];
    if (n + NS < mine) {
      c.t += step;
      mask1 = issue_tile<D, NT, E8>(p, ring, full, c, stage, kx1, vx1);
    }
  }
  __syncthreads();  // every tile of every warp is read
  // over the rings: O [W + 1][HP][D], then reference and sum [W + 1][HP][2]
  float* so = reinterpret_cast<float*>(base);
  float* sml = so + Mem::kUnits * HP * D;
  store(st, so + warp * HP * D, sml + warp * HP * 2, G);
  __syncthreads();
  for (int x = threadIdx.x; x < G * D; x += 32 * W) {  // the CTA's state
    const int g = x / D;
    float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, sml[(w * HP + g) * 2]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float mw = sml[(w * HP + g) * 2], e = mw == M ? 1.f : ptx::ex2(mw - M);
      L = fmaf(sml[(w * HP + g) * 2 + 1], e, L);
      O = fmaf(so[w * HP * D + x], e, O);
    }
    so[W * HP * D + x] = O;
    if (x % D == 0) {
      sml[(W * HP + g) * 2] = M;
      sml[(W * HP + g) * 2 + 1] = L;
    }
  }
  auto all = [&]() {
    if (p.cluster > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
  };
  all();
  // this CTA's share of the outputs (a CTA that gave up leaves no number behind: its
  // cluster's outputs are then undefined, and the error word says so)
  const int share = (G * D + p.cluster - 1) / p.cluster;
  const int end = (rank + 1) * share < G * D ? (rank + 1) * share : G * D;
  for (int x = rank * share + threadIdx.x; x < end; x += 32 * W) {
    const int g = x / D;
    const float* ml = sml + (W * HP + g) * 2;
    const float* o = so + W * HP * D + x;
    const float b2 = p.sink ? p.sink[c.h * G + g] * 1.4426950408889634f : -INFINITY;
    float mr[8], lr[8], ors[8], M = b2;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      mr[r] = r < p.cluster ? rows::cluster_ld(ml, r) : -INFINITY;
      lr[r] = r < p.cluster ? rows::cluster_ld(ml + 1, r) : 0.f;
      ors[r] = r < p.cluster ? rows::cluster_ld(o, r) : 0.f;
      M = fmaxf(M, mr[r]);
    }
    float z = b2 == -INFINITY ? 0.f : ptx::ex2(b2 - M), O = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float e = mr[r] == M ? 1.f : ptx::ex2(mr[r] - M);
      z = fmaf(lr[r], e, z);
      O = fmaf(ors[r], e, O);
    }
    reinterpret_cast<__nv_bfloat16*>(p.o)[bh0 * D + x] = __float2bfloat16_rn(z == 0.f ? 0.f : O / z);
    if (x % D == 0 && p.lse) p.lse[bh0 + g] = z == 0.f ? -INFINITY : (M + __log2f(z)) * 0.6931471805599453f;
  }
  if (p.cluster > 1) all();  // no CTA leaves while another reads its shared memory
}

template <int D, int NT, bool E8>
cudaError_t launch_cluster(const DecodePagedParams& p, cudaStream_t stream) {
  constexpr size_t smem = ClusterSmem<Tile<D, NT, E8>, D>::kBytes;
  auto kern = decode_paged_cluster_kernel<D, NT, E8>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kern, smem, &done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, (unsigned)(p.B * p.H_kv * p.cluster), 1, 32 * decode_rows_warps(D), smem, p.cluster, p, stream);
}

template <int D, int NT, bool E8>
cudaError_t launch_nt(const DecodePagedParams& p, cudaStream_t stream) {
  if (p.cluster) return launch_cluster<D, NT, E8>(p, stream);
  using T = Tile<D, NT, E8>;
  constexpr size_t most = paged_smem<T>(decode_rows_warps(D));
  static_assert(most <= 227 * 1024, "shared memory");
  if (p.warps < 1 || p.warps > decode_rows_warps(D)) return cudaErrorInvalidValue;
  auto kern = decode_paged_kernel<D, NT, E8>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kern, most, &done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, (unsigned)p.ctas, 1, 32 * p.warps, paged_smem<T>(p.warps), 1, p, stream);
}

}  // namespace

cudaError_t launch_decode_paged(const DecodePagedParams& p, int d, bool e4m3, cudaStream_t stream) {
  const int nt = (p.H / p.H_kv + 7) / 8;
  switch ((d * 4 + nt) * 2 + (e4m3 ? 1 : 0)) {
#define MATTN_CASE(D, NT)                                                 \
  case (D * 4 + NT) * 2: return launch_nt<D, NT, false>(p, stream);       \
  case (D * 4 + NT) * 2 + 1: return launch_nt<D, NT, true>(p, stream);
    MATTN_CASE(64, 1)
    MATTN_CASE(64, 2)
    MATTN_CASE(128, 1)
    MATTN_CASE(128, 2)
    MATTN_CASE(256, 1)
    MATTN_CASE(256, 2)
#undef MATTN_CASE
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mattn
