// Device pieces that the packed forwards (attention_packed.cu, attention_packed_256.cu)
// share: their sequences and key tiles, values that are not finite, output rows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_ops.h"
#include "ptx.cuh"

namespace mattn {
namespace {

// Sequence b's rows and keys, inside the packed rows whatever the arrays hold.
struct Sequence {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Sequence sequence(const PackedParams& p, int b) {
  auto in = [](int x, int n) { return x < 0 ? 0 : (x > n ? n : x); };
  Sequence s;
  s.q0 = in(__ldg(p.cu_q + b), p.T);
  s.nq = in(__ldg(p.cu_q + b + 1), p.T) - s.q0;
  s.k0 = in(__ldg(p.cu_k + b), p.T_k);
  s.nk = in(__ldg(p.cu_k + b + 1), p.T_k) - s.k0;
  if (s.nq < 0) s.nq = 0;
  if (s.nk < 0) s.nk = 0;
  return s;
}

// The key tiles [lo, hi] of 2^SHIFT keys that the n rows at positions pos, pos + 1, .. see
// (n < 1 or lo > hi: none).
template <int SHIFT>
__device__ __forceinline__ void seen_tiles(const PackedParams& p, int pos, int n, int keys, int* lo, int* hi) {
  int last = keys - 1, first = 0;
  if (p.causal) {
    last = min(last, pos + n - 1);
    if (p.window) first = max(0, pos - p.window + 1);
  }
  *lo = first >> SHIFT;
  *hi = n > 0 && last >= first ? last >> SHIFT : -1;
  if (*hi < 0) *lo = 0;
}

// Whether a pair's rows and keys lie in the packed rows.
__device__ __forceinline__ bool in_bounds(const PackedParams& p, const PackedPair& x) {
  return !(x.q_row < 0 || x.q_row > p.T || x.rows > p.T - x.q_row || x.k_row < 0 || x.k_row > p.T_k || x.keys < 0 ||
           x.keys > p.T_k - x.k_row || x.pos0 < -p.T || x.pos0 > p.T_k);
}

// The 16-bit halves of x that are no infinity or NaN, and zeros for those that are.
__device__ __forceinline__ uint32_t clean(uint32_t x) { return x & ~__vcmpeq2(x & 0x7f807f80u, 0x7f807f80u); }

// A wait that may take as long as an item, whatever its keys take: `once` waits for up to the limit;
// given up after a limit without a K tile more (`tiles`, which their producer counts).  Every other
// wait is one for a tile's work.
template <class Once>
__device__ __forceinline__ bool item_wait(volatile uint32_t* tiles, volatile int* abort_flag, Once once) {
  for (uint32_t seen = *tiles;;) {
    if (once()) return true;
    const uint32_t now = *tiles;
    if (now == seen || *abort_flag) return false;
    seen = now;
  }
}

__device__ __forceinline__ void let_copies_land(volatile int* abort_flag) {
  if (!*abort_flag) return;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 0; it < 0x10000000u && ptx::globaltimer_ns() - t0 < 2000000ull; ++it) { }
}

// A weight is off by 2^-8 of itself at most once it is bf16, as P V takes it.  Over many keys
// such errors add up to the output's own rounding or less; over few, where outputs are largest,
// they are kept out of it as far as they are common to a row's weights (all of it for one
// key): the output is divided by the sum of the rounded weights.  The LSE takes that of the
// weights as they were.  So the rows whose last key is among their sequence's first 128, or whose
// window is of 64 keys at most: a row's own keys decide, so that a chunk's rows get the bits of the
// whole prompt's.  (Windows of 65 to 128 keys too took 10% more: 4 prompts of 4,096 with 8 heads of
// 128 34.4 us for 31.1.)  Eight prompts of 700 tokens in all 0.0020 off the 64-bit form where the
// other sum left 0.0023, in 11.2 us for 10.8.
__device__ __forceinline__ bool few_keys(const PackedParams& p, int hi) {  // hi: the row's last key
  return hi < 128 || (p.window && p.window <= 64);
}
// This thread's sum of the rounded weights in N columns (pairs) of tensor memory.
template <int N>
__device__ __forceinline__ float rounded_sum(uint32_t p_tmem) {
  float a = 0.f, b = 0.f;
#pragma unroll 1
  for (int c = 0; c < N; c += 16) {
    float x[16];
    ptx::tmem_ld16(p_tmem + c, x);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      a += __uint_as_float(__float_as_uint(x[k]) << 16);
      b += __uint_as_float(__float_as_uint(x[k]) & 0xffff0000u);
    }
  }
  return a + b;
}

// 32 bytes of an output row, written once and not read again here: first out of L2.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&x)[8], uint64_t policy) {
  asm volatile("st.global.L1::no_allocate.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(p),
               "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "l"(policy)
               : "memory");
}

}  // namespace
}  // namespace mattn
