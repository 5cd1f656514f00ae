// Decode attention over the sequences' own keys or their selected blocks (the
// row worker of decode_rows.cuh on every warp), and the merge of all states
// of a decode step's operators, for sm_103a.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode_ops.h"
#include "decode_rows.cuh"
#include "kernel_params.h"
#include "ptx.cuh"

namespace mattn {
namespace {

constexpr float kLog2eR = 1.4426950408889634f;
constexpr float kLn2R = 0.6931471805599453f;

template <int D>
constexpr size_t rows_smem(int warps) {
  return 1024 + (size_t)warps * (rows::Geo<D>::kRing + rows::Geo<D>::NS * 8) + 16;
}

// One CTA per SM it runs on, of p.warps warps; warp w of the grid is warp
// w / grid of CTA w % grid, so that few shares spread over the SMs.
template <int D, int NT>
__global__ void __launch_bounds__(32 * decode_rows_warps(D), 1)
    decode_rows_kernel(const __grid_constant__ DecodeRowsParams p) {
  using Geo = rows::Geo<D>;
  const int warps = blockDim.x >> 5;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + warps * Geo::kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + warps * Geo::NS);
  if (threadIdx.x < warps * Geo::NS) ptx::mbar_init(full + threadIdx.x, 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  ptx::fence_barrier_init();
  __syncthreads();
  after_previous();
  const int warp = threadIdx.x >> 5;
  rows::work<D, NT>(p, warp * gridDim.x + blockIdx.x, gridDim.x * warps, ring + warp * Geo::kRing,
                    full + warp * Geo::NS, abort_flag);
}

template <int D, int NT>
cudaError_t launch_nt(const DecodeRowsParams& p, cudaStream_t stream) {
  constexpr size_t most = rows_smem<D>(decode_rows_warps(D));
  static_assert(most <= 227 * 1024, "shared memory");
  if (p.warps < 1 || p.warps > decode_rows_warps(D)) return cudaErrorInvalidValue;
  auto kern = decode_rows_kernel<D, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kern, most, &done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, (unsigned)p.ctas, 1, 32 * p.warps, rows_smem<D>(p.warps), 1, p, stream);
}

// Few groups or short lists: a cluster of CTAs per (sequence, key/value head),
// one warp's tile after another's, no states in memory and no second launch.
// The warps of a CTA meet in its shared memory, the CTAs of the cluster in each
// other's, each CTA finishing a share of the G x D outputs.
constexpr int kListIds = 1024;  // list entries that fit the kernel's table

template <int D, int NT, int W>
struct ListSmem {
  static constexpr int kWarps = W, HP = 8 * NT;
  static constexpr size_t kRing = (size_t)kWarps * rows::Geo<D>::kRing;
  // over the ring, once every tile is read: the warps' states, then the CTA's
  static constexpr size_t kStates = (size_t)(kWarps + 1) * HP * (D + 2) * 4;
  static_assert(kStates <= kRing, "the states must fit in the ring");
  static constexpr size_t kBytes = 1024 + kRing + kWarps * rows::Geo<D>::NS * 8 + 16 + kListIds * 4;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D, int NT, int W>
__global__ void __launch_bounds__(32 * W, 1)
    decode_lists_kernel(const __grid_constant__ DecodeRowsParams p) {
  using Geo = rows::Geo<D>;
  using Mem = ListSmem<D, NT, W>;
  constexpr int kWarps = Mem::kWarps, MT = Geo::MT, NS = Geo::NS, HP = Mem::HP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring_all = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_all = reinterpret_cast<uint64_t*>(ring_all + Mem::kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full_all + kWarps * NS);
  int* ids = reinterpret_cast<int*>(full_all + kWarps * NS + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.cluster, bkv = blockIdx.x / p.cluster;
  const int b = bkv / p.H_kv, G = p.H / p.H_kv;
  const int64_t bh0 = (int64_t)bkv * G;
  if (threadIdx.x < kWarps * NS) ptx::mbar_init(full_all + threadIdx.x, 1);
  if (threadIdx.x == 0) *abort_flag = 0;
  ptx::fence_barrier_init();
  after_previous();
  for (int i = threadIdx.x; i < p.top_k; i += 32 * kWarps) ids[i] = __ldg(p.ids + (int64_t)bkv * p.top_k + i);
  const int len = rows::cached_keys(p, b);
  __syncthreads();

  uint8_t* ring = ring_all + warp * Geo::kRing;
  uint64_t* full = full_all + warp * NS;
  const int blocks = (len + p.block - 1) / p.block;
  const int first = rank + warp * p.cluster, step = p.cluster * kWarps;  // this warp's tiles: first, first + step, ..
  const int mine = first < p.list_tiles ? (p.list_tiles - first + step - 1) / step : 0;
  auto issue = [&](int n) -> uint32_t {
    int pos[MT], cnt[MT];
#pragma unroll
    for (int x = 0; x < MT; ++x) {
      const int box = (first + n * step) * MT + x, j = box / p.box16;
      const int id = j < p.top_k ? ids[j] : -1;
      pos[x] = (uint32_t)id < (uint32_t)blocks ? id * p.block + ((box - j * p.box16) << 4) : len;
      const int left = len - pos[x];
      cnt[x] = left < 0 ? 0 : (left < 16 ? left : 16);
    }
    return rows::issue_tile<D>(p, ring, full, n & 1, bkv, pos, cnt);
  };
  uint32_t masks[2] = {0, 0};
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (n < mine && (n || p.selftest != 1)) masks[n] = issue(n);
  rows::State<D, NT> st;
  st.begin(p.q, bh0, G);
  const uint32_t at_k = rows::lane_k(ptx::smem_addr(ring)), at_v = rows::lane_v(ptx::smem_addr(ring) + Geo::kTensor);
  for (int n = 0; n < mine; ++n) {
    const int stage = n & 1;
    const uint32_t mask = stage ? masks[1] : masks[0];
    if (!rows::await(p, full + stage, (n >> 1) & 1, abort_flag)) break;
    if (mask)  // warp-uniform
      st.step(at_k + stage * Geo::kStage, at_v + stage * Geo::kStage, ring + stage * Geo::kStage + Geo::kTensor, mask,
              p.scale_log2);
    __syncwarp();
    if (n + NS < mine) {
      if (mask != Geo::kAll) ptx::fence_proxy_async_shared();  // the zeros of step before the copy that overwrites them
      __syncwarp();
      const uint32_t x = issue(n + NS);
      if (stage) masks[1] = x;
      else masks[0] = x;
    }
  }
  __syncthreads();  // every tile of every warp is read
  // the warps' states: O [kWarps + 1][HP][D], then reference and sum [kWarps + 1][HP][2]
  float* so = reinterpret_cast<float*>(ring_all);
  float* sml = so + (kWarps + 1) * HP * D;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float s = st.sum(nt, e);
      const int head = nt * 8 + (lane & 3) * 2 + e;
      if (lane < 4) {
        sml[(warp * HP + head) * 2] = st.m[nt][e];
        sml[(warp * HP + head) * 2 + 1] = s;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        so[(warp * HP + head) * D + i * 16 + (lane >> 2)] = st.o[nt][i][e];
        so[(warp * HP + head) * D + i * 16 + 8 + (lane >> 2)] = st.o[nt][i][e + 2];
      }
    }
  __syncthreads();
  // the CTA's state
  for (int t = threadIdx.x; t < G * D; t += 32 * kWarps) {
    const int g = t / D, c = t % D;
    float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[(w * HP + g) * 2]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sml[(w * HP + g) * 2], e = mw == M ? 1.f : ptx::ex2(mw - M);
      L = fmaf(sml[(w * HP + g) * 2 + 1], e, L);
      O = fmaf(so[(w * HP + g) * D + c], e, O);
    }
    so[(kWarps * HP + g) * D + c] = O;
    if (c == 0) {
      sml[(kWarps * HP + g) * 2] = M;
      sml[(kWarps * HP + g) * 2 + 1] = L;
    }
  }
  if (p.cluster > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  // this CTA's share of the outputs (a CTA that gave up leaves no number behind:
  // its cluster's outputs are then undefined, and the error word says so)
  const int share = (G * D + p.cluster - 1) / p.cluster;
  const int t1 = (rank + 1) * share < G * D ? (rank + 1) * share : G * D;
  for (int t = rank * share + threadIdx.x; t < t1; t += 32 * kWarps) {
    const int g = t / D, c = t % D;
    const float* ml = sml + (kWarps * HP + g) * 2;
    const float* o = so + (kWarps * HP + g) * D + c;
    const float b2 = p.sink ? p.sink[(bkv % p.H_kv) * G + g] * kLog2eR : -INFINITY;
    float mr[8], M = b2;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      mr[r] = r < p.cluster ? rows::cluster_ld(ml, r) : -INFINITY;
      M = fmaxf(M, mr[r]);
    }
    float z = b2 == -INFINITY ? 0.f : ptx::ex2(b2 - M), O = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r < p.cluster) {
        const float e = mr[r] == M ? 1.f : ptx::ex2(mr[r] - M);
        z = fmaf(rows::cluster_ld(ml + 1, r), e, z);
        O = fmaf(rows::cluster_ld(o, r), e, O);
      }
    reinterpret_cast<__nv_bfloat16*>(p.o)[(bh0 + g) * D + c] = __float2bfloat16_rn(z == 0.f ? 0.f : O / z);
    if (c == 0 && p.lse) p.lse[bh0 + g] = z == 0.f ? -INFINITY : (M + __log2f(z)) * kLn2R;
  }
  if (p.cluster > 1) {  // no CTA leaves while another reads its shared memory
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <int D, int NT, int W>
cudaError_t launch_lists_w(const DecodeRowsParams& p, cudaStream_t stream) {
  auto kern = decode_lists_kernel<D, NT, W>;
  const size_t smem = ListSmem<D, NT, W>::kBytes;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(kern, smem, &done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, (unsigned)(p.B * p.H_kv * p.cluster), 1, 32 * W, smem, p.cluster, p,
                        stream);
}

template <int D, int NT>
cudaError_t launch_lists_nt(const DecodeRowsParams& p, cudaStream_t stream) {
  constexpr int W = decode_rows_warps(D);
  if (p.warps == W) return launch_lists_w<D, NT, W>(p, stream);
  if (p.warps == W / 2) return launch_lists_w<D, NT, W / 2>(p, stream);
  return cudaErrorInvalidValue;
}

// The merge.  Row (b, h)'s states: `na` of the prefix, then the pieces of its
// own list.  o = sum_s 2^(m_s - M) O_s / (sum_s 2^(m_s - M) l_s + exp(sink)).
// LPS lanes take a state (16 bytes each) of SL <= 128 dims of one row; WPR warps
// share them: four and 32 dims where there are few rows, down to one and 128.
// Bound by what each warp issues and by its chain of loads (the prefix's states,
// beside the place of the own ones; the own ones): a handful of states a warp,
// their references and values loaded together, pointers moved and not formed
// anew (2,048 rows of 18 states: 7.6 us with 16 states in flight a warp and a
// warp a row).

struct Running {
  float m, l;
  float4 o;
};

// Adds n states, `step` apart: reference and sum at `ml`, the lane's dims at `o`
// (ml_step and o_step floats from one to the next).
template <int kMergeBatch>
__device__ __forceinline__ void add_states(Running& r, const float* ml, const float* o, int n, int64_t ml_step,
                                           int64_t o_step) {
  for (; n > 0; n -= kMergeBatch) {
    float2 a[kMergeBatch];
    float4 x[kMergeBatch];
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      a[i] = make_float2(-INFINITY, 0.f);
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        a[i] = *reinterpret_cast<const float2*>(ml);
        x[i] = *reinterpret_cast<const float4*>(o);
        ml += ml_step;
        o += o_step;
      }
    }
    float m = r.m;
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) m = fmaxf(m, a[i].x);
    const float k = r.m == m ? 1.f : ptx::ex2(r.m - m);
    r.m = m;
    r.l *= k;
    r.o = make_float4(r.o.x * k, r.o.y * k, r.o.z * k, r.o.w * k);
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      const float e = a[i].x == m ? 1.f : ptx::ex2(a[i].x - m);
      r.l = fmaf(a[i].y, e, r.l);
      r.o.x = fmaf(x[i].x, e, r.o.x);
      r.o.y = fmaf(x[i].y, e, r.o.y);
      r.o.z = fmaf(x[i].z, e, r.o.z);
      r.o.w = fmaf(x[i].w, e, r.o.w);
    }
  }
}

template <int D, int SL, int WPR, int NB>
__global__ void __launch_bounds__(128) decode_merge_kernel(const __grid_constant__ MergeParams p) {
  constexpr int LPS = SL / 4, SPW = 32 / LPS, U = WPR * SPW;
  static_assert(SL <= 128, "a warp's lanes hold four dims each");
  static_assert(WPR == 4 || WPR == 2 || WPR == 1, "a CTA has four warps");
  __shared__ float sm_all[4 * SPW], sl_all[4 * SPW], so_all[4 * SPW][SL];
  const int all = threadIdx.x >> 5, warp = all % WPR, lane = threadIdx.x & 31;
  const int mine = all / WPR * U;  // the row's first unit in shared memory
  float *sm = sm_all + mine, *sl = sl_all + mine;
  float(*so)[SL] = so_all + mine;
  const int sub = lane / LPS, part = lane % LPS, unit = warp * SPW + sub;
  const int64_t bh = (int64_t)blockIdx.x * (4 / WPR) + all / WPR;
  if (bh >= (int64_t)p.B * p.H) return;  // (all warps of a row)
  const int c0 = blockIdx.y * SL;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H), G = p.H / p.H_kv;
  const int g = b * p.H_kv + h / G;
  const int64_t ra = (((int64_t)(h / G) * p.B + b) * G + h % G) * p.na;
  after_previous();
  // the pieces of the group's own list: warps w0 .. w0 + nb - 1 of decode_rows
  int tiles = 0, per = 1, start = 0;
  if (p.group_start) {
    per = p.group_start[p.B * p.H_kv];
    start = p.group_start[g];
    tiles = p.list_tiles;
    if (!tiles) {
      int len = p.seq_lens ? p.seq_lens[b] : p.L;
      len = len < 0 ? 0 : (len > p.L ? p.L : len);
      tiles = key_span(len, p.window, p.first, p.tile_shift).tiles;
    }
  }
  const float b2 = p.sink ? p.sink[h] * kLog2eR : -INFINITY;
  Running r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  // this unit's states: unit, unit + U, ..
  add_states<NB>(r, p.a_ml + (ra + unit) * 2, p.a_o + (ra + unit) * D + c0 + part * 4, (p.na - unit + U - 1) / U, U * 2, U * D);
  if (tiles) {
    // state s of the own list: slot w0 + s + g, head h % G of the group
    const ListPieces own = list_pieces(start, tiles, per, p.warps);
    const int64_t at = ((int64_t)own.w0 + g + unit) * G + h % G;
    add_states<NB>(r, p.b_ml + at * 2, p.b_o + at * D + c0 + part * 4, (own.n - unit + U - 1) / U, (int64_t)U * G * 2,
               (int64_t)U * G * D);
  }
  if (part == 0) {
    sm[unit] = r.m;
    sl[unit] = r.l;
  }
  *reinterpret_cast<float4*>(&so[unit][part * 4]) = r.o;
  if (WPR == 4) __syncthreads();
  else if (WPR == 2) asm volatile("bar.sync %0, 64;" ::"r"(1 + all / WPR) : "memory");
  else __syncwarp();
  float M = b2;
#pragma unroll
  for (int u = 0; u < U; ++u) M = fmaxf(M, sm[u]);
  float e[U], z = b2 == -INFINITY ? 0.f : ptx::ex2(b2 - M);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    e[u] = sm[u] == M ? 1.f : ptx::ex2(sm[u] - M);
    z = fmaf(sl[u], e[u], z);
  }
  for (int c = warp * 32 + lane; c < SL; c += WPR * 32) {
    float x = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) x = fmaf(so[u][c], e[u], x);
    reinterpret_cast<__nv_bfloat16*>(p.o)[bh * D + c0 + c] = __float2bfloat16_rn(z == 0.f ? 0.f : x / z);
  }
  if (lane == 0 && warp == 0 && blockIdx.y == 0 && p.lse) p.lse[bh] = z == 0.f ? -INFINITY : (M + __log2f(z)) * kLn2R;
}

template <int D, int SL, int WPR, int NB = 4>
cudaError_t launch_merge_sl(const MergeParams& p, cudaStream_t stream) {
  const int rows = p.B * p.H;
  return launch_chained(decode_merge_kernel<D, SL, WPR, NB>,
                        (unsigned)((rows + 4 / WPR - 1) / (4 / WPR)), D / SL, 128, 0, 1, p, stream);
}

template <int D>
cudaError_t launch_merge_d(const MergeParams& p, cudaStream_t stream) {
  // Warps of a row: four while they fill the SMs once, or twice where a row has the
  // states for them (shared prefix of 32K, 512 own keys, 8 key/value heads of 128, in us with
  // four, two and one: 1,536 rows 43.5, 47.3, 46.9; 2,048 54.4, 57.5, 56.7; 4,096 83.2,
  // 84.4, 80.1; 8,192 166.9, 168.4, 158.7).
  constexpr int SL = D < 128 ? D : 128;
  const int64_t warps = (int64_t)p.B * p.H * (D / SL), most = kPlanSms * 36;
  if (p.many && p.B * p.H <= kPlanSms) return launch_merge_sl<D, 32, 4, 16>(p, stream);
  if (p.B * p.H <= kPlanSms) return launch_merge_sl<D, 32, 4>(p, stream);
  if (warps * 4 <= (p.states >= 8 ? 2 * most : most)) return launch_merge_sl<D, SL, 4>(p, stream);
  if (warps * 2 <= most) return launch_merge_sl<D, SL, 2>(p, stream);
  return launch_merge_sl<D, SL, 1>(p, stream);
}

}  // namespace

cudaError_t launch_decode_rows(const DecodeRowsParams& p, int d, cudaStream_t stream) {
  const int nt = (p.H / p.H_kv + 7) / 8;
  switch (d * 4 + nt) {
    case 64 * 4 + 1: return launch_nt<64, 1>(p, stream);
    case 64 * 4 + 2: return launch_nt<64, 2>(p, stream);
    case 128 * 4 + 1: return launch_nt<128, 1>(p, stream);
    case 128 * 4 + 2: return launch_nt<128, 2>(p, stream);
    case 256 * 4 + 1: return launch_nt<256, 1>(p, stream);
    case 256 * 4 + 2: return launch_nt<256, 2>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_lists(const DecodeRowsParams& p, int d, cudaStream_t stream) {
  const int nt = (p.H / p.H_kv + 7) / 8;
  switch (d * 4 + nt) {
    case 64 * 4 + 1: return launch_lists_nt<64, 1>(p, stream);
    case 64 * 4 + 2: return launch_lists_nt<64, 2>(p, stream);
    case 128 * 4 + 1: return launch_lists_nt<128, 1>(p, stream);
    case 128 * 4 + 2: return launch_lists_nt<128, 2>(p, stream);
    case 256 * 4 + 1: return launch_lists_nt<256, 1>(p, stream);
    case 256 * 4 + 2: return launch_lists_nt<256, 2>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_merge(const MergeParams& p, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_merge_d<64>(p, stream);
    case 128: return launch_merge_d<128>(p, stream);
    case 256: return launch_merge_d<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

// Warps of a CTA of decode_rows_kernel, whose lists come to `tiles` tiles at most:
// half where each would have few (32 groups of 256 tiles of 128: 18.7 us with 12 warps,
// 17.0 with 6; 192 groups: 68.2 and 69.1).
int decode_share_warps(int64_t tiles, int d) {
  const int warps = decode_rows_warps(d);
  return tiles <= (int64_t)10 * kPlanSms * warps ? warps / 2 : warps;
}

// How block lists are read.  Clusters (decode_lists_kernel) need no states in
// memory and no merge, but leave SMs idle; equal shares (decode_rows_kernel)
// take them all.  More groups than SMs: CTAs of half the warps, two an SM, of
// which one loads while the other finishes (512 groups of 2,048 keys of 128: 91.7 us with
// 12 warps, 84.3 with 6, 90.0 in shares), but for a last wave that leaves the SMs
// half empty: shares where the waves' places are more than 7/5 of the groups and
// the lists long enough for the states and the merge (312 groups of 2,048 keys of 128:
// 68.5 and 60.0, 384: 72.4 and 72.8, 456: 76.6 and 80.7, 640: 114.1 and 111.9, 768: 121.0 and
// 130.4; 312 of 1,024 keys of 256: 77.9 and 61.8; 312 of 1,024 keys of 64, 32 tiles: 19.1 and
// 21.6).  Else by the rounds of a tile per warp: 128 groups of 4,096 keys 44.4 us in
// clusters and 48.1 in shares, 4 groups of 2,048 keys of 256 9.4 and 8.0.
ListPlan decode_list_plan(int64_t groups, int top_k, int list_tiles, int d) {
  const int full = decode_rows_warps(d), shared = decode_share_warps(groups * list_tiles, d);
  const ListPlan shares{0, shared};
  if (top_k > kListIds) return shares;
  if (groups > kPlanSms) {
    const int64_t wave = 2 * kPlanSms, places = (groups + wave - 1) / wave * wave;
    if (places > wave && places * 5 > groups * 7 && list_tiles >= 64) return shares;
    return {1, full / 2};
  }
  int cluster = 1;
  while (cluster < 8 && groups * cluster * 2 <= kPlanSms && cluster * full < list_tiles) cluster *= 2;
  const int64_t rounds = (list_tiles + cluster * full - 1) / (cluster * full);
  const int64_t share_rounds = (groups * list_tiles + kPlanSms * shared - 1) / (kPlanSms * shared);
  if (rounds * 4 > share_rounds * 5) return shares;
  return {cluster, full};
}

}  // namespace mattn
