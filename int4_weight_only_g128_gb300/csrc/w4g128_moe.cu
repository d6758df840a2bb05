// The mixture-of-experts layer on packed int4-g128 experts (w4g128_moe), for
// 1..16 rows: three or four programmatic dependent launches,
//   route    one cluster of 8 CTAs: the logits of every (row, expert), the
//            picks and weights of each row, the list of picked experts with the
//            rows that each serves; the other CTAs put x in MMA operand order;
//   expert 0 gate and up of the picked experts, silu(g) u -> activations;
//   expert 1 down of the picked experts -> fp32 rows per (row, pick);
//   combine  weighted sum over a row's picks, residual, bf16 (one or two rows:
//            by the CTAs of expert 1).
// The bytes are the picked experts' weights, read once: the expert kernels are
// grouped weight streams.  One persistent kernel with grid barriers in place
// of the expert kernels measured slower (43.1 us against 38.9 us for one
// row, 5120 x 1408, 8 of 64 experts): a cooperative launch starts 2.7 us after
// the routing, and a barrier costs 2 us more than the slowest CTA, where the
// next launch's CTAs are on the SMs with their first copies already.
//
// A unit is (picked expert, 2 or 4 tiles of 16 output columns), its depth K =
// 128 G rows cut into G groups.  A team of 4 or 8 warps works on a unit and
// takes its (unit, group) items in turn, each warp through a ring of its own
// filled by cp.async (bulk copies cost a fence and some forty instructions of
// one lane per item: 409 instructions an item against 265).  The item's product
// is one warp MMA per packed word: the 16 columns are the A operand, the rows
// that picked the expert the B columns.
// x and the activations enter as fp16, a row scaled by the power of two that
// puts its largest magnitude in [2^14, 2^15); the weights as fp16 1024 + q and
// 1024 + 16 q, both from one word with one shift and four LOP3 (bf16 takes two
// shifts more: 48.4 against 46.6 us, the down projection of 16 rows of 5120).
//   gate and up: x is bf16; values down to 2^-31 of the row's largest are
//     exact, smaller ones off by at most 2^-39 of it;
//   down: an activation is rounded to fp16 where it is computed, scaled by its
//     16-column tile's largest, since the row's is not known yet (2^-11
//     relative, an eighth of bf16's rounding); the tile's exponent goes along,
//     and the operand is brought to the row's exponent when it is used, by
//     2^-24 at most and what is beyond before that.  It errs there by half a
//     step, 2^-39 of the row's largest, and where it is stored by as much of the
//     tile's.
// The bias and the group minimum are undone by X = sum_k x per (row, group):
//   sum_k x w = scale sum_k x (bias + q) + (min - bias scale) X,
// and an MMA with an all-ones A leaves X in the registers that need it, once
// for the tiles of an item (8 products beside 16 or 32; stored sums cost as
// many loads as x itself, and latency).  The x of the next item is loaded a
// whole item ahead.
// The groups g of a unit fall into 8 parts by g mod 8, summed in rising order,
// and the parts are added as ((0 + 4) + (2 + 6)) + ((1 + 5) + (3 + 7)), whether
// 8 warps hold one part each or 4 warps two each: bits do not depend on the
// grid, nor on which other rows share the expert.
//
// Measured: 16 rows, 5120 x 1408, 6 of 96 experts (712 MB): 129 us a call, 82% of
// the measured copy rate; gate and up 72 us (6.1 TB/s), down 47 us (4.7 TB/s:
// units of 11 groups, a barrier of the team and a fold for every 2.75 items of a
// warp).  One row, 8 of 64 experts (93 MB): 34.8 us: routing 5.0, lists and first
// copies 2.6, gate and up 12, the change of kernels 2, down 7.5, adding up 2, the
// rest launches: what is left above the 13.7 us of bytes is latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "w4g128_ops.h"
#include "w4g128_divide.cuh"
#include "w4g128_internal.h"
#include "w4g128_ptx.cuh"

namespace w4g128 {
namespace {

constexpr int kMaxM = W4G128_MAX_M;
constexpr int kMaxPicks = kMaxM * W4G128_MAX_TOP_K;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kParts = 8;             // partial sums of a unit
constexpr size_t kStatusBytes = 256;
constexpr uint32_t kBias = 0x64006400u;  // fp16 1024.0 twice
constexpr uint32_t kOne = 0x3C003C00u;   // fp16 1.0 twice
constexpr int kLeastHalf = 24;           // fp16 has no power of two below 2^-24

// Picked experts in rising order with the picks (row * top_k + place, places in
// rising expert order) that each serves: one entry for up to 8 rows, what an
// MMA has B columns for.  An expert of more rows has two entries; its weights
// are then dequantised twice and read twice, one entry's units after the other's:
// the second time from the L2, as far as that still holds them.  16 rows that
// all pick 8 experts, 4096 x 14336 (94 MB each): 5% more DRAM bytes than once in
// gate and up, 11% in down, 266 us a call against 142 with 8 rows; 4096 x 4096:
// no more bytes, 89 us against 56.
struct alignas(16) Lists {
  int entries;
  uint16_t expert[kMaxPicks];
  uint16_t first[kMaxPicks + 2];  // an entry's first pick, and one more
  uint16_t pick[kMaxPicks];
};
static_assert(sizeof(Lists) / 16 <= kThreads, "copied by one 16-byte load per thread");

struct Params {
  const uint16_t *x, *residual, *router;
  uint16_t* y;
  const uint8_t *gate_up, *down;
  int M, D, F, E, top_k, renormalize;
  Divisor by_top_k;
  Divisor by_per;     // units of an expert, of the launch
  int lead;           // how far ahead its units are drawn
  unsigned* status;
  unsigned* next;     // [2]: units handed out beyond the first ones, of each expert kernel
  Lists* lists;
  float* weights;     // [M][top_k], by pick
  uint8_t* xp;        // [M][D / 128][256]: x as scaled fp16 in operand order
  float* unscale;     // [M]: the factor that undoes the scale
  uint8_t* act;       // [M top_k][F / 128][256]: activations as scaled fp16 in operand order
  uint8_t* act_exp;   // [M top_k][F / 16]: the biased exponents of the tiles' largest
  unsigned* act_top;  // [M top_k]: the largest of them
  float* part;        // [M top_k][D]
  unsigned* done;     // [D / 32]: finished entries of the columns of a unit of expert 1
};

__device__ __forceinline__ float low_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Operand order of one 128-value group of a row: lane quad member c loads its
// B registers of k steps 2i and 2i + 1 as the 16 bytes at 64 i + 16 c: values
// 16 s + 2c, 16 s + 2c + 1 | 16 s + 8 + 2c, + 1 for s = 2i, then for s = 2i + 1.

// ---------------------------------------------------------------- route
constexpr int kRouteCtas = 8;  // of the cluster that routes
constexpr int kRouteThreads = 512;

// The cluster splits the depth: each CTA multiplies its slice for every row and
// expert with the warp MMA (x rows by 8 experts; a lane's 16 bytes are operand
// registers as they are, since x and the router agree on the order of the
// depth), and leaves the sums with the CTA that finishes the row.
struct RouteShared {
  float sums[kRouteCtas * 2 * W4G128_MAX_EXPERTS];  // [slice][row / 8][expert], slices * E <= 8 * 512
  // CTA 0: every row's picks
  uint16_t chosen[kMaxPicks];
  alignas(4) uint16_t rows[W4G128_MAX_EXPERTS];   // bit m: row m picked it
  uint16_t index[W4G128_MAX_EXPERTS];             // its place among the picked
};

// Rising with the value; NaN below everything, and 0 is left for "taken".
__device__ __forceinline__ uint32_t rank_of(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 ranks as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One warp: the picks of row m from the sums of its logits; experts i * 32 +
// lane, i < PER.
template <int PER>
__device__ __forceinline__ void pick_row(const Params& p, int m, int slices, const RouteShared& s, uint16_t* chosen) {
  const int lane = threadIdx.x & 31;
  float v[PER];
  uint32_t rank[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    rank[i] = 0u;
    v[i] = 0.f;
    if (e < p.E) {
#pragma unroll 8
      for (int j = 0; j < slices; ++j) v[i] += s.sums[(j * 2 + m / 8) * p.E + e];
      rank[i] = rank_of(v[i]);
    }
  }
  float all = 0.f, top = 0.f, mine = 0.f;  // mine: the exponential of this lane's pick
  int my_expert = 0;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t best = 0u;
    int at = 0;
    float val = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (rank[i] > best) {
        best = rank[i];
        at = i * 32 + lane;
        val = v[i];
      }
    }
    const uint32_t win = __reduce_max_sync(~0u, best);
    const int e = static_cast<int>(__reduce_min_sync(~0u, best == win ? static_cast<unsigned>(at) : ~0u));
    val = __shfl_sync(~0u, val, e & 31);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 32 + lane == e) rank[i] = 0u;
    if (j == 0) {
      top = val;
      if (!p.renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i * 32 + lane < p.E) all += expf(v[i] - top);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(~0u, all, d);
      }
    }
    const float x = expf(val - top);
    if (p.renormalize) all += x;  // the same in every lane, by falling logit
    if (lane == j) {
      mine = x;
      my_expert = e;
    }
  }
  int place = 0;  // by rising expert
  for (int j = 0; j < p.top_k; ++j) place += __shfl_sync(~0u, my_expert, j) < my_expert;
  if (lane < p.top_k) {
    p.weights[m * p.top_k + place] = mine / all;
    if (chosen != nullptr) {
      chosen[m * p.top_k + place] = static_cast<uint16_t>(my_expert);
    } else {  // one row: its picks are the lists
      p.lists->expert[place] = static_cast<uint16_t>(my_expert);
      p.lists->first[place] = static_cast<uint16_t>(place);
      p.lists->pick[place] = static_cast<uint16_t>(place);
      if (lane == 0) {
        p.lists->entries = p.top_k;
        p.lists->first[p.top_k] = static_cast<uint16_t>(p.top_k);
      }
    }
  }
}

// CTA 0: the lists from every row's picks.
__device__ __forceinline__ void make_lists(const Params& p, RouteShared& s) {
  const int tid = threadIdx.x, lane = tid & 31, picks = p.M * p.top_k;
  for (int i = tid; i < picks; i += kRouteThreads) {
    const int e = s.chosen[i];  // two experts' marks share a word
    atomicOr(reinterpret_cast<unsigned*>(s.rows) + e / 2, (1u << (i / p.by_top_k)) << (e % 2 * 16));
  }
  __syncthreads();
  if (tid < 32) {
    int entries = 0, before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const unsigned rows = e < p.E ? s.rows[e] : 0u;
      const unsigned any = __ballot_sync(~0u, rows != 0u);
      if (any == 0u) continue;
      // picks below, and experts' second entries above bit 16
      const int own = __popc(rows), mine = own + (own > 8 ? 1 << 16 : 0);
      int n = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(~0u, n, d);
        if (lane >= d) n += t;
      }
      const int all = __shfl_sync(~0u, n, 31);
      n -= mine;
      if (rows) {
        const int a = entries + __popc(any & ((1u << lane) - 1u)) + (n >> 16);
        const int first = before + (n & 0xFFFF);
        p.lists->expert[a] = static_cast<uint16_t>(e);
        p.lists->first[a] = static_cast<uint16_t>(first);
        s.index[e] = static_cast<uint16_t>(first);
        if (own > 8) {
          p.lists->expert[a + 1] = static_cast<uint16_t>(e);
          p.lists->first[a + 1] = static_cast<uint16_t>(first + 8);
        }
      }
      entries += __popc(any) + (all >> 16);
      before += all & 0xFFFF;
    }
    if (lane == 0) {
      p.lists->entries = entries;
      p.lists->first[entries] = static_cast<uint16_t>(before);
    }
  }
  __syncthreads();
  for (int i = tid; i < picks; i += kRouteThreads) {
    const int e = s.chosen[i], m = i / p.by_top_k;
    p.lists->pick[s.index[e] + __popc(s.rows[e] & ((1u << m) - 1u))] = static_cast<uint16_t>(i);
  }
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// For a biased exponent e of a largest magnitude: 2^s that brings it to [2^14,
// 2^15), and 2^-s, both normal for 15 <= e <= 254.
__device__ __forceinline__ float scale_up(int e) { return __int_as_float((268 - e) << 23); }
__device__ __forceinline__ float scale_back(int e) { return __int_as_float((e - 14) << 23); }
__device__ __forceinline__ int exponent_of(float top) {
  return min(max(static_cast<int>(__float_as_uint(top) >> 23), 15), 254);
}

// x in operand order, by the clusters behind the routing one, a row a CTA.  The
// scale puts the row's largest magnitude in [2^14, 2^15).
__device__ __forceinline__ void pack_x(const Params& p) {
  __shared__ float s_top[kRouteThreads / 32];
  const int tid = threadIdx.x, cta = blockIdx.x - kRouteCtas;
  for (int i = cta * kRouteThreads + tid; i < p.D / 32; i += (gridDim.x - kRouteCtas) * kRouteThreads) p.done[i] = 0u;
  const int units = p.D / 8;  // 16 bytes each
  for (int m = cta; m < p.M; m += gridDim.x - kRouteCtas) {
    const uint4* x = reinterpret_cast<const uint4*>(p.x + static_cast<long long>(m) * p.D);
    float top = 0.f;
    for (int u = tid; u < units; u += kRouteThreads) {
      const uint4 q = __ldg(x + u);
      const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(low_f(v[j])), fabsf(high_f(v[j]))));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    __syncthreads();  // (the row before has read s_top)
    if (tid % 32 == 0) s_top[tid / 32] = top;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRouteThreads / 32; ++j) top = fmaxf(top, s_top[j]);
    const int e = exponent_of(top);
    const float up = scale_up(e);
    if (tid == 0) p.unscale[m] = scale_back(e);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(x);
    for (int u = tid; u < units; u += kRouteThreads) {
      const int group = u / 16, i = u / 4 % 4, c = u % 4;
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = __ldg(words + group * 64 + 16 * i + c + 4 * j);
        const __half2 q = __floats2half2_rn(low_f(v) * up, high_f(v) * up);
        h[j] = *reinterpret_cast<const uint32_t*>(&q);
      }
      reinterpret_cast<uint4*>(p.xp)[static_cast<long long>(m) * units + u] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

// WIDE: more than 8 rows.
template <bool WIDE>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(kRouteThreads)
route_kernel(const __grid_constant__ Params p) {
  __shared__ RouteShared s;
  constexpr int kRouteWarps = kRouteThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive_relaxed();  // every CTA of the cluster runs before any writes into another
  if (blockIdx.x >= kRouteCtas) {
    grid_dependency_wait();
    grid_dependents_launch();
    pack_x(p);
    cluster_wait_acquire();
    return;
  }
  const int rank = static_cast<int>(cluster_ctarank());
  const int r = lane >> 2, c = lane & 3;
  // tiles of 8 experts; where there are few, up to 4 warps share one and split its depth
  const int tiles = (p.E + 7) / 8;
  const int log_sub = tiles * 4 <= kRouteWarps ? 2 : tiles * 2 <= kRouteWarps ? 1 : 0, sub = 1 << log_sub;
  const int slices = kRouteCtas * sub, slice = rank * sub + (warp & (sub - 1));
  const int steps = p.D / 32, k0 = steps * slice >> (3 + log_sub), k1 = steps * (slice + 1) >> (3 + log_sub);
  static_assert(kRouteCtas == 8, "2^3");
  // the router does not depend on the kernels before: into the L2 while they finish
  for (int t = warp >> log_sub; t < tiles; t += kRouteWarps >> log_sub) {
    const char* w = reinterpret_cast<const char*>(p.router + static_cast<long long>(min(t * 8 + lane % 8, p.E - 1)) * p.D);
    for (int at = k0 * 64 + lane / 8 * 128; at < k1 * 64; at += 512)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(w + at));
  }
  grid_dependency_wait();
  grid_dependents_launch();
  if (rank == 0) {
    if (tid == 0) {
      *reinterpret_cast<unsigned long long*>(p.status) = 0ull;
      p.next[0] = p.next[1] = 0u;
    }
    if (tid < p.M * p.top_k) p.act_top[tid] = 0u;
    for (int e = tid; e < W4G128_MAX_EXPERTS / 2; e += kRouteThreads) reinterpret_cast<uint32_t*>(s.rows)[e] = 0u;
  }
  const uint4* xa = reinterpret_cast<const uint4*>(p.x + static_cast<long long>(min(r, p.M - 1)) * p.D) + c;
  const uint4* xb = reinterpret_cast<const uint4*>(p.x + static_cast<long long>(min(r + 8, p.M - 1)) * p.D) + c;
  bool waited = false;
  for (int t = warp >> log_sub; t < tiles; t += kRouteWarps >> log_sub) {
    // rows and experts beyond the last repeat it; nothing of theirs is kept
    const uint4* w = reinterpret_cast<const uint4*>(p.router + static_cast<long long>(min(t * 8 + r, p.E - 1)) * p.D) + c;
    float d[4] = {};
    constexpr int kBatch = WIDE ? 5 : 8;  // steps in flight
    for (int k = k0; k < k1; k += kBatch) {
      uint4 a[kBatch], b[kBatch], v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (k + i < k1) {
          v[i] = __ldg(w + (k + i) * 4);
          a[i] = __ldg(xa + (k + i) * 4);
          b[i] = WIDE ? __ldg(xb + (k + i) * 4) : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (k + i < k1) {
          mma_bf16(d, a[i].x, b[i].x, a[i].y, b[i].y, v[i].x, v[i].y);
          mma_bf16(d, a[i].z, b[i].z, a[i].w, b[i].w, v[i].z, v[i].w);
        }
      }
    }
    if (!waited) cluster_wait_acquire();
    waited = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = r + 8 * (i >> 1), e = t * 8 + 2 * c + (i & 1);
      if (m < p.M && e < p.E)
        *static_cast<float*>(__cluster_map_shared_rank(&s.sums[(slice * 2 + (m >> 3)) * p.E + e], m & 7)) = d[i];
    }
  }
  if (!waited) cluster_wait_acquire();
  cluster_arrive_release();
  cluster_wait_acquire();
  const int m = rank + 8 * warp;  // two warps, a row each
  if (warp < 2 && m < p.M) {
    uint16_t* chosen = p.M == 1 ? nullptr : static_cast<uint16_t*>(__cluster_map_shared_rank(s.chosen, 0));
    if (p.E <= 128) pick_row<4>(p, m, slices, s, chosen);
    else pick_row<W4G128_MAX_EXPERTS / 32>(p, m, slices, s, chosen);
  }
  if (p.M == 1) return;  // (nothing is left in another CTA)
  cluster_arrive_release();
  cluster_wait_acquire();
  if (rank == 0) make_lists(p, s);
}

// ---------------------------------------------------------------- expert streams
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The A fragment of one packed word: columns r as 1024 + q, columns r + 8 as 1024 + 16 q.
__device__ __forceinline__ void operand(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t v = w >> 8;
  a[0] = lop3_and_or(w, 0x000F000Fu, kBias);
  a[1] = lop3_and_or(w, 0x00F000F0u, kBias);
  a[2] = lop3_and_or(v, 0x000F000Fu, kBias);
  a[3] = lop3_and_or(v, 0x00F000F0u, kBias);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// TILES of 16 columns per item: 4, or 2 in a down projection with few units (4:
// half the loads of x and half the work per unit).
template <int TILES>
struct Stream {
  static constexpr int kStage = TILES * kBlockBytes;
  static constexpr int kStages = TILES == 2 ? 3 : 2;  // items of a warp on their way
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kCols = TILES * kTileN;
  static constexpr int kPart = 8 * kCols;  // floats that a warp leaves of a unit: [row][column]
  static constexpr int kBytes = kRing + 2 * kWarps * kPart * 4;
};

template <int TEAM>
__device__ __forceinline__ void team_barrier(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TEAM * 32) : "memory");
}

// Two neighbouring columns of y: the sum of the row's picks, and the residual.
__device__ __forceinline__ void add_picks(const Params& p, int m, int n) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int j = 0; j < p.top_k; ++j) {
    const float w = __ldcg(p.weights + m * p.top_k + j);
    const float2 v = __ldcg(reinterpret_cast<const float2*>(p.part + static_cast<long long>(m * p.top_k + j) * p.D + n));
    s.x = fmaf(w, v.x, s.x);
    s.y = fmaf(w, v.y, s.y);
  }
  const long long at = static_cast<long long>(m) * p.D + n;
  if (p.residual) {
    const uint32_t r = *reinterpret_cast<const uint32_t*>(p.residual + at);
    s.x += low_f(r);
    s.y += high_f(r);
  }
  const __nv_bfloat162 y = __floats2bfloat162_rn(s.x, s.y);
  *reinterpret_cast<uint32_t*>(p.y + at) = *reinterpret_cast<const uint32_t*>(&y);
}

__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i < p.D / 2) add_picks(p, blockIdx.y, 2 * i);
}

// The same within expert 1, for one or two rows: a team counts its finished
// units by their columns, 32 at a time or at its end, and who counts a column's
// last entry adds up.  A launch less (small experts, one row: 18.8 -> 16.2 us);
// with more rows the few teams that finish last add up everything, which took
// longer than the launch (16 rows of 5120: 137 -> 162 us).
template <int COLS, int TEAM>
__device__ __forceinline__ void count_units(const Params& p, int entries, uint16_t* places, uint32_t* s_count, int team,
                                            int member, int finished) {
  const int lane = threadIdx.x & 31;
  team_barrier<TEAM>(team);  // every member has written its rows
  if (member == 0) {
    bool last = false;
    uint16_t place = 0;
    if (lane < finished) {
      place = places[lane];
      __threadfence();
      last = atomicAdd(p.done + place, 1u) == static_cast<unsigned>(entries) - 1u;
      __threadfence();
    }
    const uint32_t mask = __ballot_sync(~0u, last);
    if (last) places[__popc(mask & ((1u << lane) - 1u))] = place;
    if (lane == 0) *s_count = __popc(mask);
  }
  team_barrier<TEAM>(team);
  const int log_rows = p.M - 1, total = static_cast<int>(*s_count) * (COLS / 2) << log_rows;  // 1 or 2 rows
  for (int o = member * 32 + lane; o < total; o += TEAM * 32) {
    const int at = o / (COLS / 2);
    add_picks(p, at & log_rows, places[at >> log_rows] * COLS + o % (COLS / 2) * 2);
  }
}

// PHASE 0: gate and up, a unit is TILES / 2 gate tiles and their up tiles; 1:
// down, a unit is TILES neighbouring tiles.  TEAM: warps that share a unit.
// ADD: the rows' picks are added up here.
template <int PHASE, int TILES, int TEAM, bool ADD>
__global__ void __launch_bounds__(kThreads, 2) expert_kernel(const __grid_constant__ Params p) {
  using S = Stream<TILES>;
  constexpr int kSide = PHASE == 0 ? TILES / 2 : TILES;  // neighbouring tiles
  constexpr int kTeams = kWarps / TEAM;
  constexpr int kMine = kParts / TEAM;  // parts of a unit that one warp sums
  static_assert(TEAM == 4 || TEAM == 8, "the order of the parts' sums");
  constexpr int kQueue = 8;             // units of a team that are known: the current one and the next
  constexpr uint32_t kEnd = ~0u;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Lists lists;
  __shared__ uint32_t s_unit[kTeams][kQueue];
  __shared__ uint32_t s_item[kWarps][S::kStages + 1];  // items on their way: entry and group, or the end
  __shared__ uint16_t s_place[kTeams][32];             // places of finished units
  __shared__ uint32_t s_last[kTeams];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // (uniform, and known to be)
  const int team = warp / TEAM, member = warp % TEAM;

  // The lists: of the preceding kernel (phase 0), or of the one before, which
  // had completed when the preceding one let this one launch (phase 1).
  if (PHASE == 0) {
    grid_dependency_wait();
    grid_dependents_launch();
  }
  if (tid < static_cast<int>(sizeof(Lists) / 16))
    reinterpret_cast<uint4*>(&lists)[tid] = __ldcg(reinterpret_cast<const uint4*>(p.lists) + tid);

  const int K = PHASE == 0 ? p.D : p.F;
  const int G = K / kGroup;
  // A team's units: share, share + shares, .. at first, so that the teams work
  // side by side; then whatever is next (the counter), because SMs differ in
  // how fast they stream (by a third, measured).  A unit is drawn `lead` units
  // before it is worked on, so that the copies can run ahead of it; where a
  // warp may find no item in a unit, all units are handed out evenly.
  const int share = blockIdx.x + gridDim.x * team, shares = gridDim.x * kTeams;
  const int lead = p.lead;
  const bool drawn = G >= kParts && lead < kQueue;
  static_assert(S::kStages + 2 < kQueue, "the longest lead fits the queue");
  __syncthreads();
  const int units = lists.entries * static_cast<int>(p.by_per.d);
  auto locate = [&](int u) -> uint32_t {  // entry and place, or the end
    return u < units ? static_cast<uint32_t>(u / p.by_per) << 16 | static_cast<uint32_t>(u % p.by_per) : kEnd;
  };
  if (member == 0 && lane < kQueue) s_unit[team][lane] = locate(share + lane * shares);
  __syncthreads();
  auto unit_at = [&](int n) { return drawn ? s_unit[team][n % kQueue] : locate(share + n * shares); };
  const uint8_t* weights = PHASE == 0 ? p.gate_up : p.down;
  const long long quad_bytes = static_cast<long long>(G) * kQuadBytes;
  const long long expert_bytes = (PHASE == 0 ? p.F / 32 : p.D / 64) * quad_bytes;
  const uint32_t ring = smem_addr(smem) + warp * S::kStages * S::kStage;
  const uint8_t* ring_ptr = smem + warp * S::kStages * S::kStage;

  // A warp's items: in each unit of its team the groups of its parts, part by
  // part in the order in which they are added.  The members take turns from
  // unit to unit, so that they stay even where the groups do not divide.
  auto turn = [&](int u) { return static_cast<int>(static_cast<unsigned>(member - u * G) % TEAM); };
  auto part_at = [](int m, int i) { return m + 4 * i; };

  // The copies run kStages items ahead: the unit's number in the team's order,
  // the part's and the group, and this lane's 16 bytes in group 0 of its tiles.
  int c_n = 0, c_turn = turn(0), c_i = 0, c_group = c_turn;
  uint32_t c_unit = unit_at(0);
  const uint8_t *c_src = nullptr, *c_src2 = nullptr;
  auto place = [&] {
    const int t = static_cast<int>(c_unit & 0xFFFFu) * kSide;
    const uint8_t* base = weights + lists.expert[c_unit >> 16] * expert_bytes + 16 * lane;
    c_src = base + (t / kQuadTiles) * quad_bytes + (t % kQuadTiles) * kBlockBytes;
    if (PHASE == 0) {
      const int t2 = t + p.F / kTileN;
      c_src2 = base + (t2 / kQuadTiles) * quad_bytes + (t2 % kQuadTiles) * kBlockBytes;
    }
  };
  auto settle = [&] {  // to the warp's next item, once c_group is past the depth
    while (c_group >= G && c_unit != kEnd) {
      if (++c_i == kMine) {
        c_i = 0;
        c_unit = unit_at(++c_n);
        if (c_unit == kEnd) return;
        c_turn = turn(c_n);
        place();
      }
      c_group = part_at(c_turn, c_i);
    }
  };
  int c_slot = 0;
  auto copy = [&](int stage) {
    if (lane == 0) s_item[warp][c_slot] = c_unit != kEnd ? (c_unit & 0xFFFF0000u) | static_cast<uint32_t>(c_group) : kEnd;
    c_slot = c_slot == S::kStages ? 0 : c_slot + 1;
    if (c_unit != kEnd) {
      const uint32_t dst = ring + stage * S::kStage + 16 * lane;
      const int off = c_group * kQuadBytes;
      constexpr int kRun = kSide * kBlockBytes;  // contiguous bytes
#pragma unroll
      for (int i = 0; i < kRun / 512; ++i) {
        cp_async16(dst + 512 * i, c_src + off + 512 * i);
        if (PHASE == 0) cp_async16(dst + kRun + 512 * i, c_src2 + off + 512 * i);
      }
      constexpr int kRest = kRun % 512, kAt = kRun - kRest;  // a few lanes more, for each side
      if (lane < kRest / 16) cp_async16(dst + kAt, c_src + off + kAt);
      if (PHASE == 0 && lane < kRest / 16) cp_async16(dst + kRun + kAt, c_src2 + off + kAt);
      c_group += kParts;
      settle();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (c_unit != kEnd) {
    place();
    settle();
  }
#pragma unroll 1
  for (int i = 0; i < S::kStages; ++i) copy(i);
  if (PHASE == 1) {
    grid_dependency_wait();  // the weights are on their way while the activations are finished
    grid_dependents_launch();
  }

  const int r = lane >> 2, c = lane & 3;
  int stage = 0;
  float* parts = reinterpret_cast<float*>(smem + S::kRing) + team * 2 * TEAM * S::kPart;  // two halves that take turns

  // This lane's part of an item's B operand: of row r of the entry.  Columns
  // beyond the entry's rows repeat the last row; nothing of theirs is kept.
  struct Operand {
    uint4 v[4];
    uint2 exps;  // PHASE 1: of the group's 8 tiles
    int scale;   // of the row: PHASE 0 the bits of what undoes it, 1 the exponent
  };
  int x_entry = -1;
  const uint8_t *x_row = nullptr, *x_exps = nullptr;
  const int* x_scale = nullptr;
  auto load_x = [&](uint32_t which, Operand& x) {  // (nothing here waits for a load)
    if (which == kEnd) return;
    const int a = static_cast<int>(which >> 16), group = static_cast<int>(which & 0xFFFFu);
    if (a != x_entry) {
      x_entry = a;
      const int pick = lists.pick[min(lists.first[a] + r, lists.first[a + 1] - 1)];
      const int row = PHASE == 0 ? pick / p.by_top_k : pick;
      x_row = (PHASE == 0 ? p.xp : p.act) + static_cast<long long>(row) * K * 2 + 16 * c;
      x_scale = (PHASE == 0 ? reinterpret_cast<const int*>(p.unscale) : reinterpret_cast<const int*>(p.act_top)) + row;
      if (PHASE == 1) x_exps = p.act_exp + static_cast<long long>(row) * (G * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = *reinterpret_cast<const uint4*>(x_row + group * 256 + i * 64);
    if (PHASE == 1) x.exps = *reinterpret_cast<const uint2*>(x_exps + group * 8);
    x.scale = *x_scale;
  };
  __syncwarp();
  int next_slot = 1;  // of the item after the current one
  Operand x = {};
  load_x(s_item[warp][0], x);
  int scale = 0;  // of row r of the unit in hand

  auto item = [&](float (&acc)[TILES][4]) {
    Operand xn = {};
    __syncwarp();  // the descriptor below may be of the copies just issued
    load_x(s_item[warp][next_slot], xn);
    next_slot = next_slot == S::kStages ? 0 : next_slot + 1;
    scale = x.scale;
    if (PHASE == 1) {  // a tile is a k step: to the row's exponent
      int below[8], most = 0;  // binary orders between the tile's largest and the row's
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        below[s] = x.scale - static_cast<int>((s < 4 ? x.exps.x : x.exps.y) >> (8 * (s % 4)) & 0xFFu);
        most = max(most, below[s]);
      }
      auto lower = [&](int s, int orders) {
        const float f = __int_as_float(max(127 - orders, 0) << 23);
        const __half2 h = __floats2half2_rn(f, f);
        const uint32_t f2 = *reinterpret_cast<const uint32_t*>(&h);
        if (s % 2) {
          x.v[s / 2].z = hmul2(x.v[s / 2].z, f2);
          x.v[s / 2].w = hmul2(x.v[s / 2].w, f2);
        } else {
          x.v[s / 2].x = hmul2(x.v[s / 2].x, f2);
          x.v[s / 2].y = hmul2(x.v[s / 2].y, f2);
        }
      };
      if (most > kLeastHalf) {  // rare: in two steps, the first one where fp16 has bits to spare
#pragma unroll
        for (int s = 0; s < 8; ++s) lower(s, max(below[s] - kLeastHalf, 0));
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) lower(s, min(below[s], kLeastHalf));
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
    __syncwarp();
    const uint8_t* st = ring_ptr + stage * S::kStage;
    float d[TILES][4] = {}, X[4] = {};
    const uint32_t ones[4] = {kOne, kOne, kOne, kOne};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 q[TILES];
#pragma unroll
      for (int t = 0; t < TILES; ++t) q[t] = *reinterpret_cast<const uint4*>(st + t * kBlockBytes + 512 * h + 16 * lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = 4 * h + j;
        const uint32_t b0 = s % 2 ? x.v[s / 2].z : x.v[s / 2].x, b1 = s % 2 ? x.v[s / 2].w : x.v[s / 2].y;
        mma(X, ones, b0, b1);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          uint32_t w[4];
          operand(j == 0 ? q[t].x : j == 1 ? q[t].y : j == 2 ? q[t].z : q[t].w, w);
          mma(d[t], w, b0, b1);
        }
      }
    }
    uint2 meta[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) meta[t] = *reinterpret_cast<const uint2*>(st + t * kBlockBytes + kCodeBytes + 8 * r);
    __syncwarp();  // the stage is read out
    copy(stage);
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      float s0 = low_f(meta[t].x), s1 = low_f(meta[t].y);
      const float b0 = fmaf(-1024.f, s0, high_f(meta[t].x));
      const float b1 = fmaf(-64.f, s1, high_f(meta[t].y));
      s1 *= 0.0625f;  // these columns carry 16 q
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        acc[t][k] = fmaf(s0, d[t][k], fmaf(b0, X[k], acc[t][k]));
        acc[t][2 + k] = fmaf(s1, d[t][2 + k], fmaf(b1, X[k], acc[t][2 + k]));
      }
    }
    x = xn;
  };

  [[maybe_unused]] int finished = 0;  // units that the team has not counted yet
  for (int u = 0;; ++u) {
    const uint32_t unit = unit_at(u);
    if (unit == kEnd) break;
    const int a = static_cast<int>(unit >> 16), at = static_cast<int>(unit & 0xFFFFu) * kSide;  // entry, first tile
    const int first = lists.first[a], count = lists.first[a + 1] - first;
    const bool draws = drawn && member == 0 && lane == 0 && u + lead >= kQueue;
    int draw = 0;
    if (draws) draw = static_cast<int>(atomicAdd(p.next + PHASE, 1u));
    float* part = parts + (u & 1) * TEAM * S::kPart;
    const int mine = turn(u);
    float sum[TILES][4];
#pragma unroll
    for (int h = 0; h < kMine; ++h) {
      float acc[TILES][4] = {};
      for (int g = part_at(mine, h); g < G; g += kParts) item(acc);
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[t][i] = h == 0 ? acc[t][i] : sum[t][i] + acc[t][i];
    }
    const float back = PHASE == 0 ? __int_as_float(scale) : scale_back(max(scale, 15));
    float* out = part + mine * S::kPart + 2 * c * S::kCols + r;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float f = __shfl_sync(~0u, back, (2 * c + k) * 4);  // of row 2c + k (a warp without items: of no matter)
      if (2 * c + k < count)
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          out[k * S::kCols + t * kTileN] = sum[t][k] * f;
          out[k * S::kCols + t * kTileN + 8] = sum[t][2 + k] * f;
        }
    }
    // One barrier of the team per unit: the other half of the buffer, and the
    // drawn unit's place in the queue, are free again once every member is past
    // the next one.
    if (draws) s_unit[team][(u + lead) % kQueue] = locate(kQueue * shares + draw);
    team_barrier<TEAM>(team);
    auto join = [&](const float* q) {  // (parts beyond the depth are 0)
      if constexpr (TEAM == 4) return (q[0] + q[2 * S::kPart]) + (q[S::kPart] + q[3 * S::kPart]);
      else
        return ((q[0] + q[4 * S::kPart]) + (q[2 * S::kPart] + q[6 * S::kPart])) +
               ((q[S::kPart] + q[5 * S::kPart]) + (q[3 * S::kPart] + q[7 * S::kPart]));
    };
    // the folding warps take turns
    const int from = ((member + u) % TEAM) * 32 + lane;
    if (PHASE == 0) {
      constexpr int kGate = kSide * kTileN;  // columns of activations
      const unsigned tile_lanes = 0xFFFFu << (lane & 16);
      for (int o = from; o < count * kGate; o += TEAM * 32) {  // 16 lanes a tile
        const int m = o / kGate, col = o % kGate, n = at * kTileN + col;
        const int pick = lists.pick[first + m];
        const float v = join(part + m * S::kCols + col), w = join(part + m * S::kCols + col + kGate);
        const float act = v * __frcp_rn(1.f + expf(-v)) * w;
        // (magnitudes order like their bits)
        const int e = exponent_of(__uint_as_float(__reduce_max_sync(tile_lanes, __float_as_uint(act) & 0x7FFFFFFFu)));
        // column n: k step n / 16 % 8 of its group
        uint8_t* dst = p.act + static_cast<long long>(pick) * p.F * 2 + n / 128 * 256 + n / 32 % 4 * 64 + n % 8 / 2 * 16 +
                       (n / 16 % 2 * 2 + n / 8 % 2) * 4 + (n & 1) * 2;
        *reinterpret_cast<__half*>(dst) = __float2half_rn(act * scale_up(e));
        if (lane % 16 == 0) {
          p.act_exp[static_cast<long long>(pick) * (p.F / kTileN) + n / kTileN] = static_cast<uint8_t>(e);
          atomicMax(p.act_top + pick, static_cast<unsigned>(e));
        }
      }
    } else {
      for (int o = from; o < count * S::kCols; o += TEAM * 32) {
        const int m = o / S::kCols, col = o % S::kCols;
        p.part[static_cast<long long>(lists.pick[first + m]) * p.D + at * kTileN + col] = join(part + m * S::kCols + col);
      }
      if constexpr (ADD) {
        if (member == 0 && lane == 0) s_place[team][finished] = static_cast<uint16_t>(at / kSide);
        if (++finished == 32) {
          count_units<S::kCols, TEAM>(p, lists.entries, s_place[team], &s_last[team], team, member, finished);
          finished = 0;
        }
      }
    }
  }
  if constexpr (ADD)
    if (finished > 0) count_units<S::kCols, TEAM>(p, lists.entries, s_place[team], &s_last[team], team, member, finished);
}

int check(const w4g128_moe_args* a) {
  if (a == nullptr || a->x == nullptr || a->y == nullptr || a->router == nullptr || a->gate_up == nullptr ||
      a->down == nullptr || a->x == a->y)
    return W4G128_ERR_INVALID_ARG;
  if (a->M < 1 || a->M > W4G128_MAX_M || a->top_k < 1 || a->top_k > W4G128_MAX_TOP_K || (a->renormalize & ~1) != 0)
    return W4G128_ERR_INVALID_ARG;
  auto depth_ok = [](int k) { return k >= 128 && k <= 65536 && k % 128 == 0; };
  if (!depth_ok(a->D) || !depth_ok(a->F) || a->E < 1 || a->E > W4G128_MAX_EXPERTS) return W4G128_ERR_SHAPE;
  if (a->top_k > a->E) return W4G128_ERR_INVALID_ARG;
  auto off = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) != 0; };
  if (off(a->x) || off(a->residual) || off(a->y) || off(a->router) || off(a->gate_up) || off(a->down))
    return W4G128_ERR_ALIGN;
  return W4G128_OK;
}

struct Layout {
  size_t lists, weights, xp, unscale, act, act_exp, act_top, part, done, total;
};
Layout layout(const w4g128_moe_args& a) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  const size_t M = a.M, picks = M * a.top_k;
  Layout l;
  l.lists = kStatusBytes;
  l.weights = l.lists + up(sizeof(Lists));
  l.xp = l.weights + up(picks * 4);
  l.unscale = l.xp + up(M * a.D * 2);
  l.act = l.unscale + up(M * 4);
  l.act_exp = l.act + up(picks * a.F * 2);
  l.act_top = l.act_exp + up(picks * (a.F / 16));
  l.part = l.act_top + up(picks * 4);
  l.done = l.part + up(picks * a.D * 4);
  l.total = l.done + up(a.D / 32 * 4);
  return l;
}

template <int PHASE, int TILES, int TEAM, bool ADD = false>
cudaError_t launch_expert(cudaLaunchConfig_t& cfg, Params& p, int sms, long long units) {
  const int fewest = std::max((PHASE == 0 ? p.D : p.F) / kGroup / kParts * (kParts / TEAM), 1);  // items of a warp in a unit
  p.lead = 1 + (Stream<TILES>::kStages + fewest) / fewest;
  p.by_per = divisor((PHASE == 0 ? p.F : p.D) / ((PHASE == 0 ? TILES / 2 : TILES) * kTileN));
  constexpr int kBytes = Stream<TILES>::kBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(expert_kernel<PHASE, TILES, TEAM, ADD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(2 * sms, units)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  return cudaLaunchKernelEx(&cfg, expert_kernel<PHASE, TILES, TEAM, ADD>, p);
}

// Gate and up in wide items (one row of 5120, 8 experts of 1408: 34.2 us a call,
// 34.9 narrow; of 4096, 6 experts: 25.7 and 27.0).  Down wide and in small teams,
// too, where every SM has units (one row of 7168, 8 experts of 2048: 47.2 us, 50.1
// narrow; 16 rows of 4096, 8 experts of 4096: 51.3 and 54.8), else narrow in large
// teams (one row of 2048, 4 experts of 768: 12.8 us, in small teams 13.4).
cudaError_t launch_experts(cudaLaunchConfig_t& cfg, Params& p, int sms) {
  const long long most = std::min(p.M * p.top_k, p.E);  // picked experts
  const long long gate = most * (p.F / 32), down = most * (p.D / 64);
  const bool wide = down >= 2 * sms;
  cudaError_t e = launch_expert<0, 4, 8>(cfg, p, sms, gate);
  if (e != cudaSuccess) return e;
  if (p.M <= 2)
    return wide ? launch_expert<1, 4, 4, true>(cfg, p, sms, down) : launch_expert<1, 2, 8, true>(cfg, p, sms, 2 * down);
  e = wide ? launch_expert<1, 4, 4>(cfg, p, sms, down) : launch_expert<1, 2, 8>(cfg, p, sms, 2 * down);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((p.D / 2 + 127) / 128, p.M);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, combine_kernel, p);
}

cudaError_t launch(Params& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(kRouteCtas * (1 + (p.M + kRouteCtas - 1) / kRouteCtas));
  cfg.blockDim = dim3(kRouteThreads);
  e = p.M <= 8 ? cudaLaunchKernelEx(&cfg, route_kernel<false>, p) : cudaLaunchKernelEx(&cfg, route_kernel<true>, p);
  if (e != cudaSuccess) return e;
  return launch_experts(cfg, p, sms);
}

}  // namespace
}  // namespace w4g128

extern "C" {

size_t w4g128_moe_workspace_bytes(const w4g128_moe_args* args) {
  return w4g128::check(args) == W4G128_OK ? w4g128::layout(*args).total : 0;
}

int w4g128_moe(const w4g128_moe_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace w4g128;
  int rc = check(a);
  if (rc != W4G128_OK) return rc;
  if (ws == nullptr) return W4G128_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0) return W4G128_ERR_ALIGN;
  const Layout l = layout(*a);
  if (ws_bytes < l.total) return W4G128_ERR_WORKSPACE;
  rc = fault_hook();
  if (rc != W4G128_OK) return rc;
  if (!device_is_sm103()) return W4G128_ERR_DEVICE;
  auto* base = static_cast<uint8_t*>(ws);
  Params p;
  p.x = a->x; p.residual = a->residual; p.router = a->router; p.y = a->y;
  p.gate_up = static_cast<const uint8_t*>(a->gate_up);
  p.down = static_cast<const uint8_t*>(a->down);
  p.M = a->M; p.D = a->D; p.F = a->F; p.E = a->E; p.top_k = a->top_k; p.renormalize = a->renormalize;
  p.by_top_k = divisor(p.top_k);
  p.status = reinterpret_cast<unsigned*>(base);
  p.next = reinterpret_cast<unsigned*>(base + 16);
  p.lists = reinterpret_cast<Lists*>(base + l.lists);
  p.weights = reinterpret_cast<float*>(base + l.weights);
  p.xp = base + l.xp;
  p.unscale = reinterpret_cast<float*>(base + l.unscale);
  p.act = base + l.act;
  p.act_exp = base + l.act_exp;
  p.act_top = reinterpret_cast<unsigned*>(base + l.act_top);
  p.part = reinterpret_cast<float*>(base + l.part);
  p.done = reinterpret_cast<unsigned*>(base + l.done);
  if (launch(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
