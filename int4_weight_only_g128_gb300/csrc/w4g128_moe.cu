// The mixture-of-experts layer on packed int4-g128 experts (w4g128_moe), for
// 1..16 rows: four programmatic dependent launches,
//   route    logits of every (row, expert), and x in MMA operand order;
//   expert 0 gate and up of the picked experts, silu(g) u -> activations;
//   expert 1 down of the picked experts -> fp32 rows per (row, pick);
//   combine  weighted sum over a row's picks, residual, bf16.
// The bytes are the picked experts' weights, read once: the expert kernels
// are grouped weight streams.  Which experts, and which rows each serves, is
// known on the device only, so every CTA of an expert kernel derives the lists
// itself from the M x E logits (top-k per row, one warp each).
//
// A unit is (picked expert, 16 output columns), its depth K = 128 G rows cut
// into G groups.  A CTA takes a contiguous range of units and its 8 warps take
// the range's (unit, group) items in turn, each through its own ring of bulk
// copies (one 1088-byte block, or a gate and an up block, per stage).  The
// item's product is one warp MMA per packed word: the 16 columns are the A
// operand (bf16 128 + q, exact: one shift and one LOP3 per operand register),
// the rows that picked the expert are the B columns.  The bias of 128 and the
// group minimum need X = sum_k x, which an MMA with an all-ones A gives in the
// very registers that need it:
//   sum_k x w = scale sum_k x (128 + q) + (min - 128 scale) X.
// Group g of a unit is summed by whichever warp holds it into partial g mod 8
// in rising order, and the 8 partials are added in order: bits do not depend
// on the grid, nor on which other rows share the expert.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "w4g128_ops.h"
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
constexpr uint32_t kBias = 0x43004300u;  // bf16 128.0 twice
constexpr uint32_t kOnes = 0x3F803F80u;  // bf16 1.0 twice

struct Params {
  const uint16_t *x, *residual, *router;
  uint16_t* y;
  const uint8_t *gate_up, *down;
  int M, D, F, E, top_k, renormalize;
  unsigned* status;
  float* logits;   // [M][E]
  float* weights;  // [M][top_k], picks in rising expert order
  uint8_t* xp;     // [M][D / 128][256]: x in operand order
  uint8_t* act;    // [M top_k][F / 128][256]: activations in operand order
  float* part;     // [M top_k][D]
};

__device__ __forceinline__ float low_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Operand order of one 128-value group of a row: lane quad member c loads its
// B registers of k steps 2i and 2i + 1 as the 16 bytes at 64 i + 16 c: values
// 16 s + 2c, 16 s + 2c + 1 | 16 s + 8 + 2c, + 1 for s = 2i, then for s = 2i + 1.

// ---------------------------------------------------------------- route
// One CTA per expert; a thread sums its 8-value pieces of the depth for every
// row, then lanes and warps in a fixed order.
template <int MT>
__global__ void __launch_bounds__(kThreads) route_kernel(const __grid_constant__ Params p) {
  __shared__ float s_sum[kWarps][MT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, e = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  if (e == 0 && tid == 0) *reinterpret_cast<unsigned long long*>(p.status) = 0ull;

  const uint4* w = reinterpret_cast<const uint4*>(p.router + static_cast<long long>(e) * p.D);
  const uint4* x = reinterpret_cast<const uint4*>(p.x);
  const int n = p.D / 8;
  float sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) sum[m] = 0.f;
  for (int i = tid; i < n; i += kThreads) {
    const uint4 wv = __ldg(w + i);
    const uint32_t ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m < p.M) {
        const uint4 xv = __ldg(x + static_cast<long long>(m) * n + i);
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[m] = fmaf(low_f(xs[j]), low_f(ws[j]), sum[m]);
          sum[m] = fmaf(high_f(xs[j]), high_f(ws[j]), sum[m]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum[m] += __shfl_xor_sync(~0u, sum[m], d);
    if (lane == 0) s_sum[warp][m] = sum[m];
  }
  __syncthreads();
  if (tid < p.M) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) t += s_sum[j][tid];
    p.logits[tid * p.E + e] = t;
  }

  const uint32_t* xw = reinterpret_cast<const uint32_t*>(p.x);
  const int units = p.M * n;  // 16 bytes each
  for (int u = e * kThreads + tid; u < units; u += p.E * kThreads) {
    const int group = u / 16, i = u / 4 % 4, c = u % 4;  // (rows follow one another in whole groups)
    const uint32_t* src = xw + group * 64 + 16 * i + c;
    reinterpret_cast<uint4*>(p.xp)[u] = make_uint4(__ldg(src), __ldg(src + 4), __ldg(src + 8), __ldg(src + 12));
  }
}

// ---------------------------------------------------------------- the lists
// Picked experts in rising order with the picks (row * top_k + place, places in
// rising expert order) that each serves.
struct Lists {
  uint16_t expert[kMaxPicks];      // of a picked expert
  uint16_t first[kMaxPicks + 1];   // its first entry
  uint16_t pick[kMaxPicks];        // entries
  float weight[kMaxPicks];         // by pick
  int experts;
  // scratch
  uint16_t chosen[kMaxPicks];      // by pick: the expert
  alignas(4) uint16_t rows[W4G128_MAX_EXPERTS];  // bit m: row m picked it
  uint16_t index[W4G128_MAX_EXPERTS];  // its place among the picked
};

// Rising with the value; NaN below everything, and 0 is left for "taken".
__device__ __forceinline__ uint32_t rank_of(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 ranks as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ void make_lists(const Params& p, Lists& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = W4G128_MAX_EXPERTS / 32;
  for (int e = tid; e < p.E; e += kThreads) s.rows[e] = 0;
  __syncthreads();
  for (int m = warp; m < p.M; m += kWarps) {
    float v[kPer];
    uint32_t rank[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 32 + lane;
      rank[i] = 0u;
      if (e < p.E) {
        v[i] = __ldcg(p.logits + m * p.E + e);
        rank[i] = rank_of(v[i]);
      }
    }
    float all = 0.f, top = 0.f, mine = 0.f;  // mine: this lane's pick's exponential
    int my_expert = 0;
    for (int j = 0; j < p.top_k; ++j) {
      uint32_t best = 0u;
      int at = 0;
      float val = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
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
      for (int i = 0; i < kPer; ++i)
        if (i * 32 + lane == e) rank[i] = 0u;
      if (j == 0) {
        top = val;
        if (!p.renormalize) {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
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
    // places by rising expert
    int place = 0;
    for (int j = 0; j < p.top_k; ++j) place += __shfl_sync(~0u, my_expert, j) < my_expert;
    if (lane < p.top_k) {
      s.chosen[m * p.top_k + place] = static_cast<uint16_t>(my_expert);
      s.weight[m * p.top_k + place] = mine / all;
      // two rows' marks share a word
      atomicOr(reinterpret_cast<unsigned*>(s.rows) + my_expert / 2, (1u << m) << (my_expert % 2 * 16));
    }
  }
  __syncthreads();
  if (warp == 0) {
    int experts = 0, picks = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const unsigned rows = e < p.E ? s.rows[e] : 0u;
      const unsigned any = __ballot_sync(~0u, rows != 0u);
      int n = __popc(rows);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(~0u, n, d);
        if (lane >= d) n += t;
      }
      if (rows) {
        const int a = experts + __popc(any & ((1u << lane) - 1u));
        s.expert[a] = static_cast<uint16_t>(e);
        s.index[e] = static_cast<uint16_t>(a);
        s.first[a] = static_cast<uint16_t>(picks + n - __popc(rows));
      }
      experts += __popc(any);
      picks += __shfl_sync(~0u, n, 31);
    }
    if (lane == 0) {
      s.experts = experts;
      s.first[experts] = static_cast<uint16_t>(picks);
    }
  }
  __syncthreads();
  for (int i = tid; i < p.M * p.top_k; i += kThreads) {
    const int e = s.chosen[i], m = i / p.top_k;
    s.pick[s.first[s.index[e]] + __popc(s.rows[e] & ((1u << m) - 1u))] = static_cast<uint16_t>(i);
  }
  __syncthreads();
}

// ---------------------------------------------------------------- expert streams
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// PHASE 0: gate and up (two tiles per unit); 1: down.  NT: 8-row B tiles.
template <int PHASE, int NT>
struct Stream {
  static constexpr int kTiles = PHASE == 0 ? 2 : 1;
  static constexpr int kStage = kTiles * kBlockBytes;
  static constexpr int kStages = PHASE == 0 ? 4 : 8;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kCols = kTiles * kTileN;
  static constexpr int kPartFloats = kParts * NT * 8 * kCols;  // one unit's partials, [part][row][column]
  static constexpr int kBytes = kRing + 2 * kPartFloats * 4 + kWarps * kStages * 8;
};

template <int PHASE, int NT>
__global__ void __launch_bounds__(kThreads, 2) expert_kernel(const __grid_constant__ Params p) {
  using S = Stream<PHASE, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Lists lists;
  float* parts = reinterpret_cast<float*>(smem + S::kRing);
  const uint32_t bars = smem_addr(smem + S::kRing + 2 * S::kPartFloats * 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kWarps * S::kStages) mbar_init(bars + 8 * tid, 1);
  fence_mbar_init();

  // The logits: of the preceding kernel (phase 0), or of the one before, which
  // had completed when the preceding one let this one launch (phase 1).
  if (PHASE == 0) {
    grid_dependency_wait();
    grid_dependents_launch();
  }
  make_lists(p, lists);
  if (PHASE == 0 && blockIdx.x == 0)
    for (int i = tid; i < p.M * p.top_k; i += kThreads) p.weights[i] = lists.weight[i];

  const int K = PHASE == 0 ? p.D : p.F, N = PHASE == 0 ? 2 * p.F : p.D;
  const int G = K / kGroup;
  const int tiles = PHASE == 0 ? p.F / kTileN : p.D / kTileN;  // units of an expert
  const long long units = static_cast<long long>(lists.experts) * tiles;
  const long long u0 = units * blockIdx.x / gridDim.x;
  const int nu = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - u0);
  const uint8_t* weights = PHASE == 0 ? p.gate_up : p.down;
  const long long expert_bytes = static_cast<long long>(N / kTileN) * G * kBlockBytes;
  const uint64_t policy = l2_policy_evict_first();
  const uint32_t ring = smem_addr(smem) + warp * S::kStages * S::kStage;
  const uint8_t* ring_ptr = smem + warp * S::kStages * S::kStage;
  const uint32_t bar = bars + 8 * warp * S::kStages;
  bool good = true;

  // This warp's items are numbers warp, warp + 8, .. of the CTA's (unit, group) list.
  struct Cursor {
    int unit, group;
  };
  auto advance = [&](Cursor& c) {
    c.group += kWarps;
    while (c.group >= G) {
      c.group -= G;
      ++c.unit;
    }
  };
  auto issue = [&](const Cursor& c, int stage) {  // one lane
    const long long u = u0 + c.unit;
    const int a = static_cast<int>(u / tiles), t = static_cast<int>(u % tiles);
    const uint8_t* base = weights + lists.expert[a] * expert_bytes + static_cast<long long>(c.group) * kQuadBytes;
    const long long quad = static_cast<long long>(G) * kQuadBytes;
    mbar_arrive_expect_tx(bar + 8 * stage, S::kStage);
    const uint32_t dst = ring + stage * S::kStage;
    bulk_g2s(dst, base + (t / kQuadTiles) * quad + (t % kQuadTiles) * kBlockBytes, kBlockBytes, bar + 8 * stage, policy);
    if (PHASE == 0) {
      const int t2 = t + tiles;
      bulk_g2s(dst + kBlockBytes, base + (t2 / kQuadTiles) * quad + (t2 % kQuadTiles) * kBlockBytes, kBlockBytes,
               bar + 8 * stage, policy);
    }
  };
  Cursor head{0, warp};  // next to issue
  while (head.group >= G) {
    head.group -= G;
    ++head.unit;
  }
  Cursor cur = head;
  if (lane == 0) {
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) {
      if (head.unit < nu) issue(head, i);
      advance(head);
    }
  }
  if (PHASE == 1) {
    grid_dependency_wait();  // the weights are on their way while the activations are finished
    grid_dependents_launch();
  }

  const int r = lane >> 2, c = lane & 3;
  int stage = 0;
  uint32_t parity = 0;
  for (int u = 0; u < nu; ++u) {
    const int a = static_cast<int>((u0 + u) / tiles);
    const int first = lists.first[a], count = lists.first[a + 1] - first;
    float* part = parts + (u & 1) * S::kPartFloats;
    if (cur.unit == u) {
      const uint8_t* row[NT];  // this lane's B row (r of each 8-row tile) in operand order
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int i = n * 8 + r;
        const int pick = i < count ? lists.pick[first + i] : 0;
        row[n] = i < count ? (PHASE == 0 ? p.xp + static_cast<long long>(pick / p.top_k) * p.D * 2
                                         : p.act + static_cast<long long>(pick) * p.F * 2) + 16 * c
                           : nullptr;
      }
      const bool two = NT == 2 && count > 8;
      float acc[S::kTiles][NT][4];
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[t][n][0] = acc[t][n][1] = acc[t][n][2] = acc[t][n][3] = 0.f;
      const int slot = cur.group % kParts;
      while (cur.unit == u) {
        uint4 xv[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            xv[n][i] = row[n] ? *reinterpret_cast<const uint4*>(row[n] + cur.group * 256 + i * 64) : make_uint4(0, 0, 0, 0);
        // (after a wait has given up, the copies still in flight get a short one each)
        good = mbar_wait_bounded(bar + 8 * stage, parity, good ? kDefaultWaitNs : 1000000ull) && good;
        const uint8_t* st = ring_ptr + stage * S::kStage;
        float d[S::kTiles][NT][4] = {}, X[NT][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 q[S::kTiles];
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t)
            q[t] = *reinterpret_cast<const uint4*>(st + t * kBlockBytes + 512 * h + 16 * lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int s = 4 * h + j;
            uint32_t b[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 v = xv[n][s / 2];
              b[n][0] = s % 2 ? v.z : v.x;
              b[n][1] = s % 2 ? v.w : v.y;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n == 0 || two) mma(X[n], kOnes, kOnes, kOnes, kOnes, b[n][0], b[n][1]);
#pragma unroll
            for (int t = 0; t < S::kTiles; ++t) {
              const uint32_t w = j == 0 ? q[t].x : j == 1 ? q[t].y : j == 2 ? q[t].z : q[t].w;
              const uint32_t a0 = lop3_and_or(w, 0x000F000Fu, kBias), a1 = lop3_and_or(w >> 4, 0x000F000Fu, kBias);
              const uint32_t a2 = lop3_and_or(w >> 8, 0x000F000Fu, kBias), a3 = lop3_and_or(w >> 12, 0x000F000Fu, kBias);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                if (n == 0 || two) mma(d[t][n], a0, a1, a2, a3, b[n][0], b[n][1]);
            }
          }
        }
        uint2 meta[S::kTiles];
#pragma unroll
        for (int t = 0; t < S::kTiles; ++t)
          meta[t] = *reinterpret_cast<const uint2*>(st + t * kBlockBytes + kCodeBytes + 8 * r);
        __syncwarp();  // the stage is read out
        if (lane == 0 && head.unit < nu) {
          fence_proxy_async_smem();
          issue(head, stage);
        }
        if (lane == 0) advance(head);
        if (++stage == S::kStages) {
          stage = 0;
          parity ^= 1;
        }
#pragma unroll
        for (int t = 0; t < S::kTiles; ++t) {
          const float s0 = low_f(meta[t].x), s1 = low_f(meta[t].y);
          const float b0 = fmaf(-128.f, s0, high_f(meta[t].x)), b1 = fmaf(-128.f, s1, high_f(meta[t].y));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[t][n][0] = fmaf(s0, d[t][n][0], fmaf(b0, X[n][0], acc[t][n][0]));
            acc[t][n][1] = fmaf(s0, d[t][n][1], fmaf(b0, X[n][1], acc[t][n][1]));
            acc[t][n][2] = fmaf(s1, d[t][n][2], fmaf(b1, X[n][0], acc[t][n][2]));
            acc[t][n][3] = fmaf(s1, d[t][n][3], fmaf(b1, X[n][1], acc[t][n][3]));
          }
        }
        advance(cur);
      }
#pragma unroll
      for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int m = n * 8 + 2 * c + (i & 1);
            if (m < count) part[(slot * NT * 8 + m) * S::kCols + t * kTileN + r + 8 * (i >> 1)] = acc[t][n][i];
          }
    }
    // One barrier per unit: the other half of the buffer is free again once
    // every warp is past the next one.
    __syncthreads();
    const int o = (tid + 32 * (u & 7)) % kThreads;  // the folding warps take turns
    if (o < count * kTileN) {
      const int m = o / kTileN, col = o % kTileN;
      const int pick = lists.pick[first + m];
      const int n = static_cast<int>((u0 + u) % tiles) * kTileN + col;
      const int used = G < kParts ? G : kParts;
      float v = 0.f, w = 0.f;
      for (int k = 0; k < used; ++k) {
        const float* q = part + (k * NT * 8 + m) * S::kCols + col;
        v += q[0];
        if (PHASE == 0) w += q[kTileN];
      }
      if (PHASE == 0) {
        const float act = v / (1.f + expf(-v)) * w;
        const int k = n % kGroup, s = k / 16, h = k % 16 / 8, cc = k % 8 / 2;
        uint8_t* dst = p.act + static_cast<long long>(pick) * p.F * 2 + n / kGroup * 256 + s / 2 * 64 + cc * 16 +
                       (s % 2 * 2 + h) * 4 + (k & 1) * 2;
        *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(act);
      } else {
        p.part[static_cast<long long>(pick) * p.D + n] = v;
      }
    }
  }
  if (!good) atomicCAS(p.status, 0u, static_cast<unsigned>(W4G128_ERR_TIMEOUT));
}

// ---------------------------------------------------------------- combine
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  const int m = blockIdx.y, i = blockIdx.x * 128 + threadIdx.x;  // 4 columns
  if (i >= p.D / 4) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < p.top_k; ++j) {
    const float w = p.weights[m * p.top_k + j];
    const float4 v = reinterpret_cast<const float4*>(p.part + static_cast<long long>(m * p.top_k + j) * p.D)[i];
    s.x = fmaf(w, v.x, s.x);
    s.y = fmaf(w, v.y, s.y);
    s.z = fmaf(w, v.z, s.z);
    s.w = fmaf(w, v.w, s.w);
  }
  const long long at = static_cast<long long>(m) * p.D + 4 * i;
  if (p.residual) {
    const uint2 r = *reinterpret_cast<const uint2*>(p.residual + at);
    s.x += low_f(r.x);
    s.y += high_f(r.x);
    s.z += low_f(r.y);
    s.w += high_f(r.y);
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(s.x, s.y), b = __floats2bfloat162_rn(s.z, s.w);
  *reinterpret_cast<uint2*>(p.y + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
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
  size_t logits, weights, xp, act, part, total;
};
Layout layout(const w4g128_moe_args& a) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  const size_t M = a.M, picks = M * a.top_k;
  Layout l;
  l.logits = kStatusBytes;
  l.weights = l.logits + up(M * a.E * 4);
  l.xp = l.weights + up(picks * 4);
  l.act = l.xp + up(M * a.D * 2);
  l.part = l.act + up(picks * a.F * 2);
  l.total = l.part + up(picks * a.D * 4);
  return l;
}

template <int PHASE, int NT>
cudaError_t launch_expert(cudaLaunchConfig_t& cfg, const Params& p, int sms) {
  using S = Stream<PHASE, NT>;
  const cudaError_t e = cudaFuncSetAttribute(expert_kernel<PHASE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(std::min(p.M * p.top_k, p.E)) * (PHASE == 0 ? p.F : p.D) / kTileN;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(2 * sms, units)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  return cudaLaunchKernelEx(&cfg, expert_kernel<PHASE, NT>, p);
}

cudaError_t launch(const Params& p, cudaStream_t stream) {
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
  cfg.gridDim = dim3(p.E);
  cfg.blockDim = dim3(kThreads);
  if (p.M == 1) e = cudaLaunchKernelEx(&cfg, route_kernel<1>, p);
  else if (p.M <= 4) e = cudaLaunchKernelEx(&cfg, route_kernel<4>, p);
  else e = cudaLaunchKernelEx(&cfg, route_kernel<16>, p);
  if (e != cudaSuccess) return e;
  e = p.M <= 8 ? launch_expert<0, 1>(cfg, p, sms) : launch_expert<0, 2>(cfg, p, sms);
  if (e != cudaSuccess) return e;
  e = p.M <= 8 ? launch_expert<1, 1>(cfg, p, sms) : launch_expert<1, 2>(cfg, p, sms);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((p.D / 4 + 127) / 128, p.M);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, combine_kernel, p);
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
  p.status = reinterpret_cast<unsigned*>(base);
  p.logits = reinterpret_cast<float*>(base + l.logits);
  p.weights = reinterpret_cast<float*>(base + l.weights);
  p.xp = base + l.xp;
  p.act = base + l.act;
  p.part = reinterpret_cast<float*>(base + l.part);
  if (launch(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
