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
// A unit is (picked expert, one or two tiles of 16 output columns), its depth
// K = 128 G rows cut into G groups.  A CTA takes a contiguous range of units
// and its 8 warps take the range's (unit, group) items in turn, each through
// its own ring of bulk copies (two 1088-byte blocks per stage: a gate and an
// up block, or two neighbours of the down projection).  The item's product is
// one warp MMA per packed word: the 16 columns are the A operand, the rows
// that picked the expert the B columns.
//   gate and up: x as fp16, each (row, group) scaled by a power of two (exact
//     within 2^29 of the group's largest value), weights as fp16 1024 + q and
//     1024 + 16 q, both from one word with one shift and four LOP3;
//   down: activations as bf16 (their range is not known when they are
//     rounded), weights as bf16 128 + q, with two more shifts a word.
// The bias and the group minimum are undone by X = sum_k x per (row, group):
//   sum_k x w = scale sum_k x (bias + q) + (min - bias scale) X;
// the route kernel leaves X of x, and the activations come with the sums of
// their 16-column tiles (an all-ones A would give X for free of addresses, but
// costs a third of the tensor work, which measured 41% busy: dropped).
// The groups g of a unit fall into 8 parts by g mod 8, summed in rising order,
// and the parts are added as ((0 + 4) + (2 + 6)) + ((1 + 5) + (3 + 7)), whether
// 8 warps hold one part each or 2 warps four each: bits do not depend on the
// grid, nor on which other rows share the expert.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

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
constexpr uint32_t kBias16 = 0x64006400u;   // fp16 1024.0 twice
constexpr uint32_t kBiasB16 = 0x43004300u;  // bf16 128.0 twice

struct Params {
  const uint16_t *x, *residual, *router;
  uint16_t* y;
  const uint8_t *gate_up, *down;
  int M, D, F, E, top_k, renormalize;
  unsigned* status;
  float* logits;   // [M][E]
  float* weights;  // [M][top_k], picks in rising expert order
  uint8_t* xp;     // [M][D / 128][256]: x as scaled fp16 in operand order
  float2* xs;      // [M][D / 128]: X, and the factor that undoes the scale
  uint8_t* act;    // [M top_k][F / 128][256]: activations (bf16) in operand order
  float* acts;     // [M top_k][F / 16]: sums of 16 activations
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

  // x in operand order: 16 lanes per (row, group); rows follow one another in
  // whole groups.  The scale puts the group's largest magnitude in [2^14, 2^15).
  const uint32_t* xw = reinterpret_cast<const uint32_t*>(p.x);
  const int units = p.M * n;  // 16 bytes each, a multiple of 16
  for (int u0 = (e * kWarps + warp) * 32; u0 < units; u0 += p.E * kThreads) {
    const int u = u0 + lane;
    const bool real = u < units;  // (all 16 lanes of a group or none)
    const int group = u / 16, i = u / 4 % 4, c = u % 4;
    uint32_t v[4] = {};
    if (real) {
      const uint32_t* src = xw + static_cast<long long>(group) * 64 + 16 * i + c;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __ldg(src + 4 * j);
    }
    float top = 0.f, X = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      top = fmaxf(top, fmaxf(fabsf(low_f(v[j])), fabsf(high_f(v[j]))));
      X += low_f(v[j]) + high_f(v[j]);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      X += __shfl_xor_sync(~0u, X, d);
    }
    // 2^s with s = 14 - exponent(top), kept where 2^s and 2^-s are normal
    const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int s = min(max(14 - ex, -113), 126);
    const float up = __int_as_float((127 + s) << 23);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 q = __floats2half2_rn(low_f(v[j]) * up, high_f(v[j]) * up);
      h[j] = *reinterpret_cast<const uint32_t*>(&q);
    }
    if (real) {
      reinterpret_cast<uint4*>(p.xp)[u] = make_uint4(h[0], h[1], h[2], h[3]);
      if (lane % 16 == 0) p.xs[group] = make_float2(X, __int_as_float((127 - s) << 23));
    }
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
      if (i * 32 >= p.E) continue;  // (for every lane)
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
        if (i * 32 >= p.E) break;
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
      for (int i = 0; i < kPer; ++i) {
        if (i * 32 >= p.E) break;
        if (i * 32 + lane == e) rank[i] = 0u;
      }
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
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The A fragment of one packed word.  fp16: columns r as 1024 + q, columns
// r + 8 as 1024 + 16 q.  bf16: 128 + q.
template <bool BF16>
__device__ __forceinline__ void operand(uint32_t w, uint32_t (&a)[4]) {
  if constexpr (BF16) {
    a[0] = lop3_and_or(w, 0x000F000Fu, kBiasB16);
    a[1] = lop3_and_or(w >> 4, 0x000F000Fu, kBiasB16);
    a[2] = lop3_and_or(w >> 8, 0x000F000Fu, kBiasB16);
    a[3] = lop3_and_or(w >> 12, 0x000F000Fu, kBiasB16);
  } else {
    const uint32_t v = w >> 8;
    a[0] = lop3_and_or(w, 0x000F000Fu, kBias16);
    a[1] = lop3_and_or(w, 0x00F000F0u, kBias16);
    a[2] = lop3_and_or(v, 0x000F000Fu, kBias16);
    a[3] = lop3_and_or(v, 0x00F000F0u, kBias16);
  }
}

constexpr int kTiles = 2;  // of 16 columns, per item
constexpr int kStage = kTiles * kBlockBytes;
constexpr int kCols = kTiles * kTileN;
template <int NT>  // 8-row B tiles
struct Stream {
  static constexpr int kStages = NT == 1 ? 5 : 4;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kPart = NT * 8 * kCols;  // floats that a warp leaves of a unit: [row][column]
  static constexpr int kBytes = kRing + 2 * kWarps * kPart * 4;
};

// A picked expert's rows, from one lane's point of view: its B row (r of each
// 8-row tile) in operand order, and where the sums of rows 2c, 2c + 1 are.
// Columns beyond the count repeat the last row; nothing of theirs is kept.
template <int NT>
struct Rows {
  const uint8_t* x[NT];
  const float* sums[NT][2];
};

// PHASE 0: gate and up, a unit is a gate tile and its up tile; 1: down, a unit
// is two neighbouring tiles.  TEAM: warps that share a unit.
template <int PHASE, int NT, int TEAM>
__global__ void __launch_bounds__(kThreads, 2) expert_kernel(const __grid_constant__ Params p) {
  using S = Stream<NT>;
  constexpr bool kBf16 = PHASE == 1;
  constexpr int kTeams = kWarps / TEAM;
  constexpr int kMine = kParts / TEAM;  // parts of a unit that one warp sums
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Lists lists;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // (uniform, and known to be)
  const int team = warp / TEAM, member = warp % TEAM;

  // The logits: of the preceding kernel (phase 0), or of the one before, which
  // had completed when the preceding one let this one launch (phase 1).
  if (PHASE == 0) {
    grid_dependency_wait();
    grid_dependents_launch();
  }
  make_lists(p, lists);
  if (PHASE == 0 && blockIdx.x == 0)
    for (int i = tid; i < p.M * p.top_k; i += kThreads) p.weights[i] = lists.weight[i];

  const int K = PHASE == 0 ? p.D : p.F;
  const int G = K / kGroup;
  const int per = PHASE == 0 ? p.F / kTileN : p.D / kCols;  // units of an expert
  const int units = lists.experts * per;
  const int share = blockIdx.x * kTeams + team, shares = gridDim.x * kTeams;
  const int u0 = static_cast<int>(static_cast<long long>(units) * share / shares);
  const int nu = static_cast<int>(static_cast<long long>(units) * (share + 1) / shares) - u0;
  const uint8_t* weights = PHASE == 0 ? p.gate_up : p.down;
  const long long quad_bytes = static_cast<long long>(G) * kQuadBytes;
  const long long expert_bytes = (PHASE == 0 ? p.F / 32 : p.D / 64) * quad_bytes;
  const uint32_t ring = smem_addr(smem) + warp * S::kStages * kStage;
  const uint8_t* ring_ptr = smem + warp * S::kStages * kStage;

  // A warp's items: in each unit of its team the groups of its parts, part by
  // part in the order in which they are added.  The members take turns from
  // unit to unit, so that they stay even where the groups do not divide.
  auto turn = [&](int u) { return static_cast<int>(static_cast<unsigned>(member - u * G) % TEAM); };
  auto part_at = [](int m, int i) { return m + 4 * (i & 1) + 2 * (i >> 1); };

  // The copies run kStages items ahead.
  int c_unit = 0, c_turn = turn(0), c_i = 0, c_group = c_turn;
  int c_expert = u0 / per, c_at = u0 % per;
  const uint8_t *c_src = nullptr, *c_src2 = nullptr;
  auto place = [&] {  // this lane's 16 bytes in group 0 of the unit's tiles
    const uint8_t* base = weights + lists.expert[c_expert] * expert_bytes + 16 * lane;
    if (PHASE == 0) {
      const int t2 = c_at + per;
      c_src = base + (c_at / kQuadTiles) * quad_bytes + (c_at % kQuadTiles) * kBlockBytes;
      c_src2 = base + (t2 / kQuadTiles) * quad_bytes + (t2 % kQuadTiles) * kBlockBytes;
    } else {
      c_src = base + (c_at / 2) * quad_bytes + (c_at % 2) * kStage;
    }
  };
  auto settle = [&] {  // to the warp's next item, once c_group is past the depth
    while (c_group >= G && c_unit < nu) {
      if (++c_i == kMine) {
        c_i = 0;
        if (++c_unit == nu) return;
        if (++c_at == per) {
          c_at = 0;
          ++c_expert;
        }
        c_turn = turn(c_unit);
        place();
      }
      c_group = part_at(c_turn, c_i);
    }
  };
  auto copy = [&](int stage) {
    if (c_unit < nu) {
      const uint32_t dst = ring + stage * kStage + 16 * lane;
      const int off = c_group * kQuadBytes;
      if (PHASE == 0) {
        cp_async16(dst, c_src + off);
        cp_async16(dst + 512, c_src + off + 512);
        cp_async16(dst + kBlockBytes, c_src2 + off);
        cp_async16(dst + kBlockBytes + 512, c_src2 + off + 512);
        // the 64 bytes of scales and minima behind each: 4 + 4 lanes
        if (lane < 4) cp_async16(dst + 1024, c_src + off + 1024);
        else if (lane < 8) cp_async16(dst + kBlockBytes + 1024 - 64, c_src2 + off + 1024 - 64);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dst + 512 * i, c_src + off + 512 * i);
        if (lane < (kStage - 2048) / 16) cp_async16(dst + 2048, c_src + off + 2048);
      }
      c_group += kParts;
      settle();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (nu > 0) {
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
  int at = u0 % per, a = u0 / per;
  int first = 0, count = 0;
  Rows<NT> rows = {};
  float* parts = reinterpret_cast<float*>(smem + S::kRing) + team * 2 * TEAM * S::kPart;  // two halves that take turns

  // One item: d += .., for NA of the B tiles.
  auto item = [&](auto na, int group, float (&acc)[kTiles][NT][4]) {
    constexpr int NA = decltype(na)::value;
    uint4 xv[NA][4];
    float2 xs[NA][2];  // X, and (phase 0) the factor of the products
#pragma unroll
    for (int n = 0; n < NA; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[n][i] = *reinterpret_cast<const uint4*>(rows.x[n] + group * 256 + i * 64);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (PHASE == 0) {
          xs[n][k] = reinterpret_cast<const float2*>(rows.sums[n][k])[group];
        } else {
          const float4 v = reinterpret_cast<const float4*>(rows.sums[n][k])[group * 2];
          const float4 w = reinterpret_cast<const float4*>(rows.sums[n][k])[group * 2 + 1];
          xs[n][k].x = ((v.x + v.y) + (v.z + v.w)) + ((w.x + w.y) + (w.z + w.w));
        }
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
    __syncwarp();
    const uint8_t* st = ring_ptr + stage * kStage;
    float d[kTiles][NA][4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 q[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) q[t] = *reinterpret_cast<const uint4*>(st + t * kBlockBytes + 512 * h + 16 * lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = 4 * h + j;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          uint32_t w[4];
          operand<kBf16>(j == 0 ? q[t].x : j == 1 ? q[t].y : j == 2 ? q[t].z : q[t].w, w);
#pragma unroll
          for (int n = 0; n < NA; ++n)
            mma<kBf16>(d[t][n], w, s % 2 ? xv[n][s / 2].z : xv[n][s / 2].x, s % 2 ? xv[n][s / 2].w : xv[n][s / 2].y);
        }
      }
    }
    uint2 meta[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) meta[t] = *reinterpret_cast<const uint2*>(st + t * kBlockBytes + kCodeBytes + 8 * r);
    __syncwarp();  // the stage is read out
    copy(stage);
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      float s0 = low_f(meta[t].x), s1 = low_f(meta[t].y);
      const float b0 = fmaf(kBf16 ? -128.f : -1024.f, s0, high_f(meta[t].x));
      const float b1 = fmaf(kBf16 ? -128.f : -64.f, s1, high_f(meta[t].y));
      if (!kBf16) s1 *= 0.0625f;  // these columns carry 16 q
#pragma unroll
      for (int n = 0; n < NA; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float f0 = kBf16 ? s0 : s0 * xs[n][k].y, f1 = kBf16 ? s1 : s1 * xs[n][k].y;
          acc[t][n][k] = fmaf(f0, d[t][n][k], fmaf(b0, xs[n][k].x, acc[t][n][k]));
          acc[t][n][2 + k] = fmaf(f1, d[t][n][2 + k], fmaf(b1, xs[n][k].x, acc[t][n][2 + k]));
        }
    }
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;

  int expert_seen = -1;
  for (int u = 0; u < nu; ++u) {
    if (a != expert_seen) {
      expert_seen = a;
      first = lists.first[a];
      count = lists.first[a + 1] - first;
      auto source = [&](int i) {
        const int pick = lists.pick[first + min(i, count - 1)];
        return static_cast<long long>(PHASE == 0 ? pick / p.top_k : pick);
      };
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        rows.x[n] = (PHASE == 0 ? p.xp : p.act) + source(n * 8 + r) * K * 2 + 16 * c;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const long long m = source(n * 8 + 2 * c + k);
          rows.sums[n][k] = PHASE == 0 ? reinterpret_cast<const float*>(p.xs) + m * (G * 2) : p.acts + m * (G * 8);
        }
      }
    }
    float* part = parts + (u & 1) * TEAM * S::kPart;
    const int mine = turn(u);
    float sum[kTiles][NT][4];
#pragma unroll
    for (int q = 0; q < (kMine + 1) / 2; ++q) {
      float two[kTiles][NT][4];
#pragma unroll
      for (int h = 0; h < (kMine > 1 ? 2 : 1); ++h) {
        float acc[kTiles][NT][4] = {};
        const int v = part_at(mine, 2 * q + h);
        if (NT == 2 && count > 8) {
          if constexpr (NT == 2)
            for (int g = v; g < G; g += kParts) item(Two{}, g, acc);
        } else {
          for (int g = v; g < G; g += kParts) item(One{}, g, acc);
        }
#pragma unroll
        for (int i = 0; i < kTiles * NT * 4; ++i) (&two[0][0][0])[i] = h == 0 ? (&acc[0][0][0])[i] : (&two[0][0][0])[i] + (&acc[0][0][0])[i];
      }
#pragma unroll
      for (int i = 0; i < kTiles * NT * 4; ++i) (&sum[0][0][0])[i] = q == 0 ? (&two[0][0][0])[i] : (&sum[0][0][0])[i] + (&two[0][0][0])[i];
    }
    float* out = part + mine * S::kPart;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = n * 8 + 2 * c + (i & 1);
          if (m < count) out[m * kCols + t * kTileN + r + 8 * (i >> 1)] = sum[t][n][i];
        }
    // One barrier of the team per unit: the other half of the buffer is free
    // again once every member is past the next one.
    if constexpr (TEAM == kWarps) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TEAM * 32) : "memory");
    const int tt = member * 32 + lane;
    auto join = [&](const float* q) {  // (parts beyond the depth are 0)
      if constexpr (TEAM == 2) return q[0] + q[S::kPart];
      else
        return ((q[0] + q[4 * S::kPart]) + (q[2 * S::kPart] + q[6 * S::kPart])) +
               ((q[S::kPart] + q[5 * S::kPart]) + (q[3 * S::kPart] + q[7 * S::kPart]));
    };
    if (PHASE == 0) {
      const int o = (tt + 32 * (u % TEAM)) % (TEAM * 32);  // the folding warps take turns
      const int m = o / kTileN, col = o % kTileN;
      if (o / 32 * 2 < count) {  // whole warps
        float act = 0.f;
        if (m < count) {
          const int pick = lists.pick[first + m];
          const float v = join(part + m * kCols + col), w = join(part + m * kCols + col + kTileN);
          const __nv_bfloat16 b = __float2bfloat16_rn(v / (1.f + expf(-v)) * w);
          act = __bfloat162float(b);
          // columns 16 at + col: k step at % 8 of the group
          uint8_t* dst = p.act + static_cast<long long>(pick) * p.F * 2 + at / 8 * 256 + at % 8 / 2 * 64 + col % 8 / 2 * 16 +
                         (at % 2 * 2 + col / 8) * 4 + (col & 1) * 2;
          *reinterpret_cast<__nv_bfloat16*>(dst) = b;
        }
#pragma unroll
        for (int k = 8; k > 0; k >>= 1) act += __shfl_xor_sync(~0u, act, k);
        if (m < count && col == 0)
          p.acts[static_cast<long long>(lists.pick[first + m]) * (p.F / kTileN) + at] = act;
      }
    } else {
      for (int o = (tt + 32 * (u % TEAM)) % (TEAM * 32); o < count * kCols; o += TEAM * 32) {
        const int m = o / kCols, col = o % kCols;
        p.part[static_cast<long long>(lists.pick[first + m]) * p.D + at * kCols + col] = join(part + m * kCols + col);
      }
    }
    if (++at == per) {
      at = 0;
      ++a;
    }
  }
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
  size_t logits, weights, xp, xs, act, acts, part, total;
};
Layout layout(const w4g128_moe_args& a) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  const size_t M = a.M, picks = M * a.top_k;
  Layout l;
  l.logits = kStatusBytes;
  l.weights = l.logits + up(M * a.E * 4);
  l.xp = l.weights + up(picks * 4);
  l.xs = l.xp + up(M * a.D * 2);
  l.act = l.xs + up(M * (a.D / 128) * 8);
  l.acts = l.act + up(picks * a.F * 2);
  l.part = l.acts + up(picks * (a.F / 16) * 4);
  l.total = l.part + up(picks * a.D * 4);
  return l;
}

template <int PHASE, int NT, int TEAM>
cudaError_t launch_expert(cudaLaunchConfig_t& cfg, const Params& p, int sms, long long units) {
  constexpr int kBytes = Stream<NT>::kBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(expert_kernel<PHASE, NT, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(2 * sms, units)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  return cudaLaunchKernelEx(&cfg, expert_kernel<PHASE, NT, TEAM>, p);
}

template <int NT>
cudaError_t launch_experts(cudaLaunchConfig_t& cfg, const Params& p, int sms) {
  const long long most = std::min(p.M * p.top_k, p.E);  // picked experts
  const cudaError_t e = launch_expert<0, NT, 8>(cfg, p, sms, most * (p.F / kTileN));
  if (e != cudaSuccess) return e;
  const long long units = most * (p.D / kCols);
  // small teams where every team has several units
  return units >= 16 * sms ? launch_expert<1, NT, 2>(cfg, p, sms, units) : launch_expert<1, NT, 8>(cfg, p, sms, units);
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
  e = p.M <= 8 ? launch_experts<1>(cfg, p, sms) : launch_experts<2>(cfg, p, sms);
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
  p.xs = reinterpret_cast<float2*>(base + l.xs);
  p.act = base + l.act;
  p.acts = reinterpret_cast<float*>(base + l.acts);
  p.part = reinterpret_cast<float*>(base + l.part);
  if (launch(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
