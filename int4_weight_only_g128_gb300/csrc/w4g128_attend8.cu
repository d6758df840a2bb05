// Attention of 1..16 new tokens per sequence over a paged cache of e4m3 codes
// with a scale for each block of positions and head (w4g128_attend8).
//
// As in w4g128_attend, rows of one key/value head (new tokens x query heads that
// share it) are the 16-row tiles of a warp MMA and the work is the cache's bytes:
// half as many, so that what is left is latency and the conversion of the codes.
//   * Every code is an fp16 value, so both products are fp16 x fp16 -> fp32.  q,
//     bf16, becomes fp16 scaled by a power of two for each row (exact down to
//     2^-31 of the row's largest value).
//   * A key's scale multiplies its score.  A value's scale enters the softmax
//     weight: with score s_j (base 2) and value scale v_j, P_j = 2^(s_j + log2 v_j - m),
//     rounded to fp16 as an operand, and the row's sum takes P_j / v_j.  The
//     reference m follows the maximum of s_j + log2 v_j, so P_j stays in fp16's range
//     whatever the scales are, and depends on the row alone.
//   * Codes are read by ldmatrix as pairs: K's depth and V's columns then come in
//     another order than the MMA's, the same for q (laid out so) and for the result.
//   * The 16-position tiles of a sequence go in turn to all the groups of warps that
//     work on it, whatever its length, so all of them have the same share and no CTA
//     depends on how long a sequence may become.  A group keeps a ring of cp.async
//     stages and a running reference and sums of its own.
//   * The CTAs of a head are a cluster, which joins their sums through its shared
//     memory.  Only if one cluster is too small for the call does a second kernel
//     join several.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "w4g128_divide.cuh"
#include "w4g128_e4m3.cuh"
#include "w4g128_internal.h"
#include "w4g128_ops.h"
#include "w4g128_ptx.cuh"

namespace w4g128 {
namespace {

constexpr int kTile = 16;  // positions per tile
constexpr size_t kStatusBytes = 256;
constexpr float kNone = -INFINITY;
constexpr float kSlack = 8.f;  // a reference follows its maximum when that is above it by more (base 2)
constexpr float kLift = 6.f;   // weights are up to 2^(kSlack + kLift): fp16 holds them down to 2^-30 of the largest
constexpr float kLowestScale = 0x1p-80f;  // of a value: smaller ones count as this, so that weights over scales stay in range
constexpr float kLowWeight = 0x1p-90f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMostCluster = 16;

struct Params {
  const uint16_t* q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *table, *offsets, *lens;
  uint16_t* out;
  long long q_row, out_row, page_stride, slot_stride, head_stride, scale_page, scale_head, table_row;
  int rows, count, q_heads, kv_heads, group, pages, block_log2, max_len, max_new, window, sinks;
  int clusters, row_groups;  // of a sequence and head
  Divisor by_group, by_page, by_clusters, by_row_groups, by_kv_heads;
  float scale2;              // |scale| log2(e); scale < 0: q's signs are flipped, scale = 0: q counts as 0
  uint32_t flip_q, keep_q;
  unsigned long long* status;
  float* part;               // [count][kv_heads][clusters][max_new * group][head_dim]: unnormalised sums
  float2* stat;              // [count][kv_heads][clusters][max_new * group]: reference and sum
};

struct Seq {
  bool ok;
  int first_row, n, len, start;  // start: the first new row's position (negative rows are empty)
  int first;                     // the first real row's position
  int lo, sink;                  // visible to some row: [0, sink) and [lo, len)
};

__device__ __forceinline__ Seq sequence(const Params& p, int b) {
  Seq s;
  s.first_row = p.offsets[b];
  s.n = p.offsets[b + 1] - s.first_row;
  s.len = p.lens[b];
  s.ok = s.first_row >= 0 && s.n >= 0 && s.n <= p.max_new && s.first_row <= p.rows - s.n && s.len >= 0 &&
         s.len <= p.max_len;
  s.start = s.len - s.n;
  s.first = max(s.start, 0);
  s.lo = p.window > 0 ? max(0, s.first - p.window + 1) : 0;
  s.sink = p.window > 0 ? min(p.sinks, s.lo) : 0;
  return s;
}

__device__ __forceinline__ bool visible(const Params& p, int row_pos, int pos) {
  return pos <= row_pos && (p.window == 0 || row_pos - pos < p.window || pos < p.sinks);
}

// One CTA looks all lengths, row ranges and visible page ids over, beside the others.
__device__ void check_all(const Params& p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int parts = max(1, warps / p.count);  // warps that share a sequence
  bool bad = false;
  for (int b = warp / parts; b < p.count; b += warps / parts) {
    const Seq s = sequence(p, b);
    bad |= !s.ok;
    if (!s.ok || s.n == 0) continue;
    const int sink_pages = (s.sink + static_cast<int>(p.by_page.d) - 1) / p.by_page;
    const int end = s.len > 0 ? (s.len - 1) / p.by_page + 1 : 0;
    const int low = max(s.lo / p.by_page, sink_pages), all = sink_pages + end - low;
    for (int i = (warp % parts) * 32 + lane; i < all; i += parts * 32) {
      const int id = p.table[static_cast<long long>(b) * p.table_row + (i < sink_pages ? i : low + i - sink_pages)];
      bad |= id < 0 || id >= p.pages;
    }
  }
  if (__syncthreads_or(bad)) bad = true;
  if (threadIdx.x == 0) st_relaxed_u64(p.status, bad ? W4G128_ERR_CACHE : W4G128_OK);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 or 4 bytes, or zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_fast(float x) {  // 2^-22
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse_fast(float x) {  // 1 ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float low_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t low_codes(uint32_t v) { return e4m3x2_to_half2(static_cast<uint16_t>(v)); }
__device__ __forceinline__ uint32_t high_codes(uint32_t v) { return e4m3x2_to_half2(static_cast<uint16_t>(v >> 16)); }
// Bit 7 of each byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t v) { return ((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_v2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// KG groups of warps with tiles of their own, RT row tiles, DS warps per row tile.
constexpr int groups_of(int head_dim) { return head_dim == 256 ? 2 : 4; }
template <int D, int RT>
struct Shape {
  static constexpr int kDs = D == 256 ? 2 : 1;
  static constexpr int kKg = groups_of(D);
  static constexpr int kGroup = RT * kDs * 32;  // threads of a group
  static constexpr int kThreads = kKg * kGroup;
  static constexpr int kRows = RT * 16;
  static constexpr int kTileBytes = kTile * D;  // K or V of one tile
  static constexpr int kStageBytes = 2 * kTileBytes + 2 * kTile * 4;  // and their positions' scales
  // stages: what 512 threads an SM (128 registers each) leave room for
  static constexpr int kStages = RT == 1 ? (D == 64 ? 6 : D == 128 ? 3 : 2) : D == 64 ? 8 : D == 256 && RT == 2 ? 5 : 6;
  static constexpr bool kQInRegs = D == 64;  // else its fragments are read from shared memory for each tile
  static constexpr int kQBytes = kQInRegs ? 0 : kRows * 2 * D;
  static constexpr int kRing = kKg * kStages * kStageBytes;
  static constexpr int kHalf = D / kDs;      // columns of a warp
  static constexpr int kSumRow = D + 16;     // floats of a row's sums (free of bank conflicts)
  static constexpr int kLeft = kRows * (kSumRow + 2) * 4;  // a group's sums, references and sums of weights
  static constexpr int kBytes = kQBytes + (kRing > kKg * kLeft ? kRing : kKg * kLeft);
  static constexpr int kExchange = kDs == 2 ? kKg * RT * 2 * 32 : 1;  // float4: [group][row tile][half]..
};

template <int D, int RT>
__global__ void __launch_bounds__(Shape<D, RT>::kThreads, 512 / Shape<D, RT>::kThreads)
attend8_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, RT>;
  constexpr int kSteps = S::kHalf / 16;  // of Q K^T, per warp
  constexpr int kPieces = D / 16;        // 16-byte pieces of a row of codes
  constexpr int kPer = 2 * kTile * kPieces / S::kGroup;  // pieces of a tile's K and V that one thread copies
  constexpr int kStep = S::kGroup / kPieces;             // rows between them
  static_assert(S::kGroup % kPieces == 0 && 2 * kTile % kStep == 0, "a thread copies one column of pieces");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float4 s_half[S::kExchange][2];
  __shared__ float s_factor[S::kQInRegs ? 1 : S::kRows];  // a row's score factor

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);
  const int kg = warp / (RT * S::kDs), rt = warp / S::kDs % RT, half = warp % S::kDs;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
  const int cluster = static_cast<int>(blockIdx.x) / ctas;

  grid_dependency_wait();
  if (cluster == 0) {
    if (rank == 0) check_all(p);
    return;
  }
  // cluster - 1 = ((b kv_heads + head) row_groups + rg) clusters + cl
  int rest = (cluster - 1) / p.by_clusters;
  const int cl = cluster - 1 - rest * p.clusters;
  int up = rest / p.by_row_groups;
  const int rg = rest - up * p.row_groups;
  const int b = up / p.by_kv_heads;
  const int head = up - b * p.kv_heads;

  const int groups = p.clusters * ctas * S::kKg;  // of this head and sequence
  const int mine = (cl * ctas + rank) * S::kKg + kg;
  const int* table = p.table + static_cast<long long>(b) * p.table_row;
  // Without a window the first tiles are known before the length is: their page
  // ids come along with it, a tile a lane.
  int ids = -1, ids_next = -1;
  if (p.window == 0) {
    const int a = (mine + lane * groups) * kTile;
    if (a < p.max_len) ids = table[a / p.by_page];
  }
  const Seq s = sequence(p, b);
  if (!s.ok) return;
  const int live_rows = s.n * p.group;
  if (rg * S::kRows >= live_rows) return;

  // Q, asked for before the table is waited for.
  const int r = lane >> 2, c = lane & 3;
  const int row0 = (rg * RT + rt) * 16 + r;
  const bool busy = (rg * RT + rt) * 16 < live_rows;  // (of the warp)
  const int pos_a = row0 < live_rows ? s.start + row0 / p.by_group : -1;  // the rows' positions
  const int pos_b = row0 + 8 < live_rows ? s.start + (row0 + 8) / p.by_group : -1;
  auto q_row = [&](int row) {
    const int i = row / p.by_group;
    return p.q + static_cast<long long>(s.first_row + i) * p.q_row +
           static_cast<long long>(head * p.group + row - i * p.group) * D;
  };
  constexpr int kQPer = S::kQInRegs ? 1 : S::kRows * (D / 8) / S::kThreads;  // pieces of 8 values of a thread
  static_assert(S::kQInRegs || S::kRows * (D / 8) % S::kThreads == 0, "each thread loads as many pieces of Q");
  [[maybe_unused]] uint32_t qf[S::kQInRegs ? kSteps : 1][4] = {};
  [[maybe_unused]] uint4 q_part[kQPer] = {};
  if constexpr (S::kQInRegs) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      if (row0 + 8 * side < live_rows) {
        const uint2* from = reinterpret_cast<const uint2*>(q_row(row0 + 8 * side)) + c;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint2 v = __ldg(from + k * 4);
          qf[k][side] = v.x;
          qf[k][side + 2] = v.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kQPer; ++e) {
      const int i = tid + e * S::kThreads, row = rg * S::kRows + i / (D / 8);
      if (row < live_rows) q_part[e] = __ldg(reinterpret_cast<const uint4*>(q_row(row)) + i % (D / 8));
    }
  }

  // This group's tiles: every groups-th, of the sinks' and then of the others.
  const int sink_tiles = (s.sink + kTile - 1) / kTile, end_tile = (s.len + kTile - 1) / kTile;
  const int low_tile = max(s.lo / kTile, sink_tiles);
  int of_sinks = 0, low = mine;
  if (p.window > 0) {
    of_sinks = mine < sink_tiles ? (sink_tiles - 1 - mine) / groups + 1 : 0;
    if (mine < low_tile) low = mine + (low_tile - mine + groups - 1) / groups * groups;
  }
  const int total = of_sinks + (low < end_tile ? (end_tile - 1 - low) / groups + 1 : 0);
  auto tile_of = [&](int k) { return k < of_sinks ? mine + k * groups : low + (k - of_sinks) * groups; };
  auto ids_from = [&](int k) { return k < total ? table[tile_of(k) * kTile / p.by_page] : -1; };
  if (p.window == 0) ids = lane < total ? ids : -1;
  else ids = ids_from(lane);
  if (total > 32) ids_next = ids_from(32 + lane);

  float acc[S::kHalf / 8][4];  // [2 i]: columns 16 i + 4 c, + 2 of rows r and r + 8; [2 i + 1]: + 1, + 3
#pragma unroll
  for (int i = 0; i < S::kHalf / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  float m_a = kNone, m_b = kNone, l_a = 0.f, l_b = 0.f;

  uint8_t* ring = smem + S::kQBytes + kg * S::kStages * S::kStageBytes;
  const uint32_t ring_at = smem_addr(ring);
  auto group_sync = [&] {
    if constexpr (S::kGroup == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(kg + 1), "n"(S::kGroup) : "memory");
  };
  auto swizzled = [](int j, int piece) { return j * D + ((piece ^ (D == 64 ? (j >> 1) & 3 : j & 7)) << 4); };

  // A thread copies one column of pieces: rows j0, j0 + kStep, .. of K, then of V.
  const int gl = (warp % (RT * S::kDs)) * 32 + lane;
  const int ch = gl % kPieces, j0 = gl / kPieces;
  const uint8_t* k_base = p.k_cache + head * p.head_stride + ch * 16;
  const long long v_off = p.v_cache - p.k_cache;
  const float* scale_base = ((gl & 16) ? p.v_scale : p.k_scale) + head * p.scale_head;
  uint32_t okays = 0u;  // of the tiles on their way, by their number mod 32: on a page
  auto issue = [&](int k, int stage) {
    if (k < total) {
      if (k > 0 && (k & 31) == 0) {
        ids = ids_next;
        ids_next = ids_from(k + 32 + lane);
      }
      const int a = tile_of(k) * kTile, page = a / p.by_page;
      const int id = __shfl_sync(~0u, ids, k & 31);
      const bool ok = id >= 0 && id < p.pages;
      okays = (okays & ~(1u << (k & 31))) | (ok ? 1u : 0u) << (k & 31);
      const int slot = a - page * static_cast<int>(p.by_page.d);
      const uint8_t* src = k_base + (ok ? id * p.page_stride + slot * p.slot_stride : 0);
      const uint32_t dst = ring_at + stage * S::kStageBytes;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int jj = j0 + e * kStep, j = jj % kTile;
        const bool is_v = jj >= kTile;
        const bool real = ok && a + j < s.len;
        cp_async16_or_zero(dst + (is_v ? S::kTileBytes : 0) + swizzled(j, ch),
                           real ? src + (is_v ? v_off : 0) + j * p.slot_stride : p.k_cache, real);
      }
      if (gl < 32) {
        const int j = gl & 15;
        const bool real = ok && a + j < s.len;
        cp_async4_or_zero(dst + 2 * S::kTileBytes + gl * 4,
                          real ? scale_base + id * p.scale_page + ((slot + j) >> p.block_log2) : p.k_scale, real);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) issue(i, i);

  // q as fp16, its row's largest value brought to 2^14 .. 2^15 (a negative scale
  // goes into q's signs, a scale of 0 makes q 0).
  auto signed_q = [&](uint32_t v) { return (v & p.keep_q) ^ p.flip_q; };
  auto largest = [](uint32_t v, float top) {
    const float x = fabsf(low_f(v)), y = fabsf(high_f(v));
    return fmaxf(top, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
  };
  auto shift_for = [](float top) {
    return min(max(14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), -112), 110);
  };
  auto power = [](int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); };
  float factor_a = 0.f, factor_b = 0.f;
  if constexpr (S::kQInRegs) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) top = largest(qf[k][side], largest(qf[k][side + 2], top));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      const int e = shift_for(top);
      const float by = power(e);
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = side; i < 4; i += 2) {
          const uint32_t v = signed_q(qf[k][i]);
          qf[k][i] = pack_half(low_f(v) * by, high_f(v) * by);
        }
      (side ? factor_b : factor_a) = p.scale2 * power(-e);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kQPer; ++e) {
      const int i = tid + e * S::kThreads, j = i / (D / 8), piece = i % (D / 8);
      uint32_t w[4] = {signed_q(q_part[e].x), signed_q(q_part[e].y), signed_q(q_part[e].z), signed_q(q_part[e].w)};
      float top = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) top = largest(w[u], top);
#pragma unroll
      for (int d = 1; d < D / 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      const int shift = shift_for(top);
      const float by = power(shift);
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = pack_half(low_f(w[u]) * by, high_f(w[u]) * by);
      if (piece == 0) s_factor[j] = p.scale2 * power(-shift);
      // The 16 depths of a step in the order in which K's pairs of pairs come: 0 1 4 5 8 9 12 13, then the others.
      const int step = piece >> 1, odd = piece & 1;
      uint8_t* to = smem + j * 2 * D;
      *reinterpret_cast<uint2*>(to + (((2 * step) ^ (j & 7)) << 4) + odd * 8) = make_uint2(w[0], w[2]);
      *reinterpret_cast<uint2*>(to + (((2 * step + 1) ^ (j & 7)) << 4) + odd * 8) = make_uint2(w[1], w[3]);
    }
    __syncthreads();
    factor_a = s_factor[rt * 16 + r];
    factor_b = s_factor[rt * 16 + r + 8];
  }

  // ldmatrix: this lane's row of a tile of K or V and its pieces (2 i + lane / 16),
  // and of Q (rows 0-7, 8-15 of pieces 2 k, then of 2 k + 1).
  const int lj = lane & 15, lp = lane >> 4;
  const uint32_t q_at = smem_addr(smem) + rt * 16 * 2 * D + lj * 2 * D;
  const int last_pos = s.len - 1;  // of the sequence's last row
  int stage = 0;
#pragma unroll 1
  for (int k = 0; k < total; ++k) {
    cp_async_wait_group<S::kStages - 2>();
    group_sync();  // the tile is there for the group, and the stage refilled next is read out
    issue(k + S::kStages - 1, stage == 0 ? S::kStages - 1 : stage - 1);
    const int stage_bytes = stage * S::kStageBytes;
    const uint32_t tile = ring_at + stage_bytes;
    const int a = tile_of(k) * kTile;
    if (busy) {
      float sc[2][4] = {}, odd_k[2][4] = {};  // two chains of products each
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) {
        uint32_t kb[4], qk[2][4];
        ldmatrix4(kb, tile + swizzled(lj, half * (kPieces / S::kDs) + 2 * i + lp));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (S::kQInRegs) {
#pragma unroll
            for (int e = 0; e < 4; ++e) qk[u][e] = qf[2 * i + u][e];
          } else {
            ldmatrix4(qk[u], q_at + (((2 * (half * kSteps + 2 * i + u) + lp) ^ (lj & 7)) << 4));
          }
        }
        mma(sc[0], qk[0], low_codes(kb[0]), high_codes(kb[0]));
        mma(sc[1], qk[0], low_codes(kb[1]), high_codes(kb[1]));
        mma(odd_k[0], qk[1], low_codes(kb[2]), high_codes(kb[2]));
        mma(odd_k[1], qk[1], low_codes(kb[3]), high_codes(kb[3]));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[h][i] += odd_k[h][i];
      if constexpr (S::kDs == 2) {  // the other half of the depth (read out before the group's next barrier)
        float4* ex = &s_half[(kg * RT + rt) * 2 * 32][0];
        ex[(half * 32 + lane) * 2] = make_float4(sc[0][0], sc[0][1], sc[0][2], sc[0][3]);
        ex[(half * 32 + lane) * 2 + 1] = make_float4(sc[1][0], sc[1][1], sc[1][2], sc[1][3]);
        asm volatile("bar.sync %0, 64;" ::"r"(S::kKg + 1 + kg * RT + rt) : "memory");
        const float4 u = ex[((half ^ 1) * 32 + lane) * 2], v = ex[((half ^ 1) * 32 + lane) * 2 + 1];
        sc[0][0] += u.x; sc[0][1] += u.y; sc[0][2] += u.z; sc[0][3] += u.w;
        sc[1][0] += v.x; sc[1][1] += v.y; sc[1][2] += v.z; sc[1][3] += v.w;
      }
      // the scales of this lane's positions 2 c, 2 c + 1, + 8
      const float* scales = reinterpret_cast<const float*>(ring + stage_bytes + 2 * S::kTileBytes);
      float inverse[2][2], log_v[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 ks = *reinterpret_cast<const float2*>(scales + h * 8 + 2 * c);
        const float2 vs = *reinterpret_cast<const float2*>(scales + kTile + h * 8 + 2 * c);
        const float v0 = fmaxf(vs.x, kLowestScale), v1 = fmaxf(vs.y, kLowestScale);
        const float log0 = log_v[h][0] = log2_fast(v0), log1 = log_v[h][1] = log2_fast(v1);
        inverse[h][0] = inverse_fast(v0);
        inverse[h][1] = inverse_fast(v1);
        sc[h][0] = fmaf(sc[h][0] * factor_a, ks.x, log0);
        sc[h][1] = fmaf(sc[h][1] * factor_a, ks.y, log1);
        sc[h][2] = fmaf(sc[h][2] * factor_b, ks.x, log0);
        sc[h][3] = fmaf(sc[h][3] * factor_b, ks.y, log1);
      }
      const bool page_ok = (okays >> (k & 31)) & 1u;
      // every row sees the whole tile
      const bool inside = s.start >= 0 && a + kTile - 1 <= s.first && page_ok &&
                          (p.window == 0 || last_pos - a < p.window || a + kTile <= p.sinks);
      auto sees = [&](int row_pos, int pos) { return visible(p, row_pos, pos) && page_ok; };
      if (!inside) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!sees(i < 2 ? pos_a : pos_b, a + h * 8 + 2 * c + (i & 1))) sc[h][i] = kNone;
      }
      float ta = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      float tb = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
      auto above = [&](float top, float m) { return top - m > kSlack; };  // (m may be that of no score)
      if (__any_sync(~0u, above(ta, m_a) || above(tb, m_b))) {
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          ta = fmaxf(ta, __shfl_xor_sync(~0u, ta, d));
          tb = fmaxf(tb, __shfl_xor_sync(~0u, tb, d));
        }
        const float na = above(ta, m_a) ? ta : m_a, nb = above(tb, m_b) ? tb : m_b;
        const float ga = na == m_a ? 1.f : exp2_fast(m_a - na);
        const float gb = nb == m_b ? 1.f : exp2_fast(m_b - nb);
        m_a = na;
        m_b = nb;
        l_a *= ga;
        l_b *= gb;
#pragma unroll
        for (int i = 0; i < S::kHalf / 8; ++i) {
          acc[i][0] *= ga;
          acc[i][1] *= ga;
          acc[i][2] *= gb;
          acc[i][3] *= gb;
        }
      }
      const float ra = m_a == kNone ? 0.f : kLift - m_a, rb = m_b == kNone ? 0.f : kLift - m_b;
      uint32_t pf[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float w0 = exp2_fast(sc[h][0] + ra), w1 = exp2_fast(sc[h][1] + ra);
        const float w2 = exp2_fast(sc[h][2] + rb), w3 = exp2_fast(sc[h][3] + rb);
        float u0 = w0 * inverse[h][0], u1 = w1 * inverse[h][1], u2 = w2 * inverse[h][0], u3 = w3 * inverse[h][1];
        // (beside values of much larger scales, P may be below fp32's range and the weight not)
        if (__any_sync(~0u, fminf(fminf(w0, w1), fminf(w2, w3)) < kLowWeight)) {
          if (w0 < kLowWeight) u0 = exp2_fast(sc[h][0] + ra - log_v[h][0]);
          if (w1 < kLowWeight) u1 = exp2_fast(sc[h][1] + ra - log_v[h][1]);
          if (w2 < kLowWeight) u2 = exp2_fast(sc[h][2] + rb - log_v[h][0]);
          if (w3 < kLowWeight) u3 = exp2_fast(sc[h][3] + rb - log_v[h][1]);
        }
        l_a += u0 + u1;
        l_b += u2 + u3;
        pf[2 * h] = pack_half(w0, w1);
        pf[2 * h + 1] = pack_half(w2, w3);
      }

      bool odd = false;  // NaN codes in a tile that not every row sees whole
      const uint8_t* v_tile = ring + stage_bytes + S::kTileBytes;
      if (!inside) {
        const uint4* v = reinterpret_cast<const uint4*>(v_tile);
        for (int i = lane; i < S::kTileBytes / 16; i += 32) {
          const uint4 u = v[i];
          odd |= (nan_codes(u.x) | nan_codes(u.y) | nan_codes(u.z) | nan_codes(u.w)) != 0u;
        }
        odd = __any_sync(~0u, odd);
      }
#pragma unroll
      for (int i = 0; i < S::kHalf / 32; ++i) {
        uint32_t vb[4];
        ldmatrix4_trans(vb, tile + S::kTileBytes + swizzled(lj, half * (kPieces / S::kDs) + 2 * i + lp));
        if (odd) {
#pragma unroll
          for (int e = 0; e < 4; ++e) vb[e] &= ~((nan_codes(vb[e]) >> 7) * 0xFFu);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) vb[e] = __byte_perm(vb[e], 0u, 0x3120);  // a column's two positions together
        mma(acc[4 * i], pf, low_codes(vb[0]), low_codes(vb[1]));
        mma(acc[4 * i + 1], pf, high_codes(vb[0]), high_codes(vb[1]));
        mma(acc[4 * i + 2], pf, low_codes(vb[2]), low_codes(vb[3]));
        mma(acc[4 * i + 3], pf, high_codes(vb[2]), high_codes(vb[3]));
      }
      if (odd) {  // a row that sees a NaN code has NaN in its column
        for (int j = 0; j < kTile; ++j) {
          const bool va = sees(pos_a, a + j), vb = sees(pos_b, a + j);
#pragma unroll
          for (int i = 0; i < S::kHalf / 16; ++i) {
            const uint32_t bad =
                nan_codes(*reinterpret_cast<const uint32_t*>(v_tile + swizzled(j, half * (kPieces / S::kDs) + i) + 4 * c));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((bad >> (8 * e + 7)) & 1u) {
                if (va) acc[2 * i + (e & 1)][e >> 1] = NAN;
                if (vb) acc[2 * i + (e & 1)][2 + (e >> 1)] = NAN;
              }
            }
          }
        }
      }
    }
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    l_a += __shfl_xor_sync(~0u, l_a, d);
    l_b += __shfl_xor_sync(~0u, l_b, d);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the ring becomes the exchange

  // Join the CTA's groups, then the cluster's CTAs, each time in order.
  float* left = reinterpret_cast<float*>(smem + S::kQBytes);
  constexpr int kLeft = S::kLeft / 4, kStat = S::kRows * S::kSumRow;
  const int rows_here = min(S::kRows, live_rows - rg * S::kRows);
  {
    float* mine_left = left + kg * kLeft;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int row = rt * 16 + r + 8 * side;
      if (row < rows_here) {
        float* to = mine_left + row * S::kSumRow + half * S::kHalf + 4 * c;
#pragma unroll
        for (int i = 0; i < S::kHalf / 16; ++i)
          *reinterpret_cast<float4*>(to + 16 * i) = make_float4(acc[2 * i][2 * side], acc[2 * i + 1][2 * side],
                                                                acc[2 * i][2 * side + 1], acc[2 * i + 1][2 * side + 1]);
        if (c == 0 && half == 0)
          *reinterpret_cast<float2*>(mine_left + kStat + 2 * row) = make_float2(side ? m_b : m_a, side ? l_b : l_a);
      }
    }
  }
  __syncthreads();
  const int units = rows_here * (D / 4);  // of 4 columns
  float4 sum;
  float2 st;
  auto join = [&](auto&& stat_of, auto&& sums_of, int n) {
    float top = kNone;
    for (int i = 0; i < n; ++i) top = fmaxf(top, stat_of(i).x);
    const float ref = top == kNone ? 0.f : top;
    sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float2 t = stat_of(i);
      const float w = exp2_fast(t.x - ref);
      const float4 v = sums_of(i);
      l = fmaf(t.y, w, l);
      sum.x = fmaf(v.x, w, sum.x);
      sum.y = fmaf(v.y, w, sum.y);
      sum.z = fmaf(v.z, w, sum.z);
      sum.w = fmaf(v.w, w, sum.w);
    }
    st = make_float2(top, l);
  };
  auto emit = [&](int u) {
    const int row = rg * S::kRows + u / (D / 4), col = u % (D / 4) * 4;
    if (p.clusters == 1) {
      const float inv = st.y == 0.f ? 0.f : 1.f / st.y;  // no visible position: zeros
      const int i = row / p.by_group;
      uint16_t* o = p.out + static_cast<long long>(s.first_row + i) * p.out_row +
                    static_cast<long long>(head * p.group + row - i * p.group) * D + col;
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
    } else {
      const long long at =
          ((static_cast<long long>(b) * p.kv_heads + head) * p.clusters + cl) * (p.max_new * p.group) + row;
      *reinterpret_cast<float4*>(p.part + at * D + col) = sum;
      if (col == 0) p.stat[at] = st;
    }
  };
  for (int u = tid; u < units; u += S::kThreads) {
    const int row = u / (D / 4), col = u % (D / 4) * 4;
    join([&](int i) { return *reinterpret_cast<const float2*>(left + i * kLeft + kStat + 2 * row); },
         [&](int i) { return *reinterpret_cast<const float4*>(left + i * kLeft + row * S::kSumRow + col); }, S::kKg);
    if (ctas == 1) {
      emit(u);
    } else {  // (each sum's place of group 0 is read by this thread alone; its row's statistics go to places of their own)
      *reinterpret_cast<float4*>(left + row * S::kSumRow + col) = sum;
      if (col == 0) *reinterpret_cast<float2*>(left + row * S::kSumRow + D) = st;
    }
  }
  if (ctas == 1) return;
  cluster_arrive_release();
  cluster_wait_acquire();
  const uint32_t left_at = smem_addr(left);
  const int share = (units + ctas - 1) / ctas;
  for (int v = tid; v < share && rank * share + v < units; v += S::kThreads) {
    const int u = rank * share + v, row = u / (D / 4), col = u % (D / 4) * 4;
    const uint32_t at = left_at + row * S::kSumRow * 4;
    join([&](int i) { return ld_cluster_v2(cluster_map(at + D * 4, i)); },
         [&](int i) { return ld_cluster_v4(cluster_map(at + col * 4, i)); }, ctas);
    emit(u);
  }
  cluster_arrive_release();  // no CTA leaves while another reads its sums
  cluster_wait_acquire();
}

// Joins a row's clusters, in order.
template <int D>
__global__ void __launch_bounds__(D / 2) join8_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  const int b = blockIdx.z, i = blockIdx.y, hq = blockIdx.x;
  const Seq s = sequence(p, b);
  if (!s.ok || i >= s.n) return;
  const int head = hq / p.by_group, row = i * p.group + hq - head * p.group;
  const int step = p.max_new * p.group;
  const long long at = (static_cast<long long>(b) * p.kv_heads + head) * p.clusters * step + row;
  float top = kNone, l = 0.f, x = 0.f, y = 0.f;
#pragma unroll 8
  for (int z = 0; z < p.clusters; ++z) {
    const float2 st = p.stat[at + static_cast<long long>(z) * step];
    const float2 v = *reinterpret_cast<const float2*>(p.part + (at + static_cast<long long>(z) * step) * D + 2 * threadIdx.x);
    const float next = fmaxf(top, st.x), ref = next == kNone ? 0.f : next;
    const float old = exp2_fast(top - ref), w = exp2_fast(st.x - ref);
    top = next;
    l = fmaf(st.y, w, l * old);
    x = fmaf(v.x, w, x * old);
    y = fmaf(v.y, w, y * old);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint32_t*>(p.out + static_cast<long long>(s.first_row + i) * p.out_row +
                              static_cast<long long>(hq) * D)[threadIdx.x] = pack_bf16(x * inv, y * inv);
}

// CTAs of a cluster, and clusters, of one sequence and head.  Not by max_new: a
// row's sums are the same whatever rows are beside it.
struct Split {
  int ctas, clusters;
};
Split split_for(const w4g128_attend8_args& a) {
  long long span = a.max_len;
  if (a.window > 0) span = std::min<long long>(span, static_cast<long long>(a.window) + a.sinks + 2 * kTile);
  const long long pairs = static_cast<long long>(a.kv_heads) * a.count;
  const long long tiles = (span + kTile - 1) / kTile, groups = groups_of(a.head_dim);
  const long long target = a.count < 16 ? 304 : 608;
  long long want = std::max<long long>(1, target / pairs);
  want = std::min(want, (tiles + groups - 1) / groups);
  if (want <= kMostCluster) return {static_cast<int>(want), 1};
  return {8, static_cast<int>(want / 8)};
}

int check(const w4g128_attend8_args* a) {
  if (a == nullptr || a->q == nullptr || a->k_cache == nullptr || a->v_cache == nullptr || a->k_scale == nullptr ||
      a->v_scale == nullptr || a->page_table == nullptr || a->row_offsets == nullptr || a->lens == nullptr ||
      a->out == nullptr)
    return W4G128_ERR_INVALID_ARG;
  if (a->rows < 1 || a->rows > (1 << 20) || a->count < 1 || a->count > W4G128_MAX_SEQUENCES || a->max_new < 1 ||
      a->max_new > W4G128_MAX_M || a->window < 0 || a->sinks < 0 || (a->sinks > 0 && a->window == 0) ||
      !(std::fabs(a->scale) <= 16384.f))
    return W4G128_ERR_INVALID_ARG;
  if (a->kv_heads < 1 || a->kv_heads > 256 || a->q_heads < a->kv_heads || a->q_heads % a->kv_heads != 0 ||
      a->q_heads / a->kv_heads > 16 || (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256))
    return W4G128_ERR_SHAPE;
  if (a->pages < 1 || a->page_size < 16 || a->page_size % 16 != 0 || a->max_len < 1 || a->max_len > (1 << 24) ||
      a->block < 1 || a->block > 64 || (a->block & (a->block - 1)) != 0 || a->page_size % a->block != 0)
    return W4G128_ERR_SHAPE;
  const long long dim = a->head_dim;
  if (a->q_row < a->q_heads * dim || a->out_row < a->q_heads * dim || a->slot_stride < dim || a->page_stride < dim ||
      a->head_stride < dim || a->scale_page < a->page_size / a->block || a->scale_head < a->page_size / a->block ||
      a->table_row < (a->max_len - 1) / a->page_size + 1)
    return W4G128_ERR_SHAPE;
  auto off = [](const void* q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0; };
  if (off(a->q, 16) || off(a->k_cache, 16) || off(a->v_cache, 16) || off(a->out, 16) || off(a->k_scale, 4) ||
      off(a->v_scale, 4) || off(a->page_table, 4) || off(a->row_offsets, 4) || off(a->lens, 4))
    return W4G128_ERR_ALIGN;
  if (a->q_row % 8 != 0 || a->out_row % 8 != 0) return W4G128_ERR_ALIGN;
  for (long long v : {a->page_stride, a->slot_stride, a->head_stride})
    if (v % 16 != 0) return W4G128_ERR_ALIGN;
  return W4G128_OK;
}

size_t bytes_for(const w4g128_attend8_args& a) {
  const Split split = split_for(a);
  if (split.clusters == 1) return kStatusBytes;
  return kStatusBytes + static_cast<size_t>(a.count) * split.clusters * a.q_heads * a.max_new * (a.head_dim + 2) * 4;
}

template <int D, int RT>
cudaError_t launch(cudaLaunchConfig_t& cfg, Params& p, int ctas) {
  using S = Shape<D, RT>;
  cudaError_t e = cudaFuncSetAttribute(attend8_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(attend8_kernel<D, RT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  p.row_groups = (p.max_new * p.group + S::kRows - 1) / S::kRows;
  p.by_row_groups = divisor(p.row_groups);
  const long long clusters = 1 + static_cast<long long>(p.count) * p.kv_heads * p.row_groups * p.clusters;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ctas));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  return cudaLaunchKernelEx(&cfg, attend8_kernel<D, RT>, p);
}

template <int D>
cudaError_t launch_dim(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, Params& p, int ctas) {
  cfg.attrs = attr;
  cfg.numAttrs = 2;  // with the cluster
  const int rows = p.max_new * p.group;
  const cudaError_t e = rows <= 16 ? launch<D, 1>(cfg, p, ctas) : rows <= 32 ? launch<D, 2>(cfg, p, ctas)
                                                                             : launch<D, 4>(cfg, p, ctas);
  if (e != cudaSuccess || p.clusters == 1) return e;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.q_heads, p.max_new, p.count);
  cfg.blockDim = dim3(D / 2);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join8_kernel<D>, p);
}

}  // namespace
}  // namespace w4g128

extern "C" {

size_t w4g128_attend8_workspace_bytes(const w4g128_attend8_args* args) {
  return w4g128::check(args) == W4G128_OK ? w4g128::bytes_for(*args) : 0;
}

int w4g128_attend8(const w4g128_attend8_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace w4g128;
  int rc = check(a);
  if (rc != W4G128_OK) return rc;
  if (ws == nullptr) return W4G128_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0) return W4G128_ERR_ALIGN;
  if (ws_bytes < bytes_for(*a)) return W4G128_ERR_WORKSPACE;
  rc = fault_hook();
  if (rc != W4G128_OK) return rc;
  if (!device_is_sm103()) return W4G128_ERR_DEVICE;
  const Split split = split_for(*a);
  Params p;
  p.q = a->q;
  p.k_cache = static_cast<const uint8_t*>(a->k_cache); p.v_cache = static_cast<const uint8_t*>(a->v_cache);
  p.k_scale = a->k_scale; p.v_scale = a->v_scale;
  p.table = a->page_table; p.offsets = a->row_offsets; p.lens = a->lens; p.out = a->out;
  p.q_row = a->q_row; p.out_row = a->out_row;
  p.page_stride = a->page_stride; p.slot_stride = a->slot_stride; p.head_stride = a->head_stride;
  p.scale_page = a->scale_page; p.scale_head = a->scale_head; p.table_row = a->table_row;
  p.rows = a->rows; p.count = a->count; p.q_heads = a->q_heads; p.kv_heads = a->kv_heads;
  p.group = a->q_heads / a->kv_heads;
  p.pages = a->pages; p.max_len = a->max_len; p.max_new = a->max_new;
  p.block_log2 = -1;
  for (int v = a->block; v > 0; v >>= 1) ++p.block_log2;
  p.window = a->window; p.sinks = a->sinks;
  p.clusters = split.clusters;
  p.by_clusters = divisor(split.clusters);
  p.by_kv_heads = divisor(a->kv_heads);
  p.by_group = divisor(p.group);
  p.by_page = divisor(a->page_size);
  p.scale2 = a->scale == 0.f ? 1.f : std::fabs(a->scale) * kLog2e;
  p.flip_q = a->scale < 0.f ? 0x80008000u : 0u;
  p.keep_q = a->scale == 0.f ? 0u : 0xFFFFFFFFu;
  auto* base = static_cast<uint8_t*>(ws);
  p.status = reinterpret_cast<unsigned long long*>(base);
  p.part = reinterpret_cast<float*>(base + kStatusBytes);
  p.stat = reinterpret_cast<float2*>(p.part + static_cast<size_t>(p.count) * p.clusters * p.q_heads * p.max_new * a->head_dim);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split.ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->head_dim == 64 ? launch_dim<64>(cfg, attr, p, split.ctas)
                        : a->head_dim == 128 ? launch_dim<128>(cfg, attr, p, split.ctas)
                                             : launch_dim<256>(cfg, attr, p, split.ctas);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
