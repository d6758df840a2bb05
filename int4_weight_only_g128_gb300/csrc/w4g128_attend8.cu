// Attention of 1..16 new tokens per sequence over a paged cache of e4m3 codes
// with a scale for each block of positions and head (w4g128_attend8).
//
// As in w4g128_attend, rows of one key/value head (new tokens x query heads that
// share it) are the 16-row tiles of a warp MMA and the work is the cache's bytes:
// half as many, so that what is left is latency and the conversion of the codes.
//   * Every code is an fp16 value, so both products are fp16 x fp16 -> fp32, and the
//     codes are converted on their way into them.  q, bf16, becomes fp16 scaled by a
//     power of two for each row (exact down to 2^-31 of the row's largest value).
//     (The warp MMA of e4m3 operands is made of conversions and fp16 products here:
//     with q as the sum of two e4m3 values it took 936 instructions a tile, and 33
//     us where fp16 products took 25.6.)
//   * A key's scale multiplies its score.  A value's scale enters the softmax
//     weight: with score s_j (base 2) and value scale v_j, P_j = 2^(s_j + log2 v_j - m),
//     rounded to fp16 as an operand, and the row's sum takes P_j / v_j.  The
//     reference m follows the maximum of s_j + log2 v_j, so P_j stays in fp16's range
//     whatever the scales are, and depends on the row alone.  Where m rises by a value
//     scale, the sum of P_j / v_j so far is large and its factor may be below fp32's
//     range: it is applied as its root, twice.
//   * Codes are read by ldmatrix as pairs: K's depth and V's columns then come in
//     another order than the MMA's, the same for q (laid out so) and for the result.
//   * The 16-position tiles of a sequence go in turn to all the groups of warps that
//     work on it, whatever its length, so all of them have the same share and no CTA
//     depends on how long a sequence may become.  A group keeps a ring of cp.async
//     stages and a running reference and sums of its own.
//   * Few CTAs of a head are a cluster, which joins their sums through its shared
//     memory; otherwise a second kernel joins them.
//
// What bounds it: one sequence of 32771 with 8 rows, 32 heads on 8 of 128 and pages of
// 64, takes 24.9 us, 2.7 TB/s.  Its bytes alone take 9.9 us, its fp16 products 7.2.  With
// each group's first tile alone the call takes 10.3 us: 3.3 until the first lengths and
// ids are there, 2.2 in joining a CTA's groups and writing their sums, 2.1 in the second
// kernel.  The loop's other 14 us are neither the copies nor the products alone (without
// copies 1.3 us less, without the products 6 less), but both, the conversions and the
// softmax at the 8 warps an SM whose sums the registers hold.
// 16 ragged sequences of up to 9001 on 4 heads of 64 take 18.9 us, two with a window of
// 4096 and 16 rows each on 4 heads of 256 20.5, one of 611 with one row 4.8.  The framework's
// attention over bf16 takes 29.7, 18.2, 22.7 and 6.0 on these shapes: ragged lengths with a
// scale for each slot gain nothing by half the bytes.
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
constexpr float kLowWeight = 0x1p-120f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMostCluster = 16;
constexpr int kMostChunk = 64;  // tiles
constexpr int kMostCtas = 16384;  // whole chunks of a call, and so many partial results
constexpr int kChunkedFrom = 4;  // sequences
constexpr int kMostCheckers = 16;

struct Params {
  const uint16_t* q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *table, *offsets, *lens;
  uint16_t* out;
  long long q_row, out_row, page_stride, slot_stride, head_stride, scale_page, scale_head, table_row;
  int rows, count, q_heads, kv_heads, group, pages, block_log2, max_len, max_new, window, sinks;
  int clusters, row_groups;  // of a sequence and head
  int checkers;              // CTAs that look for errors; several leave their results to the second kernel
  int chunk;                 // tiles of one CTA, where a sequence is cut into chunks; or 0
  Divisor by_group, by_page, by_clusters, by_row_groups, by_kv_heads;
  float scale2;              // |scale| log2(e); scale < 0: q's signs are flipped, scale = 0: q counts as 0
  uint32_t flip_q, keep_q;
  unsigned long long* status;
  float* part;               // [count][kv_heads][clusters][max_new * group][head_dim]: unnormalised sums
  float2* stat;              // [count][kv_heads][clusters][max_new * group]: half the reference, and the sum
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

// The first CTAs (one, but for many pages) look all lengths, row ranges and visible page ids over, beside the others.
__device__ void check_all(const Params& p, int which) {
  const int lane = threadIdx.x & 31, warps = (blockDim.x >> 5) * p.checkers;
  const int warp = which * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int parts = max(1, warps / p.count);  // warps that share a sequence
  constexpr int kBatch = 8;
  bool bad = false;
  for (int b = warp / parts; b < p.count; b += warps / parts) {
    const Seq s = sequence(p, b);
    bad |= !s.ok;
    if (!s.ok || s.n == 0) continue;
    const int sink_pages = (s.sink + static_cast<int>(p.by_page.d) - 1) / p.by_page;
    const int end = s.len > 0 ? (s.len - 1) / p.by_page + 1 : 0;
    const int low = max(s.lo / p.by_page, sink_pages), all = sink_pages + end - low;
    const int* table = p.table + static_cast<long long>(b) * p.table_row;
    for (int i = (warp % parts) * 32 + lane; i < all; i += kBatch * parts * 32) {  // (many on their way at once)
      int id[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int at = i + j * parts * 32;
        id[j] = at < all ? table[at < sink_pages ? at : low + at - sink_pages] : 0;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) bad |= id[j] < 0 || id[j] >= p.pages;
    }
  }
  if (__syncthreads_or(bad)) bad = true;
  if (threadIdx.x == 0) st_relaxed_u64(p.status + (p.checkers == 1 ? 0 : 1 + which), bad ? W4G128_ERR_CACHE : W4G128_OK);
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
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ float inverse_fast(float x) {  // 1 ulp; above 2^126 too, where the inverse itself would flush
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(0.25f * x));
  return 0.25f * y;
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
__device__ __forceinline__ void st_cluster_v2(uint32_t a, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// A sum of weights holds P / v: from 2^-122, the reference's own weight over the largest scale, to
// 2^118, 2^24 weights over the smallest.  So where the factor 2^x that brings it to another
// reference flushes to 0, their product need not: the sum takes the factor's root twice, and is
// there for x down to -252, below which it is 2^-134 at most.  Parts hand on half their references.
//
// Sums over parts with (half) references and sums of weights of their own; top: the largest reference.
struct Joined {
  float top, ref, l = 0.f;
  float4 sum = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ explicit Joined(float t) : top(t), ref(t == kNone ? 0.f : t) {}
  __device__ __forceinline__ void add(const float2& st, const float4& v) {
    const float root = exp2_fast(st.x - ref), w = root * root;
    l = fmaf(st.y * root, root, l);
    sum.x = fmaf(v.x, w, sum.x);
    sum.y = fmaf(v.y, w, sum.y);
    sum.z = fmaf(v.z, w, sum.z);
    sum.w = fmaf(v.w, w, sum.w);
  }
  __device__ __forceinline__ float2 stat() const { return make_float2(top, l); }
};

// KG groups of warps with tiles of their own; RT row tiles, MT of them a warp: two, which
// share K's and V's fragments and their conversion, where a thread's sums leave room.
constexpr int groups_of(int head_dim) { return head_dim == 256 ? 2 : 4; }
template <int D, int RT>
struct Shape {
  static constexpr int kKg = groups_of(D);
  static constexpr int kMt = D == 256 || RT == 1 ? 1 : 2;
  // Warps that share a row tile's columns, each with all its scores: two for the widest heads'
  // few rows, which have few warps otherwise (3 of 4100 with 4 rows on 4 heads: 17.5 us -> 14.6; 32 rows
  // have 8 warps an SM either way: a batch of 16 took 20.3 us with one, 31.4 with two).
  static constexpr int kCols = D == 256 && RT == 1 ? 2 : 1;
  static constexpr int kGroup = RT / kMt * kCols * 32;  // threads of a group
  static constexpr int kThreads = kKg * kGroup;
  // warps an SM, by the registers of a thread's sums: 128 of them leave room for 8, 64 for 12, 32 for 16
  // (16 with 64 spill: 16 ragged sequences on heads of 64 23.3 us, 19.0 with 12)
  static constexpr int kSums = kMt * D / kCols / 2;
  static constexpr int kWarps = kSums == 128 ? 8 : kSums == 64 ? 12 : 16;
  static constexpr int kCtas = kWarps * 32 / kThreads > 0 ? kWarps * 32 / kThreads : 1;
  static constexpr int kRows = RT * 16;
  static constexpr int kTileBytes = kTile * D;  // K or V of one tile
  static constexpr int kStageBytes = 2 * kTileBytes + 2 * kTile * 4;  // K, V and their positions' scales
  static constexpr int kQBytes = kRows * 2 * D;
  static constexpr int kRoom = (227 * 1024 / kCtas - 1536 - kQBytes) / kKg / kStageBytes;
  // (3: more only take room from the L1 cache; one of 32771 25.1 us, with 6 25.4; 16 of 3000 25.2, 26.5)
  static constexpr int kStages = kRoom < 3 ? kRoom : 3;
  static constexpr int kRing = kKg * kStages * kStageBytes;
  static constexpr int kSumRow = D + 16;     // floats of a row's sums (free of bank conflicts)
  static constexpr int kLeft = kRows * (kSumRow + 2) * 4;  // a group's sums, references and sums of weights
  static constexpr int kBytes = kQBytes + kRing > kKg * kLeft ? kQBytes + kRing : kKg * kLeft;
  // what a cluster's CTAs send to one another
  static constexpr int received(int ctas) { return (kRows + ctas - 1) / ctas * ctas * (D + 2) * 4; }
  static constexpr int kMostBytes = kBytes + (kRows + kMostCluster - 1) * (D + 2) * 4;
  static_assert(kMostBytes + 512 <= 227 * 1024, "room for what a cluster's CTAs send");
  static_assert(kStages >= 2, "a stage on its way while another is read");
};

template <int D, int RT, bool ONE>  // ONE: a scale for each tile at most (blocks of 16 and more)
__global__ void __launch_bounds__(Shape<D, RT>::kThreads, Shape<D, RT>::kCtas)
attend8_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, RT>;
  constexpr int MT = S::kMt, kCols = S::kCols;
  constexpr int kSteps = D / 16;   // of Q K^T
  constexpr int kPieces = D / 16;  // 16-byte pieces of a row of codes
  constexpr int kPer = 2 * kTile * kPieces / S::kGroup;  // pieces of a tile's K and V that one thread copies
  constexpr int kStep = S::kGroup / kPieces;             // rows between them
  constexpr int kScales = 2 * S::kTileBytes;             // a stage's scales
  static_assert(S::kGroup % kPieces == 0 && 2 * kTile % kStep == 0, "a thread copies one column of pieces");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_factor[S::kRows];  // a row's score factor

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);
  const int kg = warp * 32 / S::kGroup, in_group = warp - kg * (S::kGroup / 32);
  const int rw = in_group / kCols, part = in_group % kCols;  // this warp's rows: rw MT 16 .., and its part of the columns
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_nctarank());
  const int cluster = static_cast<int>(blockIdx.x) / ctas;

  if (ctas > 1) cluster_arrive_relaxed();  // a CTA runs before another sends it sums
  grid_dependency_wait();
  if (cluster < p.checkers) {
    if (rank == 0) check_all(p, cluster);
    if (ctas > 1) cluster_wait_acquire();
    return;
  }
  // work = ((b kv_heads + head) row_groups + rg) clusters + cl
  const int work = cluster - p.checkers, rest = work / p.by_clusters;
  const int cl = work - rest * p.clusters;
  const int up = rest / p.by_row_groups;
  const int rg = rest - up * p.row_groups;
  const int b = up / p.by_kv_heads;
  const int head = up - b * p.kv_heads;

  // All groups of this head and sequence take tiles in turn, or those of a CTA the tiles of a chunk.
  const int groups = p.chunk > 0 ? S::kKg : p.clusters * ctas * S::kKg;
  const int mine = p.chunk > 0 ? cl * p.chunk + kg : (cl * ctas + rank) * S::kKg + kg;
  const int* table = p.table + static_cast<long long>(b) * p.table_row;
  // Without a window the first tiles are known before the length is: their page
  // ids come along with it, a tile a lane.
  int ids = -1, ids_next = -1;
  if (p.window == 0) {
    const int a = (mine + lane * groups) * kTile;
    if (a < p.max_len) ids = table[a / p.by_page];
  }
  const Seq s = sequence(p, b);
  const int live_rows = s.n * p.group;
  if (!s.ok || rg * S::kRows >= live_rows || (p.chunk > 0 && cl > 0 && cl * p.chunk * kTile >= s.len)) {
    if (ctas > 1) cluster_wait_acquire();
    return;
  }

  // Q, asked for before the table is waited for.
  const int r = lane >> 2, c = lane & 3;
  const int row_w = rg * S::kRows + rw * MT * 16;  // the warp's first row
  const bool busy = row_w < live_rows;             // (of the warp)
  int pos_a[MT], pos_b[MT];                        // the positions of rows r and r + 8
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = row_w + m * 16 + r;
    pos_a[m] = row < live_rows ? s.start + row / p.by_group : -1;
    pos_b[m] = row + 8 < live_rows ? s.start + (row + 8) / p.by_group : -1;
  }
  constexpr int kQPer = S::kRows * (D / 8) / S::kThreads;  // pieces of 8 values of a thread
  static_assert(S::kRows * (D / 8) % S::kThreads == 0, "each thread loads as many pieces of Q");
  uint4 q_part[kQPer] = {};
#pragma unroll
  for (int e = 0; e < kQPer; ++e) {
    const int i = tid + e * S::kThreads, row = rg * S::kRows + i / (D / 8);
    if (row < live_rows) {
      const int at = row / p.by_group;
      q_part[e] = __ldg(reinterpret_cast<const uint4*>(p.q + static_cast<long long>(s.first_row + at) * p.q_row +
                                                       static_cast<long long>(head * p.group + row - at * p.group) * D) +
                        i % (D / 8));
    }
  }

  // This group's tiles: every groups-th, of the sinks' and then of the others.
  const int sink_tiles = (s.sink + kTile - 1) / kTile;
  int end_tile = (s.len + kTile - 1) / kTile;
  if (p.chunk > 0) end_tile = min(end_tile, (cl + 1) * p.chunk);
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
  // Of 32 tiles, one a lane: where its codes and scales are, -1 where that is no page.
  long long codes_at, scales_at;
  auto locate = [&](int k) {
    const int a = tile_of(k) * kTile, slot = a - a / p.by_page * static_cast<int>(p.by_page.d);
    const bool ok = k < total && ids >= 0 && ids < p.pages;
    codes_at = ok ? ids * p.page_stride + slot * p.slot_stride : -1;
    scales_at = ids * p.scale_page + (slot >> p.block_log2);
  };
  locate(lane);

  uint8_t* ring = smem + S::kQBytes + kg * S::kStages * S::kStageBytes;
  const uint32_t ring_at = smem_addr(ring);
  auto group_sync = [&] {
    if constexpr (S::kGroup == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(kg + 1), "n"(S::kGroup) : "memory");
  };
  auto swizzled = [](int j, int piece) { return j * D + ((piece ^ (D == 64 ? (j >> 1) & 3 : j & 7)) << 4); };

  // A thread copies one column of pieces: rows j0, j0 + kStep, .. of K, then of V.
  const int gl = in_group * 32 + lane;
  const int ch = gl % kPieces, j0 = gl / kPieces;
  const uint8_t* k_base = p.k_cache + head * p.head_stride + ch * 16;
  const long long v_off = p.v_cache - p.k_cache;
  // (a tile begins a block or lies in one: its position j is in the block j / block after its first)
  const float* scale_base = ((gl & 16) ? p.v_scale : p.k_scale) + head * p.scale_head + ((gl & 15) >> p.block_log2);
  const long long row_step = kStep * p.slot_stride;
  const long long first_row = j0 % kTile * p.slot_stride + (j0 >= kTile ? v_off : 0);
  uint32_t okays = 0u;  // of the tiles on their way, by their number mod 32: on a page
  auto issue = [&](int turn, int stage) {
    if (turn < total) {
      if (turn > 0 && (turn & 31) == 0) {
        ids = ids_next;
        ids_next = ids_from(turn + 32 + lane);
        locate(turn + lane);
      }
      const int a = tile_of(turn) * kTile;
      const long long codes = __shfl_sync(~0u, codes_at, turn & 31), scales = __shfl_sync(~0u, scales_at, turn & 31);
      const bool ok = codes >= 0;
      okays = (okays & ~(1u << (turn & 31))) | (ok ? 1u : 0u) << (turn & 31);
      const uint32_t dst = ring_at + stage * S::kStageBytes;
      const uint32_t scale_dst = dst + kScales + gl * 4;
      const uint8_t* src = k_base + (ok ? codes : 0);
      if (ok && a + kTile <= s.len) {  // a whole tile
        src += first_row;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int jj = j0 + e * kStep;
          if (e * kStep == kTile) src += v_off - kTile * p.slot_stride;
          cp_async16(dst + (jj >= kTile ? S::kTileBytes : 0) + swizzled(jj % kTile, ch), src);
          src += row_step;
        }
        if (gl < 32) cp_async4(scale_dst, scale_base + scales);
      } else {  // zeros behind the end, and for what is no page
#pragma unroll 1
        for (int e = 0; e < kPer; ++e) {
          const int jj = j0 + e * kStep, j = jj % kTile;
          const bool is_v = jj >= kTile, real = ok && a + j < s.len;
          cp_async16_or_zero(dst + (is_v ? S::kTileBytes : 0) + swizzled(j, ch),
                             real ? src + (is_v ? v_off : 0) + j * p.slot_stride : p.k_cache, real);
        }
        if (gl < 32) {
          const int j = gl & 15;
          const bool real = ok && a + j < s.len;
          cp_async4_or_zero(scale_dst, real ? scale_base + scales : p.k_scale, real);
        }
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
  auto power = [](int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); };
#pragma unroll
  for (int e = 0; e < kQPer; ++e) {
    const int i = tid + e * S::kThreads, j = i / (D / 8), piece = i % (D / 8);
    const uint32_t w[4] = {signed_q(q_part[e].x), signed_q(q_part[e].y), signed_q(q_part[e].z), signed_q(q_part[e].w)};
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = largest(w[u], top);
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const int shift = min(max(14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), -112), 110);
    const float by = power(shift);
    uint32_t half[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) half[u] = pack_half(low_f(w[u]) * by, high_f(w[u]) * by);
    if (piece == 0) s_factor[j] = p.scale2 * power(-shift);
    // The 16 depths of a step in the order in which K's codes come: 0 1 4 5 8 9 12 13, then the others.
    uint8_t* to = smem + j * 2 * D + (piece & 1) * 8;
    *reinterpret_cast<uint2*>(to + (((piece & ~1) ^ (j & 7)) << 4)) = make_uint2(half[0], half[2]);
    *reinterpret_cast<uint2*>(to + (((piece | 1) ^ (j & 7)) << 4)) = make_uint2(half[1], half[3]);
  }
  __syncthreads();

  float factor[MT][2];
  float acc[MT][D / 8 / kCols][4];  // [2 i]: columns 16 i + 4 c, + 2 of rows r and r + 8; [2 i + 1]: + 1, + 3
  float ref[MT][2], l[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      factor[m][side] = s_factor[(rw * MT + m) * 16 + r + 8 * side];
      ref[m][side] = kNone;
      l[m][side] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8 / kCols; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
  }

  // ldmatrix: this lane's row and its pieces 2 i + lane / 16, in a tile of K or V and
  // in a row tile of Q (the pieces from 8 on 128 bytes further).
  const int lj = lane & 15, lp = lane >> 4;
  constexpr int kAt = kPieces / 2 < 4 ? kPieces / 2 : 4;
  uint32_t at[kAt];
#pragma unroll
  for (int i = 0; i < kAt; ++i) at[i] = swizzled(lj, 2 * i + lp);
  auto piece_at = [&](int i) { return at[i % kAt] + i / kAt * 128; };
  constexpr int kColPieces = D / 32 / kCols, kColAt = kColPieces < 4 ? kColPieces : 4;  // (pairs of pieces of this warp's columns)
  uint32_t col_at[kColAt];
#pragma unroll
  for (int i = 0; i < kColAt; ++i) col_at[i] = kCols == 1 ? at[i] : swizzled(lj, 2 * (i + part * kColPieces) + lp);
  uint32_t q_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q_at[i] = smem_addr(smem) + (rw * MT * 16 + lj) * 2 * D + (((2 * i + lp) ^ (lj & 7)) << 4);
  const int last_pos = s.len - 1;  // of the sequence's last row
  float log_top = kNone;  // of the tiles so far, the largest value scale (base 2)
  int stage = 0;
#pragma unroll 1
  for (int turn = 0; turn < total; ++turn) {
    cp_async_wait_group<S::kStages - 2>();
    group_sync();  // the tile is there for the group, and the stage refilled next is read out
    issue(turn + S::kStages - 1, stage == 0 ? S::kStages - 1 : stage - 1);
    const uint32_t tile = ring_at + stage * S::kStageBytes;
    const uint8_t* tile_ptr = ring + stage * S::kStageBytes;
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
    if (!busy) continue;

    float sc[MT][2][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) sc[m][h][0] = sc[m][h][1] = sc[m][h][2] = sc[m][h][3] = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps / 2; ++i) {  // 32 depths of positions 0-7 and 8-15
      uint32_t kb[4];
      ldmatrix4(kb, tile + piece_at(i));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t qk[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) ldmatrix4(qk[m], q_at[(2 * i + u) & 3] + m * 32 * D + (2 * i + u) / 4 * 128);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t k0 = low_codes(kb[2 * u + h]), k1 = high_codes(kb[2 * u + h]);
#pragma unroll
          for (int m = 0; m < MT; ++m) mma(sc[m][h], qk[m], k0, k1);
        }
      }
    }

    // Scores in base 2, each with its value's scale; what a row does not see is none.
    constexpr int kOwn = ONE ? 1 : 4;  // scales of this lane's positions 2 c, 2 c + 1, + 8
    float log_v[kOwn], inverse[kOwn], ks[kOwn];
    const float* scales = reinterpret_cast<const float*>(tile_ptr + kScales);
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      const int j = ONE ? 0 : (e >> 1) * 8 + 2 * c + (e & 1);
      ks[e] = scales[j];
      const float v = fmaxf(scales[kTile + j], kLowestScale);
      log_v[e] = log2_fast(v);
      inverse[e] = inverse_fast(v);
    }
    const int a = tile_of(turn) * kTile;
    const bool on_page = (okays >> (turn & 31)) & 1u;
    auto sees = [&](int row_pos, int pos) { return visible(p, row_pos, pos) && on_page; };
    // every row sees the whole tile
    const bool inside = s.start >= 0 && a + kTile - 1 <= s.first && on_page &&
                        (p.window == 0 || last_pos - a < p.window || a + kTile <= p.sinks);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float f[2][kOwn];
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        f[0][e] = factor[m][0] * ks[e];
        f[1][e] = factor[m][1] * ks[e];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = ONE ? 0 : h * 2 + (i & 1);
          sc[m][h][i] = fmaf(sc[m][h][i], f[i >> 1][e], log_v[e]);
        }
    }
    if (!inside) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!sees(i < 2 ? pos_a[m] : pos_b[m], a + h * 8 + 2 * c + (i & 1))) sc[m][h][i] = kNone;
    }

    // The references, and the weights.
    float top[MT][2];
    bool above = false;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        top[m][side] = fmaxf(fmaxf(sc[m][0][2 * side], sc[m][0][2 * side + 1]), fmaxf(sc[m][1][2 * side], sc[m][1][2 * side + 1]));
        above = above || top[m][side] - ref[m][side] > kSlack;  // (ref may be that of no score)
      }
    if (__any_sync(~0u, above)) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float gain[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          float x = top[m][side];
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
          const float was = ref[m][side], now = x - was > kSlack ? x : was;
          const float root = now == was ? 1.f : exp2_fast(0.5f * (was - now));
          gain[side] = root * root;
          ref[m][side] = now;
          l[m][side] *= root;
          l[m][side] *= root;
        }
#pragma unroll
        for (int i = 0; i < D / 8 / kCols; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][i][e] *= gain[e >> 1];
      }
    }
    // (the rounded score less the reference, which is a rounded score: the largest weight is 2^kLift, however large they are)
    auto exponent = [&](int m, int h, int i) {
      return sc[m][h][i] + (ref[m][i >> 1] == kNone ? 0.f : kLift - ref[m][i >> 1]);
    };
    uint32_t pf[MT][4];
    float least = INFINITY;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float wt[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wt[h][i] = exp2_fast(exponent(m, h, i));
          if constexpr (!ONE) least = fminf(least, wt[h][i]);
        }
        pf[m][2 * h] = pack_half(wt[h][0], wt[h][1]);
        pf[m][2 * h + 1] = pack_half(wt[h][2], wt[h][3]);
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int i = 2 * side;
        l[m][side] += ONE ? ((wt[0][i] + wt[0][i + 1]) + (wt[1][i] + wt[1][i + 1])) * inverse[0]
                          : (wt[0][i] * inverse[0] + wt[0][i + 1] * inverse[kOwn > 1 ? 1 : 0]) +
                                (wt[1][i] * inverse[kOwn > 1 ? 2 : 0] + wt[1][i + 1] * inverse[kOwn > 1 ? 3 : 0]);
      }
    }
    // Beside values of scales 2^60 times as large and more, P may be below fp32's
    // range and the weight not.  (Where it is below it without that, the weight is
    // below 2^-60 of the row's sum, whose bits it does not reach.)
    bool low;
    if constexpr (ONE) {
      log_top = fmaxf(log_top, log_v[0]);
      low = log_top - log_v[0] > 60.f;
    } else {
      low = least < kLowWeight;
      if (low && !inside) {  // most of it is masked
        low = false;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) low = low || (sc[m][h][i] > kNone && sc[m][h][i] - ref[m][i >> 1] < -100.f);
      }
    }
    if (low) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = ONE ? 0 : h * 2 + (i & 1);
            const float x = exponent(m, h, i), w = exp2_fast(x);
            if (w < kLowWeight) {  // (a sum of large scales' weights is small itself: 2^x would flush beside it)
              const float root = exp2_fast(0.5f * (x - log_v[e]));
              l[m][i >> 1] += root * root - w * inverse[e];
            }
          }
    }

    uint32_t nans = 0u;
#pragma unroll
    for (int i = 0; i < kColPieces; ++i) {  // 32 columns; NaN codes in a tile that not every row sees whole are left out
      uint32_t vb[4];
      ldmatrix4_trans(vb, tile + S::kTileBytes + col_at[i % kColAt] + i / kColAt * 128);
      if (!inside) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t bad = nan_codes(vb[e]);
          nans |= bad;
          vb[e] &= ~((bad >> 7) * 0xFFu);
        }
      }
      uint32_t even_v[4], odd_v[4];  // a column's two positions together
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t both = __byte_perm(vb[e], 0u, 0x3120);
        even_v[e] = low_codes(both);
        odd_v[e] = high_codes(both);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma(acc[m][4 * i], pf[m], even_v[0], even_v[1]);
        mma(acc[m][4 * i + 1], pf[m], odd_v[0], odd_v[1]);
        mma(acc[m][4 * i + 2], pf[m], even_v[2], even_v[3]);
        mma(acc[m][4 * i + 3], pf[m], odd_v[2], odd_v[3]);
      }
    }
    if (__any_sync(~0u, nans != 0u)) {  // a row that sees a NaN code has NaN in its column
      const uint8_t* v_tile = tile_ptr + S::kTileBytes;
      for (int j = 0; j < kTile; ++j) {
#pragma unroll
        for (int i = 0; i < D / 16 / kCols; ++i) {
          const uint32_t bad =
              nan_codes(*reinterpret_cast<const uint32_t*>(v_tile + swizzled(j, i + part * (D / 16 / kCols)) + 4 * c));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const bool va = sees(pos_a[m], a + j), vb = sees(pos_b[m], a + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((bad >> (8 * e + 7)) & 1u) {
                if (va) acc[m][2 * i + (e & 1)][e >> 1] = NAN;
                if (vb) acc[m][2 * i + (e & 1)][2 + (e >> 1)] = NAN;
              }
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      l[m][side] += __shfl_xor_sync(~0u, l[m][side], 1);
      l[m][side] += __shfl_xor_sync(~0u, l[m][side], 2);
    }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // q and the ring become the exchange

  // Join the CTA's groups, then the cluster's CTAs, each time in order.
  float* left = reinterpret_cast<float*>(smem);
  constexpr int kLeft = S::kLeft / 4, kStat = S::kRows * S::kSumRow;
  const int rows_here = min(S::kRows, live_rows - rg * S::kRows);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int row = (rw * MT + m) * 16 + r + 8 * side;
      if (row < rows_here) {
        float* to = left + kg * kLeft + row * S::kSumRow + part * (D / kCols) + 4 * c;
#pragma unroll
        for (int i = 0; i < D / 16 / kCols; ++i)
          *reinterpret_cast<float4*>(to + 16 * i) = make_float4(acc[m][2 * i][2 * side], acc[m][2 * i + 1][2 * side],
                                                                acc[m][2 * i][2 * side + 1], acc[m][2 * i + 1][2 * side + 1]);
        if (c == 0 && part == 0)
          *reinterpret_cast<float2*>(left + kg * kLeft + kStat + 2 * row) = make_float2(0.5f * ref[m][side], l[m][side]);
      }
    }
  __syncthreads();
  const int units = rows_here * (D / 4);  // of 4 columns
  auto emit = [&](int row, int col, const float4& sum, const float2& st) {  // (row: of this CTA's)
    row += rg * S::kRows;
    if (p.clusters == 1) {
      const float inv = st.y == 0.f ? 0.f : 1.f / st.y;  // no visible position: zeros
      const int i = row / p.by_group;
      uint16_t* o = p.out + static_cast<long long>(s.first_row + i) * p.out_row +
                    static_cast<long long>(head * p.group + row - i * p.group) * D + col;
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
    } else {
      const long long to =
          ((static_cast<long long>(b) * p.kv_heads + head) * p.clusters + cl) * (p.max_new * p.group) + row;
      *reinterpret_cast<float4*>(p.part + to * D + col) = sum;
      if (col == 0) p.stat[to] = st;
    }
  };
  // A cluster's row is joined by its CTA of rank row % ctas, in its place row / ctas.
  float* received = reinterpret_cast<float*>(smem + S::kBytes);
  float2* received_stat = reinterpret_cast<float2*>(received + (S::kRows + ctas - 1) / ctas * ctas * D);
  if (ctas > 1) cluster_wait_acquire();
  for (int u = tid; u < units; u += S::kThreads) {
    const int row = u / (D / 4), col = u % (D / 4) * 4;
    float2 stats[S::kKg];
    float4 sums[S::kKg];
    float top = kNone;
#pragma unroll
    for (int i = 0; i < S::kKg; ++i) {
      stats[i] = *reinterpret_cast<const float2*>(left + i * kLeft + kStat + 2 * row);
      sums[i] = *reinterpret_cast<const float4*>(left + i * kLeft + row * S::kSumRow + col);
      top = fmaxf(top, stats[i].x);
    }
    Joined joined(top);
#pragma unroll
    for (int i = 0; i < S::kKg; ++i) joined.add(stats[i], sums[i]);
    if (ctas == 1) {
      emit(row, col, joined.sum, joined.stat());
    } else {
      const int slot = row / ctas, owner = row - slot * ctas;
      const int place = slot * ctas + rank;
      st_cluster_v4(cluster_map(smem_addr(received + place * D + col), owner), joined.sum);
      if (col == 0) st_cluster_v2(cluster_map(smem_addr(received_stat + place), owner), joined.stat());
    }
  }
  if (ctas == 1) return;
  cluster_arrive_release();
  cluster_wait_acquire();
  for (int u = tid;; u += S::kThreads) {
    const int slot = u / (D / 4), col = u % (D / 4) * 4, row = slot * ctas + rank;
    if (row >= rows_here) break;
    const float2* stats = received_stat + slot * ctas;
    const float* sums = received + slot * ctas * D + col;
    float top = kNone;
#pragma unroll 4
    for (int i = 0; i < ctas; ++i) top = fmaxf(top, stats[i].x);
    Joined joined(top);
#pragma unroll 4
    for (int i = 0; i < ctas; ++i) joined.add(stats[i], *reinterpret_cast<const float4*>(sums + i * D));
    emit(row, col, joined.sum, joined.stat());
  }
}

// Joins a row's CTAs (or clusters): the warps take them in turn and are added in order.
template <int D, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) join8_kernel(const __grid_constant__ Params p) {
  constexpr int kPer = D / 32, kBatch = kWarps == 4 ? 5 : 3;
  __shared__ float s_sum[kWarps][D];
  __shared__ float2 s_stat[kWarps];
  grid_dependency_wait();
  const int b = blockIdx.z, i = blockIdx.y, hq = blockIdx.x;
  if (p.checkers > 1 && (b | i | hq) == 0 && threadIdx.x < 32) {
    const bool bad = static_cast<int>(threadIdx.x) < p.checkers && p.status[1 + threadIdx.x] != W4G128_OK;
    if (__any_sync(~0u, bad)) {
      if (threadIdx.x == 0) st_relaxed_u64(p.status, W4G128_ERR_CACHE);
    } else if (threadIdx.x == 0) {
      st_relaxed_u64(p.status, W4G128_OK);
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = hq / p.by_group, row = i * p.group + hq - head * p.group;
  const int step = p.max_new * p.group;
  const long long at = (static_cast<long long>(b) * p.kv_heads + head) * p.clusters * step + row;
  // (on their way before the sequence is known: what no CTA wrote is not looked at)
  float2 st[kBatch];
  float v[kBatch][kPer];
  auto load = [&](int z) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (z + kWarps * j < p.clusters) {
        const long long from = at + static_cast<long long>(z + kWarps * j) * step;
        st[j] = p.stat[from];
        const float* o = p.part + from * D + lane * kPer;
        if constexpr (kPer == 2) *reinterpret_cast<float2*>(v[j]) = *reinterpret_cast<const float2*>(o);
        else
#pragma unroll
          for (int k = 0; k < kPer; k += 4) *reinterpret_cast<float4*>(&v[j][k]) = *reinterpret_cast<const float4*>(o + k);
      }
    }
  };
  load(warp);
  const Seq s = sequence(p, b);
  if (!s.ok || i >= s.n) return;
  const int parts = p.chunk > 0 ? max(1, (s.len + p.chunk * kTile - 1) / (p.chunk * kTile)) : p.clusters;  // (chunks alive)
  float top = kNone, l = 0.f, sum[kPer] = {};
  for (int z = warp; z < parts; z += kWarps * kBatch) {
    if (z > warp) load(z);
    float next = top;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (z + kWarps * j < parts) next = fmaxf(next, st[j].x);
    const float ref = next == kNone ? 0.f : next, old_root = exp2_fast(top - ref), old = old_root * old_root;
    top = next;
    l = l * old_root * old_root;
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum[k] *= old;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (z + kWarps * j < parts) {
        const float root = exp2_fast(st[j].x - ref), w = root * root;
        l = fmaf(st[j].y * root, root, l);
#pragma unroll
        for (int k = 0; k < kPer; ++k) sum[k] = fmaf(v[j][k], w, sum[k]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) s_sum[warp][lane * kPer + k] = sum[k];
  if (lane == 0) s_stat[warp] = make_float2(top, l);
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  const int k = threadIdx.x;
  top = kNone;
#pragma unroll
  for (int j = 0; j < kWarps; ++j) top = fmaxf(top, s_stat[j].x);
  const float ref = top == kNone ? 0.f : top;
  float x = 0.f, y = 0.f;
  l = 0.f;
#pragma unroll
  for (int j = 0; j < kWarps; ++j) {
    const float root = exp2_fast(s_stat[j].x - ref), w = root * root;
    const float2 u = *reinterpret_cast<const float2*>(&s_sum[j][2 * k]);
    l = fmaf(s_stat[j].y * root, root, l);
    x = fmaf(u.x, w, x);
    y = fmaf(u.y, w, y);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint32_t*>(p.out + static_cast<long long>(s.first_row + i) * p.out_row + static_cast<long long>(hq) * D)[k] =
      pack_bf16(x * inv, y * inv);
}

// How a sequence and head is shared out.  Not by max_new: a row's sums are the same whatever
// rows are beside it.
//   * All CTAs of one sequence take its tiles in turn: as many as the GPU holds of those for
//     32 rows on heads of 64 and 128 (one of 32771 with 8 rows, 8 heads of 128: 24.9 us with
//     303, 29.8 with 220, 34.0 with 455), of those for 64 rows on heads of 256, here with 151
//     and with 303: 2 with a window of 4096 and 64 rows each on 4 heads 20.6 us and 30.3, one
//     of 32771 with 64 rows 44.9 and 51.4, with 4 rows 27.3 and 22.0, 3 of 4100 with 4 rows
//     each 14.6 and 12.9.
//   * Few CTAs are joined in a cluster (one of 611 on 8 heads: 4.9 us, and 5.7 with a second
//     kernel).
//   * From 4 sequences on, whose lengths are their own, a CTA takes a chunk of positions, so
//     that a sequence has CTAs by its length: chunks that cut max_len of all into two or
//     three CTAs for each that the GPU holds.  Heads of 64, 16 ragged on 4 heads: 19.0 us
//     with 1213, 24.6, 20.1 and 26.5 with 606, 909 and 1820.  Heads of 128, 16 ragged of up
//     to 6000 on 8 heads and 16 of 3000: 23.2 and 25.2 us with 909, 24.9 and 28.3 with 455,
//     24.9 and 28.6 with 606, 25.7 and 28.3 with 1213.  Heads of 256, 8 ragged of up to 9000
//     on 4 heads and 8 of 9000: 27.8 and 36.4 us with 455, 41.5 and 44.2 with 303, 26.4 and
//     45.1 with 606, 23.3 and 38.6 with 909.
//   * A chunk has an end, so that the last ones of long calls end together (64 ragged ones of
//     up to 9000 on 8 heads of 256: 130 us with 64 tiles at most, 151 with 128).
//   * But max_len may be far above the lengths: there are 16384 whole chunks at most, most of
//     them without a position.  With max_len 131072, with this limit, without one and with
//     8192: 64 of 4000 on 8 heads of 128 143 us, 190 and 130; 256 of up to 1000 on 8 of 64
//     51, 337 and 40; 64 of up to 9000 on 8 of 256 210, 229 and 308.
struct Split {
  int ctas, clusters, chunk;  // CTAs of a cluster; clusters of one sequence and head; tiles of a chunk, or 0
};
Split split_for(const w4g128_attend8_args& a) {
  long long span = a.max_len;
  if (a.window > 0) span = std::min<long long>(span, static_cast<long long>(a.window) + a.sinks + 2 * kTile);
  const long long pairs = static_cast<long long>(a.kv_heads) * a.count;
  const long long tiles = (span + kTile - 1) / kTile, groups = groups_of(a.head_dim);
  const long long target = a.head_dim == 64 ? 455 : a.head_dim == 128 ? 303 : 151;
  const long long most = std::max<long long>(1, target / pairs), whole = (tiles + groups - 1) / groups;
  const long long want = std::min(most, whole);
  const bool chunks = a.count >= kChunkedFrom && a.window == 0 && whole > most;
  if (!chunks && want <= kMostCluster && want * pairs <= 128) return {static_cast<int>(want), 1, 0};
  if (chunks) {
    const long long some = a.head_dim == 64 ? 1213 : a.head_dim == 128 ? 909 : 455;
    auto of_ctas = [&](long long n) { return (tiles * pairs + n * groups - 1) / (n * groups) * groups; };
    const long long chunk = std::max(std::min<long long>(kMostChunk, of_ctas(some)), of_ctas(kMostCtas));
    return {1, static_cast<int>((tiles + chunk - 1) / chunk), static_cast<int>(chunk)};
  }
  return {1, static_cast<int>(want), 0};
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
  const auto kernel = p.block_log2 >= 4 ? attend8_kernel<D, RT, true> : attend8_kernel<D, RT, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kMostBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  p.row_groups = (p.max_new * p.group + S::kRows - 1) / S::kRows;
  p.by_row_groups = divisor(p.row_groups);
  const long long clusters = p.checkers + static_cast<long long>(p.count) * p.kv_heads * p.row_groups * p.clusters;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ctas));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kBytes + (ctas > 1 ? S::received(ctas) : 0);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D>
cudaError_t launch_dim(cudaLaunchConfig_t& cfg, Params& p, int ctas) {
  cfg.numAttrs = ctas > 1 ? 2 : 1;  // with the cluster
  const int rows = p.max_new * p.group;
  const cudaError_t e = rows <= 16 ? launch<D, 1>(cfg, p, ctas) : rows <= 32 ? launch<D, 2>(cfg, p, ctas)
                                                                             : launch<D, 4>(cfg, p, ctas);
  if (e != cudaSuccess || p.clusters == 1) return e;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.q_heads, p.max_new, p.count);
  cfg.dynamicSmemBytes = 0;
  // 4 warps for up to 20, which they ask for at once, otherwise 16 (16 ragged sequences in 12 chunks: 19.0 us, 20.1
  // with 8 and 22.8 with 16; one of 100003 on one head: 14.5 with 16, 17.1 with 8 and 20.6 with 4).
  const bool few = p.clusters <= 20;
  cfg.blockDim = dim3(few ? 128 : 512);
  return few ? cudaLaunchKernelEx(&cfg, join8_kernel<D, 4>, p) : cudaLaunchKernelEx(&cfg, join8_kernel<D, 16>, p);
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
  p.chunk = split.chunk;
  // One CTA looks the page ids over, beside the others, and more from 32768 on (256
  // sequences of 8000 on one head of 64, pages of 16: 60.6 us, and 146 with one; one of
  // 1000003 on one head of 64: 35.9 and 69.6).
  const long long ids = static_cast<long long>(a->count) * ((a->max_len - 1) / a->page_size + 1);
  p.checkers = split.clusters == 1 ? 1 : static_cast<int>(std::min<long long>(kMostCheckers, std::max<long long>(1, ids / 16384)));
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
  cfg.attrs = attr;
  const cudaError_t e = a->head_dim == 64 ? launch_dim<64>(cfg, p, split.ctas)
                        : a->head_dim == 128 ? launch_dim<128>(cfg, p, split.ctas) : launch_dim<256>(cfg, p, split.ctas);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
