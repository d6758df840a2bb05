// Attention of 1..16 new tokens per sequence over a paged cache
// (w4g128_attend): split over the positions, joined by a second kernel.
//
// Rows of one key/value head (new tokens x query heads that share it) are the
// 16-row tiles of a warp MMA (m16n8k16, bf16 -> fp32): with at most 256 rows
// against every position, the work is the cache's bytes, and the point is to
// read each byte once and keep enough of them in flight.
//   * A sequence is cut into chunks of C positions at multiples of C; one CTA
//     takes one (chunk, head, up to 64 rows).  C follows from the cache's and
//     the batch's shape alone, so a row's sums never depend on the rows beside it.
//   * The CTA's groups of warps take the chunk's 16-position tiles in turn,
//     each with its own ring of cp.async stages and its own running maximum
//     and sum: no barrier of the whole CTA until the end.  A group is RT warps,
//     one per 16 rows, sharing the group's tiles; with 256-wide heads two warps
//     share a row tile, each with half of the depth of Q K^T (the halves are
//     exchanged) and half of the columns of P V, so that a warp's registers
//     stay at 128 and an SM holds 16 warps.
//   * A tile lies in one page (page sizes are multiples of 16): one table
//     lookup per tile, made before the loop.
//   * S = Q K^T lands in the registers that P V wants it in; K comes by
//     ldmatrix, V by ldmatrix.trans, from rows whose 16-byte pieces are
//     exchanged by the low bits of the position, free of bank conflicts.
// Measured, one sequence of 32771, 8 heads of 128, 8 new tokens of 32 query
// heads (134 MB): 29.4 us a call, 67% of the measured copy rate; the tile loop
// streams at 6.7 TB/s, the rest is each CTA's start (length, table: 2.4 us), the
// join of its groups (1.5 us) and the second kernel (4 us).  With 64 rows the
// tile loop's latency binds: two of window 4096, 4 heads of 256, 16 new tokens
// take 22.6 us against 5.1 us of bytes and 1.1 us of operations at the measured
// bf16 rate; under ncu an active SM issues 1.5 instructions a clock, its tensor
// pipe is busy 22% and its shared memory 60% of the time.  Warp MMAs fed by
// ldmatrix go no faster; tcgen05 with the rows as one tile of 64 or 128 would,
// and is not built.  Not kept there: two row tiles a warp at 255 registers
// (8 long 34.9 us, 30.5 without), two position tiles a turn of the loop (22.8
// and 22.7: the same).
// Positions masked for some row hold arbitrary bits, and 0 x NaN is NaN: tiles
// at a mask's edge are searched for non-finite values, which are then applied
// to the rows that see them one by one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "w4g128_ops.h"
#include "w4g128_divide.cuh"
#include "w4g128_internal.h"
#include "w4g128_ptx.cuh"
#include "w4g128_status.cuh"

namespace w4g128 {
namespace {

constexpr int kTile = 16;        // positions per tile
constexpr int kMaxChunk = 2048;  // positions per chunk, at most
constexpr size_t kStatusBytes = 256;
constexpr float kNone = -INFINITY;
// A row's reference follows its maximum only when that is above it by more than
// this (base 2): weights up to 2^8 cost no precision, and most tiles neither
// exchange their maxima nor rescale the sums (per call, 16 new tokens of 64 heads
// on 8 at 32771, 128 rows a head: 98.6 -> 89.4 us; 16 ragged sequences 21.3 -> 19.3).
constexpr float kSlack = 8.f;
constexpr uint32_t kOnes = 0x3F803F80u;  // bf16 1.0 twice
constexpr float kLog2e = 1.44269504088896340736f;

struct Params {
  const uint16_t *q, *k_new, *v_new;
  uint16_t *k_cache, *v_cache;
  const int *table, *offsets, *lens;
  uint16_t* out;
  long long q_row, kv_row, out_row, page_stride, slot_stride, head_stride, table_row;
  int rows, count, q_heads, kv_heads, group, pages, page_size, max_len, max_new, window, sinks;
  int chunk, splits;  // positions per chunk; chunks a sequence may need
  Divisor by_chunk, by_group, by_page, by_row_groups;
  float scale2;       // |scale| log2(e); scale < 0: q's signs are flipped, scale = 0: q counts as 0
  uint32_t flip_q, keep_q;
  unsigned long long *status, *pending;
  float* part;        // [count][splits][kv_heads][max_new * group][head_dim]: unnormalised sums
  float2* stat;       // [count][splits][kv_heads][max_new * group]: maximum (base 2) and sum
};

// What the rows of one sequence see.
struct Seq {
  bool ok;
  int first_row, n, len, start;  // start: the first new row's position (negative rows are empty)
  int first;                     // the first real row's position
  int lo, sink;                  // visible to some row: [0, sink) and [lo, len)
  int sink_chunks, lo_chunk, chunks;
  __device__ int chunk_id(int z) const { return z < sink_chunks ? z : lo_chunk + z - sink_chunks; }
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
  s.lo_chunk = s.lo / p.by_chunk;
  s.sink_chunks = min((s.sink + p.chunk - 1) / p.by_chunk, s.lo_chunk);
  s.chunks = s.ok && s.n > 0 && s.len > 0 ? s.sink_chunks + (s.len - 1) / p.by_chunk - s.lo_chunk + 1 : 0;
  return s;
}

// The sequence's length and rows, and the pages that its rows see.
__device__ __forceinline__ bool in_range(const Params& p, int b) {
  const Seq s = sequence(p, b);
  bool ok = s.ok;
  if (ok && s.n > 0) {
    for (int a = 0; a < s.len; a += kTile) {
      const int id = p.table[static_cast<long long>(b) * p.table_row + a / p.by_page];
      ok = ok && ((a >= s.sink && a + kTile <= s.lo) || (id >= 0 && id < p.pages));
    }
  }
  return ok;
}

__device__ __forceinline__ bool visible(const Params& p, int row_pos, int pos) {
  return pos <= row_pos && (p.window == 0 || row_pos - pos < p.window || pos < p.sinks);
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes, or zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ bool non_finite2(uint32_t v) {  // either bf16 of the word
  return (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t finite_or_zero2(uint32_t v) {
  if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
  if ((v & 0x7F800000u) == 0x7F800000u) v &= 0x0000FFFFu;
  return v;
}

// KG groups of warps with tiles of their own, RT row tiles, DS warps per row tile.
template <int D, int RT>
struct Shape {
  static constexpr int kDs = D == 256 ? 2 : 1;
  static constexpr int kKg = D == 256 ? 2 : 4;
  static constexpr int kGroup = RT * kDs * 32;  // threads of a group
  static constexpr int kThreads = kKg * kGroup;
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kTileBytes = kTile * kRowBytes;  // K or V of one tile
  // stages: what 512 threads an SM (128 registers each) leave room for
  static constexpr int kStages = RT == 1 ? (D == 64 ? 3 : 2) : RT == 2 ? (D == 64 ? 4 : D == 128 ? 3 : 2)
                                                                       : (D == 64 ? 6 : D == 128 ? 5 : 4);
  static constexpr bool kQInRegs = D == 64;  // else its fragments are read from shared memory for each tile
  static constexpr int kQBytes = kQInRegs ? 0 : RT * 16 * kRowBytes;
  static constexpr int kRing = kKg * kStages * 2 * kTileBytes;
  static constexpr int kHalf = D / kDs;  // columns of a warp
  static constexpr int kLeft = 16 * (kHalf + 2) * 4;  // a warp's sums, maxima and sums of weights
  static constexpr int kJoin = (kKg - 1) * RT * kDs * kLeft;
  static constexpr int kBytes = kQBytes + (kRing > kJoin ? kRing : kJoin);
  static constexpr int kExchange = kDs == 2 ? kKg * RT * 2 * 32 : 1;  // float4: [group][row tile][half]..
};

template <int D, int RT>
__global__ void __launch_bounds__(Shape<D, RT>::kThreads, 512 / Shape<D, RT>::kThreads)
attend_kernel(const __grid_constant__ Params p) {
  using S = Shape<D, RT>;
  constexpr int kSteps = S::kHalf / 16;     // of Q K^T, per warp
  constexpr int kPieces = D / 8;            // 16-byte pieces of a row
  constexpr int kPer = kTile * kPieces / S::kGroup;  // pieces of a K tile that one thread copies
  constexpr int kRows = S::kGroup / kPieces;         // rows between them
  static_assert(S::kGroup % kPieces == 0 && kTile % kRows == 0, "a thread copies one column of pieces");
  static_assert(kMaxChunk / kTile <= S::kThreads, "one thread per tile of a chunk");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_tile[kMaxChunk / kTile];  // a tile's first element in the caches, or -1: not a page
  __shared__ float4 s_half[S::kExchange][2];

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);
  const int kg = warp / (RT * S::kDs), rt = warp / S::kDs % RT, half = warp % S::kDs;
  const int head = static_cast<int>(blockIdx.y) / p.by_row_groups;
  const int rg = static_cast<int>(blockIdx.y - head * p.by_row_groups.d);
  const int b = blockIdx.z, z = blockIdx.x;

  grid_dependency_wait();
  // (max_len is at most a chunk: this kernel is the call.  It reports errors itself: noted ones would stay in the
  // pending word, which only the second kernel empties, and reach the next call on the workspace that has one)
  const bool direct = p.splits == 1;
  if (direct && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    bool bad = false;
    for (int i = tid; i < p.count; i += S::kThreads) bad |= !in_range(p, i);
    if (__syncthreads_or(bad)) bad = true;
    if (tid == 0) st_relaxed_u64(p.status, bad ? W4G128_ERR_CACHE : W4G128_OK);
  }
  // Without a window this chunk's positions are known before the length is: its
  // page ids come along with it.
  const int ahead_pos = z * p.chunk + tid * kTile;
  int ahead_id = -1;
  if (p.window == 0 && tid < p.chunk / kTile && ahead_pos < p.max_len)
    ahead_id = p.table[static_cast<long long>(b) * p.table_row + ahead_pos / p.by_page];
  const Seq s = sequence(p, b);
  if (!s.ok) {
    if (!direct && z == 0 && blockIdx.y == 0 && tid == 0) note_error(p.pending, W4G128_ERR_CACHE);
    return;
  }
  const int live_rows = s.n * p.group;
  if (rg * 16 * RT >= live_rows) return;
  if (z >= s.chunks && !(direct && z == 0)) return;  // (direct: empty rows are written as zeros)

  const int p0 = s.chunks ? s.chunk_id(z) * p.chunk : 0;
  const int p1 = s.chunks ? min(p0 + p.chunk, s.len) : 0;
  const int fresh = p.k_new != nullptr ? s.first : s.len;  // positions from here on come from k_new, v_new

  // Q, asked for before the table is waited for: this lane's part of the A
  // fragments of rows r and r + 8, or this thread's pieces for shared memory.
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
  constexpr int kQPer = RT * 16 * kPieces / S::kThreads;
  static_assert(S::kQInRegs || RT * 16 * kPieces % S::kThreads == 0, "each thread loads as many pieces of Q");
  [[maybe_unused]] uint32_t qf[S::kQInRegs ? kSteps : 1][4] = {};
  [[maybe_unused]] uint4 q_part[S::kQInRegs ? 1 : kQPer] = {};
  if constexpr (S::kQInRegs) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      if (row0 + 8 * side < live_rows) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(q_row(row0 + 8 * side) + half * S::kHalf) + c;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          qf[k][side] = __ldg(from + k * 8);
          qf[k][side + 2] = __ldg(from + k * 8 + 4);
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kQPer; ++e) {
      const int i = tid + e * S::kThreads, row = rg * RT * 16 + i / kPieces;
      if (row < live_rows) q_part[e] = __ldg(reinterpret_cast<const uint4*>(q_row(row)) + i % kPieces);
    }
  }

  // where this chunk's tiles are
  const int tiles = (p1 - p0 + kTile - 1) / kTile;
  for (int t = tid; t < tiles; t += S::kThreads) {
    const int a = p0 + t * kTile;
    const bool seen = a < s.sink || (a + kTile > s.lo && a < s.len);
    const int page = a / p.by_page;
    const int id = !seen ? -1 : p.window == 0 ? ahead_id : p.table[static_cast<long long>(b) * p.table_row + page];
    const bool ok = id >= 0 && id < p.pages;
    if (seen && !ok && !direct) note_error(p.pending, W4G128_ERR_CACHE);
    s_tile[t] = ok ? id * p.page_stride + (a - page * p.page_size) * p.slot_stride + head * p.head_stride : -1;
  }

  __syncthreads();

  float acc[S::kHalf / 8][4];
#pragma unroll
  for (int i = 0; i < S::kHalf / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  // references (running maxima, up to the slack) of the raw scores of rows r and r + 8, and the sums of the
  // weights (sum[0] and sum[2]: a product with ones)
  float m_a = kNone, m_b = kNone, sum[4] = {};

  const uint32_t ring = smem_addr(smem) + S::kQBytes + kg * S::kStages * 2 * S::kTileBytes;
  auto group_sync = [&] {
    if constexpr (S::kGroup == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(kg + 1), "n"(S::kGroup) : "memory");
  };
  // The group's tiles that some row sees, in rising order.
  auto next_tile = [&](int t) {
    if (p.window > 0) {
      while (t < tiles) {
        const int a = p0 + t * kTile;
        if (a < s.sink || a + kTile > s.lo) break;
        t += S::kKg;
      }
    }
    return t;
  };

  // A thread copies one column of 16-byte pieces: rows j0, j0 + kRows, ..  The
  // pieces of a row are exchanged by the row's low bits.
  const int gl = (warp % (RT * S::kDs)) * 32 + lane;
  const int ch = gl % kPieces, j0 = gl / kPieces;
  const uint16_t* k_base = p.k_cache + j0 * p.slot_stride + ch * 8;
  const long long v_off = p.v_cache - p.k_cache;
  const long long row_step = kRows * p.slot_stride;
  uint32_t put[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    put[i] = ring + (j0 + i * kRows) * S::kRowBytes + ((ch ^ ((j0 + i * kRows) & 7)) << 4);
  auto issue = [&](int t, int stage) {
    if (t < tiles) {
      const int a = p0 + t * kTile;
      const long long where = s_tile[t];
      const uint32_t dst = stage * 2 * S::kTileBytes;
      if (a + kTile <= fresh && where >= 0) {  // a whole tile of the cache
        const uint16_t* src = k_base + where;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          cp_async16(put[i] + dst, src);
          cp_async16(put[i] + dst + S::kTileBytes, src + v_off);
          src += row_step;
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
          const int j = j0 + i * kRows, pos = a + j;
          const bool is_new = pos >= fresh;
          const bool real = pos < s.len && (is_new || where >= 0);
          const long long src = is_new ? static_cast<long long>(s.first_row + pos - s.start) * p.kv_row +
                                             static_cast<long long>(head) * D + ch * 8
                                       : where + j * p.slot_stride + ch * 8;
          const uint32_t at = ring + dst + j * S::kRowBytes + ((ch ^ (j & 7)) << 4);
          const uint16_t* kb = is_new ? p.k_new : p.k_cache;
          const uint16_t* vb = is_new ? p.v_new : p.v_cache;
          cp_async16_or_zero(at, real ? kb + src : p.k_cache, real);
          cp_async16_or_zero(at + S::kTileBytes, real ? vb + src : p.k_cache, real);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  int ahead = next_tile(kg);  // (chunks start at multiples of 64: a tile's group follows from its position)
  int t = ahead;
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) {
    issue(ahead, i);
    ahead = next_tile(ahead + S::kKg);
  }

  // (a negative scale goes into q's signs, a scale of 0 makes q 0)
  auto signed_q = [&](uint32_t v) { return (v & p.keep_q) ^ p.flip_q; };
  if constexpr (S::kQInRegs) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[k][i] = signed_q(qf[k][i]);
  } else {
#pragma unroll
    for (int e = 0; e < kQPer; ++e) {
      const int i = tid + e * S::kThreads, j = i / kPieces, piece = i % kPieces;
      const uint4 v = q_part[e];
      *reinterpret_cast<uint4*>(smem + j * S::kRowBytes + ((piece ^ (j & 7)) << 4)) =
          make_uint4(signed_q(v.x), signed_q(v.y), signed_q(v.z), signed_q(v.w));
    }
  }
  if constexpr (!S::kQInRegs) __syncthreads();

  // ldmatrix: this lane's row of a K and of a V tile, and its pieces 0, 2, 4, 6
  // (the others follow at constant distances).
  const int kj = (lane & 7) + ((lane >> 4) << 3), vj = (lane & 7) + (((lane >> 3) & 1) << 3);
  uint32_t k_at[4], v_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k_at[i] = kj * S::kRowBytes + half * 2 * S::kHalf + (((2 * i + ((lane >> 3) & 1)) ^ (kj & 7)) << 4);
    v_at[i] = vj * S::kRowBytes + half * 2 * S::kHalf + (((2 * i + (lane >> 4)) ^ (vj & 7)) << 4) + S::kTileBytes;
  }
  const uint32_t q_tile = smem_addr(smem) + rt * 16 * S::kRowBytes - S::kTileBytes;
  const int last_pos = s.len - 1;  // of the sequence's last row
  int stage = 0;
  while (t < tiles) {
    cp_async_wait_group<S::kStages - 2>();
    group_sync();  // the tile is there for the group, and the stage refilled next is read out
    issue(ahead, stage == 0 ? S::kStages - 1 : stage - 1);
    ahead = next_tile(ahead + S::kKg);
    const uint32_t tile = ring + stage * 2 * S::kTileBytes;
    const int a = p0 + t * kTile;
    if (busy) {
      float sc[2][4] = {}, odd_k[2][4] = {};  // two chains of products each
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t kb[4], qk[4];
        ldmatrix4(kb, tile + k_at[k & 3] + (k >> 2) * 128);
        if constexpr (S::kQInRegs) {
#pragma unroll
          for (int i = 0; i < 4; ++i) qk[i] = qf[k][i];
        } else {  // (rows and pieces lie as in a V tile)
          ldmatrix4(qk, q_tile + v_at[k & 3] + (k >> 2) * 128);
        }
        mma((k & 1) ? odd_k[0] : sc[0], qk, kb[0], kb[1]);
        mma((k & 1) ? odd_k[1] : sc[1], qk, kb[2], kb[3]);
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
      const bool page_ok = s_tile[t] >= 0;
      // every row sees the whole tile
      const bool inside = s.start >= 0 && a + kTile - 1 <= s.first && page_ok &&
                          (p.window == 0 || last_pos - a < p.window || a + kTile <= p.sinks);
      auto sees = [&](int row_pos, int pos) { return visible(p, row_pos, pos) && (page_ok || pos >= fresh); };
      if (!inside) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!sees(i < 2 ? pos_a : pos_b, a + h * 8 + 2 * c + (i & 1))) sc[h][i] = kNone;
      }
      float ta = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      float tb = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
      auto above = [&](float top, float m) { return (top - m) * p.scale2 > kSlack; };  // (m may be that of no score)
      if (__any_sync(~0u, above(ta, m_a) || above(tb, m_b))) {
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          ta = fmaxf(ta, __shfl_xor_sync(~0u, ta, d));
          tb = fmaxf(tb, __shfl_xor_sync(~0u, tb, d));
        }
        const float na = above(ta, m_a) ? ta : m_a, nb = above(tb, m_b) ? tb : m_b;
        const float ga = na == m_a ? 1.f : exp2_fast((m_a - na) * p.scale2);
        const float gb = nb == m_b ? 1.f : exp2_fast((m_b - nb) * p.scale2);
        m_a = na;
        m_b = nb;
        sum[0] *= ga;
        sum[2] *= gb;
#pragma unroll
        for (int i = 0; i < S::kHalf / 8; ++i) {
          acc[i][0] *= ga;
          acc[i][1] *= ga;
          acc[i][2] *= gb;
          acc[i][3] *= gb;
        }
      }
      const float ra = m_a == kNone ? 0.f : -m_a * p.scale2, rb = m_b == kNone ? 0.f : -m_b * p.scale2;
      auto weight = [&](float x, float ref) { return exp2_fast(fmaf(x, p.scale2, ref)); };
      uint32_t pf[4];
      pf[0] = pack_bf16(weight(sc[0][0], ra), weight(sc[0][1], ra));
      pf[1] = pack_bf16(weight(sc[0][2], rb), weight(sc[0][3], rb));
      pf[2] = pack_bf16(weight(sc[1][0], ra), weight(sc[1][1], ra));
      pf[3] = pack_bf16(weight(sc[1][2], rb), weight(sc[1][3], rb));
      mma(sum, pf, kOnes, kOnes);

      bool odd = false;  // non-finite values in a tile that not every row sees whole
      const uint8_t* v_tile = smem + S::kQBytes + (kg * S::kStages + stage) * 2 * S::kTileBytes + S::kTileBytes;
      if (!inside) {
        const uint4* v = reinterpret_cast<const uint4*>(v_tile);
        for (int i = lane; i < S::kTileBytes / 16; i += 32) {
          const uint4 u = v[i];
          odd |= non_finite2(u.x) || non_finite2(u.y) || non_finite2(u.z) || non_finite2(u.w);
        }
        odd = __any_sync(~0u, odd);
      }
      if (!odd) {
#pragma unroll
        for (int i = 0; i < S::kHalf / 16; ++i) {
          uint32_t vb[4];
          ldmatrix4_trans(vb, tile + v_at[i & 3] + (i >> 2) * 128);
          mma(acc[2 * i], pf, vb[0], vb[1]);
          mma(acc[2 * i + 1], pf, vb[2], vb[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < S::kHalf / 16; ++i) {
          uint32_t vb[4];
          ldmatrix4_trans(vb, tile + v_at[i & 3] + (i >> 2) * 128);
#pragma unroll
          for (int e = 0; e < 4; ++e) vb[e] = finite_or_zero2(vb[e]);
          mma(acc[2 * i], pf, vb[0], vb[1]);
          mma(acc[2 * i + 1], pf, vb[2], vb[3]);
        }
        for (int j = 0; j < kTile; ++j) {
          const uint32_t wa = j < 8 ? pf[0] : pf[2], wb = j < 8 ? pf[1] : pf[3];
          const int from = (lane & ~3) | ((j & 7) >> 1);
          const uint32_t ua = __shfl_sync(~0u, wa, from), ub = __shfl_sync(~0u, wb, from);
          const float fa = (j & 1) ? high_f(ua) : low_f(ua), fb = (j & 1) ? high_f(ub) : low_f(ub);
          const bool va = sees(pos_a, a + j), vb = sees(pos_b, a + j);
#pragma unroll
          for (int i = 0; i < S::kHalf / 8; ++i) {
            const uint32_t u = *reinterpret_cast<const uint32_t*>(v_tile + j * S::kRowBytes + half * 2 * S::kHalf +
                                                                  ((i ^ (j & 7)) << 4) + 4 * c);
            if ((u & 0x7F80u) == 0x7F80u) {
              if (va) acc[i][0] += fa * low_f(u);
              if (vb) acc[i][2] += fb * low_f(u);
            }
            if ((u & 0x7F800000u) == 0x7F800000u) {
              if (va) acc[i][1] += fa * high_f(u);
              if (vb) acc[i][3] += fb * high_f(u);
            }
          }
        }
      }
    }
    t = next_tile(t + S::kKg);
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
  }
  float l_a = sum[0], l_b = sum[2];
  // from here on the maxima are those of the exponents
  if (m_a != kNone) m_a *= p.scale2;
  if (m_b != kNone) m_b *= p.scale2;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the ring becomes the exchange

  // Join the groups in order: the others leave theirs, group 0 adds.
  float* ex = reinterpret_cast<float*>(smem + S::kQBytes);
  constexpr int kLeft = S::kLeft / 4;
  const int slot = rt * S::kDs + half;
  if (kg > 0) {
    float* e = ex + ((kg - 1) * RT * S::kDs + slot) * kLeft;
#pragma unroll
    for (int i = 0; i < S::kHalf / 8; ++i)
      reinterpret_cast<float4*>(e)[i * 32 + lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    if (c == 0) {
      float2* st = reinterpret_cast<float2*>(e + 16 * S::kHalf);
      st[r] = make_float2(m_a, l_a);
      st[r + 8] = make_float2(m_b, l_b);
    }
  }
  __syncthreads();
  if (kg > 0) {
    // Meanwhile the new rows go to their pages; nobody reads those slots in this call.
    if (rg == 0 && p1 > fresh) {
      const int a = max(p0, fresh);
      for (int i = tid - S::kGroup; i < (p1 - a) * kPieces; i += S::kThreads - S::kGroup) {
        const int pos = a + i / kPieces, piece = i % kPieces;
        const long long where = s_tile[(pos - p0) / kTile];
        if (where < 0) continue;
        const long long src = static_cast<long long>(s.first_row + pos - s.start) * p.kv_row +
                              static_cast<long long>(head) * D + piece * 8;
        const long long dst = where + (pos - p0) % kTile * p.slot_stride + piece * 8;
        *reinterpret_cast<uint4*>(p.k_cache + dst) = __ldg(reinterpret_cast<const uint4*>(p.k_new + src));
        *reinterpret_cast<uint4*>(p.v_cache + dst) = __ldg(reinterpret_cast<const uint4*>(p.v_new + src));
      }
    }
    return;
  }
  float2 sa[S::kKg], sb[S::kKg];
  sa[0] = make_float2(m_a, l_a);
  sb[0] = make_float2(m_b, l_b);
  float top_a = m_a, top_b = m_b;
#pragma unroll
  for (int g = 1; g < S::kKg; ++g) {
    const float2* st = reinterpret_cast<const float2*>(ex + ((g - 1) * RT * S::kDs + slot) * kLeft + 16 * S::kHalf);
    sa[g] = st[r];
    sb[g] = st[r + 8];
    top_a = fmaxf(top_a, sa[g].x);
    top_b = fmaxf(top_b, sb[g].x);
  }
  const float ra = top_a == kNone ? 0.f : top_a, rb = top_b == kNone ? 0.f : top_b;
  float wa = exp2_fast(sa[0].x - ra), wb = exp2_fast(sb[0].x - rb);
  l_a = sa[0].y * wa;
  l_b = sb[0].y * wb;
#pragma unroll
  for (int i = 0; i < S::kHalf / 8; ++i) {
    acc[i][0] *= wa;
    acc[i][1] *= wa;
    acc[i][2] *= wb;
    acc[i][3] *= wb;
  }
#pragma unroll
  for (int g = 1; g < S::kKg; ++g) {
    wa = exp2_fast(sa[g].x - ra);
    wb = exp2_fast(sb[g].x - rb);
    l_a = fmaf(sa[g].y, wa, l_a);
    l_b = fmaf(sb[g].y, wb, l_b);
    const float4* e = reinterpret_cast<const float4*>(ex + ((g - 1) * RT * S::kDs + slot) * kLeft);
#pragma unroll
    for (int i = 0; i < S::kHalf / 8; ++i) {
      const float4 v = e[i * 32 + lane];
      acc[i][0] = fmaf(v.x, wa, acc[i][0]);
      acc[i][1] = fmaf(v.y, wa, acc[i][1]);
      acc[i][2] = fmaf(v.z, wb, acc[i][2]);
      acc[i][3] = fmaf(v.w, wb, acc[i][3]);
    }
  }

#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int row = row0 + 8 * side;
    if (row >= live_rows) continue;
    const float l = side ? l_b : l_a;
    if (direct) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no visible position: zeros
      const int i_new = row / p.by_group;
      uint32_t* o = reinterpret_cast<uint32_t*>(
          p.out + static_cast<long long>(s.first_row + i_new) * p.out_row +
          static_cast<long long>(head * p.group + row - i_new * p.group) * D + half * S::kHalf);
#pragma unroll
      for (int i = 0; i < S::kHalf / 8; ++i) o[i * 4 + c] = pack_bf16(acc[i][2 * side] * inv, acc[i][2 * side + 1] * inv);
    } else {
      const long long at =
          ((static_cast<long long>(b) * p.splits + z) * p.kv_heads + head) * (p.max_new * p.group) + row;
      float2* o = reinterpret_cast<float2*>(p.part + at * D + half * S::kHalf);
#pragma unroll
      for (int i = 0; i < S::kHalf / 8; ++i) o[i * 4 + c] = make_float2(acc[i][2 * side], acc[i][2 * side + 1]);
      if (c == 0 && half == 0) p.stat[at] = make_float2(side ? top_b : top_a, l);
    }
  }
}

// Joins a row's chunks: W warps take the chunks by their number mod W, each
// joins its own in rising order with a running maximum, and the W are added in
// order.  Latency is all there is to it.  A sequence alone without a window may
// have hundreds of chunks: 8 warps, and the first 32 chunks' sums are on their
// way while the length is read (those beyond it are not looked at); 100003
// positions on one head take 20.4 us a call for 27.1, 32771 on 8 heads 27.9 for
// 29.9.  A batch with more than 16 chunks a sequence does the same (two of 4099,
// 4 heads: 11.8 for 12.7).  Others and windows have few chunks and many rows to
// join, whose idle warps cost more: 4 (16 sequences, 3 new: 21.4, 23.2 with 8).
template <int D, int W>
__global__ void __launch_bounds__(W * 32) join_kernel(const __grid_constant__ Params p) {
  constexpr int kPer = D / 32;
  constexpr int kBatch = 4;
  __shared__ float s_sum[W][D];
  __shared__ float2 s_stat[W];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z, i = blockIdx.y, hq = blockIdx.x;
  const int head = hq / p.by_group, row = i * p.group + hq - head * p.group;
  const long long step = static_cast<long long>(p.kv_heads) * (p.max_new * p.group);
  const long long at0 = (static_cast<long long>(b) * p.splits * p.kv_heads + head) * (p.max_new * p.group) + row;

  float2 st[kBatch];
  float v[kBatch][kPer];
  auto load = [&](int z, int end) {  // chunks z, z + W, .. below end
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (z + W * j < end) {
        const long long at = at0 + (z + W * j) * step;
        st[j] = p.stat[at];
        const float* o = p.part + at * D + lane * kPer;
        if constexpr (kPer == 2) *reinterpret_cast<float2*>(v[j]) = *reinterpret_cast<const float2*>(o);
        else
#pragma unroll
          for (int k = 0; k < kPer; k += 4) *reinterpret_cast<float4*>(&v[j][k]) = *reinterpret_cast<const float4*>(o + k);
      }
    }
  };
  if constexpr (W == 8) load(warp, p.splits);
  if (b == 0 && i == 0 && hq == 0 && threadIdx.x == 0) publish_errors(p.status, p.pending);
  const Seq s = sequence(p, b);
  if (!s.ok || i >= s.n) return;

  float top = kNone, l = 0.f, sum[kPer] = {};
  auto add = [&](int z, int end) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (z + W * j < end) {
        const float next = fmaxf(top, st[j].x), ref = next == kNone ? 0.f : next;
        const float old = exp2_fast(top - ref), w = exp2_fast(st[j].x - ref);
        top = next;
        l = fmaf(st[j].y, w, l * old);
#pragma unroll
        for (int k = 0; k < kPer; ++k) sum[k] = fmaf(v[j][k], w, sum[k] * old);
      }
    }
  };
  if (W == 8 || p.window == 0) {
    if constexpr (W != 8) load(warp, s.chunks);
    add(warp, s.chunks);
    for (int z = warp + W * kBatch; z < s.chunks; z += W * kBatch) {
      load(z, s.chunks);
      add(z, s.chunks);
    }
  } else {  // the sinks' chunks are numbers 0 .., the others lo_chunk ..
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int z0 = side ? s.sink_chunks : 0, end = side ? s.chunks : s.sink_chunks;
      for (int z = z0 + ((warp - (side ? s.lo_chunk : 0)) & (W - 1)); z < end; z += W * kBatch) {
        load(z, end);
        add(z, end);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) s_sum[warp][lane * kPer + k] = sum[k];
  if (lane == 0) s_stat[warp] = make_float2(top, l);
  __syncthreads();
  top = kNone;
#pragma unroll
  for (int j = 0; j < W; ++j) top = fmaxf(top, s_stat[j].x);
  const float ref = top == kNone ? 0.f : top;
  float w[W];
  l = 0.f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    w[j] = exp2_fast(s_stat[j].x - ref);
    l = fmaf(s_stat[j].y, w[j], l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (threadIdx.x < D / 2) {
    const int k = threadIdx.x;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float2 u = *reinterpret_cast<const float2*>(&s_sum[j][2 * k]);
      x = fmaf(u.x, w[j], x);
      y = fmaf(u.y, w[j], y);
    }
    reinterpret_cast<uint32_t*>(p.out + static_cast<long long>(s.first_row + i) * p.out_row + static_cast<long long>(hq) * D)[k] =
        pack_bf16(x * inv, y * inv);
  }
}

// Positions per chunk: the multiple of 64 that cuts the call's positions (span
// x heads x sequences) into a few chunks for each SM.  One sequence: 304, as
// many CTAs of 32 rows as the GPU holds at once.  A batch: 608, as its sequences
// have lengths of their own, half of max_len on average, and 684 for 16 or more
// sequences, whose CTAs even out.  A window: 304, and 152 for heads of 256.  Not
// less than 128 past 2048 positions: the second kernel takes 32 chunks at once.
// Measured, us per call.  One sequence of 32771, 8 heads of 128, 32 rows: 30.6 at
// 304, 38.5 at 456 (a second wave).
// Batches of lengths up to L, at 608 and 684 (heads x width, rows a head):
//   4 of 9001, 4 x 64, 18: 8.6 and 11.0;  8 of 6000, 8 x 128, 24: 24.2 and 28.1;
//   8 of 6000, 8 x 128, 4 and 12: 16.4 and 15.3, 19.6 and 19.2;
//   12 of 9001, 4 x 64, 6 and 18: 11.3 and 10.2, 15.5 and 15.3;
//   16 and 32 of 9001, 4 x 64, 18: 18.2 and 18.0, 29.6 and 29.3;
//   16, 24, 32 of 6000, 8 x 128, 4: 26.5 and 25.4, 37.4 and 34.5, 42.3 and 42.4;
//   16, 32, 64 of 4000, 2 x 256, 24: 20.6 and 21.5, 30.8 and 29.2, 53.6 and 49.6;
//   32 of 3000, 4 x 128, 24: 23.7 and 24.4;  64 of 20000, 1 x 128, 8: 39.8 and 38.3.
// So 684 loses up to a third below 16 sequences and up to 4% from there on, and
// gains up to 8%; 304 is slower than both by up to a half.
// Windows of 4096 at 152 and 304, heads of 256:
//   64 rows, 2 x 4 and 1 x 8 heads (one wave of CTAs): 22.6 and 29.1;
//   64 rows, 8 x 2 and 8 x 4: 46.9 and 42.2, 89.7 and 75.9;
//   4 rows, 2 x 4 and 8 x 2: 13.0 and 11.8, 23.2 and 19.0;
// of 128: 64 rows, 1 x 8: 12.7 and 18.2;  4 rows, 2 x 8, 8 x 2 and 8 x 8: 12.4 and
// 10.3, 13.3 and 10.7, 35.0 and 28.7.  A rule by rows and waves would serve both;
// this one goes by the width alone.
// Chunks of 128 for 64: 4 of 4099, 2 heads of 256: 12.4 for 17.5; one of 2049, 8
// heads of 128: 6.9 for 7.7; but one of 611: 7.4 for 6.6.  max_len far above the
// lengths makes few chunks: one token at 4096, 8 heads of 128: 6.9 with 4096, 26.2
// with 131072.
int chunk_for(const w4g128_attend_args& a) {
  long long span = a.max_len;
  if (a.window > 0) span = std::min<long long>(span, static_cast<long long>(a.window) + a.sinks + 16);
  const long long all = span * a.kv_heads * a.count;
  const int target = a.window > 0 ? (a.head_dim == 256 ? 152 : 304) : a.count == 1 ? 304 : a.count < 16 ? 608 : 684;
  const long long least = a.window == 0 && a.max_len > 2048 ? 128 : 64;
  const long long chunk = std::max(least, (all + 64LL * target - 1) / (64LL * target) * 64);
  return static_cast<int>(std::min<long long>(chunk, kMaxChunk));
}

// Most chunks that a sequence's rows can see: all of them, or the window's
// span of at most window + max_new - 1 positions and the sinks' chunks.
int splits_for(const w4g128_attend_args& a, int chunk) {
  const long long all = (static_cast<long long>(a.max_len) + chunk - 1) / chunk;
  if (a.window == 0) return static_cast<int>(all);
  const long long span = (static_cast<long long>(a.window) + a.max_new - 1 + chunk - 1) / chunk + 1;
  const long long sinks = (static_cast<long long>(a.sinks) + chunk - 1) / chunk;
  return static_cast<int>(std::min(all, span + sinks));
}

int check(const w4g128_attend_args* a) {
  if (a == nullptr || a->q == nullptr || a->k_cache == nullptr || a->v_cache == nullptr || a->page_table == nullptr ||
      a->row_offsets == nullptr || a->lens == nullptr || a->out == nullptr || (a->k_new == nullptr) != (a->v_new == nullptr))
    return W4G128_ERR_INVALID_ARG;
  if (a->rows < 1 || a->rows > (1 << 20) || a->count < 1 || a->count > W4G128_MAX_SEQUENCES || a->max_new < 1 ||
      a->max_new > W4G128_MAX_M || a->window < 0 || a->sinks < 0 || (a->sinks > 0 && a->window == 0) ||
      !std::isfinite(a->scale * kLog2e))
    return W4G128_ERR_INVALID_ARG;
  if (a->kv_heads < 1 || a->kv_heads > 256 || a->q_heads < a->kv_heads || a->q_heads % a->kv_heads != 0 ||
      a->q_heads / a->kv_heads > 16 || (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256))
    return W4G128_ERR_SHAPE;
  if (a->pages < 1 || a->page_size < 16 || a->page_size % 16 != 0 || a->max_len < 1 || a->max_len > (1 << 24))
    return W4G128_ERR_SHAPE;
  const long long dim = a->head_dim;
  if (a->q_row < a->q_heads * dim || a->out_row < a->q_heads * dim || (a->k_new && a->kv_row < a->kv_heads * dim) ||
      a->slot_stride < dim || a->page_stride < dim || a->head_stride < dim ||
      a->table_row < (a->max_len - 1) / a->page_size + 1)
    return W4G128_ERR_SHAPE;
  auto off = [](const void* q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0; };
  if (off(a->q, 16) || off(a->k_new, 16) || off(a->v_new, 16) || off(a->k_cache, 16) || off(a->v_cache, 16) ||
      off(a->out, 16) || off(a->page_table, 4) || off(a->row_offsets, 4) || off(a->lens, 4))
    return W4G128_ERR_ALIGN;
  for (long long v : {a->q_row, a->kv_row, a->out_row, a->page_stride, a->slot_stride, a->head_stride})
    if (v % 8 != 0) return W4G128_ERR_ALIGN;
  return W4G128_OK;
}

size_t bytes_for(const w4g128_attend_args& a) {
  const int splits = splits_for(a, chunk_for(a));
  if (splits == 1) return kStatusBytes;
  return kStatusBytes + static_cast<size_t>(a.count) * splits * a.q_heads * a.max_new * (a.head_dim + 2) * 4;
}

template <int D, int RT>
cudaError_t launch_attend(cudaLaunchConfig_t& cfg, Params& p) {
  using S = Shape<D, RT>;
  const cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  const int row_groups = (p.max_new * p.group + 16 * RT - 1) / (16 * RT);
  p.by_row_groups = divisor(row_groups);
  cfg.gridDim = dim3(p.splits, p.kv_heads * row_groups, p.count);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  return cudaLaunchKernelEx(&cfg, attend_kernel<D, RT>, p);
}

template <int D>
cudaError_t launch_dim(cudaLaunchConfig_t& cfg, Params& p) {
  const int rows = p.max_new * p.group;
  const cudaError_t e = rows <= 16 ? launch_attend<D, 1>(cfg, p) : rows <= 32 ? launch_attend<D, 2>(cfg, p)
                                                                              : launch_attend<D, 4>(cfg, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  cfg.gridDim = dim3(p.q_heads, p.max_new, p.count);
  cfg.dynamicSmemBytes = 0;
  if (p.window == 0 && (p.count == 1 || p.splits > 16)) {
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, join_kernel<D, 8>, p);
  }
  cfg.blockDim = dim3(128);
  return cudaLaunchKernelEx(&cfg, join_kernel<D, 4>, p);
}

}  // namespace
}  // namespace w4g128

extern "C" {

size_t w4g128_attend_workspace_bytes(const w4g128_attend_args* args) {
  return w4g128::check(args) == W4G128_OK ? w4g128::bytes_for(*args) : 0;
}

int w4g128_attend(const w4g128_attend_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace w4g128;
  int rc = check(a);
  if (rc != W4G128_OK) return rc;
  if (ws == nullptr) return W4G128_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0) return W4G128_ERR_ALIGN;
  if (ws_bytes < bytes_for(*a)) return W4G128_ERR_WORKSPACE;
  rc = fault_hook();
  if (rc != W4G128_OK) return rc;
  if (!device_is_sm103()) return W4G128_ERR_DEVICE;
  Params p;
  p.q = a->q; p.k_new = a->k_new; p.v_new = a->v_new; p.k_cache = a->k_cache; p.v_cache = a->v_cache;
  p.table = a->page_table; p.offsets = a->row_offsets; p.lens = a->lens; p.out = a->out;
  p.q_row = a->q_row; p.kv_row = a->kv_row; p.out_row = a->out_row;
  p.page_stride = a->page_stride; p.slot_stride = a->slot_stride; p.head_stride = a->head_stride;
  p.table_row = a->table_row;
  p.rows = a->rows; p.count = a->count; p.q_heads = a->q_heads; p.kv_heads = a->kv_heads;
  p.group = a->q_heads / a->kv_heads;
  p.pages = a->pages; p.page_size = a->page_size; p.max_len = a->max_len; p.max_new = a->max_new;
  p.window = a->window; p.sinks = a->sinks;
  p.chunk = chunk_for(*a);
  p.splits = splits_for(*a, p.chunk);
  p.by_chunk = divisor(p.chunk);
  p.by_group = divisor(p.group);
  p.by_page = divisor(p.page_size);
  p.scale2 = a->scale == 0.f ? 1.f : std::fabs(a->scale) * kLog2e;
  p.flip_q = a->scale < 0.f ? 0x80008000u : 0u;
  p.keep_q = a->scale == 0.f ? 0u : 0xFFFFFFFFu;
  auto* base = static_cast<uint8_t*>(ws);
  p.status = reinterpret_cast<unsigned long long*>(base);
  p.pending = p.status + 1;
  p.part = reinterpret_cast<float*>(base + kStatusBytes);
  p.stat = reinterpret_cast<float2*>(p.part + static_cast<size_t>(p.count) * p.splits * p.q_heads * p.max_new * a->head_dim);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a->head_dim == 64 ? launch_dim<64>(cfg, p)
                        : a->head_dim == 128 ? launch_dim<128>(cfg, p) : launch_dim<256>(cfg, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
