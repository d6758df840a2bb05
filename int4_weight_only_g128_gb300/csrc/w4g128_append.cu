// Rotated queries, and rotated keys and values put into a paged cache
// (w4g128_append), in one launch.
//
// A head's row is pieces of 8 values, 16 bytes, and every byte is read and written once.
//   * few rows (a decode or verify step): a warp for each head, a piece a lane; the other
//     side of its pairs comes by shuffle.  What takes time is the chain length -> rows ->
//     cosines -> store: 2.9 us for one token, 3.1 for 16 sequences of up to 3 rows in 8
//     bits, of which the launch alone is most.
//   * many: a lane has two pieces, both sides of 8 pairs, and works on two values with
//     one instruction, since here instructions count (a piece a lane, with shuffles and
//     an address for each, took 41.0 us where this takes 33.2).  Row by row what needs no
//     block, by blocks what goes into 8 bits, each on its part of the CTAs.  A prompt of
//     8191 rows (32 + 2 x 8 heads of 128, blocks of 64) takes 33.2 us, 5.5 TB/s of the 184
//     MB that it reads and writes; of as many into bf16 (201 MB) 35.3, 5.7 TB/s.  Two
//     prompts of 2049 rows of 16 + 2 x 4 heads of 256 in bf16 take 21.2, 4.8 TB/s, for 100
//     MB: start and end take 3 us of it, and 12294 pieces of work on 2424 warps a sixth
//     round for some.
// The angle p f of position p is a 64-bit integer of 2^-64 turns, p times f / 2 pi
// rounded to that: exact modulo a turn but for p 2^-64 and the 2^-53 of f / 2 pi in
// 64 bits.  Its multiple of a quarter turn goes into signs, so that the fp32
// argument is at most an eighth and its rounding costs 2^-27 turns at most.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "w4g128_divide.cuh"
#include "w4g128_e4m3.cuh"
#include "w4g128_internal.h"
#include "w4g128_ops.h"
#include "w4g128_ptx.cuh"

namespace w4g128 {
namespace {

constexpr int kChunk = 64;  // positions, a multiple of every block
constexpr int kThreads = 256;
constexpr int kFewRows = 16;
// CTAs of a prompt's call: two an SM, but the one that looks for errors (a third an SM, with the registers that leaves, takes 27 us where this takes 21)
constexpr int kWorkers = 303;
constexpr size_t kWorkspace = 256;
constexpr int kLowestScale = -100;

struct Params {
  const uint16_t *q, *k_new, *v_new;
  uint16_t* q_out;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const double* freqs;
  const int *table, *offsets, *lens;
  long long q_row, q_out_row, kv_row, page_stride, slot_stride, head_stride, scale_page, scale_head, table_row;
  int rows, count, q_heads, kv_heads, half, interleaved, pages, block_log2, max_len, max_new;
  int chunks;       // that the new rows of a sequence may touch
  int row_workers;  // CTAs that work row by row
  Divisor by_page, by_half, by_kv, by_new, by_parts;
  int ragged;          // whether some sequences are known to have fewer new rows than max_new
  unsigned row_items;  // parts of rows that are worked on one by one, if none are
  unsigned long long* status;
};

// A sequence's new rows.
struct Span {
  bool ok;
  int first_row, n, len, start, first;  // start: the first new row's position; first: the first real one's
};

__device__ __forceinline__ Span span_of(const Params& p, int b) {
  Span s;
  s.first_row = p.offsets[b];
  s.n = p.offsets[b + 1] - s.first_row;
  s.len = p.lens[b];
  s.ok = s.first_row >= 0 && s.n >= 0 && s.n <= p.max_new && s.first_row <= p.rows - s.n && s.len >= 0 &&
         s.len <= p.max_len;
  s.start = s.len - s.n;
  s.first = max(s.start, 0);
  return s;
}

// One CTA looks all lengths, row ranges and page ids over, beside the others.
__device__ void check_all(const Params& p) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  auto page_bad = [&](int b, int page) {
    const int id = p.table[static_cast<long long>(b) * p.table_row + page];
    return id < 0 || id >= p.pages;
  };
  for (int b0 = 0; b0 < p.count; b0 += kThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int from = 0, to = 0;  // pages of the new rows
    if (b < p.count) {
      const Span s = span_of(p, b);
      bad |= !s.ok;
      if (s.ok && s.first < s.len) {
        from = s.first / p.by_page;
        to = (s.len - 1) / p.by_page + 1;
      }
    }
    const bool many = to - from > 4;
    if (!many)
      for (int page = from; page < to; ++page) bad |= page_bad(b, page);
    for (unsigned left = __ballot_sync(~0u, many); left != 0u; left &= left - 1) {  // a prompt: the warp together
      const int src = __ffs(left) - 1;
      const int at = __shfl_sync(~0u, b, src), end = __shfl_sync(~0u, to, src);
      for (int page = __shfl_sync(~0u, from, src) + lane; page < end; page += 32) bad |= page_bad(at, page);
    }
  }
  if (__syncthreads_or(bad)) bad = true;
  if (threadIdx.x == 0) st_relaxed_u64(p.status, bad ? W4G128_ERR_CACHE : W4G128_OK);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The scale that a block of magnitude `top` (its bits) gets anew, and its inverse: powers of two.
__device__ __forceinline__ int fresh_exponent(uint32_t top) {
  return max(static_cast<int>(top >> 23) - 127 - 5, kLowestScale);
}
__device__ __forceinline__ float exp2_of(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// 2^-64 turns a position of one frequency.
__device__ __forceinline__ unsigned long long turn_step(double freq) {
  double turns = freq * 0.15915494309189533576888376337251;  // 1 / (2 pi)
  turns -= floor(turns);
  return __double2ull_rz(turns * 18446744073709551616.0);
}
// Cosine and sine of `pos` steps.
__device__ __forceinline__ float2 turned(unsigned long long step, int pos) {
  const unsigned long long full = static_cast<unsigned long long>(pos) * step;
  const uint32_t turn = static_cast<uint32_t>((full + 0x80000000ull) >> 32);  // 2^-32 turns
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(turn - (quarter << 30))) * 0x1p-31f;  // half turns
  float sn, cs;
  sincospif(x, &sn, &cs);
  const float c = (quarter & 1u) ? -sn : cs, d = (quarter & 1u) ? cs : sn;
  return (quarter & 2u) ? make_float2(-c, -d) : make_float2(c, d);
}

// A lane's piece of 8 values of a head, the pairs it belongs to and their angles.
template <int D>
struct Piece {
  static constexpr int kPieces = D / 8;       // of a row
  static constexpr int kRows = 32 / kPieces;  // rows, or heads of a row, of a warp at once
  int sub, piece, first_pair, from;           // from: the lane with the other side of the pairs
  bool turns, second, interleaved;
  float c[8], s[8];  // of its pairs (interleaved: 4; else the sine has the sign of this lane's side)

  __device__ __forceinline__ Piece(const Params& p, int lane) {
    sub = lane / kPieces;
    piece = lane % kPieces;
    const int side = p.half / 8;  // pieces of one side of the pairs
    interleaved = p.interleaved != 0;
    turns = piece < 2 * side;
    second = !interleaved && piece >= side;
    first_pair = !turns ? 0 : interleaved ? piece * 4 : (second ? piece - side : piece) * 8;
    from = !turns || interleaved ? lane : second ? lane - side : lane + side;
  }
  // Its angles, from the cosines and sines of a row.
  __device__ __forceinline__ void look(const float* cosines, const float* sines) {
    if (!turns) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && interleaved) break;
      const float4 x = *reinterpret_cast<const float4*>(cosines + first_pair + 4 * h);
      const float4 y = *reinterpret_cast<const float4*>(sines + first_pair + 4 * h);
      c[4 * h] = x.x; c[4 * h + 1] = x.y; c[4 * h + 2] = x.z; c[4 * h + 3] = x.w;
      s[4 * h] = y.x; s[4 * h + 1] = y.y; s[4 * h + 2] = y.z; s[4 * h + 3] = y.w;
    }
    if (interleaved || second) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = -s[i];
  }
  // All lanes of the warp; only: whether this lane's piece is rotated at all.
  __device__ __forceinline__ void rotate(const uint4& raw, bool only, float (&x)[8]) const {
    unpack(raw, x);
    if (interleaved) {
      if (!turns || !only) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = fmaf(a, c[i], -(b * s[i]));
        x[2 * i + 1] = fmaf(b, c[i], a * s[i]);
      }
      return;
    }
    uint4 other;
    other.x = __shfl_sync(~0u, raw.x, from);
    other.y = __shfl_sync(~0u, raw.y, from);
    other.z = __shfl_sync(~0u, raw.z, from);
    other.w = __shfl_sync(~0u, raw.w, from);
    if (!turns || !only) return;
    float y[8];
    unpack(other, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], y[i] * s[i]);
  }
};

__device__ __forceinline__ uint4 packed(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// What is not finite becomes NaN, which takes no part in a maximum.
__device__ __forceinline__ float magnitude(float (&x)[8]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = fmaf(x[e], 0.f, x[e]);
    top = fmaxf(top, fabsf(x[e]));
  }
  return top;
}
// A power of two whose inverse is a normal number too: up to 2^126.
__device__ __forceinline__ bool has_inverse(float scale) {
  return (__float_as_uint(scale) & 0x007FFFFFu) == 0u && scale < 0x1p127f;
}
__device__ __forceinline__ uint2 coded(const float (&x)[8], float scale) {
  uint32_t code[4];
  if (has_inverse(scale)) {
    const float inverse = exp2_of(127 - static_cast<int>(__float_as_uint(scale) >> 23));
#pragma unroll
    for (int e = 0; e < 4; ++e) code[e] = to_e4m3x2(x[2 * e] * inverse, x[2 * e + 1] * inverse);
  } else {  // (a scale that another program set need not be one)
#pragma unroll
    for (int e = 0; e < 4; ++e) code[e] = to_e4m3x2(__fdiv_rn(x[2 * e], scale), __fdiv_rn(x[2 * e + 1], scale));
  }
  return make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
}
// Codes in a scale that is `factor` times smaller than before.
__device__ __forceinline__ uint2 recoded(const uint2& old, float factor) {
  uint32_t code[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t h = e4m3x2_to_half2(static_cast<uint16_t>((e < 2 ? old.x : old.y) >> (e & 1) * 16));
    float a, d;
    asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(a), "=f"(d) : "r"(h));
    code[e] = to_e4m3x2(a * factor, d * factor);
  }
  return make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
}
// The scale of a block of magnitude `top` (its bits) that has positions already (held), in the scale `was`.
__device__ __forceinline__ float scale_for(uint32_t top, bool held, float was, bool& keeps) {
  keeps = held && was > 0.f && __uint_as_float(top) <= kE4M3Max * was;
  return keeps ? was : exp2_of(fresh_exponent(top));
}

// The rows of a chunk: where they go, and their cosines and sines.
struct Rows {
  int p0, live, row0;  // the first position, their number, the first row
};
__device__ __forceinline__ Rows rows_of(const Params& p, const Span& s, int chunk) {
  const int c0 = (s.first & ~(kChunk - 1)) + chunk * kChunk;
  Rows r;
  r.p0 = max(c0, s.first);
  r.live = s.ok && s.n > 0 ? min(c0 + kChunk, s.len) - r.p0 : 0;
  r.row0 = s.first_row + r.p0 - s.start;
  return r;
}
__device__ __forceinline__ void prepare_rows(const Params& p, int b, const Rows& rows, double freq, int pair, int pair_group,
                                             long long* at, long long* block, float* trig) {
  if (static_cast<int>(threadIdx.x) < rows.live) {
    const int pos = rows.p0 + static_cast<int>(threadIdx.x), page = pos / p.by_page;
    const int slot = pos - page * static_cast<int>(p.by_page.d);
    const int id = p.table[static_cast<long long>(b) * p.table_row + page];
    const bool ok = id >= 0 && id < p.pages;
    at[threadIdx.x] = ok ? id * p.page_stride + slot * p.slot_stride : -1;
    block[threadIdx.x] = id * p.scale_page + (p.block_log2 >= 0 ? slot >> p.block_log2 : 0);
  }
  if (p.half > 0) {
    const int groups = kThreads / p.by_half;
    if (pair_group < groups) {
      const unsigned long long step = turn_step(freq);
      for (int r = pair_group; r < rows.live; r += groups) {
        const float2 v = turned(step, rows.p0 + r);
        trig[r * p.half + pair] = v.x;
        trig[(rows.live + r) * p.half + pair] = v.y;
      }
    }
  }
}

// Up to 16 new rows a sequence: a warp for each head of q, k and v.
template <int D>
__global__ void __launch_bounds__(kThreads) append_few_kernel(const __grid_constant__ Params p) {
  using P = Piece<D>;
  constexpr int kPasses = kFewRows / P::kRows, kWarps = kThreads / 32;
  extern __shared__ __align__(16) float s_trig[];      // [live rows][half] cosines, then sines
  __shared__ long long s_at[kFewRows], s_block[kFewRows];  // a row's slot and scale in the caches; -1: no page
  __shared__ unsigned s_top[kWarps][kChunk];           // a block's magnitude
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);

  grid_dependency_wait();
  if (blockIdx.z == 0) {
    if (blockIdx.x == 0 && blockIdx.y == 0) check_all(p);
    return;
  }
  const int pair_group = p.half > 0 ? tid / p.by_half : 0;
  const int pair = tid - pair_group * p.half;
  double freq = 0.0;
  if (p.half > 0) freq = p.freqs[pair];
  const int b = blockIdx.z - 1;
  const Rows rows = rows_of(p, span_of(p, b), blockIdx.x);
  if (rows.live <= 0) return;
  for (int i = tid; i < kWarps * kChunk; i += kThreads) (&s_top[0][0])[i] = 0u;
  prepare_rows(p, b, rows, freq, pair, pair_group, s_at, s_block, s_trig);
  __syncthreads();

  const int u = blockIdx.y * kWarps + warp;
  if (u >= 2 * p.kv_heads + p.q_heads) return;
  const int live = rows.live;
  P my(p, lane);
  const bool is_q = u >= 2 * p.kv_heads, is_v = !is_q && u >= p.kv_heads;
  const int head = is_q ? u - 2 * p.kv_heads : is_v ? u - p.kv_heads : u;
  const long long stride = is_q ? p.q_row : p.kv_row;
  const uint16_t* src = (is_q ? p.q : is_v ? p.v_new : p.k_new) + rows.row0 * stride + static_cast<long long>(head) * D + my.piece * 8;
  uint4 raw[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * P::kRows + my.sub;
    raw[i] = r < live ? *reinterpret_cast<const uint4*>(src + r * stride) : make_uint4(0u, 0u, 0u, 0u);
  }
  auto value = [&](int i, int r, float (&x)[8]) {  // (rows behind the last look at the last's angles)
    const int at = min(r, live - 1);
    if (!is_v) my.look(s_trig + at * p.half, s_trig + (live + at) * p.half);
    my.rotate(raw[i], !is_v, x);
  };
  const long long in_slot = head * p.head_stride + my.piece * 8;
  if (is_q || p.block_log2 < 0) {
    uint16_t* out = p.q_out + rows.row0 * p.q_out_row + static_cast<long long>(head) * D + my.piece * 8;
    uint16_t* cache = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + in_slot;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i * P::kRows >= live) break;
      const int r = i * P::kRows + my.sub;
      float x[8];
      value(i, r, x);
      if (r < live && (is_q || s_at[r] >= 0))
        *reinterpret_cast<uint4*>(is_q ? out + r * p.q_out_row : cache + s_at[r]) = is_v ? raw[i] : packed(x);
    }
    return;
  }

  // 8 bits: the magnitudes of the rows' blocks, then their scales and codes.
  float* scales = (is_v ? p.v_scale : p.k_scale) + head * p.scale_head;
  uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + in_slot;
  const int held = rows.p0 & ((1 << p.block_log2) - 1);  // positions that the first row's block has already
  const bool real0 = s_at[0] >= 0;
  float was = 0.f;
  if (held > 0 && real0) was = scales[s_block[0]];
  unsigned* tops = s_top[warp];
  auto block_of = [&](int r) { return (held + r) >> p.block_log2; };
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (i * P::kRows >= live) break;
    const int r = i * P::kRows + my.sub;
    float x[8];
    value(i, r, x);
    float top = magnitude(x);
#pragma unroll
    for (int d = 1; d < P::kPieces; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (my.piece == 0 && r < live) atomicMax(&tops[block_of(r)], __float_as_uint(top));
  }
  __syncwarp();
  bool keeps;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (i * P::kRows >= live) break;
    const int r = i * P::kRows + my.sub;
    float x[8];
    value(i, r, x);
    if (r >= live || s_at[r] < 0) continue;
    magnitude(x);
    const float scale = scale_for(tops[block_of(r)], held > 0 && block_of(r) == 0, was, keeps);
    *reinterpret_cast<uint2*>(cache + s_at[r]) = coded(x, scale);
    if (my.piece == 0 && !keeps && (r == 0 || block_of(r) != block_of(r - 1))) scales[s_block[r]] = scale;
  }
  if (held > 0 && real0) {
    const float scale = scale_for(tops[0], true, was, keeps);
    if (!keeps) {  // what the block has goes to the larger scale
      for (int i = my.sub; i < held; i += P::kRows) {
        uint2* at = reinterpret_cast<uint2*>(cache + s_at[0] - (held - i) * p.slot_stride);
        *at = recoded(*at, was / scale);
      }
    }
  }
}

// Prompts.  Queries, and keys and values of a bf16 cache, go row by row: a warp reads
// a row's heads as they lie and writes them as they lie, its angles in registers.
// Keys and values of an 8-bit cache go by blocks: a CTA takes 64 positions and, one
// after another, heads of k and v, whose rows its 8 warps keep in registers between
// the maximum that decides a block's scale and the codes.  Both at once, each on a
// part of the CTAs.
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float low_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
// Two values, each operation on both (as one instruction).
__device__ __forceinline__ unsigned long long two(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long mul_two(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma_two(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// A lane's two pieces of 8 values of a head: both sides of 8 pairs, or, interleaved,
// neighbours that hold 8 pairs; of what is not rotated any two.
template <int D>
struct Duo {
  static constexpr int kDuos = D / 16;      // of a row
  static constexpr int kHeads = 32 / kDuos; // of a warp at once
  int sub, duo, first, second;              // the pieces' first values
  bool turns, interleaved;
  unsigned long long c[4], s[4], minus_s[4];  // of its pairs, two by two

  __device__ __forceinline__ Duo(const Params& p, int lane) {
    sub = lane / kDuos;
    duo = lane % kDuos;
    const int side = p.half / 8;  // pieces of one side of the pairs
    interleaved = p.interleaved != 0;
    turns = duo < side;
    first = (interleaved ? 2 * duo : turns ? duo : duo + side) * 8;
    second = interleaved ? first + 8 : first + (turns ? side : kDuos - side) * 8;
  }
  __device__ __forceinline__ void look(const float* cosines, const float* sines) {
    if (!turns) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 x = *reinterpret_cast<const float4*>(cosines + 8 * duo + 4 * h);
      const float4 y = *reinterpret_cast<const float4*>(sines + 8 * duo + 4 * h);
      c[2 * h] = two(x.x, x.y); c[2 * h + 1] = two(x.z, x.w);
      s[2 * h] = two(y.x, y.y); s[2 * h + 1] = two(y.z, y.w);
      minus_s[2 * h] = two(-y.x, -y.y); minus_s[2 * h + 1] = two(-y.z, -y.w);
    }
  }
  // The values of both pieces, two by two, rotated.
  __device__ __forceinline__ void turn(const uint4& one, const uint4& other, unsigned long long (&x)[8]) const {
    unpack(one, other, x);
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, b, c0, c1, s0, s1;
        split(x[i], a, b);
        split(c[i / 2], c0, c1);
        split(s[i / 2], s0, s1);
        const float cs = i & 1 ? c1 : c0, sn = i & 1 ? s1 : s0;
        x[i] = two(fmaf(a, cs, -(b * sn)), fmaf(b, cs, a * sn));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned long long a = x[i], b = x[4 + i];
        x[i] = fma_two(a, c[i], mul_two(b, minus_s[i]));
        x[4 + i] = fma_two(b, c[i], mul_two(a, s[i]));
      }
    }
  }
  __device__ __forceinline__ static void unpack(const uint4& one, const uint4& other, unsigned long long (&x)[8]) {
    const uint32_t v[8] = {one.x, one.y, one.z, one.w, other.x, other.y, other.z, other.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = two(low_f(v[i]), high_f(v[i]));
  }
  __device__ __forceinline__ void rotate(uint4& one, uint4& other) const {
    unsigned long long x[8];
    turn(one, other, x);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      split(x[i], lo, hi);
      v[i] = pack_bf16(lo, hi);
    }
    one = make_uint4(v[0], v[1], v[2], v[3]);
    other = make_uint4(v[4], v[5], v[6], v[7]);
  }
};

// The largest finite magnitude; what is infinite becomes NaN, which takes no part.
__device__ __forceinline__ float magnitude_two(unsigned long long (&x)[8]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    split(x[i], lo, hi);
    top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
  }
  if (top == INFINITY) {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      split(x[i], lo, hi);
      lo = fmaf(lo, 0.f, lo);
      hi = fmaf(hi, 0.f, hi);
      x[i] = two(lo, hi);
      top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
    }
  }
  return top;
}
// The codes of 8 values.
__device__ __forceinline__ uint2 coded_two(const unsigned long long* x, float scale) {
  uint32_t code[4];
  if (has_inverse(scale)) {
    const float inverse = exp2_of(127 - static_cast<int>(__float_as_uint(scale) >> 23));
    const unsigned long long by = two(inverse, inverse);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      split(mul_two(x[e], by), lo, hi);
      code[e] = to_e4m3x2(lo, hi);
    }
  } else {  // (a scale that another program set need not be one)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      split(x[e], lo, hi);
      code[e] = to_e4m3x2(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale));
    }
  }
  return make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
}

// Of ragged sequences: sums[b] is how many rows (or chunks) those before b have, so
// that workers share what there is.  All threads of the CTA.
__device__ void sum_up(const Params& p, bool chunks, int* sums) {
  __shared__ int s_warps[kThreads / 32];
  constexpr int kPer = W4G128_MAX_SEQUENCES / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int v[kPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = tid * kPer + j;
    v[j] = 0;
    if (b < p.count) {
      const Span s = span_of(p, b);
      if (s.ok && s.n > 0 && s.len > 0) v[j] = chunks ? (s.len - 1) / kChunk - s.first / kChunk + 1 : s.n;
    }
    sum += v[j];
  }
  int before = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) s_warps[warp] = before;
  __syncthreads();
  before -= sum;
  for (int i = 0; i < warp; ++i) before += s_warps[i];
  if (tid == 0) sums[0] = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    before += v[j];
    if (tid * kPer + j < p.count) sums[tid * kPer + j + 1] = before;
  }
  __syncthreads();
}
// The sequence that the row (or chunk) `which` of all belongs to.
__device__ __forceinline__ int sequence_of(const int* sums, int count, int which) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sums[mid] <= which) lo = mid;
    else hi = mid;
  }
  return lo;
}

constexpr int kRowBatch = 4;  // pairs of pieces of a lane at once: 8 heads of 256, 16 of 128, 32 of 64
template <int D>
__device__ void append_rows(const Params& p, int worker, int workers, float* trig, int* sums) {
  using P = Duo<D>;
  constexpr int kWarps = kThreads / 32, kHeads = kRowBatch * P::kHeads;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  constexpr int kSteps = D / 64;  // pairs of a lane
  unsigned long long step[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) step[i] = i * 32 + lane < p.half ? turn_step(p.freqs[i * 32 + lane]) : 0ull;
  float* cosines = trig + warp * D;
  float* sines = cosines + D / 2;
  P my(p, lane);
  const int heads = p.q_heads + (p.block_log2 < 0 ? 2 * p.kv_heads : 0);
  if (p.ragged) sum_up(p, false, sums);
  const unsigned all = p.ragged ? static_cast<unsigned>(min(sums[p.count], p.rows)) * p.by_parts.d : p.row_items, stride = workers * kWarps;
  struct Item {  // a part of a row's heads
    bool real, queries;  // queries: all of them
    int pos, h0, id;     // id: of the row's page, where it is asked for
    long long row;
    uint4 raw[2 * kRowBatch];
  };
  const uint16_t* q = p.q + my.sub * D;
  uint16_t* q_out = p.q_out + my.sub * D;
  auto load = [&](unsigned item, Item& it) {
    it.real = false;
    if (item >= all) return;
    const int which = static_cast<int>(item) / p.by_parts;
    const int h0 = (static_cast<int>(item) - which * static_cast<int>(p.by_parts.d)) * kHeads;
    const int b = p.ragged ? sequence_of(sums, p.count, which) : which / p.by_new;
    const int i_new = which - (p.ragged ? sums[b] : b * p.max_new);
    const Span s = span_of(p, b);
    it.pos = s.start + i_new;
    it.row = s.first_row + i_new;
    it.h0 = h0;
    it.queries = h0 + kHeads <= p.q_heads;
    it.real = s.ok && i_new < s.n && it.pos >= 0;
    if (!it.real) return;
    if (it.queries) {
      const uint16_t* from = q + it.row * p.q_row + static_cast<long long>(h0) * D;
#pragma unroll
      for (int i = 0; i < kRowBatch; ++i) {
        it.raw[2 * i] = *reinterpret_cast<const uint4*>(from + i * P::kHeads * D + my.first);
        it.raw[2 * i + 1] = *reinterpret_cast<const uint4*>(from + i * P::kHeads * D + my.second);
      }
      return;
    }
    if (p.block_log2 < 0) it.id = p.table[static_cast<long long>(b) * p.table_row + it.pos / p.by_page];
#pragma unroll
    for (int i = 0; i < kRowBatch; ++i) {
      const int h = h0 + i * P::kHeads + my.sub;
      const uint16_t* from = h < p.q_heads ? p.q + it.row * p.q_row + static_cast<long long>(h) * D
                                           : (h < p.q_heads + p.kv_heads ? p.k_new : p.v_new) + it.row * p.kv_row +
                                                 static_cast<long long>((h - p.q_heads) % p.by_kv) * D;
      it.raw[2 * i] = h < heads ? *reinterpret_cast<const uint4*>(from + my.first) : make_uint4(0u, 0u, 0u, 0u);
      it.raw[2 * i + 1] = h < heads ? *reinterpret_cast<const uint4*>(from + my.second) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  Item next;
  load(worker * kWarps + warp, next);
  for (unsigned item = worker * kWarps + warp; item < all; item += stride) {
    Item it = next;
    load(item + stride, next);  // on its way while this one is worked on
    if (!it.real) continue;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i * 32 + lane < p.half) {
        const float2 v = turned(step[i], it.pos);
        cosines[i * 32 + lane] = v.x;
        sines[i * 32 + lane] = v.y;
      }
    }
    __syncwarp();
    my.look(cosines, sines);
#pragma unroll
    for (int i = 0; i < kRowBatch; ++i)
      if (my.turns && it.h0 + i * P::kHeads + my.sub < p.q_heads + p.kv_heads) my.rotate(it.raw[2 * i], it.raw[2 * i + 1]);
    if (it.queries) {
      uint16_t* to = q_out + it.row * p.q_out_row + static_cast<long long>(it.h0) * D;
#pragma unroll
      for (int i = 0; i < kRowBatch; ++i) {
        *reinterpret_cast<uint4*>(to + i * P::kHeads * D + my.first) = it.raw[2 * i];
        *reinterpret_cast<uint4*>(to + i * P::kHeads * D + my.second) = it.raw[2 * i + 1];
      }
      continue;
    }
    long long at = -1;
    if (p.block_log2 < 0 && it.id >= 0 && it.id < p.pages)
      at = it.id * p.page_stride + (it.pos - it.pos / p.by_page * static_cast<int>(p.by_page.d)) * p.slot_stride;
#pragma unroll
    for (int i = 0; i < kRowBatch; ++i) {
      const int h = it.h0 + i * P::kHeads + my.sub;
      const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.kv_heads;
      if (h >= heads || (!is_q && at < 0)) continue;
      const int kv = (h - p.q_heads) % p.by_kv;
      uint16_t* to = is_q ? p.q_out + it.row * p.q_out_row + static_cast<long long>(h) * D
                          : static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + at + kv * p.head_stride;
      *reinterpret_cast<uint4*>(to + my.first) = it.raw[2 * i];
      *reinterpret_cast<uint4*>(to + my.second) = it.raw[2 * i + 1];
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) append_rows_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) float s_trig[kThreads / 32 * D];
  __shared__ int s_sums[W4G128_MAX_SEQUENCES + 1];
  grid_dependency_wait();
  if (blockIdx.x == 0) check_all(p);
  else append_rows<D>(p, static_cast<int>(blockIdx.x) - 1, static_cast<int>(gridDim.x) - 1, s_trig, s_sums);
}

constexpr int kBlockStages = 2;  // (3 take room from the L1 cache: 32.9 us for 8191 rows, and 32.6)

template <int D>
__global__ void __launch_bounds__(kThreads, 2) append_many_kernel(const __grid_constant__ Params p) {
  using P = Duo<D>;
  constexpr int kWarps = kThreads / 32, kWarpRows = kChunk / kWarps;  // a warp's rows of a chunk, side by side
  constexpr int kPasses = kWarpRows / P::kHeads;  // (a warp has as many rows at once as heads of a row above)
  constexpr int kStages = kBlockStages;
  extern __shared__ __align__(16) uint8_t s_many[];    // the stages; [live rows][half] cosines, then sines
  __shared__ long long s_at[kChunk], s_block[kChunk];  // a row's slot and scale in the caches; -1: no page
  __shared__ unsigned s_top[3][kChunk];                // a block's magnitude, of three heads in turn
  __shared__ int s_sums[W4G128_MAX_SEQUENCES + 1];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);

  grid_dependency_wait();
  if (blockIdx.x == 0) {
    check_all(p);
    return;
  }
  const int worker = static_cast<int>(blockIdx.x) - 1;
  if (worker < p.row_workers) {
    append_rows<D>(p, worker, p.row_workers, reinterpret_cast<float*>(s_many), s_sums);
    return;
  }

  const int pair_group = p.half > 0 ? tid / p.by_half : 0;
  const int pair = tid - pair_group * p.half;
  double freq = 0.0;
  if (p.half > 0) freq = p.freqs[pair];
  P my(p, lane);
  uint4* ring = reinterpret_cast<uint4*>(s_many) + tid;
  float* s_trig = reinterpret_cast<float*>(s_many + kThreads * kPasses * kStages * 32);
  // An equal share of all (sequence, chunk, head), in order, chunk by chunk.
  const int units = 2 * p.kv_heads, workers = static_cast<int>(gridDim.x) - 1 - p.row_workers;
  if (p.ragged) sum_up(p, true, s_sums);
  const long long all = (p.ragged ? s_sums[p.count] : static_cast<long long>(p.count) * p.chunks) * units;
  const long long end = all * (worker - p.row_workers + 1) / workers;
  for (long long item = all * (worker - p.row_workers) / workers; item < end;) {
    const long long which = item / units;
    const int u_first = static_cast<int>(item - which * units);
    const int u_end = static_cast<int>(min(static_cast<long long>(units), u_first + (end - item)));
    item += u_end - u_first;
    const int b = p.ragged ? sequence_of(s_sums, p.count, static_cast<int>(which)) : static_cast<int>(which / p.chunks);
    const int chunk = static_cast<int>(which - (p.ragged ? s_sums[b] : static_cast<long long>(b) * p.chunks));
    const Rows rows = rows_of(p, span_of(p, b), chunk);
    if (rows.live <= 0) continue;
    __syncthreads();  // the last chunk's rows are done with
    for (int i = tid; i < 3 * kChunk; i += kThreads) (&s_top[0][0])[i] = 0u;
    prepare_rows(p, b, rows, freq, pair, pair_group, s_at, s_block, s_trig);
    __syncthreads();

    const int live = rows.live, lead = rows.p0 & (kChunk - 1);  // rows lie `lead` into the chunk
    const int held = rows.p0 & ((1 << p.block_log2) - 1);       // positions that the first row's block has already
    const bool real0 = s_at[0] >= 0;
    const bool one = (1 << p.block_log2) >= kWarpRows;  // a warp's rows share a block
    auto row_of = [&](int i) { return warp * kWarpRows + i * P::kHeads + my.sub - lead; };  // among the live ones, or outside
    auto block_of = [&](int r) { return (lead + r) >> p.block_log2; };
    const int block0 = block_of(0);
    auto issue = [&](int u, int stage) {
      if (u < u_end) {
        const uint16_t* src = (u >= p.kv_heads ? p.v_new : p.k_new) + rows.row0 * p.kv_row +
                              static_cast<long long>(u >= p.kv_heads ? u - p.kv_heads : u) * D;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int r = row_of(i);
          if (r >= 0 && r < live) {
            cp_async16(smem_addr(ring + (stage * kPasses + i) * 2 * kThreads), src + r * p.kv_row + my.first);
            cp_async16(smem_addr(ring + ((stage * kPasses + i) * 2 + 1) * kThreads), src + r * p.kv_row + my.second);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue(u_first + i, i);
    int stage = 0;
    int turn = 0;
    for (int u = u_first; u < u_end; ++u) {
      const bool is_v = u >= p.kv_heads;
      const int head = is_v ? u - p.kv_heads : u;
      float* scales = (is_v ? p.v_scale : p.k_scale) + head * p.scale_head;
      uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + head * p.head_stride;
      float was = 0.f;
      if (held > 0 && real0) was = scales[s_block[0]];
      unsigned* tops = s_top[turn];
      issue(u + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      cp_async_wait_group<kStages - 1>();
      unsigned long long x[kPasses][8];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int r = row_of(i);
        uint4 first = make_uint4(0u, 0u, 0u, 0u), second = first;
        if (r >= 0 && r < live) {
          first = ring[(stage * kPasses + i) * 2 * kThreads];
          second = ring[((stage * kPasses + i) * 2 + 1) * kThreads];
        }
        if (!is_v && my.turns) {
          const int look = min(max(r, 0), live - 1);
          my.look(s_trig + look * p.half, s_trig + (live + look) * p.half);
          my.turn(first, second, x[i]);
        } else {
          P::unpack(first, second, x[i]);
        }
        const float t = magnitude_two(x[i]);
        top = one ? fmaxf(top, t) : t;
        if (!one) {
#pragma unroll
          for (int d = 1; d < P::kDuos; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
          if (my.duo == 0 && r >= 0 && r < live) atomicMax(&tops[block_of(r)], __float_as_uint(top));
        }
      }
      if (one) {  // (rows outside are zeros)
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        if (lane == 0) atomicMax(&tops[(warp * kWarpRows) >> p.block_log2], __float_as_uint(top));
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
      __syncthreads();
      if (tid < kChunk) s_top[turn == 0 ? 2 : turn - 1][tid] = 0u;  // the head's after the next: nobody looks there any more, nor yet
      turn = turn == 2 ? 0 : turn + 1;
      bool keeps;
      float scale = 0.f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int r = row_of(i);
        if (!one || i == 0) {
          const int block = (warp * kWarpRows + (one ? 0 : i * P::kHeads + my.sub)) >> p.block_log2;
          scale = scale_for(tops[block], held > 0 && block == block0, was, keeps);
        }
        if (r < 0 || r >= live || s_at[r] < 0) continue;
        *reinterpret_cast<uint2*>(cache + s_at[r] + my.first) = coded_two(x[i], scale);
        *reinterpret_cast<uint2*>(cache + s_at[r] + my.second) = coded_two(x[i] + 4, scale);
        if (my.duo == 0 && !keeps && (r == 0 || block_of(r) != block_of(r - 1))) scales[s_block[r]] = scale;
      }
      if (held > 0 && real0) {
        scale = scale_for(tops[block0], true, was, keeps);
        if (!keeps) {  // what the block has goes to the larger scale
          for (int i = warp * P::kHeads + my.sub; i < held; i += kWarps * P::kHeads) {
            uint8_t* at = cache + s_at[0] - (held - i) * p.slot_stride;
            for (int from : {my.first, my.second}) {
              uint2* piece = reinterpret_cast<uint2*>(at + from);
              *piece = recoded(*piece, was / scale);
            }
          }
        }
      }
    }
  }
}

int check(const w4g128_append_args* a) {
  if (a == nullptr || a->k_new == nullptr || a->v_new == nullptr || a->k_cache == nullptr || a->v_cache == nullptr ||
      a->page_table == nullptr || a->row_offsets == nullptr || a->lens == nullptr ||
      (a->q == nullptr) != (a->q_out == nullptr) || (a->q == nullptr) != (a->q_heads == 0))
    return W4G128_ERR_INVALID_ARG;
  if ((a->block == 0) != (a->k_scale == nullptr) || (a->block == 0) != (a->v_scale == nullptr) ||
      (a->rot_dim == 0) != (a->freqs == nullptr))
    return W4G128_ERR_INVALID_ARG;
  if (a->rows < 1 || a->rows > (1 << 20) || a->count < 1 || a->count > W4G128_MAX_SEQUENCES || a->max_new < 1 ||
      a->max_new > (1 << 20) || a->interleaved < 0 || a->interleaved > 1 ||
      (a->q != nullptr && a->q == a->q_out && a->q_row != a->q_out_row))
    return W4G128_ERR_INVALID_ARG;
  if (a->kv_heads < 1 || a->kv_heads > 256 || a->q_heads < 0 || a->q_heads > 4096 ||
      (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256) || a->rot_dim < 0 || a->rot_dim > a->head_dim ||
      a->rot_dim % 16 != 0)
    return W4G128_ERR_SHAPE;
  if (a->pages < 1 || a->page_size < 16 || a->page_size % 16 != 0 || a->max_len < 1 || a->max_len > (1 << 24))
    return W4G128_ERR_SHAPE;
  if (a->block != 0 && (a->block < 0 || a->block > kChunk || (a->block & (a->block - 1)) != 0 || a->page_size % a->block != 0))
    return W4G128_ERR_SHAPE;
  const long long dim = a->head_dim;
  if ((a->q && (a->q_row < a->q_heads * dim || a->q_out_row < a->q_heads * dim)) || a->kv_row < a->kv_heads * dim ||
      a->slot_stride < dim || a->page_stride < dim || a->head_stride < dim ||
      a->table_row < (a->max_len - 1) / a->page_size + 1)
    return W4G128_ERR_SHAPE;
  if (a->block != 0 && (a->scale_page < a->page_size / a->block || a->scale_head < a->page_size / a->block))
    return W4G128_ERR_SHAPE;
  auto off = [](const void* q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0; };
  if (off(a->q, 16) || off(a->q_out, 16) || off(a->k_new, 16) || off(a->v_new, 16) || off(a->k_cache, 16) ||
      off(a->v_cache, 16) || off(a->k_scale, 4) || off(a->v_scale, 4) || off(a->freqs, 8) || off(a->page_table, 4) ||
      off(a->row_offsets, 4) || off(a->lens, 4))
    return W4G128_ERR_ALIGN;
  for (long long v : {a->q_row, a->q_out_row, a->kv_row})
    if (v % 8 != 0) return W4G128_ERR_ALIGN;
  for (long long v : {a->page_stride, a->slot_stride, a->head_stride})
    if (v % (a->block != 0 ? 16 : 8) != 0) return W4G128_ERR_ALIGN;
  return W4G128_OK;
}

template <int D>
cudaError_t launch(cudaLaunchConfig_t& cfg, Params& p) {
  p.chunks = (p.max_new + kChunk - 2) / kChunk + 1;
  cfg.blockDim = dim3(kThreads);
  // A warp for each head while there are few rows: up to 64 of up to 32 sequences, 8 of
  // one, in a bf16 cache (16 of 4 rows, 32 + 2 x 8 heads of 128: 3.5 us, and 3.8 row by
  // row; 64 of one 4.6 and 3.8; one of 8 3.4 and 3.8; of 16 4.7 and 3.7; 256 of one 11.5
  // and 4.0); in 8 bits always but for few sequences of more than 4 rows (one of 4 3.7 us,
  // and 3.9 by blocks; 4 of 8 5.3 and 4.1; 8 of 8 5.4 and 5.1; 16 of 8 6.6 and 7.5; 256 of
  // one 12.5 and 44).
  const bool few = p.max_new <= kFewRows && (p.block_log2 < 0 ? p.count <= 32 && p.max_new <= 8 && p.count * p.max_new <= 64
                                                              : p.max_new <= 4 || p.count > 8);
  if (few) {
    const int units = 2 * p.kv_heads + p.q_heads;
    cfg.gridDim = dim3(p.chunks, (units + kThreads / 32 - 1) / (kThreads / 32), p.count + 1);  // (the first CTA looks for errors)
    cfg.dynamicSmemBytes = static_cast<size_t>(2 * kFewRows) * p.half * sizeof(float);
    return cudaLaunchKernelEx(&cfg, append_few_kernel<D>, p);
  }
  // Row by row: a part of a row's heads at a time, while their number fits.
  constexpr int kHeads = kRowBatch * Duo<D>::kHeads;
  const int heads = p.q_heads + (p.block_log2 < 0 ? 2 * p.kv_heads : 0);
  const long long rows = static_cast<long long>(p.count) * p.max_new;
  const int parts = std::max(1, (heads + kHeads - 1) / kHeads);
  // Fewer rows than count max_new: each CTA first adds the sequences' up, so that all share
  // what there is (a prompt of 8191 beside 63 single tokens into bf16 36.7 us, by max_new
  // 266; into blocks of 16 48 and 1356; where all have max_new that costs up to 1.2 us: 256
  // of one row 4.0 without, 5.2 with it).
  p.ragged = rows > p.rows ? 1 : 0;
  p.by_new = divisor(p.max_new);
  p.by_parts = divisor(parts);  // (at most 2^20 rows of 576 parts)
  p.row_items = p.ragged ? 0 : static_cast<unsigned>(rows * parts);
  if (p.block_log2 < 0) {
    cfg.gridDim = dim3(1 + kWorkers);
    return cudaLaunchKernelEx(&cfg, append_rows_kernel<D>, p);
  }
  const int stages = kChunk * D * 2 * kBlockStages;
  const int most = stages + kChunk * D * static_cast<int>(sizeof(float));
  const cudaError_t e = cudaFuncSetAttribute(append_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  // A value of k or v costs three times a query's (a prompt of 8191, 32 + 2 x 8 heads of
  // 128, 64 rotated pairs: 32.6 us, with 2.5 times 37.6, with 3.5 times 34.3).
  const long long kv_work = 3 * 2 * p.kv_heads;
  p.row_workers = p.q_heads == 0 ? 0 : static_cast<int>(std::min<long long>(kWorkers - 1, 1 + kWorkers * p.q_heads * 2 / (2 * p.q_heads + kv_work)));
  cfg.gridDim = dim3(1 + kWorkers);
  cfg.dynamicSmemBytes = stages + 2 * kChunk * p.half * static_cast<int>(sizeof(float));
  return cudaLaunchKernelEx(&cfg, append_many_kernel<D>, p);
}

}  // namespace
}  // namespace w4g128

extern "C" {

size_t w4g128_append_workspace_bytes(const w4g128_append_args* args) {
  return w4g128::check(args) == W4G128_OK ? w4g128::kWorkspace : 0;
}

int w4g128_append(const w4g128_append_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace w4g128;
  int rc = check(a);
  if (rc != W4G128_OK) return rc;
  if (ws == nullptr) return W4G128_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0) return W4G128_ERR_ALIGN;
  if (ws_bytes < kWorkspace) return W4G128_ERR_WORKSPACE;
  rc = fault_hook();
  if (rc != W4G128_OK) return rc;
  if (!device_is_sm103()) return W4G128_ERR_DEVICE;
  Params p;
  p.q = a->q; p.q_out = a->q_out; p.k_new = a->k_new; p.v_new = a->v_new; p.k_cache = a->k_cache; p.v_cache = a->v_cache;
  p.k_scale = a->k_scale; p.v_scale = a->v_scale; p.freqs = a->freqs;
  p.table = a->page_table; p.offsets = a->row_offsets; p.lens = a->lens;
  p.q_row = a->q_row; p.q_out_row = a->q_out_row; p.kv_row = a->kv_row;
  p.page_stride = a->page_stride; p.slot_stride = a->slot_stride; p.head_stride = a->head_stride;
  p.scale_page = a->scale_page; p.scale_head = a->scale_head; p.table_row = a->table_row;
  p.rows = a->rows; p.count = a->count; p.q_heads = a->q_heads; p.kv_heads = a->kv_heads; p.half = a->rot_dim / 2;
  p.interleaved = a->interleaved; p.pages = a->pages; p.max_len = a->max_len; p.max_new = a->max_new;
  p.block_log2 = -1;
  for (int v = a->block; v > 0; v >>= 1) ++p.block_log2;
  p.by_page = divisor(a->page_size);
  p.by_half = divisor(std::max(p.half, 1));
  p.by_kv = divisor(a->kv_heads);
  p.status = static_cast<unsigned long long*>(ws);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a->head_dim == 64 ? launch<64>(cfg, p) : a->head_dim == 128 ? launch<128>(cfg, p) : launch<256>(cfg, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
