// Rotated queries, and rotated keys and values put into a paged cache
// (w4g128_append), in one launch.
//
// A CTA takes 64 positions of a sequence at a multiple of 64 (so whole blocks of
// an 8-bit cache, whose scale all of a block's rows decide) and some of the heads
// of q, k and v.  It computes the cosines and sines of its rows once, for all its
// heads.  A head's rows are pieces of 8 values, 16 bytes a lane; the other half of
// a rotated pair is in another lane of the same warp (or the same piece), so it
// comes by shuffle and every byte is read and written once.
//   * up to 16 new rows a sequence (a decode or verify step): a warp for each
//     head.  What takes time is the chain length -> rows -> cosines -> store.
//   * prompts: the 8 warps share a head's rows, kept in registers between the
//     maximum that decides an 8-bit block's scale and the codes.
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
  Divisor by_page, by_half;
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

template <int D, int TEAM>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Params p) {
  constexpr int kPieces = D / 8;       // of a row
  constexpr int kRows = 32 / kPieces;  // rows of a warp at once
  constexpr int kMaxLive = TEAM == 1 ? kFewRows : kChunk;
  constexpr int kPasses = kMaxLive / (kRows * TEAM);
  constexpr int kTeams = kThreads / 32 / TEAM;
  extern __shared__ __align__(16) float s_trig[];    // [live rows][half] cosines, then sines
  __shared__ long long s_at[kChunk], s_block[kChunk];  // a row's slot and scale in the caches; -1: no page
  __shared__ unsigned s_top[3][kTeams][kChunk];        // a block's magnitude, of three heads in turn
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);
  const int team = warp / TEAM, member = warp % TEAM;

  grid_dependency_wait();
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0 && blockIdx.z == 0) check_all(p);
    return;
  }
  const int b = blockIdx.z;
  const int pair_group = p.half > 0 ? tid / p.by_half : 0;
  const int pair = tid - pair_group * p.half;
  double freq = 0.0;
  if (p.half > 0) freq = p.freqs[pair];
  const Span s = span_of(p, b);
  if (!s.ok || s.n == 0) return;
  const int c0 = (s.first & ~(kChunk - 1)) + static_cast<int>(blockIdx.x) * kChunk;
  const int p0 = max(c0, s.first), p1 = min(c0 + kChunk, s.len);
  const int live = p1 - p0;
  if (live <= 0) return;
  const int row0 = s.first_row + p0 - s.start;

  for (int i = tid; i < 3 * kTeams * kChunk; i += kThreads) (&s_top[0][0][0])[i] = 0u;
  if (tid < live) {
    const int pos = p0 + tid, page = pos / p.by_page;
    const int slot = pos - page * static_cast<int>(p.by_page.d);
    const int id = p.table[static_cast<long long>(b) * p.table_row + page];
    const bool ok = id >= 0 && id < p.pages;
    s_at[tid] = ok ? id * p.page_stride + slot * p.slot_stride : -1;
    s_block[tid] = id * p.scale_page + (p.block_log2 >= 0 ? slot >> p.block_log2 : 0);
  }
  if (p.half > 0) {
    const int groups = kThreads / p.by_half;
    if (pair_group < groups) {
      double turns = freq * 0.15915494309189533576888376337251;  // 1 / (2 pi)
      turns -= floor(turns);
      const unsigned long long step = __double2ull_rz(turns * 18446744073709551616.0);
      for (int r = pair_group; r < live; r += groups) {
        const unsigned long long full = static_cast<unsigned long long>(p0 + r) * step;
        const uint32_t turn = static_cast<uint32_t>((full + 0x80000000ull) >> 32);  // 2^-32 turns
        const uint32_t quarter = (turn + 0x20000000u) >> 30;
        const float x = static_cast<float>(static_cast<int>(turn - (quarter << 30))) * 0x1p-31f;  // half turns
        float sn, cs;
        sincospif(x, &sn, &cs);
        const float c = (quarter & 1u) ? -sn : cs, d = (quarter & 1u) ? cs : sn;
        s_trig[r * p.half + pair] = (quarter & 2u) ? -c : c;
        s_trig[(live + r) * p.half + pair] = (quarter & 2u) ? -d : d;
      }
    }
  }
  __syncthreads();

  const int sub = lane / kPieces, piece = lane % kPieces;
  const int turn_pieces = p.half / 8;  // of one side of the pairs
  auto row_of = [&](int pass) { return (pass * TEAM + member) * kRows + sub; };
  auto rotate = [&](const uint4& raw, int r, float (&x)[8]) {
    unpack(raw, x);
    if (p.half == 0) return;
    if (p.interleaved) {
      if (piece >= 2 * turn_pieces || r >= live) return;
      const float4 c = *reinterpret_cast<const float4*>(&s_trig[r * p.half + piece * 4]);
      const float4 d = *reinterpret_cast<const float4*>(&s_trig[(live + r) * p.half + piece * 4]);
      const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], e = x[2 * i + 1];
        x[2 * i] = fmaf(a, cs[i], -(e * sn[i]));
        x[2 * i + 1] = fmaf(e, cs[i], a * sn[i]);
      }
      return;
    }
    const bool second = piece >= turn_pieces;
    const int from = piece < turn_pieces ? lane + turn_pieces : piece < 2 * turn_pieces ? lane - turn_pieces : lane;
    uint4 other;
    other.x = __shfl_sync(~0u, raw.x, from);
    other.y = __shfl_sync(~0u, raw.y, from);
    other.z = __shfl_sync(~0u, raw.z, from);
    other.w = __shfl_sync(~0u, raw.w, from);
    if (piece >= 2 * turn_pieces || r >= live) return;
    float y[8];
    unpack(other, y);
    const int i0 = (second ? piece - turn_pieces : piece) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c = *reinterpret_cast<const float4*>(&s_trig[r * p.half + i0 + 4 * h]);
      const float4 d = *reinterpret_cast<const float4*>(&s_trig[(live + r) * p.half + i0 + 4 * h]);
      const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * h + i;
        x[e] = second ? fmaf(x[e], cs[i], y[e] * sn[i]) : fmaf(x[e], cs[i], -(y[e] * sn[i]));
      }
    }
  };
  auto packed = [&](const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  };

  const int units = 2 * p.kv_heads + p.q_heads;
  int turn = 0;
  for (int u0 = blockIdx.y * kTeams; u0 < units; u0 += gridDim.y * kTeams) {
    const int u = u0 + team;
    if (TEAM == 1 && u >= units) break;  // (one head a team: a larger team is all of the CTA)
    const bool is_q = u >= 2 * p.kv_heads, is_v = !is_q && u >= p.kv_heads;
    const int head = is_q ? u - 2 * p.kv_heads : is_v ? u - p.kv_heads : u;
    const uint16_t* src = is_q ? p.q + static_cast<long long>(row0) * p.q_row
                               : (is_v ? p.v_new : p.k_new) + static_cast<long long>(row0) * p.kv_row;
    const long long stride = is_q ? p.q_row : p.kv_row;
    src += static_cast<long long>(head) * D + piece * 8;
    uint4 raw[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = row_of(i);
      raw[i] = r < live ? *reinterpret_cast<const uint4*>(src + r * stride) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (is_q) {
      uint16_t* dst = p.q_out + static_cast<long long>(row0) * p.q_out_row + static_cast<long long>(head) * D + piece * 8;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (i * TEAM * kRows >= live) break;
        const int r = row_of(i);
        float x[8];
        rotate(raw[i], r, x);
        if (r < live) *reinterpret_cast<uint4*>(dst + r * p.q_out_row) = packed(x);
      }
      continue;
    }
    const long long in_slot = head * p.head_stride + piece * 8;
    if (p.block_log2 < 0) {
      uint16_t* cache = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + in_slot;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (i * TEAM * kRows >= live) break;
        const int r = row_of(i);
        float x[8];
        if (!is_v) rotate(raw[i], r, x);
        if (r < live && s_at[r] >= 0) *reinterpret_cast<uint4*>(cache + s_at[r]) = is_v ? raw[i] : packed(x);
      }
      continue;
    }

    // 8 bits: the magnitudes of the rows' blocks, then their scales and codes.
    float* scales = (is_v ? p.v_scale : p.k_scale) + head * p.scale_head;
    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + in_slot;
    const int held = p0 & ((1 << p.block_log2) - 1);  // positions that the first row's block has already
    const bool real0 = s_at[0] >= 0;
    float was = 0.f;
    if (held > 0 && real0) was = scales[s_block[0]];
    unsigned* tops = s_top[turn][team];
    const int block0 = (p0 - c0) >> p.block_log2;
    auto block_of = [&](int r) { return (p0 - c0 + r) >> p.block_log2; };
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i * TEAM * kRows >= live) break;
      const int r = row_of(i);
      float x[8];
      if (is_v) unpack(raw[i], x);
      else rotate(raw[i], r, x);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(x[e]);
        top = fmaxf(top, a < INFINITY ? a : 0.f);
      }
#pragma unroll
      for (int d = 1; d < kPieces; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      if (piece == 0 && r < live) atomicMax(&tops[block_of(r)], __float_as_uint(top));
    }
    if constexpr (TEAM == 1) __syncwarp();
    else __syncthreads();
    {  // the magnitudes of the head after the next: nobody looks at them any more, nor yet
      unsigned* later = s_top[turn == 0 ? 2 : turn - 1][team];
      for (int i = member * 32 + lane; i < kChunk; i += TEAM * 32) later[i] = 0u;
    }
    turn = turn == 2 ? 0 : turn + 1;
    // The scale of a row's block, and what turns values into codes.
    auto scale_for = [&](int block, bool& keeps) {
      const uint32_t top = tops[block];
      keeps = held > 0 && block == block0 && was > 0.f && __uint_as_float(top) <= kE4M3Max * was;
      return keeps ? was : exp2_of(fresh_exponent(top));
    };
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i * TEAM * kRows >= live) break;
      const int r = row_of(i);
      float x[8];
      if (is_v) unpack(raw[i], x);
      else rotate(raw[i], r, x);
      if (r >= live || s_at[r] < 0) continue;
      bool keeps;
      const float scale = scale_for(block_of(r), keeps);
      // (a scale that another program set need not be a power of two)
      const bool power = (__float_as_uint(scale) & 0x007FFFFFu) == 0u;
      const float inverse = 1.f / scale;
      uint32_t code[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a = x[2 * e], d = x[2 * e + 1];
        a = fabsf(a) < INFINITY ? (power ? a * inverse : a / scale) : NAN;
        d = fabsf(d) < INFINITY ? (power ? d * inverse : d / scale) : NAN;
        code[e] = to_e4m3x2(a, d);
      }
      *reinterpret_cast<uint2*>(cache + s_at[r]) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
      const bool leads = r == 0 || block_of(r) != block_of(r - 1);
      if (piece == 0 && leads && !keeps) scales[s_block[r]] = scale;
    }
    if (held > 0 && real0) {
      bool keeps;
      const float scale = scale_for(block0, keeps);
      if (!keeps) {  // what the block has goes to the larger scale
        const float factor = was / scale;
        for (int i = (member * 32 + lane) / kPieces; i < held; i += TEAM * kRows) {
          uint2* at = reinterpret_cast<uint2*>(cache + s_at[0] - (held - i) * p.slot_stride);
          const uint2 old = *at;
          uint32_t code[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t h = e4m3x2_to_half2(static_cast<uint16_t>((e < 2 ? old.x : old.y) >> (e & 1) * 16));
            float a, d;
            asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(a), "=f"(d) : "r"(h));
            code[e] = to_e4m3x2(a * factor, d * factor);
          }
          *at = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
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

template <int D, int TEAM>
cudaError_t launch(cudaLaunchConfig_t& cfg, const Params& p) {
  const int most = TEAM == 1 ? kFewRows : kChunk;
  cfg.dynamicSmemBytes = static_cast<size_t>(2 * most) * p.half * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(append_kernel<D, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             2 * kChunk * (D / 2) * static_cast<int>(sizeof(float)));
  if (e != cudaSuccess) return e;
  const int units = 2 * p.kv_heads + p.q_heads;
  const int chunks = (p.max_new + kChunk - 2) / kChunk + 1;  // that the new rows may touch
  int slices = (units + 7) / 8;
  if (TEAM > 1) {
    const long long ctas = static_cast<long long>(chunks) * p.count;
    slices = static_cast<int>(std::min<long long>(units, std::max<long long>(1, (608 + ctas - 1) / ctas)));
  }
  cfg.gridDim = dim3(chunks + 1, slices, p.count);  // (the last chunk's first CTA looks for errors)
  cfg.blockDim = dim3(kThreads);
  return cudaLaunchKernelEx(&cfg, append_kernel<D, TEAM>, p);
}

template <int D>
cudaError_t launch_dim(cudaLaunchConfig_t& cfg, const Params& p) {
  return p.max_new <= kFewRows ? launch<D, 1>(cfg, p) : launch<D, kThreads / 32>(cfg, p);
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
  p.status = static_cast<unsigned long long*>(ws);
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
