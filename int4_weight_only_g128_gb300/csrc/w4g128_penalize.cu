// Penalties, biases and masks on logits (w4g128_penalize), in one launch.
//
// A row's vocabulary is cut into slices, a CTA each.  In shared memory a CTA has a
// word for each of its tokens: the times it occurs in the answer, and in the top bit
// whether it occurs at all.  Every CTA reads the whole history (from the L2: 131 KB
// for 32771 tokens) and counts its own tokens by additions of whole numbers, whose
// order does not matter.  (Each CTA its part of the history, counted where a token
// belongs by additions to the shared memory of a cluster's CTAs, took 19.8 us where
// this takes 5.5: the frequent tokens' additions wait for one another across the
// cluster.)  In the same way a list's biases leave their places in the list, of which
// the largest stays.  Then the CTA goes over its slice, 8 tokens a thread at a time;
// the logits and mask words are on their way while the tokens are counted.  A chain of
// loads (settings, history) bounds one row; 16 rows of 248320 with 4099 tokens and
// 300 biases take 11.0 us, 1.5 TB/s (its bytes alone take 2.4 us), and 4.7 without
// the counting, a chain of loads, additions and barriers.  Registers (59 a thread) leave
// two CTAs of 512 threads to an SM, 304 at once: its 496 run in two waves, the second
// nearly as long as the first.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "w4g128_internal.h"
#include "w4g128_ops.h"
#include "w4g128_ptx.cuh"

namespace w4g128 {
namespace {

constexpr int kBatch = 2;  // loads of 4 tokens on their way at once
constexpr int kMostHistory = 1 << 30;
constexpr int kNear = 512;
constexpr int kMostBias = 65535;
constexpr uint32_t kSeen = 0x80000000u;
constexpr int kMostSlice = 8192;

struct Params {
  const uint16_t* logits;
  uint16_t* out;
  const int* history;
  const long long* history_start;
  const int *history_len, *prompt_len;
  const float *repetition, *presence, *frequency;
  const int* bias_tokens;
  const float* bias_values;
  const int* bias_offsets;
  const uint32_t* mask;
  long long row_stride, out_stride, mask_row, history_size;
  int bias_size, vocab, slice;  // slice: tokens a CTA, a multiple of 8
};

__device__ __forceinline__ float bf16_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ uint32_t f_bf16(float x) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

template <int T>
__global__ void __launch_bounds__(T) penalize_kernel(const __grid_constant__ Params p) {
  constexpr int kAhead = 8192 / 8 / T;  // pieces of 8 logits that a thread asks for ahead
  __shared__ float s_bias[kNear];       // a list's first values
  extern __shared__ __align__(16) uint32_t s_words[];  // [slice] counts, if any; [slice] 16-bit places in the list, if any
  const int tid = threadIdx.x, row = blockIdx.y;
  const int rank = blockIdx.x;
  const bool may_count = p.history != nullptr, may_bias = p.bias_tokens != nullptr;
  uint32_t* counts = s_words;
  uint32_t* places = may_count ? s_words + p.slice : s_words;

  if (may_count)
    for (int i = tid * 4; i < p.slice; i += T * 4) *reinterpret_cast<uint4*>(counts + i) = make_uint4(0u, 0u, 0u, 0u);
  if (may_bias)
    for (int i = tid * 4; i < p.slice / 2; i += T * 4) *reinterpret_cast<uint4*>(places + i) = make_uint4(0u, 0u, 0u, 0u);
  grid_dependency_wait();

  // Pieces of 8 tokens start where the row's logits are 16-byte aligned.
  const uint16_t* in = p.logits + row * p.row_stride;
  uint16_t* out = p.out + row * p.out_stride;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(in) & 15u) / 2);  // piece 0 starts at token -shift
  const bool out_whole = ((reinterpret_cast<uintptr_t>(out) & 15u) / 2) == static_cast<unsigned>(shift);
  const int first = rank * p.slice - shift;  // this CTA's first token
  const uint32_t* mask = p.mask != nullptr ? p.mask + row * p.mask_row : nullptr;
  const int words = (p.vocab + 31) / 32;
  uint4 ahead[kAhead];
  uint32_t allowed_ahead[kAhead];
  auto load = [&](int t0, uint4& v, uint32_t& allowed) {
    v = make_uint4(0u, 0u, 0u, 0u);
    allowed = 0xFFu;
    if (t0 >= 0 && t0 + 8 <= p.vocab) {
      v = *reinterpret_cast<const uint4*>(in + t0);
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (t0 + e >= 0 && t0 + e < p.vocab) w[e / 2] |= static_cast<uint32_t>(in[t0 + e]) << (e & 1) * 16;
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (mask != nullptr) {  // the 8 bits from t0 on (of a token outside: any)
      const int w0 = t0 >> 5;
      const uint32_t lo = w0 >= 0 && w0 < words ? mask[w0] : 0u;
      uint32_t hi = 0u;
      if ((t0 & 31) > 24 && w0 + 1 < words) hi = mask[w0 + 1];
      allowed = __funnelshift_r(lo, hi, t0 & 31) & 0xFFu;
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int at = (i * T + tid) * 8;
    if (at < p.slice && first + at < p.vocab) load(first + at, ahead[i], allowed_ahead[i]);
  }

  float repetition = 1.f, presence = 0.f, frequency = 0.f;
  if (p.repetition != nullptr) repetition = p.repetition[row];
  if (p.presence != nullptr) presence = p.presence[row];
  if (p.frequency != nullptr) frequency = p.frequency[row];
  const float inverse = 1.f / repetition;
  int b0 = 0, listed = 0, listed_token = -1;
  float listed_value = 0.f;
  if (may_bias) {  // this thread's first entry, on its way while the history is counted
    b0 = max(p.bias_offsets[row], 0);
    // (both ends from 0 on before they are subtracted: an end near -2^31 would wrap)
    listed = min(max(max(min(p.bias_offsets[row + 1], p.bias_size), 0) - b0, 0), kMostBias);
    if (tid < listed) {
      listed_token = p.bias_tokens[b0 + tid];
      listed_value = p.bias_values[b0 + tid];
    }
  }
  if (may_count) {
    long long begin = p.history_start != nullptr ? p.history_start[row] : 0;
    const int given = min(max(p.history_len[row], 0), kMostHistory);
    int prompt = p.prompt_len != nullptr ? p.prompt_len[row] : 0;
    // (what lies outside the buffer is not read)
    const int skip = begin >= 0 ? 0 : begin < -given ? given : static_cast<int>(-begin);
    begin += skip;
    const int len = static_cast<int>(min(static_cast<long long>(given - skip), max(p.history_size - begin, 0ll)));
    prompt = prompt > skip ? prompt - skip : 0;
    const int* tokens = p.history + begin;
    const int whole = min(len, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(tokens) & 15u)) / 4 & 3u));
    // (a place before the row's first token, for a token below 0, is never written out)
    const unsigned mine = static_cast<unsigned>(max(min(p.slice, p.vocab - first), 0));  // (the last slice may lie behind)
    __syncthreads();
    auto count = [&](int t, bool asked) {
      const unsigned at = static_cast<unsigned>(t) - static_cast<unsigned>(first);
      if (at < mine) {
        if (asked) atomicOr(&counts[at], kSeen);
        else atomicAdd(&counts[at], 1u);
      }
    };
    if (tid < whole) count(tokens[tid], tid < prompt);  // up to a 16-byte boundary
    const int4* four = reinterpret_cast<const int4*>(tokens + whole);
    const int quads = (len - whole) / 4;
    for (int q0 = tid & ~31; q0 < quads; q0 += kBatch * T) {
      int4 t[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (q0 + j * T >= quads) break;  // (of the warp)
        const int q = q0 + j * T + (tid & 31);
        t[j] = q < quads ? __ldg(four + q) : make_int4(-8, -8, -8, -8);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (q0 + j * T >= quads) break;
        const int left = prompt - whole - 4 * (q0 + j * T + (tid & 31));  // of the prompt, from here on
        count(t[j].x, left > 0);
        count(t[j].y, left > 1);
        count(t[j].z, left > 2);
        count(t[j].w, left > 3);
      }
    }
    const int rest = whole + 4 * quads + tid;
    if (rest < len) count(tokens[rest], rest < prompt);
  }
  if (may_bias) {  // each CTA looks for its own tokens
    if (!may_count) __syncthreads();
    for (int i = tid; i < listed; i += T) {
      const int t = i == tid ? listed_token : p.bias_tokens[b0 + i];
      const unsigned at = static_cast<unsigned>(t) - static_cast<unsigned>(first);
      if (i < kNear) s_bias[i] = i == tid ? listed_value : p.bias_values[b0 + i];
      if (t >= 0 && t < p.vocab && at < static_cast<unsigned>(p.slice)) {
        uint32_t* word = places + at / 2;
        const unsigned up = (at & 1u) * 16u;
        uint32_t seen = *word;
        while (((seen >> up) & 0xFFFFu) < static_cast<uint32_t>(i + 1)) {
          const uint32_t prev = atomicCAS(word, seen, (seen & ~(0xFFFFu << up)) | static_cast<uint32_t>(i + 1) << up);
          if (prev == seen) break;
          seen = prev;
        }
      }
    }
  }
  if (may_count || may_bias) __syncthreads();

  auto finish = [&](int at, const uint4& v, uint32_t allowed) {
    const int t0 = first + at;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[8] = {}, place[4] = {}, counted = 0u, placed = 0u;
    if (may_count) {
      const uint4 a = *reinterpret_cast<const uint4*>(counts + at), b = *reinterpret_cast<const uint4*>(counts + at + 4);
      c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
      c[4] = b.x; c[5] = b.y; c[6] = b.z; c[7] = b.w;
      counted = a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w;
    }
    if (may_bias) {
      const uint4 a = *reinterpret_cast<const uint4*>(places + at / 2);
      place[0] = a.x; place[1] = a.y; place[2] = a.z; place[3] = a.w;
      placed = a.x | a.y | a.z | a.w;
    }
    if ((counted | placed) != 0u) {  // few pieces have a token of the history or of the list
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[e] = bf16_f((w[e / 2] >> (e & 1) * 16) & 0xFFFFu);
        const float times = static_cast<float>(c[e] & ~kSeen);
        float x = z[e] * (z[e] > 0.f ? inverse : repetition);
        x = __fsub_rn(x, __fmul_rn(frequency, times));
        x = __fsub_rn(x, times > 0.f ? presence : 0.f);
        if (c[e] != 0u) z[e] = x;
      }
      if (placed != 0u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t where = (place[e / 2] >> (e & 1) * 16) & 0xFFFFu;
          if (where != 0u) z[e] = __fadd_rn(z[e], where <= kNear ? s_bias[where - 1] : p.bias_values[b0 + static_cast<int>(where) - 1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f_bf16(z[2 * e]) | f_bf16(z[2 * e + 1]) << 16;
    }
    if (allowed != 0xFFu) {  // -inf
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t keep = ((allowed >> 2 * e & 1u) ? 0x0000FFFFu : 0u) | ((allowed >> 2 * e & 2u) ? 0xFFFF0000u : 0u);
        w[e] = (w[e] & keep) | (0xFF80FF80u & ~keep);
      }
    }
    if (out_whole && t0 >= 0 && t0 + 8 <= p.vocab) {
      *reinterpret_cast<uint4*>(out + t0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (t0 + e >= 0 && t0 + e < p.vocab) out[t0 + e] = static_cast<uint16_t>(w[e / 2] >> (e & 1) * 16);
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int at = (i * T + tid) * 8;
    if (at < p.slice && first + at < p.vocab) finish(at, ahead[i], allowed_ahead[i]);
  }
  for (int at = (kAhead * T + tid) * 8; at < p.slice && first + at < p.vocab; at += T * 8) {
    uint4 v;
    uint32_t allowed;
    load(first + at, v, allowed);
    finish(at, v, allowed);
  }
}

int check(const w4g128_penalize_args* a) {
  if (a == nullptr || a->logits == nullptr || a->out == nullptr) return W4G128_ERR_INVALID_ARG;
  if ((a->history != nullptr && a->history_len == nullptr) ||
      (a->bias_tokens != nullptr && (a->bias_values == nullptr || a->bias_offsets == nullptr)))
    return W4G128_ERR_INVALID_ARG;
  if (a->rows < 1 || a->rows > W4G128_MAX_SAMPLE_ROWS || a->history_size < 0 || a->bias_size < 0 ||
      (a->out == a->logits && a->out_stride != a->row_stride))
    return W4G128_ERR_INVALID_ARG;
  if (a->vocab < 1 || a->vocab > W4G128_MAX_VOCAB || a->row_stride < a->vocab || a->out_stride < a->vocab ||
      (a->mask != nullptr && a->mask_row != 0 && a->mask_row < (a->vocab + 31) / 32))
    return W4G128_ERR_SHAPE;
  auto off = [](const void* q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0; };
  if (off(a->logits, 2) || off(a->out, 2) || off(a->history_start, 8)) return W4G128_ERR_ALIGN;
  const void* words[] = {a->history, a->history_len, a->prompt_len, a->repetition, a->presence, a->frequency,
                         a->bias_tokens, a->bias_values, a->bias_offsets, a->mask};
  for (const void* q : words)
    if (off(q, 4)) return W4G128_ERR_ALIGN;
  return W4G128_OK;
}

}  // namespace
}  // namespace w4g128

extern "C" {

int w4g128_penalize(const w4g128_penalize_args* a, void* stream) {
  using namespace w4g128;
  int rc = check(a);
  if (rc != W4G128_OK) return rc;
  rc = fault_hook();
  if (rc != W4G128_OK) return rc;
  if (!device_is_sm103()) return W4G128_ERR_DEVICE;
  Params p;
  p.logits = a->logits; p.out = a->out;
  p.history = a->history_size > 0 ? a->history : nullptr;
  p.history_start = a->history_start; p.history_len = a->history_len; p.prompt_len = a->prompt_len;
  p.repetition = a->repetition; p.presence = a->presence; p.frequency = a->frequency;
  p.bias_tokens = a->bias_size > 0 ? a->bias_tokens : nullptr;
  p.bias_values = a->bias_values; p.bias_offsets = a->bias_offsets; p.mask = a->mask;
  p.row_stride = a->row_stride; p.out_stride = a->out_stride; p.mask_row = a->mask_row; p.history_size = a->history_size;
  p.bias_size = a->bias_size; p.vocab = a->vocab;
  // Slices of 8192 tokens, or of 2048 where that makes no more CTAs than two an SM, all at
  // once (one row of 32000: 3.3 us, and 4.0 with 8192; 16 rows of 248320: 11.0 us with 8192
  // in two waves, 14.5 with 4096 in four and 22 with 2048 in seven).  Long histories take
  // more threads (one row with 32771 tokens: 5.5 us, and 8.5 with 512; with 613 tokens 3.4
  // and 3.3, 16 rows with 4099 15.7 and 11.0).
  p.slice = static_cast<long long>(a->rows) * ((a->vocab + 7 + 2047) / 2048) <= 304 ? 2048 : kMostSlice;
  const int ctas = (a->vocab + 7 + p.slice - 1) / p.slice;
  const bool wide = a->history_size / a->rows > 8192;
  const size_t shared = (p.history ? 4 : 0) * static_cast<size_t>(p.slice) + (p.bias_tokens ? 2 : 0) * static_cast<size_t>(p.slice);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, a->rows);
  cfg.blockDim = dim3(wide ? 1024 : 512);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = wide ? penalize_kernel<1024> : penalize_kernel<512>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 6 * kMostSlice);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}

}  // extern "C"
