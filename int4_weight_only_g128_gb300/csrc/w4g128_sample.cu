// Token sampling (w4g128_sample): temperature, top-k, top-p, min-p and the
// draw itself, one launch, one read of the logits.
//
// A bf16 logit has at most 65536 values, so the row's whole distribution is a
// histogram over 16-bit keys ordered like the values, and every token with the
// same value has the same weight: the sort, the softmax and the cumulative sum
// over the vocabulary become a scan over bins.  One row is one cluster of 16, 8,
// 6 or 4 CTAs.  Each counts its slice of the row into its own 65536 16-bit
// counters (128 KB of shared memory; a slice has at most 65535 tokens) and marks
// the units of 8 bins that it touched, a few hundred of 8192 in an ordinary row.
// The touched units of all copies, in order, are cut evenly among the CTAs; each
// merges its run over distributed shared memory, weighs the bins and scans
// (count, mass).  The filters keep prefixes of the order, so
// each is one point of the scan that one thread finds and tells the cluster.
// The chosen bin and the rank within it lead back to the token: every CTA
// counts the bin in its slice once more, and the one that holds the rank finds
// the place.
//
// Masses are exact integers (weights as 62-bit fractions of the largest, sums
// in 128 bits): prefix sums agree to the bit whatever their order, so exactly
// one thread owns each crossing, and the cluster's size changes no result.
// FP64 runs at 2 operations a cycle and SM here, so the weights come from an
// fp32 pair evaluation (exp2_neg) instead: about 1e-14 relative, with 35
// full-rate operations a bin.
//
// Bound: latency.  A row of 248320 logits is 0.5 MB, 0.1 us of HBM; the chain
// load, count, merge, scan and five or six cluster barriers is what takes time.
// Measured, one row of 248320 with top-p (16 CTAs), 15.1 us a call: launch and
// clearing 1.4, counting 2.6, marks and largest 1.3, the run 1.6, merge and
// weights 1.5, scan 1.7, top-p 1.2, draw 1.4, search 2.0.  16 rows (6 CTAs each):
// 20.8 us, of which counting 6.4 (shared-memory atomics, 8 cycles a warp).
#include <cuda_runtime.h>

#include <cstdint>

#include "w4g128_ops.h"
#include "w4g128_internal.h"
#include "w4g128_ptx.cuh"

namespace w4g128 {
namespace {

typedef unsigned __int128 u128;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 65536;
constexpr int kUnit = 8;                  // bins that are marked, merged and handed out together
constexpr int kUnits = kBins / kUnit;
constexpr int kWords = kUnits / 32;       // of the marks
constexpr size_t kHistBytes = kBins * 2;  // 16-bit counters; later the weights of a long run
constexpr int run_units(int ctas) { return (kUnits + ctas - 1) / ctas; }  // at most
constexpr size_t smem_for(int ctas) { return kHistBytes + run_units(ctas) * kUnit * 4; }  // and a run's merged counts
constexpr uint32_t kMinusInf = 0x007Fu;  // key of -inf: what is not above it is never chosen
constexpr uint32_t kPlusInf = 0xFF80u;

// a slice: its share of the 16-byte vectors and the ragged ends of up to 7 tokens
constexpr bool slice_fits(int vocab, int ctas) { return (vocab / 8 + ctas - 1) / ctas * 8 + 14 <= 65535; }
static_assert(slice_fits(W4G128_MAX_VOCAB, 8), "a slice's count of one bin fits 16 bits");
static_assert(kWords % 32 == 0 && kWarps == 32, "a warp per 32 words of marks, in blocks of 32 words");
constexpr int kBlocks = 8;  // of 1024 vectors, a slice's at most
static_assert(65535 / 8 <= kBlocks * kThreads, "a slice's vectors");

// 2^(-j / 32) as unevaluated sums of two floats, by square roots of 1/2.
constexpr double root(double v) {
  double r = 1.0;
  for (int i = 0; i < 60; ++i) r = 0.5 * (r + v / r);  // Newton's iteration
  return r;
}
struct Table {
  float hi[32], lo[32];
};
constexpr Table make_table() {
  double half[5] = {};  // 2^(-1/2), 2^(-1/4), .. 2^(-1/32)
  half[0] = root(0.5);
  for (int i = 1; i < 5; ++i) half[i] = root(half[i - 1]);
  Table t = {};
  for (int j = 0; j < 32; ++j) {
    double v = 1.0;
    for (int i = 0; i < 5; ++i)
      if (j >> (4 - i) & 1) v *= half[i];
    t.hi[j] = static_cast<float>(v);
    t.lo[j] = static_cast<float>(v - static_cast<double>(t.hi[j]));
  }
  return t;
}
__constant__ Table c_table = make_table();

// The order-preserving key of a bf16 pattern; -0 becomes +0, NaN becomes 0.
__device__ __forceinline__ uint32_t key_of(uint32_t b) {
  if ((b & 0x7FFFu) > 0x7F80u) return 0u;
  if (b == 0x8000u) b = 0u;
  return (b & 0x8000u) ? (b ^ 0xFFFFu) : (b | 0x8000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  const uint32_t b = (key & 0x8000u) ? (key ^ 0x8000u) : (key ^ 0xFFFFu);
  return __uint_as_float(b << 16);
}

struct Pair {  // an unevaluated sum hi + lo, |lo| <= ulp(hi) / 2
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}

// 2^-y as a fraction of 2^62, for y = y.hi + y.lo >= 0 (0 from y = 62.5 on).
// y = k / 32 + r with |r| <= 1/64; 2^-r = e^z, z = -r ln 2, |z| <= 0.011, by
// the first six terms of its series (the next one is below 3e-15), the sum
// carried as a pair; times 2^(-(k mod 32) / 32) from the table, and shifted.
__device__ __forceinline__ uint64_t exp2_neg(Pair y, const float2* table) {
  if (!(y.hi < 62.5f)) return 0ull;
  const float kf = rintf(y.hi * 32.f);
  const int k = static_cast<int>(kf);
  const Pair r = two_sum(__fsub_rn(y.hi, kf * 0.03125f), y.lo);  // the difference is exact
  // ln 2 as a pair
  constexpr float kL = 0.693147182464599609375f, kLl = -1.904654323148236e-9f;
  Pair z = two_prod(-r.hi, kL);
  z.lo = __fadd_rn(z.lo, __fmaf_rn(-r.hi, kLl, -r.lo * kL));
  const Pair s = two_prod(z.hi, z.hi);
  const float cube = __fmul_rn(s.hi, z.hi);
  float tail = __fmaf_rn(z.hi, 1.f / 120.f, 1.f / 24.f);
  tail = __fmaf_rn(tail, z.hi, 1.f / 6.f);
  tail = __fmul_rn(tail, cube);
  const Pair a = two_sum(1.f, z.hi);
  const Pair b = two_sum(a.hi, 0.5f * s.hi);
  float lo = __fadd_rn(__fadd_rn(a.lo, b.lo), z.lo);
  lo = __fadd_rn(lo, __fmaf_rn(z.hi, z.lo, 0.5f * s.lo));
  lo = __fadd_rn(lo, tail);
  const Pair e = two_sum(b.hi, lo);
  const float2 t = table[k & 31];
  const Pair m = two_prod(e.hi, t.x);
  const float mlo = __fadd_rn(m.lo, __fmaf_rn(e.hi, t.y, e.lo * t.x));
  const float scale = __int_as_float((127 + 62 - (k >> 5)) << 23);  // 2^(62 - floor), floor <= 62
  return static_cast<uint64_t>(__float2ll_rn(m.hi * scale) + __float2ll_rn(mlo * scale));
}

struct Params {
  const uint16_t* logits;
  long long row_stride;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int* tokens;
  float* logprobs;
  int vocab;
};

struct Settings {
  // log2(e) / temperature, for logits times `down`: above a temperature of 1 2^64 moves from one to the other, so that
  // neither a difference of logits (up to 2^129) nor a rate (down to 2^-128) leaves the range where a pair is precise
  Pair rate;
  float down;
  float min_p, top_p, u;
  int top_k;
};

struct Sum {  // a number of tokens and their mass
  uint32_t n;
  u128 m;
};
__device__ __forceinline__ u128 shfl_up128(u128 v, int d) {
  const uint64_t lo = __shfl_up_sync(~0u, static_cast<uint64_t>(v), d);
  const uint64_t hi = __shfl_up_sync(~0u, static_cast<uint64_t>(v >> 64), d);
  return (static_cast<u128>(hi) << 64) | lo;
}

// floor(z f / 2^64), and whether that is exact.
__device__ __forceinline__ u128 scaled_floor(u128 z, uint64_t f, bool* exact) {
  const uint64_t zl = static_cast<uint64_t>(z), zh = static_cast<uint64_t>(z >> 64);
  const u128 low = static_cast<u128>(zl) * f;
  *exact = static_cast<uint64_t>(low) == 0ull;
  return static_cast<u128>(zh) * f + (low >> 64);  // zh < 2^18
}

__device__ __forceinline__ float as_float(u128 v) {
  return fmaf(static_cast<float>(static_cast<uint64_t>(v >> 64)), 18446744073709551616.f,
              static_cast<float>(static_cast<uint64_t>(v)));
}

// floor(d / w) for a quotient known to be below 2^20 (w > 0): the float
// quotient is off by less than 1.
__device__ __forceinline__ uint32_t small_quotient(u128 d, uint64_t w) {
  uint32_t q = static_cast<uint32_t>(as_float(d) / static_cast<float>(w));
  while (static_cast<u128>(q) * w > d) --q;
  while (static_cast<u128>(q + 1) * w <= d) ++q;
  return q;
}

// A fraction in [0, 1) in units of 2^-64 (exact from 2^-40 up).
__device__ __forceinline__ uint64_t fraction64(float v) {
  return static_cast<uint64_t>(v * 18446744073709551616.f);
}

template <class T>
__device__ __forceinline__ T* peer(T* p, uint32_t rank) {
  return static_cast<T*>(__cluster_map_shared_rank(p, rank));
}
__device__ __forceinline__ void cluster_sync_all() {
  cluster_arrive_release();
  cluster_wait_acquire();
}

template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const Params p) {
  constexpr int kRunUnits = (kUnits + CTAS - 1) / CTAS;  // at most
  constexpr int kMost = kRunUnits * kUnit;               // bins of a run
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* hist = smem;                // bin b: bits 16 (b & 1) .. of word b / 2
  uint32_t* counts = smem + kBins / 2;  // of the run's bins, falling
  static_assert(kMost * 8 <= static_cast<int>(kHistBytes), "a run's weights fit over the counters");
  __shared__ uint32_t s_marks[kWords];  // unit kUnits - 1 - i: bit i % 32 of word i / 32
  __shared__ uint16_t s_run[kRunUnits];  // the run's units, falling
  __shared__ uint64_t s_weight[kThreads];      // of a short run's bins
  __shared__ uint2 s_all[kWords];              // the marks of all copies, and the marked units before the word
  __shared__ uint32_t s_word[kWords / 32];
  __shared__ float2 table[32];
  __shared__ Settings s_set;
  __shared__ uint32_t s_red[kWarps];
  __shared__ uint32_t s_max[CTAS], s_own[CTAS];
  __shared__ uint16_t s_block[kBlocks][kWarps];  // the chosen bin's tokens, by block and warp
  __shared__ uint32_t s_ends[2];                 // and in the ragged ends
  __shared__ Sum s_warp[kWarps], s_ok[kWarps], s_tot[CTAS], s_totok[CTAS];
  __shared__ Sum s_before, s_total, s_passed;  // of the CTAs before this one, and of all
  __shared__ Sum s_topk, s_topp;          // what each filter keeps
  __shared__ uint32_t s_key, s_rank;      // the chosen bin, and the token's place among its equals

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int row = blockIdx.x / CTAS;

  cluster_arrive_relaxed();  // every CTA of the cluster runs before any writes into another
  for (int i = tid; i < kBins / 8; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid < 32) table[tid] = make_float2(c_table.hi[tid], c_table.lo[tid]);
  grid_dependency_wait();

  // The row's settings, read once: a load where each is used would cost its latency there.
  const bool reads = tid == kThreads - 1;
  float T = 1.f;
  Settings set = {{0.f, 0.f}, 1.f, 0.f, 1.f, 0.f, 0};
  if (reads) {
    if (p.temperature) T = p.temperature[row];
    if (p.min_p) set.min_p = p.min_p[row];
    if (p.top_p) set.top_p = p.top_p[row];
    if (p.top_k) set.top_k = p.top_k[row];
    set.u = p.u[row];
  }
  __syncthreads();

  // Count the slice: 16-byte vectors inside the row, the ragged ends by CTA 0
  // and the last CTA, so that slices are index ranges in rank order.
  const uint16_t* base = p.logits + static_cast<long long>(row) * p.row_stride;
  const int head = min(p.vocab, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(base) & 15u)) & 15u) / 2);
  const int nvec = (p.vocab - head) / 8;
  const int v0 = static_cast<int>(static_cast<long long>(nvec) * rank / CTAS);
  const int v1 = static_cast<int>(static_cast<long long>(nvec) * (rank + 1) / CTAS);
  const int tail = head + 8 * nvec;
  const bool first = rank == 0, last = rank == CTAS - 1;
  uint32_t top = 0;
  auto count = [&](uint32_t bits) {
    const uint32_t k = key_of(bits);
    if (k > kMinusInf) {
      atomicAdd(&hist[k >> 1], (k & 1u) ? 0x10000u : 1u);
      top = max(top, k);
    }
  };
  const uint4* vec = reinterpret_cast<const uint4*>(base + head);
  for (int i = v0 + tid; i < v1; i += 4 * kThreads) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * kThreads < v1) v[j] = __ldg(vec + i + j * kThreads);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j * kThreads < v1) {
        const uint32_t q[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          count(q[k] & 0xFFFFu);
          count(q[k] >> 16);
        }
      }
    }
  }
  if (reads) {  // (for behind the next barriers)
    const bool greedy = !(T > 0.f);
    if (greedy) {
      T = 1.f;
      set.min_p = 0.f;
      set.top_p = 1.f;
      set.top_k = 1;
    }
    const bool hot = T > 1.f;
    const double c = (hot ? 1.4426950408889634 * 18446744073709551616. : 1.4426950408889634) / static_cast<double>(T);
    if (hot) set.down = 1.f / 18446744073709551616.f;
    const float hi = static_cast<float>(c);
    set.rate = {hi, static_cast<float>(c - static_cast<double>(hi))};
    s_set = set;
  }
  if (first && tid < head) count(base[tid]);
  if (last && tail + tid < p.vocab) count(base[tail + tid]);
  top = __reduce_max_sync(~0u, top);
  if (lane == 0) s_red[warp] = top;
  __syncthreads();
  // mark the touched units, the highest first
#pragma unroll
  for (int i = 0; i < kUnits / kThreads; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(hist)[kUnits - 1 - (i * kThreads + tid)];
    const uint32_t any = __ballot_sync(~0u, (v.x | v.y | v.z | v.w) != 0u);
    if (lane == 0) s_marks[i * kWarps + warp] = any;
  }
  cluster_wait_acquire();
  if (warp == 0) {
    top = __reduce_max_sync(~0u, s_red[lane]);
    if (lane < CTAS) *peer(&s_max[rank], lane) = top;
  }
  cluster_sync_all();

  uint32_t maxkey = 0;
#pragma unroll
  for (int j = 0; j < CTAS; ++j) maxkey = max(maxkey, s_max[j]);
  if (maxkey == 0u) {  // nothing is allowed, and no remote access is outstanding
    if (rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      if (p.logprobs) p.logprobs[row] = __int_as_float(0xFF800000);
    }
    return;
  }

  // All touched units, and this CTA's run of them: unit i of all goes to place i - r0.
  if (tid < kWords) {
    uint32_t marks = 0;
#pragma unroll
    for (int j = 0; j < CTAS; ++j) marks |= peer(s_marks, j)[tid];
    uint32_t ahead = __popc(marks);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(~0u, ahead, d);
      if (lane >= d) ahead += v;
    }
    if (lane == 31) s_word[warp] = ahead;
    s_all[tid] = make_uint2(marks, ahead - __popc(marks));
  }
  __syncthreads();
  uint32_t touched = 0, ahead[kWords / 32];
#pragma unroll
  for (int j = 0; j < kWords / 32; ++j) {
    ahead[j] = touched;
    touched += s_word[j];
  }
  const int r0 = static_cast<int>(touched * rank / CTAS), r1 = static_cast<int>(touched * (rank + 1) / CTAS);
#pragma unroll
  for (int k = 0; k < kWords / 32; ++k) {  // word k * 32 + warp, bit lane
    const uint2 w = s_all[k * kWarps + warp];
    const int i = static_cast<int>(ahead[k] + w.y + __popc(w.x & ((1u << lane) - 1u))) - r0;
    if ((w.x >> lane & 1u) && i >= 0 && i < r1 - r0)
      s_run[i] = static_cast<uint16_t>(kUnits - 1 - ((k * kWarps + warp) * 32 + lane));
  }
  __syncthreads();

  // Merge: one thread per (unit, copy).
  constexpr int kLanes = CTAS > 8 ? 16 : CTAS > 4 ? 8 : 4;
  const int bins = (r1 - r0) * kUnit;
  for (int u0 = warp * (32 / kLanes); u0 < r1 - r0; u0 += kWarps * (32 / kLanes)) {
    const int u = u0 + lane / kLanes, j = lane % kLanes;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (u < r1 - r0 && j < CTAS) v = reinterpret_cast<const uint4*>(peer(hist, j))[s_run[u]];
    uint32_t c[8] = {v.x & 0xFFFFu, v.x >> 16, v.y & 0xFFFFu, v.y >> 16, v.z & 0xFFFFu, v.z >> 16, v.w & 0xFFFFu, v.w >> 16};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) c[i] += __shfl_xor_sync(~0u, c[i], d);
    if (u < r1 - r0) {  // falling
      if (j == 0) reinterpret_cast<uint4*>(counts)[2 * u] = make_uint4(c[7], c[6], c[5], c[4]);
      if (j == 1) reinterpret_cast<uint4*>(counts)[2 * u + 1] = make_uint4(c[3], c[2], c[1], c[0]);
    }
  }
  // A long run's weights take the counters' place once all have read them.
  const bool shortrun = (touched + CTAS - 1) / CTAS * kUnit <= kThreads;  // the same for the whole cluster
  uint64_t* weights = shortrun ? s_weight : reinterpret_cast<uint64_t*>(hist);
  if (shortrun) __syncthreads();
  else cluster_sync_all();
  auto key_at = [&](int i) { return static_cast<uint32_t>(s_run[i / kUnit]) * kUnit + (kUnit - 1 - i % kUnit); };

  // Weigh the occupied bins, neighbours by neighbouring threads.
  const Pair rate = s_set.rate;
  const float down = s_set.down, vmax = value_of(maxkey) * down;
  for (int i = tid; i < bins; i += kThreads) {
    if (counts[i]) {
      const uint32_t key = key_at(i);
      uint64_t w = 1ull << 62;
      if (key != maxkey) {
        if (maxkey == kPlusInf) {
          w = 0ull;
        } else {
          const Pair d = two_sum(vmax, -value_of(key) * down);
          Pair y = two_prod(d.hi, rate.hi);
          y.lo = __fadd_rn(y.lo, __fmaf_rn(d.hi, rate.lo, d.lo * rate.hi));
          w = exp2_neg(two_sum(y.hi, y.lo), table);
        }
      }
      weights[i] = w;
    }
  }
  __syncthreads();

  // Scan, some neighbouring bins per thread.
  const int per_thread = (bins + kThreads - 1) / kThreads;
  const int b0 = min(bins, tid * per_thread), b1 = min(bins, b0 + per_thread);
  const float minp = s_set.min_p;
  const bool use_minp = minp > 0.f;
  const uint64_t least = use_minp ? static_cast<uint64_t>(fminf(minp, 1.f) * 4611686018427387904.f) : 0ull;
  Sum mine{0u, 0}, ok{0u, 0};
  for (int i = b0; i < b1; ++i) {
    const uint32_t c = counts[i];
    if (c) {
      const uint64_t w = weights[i];
      const u128 m = static_cast<u128>(w) * c;
      mine.n += c;
      mine.m += m;
      if (w >= least) {
        ok.n += c;
        ok.m += m;
      }
    }
  }
  Sum inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t n = __shfl_up_sync(~0u, inc.n, d);
    const u128 m = shfl_up128(inc.m, d);
    if (lane >= d) {
      inc.n += n;
      inc.m += m;
    }
  }
  if (lane == 31) s_warp[warp] = inc;
  if (use_minp) {  // the same for every thread of the cluster
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t n = __shfl_up_sync(~0u, ok.n, d);
      const u128 m = shfl_up128(ok.m, d);
      if (lane >= d) {
        ok.n += n;
        ok.m += m;
      }
    }
    if (lane == 31) s_ok[warp] = ok;
  }
  __syncthreads();
  auto sum_all = [&](Sum t) {  // over a warp
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      t.n += __shfl_xor_sync(~0u, t.n, d);
      const uint64_t lo = __shfl_xor_sync(~0u, static_cast<uint64_t>(t.m), d);
      const uint64_t hi = __shfl_xor_sync(~0u, static_cast<uint64_t>(t.m >> 64), d);
      t.m += (static_cast<u128>(hi) << 64) | lo;
    }
    return t;
  };
  if (warp == 0) {
    Sum t = s_warp[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t n = __shfl_up_sync(~0u, t.n, d);
      const u128 m = shfl_up128(t.m, d);
      if (lane >= d) {
        t.n += n;
        t.m += m;
      }
    }
    s_warp[lane] = t;  // inclusive
    __syncwarp();
    if (lane < CTAS) *peer(&s_tot[rank], lane) = s_warp[kWarps - 1];
  } else if (warp == 1 && use_minp) {
    const Sum t = sum_all(s_ok[lane]);
    if (lane < CTAS) *peer(&s_totok[rank], lane) = t;
  }
  cluster_sync_all();
  if (warp == 0) {
    const Sum none{0u, 0};
    const Sum t = lane < CTAS ? s_tot[lane] : none;
    const Sum all = sum_all(t), up = sum_all(lane < static_cast<int>(rank) ? t : none);
    if (lane == 0) {
      s_total = all;
      s_before = up;
    }
  } else if (warp == 1 && use_minp) {
    const Sum t = sum_all(lane < CTAS ? s_totok[lane] : Sum{0u, 0});
    if (lane == 0) s_passed = t;
  }
  __syncthreads();
  const Sum total = s_total;
  Sum passed = s_passed, before = s_before;  // before: of the bins above this thread's
  if (warp > 0) {
    before.n += s_warp[warp - 1].n;
    before.m += s_warp[warp - 1].m;
  }
  before.n += inc.n - mine.n;
  before.m += inc.m - mine.m;

  // top-k: the kept count and mass
  const int kreq = s_set.top_k;
  Sum kept = total;
  if (kreq > 0 && static_cast<uint32_t>(kreq) < total.n) {
    const uint32_t K = static_cast<uint32_t>(kreq);
    if (before.n < K && K <= before.n + mine.n) {
      uint32_t left = K - before.n;
      u128 m = before.m;
      for (int i = b0; left > 0u; ++i) {
        const uint32_t take = min(left, counts[i]);
        if (take) m += static_cast<u128>(weights[i]) * take;
        left -= take;
      }
      for (int j = 0; j < CTAS; ++j) *peer(&s_topk, j) = Sum{K, m};
    }
    cluster_sync_all();
    kept = s_topk;
  }
  // top-p: the tokens whose predecessors' mass is below the fraction
  const float top_p = s_set.top_p;
  if (top_p < 1.f) {
    bool exact;
    u128 goal = scaled_floor(kept.m, top_p > 0.f ? fraction64(top_p) : 0ull, &exact);
    if (!exact || goal == 0) goal += 1;  // before < fraction as integers: before < ceil; the first token stays
    if (before.m < goal && goal <= before.m + mine.m) {
      Sum k = before;
      for (int i = b0; i < b1; ++i) {
        const uint32_t c = counts[i];
        if (c == 0u) continue;
        const uint64_t w = weights[i];
        const u128 m = static_cast<u128>(w) * c;
        if (w > 0ull && k.m + m >= goal) {
          const uint32_t take = small_quotient(goal - k.m - 1, w) + 1;  // ceil((goal - before) / w)
          k.n += take;
          k.m += static_cast<u128>(w) * take;
          break;
        }
        k.n += c;
        k.m += m;
      }
      // top-k ends inside a bin: it may keep fewer of equal tokens
      if (k.n > kept.n) k = kept;
      for (int j = 0; j < CTAS; ++j) *peer(&s_topp, j) = k;
    }
    cluster_sync_all();
    kept = s_topp;
  }
  if (use_minp) {
    if (minp > 1.f) passed = Sum{1u, static_cast<u128>(1ull << 62)};
    if (passed.n < kept.n) kept = passed;
  }

  // The draw.
  float uu = s_set.u;
  if (!(uu > 0.f)) uu = 0.f;
  bool exact;
  const u128 goal = scaled_floor(kept.m, uu < 1.f ? fraction64(uu) : ~0ull, &exact);  // below kept.m
  uint64_t drawn = 0;  // the weight, where it is this thread's
  if (before.m <= goal && goal < before.m + mine.m) {
    u128 m = before.m;
    for (int i = b0; i < b1; ++i) {
      const uint32_t c = counts[i];
      if (c == 0u) continue;
      const uint64_t w = weights[i];
      const u128 next = m + static_cast<u128>(w) * c;
      if (goal < next) {
        const uint32_t j = small_quotient(goal - m, w);
        for (int r = 0; r < CTAS; ++r) {
          *peer(&s_key, r) = key_at(i);
          *peer(&s_rank, r) = j;
        }
        drawn = w;
        break;
      }
      m = next;
    }
  }
  cluster_sync_all();

  if (drawn != 0 && p.logprobs) {
    // log(w / kept): near 1 from the exact remainder, so that it keeps its relative precision
    const float gone = as_float(kept.m - drawn) / as_float(kept.m);
    p.logprobs[row] = gone < 0.5f ? log1pf(-gone) : logf(static_cast<float>(drawn) / as_float(kept.m));
  }

  // Back to the token: the (rank)-th occurrence of the key in index order, by
  // blocks of 1024 vectors; the ragged ends are the first CTA's block before and
  // the last CTA's block behind the vectors.
  const uint32_t key = s_key;
  const int blocks = (v1 - v0 + kThreads - 1) / kThreads;
  // by their bit patterns: +0 and -0 are one key
  const uint32_t bits1 = (key & 0x8000u) ? (key ^ 0x8000u) : (key ^ 0xFFFFu);
  const uint32_t pattern = bits1 * 0x10001u, mask = bits1 == 0u ? 0x7FFF7FFFu : ~0u;
  auto hits = [&](const uint4& v) {  // bit i: value i of the vector
    const uint32_t x[4] = {(v.x & mask) ^ pattern, (v.y & mask) ^ pattern, (v.z & mask) ^ pattern, (v.w & mask) ^ pattern};
    uint32_t any = 0, m = 0;  // any: a half of a word is 0
#pragma unroll
    for (int k = 0; k < 4; ++k) any |= (x[k] - 0x00010001u) & ~x[k];
    if (any & 0x80008000u) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m |= ((x[k] & 0xFFFFu) == 0u ? 1u << (2 * k) : 0u) | (x[k] < 0x10000u ? 2u << (2 * k) : 0u);
    }
    return m;
  };
  uint64_t found = 0;  // 8 bits a block
  uint32_t ends = 0;   // of the ragged ends, this thread's value
  if (first && tid < head) ends = key_of(base[tid]) == key;
  if (last && tail + tid < p.vocab) ends |= (key_of(base[tail + tid]) == key) << 1;
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int i = v0 + j * kThreads + tid;
    if (i < v1) found |= static_cast<uint64_t>(hits(__ldg(vec + i))) << (8 * j);
  }
  const uint32_t in_head = __popc(__ballot_sync(~0u, ends & 1u)), in_tail = __popc(__ballot_sync(~0u, ends & 2u));
  if (tid == 0) {  // (fewer than 8 values: warp 0's)
    s_ends[0] = in_head;
    s_ends[1] = in_tail;
  }
  for (int j = 0; j < blocks; ++j) {
    const uint32_t n = __reduce_add_sync(~0u, __popc(static_cast<uint32_t>(found >> (8 * j)) & 0xFFu));
    if (lane == 0) s_block[j][warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t n = 0;
    for (int j = 0; j < blocks; ++j) n += s_block[j][lane];
    n = __reduce_add_sync(~0u, n) + s_ends[0] + s_ends[1];
    if (lane < CTAS) *peer(&s_own[rank], lane) = n;
  }
  cluster_sync_all();  // no remote access is left
  uint32_t nth = s_rank;
  for (int j = 0; j < static_cast<int>(rank); ++j) {
    if (nth < s_own[j]) return;
    nth -= s_own[j];
  }
  if (nth >= s_own[rank]) return;
  if (first) {
    if (nth < s_ends[0]) {
      const uint32_t heads = __ballot_sync(~0u, ends & 1u);
      if (warp == 0 && (ends & 1u) && __popc(heads & ((1u << lane) - 1u)) == static_cast<int>(nth)) p.tokens[row] = tid;
      return;
    }
    nth -= s_ends[0];
  }
  for (int j = 0; j < blocks; ++j) {
    const uint32_t mine_n = s_block[j][lane];
    const uint32_t all = __reduce_add_sync(~0u, mine_n);
    if (nth >= all) {
      nth -= all;
      continue;
    }
    const uint32_t below = __reduce_add_sync(~0u, lane < warp ? mine_n : 0u);
    const uint32_t bits = static_cast<uint32_t>(found >> (8 * j)) & 0xFFu;
    uint32_t pre = __popc(bits);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(~0u, pre, d);
      if (lane >= d) pre += v;
    }
    pre += below;
    const uint32_t at = pre - __popc(bits);
    if (at <= nth && nth < pre) {
      uint32_t rest = bits;
      for (uint32_t i = at; i < nth; ++i) rest &= rest - 1;
      p.tokens[row] = head + 8 * (v0 + j * kThreads + tid) + __ffs(rest) - 1;
    }
    return;
  }
  // behind the vectors
  if (warp == 0) {
    const uint32_t tails = __ballot_sync(~0u, ends & 2u);
    if ((ends & 2u) && __popc(tails & ((1u << lane) - 1u)) == static_cast<int>(nth)) p.tokens[row] = tail + tid;
  }
}

template <int CTAS>
cudaError_t configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* cluster, int rows) {
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem_for(CTAS)));
  if (e == cudaSuccess && CTAS > 8)
    e = cudaFuncSetAttribute(sample_kernel<CTAS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  cluster->id = cudaLaunchAttributeClusterDimension;
  cluster->val.clusterDim.x = CTAS;
  cluster->val.clusterDim.y = 1;
  cluster->val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * CTAS);
  cfg.dynamicSmemBytes = smem_for(CTAS);
  return e;
}

// Clusters of this size that the device holds at once (0: none).
template <int CTAS>
int held() {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(kThreads);
  if (configure<CTAS>(cfg, attr, 1) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<CTAS>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

// The largest cluster of which the device holds one for each row at once, so
// that no row waits for another; beyond that 4, where a slice still fits.  16
// CTAs halve the counting of 8, but wait longer for each other: one row of 32000
// takes 14.0 us with 16 and 13.0 with 8, of 65000 14.3 and 14.1, of 131072 15.3
// and 15.5, of 248320 15.9 and 17.5.
int cluster_for(int rows, int vocab) {
  static const int most16 = held<16>(), most8 = held<8>(), most6 = held<6>();  // (devices that run this are alike)
  if (rows <= most16 && vocab > 65536) return 16;
  if (rows <= most8) return 8;
  if (rows <= most6 && slice_fits(vocab, 6)) return 6;
  return slice_fits(vocab, 4) ? 4 : 8;
}

template <int CTAS>
cudaError_t launch(const Params& p, int rows, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(kThreads);
  const cudaError_t e = configure<CTAS>(cfg, attr + 1, rows);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, sample_kernel<CTAS>, p);
}

}  // namespace
}  // namespace w4g128

extern "C" int w4g128_sample(const w4g128_sample_args* a, void* stream) {
  using namespace w4g128;
  if (a == nullptr || a->logits == nullptr || a->u == nullptr || a->tokens == nullptr) return W4G128_ERR_INVALID_ARG;
  if (a->rows < 1 || a->rows > W4G128_MAX_SAMPLE_ROWS) return W4G128_ERR_INVALID_ARG;
  if (a->vocab < 1 || a->vocab > W4G128_MAX_VOCAB || a->row_stride < a->vocab) return W4G128_ERR_SHAPE;
  auto off = [](const void* q, uintptr_t n) { return (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0; };
  if (off(a->logits, 2) || off(a->temperature, 4) || off(a->top_k, 4) || off(a->top_p, 4) || off(a->min_p, 4) ||
      off(a->u, 4) || off(a->tokens, 4) || off(a->logprobs, 4))
    return W4G128_ERR_ALIGN;
  const int fault = fault_hook();
  if (fault != W4G128_OK) return fault;
  if (!device_is_sm103()) return W4G128_ERR_DEVICE;
  const Params p{a->logits, a->row_stride, a->temperature, a->top_k, a->top_p, a->min_p, a->u,
                 a->tokens, a->logprobs, a->vocab};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int ctas = cluster_for(a->rows, a->vocab);
  const cudaError_t e = ctas == 16  ? launch<16>(p, a->rows, s)
                        : ctas == 8 ? launch<8>(p, a->rows, s)
                        : ctas == 6 ? launch<6>(p, a->rows, s)
                                    : launch<4>(p, a->rows, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return W4G128_ERR_CUDA;
  }
  return W4G128_OK;
}
