// Device helpers of the kernels around the paged cache: error codes, programmatic launches, division.
#pragma once

#include "common.cuh"

namespace gdn {

// beside DeviceError's:
constexpr int kDevErrCache = 3;   // kv_lens, a page id or a position out of its range
constexpr int kDevErrPlan = 4;    // requests that the free pages, the table or the token rows do not hold
constexpr int kDevErrDraft = 5;   // a token outside the vocabulary, a draft without probabilities, a row without weight

// Raises the error flag for a cu_seqlens with an inconsistent sequence: thread `i` of `n`
// looks at every n-th one.
__device__ __forceinline__ void check_seqs(const int32_t* cu, int num_seqs, int total, int64_t i, int64_t n, int* err) {
  if (cu == nullptr) return;
  for (int64_t s = i; s < num_seqs; s += n) {
    int bos, eos;
    if (!seq_bounds(cu, num_seqs, total, (int)s, bos, eos)) raise_error(err, kDevErrSeqlens);
  }
}

// Zeros to the rows of sequences with nothing to attend.  A few rows are a warp's work (zero_few); but one inactive slot may hold
// most of a padded step's rows, and above kFewWords 16-byte words of output the whole grid takes part (zero_many).
constexpr int64_t kFewWords = 2048;
__device__ __forceinline__ void zero_few(void* out, int64_t at, int64_t words) {
  uint4* o = static_cast<uint4*>(out) + at;
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < (int)words; i += 32) o[i] = make_uint4(0, 0, 0, 0);
}
// All sequences of more words, by one range per CTA of their rows laid end to end.  `load` gives a sequence's bounds and length
// {bos, n, len}; row: words per token; THREADS threads of each CTA call it, `sync` is a barrier of theirs and scratch
// THREADS / 32 + 2 numbers in shared memory.
template <int THREADS, typename Load, typename Sync>
__device__ __forceinline__ void zero_many(Load load, int num_seqs, int64_t row, void* out, int tid, int64_t* scratch, Sync sync) {
  constexpr int WARPS = THREADS / 32;
  const int lane = tid & 31, warp = tid >> 5;
  const int per = (num_seqs + THREADS - 1) / THREADS, s_lo = min(num_seqs, tid * per), s_hi = min(num_seqs, s_lo + per);
  auto words = [&](int s) {
    const auto q = load(s);
    return q.len == 0 && q.n * row > kFewWords ? q.n * row : 0;
  };
  int64_t sum = 0;
#pragma unroll 1
  for (int s = s_lo; s < s_hi; ++s) sum += words(s);
  int64_t inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  sync();
  int64_t before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  if (total == 0) return;
  auto cut = [&](unsigned c) { return c == gridDim.x ? total : total * c / gridDim.x & ~(int64_t)7; };     // (whole lines)
  const int64_t lo = cut(blockIdx.x), hi = cut(blockIdx.x + 1);
  if (before <= lo && lo < before + sum) {         // the sequence that the range starts in
    int64_t at = before;
#pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
      const int64_t w = words(s);
      if (lo < at + w) {
        scratch[WARPS] = at;
        scratch[WARPS + 1] = s;
        break;
      }
      at += w;
    }
  }
  sync();
  if (lo >= hi) return;
  int64_t at = scratch[WARPS];
#pragma unroll 1
  for (int base = (int)scratch[WARPS + 1]; base < num_seqs && at < hi; base += 32) {
    int bos = 0, n = 0;
    if (base + lane < num_seqs) {
      const auto q = load(base + lane);
      bos = q.bos;
      n = q.len == 0 && q.n * row > kFewWords ? q.n : 0;
    }
    uint32_t idle = __ballot_sync(0xffffffffu, n > 0);
#pragma unroll 1
    while (idle != 0 && at < hi) {
      const int from = __ffs(idle) - 1;
      idle &= idle - 1;
      uint4* o = static_cast<uint4*>(out) + __shfl_sync(0xffffffffu, bos, from) * row;
      const int64_t w = __shfl_sync(0xffffffffu, n, from) * row, end = min(hi - at, w);
#pragma unroll 4
      for (int64_t i = max(lo - at, (int64_t)0) + tid; i < end; i += THREADS) o[i] = make_uint4(0, 0, 0, 0);
      at += w;
    }
  }
}

// Programmatic launches: until the kernels before this one have ended and their writes are
// visible; and leave for the next kernel to be set up (it waits in turn).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// x / d for 0 <= x < 2^31 by one multiplication (d > 0; Granlund and Montgomery's division by an
// invariant integer): with 2^k the first power of two that is at least d and m = floor(2^32 (2^k - d) / d) + 1, x / d = (hi32(x m) + x) >> k.
struct Div {
  uint32_t d, m, k;
  static Div of(uint32_t d) {
    uint32_t k = 0;
    while ((uint64_t)1 << k < d) ++k;
    return {d, (uint32_t)(((((uint64_t)1 << k) - d) << 32) / d + 1), k};
  }
  __device__ __forceinline__ int quot(int x) const { return (int)((__umulhi((uint32_t)x, m) + (uint32_t)x) >> k); }
};

}  // namespace gdn
