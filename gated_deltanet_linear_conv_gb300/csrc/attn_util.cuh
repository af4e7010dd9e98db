// Device helpers of norm_rope.cu and paged_attn.cu.
#pragma once

#include "common.cuh"

namespace gdn {

constexpr int kDevErrCache = 3;   // beside DeviceError's: kv_lens, a page id or a position out of its range

// Raises the error flag for a cu_seqlens with an inconsistent sequence: thread `i` of `n`
// looks at every n-th one.
__device__ __forceinline__ void check_seqs(const int32_t* cu, int num_seqs, int total, int64_t i, int64_t n, int* err) {
  if (cu == nullptr) return;
  for (int64_t s = i; s < num_seqs; s += n) {
    int bos, eos;
    if (!seq_bounds(cu, num_seqs, total, (int)s, bos, eos)) raise_error(err, kDevErrSeqlens);
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
