// Host-callable launchers of the softmax attention over a paged cache, shared between
// api.cu, norm_rope.cu and paged_attn.cu.
#pragma once

#include "launch.h"

namespace gdn {

struct HeadsIn { const void* p; int64_t ts, hs; };    // element (t, h, i) at t * ts + h * hs + i
struct PagedCache {
  void* k; void* v;                              // element (page, h, slot, i) at page * ps + h * hs + slot * ss + i
  int64_t ps, hs, ss;
  const int32_t* bt;                             // [N, max_pages]
  const int32_t* lens;                           // [N]
  int num_pages, page_size, max_pages;
  // the axes 0 slot, 1 head, 2 page by increasing stride, and those strides (of an axis with
  // one entry, whose stride is never used: one that fits the order)
  int order[3];
  int64_t sorted[3];
};

struct NormRopeArgs {
  HeadsIn q, k, v;                               // q.p null: no q; v.p null: no cache
  void* q_out; void* k_out;                      // [T, Nq, D] / [T, Nkv, D]; k_out null: k and v go to the cache
  PagedCache c;
  const float* qw; const float* kw;              // [D] or null (no norm)
  const float* table;                            // [max_pos, rot] cosines | sines, or null with rot = 0
  const int32_t* pos;                            // [T] or null
  const int32_t* cu;
  int num_seqs, total, Nq, Nkv, D, rot, inter, max_pos;
  float eps;
  int in_bf16, q_bf16, kv_bf16;                  // kv: the type of k_out or of the cache
  int* err;
};
cudaError_t launch_norm_rope(const NormRopeArgs& p, cudaStream_t s);

struct PagedAttnArgs {
  HeadsIn q, gate;                               // gate.p null: no gate
  PagedCache c;
  void* o;                                       // [T, Nq, D]
  const int32_t* cu;
  int num_seqs, total, Nq, Nkv, D;
  float scale;
  int in_bf16, out_bf16;
  void* ws;
  int* err;
  unsigned long long wait_ns = 2000000000ull;    // bound of every wait
  int skip = 0;                                  // test hook: copies never issued (1 query rows, 2 keys and values)
};
size_t paged_attn_workspace_bytes(int Nq, int Nkv, int D, bool bf, int64_t table_tokens);
cudaError_t launch_paged_attn(const PagedAttnArgs& p, cudaStream_t s);

// Launch that may begin while the kernel before it on the stream still runs: the kernel has to
// wait (pdl_wait) in every thread before it touches global memory, so that its end implies the
// end of all that was launched before it.  Its start-up overlaps the other's end.
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*fn)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

}  // namespace gdn
