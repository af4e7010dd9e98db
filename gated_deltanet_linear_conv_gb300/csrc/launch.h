// Internal launcher interface between the C-ABI layer (api.cu) and the
// kernel translation units.  Arguments are already validated by the caller.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

struct ConvGatingArgs {
  const void* x;          // mixed_qkv [T, C]
  const void* w;          // [C, 4]
  const void* bias;       // [C] or null
  const void* state_in;   // [N, C, 3] or null
  void* state_out;        // [N, C, 3] or null
  const void* a;          // [T, Nv]
  const void* b;          // [T, Nv]
  const float* A_log;     // [Nv]
  const float* dt_bias;   // [Nv]
  void* q;                // [T, Nk, Dk]
  void* k;                // [T, Nk, Dk]
  void* v;                // [T, Nv, Dv]
  float* g;               // [T, Nv]
  float* beta;            // [T, Nv]
  const int32_t* cu;      // [N + 1] or null
  int num_seqs, total, Nk, Nv, Dk, Dv, C;
  float q_scale, l2_eps;
  int in_bf16, out_bf16;
  int* err;
};
cudaError_t launch_conv_gating(const ConvGatingArgs& p, cudaStream_t s);
// The conv state after every token ([tokens, C, 3], the input element type).
cudaError_t launch_conv_state_steps(const ConvGatingArgs& p, void* steps, cudaStream_t s);

struct GatingArgs {
  const void* a; const void* b; const float* A_log; const float* dt_bias;
  float* g; float* beta; int64_t rows; int Nv; int in_bf16;
};
cudaError_t launch_gating(const GatingArgs& p, cudaStream_t s);

struct RmsNormArgs {
  const void* x; const void* z; const float* w; void* y;
  int64_t rows; int dim; float eps; int x_bf16, z_bf16, out_bf16;
};
cudaError_t launch_gated_rmsnorm(const RmsNormArgs& p, cudaStream_t s);

struct DecodeArgs {
  const void* q; const void* k; const void* v;   // [T, Nk, Dk] / [T, Nv, Dv]
  const float* g; const float* beta;             // [T, Nv]
  float* state;                                  // [N, Nv, Dk, Dv]
  void* o;                                       // [T, Nv, Dv]
  const int32_t* cu;
  int num_seqs, total, Nk, Nv, Dk, Dv;
  float scale;
  int in_bf16, out_bf16;
  int* err;
  float* step_states;                            // [T, Nv, Dk, Dv] state after each token, or null
};
cudaError_t launch_recurrent_decode(const DecodeArgs& p, cudaStream_t s);

struct DecodeFusedArgs {
  const void* x; const void* w; const void* bias; void* conv_state;
  const void* a; const void* b; const float* A_log; const float* dt_bias;
  float* state; const void* z; const float* norm_w; void* y;
  int B, Nk, Nv, Dk, Dv, C;
  float q_scale, l2_eps, norm_eps;
  int in_bf16, out_bf16;
};
cudaError_t launch_decode_fused(const DecodeFusedArgs& p, cudaStream_t s);

struct ChunkArgs {
  const void* q; const void* k; const void* v;   // [T, Nk, Dk] / [T, Nv, Dv]
  const float* g; const float* beta;             // [T, Nv]
  const float* S0;                               // [N, Nv, Dk, Dv] or null
  float* ST;                                     // [N, Nv, Dk, Dv] or null
  void* o;                                       // [T, Nv, Dv]
  const int32_t* cu;
  int num_seqs, total, Nk, Nv, Dk, Dv;
  float scale;
  int in_bf16, out_bf16;
  void* workspace; size_t workspace_bytes;
  int* err;
  // gated RMSNorm fused into the output (tensor-core path): o holds y then
  const void* z;                                 // [T, Nv, Dv] bf16, or null (plain o)
  const float* norm_w;                           // [Dv]
  float norm_eps;
  // bound of each wait of the scan on a flag or barrier, in ns of device time (0: the default)
  unsigned long long wait_ns;
  int no_solve;                                  // test hook: the one-sequence launch runs no solve
  int no_split;                                  // never split a long sequence (smaller workspace)
  // one-sequence launch with z: the scan writes o into o's buffer and spare solve groups apply
  // the gated norm in place, block by block (set by the launcher, not by callers)
  int side_norm;
};
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
// Portable fp32 CUDA-core implementation of the chunk form.
cudaError_t launch_chunk_simt(const ChunkArgs& p, cudaStream_t s);
// tcgen05 tensor-core implementation (bf16 q/k/v, Dk = Dv = 128).
bool chunk_tc_supported(const ChunkArgs& p);
// Workspace bytes of a call on the current device (allow_split: a long single sequence may
// run split in two segments, which needs extra scratch).
size_t chunk_tc_workspace_bytes(int num_seqs, int total, int Nv, bool allow_split = true);
cudaError_t launch_chunk_tc(const ChunkArgs& p, cudaStream_t s);
// Fixed-size device scratch owned by the library (see gdn_chunk_prefill_static).
constexpr size_t kStaticScratchBytes = (size_t)32 << 20;
cudaError_t static_scratch(void** ptr);

// ---- softmax attention over a paged cache (norm_rope.cu, paged_attn.cu)
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
};
size_t paged_attn_workspace_bytes(int num_seqs, int total, int Nq, int Nkv, int D, bool bf, int64_t table_tokens);
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
