// C-ABI layer of the GB300 Gated DeltaNet library: argument validation on the
// host, then the launch of the kernels of each call.  Declarations and the
// contract of every entry point are in include/gdn.h.

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "gdn.h"
#include "launch.h"
#include "paged_attn.h"

namespace {

thread_local char g_err[512] = "no error";

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t e, const char* where) {
  return fail(GDN_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

// Sticky device error flag, one per device that loads the library.
__device__ int g_device_error;

constexpr int kMaxDevices = 64;
std::mutex g_flag_mu;
int* g_flag_ptr[kMaxDevices];

// Device address of the error flag on the current device (looked up once).
int get_flag(int** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(GDN_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lock(g_flag_mu);
  if (g_flag_ptr[dev] == nullptr) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_device_error);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(device error flag)");
    g_flag_ptr[dev] = static_cast<int*>(ptr);
  }
  *out = g_flag_ptr[dev];
  return GDN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(int d) { return d == GDN_BF16 || d == GDN_F32; }

#define REQUIRE_PTR(p)                                                                  \
  do {                                                                                  \
    if ((p) == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, #p);    \
    if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, #p); \
  } while (0)
#define OPTIONAL_PTR(p)                                                                 \
  do {                                                                                  \
    if ((p) != nullptr && !aligned16(p))                                                \
      return fail(GDN_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, #p);      \
  } while (0)

int check_dims(const char* fn, const gdn_dims* d, const int32_t* cu) {
  if (d == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: dims is NULL", fn);
  if (d->num_seqs < 1) return fail(GDN_ERR_INVALID_ARG, "%s: num_seqs = %d < 1", fn, d->num_seqs);
  if (d->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "%s: total_tokens < 0", fn);
  if (d->num_k_heads < 1 || d->num_v_heads < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: head counts must be >= 1", fn);
  if (d->num_v_heads % d->num_k_heads != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: num_v_heads (%d) is not a multiple of num_k_heads (%d)",
                fn, d->num_v_heads, d->num_k_heads);
  if ((d->head_k_dim != 64 && d->head_k_dim != 128) || (d->head_v_dim != 64 && d->head_v_dim != 128))
    return fail(GDN_ERR_UNSUPPORTED, "%s: head dims (%d, %d) not in {64, 128}", fn,
                d->head_k_dim, d->head_v_dim);
  if (cu == nullptr && d->total_tokens % d->num_seqs != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: total_tokens %% num_seqs != 0 without cu_seqlens", fn);
  OPTIONAL_PTR(cu);
  return GDN_OK;
}

// Checks of the paged-attention calls.
int check_attn_dims(const char* fn, const gdn_attn_dims* d, const int32_t* cu) {
  if (d == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: dims is NULL", fn);
  if (d->num_seqs < 1) return fail(GDN_ERR_INVALID_ARG, "%s: num_seqs = %d < 1", fn, d->num_seqs);
  if (d->total_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "%s: total_tokens < 0", fn);
  if (d->num_q_heads < 1 || d->num_kv_heads < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: head counts must be >= 1", fn);
  if (d->num_q_heads % d->num_kv_heads != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: num_q_heads (%d) is not a multiple of num_kv_heads (%d)", fn,
                d->num_q_heads, d->num_kv_heads);
  if (d->num_q_heads > 65535) return fail(GDN_ERR_UNSUPPORTED, "%s: more than 65535 query heads", fn);
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return fail(GDN_ERR_UNSUPPORTED, "%s: head dim %d not in {64, 128, 256}", fn, d->head_dim);
  if (cu == nullptr && d->total_tokens % d->num_seqs != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: total_tokens %% num_seqs != 0 without cu_seqlens", fn);
  OPTIONAL_PTR(cu);
  return GDN_OK;
}

int check_heads(const char* fn, const char* name, const gdn_heads* h, int dtype) {
  if (h == nullptr || h->data == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  const int64_t unit = dtype == GDN_BF16 ? 8 : 4;
  if (!aligned16(h->data)) return fail(GDN_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, name);
  if (h->token_stride < 0 || h->head_stride < 0 || h->token_stride % unit != 0 || h->head_stride % unit != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s: the strides of %s must be multiples of 16 bytes, >= 0", fn, name);
  return GDN_OK;
}

int check_norm_rope(const char* fn, const gdn_attn_dims* d, const gdn_norm_rope* nr) {
  OPTIONAL_PTR(nr->q_norm_w);
  OPTIONAL_PTR(nr->k_norm_w);
  OPTIONAL_PTR(nr->positions);
  if (nr->rotary_dim < 0 || nr->rotary_dim > d->head_dim)
    return fail(GDN_ERR_INVALID_ARG, "%s: rotary_dim %d not in [0, head_dim]", fn, nr->rotary_dim);
  if (nr->rotary_dim % 16 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "%s: rotary_dim %d is not a multiple of 16", fn, nr->rotary_dim);
  if (nr->rotary_dim > 0) {
    const float* cos_sin = nr->cos_sin;
    REQUIRE_PTR(cos_sin);
    if (nr->max_positions < 1) return fail(GDN_ERR_INVALID_ARG, "%s: max_positions < 1", fn);
    if (nr->interleaved != 0 && nr->interleaved != 1)
      return fail(GDN_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1", fn);
  }
  return GDN_OK;
}

// The cache's axes 0 slot, 1 head, 2 page by increasing stride; axes of one entry last, with
// the largest stride of the others.
void cache_axes(const gdn_paged_cache* c, int num_kv_heads, int head_dim, int order[3], int64_t stride[3]) {
  const int64_t st[3] = {c->slot_stride, c->head_stride, c->page_stride};
  const int ext[3] = {c->page_size, num_kv_heads, c->num_pages};
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if (ext[i] <= 1) continue;
    int j = n++;
    for (; j > 0 && stride[j - 1] > st[i]; --j) {
      stride[j] = stride[j - 1];
      order[j] = order[j - 1];
    }
    stride[j] = st[i];
    order[j] = i;
  }
  const int64_t top = n > 0 ? stride[n - 1] : head_dim;
  for (int i = 0; i < 3; ++i) {
    if (ext[i] > 1) continue;
    stride[n] = top;
    order[n++] = i;
  }
}

int check_cache(const char* fn, const gdn_attn_dims* d, const gdn_paged_cache* c, int dtype) {
  if (c == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: cache is NULL", fn);
  const void *cache_k = c->k, *cache_v = c->v;
  const int32_t *block_table = c->block_table, *kv_lens = c->kv_lens;
  REQUIRE_PTR(cache_k);
  REQUIRE_PTR(cache_v);
  REQUIRE_PTR(block_table);
  REQUIRE_PTR(kv_lens);
  if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1)
    return fail(GDN_ERR_INVALID_ARG, "%s: num_pages, page_size and max_pages must be >= 1", fn);
  const int64_t unit = dtype == GDN_BF16 ? 8 : 4, most = (int64_t)1 << (dtype == GDN_BF16 ? 39 : 38);
  const int64_t st[3] = {c->page_stride, c->head_stride, c->slot_stride};
  for (int i = 0; i < 3; ++i)
    if (st[i] <= 0 || st[i] % unit != 0 || st[i] >= most)
      return fail(GDN_ERR_INVALID_ARG, "%s: the cache strides must be positive multiples of 16 bytes below 2^40 bytes",
                  fn);
  const int ext[3] = {c->page_size, d->num_kv_heads, c->num_pages};
  int order[3];
  int64_t stride[3], span = d->head_dim;
  cache_axes(c, d->num_kv_heads, d->head_dim, order, stride);
  for (int i = 0; i < 3 && ext[order[i]] > 1; ++i) {
    if (stride[i] < span) return fail(GDN_ERR_INVALID_ARG, "%s: the cache's strides make entries overlap", fn);
    if (i > 0 && stride[i] % stride[i - 1] != 0)
      return fail(GDN_ERR_UNSUPPORTED, "%s: the cache's strides are not multiples of one another", fn);
    if (stride[i] > ((int64_t)1 << 60) / ext[order[i]])              // (their product may pass 64 bits)
      return fail(GDN_ERR_INVALID_ARG, "%s: the cache's strides span more than 2^60 elements", fn);
    span = stride[i] * ext[order[i]];
  }
  return GDN_OK;
}

gdn::HeadsIn heads_in(const gdn_heads* h) {
  return h == nullptr ? gdn::HeadsIn{nullptr, 0, 0} : gdn::HeadsIn{h->data, h->token_stride, h->head_stride};
}

gdn::PagedCache paged_cache(const gdn_attn_dims* d, const gdn_paged_cache* c) {
  gdn::PagedCache p{c->k, c->v, c->page_stride, c->head_stride, c->slot_stride, c->block_table, c->kv_lens,
                    c->num_pages, c->page_size, c->max_pages, {}, {}};
  cache_axes(c, d->num_kv_heads, d->head_dim, p.order, p.sorted);
  return p;
}

#define CHECK(call)                   \
  do {                                \
    const int st_ = (call);           \
    if (st_ != GDN_OK) return st_;    \
  } while (0)

// The part common to gdn_qk_norm_rope and gdn_paged_kv_append (cache null: dense k_out).
int norm_rope(const char* fn, const gdn_attn_dims* dims, const int32_t* cu, const gdn_heads* q, const gdn_heads* k,
              const gdn_heads* v, int in_dtype, const gdn_norm_rope* nr, const gdn_paged_cache* cache, int kv_dtype,
              void* q_out, int q_dtype, void* k_out, void* stream) {
  CHECK(check_attn_dims(fn, dims, cu));
  if (!valid_dtype(in_dtype) || !valid_dtype(kv_dtype) || !valid_dtype(q_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  if (nr != nullptr) CHECK(check_norm_rope(fn, dims, nr));
  if (dims->total_tokens == 0) return GDN_OK;
  if (q != nullptr) {
    CHECK(check_heads(fn, "q", q, in_dtype));
    REQUIRE_PTR(q_out);
  }
  if (k != nullptr) CHECK(check_heads(fn, "k", k, in_dtype));
  if (v != nullptr) CHECK(check_heads(fn, "v", v, in_dtype));
  if (cache != nullptr) CHECK(check_cache(fn, dims, cache, kv_dtype));
  else if (k != nullptr) REQUIRE_PTR(k_out);
  int* flag = nullptr;
  CHECK(get_flag(&flag));
  gdn::NormRopeArgs p{};
  p.q = heads_in(q); p.k = heads_in(k); p.v = heads_in(v);
  p.q_out = q_out; p.k_out = k_out;
  if (cache != nullptr) p.c = paged_cache(dims, cache);
  if (nr != nullptr) {
    p.qw = nr->q_norm_w; p.kw = nr->k_norm_w; p.eps = nr->norm_eps;
    p.rot = nr->rotary_dim; p.inter = nr->interleaved; p.max_pos = nr->max_positions;
    p.table = nr->cos_sin; p.pos = nr->positions;
  }
  p.cu = cu; p.num_seqs = dims->num_seqs; p.total = dims->total_tokens;
  p.Nq = q != nullptr ? dims->num_q_heads : 0;
  p.Nkv = k != nullptr ? dims->num_kv_heads : 0;
  p.D = dims->head_dim;
  p.in_bf16 = in_dtype == GDN_BF16; p.q_bf16 = q_dtype == GDN_BF16; p.kv_bf16 = kv_dtype == GDN_BF16;
  p.err = flag;
  cudaError_t e = gdn::launch_norm_rope(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

// gdn_paged_attn_decode, and the test hook of its waits (wait_ns > 0).
int attn_decode(const char* fn, const gdn_attn_dims* dims, const int32_t* cu_seqlens, const gdn_heads* q,
                const gdn_heads* gate, int in_dtype, const gdn_paged_cache* cache, float scale, void* o, int out_dtype,
                void* workspace, size_t workspace_bytes, int64_t wait_ns, int skip, void* stream) {
  CHECK(check_attn_dims(fn, dims, cu_seqlens));
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  if (dims->total_tokens == 0) return GDN_OK;
  CHECK(check_heads(fn, "q", q, in_dtype));
  if (gate != nullptr) CHECK(check_heads(fn, "gate", gate, in_dtype));
  CHECK(check_cache(fn, dims, cache, in_dtype));
  REQUIRE_PTR(o);
  const size_t need = gdn::paged_attn_workspace_bytes(dims->num_q_heads, dims->num_kv_heads, dims->head_dim,
                                                      in_dtype == GDN_BF16,
                                                      (int64_t)cache->max_pages * cache->page_size);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
    return fail(GDN_ERR_INVALID_ARG, "%s: workspace of %zu bytes (16-byte aligned) required, got %zu", fn, need,
                workspace_bytes);
  int* flag = nullptr;
  CHECK(get_flag(&flag));
  gdn::PagedAttnArgs p{};
  p.q = heads_in(q); p.gate = heads_in(gate); p.c = paged_cache(dims, cache); p.o = o;
  p.cu = cu_seqlens; p.num_seqs = dims->num_seqs; p.total = dims->total_tokens;
  p.Nq = dims->num_q_heads; p.Nkv = dims->num_kv_heads; p.D = dims->head_dim;
  p.scale = scale; p.in_bf16 = in_dtype == GDN_BF16; p.out_bf16 = out_dtype == GDN_BF16;
  p.ws = workspace; p.err = flag;
  if (wait_ns > 0) p.wait_ns = (unsigned long long)wait_ns;
  p.skip = skip;
  cudaError_t e = gdn::launch_paged_attn(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_version(void) { return (1 << 16) | 0; }

const char* gdn_last_error_string(void) { return g_err; }

int gdn_check_device_error(void* stream) {
  int* flag = nullptr;
  int st = get_flag(&flag);
  if (st != GDN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int host = 0;
  e = cudaMemcpy(&host, flag, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "read device error flag");
  if (host != 0) {
    const int zero = 0;
    e = cudaMemcpy(flag, &zero, sizeof(int), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "clear device error flag");
    return fail(GDN_ERR_DEVICE, "device error %d (%s)", host,
                host == 1   ? "inconsistent cu_seqlens"
                : host == 2 ? "bounded wait timed out"
                : host == 3 ? "kv_lens, a page id or a position out of range"
                            : "?");
  }
  return GDN_OK;
}

int gdn_conv_gating(const gdn_dims* dims, const int32_t* cu_seqlens, const void* mixed_qkv,
                    int in_dtype, const void* conv_w, const void* conv_bias,
                    const void* conv_state_in, void* conv_state_out, const void* a, const void* b,
                    const float* A_log, const float* dt_bias, float q_scale, float l2_eps,
                    void* q, void* k, void* v, int out_dtype, float* g, float* beta,
                    void* stream) {
  const char* fn = "gdn_conv_gating";
  int st = check_dims(fn, dims, cu_seqlens);
  if (st != GDN_OK) return st;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  const int kd = dims->num_k_heads * dims->head_k_dim;
  const int vd = dims->num_v_heads * dims->head_v_dim;
  if (kd % 128 != 0 || vd % 128 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "%s: Nk*Dk and Nv*Dv must be multiples of 128", fn);
  REQUIRE_PTR(conv_w);
  REQUIRE_PTR(A_log);
  REQUIRE_PTR(dt_bias);
  OPTIONAL_PTR(conv_bias);
  OPTIONAL_PTR(conv_state_in);
  OPTIONAL_PTR(conv_state_out);
  if (dims->total_tokens > 0) {
    REQUIRE_PTR(mixed_qkv);
    REQUIRE_PTR(a);
    REQUIRE_PTR(b);
    REQUIRE_PTR(q);
    REQUIRE_PTR(k);
    REQUIRE_PTR(v);
    REQUIRE_PTR(g);
    REQUIRE_PTR(beta);
  }
  int* flag = nullptr;
  st = get_flag(&flag);
  if (st != GDN_OK) return st;
  gdn::ConvGatingArgs p{};
  p.x = mixed_qkv; p.w = conv_w; p.bias = conv_bias;
  p.state_in = conv_state_in; p.state_out = conv_state_out;
  p.a = a; p.b = b; p.A_log = A_log; p.dt_bias = dt_bias;
  p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta;
  p.cu = cu_seqlens; p.num_seqs = dims->num_seqs; p.total = dims->total_tokens;
  p.Nk = dims->num_k_heads; p.Nv = dims->num_v_heads;
  p.Dk = dims->head_k_dim; p.Dv = dims->head_v_dim; p.C = 2 * kd + vd;
  p.q_scale = q_scale; p.l2_eps = l2_eps;
  p.in_bf16 = in_dtype == GDN_BF16; p.out_bf16 = out_dtype == GDN_BF16;
  p.err = flag;
  cudaError_t e = gdn::launch_conv_gating(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_conv_state_steps(const gdn_dims* dims, const int32_t* cu_seqlens, const void* mixed_qkv, int in_dtype,
                         const void* conv_state_in, void* step_states, void* stream) {
  const char* fn = "gdn_conv_state_steps";
  int st = check_dims(fn, dims, cu_seqlens);
  if (st != GDN_OK) return st;
  if (!valid_dtype(in_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  OPTIONAL_PTR(conv_state_in);
  if (dims->total_tokens > 0) {
    REQUIRE_PTR(mixed_qkv);
    REQUIRE_PTR(step_states);
  }
  int* flag = nullptr;
  st = get_flag(&flag);
  if (st != GDN_OK) return st;
  gdn::ConvGatingArgs p{};
  p.x = mixed_qkv;
  p.state_in = conv_state_in;
  p.cu = cu_seqlens;
  p.num_seqs = dims->num_seqs;
  p.total = dims->total_tokens;
  p.C = 2 * dims->num_k_heads * dims->head_k_dim + dims->num_v_heads * dims->head_v_dim;
  p.in_bf16 = in_dtype == GDN_BF16;
  p.err = flag;
  cudaError_t e = gdn::launch_conv_state_steps(p, step_states, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_gating(int64_t rows, int32_t num_v_heads, const void* a, const void* b, int in_dtype,
               const float* A_log, const float* dt_bias, float* g, float* beta, void* stream) {
  const char* fn = "gdn_gating";
  if (rows < 0 || num_v_heads < 1) return fail(GDN_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (!valid_dtype(in_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  REQUIRE_PTR(A_log);
  REQUIRE_PTR(dt_bias);
  if (rows > 0) {
    REQUIRE_PTR(a);
    REQUIRE_PTR(b);
    REQUIRE_PTR(g);
    REQUIRE_PTR(beta);
  }
  gdn::GatingArgs p{a, b, A_log, dt_bias, g, beta, rows, num_v_heads, in_dtype == GDN_BF16};
  cudaError_t e = gdn::launch_gating(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_chunk_prefill_workspace_size(const gdn_dims* dims, size_t* bytes) {
  const char* fn = "gdn_chunk_prefill_workspace_size";
  if (dims == nullptr || bytes == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: NULL argument", fn);
  int st = check_dims(fn, dims, nullptr);
  if (st != GDN_OK && st != GDN_ERR_INVALID_ARG) return st;   // equal split not required here
  *bytes = (dims->head_k_dim == 128 && dims->head_v_dim == 128)
               ? gdn::chunk_tc_workspace_bytes(dims->num_seqs, dims->total_tokens, dims->num_v_heads)
               : 0;
  return GDN_OK;
}

static int chunk_common(const char* fn, const gdn_dims* dims, const int32_t* cu_seqlens,
                        const void* q, const void* k, const void* v, int in_dtype,
                        const float* g, const float* beta, const float* initial_state,
                        float* final_state, void* o, int out_dtype, gdn::ChunkArgs* p) {
  int st = check_dims(fn, dims, cu_seqlens);
  if (st != GDN_OK) return st;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  OPTIONAL_PTR(initial_state);
  OPTIONAL_PTR(final_state);
  if (dims->total_tokens > 0) {
    REQUIRE_PTR(q);
    REQUIRE_PTR(k);
    REQUIRE_PTR(v);
    REQUIRE_PTR(g);
    REQUIRE_PTR(beta);
    REQUIRE_PTR(o);
  }
  int* flag = nullptr;
  st = get_flag(&flag);
  if (st != GDN_OK) return st;
  *p = gdn::ChunkArgs{};
  p->q = q; p->k = k; p->v = v; p->g = g; p->beta = beta;
  p->S0 = initial_state; p->ST = final_state; p->o = o;
  p->cu = cu_seqlens; p->num_seqs = dims->num_seqs; p->total = dims->total_tokens;
  p->Nk = dims->num_k_heads; p->Nv = dims->num_v_heads;
  p->Dk = dims->head_k_dim; p->Dv = dims->head_v_dim;
  p->in_bf16 = in_dtype == GDN_BF16; p->out_bf16 = out_dtype == GDN_BF16;
  p->err = flag;
  return GDN_OK;
}

int gdn_chunk_prefill(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q,
                      const void* k, const void* v, int in_dtype, const float* g,
                      const float* beta, float scale, const float* initial_state,
                      float* final_state, void* o, int out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_chunk_prefill";
  gdn::ChunkArgs p;
  int st = chunk_common(fn, dims, cu_seqlens, q, k, v, in_dtype, g, beta, initial_state,
                        final_state, o, out_dtype, &p);
  if (st != GDN_OK) return st;
  p.scale = scale;
  p.workspace = workspace;
  p.workspace_bytes = workspace_bytes;
  // bf16 q/k/v with 128-wide heads run on the tensor cores; fp32 inputs and
  // other head sizes run the fp32 CUDA-core kernel.
  const bool tc = gdn::chunk_tc_supported(p);
  if (tc && dims->total_tokens > 0) {
    const size_t need = gdn::chunk_tc_workspace_bytes(dims->num_seqs, dims->total_tokens, dims->num_v_heads);
    if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))
      return fail(GDN_ERR_INVALID_ARG, "%s: workspace of %zu bytes (16-byte aligned) required, got %zu", fn,
                  need, workspace_bytes);
  }
  cudaError_t e = tc ? gdn::launch_chunk_tc(p, static_cast<cudaStream_t>(stream))
                     : gdn::launch_chunk_simt(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_chunk_prefill_gated_norm(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q,
                                 const void* k, const void* v, int in_dtype, const float* g,
                                 const float* beta, float scale, const float* initial_state,
                                 float* final_state, const void* z, int z_dtype, const float* norm_w,
                                 float norm_eps, void* y, int out_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const char* fn = "gdn_chunk_prefill_gated_norm";
  gdn::ChunkArgs p;
  int st = chunk_common(fn, dims, cu_seqlens, q, k, v, in_dtype, g, beta, initial_state,
                        final_state, y, out_dtype, &p);
  if (st != GDN_OK) return st;
  if (!valid_dtype(z_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  if (!gdn::chunk_tc_supported(p))
    return fail(GDN_ERR_UNSUPPORTED, "%s: needs bf16 q/k/v and 128-wide heads", fn);
  if (z_dtype != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "%s: z must be bf16", fn);
  REQUIRE_PTR(norm_w);
  if (dims->total_tokens > 0) {
    REQUIRE_PTR(z);
    const size_t need = gdn::chunk_tc_workspace_bytes(dims->num_seqs, dims->total_tokens, dims->num_v_heads);
    if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))
      return fail(GDN_ERR_INVALID_ARG, "%s: workspace of %zu bytes (16-byte aligned) required, got %zu", fn,
                  need, workspace_bytes);
  }
  p.scale = scale;
  p.workspace = workspace;
  p.workspace_bytes = workspace_bytes;
  p.z = z;
  p.norm_w = norm_w;
  p.norm_eps = norm_eps;
  cudaError_t e = gdn::launch_chunk_tc(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_chunk_prefill_fp32(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q,
                           const void* k, const void* v, int in_dtype, const float* g,
                           const float* beta, float scale, const float* initial_state,
                           float* final_state, void* o, int out_dtype, void* stream) {
  const char* fn = "gdn_chunk_prefill_fp32";
  gdn::ChunkArgs p;
  int st = chunk_common(fn, dims, cu_seqlens, q, k, v, in_dtype, g, beta, initial_state,
                        final_state, o, out_dtype, &p);
  if (st != GDN_OK) return st;
  p.scale = scale;
  cudaError_t e = gdn::launch_chunk_simt(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_chunk_prefill_static(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q,
                             const void* k, const void* v, int in_dtype, const float* g,
                             const float* beta, float scale, const float* initial_state,
                             float* final_state, void* o, int out_dtype, void* stream) {
  const char* fn = "gdn_chunk_prefill_static";
  gdn::ChunkArgs p;
  int st = chunk_common(fn, dims, cu_seqlens, q, k, v, in_dtype, g, beta, initial_state,
                        final_state, o, out_dtype, &p);
  if (st != GDN_OK) return st;
  if (!gdn::chunk_tc_supported(p))
    return fail(GDN_ERR_UNSUPPORTED, "%s: needs bf16 q/k/v and 128-wide heads", fn);
  const size_t need = gdn::chunk_tc_workspace_bytes(dims->num_seqs, dims->total_tokens, dims->num_v_heads, false);
  if (need > gdn::kStaticScratchBytes)
    return fail(GDN_ERR_INVALID_ARG,
                "%s: this problem needs %zu bytes of scratch, more than the library's fixed %zu bytes; "
                "use gdn_chunk_prefill with a caller workspace", fn, need, gdn::kStaticScratchBytes);
  void* scratch = nullptr;
  cudaError_t e = gdn::static_scratch(&scratch);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  p.scale = scale;
  p.workspace = scratch;
  p.workspace_bytes = gdn::kStaticScratchBytes;
  p.no_split = 1;                 // the layout checked above
  e = gdn::launch_chunk_tc(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_test_chunk_wait_timeout(const gdn_dims* dims, const void* q, const void* k, const void* v,
                                const float* g, const float* beta, void* o, void* workspace,
                                size_t workspace_bytes, int64_t wait_ns, void* stream) {
  const char* fn = "gdn_test_chunk_wait_timeout";
  gdn::ChunkArgs p;
  int st = chunk_common(fn, dims, nullptr, q, k, v, GDN_BF16, g, beta, nullptr, nullptr, o, GDN_BF16, &p);
  if (st != GDN_OK) return st;
  if (dims->num_seqs != 1 || dims->total_tokens < 1 || !gdn::chunk_tc_supported(p))
    return fail(GDN_ERR_UNSUPPORTED, "%s: needs one sequence of bf16 q/k/v with 128-wide heads", fn);
  if (wait_ns < 1000000 || wait_ns > 10000000000ll)
    return fail(GDN_ERR_INVALID_ARG, "%s: wait_ns must lie in [1 ms, 10 s]", fn);
  const size_t need = gdn::chunk_tc_workspace_bytes(dims->num_seqs, dims->total_tokens, dims->num_v_heads);
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))
    return fail(GDN_ERR_INVALID_ARG, "%s: workspace of %zu bytes (16-byte aligned) required", fn, need);
  p.scale = 1.0f;
  p.workspace = workspace;
  p.workspace_bytes = workspace_bytes;
  p.wait_ns = (unsigned long long)wait_ns;
  p.no_solve = 1;
  cudaError_t e = gdn::launch_chunk_tc(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

static int recurrent_decode(const char* fn, const gdn_dims* dims, const int32_t* cu_seqlens, const void* q,
                            const void* k, const void* v, int in_dtype, const float* g,
                            const float* beta, float scale, float* state, float* step_states, void* o,
                            int out_dtype, void* stream) {
  int st = check_dims(fn, dims, cu_seqlens);
  if (st != GDN_OK) return st;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  REQUIRE_PTR(state);
  OPTIONAL_PTR(step_states);
  if (dims->total_tokens > 0) {
    REQUIRE_PTR(q);
    REQUIRE_PTR(k);
    REQUIRE_PTR(v);
    REQUIRE_PTR(g);
    REQUIRE_PTR(beta);
    REQUIRE_PTR(o);
  }
  int* flag = nullptr;
  st = get_flag(&flag);
  if (st != GDN_OK) return st;
  gdn::DecodeArgs p{};
  p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.state = state; p.o = o;
  p.step_states = step_states;
  p.cu = cu_seqlens; p.num_seqs = dims->num_seqs; p.total = dims->total_tokens;
  p.Nk = dims->num_k_heads; p.Nv = dims->num_v_heads;
  p.Dk = dims->head_k_dim; p.Dv = dims->head_v_dim;
  p.scale = scale; p.in_bf16 = in_dtype == GDN_BF16; p.out_bf16 = out_dtype == GDN_BF16;
  p.err = flag;
  cudaError_t e = gdn::launch_recurrent_decode(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_recurrent_decode(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q,
                         const void* k, const void* v, int in_dtype, const float* g,
                         const float* beta, float scale, float* state, void* o, int out_dtype,
                         void* stream) {
  return recurrent_decode("gdn_recurrent_decode", dims, cu_seqlens, q, k, v, in_dtype, g, beta, scale, state,
                          nullptr, o, out_dtype, stream);
}

int gdn_recurrent_decode_steps(const gdn_dims* dims, const int32_t* cu_seqlens, const void* q,
                               const void* k, const void* v, int in_dtype, const float* g,
                               const float* beta, float scale, float* state, float* step_states, void* o,
                               int out_dtype, void* stream) {
  if (step_states == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "gdn_recurrent_decode_steps: step_states is NULL");
  return recurrent_decode("gdn_recurrent_decode_steps", dims, cu_seqlens, q, k, v, in_dtype, g, beta, scale,
                          state, step_states, o, out_dtype, stream);
}

int gdn_gated_rmsnorm(int64_t rows, int32_t dim, const void* x, int x_dtype, const void* z,
                      int z_dtype, const float* w, float eps, void* y, int out_dtype,
                      void* stream) {
  const char* fn = "gdn_gated_rmsnorm";
  if (rows < 0) return fail(GDN_ERR_INVALID_ARG, "%s: rows < 0", fn);
  if (dim != 64 && dim != 128) return fail(GDN_ERR_UNSUPPORTED, "%s: dim %d not in {64, 128}", fn, dim);
  if (!valid_dtype(x_dtype) || !valid_dtype(z_dtype) || !valid_dtype(out_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  REQUIRE_PTR(w);
  if (rows > 0) {
    REQUIRE_PTR(x);
    REQUIRE_PTR(z);
    REQUIRE_PTR(y);
  }
  gdn::RmsNormArgs p{x, z, w, y, rows, dim, eps, x_dtype == GDN_BF16, z_dtype == GDN_BF16,
                     out_dtype == GDN_BF16};
  cudaError_t e = gdn::launch_gated_rmsnorm(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_decode_fused(const gdn_dims* dims, const void* mixed_qkv, int in_dtype,
                     const void* conv_w, const void* conv_bias, void* conv_state, const void* a,
                     const void* b, const float* A_log, const float* dt_bias, float q_scale,
                     float l2_eps, float* state, const void* z, const float* norm_w,
                     float norm_eps, void* y, int out_dtype, void* stream) {
  const char* fn = "gdn_decode_fused";
  int st = check_dims(fn, dims, nullptr);
  if (st != GDN_OK) return st;
  if (dims->total_tokens != dims->num_seqs)
    return fail(GDN_ERR_INVALID_ARG, "%s: needs exactly one token per sequence", fn);
  if (dims->num_v_heads / dims->num_k_heads > 32)
    return fail(GDN_ERR_UNSUPPORTED, "%s: Nv/Nk > 32", fn);
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
    return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  REQUIRE_PTR(mixed_qkv);
  REQUIRE_PTR(conv_w);
  OPTIONAL_PTR(conv_bias);
  REQUIRE_PTR(conv_state);
  REQUIRE_PTR(a);
  REQUIRE_PTR(b);
  REQUIRE_PTR(A_log);
  REQUIRE_PTR(dt_bias);
  REQUIRE_PTR(state);
  REQUIRE_PTR(z);
  REQUIRE_PTR(norm_w);
  REQUIRE_PTR(y);
  gdn::DecodeFusedArgs p{};
  p.x = mixed_qkv; p.w = conv_w; p.bias = conv_bias; p.conv_state = conv_state;
  p.a = a; p.b = b; p.A_log = A_log; p.dt_bias = dt_bias;
  p.state = state; p.z = z; p.norm_w = norm_w; p.y = y;
  p.B = dims->num_seqs; p.Nk = dims->num_k_heads; p.Nv = dims->num_v_heads;
  p.Dk = dims->head_k_dim; p.Dv = dims->head_v_dim;
  p.C = 2 * p.Nk * p.Dk + p.Nv * p.Dv;
  p.q_scale = q_scale; p.l2_eps = l2_eps; p.norm_eps = norm_eps;
  p.in_bf16 = in_dtype == GDN_BF16; p.out_bf16 = out_dtype == GDN_BF16;
  cudaError_t e = gdn::launch_decode_fused(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return GDN_OK;
}

int gdn_qk_norm_rope(const gdn_attn_dims* dims, const int32_t* cu_seqlens, const gdn_heads* q,
                     const gdn_heads* k, int in_dtype, const gdn_norm_rope* nr, void* q_out,
                     void* k_out, int out_dtype, void* stream) {
  const char* fn = "gdn_qk_norm_rope";
  if (q == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: q is NULL", fn);
  if (nr == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: nr is NULL", fn);
  return norm_rope(fn, dims, cu_seqlens, q, k, nullptr, in_dtype, nr, nullptr, out_dtype, q_out, out_dtype, k_out,
                   stream);
}

int gdn_paged_kv_append(const gdn_attn_dims* dims, const int32_t* cu_seqlens, const gdn_heads* q,
                        const gdn_heads* k, const gdn_heads* v, int in_dtype,
                        const gdn_norm_rope* nr, const gdn_paged_cache* cache, int cache_dtype,
                        void* q_out, int q_dtype, void* stream) {
  const char* fn = "gdn_paged_kv_append";
  if (k == nullptr || v == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: %s is NULL", fn, k == nullptr ? "k" : "v");
  if (cache == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: cache is NULL", fn);
  return norm_rope(fn, dims, cu_seqlens, q, k, v, in_dtype, nr, cache, cache_dtype, q_out, q_dtype, nullptr, stream);
}

int gdn_paged_attn_decode_workspace_size(const gdn_attn_dims* dims, int in_dtype, int64_t table_tokens,
                                         size_t* bytes) {
  const char* fn = "gdn_paged_attn_decode_workspace_size";
  if (dims == nullptr || bytes == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (!valid_dtype(in_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", fn);
  if (table_tokens < 0) return fail(GDN_ERR_INVALID_ARG, "%s: table_tokens < 0", fn);
  gdn_attn_dims d = *dims;
  if (d.num_seqs > 1) d.num_seqs = 1;            // the bounds come with the call: no equal split required here
  CHECK(check_attn_dims(fn, &d, nullptr));
  *bytes = gdn::paged_attn_workspace_bytes(dims->num_q_heads, dims->num_kv_heads, dims->head_dim, in_dtype == GDN_BF16,
                                           table_tokens);
  return GDN_OK;
}

int gdn_paged_attn_decode(const gdn_attn_dims* dims, const int32_t* cu_seqlens, const gdn_heads* q,
                          const gdn_heads* gate, int in_dtype, const gdn_paged_cache* cache,
                          float scale, void* o, int out_dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return attn_decode("gdn_paged_attn_decode", dims, cu_seqlens, q, gate, in_dtype, cache, scale, o, out_dtype, workspace,
                     workspace_bytes, 0, 0, stream);
}

int gdn_test_paged_attn_wait_timeout(const gdn_attn_dims* dims, const int32_t* cu_seqlens, const gdn_heads* q,
                                     int in_dtype, const gdn_paged_cache* cache, void* o, void* workspace,
                                     size_t workspace_bytes, int64_t wait_ns, int skip, void* stream) {
  const char* fn = "gdn_test_paged_attn_wait_timeout";
  if (wait_ns < 1000000 || wait_ns > 10000000000ll)
    return fail(GDN_ERR_INVALID_ARG, "%s: wait_ns must lie in [1 ms, 10 s]", fn);
  if (skip < 1 || skip > 3) return fail(GDN_ERR_INVALID_ARG, "%s: skip must be 1, 2 or 3", fn);
  return attn_decode(fn, dims, cu_seqlens, q, nullptr, in_dtype, cache, 1.0f, o, in_dtype, workspace, workspace_bytes,
                     wait_ns, skip, stream);
}

}  // extern "C"
