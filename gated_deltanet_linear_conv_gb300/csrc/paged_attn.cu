// Attention of the new tokens of each sequence over its paged cache ([QDA], the
// full-attention layers and section "Cache"):
//   o[t, h] = sum_j softmax_j(scale q[t, h] . k_j) v_j, then * sigmoid(gate[t, h]).
//
// One CTA per (token, query head).  Each warp walks every fourth cached token with a
// running maximum m, sum l and output o of its own: for a new score x,
//   m' = max(m, x);  l <- l e^(m - m') + e^(x - m');  o <- o e^(m - m') + e^(x - m') v,
// and the warps are joined at the end with the same rule.

#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;

template <typename Tin, typename Tout, int D>
__global__ void __launch_bounds__(kWarps * 32)
paged_attn_kernel(PagedAttnArgs p) {
  constexpr int E = D / 32;                        // elements per lane
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, h = blockIdx.y;
  const int kvh = h / (p.Nq / p.Nkv);
  const int s = find_seq(p.cu, p.num_seqs, p.total, t);
  int bos, eos;
  if (h == 0) check_seqs(p.cu, p.num_seqs, p.total, (int64_t)t * blockDim.x + threadIdx.x,
                         (int64_t)p.total * blockDim.x, p.err);
  if (!seq_bounds(p.cu, p.num_seqs, p.total, s, bos, eos) || t < bos || t >= eos) return;
  int len = __ldg(p.c.lens + s);
  if (len != 0 && (len < eos - bos || (int64_t)len > (int64_t)p.c.max_pages * p.c.page_size)) {
    if (threadIdx.x == 0) raise_error(p.err, kDevErrCache);
    len = 0;
  }
  const int end = len == 0 ? 0 : len - (eos - t) + 1;     // sees the cache indices below this
  float q[E], o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = to_f32(static_cast<const Tin*>(p.q.p)[t * p.q.ts + h * p.q.hs + i * 32 + lane]) * p.scale;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < end; j += kWarps) {
    const int page = __ldg(p.c.bt + (int64_t)s * p.c.max_pages + j / p.c.page_size);
    const bool ok = page >= 0 && page < p.c.num_pages;
    if (!ok && lane == 0) raise_error(p.err, kDevErrCache);
    const int64_t at = (ok ? page : 0) * p.c.ps + kvh * p.c.hs + (j % p.c.page_size) * p.c.ss + lane;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) x += ok ? q[i] * to_f32(static_cast<const Tin*>(p.c.k)[at + i * 32]) : 0.f;
    x = group_sum(x, 32);
    const float mn = fmaxf(m, x);
    const float base = mn == -INFINITY ? 0.f : mn;   // scores of -inf so far: weights of 0
    const float a = expf(m - base), e = expf(x - base);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < E; ++i)
      o[i] = o[i] * a + (ok ? e * to_f32(static_cast<const Tin*>(p.c.v)[at + i * 32]) : 0.f);
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) so[warp][i * 32 + lane] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kWarps * 32) {
    float mt = -INFINITY, lt = 0.f, ot = 0.f;
    for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm[w]);
    for (int w = 0; w < kWarps; ++w) {
      if (sm[w] == -INFINITY) continue;            // a warp without tokens
      const float a = expf(sm[w] - mt);
      lt += sl[w] * a;
      ot += so[w][i] * a;
    }
    float y = lt == 0.f ? 0.f : ot / lt;
    if (p.gate.p != nullptr)
      y *= sigmoidf_(to_f32(static_cast<const Tin*>(p.gate.p)[t * p.gate.ts + h * p.gate.hs + i]));
    static_cast<Tout*>(p.o)[((int64_t)t * p.Nq + h) * D + i] = from_f32<Tout>(y);
  }
}

template <typename Tin, typename Tout>
cudaError_t launch_t(const PagedAttnArgs& p, cudaStream_t s) {
  const dim3 grid(p.total, p.Nq);
  if (p.D == 64) paged_attn_kernel<Tin, Tout, 64><<<grid, kWarps * 32, 0, s>>>(p);
  else if (p.D == 128) paged_attn_kernel<Tin, Tout, 128><<<grid, kWarps * 32, 0, s>>>(p);
  else paged_attn_kernel<Tin, Tout, 256><<<grid, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t paged_attn_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_paged_attn(const PagedAttnArgs& p, cudaStream_t s) {
  if (p.in_bf16) return p.out_bf16 ? launch_t<bf16, bf16>(p, s) : launch_t<bf16, float>(p, s);
  return p.out_bf16 ? launch_t<float, bf16>(p, s) : launch_t<float, float>(p, s);
}

}  // namespace gdn
