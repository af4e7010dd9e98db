// Per-head RMSNorm and position rotation of queries and keys, with dense outputs or
// with k and v written into a paged cache ([QDA], the full-attention layers: q_norm,
// k_norm, partial rotation; section "Cache").
//
// A row is one (token, head) vector x[D]:
//   u = x / sqrt(mean(x^2) + eps) * w;  pairs (a, b) of the first r elements become
//   (a c - b s, b c + a s), with a, b = u[i], u[i + r/2] or u[2i], u[2i + 1].
// D/8 lanes hold a row, 8 elements each; r is a multiple of 16, so a lane's 8 elements
// are rotated or passed as a whole and, in the half-split pairing, their partners are
// the 8 elements of one other lane.

#include "common.cuh"
#include "launch.h"

namespace gdn {
namespace {

template <typename Tin, typename Tq, typename Tkv, int D, bool CACHE>
__global__ void __launch_bounds__(256)
norm_rope_kernel(NormRopeArgs p) {
  constexpr int LPR = D / 8;                       // lanes per row
  constexpr int RPW = 32 / LPR;                    // rows per warp
  const int lane = threadIdx.x & 31;
  const int c = lane % LPR;                        // this lane's 8-element chunk of its row
  const int rows_per_token = p.Nq + (CACHE ? 2 : 1) * p.Nkv;
  const int64_t rows = (int64_t)p.total * rows_per_token;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5) * RPW;
  const int64_t first = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * RPW;
  check_seqs(p.cu, p.num_seqs, p.total, (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
             (int64_t)gridDim.x * blockDim.x, p.err);
  for (int64_t r0 = first; r0 < rows; r0 += step) {
    const int64_t row = r0 + lane / LPR;
    const bool live = row < rows;
    const int t = live ? (int)(row / rows_per_token) : 0;
    const int h = live ? (int)(row % rows_per_token) : 0;
    const bool is_q = h < p.Nq, is_v = h >= p.Nq + p.Nkv;
    const HeadsIn in = is_q ? p.q : is_v ? p.v : p.k;
    const int hh = is_q ? h : is_v ? h - p.Nq - p.Nkv : h - p.Nq;

    // where the token stands: its sequence, its index there and in the cache
    const int s = find_seq(p.cu, p.num_seqs, p.total, t);
    int bos = 0, eos = 0, err = 0;
    bool ok = live && seq_bounds(p.cu, p.num_seqs, p.total, s, bos, eos) && t >= bos && t < eos;
    int pos = t - bos, page = 0, slot = 0;
    if (CACHE && ok) {
      const int len = __ldg(p.c.lens + s);
      if (len == 0) {
        ok = false;                                // an inactive sequence: nothing to write
      } else if (len < eos - bos || (int64_t)len > (int64_t)p.c.max_pages * p.c.page_size) {
        err = kDevErrCache;
        ok = false;
      } else {
        pos = len - (eos - bos) + (t - bos);
        page = __ldg(p.c.bt + (int64_t)s * p.c.max_pages + pos / p.c.page_size);
        slot = pos % p.c.page_size;
        if (page < 0 || page >= p.c.num_pages) {
          err = kDevErrCache;
          ok = false;
        }
      }
    }
    if (p.rot > 0 && ok) {
      if (p.pos != nullptr) pos = __ldg(p.pos + t);
      if (pos < 0 || pos >= p.max_pos) {
        err = kDevErrCache;
        ok = false;
      }
    }
    if (live && err != 0 && c == 0) raise_error(p.err, err);

    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (ok) load8(static_cast<const Tin*>(in.p) + t * in.ts + hh * in.hs + c * 8, x);
    const float* w = is_v ? nullptr : is_q ? p.qw : p.kw;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    ss = group_sum(ss, LPR);
    if (w != nullptr) {
      const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
      float wf[8];
      load8(w + c * 8, wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wf[i];
    }
    if (p.rot > 0) {
      const float* cs = p.table + (ok ? (int64_t)pos * p.rot : 0);
      const bool turn = ok && !is_v && c * 8 < p.rot;
      if (p.inter) {
        if (turn) {
          float co[4], si[4];
          load4(cs + c * 4, co);
          load4(cs + p.rot / 2 + c * 4, si);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * co[i] - b * si[i];
            x[2 * i + 1] = b * co[i] + a * si[i];
          }
        }
      } else {
        const int half = p.rot / 16;               // chunks in half of the rotated part
        const bool low = c < half;
        const int partner = lane - c + (c * 8 < p.rot ? (low ? c + half : c - half) : c);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
        if (turn) {
          const int at = (low ? c : c - half) * 8;
          float co[8], si[8];
          load8(cs + at, co);
          load8(cs + p.rot / 2 + at, si);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * co[i] + (low ? -y[i] : y[i]) * si[i];
        }
      }
    }
    if (!ok) continue;
    if (is_q) {
      store8(static_cast<Tq*>(p.q_out) + ((int64_t)t * p.Nq + hh) * D + c * 8, x);
    } else if (CACHE) {
      Tkv* dst = static_cast<Tkv*>(is_v ? p.c.v : p.c.k);
      store8(dst + page * p.c.ps + hh * p.c.hs + slot * p.c.ss + c * 8, x);
    } else {
      store8(static_cast<Tkv*>(p.k_out) + ((int64_t)t * p.Nkv + hh) * D + c * 8, x);
    }
  }
}

template <typename Tin, typename Tq, typename Tkv, int D>
cudaError_t launch_d(const NormRopeArgs& p, cudaStream_t s) {
  const bool cache = p.k_out == nullptr && p.v.p != nullptr;
  const int64_t rows = (int64_t)p.total * (p.Nq + (cache ? 2 : 1) * p.Nkv);
  const int rows_per_block = 8 * 32 / (D / 8);
  const int64_t need = (rows + rows_per_block - 1) / rows_per_block;
  const int blocks = (int)std::min<int64_t>(need, (int64_t)num_sms() * 8);
  if (blocks == 0) return cudaSuccess;
  if (cache) norm_rope_kernel<Tin, Tq, Tkv, D, true><<<blocks, 256, 0, s>>>(p);
  else norm_rope_kernel<Tin, Tq, Tkv, D, false><<<blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename Tin, typename Tq, typename Tkv>
cudaError_t launch_t(const NormRopeArgs& p, cudaStream_t s) {
  return p.D == 64 ? launch_d<Tin, Tq, Tkv, 64>(p, s)
                   : p.D == 128 ? launch_d<Tin, Tq, Tkv, 128>(p, s) : launch_d<Tin, Tq, Tkv, 256>(p, s);
}

template <typename Tin>
cudaError_t launch_in(const NormRopeArgs& p, cudaStream_t s) {
  if (p.q_bf16) return p.kv_bf16 ? launch_t<Tin, bf16, bf16>(p, s) : launch_t<Tin, bf16, float>(p, s);
  return p.kv_bf16 ? launch_t<Tin, float, bf16>(p, s) : launch_t<Tin, float, float>(p, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& p, cudaStream_t s) {
  return p.in_bf16 ? launch_in<bf16>(p, s) : launch_in<float>(p, s);
}

}  // namespace gdn
