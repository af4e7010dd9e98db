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

// Eight consecutive elements as loaded.
template <typename T> struct Chunk;
template <> struct Chunk<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
};
template <> struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

constexpr int kThreads = 128;
constexpr int kRows = 4;                           // rows of a token that a lane group holds at once

// A group of D/8 lanes takes kRows consecutive rows (q heads, then k heads, then v heads) of
// one token: their loads go out together and first, the token's metadata and its table
// entries, read once for all of them, behind.  Block x: tokens, block y: rows.
template <typename Tin, typename Tq, typename Tkv, int D, bool CACHE>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const __grid_constant__ NormRopeArgs p) {
  constexpr int LPR = D / 8;                       // lanes per row
  const int c = threadIdx.x % LPR;                 // this lane's 8-element chunk of its rows
  const int t = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  const int h0 = blockIdx.y * kRows;
  const int rows = p.Nq + (CACHE ? 2 : 1) * p.Nkv;
  const bool live = t < p.total;
  const int lane = threadIdx.x & 31;

  pdl_launch_next();
  pdl_wait();
  Chunk<Tin> raw[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int h = h0 + u;
    if (live && h < rows) {
      const HeadsIn& in = h < p.Nq ? p.q : h < p.Nq + p.Nkv ? p.k : p.v;
      const int hh = h < p.Nq ? h : h < p.Nq + p.Nkv ? h - p.Nq : h - p.Nq - p.Nkv;
      raw[u].load(static_cast<const Tin*>(in.p) + t * in.ts + hh * in.hs + c * 8);
    }
  }
  // where the token stands: its sequence, its index there and in the cache
  if (blockIdx.y == 0) check_seqs(p.cu, p.num_seqs, p.total, (int64_t)blockIdx.x * kThreads + threadIdx.x,
                                  (int64_t)gridDim.x * kThreads, p.err);
  bool ok = live;
  int pos = 0, page = 0, slot = 0;
  if (CACHE || (p.rot > 0 && p.pos == nullptr) || p.cu != nullptr) {
    const int s = find_seq(p.cu, p.num_seqs, p.total, t);
    int bos = 0, eos = 0;
    ok = ok && seq_bounds(p.cu, p.num_seqs, p.total, s, bos, eos) && t >= bos && t < eos;
    pos = t - bos;
    if (CACHE && ok) {
      bool bad = false;
      const int len = __ldg(p.c.lens + s);
      if (len == 0) {
        ok = false;                                // an inactive sequence: nothing to write
      } else if (len < eos - bos || (int64_t)len > (int64_t)p.c.max_pages * p.c.page_size) {
        bad = true;
      } else {
        pos = len - (eos - bos) + (t - bos);
        page = __ldg(p.c.bt + (int64_t)s * p.c.max_pages + pos / p.c.page_size);
        slot = pos % p.c.page_size;
        bad = page < 0 || page >= p.c.num_pages;
      }
      if (bad) {
        ok = false;
        if (c == 0) raise_error(p.err, kDevErrCache);
      }
    }
  }
  if (p.rot > 0 && ok) {
    if (p.pos != nullptr) pos = __ldg(p.pos + t);
    if (pos < 0 || pos >= p.max_pos) {
      ok = false;
      if (c == 0) raise_error(p.err, kDevErrCache);
    }
  }
  // this lane's cosines and sines: 8 of each half-split, 4 interleaved
  const int half = p.rot / 16;                     // chunks in half of the rotated part
  const bool turn = c * 8 < p.rot;
  const bool low = c < half;
  const int partner = lane - c + (turn ? (low ? c + half : c - half) : c);
  float co[8], si[8];
  if (turn && ok && h0 < p.Nq + p.Nkv) {
    const float* cs = p.table + (int64_t)pos * p.rot;
    if (p.inter) {
      load4(cs + c * 4, *reinterpret_cast<float(*)[4]>(co));
      load4(cs + p.rot / 2 + c * 4, *reinterpret_cast<float(*)[4]>(si));
    } else {
      load8(cs + (low ? c : c - half) * 8, co);
      load8(cs + p.rot / 2 + (low ? c : c - half) * 8, si);
    }
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int h = h0 + u;
    if (h >= rows) break;                          // (the same for the whole block)
    const bool is_q = h < p.Nq, is_v = h >= p.Nq + p.Nkv;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) raw[u].get(x);
    const float* w = is_v ? nullptr : is_q ? p.qw : p.kw;
    if (w != nullptr) {
      float ss = 0.f, wf[8];
      load8(w + c * 8, wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      ss = group_sum(ss, LPR);
      const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wf[i];
    }
    if (p.rot > 0 && !is_v) {
      if (p.inter) {
        if (turn) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * co[i] - b * si[i];
            x[2 * i + 1] = b * co[i] + a * si[i];
          }
        }
      } else {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
        if (turn) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * co[i] + (low ? -y[i] : y[i]) * si[i];
        }
      }
    }
    if (!ok) continue;
    if (is_q) {
      store8(static_cast<Tq*>(p.q_out) + ((int64_t)t * p.Nq + h) * D + c * 8, x);
    } else if (CACHE) {
      const int hh = is_v ? h - p.Nq - p.Nkv : h - p.Nq;
      Tkv* dst = static_cast<Tkv*>(is_v ? p.c.v : p.c.k);
      store8(dst + page * p.c.ps + hh * p.c.hs + slot * p.c.ss + c * 8, x);
    } else {
      store8(static_cast<Tkv*>(p.k_out) + ((int64_t)t * p.Nkv + h - p.Nq) * D + c * 8, x);
    }
  }
}

template <typename Tin, typename Tq, typename Tkv, int D>
cudaError_t launch_d(const NormRopeArgs& p, cudaStream_t s) {
  const bool cache = p.k_out == nullptr && p.v.p != nullptr;
  const int rows = p.Nq + (cache ? 2 : 1) * p.Nkv;
  if (p.total == 0 || rows == 0) return cudaSuccess;
  const int per_block = kThreads / (D / 8);
  const dim3 grid((p.total + per_block - 1) / per_block, (rows + kRows - 1) / kRows);
  return cache ? launch_early(norm_rope_kernel<Tin, Tq, Tkv, D, true>, grid, dim3(kThreads), 0, s, p)
               : launch_early(norm_rope_kernel<Tin, Tq, Tkv, D, false>, grid, dim3(kThreads), 0, s, p);
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
