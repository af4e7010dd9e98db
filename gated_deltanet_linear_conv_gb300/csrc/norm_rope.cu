// Per-head RMSNorm and position rotation of queries and keys, with dense outputs or
// with k and v written into a paged cache ([QDA], the full-attention layers: q_norm,
// k_norm, partial rotation; section "Cache").
//
// A row is one (token, head) vector x[D]:
//   u = x / sqrt(mean(x^2) + eps) * w;  pairs (a, b) of the first r elements become
//   (a c - b s, b c + a s), with a, b = u[i], u[i + r/2] or u[2i], u[2i + 1].
//
// Bound: HBM, each row read once and written once.  4096 tokens of 40 heads of 128 in bf16 take 17.1 us,
// 75 % of the copy rate (prompts of 16 sequences into pages 25.5, 72 %): 118 to 128 registers leave four
// blocks of four warps per SM, 19 to 20 % of its warps are active, and at that few the latency of
// shared memory and arithmetic shows (issue slots 57 and 52 % active).  What keeps the row loop short:
//  - D/16 lanes hold a row, each two 8-element chunks, D/16 chunks apart: what is done per
//    warp and step serves up to eight rows;
//  - the norm's weights are folded into the token's cosines and sines once, and its factor
//    multiplies the rotated row (both are linear): y = inv (x o (c w) + x' o (+-s w'));
//  - rows come through shared memory by asynchronous copies, kDepth rows ahead, and a lane
//    reads its partners x' there (r is a multiple of 16: a chunk is rotated or passed as a
//    whole and, in the half-split pairing, its partners are one other chunk);
//  - addresses walk by the head stride; element pairs go through the packed fp32x2 operations.

#include "attn_util.cuh"
#include "paged_attn.h"
#include "tc_util.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kDepth = 4;                          // rows in flight per lane group
constexpr int kResident = 4;                       // blocks per SM
// What a block does before its rows costs about so many rows.  0, 5, 10 and 20: prompts of 16 sequences,
// 48 rows of 128 a token, 71.4, 25.8, 25.7 and 31.6 us; 4096 tokens of 40 rows 39.9, 17.5, 17.4 and 17.4.
constexpr int kSetup = 10;
constexpr int kPiece = kThreads * 32;              // bytes of the 16-byte pieces of a step's chunks

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The eight elements of a chunk from shared memory: one 16-byte piece, or two kPiece apart.
__device__ __forceinline__ void fetch(uint32_t at, float2 (&f)[4], bf16) {
  uint32_t w[4];
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
}
__device__ __forceinline__ void fetch(uint32_t at, float2 (&f)[4], float) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(f[2 * i].x), "=f"(f[2 * i].y), "=f"(f[2 * i + 1].x),
                 "=f"(f[2 * i + 1].y) : "r"(at + i * kPiece) : "memory");
}
__device__ __forceinline__ void load_w(const float* p, float2 (&f)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void put(bf16* p, const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __float22bfloat162_rn(f[i]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put(float* p, const float2 (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
__device__ __forceinline__ float rsqrt_approx(float x) {           // 2^-22 relative
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A group of D/16 lanes takes `span` consecutive rows (q heads, then k heads, then v heads) of
// one token, whose metadata and table entries it reads once, behind the first copies.
// Block x: tokens, block y: row ranges.
template <typename Tin, typename Tq, typename Tkv, int D, bool CACHE>
__global__ void __launch_bounds__(kThreads, kResident)
norm_rope_kernel(const __grid_constant__ NormRopeArgs p, int span, Div by_len, Div by_page) {
  constexpr int LPR = D / 16;                      // lanes per row
  constexpr int PIECES = (int)sizeof(Tin) / 2;     // 16-byte pieces of a chunk
  constexpr int BYTES = kPiece * PIECES;           // a step: one row per group
  __shared__ __align__(16) uint8_t ring[kDepth * BYTES];
  const int c = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int t = blockIdx.x * (kThreads / LPR) + group;
  const int k_lo = p.Nq, v_lo = p.Nq + p.Nkv, rows = v_lo + (CACHE ? p.Nkv : 0);
  const int h_lo = blockIdx.y * span, h_hi = min(rows, h_lo + span);
  const bool in_range = t < p.total;
  const uint32_t base = tc::smem_u32(ring) + group * (2 * LPR * 16);

  pdl_launch_next();
  pdl_wait();
  // the copies' cursor: row ch, its source for this lane, the stride to the next row
  const Tin* src = nullptr;
  int64_t src_step = 0;
  int ch = h_lo;
  auto seek = [&]() {
    const HeadsIn& in = ch < k_lo ? p.q : ch < v_lo ? p.k : p.v;
    const int hh = ch < k_lo ? ch : ch < v_lo ? ch - k_lo : ch - v_lo;
    src = static_cast<const Tin*>(in.p) + t * in.ts + hh * in.hs + c * 8;
    src_step = in.hs;
  };
  auto copy_row = [&](uint32_t at) {               // one group of copies, empty behind the last row
    if (in_range && ch < h_hi) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          copy16(base + at + (c + j * LPR) * 16 + i * kPiece, src + j * (D / 2) + i * 4);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++ch;
    src += src_step;
    if (ch == k_lo || ch == v_lo) seek();
  };
  seek();
#pragma unroll 1
  for (int u = 0; u < kDepth; ++u) copy_row(u * BYTES);

  // where the token stands: its sequence, its index there and in the cache
  if (blockIdx.y == 0) check_seqs(p.cu, p.num_seqs, p.total, (int64_t)blockIdx.x * kThreads + threadIdx.x,
                                  (int64_t)gridDim.x * kThreads, p.err);
  bool ok = in_range;
  int pos = 0, page = 0, slot = 0;
  if (CACHE || (p.rot > 0 && p.pos == nullptr) || p.cu != nullptr) {
    int s, bos, eos;
    if (p.cu == nullptr) {
      s = by_len.quot(t);
      bos = s * by_len.d;
      eos = bos + by_len.d;
    } else {
      s = find_seq(p.cu, p.num_seqs, p.total, t);
      ok = ok && seq_bounds(p.cu, p.num_seqs, p.total, s, bos, eos) && t >= bos && t < eos;
    }
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
        const int at = by_page.quot(pos);
        page = __ldg(p.c.bt + (int64_t)s * p.c.max_pages + at);
        slot = pos - at * p.c.page_size;
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

  // this lane's chunks: c and c + LPR; the chunk of each one's partners
  const int half = p.rot / 16;                     // chunks in half of the rotated part
  bool turn[2];
  int chunk[2], mate[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    chunk[j] = c + j * LPR;
    turn[j] = chunk[j] * 8 < p.rot;
    mate[j] = !turn[j] || p.inter ? chunk[j] : chunk[j] < half ? chunk[j] + half : chunk[j] - half;
  }
  uint32_t at = 0;
#pragma unroll 1
  for (int h = h_lo; h < h_hi;) {
    const int kind = h < k_lo ? 0 : h < v_lo ? 1 : 2;
    const int end = min(h_hi, kind == 0 ? k_lo : kind == 1 ? v_lo : rows);
    const float* w = kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr;
    const bool norm = w != nullptr, rotate = kind < 2 && p.rot > 0;
    // factors of this lane's elements and of their partners: weights, then cosines and sines
    float2 fx[2][4], fy[2][4];
    if (norm || rotate) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (norm) {
          load_w(w + chunk[j] * 8, fx[j]);
          load_w(w + mate[j] * 8, fy[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) fx[j][i] = fy[j][i] = make_float2(1.f, 1.f);
        }
        if (rotate && turn[j] && ok) {
          const float* cs = p.table + (int64_t)pos * p.rot;
          const float* sn = cs + p.rot / 2;
          if (p.inter) {
            const float4 co = *reinterpret_cast<const float4*>(cs + chunk[j] * 4);
            const float4 si = *reinterpret_cast<const float4*>(sn + chunk[j] * 4);
            const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              fy[j][i] = make_float2(-ss[i] * fx[j][i].y, ss[i] * fx[j][i].x);
              fx[j][i] = make_float2(cc[i] * fx[j][i].x, cc[i] * fx[j][i].y);
            }
          } else {
            const int low = min(chunk[j], mate[j]) * 8;
            const float2 sign = chunk[j] < half ? make_float2(-1.f, -1.f) : make_float2(1.f, 1.f);
            float2 co[4], si[4];
            load_w(cs + low, co);
            load_w(sn + low, si);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              fx[j][i] = __fmul2_rn(fx[j][i], co[i]);
              fy[j][i] = __fmul2_rn(__fmul2_rn(fy[j][i], si[i]), sign);
            }
          }
        }
      }
    }
    // where the rows go: a q row of its token, a k or v row of its token or its cache slot
    Tq* qo = static_cast<Tq*>(p.q_out) + ((int64_t)t * p.Nq + h) * D + c * 8;
    Tkv* ko = kind == 0  ? nullptr
              : CACHE ? static_cast<Tkv*>(kind == 1 ? p.c.k : p.c.v) + page * p.c.ps + slot * p.c.ss +
                            (h - (kind == 1 ? k_lo : v_lo)) * p.c.hs + c * 8
                      : static_cast<Tkv*>(p.k_out) + ((int64_t)t * p.Nkv + h - k_lo) * D + c * 8;
    const int64_t k_step = CACHE ? p.c.hs : D;
#pragma unroll 1
    for (; h < end; ++h) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      __syncwarp();
      float2 x[2][4], y[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) fetch(base + at + chunk[j] * 16, x[j], Tin());
      if (rotate && !p.inter) {
#pragma unroll
        for (int j = 0; j < 2; ++j) fetch(base + at + mate[j] * 16, y[j], Tin());
      }
      __syncwarp();                                // read by all lanes before it is copied over
      copy_row(at);
      at = at == (kDepth - 1) * BYTES ? 0 : at + BYTES;
      float2 inv = make_float2(1.f, 1.f);
      if (norm) {
        float2 s2 = __fmul2_rn(x[0][0], x[0][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) s2 = __ffma2_rn(x[i / 4][i % 4], x[i / 4][i % 4], s2);
        const float ss = group_sum(s2.x + s2.y, LPR);
        inv.x = inv.y = rsqrt_approx(fmaf(ss, 1.0f / D, p.eps));
      }
      if (norm || rotate) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 mate_x = p.inter ? make_float2(x[j][i].y, x[j][i].x) : y[j][i];
            float2 r = __fmul2_rn(x[j][i], fx[j][i]);
            if (rotate && turn[j]) r = __ffma2_rn(mate_x, fy[j][i], r);
            x[j][i] = norm ? __fmul2_rn(r, inv) : r;
          }
      }
      if (ok) {
        if (kind == 0) {
          put(qo, x[0]);
          put(qo + D / 2, x[1]);
        } else {
          put(ko, x[0]);
          put(ko + D / 2, x[1]);
        }
      }
      qo += D;
      ko += k_step;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename Tin, typename Tq, typename Tkv, int D>
cudaError_t launch_d(const NormRopeArgs& p, cudaStream_t s) {
  const bool cache = p.k_out == nullptr && p.v.p != nullptr;
  const int rows = p.Nq + (cache ? 2 : 1) * p.Nkv;
  if (p.total == 0 || rows == 0) return cudaSuccess;
  const int per_block = kThreads / (D / 16), tblocks = (p.total + per_block - 1) / per_block;
  // Row ranges per token block: the count with the shortest sum of rounds, each a block's set-up
  // and its rows.  (A round that is only just begun is what this avoids: 16 prompts, 313 token
  // blocks of 48 rows, take 29.4 us in two ranges, just over one round, and 25.2 us in three.)
  int span = rows;
  int64_t best = INT64_MAX;
  const int64_t round = (int64_t)kResident * num_sms();
  for (int r = 1; r <= std::min(rows, 64); ++r) {
    const int s_r = (rows + r - 1) / r, used = (rows + s_r - 1) / s_r;
    const int64_t cost = ((int64_t)tblocks * used + round - 1) / round * (kSetup + s_r);
    if (cost < best) {
      best = cost;
      span = s_r;
    }
    if ((int64_t)tblocks * used >= 16 * round) break;              // more rounds than that differ little
  }
  const Div by_len = Div::of(std::max(1, p.total / p.num_seqs)), by_page = Div::of(std::max(1, p.c.page_size));
  const dim3 grid(tblocks, (rows + span - 1) / span);
  return cache ? launch_early(norm_rope_kernel<Tin, Tq, Tkv, D, true>, grid, dim3(kThreads), 0, s, p, span,
                              by_len, by_page)
               : launch_early(norm_rope_kernel<Tin, Tq, Tkv, D, false>, grid, dim3(kThreads), 0, s, p, span,
                              by_len, by_page);
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
