// Cached tokens of a 4-bit paged cache as dense keys and values: element i of a row is n_i s + m with the
// step s and least value m of its group of 64, in float32, rounded once when stored.
//
// Bound: HBM, 4.5 bits in and 16 or 32 out per element.  A lane takes eight neighbours (one word of
// nibbles in, 16 or 32 bytes out), so that a row's stores are whole lines; a token's page is looked up
// once for all its rows, of which kStep are in flight per lane.

#include "attn_util.cuh"
#include "paged_attn.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = 4;

// The eight values of a word of nibbles, n s + m.  A nibble at bit b of 2^23's mantissa makes 2^23 + n 2^b, so that a mask
// and an exact subtraction give n 2^b, and s 2^-b takes the factor off (s is 0 or above 2^-101); the upper three are moved down first.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t scales, float (&x)[8]) {
  const float s = __uint_as_float(scales << 16), m = __uint_as_float(scales & 0xffff0000u);
  const float2 m2 = make_float2(m, m), off = make_float2(-8388608.f, -8388608.f);
  const float2 s04 = __fmul2_rn(make_float2(s, s), make_float2(1.f, 0x1p-4f));
  const float2 s8c = __fmul2_rn(make_float2(s, s), make_float2(0x1p-8f, 0x1p-12f));
  const float s16 = s * 0x1p-16f;
  const uint32_t v = w >> 20;
  auto at = [](uint32_t word, int b) { return __uint_as_float((word & (15u << b)) | 0x4b000000u); };
  const float2 n[4] = {make_float2(at(w, 0), at(w, 4)), make_float2(at(w, 8), at(w, 12)), make_float2(at(w, 16), at(v, 0)),
                       make_float2(at(v, 4), at(v, 8))};
  const float2 f[4] = {s04, s8c, make_float2(s16, s), make_float2(s04.y, s8c.x)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 y = __ffma2_rn(__fadd2_rn(n[k], off), f[k], m2);
    x[2 * k] = y.x;
    x[2 * k + 1] = y.y;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4ReadArgs p, int span, Div by_len,
                                                            Div by_page) {
  constexpr int LPR = D / 8;                       // lanes per row
  const int c = threadIdx.x % LPR;
  const int64_t t64 = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  // k heads, then v heads, of the outputs that are given
  const int r_lo = (p.k_out == nullptr ? p.Nkv : 0) + blockIdx.y * span;
  const int r_hi = min(p.v_out == nullptr ? p.Nkv : 2 * p.Nkv, r_lo + span);
  pdl_launch_next();
  pdl_wait();
  if (blockIdx.y == 0)
    check_seqs(p.cu, p.num_seqs, p.total, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads, p.err);
  if (t64 >= p.total) return;
  const int t = (int)t64;
  int s, bos, eos;
  bool ok = true;
  if (p.cu == nullptr) {
    s = by_len.quot(t);
    bos = s * by_len.d;
    eos = bos + by_len.d;
  } else {
    s = find_seq(p.cu, p.num_seqs, p.total, t);
    ok = seq_bounds(p.cu, p.num_seqs, p.total, s, bos, eos) && t >= bos && t < eos;
  }
  int page = 0, slot = 0;
  if (ok) {
    const int len = __ldg(p.c.lens + s);
    bool bad = false;
    if (len == 0) {
      ok = false;                                  // an inactive sequence: its rows are zero
    } else if (len < eos - bos || (int64_t)len > (int64_t)p.c.max_pages * p.c.page_size) {
      bad = true;
    } else {
      const int pos = len - (eos - bos) + (t - bos), at = by_page.quot(pos);
      page = __ldg(p.c.bt + (int64_t)s * p.c.max_pages + at);
      slot = pos - at * p.c.page_size;
      bad = page < 0 || page >= p.c.num_pages;
    }
    if (bad) {
      ok = false;
      if (c == 0) raise_error(p.err, kDevErrCache);
    }
  }
  const int64_t at = page * p.c.ps + slot * p.c.ss + c * 4, scale_at = page * p.c.sps + slot * p.c.sss + c / 8;
#pragma unroll 1
  for (int r0 = r_lo; r0 < r_hi; r0 += kStep) {
    uint32_t w[kStep], sm[kStep];
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      const int r = r0 + i, h = r < p.Nkv ? r : r - p.Nkv;
      w[i] = sm[i] = 0;
      if (!ok || r >= r_hi) continue;
      w[i] = __ldg(reinterpret_cast<const uint32_t*>((r < p.Nkv ? p.c.k : p.c.v) + at + h * p.c.hs));
      sm[i] = __ldg((r < p.Nkv ? p.c.ks : p.c.vs) + scale_at + h * p.c.shs);
    }
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      const int r = r0 + i, h = r < p.Nkv ? r : r - p.Nkv;
      if (r >= r_hi) break;
      T* out = static_cast<T*>(r < p.Nkv ? p.k_out : p.v_out);
      float x[8];
      unpack(w[i], sm[i], x);
      store8(out + ((int64_t)t * p.Nkv + h) * D + c * 8, x);
    }
  }
}

template <typename T, int D>
cudaError_t launch_d(const Kv4ReadArgs& p, cudaStream_t s) {
  const int per_block = kThreads / (D / 8), rows = ((p.k_out != nullptr) + (p.v_out != nullptr)) * p.Nkv;
  const int64_t tblocks = ((int64_t)p.total + per_block - 1) / per_block;
  // rows of a token in one block, or split where the tokens alone do not fill the device
  const int64_t want = 8 * num_sms();
  const int parts = (int)std::min<int64_t>((rows + kStep - 1) / kStep, std::max<int64_t>(1, want / tblocks));
  const int span = ((rows + parts - 1) / parts + kStep - 1) / kStep * kStep;
  return launch_early(kv4_read_kernel<T, D>, dim3((unsigned)tblocks, (rows + span - 1) / span), dim3(kThreads), 0, s, p, span,
                      Div::of(std::max(1, p.total / p.num_seqs)), Div::of(p.c.page_size));
}

template <typename T>
cudaError_t launch_t(const Kv4ReadArgs& p, cudaStream_t s) {
  return p.D == 64 ? launch_d<T, 64>(p, s) : p.D == 128 ? launch_d<T, 128>(p, s) : launch_d<T, 256>(p, s);
}

}  // namespace

cudaError_t launch_kv4_read(const Kv4ReadArgs& p, cudaStream_t s) {
  return p.out_bf16 ? launch_t<bf16>(p, s) : launch_t<float>(p, s);
}

}  // namespace gdn
