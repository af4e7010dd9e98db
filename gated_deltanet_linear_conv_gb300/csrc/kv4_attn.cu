// Attention of the new tokens of each sequence over a paged cache in 4 bits:
//   o[t, h] = sum_j softmax_j(scale q[t, h] . k_j) v_j, then * sigmoid(gate[t, h]),
// with element i of a key or value n_i s_g + m_g, s_g and m_g the step and least value of its
// group g of 64 elements.  The groups' scales stay out of the products:
//   q . k = sum_g s_g (q_g . n_g) + m_g sum(q_g),      o_g = sum_j (p_j s_jg) n_jg + sum_j p_j m_jg,
// so that the matrix instructions multiply whole numbers 0 .. 15, and a value never has to be
// made.  m16n8k16 in f16: a nibble in the low bits of a half-word is the subnormal number n 2^-24,
// one four bits higher 16 n 2^-24, so that a word of eight nibbles becomes four operands by four
// or five masks and byte moves; what the factor of 16 needs is done once, to q before and to o after.  (f16
// products with subnormal numbers are exact, and the sums are float32.)  ldmatrix brings the words to the lanes
// that need them: half-words of four nibbles for its elements, transposed for the values.
//
// Bound: the cache's bytes at HBM rate, 9/16 of a byte per element.  At that rate an SM has 400 issue slots per 16 tokens
// of a kv head of 128; this kernel needs 313, so the arithmetic is kept at word granularity
// throughout.  256 sequences of 512 to 8192, 8 kv heads of 128 (1.26 GB): 247 us, 5.1 TB/s, 75 % of the copy
// rate (in an earlier form of the same time the copies alone 194 us, the arithmetic alone 200) at the 12 warps per SM that 168
// registers leave.
//
// Rows: eight rows (a new token and query head each, all of one kv head) are an octet, the
// narrow side of the products; keys are the 16-row side, so no row of a product is padding:
//   S^T [16 tokens x 8 rows] = K Q^T,   O^T [16 columns of d x 8 rows] += V^T W^T.
// A unit is one pass over a sequence: (sequence, kv head, NT octets).
//
// Weights enter the second product in f16, w = 8 p_j s_jg / r with r, of a row and group, a power of two next to the
// greatest p_j s_jg so far (2^-11 relative; a bf16 output rounds by 2^-8), so that neither what a row does not see nor other rows
// cost it digits, and neither large nor small values leave f16's range; p itself, l = sum p and sum p m are
// float32.  (Bits do differ with the batch: by it go the cuts of units, and when a warp's rows are brought up to date.)
// The running maximum and r are brought up to date only when a lane's weights of a row over that maximum, 2 or 4
// tokens, sum to more than 2^7 or some w passes f16's range: most slices need no exchange between lanes and no
// rescaling.  (One r for all rows took 1 % less, 4 % in two octets, and let rows with other numbers cost each other digits.)
//
// Work split as in the 16-bit kernel: all slices of 16 or 32 tokens of all units lie end to end (a gap of COST for a
// unit's start and join), and each CTA takes an equal range, computed on the device from kv_lens;
// pieces of units that cross ranges go to the workspace, and a second kernel joins them in order.  With short
// tables ranges end at unit borders and nothing is joined.  Inside a CTA four warps take the slices of a piece
// in turn, each with its own ring of stages filled by asynchronous 16-byte copies: a warp waits
// for its own copies only, so the stream needs no barrier between warps and any page size and stride will do.

#include <cuda_fp16.h>

#include "attn_util.cuh"
#include "paged_attn.h"
#include "tc_util.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// Ranges end at unit borders with tables up to kAlignTokens, and up to kAlignMany where there are as many units as CTAs.  Whole
// units against cut ones, us: one sequence of 1000, 16 heads over 2 of 256, 15.6 and 13.6, of 500 10.8 and 13.3; 256 of
// 100 to 900, 32 heads over 8 of 128, 53.2 and 54.5; 32 of 500 to 2000 26.3 and 21.7.
constexpr int kAlignTokens = 512, kAlignMany = 1024;
// A unit's start and join, in tokens, of one octet of rows (below) and of more, which have dearer starts and joins.  160, 320,
// 512 and 640, us: 256 sequences of 512 to 8192, 32 heads over 8 of 128, 269, 260, 262 and 266; 32 of 500 to 2000 26.8, 22.5,
// 23.0 and 23.0; one of 2000, 16 over 2 of 256, 11.5, 13.5, 15.0 and 15.5.  Two octets (24 heads over 8 of 64, 4 or 5 tokens):
// 16 sequences of 0 to 8192 36.7, 28.0, 26.2 and 26.5; 64 of 1000 to 3000 39.8, 39.0, 38.2 and 38.7; 128 of 100 to 9000 150, 137,
// 132 and 133; of 128-wide heads (32 over 8, 3 tokens) 16 of 0 to 8192 42.3, 37.2, 37.1 and 37.9, 64 of 1000 to 3000 66.4,
// 63.6, 63.6 and 64.6.  Four of 64-wide ones (9 tokens): 16 of 0 to 8192 42.2, 38.8, 37.4 and 38.0; 64 of 1000 to 3000 67.9,
// 65.0, 63.9 and 64.9.
constexpr int kUnitCost = 320, kManyUnitCost = 512;
// Tokens of a range at least, where units are cut.  96, 192 and 384, us: one sequence of 1000, 16 heads over 2 of 256, 13.6,
// 14.3 and 18.6; of 8000, 32 over 8 of 128, 13.1, 13.7 and 15.1; 32 of 500 to 2000 21.5, 21.4 and 21.6.
constexpr int kMinTokens = 96;
constexpr int kMaxCtas = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3e38f;                  // the running maximum before the first score
constexpr float kMostWeight = 128.f;               // sum of a lane's weights over the running maximum, by rows
constexpr float kWeight = 8.f;
constexpr float kNoStep = 0x1p120f;                // kWeight / r before the first step

template <int D_, int NT_>
struct Cfg {
  static constexpr int D = D_, NT = NT_;
  static constexpr int NG = D / 64;                // groups of a row
  static constexpr int ROWS = 8 * NT;
  static constexpr int SIZE = NG * NT;             // 16 accumulators each
  static constexpr int OCC = SIZE <= 1 ? 4 : SIZE <= 2 ? 3 : 2;    // CTAs per SM, by the registers they want
  // Blocks of 16 tokens in a slice, a warp's step: two where the registers suffice.  1 and 2, us: 256 sequences as above 293 and
  // 260; 64 of 1000 to 9000, 24 heads over 8 of 64, 57.6 and 52.6; two octets of 64-wide heads, 16 x 5 tokens of 4096 26.7 and
  // 24.7, 64 x 4 of 1000 to 3000 40.6 and 38.2.
  static constexpr int U = NT == 1 || SIZE == 2 ? 2 : 1;
  static constexpr int SLICE = 16 * U;
  static constexpr int COST = (NT > 1 ? kManyUnitCost : kUnitCost) / SLICE;
  static constexpr int KV = SLICE * D / 2;         // bytes of a slice's keys (or values)
  static constexpr int SC = SLICE * NG * 4;        // of their scales
  static constexpr int STAGE = 2 * (KV + SC);
  // Slices in a warp's ring.  As many and one more, us: one sequence of 131072, 16 heads over 2 of 256, 24.9 and 26.3; 64 x 9
  // tokens of 1000 to 3000, 24 over 8 of 64, 65.1 and 65.8; 64 of 1000 to 9000 and 256 sequences as above no difference.
  static constexpr int STAGES = U == 2 ? 2 : 3;
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int JP = D + 4;                 // join row pitch (floats)
  static constexpr int JOIN = kWarps * 8 * (JP + 2) * 4;
  static constexpr int Q = NT * NG * 1024 + ROWS * 4;              // q operands, and a factor of each row's products
  static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + Q;
  static_assert((SMEM + 1024) * OCC <= 228 * 1024 && STAGE % 128 == 0 && KV % 128 == 0, "ring");   // (addresses within a stage go by xor)
};

struct Params {
  Kv4AttnArgs a;
  int G;
  Div by_G, by_page;
  uint32_t ps, hs, ss, sps, shs, sss;              // strides: of k and v in 16 bytes, of the scales in rows of them
  int whole;                                       // pages hold whole blocks of 16 tokens: a block lies in one page
  int align;
  float c;                                         // scale * log2(e)
  struct Rec* rec;                                 // [grid]
  float* part_ml;                                  // [2 * grid][ROWS][2]
  float* part_o;                                   // [2 * grid][ROWS][D]
};
// A unit that starts in a CTA's range and ends behind it; CTA c's is record c.
struct Rec {
  int valid, bos, x0, rows, kvh;
  int pieces;                                      // CTAs c .. c + pieces - 1 hold its pieces
};

__host__ __device__ constexpr size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / x of a power of two
__device__ __forceinline__ float inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t add_half(uint32_t a, uint32_t b) {
  const __half2 s = __hadd2_rn(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}
__device__ __forceinline__ bool finite_half(uint32_t a) {
  return __hble2(*reinterpret_cast<const __half2*>(&a), __half2half2(__ushort_as_half(0x7bff)));
}
// `size` bytes to shared memory; zeros where `take` is not set (src is not read then).
template <int SIZE>
__device__ __forceinline__ void copy(uint32_t dst, const void* src, bool take) {
  const uint32_t n = take ? SIZE : 0;
  if constexpr (SIZE == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(SIZE), "r"(n) : "memory");
}
// Four 8x8 matrices of half-words, row i of matrix k at the address of lane 8 k + i: as they lie, or transposed.
__device__ __forceinline__ void ldsm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N]) {
  if constexpr (N == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
  else if constexpr (N == 2) asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  else asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ float step_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float least_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Where the 16-byte piece c of a row lies in a slice: eight rows' pieces c cover all banks.
template <int NG>
__device__ __forceinline__ uint32_t piece_at(int row, int c) {
  return row * (32 * NG) + ((c ^ (NG == 1 ? row >> 2 & 1 : NG == 2 ? row >> 1 & 3 : row & 7)) * 16);
}

// A sequence as the call sees it; metadata out of range reads as length 0.
struct Seq { int bos, n, len; };
__device__ __forceinline__ Seq load_seq(const Kv4AttnArgs& a, int s, int* err = nullptr) {
  int bos, eos;
  const bool ok = seq_bounds(a.cu, a.num_seqs, a.total, s, bos, eos);
  int len = __ldg(a.c.lens + s);
  const int n = eos - bos;
  const int64_t most = min((int64_t)a.c.max_pages * a.c.page_size, (int64_t)0x7fffff00);
  if (n > 0 && len != 0 && (len < n || len > most)) {
    if (err != nullptr) raise_error(err, kDevErrCache);
    len = 0;
  }
  if (!ok && err != nullptr) raise_error(err, kDevErrSeqlens);
  return {bos, n, n > 0 ? len : 0};
}
template <typename C>
__device__ __forceinline__ int seq_slices(const Seq& q) { return (q.len + C::SLICE - 1) / C::SLICE; }
template <typename C>
__device__ __forceinline__ int seq_groups(const Params& p, const Seq& q) {     // passes per kv head
  return (int)(((int64_t)q.n * p.G + C::ROWS - 1) / C::ROWS);
}
template <typename C>
__device__ __forceinline__ int64_t seq_work(const Params& p, const Seq& q) {
  return q.len == 0 ? 0 : (int64_t)(seq_slices<C>(q) + C::COST) * seq_groups<C>(p, q) * p.a.Nkv;
}
__device__ __noinline__ int64_t div_long(int64_t x, int64_t d) { return x / d; }

// Bounds of the ranges: CTA c of n takes [at(c), at(c + 1)).
struct Ranges {
  int64_t q;
  int r, n;
  __device__ __forceinline__ Ranges(int64_t total, int ctas) : n(ctas) {
    q = total >> 32 ? div_long(total, ctas) : (uint32_t)total / (uint32_t)ctas;
    r = (int)(total - q * ctas);
  }
  __device__ __forceinline__ int64_t at(int c) const { return q * c + min(c, r); }
  __device__ __forceinline__ int before(int64_t end) const {       // CTAs that start before position end > 0
    const int64_t wide = (q + 1) * r;
    return end <= wide ? (int)div_long(end + q, q + 1) : r + (int)div_long(end - wide + q - 1, q);
  }
};

// (Two sequences of 300 tokens beside an inactive slot of 64 and 512 rows of 32 heads of 128, us: by one warp 98 and 715, by the
// grid 11.6 and 11.6; without the slot 8.3.)
__device__ __noinline__ void zero_slots(const Kv4AttnArgs& a, int64_t* scratch) {
  zero_many<kThreads>([&](int s) { return load_seq(a, s); }, a.num_seqs, (int64_t)a.Nq * a.D / 8, a.o, threadIdx.x, scratch,
                      [] { __syncthreads(); });
}

// Four elements of (token t, head h) from d: the gate, and y = o * sigmoid(gate).
__device__ __forceinline__ void gate4(const Kv4AttnArgs& a, int t, int h, int d, float (&g)[4]) {
  if (a.gate.p != nullptr) load4(static_cast<const bf16*>(a.gate.p) + t * a.gate.ts + h * a.gate.hs + d, g);
}
__device__ __forceinline__ void finish4(const Kv4AttnArgs& a, int t, int h, int d, int D, const float (&g)[4], float (&y)[4]) {
  if (a.gate.p != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= rcp(1.f + ex2(-kLog2e * g[i]));
  }
  store4(static_cast<bf16*>(a.o) + ((int64_t)t * a.Nq + h) * D + d, y);
}

// ------------------------------------------------------------------ a warp's share of a piece
template <typename C>
struct Warp {
  static constexpr int NG = C::NG, NT = C::NT, D = C::D;
  float qs[NT][NG][2], cm[NT][2];                  // sum(q_g) and factor of the scores, of columns 2t, 2t + 1
  int lim[NT][2];                                  // tokens that those columns see
  float o[NT][NG][4][4], om[NT][NG][2];            // sums of w n, and (this lane's tokens) of p m
  float m[NT][2], l[NT][2];
  uint32_t x_at, s_at;                             // in a stage: this lane's first matrix row, its first token's scales
  uint32_t q_at;                                   // this lane's q operands: 16 bytes for each octet, group and half of it
  float vs[NT][NG][2];                             // kWeight / r, of columns 2t, 2t + 1

  // Every warp of the CTA writes the same q operands to `qs_`: each reads what it wrote itself.  Returns whether some row has
  // a factor of its products, 2^part below, that is not 1: only slice<true> heeds them.
  __device__ __forceinline__ bool start(const Params& p, const Seq& q, int x0, int rows, int kvh, uint32_t qs_, int lane) {
    q_at = qs_ + lane * 16;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t fs = qs_ + NT * NG * 1024;
    bool far = false;
    // matrices of a group's product: tokens 0..7 and 8..15 of its first 32 elements, then of its others
    x_at = piece_at<NG>(lane & 15, lane >> 4);
    s_at = 2 * C::KV + g * (NG * 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g, x = x0 + r;
      const bool live = r < rows;
      const int tok = p.by_G.quot(x), h = x - tok * p.G;
      const bf16* src = static_cast<const bf16*>(p.a.q.p) + (q.bos + tok) * p.a.q.ts + (kvh * p.G + h) * p.a.q.hs + 8 * t;
      auto load = [&](int gr, float (&v)[16]) {
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
        if (live) {
          load8(src + gr * 64, a);
          load8(src + gr * 64 + 32, b);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = a[i];
          v[8 + i] = b[i];
        }
      };
      float top = 0.f, sum[NG];
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float v[16];
        load(gr, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(v[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // by a power of two, so that the row's largest lies in [2^10, 2^11) (below that where float32 has no greater power):
      // bf16's digits all fit f16
      const int ex = (int)(__float_as_uint(top) >> 23), by = ex == 255 ? 127 : min(254, 264 - ex);
      const float up = __uint_as_float((uint32_t)by << 23);
      // A score is c 2^e times the sum of its products with the row, e = 24 + 127 - by.  Where queries from 2^113 on bring that
      // factor to float32's end, the products get a part of it: a sum that leaves float32 then is one whose score does.
      const int e2 = 151 - by, part = min(127, max(0, (int)(__float_as_uint(p.c) >> 23 & 255) + e2 - 253));
      auto power = [](int i) { return __uint_as_float((uint32_t)(127 + i) << 23); };
      const int e3 = e2 - part;                    // (in two steps: 2^e3 alone may leave the range)
      const float factor = p.c * power(e3 >> 1) * power(e3 - (e3 >> 1));
      far = far || part > 0;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float v[16];                               // (read again: kept, the row would cost 16 NG registers)
        load(gr, v);
        sum[gr] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[i] *= up;
          sum[gr] += v[i];
        }
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
        sum[gr] = (sum[gr] + __shfl_xor_sync(0xffffffffu, sum[gr], 2)) * (5.9604644775390625e-8f * power(part));
        // of step st of half w: elements 2 st, 2 st + 4 (low nibbles), 2 st + 1, 2 st + 5 (high ones)
#pragma unroll
        for (int w = 0; w < 2; ++w)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(q_at + ((nt * NG + gr) * 2 + w) * 512),
                       "r"(pack_half(v[8 * w], v[8 * w + 4])), "r"(pack_half(v[8 * w + 1] * 0.0625f, v[8 * w + 5] * 0.0625f)),
                       "r"(pack_half(v[8 * w + 2], v[8 * w + 6])), "r"(pack_half(v[8 * w + 3] * 0.0625f, v[8 * w + 7] * 0.0625f))
                       : "memory");
      }
      if (t == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(fs + r * 4), "f"(power(part)) : "memory");
      // of the columns: from the lanes that hold those rows
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = (2 * t + e) * 4;
        cm[nt][e] = __shfl_sync(0xffffffffu, factor, from);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) qs[nt][gr][e] = __shfl_sync(0xffffffffu, sum[gr], from);
        const int c = nt * 8 + 2 * t + e;
        lim[nt][e] = c < rows ? q.len - q.n + p.by_G.quot(x0 + c) + 1 : 0;
        m[nt][e] = kLowest;
        l[nt][e] = 0.f;
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        om[nt][gr][0] = om[nt][gr][1] = 0.f;
        vs[nt][gr][0] = vs[nt][gr][1] = kNoStep;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][gr][i][e] = 0.f;
      }
    }
    return __any_sync(0xffffffffu, far);
  }

  // The tokens from tok0 in stage `at`.  TAIL: some column does not see all of them, or start() said so.
  template <bool TAIL>
  __device__ __forceinline__ void slice(uint32_t at, int tok0, int lane) {
    constexpr int U = C::U;
    const int ra = lane >> 2;                      // this lane's tokens: ra and ra + 8 of each 16
    constexpr uint32_t kRow = D / 2;
    const uint32_t xat = at + x_at, sat = at + s_at;               // (a group further on is 32 bytes away by xor)
    float s[U][NT][4], more[NT][2];
    uint32_t ka[U][NG], kb[U][NG];
    if (TAIL) {
      const uint32_t f_at = q_at + NT * NG * 1024 - lane * 16 + (lane & 3) * 8;    // of columns 2t, 2t + 1 (see start)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(more[nt][0]), "=f"(more[nt][1]) : "r"(f_at + nt * 32) : "memory");
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      lds_words<NG>(sat + u * 16 * NG * 4, ka[u]);
      lds_words<NG>(sat + (u * 16 + 8) * NG * 4, kb[u]);
    }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      uint32_t qf[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int w = 0; w < 2; ++w) lds_words<4>(q_at + ((nt * NG + gr) * 2 + w) * 512, qf[nt][w]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t words[4];                         // eight nibbles of token ra, of ra + 8; of the group's other half
        ldsm4((xat ^ (32 * gr)) + u * 16 * kRow, words);
        float acc[NT][4];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const uint32_t x = words[2 * w] >> (8 * st), y = words[2 * w + 1] >> (8 * st);
            const uint32_t a0 = x & 0x000f000fu, a1 = y & 0x000f000fu, a2 = x & 0x00f000f0u, a3 = y & 0x00f000f0u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (w == 0 && st == 0) mma_first(acc[nt], a0, a1, a2, a3, qf[nt][w][2 * st], qf[nt][w][2 * st + 1]);
              else mma(acc[nt], a0, a1, a2, a3, qf[nt][w][2 * st], qf[nt][w][2 * st + 1]);
            }
          }
        const float sa = step_of(ka[u][gr]), ma = least_of(ka[u][gr]), sb = step_of(kb[u][gr]), mb = least_of(kb[u][gr]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (TAIL) {
              acc[nt][e] *= more[nt][e];
              acc[nt][2 + e] *= more[nt][e];
            }
            const float fa = gr == 0 ? ma * qs[nt][gr][e] : fmaf(ma, qs[nt][gr][e], s[u][nt][e]);
            const float fb = gr == 0 ? mb * qs[nt][gr][e] : fmaf(mb, qs[nt][gr][e], s[u][nt][2 + e]);
            s[u][nt][e] = fmaf(sa, acc[nt][e], fa);
            s[u][nt][2 + e] = fmaf(sb, acc[nt][2 + e], fb);
          }
      }
    }
    auto sees = [&](int u, int nt, int e) { return tok0 + u * 16 + ra + (e < 2 ? 0 : 8) < lim[nt][e & 1]; };
    uint32_t va[U][NG], vb[U][NG];
    float p[U][NT][4], add[NT][2];                 // weights, their sums
    uint32_t b0[U][NG][NT], b1[U][NG][NT];         // weights times steps in r / kWeight
    bool raise;
    auto weights = [&]() {
      raise = false;
      uint32_t top = 0;                            // (sums of halves: infinite where a weight is)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (rounded like the maximum it is compared with: far from 0 a fused difference would not be 0 for equal scores)
            p[u][nt][e] = __fsub_rn(__fmul_rn(s[u][nt][e], cm[nt][e & 1]), m[nt][e & 1]);
            if (TAIL && !sees(u, nt, e)) p[u][nt][e] = -INFINITY;
            p[u][nt][e] = ex2(p[u][nt][e]);
          }
        add[nt][0] = p[0][nt][0] + p[0][nt][2];
        add[nt][1] = p[0][nt][1] + p[0][nt][3];
        if (U == 2) {
          add[nt][0] += p[U - 1][nt][0] + p[U - 1][nt][2];
          add[nt][1] += p[U - 1][nt][1] + p[U - 1][nt][3];
        }
        raise = raise || !(add[nt][0] <= kMostWeight) || !(add[nt][1] <= kMostWeight);         // (also for a NaN, which hides others)
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const float sa = step_of(va[u][gr]), sb = step_of(vb[u][gr]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[e] = p[u][nt][e] * vs[nt][gr][e & 1] * (e < 2 ? sa : sb);
              if (TAIL && !sees(u, nt, e)) w[e] = 0.f;             // (what a column does not see may hold anything)
            }
            b0[u][gr][nt] = pack_half(w[0], w[1]);
            b1[u][gr][nt] = pack_half(w[2], w[3]);
            const uint32_t both = add_half(b0[u][gr][nt], b1[u][gr][nt]);
            top = u == 0 && gr == 0 && nt == 0 ? both : add_half(top, both);
          }
        }
      raise = raise || !finite_half(top);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      lds_words<NG>(sat + C::SC + u * 16 * NG * 4, va[u]);
      lds_words<NG>(sat + C::SC + (u * 16 + 8) * NG * 4, vb[u]);
    }
    weights();
    // sums instead of maxima: no term exceeds one, and they are additions where the integer pipe is the busier one
    if (__any_sync(0xffffffffu, raise)) {
      float x[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][nt][e] = TAIL && !sees(u, nt, e) ? -INFINITY : __fmul_rn(s[u][nt][e], cm[nt][e & 1]);
      lift(x, va, vb);
      weights();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt][0] += add[nt][0];
      l[nt][1] += add[nt][1];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const float ma = least_of(va[u][gr]), mb = least_of(vb[u][gr]);
        uint32_t c0[NT], c1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float(&pt)[4] = p[u][nt];
          if (TAIL) {                              // (0 * NaN is NaN)
#pragma unroll
            for (int e = 0; e < 4; ++e) om[nt][gr][e & 1] += sees(u, nt, e) ? pt[e] * (e < 2 ? ma : mb) : 0.f;
          } else {
            om[nt][gr][0] = fmaf(pt[0], ma, fmaf(pt[2], mb, om[nt][gr][0]));
            om[nt][gr][1] = fmaf(pt[1], ma, fmaf(pt[3], mb, om[nt][gr][1]));
          }
          c0[nt] = movm(b0[u][gr][nt]);
          c1[nt] = movm(b1[u][gr][nt]);
        }
        uint32_t words[4];                         // of tokens 2t and 2t + 1, four nibbles each; of 2t + 8, 2t + 9; of the other half
        ldsm4t((xat ^ (32 * gr)) + C::KV + u * 16 * kRow, words);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            // both nibbles of a byte, low + 16 high, stand for the high one: give() takes the low one's share off
            const uint32_t a1 = __byte_perm(words[2 * w], 0, st == 0 ? 0x4240 : 0x4341), a0 = a1 & 0x000f000fu;
            const uint32_t a3 = __byte_perm(words[2 * w + 1], 0, st == 0 ? 0x4240 : 0x4341), a2 = a3 & 0x000f000fu;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(o[nt][gr][2 * w + st], a0, a1, a2, a3, c0[nt], c1[nt]);
          }
      }
    }
  }

  // New maxima and references, the sums so far brought to them.
  __device__ __forceinline__ void lift(const float (&s)[C::U][NT][4], const uint32_t (&va)[C::U][NG],
                                       const uint32_t (&vb)[C::U][NG]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
        if (C::U == 2) mx = fmaxf(mx, fmaxf(s[C::U - 1][nt][e], s[C::U - 1][nt][2 + e]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float now = fmaxf(m[nt][e], mx);
        const float f = now == m[nt][e] ? 1.f : ex2(m[nt][e] - now);
        m[nt][e] = now;
        l[nt][e] *= f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          float top = 0.f;                         // (fmaxf passes over a NaN, which only makes its own columns NaN)
#pragma unroll
          for (int u = 0; u < C::U; ++u)
            top = fmaxf(top, fmaxf(ex2(s[u][nt][e] - now) * step_of(va[u][gr]), ex2(s[u][nt][2 + e] - now) * step_of(vb[u][gr])));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          top = fmaxf(top, f * kWeight * inverse(vs[nt][gr][e]));
          float fo = f;
          const float was = top * vs[nt][gr][e];
          if (was > 2.f * kWeight || was < 0.5f * kWeight) {
            const uint32_t ex = min(max(__float_as_uint(top) >> 23, 27u), 251u);
            const float to = __uint_as_float((254 - ex) << 23) * kWeight;              // kWeight / 2^floor(log2(top))
            fo = fo * inverse(vs[nt][gr][e]) * to; // (in this order at most 2: top is not below the first two)
            vs[nt][gr][e] = to;
          }
          om[nt][gr][e] *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[nt][gr][i][e] *= fo;
            o[nt][gr][i][2 + e] *= fo;
          }
        }
      }
    }
  }

  // Octet nt's rows into the join buffers.
  __device__ __forceinline__ void give(int nt, float* jo, float* jm, float* jl, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l[nt][e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (g == 0) {
        jm[2 * t + e] = m[nt][e];
        jl[2 * t + e] = v;
      }
    }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float back = inverse(vs[nt][gr][e]);  // r / kWeight (times 2^24 it could pass the range)
        float x = om[nt][gr][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float y[4];
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const float low = o[nt][gr][2 * w + st][e] * 16777216.f, both = o[nt][gr][2 * w + st][2 + e] * 16777216.f;
            y[2 * st] = fmaf(low, back, x);
            y[2 * st + 1] = fmaf(both - low, back * 0.0625f, x);
          }
          *reinterpret_cast<float4*>(jo + (2 * t + e) * C::JP + gr * 64 + w * 32 + g * 4) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    }
  }
};

// ------------------------------------------------------------------ the main kernel
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (Cfg<D, NT>::OCC)) kv4_attn_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  // (all of a CTA's shared memory is its ring and q operands: what the start and the joins need lies in the ring)
  int64_t* scan = reinterpret_cast<int64_t*>(smem);                // [kWarps] warp sums
  volatile int64_t* from = scan + kWarps;                          // where the range starts: the sequence's first slice
  volatile int* from_seq = reinterpret_cast<int*>(scan + kWarps + 1);
  const Kv4AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_next();
  pdl_wait();
  // all work, and the sequence that this CTA's range starts in
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int s_lo = min(a.num_seqs, tid * per), s_hi = min(a.num_seqs, s_lo + per);
  int64_t sum = 0;
  const int64_t row = (int64_t)a.Nq * (D / 8);     // 16-byte words of a token's output
  bool many = false;                               // see zero_many
#pragma unroll 1
  for (int s = s_lo; s < s_hi; ++s) {
    const Seq q = load_seq(a, s);
    sum += seq_work<C>(p, q);
    many = many || (q.len == 0 && q.n * row > kFewWords);
  }
  int64_t inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  many = __syncthreads_or(many);
  int64_t before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const Ranges rg(total, (int)max((int64_t)1, min((int64_t)gridDim.x, total / ((p.align ? 1 : kMinTokens / C::SLICE) + C::COST))));
  const bool mine = (int)blockIdx.x < rg.n;
  const int64_t lo = mine ? rg.at(blockIdx.x) : total, hi = mine ? rg.at(blockIdx.x + 1) : total;
  if (before <= lo && lo < before + sum) {
    int64_t at = before;
#pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
      const int64_t w = seq_work<C>(p, load_seq(a, s));
      if (lo < at + w) {
        *from = at;
        *from_seq = s;
        break;
      }
      at += w;
    }
  }
  // sequences with nothing to attend: their rows are zero; every sequence's metadata is checked once
#pragma unroll 1
  for (int s = blockIdx.x * kWarps + warp; s < a.num_seqs; s += gridDim.x * kWarps) {
    const Seq q = load_seq(a, s, lane == 0 ? a.err : nullptr);
    if (q.n > 0 && q.len == 0 && q.n * row <= kFewWords) zero_few(a.o, q.bos * row, q.n * row);
  }
  if (many) zero_slots(a, scan + kWarps + 2);
  __syncthreads();
  Rec rec{};
  if (lo < hi) {
    int s = *from_seq;
    Seq q = load_seq(a, s);
    int64_t seq_at = *from, pos = lo;
    __syncthreads();                               // before the first copies into the ring
    int slices = seq_slices<C>(q), groups = seq_groups<C>(p, q), cost = slices + C::COST;
    int unit = (int)div_long(pos - seq_at, cost);
    if (p.align && seq_at + (int64_t)unit * cost < pos) ++unit;    // the first unit that starts here
    if (p.align) pos = seq_at + (int64_t)unit * cost;
    const uint32_t ring = tc::smem_u32(smem) + warp * (C::STAGES * C::STAGE);
    float* jo = reinterpret_cast<float*>(smem);
    float(*jm)[8] = reinterpret_cast<float(*)[8]>(jo + kWarps * 8 * C::JP);
    float(*jl)[8] = jm + kWarps;
    const uint32_t qat = tc::smem_u32(smem) + C::SMEM - C::Q;
#pragma unroll 1
    while (pos < hi) {
      if (unit >= groups * a.Nkv) {
        seq_at += (int64_t)cost * groups * a.Nkv;
        do {
          if (++s >= a.num_seqs) break;            // (cannot be: pos < hi <= total)
          q = load_seq(a, s);
        } while (q.len == 0);
        if (s >= a.num_seqs) break;
        slices = seq_slices<C>(q);
        groups = seq_groups<C>(p, q);
        cost = slices + C::COST;
        unit = 0;
        continue;
      }
      const int64_t unit_at = seq_at + (int64_t)unit * cost;
      const int t0 = max(0, (int)(pos - unit_at) - C::COST);
      const int t1 = p.align ? slices : (int)min((int64_t)slices, hi - unit_at - C::COST);
      if (t1 <= t0) break;                         // the range ends before the unit's first slice
      const int kvh = unit / groups, x0 = (unit % groups) * C::ROWS;
      const int rows = (int)min((int64_t)C::ROWS, (int64_t)q.n * p.G - x0);

      // ---------------------------------------------------------- the stream of this warp
      const int32_t* bt = a.c.bt + (int64_t)s * a.c.max_pages;
      constexpr int CPR = D / 32, HALF = CPR / 2;  // 16-byte pieces of a row; of 16 rows, per lane
      // this lane's pieces: row lane / CPR (+ 32 / CPR for each further one) at piece_at()
      const uint32_t to = ring + piece_at<C::NG>(lane / CPR, lane % CPR);
      auto to_at = [&](int i) {                    // (rows 4, 8 and 12 on in 256-wide heads, 8 in 128-wide ones: see piece_at)
        return C::NG == 4 ? (to ^ (i & 1) * 64) + i * 512 : to + i * 512;
      };
      const bool whole = p.whole;
      const uint64_t own = (uint64_t)kvh * p.hs + lane % CPR + (whole ? (uint64_t)(lane / CPR) * p.ss : 0);
      const uint64_t sown = (uint64_t)kvh * p.shs + (whole ? (uint64_t)(lane & 15) * p.sss : 0);
      // page and slot of a token of the next slice to copy: this lane's (U = 1: of lane % 16), or, where 16 tokens lie in one
      // page, the first of its 16
      int page, slot;
      auto lookup = [&](int sl) {
        const int tok = sl * C::SLICE + (lane & (C::SLICE - 1) & (whole ? 16 : 31));
        page = -1;
        slot = 0;
        if (sl < t1 && tok < q.len) {
          const int at = p.by_page.quot(tok);
          slot = tok - at * a.c.page_size;
          page = __ldg(bt + at);
          if ((uint32_t)page >= (uint32_t)a.c.num_pages) {
            raise_error(a.err, kDevErrCache);
            page = -1;
          }
        }
      };
      auto issue = [&](int sl, int st) {           // one group of copies, empty behind the piece's end
        if (sl < t1) {
          const uint32_t dst = st * C::STAGE;
#pragma unroll
          for (int u = 0; u < C::U; ++u) {
            uint64_t off = 0;
            bool take = false;
            if (whole) {
              // (rows behind the sequence's last are the page's own, and no column sees them)
              const int pr = C::U == 1 ? page : __shfl_sync(0xffffffffu, page, 16 * u);
              const int sr = C::U == 1 ? slot : __shfl_sync(0xffffffffu, slot, 16 * u);
              take = pr >= 0;
              off = own + (uint64_t)(uint32_t)max(pr, 0) * p.ps + (uint64_t)(uint32_t)sr * p.ss;
            }
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
              if (!whole) {
                const int row = 16 * u + (lane + 32 * i) / CPR;
                const int pr = __shfl_sync(0xffffffffu, page, row), sr = __shfl_sync(0xffffffffu, slot, row);
                take = pr >= 0;
                off = own + (uint64_t)(uint32_t)max(pr, 0) * p.ps + (uint64_t)(uint32_t)sr * p.ss;
              }
              copy<16>(to_at(i) + dst + u * (16 * D / 2), a.c.k + off * 16, take);
              copy<16>(to_at(i) + dst + u * (16 * D / 2) + C::KV, a.c.v + off * 16, take);
              if (whole) off += (uint64_t)(32 / CPR) * p.ss;
            }
          }
          // the scales of row lane (U = 1: of keys, then of values)
          const uint64_t soff = (sown + (uint64_t)(uint32_t)max(page, 0) * p.sps + (uint64_t)(uint32_t)slot * p.sss) * C::NG;
          const uint32_t sto = ring + 2 * C::KV + dst + lane * (4 * C::NG);
          if (C::U == 1) {
            copy<4 * C::NG>(sto, (lane < 16 ? a.c.ks : a.c.vs) + soff, page >= 0);
          } else {
            copy<4 * C::NG>(sto, a.c.ks + soff, page >= 0);
            copy<4 * C::NG>(sto + C::SC, a.c.vs + soff, page >= 0);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      lookup(t0 + warp);
#pragma unroll 1
      for (int i = 0; i < C::STAGES - 1; ++i) {
        issue(t0 + warp + i * kWarps, i);
        lookup(t0 + warp + (i + 1) * kWarps);
      }
      Warp<C> w;
      const bool far = w.start(p, q, x0, rows, kvh, qat, lane);
      __syncwarp();
      const int all = far ? 0 : q.len - q.n + p.by_G.quot(x0) + 1; // the first row's token sees least
      const int most = q.len - q.n + p.by_G.quot(x0 + rows - 1) + 1;
      int st = 0;
#pragma unroll 1
      for (int sl = t0 + warp; sl < t1; sl += kWarps) {
        asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
        __syncwarp();                              // all lanes' copies have landed, and all are done with the stage before
        const int next = sl + (C::STAGES - 1) * kWarps;
        issue(next, st == 0 ? C::STAGES - 1 : st - 1);
        lookup(next + kWarps);
        const int tok0 = sl * C::SLICE;
        if (tok0 + C::SLICE <= all) w.template slice<false>(ring + st * C::STAGE, tok0, lane);
        else if (tok0 < most) w.template slice<true>(ring + st * C::STAGE, tok0, lane);
        st = st == C::STAGES - 1 ? 0 : st + 1;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");

      // ---------------------------------------------------------- the warps' shares joined
      const int slot_out = t0 == 0 && t1 == slices ? -1 : 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
      if (tid == 0 && t0 == 0 && t1 < slices)
        rec = {1, q.bos, x0, rows, kvh, rg.before(unit_at + cost) - (int)blockIdx.x};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= rows) break;
        __syncthreads();                           // the stages, or the octet before, are no longer read
        w.give(nt, jo + warp * 8 * C::JP, jm[warp], jl[warp], lane);
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < 8 * (D / 4); i += kThreads) {
          const int r = i / (D / 4), e = i % (D / 4) * 4, row = nt * 8 + r;
          if (row >= rows) break;
          float mt = kLowest, lt = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kWarps; ++k) mt = fmaxf(mt, jm[k][r]);
#pragma unroll
          for (int k = 0; k < kWarps; ++k) {
            const float f = ex2(jm[k][r] - mt);
            const float4 v = *reinterpret_cast<const float4*>(jo + (k * 8 + r) * C::JP + e);
            lt = fmaf(jl[k][r], f, lt);
            y[0] = fmaf(v.x, f, y[0]); y[1] = fmaf(v.y, f, y[1]);
            y[2] = fmaf(v.z, f, y[2]); y[3] = fmaf(v.w, f, y[3]);
          }
          if (slot_out >= 0) {
            const int64_t at = (int64_t)slot_out * C::ROWS + row;
            store4(p.part_o + at * D + e, y);
            if (e == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(mt, lt);
          } else {
            const float inv = lt == 0.f ? 0.f : rcp(lt);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] *= inv;
            const int t = p.by_G.quot(x0 + row), h = kvh * p.G + x0 + row - t * p.G;
            float gt[4];
            gate4(a, q.bos + t, h, e, gt);
            finish4(a, q.bos + t, h, e, D, gt, y);
          }
        }
      }
      __syncthreads();                             // before the next piece's copies
      pos = unit_at + cost;
      ++unit;
    }
  }
  if (tid == 0 && !p.align) p.rec[blockIdx.x] = rec;
}

// ------------------------------------------------------------------ the join
// Three forms, by how many units can be cut, so that neither blocks start for nothing nor many pieces wait for one
// another: COLS columns of a row go to COLS/4 lanes, the pieces to PG groups of them in turn, whose sums are
// joined through shared memory in order.  PG = 1, about as many units as CTAs (about two pieces each): block (c, y)
// joins the unit that starts in CTA c's range and ends behind it, if there is one.  PG > 1: blocks (u, y) join the
// unit of the u-th CTA with a record.  BATCH pieces of a group are loaded at a time: for PG = 16, where a unit may have
// hundreds, 4 and 10, us: one sequence of 131072, 16 heads over 2 of 256, 26.5 and 24.9 (33.2 with PG = 4); of 30000, 32 over 8
// of 128, 16.7 and 16.1 (20.6 with PG = 4).
constexpr int kJoinThreads = 256;
template <int D, int COLS, int PG, int BATCH = 4>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const __grid_constant__ Params p, int ctas, int rows) {
  constexpr int LPR = COLS / 4, RPB = kJoinThreads / (LPR * PG);   // lanes across a row, rows of a block
  constexpr int PER = (kMaxCtas + kJoinThreads - 1) / kJoinThreads;
  static_assert(RPB >= 1, "rows");
  __shared__ int count[kJoinThreads / 32], found;
  __shared__ Rec found_rec;
  __shared__ __align__(16) float so[PG > 1 ? PG * RPB : 1][COLS + 4];
  __shared__ float sml[PG > 1 ? PG * RPB : 1][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_next();
  pdl_wait();
  int c0 = blockIdx.x;
  Rec u;
  if constexpr (PG == 1) {
    u = p.rec[c0];
    if (!u.valid) return;
  } else {
    // every record is loaded at once, so that finding the one costs no second load
    Rec r[PER];
    uint32_t mask[PER];
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (warp * PER + i) * 32 + lane;
      r[i].valid = 0;
      if (c < ctas) r[i] = p.rec[c];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      mask[i] = __ballot_sync(0xffffffffu, r[i].valid != 0);
      cnt += __popc(mask[i]);
    }
    if (lane == 0) count[warp] = cnt;
    if (tid == 0) found = -1;
    __syncthreads();
    int at = 0;
    for (int i = 0; i < warp; ++i) at += count[i];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (r[i].valid != 0 && at + __popc(mask[i] & ((1u << lane) - 1)) == (int)blockIdx.x) {
        found = (warp * PER + i) * 32 + lane;
        found_rec = r[i];
      }
      at += __popc(mask[i]);
    }
    __syncthreads();
    c0 = found;
    if (c0 < 0) return;
    u = found_rec;
  }
  const int k0 = tid / (LPR * RPB), rl = tid / LPR % RPB, row = blockIdx.y * RPB + rl;
  const int c = tid % LPR * 4, e = blockIdx.z * COLS + c;
  if (blockIdx.y * RPB >= u.rows) return;
  const bool live = row < u.rows;
  float m = kLowest, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f}, gt[4];
  const int t = p.by_G.quot(u.x0 + row), h = u.kvh * p.G + u.x0 + row - t * p.G;
  if (live && k0 == 0) gate4(p.a, u.bos + t, h, e, gt);            // (needed at the end)
#pragma unroll 1
  for (int k = k0; live && k < u.pieces; k += BATCH * PG) {
    float2 ml[BATCH];
    float v[BATCH][4];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      ml[j] = make_float2(kLowest, 0.f);
      v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.f;
      const int i = k + j * PG;
      if (i < u.pieces) {
        // CTA c0's last piece (slot 2 c0 + 1), then the first ones of the CTAs behind it
        const int64_t x = ((int64_t)2 * (c0 + i) + (i == 0 ? 1 : 0)) * rows + row;
        ml[j] = *reinterpret_cast<const float2*>(p.part_ml + x * 2);
        load4(p.part_o + x * D + e, v[j]);
      }
    }
    float now = m;
#pragma unroll
    for (int j = 0; j < BATCH; ++j) now = fmaxf(now, ml[j].x);
    const float f0 = ex2(m - now);
    l *= f0;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= f0;
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const float f = ex2(ml[j].x - now);
      l = fmaf(ml[j].y, f, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fmaf(v[j][i], f, y[i]);
    }
    m = now;
  }
  if constexpr (PG > 1) {
    store4(&so[k0 * RPB + rl][c], y);
    if (c == 0) {
      sml[k0 * RPB + rl][0] = m;
      sml[k0 * RPB + rl][1] = l;
    }
    __syncthreads();
    if (k0 != 0) return;
    float mt = kLowest;
    l = y[0] = y[1] = y[2] = y[3] = 0.f;
#pragma unroll
    for (int k = 0; k < PG; ++k) mt = fmaxf(mt, sml[k * RPB + rl][0]);
#pragma unroll
    for (int k = 0; k < PG; ++k) {
      const float f = ex2(sml[k * RPB + rl][0] - mt);
      float v[4];
      load4(&so[k * RPB + rl][c], v);
      l = fmaf(sml[k * RPB + rl][1], f, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fmaf(v[i], f, y[i]);
    }
  }
  if (!live) return;
  const float inv = l == 0.f ? 0.f : rcp(l);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] *= inv;
  finish4(p.a, u.bos + t, h, e, D, gt, y);
}

// ------------------------------------------------------------------ host
// Octets per pass at most: as many as registers hold the sums and queries of.  Twice as many, us (an earlier form of the kernel,
// registers spilled): 16 x 4 tokens of 4096, 64 heads over 8 of 128, 71 against 56; 16 x 2, 32 over 4 of 256, 50 against 41.
constexpr int most_octets(int D) { return D == 256 ? 1 : D == 128 ? 2 : 4; }
constexpr int occupancy(int D, int nt) { return D / 64 * nt <= 1 ? 4 : D / 64 * nt <= 2 ? 3 : 2; }
int grid_of(int D, int nt) { return std::min(occupancy(D, nt) * num_sms(), kMaxCtas); }
size_t workspace_of(int D, int nt) {
  const size_t grid = grid_of(D, nt), rows = 8 * nt;
  return align16(sizeof(Rec) * grid) + align16(2 * grid * rows * 2 * 4) + 2 * grid * rows * D * 4;
}

template <int D, int NT>
cudaError_t launch_c(const Kv4AttnArgs& a, cudaStream_t s) {
  using C = Cfg<D, NT>;
  static_assert(C::OCC == occupancy(D, NT), "grid");
  const auto fn = kv4_attn_kernel<D, NT>;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  const int grid = grid_of(D, NT);
  Params p{};
  p.a = a;
  p.G = a.Nq / a.Nkv;
  p.by_G = Div::of(p.G);
  p.by_page = Div::of(a.c.page_size);
  p.ps = (uint32_t)(a.c.ps / 16); p.hs = (uint32_t)(a.c.hs / 16); p.ss = (uint32_t)(a.c.ss / 16);
  p.sps = (uint32_t)(a.c.sps / C::NG); p.shs = (uint32_t)(a.c.shs / C::NG); p.sss = (uint32_t)(a.c.sss / C::NG);
  p.whole = a.c.page_size % 16 == 0;
  // at most so many units
  const int64_t rows = (int64_t)p.G * (a.cu == nullptr ? a.total / a.num_seqs : a.total);
  const int64_t units = (int64_t)a.Nkv * (a.cu == nullptr ? (rows + C::ROWS - 1) / C::ROWS * a.num_seqs
                                                          : a.num_seqs + rows / C::ROWS);
  const int64_t table = (int64_t)a.c.max_pages * a.c.page_size;
  p.align = table <= kAlignTokens || (table <= kAlignMany && units >= grid);
  p.c = a.scale * kLog2e;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.rec = reinterpret_cast<Rec*>(ws);
  ws += align16(sizeof(Rec) * grid);
  p.part_ml = reinterpret_cast<float*>(ws);
  ws += align16((size_t)2 * grid * C::ROWS * 2 * 4);
  p.part_o = reinterpret_cast<float*>(ws);
  e = launch_early(fn, dim3(grid), dim3(kThreads), C::SMEM, s, p);
  if (e != cudaSuccess || p.align) return e;
  if (units * 2 >= grid) {
    constexpr int RPB = kJoinThreads / (D / 4);
    return launch_early(kv4_join_kernel<D, D, 1>, dim3(grid, (C::ROWS + RPB - 1) / RPB), dim3(kJoinThreads), 0, s, p, grid,
                        (int)C::ROWS);
  }
  const int n = (int)units;
  if (n * 32 >= grid)
    return launch_early(kv4_join_kernel<D, D, 4>, dim3(n, C::ROWS / (kJoinThreads / D)), dim3(kJoinThreads), 0, s, p, grid,
                        (int)C::ROWS);
  return launch_early(kv4_join_kernel<D, 64, 16, 10>, dim3(n, C::ROWS, D / 64), dim3(kJoinThreads), 0, s, p, grid, (int)C::ROWS);
}

template <int D>
cudaError_t launch_d(const Kv4AttnArgs& a, int nt, cudaStream_t s) {
  if constexpr (most_octets(D) >= 4) {
    if (nt == 4) return launch_c<D, 4>(a, s);
  }
  if constexpr (most_octets(D) >= 2) {
    if (nt == 2) return launch_c<D, 2>(a, s);
  }
  return launch_c<D, 1>(a, s);
}

}  // namespace

// For the most rows of a pass, so that one workspace serves calls of any numbers of tokens.
size_t kv4_attn_workspace_bytes(int D, int64_t table_tokens) {
  if (table_tokens <= kAlignTokens) return 0;
  size_t most = 0;
  for (int nt = 1; nt <= most_octets(D); nt *= 2) most = std::max(most, workspace_of(D, nt));
  return most;
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t s) {
  // octets per pass: enough for the rows of an even batch
  const int64_t want = (int64_t)((a.total + a.num_seqs - 1) / a.num_seqs) * (a.Nq / a.Nkv);
  int nt = 1;
  while (nt * 8 < want && nt < most_octets(a.D)) nt *= 2;
  return a.D == 64 ? launch_d<64>(a, nt, s) : a.D == 128 ? launch_d<128>(a, nt, s) : launch_d<256>(a, nt, s);
}

}  // namespace gdn
