// Per-head RMSNorm and position rotation of queries and keys, with dense outputs or
// with k and v written into a paged cache ([QDA], the full-attention layers: q_norm,
// k_norm, partial rotation; section "Cache"), in its element type or in 4 bits.
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
//
// In 4 bits a group of 64 elements x of a k or v row (after norm and rotation, in float32) is held as a step s =
// (max - min) / 15 and a least value m = min, both rounded to bf16, and n = (x - m) / s rounded to 0 .. 15 (halves to
// even): x ~ n s + m.  Eight lanes hold a group (four in a 64-wide row), so its extremes take three exchanges each.
// Where a float32 result lies so near to where a rounding turns that its error could decide, the row is done again
// in pairs of floats, so that the stored bits are those of the formulas whatever the order of sums.  The prompts of 16
// sequences above take 28.0 us into 4 bits (19.0 into 16 on the same host), a token of each of 256 sequences 6.8 (3.9).

#include "attn_util.cuh"
#include "paged_attn.h"
#include "tc_util.cuh"

#include <type_traits>

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kDepth = 4;                          // rows in flight per lane group
constexpr int kResident = 4, kResident4 = 3;       // blocks per SM (4 bits: more registers)
// What a block does before its rows costs about so many rows.  0, 5, 10 and 20: prompts of 16 sequences,
// 48 rows of 128 a token, 71.4, 25.8, 25.7 and 31.6 us; 4096 tokens of 40 rows 39.9, 17.5, 17.4 and 17.4.
constexpr int kSetup = 10;
// Into 4 bits, where a k or v row counts as kRow4 and ranges with such rows go first.  The rule above and this one, us: the
// prompts 32.5 and 28.1, 256 tokens of them 8.5 and 7.0, 2048 25.5 and 17.0, 16384 108 and 98.
constexpr int kSetup4 = 4, kRow4 = 8;
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

struct Kv4 {};                                     // the cache's type: 4 bits and group scales

constexpr float kFloatMost = 3.40282347e38f;
// How far a value after norm and rotation in float32 is off, relative to the row's largest: half of the 14 steps
// (2^-24) of the mean square, 2.2 of the root (2^-22.9) and 5 of the products make 14.2 of |a c| + |b s|, which is at
// most the root of (a^2 + b^2) (c^2 + s^2), the sum of the pair's squares after the rotation, whatever c and s: 20.1
// steps of the larger.
constexpr float kRowError = 0x1.6p-20f;            // 22 steps

// x / s by Markstein's correction of a quotient by its exact remainder (r = 1 / s), correctly rounded but for results next to
// the smallest numbers: a quotient that is a half, where the rounding turns, comes out as it is.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// bf16(x) is the same for all values within e of x.
__device__ __forceinline__ bool sure(float x, float e) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x - e)) == __bfloat16_as_ushort(__float2bfloat16_rn(x + e));
}
// The step and the least value as one word; below 2^-100 the quotients' reciprocals and remainders would leave the
// range of normal numbers: the step is 0.
__device__ __forceinline__ uint32_t scales(float range, float lo, float& s, float& m) {
  bf16 sb = __float2bfloat16_rn(range);
  s = __bfloat162float(sb);
  if (!(s >= 0x1p-100f)) {
    s = 0.f;
    sb = __float2bfloat16_rn(0.f);
  }
  const bf16 mb = __float2bfloat16_rn(lo);
  m = __bfloat162float(mb);
  return (uint32_t)__bfloat16_as_ushort(sb) | (uint32_t)__bfloat16_as_ushort(mb) << 16;
}
constexpr uint32_t kNanScales = 0x7fc00000u;

// (NaN if either is)
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A row's groups (this lane's two chunks are of one group where D = 64, else of one each): its nibbles and scales.  A group
// with an infinity or NaN, or whose range passes float32, reads as NaN.  `exact`: the elements are what the formulas
// start from, else they are off by kRowError.  Returns whether that or a rounding could have changed one of the numbers
// (kOpenNumber) or scales (kOpenScale), and, of all lanes of a row whose largest element is not in 2^-60 .. 2^120 and
// not 0, kOutOfRange: a product on the way may have left float32's range, and kRowError does not hold.
//
// Seven operations an element, most on pairs: the quotient (see above) rounds by the addition of 1.5 2^23, whose sum holds
// n in its low bits; the remainder, exact next to where the rounding turns, tells how far from there the element is.
// Only the one nearest counts.  Quotients below 0 or above 15 want m's rounding to be near s: seldom.
constexpr int kOpenNumber = 1, kOpenScale = 2, kOutOfRange = 4;
template <typename Tin, int D>
__device__ __forceinline__ int quantise(const float2 (&x)[2][4], bool exact, uint32_t (&nib)[2], uint32_t (&word)[2]) {
  constexpr int LPR = D / 16, LANES = LPR < 8 ? LPR : 8;           // lanes of a row, of a group
  constexpr float kMagic = 12582912.f;
  float lo[2], hi[2], e = 0.f;
  int open = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    lo[j] = hi[j] = x[j][0].x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[j] = min_nan(lo[j], min_nan(x[j][i].x, x[j][i].y));
      hi[j] = max_nan(hi[j], max_nan(x[j][i].x, x[j][i].y));
    }
  }
  if (D == 64) {
    lo[0] = lo[1] = min_nan(lo[0], lo[1]);
    hi[0] = hi[1] = max_nan(hi[0], hi[1]);
  }
#pragma unroll
  for (int j = 0; j < (D == 64 ? 1 : 2); ++j)
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) {
      lo[j] = min_nan(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], off));
      hi[j] = max_nan(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], off));
    }
  if (D == 64) {
    lo[1] = lo[0];
    hi[1] = hi[0];
  }
  if (!exact) {
    e = max_nan(max_nan(fabsf(lo[0]), fabsf(hi[0])), max_nan(fabsf(lo[1]), fabsf(hi[1])));
    if (LPR > LANES) e = max_nan(e, __shfl_xor_sync(0xffffffffu, e, LANES));
    if (!(e >= 0x1p-60f && e <= 0x1p120f) && e != 0.f) open = kOutOfRange;
    e *= kRowError;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float range = hi[j] - lo[j], fifteenth = range * (1.f / 15.f);
    float s, m;
    word[j] = scales(fifteenth, lo[j], s, m);
    const bool fine = range <= kFloatMost;
    const float r = s > 0.f ? rcp_approx(s) : 0.f; // (what its error changes shows in the remainder)
    // where a difference from m is sure to be exact (short numbers, not too far apart), halves decide as they are
    const bool shorts = sizeof(Tin) == 2 && exact;
    uint32_t lost = shorts && m != 0.f && fabsf(m) < 0x1p-15f * range;
    const float2 m2 = make_float2(-m, -m), r2 = make_float2(r, r), s2 = make_float2(-s, -s);
    const float2 up2 = make_float2(kMagic, kMagic), down2 = make_float2(-kMagic, -kMagic);
    float worst = 0.f;
    float2 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = x[j][i], d = __fadd2_rn(v, m2), q = __fmul2_rn(d, r2);
      t[i] = __fadd2_rn(__ffma2_rn(__ffma2_rn(q, s2, d), r2, q), up2);
      const float2 rem = __ffma2_rn(__fadd2_rn(t[i], down2), s2, d);
      worst = fmaxf(worst, fmaxf(fabsf(rem.x), fabsf(rem.y)));
      if (shorts) {
        const float2 back = __fadd2_rn(d, make_float2(m, m));
        lost |= (__float_as_uint(back.x) ^ __float_as_uint(v.x)) & 0x7fffffffu;        // (-0 + 0 is 0)
        lost |= (__float_as_uint(back.y) ^ __float_as_uint(v.y)) & 0x7fffffffu;
      }
    }
    if (fabsf(m) * 0x1p-8f > 0.4f * s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[i].x = fminf(fmaxf(t[i].x, kMagic), kMagic + 15.f);
        t[i].y = fminf(fmaxf(t[i].y, kMagic), kMagic + 15.f);
      }
    }
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += (__float_as_uint(t[i].x) << (8 * i)) + (__float_as_uint(t[i].y) << (8 * i + 4));
    // 0x4b400000 is the magic number's pattern
    nib[j] = fine ? sum - 0x4b400000u * 0x11111111u : 0u;
    const float et = shorts ? 0.f : fmaf(s, 0x1p-19f, e);
    if (fine) {
      if (s > 0.f && (lost != 0 || !(worst <= 0.5f * s - et))) open |= kOpenNumber;
      // (two ends' errors, 2 e / 15, two roundings, and the constant's)
      if (!sure(fifteenth, fmaf(fifteenth, 0x1p-22f, 0.134f * e)) || !sure(lo[j], e)) open |= kOpenScale;
    } else {
      word[j] = kNanScales;
    }
  }
  return open;
}

// Pairs of floats whose sum stands for a number to some 46 bits: sums, products and the error of each by the exact
// operations of Dekker and Knuth (and the product's by one fused operation).
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair norm2(float a, float b) {          // |a| >= |b|
  const float h = __fadd_rn(a, b);
  return {h, __fsub_rn(b, __fsub_rn(h, a))};
}
__device__ __forceinline__ Pair sum2(float a, float b) {
  const float h = __fadd_rn(a, b), t = __fsub_rn(h, a);
  return {h, __fadd_rn(__fsub_rn(a, __fsub_rn(h, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair product2(float a, float b) {
  const float h = __fmul_rn(a, b);
  return {h, __fmaf_rn(a, b, -h)};
}
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  const Pair t = sum2(a.h, b.h);
  return norm2(t.h, __fadd_rn(t.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair operator*(const Pair& a, const Pair& b) {
  const Pair t = product2(a.h, b.h);
  return norm2(t.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, t.l)));
}
__device__ __forceinline__ bool operator<(const Pair& a, const Pair& b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }

// The same with what float32 cannot decide done again from the stored row in pairs of floats (one row in a hundred has such
// a value): what 4 bits hold does not depend on the order of any sum.  (In float64 this took 8 us on GB300, which has
// few units for it, longer than the rest of a decode step's append.)  Only the elements in question are done again: where
// a scale is open those that can be a group's least or greatest, then those next to where a rounding turns.  x[8 j + i]:
// this lane's elements in float32, off by kRowError if not `as_is`; `row` null: no such row (its lanes only take part).
template <typename Tin, int D>
__device__ __noinline__ void quantise_closely(const float (&x)[16], int open, bool as_is, const Tin* row, const float* w,
                                              const float* cs, int rot, int inter, float eps, uint32_t (&nib)[2],
                                              uint32_t (&word)[2]) {
  constexpr int LPR = D / 16, LANES = LPR < 8 ? LPR : 8;
  const int c = threadIdx.x % LPR, half = rot / 16;
  float e = 0.f;
  if (!as_is) {
#pragma unroll
    for (int i = 0; i < 16; ++i) e = fmaxf(e, fabsf(x[i]));
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, off));
    e *= kRowError;
  }
  Pair inv{1.f, 0.f};
  if (w != nullptr) {
    Pair ss[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (row != nullptr) load8(row + (c + j * LPR) * 8, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const Pair q = product2(v[i], v[i]), t = sum2(ss[j].h, q.h);
        ss[j] = {t.h, __fadd_rn(ss[j].l, __fadd_rn(t.l, q.l))};
      }
    }
    Pair ms = norm2(ss[0].h, ss[0].l) + norm2(ss[1].h, ss[1].l);
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1)
      ms = ms + Pair{__shfl_xor_sync(0xffffffffu, ms.h, off), __shfl_xor_sync(0xffffffffu, ms.l, off)};
    ms = Pair{ms.h * (1.f / D), ms.l * (1.f / D)} + Pair{eps, 0.f};
    // from the float32 root y: 1 / sqrt(ms) = y (1 - d)^(-1/2), d = 1 - ms y^2 some 2^-21, by its series to d^2
    const float y = rsqrt_approx(ms.h);
    const Pair one = ms * product2(y, y);
    const float d = __fsub_rn(__fsub_rn(1.f, one.h), one.l);
    inv = norm2(y, y * d * fmaf(0.375f, d, 0.5f));
  }
  auto exact = [&](int k) -> Pair {                // element k of this lane
    const int chunk = c + (k >> 3) * LPR, at = chunk * 8 + (k & 7);
    const float a0 = to_f32(row[at]);
    Pair a = w == nullptr ? Pair{a0, 0.f} : product2(a0, w[at]) * inv;
    if (cs == nullptr || at >= rot) return a;
    const int other = inter ? at ^ 1 : chunk < half ? at + rot / 2 : at - rot / 2, p = inter ? at / 2 : min(at, other);
    const float b0 = to_f32(row[other]), sn = cs[rot / 2 + p];
    const Pair b = w == nullptr ? Pair{b0, 0.f} : product2(b0, w[other]) * inv;
    return a * Pair{cs[p], 0.f} + b * Pair{at < other ? -sn : sn, 0.f};
  };
  uint32_t todo = 0;
  bool moved[2] = {false, false};                  // a group whose scales came out otherwise
  if (__any_sync(0xffffffffu, open & kOpenScale)) {
    // least and greatest (D = 64: both chunks are of one group)
    float l[2], h[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      l[j] = h[j] = x[8 * j];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        l[j] = min_nan(l[j], x[8 * j + i]);
        h[j] = max_nan(h[j], x[8 * j + i]);
      }
    }
    if (D == 64) {
      l[0] = l[1] = min_nan(l[0], l[1]);
      h[0] = h[1] = max_nan(h[0], h[1]);
    }
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[j] = min_nan(l[j], __shfl_xor_sync(0xffffffffu, l[j], off));
        h[j] = max_nan(h[j], __shfl_xor_sync(0xffffffffu, h[j], off));
      }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (row != nullptr && h[i / 8] - l[i / 8] <= kFloatMost &&
          (x[i] <= l[i / 8] + 2.f * e || x[i] >= h[i / 8] - 2.f * e))
        todo |= 1u << i;
    Pair lo[2], hi[2];
    lo[0] = lo[1] = {INFINITY, 0.f};
    hi[0] = hi[1] = {-INFINITY, 0.f};
    while (todo != 0) {
      const int k = __ffs(todo) - 1;
      todo &= todo - 1;
      const Pair v = exact(k);
      if (D == 64 || k < 8) {
        if (v < lo[0]) lo[0] = v;
        if (hi[0] < v) hi[0] = v;
      } else {
        if (v < lo[1]) lo[1] = v;
        if (hi[1] < v) hi[1] = v;
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < (D == 64 ? 1 : 2); ++j) {
#pragma unroll
      for (int off = LANES / 2; off > 0; off >>= 1) {
        const Pair a{__shfl_xor_sync(0xffffffffu, lo[j].h, off), __shfl_xor_sync(0xffffffffu, lo[j].l, off)};
        const Pair b{__shfl_xor_sync(0xffffffffu, hi[j].h, off), __shfl_xor_sync(0xffffffffu, hi[j].l, off)};
        if (a < lo[j]) lo[j] = a;
        if (hi[j] < b) hi[j] = b;
      }
      if (!(h[j] - l[j] <= kFloatMost) || row == nullptr) continue;
      const Pair range = hi[j] + Pair{-lo[j].h, -lo[j].l};
      const float f = __fdiv_rn(range.h, 15.f);
      float s, m;
      const uint32_t now = scales(__fadd_rn(f, __fadd_rn(__fmaf_rn(-f, 15.f, range.h), range.l) * (1.f / 15.f)), lo[j].h, s, m);
      moved[j] = now != word[j];
      word[j] = now;
    }
    if (D == 64) moved[1] = moved[0];
  }
  // the elements
  float s[2], m[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t wd = word[D == 64 ? 0 : j];
    s[j] = __uint_as_float(wd << 16);
    m[j] = __uint_as_float(wd & 0xffff0000u);
    if (moved[j]) {
      const float r = s[j] > 0.f ? __frcp_rn(s[j]) : 0.f;
      nib[j] = 0;
#pragma unroll 1
      for (int i = 0; i < 8; ++i)
        nib[j] |= (uint32_t)fminf(fmaxf(rintf(quotient(x[8 * j + i] - m[j], s[j], r)), 0.f), 15.f) << (4 * i);
    }
    if (!(s[j] > 0.f) || row == nullptr) continue; // (one value, or NaN)
    const float near = 0.5f * s[j] - fmaf(s[j], 0x1p-18f, e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float rem = __fmaf_rn(-(float)((nib[j] >> (4 * i)) & 15u), s[j], x[8 * j + i] - m[j]);
      if (!(fabsf(rem) <= near)) todo |= 1u << (8 * j + i);
    }
  }
  while (todo != 0) {
    const int k = __ffs(todo) - 1, at = 4 * (k & 7);
    const bool up = k >= 8;
    todo &= todo - 1;
    const float sj = up ? s[1] : s[0];
    const Pair d = exact(k) + Pair{-(up ? m[1] : m[0]), 0.f};
    // from the pair: float32's own number is off by more than one where a group's range is a few of its values' last digits
    const uint32_t n = (uint32_t)fminf(fmaxf(rintf(__fmul_rn(d.h, rcp_approx(sj))), 0.f), 15.f);
    // above (n + 1/2) s, below (n - 1/2) s, or on one of them: these differences are exact next to 0
    const float over = __fadd_rn(__fmaf_rn(-((float)n + 0.5f), sj, d.h), d.l);
    const float under = __fadd_rn(__fmaf_rn(-((float)n - 0.5f), sj, d.h), d.l);
    uint32_t to = n;                               // (off by one at most)
    if (n < 15 && (over > 0.f || (over == 0.f && n % 2 == 1))) to = n + 1;
    if (n > 0 && (under < 0.f || (under == 0.f && n % 2 == 1))) to = n - 1;
    if (up) nib[1] = (nib[1] & ~(15u << at)) | to << at;
    else nib[0] = (nib[0] & ~(15u << at)) | to << at;
  }
  __syncwarp();
}

// A row whose mean square or result leaves the range in which float32 keeps its digits: all of it in float64.
template <typename Tin, int D>
__device__ __noinline__ void quantise_wild(const Tin* row, const float* w, const float* cs, int rot, int inter, float eps,
                                           uint32_t (&nib)[2], uint32_t (&word)[2]) {
  constexpr int LPR = D / 16, LANES = LPR < 8 ? LPR : 8;
  const int c = threadIdx.x % LPR, half = rot / 16;
  double inv = 1.0, x[16], lo[2] = {INFINITY, INFINITY}, hi[2] = {-INFINITY, -INFINITY};
  if (w != nullptr) {
    double ss = 0.0;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const double v = row == nullptr ? 0.0 : (double)to_f32(row[(c + i / 8 * LPR) * 8 + i % 8]);
      ss = fma(v, v, ss);
    }
#pragma unroll 1
    for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    inv = 1.0 / sqrt(ss / D + (double)eps);
  }
  bool fine[2] = {true, true};
#pragma unroll 1
  for (int k = 0; k < 16; ++k) {
    const int chunk = c + (k >> 3) * LPR, at = chunk * 8 + (k & 7), j = D == 64 ? 0 : k >> 3;
    x[k] = 0.0;
    if (row != nullptr) {
      x[k] = (double)to_f32(row[at]) * (w == nullptr ? 1.0 : inv * (double)w[at]);
      if (cs != nullptr && at < rot) {
        const int other = inter ? at ^ 1 : chunk < half ? at + rot / 2 : at - rot / 2, p = inter ? at / 2 : min(at, other);
        const double b = (double)to_f32(row[other]) * (w == nullptr ? 1.0 : inv * (double)w[other]);
        x[k] = fma(at < other ? -b : b, (double)cs[rot / 2 + p], x[k] * (double)cs[p]);
      }
    }
    fine[j] = fine[j] && fabs(x[k]) <= (double)kFloatMost;
    lo[j] = fmin(lo[j], x[k]);
    hi[j] = fmax(hi[j], x[k]);
  }
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const int from = D == 64 ? 0 : j;
    double a = fine[from] ? lo[from] : -INFINITY, b = hi[from];
#pragma unroll 1
    for (int off = LANES / 2; off > 0; off >>= 1) {
      a = fmin(a, __shfl_xor_sync(0xffffffffu, a, off));
      b = fmax(b, __shfl_xor_sync(0xffffffffu, b, off));
    }
    float s, m;
    word[j] = scales(__double2float_rn((b - a) / 15.0), __double2float_rn(a), s, m);
    nib[j] = 0;
    if (!(b - a <= (double)kFloatMost)) {
      word[j] = kNanScales;
    } else if (s > 0.f) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i)
        nib[j] |= (uint32_t)fmin(fmax(rint((x[8 * j + i] - (double)m) / (double)s), 0.0), 15.0) << (4 * i);
    }
  }
}

// A group of D/16 lanes takes `span` consecutive rows (q heads, then k heads, then v heads) of
// one token, whose metadata and table entries it reads once, behind the first copies.
// Block x: tokens, block y: row ranges.
template <typename Tin, typename Tq, typename Tkv, int D, bool CACHE>
__global__ void __launch_bounds__(kThreads, std::is_same<Tkv, Kv4>::value ? kResident4 : kResident)
norm_rope_kernel(const __grid_constant__ NormRopeArgs p, const __grid_constant__ PagedCache4 p4, int span, Div by_len,
                 Div by_page) {
  constexpr bool FOUR = std::is_same<Tkv, Kv4>::value;
  using Tout = typename std::conditional<FOUR, uint8_t, Tkv>::type;
  constexpr int LPR = D / 16;                      // lanes per row
  constexpr int PIECES = (int)sizeof(Tin) / 2;     // 16-byte pieces of a chunk
  constexpr int BYTES = kPiece * PIECES;           // a step: one row per group
  __shared__ __align__(16) uint8_t ring[kDepth * BYTES];
  const int c = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int t = blockIdx.x * (kThreads / LPR) + group;
  const int k_lo = p.Nq, v_lo = p.Nq + p.Nkv, rows = v_lo + (CACHE ? p.Nkv : 0);
  const int h_lo = (FOUR ? gridDim.y - 1 - blockIdx.y : blockIdx.y) * span, h_hi = min(rows, h_lo + span);
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
    Tout* ko = kind == 0 || FOUR ? nullptr
              : CACHE ? static_cast<Tout*>(kind == 1 ? p.c.k : p.c.v) + page * p.c.ps + slot * p.c.ss +
                            (h - (kind == 1 ? k_lo : v_lo)) * p.c.hs + c * 8
                      : static_cast<Tout*>(p.k_out) + ((int64_t)t * p.Nkv + h - k_lo) * D + c * 8;
    const int64_t k_step = CACHE ? p.c.hs : D;
    uint8_t* k4 = nullptr;
    uint32_t* k4s = nullptr;
    if (FOUR && kind != 0) {
      const int hh = h - (kind == 1 ? k_lo : v_lo);
      k4 = (kind == 1 ? p4.k : p4.v) + page * p4.ps + slot * p4.ss + hh * p4.hs + c * 4;
      k4s = (kind == 1 ? p4.ks : p4.vs) + page * p4.sps + slot * p4.sss + hh * p4.shs;
    }
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
      bool wild = false;                           // see quantise_wild
      if (norm) {
        float2 s2 = __fmul2_rn(x[0][0], x[0][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) s2 = __ffma2_rn(x[i / 4][i % 4], x[i / 4][i % 4], s2);
        const float ss = group_sum(s2.x + s2.y, LPR);
        const float ms = fmaf(ss, 1.0f / D, p.eps);
        inv.x = inv.y = rsqrt_approx(ms);
        wild = !(ms >= 0x1p-80f && ms <= 0x1p120f);
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
      if constexpr (FOUR) {
        if (kind != 0) {                           // (all lanes of a warp together: a group's exchanges need them)
          uint32_t nib[2], word[2];
          const int open = quantise<Tin, D>(x, !(norm || rotate), nib, word);
          wild = wild || (open & kOutOfRange) != 0;
          const bool any_wild = __any_sync(0xffffffffu, ok && wild);
          if (any_wild || __any_sync(0xffffffffu, ok && open != 0)) {
            const HeadsIn& in = kind == 1 ? p.k : p.v;
            const Tin* row = static_cast<const Tin*>(in.p) + t * in.ts + (h - (kind == 1 ? k_lo : v_lo)) * in.hs;
            const float* cs = rotate && ok ? p.table + (int64_t)pos * p.rot : nullptr;
            float xs[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) xs[i] = i % 2 ? x[i / 8][i % 8 / 2].y : x[i / 8][i % 8 / 2].x;
            quantise_closely<Tin, D>(xs, open, !(norm || rotate), ok && !wild ? row : nullptr, w, cs, p.rot, p.inter, p.eps,
                                     nib, word);
            if (any_wild) {
              uint32_t wn[2], ww[2];
              quantise_wild<Tin, D>(ok && wild ? row : nullptr, w, cs, p.rot, p.inter, p.eps, wn, ww);
              if (wild) {
                nib[0] = wn[0]; nib[1] = wn[1];
                word[0] = ww[0]; word[1] = ww[1];
              }
            }
          }
          if (ok) {
            *reinterpret_cast<uint32_t*>(k4) = nib[0];
            *reinterpret_cast<uint32_t*>(k4 + D / 4) = nib[1];
            if (D == 64) {
              if (c == 0) *k4s = word[0];
            } else if (c % 8 == 0) {
              k4s[c / 8] = word[0];
              k4s[(c + LPR) / 8] = word[1];
            }
          }
          k4 += p4.hs;
          k4s += p4.shs;
        }
      }
      if (ok) {
        if (kind == 0) {
          put(qo, x[0]);
          put(qo + D / 2, x[1]);
        } else if constexpr (!FOUR) {
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
  constexpr bool FOUR = std::is_same<Tkv, Kv4>::value;
  const bool cache = FOUR || (p.k_out == nullptr && p.v.p != nullptr);
  const int rows = p.Nq + (cache ? 2 : 1) * p.Nkv;
  if (p.total == 0 || rows == 0) return cudaSuccess;
  const int per_block = kThreads / (D / 16), tblocks = (p.total + per_block - 1) / per_block;
  // Row ranges per token block: the count with the shortest sum of rounds, each a block's set-up
  // and its rows.  (A round that is only just begun is what this avoids: 16 prompts, 313 token
  // blocks of 48 rows, take 29.4 us in two ranges, just over one round, and 25.2 us in three.)
  int span = rows;
  int64_t best = INT64_MAX;
  const int64_t round = (int64_t)(FOUR ? kResident4 : kResident) * num_sms();
  for (int r = 1; r <= std::min(rows, 64); ++r) {
    const int s_r = (rows + r - 1) / r, used = (rows + s_r - 1) / s_r;
    const int64_t blocks = (int64_t)tblocks * used, rounds = (blocks + round - 1) / round;
    int64_t cost = rounds * (kSetup + s_r);
    if (FOUR) {
      // ranges of rows to quantise go first; behind them the SMs run empty for about one of the others
      const int more = kRow4 - 1, least = kSetup4 + s_r + more * std::max(0, s_r - p.Nq);
      const int most = kSetup4 + s_r + more * std::min(s_r, 2 * p.Nkv);
      cost = blocks <= round || used == 1 ? rounds * most
             : std::max<int64_t>(most, tblocks * ((int64_t)used * kSetup4 + p.Nq + 2 * kRow4 * p.Nkv) / round + least);
    }
    if (cost < best) {
      best = cost;
      span = s_r;
    }
    if (blocks >= 16 * round) break;              // more rounds than that differ little
  }
  const Div by_len = Div::of(std::max(1, p.total / p.num_seqs)), by_page = Div::of(std::max(1, p.c.page_size));
  const dim3 grid(tblocks, (rows + span - 1) / span);
  const PagedCache4 p4 = FOUR ? *p.c4 : PagedCache4{};
  if constexpr (!FOUR) {
    if (!cache)
      return launch_early(norm_rope_kernel<Tin, Tq, Tkv, D, false>, grid, dim3(kThreads), 0, s, p, p4, span, by_len, by_page);
  }
  return launch_early(norm_rope_kernel<Tin, Tq, Tkv, D, true>, grid, dim3(kThreads), 0, s, p, p4, span, by_len, by_page);
}

template <typename Tin, typename Tq, typename Tkv>
cudaError_t launch_t(const NormRopeArgs& p, cudaStream_t s) {
  return p.D == 64 ? launch_d<Tin, Tq, Tkv, 64>(p, s)
                   : p.D == 128 ? launch_d<Tin, Tq, Tkv, 128>(p, s) : launch_d<Tin, Tq, Tkv, 256>(p, s);
}

template <typename Tin>
cudaError_t launch_in(const NormRopeArgs& p, cudaStream_t s) {
  if (p.c4 != nullptr) return p.q_bf16 ? launch_t<Tin, bf16, Kv4>(p, s) : launch_t<Tin, float, Kv4>(p, s);
  if (p.q_bf16) return p.kv_bf16 ? launch_t<Tin, bf16, bf16>(p, s) : launch_t<Tin, bf16, float>(p, s);
  return p.kv_bf16 ? launch_t<Tin, float, bf16>(p, s) : launch_t<Tin, float, float>(p, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& p, cudaStream_t s) {
  return p.in_bf16 ? launch_in<bf16>(p, s) : launch_in<float>(p, s);
}

}  // namespace gdn
