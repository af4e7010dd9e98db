// Attention of the new tokens of each sequence over its paged cache ([QDA], the
// full-attention layers and section "Cache"):
//   o[t, h] = sum_j softmax_j(scale q[t, h] . k_j) v_j, then * sigmoid(gate[t, h]).
//
// Bound: every visible key and value is read once per call and used by the G = Nq / Nkv
// query heads of its head, 2 G flops per byte in bf16 (G / 2 per byte pair in float32): far
// below the matrix ridge, so the kernel is a stream of the cache at HBM rate with the
// softmax riding along (one pass, running maximum and sum).
//
// Rows.  The 8 columns of a product tile (an octet) are query heads of one token and one
// kv head; all its columns see the same cache indices.  A unit is (sequence, kv head, NT
// consecutive octets); its cache indices split into tiles of 16 KB of K and 16 KB of V.
//
// Work split.  All tiles of all units, laid end to end, are cut into one equal range per
// CTA (one CTA per SM), from kv_lens as they stand on the device: ragged batches and a
// single long context keep every SM equally busy, and neither the host nor a captured
// graph needs the lengths.  A unit inside one range is finished by its CTA; the pieces of
// a unit that crosses ranges (at most one cut per CTA) go to the workspace, unnormalised
// with their maxima and sums, and a second small kernel joins them in order.  With short
// tables (no unit can exceed kAlignTiles tiles) ranges end at unit borders instead and no
// second kernel runs.
//
// Inside a CTA a producer warp walks the range: it looks the page ids up and issues TMA
// boxes of gcd(page size, tile) slots (so any page size tiles exactly; slots past the end
// of a sequence come as the out-of-range zero fill) into a ring of stages, and the query
// rows of each unit by bulk copies.  Consumer warps each take 16-token (bf16) or 4-token
// (float32) slices with a maximum, sum and output of their own, joined through shared
// memory once per unit.

#include <numeric>

#include "common.cuh"
#include "launch.h"
#include "tc_util.cuh"
#include "tmap.cuh"

namespace gdn {
namespace {

constexpr int kStageHalf = 16384;                  // bytes of K (and of V) in a stage
constexpr int kAlignTiles = 8;                     // no unit longer than this: ranges end at unit borders
constexpr int kMinTiles = 2;                       // tiles of a range at least (fewer CTAs for little work)
constexpr int kMaxCtas = 256;                      // CTAs, and so pieces of a unit, at most
constexpr uint64_t kWaitNs = 2000000000ull;        // bound of every wait
constexpr uint32_t kPollCap = 1u << 28;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ shapes
template <typename T, int D, int NT_>
struct Cfg {
  static constexpr bool BF = sizeof(T) == 2;
  static constexpr int NT = NT_;                                   // octets per pass
  static constexpr int ROWS = NT * 8;
  static constexpr int CW = 8;                                     // consumer warps
  static constexpr int DS = BF && D == 256 ? 2 : 1;                // warps that share a slice, each with D / DS of its output
  static constexpr int TG = CW / DS;                               // slices in work at a time
  static constexpr int THREADS = (CW + 1) * 32;
  static constexpr int TILE = kStageHalf / (D * (int)sizeof(T));   // tokens per stage
  static constexpr int SLICE = BF ? 16 : 4;                        // tokens per warp step
  static constexpr int SL = TILE / SLICE;                          // slices per stage
  static constexpr int USERS = SL < TG ? SL : TG;                  // slices of a stage in work at a time
  static constexpr int QPITCH = D * (int)sizeof(T) + 16;           // bytes; padded: ldmatrix without conflicts
  static constexpr int QBYTES = ROWS * QPITCH;
  static constexpr int JP = D + 4;                                 // join row pitch (floats)
  static constexpr int JOIN = TG * 8 * JP * 4 + TG * 8 * 2 * 4;
  static constexpr int HEAD = 1024;
  static constexpr int FIXED = HEAD + 2 * QBYTES + JOIN;
  static constexpr int MOST = 227 * 1024 - 1024;                   // 1024: alignment of the ring
  // Where a stage has fewer slices than there are warps, GROUPS sets of warps take the stages
  // in turn; the ring is a multiple of them, so that a stage always has the same readers (a
  // warp two rounds ahead of another's would take a phase that is still to come for done).
  static constexpr int GROUPS = TG / USERS;
  static constexpr int FIT = (MOST - FIXED) / (2 * kStageHalf) < 6 ? (MOST - FIXED) / (2 * kStageHalf) : 6;
  static constexpr int STAGES = FIT - FIT % GROUPS;
  static constexpr int SMEM = FIXED + STAGES * 2 * kStageHalf + 1024;
  static_assert(STAGES >= 3 && TG % USERS == 0 && STAGES % GROUPS == 0, "ring");
};

// One piece of a unit, from the producer to the consumers (and, unjoined, to the join kernel).
struct Piece {
  int tile0, tile1;        // tiles [tile0, tile1); tile0 < 0: no more pieces
  int slot;                // -1: the whole unit (write the output); else workspace slot of the piece
  int len, n, bos;         // cached length, new tokens, first token of the sequence
  int x0, nvalid, kvh;     // first octet, octets present, kv head
};
// A unit that starts in a CTA's range and ends behind it; CTA c's is record c.
struct SplitRec {
  int valid, bos, x0, nvalid, kvh, geff;
  int64_t end, total;      // the unit's end in the laid-out tiles; all tiles
};
static_assert(sizeof(SplitRec) == 40, "");

__host__ __device__ constexpr size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

struct Params {
  PagedAttnArgs a;
  int G, NG;               // query heads per kv head, octets per token
  int box, align;          // slots per TMA box; ranges end at unit borders
  float c;                 // scale * log2(e)
  SplitRec* rec;           // [grid]
  float* part_o;           // [2 * grid][ROWS][D]
  float* part_ml;          // [2 * grid][ROWS][2]
};

// ------------------------------------------------------------------ small helpers
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Bounded wait of a whole warp on a phase; gives up when another warp aborted or the time
// ran out, all lanes alike.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = tc::mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = now_ns();
    for (uint32_t i = 0; i < kPollCap && !ok; ++i) {
      ok = tc::mbar_try_wait(bar, parity);
      if (*abort != 0 || now_ns() - t0 > kWaitNs) break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// One box of the 4-D map {D, slot, kv head, page}.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A sequence as the call sees it: new tokens [bos, bos + n), cached length (0: nothing to
// attend, its rows are zero).  Metadata out of range reads as length 0.
struct Seq { int bos, n, len; };
__device__ __forceinline__ Seq load_seq(const PagedAttnArgs& a, int s, int* err = nullptr) {
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
__device__ __forceinline__ int seq_tiles(const Seq& q) { return (q.len + C::TILE - 1) / C::TILE; }
template <typename C>
__device__ __forceinline__ int seq_groups(const Params& p, const Seq& q) {   // octet groups per kv head
  return (int)(((int64_t)q.n * p.NG + C::NT - 1) / C::NT);
}

// y = o * sigmoid(gate), four elements of (token t, head h) from d.
template <typename T>
__device__ __forceinline__ void finish4(const PagedAttnArgs& a, int t, int h, int d, int D, float (&y)[4]) {
  if (a.gate.p != nullptr) {
    float g[4];
    load4(static_cast<const T*>(a.gate.p) + t * a.gate.ts + h * a.gate.hs + d, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= sigmoidf_(g[i]);
  }
  const int64_t at = ((int64_t)t * a.Nq + h) * D + d;
  if (a.out_bf16) store4(static_cast<bf16*>(a.o) + at, y);
  else store4(static_cast<float*>(a.o) + at, y);
}

// ------------------------------------------------------------------ consumers
// Per warp: running maxima m (of scale log2(e) q.k), sums l and outputs o of the slices it took.

// bf16 on the matrix instructions, transposed: S^T [16 tokens x 8 heads] = K Q^T, then
// O^T [D x 8 heads] += V^T P^T.  With at most 8 heads on the narrow side no row of a
// product is padding, half the instructions and accumulators of the other orientation; the
// score tile turns into the second product's operand by an 8x8 transpose in registers.
// The weights enter it as the sum of two bf16 values (2^-16 relative; one value would
// add an error as large as the output's own rounding), the sum l takes them in float32.
template <int D, int NT>
struct TcWarp {
  using C = Cfg<bf16, D, NT>;
  static constexpr int KS = D / 16;
  static constexpr int OS = KS / C::DS;            // 16-row blocks of O^T that this warp holds
  static constexpr bool QREG = NT * D <= 256;      // query fragments stay in registers
  static constexpr int CH = NT <= 2 ? 2 : 1;       // score accumulators: shorter chains of dependent products
  float o[NT][OS][4];
  float m[NT][2], l[NT][2];
  uint32_t qf[QREG ? NT : 1][QREG ? KS : 1][2];
  uint32_t qaddr;
  int d0;                                          // first of this warp's blocks

  __device__ __forceinline__ void start(const uint8_t* q, int share, int lane) {
    d0 = share * OS;
    // x4: two k steps of one octet; lanes 8i..8i+7 give the rows of matrix i
    qaddr = tc::smem_u32(q) + (lane & 7) * C::QPITCH + (lane >> 3) * 16;
    if (QREG) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          uint32_t r[4];
          ldsm4(qaddr + nt * 8 * C::QPITCH + ks * 32, r);
          qf[nt][ks][0] = r[0]; qf[nt][ks][1] = r[1];
          qf[nt][ks + 1][0] = r[2]; qf[nt][ks + 1][1] = r[3];
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < OS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }
  }

  // Slice of the 16 tokens from tok0, rows j0.. of the stage; lim(nt): tokens octet nt sees.
  template <typename Lim>
  __device__ __forceinline__ void slice(uint8_t* ks_, uint8_t* vs_, int j0, int tok0, int nvalid, float c, Lim lim,
                                        int lane) {
    float s[NT][4], s1[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = s1[nt][e] = 0.f;
    {
      const int row = j0 + (lane & 15);
      const uint32_t base = tc::smem_u32(ks_) + row * 128;
      const uint32_t sw = (uint32_t)(row & 7);
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
        uint32_t a0[4], a1[4];
        const uint32_t blk = base + (ks >> 2) * (C::TILE * 128);
        ldsm4(blk + (((uint32_t)((ks & 3) * 2 + (lane >> 4)) ^ sw) << 4), a0);
        ldsm4(blk + (((uint32_t)((ks & 3) * 2 + 2 + (lane >> 4)) ^ sw) << 4), a1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (QREG) {
            mma16816(s[nt], a0, qf[nt][ks][0], qf[nt][ks][1]);
            mma16816(CH == 2 ? s1[nt] : s[nt], a1, qf[nt][ks + 1][0], qf[nt][ks + 1][1]);
          } else {
            uint32_t r[4];
            ldsm4(qaddr + nt * 8 * C::QPITCH + ks * 32, r);
            mma16816(s[nt], a0, r[0], r[1]);
            mma16816(CH == 2 ? s1[nt] : s[nt], a1, r[2], r[3]);
          }
        }
      }
    }
    const bool tail = tok0 + 16 > lim(0);          // octets come in order of their token: lim(0) is the least
    const int g = lane >> 2;
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = (CH == 2 ? s[nt][e] + s1[nt][e] : s[nt][e]) * c;
      if (tail) {
        const int last = lim(nt) - tok0;
        if (g >= last) s[nt][0] = s[nt][1] = -INFINITY;
        if (g + 8 >= last) s[nt][2] = s[nt][3] = -INFINITY;
      }
      float mx[2] = {fmaxf(s[nt][0], s[nt][2]), fmaxf(s[nt][1], s[nt][3])};
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
      }
      const bool up = mx[0] > m[nt][0] || mx[1] > m[nt][1];
      if (__any_sync(0xffffffffu, up)) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[nt][e], mx[e]);
          al[e] = mn == m[nt][e] ? 1.f : exp2f(m[nt][e] - mn);     // (-inf stays -inf: no change)
          m[nt][e] = mn;
          l[nt][e] *= al[e];
        }
#pragma unroll
        for (int i = 0; i < OS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] *= al[e & 1];
      }
      const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
      const float p0 = exp2f(s[nt][0] - b0), p1 = exp2f(s[nt][1] - b1);
      const float p2 = exp2f(s[nt][2] - b0), p3 = exp2f(s[nt][3] - b1);
      l[nt][0] += p0 + p2;
      l[nt][1] += p1 + p3;
      const uint32_t h0 = pack_bf16(p0, p1), h1 = pack_bf16(p2, p3);
      const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h0));
      const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h1));
      hi[nt][0] = movm(h0);
      hi[nt][1] = movm(h1);
      lo[nt][0] = movm(pack_bf16(p0 - f0.x, p1 - f0.y));
      lo[nt][1] = movm(pack_bf16(p2 - f1.x, p3 - f1.y));
    }
    const int vrow = j0 + (lane & 7) + ((lane >> 4) << 3);
    const uint32_t vbase = tc::smem_u32(vs_) + vrow * 128;
    const uint32_t vsw = (uint32_t)(vrow & 7);
    auto vfrag = [&](int b, uint32_t (&a)[4]) {
      const int i = d0 + b;
      const uint32_t ch = (uint32_t)((i & 3) * 2 + ((lane >> 3) & 1));
      ldsm4t(vbase + (i >> 2) * (C::TILE * 128) + ((ch ^ vsw) << 4), a);
    };
    if (!tail) {
#pragma unroll
      for (int i = 0; i < OS; ++i) {
        uint32_t a[4];
        vfrag(i, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(o[nt][i], a, hi[nt][0], hi[nt][1]);
          mma16816(o[nt][i], a, lo[nt][0], lo[nt][1]);
        }
      }
    } else {
      // The end of the visible range: rows that an octet does not see may hold anything, and
      // 0 * NaN is NaN.  They are cleared in the stage, from the octet that sees most to the
      // one that sees least; a warp clears the columns that it reads.
#pragma unroll
      for (int nt = NT - 1; nt >= 0; --nt) {
        if (nt >= nvalid) continue;
        const int last = max(0, min(16, lim(nt) - tok0));
        for (int e = lane; e < (16 - last) * (2 * OS); e += 32) {
          const int r = j0 + last + e / (2 * OS), ch = 2 * d0 + e % (2 * OS);
          *reinterpret_cast<uint4*>(vs_ + (ch >> 3) * (C::TILE * 128) + r * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < OS; ++i) {
          uint32_t a[4];
          vfrag(i, a);
          mma16816(o[nt][i], a, hi[nt][0], hi[nt][1]);
          mma16816(o[nt][i], a, lo[nt][0], lo[nt][1]);
        }
        __syncwarp();
      }
      tc::fence_proxy_async_smem();                // before the ring's next copy into these rows
    }
  }

  // This warp's share of octet nt into the join buffers.
  __device__ __forceinline__ void give(int nt, float* jo, float* jm, float* jl, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l[nt][e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (g == 0 && d0 == 0) {
        jm[2 * t + e] = m[nt][e];
        jl[2 * t + e] = v;
      }
    }
#pragma unroll
    for (int i = 0; i < OS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) jo[(2 * t + (e & 1)) * C::JP + (d0 + i) * 16 + g + (e >> 1) * 8] = o[nt][i][e];
  }
};

// float32 on the CUDA cores: the lanes of a warp span a head row, four tokens at a time.
// The 8 x 4 partial dot products are summed over the lanes by folding halves onto each
// other (9 exchanges per token), which leaves lane 4 h + i with the score of head h and
// token i: one exponential per lane.
template <int D>
struct SimtWarp {
  using C = Cfg<float, D, 1>;
  static constexpr int E = D / 32;                 // elements per lane
  static constexpr int V = E < 4 ? E : 4;          // per load
  float q[8][E], o[8][E];
  float m, l;                                      // of head lane / 4

  // element i of a lane sits at column (i / V) * 32 V + lane V + i % V
  static __device__ __forceinline__ void row(const uint8_t* base, int r, int lane, float (&x)[E]) {
    const float* p = reinterpret_cast<const float*>(base) + r * D + lane * V;
    if (V == 4) {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(p + i * 32);
        x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;
      }
    } else {
      const float2 f = *reinterpret_cast<const float2*>(p);
      x[0] = f.x; x[1] = f.y;
    }
  }
  __device__ __forceinline__ void start(const uint8_t* qs, int, int lane) {
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      row(qs + h * C::QPITCH, 0, lane, q[h]);
#pragma unroll
      for (int i = 0; i < E; ++i) o[h][i] = 0.f;
    }
    m = -INFINITY;
    l = 0.f;
  }
  template <typename Lim>
  __device__ __forceinline__ void slice(uint8_t* ks_, uint8_t* vs_, int j0, int tok0, int, float c, Lim lim, int lane) {
    const int last = lim(0) - tok0;                // tokens of the slice that are visible (> 0)
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float k[E], d[8];
      row(ks_, j0 + i, lane, k);
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        d[h] = q[h][0] * k[0];
#pragma unroll
        for (int e = 1; e < E; ++e) d[h] = fmaf(q[h][e], k[e], d[h]);
      }
#pragma unroll
      for (int w = 4, off = 16; w >= 1; w >>= 1, off >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int h = 0; h < w; ++h) {
          const float keep = up ? d[h + w] : d[h], send = up ? d[h] : d[h + w];
          d[h] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
      }
      d[0] += __shfl_xor_sync(0xffffffffu, d[0], 2);
      d[0] += __shfl_xor_sync(0xffffffffu, d[0], 1);
      if ((lane & 3) == i) s = d[0];
    }
    s = (lane & 3) < last ? s * c : -INFINITY;
    float mx = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx > m)) {
      const float mn = fmaxf(m, mx);
      const float al = mn == m ? 1.f : exp2f(m - mn);
      m = mn;
      l *= al;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const float a = __shfl_sync(0xffffffffu, al, 4 * h);
#pragma unroll
        for (int e = 0; e < E; ++e) o[h][e] *= a;
      }
    }
    const float p = exp2f(s - (m == -INFINITY ? 0.f : m));
    l += p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < last) {                              // rows behind may hold anything: not read into o
        float v[E];
        row(vs_, j0 + i, lane, v);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float w = __shfl_sync(0xffffffffu, p, 4 * h + i);
#pragma unroll
          for (int e = 0; e < E; ++e) o[h][e] = fmaf(w, v[e], o[h][e]);
        }
      }
    }
  }
  __device__ __forceinline__ void give(int, float* jo, float* jm, float* jl, int lane) {
    float v = l;
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    if ((lane & 3) == 0) {
      jm[lane >> 2] = m;
      jl[lane >> 2] = v;
    }
#pragma unroll
    for (int h = 0; h < 8; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) jo[h * C::JP + (e / V) * 32 * V + lane * V + e % V] = o[h][e];
  }
};
template <typename T, int D, int NT> struct WarpOf { using type = TcWarp<D, NT>; };
template <int D, int NT> struct WarpOf<float, D, NT> { using type = SimtWarp<D>; };

// ------------------------------------------------------------------ the main kernel
template <typename T, int D, int NT>
__global__ void __launch_bounds__(Cfg<T, D, NT>::THREADS, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ Params p) {
  using C = Cfg<T, D, NT>;
  constexpr int COLS = 128 / (int)sizeof(T);       // columns of a box (128 bytes, swizzled) in bf16
  constexpr int CB = C::BF ? D / COLS : 1;         // boxes across a row; float32: whole rows, not swizzled
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* ring = tc::smem_aligned<1024>(raw);
  uint8_t* qs = ring + C::STAGES * 2 * kStageHalf;
  float* jo = reinterpret_cast<float*>(qs + 2 * C::QBYTES);
  float* jm = jo + C::TG * 8 * C::JP;
  float* jl = jm + C::TG * 8;
  uint8_t* head = reinterpret_cast<uint8_t*>(jl + C::TG * 8);
  uint64_t* full = reinterpret_cast<uint64_t*>(head);
  uint64_t* empty = full + C::STAGES;
  uint64_t* qfull = empty + C::STAGES;
  uint64_t* qempty = qfull + 2;
  Piece* piece = reinterpret_cast<Piece*>(head + 256);             // [2]
  int64_t* scan = reinterpret_cast<int64_t*>(head + 512);          // [CW + 1] warp sums, then the start
  volatile int* abort = reinterpret_cast<int*>(head + 768);
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, C::USERS * C::DS);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(qfull + i, 1);
      tc::mbar_init(qempty + i, C::CW);
    }
    *abort = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&mk);
    tc::prefetch_tmap(&mv);
  }
  // all tiles, and the sequence that this CTA's range starts in
  const int per = (a.num_seqs + C::THREADS - 1) / C::THREADS;
  const int s_lo = min(a.num_seqs, tid * per), s_hi = min(a.num_seqs, s_lo + per);
  int64_t sum = 0;
  for (int s = s_lo; s < s_hi; ++s) {
    const Seq q = load_seq(a, s);
    sum += (int64_t)seq_tiles<C>(q) * seq_groups<C>(p, q) * a.Nkv;
  }
  int64_t inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
  for (int w = 0; w <= C::CW; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int64_t geff = max((int64_t)1, min((int64_t)gridDim.x, total / kMinTiles));
  const bool mine = (int64_t)blockIdx.x < geff;
  const int64_t lo = mine ? total * blockIdx.x / geff : total;
  const int64_t hi = mine ? total * (blockIdx.x + 1) / geff : total;
  __syncthreads();
  if (before <= lo && lo < before + sum) {
    int64_t at = before;
    for (int s = s_lo; s < s_hi; ++s) {
      const Seq q = load_seq(a, s);
      const int64_t w = (int64_t)seq_tiles<C>(q) * seq_groups<C>(p, q) * a.Nkv;
      if (lo < at + w) {
        scan[0] = s;
        scan[1] = at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();

  if (warp == C::CW) {
    // ------------------------------------------------------------ producer
    int s = lo < hi ? (int)scan[0] : a.num_seqs;
    int64_t seq_at = lo < hi ? scan[1] : 0, pos = lo;
    SplitRec rec{};
    int it = 0, npiece = 0;
    bool ok = true;
    Seq q{0, 0, 0};
    int tiles = 0, groups = 0;
    if (s < a.num_seqs) {
      q = load_seq(a, s);
      tiles = seq_tiles<C>(q);
      groups = seq_groups<C>(p, q);
      if (p.align) pos = seq_at + (pos - seq_at + tiles - 1) / tiles * tiles;   // the first unit that starts here
    }
    while (ok && pos < hi) {
      if (pos >= seq_at + (int64_t)tiles * groups * a.Nkv) {
        // the next sequence with work: the warp looks at 32 of them at a time
        seq_at += (int64_t)tiles * groups * a.Nkv;
        int base = s + 1;
        for (;;) {
          Seq c{0, 0, 0};
          if (base + lane < a.num_seqs) c = load_seq(a, base + lane);
          const uint32_t has = __ballot_sync(0xffffffffu, c.len > 0);
          if (has != 0) {
            const int w = __ffs(has) - 1;
            s = base + w;
            q.bos = __shfl_sync(0xffffffffu, c.bos, w);
            q.n = __shfl_sync(0xffffffffu, c.n, w);
            q.len = __shfl_sync(0xffffffffu, c.len, w);
            break;
          }
          base += 32;
          if (base >= a.num_seqs) break;           // (cannot be: pos < hi <= total)
        }
        if (base >= a.num_seqs) break;
        tiles = seq_tiles<C>(q);
        groups = seq_groups<C>(p, q);
        continue;
      }
      const int unit = (int)((pos - seq_at) / tiles);
      const int t0 = (int)((pos - seq_at) % tiles);
      const int t1 = p.align ? tiles : (int)min((int64_t)tiles, t0 + (hi - pos));
      const int kvh = unit / groups, x0 = (unit % groups) * NT;
      const int nvalid = min(NT, q.n * p.NG - x0);
      const int qslot = npiece & 1;
      ok = wait_bar(qempty + qslot, ((npiece >> 1) & 1) ^ 1, abort);
      if (!ok) break;
      if (lane == 0) {
        Piece d;
        d.tile0 = t0; d.tile1 = t1;
        d.slot = t0 == 0 && t1 == tiles ? -1 : 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
        d.len = q.len; d.n = q.n; d.bos = q.bos; d.x0 = x0; d.nvalid = nvalid; d.kvh = kvh;
        piece[qslot] = d;
        if (t0 == 0 && t1 < tiles)
          rec = {1, q.bos, x0, nvalid, kvh, (int)geff, pos + tiles, total};
      }
      // query rows: octet x of the sequence is token x / NG, heads (x % NG) * 8 .. of the kv head's G
      int rows = 0;
      for (int x = x0; x < x0 + nvalid; ++x) rows += min(8, p.G - (x % p.NG) * 8);
      if (lane == 0) tc::mbar_arrive_expect_tx(qfull + qslot, (uint32_t)(rows * D * sizeof(T)));
      __syncwarp();
      for (int r = lane; r < nvalid * 8; r += 32) {
        const int x = x0 + r / 8, oct = x % p.NG, h = oct * 8 + r % 8;
        if (h < p.G)
          tc::bulk_load(qs + qslot * C::QBYTES + r * C::QPITCH,
                        static_cast<const T*>(a.q.p) + (q.bos + x / p.NG) * a.q.ts + (kvh * p.G + h) * a.q.hs,
                        D * sizeof(T), qfull + qslot);
      }
      ++npiece;
      const int32_t* bt = a.c.bt + (int64_t)s * a.c.max_pages;
      const int nbox = C::TILE / p.box;
      // page and slot of this lane's first box, one tile ahead of its use
      auto lookup = [&](int tile, int b, int& page, int& off) {
        const int tok = tile * C::TILE + b * p.box;
        page = a.c.num_pages;                      // out of range: zero fill
        off = 0;
        if (tok < q.len && b < nbox) {
          const int pg = __ldg(bt + tok / a.c.page_size);
          off = tok % a.c.page_size;
          if (pg >= 0 && pg < a.c.num_pages) page = pg;
          else raise_error(a.err, kDevErrCache);
        }
      };
      int page, off;
      lookup(t0, lane, page, off);
      for (int tile = t0; tile < t1; ++tile, ++it) {
        int npage = 0, noff = 0;
        if (tile + 1 < t1) lookup(tile + 1, lane, npage, noff);
        const int st = it % C::STAGES;
        ok = wait_bar(empty + st, ((it / C::STAGES) & 1) ^ 1, abort);
        if (!ok) break;
        uint8_t* kd = ring + st * 2 * kStageHalf;
        if (lane == 0) tc::mbar_arrive_expect_tx(full + st, 2 * kStageHalf);
        __syncwarp();
        for (int b = lane; b < nbox; b += 32) {
          if (b >= 32) lookup(tile, b, page, off);
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            const int dst = cb * (C::TILE * 128) + b * p.box * (kStageHalf / C::TILE / CB);
            tma_load_4d(kd + dst, &mk, full + st, cb * COLS, off, kvh, page);
            tma_load_4d(kd + kStageHalf + dst, &mv, full + st, cb * COLS, off, kvh, page);
          }
        }
        page = npage;
        off = noff;
      }
      pos += t1 - t0;
    }
    if (ok) {
      const int qslot = npiece & 1;
      ok = wait_bar(qempty + qslot, ((npiece >> 1) & 1) ^ 1, abort);
      if (ok && lane == 0) {
        piece[qslot].tile0 = -1;
        tc::mbar_arrive(qfull + qslot);
      }
    }
    if (lane == 0 && !p.align) p.rec[blockIdx.x] = rec;
    if (!ok) {
      if (lane == 0) {
        *abort = 1;
        raise_error(a.err, kDevErrTimeout);
      }
      // copies in flight land before the CTA's shared memory goes
      const int zero = 0;
      for (int i = max(0, it - C::STAGES); i < it; ++i)
        wait_bar(full + i % C::STAGES, (i / C::STAGES) & 1, const_cast<volatile int*>(&zero));
      for (int i = max(0, npiece - 2); i < npiece; ++i)
        wait_bar(qfull + (i & 1), (i >> 1) & 1, const_cast<volatile int*>(&zero));
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // sequences with nothing to attend: their rows are zero; every sequence's metadata is checked once
  for (int s = blockIdx.x * C::CW + warp; s < a.num_seqs; s += gridDim.x * C::CW) {
    const Seq q = load_seq(a, s, lane == 0 ? a.err : nullptr);
    if (q.n > 0 && q.len == 0) {
      const int64_t b = (int64_t)q.bos * a.Nq * D, e = b + (int64_t)q.n * a.Nq * D;
      const float z[4] = {0.f, 0.f, 0.f, 0.f};
      for (int64_t i = b + lane * 4; i < e; i += 128) {
        if (a.out_bf16) store4(static_cast<bf16*>(a.o) + i, z);
        else store4(static_cast<float*>(a.o) + i, z);
      }
    }
  }
  const int tw = warp % C::TG;                     // which slices; warps tw + k TG share them
  typename WarpOf<T, D, NT>::type w;
  int it = 0;
  for (int np = 0;; ++np) {
    const int qslot = np & 1;
    bool ok = wait_bar(qfull + qslot, (np >> 1) & 1, abort);
    Piece d{};
    if (ok) {
      d = piece[qslot];
      if (d.tile0 < 0) break;
      w.start(qs + qslot * C::QBYTES, warp / C::TG, lane);
      auto lim = [&](int nt) { return d.len - d.n + (d.x0 + min(nt, d.nvalid - 1)) / p.NG + 1; };
      const int most = lim(NT - 1);
      for (int tile = d.tile0; tile < d.tile1; ++tile, ++it) {
        int j = C::SL >= C::TG ? tw : tw - (it * C::SL) % C::TG;           // this warp's first slice of the stage
        if (j < 0 || j >= C::SL) continue;
        const int st = it % C::STAGES;
        if (!wait_bar(full + st, (it / C::STAGES) & 1, abort)) {
          ok = false;
          break;
        }
        uint8_t* kd = ring + st * 2 * kStageHalf;
        for (; j < C::SL; j += C::TG) {
          const int tok0 = tile * C::TILE + j * C::SLICE;
          if (tok0 < most) w.slice(kd, kd + kStageHalf, j * C::SLICE, tok0, d.nvalid, p.c, lim, lane);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty + st);
      }
    }
    if (!ok && lane == 0) {
      *abort = 1;
      raise_error(a.err, kDevErrTimeout);
    }
    // the warps' shares joined, octet by octet
    bool quit = false;
    for (int nt = 0; nt < NT; ++nt) {
      if (nt > 0 && nt >= d.nvalid) break;
      if (ok) {
#pragma unroll
        for (int k = 0; k < NT; ++k)
          if (k == nt) w.give(k, jo + tw * 8 * C::JP, jm + tw * 8, jl + tw * 8, lane);
      }
      if (tc::named_sync_or(1, C::CW * 32, !ok)) {
        quit = true;
        break;
      }
      const int x = d.x0 + nt, oct = x % p.NG;
      for (int i = tid; i < 8 * (D / 4); i += C::CW * 32) {
        const int h = i / (D / 4), e = (i % (D / 4)) * 4;
        if (oct * 8 + h >= p.G) break;
        float mt = -INFINITY, lt = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < C::TG; ++k) mt = fmaxf(mt, jm[k * 8 + h]);
        const float base = mt == -INFINITY ? 0.f : mt;
#pragma unroll
        for (int k = 0; k < C::TG; ++k) {
          const float f = exp2f(jm[k * 8 + h] - base);
          const float4 v = *reinterpret_cast<const float4*>(jo + (k * 8 + h) * C::JP + e);
          lt = fmaf(jl[k * 8 + h], f, lt);
          y[0] = fmaf(v.x, f, y[0]); y[1] = fmaf(v.y, f, y[1]);
          y[2] = fmaf(v.z, f, y[2]); y[3] = fmaf(v.w, f, y[3]);
        }
        if (d.slot < 0) {
          const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] *= inv;
          finish4<T>(a, d.bos + x / p.NG, d.kvh * p.G + oct * 8 + h, e, D, y);
        } else {
          const int64_t r = (int64_t)d.slot * C::ROWS + nt * 8 + h;
          store4(p.part_o + r * D + e, y);
          if (e == 0) *reinterpret_cast<float2*>(p.part_ml + r * 2) = make_float2(mt, lt);
        }
      }
      tc::named_sync(1, C::CW * 32);
    }
    if (quit) break;
    if (lane == 0) tc::mbar_arrive(qempty + qslot);
  }
}

// ------------------------------------------------------------------ the join
// Block (c, row) joins one row of the unit that starts in CTA c's range and ends behind it,
// its pieces in order.  All loads of a block but the record are independent: first the
// maxima and sums (a thread per piece) for the weights, beside them the outputs, NP pieces
// at a time.  Launched while the main kernel runs; the first step is to wait for its end.
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
paged_attn_join_kernel(const __grid_constant__ Params p) {
  constexpr int LPR = D / 4;                       // threads across a row
  constexpr int NP = kJoinThreads / LPR;           // pieces in flight
  __shared__ float sw[kMaxCtas], so[NP][D], red[2][kJoinThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const SplitRec r = p.rec[blockIdx.x];
  const int row = blockIdx.y, x = r.x0 + row / 8, h = (x % p.NG) * 8 + row % 8;
  if (!r.valid || row >= r.nvalid * 8 || h >= p.G) return;
  // CTA c0's last piece, then the first one of every CTA whose range starts before the unit's end
  const int c0 = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)((r.end * r.geff + r.total - 1) / r.total) - c0;
  auto at = [&](int i) { return ((int64_t)2 * (c0 + i) + (i == 0 ? 1 : 0)) * (gridDim.y) + row; };
  float2 ml = make_float2(-INFINITY, 0.f);
  if (tid < n) ml = *reinterpret_cast<const float2*>(p.part_ml + at(tid) * 2);
  float m = ml.x;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) m = fmaxf(m, red[0][i]);
  const float w = exp2f(ml.x - (m == -INFINITY ? 0.f : m));
  float l = w * ml.y;
  if (tid < n) sw[tid] = w;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) l += red[1][i];
  const int k = tid / LPR, e = (tid % LPR) * 4;
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = k; i < n; i += NP) {
    float v[4];
    load4(p.part_o + at(i) * D + e, v);
    const float f = sw[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmaf(v[j], f, y[j]);
  }
  store4(&so[k][e], y);
  __syncthreads();
  if (k != 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 1; i < NP; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += so[i][e + j];
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] *= inv;
  finish4<T>(p.a, r.bos + x / p.NG, r.kvh * p.G + h, e, D, y);
}

// ------------------------------------------------------------------ host
// Octets per pass: enough for the new tokens of an even batch (a unit's rows then read
// the cache once), up to the four whose outputs fit the registers.
int octets_per_pass(int num_seqs, int total, int Nq, int Nkv, int D, bool bf) {
  if (!bf) return 1;
  const int64_t want = (int64_t)((total + num_seqs - 1) / num_seqs) * ((Nq / Nkv + 7) / 8);
  int nt = 1;
  while (nt < want && nt < 4) nt *= 2;
  return nt;
}

// A 4-D map over the cache, {D, slot, head, page}, box {cols, box, 1, 1}.
bool cache_map(CUtensorMap* map, const void* base, const PagedAttnArgs& a, int cols, int box) {
  EncodeTiledFn enc = tmap_encoder();
  if (enc == nullptr) return false;
  const int es = a.in_bf16 ? 2 : 4;
  cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.c.page_size, (cuuint64_t)a.Nkv, (cuuint64_t)a.c.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)a.c.ss * es, (cuuint64_t)a.c.hs * es, (cuuint64_t)a.c.ps * es};
  cuuint32_t bx[4] = {(cuuint32_t)cols, (cuuint32_t)box, 1, 1};
  cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, a.in_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
             const_cast<void*>(base), dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             a.in_bf16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int NT>
cudaError_t launch_c(const PagedAttnArgs& a, cudaStream_t s) {
  using C = Cfg<T, D, NT>;
  const auto fn = paged_attn_kernel<T, D, NT>;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  const int grid = std::min(num_sms(), kMaxCtas);
  Params p{};
  p.a = a;
  p.G = a.Nq / a.Nkv;
  p.NG = (p.G + 7) / 8;
  p.box = std::gcd(a.c.page_size, C::TILE);
  p.align = ((int64_t)a.c.max_pages * a.c.page_size + C::TILE - 1) / C::TILE <= kAlignTiles;
  p.c = a.scale * kLog2e;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.rec = reinterpret_cast<SplitRec*>(ws);
  ws += align16(sizeof(SplitRec) * grid);
  p.part_ml = reinterpret_cast<float*>(ws);
  ws += align16((size_t)2 * grid * C::ROWS * 2 * 4);
  p.part_o = reinterpret_cast<float*>(ws);
  CUtensorMap mk, mv;
  const int cols = C::BF ? 64 : D;
  if (!cache_map(&mk, a.c.k, a, cols, p.box) || !cache_map(&mv, a.c.v, a, cols, p.box)) return cudaErrorInvalidValue;
  fn<<<grid, C::THREADS, C::SMEM, s>>>(mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.align) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, C::ROWS);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<T, D>, p);
}

template <int D>
cudaError_t launch_bf16(const PagedAttnArgs& a, int nt, cudaStream_t s) {
  if (nt == 1) return launch_c<bf16, D, 1>(a, s);
  if (nt == 2) return launch_c<bf16, D, 2>(a, s);
  return launch_c<bf16, D, 4>(a, s);
}

}  // namespace

size_t paged_attn_workspace_bytes(int num_seqs, int total, int Nq, int Nkv, int D) {
  // the same for every type and table: the caller may size it before those are known
  const int rows = octets_per_pass(num_seqs, total, Nq, Nkv, D, true) * 8;
  const size_t grid = std::min(num_sms(), kMaxCtas);
  return align16(sizeof(SplitRec) * grid) + align16(2 * grid * rows * 2 * 4) + 2 * grid * rows * D * 4;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
  const int nt = octets_per_pass(a.num_seqs, a.total, a.Nq, a.Nkv, a.D, a.in_bf16);
  if (a.in_bf16)
    return a.D == 64 ? launch_bf16<64>(a, nt, s) : a.D == 128 ? launch_bf16<128>(a, nt, s) : launch_bf16<256>(a, nt, s);
  return a.D == 64 ? launch_c<float, 64, 1>(a, s)
                   : a.D == 128 ? launch_c<float, 128, 1>(a, s) : launch_c<float, 256, 1>(a, s);
}

}  // namespace gdn
