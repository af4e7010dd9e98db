// Attention of the new tokens of each sequence over its paged cache ([QDA], the
// full-attention layers and section "Cache"):
//   o[t, h] = sum_j softmax_j(scale q[t, h] . k_j) v_j, then * sigmoid(gate[t, h]).
//
// Bound: a pass reads every key and value of a sequence and kv head once, for the G = Nq / Nkv
// query heads of that head, 2 G flops per byte in bf16 and G in float32 for each new token:
// in bf16 far below the matrix ridge, so the kernel is a stream of the cache at HBM rate with
// the softmax riding along (running maximum and sum).  float32 is that for one token; with
// more, the CUDA cores bound it.
//
// Rows.  The 8 columns of a product tile (an octet) are query heads of one token and one
// kv head; all its columns see the same cache indices.  A unit is one pass: (sequence, kv head,
// NT consecutive octets); its cache indices split into tiles of at most 8 KB of K and 8 KB of V.
// A sequence with more octets per kv head (more than four in bf16, fewer in float32) takes more
// passes, and each streams the whole sequence: also tiles behind the last index that the pass's
// tokens see, which the consumers skip.  With a few new tokens that is next to nothing; for a
// whole prompt it is half of the traffic.
//
// Work split.  All tiles of all units, laid end to end with a gap of kUnitCost for each
// unit's start and join, are cut into one equal range per CTA (two CTAs per SM, one's starts
// and joins under the other's stream), from kv_lens as they stand on the device: ragged
// batches and a single long context keep every SM equally busy, and neither the host nor a
// captured graph needs the lengths.  A unit inside one
// range is finished by its CTA; the pieces of a unit that crosses ranges (at most one cut
// per CTA) go to the workspace, unnormalised with their maxima and sums, and a second small
// kernel joins them in order.  With short tables (at most kAlignTiles full tiles of tokens; fewer
// than twice as many tiles where pages do not fill a tile) ranges end at unit borders instead
// and no second kernel runs.
//
// Where the time goes, from copies of the kernel that leave a step out (us; 16 sequences of 512 to
// 8192 with four tokens, 16 heads over 2 of 256 | one sequence of 131072, the same heads | float32,
// 32 sequences of 100 to 4000, 8 heads over 2 of 128): stream with its start and end 23.7 | 44.2 |
// 26.0 (at the copy rate 17.3 | 40.3 | 20.5), arithmetic 4.1 | 2.4 | 2.1 more, pieces to the workspace 2.1
// | 0.6 | 0, their join 6.5 | 4.4 | 2.8; together 36.5 | 51.7 | 30.7.
//
// Inside a CTA a producer warp walks the range: it looks the page ids up and issues TMA
// boxes that end where pages do (boxes past the end of a sequence come as the out-of-range
// zero fill) into a ring of stages, and the query rows of each unit by bulk copies.  Four
// consumer warps take 16-token (bf16) or 4-token (float32) slices with a maximum, sum and
// output of their own, joined through shared memory once per unit.  With many rows in bf16
// (NT * D > 256) DS of them share a slice: each computes the weights of NT / DS octets, they
// exchange them, and each accumulates D / DS columns of the output of all octets, so that a
// warp never holds more than 64 accumulators.
//
// Why not the tensor memory's products: with keys on the 128-row side the 8 to 32 rows of a pass
// would be their columns, and possible; but the matrix instructions used here are 12 to 33 % busy, so
// for these calls their rate is not what bounds.  Many rows (prompts) are another matter.

#include "attn_util.cuh"
#include "paged_attn.h"
#include "tc_util.cuh"
#include "tmap.cuh"

namespace gdn {
namespace {

constexpr int kStageHalf = 8192;                   // bytes of K (and of V) in a stage
// Tables of at most so many full tiles: ranges end at unit borders, no workspace.  Whole units against
// cut ones in bf16, us: 64 sequences of 8 tiles 12.6 and 14.5 (256-wide heads), 11.8 and 12.2
// (128-wide); of 16 tiles 19.2 and 17.5, 18.0 and 15.5; one sequence of 16 tiles 16.7 and 11.1; 64
// of 32 tiles 31 and 23.  The cut is the faster one from somewhat below 16 tiles on; the limit is
// also what tables need no workspace by, and stays.
constexpr int kAlignTiles = 16;
// Tiles of a range at least: fewer CTAs for little work, so fewer pieces to join.  1, 2, 4, 8 and 16: one
// sequence of 600 tokens, 2 kv heads of 256, 10.0, 10.1, 11.3, 14.3 and 19.8 us; 8 of 2000 of 128 11.5,
// 11.5, 11.5, 14.1 and 19.6.
constexpr int kMinTiles = 4;
// A unit's start and join, in tiles, where ranges are cut.  0, 2, 4 and 8: 700 sequences of 1 to 1500
// tokens 110, 101.7, 103.6 and 110 us; 16 x 4 tokens of 512 to 8192 38.4, 36.8, 36.5 and 36.6.
constexpr int kUnitCost = 4;
constexpr int kOcc = 2;                            // CTAs per SM
constexpr int kMaxCtas = 512;                      // CTAs, and so pieces of a unit, at most
constexpr uint32_t kPollCap = 1u << 28;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ shapes
template <typename T, int D, int NT_, int RG_ = 8>
struct Cfg {
  static constexpr bool BF = sizeof(T) == 2;
  static constexpr int NT = NT_;                                   // octets per pass
  static constexpr int RG = RG_;                                   // rows of an octet: 8, or 4 where four heads are all
  static constexpr int ROWS = NT * RG;
  static constexpr int CW = 4;                                     // consumer warps
  static constexpr int THREADS = (CW + 1) * 32;
  static constexpr int DS = BF && NT * D > 256 ? NT * D / 256 : 1; // warps that share a slice
  static constexpr int TG = CW / DS;                               // slices in work at a time
  static constexpr int TILE = kStageHalf / (D * (int)sizeof(T));   // tokens per stage
  static constexpr int SLICE = BF ? 16 : 4;                        // tokens per warp step
  static constexpr int SL = TILE / SLICE;                          // slices per stage
  static constexpr int USERS = SL < TG ? SL : TG;                  // slices of a stage in work at a time
  static constexpr int QPITCH = D * (int)sizeof(T) + 16;           // bytes; padded: ldmatrix without conflicts
  static constexpr int QBYTES = ROWS * QPITCH;
  static constexpr int JP = D + 4;                                 // join row pitch (floats)
  static constexpr int JOIN = TG * ROWS * (JP + 2) * 4;
  static constexpr int XW = NT * 32 * 16, XA = NT * 8 * 4;         // weights and factors of a shared slice
  static constexpr int XBYTES = DS > 1 ? TG * 2 * (XW + XA) : 0;
  static constexpr int HEAD = 1024;
  static constexpr int FIXED = HEAD + QBYTES + JOIN + XBYTES;
  static constexpr int MOST = 113 * 1024 - 1024;                   // two CTAs per SM; 1024: alignment of the ring
  // Where a stage has fewer slices than are in work, GROUPS sets of warps take the stages
  // in turn; the ring is a multiple of them, so that a stage always has the same readers (a
  // warp two rounds ahead of another's would take a phase that is still to come for done).
  static constexpr int GROUPS = TG / USERS;
  static constexpr int FIT = (MOST - FIXED) / (2 * kStageHalf) < 6 ? (MOST - FIXED) / (2 * kStageHalf) : 6;
  static constexpr int STAGES = FIT - FIT % GROUPS;
  static constexpr int SMEM = FIXED + STAGES * 2 * kStageHalf + 1024;
  static_assert(SL >= 1 && STAGES >= 3 && TG % USERS == 0 && STAGES % GROUPS == 0, "ring");
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
  int valid, bos, x0, nvalid, kvh;
  int pieces;              // CTAs c .. c + pieces - 1 hold its pieces
};

__device__ __noinline__ int64_t div_long(int64_t x, int64_t d) { return x / d; }
// x / d for x / d < 2^31, by the short division where x allows it.
__device__ __forceinline__ int div_small(int64_t x, int d) {
  return x >> 32 ? (int)div_long(x, d) : (int)((uint32_t)x / (uint32_t)d);
}

// Bounds of the ranges: CTA c of n takes [at(c), at(c + 1)) of `total` tiles.
struct Ranges {
  int64_t q;
  int r, n;
  __device__ __forceinline__ Ranges(int64_t total, int ctas) : n(ctas) {
    q = total >> 32 ? div_long(total, ctas) : (uint32_t)total / (uint32_t)ctas;
    r = (int)(total - q * ctas);
  }
  __device__ __forceinline__ int64_t at(int c) const { return q * c + min(c, r); }
  // CTAs that start before position `end` > 0
  __device__ __forceinline__ int before(int64_t end) const {
    const int64_t wide = (q + 1) * r;
    return end <= wide ? (int)div_long(end + q, q + 1) : r + (int)div_long(end - wide + q - 1, q);
  }
};

__host__ __device__ constexpr size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

struct Params {
  PagedAttnArgs a;
  int G, NG, rg_log;           // query heads per kv head, octets per token, log2 of the rows of an octet
  Div by_NG, by_page, by_tile;
  int box, nbox, tile;     // slots per TMA box, boxes per tile, tokens per tile (<= C::TILE)
  int align;               // ranges end at unit borders
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

// Kernels of a few us run their code about once: what is not on the common path is kept out
// of line, since every line of code that is fetched on the way costs time.

// Bounded wait of a whole warp on a phase; gives up when another warp aborted or the time
// ran out, all lanes alike.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  const uint64_t t0 = now_ns();
#pragma unroll 1
  for (uint32_t i = 0; i < kPollCap; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*abort != 0 || now_ns() - t0 > limit) break;
  }
  return false;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  bool ok = tc::mbar_try_wait(bar, parity);
  if (!ok) ok = wait_slow(bar, parity, abort, limit);
  return __all_sync(0xffffffffu, ok);
}

// 2^x and 1 / x by the hardware's approximations (2^-22 and 2^-23 relative; results below
// 2^-126 become 0, -inf gives 0).
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

// One box of a 4-D map.
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
__device__ __forceinline__ int seq_tiles(const Params& p, const Seq& q) { return p.by_tile.quot(q.len + p.tile - 1); }
template <typename C>
__device__ __forceinline__ int seq_groups(const Params& p, const Seq& q) {   // octet groups per kv head
  return (int)(((int64_t)q.n * p.NG + C::NT - 1) / C::NT);
}

template <typename C>
__device__ __forceinline__ int64_t seq_work(const Params& p, const Seq& q) {
  return q.len == 0 ? 0 : (int64_t)(seq_tiles(p, q) + kUnitCost) * seq_groups<C>(p, q) * p.a.Nkv;
}

// The next sequence behind s with anything to attend (the warp looks at 32 at a time); its
// index, num_seqs when there is none.
__device__ __noinline__ int next_seq(const PagedAttnArgs& a, int s, Seq* q) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int base = s + 1; base < a.num_seqs; base += 32) {
    const Seq c = base + lane < a.num_seqs ? load_seq(a, base + lane) : Seq{0, 0, 0};
    const uint32_t has = __ballot_sync(0xffffffffu, c.len > 0);
    if (has != 0) {
      const int w = __ffs(has) - 1;
      q->bos = __shfl_sync(0xffffffffu, c.bos, w);
      q->n = __shfl_sync(0xffffffffu, c.n, w);
      q->len = __shfl_sync(0xffffffffu, c.len, w);
      return base + w;
    }
  }
  return a.num_seqs;
}
// The rows of a sequence with nothing to attend, by a warp.
__device__ __noinline__ void zero_rows(const PagedAttnArgs& a, const Seq& q) {
  const int64_t b = (int64_t)q.bos * a.Nq * a.D, e = b + (int64_t)q.n * a.Nq * a.D;
  const float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int64_t i = b + (threadIdx.x & 31) * 4; i < e; i += 128) {
    if (a.out_bf16) store4(static_cast<bf16*>(a.o) + i, z);
    else store4(static_cast<float*>(a.o) + i, z);
  }
}

// Four elements of (token t, head h) from d: the gate, and y = o * sigmoid(gate).
template <typename T>
__device__ __forceinline__ void gate4(const PagedAttnArgs& a, int t, int h, int d, float (&g)[4]) {
  if (a.gate.p != nullptr) load4(static_cast<const T*>(a.gate.p) + t * a.gate.ts + h * a.gate.hs + d, g);
}
__device__ __forceinline__ void finish4(const PagedAttnArgs& a, int t, int h, int d, int D, const float (&g)[4],
                                        float (&y)[4]) {
  if (a.gate.p != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= rcp(1.f + ex2(-kLog2e * g[i]));
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
  static constexpr int NO = NT / C::DS;            // octets whose weights it computes
  static_assert(OS * NT <= 16 && NO >= 1, "64 accumulators");
  float o[NT][OS][4];
  float m[NO][2], l[NO][2];
  uint32_t qf[NO][KS][2];
  int d0, n0;                                      // first of its blocks and octets
  uint32_t xw;                                     // exchange buffer of the warps that share its slices
  uint32_t flip;

  __device__ __forceinline__ void start(const uint8_t* q, int share, uint8_t* x, int lane) {
    d0 = share * OS;
    n0 = share * NO;
    xw = tc::smem_u32(x);
    flip = 0;
    // x4: two k steps of one octet; lanes 8i..8i+7 give the rows of matrix i
    const uint32_t qaddr = tc::smem_u32(q) + (n0 * 8 + (lane & 7)) * C::QPITCH + (lane >> 3) * 16;
#pragma unroll
    for (int k = 0; k < NO; ++k) {
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
        uint32_t r[4];
        ldsm4(qaddr + k * 8 * C::QPITCH + ks * 32, r);
        qf[k][ks][0] = r[0]; qf[k][ks][1] = r[1];
        qf[k][ks + 1][0] = r[2]; qf[k][ks + 1][1] = r[3];
      }
      m[k][0] = m[k][1] = -INFINITY;
      l[k][0] = l[k][1] = 0.f;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < OS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
  }

  static constexpr bool QREG = true;
  // Slice of the 16 tokens from tok0, rows j0.. of the stage; lim(nt): tokens octet nt sees.
  template <typename Lim>
  __device__ __forceinline__ void slice(uint8_t* ks_, uint8_t* vs_, int j0, int tok0, int nvalid, float c, Lim lim,
                                        int tw, int lane) {
    float s[NO][4], s1[NO][4];                     // two accumulators: half the chain of dependent products
#pragma unroll
    for (int k = 0; k < NO; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[k][e] = s1[k][e] = 0.f;
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
        for (int k = 0; k < NO; ++k) {
          mma16816(s[k], a0, qf[k][ks][0], qf[k][ks][1]);
          mma16816(s1[k], a1, qf[k][ks + 1][0], qf[k][ks + 1][1]);
        }
      }
    }
    const bool tail = tok0 + 16 > lim(0);          // octets come in order of their token: lim(0) is the least
    const int g = lane >> 2, t = lane & 3;
    uint32_t w[NT][4];                             // weights: high parts of both 8-token halves, low parts
    float al[NT][2];                               // factors of the outputs so far
#pragma unroll
    for (int k = 0; k < NO; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[k][e] = (s[k][e] + s1[k][e]) * c;
      if (tail) {
        const int last = lim(n0 + k) - tok0;
        if (g >= last) s[k][0] = s[k][1] = -INFINITY;
        if (g + 8 >= last) s[k][2] = s[k][3] = -INFINITY;
      }
      float mx[2] = {fmaxf(s[k][0], s[k][2]), fmaxf(s[k][1], s[k][3])};
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[k][e], mx[e]);
        al[k][e] = mn == m[k][e] ? 1.f : ex2(m[k][e] - mn);      // (-inf stays -inf: no change)
        m[k][e] = mn;
      }
      const float b0 = m[k][0] == -INFINITY ? 0.f : m[k][0], b1 = m[k][1] == -INFINITY ? 0.f : m[k][1];
      const float p0 = ex2(s[k][0] - b0), p1 = ex2(s[k][1] - b1);
      const float p2 = ex2(s[k][2] - b0), p3 = ex2(s[k][3] - b1);
      l[k][0] = fmaf(l[k][0], al[k][0], p0 + p2);
      l[k][1] = fmaf(l[k][1], al[k][1], p1 + p3);
      const uint32_t h0 = pack_bf16(p0, p1), h1 = pack_bf16(p2, p3);
      const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h0));
      const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h1));
      w[k][0] = movm(h0);
      w[k][1] = movm(h1);
      w[k][2] = movm(pack_bf16(p0 - f0.x, p1 - f0.y));
      w[k][3] = movm(pack_bf16(p2 - f1.x, p3 - f1.y));
    }
    if (C::DS > 1) {
      // all octets' weights and factors through the exchange buffer; two of them in turn: a
      // warp writes one again only after a barrier that the others reach behind their reads
      const uint32_t xb = xw + flip * (C::XW + C::XA);
      flip ^= 1;
#pragma unroll
      for (int k = 0; k < NO; ++k) {
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(xb + ((n0 + k) * 32 + lane) * 16), "r"(w[k][0]),
                     "r"(w[k][1]), "r"(w[k][2]), "r"(w[k][3]) : "memory");
        if (g == 0)
          asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(xb + C::XW + ((n0 + k) * 8 + 2 * t) * 4), "f"(al[k][0]),
                       "f"(al[k][1]) : "memory");
      }
      tc::named_sync(2 + tw, C::DS * 32);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[nt][0]), "=r"(w[nt][1]), "=r"(w[nt][2]), "=r"(w[nt][3])
                     : "r"(xb + (nt * 32 + lane) * 16) : "memory");
        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(al[nt][0]), "=f"(al[nt][1])
                     : "r"(xb + C::XW + (nt * 8 + 2 * t) * 4) : "memory");
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (__any_sync(0xffffffffu, al[nt][0] != 1.f || al[nt][1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < OS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] *= al[nt][e & 1];
      }
    }
    const int vrow = j0 + (lane & 7) + ((lane >> 4) << 3);
    const uint32_t vbase = tc::smem_u32(vs_) + vrow * 128;
    const uint32_t vsw = (uint32_t)(vrow & 7);
    auto vfrag = [&](int b, uint32_t (&a)[4]) {
      const int i = d0 + b;
      const uint32_t ch = (uint32_t)((i & 3) * 2 + ((lane >> 3) & 1));
      ldsm4t(vbase + (i >> 2) * (C::TILE * 128) + ((ch ^ vsw) << 4), a);
    };
    // Rows that an octet does not see may hold anything, and 0 * NaN is NaN: at the end of the
    // visible range they are cleared in the stage, in the columns that this warp reads, once
    // where all octets see the same (mixed: the slice holds new tokens that only some see).
    auto clear = [&](int last) {
#pragma unroll 1
      for (int e = lane; e < (16 - last) * (2 * OS); e += 32) {
        const int r = j0 + last + e / (2 * OS), ch = 2 * d0 + e % (2 * OS);
        *reinterpret_cast<uint4*>(vs_ + (ch >> 3) * (C::TILE * 128) + r * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    };
    const bool mixed = tail && min(lim(NT - 1), tok0 + 16) > lim(0);
    if (NT > 1 && mixed) {
      // from the octet that sees most to the one that sees least
#pragma unroll
      for (int nt = NT - 1; nt >= 0; --nt) {
        if (nt >= nvalid) continue;
        clear(max(0, min(16, lim(nt) - tok0)));
#pragma unroll
        for (int i = 0; i < OS; ++i) {
          uint32_t a[4];
          vfrag(i, a);
          mma16816(o[nt][i], a, w[nt][0], w[nt][1]);
          mma16816(o[nt][i], a, w[nt][2], w[nt][3]);
        }
        __syncwarp();
      }
    } else {
      if (tail) clear(max(0, min(16, lim(0) - tok0)));
#pragma unroll
      for (int i = 0; i < OS; ++i) {
        uint32_t a[4];
        vfrag(i, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a, w[nt][0], w[nt][1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a, w[nt][2], w[nt][3]);
      }
    }
    if (tail) tc::fence_proxy_async_smem();        // before the ring's next copy into the cleared rows
  }

  // This warp's share into the join buffers (any: it took a slice).
  __device__ __forceinline__ void give(float* jo, float* jm, float* jl, bool any, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k = 0; k < NO; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[k][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (g == 0) {
          jm[(n0 + k) * 8 + 2 * t + e] = m[k][e];
          jl[(n0 + k) * 8 + 2 * t + e] = v;
        }
      }
    if (!any) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < OS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          jo[(nt * 8 + 2 * t + (e & 1)) * C::JP + (d0 + i) * 16 + g + (e >> 1) * 8] = o[nt][i][e];
  }
};

// float32 on the CUDA cores, four tokens at a time.  Eight lanes span a head row; the four
// groups of eight take two rows of an octet each (or one, where an octet has four), so that
// a dot product is summed over 8 lanes only: with 32 lanes across the row the exchanges were
// half of the instructions (147 per token and warp, 54 % of the issue slots), with 4 the reads
// of shared memory bound it.  The sums end with one score of the 8 x 4 per lane and octet: one
// exponential each.  NT octets share what is read of the cache; their reductions run side by
// side, without a branch between them.  6 new tokens of 149 sequences of 6511 (64-wide heads, 8
// per kv head, pages of 20) took 995 us with one octet at a time, 886 with four, 591 with the two
// whose queries and outputs stay in registers (440 with what followed elsewhere).  Element pairs go through the packed fp32x2
// operations.  Slower were products in three tf32 parts on the matrix instructions (but for
// 64-wide heads: the splits cost more than they save) and a token per lane group with all rows in
// each (a quarter of the shared memory reads, but longer chains: 34.8 against 30.8 us for 32
// ragged sequences of up to 4000, 111 against 87 for 16 x 4096 with four new tokens each).
template <int D, int NT, int RG>
struct SimtWarp {
  using C = Cfg<float, D, NT, RG>;
  static constexpr int E = D / 32;                 // 4-element chunks per lane: columns 32 i + 4 (lane % 8)
  static constexpr int H = RG / 4;                 // rows of an octet per lane group
  static constexpr bool QREG = NT * H * E < 16;    // queries in registers; at 64 of them they stay in shared memory
  float2 q[QREG ? NT : 1][QREG ? H : 1][QREG ? E : 1][2], o[NT][H][E][2];
  float m[NT], l[NT];                              // of row `mine`
  uint32_t q_at;

  static __device__ __forceinline__ int mine(int lane) { return RG == 8 ? lane >> 2 : lane >> 3; }
  // lane that holds the score of this lane group's row h, token i
  static __device__ __forceinline__ int holder(int lane, int h, int i) { return (lane & 24) + h * 4 + i; }
  static __device__ __forceinline__ void chunk(uint32_t at, float2 (&x)[2]) {
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x[0].x), "=f"(x[0].y), "=f"(x[1].x), "=f"(x[1].y)
                 : "r"(at) : "memory");
  }
  __device__ __forceinline__ void start(const uint8_t* qs, int, uint8_t*, int lane) {
    q_at = tc::smem_u32(qs) + (lane >> 3) * H * C::QPITCH + (lane & 7) * 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (QREG) chunk(q_at + (nt * RG + h) * C::QPITCH + e * 128, q[nt][h][e]);
          o[nt][h][e][0] = o[nt][h][e][1] = make_float2(0.f, 0.f);
        }
      m[nt] = -INFINITY;
      l[nt] = 0.f;
    }
  }
  template <typename Lim>
  __device__ __forceinline__ void slice(uint8_t* ks_, uint8_t* vs_, int j0, int tok0, int, float c, Lim lim,
                                        int, int lane) {
    const uint32_t k_at = tc::smem_u32(ks_) + j0 * (D * 4) + (lane & 7) * 16;
    const uint32_t v_at = tc::smem_u32(vs_) + j0 * (D * 4) + (lane & 7) * 16;
    float2 a[4][NT][H];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float2 k[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) chunk(k_at + i * (D * 4) + e * 128, k[i]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          float2 qe[2];
          if (QREG) {
            qe[0] = q[nt][h][e][0];
            qe[1] = q[nt][h][e][1];
          } else {
            chunk(q_at + (nt * RG + h) * C::QPITCH + e * 128, qe);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i][nt][h] = e == 0 ? __fmul2_rn(qe[0], k[i][0]) : __ffma2_rn(qe[0], k[i][0], a[i][nt][h]);
            a[i][nt][h] = __ffma2_rn(qe[1], k[i][1], a[i][nt][h]);
          }
        }
      }
    }
    // step by step for all octets, without a branch between them: each step's exchanges overlap
    float p[NT], al[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      p[nt] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float d;
        if (H == 2) {                              // lanes 4..7 of a group go on with the second row
          const bool up = (lane & 4) != 0;
          const float d0 = a[i][nt][0].x + a[i][nt][0].y, d1 = a[i][nt][H - 1].x + a[i][nt][H - 1].y;
          d = (up ? d1 : d0) + __shfl_xor_sync(0xffffffffu, up ? d0 : d1, 4);
        } else {
          d = a[i][nt][0].x + a[i][nt][0].y;
          d += __shfl_xor_sync(0xffffffffu, d, 4);
        }
        d += __shfl_xor_sync(0xffffffffu, d, 2);
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        if ((lane & 3) == i) p[nt] = d;
      }
    }
    int last[NT];                                  // tokens of the slice that an octet sees (not falling with nt)
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      last[nt] = lim(nt) - tok0;
      p[nt] = (lane & 3) < last[nt] ? p[nt] * c : -INFINITY;
      float mx = fmaxf(p[nt], __shfl_xor_sync(0xffffffffu, p[nt], 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[nt], mx);
      al[nt] = mn == m[nt] ? 1.f : ex2(m[nt] - mn);
      up = up || al[nt] != 1.f;
      m[nt] = mn;
      p[nt] = ex2(p[nt] - (mn == -INFINITY ? 0.f : mn));
      l[nt] = fmaf(l[nt], al[nt], p[nt]);
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float f = __shfl_sync(0xffffffffu, al[nt], holder(lane, h, 0));
#pragma unroll
          for (int e = 0; e < E; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k) o[nt][h][e][k] = __fmul2_rn(o[nt][h][e][k], make_float2(f, f));
        }
    }
    auto values = [&](int i, bool all) {           // a token's values into the octets that see it
      float2 v[E][2];
#pragma unroll
      for (int e = 0; e < E; ++e) chunk(v_at + i * (D * 4) + e * 128, v[e]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (!all && i >= last[nt]) continue;       // what an octet does not see may hold anything
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float x = __shfl_sync(0xffffffffu, p[nt], holder(lane, h, i));
#pragma unroll
          for (int e = 0; e < E; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k) o[nt][h][e][k] = __ffma2_rn(make_float2(x, x), v[e][k], o[nt][h][e][k]);
        }
      }
    };
    if (last[0] >= 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) values(i, true);
    } else {
#pragma unroll 1
      for (int i = 0; i < min(4, last[NT - 1]); ++i) values(i, false);
    }
  }
  __device__ __forceinline__ void give(float* jo, float* jm, float* jl, bool any, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float v = l[nt];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      if ((lane & 3) == 0 && (RG == 8 || (lane & 4) == 0)) {
        jm[nt * RG + mine(lane)] = m[nt];
        jl[nt * RG + mine(lane)] = v;
      }
    }
    if (!any) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e)
          *reinterpret_cast<float4*>(jo + (nt * RG + (lane >> 3) * H + h) * C::JP + e * 32 + (lane & 7) * 4) =
              make_float4(o[nt][h][e][0].x, o[nt][h][e][0].y, o[nt][h][e][1].x, o[nt][h][e][1].y);
  }
};
template <typename T, int D, int NT, int RG> struct WarpOf { using type = TcWarp<D, NT>; };
template <int D, int NT, int RG> struct WarpOf<float, D, NT, RG> { using type = SimtWarp<D, NT, RG>; };

// ------------------------------------------------------------------ the main kernel
template <typename T, int D, int NT, int RG>
__global__ void __launch_bounds__(Cfg<T, D, NT, RG>::THREADS, kOcc)
paged_attn_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ Params p) {
  using C = Cfg<T, D, NT, RG>;
  constexpr int COLS = 128 / (int)sizeof(T);       // columns of a box (128 bytes, swizzled) in bf16
  constexpr int CB = C::BF ? D / COLS : 1;         // boxes across a row; float32: whole rows, not swizzled
  extern __shared__ __align__(16) uint8_t raw[];
  uint8_t* ring = tc::smem_aligned<1024>(raw);
  uint8_t* qs = ring + C::STAGES * 2 * kStageHalf;
  uint8_t* xs = qs + C::QBYTES;
  float* jo = reinterpret_cast<float*>(xs + C::XBYTES);
  float* jm = jo + C::TG * C::ROWS * C::JP;
  float* jl = jm + C::TG * C::ROWS;
  uint8_t* head = reinterpret_cast<uint8_t*>(jl + C::TG * C::ROWS);
  uint64_t* full = reinterpret_cast<uint64_t*>(head);
  uint64_t* empty = full + C::STAGES;
  uint64_t* qfull = empty + C::STAGES;
  uint64_t* qempty = qfull + 1;
  Piece* piece = reinterpret_cast<Piece*>(head + 256);
  int64_t* scan = reinterpret_cast<int64_t*>(head + 512);          // [CW + 1] warp sums
  int64_t* from = scan + C::CW + 1;                                // where the range starts: the sequence's first tile
  int* from_seq = reinterpret_cast<int*>(from + 1);                // and the sequence: index, bos, n, len
  volatile int* abort = reinterpret_cast<int*>(head + 768);
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_launch_next();
  if (tid == C::CW * 32) {
#pragma unroll 1
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, C::USERS * C::DS);
    }
    tc::mbar_init(qfull, 1);
    tc::mbar_init(qempty, C::CW);
    *abort = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&mk);
    tc::prefetch_tmap(&mv);
  }
  // rows of an octet without a query head are never copied: finite, or their columns would be
  // rescaled at every slice
#pragma unroll 1
  for (int i = tid; i < C::QBYTES / 16; i += C::THREADS) reinterpret_cast<uint4*>(qs)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  pdl_wait();
  // all tiles, and the sequence that this CTA's range starts in
  const int per = (a.num_seqs + C::THREADS - 1) / C::THREADS;
  const int s_lo = min(a.num_seqs, tid * per), s_hi = min(a.num_seqs, s_lo + per);
  int64_t sum = 0;
#pragma unroll 1
  for (int s = s_lo; s < s_hi; ++s) sum += seq_work<C>(p, load_seq(a, s));
  int64_t inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w <= C::CW; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const Ranges rg(total, (int)max((int64_t)1, min((int64_t)gridDim.x, total / kMinTiles)));
  const bool mine = (int)blockIdx.x < rg.n;
  const int64_t lo = mine ? rg.at(blockIdx.x) : total;
  const int64_t hi = mine ? rg.at(blockIdx.x + 1) : total;
  if (before <= lo && lo < before + sum) {
    int64_t at = before;
#pragma unroll 1
    for (int s = s_lo; s < s_hi; ++s) {
      const Seq q = load_seq(a, s);
      const int64_t w = seq_work<C>(p, q);
      if (lo < at + w) {
        *from = at;
        from_seq[0] = s;
        from_seq[1] = q.bos;
        from_seq[2] = q.n;
        from_seq[3] = q.len;
        break;
      }
      at += w;
    }
  }
  __syncthreads();

  if (warp == C::CW) {
    // ------------------------------------------------------------ producer
    SplitRec rec{};
    int it = 0, npiece = 0;
    const int boxes = a.skip & 2 ? 0 : p.nbox;     // (no copies: the test of waits that run out)
    bool ok = true;
    if (lo < hi) {
      int s = from_seq[0];
      Seq q{from_seq[1], from_seq[2], from_seq[3]};
      int tiles = seq_tiles(p, q), groups = seq_groups<C>(p, q);
      int64_t seq_at = *from, pos = lo;
      int cost = tiles + kUnitCost;                // of a unit; its tiles lie at the end
      int unit = div_small(pos - seq_at, cost);
      if (p.align && seq_at + (int64_t)unit * cost < pos) ++unit;          // the first unit that starts here
      if (p.align) pos = seq_at + (int64_t)unit * cost;
#pragma unroll 1
      while (pos < hi) {
        if (unit >= groups * a.Nkv) {
          seq_at += (int64_t)cost * groups * a.Nkv;
          s = next_seq(a, s, &q);
          if (s >= a.num_seqs) break;              // (cannot be: pos < hi <= total)
          tiles = seq_tiles(p, q);
          groups = seq_groups<C>(p, q);
          cost = tiles + kUnitCost;
          unit = 0;
          continue;
        }
        const int64_t unit_at = seq_at + (int64_t)unit * cost;
        const int t0 = max(0, (int)(pos - unit_at) - kUnitCost);
        const int t1 = p.align ? tiles : (int)min((int64_t)tiles, hi - unit_at - kUnitCost);
        if (t1 <= t0) break;                       // the range ends before the unit's first tile
        const int kvh = unit / groups, x0 = (unit % groups) * NT;
        const int nvalid = min(NT, q.n * p.NG - x0);
        const int32_t* bt = a.c.bt + (int64_t)s * a.c.max_pages;
        // page and slot of this lane's first box, one tile ahead of its use
        auto lookup = [&](int tile, int b, int& page, int& off) {
          const int tok = tile * p.tile + b * p.box;
          page = a.c.num_pages;                    // out of range: zero fill
          off = 0;
          if (tok < q.len && b < p.nbox) {
            const int at = p.by_page.quot(tok);
            const int pg = __ldg(bt + at);
            off = tok - at * a.c.page_size;
            if (pg >= 0 && pg < a.c.num_pages) page = pg;
            else raise_error(a.err, kDevErrCache);
          }
        };
        int page, off;
        lookup(t0, lane, page, off);
#pragma unroll 1
        for (int tile = t0; tile < t1; ++tile, ++it) {
          int npage = 0, noff = 0;
          const int st = it % C::STAGES;
          ok = wait_bar(empty + st, ((it / C::STAGES) & 1) ^ 1, abort, p.a.wait_ns);
          if (!ok) break;
          uint8_t* kd = ring + st * 2 * kStageHalf;
          if (lane == 0) tc::mbar_arrive_expect_tx(full + st, p.tile * (2 * kStageHalf / C::TILE));
          __syncwarp();
#pragma unroll 1
          for (int b = lane; b < boxes; b += 32) {
            if (b >= 32) lookup(tile, b, page, off);
            auto axis = [&](int i) { return a.c.order[i] == 0 ? off : a.c.order[i] == 1 ? kvh : page; };
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
              const int dst = cb * (C::TILE * 128) + b * p.box * (kStageHalf / C::TILE / CB);
              tma_load_4d(kd + dst, &mk, full + st, cb * COLS, axis(0), axis(1), axis(2));
              tma_load_4d(kd + kStageHalf + dst, &mv, full + st, cb * COLS, axis(0), axis(1), axis(2));
            }
          }
          if (tile + 1 < t1) lookup(tile + 1, lane, npage, noff);
          page = npage;
          off = noff;
          if (tile != t0) continue;
          // behind its first tile: the piece and its query rows.  Octet x of the sequence is token
          // x / NG, heads (x % NG) * 8 .. of the kv head's G
          ok = wait_bar(qempty, (npiece & 1) ^ 1, abort, p.a.wait_ns);
          if (!ok) {
            ++it;                                  // (this tile is in flight)
            break;
          }
          int rows = 0;
          auto head_of = [&](int r, int& tok) {    // head within the kv head's, and token, of row r
            const int x = x0 + r / RG;
            tok = p.by_NG.quot(x);
            return (x - tok * p.NG) * RG + r % RG;
          };
          int tok;
#pragma unroll 1
          for (int r = lane; r < nvalid * RG; r += 32) rows += head_of(r, tok) < p.G;
          rows = __reduce_add_sync(0xffffffffu, rows);
          if (lane == 0) {
            Piece d;
            d.tile0 = t0; d.tile1 = t1;
            d.slot = t0 == 0 && t1 == tiles ? -1 : 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
            d.len = q.len; d.n = q.n; d.bos = q.bos; d.x0 = x0; d.nvalid = nvalid; d.kvh = kvh;
            *piece = d;
            if (t0 == 0 && t1 < tiles)
              rec = {1, q.bos, x0, nvalid, kvh, rg.before(unit_at + cost) - (int)blockIdx.x};
            tc::mbar_arrive_expect_tx(qfull, (uint32_t)(rows * D * sizeof(T)));
          }
          __syncwarp();
#pragma unroll 1
          for (int r = lane; r < nvalid * RG; r += 32) {
            const int h = head_of(r, tok);
            if (h < p.G && !(a.skip & 1)) {
              tc::bulk_load(qs + r * C::QPITCH,
                            static_cast<const T*>(a.q.p) + (q.bos + tok) * a.q.ts + (kvh * p.G + h) * a.q.hs,
                            D * sizeof(T), qfull);
              if (a.gate.p != nullptr && t1 - t0 == tiles) {   // needed at the end of the piece
                const T* gp = static_cast<const T*>(a.gate.p) + (q.bos + tok) * a.gate.ts + (kvh * p.G + h) * a.gate.hs;
#pragma unroll 1
                for (int i = 0; i < D; i += 128 / (int)sizeof(T))
                  asm volatile("prefetch.global.L2 [%0];" ::"l"(gp + i));
              }
            }
          }
          ++npiece;
        }
        if (!ok) break;
        pos = unit_at + cost;
        ++unit;
      }
    }
    if (ok) {
      ok = wait_bar(qempty, (npiece & 1) ^ 1, abort, p.a.wait_ns);
      if (ok && lane == 0) {
        piece->tile0 = -1;
        tc::mbar_arrive(qfull);
      }
    }
    if (lane == 0 && !p.align) p.rec[blockIdx.x] = rec;
    if (!ok && lane == 0) {
      *abort = 1;
      raise_error(a.err, kDevErrTimeout);
    }
    // every copy lands before the CTA's shared memory goes, whatever the consumers do
    int none = 0;
#pragma unroll 1
    for (int i = max(0, it - C::STAGES); i < it; ++i) wait_bar(full + i % C::STAGES, (i / C::STAGES) & 1, &none, p.a.wait_ns);
    if (!ok && npiece > 0) wait_bar(qfull, (npiece - 1) & 1, &none, p.a.wait_ns);
    return;
  }

  // -------------------------------------------------------------- consumers
  // sequences with nothing to attend: their rows are zero; every sequence's metadata is checked once
#pragma unroll 1
  for (int s = blockIdx.x * C::CW + warp; s < a.num_seqs; s += gridDim.x * C::CW) {
    const Seq q = load_seq(a, s, lane == 0 ? a.err : nullptr);
    if (q.n > 0 && q.len == 0) zero_rows(a, q);
  }
  const int tw = warp % C::TG;                     // which slices; warps tw + k TG share them
  // The slices go round the warps from stage to stage.  In float32 also where tiles are not full:
  // five slices of four tokens on four warps took 592 us for the case at SimtWarp (in tiles of
  // 20), this way 461.  In bf16 the arithmetic is not what bounds such tiles, and a count that is
  // no constant cost full ones (45.0 against 47.5 us for 35 ragged sequences, 64-wide heads).
  const int turn = C::BF || C::SL < C::TG ? C::SL : (p.tile + C::SLICE - 1) / C::SLICE;
  typename WarpOf<T, D, NT, RG>::type w;
  int it = 0;
  // After a wait that ran out a warp leaves its piece and goes to the next barrier of all consumers,
  // where they agree to stop; on the way it meets the warps that share its slices at each slice's
  // barrier, so that none is left short of a warp.  It hands no stage back: one that did not fill
  // must not be armed again.
#pragma unroll 1
  for (int np = 0;; ++np) {
    bool ok = wait_bar(qfull, np & 1, abort, p.a.wait_ns);
    if (tc::named_sync_or(1, C::CW * 32, !ok)) {
      if (lane == 0) {
        *abort = 1;
        raise_error(a.err, kDevErrTimeout);
      }
      break;
    }
    const Piece d = *piece;
    if (d.tile0 < 0) break;
    w.start(qs, warp / C::TG, xs + tw * 2 * (C::XW + C::XA), lane);
    __syncwarp();
    if (decltype(w)::QREG && lane == 0) tc::mbar_arrive(qempty);
    auto lim = [&](int nt) { return d.len - d.n + p.by_NG.quot(d.x0 + min(nt, d.nvalid - 1)) + 1; };
    const int most = lim(NT - 1);
    bool any = false;
#pragma unroll 1
    for (int tile = d.tile0; tile < d.tile1; ++tile, ++it) {
      int j = (tw - it * turn) & (C::TG - 1);      // this warp's first slice of the stage
      if (j >= C::SL) continue;
      const int st = it % C::STAGES;
      if (!wait_bar(full + st, (it / C::STAGES) & 1, abort, p.a.wait_ns)) {
        ok = false;
        if (lane == 0) *abort = 1;                 // ends the waits of the others
        if (C::DS > 1) {
#pragma unroll 1
          for (; tile < d.tile1; ++tile, ++it)
#pragma unroll 1
            for (j = (tw - it * turn) & (C::TG - 1); j < C::SL; j += C::TG)
              if (tile * p.tile + j * C::SLICE < min(most, (tile + 1) * p.tile)) tc::named_sync(2 + tw, C::DS * 32);
        }
        break;
      }
      uint8_t* kd = ring + st * 2 * kStageHalf;
#pragma unroll 1
      for (; j < C::SL; j += C::TG) {
        const int tok0 = tile * p.tile + j * C::SLICE, end = (tile + 1) * p.tile;
        if (tok0 < min(most, end)) {
          auto seen = [&](int nt) { return min(lim(nt), end); };           // rows behind the tile's last are not loaded
          w.slice(kd, kd + kStageHalf, j * C::SLICE, tok0, d.nvalid, p.c, seen, tw, lane);
          any = true;
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty + st);
    }
    // the warps' shares joined
    w.give(jo + tw * C::ROWS * C::JP, jm + tw * C::ROWS, jl + tw * C::ROWS, any, lane);
    if (tc::named_sync_or(1, C::CW * 32, !ok)) {
      if (lane == 0) {
        *abort = 1;
        raise_error(a.err, kDevErrTimeout);
      }
      break;
    }
    // a thread per row: each share's weight in the row (in place of its maximum)
    if (tid < d.nvalid * RG) {
      float mt = -INFINITY, lt = 0.f, f[C::TG];
#pragma unroll
      for (int k = 0; k < C::TG; ++k) mt = fmaxf(mt, jm[k * C::ROWS + tid]);
      const float base = mt == -INFINITY ? 0.f : mt;
#pragma unroll
      for (int k = 0; k < C::TG; ++k) {
        f[k] = ex2(jm[k * C::ROWS + tid] - base);
        lt = fmaf(jl[k * C::ROWS + tid], f[k], lt);
      }
      const float inv = d.slot >= 0 ? 1.f : lt == 0.f ? 0.f : rcp(lt);
#pragma unroll
      for (int k = 0; k < C::TG; ++k) jm[k * C::ROWS + tid] = f[k] * inv;
      if (d.slot >= 0)
        *reinterpret_cast<float2*>(p.part_ml + ((int64_t)d.slot * C::ROWS + tid) * 2) = make_float2(mt, lt);
    }
    tc::named_sync(1, C::CW * 32);
    auto joined = [&](int r, int e, float (&y)[4]) {
      y[0] = y[1] = y[2] = y[3] = 0.f;
#pragma unroll
      for (int k = 0; k < C::TG; ++k) {
        const float f = jm[k * C::ROWS + r];
        if (f == 0.f) continue;                    // (the outputs of a share without slices are not written)
        const float4 v = *reinterpret_cast<const float4*>(jo + (k * C::ROWS + r) * C::JP + e);
        y[0] = fmaf(v.x, f, y[0]); y[1] = fmaf(v.y, f, y[1]);
        y[2] = fmaf(v.z, f, y[2]); y[3] = fmaf(v.w, f, y[3]);
      }
    };
    const int groups4 = d.nvalid * RG * (D / 4);
    if (d.slot >= 0) {
      float* po = p.part_o + (int64_t)d.slot * C::ROWS * D;
#pragma unroll 4
      for (int i = tid; i < groups4; i += C::CW * 32) {
        float y[4];
        joined(i / (D / 4), i % (D / 4) * 4, y);
        store4(po + i * 4, y);
      }
    } else {
      // the next four columns' gate loaded ahead
      auto place = [&](int i, int& tok) {          // head of group i (-1: no such row), and token
        const int r = i / (D / 4), x = d.x0 + r / RG, t = p.by_NG.quot(x), h = (x - t * p.NG) * RG + r % RG;
        tok = d.bos + t;
        return i < groups4 && h < p.G ? d.kvh * p.G + h : -1;
      };
      int tok, hd = place(tid, tok);
      float gt[4];
      if (hd >= 0) gate4<T>(a, tok, hd, tid % (D / 4) * 4, gt);
#pragma unroll 1
      for (int i = tid; i < groups4; i += C::CW * 32) {
        int ntok, nhd = place(i + C::CW * 32, ntok);
        float ngt[4];
        if (nhd >= 0) gate4<T>(a, ntok, nhd, (i + C::CW * 32) % (D / 4) * 4, ngt);
        if (hd >= 0) {
          float y[4];
          joined(i / (D / 4), i % (D / 4) * 4, y);
          finish4(a, tok, hd, i % (D / 4) * 4, D, gt, y);
        }
        tok = ntok;
        hd = nhd;
#pragma unroll
        for (int k = 0; k < 4; ++k) gt[k] = ngt[k];
      }
    }
    tc::named_sync(1, C::CW * 32);
    if (!decltype(w)::QREG && lane == 0) tc::mbar_arrive(qempty);
  }
}

// ------------------------------------------------------------------ the join
// Launched while the main kernel runs; the first step is to wait for its end.  Three forms,
// by how many units can be cut at most, so that neither blocks start for nothing nor many
// pieces wait for one another.  The whole call with the third form below, with PG = 4 and with PG =
// 1, us, bf16, 131072 tokens in all, so many units of 256-wide heads: 1 unit 33, 45 and 65; 2 52, 58 and 69; 8
// 51, 52 and 55; 16 53.5, 51.3 and 52.0; 32 57.7, 50.9 and 51.3; 128 81, 53.5 and 51.1; with more units
// than half of the CTAs, 160 (PG = 4: 54.8) and 256 (57.9), PG = 1 takes 51.2 and 52.2.
//
// PG = 1, about as many units as CTAs (about two pieces each): blocks (c, y) join the unit that starts
// in CTA c's range and ends behind it, if there is one; a thread takes four columns of a row.
// PG = 4, fewer units: blocks (u, y) join the unit of the u-th CTA with a record; four lanes
// share four columns, each with every fourth piece.
constexpr int kJoinThreads = 256;
__device__ __forceinline__ int64_t piece_row(int c0, int i, int rows, int row) {
  // CTA c0's last piece (slot 2 c0 + 1), then the first ones of the CTAs behind it
  return ((int64_t)2 * (c0 + i) + (i == 0 ? 1 : 0)) * rows + row;
}
// The record of the nth CTA that has one, and that CTA (-1 if there are fewer), for all threads of
// the block: every record is loaded at once, so that finding the one costs no second load.
template <int THREADS>
__device__ __forceinline__ SplitRec nth_record(const Params& p, int ctas, int nth, int* found, int& cta) {
  constexpr int PER = (kMaxCtas + THREADS - 1) / THREADS, WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  SplitRec r[PER];
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
  if (lane == 0) found[warp] = cnt;
  if (tid == 0) found[WARPS] = -1;
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) at += i < warp ? found[i] : 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (r[i].valid != 0 && at + __popc(mask[i] & ((1u << lane) - 1)) == nth) {
      found[WARPS] = (warp * PER + i) * 32 + lane;
      *reinterpret_cast<SplitRec*>(found + WARPS + 1) = r[i];
    }
    at += __popc(mask[i]);
  }
  __syncthreads();
  cta = found[WARPS];
  return *reinterpret_cast<const SplitRec*>(found + WARPS + 1);
}
template <typename T, int D, int PG>
__global__ void __launch_bounds__(kJoinThreads)
paged_attn_join_kernel(const __grid_constant__ Params p, int ctas, int rows) {
  __shared__ int found[kJoinThreads / 32 + 1 + sizeof(SplitRec) / 4];
  pdl_launch_next();
  pdl_wait();
  int c0 = blockIdx.x;
  const SplitRec r = PG > 1 ? nth_record<kJoinThreads>(p, ctas, blockIdx.x, found, c0) : p.rec[c0];
  if (c0 < 0) return;
  // lanes: 32 / PG column groups side by side, PG times
  const int lane = threadIdx.x & 31, k0 = lane / (32 / PG);
  const int i = (blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5)) * (32 / PG) + lane % (32 / PG);
  const int row = i / (D / 4), e = (i % (D / 4)) * 4;
  const int oct = row >> p.rg_log, x = r.x0 + oct, t = p.by_NG.quot(x);
  const int h = ((x - t * p.NG - oct) << p.rg_log) + row;
  const bool live = r.valid && oct < r.nvalid && h < p.G;
  if (!__any_sync(0xffffffffu, live)) return;
  float gt[4], m = -INFINITY, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
  if (live && k0 == 0) gate4<T>(p.a, r.bos + t, r.kvh * p.G + h, e, gt);
#pragma unroll 1
  for (int j0 = k0; live && j0 < r.pieces; j0 += 4 * PG) {
    float2 ml[4];
    float v[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ml[j] = make_float2(-INFINITY, 0.f);
      v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.f;
      if (j0 + j * PG < r.pieces) {
        const int64_t at = piece_row(c0, j0 + j * PG, rows, row);
        ml[j] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
        load4(p.part_o + at * D + e, v[j]);
      }
    }
    const float mn = fmaxf(fmaxf(fmaxf(m, ml[0].x), fmaxf(ml[1].x, ml[2].x)), ml[3].x);
    const float base = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - base);
    l *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] *= f0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = ex2(ml[j].x - base);
      l = fmaf(ml[j].y, f, l);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = fmaf(v[j][k], f, y[k]);
    }
    m = mn;
  }
#pragma unroll
  for (int off = 32 / PG; off < 32; off <<= 1) {   // the lanes that share the columns
    const float mo = __shfl_xor_sync(0xffffffffu, m, off), mn = fmaxf(m, mo), base = mn == -INFINITY ? 0.f : mn;
    const float f0 = ex2(m - base), f1 = ex2(mo - base);
    l = l * f0 + __shfl_xor_sync(0xffffffffu, l, off) * f1;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = y[k] * f0 + __shfl_xor_sync(0xffffffffu, y[k], off) * f1;
    m = mn;
  }
  if (!live || k0 != 0) return;
  const float inv = l == 0.f ? 0.f : rcp(l);
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] *= inv;
  finish4(p.a, r.bos + t, r.kvh * p.G + h, e, D, gt, y);
}

// Few units (so many pieces): block (u, row, z) joins 64 columns of a row of the u-th CTA
// with a record.  All its loads but the records are independent: the outputs, 32 pieces at
// a time, and the maxima and sums (a thread per piece) for their weights.
constexpr int kFewThreads = 512;
template <typename T, int D>
__global__ void __launch_bounds__(kFewThreads)
paged_attn_join_few_kernel(const __grid_constant__ Params p, int ctas) {
  constexpr int LPR = 16;                          // threads across the columns
  constexpr int NP = kFewThreads / LPR;            // pieces in flight
  constexpr int WARPS = kFewThreads / 32;
  static_assert(kMaxCtas <= kFewThreads, "a thread per CTA");
  __shared__ float sw[kMaxCtas], so[WARPS][64], red[2][WARPS];
  __shared__ int found[WARPS + 1 + sizeof(SplitRec) / 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_next();
  pdl_wait();
  int c0;
  const SplitRec r = nth_record<kFewThreads>(p, ctas, blockIdx.x, found, c0);
  if (c0 < 0) return;
  const int row = blockIdx.y, oct = row >> p.rg_log, x = r.x0 + oct, t = p.by_NG.quot(x);
  const int h = ((x - t * p.NG - oct) << p.rg_log) + row;
  if (oct >= r.nvalid || h >= p.G) return;
  constexpr int U = 5;                             // loads in flight per thread (2, 3 and 10: all calls within 1 us)
  const int k = tid / LPR, col = (tid % LPR) * 4, e = blockIdx.z * 64 + col, n = r.pieces;
  float v[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (k + u * NP < n) load4(p.part_o + piece_row(c0, k + u * NP, gridDim.y, row) * D + e, v[u]);
  const float2 ml = tid < n ? *reinterpret_cast<const float2*>(p.part_ml + piece_row(c0, tid, gridDim.y, row) * 2)
                            : make_float2(-INFINITY, 0.f);
  float gt[4];
  if (k == 0) gate4<T>(p.a, r.bos + t, r.kvh * p.G + h, e, gt);
  float m = ml.x;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) m = fmaxf(m, red[0][i]);
  const float w = ex2(ml.x - (m == -INFINITY ? 0.f : m));
  float l = w * ml.y;
  sw[tid] = w;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) l += red[1][i];
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int i = k; i < n; i += U * NP) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u * NP >= n) break;
      const float f = sw[i + u * NP];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = fmaf(v[u][j], f, y[j]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int next = i + (U + u) * NP;
      if (next < n) load4(p.part_o + piece_row(c0, next, gridDim.y, row) * D + e, v[u]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] += __shfl_xor_sync(0xffffffffu, y[j], LPR);
  if (lane < LPR) store4(&so[warp][col], y);
  __syncthreads();
  if (k != 0) return;
  const float inv = l == 0.f ? 0.f : rcp(l);
#pragma unroll
  for (int i = 1; i < WARPS; ++i) {
    float o[4];
    load4(&so[i][col], o);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += o[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] *= inv;
  finish4(p.a, r.bos + t, r.kvh * p.G + h, e, D, gt, y);
}

// ------------------------------------------------------------------ host
// Rows of an octet: in float32 four where the kv head has no more heads, half the arithmetic
// of eight (with more heads, eight rows mean fewer octets).
int octet_rows(int Nq, int Nkv, bool bf) { return !bf && Nq / Nkv <= 4 ? 4 : 8; }

// Octets per pass at most: as many as the registers hold the outputs (float32: and queries) of.
int most_octets(int rg, int D, bool bf) { return bf ? 4 : std::min(rg == 8 ? 2 : 4, 2048 / (D * rg)); }

// Octets per pass: enough for the new tokens of an even batch (a unit's rows then read the cache
// once).  In float32 a pass of four takes 1.7 times one of two (16 x 4096 tokens, 128-wide heads:
// 87 and 50 us), so twos where the last four would be half empty (153 sequences with 6 octets: 46
// against 55 us).
int octets_per_pass(int num_seqs, int total, int Nq, int Nkv, int D, bool bf) {
  const int rg = octet_rows(Nq, Nkv, bf);
  const int64_t want = (int64_t)((total + num_seqs - 1) / num_seqs) * ((Nq / Nkv + rg - 1) / rg);
  const int most = most_octets(rg, D, bf);
  int nt = 1;
  while (nt < want && nt < most) nt *= 2;
  if (!bf && nt == 4 && want > 4 && (want - 1) % 4 < 2) nt = 2;
  return nt;
}

// Slots per box and boxes per tile.  A box has to end where a page does, so its slots divide a
// page's; a tile that no number of them fills stays partly empty.  The time of a tile grows with
// its boxes (of K and V, a box per 64 columns in bf16) about as `fixed` + boxes, beside its share
// of the stream: least per slot is best.  Measured for 16 x 4096 tokens in bf16, 64-, 128- and
// 256-wide heads: pages of 20, full tiles of 4-slot boxes 52, 48 and 49 us, tiles of 60 of 64,
// 30 of 32 and 10 of 16 slots 32, 34 and 41; pages of 24, full tiles of 8-slot boxes 38, 36 and
// 36 us, 48 of 64, 24 of 32 and 12 of 16 slots 33, 32 and 36.  In float32 the arithmetic goes
// by whole tiles too, and a full one is worth nearly any boxes (the case at SimtWarp: 440 us with
// eight boxes of 4 slots, 486 with three of 10, 461 with one of 20).
void tile_boxes(int page_size, int tile, bool bf, int D, int* box, int* n) {
  const int fixed = bf ? 16 : 256, per = bf ? D / 32 : 2;
  int best = 0;
  for (int d = 1; d <= std::min(page_size, tile); ++d) {
    if (page_size % d != 0) continue;
    const int k = tile / d, cost = fixed + per * k;
    if (best == 0 || (int64_t)cost * *box * *n <= (int64_t)best * d * k) {
      best = cost;
      *box = d;
      *n = k;
    }
  }
}

// Tables so short that ranges end at unit borders, by full tiles: the page size is not known where
// the workspace's size is asked for.
bool short_table(int D, bool bf, int64_t table_tokens) {
  return table_tokens <= (int64_t)kAlignTiles * (kStageHalf / (D * (bf ? 2 : 4)));
}

// A 4-D map over the cache: D, then slot, head and page by increasing stride (each stride has to
// be a multiple of the one before); boxes of `box` slots and `cols` elements.
bool cache_map(CUtensorMap* map, const void* base, const PagedAttnArgs& a, int cols, int box) {
  EncodeTiledFn enc = tmap_encoder();
  if (enc == nullptr) return false;
  const int es = a.in_bf16 ? 2 : 4;
  const int ext[3] = {a.c.page_size, a.Nkv, a.c.num_pages};
  cuuint64_t dims[4] = {(cuuint64_t)a.D}, strides[3];
  cuuint32_t bx[4] = {(cuuint32_t)cols};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = (cuuint64_t)ext[a.c.order[i]];
    strides[i] = (cuuint64_t)a.c.sorted[i] * es;
    bx[i + 1] = a.c.order[i] == 0 ? (cuuint32_t)box : 1;
  }
  cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, a.in_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
             const_cast<void*>(base), dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             a.in_bf16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int NT, int RG = 8>
cudaError_t launch_c(const PagedAttnArgs& a, cudaStream_t s) {
  using C = Cfg<T, D, NT, RG>;
  const auto fn = paged_attn_kernel<T, D, NT, RG>;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  const int grid = std::min(kOcc * num_sms(), kMaxCtas);
  Params p{};
  p.a = a;
  p.G = a.Nq / a.Nkv;
  p.NG = (p.G + RG - 1) / RG;
  p.rg_log = RG == 8 ? 3 : 2;
  p.by_NG = Div::of(p.NG);
  p.by_page = Div::of(a.c.page_size);
  tile_boxes(a.c.page_size, C::TILE, C::BF, D, &p.box, &p.nbox);
  p.tile = p.box * p.nbox;
  p.by_tile = Div::of(p.tile);
  p.align = short_table(D, C::BF, (int64_t)a.c.max_pages * a.c.page_size);
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
  e = launch_early(fn, dim3(grid), dim3(C::THREADS), C::SMEM, s, mk, mv, p);
  if (e != cudaSuccess || p.align) return e;
  // at most so many units can be cut, into so many pieces each on average
  const int64_t per_seq = a.cu == nullptr ? ((int64_t)(a.total / a.num_seqs) * p.NG + NT - 1) / NT : 0;
  const int64_t units = a.cu == nullptr ? per_seq * a.num_seqs * a.Nkv
                                        : (int64_t)a.Nkv * (a.num_seqs + (int64_t)a.total * p.NG / NT);
  const bool few = units * 16 <= grid && units * C::ROWS * (D / 64) <= 4 * num_sms();
  const bool many = units * 2 > grid;
  if (few)
    return launch_early(paged_attn_join_few_kernel<T, D>, dim3((int)units, C::ROWS, D / 64), dim3(kFewThreads), 0, s, p,
                        grid);
  if (many)
    return launch_early(paged_attn_join_kernel<T, D, 1>, dim3(grid, (C::ROWS * D / 4 + kJoinThreads - 1) / kJoinThreads),
                        dim3(kJoinThreads), 0, s, p, grid, (int)C::ROWS);
  return launch_early(paged_attn_join_kernel<T, D, 4>, dim3((int)units, C::ROWS * D / kJoinThreads), dim3(kJoinThreads), 0,
                      s, p, grid, (int)C::ROWS);
}

template <int D>
cudaError_t launch_bf16(const PagedAttnArgs& a, int nt, cudaStream_t s) {
  if (nt == 1) return launch_c<bf16, D, 1>(a, s);
  if (nt == 2) return launch_c<bf16, D, 2>(a, s);
  return launch_c<bf16, D, 4>(a, s);
}

template <int D, int RG>
cudaError_t launch_f32(const PagedAttnArgs& a, int nt, cudaStream_t s) {
  if constexpr (RG == 4 && D <= 128) {
    if (nt == 4) return launch_c<float, D, 4, RG>(a, s);
  }
  if constexpr (D * RG <= 1024) {
    if (nt == 2) return launch_c<float, D, 2, RG>(a, s);
  }
  return nt == 1 ? launch_c<float, D, 1, RG>(a, s) : cudaErrorInvalidValue;
}

}  // namespace

// For the most rows of a pass, so that one workspace serves calls of any numbers of tokens.
size_t paged_attn_workspace_bytes(int Nq, int Nkv, int D, bool bf, int64_t table_tokens) {
  if (short_table(D, bf, table_tokens)) return 0;
  const int rg = octet_rows(Nq, Nkv, bf);
  const size_t rows = (size_t)most_octets(rg, D, bf) * rg;
  const size_t grid = std::min(kOcc * num_sms(), kMaxCtas);
  return align16(sizeof(SplitRec) * grid) + align16(2 * grid * rows * 2 * 4) + 2 * grid * rows * D * 4;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
  const int nt = octets_per_pass(a.num_seqs, a.total, a.Nq, a.Nkv, a.D, a.in_bf16);
  if (a.in_bf16)
    return a.D == 64 ? launch_bf16<64>(a, nt, s) : a.D == 128 ? launch_bf16<128>(a, nt, s) : launch_bf16<256>(a, nt, s);
  if (octet_rows(a.Nq, a.Nkv, false) == 4)
    return a.D == 64 ? launch_f32<64, 4>(a, nt, s) : a.D == 128 ? launch_f32<128, 4>(a, nt, s) : launch_f32<256, 4>(a, nt, s);
  return a.D == 64 ? launch_f32<64, 8>(a, nt, s) : a.D == 128 ? launch_f32<128, 8>(a, nt, s) : launch_f32<256, 8>(a, nt, s);
}

}  // namespace gdn
