// Verification of drafted tokens (rejection sampling that keeps the target's distribution).
//
// Sequence s has n rows: its step's tokens x_0 (certain) and x_1 .. x_{n-1} (drafts).  Row i of the
// target's probabilities p judges draft x_{i+1}, drawn from row i of the draft's q:
//   kept while  u_i q_i(x_{i+1}) < p_i(x_{i+1})          (q = 1 at x where no q is given)
// At the first refused draft a token is drawn from w = max(p - q, 0) of that row (from p without x
// where no q is given), after the last row from w = p: by u of the sequence's last row, the first j
// with C_j > u W, C the running sum of w and W its end.
//
// Sums in any order give one result: w counts in whole units of 2^-42 (p and q rounded to them,
// halves to even), u in units of 2^-24, and C_j 2^24 > U W is decided in whole numbers.  A float32 p
// in [0, 1] splits exactly: with a = (p + 6) - 6, a multiple of 2^-21, and p - a,
//   p 2^42 = 2^21 (a 2^21) + (p - a) 2^42,
// both whole parts taken from the low bits of a float sum (p + 6; (p - a) 2^42 + 1.5 2^23).  Differences
// of two p's parts are whole numbers again, so a weight costs a dozen float32 and 32-bit operations
// and the sums of a tile stay in 32 bits.
//
// Bound: HBM, one row of p (and one of q) per sequence; for few sequences latency.  A cluster of CTAs
// per sequence: each judges the drafts for itself (two reads per draft, side by side), sums its
// part of the row by tiles of 1024 elements, and the CTA that holds the level u W finds the tile
// among its sums and reads that tile alone again.  256 sequences of 4 drafts, a vocabulary of 131072 in float32: 41.6 us, 82 % of
// the copy rate; one sequence, 32000: 5.7 us.

#include <cooperative_groups.h>

#include "attn_util.cuh"
#include "paged_attn.h"
#include "serving.h"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

// Runs of 16 bytes in flight per lane and row (B below): 2, 4 and 8 with as many blocks per SM as the registers leave: 51, 42
// and 46 us for the 256 sequences.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 1024;
constexpr int kPer = kTile / 32;                   // elements of a tile per lane
constexpr int kMaxTiles = kVerifyMaxVocab / kTile;

// The whole parts of p in units of 2^-21 and of the rest in units of 2^-42, each over a fixed offset
// that differences cancel; p in [0, 1].
__device__ __forceinline__ void split(float p, uint32_t& hi, uint32_t& lo) {
  const float a = __fadd_rn(p, 6.f);
  hi = __float_as_uint(a);
  lo = __float_as_uint(__fmaf_rn(__fsub_rn(p, __fsub_rn(a, 6.f)), 4398046511104.f, 12582912.f));
}

// E neighbours of a row from element `at` on, as float32; 0 behind element `n`.  E = 1 where rows start anywhere (odd
// vocabularies): 256 x 4 drafts of 50257 take 24 us in either type, of 50256 in bf16 17 and in float32 22.  Two aligned pieces
// of 16 bytes, moved together in registers, instead: 29 and 43 (half as much in flight).
template <int E, typename T>
__device__ __forceinline__ void load(const T* row, int at, int n, float (&x)[E]) {
  if constexpr (E == 1) {
    x[0] = at < n ? to_f32(row[at]) : 0.f;
  } else {                                         // 16 bytes, and n is a multiple of E
    uint4 v = make_uint4(0, 0, 0, 0);
    if (at < n) v = __ldcs(reinterpret_cast<const uint4*>(row + at));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (E == 4) {
        x[k] = __uint_as_float(w[k]);
      } else {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The row that a token is drawn from: p, less q where given, without element `skip`.
template <typename T>
struct Row {
  const T* p;
  const T* q;
  int skip;
};

// Adds the weights of E neighbours from element `at` on, whole units hi 2^21 + lo.  DRAFT: less r.q.
template <int E, bool DRAFT, typename T>
__device__ __forceinline__ void weigh(const Row<T>& r, int at, const float (&p)[E], const float (&q)[E], int32_t (&hi)[E],
                                      int32_t (&lo)[E]) {
#pragma unroll
  for (int k = 0; k < E; ++k) {
    const float pk = __saturatef(p[k]);            // NaN and what is below 0 count as 0, what is above 1 as 1
    uint32_t ph, pl, qh = __float_as_uint(6.f), ql = __float_as_uint(12582912.f);
    split(pk, ph, pl);
    if (DRAFT) split(fminf(pk, __saturatef(q[k])), qh, ql);        // (p - min(p, q) = max(p - q, 0), also in whole units)
    hi[k] = (int32_t)(ph - qh);
    lo[k] = (int32_t)(pl - ql);
    if (!DRAFT && at + k == r.skip) hi[k] = lo[k] = 0;
  }
}
// The weight of a tile, this lane's part.  B runs of E neighbours are in flight at a time.
template <int E, int B, bool DRAFT, typename T>
__device__ __forceinline__ uint64_t tile_sum(const Row<T>& r, int at, int n, int lane) {
  int32_t h = 0, l = 0;                            // 32 times 2^21 at most
#pragma unroll 1
  for (int b = 0; b < kPer / E; b += B) {
    float p[B][E], q[B][E];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      load<E>(r.p, at + ((b + i) * 32 + lane) * E, n, p[i]);
      if (DRAFT) load<E>(r.q, at + ((b + i) * 32 + lane) * E, n, q[i]);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      int32_t hi[E], lo[E];
      weigh<E, DRAFT>(r, at + ((b + i) * 32 + lane) * E, p[i], q[i], hi, lo);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        h += hi[k];
        l += lo[k];
      }
    }
  }
  return (uint64_t)((int64_t)h * (1 << 21) + l);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) draft_verify_kernel(const __grid_constant__ DraftVerifyArgs p) {
  __shared__ uint64_t sums[kMaxTiles];             // of this CTA's tiles
  __shared__ uint64_t part;                        // of this CTA
  __shared__ uint64_t piece[kTile / 32];           // of the tile that is drawn from: the sums of its runs across a warp
  __shared__ uint64_t rest_at;
  __shared__ int first, tile_at;
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1, B = VEC ? 4 : 16;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int s = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_next();
  pdl_wait();
  int bos, eos;
  const bool ok = seq_bounds(p.cu, p.num_seqs, p.total, s, bos, eos);
  const int n = eos - bos;
  if (n <= 0) {                                    // the whole cluster
    if (rank == 0 && tid == 0) {
      if (!ok) raise_error(p.err, kDevErrSeqlens);
      p.accepted[s] = 0;
      if (p.lens != nullptr) p.lens_out[s] = p.lens[s];
    }
    return;
  }
  if (p.lens != nullptr && p.lens[s] == 0) {       // an inactive slot of a padded batch
    cluster.sync();                                // (lens_out may be lens)
    if (rank == 0) {
      for (int i = tid; i < n; i += kThreads) p.out[bos + i] = -1;
      if (tid == 0) p.accepted[s] = p.lens_out[s] = 0;
    }
    return;
  }
  const T* pp = static_cast<const T*>(p.p);
  const T* qq = static_cast<const T*>(p.q);
  if (tid == 0) first = n - 1;
  __syncthreads();
  // the first refused draft
#pragma unroll 1
  for (int i = tid; i < n - 1; i += kThreads) {
    const int x = p.tokens[bos + i + 1];
    const bool known = x >= 0 && x < p.vocab && (qq == nullptr || i < p.q_rows);
    bool keep = false;
    if (known) {
      const float px = to_f32(pp[(int64_t)(bos + i) * p.p_row + x]);
      const float qx = qq == nullptr ? 1.f : to_f32(qq[s * p.q_seq + i * p.q_row + x]);
      keep = (double)p.uniform[bos + i] * (double)qx < (double)px;         // (both products' sides exact)
    } else if (rank == 0) {
      raise_error(p.err, kDevErrDraft);
    }
    if (!keep) atomicMin(&first, i);
  }
  __syncthreads();
  const int a = first;
  Row<T> row{pp + (int64_t)(bos + a) * p.p_row, nullptr, -1};
  if (a < n - 1) {
    if (qq == nullptr) row.skip = p.tokens[bos + a + 1];
    else if (a < p.q_rows) row.q = qq + s * p.q_seq + a * p.q_row;
  }
  const int tiles = (p.vocab + kTile - 1) / kTile, per = (tiles + ranks - 1) / ranks;
  const int lo_tile = min(tiles, rank * per), hi_tile = min(tiles, lo_tile + per);
  const float u = p.uniform[eos - 1];
  const uint64_t U = (uint64_t)floorf(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f) * 16777216.f);
  uint64_t before, level;
#pragma unroll 1
  for (;;) {
#pragma unroll 1
    for (int t = lo_tile + warp; t < hi_tile; t += kWarps) {
      const uint64_t sum = warp_sum64(row.q != nullptr ? tile_sum<E, B, true>(row, t * kTile, p.vocab, lane)
                                                       : tile_sum<E, B, false>(row, t * kTile, p.vocab, lane));
      if (lane == 0) sums[t - lo_tile] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      uint64_t v = 0;
#pragma unroll 1
      for (int t = lane; t < hi_tile - lo_tile; t += 32) v += sums[t];
      v = warp_sum64(v);
      if (lane == 0) part = v;
    }
    cluster.sync();
    before = 0;
    uint64_t W = 0;
#pragma unroll 1
    for (int r = 0; r < ranks; ++r) {
      const uint64_t v = *cluster.map_shared_rank(&part, r);
      if (r < rank) before += v;
      W += v;
    }
    level = (W >> 24) * U + (((W & 0xffffffu) * U) >> 24);
    cluster.sync();                                // (part may be written again, or its CTA end)
    if (W != 0) break;
    if (row.q == nullptr && row.skip < 0) {        // no weight at all: no token
      if (rank == 0 && tid == 0) {
        raise_error(p.err, kDevErrDraft);
        p.out[bos + a] = -1;
      }
      level = ~(uint64_t)0;
      break;
    }
    row.q = nullptr;                               // nothing is left of p: drawn from p itself
    row.skip = -1;
  }
  if (rank == 0) {
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads)
      if (i != a) p.out[bos + i] = i < a ? p.tokens[bos + i + 1] : -1;
    if (tid == 0) {
      p.accepted[s] = a;
      if (p.lens != nullptr) p.lens_out[s] = p.lens[s] - (n - 1 - a);
    }
  }
  if (level < before || level - before >= part) return;            // another CTA's part holds the level
  // the tile: warp 0 goes through the sums, 32 at a time
  auto scan = [&](uint64_t v) {                    // inclusive, across the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint64_t o = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += o;
    }
    return v;
  };
  if (warp == 0) {
    uint64_t rest = level - before;
#pragma unroll 1
    for (int t0 = 0; t0 < hi_tile - lo_tile; t0 += 32) {
      const uint64_t v = t0 + lane < hi_tile - lo_tile ? sums[t0 + lane] : 0, inc = scan(v);
      const uint32_t over = __ballot_sync(0xffffffffu, inc > rest);
      if (over != 0) {
        if (lane == __ffs(over) - 1) {
          tile_at = lo_tile + t0 + lane;
          rest_at = rest - (inc - v);
        }
        break;
      }
      rest -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  // its runs of E neighbours per lane, all warps side by side
  constexpr int PIECES = kPer / E;
  const int base = tile_at * kTile;
  auto run_of = [&](int i, uint64_t (&run)[E]) {   // running sums of this lane's neighbours in piece i
    const int at = base + (i * 32 + lane) * E;
    float x[E], y[E];
    int32_t hi[E], lo[E];
    load<E>(row.p, at, p.vocab, x);
    if (row.q != nullptr) {
      load<E>(row.q, at, p.vocab, y);
      weigh<E, true>(row, at, x, y, hi, lo);
    } else {
      weigh<E, false>(row, at, x, y, hi, lo);
    }
    uint64_t v = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      v += (uint64_t)((int64_t)hi[k] * (1 << 21) + lo[k]);
      run[k] = v;
    }
  };
#pragma unroll 1
  for (int i = warp; i < PIECES; i += kWarps) {
    uint64_t run[E];
    run_of(i, run);
    const uint64_t v = warp_sum64(run[E - 1]);
    if (lane == 0) piece[i] = v;
  }
  __syncthreads();
  if (warp != 0) return;
  uint64_t rest = rest_at;
  const uint64_t v = lane < PIECES ? piece[lane] : 0, inc = scan(v);
  const int i = __ffs(__ballot_sync(0xffffffffu, inc > rest)) - 1;
  rest -= __shfl_sync(0xffffffffu, inc - v, i);
  uint64_t run[E];
  run_of(i, run);
  const uint64_t all = scan(run[E - 1]);
  const uint32_t over = __ballot_sync(0xffffffffu, all > rest);
  if (lane == __ffs(over) - 1) {
    const uint64_t mine = rest - (all - run[E - 1]);
    int k = 0;
#pragma unroll
    for (int j = 0; j < E - 1; ++j) k += run[j] <= mine;
    p.out[bos + a] = base + (i * 32 + lane) * E + k;
  }
}

template <typename T>
cudaError_t launch_t(const DraftVerifyArgs& p, cudaStream_t s) {
  // CTAs per sequence: eight (a portable cluster) where the sequences alone do not fill the device.  1, 2, 4 and 8, us, most
  // drafts kept, the rule's choice in brackets: 512 x 2 drafts of 32000 in float32 [17.2], 20.2, 26.9 and 48.5; 256 x 4 of 131072
  // 43.2, [27.6], 31.3 and 39.0, of 50256 in bf16 18.8, [13.1], 16.9 and 26.0; 128 x 4 of those 15.6, 13.0, [9.9] and 14.6; 100 x 4
  // of 131072 in float32 30.7, 19.5, [16.2] and 19.6, 64 x 4 27.7, 20.0, 14.9 and [12.0], 16 x 4 26.4, 15.5, 10.3 and [8.8]; one of
  // 32000 7.4, 5.6, 5.1 and [5.2].
  int ctas = 8;
  while (ctas > 1 && ((int64_t)p.num_seqs * ctas > 4 * num_sms() || ctas * kTile > p.vocab)) ctas /= 2;
  const int64_t unit = 16 / sizeof(T);
  const bool vec = p.vocab % unit == 0 && p.p_row % unit == 0 && p.q_seq % unit == 0 && p.q_row % unit == 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.num_seqs * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return vec ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<T, true>, p) : cudaLaunchKernelEx(&cfg, draft_verify_kernel<T, false>, p);
}

}  // namespace

cudaError_t launch_draft_verify(const DraftVerifyArgs& p, cudaStream_t s) {
  return p.bf16 ? launch_t<bf16>(p, s) : launch_t<float>(p, s);
}

}  // namespace gdn
