// The paged cache's metadata of the next step from the requests' lengths: which sequence gets
// which pages, the bounds of the packed new tokens, their positions and cache slots.
//
//   after[s] = lens[s] + add[s] (0 for an ended sequence);  need[s] = ceil(after[s] / P) where add[s] > 0
//   take[s] = max(0, need[s] - held[s]) pages from the ring of free ones, sequence by sequence
//   cu = prefix sums of max(add, 0);  token i of s: position lens[s] + i, slot page * P + position % P
//
// Bound: latency.  The bytes are a few per sequence and twelve per token (a megabyte for 70,000
// tokens), so what counts is one launch and few dependent reads (7.3 us for 256 requests, 10 for the prompts of 16 sequences
// with 70,000 tokens, in a graph).  One cluster does it all: each
// CTA scans all sequences for itself (three sums), which is cheaper than to wait for one that
// does, and takes its share of the tokens and pages; a cluster barrier separates the last read of
// the state from its update, so the update may be in place.
//
// Either the whole request fits or nothing changes: the checks' outcome is the same in every CTA.

#include <cooperative_groups.h>

#include "attn_util.cuh"
#include "gdn.h"
#include "paged_attn.h"
#include "serving.h"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

// One cluster of 8 CTAs of 512 threads.  1, 4 and 8 CTAs, us: 256 requests of one token 8.5, 8.4 and 7.3, of five 11.7, 11.8 and
// 8.2; 70,000 slots of 16 prompts 51, 16 and 10; 4096 requests 27, 18 and 17.  256 and 1024 threads: 4096 requests 20 and
// 24, the prompts 15 and 12.
constexpr int kCtas = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kMost = 0x7fffffff;
constexpr uint32_t kStop = 0x80000000u;
constexpr int kRest = GDN_PLAN_REST;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {          // a, b <= kStop
  const uint32_t s = a + b;
  return s < a ? kStop : min(s, kStop);            // (both kStop: 0)
}

// Three running sums that stop at kStop: above every number of tokens or pages that a call can have, so that no request
// which reaches it fits.
struct Sums {
  uint32_t add, take, back;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {sat_add(a.add, b.add), sat_add(a.take, b.take), sat_add(a.back, b.back)};
}

// The last index i of start[0..n) with start[i] <= x (start[0] = 0, not falling).
__device__ __forceinline__ int owner(const int32_t* start, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(const __grid_constant__ PagePlanArgs p, Div by_page) {
  extern __shared__ int32_t starts[];              // cu, then the first page taken and given back, of each sequence
  __shared__ Sums warp_sum[2][kWarps];
  __shared__ int bad_any;
  const int N = p.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t *cu = starts, *taken = starts + N, *given = starts + 2 * N;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  if (tid == 0) bad_any = 0;
  pdl_launch_next();
  pdl_wait();
  const int64_t head = p.ring[0], count = p.ring[1], pages = p.num_pages;
  bool bad = head < 0 || head >= pages || count < 0 || count > pages;
  const int64_t most = (int64_t)p.max_pages * p.page_size;
  Sums base{0, 0, 0};
#pragma unroll 1
  for (int s0 = 0, turn = 0; s0 < N; s0 += kThreads, turn ^= 1) {
    const int s = s0 + tid;
    Sums x{0, 0, 0};
    if (s < N) {
      const int add = p.add[s], len = p.lens[s], held = p.held[s];
      if (held < 0 || held > p.max_pages) {
        bad = true;
      } else if (add == kRest && s == N - 1) {
        bad = bad || len != 0;
      } else if (add < 0) {
        x.back = held;
      } else if (len < 0 || len > (int64_t)held * p.page_size || (int64_t)len + add > min(most, kMost)) {
        bad = true;
      } else if (add > 0) {
        x.add = add;
        x.take = max(0, by_page.quot(len + add - 1) + 1 - held);
      }
    }
    Sums inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const Sums o{__shfl_up_sync(0xffffffffu, inc.add, off), __shfl_up_sync(0xffffffffu, inc.take, off),
                   __shfl_up_sync(0xffffffffu, inc.back, off)};
      if (lane >= off) inc = inc + o;
    }
    if (lane == 31) warp_sum[turn][warp] = inc;
    __syncthreads();
    Sums before = base;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before = before + warp_sum[turn][w];
      base = base + warp_sum[turn][w];
    }
    if (s < N) {
      // exclusive sums; where a sum has stopped nothing of it is used
      cu[s] = before.add + (inc.add - x.add);
      taken[s] = before.take + (inc.take - x.take);
      given[s] = before.back + (inc.back - x.back);
    }
  }
  bad = bad || base.add > (uint32_t)p.total || (int64_t)base.take > count ||
        count + (int64_t)base.back > pages;        // (pages both free and held: those given back would meet those being taken)
  if (bad) bad_any = 1;
  __syncthreads();
  bad = bad_any != 0;
  const int total = bad ? 0 : (int)base.add, n_take = bad ? 0 : (int)base.take, n_back = bad ? 0 : (int)base.back;
  auto free_at = [&](int64_t i) {                  // entry head + i of the ring, i < 2 pages
    int64_t at = head + i;
    if (at >= pages) at -= pages;
    if (at >= pages) at -= pages;
    return at;
  };
  const int me = rank * kThreads + tid, all = ranks * kThreads;
  // pages taken
#pragma unroll 1
  for (int i = me; i < n_take; i += all) {
    const int s = owner(taken, N, i);
    const int pg = p.free_pages[free_at(i)];
    if (pg < 0 || pg >= p.num_pages) raise_error(p.err, kDevErrCache);
    p.bt[(int64_t)s * p.max_pages + p.held[s] + (i - taken[s])] = pg;
  }
  // positions and slots of four tokens at a time; rows behind the last token: position 0, slot -1
#pragma unroll 1
  for (int64_t t0 = (int64_t)me * 4; t0 < p.total; t0 += (int64_t)all * 4) {
    int32_t pos[4] = {0, 0, 0, 0};
    int64_t slot[4] = {-1, -1, -1, -1};
    int s = -1, end = 0, len = 0, held = 0, at = -1, pg = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (int)t0 + k;
      if (t >= total) break;
      if (s < 0 || t >= end) {
        s = owner(cu, N, t);
        end = s + 1 < N ? cu[s + 1] : total;
        len = p.lens[s];
        held = p.held[s];
        at = -1;
      }
      pos[k] = len + (t - cu[s]);
      const int page = by_page.quot(pos[k]);
      if (page != at) {
        at = page;
        pg = at < held ? p.bt[(int64_t)s * p.max_pages + at] : p.free_pages[free_at(taken[s] + (at - held))];
        if (pg < 0 || pg >= p.num_pages) {
          raise_error(p.err, kDevErrCache);
          pg = -1;
        }
      }
      slot[k] = pg < 0 ? -1 : (int64_t)pg * p.page_size + (pos[k] - at * p.page_size);
    }
    if (t0 + 4 <= p.total) {
      if (p.pos != nullptr) *reinterpret_cast<int4*>(p.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.slots != nullptr) {
        *reinterpret_cast<longlong2*>(p.slots + t0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(p.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (t0 + k >= p.total) break;
        if (p.pos != nullptr) p.pos[t0 + k] = pos[k];
        if (p.slots != nullptr) p.slots[t0 + k] = slot[k];
      }
    }
  }
  // pages that go back, behind the free ones (the entries taken above are not among those
  // written here: free, held and given back pages together are at most the ring's)
#pragma unroll 1
  for (int i = me; i < n_back; i += all) {
    const int s = owner(given, N, i);
    const int pg = p.bt[(int64_t)s * p.max_pages + (i - given[s])];
    if (pg < 0 || pg >= p.num_pages) raise_error(p.err, kDevErrCache);
    p.free_pages[free_at(count + i)] = pg;
  }
  // the state's update, once every CTA has read what it needs
  cluster.sync();
#pragma unroll 1
  for (int s = me; s < N; s += all) {
    const int len = p.lens[s], held = p.held[s], ask = p.add[s], add = ask == kRest ? 0 : ask;
    const bool gone = add < 0;
    p.cu[s] = bad ? 0 : cu[s];
    p.lens_out[s] = bad ? len : gone ? 0 : len + add;
    const int need = add > 0 && !bad ? by_page.quot(len + add - 1) + 1 : 0;
    p.held_out[s] = bad ? held : gone ? 0 : max(held, need);
  }
  if (me == 0) {
    p.cu[N] = !bad && p.add[N - 1] == kRest ? p.total : total;
    p.ring_out[0] = bad ? (int32_t)head : (int32_t)free_at(n_take);
    p.ring_out[1] = (int32_t)(count - n_take + n_back);
    if (bad) raise_error(p.err, kDevErrPlan);
  }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs& p, cudaStream_t s) {
  const int smem = 3 * p.num_seqs * 4;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (smem > 40 * 1024 && (dev < 0 || dev >= 64 || !ready[dev])) {
    e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * kPlanMaxSeqs * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  constexpr int ctas = kCtas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, page_plan_kernel, p, Div::of(p.page_size));
}

}  // namespace gdn
