// kvq_block_plan.cu -- a step's block tables, packed offsets and slot maps from
// the requests' lengths.
//
// Everything is prefix sums over at most 1024 requests, one per thread: blocks
// that come back, blocks and token slots asked for, then (for those that are
// served) blocks, token slots and touched blocks.  Each CTA of one cluster does
// all of the sums for itself from the same inputs, so nothing passes between
// CTAs; the cluster's threads then share the entries to write.  New block k is
// the k-th from the top of the stack of what was free and what comes back, a
// function of the old arrays alone: entries of the stack above the old count
// are looked up in the ending request's table row, not in the stack that is
// being written.  Written places and read places are apart, except the lengths
// and the count, which may be updated in place: a cluster barrier stands between
// the last read and the first write.  Where tokens are taken back, a row's blocks
// behind its new length come back while the same entries get new ones: all that
// comes back is then on the stack, behind a second cluster barrier, before any new
// block is looked up, in the stack alone (64 requests, five tokens each: 3.9 us
// without, 4.1 with one of each taken back; 256 of 29 tokens, 8 CTAs: 5.4 and 6.1).
//
// Bound: latency.  The bytes of a step (a few 100 KB at most) take less than a
// microsecond; a launch, two rounds of loads and the sums take the rest.
#include <cooperative_groups.h>

#include "kvq_block.cuh"

namespace kvq {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;  // at most
constexpr int kPlanCtas = 8;

// Inclusive sums over the CTA of up to three values per thread.
template <int V>
__device__ __forceinline__ void sum_scan(long long (&v)[V], long long (*warp_sums)[32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v[i], o);
      if (lane >= o) v[i] += x;
    }
  __syncthreads();  // the sums of the scan before have been read
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < V; ++i) warp_sums[i][w] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    long long x = lane < (int)(blockDim.x >> 5) ? warp_sums[i][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (w) v[i] += __shfl_sync(0xffffffffu, x, w - 1);
  }
}

// The last i with at[i] <= v, for v in [at[0], at[n]): empty ranges are passed over.
__device__ __forceinline__ int range_of(const int* at, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= v) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// BACK: tokens are taken back first (an instantiation of its own: in one kernel the plan
// without it took 3.26 us in place of 2.98 for 16 requests).
template <bool BACK>
__global__ void __launch_bounds__(kPlanThreads) block_plan_kernel(const __grid_constant__ BlockPlanParams p) {
  __shared__ int s_len[kMaxBlockBatch], s_back0[kMaxBlockBatch + 1], s_new0[kMaxBlockBatch + 1], s_start[kMaxBlockBatch + 1];
  __shared__ long long s_warp[3][32];
  const BlockGeo& G = p.geo;
  const int b = threadIdx.x, rank = blockIdx.x;
  const bool mine = b < G.B;
  grid_dep_wait();
  const int free0 = min(max(p.free_before[0], 0), G.n_blocks);
  const int had = mine ? p.lens_before[b] : 0, ask = mine ? p.n_new[b] : 0;
  const int taken = BACK && mine ? p.n_back[b] : 0;  // (of a request that ends: all the same)
  const int row_tokens = G.max_blocks * kBlockTokens;  // <= 2^30
  const bool proper = had >= 0 && had <= row_tokens, can = proper && taken >= 0 && taken <= had;
  const int len = can ? had - taken : had;
  const int held = can ? (len + kBlockTokens - 1) / kBlockTokens : 0;
  const bool fits = mine && can && ask >= 0 && ask <= row_tokens - len;
  const int need = fits ? (len + ask + kBlockTokens - 1) / kBlockTokens - held : 0;
  const bool ends = mine && ask < 0;
  const int all_held = proper ? (had + kBlockTokens - 1) / kBlockTokens : 0;
  long long v[3] = {ends ? all_held : can ? all_held - held : 0, need, fits ? ask : 0};
  const int back = (int)v[0];
  sum_scan(v, s_warp);
  // more than the pool cannot come back: what would not fit the stack is left out
  const long long back_end = min(v[0], (long long)(G.n_blocks - free0));
  __shared__ int s_back;
  if (b == blockDim.x - 1) s_back = (int)back_end;
  __syncthreads();
  const int all = free0 + s_back;
  const bool served = fits && (need == 0 || v[1] <= all) && v[2] <= G.N;
  const int n = served ? ask : 0, fresh = served ? need : 0;
  const int units = n ? (len + n + kBlockTokens - 1) / kBlockTokens - len / kBlockTokens : 0;
  long long u[3] = {fresh, n, units};
  sum_scan(u, s_warp);
  if (mine) {
    s_len[b] = BACK && ends ? 0 : len;
    s_back0[b] = (int)(min(v[0] - back, (long long)(G.n_blocks - free0)));
    s_new0[b] = (int)(u[0] - fresh);
    s_start[b] = (int)(u[1] - n);
    if (b == G.B - 1) {
      s_back0[G.B] = s_back;
      s_new0[G.B] = (int)u[0];
      s_start[G.B] = (int)u[1];
    }
  }
  // every old length and count is read
  if (gridDim.x > 1) cg::this_cluster().sync();
  else __syncthreads();
  grid_dep_trigger();

  if (rank == 0 && mine) {
    p.t.lens[b] = ends ? 0 : len + n;
    p.t.start[b + 1] = (int)u[1];
    p.t.unit0[b + 1] = (int)u[2];
    if (b == 0) {
      p.t.start[0] = 0;
      p.t.unit0[0] = 0;
    }
    if (b == G.B - 1) p.t.free_count[0] = all - s_new0[G.B];
  }
  const int tid = rank * blockDim.x + b, threads = gridDim.x * blockDim.x;
  const auto came_back = [&](int i) {  // the i-th block that comes back
    const int r = range_of(s_back0, G.B, i), kept = BACK ? (s_len[r] + kBlockTokens - 1) / kBlockTokens : 0;
    return p.t.block_table[(size_t)r * G.max_blocks + kept + (i - s_back0[r])];
  };
  const auto popped = [&](int k) {  // the k-th new block
    const int at = all - 1 - k;
    if (BACK) return __ldcg(p.t.free_list + at);
    return at < free0 ? p.t.free_list[at] : came_back(at - free0);
  };
  for (int i = tid; i < s_back; i += threads) p.t.free_list[free0 + i] = came_back(i);
  if (BACK) {
    if (gridDim.x > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  const int total_new = s_new0[G.B], total = s_start[G.B];
  for (int k = tid; k < total_new; k += threads) {
    const int r = range_of(s_new0, G.B, k);
    const int at = (s_len[r] + kBlockTokens - 1) / kBlockTokens + (k - s_new0[r]);
    p.t.block_table[(size_t)r * G.max_blocks + at] = popped(k);
  }
  for (int i = tid; i < G.N; i += threads) {
    int row = -1, pos = 0, slot = -1;
    if (i < total) {
      row = range_of(s_start, G.B, i);
      pos = s_len[row] + (i - s_start[row]);
      const int j = pos / kBlockTokens, held_r = (s_len[row] + kBlockTokens - 1) / kBlockTokens;
      const int id = j < held_r ? p.t.block_table[(size_t)row * G.max_blocks + j] : popped(s_new0[row] + j - held_r);
      slot = (int)((unsigned)id * kBlockTokens + pos % kBlockTokens);
    }
    p.t.token_row[i] = row;
    p.t.position[i] = pos;
    p.t.slot[i] = slot;
  }
}

cudaError_t launch_block_plan(const BlockPlanParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // a thread per request; one CTA where a thread per token slot fits it, too
  const int ctas = p.geo.N <= kPlanThreads ? 1 : kPlanCtas;
  const int want = ctas == 1 ? p.geo.N : 512, threads = ((p.geo.B > want ? p.geo.B : want) + 31) / 32 * 32;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas == 1 ? 1 : 2;
  return p.n_back ? cudaLaunchKernelEx(&cfg, block_plan_kernel<true>, p) : cudaLaunchKernelEx(&cfg, block_plan_kernel<false>, p);
}

}  // namespace kvq
