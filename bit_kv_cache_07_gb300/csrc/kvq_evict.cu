// kvq_evict.cu -- eviction of the 32-token groups with the least accumulated
// attention weight, compacting the cache in place.
//
// Per stream with n groups of which E leave, left = n - E:
//   total_j = sum of the group's 32 recorded weights,
//   gone    = the first E groups in ascending order of (total_j, j),
//   the k-th group slot < left that was freed takes the k-th kept group from
//   the slots >= left (both ascending).
// Attention does not depend on the order of the keys (they carry their
// positions), so at most E groups move, never the whole tail, and every
// source lies behind every destination: the moves are independent of one
// another.  The fp16 window follows in order.
//
// Three launches: totals (and a copy of the window, whose slots shift); one
// CTA per stream that selects, plans the moves and compacts the record; the
// moves.  The unquantized cache, whose window lands where groups leave from,
// writes its window in a fourth.
//
// Measured: 16 x 32k tokens K8V4, 8 KV heads, a quarter leaves: 93 us (4.2 TB/s
// over the whole call), of which the moves are 60 (some 350 MB read and written
// in copies of 4 KB to 256 bytes: 5.8 TB/s), the totals 15 and the selection, a
// chain of CTA-wide steps per stream, 17; 4 ragged rows up to 8k fp16, three
// tenths: 27 us (1.7 TB/s); one sequence of 2k: 37 to 46 us, which is the host's
// time (21 on the GPU).  What bounds the large call: the totals and the
// selection before the moves, a third of it for 17 MB of record.
#include "kvq_evict.cuh"

namespace kvq {
namespace {

constexpr int kSumThreads = 256;
constexpr int kSelThreads = 1024;
constexpr int kOwn = 4;  // keys per thread of the selection in registers
constexpr int kMoveThreads = 256;

// A float as its signed 24-bit mantissa and exponent (of the last bit).
__device__ __forceinline__ void decompose(float x, int* mant, int* exp) {
  const uint32_t u = __float_as_uint(x);
  const int e = (u >> 23) & 255;
  const int m = (int)(u & 0x7FFFFFu) | (e ? 0x800000 : 0);
  *mant = (u >> 31) ? -m : m;
  *exp = e ? e : 1;
}

// Order-preserving key of a total (NaN last, -0 as 0).
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// Totals of the groups as order keys, four threads per group; then copies of
// the window rows.  The sum is exact to 2^-57 of the group's largest weight
// and does not depend on the order: mantissas are aligned to the largest
// exponent in 64-bit integers (fp64 adds are a narrow pipe on this GPU), and
// only their sum is rounded to fp64.
__global__ void __launch_bounds__(kSumThreads) evict_sum_kernel(const __grid_constant__ EvictParams p) {
  grid_dep_trigger();
  const Geometry& G = p.geo;
  if ((int)blockIdx.x < p.sum_blocks) {
    const int per = kSumThreads / 4;  // groups per CTA
    const int bps = (p.cap + per - 1) / per, s = blockIdx.x / bps, j = (blockIdx.x - s * bps) * per + (threadIdx.x >> 2);
    const int b = s / G.Hkv, T = p.tokens[b], ng = group_count(p, T);
    if ((blockIdx.x - s * bps) * per >= ng || p.evict[b] == 0) return;  // the whole CTA
    const bool have = j < ng;
    const float* m = p.mass + (size_t)s * p.max_tokens + p.S + (size_t)j * kGroupTokens + 8 * (threadIdx.x & 3);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = have ? m[i] : 0.0f;
    int mant[8], exp[8], top = 1;
    float plain = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      decompose(x[i], &mant[i], &exp[i]);
      if (mant[i]) top = max(top, exp[i]);
      plain += exp[i] == 255 ? x[i] : 0.0f;  // finite ones cannot move an infinity, their fp32 sum could
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      plain += __shfl_xor_sync(0xffffffffu, plain, o);
    }
    long long sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = top - exp[i];
      if (d < 58) sum += ((long long)mant[i] << 34) >> d;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (have && (threadIdx.x & 3) == 0) {
      // an infinity or a NaN among them: what adding them gives
      const double total = top == 255 ? (double)plain : scalbn((double)sum, top - 150 - 34);
      p.keys[(size_t)s * p.cap + j] = order_key(total);
    }
    return;
  }
  // window rows (256 bytes of K, then of V) into the workspace
  const long long rows = (long long)G.NS * p.save_rows * 2;
  for (long long i = (long long)(blockIdx.x - p.sum_blocks) * (kSumThreads / 16) + (threadIdx.x >> 4); i < rows;
       i += (long long)p.save_blocks * (kSumThreads / 16)) {
    const int row = (int)(i % p.save_rows);
    const long long sv = i / p.save_rows;
    const int s = (int)(sv >> 1), b = s / G.Hkv;
    if (p.evict[b] == 0) continue;
    int slot = row;
    if (G.fp16_mode) {
      slot = p.S + kGroupTokens * group_count(p, p.tokens[b]) + row;
      if (slot >= p.tokens[b]) continue;
    }
    const uint16_t* src = ((sv & 1) ? p.L.v_ring : p.L.k_ring) + ((size_t)s * G.ring + slot) * kHeadDim;
    reinterpret_cast<uint4*>(p.saved)[i * 16 + (threadIdx.x & 15)] = reinterpret_cast<const uint4*>(src)[threadIdx.x & 15];
  }
}

// Exclusive prefix sum over the CTA's threads; *total is the sum.
__device__ __forceinline__ int block_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[w] = x;
  __syncthreads();
  if (w == 0) {
    int t = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    sh[lane] = t;
  }
  __syncthreads();
  *total = sh[31];
  return x - v + (w ? sh[w - 1] : 0);
}
// One CTA per stream: the E-th smallest key by its bytes from the highest (each
// step counts the keys that share the bytes so far by their next one; three or
// four steps part unequal sums, where bits took some forty), ties to the lower
// slot; the lists of freed slots and of groups that fill them; the record.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int sh[32], hist[256], found[2];
  const Geometry& G = p.geo;
  const int s = blockIdx.x, b = s / G.Hkv, tid = threadIdx.x, lane = tid & 31;
  const int T = p.tokens[b], ng = group_count(p, T), E = p.evict[b], left = ng - E;
  grid_dep_wait();
  grid_dep_trigger();
  const unsigned long long* keys = p.keys + (size_t)s * p.cap;
  int* hole = p.hole + (size_t)s * p.cap;
  int* mover = p.mover + (size_t)s * p.cap;
  int* source = p.source ? p.source + (size_t)s * p.cap : nullptr;
  int nmoves = 0;
  // each thread's contiguous groups; up to kOwn of them stay in registers over
  // the counting (from L2 each of up to 64 counts would wait a round trip)
  const int per = (ng + kSelThreads - 1) / kSelThreads, j0 = min(ng, tid * per), j1 = min(ng, j0 + per);
  unsigned long long own[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) own[i] = j0 + i < j1 && E > 0 ? keys[j0 + i] : ~0ull;
  if (E > 0) {
    unsigned long long bound = ~0ull;
    int below = 0;  // keys < bound
    if (E < ng) {
      unsigned long long lo = 0;  // at most E keys are below it
      for (int shift = 56; shift >= 0 && below < E; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        auto count = [&](bool have, unsigned long long k) {  // whole warps; one add per value in a warp
          have = have && (shift == 56 || k >> (shift + 8) == lo >> (shift + 8));
          const int d = have ? (int)(k >> shift) & 255 : 256;
          const unsigned same = __match_any_sync(0xffffffffu, d);
          if (have && lane == __ffs(same) - 1) atomicAdd(&hist[d], __popc(same));
        };
#pragma unroll
        for (int i = 0; i < kOwn; ++i) count(j0 + i < j1, own[i]);
        for (int i = kOwn; i < per; ++i) count(j0 + i < j1, j0 + i < j1 ? keys[j0 + i] : 0);
        __syncthreads();
        if (tid < 32) {  // the last byte with at most E keys below it: 8 a lane
          int n[8], sum = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) n[i] = hist[8 * lane + i], sum += n[i];
          int c = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) c += y;
          }
          c += below - sum;
          int d = -1, at = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (c <= E) d = 8 * lane + i, at = c;
            c += n[i];
          }
          const int last = __reduce_max_sync(0xffffffffu, d);
          if (d == last) found[0] = d, found[1] = at;
        }
        __syncthreads();
        lo |= (unsigned long long)found[0] << shift;
        below = found[1];
      }
      bound = lo;  // with fewer than E keys below it, keys equal to it fill up the rest, by slot
    } else {
      below = -1;  // all of them
    }
    int eq = 0, total;
    for (int j = j0; j < j1; ++j) eq += keys[j] == bound;
    const int rest = E - below;
    int rank = block_scan(eq, sh, &total), nh = 0, nm = 0;
    for (int pass = 0; pass < 2; ++pass) {
      int r = rank, hk = nh, mk = nm;
      for (int j = j0; j < j1; ++j) {
        const unsigned long long k = keys[j];
        const bool gone = below < 0 || k < bound || (k == bound && r < rest);
        r += k == bound;
        if (gone && j < left) {
          if (pass) hole[hk] = j;
          ++hk;
        }
        if (!gone && j >= left) {
          if (pass) mover[mk] = j;
          ++mk;
        }
      }
      if (pass == 0) {
        nh = block_scan(hk, sh, &nmoves);
        nm = block_scan(mk, sh, &total);
      }
    }
    __syncthreads();
  }
  if (tid == 0) p.moves[s] = nmoves;
  if (source) {
    for (int j = tid; j < left; j += kSelThreads) source[j] = j;
    __syncthreads();
    for (int k = tid; k < nmoves; k += kSelThreads) source[hole[k]] = mover[k];
  }
  // the record: sinks and groups that stay, groups that move, the window,
  // zeros behind it.  In place every step reads behind what it writes.
  const float* in = p.mass + (size_t)s * p.max_tokens;
  float* out = p.mass_out + (size_t)s * p.max_tokens;
  const int first = min(p.S, T) + (ng > 0 ? kGroupTokens * left : 0);
  if (in != out)
    for (int t0 = 0; t0 < first; t0 += 8 * kSelThreads) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = t0 + i * kSelThreads + tid < first ? in[t0 + i * kSelThreads + tid] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t0 + i * kSelThreads + tid < first) out[t0 + i * kSelThreads + tid] = v[i];
    }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < nmoves * kGroupTokens; i += kSelThreads)
    out[p.S + hole[i >> 5] * kGroupTokens + (i & 31)] = in[p.S + mover[i >> 5] * kGroupTokens + (i & 31)];
  const int shift = kGroupTokens * E;
  for (int t0 = first; t0 < T - shift; t0 += kSelThreads) {
    const int t = t0 + tid;
    float v = 0.0f;
    __syncthreads();
    if (t < T - shift) v = in[t + shift];
    __syncthreads();
    if (t < T - shift) out[t] = v;
  }
  __syncthreads();
  for (int t = T - shift + tid; t < T; t += kSelThreads) out[t] = 0.0f;
}

// bytes from src to dst (apart from each other), 8 chunks of 16 per lane in flight.
__device__ __noinline__ void copy_bytes(uint8_t* __restrict__ dst, const uint8_t* __restrict__ src, int bytes, int lane) {
  for (int i = 16 * lane; i < bytes; i += 8 * 512) {
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + 512 * u < bytes) v[u] = *reinterpret_cast<const uint4*>(src + i + 512 * u);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + 512 * u < bytes) *reinterpret_cast<uint4*>(dst + i + 512 * u) = v[u];
  }
}

// The moves, one warp per group; window rows from the workspace.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p, int groups, int window) {
  const Geometry& G = p.geo;
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const long long warp = (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const long long warps = (long long)gridDim.x * (kMoveThreads / 32);
  if (groups) {
    for (long long i = warp; i < (long long)G.NS * p.most; i += warps) {
      const int s = (int)(i / p.most), k = (int)(i - (long long)s * p.most);
      if (k >= p.moves[s]) continue;
      const size_t to = p.hole[(size_t)s * p.cap + k], from = p.mover[(size_t)s * p.cap + k];
      if (G.fp16_mode) {
        const size_t base = ((size_t)s * G.ring + p.S) * 256;
        uint8_t *kr = reinterpret_cast<uint8_t*>(p.L.k_ring) + base, *vr = reinterpret_cast<uint8_t*>(p.L.v_ring) + base;
        constexpr int kBytes = kGroupTokens * kHeadDim * 2;
        copy_bytes(kr + to * kBytes, kr + from * kBytes, kBytes, lane);
        copy_bytes(vr + to * kBytes, vr + from * kBytes, kBytes, lane);
        continue;
      }
      const size_t row = (size_t)s * G.gcap;  // groups before this stream's
      auto move = [&](void* region, int bytes) {  // bytes of one group
        uint8_t* r = static_cast<uint8_t*>(region);
        copy_bytes(r + (row + to) * bytes, r + (row + from) * bytes, bytes, lane);
      };
      const bool nuq = G.kb == 3;
      move(p.L.k_codes, kGroupTokens * G.krow);
      move(p.L.k_scales, nuq ? kGroupTokens * 4 : G.gkc ? kGroupTokens * G.nkg * 4 : kHeadDim * 4);
      move(p.L.v_codes, kGroupTokens * G.vrow);
      move(p.L.v_scales, nuq ? kGroupTokens * 4 : kGroupTokens * G.nvg * 4);
      if (nuq && G.nout) {  // every row holds nout outliers: the row pointers stay
        move(p.L.k_col, kGroupTokens * G.nout);
        move(p.L.k_val, kGroupTokens * G.nout * 2);
        move(p.L.v_col, kGroupTokens * G.nout);
        move(p.L.v_val, kGroupTokens * G.nout * 2);
      }
    }
  }
  if (window) {
    const long long rows = (long long)G.NS * p.save_rows * 2;
    for (long long i = 2 * warp + (lane >> 4); i < rows; i += 2 * warps) {
      const int row = (int)(i % p.save_rows);
      const long long sv = i / p.save_rows;
      const int s = (int)(sv >> 1), b = s / G.Hkv;
      if (p.evict[b] == 0) continue;
      int slot;
      if (G.fp16_mode) {
        const int from = p.S + kGroupTokens * group_count(p, p.tokens[b]) + row;
        if (from >= p.tokens[b]) continue;
        slot = from - kGroupTokens * p.evict[b];
      } else {  // ring slot r takes slot (r + 32 E) mod ring
        const int shift = (int)((long long)kGroupTokens * p.evict[b] % G.ring);
        slot = row - shift < 0 ? row - shift + G.ring : row - shift;
      }
      uint16_t* dst = ((sv & 1) ? p.L.v_ring : p.L.k_ring) + ((size_t)s * G.ring + slot) * kHeadDim;
      reinterpret_cast<uint4*>(dst)[lane & 15] = reinterpret_cast<const uint4*>(p.saved)[i * 16 + (lane & 15)];
    }
  }
}

}  // namespace

cudaError_t launch_evict(EvictParams& p, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int per = kSumThreads / 4;
  p.sum_blocks = p.most ? p.geo.NS * ((p.cap + per - 1) / per) : 0;
  p.save_blocks = p.most && p.save_rows ? 8 * sms : 0;
  if (p.most) {
    evict_sum_kernel<<<p.sum_blocks + p.save_blocks, kSumThreads, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  e = launch_dependent(evict_select_kernel, dim3(p.geo.NS), dim3(kSelThreads), 0, st, p);
  if (e != cudaSuccess || !p.most) return e;
  const bool apart = p.geo.fp16_mode;
  e = launch_dependent(evict_move_kernel, dim3(8 * sms), dim3(kMoveThreads), 0, st, p, 1, apart ? 0 : 1);
  if (e == cudaSuccess && apart && p.save_rows)
    e = launch_dependent(evict_move_kernel, dim3(8 * sms), dim3(kMoveThreads), 0, st, p, 0, 1);
  return e;
}

}  // namespace kvq
