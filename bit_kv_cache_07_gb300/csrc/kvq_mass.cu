// kvq_mass.cu -- accumulated attention weight of every cached token (the
// record that kvq_evict goes by).
//
// For token t of stream (b, h), over the query rows r = (query head j of the
// KV head's group, row i) that attended it:
//   mass_t <- decay * mass_t + sum_r w_i exp(scale * q_r . k_t - lse_r)
// with the log-sum-exp that the attention returned: the rows' softmax is not
// computed again, one pass over the keys is enough.
#include "kvq_tree.cuh"

namespace kvq {
namespace {

constexpr int kMassThreads = 256;
constexpr int kMassRows = 64;  // query rows in shared memory at a time
constexpr uint32_t kTileBytes = kTile * kHeadDim * 2;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Keys of tile kt into shared memory as hi + lo fp16 parts (as the tree
// attention's tiles).
__device__ __forceinline__ void fill_keys(const MassParams& p, const TileCounts& tc, int s, bool quant, int kt, uint8_t* sK,
                                          uint8_t* sKlo, int tid) {
  const Geometry& G = p.geo;
  const int cb = tid & 7;
  for (int u = 0; u < 4; ++u) {
    const int t = (tid >> 3) * 4 + u, f = kt * kTile + t;
    float x[2][8];
    const bool have = f < (quant ? tc.Nq : tc.k1);
    int pos = 0;
    if (have) {
      if (quant) {
        pos = G.S + f;
#pragma unroll
        for (int h = 0; h < 2; ++h) k_chunk(G, p.L, p.k_lut_off, s, f, cb + 8 * h, x[h]);
      } else {
        const uint16_t* kr = fp16_row(G, p.L.k_sink, p.L.k_ring, s, tc, f, &pos);
#pragma unroll
        for (int h = 0; h < 2; ++h) unpack8(*reinterpret_cast<const uint4*>(kr + 8 * cb + 64 * h), x[h]);
      }
      if (G.pre_rope) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 e = spec_expi(((double)G.pos_offset + pos) * p.theta[8 * cb + i]);
          const float a = x[0][i], c = x[1][i];
          x[0][i] = a * e.x - c * e.y;
          x[1][i] = c * e.x + a * e.y;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
      if (have) split8(x[h], &hi, &lo);
      const uint32_t o = tile_off(t, cb + 8 * h);
      *reinterpret_cast<uint4*>(sK + o) = hi;
      *reinterpret_cast<uint4*>(sKlo + o) = lo;
    }
  }
}

// One CTA per tile of 128 keys at a time; warp w owns 16 keys of the tile
// (the mma's rows), the query rows pass as its columns, 64 at a time.
__global__ void __launch_bounds__(kMassThreads, 1) mass_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sK = smem, *sKlo = smem + kTileBytes, *sQ = smem + 2 * kTileBytes;
  float2* sW = reinterpret_cast<float2*>(sQ + kMassRows * kHeadDim * 2);  // (lse, weight) of the rows
  const Geometry& G = p.geo;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, tq = lane & 3;
  const uint32_t aK = (uint32_t)__cvta_generic_to_shared(sK), aKlo = (uint32_t)__cvta_generic_to_shared(sKlo),
                 aQ = (uint32_t)__cvta_generic_to_shared(sQ);
  const int M = G.g * p.n;
  const int x_end = cta_first_tile(p.ncta, p.total, blockIdx.x + 1);
  for (int x = cta_first_tile(p.ncta, p.total, blockIdx.x); x < x_end; ++x) {
    const int b = row_of(p.rows.tile0, G.B, x);
    const int T = p.rows.tokens[b];
    const TileCounts tc = tile_counts(G, T, 0);
    const int per = tc.qt + tc.ft, off = x - p.rows.tile0[b], h = off / per, k = off - h * per, s = b * G.Hkv + h;
    const bool quant = k < tc.qt;
    const int kt = quant ? k : k - tc.qt;
    __syncthreads();  // the previous tile's keys are used
    fill_keys(p, tc, s, quant, kt, sK, sKlo, tid);
    float sum[2] = {0.0f, 0.0f};  // keys 16 w + g, + 8
    const size_t head0 = (size_t)b * G.Hq_tot + (size_t)layer_head(G, h) * G.g;
    for (int r0 = 0; r0 < M; r0 += kMassRows) {
      const int nr = min(kMassRows, M - r0);
      __syncthreads();  // the previous rows are used; on the first pass, the keys are written
      for (int i = tid; i < kMassRows * 16; i += kMassThreads) {
        const int r = i >> 4, ch = i & 15;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < nr) v = *reinterpret_cast<const uint4*>(p.q + (head0 * p.n + r0 + r) * kHeadDim + 8 * ch);
        *reinterpret_cast<uint4*>(sQ + r * 256 + ((ch ^ (r & 7)) << 4)) = v;
      }
      if (tid < kMassRows) {
        float2 lw = make_float2(0.0f, 0.0f);
        if (tid < nr) {
          lw.x = p.lse[head0 * p.n + r0 + tid];
          lw.y = p.weight ? p.weight[(size_t)b * p.n + (r0 + tid) % p.n] : 1.0f;
        }
        if (lw.x == -INFINITY) lw = make_float2(0.0f, 0.0f);  // a row that saw nothing
        sW[tid] = lw;
      }
      __syncthreads();
      for (int n0 = 0; n0 < nr; n0 += 16) {
        float z[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t ka[4], kl[4], qb[4];
          const uint32_t off_k = tile_off(16 * w + (lane & 15), 2 * ks + (lane >> 4));
          ldsm4(ka, aK + off_k);
          ldsm4(kl, aKlo + off_k);
          const int r = n0 + (lane & 7) + ((lane >> 4) << 3), ch = 2 * ks + ((lane >> 3) & 1);
          ldsm4(qb, aQ + r * 256 + ((ch ^ (r & 7)) << 4));
          mma16816(z[0], ka, qb[0], qb[1]);
          mma16816(z[1], ka, qb[2], qb[3]);
          mma16816(z[0], kl, qb[0], qb[1]);
          mma16816(z[1], kl, qb[2], qb[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 lw = sW[n0 + 8 * i + 2 * tq + (e & 1)];
            if (lw.y != 0.0f) sum[e >> 1] += lw.y * ex2(fmaf(z[i][e], p.q_scale, -lw.x) * 1.4426950408889634f);
          }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      const int f = kt * kTile + 16 * w + g + 8 * e;
      if (tq == 0 && f < (quant ? tc.Nq : tc.k1)) {
        const int t = quant ? G.S + f : f < tc.S_eff ? f : G.S + tc.Nq + (f - tc.S_eff);
        float* m = p.mass + (size_t)s * p.cap + t;
        *m = fmaf(p.decay, *m, sum[e]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_attn_mass(const MassParams& p, cudaStream_t st) {
  static std::atomic<long long> memo[kMemoDevices];
  const int smem = (int)(2 * kTileBytes) + kMassRows * (kHeadDim * 2 + 8);
  cudaError_t e = ensure_smem_limit(mass_kernel, memo, smem);
  if (e != cudaSuccess) return e;
  mass_kernel<<<p.ncta, kMassThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace kvq
