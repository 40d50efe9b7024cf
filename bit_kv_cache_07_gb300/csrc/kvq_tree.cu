// kvq_tree.cu -- attention of a tree of drafted tokens over the cache and over
// the drafted tokens themselves (speculative decoding's verification).
//
// For query row r = (query head j of the KV head's group, node i):
//   z_rt = scale * q_r . k_t over the T cached tokens and the drafted tokens
//          that node i sees (bit t of its mask words),
//   out_r = sum_t exp(z_rt - m_r) v_t / l_r,  l_r = sum_t exp(z_rt - m_r),
// with the quantized part of the sum rotated back once when V is stored
// Hadamard-rotated.  A row that sees nothing gives 0 and lse = -inf.
#include "kvq_tree.cuh"

namespace kvq {
namespace {

constexpr int kTreeThreads = 256;
constexpr uint32_t kTileBytes = kTile * kHeadDim * 2;  // 32 KB

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
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Tile kt of one kind of stream s (batch row b) into shared memory: K as
// hi + lo fp16 parts, V as fp16.  Thread (tid >> 3) takes 4 consecutive keys,
// tid & 7 the channels [8 cb, 8 cb + 8) and the same of the second half (a
// RoPE pair's two channels).  Keys past the end become zeros.
__device__ __forceinline__ void fill_tile(const TreeParams& p, const TileCounts& tc, int s, int b, bool quant, int kt, int n_b,
                                          uint8_t* sK, uint8_t* sKlo, uint8_t* sV, uint32_t* flag, int tid) {
  const Geometry& G = p.geo;
  const int cb = tid & 7;
  for (int u = 0; u < 4; ++u) {
    const int t = (tid >> 3) * 4 + u, f = kt * kTile + t;
    float x[2][8], y[2][8];
    uint4 vraw[2];
    bool have = false, direct = false;
    int pos = 0;
    if (quant) {
      if (f < tc.Nq) {
        have = true;
        pos = G.S + f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          k_chunk(G, p.L, p.k_lut_off, s, f, cb + 8 * h, x[h]);
          v_chunk(G, p.L, p.v_lut_off, s, f, cb + 8 * h, y[h]);
        }
      }
    } else if (f < tc.k1 + n_b) {
      have = direct = true;
      const uint16_t *kr, *vr;
      if (f < tc.k1) {
        kr = fp16_row(G, p.L.k_sink, p.L.k_ring, s, tc, f, &pos);
        vr = fp16_row(G, p.L.v_sink, p.L.v_ring, s, tc, f, &pos);
      } else {
        const size_t row = in_stream(G, s) * p.n + (f - tc.k1);
        kr = p.kd + row * kHeadDim;
        vr = p.vd + row * kHeadDim;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unpack8(*reinterpret_cast<const uint4*>(kr + 8 * cb + 64 * h), x[h]);
        vraw[h] = *reinterpret_cast<const uint4*>(vr + 8 * cb + 64 * h);
        if (f >= tc.k1 && !finite8(vraw[h])) {
          // a drafted value that some rows must not see: it enters as zero
          // here and the merge adds it to the rows that do
          *flag = 1;
          unpack8(vraw[h], y[h]);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[h][i] = isfinite(y[h][i]) ? y[h][i] : 0.0f;
          vraw[h] = pack8(y[h]);
        }
      }
    }
    if (have && G.pre_rope && f < (quant ? tc.Nq : tc.k1)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 e = spec_expi(((double)G.pos_offset + pos) * p.theta[8 * cb + i]);
        const float a = x[0][i], c = x[1][i];
        x[0][i] = a * e.x - c * e.y;
        x[1][i] = c * e.x + a * e.y;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 hi = make_uint4(0, 0, 0, 0), lo = hi, v = hi;
      if (have) {
        split8(x[h], &hi, &lo);
        if (direct) {
          v = vraw[h];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[h][i] = fminf(fmaxf(y[h][i], -65504.0f), 65504.0f);
          v = pack8(y[h]);
        }
      }
      const uint32_t o = tile_off(t, cb + 8 * h);
      *reinterpret_cast<uint4*>(sK + o) = hi;
      *reinterpret_cast<uint4*>(sKlo + o) = lo;
      *reinterpret_cast<uint4*>(sV + o) = v;
    }
  }
}

// One CTA walks its range of tiles.  WR warps along the rows (16 each), WK
// along the keys of a tile; each (row, key) warp keeps its own softmax state
// and writes its own partial result.
template <int WR>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_attn_kernel(const __grid_constant__ TreeParams p) {
  constexpr int WK = 8 / WR, KW = kTile / WK, KC = KW < 32 ? KW : 32;  // keys per warp of a tile, per step
  constexpr int NT = KC / 8;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sK = smem, *sKlo = smem + kTileBytes, *sV = smem + 2 * kTileBytes, *sQ = smem + 3 * kTileBytes;
  uint32_t* sMask = reinterpret_cast<uint32_t*>(sQ + 16 * WR * kHeadDim * 2);  // [16 WR][8]
  __shared__ uint32_t flag;
  const Geometry& G = p.geo;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, wr = w % WR, wk = w / WR;
  const int g = lane >> 2, tq = lane & 3;
  const uint32_t aK = (uint32_t)__cvta_generic_to_shared(sK), aKlo = (uint32_t)__cvta_generic_to_shared(sKlo),
                 aV = (uint32_t)__cvta_generic_to_shared(sV), aQ = (uint32_t)__cvta_generic_to_shared(sQ);
  int x = cta_first_tile(p.ncta, p.total, blockIdx.x);
  const int x_end = cta_first_tile(p.ncta, p.total, blockIdx.x + 1);
  while (x < x_end) {
    // the piece that starts at tile x
    const int b = row_of(p.rows.tile0, G.B, x);
    const int n_b = p.rows.nodes[b], M = G.g * n_b, nrb = (M + p.rblk - 1) / p.rblk;
    const TileCounts tc = tile_counts(G, p.rows.tokens[b], p.mask ? n_b : 0);
    const int per = tc.qt + tc.ft, off = x - p.rows.tile0[b], pair = off / per, k = off - pair * per;
    const int h = pair / nrb, rb = pair - h * nrb, s = b * G.Hkv + h;
    const bool quant = k < tc.qt;
    const int k0 = quant ? k : k - tc.qt, kind_tiles = quant ? tc.qt : tc.ft;
    const int cnt = min(kind_tiles - k0, x_end - x);
    const int slot = blockIdx.x + 2 * (p.rows.pair0[b] + pair) + (quant ? 0 : 1);
    const int r0 = rb * p.rblk, nr = min(p.rblk, M - r0);
    const uint16_t* qb = p.q + ((size_t)b * G.Hq_tot + (size_t)layer_head(G, h) * G.g) * p.n * kHeadDim;
    __syncthreads();  // the previous piece is done with shared memory
    if (tid == 0) flag = 0;
    for (int i = tid; i < 16 * WR * 16; i += kTreeThreads) {
      const int r = i >> 4, ch = i & 15;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < nr) {
        const int j = (r0 + r) / n_b, node = (r0 + r) - j * n_b;
        v = *reinterpret_cast<const uint4*>(qb + ((size_t)j * p.n + node) * kHeadDim + 8 * ch);
      }
      *reinterpret_cast<uint4*>(sQ + r * 256 + ((ch ^ (r & 7)) << 4)) = v;
    }
    if (!quant && p.mask)
      for (int i = tid; i < 16 * WR * p.words; i += kTreeThreads) {
        const int r = i / p.words, wd = i - r * p.words;
        sMask[r * 8 + wd] = r < nr ? p.mask[((size_t)b * p.n + (r0 + r) % n_b) * p.words + wd] : 0;
      }
    __syncthreads();
    uint32_t qa[8][4];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const int r = 16 * wr + (lane & 15), ch = 2 * ks + (lane >> 4);
      ldsm4(qa[ks], aQ + r * 256 + ((ch ^ (r & 7)) << 4));
    }
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

    for (int kt = k0; kt < k0 + cnt; ++kt) {
      __syncthreads();  // every warp is done with the previous tile
      fill_tile(p, tc, s, b, quant, kt, p.mask ? n_b : 0, sK, sKlo, sV, &flag, tid);
      __syncthreads();
#pragma unroll 1
      for (int c0 = wk * KW; c0 < wk * KW + KW; c0 += KC) {
        float z[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
          for (int i = 0; i < NT; i += 2) {
            // keys c0 + 8 i .. + 16, channels 16 ks .. + 16
            const int t = c0 + 8 * i + (lane & 7) + ((lane >> 4) << 3), ch = 2 * ks + ((lane >> 3) & 1);
            const uint32_t off = tile_off(t, ch);
            uint32_t kb[4];
            ldsm4(kb, aK + off);
            mma16816(z[i], qa[ks], kb[0], kb[1]);
            mma16816(z[i + 1], qa[ks], kb[2], kb[3]);
            ldsm4(kb, aKlo + off);
            mma16816(z[i], qa[ks], kb[0], kb[1]);
            mma16816(z[i + 1], qa[ks], kb[2], kb[3]);
          }
        }
        // scale and mask; this thread holds rows g, g + 8 and keys c0 + 8 i + 2 tq + {0, 1}
        const int base = kt * kTile + c0;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int f = base + 8 * i + 2 * tq + (e & 1), r = 16 * wr + g + 8 * (e >> 1);
            bool ok;
            if (quant) {
              ok = f < tc.Nq;
            } else {
              const int d = f - tc.k1;
              ok = d < 0 || (p.mask && d < n_b && ((sMask[r * 8 + (d >> 5)] >> (d & 31)) & 1));
            }
            z[i][e] = ok ? z[i][e] * p.q_scale : -INFINITY;
            mx[e >> 1] = fmaxf(mx[e >> 1], z[i][e]);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          const float mn = fmaxf(m[e], mx[e]);
          const float al = mn == -INFINITY ? 1.0f : ex2(m[e] - mn);
          m[e] = mn;
          l[e] *= al;
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i][2 * e] *= al, o[i][2 * e + 1] *= al;
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            z[i][e] = ex2(z[i][e] - mu[e >> 1]);
            l[e >> 1] += z[i][e];
          }
        // O += P V; P rounds to fp16 (relative 2^-11 of each weight, as the output does)
#pragma unroll
        for (int ks = 0; ks < KC / 16; ++ks) {
          const uint32_t pa[4] = {pack2(z[2 * ks][0], z[2 * ks][1]), pack2(z[2 * ks][2], z[2 * ks][3]),
                                  pack2(z[2 * ks + 1][0], z[2 * ks + 1][1]), pack2(z[2 * ks + 1][2], z[2 * ks + 1][3])};
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int t = c0 + 16 * ks + (lane & 15), ch = i + (lane >> 4);
            uint32_t vb[4];
            ldsm4t(vb, aV + tile_off(t, ch));
            mma16816(o[i], pa, vb[0], vb[1]);
            mma16816(o[i + 1], pa, vb[2], vb[3]);
          }
        }
      }
    }
    // the piece's partial result
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      const int r = 16 * wr + g + 8 * e;
      if (r < nr) {
        const size_t at = ((size_t)slot * p.sub + wk) * p.rstride + r;
        if (tq == 0) p.part_ml[at] = make_float2(m[e], l[e]);
        float* acc = p.part_acc + at * kHeadDim;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          *reinterpret_cast<float2*>(acc + 8 * i + 2 * tq) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
      }
    }
    if (tid < p.sub) p.part_flag[(size_t)slot * p.sub + tid] = flag;
    x += cnt;
  }
}

// Join the pieces of each row: one CTA per row, 4 warps stride over the
// pieces (lane l owns channels 4 l .. 4 l + 3), quantized and fp16 pieces
// summed apart, the quantized sum rotated back once.
__global__ void __launch_bounds__(128) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  const Geometry& G = p.geo;
  const int b = blockIdx.z, h = blockIdx.y, n_b = p.rows.nodes[b], r = blockIdx.x;
  if (r >= G.g * n_b) return;
  const int j = r / n_b, node = r - j * n_b, rb = r / p.rblk, rr = r - rb * p.rblk;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int nrb = (G.g * n_b + p.rblk - 1) / p.rblk, pair = h * nrb + rb;
  const TileCounts tc = tile_counts(G, p.rows.tokens[b], p.mask ? n_b : 0);
  const int t0 = p.rows.tile0[b] + pair * (tc.qt + tc.ft);
  __shared__ float sM[4], sL[4];
  __shared__ __align__(16) float sAcc[4][2][kHeadDim];
  __shared__ uint32_t sFlag;
  if (threadIdx.x == 0) sFlag = 0;
  grid_dep_wait();
  __syncthreads();
  float M = -INFINITY, L = 0.0f;
  float4 a[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int first = kind ? t0 + tc.qt : t0, tiles = kind ? tc.ft : tc.qt;
    if (tiles == 0) continue;
    const int item = 2 * (p.rows.pair0[b] + pair) + kind;
    const int c0 = tile_owner(p.ncta, p.total, first), c1 = tile_owner(p.ncta, p.total, first + tiles - 1);
    const int np = (c1 - c0 + 1) * p.sub;
    for (int i = w; i < np; i += 4) {
      const size_t sl = (size_t)(c0 + item) * p.sub + i, at = sl * p.rstride + rr;
      const float2 ml = p.part_ml[at];
      if (kind && p.part_flag[sl]) sFlag = 1;
      if (ml.x == -INFINITY && ml.y == 0.0f) continue;  // nothing seen
      const float4 v = *reinterpret_cast<const float4*>(p.part_acc + at * kHeadDim + 4 * lane);
      const float mn = fmaxf(M, ml.x), wo = M == -INFINITY ? 0.0f : ex2(M - mn), wn = ml.x == -INFINITY ? 1.0f : ex2(ml.x - mn);
      M = mn;
      L = L * wo + ml.y * wn;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        a[q].x *= wo, a[q].y *= wo, a[q].z *= wo, a[q].w *= wo;
        if (q == kind)
          a[q].x += v.x * wn, a[q].y += v.y * wn, a[q].z += v.z * wn, a[q].w += v.w * wn;
      }
    }
  }
  if (lane == 0) sM[w] = M, sL[w] = L;
#pragma unroll
  for (int q = 0; q < 2; ++q) *reinterpret_cast<float4*>(&sAcc[w][q][4 * lane]) = a[q];
  __syncthreads();
  if (w) return;
  M = fmaxf(fmaxf(sM[0], sM[1]), fmaxf(sM[2], sM[3]));
  L = 0.0f;
  float x[2][4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float wt = sM[i] == -INFINITY ? (sL[i] == 0.0f ? 0.0f : 1.0f) : ex2(sM[i] - M);
    L += sL[i] * wt;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[q][e] += sAcc[i][q][4 * lane + e] * wt;
  }
  if (G.hadamard) {
    // Hn = H / sqrt(d): butterflies of width 1, 2 within the lane, 4 .. 64 across lanes
    float* y = x[0];
    float s0 = y[0] + y[1], s1 = y[0] - y[1], s2 = y[2] + y[3], s3 = y[2] - y[3];
    y[0] = s0 + s2, y[1] = s1 + s3, y[2] = s0 - s2, y[3] = s1 - s3;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float other = __shfl_xor_sync(0xffffffffu, y[e], d);
        y[e] = (lane & d) ? other - y[e] : y[e] + other;
      }
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= p.hadamard_c;
  }
  float res[4];
  const float inv = L != 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) res[e] = (x[0][e] + x[1][e]) * inv;
  if (sFlag) {
    // drafted values that are not finite, for the rows that see them
    const size_t row0 = in_stream(G, b * G.Hkv + h) * p.n;
    for (int i = 0; i < n_b; ++i) {
      if (!((p.mask[((size_t)b * p.n + node) * p.words + (i >> 5)] >> (i & 31)) & 1)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = half_bits_to_float(p.vd[(row0 + i) * kHeadDim + 4 * lane + e]);
        if (!isfinite(v)) res[e] += v;
      }
    }
  }
  const size_t orow = ((size_t)b * G.Hq_tot + (size_t)layer_head(G, h) * G.g + j) * p.n + node;
  *reinterpret_cast<uint2*>(p.out + orow * kHeadDim + 4 * lane) = make_uint2(pack2(res[0], res[1]), pack2(res[2], res[3]));
  if (p.lse && lane == 0) p.lse[orow] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int WR>
cudaError_t launch_t(const TreeParams& p, cudaStream_t st) {
  static std::atomic<long long> memo[kMemoDevices];
  const int smem = (int)(3 * kTileBytes) + 16 * WR * (kHeadDim * 2 + 32);
  cudaError_t e = ensure_smem_limit(tree_attn_kernel<WR>, memo, smem);
  if (e != cudaSuccess) return e;
  tree_attn_kernel<WR><<<p.ncta, kTreeThreads, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attn(const TreeParams& p, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.total > 0) e = p.rblk == 16 ? launch_t<1>(p, st) : launch_tree_tc(p, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(tree_merge_kernel, dim3(p.geo.g * p.n, p.geo.Hkv, p.geo.B), dim3(128), 0, st, p);
}

}  // namespace kvq
