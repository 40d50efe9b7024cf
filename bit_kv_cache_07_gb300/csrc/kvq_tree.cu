// kvq_tree.cu -- attention of a tree of drafted tokens over the cache and over
// the drafted tokens themselves (speculative decoding's verification).
//
// For query row r = (query head j of the KV head's group, node i):
//   z_rt = scale * q_r . k_t over the T cached tokens and the drafted tokens
//          that node i sees (bit t of its mask words),
//   out_r = sum_t exp(z_rt - m_r) v_t / l_r,  l_r = sum_t exp(z_rt - m_r),
// with the quantized part of the sum rotated back once when V is stored
// Hadamard-rotated.  A row that sees nothing gives 0 and lse = -inf.
#include "kvq_pipe.cuh"

namespace kvq {
namespace {

constexpr int kSmallRows = 16;
constexpr int kConsumerWarps = kTile / 16;
constexpr int kConsumers = 32 * kConsumerWarps;
constexpr int kThreadsSmall = kConsumers + kProducers + 32;
constexpr uint32_t kFixedSmall = 2 * kStageBytes + kSmallRows * kHeadDim * 2 + 2 * kGroupRowBytes + kTailBytes;
constexpr uint32_t kSmemSmall = 227 * 1024;

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Up to 16 query rows per KV head: a 128-row tensor-core tile would be mostly
// padding, and the dequantization of a tile costs more than its products.
// The same producers fill the tiles; 6 warps take 16 keys of each with
// mma.sync (m16n8k16), every warp with its own softmax state and partial
// result.
//
// Measured with the merge, 32 KV heads: 8 x 4k tokens KV4 and 16 nodes 175 us
// (1.0 TB/s); 64k tokens of 3-bit codes with 2 outliers a vector and RoPE, 8
// nodes 508 us (0.48 TB/s).  Bound by the producers: some 4,000 cycles a tile
// of uniform codes, 6,900 of non-uniform rotated ones, at an issue slot in two.
// Sent through the tensor-core kernel instead, the two took 173 and 702 us where
// this one took 171 and 695, and 4 nodes over 1k tokens 19 against 18: the
// producers are the same, but fewer rows are padding here.  A second team of
// producer warps for every other tile: 208 us against 170 for the first (their
// registers are taken from the consumers).
__device__ __forceinline__ void consume(const TreeParams& p, const Bars& B, const uint8_t* sQ, const uint8_t* stage0, const uint8_t* sM,
                                        Tail* tail, int x, int x_end, int tid, volatile int* gave_up) {
  auto wait = [&](uint32_t bar, int phase) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, gave_up)); };
  const int lane = tid & 31, w = tid >> 5, g = lane >> 2, tq = lane & 3;
  const uint32_t aQ = (uint32_t)__cvta_generic_to_shared(sQ), a0 = (uint32_t)__cvta_generic_to_shared(stage0),
                 aM = (uint32_t)__cvta_generic_to_shared(sM);
  int i = 0;
  for (int piece = 0; x < x_end; ++piece) {
    const Piece c = piece_at(p, x, x_end);
    const bool two = c.quant || p.geo.pre_rope, grouped = channel_scales(p.geo) && c.quant;
    const uint32_t* mask_row[2] = {nullptr, nullptr};
    if (p.mask && !c.quant)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (g + 8 * e < c.nr) mask_row[e] = p.mask + ((size_t)c.b * p.n + (g + 8 * e) % c.n_b) * p.words;
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
#pragma unroll 1
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      const uint32_t aK = a0 + st * kStageBytes, aN = aK + kTileBytes, aV = aN + kTileBytes;
      if (!wait(B.full_k + 8 * st, i >> 1)) return;
      // logits of keys 16 w + 8 n + 2 tq + {0, 1}, rows g and g + 8
      float z[2][4] = {}, zn[2][4] = {}, zg[4] = {};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t off = tile_off(16 * w + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1));
        uint32_t qa[4], kb[4];
        ldsm4(qa, aQ + q_off<kSmallRows>(lane & 15, 2 * ks + (lane >> 4)));
        ldsm4(kb, aK + off);
        mma16816(z[0], qa, kb[0], kb[1]);
        mma16816(z[1], qa, kb[2], kb[3]);
        if (two) {
          ldsm4(kb, aN + off);
          mma16816(zn[0], qa, kb[0], kb[1]);
          mma16816(zn[1], qa, kb[2], kb[3]);
        }
        if (grouped) {
          ldsm4(kb, aM + st * kGroupRowBytes + q_off<8>(lane & 7, 2 * ks + ((lane >> 3) & 1)));
          mma16816(zg, qa, kb[0], kb[1]);
        }
      }
      float base[2];  // rows g, g + 8: what the group of the warp's 16 keys shares
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // column n (min of group n), 4 + n (its scale): lane 4 g + n / 2, element n & 1
        const float a = (w >> 1) & 1 ? zg[2 * e + 1] : zg[2 * e];
        const float mn = __shfl_sync(0xffffffffu, a, (lane & ~3) + (w >> 2)), sc = __shfl_sync(0xffffffffu, a, (lane & ~3) + 2 + (w >> 2));
        base[e] = grouped ? fmaf((float)(1 << (p.geo.kb - 1)), sc, mn) : 0.0f;
      }
      mbar_arrive_warp(B.empty_k + 8 * st);
      const int f0 = (c.k0 + t) * kTile + 32 * (w >> 1);
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t ok = seen(p, c, mask_row[e], f0) >> (16 * (w & 1));
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float& y = z[n][2 * e + q];
            y = (ok >> (8 * n + 2 * tq + q)) & 1 ? (y - zn[n][2 * e + q] + base[e]) * p.q_scale : -INFINITY;
            mx[e] = fmaxf(mx[e], y);
          }
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      }
      // the reference lies 12 octaves below the maximum it was taken from and moves when a logit passes it by 15:
      // weights stay in fp16's range, down to 2^-37 of the largest (kvq_tree_tc.cu), and O is rarely rescaled
      const bool move[2] = {mx[0] > m[0] + 15.0f, mx[1] > m[1] + 15.0f};
      if (__any_sync(0xffffffffu, move[0] || move[1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float to = mx[e] - 12.0f, al = move[e] ? ex2(m[e] - to) : 1.0f;
          if (move[e]) m[e] = to;
          l[e] *= al;
#pragma unroll
          for (int n = 0; n < 16; ++n) o[n][2 * e] *= al, o[n][2 * e + 1] *= al;
        }
      }
      const float mu[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[n][e] = ex2(z[n][e] - mu[e >> 1]);
          l[e >> 1] += z[n][e];
        }
      if (!wait(B.full_v + 8 * st, i >> 1)) return;
      // O += P V with P in two fp16 parts (22 bits): the products are few, and V's
      // own rounding stays the only one before the output's
      uint32_t pa[4], pn[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(z[e >> 1][2 * (e & 1)], z[e >> 1][2 * (e & 1) + 1], &pa[e], &pn[e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) pn[e] ^= 0x80008000u;
#pragma unroll
      for (int n = 0; n < 16; n += 2) {
        uint32_t vb[4];
        ldsm4t(vb, aV + tile_off(16 * w + (lane & 15), n + (lane >> 4)));
        mma16816(o[n], pa, vb[0], vb[1]);
        mma16816(o[n + 1], pa, vb[2], vb[3]);
        mma16816(o[n], pn, vb[0], vb[1]);
        mma16816(o[n + 1], pn, vb[2], vb[3]);
      }
      mbar_arrive_warp(B.empty_v + 8 * st);
    }
    // the piece's partial result; this thread holds slots 8 n + 2 tq + {0, 1} of the values' channel order
    const bool paired = c.quant && p.geo.vb != 3 && paired_order(p.geo.vb);
    if (tid == 0 && !c.quant) {
      const uint32_t bad = *(volatile int*)&tail->bad_piece[piece & 3] == piece + 1;
      for (int e = 0; e < p.sub; ++e) p.part_flag[(size_t)c.slot * p.sub + e] = bad;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      const int r = g + 8 * e;
      if (r < c.nr) {
        const size_t at = ((size_t)c.slot * p.sub + w) * p.rstride + r;
        if (tq == 0) p.part_ml[at] = make_float2(m[e], l[e]);
        float* acc = p.part_acc + at * kHeadDim;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          if (paired) acc[8 * n + tq] = o[n][2 * e], acc[8 * n + tq + 4] = o[n][2 * e + 1];
          else *reinterpret_cast<float2*>(acc + 8 * n + 2 * tq) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
        }
      }
    }
    x += c.cnt;
  }
}

// FP16: the unquantized cache, without the quantized tiles' code (8 x 16k tokens, 8
// KV heads, 16 rows each: 193 us, 2.8 TB/s; with it 230).
template <bool FP16>
__global__ void __launch_bounds__(kThreadsSmall, 1) tree_small_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *stage0 = smem, *sQ = stage0 + 2 * kStageBytes, *sM = sQ + kSmallRows * kHeadDim * 2;
  Tail* tail = reinterpret_cast<Tail*>(sM + 2 * kGroupRowBytes);
  uint8_t* raw0 = sM + 2 * kGroupRowBytes + kTailBytes;
  volatile int* gave_up = &tail->gave_up;
  grid_dep_trigger();  // the merge may be launched; it waits for this grid's end
  const int tid = threadIdx.x;
  const Bars B = bars_at((uint32_t)__cvta_generic_to_shared(tail->bars));
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.full_k + 8 * i, kProducers / 32);
      mbar_init(B.full_v + 8 * i, kProducers / 32);
      mbar_init(B.empty_k + 8 * i, kConsumerWarps);
      mbar_init(B.empty_v + 8 * i, kConsumerWarps);
    }
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(B.raw_full + 8 * i, 1);
      mbar_init(B.raw_empty + 8 * i, kProducers / 32);
    }
    *gave_up = 0;
    for (int i = 0; i < 4; ++i) tail->bad_piece[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  put_tables<true>(p, tail, raw0, tid);
  __syncthreads();
  const int x = cta_first_tile(p.ncta, p.total, blockIdx.x), x_end = cta_first_tile(p.ncta, p.total, blockIdx.x + 1);
  if (tid < kConsumers) {
    consume(p, B, sQ, stage0, sM, tail, x, x_end, tid, gave_up);
  } else if (tid < kConsumers + kProducers) {
    produce<kSmallRows, true, FP16>(p, B, sQ, stage0, sM, raw0, tail, x, x_end, tid - kConsumers, gave_up);
  } else {
    if ((tid & 31) == 0) load_tiles<true>(p, B, (uint32_t)__cvta_generic_to_shared(raw0), x, x_end, gave_up);
    __syncwarp();
  }
  __syncthreads();
  if (*gave_up) {  // a wait ran out: every row of the range becomes NaN
    for (int y = x; y < x_end;) {
      const Piece c = piece_at(p, y, x_end);
      for (int r = tid; r < c.nr * p.sub; r += kThreadsSmall)
        p.part_ml[((size_t)c.slot * p.sub + r / c.nr) * p.rstride + r % c.nr] = make_float2(NAN, NAN);
      y += c.cnt;
    }
  }
}

// Join the pieces of each row: one CTA per row.  The partial maxima and sums
// first, one per thread, and from them every partial result's weight; then
// 4 warps add the weighted partial results (lane l owns channels 4 l .. 4 l +
// 3), all loads independent.  Quantized and fp16 pieces are summed apart, the
// quantized sum rotated back once.  Bound by reading the partial results, which
// are in L2: 19 to 23 us of 8 x 32 KV heads x 16 rows (6 partial results a piece)
// and of 8 x 8 x 128, timed alone on a cold L2.
constexpr int kMergeThreads = 128;
constexpr int kMaxParts = kMaxSpecCtas * kConsumerWarps;  // of one kind of a row
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  const Geometry& G = p.geo;
  const int b = blockIdx.z, h = blockIdx.y, n_b = p.rows.nodes[b], r = blockIdx.x;
  if (r >= G.g * n_b) return;
  const int j = r / n_b, node = r - j * n_b, rb = r / p.rblk, rr = r - rb * p.rblk;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int nrb = (G.g * n_b + p.rblk - 1) / p.rblk, pair = h * nrb + rb;
  const TileCounts tc = tile_counts(G, p.rows.tokens[b], p.mask ? n_b : 0);
  __shared__ float sW[2 * kMaxParts];
  __shared__ float sM[4], sL[4];
  __shared__ __align__(16) float sAcc[4][2][kHeadDim];
  __shared__ uint32_t sFlag;
  if (tid == 0) sFlag = 0;
  const PartSpan span[2] = {part_span(p, tc, b, pair, 0), part_span(p, tc, b, pair, 1)};
  const size_t at0[2] = {span[0].at, span[1].at};
  const int np[2] = {span[0].n, span[1].n};
  grid_dep_wait();
  __syncthreads();
  const int all = np[0] + np[1];
  auto index = [&](int i) { return i < np[0] ? at0[0] + i : at0[1] + (i - np[0]); };
  float M = -INFINITY;
  bool bad = false;  // not a number somewhere: the row becomes that
  for (int i = tid; i < all; i += kMergeThreads) {
    const size_t sl = index(i);
    const float2 ml = p.part_ml[sl * p.rstride + rr];
    if (i >= np[0] && names_drafted(p, ml, p.part_flag[sl])) sFlag = 1;
    M = fmaxf(M, ml.x);
    bad = bad || ml.x != ml.x || ml.y != ml.y;
  }
  M = warp_max(M);
  if (lane == 0) sM[w] = M;
  bad = __syncthreads_or(bad);
  M = fmaxf(fmaxf(sM[0], sM[1]), fmaxf(sM[2], sM[3]));
  float L = 0.0f;
  for (int i = tid; i < all; i += kMergeThreads) {
    const float2 ml = p.part_ml[index(i) * p.rstride + rr];
    const float wt = ml.x == -INFINITY ? 0.0f : ex2(ml.x - M);
    sW[i] = wt;
    L += wt * ml.y;
  }
  L = warp_sum(L);
  if (lane == 0) sL[w] = L;
  __syncthreads();
  L = bad ? NAN : sL[0] + sL[1] + sL[2] + sL[3];
  float4 a[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const float* acc = p.part_acc + (at0[kind] * p.rstride + rr) * kHeadDim + 4 * lane;
    const float* wt = sW + (kind ? np[0] : 0);
#pragma unroll 4
    for (int i = w; i < np[kind]; i += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(acc + (size_t)i * p.rstride * kHeadDim));
      const float c = wt[i];
      if (c != 0.0f) a[kind].x += v.x * c, a[kind].y += v.y * c, a[kind].z += v.z * c, a[kind].w += v.w * c;
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) *reinterpret_cast<float4*>(&sAcc[w][q][4 * lane]) = a[q];
  __syncthreads();
  if (w) return;
  float x[2][4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[q][e] += sAcc[i][q][4 * lane + e];
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

template <bool FP16>
cudaError_t launch_small(TreeParams& p, cudaStream_t st) {
  p.raw = raw_slot(p.geo, true, kSmemSmall - kFixedSmall);
  if (kFixedSmall + raw_bytes(p.geo, p.raw, true) > kSmemSmall) return cudaErrorInvalidValue;
  static std::atomic<long long> memo[kMemoDevices];
  const cudaError_t e = ensure_smem_limit(tree_small_kernel<FP16>, memo, (int)kSmemSmall);
  if (e != cudaSuccess) return e;
  tree_small_kernel<FP16><<<p.ncta, kThreadsSmall, kSmemSmall, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attn(TreeParams& p, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.total > 0) e = p.rblk != kSmallRows ? launch_tree_tc(p, st) : p.geo.fp16_mode ? launch_small<true>(p, st) : launch_small<false>(p, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(tree_merge_kernel, dim3(p.geo.g * p.n, p.geo.Hkv, p.geo.B), dim3(128), 0, st, p);
}

}  // namespace kvq
