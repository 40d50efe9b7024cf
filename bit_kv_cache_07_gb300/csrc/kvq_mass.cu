// kvq_mass.cu -- accumulated attention weight of every cached token (the
// record that kvq_evict goes by).
//
// For token t of stream (b, h), over the query rows r = (query head j of the
// KV head's group, row i) that attended it:
//   mass_t <- decay * mass_t + sum_r w_i exp(scale * q_r . k_t - lse_r)
// with the log-sum-exp that the attention returned: the rows' softmax is not
// computed again, one pass over the keys is enough.
//
// The tile kernels' copies and producers, for keys alone; 6 warps take 16
// keys of a tile each as the rows of mma.sync (m16n8k16), the query rows pass
// as its columns, 8 at a time, so that a key's weights are summed within a
// quad of lanes.
#include "kvq_pipe.cuh"

namespace kvq {
namespace {

constexpr int kConsumerWarps = kTile / 16;
constexpr int kConsumers = 32 * kConsumerWarps;
constexpr int kThreadsMass = kConsumers + kProducers + 32;
constexpr uint32_t kFixedMass = 2 * kKeyStageBytes + 2 * kGroupRowBytes + kTailBytes;
constexpr uint32_t kSmemMass = 227 * 1024;

// 8 query rows as the mma's columns: this thread's operand words (row g of
// the 8, channels 16 ks + 2 tq, + 1 and + 8, + 9), in the keys' channel order.
__device__ __forceinline__ void load_rows(const uint16_t* q, int left, bool paired, int lane, uint32_t (&b)[8][2]) {
  const int g = lane >> 2, tq = lane & 3;
  const bool have = g < left;
  const uint16_t* row = q + (size_t)g * kHeadDim;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // slots 2 tq, 2 tq + 1 of chunk 2 ks + h: channels 2 tq, 2 tq + 1, or (paired) tq, tq + 4
      const uint16_t* c = row + 8 * (2 * ks + h);
      uint32_t w = 0;
      if (have) w = paired ? (uint32_t)__ldg(c + tq) | (uint32_t)__ldg(c + tq + 4) << 16 : __ldg(reinterpret_cast<const uint32_t*>(c) + tq);
      b[ks][h] = w;
    }
}
// Their log-sum-exps and weights: columns 2 tq, 2 tq + 1.
__device__ __forceinline__ void load_weights(const TreeParams& p, size_t row0, int b, int r0, int M, int tq, float2 (&lw)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + 2 * tq + e;
    lw[e] = make_float2(0.0f, 0.0f);
    if (r < M) {
      const float lse = __ldg(p.row_lse + row0 + r), wt = p.weight ? __ldg(p.weight + (size_t)b * p.n + r % p.n) : 1.0f;
      if (lse != -INFINITY) lw[e] = make_float2(lse, wt);  // (a row that saw nothing)
    }
  }
}

// ONE: at most 8 rows per KV head, whose operand stays in registers.
template <bool ONE>
__device__ __forceinline__ void weigh(const TreeParams& p, const Bars& B, const uint8_t* stage0, const uint8_t* sM, int x, int x_end,
                                      int tid, volatile int* gave_up) {
  auto wait = [&](uint32_t bar, int phase) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, gave_up)); };
  const Geometry& G = p.geo;
  const int lane = tid & 31, w = tid >> 5, g = lane >> 2, tq = lane & 3, M = G.g * p.n;
  const uint32_t a0 = (uint32_t)__cvta_generic_to_shared(stage0), aM = (uint32_t)__cvta_generic_to_shared(sM);
  int i = 0;
  while (x < x_end) {
    const Piece c = piece_at(p, x, x_end);
    const bool two = c.quant || G.pre_rope, grouped = channel_scales(G) && c.quant;
    const bool paired = c.quant && !G.pre_rope && G.kb != 3 && paired_order(G.kb);
    const size_t row0 = ((size_t)c.b * G.Hq_tot + (size_t)layer_head(G, c.h) * G.g) * p.n;
    const uint16_t* q = p.q + row0 * kHeadDim;
    uint32_t qb[8][2];
    float2 lw[2];
    if (ONE) {
      load_rows(q, M, paired, lane, qb);
      load_weights(p, row0, c.b, 0, M, tq, lw);
    }
#pragma unroll 1
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      const uint32_t aK = a0 + st * kKeyStageBytes, aN = aK + kTileBytes;
      if (!wait(B.full_k + 8 * st, i >> 1)) return;
      float sum[2] = {0.0f, 0.0f};  // keys 16 w + g, + 8
#pragma unroll 1
      for (int r0 = 0; r0 < M; r0 += 8) {
        if (!ONE) {
          load_rows(q + (size_t)r0 * kHeadDim, M - r0, paired, lane, qb);
          load_weights(p, row0, c.b, r0, M, tq, lw);
        }
        float z[4] = {}, zn[4] = {}, zg[4] = {};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t ka[4];
          const uint32_t off = tile_off(16 * w + (lane & 15), 2 * ks + (lane >> 4));
          ldsm4(ka, aK + off);
          mma16816(z, ka, qb[ks][0], qb[ks][1]);
          if (two) {
            ldsm4(ka, aN + off);
            mma16816(zn, ka, qb[ks][0], qb[ks][1]);
          }
          if (grouped) {  // 8 rows: the groups' min and scale rows (the mma's rows 8..15: the same)
            ldsm4(ka, aM + st * kGroupRowBytes + q_off<8>(lane & 7, 2 * ks + (lane >> 4)));
            mma16816(zg, ka, qb[ks][0], qb[ks][1]);
          }
        }
        // columns 2 tq + e: min of the warp's group (row w / 2), its scale (row 4 + w / 2)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = __shfl_sync(0xffffffffu, zg[e], 4 * (w >> 1) + tq), sc = __shfl_sync(0xffffffffu, zg[e], 16 + 4 * (w >> 1) + tq);
          const float base = grouped ? fmaf((float)(1 << (G.kb - 1)), sc, mn) : 0.0f;
          if (lw[e].y != 0.0f) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float s = z[2 * k + e] - zn[2 * k + e] + base;
              sum[k] += lw[e].y * ex2(fmaf(s, p.q_scale, -lw[e].x) * 1.4426950408889634f);
            }
          }
        }
      }
      mbar_arrive_warp(B.empty_k + 8 * st);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
        const int f = (c.k0 + t) * kTile + 16 * w + g + 8 * k;
        if (tq == 0 && f < (c.quant ? c.tc.Nq : c.tc.k1)) {
          const int pos = c.quant ? G.S + f : f < c.tc.S_eff ? f : G.S + c.tc.Nq + (f - c.tc.S_eff);
          float* m = p.mass + (size_t)c.s * p.cap + pos;
          *m = fmaf(p.decay, *m, sum[k]);
        }
      }
    }
    x += c.cnt;
  }
}

template <bool ONE>
__global__ void __launch_bounds__(kThreadsMass, 1) mass_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *stage0 = smem, *sM = stage0 + 2 * kKeyStageBytes;
  Tail* tail = reinterpret_cast<Tail*>(sM + 2 * kGroupRowBytes);
  uint8_t* raw0 = sM + 2 * kGroupRowBytes + kTailBytes;
  volatile int* gave_up = &tail->gave_up;
  const int tid = threadIdx.x;
  const Bars B = bars_at((uint32_t)__cvta_generic_to_shared(tail->bars));
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.full_k + 8 * i, kProducers / 32);
      mbar_init(B.empty_k + 8 * i, kConsumerWarps);
    }
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(B.raw_full + 8 * i, 1);
      mbar_init(B.raw_empty + 8 * i, kProducers / 32);
    }
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid < 8) tail->lut[tid] = p.k_lut_off[tid];
  if (tid < kHeadDim) tail->zeros[tid] = 0;
  __syncthreads();
  const int x = cta_first_tile(p.ncta, p.total, blockIdx.x), x_end = cta_first_tile(p.ncta, p.total, blockIdx.x + 1);
  if (tid < kConsumers) {
    weigh<ONE>(p, B, stage0, sM, x, x_end, tid, gave_up);
  } else if (tid < kConsumers + kProducers) {
    produce<0, false>(p, B, nullptr, stage0, sM, raw0, tail, x, x_end, tid - kConsumers, gave_up);
  } else {
    if ((tid & 31) == 0) load_tiles<false>(p, B, (uint32_t)__cvta_generic_to_shared(raw0), x, x_end, gave_up);
    __syncwarp();
  }
  __syncthreads();
  if (*gave_up) {  // a wait ran out: the range's entries become NaN
    for (int y = x; y < x_end;) {
      const Piece c = piece_at(p, y, x_end);
      const int f1 = min((c.k0 + c.cnt) * kTile, c.quant ? c.tc.Nq : c.tc.k1);
      for (int f = c.k0 * kTile + tid; f < f1; f += kThreadsMass)
        p.mass[(size_t)c.s * p.cap + (c.quant ? p.geo.S + f : f < c.tc.S_eff ? f : p.geo.S + c.tc.Nq + (f - c.tc.S_eff))] = NAN;
      y += c.cnt;
    }
  }
}

template <bool ONE>
cudaError_t launch_t(TreeParams& p, cudaStream_t st) {
  static std::atomic<long long> memo[kMemoDevices];
  p.raw = raw_slot(p.geo, false, kSmemMass - kFixedMass);
  if (kFixedMass + p.raw.slots * p.raw.bytes > kSmemMass) return cudaErrorInvalidValue;
  const cudaError_t e = ensure_smem_limit(mass_kernel<ONE>, memo, (int)kSmemMass);
  if (e != cudaSuccess) return e;
  mass_kernel<ONE><<<p.ncta, kThreadsMass, kSmemMass, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_mass(TreeParams& p, cudaStream_t st) {
  if (mass_stream_eligible(p.geo)) return launch_mass_stream(p, st);
  return p.geo.g * p.n <= 8 ? launch_t<true>(p, st) : launch_t<false>(p, st);
}

}  // namespace kvq
