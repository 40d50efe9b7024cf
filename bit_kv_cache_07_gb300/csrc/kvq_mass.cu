// kvq_mass.cu -- accumulated attention weight of every cached token (the
// record that kvq_evict goes by).
//
// For token t of stream (b, h), over the query rows r = (query head j of the
// KV head's group, row i) that attended it:
//   mass_t <- decay * mass_t + sum_r w_i exp(scale * q_r . k_t - lse_r)
// with the log-sum-exp that the attention returned: the rows' softmax is not
// computed again, one pass over the keys is enough.  Up to 8 rows per KV head
// over uniform codes go through kvq_mass_stream.cu; this is the kernel for
// more rows, non-uniform codes and keys cached before RoPE.
//
// The tile kernels' copies and producers, for keys alone.  A tile's keys are
// the matrix product's rows (operand A, 96 of 128), the query rows its
// columns (B, up to 256): a key's logits land in one lane of TMEM, so its
// weights are summed by one thread, in fp32 and in order.  What a group's 32
// keys share (kvq_fill.cuh: keys_channel) is computed per tile by one warp
// with mma.sync and enters the exponent together with -lse; a group's keys
// are one warp's, so it is read like a constant.
//
// Measured: 4 ragged rows up to 32k tokens of InnerQ KV4 keys, 8 KV heads, 68
// query rows each: 92 us (0.72 TB/s).  Bound by the producers' fp32 conversion of
// keys with a scale per token, at 56 % of the issue slots.
#include "kvq_tc.cuh"
#include "kvq_pipe.cuh"

namespace kvq {
namespace {

constexpr int kWeighWarps = kTile / 32;  // one per group of a tile; then the warp that prepares their offsets
constexpr int kThreadsMass = 128 + kProducers + 64;
constexpr int kMaxCols = 256;
constexpr uint32_t kQBytes = kMaxCols * kHeadDim * 2;
constexpr uint32_t kOffBytes = kTile / 32 * kMaxCols * 4;
// (operand A reads 32 rows behind a tile: the next one's, or Q's)
constexpr uint32_t kFixedMass = 2 * kKeyStageBytes + kQBytes + 2 * kGroupRowBytes + 2 * kOffBytes + kMaxCols * 4 + kTailBytes;
constexpr uint32_t kSmemMass = 227 * 1024;

// Byte offset of a 16-byte chunk of query row r (cols rows in all).
__device__ __forceinline__ uint32_t col_off(int cols, int r, int chunk) {
  return (uint32_t)((chunk >> 3) * (cols * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
}

struct MassSmem {
  uint8_t *stage0, *sQ, *sM;
  float *off, *wt;  // [2][3][kMaxCols], [kMaxCols]
};

// The piece's query rows as operand B, their weights, by 128 threads.  A row
// that does not count (weight 0, or nothing seen) is staged as zeros: its
// weights of 1 meet a factor of 0, whatever it held.
__device__ __forceinline__ void put_rows(const TreeParams& p, const Bars& B, const Piece& c, const MassSmem& m, int cols, int tid) {
  const Geometry& G = p.geo;
  const bool paired = c.quant && !G.pre_rope && G.kb != 3 && paired_order(G.kb);
  const size_t row0 = ((size_t)c.b * G.Hq_tot + (size_t)layer_head(G, c.h) * G.g) * p.n + p.r0;
  for (int r = tid; r < cols; r += 128) {
    float w = 0.0f;
    if (r < p.nr && __ldg(p.row_lse + row0 + r) != -INFINITY) w = p.weight ? __ldg(p.weight + (size_t)c.b * p.n + (p.r0 + r) % p.n) : 1.0f;
    m.wt[r] = w;
    const uint4* row = reinterpret_cast<const uint4*>(p.q + (row0 + r) * kHeadDim);
#pragma unroll
    for (int ch = 0; ch < 16; ++ch) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (w != 0.0f) v = __ldg(row + ch);
      if (paired) v = pair_chunk(v);
      *reinterpret_cast<uint4*>(m.sQ + col_off(cols, r, ch)) = v;
    }
  }
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  mbar_arrive_warp(B.q_full);
}

__device__ __forceinline__ void issue(uint32_t lead, const TreeParams& p, const Bars& B, uint32_t tmem, uint32_t stage0, uint32_t q, int cols, int x,
                                      int x_end, volatile int* gave_up) {
  auto wait = [&](uint32_t bar, int phase, volatile int* g) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase, g)); };
  const uint64_t kd = smem_desc(stage0, 16, 1024), qd = smem_desc(q, 16, 1024);  // stage 0; the rest adds to the address
  int i = 0;
  for (int piece = 0; x < x_end; ++piece) {
    const Piece c = piece_at(p, x, x_end);
    const int parts = c.quant || p.geo.pre_rope ? 2 : 1;
    if (!wait(B.q_full, piece & 1, gave_up)) return;
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      if (!wait(B.full_k + 8 * st, (i >> 1) & 1, gave_up)) return;
      if (i >= 2 && !wait(B.p_full + 8 * st, ((i >> 1) - 1) & 1, gave_up)) return;  // the accumulator is read
      tc_after();
      const uint64_t k = kd + st * (kKeyStageBytes >> 4);
      const uint32_t half = cols * 128 >> 4;  // from a row's first 64 channels to the others
      // the keys' small parts first: the sum is small while they enter, so only
      // the large parts' 8 steps cut it at its final size (InnerQ keys, 17 rows: error
      // against 64 bits 1.1e-6 to 5.9e-7, that of plain fp32 6.5e-7)
      if (parts == 2) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 channels
          mma_ss(lead, tmem + 256 * st, k + (kTileBytes >> 4) + (ks >> 2) * (kTile * 128 >> 4) + (ks & 3) * 2,
                 qd + (ks >> 2) * half + (ks & 3) * 2, idesc(cols) | kNegA, ks > 0);
      }
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_ss(lead, tmem + 256 * st, k + (ks >> 2) * (kTile * 128 >> 4) + (ks & 3) * 2, qd + (ks >> 2) * half + (ks & 3) * 2, idesc(cols),
               parts == 2 || ks > 0);
      mma_commit(lead, B.empty_k + 8 * st);
      mma_commit(lead, B.s_full + 8 * st);
    }
    x += c.cnt;
  }
}

// The offsets of a tile: off[group][row] = scale * (q . m + 2^(b-1) q . s) - lse
// (-lse alone where keys come whole), by one warp.
__device__ __forceinline__ void offsets(const TreeParams& p, const Bars& B, const MassSmem& m, int cols, int x, int x_end, int lane,
                                        volatile int* gave_up) {
  auto wait = [&](uint32_t bar, int phase) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, gave_up)); };
  const Geometry& G = p.geo;
  const uint32_t aQ = (uint32_t)__cvta_generic_to_shared(m.sQ), aM = (uint32_t)__cvta_generic_to_shared(m.sM);
  const float centre = (float)(1 << (G.kb - 1));
  int i = 0;
  Piece c = piece_at(p, x, x_end);
  put_rows(p, B, c, m, cols, 32 * kWeighWarps + lane);
  for (int piece = 0; x < x_end; ++piece) {
    const bool grouped = channel_scales(G) && c.quant;
    const float* lse = p.row_lse + ((size_t)c.b * G.Hq_tot + (size_t)layer_head(G, c.h) * G.g) * p.n + p.r0;
    if (!wait(B.q_full, piece)) return;
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      float* off = m.off + st * (kTile / 32) * kMaxCols;
      if (i >= 2 && !wait(B.p_full + 8 * st, (i >> 1) - 1)) return;  // the offsets of tile i - 2 are read
      if (!grouped) {
        for (int r = lane; r < cols; r += 32) {
          const float v = r < p.nr && m.wt[r] != 0.0f ? -__ldg(lse + r) : 0.0f;
#pragma unroll
          for (int g = 0; g < kTile / 32; ++g) off[g * kMaxCols + r] = v;
        }
      } else {
        if (!wait(B.full_k + 8 * st, i >> 1)) return;
        uint32_t a[8][4];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) ldsm4(a[ks], aM + st * kGroupRowBytes + q_off<8>(lane & 7, 2 * ks + (lane >> 4)));
#pragma unroll 1
        for (int r0 = 0; r0 < cols; r0 += 16) {
          float z[2][4] = {};
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t qb[4];
            ldsm4(qb, aQ + col_off(cols, r0 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
            mma16816(z[0], a[ks], qb[0], qb[1]);
            mma16816(z[1], a[ks], qb[2], qb[3]);
          }
          // lane 4 g + tq: q . m of group g (g < 3), q . s of group g - 4 (4 <= g < 7), rows r0 + 8 n + 2 tq + e
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float s = __shfl_down_sync(0xffffffffu, z[n][e], 16);
              const int r = r0 + 8 * n + 2 * (lane & 3) + e;
              if (lane < 4 * (kTile / 32))
                off[(lane >> 2) * kMaxCols + r] =
                    r < p.nr && m.wt[r] != 0.0f ? fmaf(fmaf(centre, s, z[n][e]), p.q_scale, -__ldg(lse + r)) : 0.0f;
            }
        }
      }
      mbar_arrive_warp(B.empty_k + 8 * st);  // the group rows are read
      mbar_arrive_warp(B.full_v + 8 * st);   // the tile's offsets are there
    }
    x += c.cnt;
    if (x < x_end) {
      // every product of this piece is done before its rows are replaced; and every reader of its weights
      if (!wait(B.s_full + 8 * ((i - 1) & 1), (i - 1) >> 1) || !wait(B.p_full + 8 * ((i - 1) & 1), (i - 1) >> 1)) return;
      c = piece_at(p, x, x_end);
      put_rows(p, B, c, m, cols, 32 * kWeighWarps + lane);
    }
  }
}

// Two logits' share of a key's sum: d = v * scale + off, sum += w * 2^(d log2 e).
__device__ __forceinline__ void add_weights(float2& sum, uint32_t v0, uint32_t v1, float scale, float2 off, float2 w) {
  const float2 d = __ffma2_rn(make_float2(__uint_as_float(v0), __uint_as_float(v1)), make_float2(scale, scale), off);
  const float2 y = __fmul2_rn(d, make_float2(1.4426950408889634f, 1.4426950408889634f));
  sum = __ffma2_rn(w, make_float2(ex2(y.x), ex2(y.y)), sum);
}

// A key's sum over the rows that count alone: a row of zeros (one that does not
// count, or padding) meets a key that is not finite as 0 * inf.
__device__ __noinline__ float counted(uint32_t logits, const float* off, const float* wt, int cols, float scale) {
  float sum = 0.0f;
#pragma unroll 1
  for (int r0 = 0; r0 < cols; r0 += 8) {
    uint32_t v[8];
    tm_load8(v, logits + r0);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (wt[r0 + e] != 0.0f) sum = fmaf(wt[r0 + e], ex2(fmaf(__uint_as_float(v[e]), scale, off[r0 + e]) * 1.4426950408889634f), sum);
  }
  return sum;
}

__device__ __forceinline__ void weigh(const TreeParams& p, const Bars& B, uint32_t tmem, const MassSmem& m, int cols, int x, int x_end,
                                      int tid, volatile int* gave_up) {
  auto wait = [&](uint32_t bar, int phase) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, gave_up)); };
  const Geometry& G = p.geo;
  const int w = tid >> 5;
  const uint32_t lane0 = (uint32_t)(tid & ~31) << 16;
  int i = 0;
  Piece c = piece_at(p, x, x_end);
  put_rows(p, B, c, m, cols, tid);
  for (int piece = 0; x < x_end; ++piece) {
    if (!wait(B.q_full, piece)) return;  // all rows' weights are there
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1, f = (c.k0 + t) * kTile + tid;
      const bool have = f < (c.quant ? c.tc.Nq : c.tc.k1);
      float* at = p.mass + (size_t)c.s * p.cap + (c.quant ? G.S + f : f < c.tc.S_eff ? f : G.S + c.tc.Nq + (f - c.tc.S_eff));
      const float old = have ? *at : 0.0f;
      const float4* off = reinterpret_cast<const float4*>(m.off + (st * (kTile / 32) + w) * kMaxCols);
      const float4* wt = reinterpret_cast<const float4*>(m.wt);
      if (!wait(B.full_v + 8 * st, i >> 1) || !wait(B.s_full + 8 * st, i >> 1)) return;
      tc_after();
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (int r0 = 0; r0 < cols; r0 += 32) {
        uint32_t v[32];
        tm_load32(v, tmem + 256 * st + lane0 + r0);
        tm_wait_ld(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 o = off[r0 / 4 + e], u = wt[r0 / 4 + e];
          add_weights(sum, v[4 * e], v[4 * e + 1], p.q_scale, make_float2(o.x, o.y), make_float2(u.x, u.y));
          add_weights(sum, v[4 * e + 2], v[4 * e + 3], p.q_scale, make_float2(o.z, o.w), make_float2(u.z, u.w));
        }
      }
      float total = sum.x + sum.y;
      if (__any_sync(0xffffffffu, total != total)) total = counted(tmem + 256 * st + lane0, &off[0].x, m.wt, cols, p.q_scale);
      tc_before();
      mbar_arrive_warp(B.p_full + 8 * st);
      if (have) *at = fmaf(p.decay, old, total);
    }
    x += c.cnt;
    if (x < x_end) {
      // (the last product is done: its logits were read; every warp is done with the weights)
      if (!wait(B.p_full + 8 * ((i - 1) & 1), (i - 1) >> 1)) return;
      c = piece_at(p, x, x_end);
      put_rows(p, B, c, m, cols, tid);
    }
  }
}

// FP16: the unquantized cache, without the quantized tiles' code (14 x 18k tokens,
// 4 KV heads, 16 rows each: 96 us, 2.7 TB/s; with it 113).
template <bool FP16>
__global__ void __launch_bounds__(kThreadsMass, 1) mass_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  MassSmem m;
  m.stage0 = smem;
  m.sQ = m.stage0 + 2 * kKeyStageBytes;
  m.sM = m.sQ + kQBytes;
  m.off = reinterpret_cast<float*>(m.sM + 2 * kGroupRowBytes);
  m.wt = m.off + 2 * kOffBytes / 4;
  Tail* tail = reinterpret_cast<Tail*>(m.wt + kMaxCols);
  uint8_t* raw0 = reinterpret_cast<uint8_t*>(tail) + kTailBytes;
  volatile int* gave_up = &tail->gave_up;
  const int tid = threadIdx.x, w = tid >> 5, cols = (p.nr + 31) / 32 * 32;
  const Bars B = bars_at((uint32_t)__cvta_generic_to_shared(tail->bars));
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.full_k + 8 * i, kProducers / 32);
      mbar_init(B.empty_k + 8 * i, 2);            // the products, the offsets' warp
      mbar_init(B.s_full + 8 * i, 1);             // logits
      mbar_init(B.p_full + 8 * i, kWeighWarps);   // logits and offsets are read
      mbar_init(B.full_v + 8 * i, 1);             // offsets (there are no values)
    }
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(B.raw_full + 8 * i, 1);
      mbar_init(B.raw_empty + 8 * i, kProducers / 32);
    }
    mbar_init(B.q_full, 4);
    mbar_init(B.done, 1);
    *gave_up = ((uint32_t)__cvta_generic_to_shared(smem) & 1023) != 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  put_tables<false>(p, tail, raw0, tid);
  constexpr int issuer = 4 + kProducers / 32;  // then the copies' warp
  if (w == issuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&tail->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *(volatile uint32_t*)&tail->tmem;
  const int x = cta_first_tile(p.ncta, p.total, blockIdx.x), x_end = cta_first_tile(p.ncta, p.total, blockIdx.x + 1);
  if (*gave_up) {
  } else if (w < kWeighWarps) {
    weigh(p, B, tmem, m, cols, x, x_end, tid, gave_up);
  } else if (w < 4) {
    offsets(p, B, m, cols, x, x_end, tid & 31, gave_up);
  } else if (w < issuer) {
    produce<0, false, FP16>(p, B, nullptr, m.stage0, m.sM, raw0, tail, x, x_end, tid - 128, gave_up);
  } else if (w == issuer) {
    const uint32_t lead = elect_lead();
    issue(lead, p, B, tmem, (uint32_t)__cvta_generic_to_shared(m.stage0), (uint32_t)__cvta_generic_to_shared(m.sQ), cols, x, x_end, gave_up);
    mma_commit(lead, B.done);  // whatever is in flight ends before TMEM is freed
    mbar_wait(B.done, 0, nullptr);
    __syncwarp();
  } else {
    if ((tid & 31) == 0) load_tiles<false>(p, B, (uint32_t)__cvta_generic_to_shared(raw0), x, x_end, gave_up);
    __syncwarp();
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (w == issuer) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
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

}  // namespace

template <bool FP16>
static cudaError_t launch(TreeParams& p, cudaStream_t st) {
  const int M = p.geo.g * p.n;
  static std::atomic<long long> memo[kMemoDevices];
  cudaError_t e = ensure_smem_limit(mass_kernel<FP16>, memo, (int)kSmemMass);
  // rows beyond one accumulator's columns: further passes add to the record
  for (p.r0 = 0; e == cudaSuccess && p.r0 < M; p.r0 += kMaxCols) {
    p.nr = M - p.r0 < kMaxCols ? M - p.r0 : kMaxCols;
    mass_kernel<FP16><<<p.ncta, kThreadsMass, kSmemMass, st>>>(p);
    e = cudaGetLastError();
    p.decay = 1.0f;
  }
  return e;
}
cudaError_t launch_attn_mass(TreeParams& p, cudaStream_t st) {
  if (p.geo.g * p.n <= 8 && mass_stream_eligible(p.geo)) return launch_mass_stream(p, st);
  p.raw = raw_slot(p.geo, false, kSmemMass - kFixedMass);
  if (kFixedMass + raw_bytes(p.geo, p.raw, false) > kSmemMass) return cudaErrorInvalidValue;
  return p.geo.fp16_mode ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace kvq
