// kvq_mass_stream.cu -- accumulated attention weight for up to 8 query rows per
// KV head, over uniform codes (and fp16 tokens) without RoPE: every call after
// a decode, and after small trees.
//
// With few rows a tile of dequantized keys costs far more than its products,
// so the codes go to the tensor cores as they are (the decode's key side,
// kvq_decode_mma.cuh): S = Kcodes . Q', Q' = q * scale_k per channel in hi + lo
// fp16 parts (q brought into (-1, 1) by a power of two per row), the codes
// centred (code - 2^(b-1): the record is fp32, and the offset of 1024 that the
// decode leaves in its codes would cost it 10 bits), the minimum's share in one
// number per row.  A thread's operand is 32 consecutive channels of a token, so
// a warp reads whole rows from global memory straight into its fragments,
// the next 32 tokens' ahead of this one's products: no shared memory for keys,
// no barrier between warps.
//
// Every warp walks an equal range of 32-token items (quantized groups, then
// fp16 items, stream after stream).
//
// Measured: 16 x 32k tokens KV2, 8 KV heads, 4 query rows each: 87 us (2.75 TB/s);
// 777 tokens KV8: 11 us, the host's time of a call.  Bound by instructions (64 %
// of the issue slots): the group's Q' and an exponential per key and row.
#include <cstring>

#include "kvq_decode_mma.cuh"
#include "kvq_tree.cuh"

namespace kvq {
namespace {

constexpr int kStreamWarps = 4;  // per CTA

struct StreamParams {
  Geometry geo;
  LayerPtrs L;
  const uint16_t* q;
  const float* row_lse;
  const float* weight;
  float* mass;
  float decay, scale;
  int n, cap, nr;      // rows per sequence, tokens of a record's row; rows of a KV head
  int nwarps, total;   // warps, 32-token items
  int tokens[kMaxRaggedRows];
  int item0[kMaxRaggedRows + 1];
};

template <int NT>
struct WarpSmem {
  alignas(16) float qw[4 * NT][kHeadDim];  // q * softmax scale, in the Q' build's channel order
  mma::MmaWarpSmem<NT> m;
  alignas(8) float qsum[4 * NT][2];  // InnerQ: sum of q n over each channel group
  float up[4 * NT];                  // the rows' powers of two
};

// The keys of a group in flight: this thread's 32-channel slices of tokens gq + 8 i.
template <int KB>
struct GroupRegs {
  uint32_t w[4][KB];  // KB words of 4 bytes: 32 channels
  uint2 s01, s23;     // {min, scale} of the lane's four Q' channels (InnerQ: unused)
  uint2 tok[4];       // InnerQ: {min, scale} of tokens gq + 8 i, both groups
};
template <int KB, bool IQ>
__device__ __forceinline__ void load_group(const StreamParams& p, int s, int grp, int lane, GroupRegs<KB>& r) {
  const Geometry& G = p.geo;
  constexpr int kRow = kHeadDim * KB / 8, kSlice = 4 * KB;
  const int gq = lane >> 2, tq = lane & 3;
  const size_t tok = (size_t)s * G.qcap + (size_t)grp * kGroupTokens;
  const uint8_t* codes = p.L.k_codes + tok * kRow;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* row = codes + (gq + 8 * i) * kRow;
    if constexpr (IQ) {
      // half the slice from each 64-channel group
      if constexpr (KB == 8) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + 16 * tq)), b = __ldg(reinterpret_cast<const uint4*>(row + 64 + 16 * tq));
        r.w[i][0] = a.x, r.w[i][1] = a.y, r.w[i][2] = a.z, r.w[i][3] = a.w;
        r.w[i][4] = b.x, r.w[i][5] = b.y, r.w[i][6] = b.z, r.w[i][7] = b.w;
      } else if constexpr (KB == 4) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + 8 * tq)), b = __ldg(reinterpret_cast<const uint2*>(row + 32 + 8 * tq));
        r.w[i][0] = a.x, r.w[i][1] = a.y, r.w[i][2] = b.x, r.w[i][3] = b.y;
      } else {
        r.w[i][0] = __ldg(reinterpret_cast<const uint32_t*>(row + 4 * tq));
        r.w[i][1] = __ldg(reinterpret_cast<const uint32_t*>(row + 16 + 4 * tq));
      }
      r.tok[i] = __ldg(reinterpret_cast<const uint2*>(p.L.k_scales + 2 * (tok + gq + 8 * i)));
    } else if constexpr (KB == 2) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + kSlice * tq));
      r.w[i][0] = a.x, r.w[i][1] = a.y;
    } else {
#pragma unroll
      for (int k = 0; k < KB / 4; ++k) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + kSlice * tq) + k);
        r.w[i][4 * k] = a.x, r.w[i][4 * k + 1] = a.y, r.w[i][4 * k + 2] = a.z, r.w[i][4 * k + 3] = a.w;
      }
    }
  }
  if constexpr (!IQ) {
    const uint32_t* sc = p.L.k_scales + ((size_t)s * G.gcap + grp) * kHeadDim;
    const int c0 = mma::qb_first_channel<KB>(lane);
    r.s01 = __ldg(reinterpret_cast<const uint2*>(sc + c0));
    r.s23 = __ldg(reinterpret_cast<const uint2*>(sc + c0 + mma::qb_pair_dist<KB>()));
  }
}

// The power of two that brings a row whose largest element is `most` into
// (-1, 1), and the one back.  Q' then stays below the scales themselves, so
// within fp16's range (with large rows over wide channels q * scale_k does not),
// and both are exact.
__device__ __forceinline__ void unit_range(float most, float* down, float* back) {
  const uint32_t e = min(__float_as_uint(most) >> 23, 252u);  // biased; most < 2^(e - 126)
  *down = __uint_as_float((253 - e) << 23);
  *back = __uint_as_float((e + 1) << 23);
}

// x as hi + 2^-11 lo, both fp16 (the rest is scaled up: unscaled it would lie in
// fp16's subnormal range and keep few bits).
constexpr float kLoUp = 2048.0f, kLoDown = 1.0f / 2048.0f;
__device__ __forceinline__ void split_scaled(float2 x, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 f = __half22float2(h);
  hi = mma::h2_as_u32(h);
  lo = mma::h2_as_u32(__floats2half2_rn((x.x - f.x) * kLoUp, (x.y - f.y) * kLoUp));
}

// Centred codes of k-step st for one token (see mma::k_frag for the order).
template <int KB>
__device__ __forceinline__ void centred_frag(const uint32_t* w, int st, uint32_t& lo, uint32_t& hi) {
  auto h2 = [](uint16_t x) { return __halves2half2(__ushort_as_half(x), __ushort_as_half(x)); };
  auto h = [](uint32_t x) { return mma::u32_as_h2(x); };
  mma::k_frag<KB>(w, st, lo, hi);
  if constexpr (KB == 8) {
    lo = mma::h2_as_u32(__hsub2(h(lo), h2(0x6480)));  // 1024 + 128
    hi = mma::h2_as_u32(__hsub2(h(hi), h2(0x6480)));
  } else if constexpr (KB == 4) {
    lo = mma::h2_as_u32(__hsub2(h(lo), h2(0x6408)));                    // 1024 + 8
    hi = mma::h2_as_u32(__hfma2(h(hi), h2(0x2C00), h2(0xD480)));        // / 16 - 72
  } else if (st & 1) {
    lo = mma::h2_as_u32(__hfma2(h(lo), h2(0x2C00), h2(0xD420)));        // / 16 - 66
    hi = mma::h2_as_u32(__hfma2(h(hi), h2(0x2400), h2(0xCC80)));        // / 64 - 18
  } else {
    lo = mma::h2_as_u32(__hsub2(h(lo), h2(0x6402)));                    // 1024 + 2
    hi = mma::h2_as_u32(__hfma2(h(hi), h2(0x3400), h2(0xDC08)));        // / 4 - 258
  }
}

// InnerQ: the rows' fragments, q * n_c in hi + lo parts, fixed over a stream
// (a scale per token multiplies the products), and sum_c q_c n_c of the two
// channel groups.
template <int KB, int NT>
__device__ __forceinline__ void build_q_token(WarpSmem<NT>& sm, const float* __restrict__ norm, int nr, int lane) {
  const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = NT == 2 ? gq : gq >> 1;
    const bool lo = NT == 2 ? nt == 1 : (gq & 1) != 0;
    unsigned char* row = reinterpret_cast<unsigned char*>(&sm.m.bq[nt][lane][0]);
#pragma unroll
    for (int c4 = 0; c4 < 4; ++c4) {
      uint32_t reg[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int ri = 4 * c4 + k;
        uint32_t hv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = mma::iq_channel(tq, mma::k_offset_of<KB>(ri >> 1, 2 * (ri & 1) + e));
          const float v = r < nr ? sm.qw[r][mma::qb_perm_pos<KB>(c)] * (norm ? __ldg(norm + c) : 1.0f) : 0.0f;
          const __half hi = __float2half_rn(v);
          hv[e] = __half_as_ushort(lo ? __float2half_rn((v - __half2float(hi)) * kLoUp) : hi);
        }
        reg[k] = hv[0] | (hv[1] << 16);
      }
      *reinterpret_cast<uint4*>(row + 16 * (c4 ^ ((lane >> 1) & 3))) = make_uint4(reg[0], reg[1], reg[2], reg[3]);
    }
  }
  for (int r = 0; r < nr; ++r) {
    float qs = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = 4 * lane + k;  // all four in group lane / 16
      qs += sm.qw[r][mma::qb_perm_pos<KB>(c)] * (norm ? __ldg(norm + c) : 1.0f);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) qs += __shfl_xor_sync(0xffffffffu, qs, o);
    if ((lane & 15) == 0) sm.qsum[r][lane >> 4] = qs;
  }
  __syncwarp();
}

// Q' of a group: fragment rows (hi and lo) and every row's bias.
template <int KB, int NT>
__device__ __forceinline__ void build_q(WarpSmem<NT>& sm, const GroupRegs<KB>& r, int nr, int lane) {
  constexpr int GT = 4 * NT;
  const float2 ms[4] = {unpack_min_scale(r.s01.x), unpack_min_scale(r.s01.y), unpack_min_scale(r.s23.x), unpack_min_scale(r.s23.y)};
  const int c0 = mma::qb_first_channel<KB>(lane);
  // pairs A = (c0, c0 + D) -> B-word 2s, B = (c0 + 1, c0 + D + 1) -> B-word 2s + 1
  const float2 skA = make_float2(ms[0].y, ms[2].y), skB = make_float2(ms[1].y, ms[3].y);
  const float2 mnA = make_float2(ms[0].x, ms[2].x), mnB = make_float2(ms[1].x, ms[3].x);
  const int tsl = lane >> 3;  // reader thread-in-group of these channels
  float bpart[GT];
#pragma unroll
  for (int h = 0; h < GT; ++h) {
    bpart[h] = 0.0f;
    if (h >= nr) continue;
    unsigned char *dhi, *dlo;
    int whi, wlo;
    if constexpr (NT == 2) {
      const int row = 4 * h + tsl;  // column h in table 0 (hi) and table 1 (lo)
      dhi = reinterpret_cast<unsigned char*>(&sm.m.bq[0][row][0]);
      dlo = reinterpret_cast<unsigned char*>(&sm.m.bq[1][row][0]);
      whi = wlo = (8 * (lane & 7)) ^ (((row >> 1) & 3) << 4);
    } else {
      dhi = reinterpret_cast<unsigned char*>(&sm.m.bq[0][8 * h + tsl][0]);  // columns 2 h (hi), 2 h + 1 (lo)
      dlo = dhi + 4 * 64;
      whi = (8 * (lane & 7)) ^ (((tsl >> 1) & 1) << 4);
      wlo = whi ^ 32;
    }
    const float4 q4 = *reinterpret_cast<const float4*>(&sm.qw[h][4 * lane]);
    const float2 qA = make_float2(q4.x, q4.y), qB = make_float2(q4.z, q4.w);
    const float2 pA = make_float2(qA.x * skA.x, qA.y * skA.y), pB = make_float2(qB.x * skB.x, qB.y * skB.y);
    uint32_t hA, lA, hB, lB;
    split_scaled(pA, hA, lA);
    split_scaled(pB, hB, lB);
    *reinterpret_cast<uint2*>(dhi + whi) = make_uint2(hA, hB);
    *reinterpret_cast<uint2*>(dlo + wlo) = make_uint2(lA, lB);
    // the minimum's share and the centre's
    const float mins = qA.x * mnA.x + qA.y * mnA.y + qB.x * mnB.x + qB.y * mnB.y;
    bpart[h] = fmaf((float)(1 << (KB - 1)), (pA.x + pA.y) + (pB.x + pB.y), mins);
  }
  const float bsum = mma::reduce_heads<GT>(bpart, lane);
  const int hb = mma::head_of_lane<GT>(lane);
  if ((lane & mma::rest_mask<GT>()) == 0 && hb < nr) sm.m.bias[hb] = bsum;
  __syncwarp();
}

// A lane's rows: NT = 1: row tq; NT = 2: rows 2 tq, 2 tq + 1.
template <int NT>
__device__ __forceinline__ int lane_row(int i, int tq) { return NT == 2 ? 2 * tq + i : tq; }

// Add the weights of tokens gq + 8 i, i = 0..3, to the record: x[i] is this
// lane's share of token i's sum.
__device__ __forceinline__ void record(float (&x)[4], float* at, bool have, float decay, float old, int tq) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] += __shfl_xor_sync(0xffffffffu, x[i], 1);
    x[i] += __shfl_xor_sync(0xffffffffu, x[i], 2);
  }
  const float mine = tq == 0 ? x[0] : tq == 1 ? x[1] : tq == 2 ? x[2] : x[3];  // token gq + 8 tq
  if (have) *at = fmaf(decay, old, mine);
}

template <int KB, int NT, bool IQ>
__global__ void __launch_bounds__(32 * kStreamWarps, 4) mass_stream_kernel(const __grid_constant__ StreamParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const Geometry& G = p.geo;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  WarpSmem<NT>& sm = reinterpret_cast<WarpSmem<NT>*>(smem)[threadIdx.x >> 5];
  const int wi = blockIdx.x * kStreamWarps + (threadIdx.x >> 5);
  if (wi >= p.nwarps) return;
  int x = cta_first_tile(p.nwarps, p.total, wi);
  const int x_end = cta_first_tile(p.nwarps, p.total, wi + 1);
  while (x < x_end) {
    const int b = row_of(p.item0, G.B, x);
    int S_eff, Nq, W;
    window_counts(G, p.tokens[b], &S_eff, &Nq, &W);
    const int ng = Nq / kGroupTokens, k1 = S_eff + W, per = ng + (k1 + 31) / 32;
    const int off = x - p.item0[b], h = off / per, k0 = off - h * per, s = b * G.Hkv + h;
    const int k_end = min(per, k0 + x_end - x);
    const size_t row0 = ((size_t)b * G.Hq_tot + (size_t)layer_head(G, h) * G.g) * p.n;
    const uint16_t* q = p.q + row0 * kHeadDim;
    float* rec = p.mass + (size_t)s * p.cap;
    // the lane's rows: log-sum-exp (log2 units) and weight; a row that saw nothing counts as 0
    float lse[NT], wt[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = lane_row<NT>(i, tq);
      lse[i] = wt[i] = 0.0f;
      if (r < p.nr) {
        const float l = __ldg(p.row_lse + row0 + r);
        if (l != -INFINITY) lse[i] = l, wt[i] = p.weight ? __ldg(p.weight + (size_t)b * p.n + r % p.n) : 1.0f;
      }
    }
    if (k0 < ng) {
      // the rows, scaled, in the Q' build's order; a row that does not count may hold anything
      const float* norm = IQ && G.knorm ? p.L.k_norm + (size_t)s * kHeadDim : nullptr;
      __syncwarp();
#pragma unroll 1
      for (int r = 0; r < p.nr; ++r) {
        float x[4], most = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = lane + 32 * j;
          x[j] = half_bits_to_float(__ldg(q + (size_t)r * kHeadDim + c)) * p.scale;
          most = fmaxf(most, fabsf(norm ? x[j] * __ldg(norm + c) : x[j]));
        }
        float down, back;
        unit_range(warp_max(most), &down, &back);
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.qw[r][mma::qb_perm_pos<KB>(lane + 32 * j)] = x[j] * down;
        if (lane == 0) sm.up[r] = back;
      }
      __syncwarp();
      if constexpr (IQ) build_q_token<KB, NT>(sm, norm, p.nr, lane);
      GroupRegs<KB> cur;
      load_group<KB, IQ>(p, s, k0, lane, cur);
      const int ke = min(k_end, ng);
#pragma unroll 1
      for (int k = k0; k < ke; ++k) {
        float* at = rec + G.S + k * kGroupTokens + gq + 8 * tq;
        const float old = *at;
        if constexpr (!IQ) {
          __syncwarp();  // the last group's Q' is read
          build_q<KB, NT>(sm, cur, p.nr, lane);
        }
        GroupRegs<KB> now = cur;
        if (k + 1 < ke) load_group<KB, IQ>(p, s, k + 1, lane, cur);  // in flight under this group's products
        uint32_t bq[NT][16];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(&sm.m.bq[nt][lane][0]) + 16 * (c ^ ((lane >> 1) & 3)));
            bq[nt][4 * c] = u.x, bq[nt][4 * c + 1] = u.y, bq[nt][4 * c + 2] = u.z, bq[nt][4 * c + 3] = u.w;
          }
        float sum[4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          // two accumulators: even and odd k-steps (InnerQ: the two channel groups); NT = 2: per part
          float S0[NT][4] = {}, S1[NT][4] = {};
#pragma unroll
          for (int st = 0; st < 8; ++st) {
            uint32_t lo0, hi0, lo1, hi1;
            centred_frag<KB>(now.w[2 * mt], st, lo0, hi0);
            centred_frag<KB>(now.w[2 * mt + 1], st, lo1, hi1);
            float(*acc)[4] = (IQ ? st >= 4 : st & 1) ? S1 : S0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma::mma16816(acc[nt], lo0, lo1, hi0, hi1, bq[nt][2 * st], bq[nt][2 * st + 1]);
          }
#pragma unroll
          for (int rh = 0; rh < 2; ++rh) {
            float add = 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const int r = lane_row<NT>(i, tq);
              // hi and lo parts: column pairs (NT = 1), or the two tables
              const float a = NT == 2 ? fmaf(S0[NT - 1][2 * rh + i], kLoDown, S0[0][2 * rh + i]) : fmaf(S0[0][2 * rh + 1], kLoDown, S0[0][2 * rh]);
              const float c = NT == 2 ? fmaf(S1[NT - 1][2 * rh + i], kLoDown, S1[0][2 * rh + i]) : fmaf(S1[0][2 * rh + 1], kLoDown, S1[0][2 * rh]);
              float z;
              if constexpr (IQ) {
                // sum_j s_j S_j + (min_j + 2^(b-1) s_j) sum q n
                const float2 qs = *reinterpret_cast<const float2*>(&sm.qsum[r < p.nr ? r : 0][0]);
                const float2 t0 = unpack_min_scale(now.tok[2 * mt + rh].x), t1 = unpack_min_scale(now.tok[2 * mt + rh].y);
                constexpr float kC = (float)(1 << (KB - 1));
                z = fmaf(t0.y, a, fmaf(kC, t0.y, t0.x) * qs.x) + fmaf(t1.y, c, fmaf(kC, t1.y, t1.x) * qs.y);
              } else {
                z = a + c + sm.m.bias[r < p.nr ? r : 0];
              }
              if (wt[i] != 0.0f) add = fmaf(wt[i], mma::ex2(fmaf(z, sm.up[r < p.nr ? r : 0], -lse[i]) * 1.4426950408889634f), add);
            }
            sum[2 * mt + rh] = add;
          }
        }
        record(sum, at, true, p.decay, old, tq);
      }
    }
    // fp16 items: k-step st takes channels 32 tq + 4 st .. + 3; columns are the rows
    if (k_end > ng) {
      uint32_t qb[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (gq < p.nr) u = __ldg(reinterpret_cast<const uint4*>(q + (size_t)gq * kHeadDim + 32 * tq) + c);
        qb[4 * c] = u.x, qb[4 * c + 1] = u.y, qb[4 * c + 2] = u.z, qb[4 * c + 3] = u.w;
      }
      float lf[2], wf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * tq + i;
        lf[i] = wf[i] = 0.0f;
        if (r < p.nr) {
          const float l = __ldg(p.row_lse + row0 + r);
          if (l != -INFINITY) lf[i] = l, wf[i] = p.weight ? __ldg(p.weight + (size_t)b * p.n + r % p.n) : 1.0f;
        }
      }
      const int slot0 = Nq % G.ring;
#pragma unroll 1
      for (int k = max(k0, ng); k < k_end; ++k) {
        const int f0 = 32 * (k - ng);
        float sum[4];
#pragma unroll 1
        for (int mt = 0; mt < 2; ++mt) {
          uint4 w[2][4];
#pragma unroll
          for (int rh = 0; rh < 2; ++rh) {
            const int f = f0 + gq + 8 * (2 * mt + rh);
            int slot = slot0 + f - S_eff;
            if (slot >= G.ring) slot -= G.ring;
            const uint16_t* row = f < S_eff ? p.L.k_sink + ((size_t)s * G.S + f) * kHeadDim : p.L.k_ring + ((size_t)s * G.ring + slot) * kHeadDim;
#pragma unroll
            for (int c = 0; c < 4; ++c) w[rh][c] = f < k1 ? __ldg(reinterpret_cast<const uint4*>(row + 32 * tq) + c) : make_uint4(0, 0, 0, 0);
          }
          float S[4] = {};
#pragma unroll
          for (int st = 0; st < 8; ++st) {
            const uint4 a = w[0][st >> 1], c = w[1][st >> 1];
            const uint32_t a0 = st & 1 ? a.z : a.x, a2 = st & 1 ? a.w : a.y, c0 = st & 1 ? c.z : c.x, c2 = st & 1 ? c.w : c.y;
            mma::mma16816(S, a0, c0, a2, c2, qb[2 * st], qb[2 * st + 1]);
          }
#pragma unroll
          for (int rh = 0; rh < 2; ++rh) {
            float add = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (wf[i] != 0.0f) add = fmaf(wf[i], mma::ex2(fmaf(S[2 * rh + i], p.scale, -lf[i]) * 1.4426950408889634f), add);
            if (mt == 0) sum[rh] = add;
            else sum[2 + rh] = add;
          }
        }
        const int f = f0 + gq + 8 * tq;
        const int pos = f < S_eff ? f : G.S + Nq + (f - S_eff);
        const bool have = f < k1;
        record(sum, rec + pos, have, p.decay, have ? rec[pos] : 0.0f, tq);
      }
    }
    x += k_end - k0;
  }
}

template <int KB, int NT, bool IQ>
cudaError_t launch_t(const StreamParams& p, cudaStream_t st) {
  static std::atomic<long long> memo[kMemoDevices];
  const int smem = (int)sizeof(WarpSmem<NT>) * kStreamWarps;
  const cudaError_t e = ensure_smem_limit(mass_stream_kernel<KB, NT, IQ>, memo, smem);
  if (e != cudaSuccess) return e;
  mass_stream_kernel<KB, NT, IQ><<<(p.nwarps + kStreamWarps - 1) / kStreamWarps, 32 * kStreamWarps, smem, st>>>(p);
  return cudaGetLastError();
}
template <int KB>
cudaError_t launch_kb(const StreamParams& p, cudaStream_t st) {
  if (p.geo.gkc) return p.nr <= 4 ? launch_t<KB, 1, true>(p, st) : launch_t<KB, 2, true>(p, st);
  return p.nr <= 4 ? launch_t<KB, 1, false>(p, st) : launch_t<KB, 2, false>(p, st);
}

}  // namespace

bool mass_stream_eligible(const Geometry& G) { return !G.pre_rope && G.kb != 3; }

cudaError_t launch_mass_stream(const TreeParams& t, cudaStream_t st) {
  StreamParams p;
  std::memset(&p, 0, sizeof(p));
  p.geo = t.geo;
  p.L = t.L;
  p.q = t.q;
  p.row_lse = t.row_lse;
  p.weight = t.weight;
  p.mass = t.mass;
  p.scale = t.q_scale;
  p.n = t.n;
  p.cap = t.cap;
  long long total = 0;
  for (int b = 0; b < p.geo.B; ++b) {
    p.tokens[b] = t.rows.tokens[b];
    int S_eff, Nq, W;
    window_counts(p.geo, p.tokens[b], &S_eff, &Nq, &W);
    p.item0[b] = (int)total;
    total += (long long)p.geo.Hkv * (Nq / kGroupTokens + (S_eff + W + 31) / 32);
  }
  p.item0[p.geo.B] = (int)total;
  p.total = (int)total;  // at most 3 (and an odd one) per tile of the caller's count
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (p.geo.sm_budget > 0 && p.geo.sm_budget < sms) sms = p.geo.sm_budget;
  const long long warps = (long long)sms * 4 * kStreamWarps;
  p.nwarps = (int)(warps < total ? warps : total);
  p.nr = p.geo.g * p.n;
  p.decay = t.decay;
  return p.geo.fp16_mode || p.geo.kb == 2 ? launch_kb<2>(p, st) : p.geo.kb == 4 ? launch_kb<4>(p, st) : launch_kb<8>(p, st);
}

}  // namespace kvq
