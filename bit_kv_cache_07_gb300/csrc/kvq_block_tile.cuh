// kvq_block_tile.cuh -- one warp's arithmetic on a tile (a block of 32 tokens of a KV
// head) for the block attention, for up to 8 NT (token, query head) rows.
//
// With y_rt = scale log2(e) 2^ek (q_r . c_t) + ev and w_rt = 2^(y_rt - ref_r) it keeps
// per row ref, l = sum 2^-ev w and O = sum w c'.  Codes become fp16 in registers (e4m3
// is a subset); weights go up to 2^12 at a new reference and to 2^15 before it moves
// (fp16 ends at 2^16).
//
// The tokens lie on the product's 16 rows and the query rows on its 8 columns
// (S^T = K Q^T, O^T = V^T P^T): decode steps of up to 8 heads per KV head fill the
// columns, and 32 matrix instructions, half the exponentials and 32 accumulators do
// where query rows on the 16 rows take twice that (64 ragged requests of 7 heads
// 53.5 us that way, 48.3 this way).  A tile's conversions (128 instructions, the larger
// part) serve all NT column tiles.  With NT 1 the weights enter in two fp16 parts (22
// bits, 16 matrix instructions more), which leaves the output its own rounding's
// error (2.1e-4 normwise against 64 bits).  With NT 2 they enter in one (2.6e-4): its
// 255 registers are full, and two take 56.5 us in place of 50.8 at 16 rows, 114 in place
// of 95 at 32 (16 x 8k tokens of 32 on 8 heads).
//
// More rows are more warps on a tile, 16 rows each, which convert it again: 32 rows by
// one warp spill their accumulators (and took 98 us where two warps took 94, 16 x 8k
// tokens, 8 new ones of 32 on 8 heads; 16 rows spill 16 to 44 bytes themselves).
#pragma once

#include "kvq_block.cuh"
#include "kvq_pipe.cuh"

namespace kvq {
namespace tile {

constexpr float kRoom = 12.0f, kMoveAt = 15.0f;

__device__ __forceinline__ void e4m3_halves(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n" : "=r"(lo), "=r"(hi) : "r"(four));
}
__device__ __forceinline__ uint32_t as_word(const __half2& h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ uint32_t pack_halves(float a, float b) { return as_word(__floats2half2_rn(a, b)); }
__device__ __forceinline__ uint32_t transposed(uint32_t a) {  // an 8 x 8 matrix of halves over the warp
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
  return d;
}

// Token (of the request's new ones) of row r of a segment's block: a row below 64 and
// what r0 lies into its token are below 2^11, so the product with ceil(2^32 / g) is exact.
__device__ __forceinline__ int token_at(const BlockAttnParams& p, const BlockSegment& s, int r) {
  const int i0 = s.r0 ? s.r0 / p.geo.g : 0, x = s.r0 - i0 * p.geo.g + r;
  return i0 + (p.geo.g > 1 ? (int)__umulhi((unsigned)x, p.g_inv) : x);
}
// Row of q and out.
__device__ __forceinline__ size_t row_at(const BlockAttnParams& p, const BlockSegment& s, int r) {
  const int i = token_at(p, s, r), j = s.r0 + r - i * p.geo.g;
  return (size_t)(s.first + i) * p.geo.Hq + s.h * p.geo.g + j;
}
__device__ __forceinline__ float log_sum(float ref, float l) { return l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f; }

struct Tile {
  const uint8_t* K;
  uint32_t V;           // shared-memory address
  float f, ev, inv_v;   // scale log2(e) 2^ek, ev, 2^-ev
  int t0;               // first token
  bool masked;          // some row does not see some token
};

// The values of two chunks (16 channels each) of 16 tokens, by ldmatrix: a pair of
// adjacent channels of two tokens per register, then sorted by channel: ev[u][o] the
// even, od[u][o] the odd channel of chunk u, tokens of octet o.
__device__ __forceinline__ void value_halves(uint32_t V, int lane, int kk, int c, uint32_t (&even)[2][2], uint32_t (&odd)[2][2]) {
  uint32_t v[4];
  const int mt = lane >> 3, tok = 16 * kk + 8 * (mt & 1) + (lane & 7);
  ldsm4t(v, V + tok * kHeadDim + (((c + (mt >> 1)) ^ (lane & 7)) << 4));
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int o = 0; o < 2; ++o) e4m3_halves(__byte_perm(v[2 * u + o], 0, 0x3120), even[u][o], odd[u][o]);
}

// Lane (gq, tq): rows 8 n + 2 tq, + 1 of the results, rows 8 n + gq of the queries.
template <int NT>
struct Rows {
  static constexpr int kRows = 8 * NT;
  static constexpr int kParts = NT == 1 ? 2 : 1;  // fp16 parts of a weight
  uint32_t q[NT][8][2];
  float O[NT][8][4], ref[NT][2], l[NT][2];  // O[n][c]: channels 16 c + 2 gq (+ 1 in the last two), rows 2 tq, 2 tq + 1 of n

  // Channel 32 tq + 4 k + {0, 1 | 2, 3} enters step k of the product as 2 tq + {0, 1 | 8, 9}.
  __device__ __forceinline__ void load_q(const BlockAttnParams& p, const BlockSegment& s, int row0, int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = min(row0 + 8 * n + (lane >> 2), s.rows - 1);  // (rows that are not there: the last one again)
      const uint4* src = reinterpret_cast<const uint4*>(p.q + row_at(p, s, r) * kHeadDim + 32 * (lane & 3));
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = __ldg(src + u);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) q[n][k][0] = w[2 * k], q[n][k][1] = w[2 * k + 1];
    }
  }
  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ref[n][i] = -INFINITY;
        l[n][i] = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) O[n][c][0] = O[n][c][1] = O[n][c][2] = O[n][c][3] = 0.0f;
    }
  }
  // row0: this warp's first row
  __device__ __forceinline__ void tile(const BlockAttnParams& p, const BlockSegment& s, const Tile& t, int lane, int row0) {
    const int gq = lane >> 2, tq = lane & 3;
    float S[NT][2][4];  // tokens 16 m + gq, + 8 (the last two), rows 2 tq, 2 tq + 1 of n
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < 2; ++m) S[n][m][0] = S[n][m][1] = S[n][m][2] = S[n][m][3] = 0.0f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // of the channels
      uint4 kc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        kc[j] = *reinterpret_cast<const uint4*>(t.K + (8 * j + gq) * kHeadDim + (((2 * tq + half) ^ gq) << 4));
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t a[4];
          e4m3_halves(reinterpret_cast<const uint32_t*>(&kc[2 * m])[k], a[0], a[2]);
          e4m3_halves(reinterpret_cast<const uint32_t*>(&kc[2 * m + 1])[k], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(S[n][m], a, q[n][4 * half + k][0], q[n][4 * half + k][1]);
        }
    }
    uint32_t w[kParts][NT][2][2];  // weights of 16 tokens, as the product's columns
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (NT > 1 && row0 + 8 * n >= s.rows) {  // no such rows
#pragma unroll
        for (int part = 0; part < kParts; ++part) w[part][n][0][0] = w[part][n][0][1] = w[part][n][1][0] = w[part][n][1][1] = 0;
        continue;
      }
      float z[2][4];
      const float base[2] = {t.ev - ref[n][0], t.ev - ref[n][1]};
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[m][e] = fmaf(S[n][m][e], t.f, base[e & 1]);
      if (t.masked) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pos = s.before + token_at(p, s, min(row0 + 8 * n + 2 * tq + i, s.rows - 1));
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = i; e < 4; e += 2) {
              const int at = t.t0 + 16 * m + gq + 8 * (e >> 1);
              if (!(at <= pos && (pos - at < p.window || at < p.n_first))) z[m][e] = -INFINITY;
            }
        }
      }
      const float h0 = fmaxf(fmaxf(z[0][0], z[0][2]), fmaxf(z[1][0], z[1][2])), h1 = fmaxf(fmaxf(z[0][1], z[0][3]), fmaxf(z[1][1], z[1][3]));
      if (__any_sync(0xffffffffu, fmaxf(h0, h1) > kMoveAt)) {  // a row's reference moves
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float high = i ? h1 : h0, top = -INFINITY;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = i; e < 4; e += 2)
              if (z[m][e] != -INFINITY) top = fmaxf(top, fmaf(S[n][m][e], t.f, t.ev));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
          }
          if (high > kMoveAt) {
            const float to = top - kRoom, a = ex2(ref[n][i] - to), base_to = t.ev - to;
            ref[n][i] = to;
            l[n][i] *= a;
#pragma unroll
            for (int c = 0; c < 8; ++c) O[n][c][i] *= a, O[n][c][2 + i] *= a;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int e = i; e < 4; e += 2)
                if (z[m][e] != -INFINITY) z[m][e] = fmaf(S[n][m][e], t.f, base_to);
          }
        }
      }
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float a = ex2(z[m][2 * o]), b = ex2(z[m][2 * o + 1]);
          sum[0] += a;
          sum[1] += b;
          const __half2 h = __floats2half2_rn(a, b);
          w[0][n][m][o] = transposed(as_word(h));
          if constexpr (kParts == 2) {
            const float2 back = __half22float2(h);
            w[1][n][m][o] = transposed(pack_halves(a - back.x, b - back.y));
          }
        }
      l[n][0] = fmaf(sum[0], t.inv_v, l[n][0]);
      l[n][1] = fmaf(sum[1], t.inv_v, l[n][1]);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        uint32_t even[2][2], odd[2][2];
        value_halves(t.V, lane, kk, c, even, odd);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t a[4] = {even[u][0], odd[u][0], even[u][1], odd[u][1]};
#pragma unroll
          for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(O[n][c + u], a, w[part][n][kk][0], w[part][n][kk][1]);
        }
      }
  }
  __device__ __forceinline__ void spoil() {
#pragma unroll
    for (int n = 0; n < NT; ++n) l[n][0] = l[n][1] = NAN;
  }
  __device__ __forceinline__ void close() {  // the lanes' sums of weights
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], o);
  }
  // Place of a row's four channels u among its 32 in the join (stores of several rows at
  // once spread over the banks).
  static __device__ __forceinline__ int place(int r, int u) { return u ^ (r >> 1 & 3) << 2; }
  __device__ __forceinline__ void dump(float4 (*join)[32], float2* ml, int lane) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * n + 2 * tq + i;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          reinterpret_cast<float2*>(&join[r][place(r, 4 * c + (gq >> 1))])[gq & 1] = make_float2(O[n][c][i], O[n][c][2 + i]);
        if (gq == 0) ml[r] = make_float2(ref[n][i], l[n][i]);
      }
  }
  __device__ __forceinline__ void put(const BlockAttnParams& p, const BlockSegment& s, int row0, int lane) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + 8 * n + 2 * tq + i;
        if (r >= s.rows) continue;
        const float inv = l[n][i] == 0.0f ? 0.0f : 1.0f / l[n][i];
        const size_t row = row_at(p, s, r);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint32_t*>(p.out + row * kHeadDim + 16 * c + 2 * gq) = pack_halves(O[n][c][i] * inv, O[n][c][2 + i] * inv);
        if (p.lse && gq == 0) p.lse[row] = log_sum(ref[n][i], l[n][i]);
      }
  }
};

}  // namespace tile
}  // namespace kvq
