// kvq_block_tile.cuh -- one warp's arithmetic on a tile (a block of 32 tokens of a KV
// head) for the block attention: Rows8 for up to 8 (token, query head) rows,
// RowsWide<MT> for 16 MT.
//
// With y_rt = scale log2(e) 2^ek (q_r . c_t) + ev and w_rt = 2^(y_rt - ref_r) both keep
// per row ref, l = sum 2^-ev w and O = sum w c'.  Codes become fp16 in registers (e4m3
// is a subset); weights go up to 2^12 at a new reference and to 2^15 before it moves
// (fp16 ends at 2^16).
//
// Rows8 puts the tokens on the product's 16 rows and the query rows on its 8 columns
// (S^T = K Q^T, O^T = V^T P^T): 32 matrix instructions a tile, no padding, half the
// exponentials, 32 accumulators.  Its weights enter in two fp16 parts (22 bits; 16
// instructions more), which brings the output to its own rounding's error (2.1e-4
// normwise against 64 bits; one part: 2.6e-4).  RowsWide puts 16 query rows on the
// rows (64 instructions a tile and row tile), its weights in one part; with MT 2 the
// conversions serve both row tiles.
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
  int window, n_first;
  __device__ __forceinline__ bool seen(int t, int pos) const { return t <= pos && (pos - t < window || t < n_first); }
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

// ------------------------------------------------------------------- up to 8 rows
// Lane (gq, tq): rows 2 tq, 2 tq + 1 of the results, row gq of the queries.
struct Rows8 {
  static constexpr int kRows = 8, kPhases = 1;
  static constexpr bool kQueriesAhead = true;
  uint32_t q[8][2];
  float O[8][4], ref[2], l[2];  // O[c]: channels 16 c + 2 gq (+ 1 in the last two), rows 2 tq, 2 tq + 1
  int see[2];                   // last position that a row sees

  // Channel 32 tq + 4 k + {0, 1 | 2, 3} enters step k of the product as 2 tq + {0, 1 | 8, 9}.
  __device__ __forceinline__ void load_q(const BlockAttnParams& p, const BlockSegment& s, int, int lane, uint4*) {
    const int r = min(lane >> 2, s.rows - 1);  // (rows that are not there: the last one again)
    const uint4* src = reinterpret_cast<const uint4*>(p.q + row_at(p, s, r) * kHeadDim + 32 * (lane & 3));
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = __ldg(src + u);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k][0] = w[2 * k], q[k][1] = w[2 * k + 1];
  }
  __device__ __forceinline__ void begin(const BlockAttnParams& p, const BlockSegment& s, int, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ref[i] = -INFINITY;
      l[i] = 0.0f;
      see[i] = s.before + token_at(p, s, min(2 * (lane & 3) + i, s.rows - 1));
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) O[c][0] = O[c][1] = O[c][2] = O[c][3] = 0.0f;
  }
  __device__ __forceinline__ void tile(const Tile& t, int lane, int, const uint4*) {
    const int gq = lane >> 2, tq = lane & 3;
    float S[2][4];  // tokens 16 m + gq, + 8 (the last two), rows 2 tq, 2 tq + 1
#pragma unroll
    for (int m = 0; m < 2; ++m) S[m][0] = S[m][1] = S[m][2] = S[m][3] = 0.0f;
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
          mma16816(S[m], a, q[4 * half + k][0], q[4 * half + k][1]);
        }
    }
    float z[2][4];
    const float base[2] = {t.ev - ref[0], t.ev - ref[1]};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[m][e] = fmaf(S[m][e], t.f, base[e & 1]);
    if (t.masked) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!t.seen(t.t0 + 16 * m + gq + 8 * (e >> 1), see[e & 1])) z[m][e] = -INFINITY;
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
            if (z[m][e] != -INFINITY) top = fmaxf(top, fmaf(S[m][e], t.f, t.ev));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
        }
        if (high > kMoveAt) {
          const float to = top - kRoom, a = ex2(ref[i] - to), base_to = t.ev - to;
          ref[i] = to;
          l[i] *= a;
#pragma unroll
          for (int c = 0; c < 8; ++c) O[c][i] *= a, O[c][2 + i] *= a;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = i; e < 4; e += 2)
              if (z[m][e] != -INFINITY) z[m][e] = fmaf(S[m][e], t.f, base_to);
        }
      }
    }
    float sum[2] = {0.0f, 0.0f};
    uint32_t hi[2][2], lo[2][2];  // weights of 16 tokens, as the product's columns
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const float a = ex2(z[m][2 * o]), b = ex2(z[m][2 * o + 1]);
        sum[0] += a;
        sum[1] += b;
        const __half2 h = __floats2half2_rn(a, b);
        const float2 back = __half22float2(h);
        hi[m][o] = transposed(as_word(h));
        lo[m][o] = transposed(pack_halves(a - back.x, b - back.y));
      }
    l[0] = fmaf(sum[0], t.inv_v, l[0]);
    l[1] = fmaf(sum[1], t.inv_v, l[1]);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        uint32_t even[2][2], odd[2][2];
        value_halves(t.V, lane, kk, c, even, odd);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t a[4] = {even[u][0], odd[u][0], even[u][1], odd[u][1]};
          mma16816(O[c + u], a, hi[kk][0], hi[kk][1]);
          mma16816(O[c + u], a, lo[kk][0], lo[kk][1]);
        }
      }
  }
  __device__ __forceinline__ void spoil() { l[0] = l[1] = NAN; }
  __device__ __forceinline__ void close() {  // the lanes' sums of weights
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  }
  // Place of a row's four channels u among its 32 in the join (stores of several rows at
  // once spread over the banks).
  static __device__ __forceinline__ int place(int r, int u) { return u ^ (r >> 1 & 3) << 2; }
  __device__ __forceinline__ void dump(int, float4 (*join)[32], float2* ml, int lane, int) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * tq + i;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        reinterpret_cast<float2*>(&join[r][place(r, 4 * c + (gq >> 1))])[gq & 1] = make_float2(O[c][i], O[c][2 + i]);
      if (gq == 0) ml[r] = make_float2(ref[i], l[i]);
    }
  }
  __device__ __forceinline__ void put(const BlockAttnParams& p, const BlockSegment& s, int, int lane) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * tq + i;
      if (r >= s.rows) continue;
      const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
      const size_t row = row_at(p, s, r);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint32_t*>(p.out + row * kHeadDim + 16 * c + 2 * gq) = pack_halves(O[c][i] * inv, O[c][2 + i] * inv);
      if (p.lse && gq == 0) p.lse[row] = log_sum(ref[i], l[i]);
    }
  }
};

// ------------------------------------------------------------------ 16 MT rows
// Lane (gq, tq): rows 16 m + gq, + 8 of the results and of the queries.
template <int MT>
struct RowsWide {
  static constexpr int kRows = 16 * MT, kPhases = MT;
  static constexpr bool kQueriesAhead = MT == 1;
  uint32_t qa[MT == 1 ? 8 : 1][4];  // MT 2: in shared memory, [tile][step][lane], each lane's own words
  float O[MT][8][2][4], ref[MT][2], l[MT][2];
  int see[MT][2];

  __device__ __forceinline__ void load_q(const BlockAttnParams& p, const BlockSegment& s, int row0, int lane, uint4* q_mine) {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint4 v[2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = min(row0 + m * 16 + gq + 8 * hf, s.rows - 1);  // (rows that are not there: the last one again)
        const uint4* src = reinterpret_cast<const uint4*>(p.q + row_at(p, s, r) * kHeadDim + 32 * tq);
#pragma unroll
        for (int u = 0; u < 4; ++u) v[hf][u] = __ldg(src + u);
      }
      const uint32_t *lo = reinterpret_cast<const uint32_t*>(v[0]), *hi = reinterpret_cast<const uint32_t*>(v[1]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (MT == 1) {
          qa[k][0] = lo[2 * k], qa[k][1] = hi[2 * k], qa[k][2] = lo[2 * k + 1], qa[k][3] = hi[2 * k + 1];
        } else {
          q_mine[(m * 8 + k) * 32 + lane] = make_uint4(lo[2 * k], hi[2 * k], lo[2 * k + 1], hi[2 * k + 1]);
        }
      }
    }
  }
  __device__ __forceinline__ void begin(const BlockAttnParams& p, const BlockSegment& s, int row0, int lane) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        ref[m][hf] = -INFINITY;
        l[m][hf] = 0.0f;
        see[m][hf] = s.before + token_at(p, s, min(row0 + 16 * m + (lane >> 2) + 8 * hf, s.rows - 1));
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) O[m][c][e >> 2][e & 3] = 0.0f;
    }
  }
  // rows: from this warp's first one on
  __device__ __forceinline__ void tile(const Tile& t, int lane, int rows, const uint4* q_mine) {
    const int gq = lane >> 2, tq = lane & 3;
    float S[MT][4][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[m][j][0] = S[m][j][1] = S[m][j][2] = S[m][j][3] = 0.0f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // of the channels
      uint4 kc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        kc[j] = *reinterpret_cast<const uint4*>(t.K + (8 * j + gq) * kHeadDim + (((2 * tq + half) ^ gq) << 4));
#pragma unroll
      for (int k = 4 * half; k < 4 * half + 4; ++k) {
        uint32_t a[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (MT == 1) {
            a[m][0] = qa[k][0], a[m][1] = qa[k][1], a[m][2] = qa[k][2], a[m][3] = qa[k][3];
          } else {
            const uint4 q = q_mine[(m * 8 + k) * 32 + lane];
            a[m][0] = q.x, a[m][1] = q.y, a[m][2] = q.z, a[m][3] = q.w;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b0, b1;
          e4m3_halves(reinterpret_cast<const uint32_t*>(&kc[j])[k & 3], b0, b1);
#pragma unroll
          for (int m = 0; m < MT; ++m) mma16816(S[m][j], a[m], b0, b1);
        }
      }
    }
    uint32_t pa[MT][2][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (16 * m + 8 * hf >= rows) {  // no such rows
          pa[m][0][hf] = pa[m][0][2 + hf] = pa[m][1][hf] = pa[m][1][2 + hf] = 0;
          continue;
        }
        float z[4][2];
        const float base = t.ev - ref[m][hf];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[j][0] = fmaf(S[m][j][2 * hf], t.f, base);
          z[j][1] = fmaf(S[m][j][2 * hf + 1], t.f, base);
        }
        if (t.masked) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!t.seen(t.t0 + 8 * j + 2 * tq + e, see[m][hf])) z[j][e] = -INFINITY;
        }
        float high = fmaxf(z[0][0], z[0][1]);
#pragma unroll
        for (int j = 1; j < 4; ++j) high = fmaxf(high, fmaxf(z[j][0], z[j][1]));
        if (__any_sync(0xffffffffu, high > kMoveAt)) {  // a row's reference moves
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (z[j][e] != -INFINITY) top = fmaxf(top, fmaf(S[m][j][2 * hf + e], t.f, t.ev));
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
          }
          if (high > kMoveAt) {
            const float to = top - kRoom, a = ex2(ref[m][hf] - to), base_to = t.ev - to;
            ref[m][hf] = to;
            l[m][hf] *= a;
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                O[m][c][q][2 * hf] *= a;
                O[m][c][q][2 * hf + 1] *= a;
              }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (z[j][e] != -INFINITY) z[j][e] = fmaf(S[m][j][2 * hf + e], t.f, base_to);
          }
        }
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[j][0] = ex2(z[j][0]);
          z[j][1] = ex2(z[j][1]);
          sum += z[j][0] + z[j][1];
          pa[m][j >> 1][2 * (j & 1) + hf] = pack_halves(z[j][0], z[j][1]);
        }
        l[m][hf] = fmaf(sum, t.inv_v, l[m][hf]);
      }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        uint32_t even[2][2], odd[2][2];
        value_halves(t.V, lane, kk, c, even, odd);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma16816(O[m][c + u][0], pa[m][kk], even[u][0], even[u][1]);
            mma16816(O[m][c + u][1], pa[m][kk], odd[u][0], odd[u][1]);
          }
      }
  }
  __device__ __forceinline__ void spoil() {
#pragma unroll
    for (int m = 0; m < MT; ++m) l[m][0] = l[m][1] = NAN;
  }
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) l[m][hf] += __shfl_xor_sync(0xffffffffu, l[m][hf], o);
  }
  static __device__ __forceinline__ int place(int r, int u) { return u ^ (r & 1) << 2; }
  __device__ __forceinline__ void dump(int m_, float4 (*join)[32], float2* ml, int lane, int rows) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (m != m_ || 16 * m + 8 * hf >= rows) continue;
        const int r = gq + 8 * hf;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float(&o)[2][4] = O[m][c];
          join[r][place(r, 4 * c + tq)] = make_float4(o[0][2 * hf], o[1][2 * hf], o[0][2 * hf + 1], o[1][2 * hf + 1]);
        }
        if (tq == 0) ml[r] = make_float2(ref[m][hf], l[m][hf]);
      }
  }
  __device__ __forceinline__ void put(const BlockAttnParams& p, const BlockSegment& s, int row0, int lane) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = row0 + 16 * m + gq + 8 * hf;
        if (r >= s.rows) continue;
        const float inv = l[m][hf] == 0.0f ? 0.0f : 1.0f / l[m][hf];
        const size_t row = row_at(p, s, r);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float(&o)[2][4] = O[m][c];
          *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 16 * c + 4 * tq) =
              make_uint2(pack_halves(o[0][2 * hf] * inv, o[1][2 * hf] * inv), pack_halves(o[0][2 * hf + 1] * inv, o[1][2 * hf + 1] * inv));
        }
        if (p.lse && tq == 0) p.lse[row] = log_sum(ref[m][hf], l[m][hf]);
      }
  }
};

}  // namespace tile
}  // namespace kvq
