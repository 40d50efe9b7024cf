// kvq_tree.cuh -- parameters, work split and tile producers of the operators
// that run many query rows per KV head over the cache: kvq_tree_attn (a tree
// of drafted tokens) and kvq_attn_mass (accumulated attention weight).
//
// Both cut a stream's tokens into tiles of 128 keys.  A tile is either
// quantized (positions [S, S + Nq)) or fp16 (sinks, window, then the drafted
// tokens).  A tile's keys are dequantized once into shared memory and used
// by every query row.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr int kTile = 128;          // keys per tile
constexpr int kMaxTreeNodes = 256;  // drafted tokens per sequence
constexpr int kMaxSpecCtas = 160;   // CTAs of the tile kernels, one per SM at most (bounds the workspace)

// Work of one call, planned on the host.  Rows of KV head h, batch row b:
// r = j * nodes[b] + i for query head j of the group and node i; they are cut
// into blocks of `rblk`.  The tiles of (b, h, row block), quantized ones first,
// are laid end to end in that order and cut into ncta equal ranges; a range
// covers one or more pieces, a piece being the part of an item (b, h, row
// block, kind) that one CTA handles.  Piece p of CTA c on item e writes its
// partial softmax to slot c + e: slots along the line strictly increase.
struct SpecRows {
  int tokens[kMaxRaggedRows];
  int nodes[kMaxRaggedRows];
  int tile0[kMaxRaggedRows + 1];  // first tile of batch row b
  int pair0[kMaxRaggedRows + 1];  // first (h, row block) pair of batch row b
};

struct TreeParams {
  Geometry geo;
  LayerPtrs L;
  const uint16_t* q;
  const uint16_t* kd;
  const uint16_t* vd;
  const uint32_t* mask;  // [B][n][words] or null (no drafted keys)
  uint16_t* out;
  float* lse;
  float2* part_ml;    // [slots][sub][rstride] (maximum in log2 units, sum)
  float* part_acc;    // [slots][sub][rstride][d]
  uint32_t* part_flag;  // [slots][sub] a drafted value of the piece is not finite
  int n, words;       // nodes per sequence (the inputs' stride), mask words per node
  int rblk, sub;      // rows per block; partial results per piece
  int rstride;        // rows of a partial result
  int ncta, total;    // CTAs, tiles
  float q_scale;      // softmax scale * log2(e)
  float hadamard_c;
  float k_lut_off[8], v_lut_off[8];
  double theta[kHeadDim / 2];               // RoPE radians per position
  unsigned long long freq[kHeadDim / 2];    // RoPE turns per position, 64-bit fractions
  SpecRows rows;
};

struct MassParams {
  Geometry geo;
  LayerPtrs L;
  const uint16_t* q;     // [B][Hq][n][d]
  const float* lse;      // [B][Hq][n]
  const float* weight;   // [B][n] or null
  float* mass;           // [NS][cap]
  int n, cap;            // query rows per sequence, tokens per stream of the record
  int ncta, total;       // CTAs, tiles
  float decay, q_scale;  // q_scale: the softmax scale
  float k_lut_off[8];
  double theta[kHeadDim / 2];
  unsigned long long freq[kHeadDim / 2];
  SpecRows rows;
};

// Tiles of a (b, h, row block): quantized, fp16.
struct TileCounts {
  int S_eff, Nq, W, k1;  // sinks present, quantized tokens, window tokens, fp16 tokens (sinks + window)
  int qt, ft;            // quantized and fp16 tiles
};
__host__ __device__ inline TileCounts tile_counts(const Geometry& G, int T, int drafted) {
  TileCounts c;
  window_counts(G, T, &c.S_eff, &c.Nq, &c.W);
  c.k1 = c.S_eff + c.W;
  c.qt = (c.Nq + kTile - 1) / kTile;
  c.ft = (c.k1 + drafted + kTile - 1) / kTile;
  return c;
}
__host__ __device__ inline int cta_first_tile(int ncta, int total, int i) { return (int)((long long)i * total / ncta); }
// The CTA whose range holds tile t.
__host__ __device__ inline int tile_owner(int ncta, int total, int t) {
  return (int)((((long long)t + 1) * ncta - 1) / total);
}
// The last row whose first entry is <= v (entries do not decrease; rows
// without work share their entry with the next row and are skipped).
__host__ __device__ inline int row_of(const int* tab, int rows, int v) {
  int lo = 0, hi = rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab[mid] <= v) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Keys with a scale per channel and group that the tile kernels take apart
// (kvq_fill.cuh: keys_channel).
__host__ __device__ inline bool channel_scales(const Geometry& G) { return !G.pre_rope && G.kb != 3 && !G.gkc && !G.fp16_mode; }

#ifdef __CUDACC__

// Byte offset of channel c of key t in a tile: two halves of 64 channels,
// rows of 128 bytes whose 16-byte chunks are XOR-swizzled by the row (the
// 128-byte swizzle of the tensor cores' shared-memory operands; ldmatrix
// reads of 8 rows touch distinct banks too).
__device__ __forceinline__ uint32_t tile_off(int t, int chunk /* c / 8 */) {
  return (uint32_t)((chunk >> 3) * (kTile * 128) + t * 128 + (((chunk & 7) ^ (t & 7)) << 4));
}

// e^{i x} for an fp64 angle: reduced modulo 2 pi in fp64, then fp32.
__device__ __forceinline__ float2 spec_expi(double x) {
  const double turns = x * 0.15915494309189533576888376337251;
  float sn, cs;
  sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
  return make_float2(cs, sn);
}
__device__ __forceinline__ float2 spec_cmul(float2 a, float2 b) {
  return make_float2(a.x * b.x - a.y * b.y, a.x * b.y + a.y * b.x);
}

// The 8 codes of one 8-channel chunk of a packed row, as integers.
__device__ __forceinline__ void chunk_codes(const uint8_t* row, int bits, int chunk, int (&c)[8]) {
  if (bits == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + chunk * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = (w.x >> (8 * i)) & 255, c[4 + i] = (w.y >> (8 * i)) & 255;
  } else if (bits == 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(row + chunk * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = (w >> (4 * i)) & 15;
  } else if (bits == 2) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(row + chunk * 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = (w >> (2 * i)) & 3;
  } else {  // 3 bits: 3 bytes, at no particular alignment
    const uint8_t* b = row + chunk * 3;
    const uint32_t w = (uint32_t)b[0] | ((uint32_t)b[1] << 8) | ((uint32_t)b[2] << 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = (w >> (3 * i)) & 7;
  }
}

// Outliers of one token that fall into an 8-channel chunk replace its values.
__device__ __forceinline__ void chunk_outliers(const uint8_t* col, const uint16_t* val, int k, int chunk, float (&x)[8]) {
  for (int j = 0; j < k; ++j) {
    const int o = (int)col[j] - 8 * chunk;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i == o) x[i] = half_bits_to_float(val[j]);
  }
}

// Dequantized channels [8 chunk, 8 chunk + 8) of quantized key i of stream s.
__device__ __forceinline__ void k_chunk(const Geometry& G, const LayerPtrs& L, const float* lut_off, int s, int i, int chunk,
                                        float (&x)[8]) {
  const size_t tok = (size_t)s * G.qcap + i;
  int c[8];
  chunk_codes(L.k_codes + tok * G.krow, G.kb, chunk, c);
  if (G.kb == 3) {
    const float2 ms = unpack_min_scale(L.k_scales[tok]);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf(ms.y, lut_off[c[j]], ms.x);
    chunk_outliers(L.k_col + tok * G.nout, L.k_val + tok * G.nout, G.nout, chunk, x);
  } else if (G.gkc) {
    const float2 ms = unpack_min_scale(L.k_scales[tok * G.nkg + 8 * chunk / G.gkc]);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf((float)c[j], ms.y, ms.x);
    if (G.knorm)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= L.k_norm[(size_t)s * kHeadDim + 8 * chunk + j];
  } else {
    const uint32_t* sc = L.k_scales + ((size_t)s * G.gcap + i / kGroupTokens) * kHeadDim + 8 * chunk;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 ms = unpack_min_scale(sc[j]);
      x[j] = fmaf((float)c[j], ms.y, ms.x);
    }
  }
}

// The same of value i (in the rotated domain when V is Hadamard-rotated).
__device__ __forceinline__ void v_chunk(const Geometry& G, const LayerPtrs& L, const float* lut_off, int s, int i, int chunk,
                                        float (&x)[8]) {
  const size_t tok = (size_t)s * G.qcap + i;
  int c[8];
  chunk_codes(L.v_codes + tok * G.vrow, G.vb, chunk, c);
  if (G.vb == 3) {
    const float2 ms = unpack_min_scale(L.v_scales[tok]);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf(ms.y, lut_off[c[j]], ms.x);
    chunk_outliers(L.v_col + tok * G.nout, L.v_val + tok * G.nout, G.nout, chunk, x);
  } else {
    const float2 ms = unpack_min_scale(L.v_scales[tok * G.nvg + 8 * chunk / G.gv]);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf((float)c[j], ms.y, ms.x);
  }
}

// fp16 key f of a stream (f < k1): its row in the sinks or the window ring,
// and its position in the sequence.
__device__ __forceinline__ const uint16_t* fp16_row(const Geometry& G, const uint16_t* sink, const uint16_t* ring, int s,
                                                    const TileCounts& tc, int f, int* pos) {
  if (f < tc.S_eff) {
    *pos = f;
    return sink + ((size_t)s * G.S + f) * kHeadDim;
  }
  const int t = G.S + tc.Nq + (f - tc.S_eff);  // window token (f >= S_eff only when all S sinks are present)
  *pos = t;
  return ring + ((size_t)s * G.ring + (t - G.S) % G.ring) * kHeadDim;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint4 r;
  __half2 h;
  h = __floats2half2_rn(x[0], x[1]), r.x = *reinterpret_cast<uint32_t*>(&h);
  h = __floats2half2_rn(x[2], x[3]), r.y = *reinterpret_cast<uint32_t*>(&h);
  h = __floats2half2_rn(x[4], x[5]), r.z = *reinterpret_cast<uint32_t*>(&h);
  h = __floats2half2_rn(x[6], x[7]), r.w = *reinterpret_cast<uint32_t*>(&h);
  return r;
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
// x as hi + lo fp16 parts: 22 bits of x (hi saturates at the fp16 range, the
// lo part takes what is left).
__device__ __forceinline__ void split8(const float (&x)[8], uint4* hi, uint4* lo) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = fminf(fmaxf(x[i], -65504.0f), 65504.0f);
  *hi = pack8(a);
  unpack8(*hi, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = x[i] - b[i];
  *lo = pack8(b);
}
__device__ __forceinline__ bool finite8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) ok = ok && (w[i] & 0x7C00u) != 0x7C00u && (w[i] & 0x7C000000u) != 0x7C000000u;
  return ok;
}

#endif  // __CUDACC__

cudaError_t launch_tree_attn(const TreeParams& p, cudaStream_t st);
cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t st);
cudaError_t launch_attn_mass(const MassParams& p, cudaStream_t st);

}  // namespace kvq
