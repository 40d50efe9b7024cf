// kvq_tree.cuh -- parameters, work split and tile producers of the operators
// that run many query rows per KV head over the cache: kvq_tree_attn (a tree
// of drafted tokens) and kvq_attn_mass (accumulated attention weight).
//
// Both cut a stream's tokens into tiles of 96 keys (three groups: two stages
// of a dequantized tile and three of its stored bytes fit shared memory).  A tile is either
// quantized (positions [S, S + Nq)) or fp16 (sinks, window, then the drafted
// tokens).  A tile's keys are dequantized once into shared memory and used
// by every query row.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr int kTile = 96;           // keys per tile
constexpr int kTileRows = 128;      // query rows of the tensor-core kernel
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

// Stored bytes of a quantized tile as copied into shared memory: byte offsets
// of its parts within a slot, and how many slots there are (2..kMaxRaw).
// Non-uniform codes are looked up two at a time: behind the slots lie the
// level pairs of K, then of V, in 16 copies, one per bank pair of a half-warp.
constexpr int kMaxRaw = 4;
constexpr int kLevelPairBytes = 64 * 16 * 8;
struct RawSlot {
  int slots, bytes, pairs;
  int ks, kcol, kval, v, vs, vcol, vval;  // K codes at 0
};
inline RawSlot raw_slot(const Geometry& G, bool values, int room) {
  RawSlot r;
  int off = kTile * G.krow;
  auto put = [&](int bytes) {
    const int at = off;
    off += (bytes + 15) / 16 * 16;
    return at;
  };
  r.ks = put(G.kb == 3 ? kTile * 4 : G.gkc ? kTile * G.nkg * 4 : kTile / kGroupTokens * kHeadDim * 4);
  r.kcol = put(kTile * G.nout);
  r.kval = put(kTile * G.nout * 2);
  r.v = put(values ? kTile * G.vrow : 0);
  r.vs = put(values ? kTile * (G.vb == 3 ? 1 : G.nvg) * 4 : 0);
  r.vcol = put(values ? kTile * G.nout : 0);
  r.vval = put(values ? kTile * G.nout * 2 : 0);
  r.bytes = (off + 127) / 128 * 128;
  if (G.kb == 3) room -= (values ? 2 : 1) * kLevelPairBytes;
  r.slots = room / (r.bytes > 0 ? r.bytes : 1);
  r.slots = r.slots > kMaxRaw ? kMaxRaw : r.slots < 2 ? 2 : r.slots;
  r.pairs = r.slots * r.bytes;
  return r;
}

// Shared memory behind a kernel's fixed part.
inline uint32_t raw_bytes(const Geometry& G, const RawSlot& r, bool values) {
  return r.pairs + (G.kb == 3 ? (values ? 2 : 1) * kLevelPairBytes : 0);
}

struct TreeParams {
  Geometry geo;
  LayerPtrs L;
  const uint16_t* q;
  const uint16_t* kd;
  const uint16_t* vd;
  const uint32_t* mask;  // [B][n][words] or null (no drafted keys)
  uint16_t* out;
  float* lse;
  // the record of attention weight: rows' log-sum-exp and weights, [NS][cap] entries
  const float* row_lse;
  const float* weight;
  float* mass;
  float decay;
  int cap;
  int r0, nr;          // rows of a KV head in this pass
  float2* part_ml;    // [slots][sub][rstride] (maximum in log2 units, sum)
  float* part_acc;    // [slots][sub][rstride][d]
  uint32_t* part_flag;  // [slots][sub] a drafted value of the piece is not finite
  int n, words;       // nodes per sequence (the inputs' stride), mask words per node
  int rblk, sub;      // rows per block; partial results per piece
  int rstride;        // rows of a partial result
  int ncta, total;    // CTAs, tiles
  RawSlot raw;        // stored bytes of a tile in shared memory
  float q_scale;      // softmax scale * log2(e) (the record: the softmax scale)
  float hadamard_c;
  float k_lut_off[8], v_lut_off[8];
  unsigned long long freq[kHeadDim / 2];    // RoPE turns per position, 64-bit fractions
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

// Where the merge finds the partial results of one kind (0: quantized tiles,
// 1: fp16 tiles) of a (b, h, row block): n of them, consecutive in (slot, sub).
struct PartSpan {
  size_t at;
  int n;
};
__host__ __device__ inline PartSpan part_span(const TreeParams& p, const TileCounts& tc, int b, int pair, int kind) {
  const int tiles = kind ? tc.ft : tc.qt;
  if (!tiles) return PartSpan{0, 0};
  const int first = p.rows.tile0[b] + pair * (tc.qt + tc.ft) + (kind ? tc.qt : 0);
  const int c0 = tile_owner(p.ncta, p.total, first), c1 = tile_owner(p.ncta, p.total, first + tiles - 1);
  return PartSpan{(size_t)(c0 + 2 * (p.rows.pair0[b] + pair) + kind) * p.sub, (c1 - c0 + 1) * p.sub};
}
// Whether a partial result of an fp16 piece names drafted values that are not
// finite.  A piece whose CTA gave up has NaN in ml and no flag written: its flag
// is whatever the scratch held and says nothing.
__host__ __device__ inline bool names_drafted(const TreeParams& p, float2 ml, uint32_t flag) {
  return p.mask && ml.x == ml.x && flag;
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

// The 8 uniform codes of one 8-channel chunk of a packed row, as integers.
__device__ __forceinline__ void chunk_codes(const uint8_t* row, int bits, int chunk, int (&c)[8]) {
  if (bits == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + chunk * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = (w.x >> (8 * i)) & 255, c[4 + i] = (w.y >> (8 * i)) & 255;
  } else if (bits == 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(row + chunk * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = (w >> (4 * i)) & 15;
  } else {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(row + chunk * 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = (w >> (2 * i)) & 3;
  }
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
__device__ __forceinline__ bool finite8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) ok = ok && (w[i] & 0x7C00u) != 0x7C00u && (w[i] & 0x7C000000u) != 0x7C000000u;
  return ok;
}

#endif  // __CUDACC__

// (they place the stored bytes of a tile in shared memory: p.raw)
cudaError_t launch_tree_attn(TreeParams& p, cudaStream_t st);
cudaError_t launch_tree_tc(TreeParams& p, cudaStream_t st);
cudaError_t launch_attn_mass(TreeParams& p, cudaStream_t st);
bool mass_stream_eligible(const Geometry& G);
cudaError_t launch_mass_stream(const TreeParams& t, cudaStream_t st);

}  // namespace kvq
