// kvq_fill.cuh -- dequantization of 128-key tiles into the shared-memory
// operands of the matrix instructions (kvq_tree_tc.cu, kvq_mass.cu): keys as
// hi + lo fp16 parts (22 bits), values as fp16, rows of 128 bytes with the
// 128-byte swizzle (tile_off).
//
// 256 threads fill a tile.  The raw codes and scales of a tile are read into
// registers first (load) and converted later (keys, values), so that a tile's
// loads are in flight while the one before it is waited for.
//
// Two mappings.  Uniform codes without RoPE: a thread owns 8 channels of 8
// consecutive keys (of one group: a channel's scale is read once for 8
// codes).  Non-uniform codes and keys cached before RoPE: a thread owns 8
// channel pairs (c, c + 64) of 4 consecutive keys.
#pragma once

#include "kvq_tree.cuh"

namespace kvq {

#ifdef __CUDACC__

// 1024 + x by the fp16 exponent, then the offset leaves: exact integers.
__device__ __forceinline__ uint32_t lop_and_or(uint32_t a, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(r) : "r"(a), "r"(mask), "r"(magic));
  return r;
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ __half2 h2_const(uint16_t bits) {
  return __halves2half2(__ushort_as_half(bits), __ushort_as_half(bits));
}

// The 8 codes of a chunk as fp16 pairs, less 2^(BITS - 1) when CENTRED.  Pair
// i holds channels (2 i, 2 i + 1) for 8-bit codes and (i, i + 4) for 4- and
// 2-bit codes (one mask takes both out of a word): the operands' channel
// order within a chunk.
template <int BITS, bool CENTRED = false>
__device__ __forceinline__ void code_pairs(uint2 w, __half2 (&c)[4]) {
  if constexpr (BITS == 8) {
    const __half2 off = h2_const(CENTRED ? 0x6480 : 0x6400);  // 1024 (+ 128)
    c[0] = __hsub2(as_h2(__byte_perm(w.x, 0x64646464u, 0x4140u)), off);
    c[1] = __hsub2(as_h2(__byte_perm(w.x, 0x64646464u, 0x4342u)), off);
    c[2] = __hsub2(as_h2(__byte_perm(w.y, 0x64646464u, 0x4140u)), off);
    c[3] = __hsub2(as_h2(__byte_perm(w.y, 0x64646464u, 0x4342u)), off);
  } else if constexpr (BITS == 4) {
    const __half2 off = h2_const(CENTRED ? 0x6408 : 0x6400), k16th = h2_const(0x2C00);  // 1024 (+ 8)
    const __half2 off16 = h2_const(CENTRED ? 0xD480 : 0xD400);                            // -64 (- 8)
    c[0] = __hsub2(as_h2(lop_and_or(w.x, 0x000F000Fu, 0x64006400u)), off);
    c[1] = __hfma2(as_h2(lop_and_or(w.x, 0x00F000F0u, 0x64006400u)), k16th, off16);
    c[2] = __hsub2(as_h2(lop_and_or(w.x >> 8, 0x000F000Fu, 0x64006400u)), off);
    c[3] = __hfma2(as_h2(lop_and_or(w.x >> 8, 0x00F000F0u, 0x64006400u)), k16th, off16);
  } else {
    // 16 bits: channels 0..3 to the low half, 4..7 to the high half
    const uint32_t x = __byte_perm(w.x, 0, 0x4140u);
    c[0] = __hsub2(as_h2(lop_and_or(x, 0x00030003u, 0x64006400u)), h2_const(CENTRED ? 0x6402 : 0x6400));
    c[1] = __hfma2(as_h2(lop_and_or(x, 0x000C000Cu, 0x64006400u)), h2_const(0x3400), h2_const(CENTRED ? 0xDC08 : 0xDC00));  // /4 - 256 (- 2)
    c[2] = __hfma2(as_h2(lop_and_or(x, 0x00300030u, 0x64006400u)), h2_const(0x2C00), h2_const(CENTRED ? 0xD420 : 0xD400));  // /16 - 64 (- 2)
    c[3] = __hfma2(as_h2(lop_and_or(x, 0x00C000C0u, 0x64006400u)), h2_const(0x2400), h2_const(CENTRED ? 0xCC80 : 0xCC00));  // /64 - 16 (- 2)
  }
}
// Whether a chunk's channels are stored in the order 0 4 1 5 2 6 3 7.
__host__ __device__ inline bool paired_order(int bits) { return bits == 4 || bits == 2; }
__device__ __forceinline__ uint4 pair_chunk(const uint4& u) {
  return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                    __byte_perm(u.y, u.w, 0x7632));
}

__device__ __forceinline__ uint32_t pack_sat(float lo, float hi) {  // to fp16, saturating at its range (NaN stays)
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// x as its fp16 value and minus what is left of it: x = hi - neg.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t* hi, uint32_t* neg) {
  *hi = pack_sat(x0, x1);
  const float2 h = __half22float2(as_h2(*hi));
  *neg = as_u32(__floats2half2_rn(h.x - x0, h.y - x1));
}

// Turns of position pos at frequency f (turns per position as a 64-bit
// fraction): the product's wrap is the reduction, so the angle is exact to
// 2^-32 turns at every position below 2^31.
__device__ __forceinline__ float2 phasor(uint32_t pos, unsigned long long f) {
  const uint32_t turns = pos * (uint32_t)(f >> 32) + __umulhi(pos, (uint32_t)f);
  float sn, cs;
  sincospif((float)(int)turns * 4.656612873077393e-10f /* 2^-31: half turns */, &sn, &cs);
  return make_float2(cs, sn);
}

// Byte offset of a 16-byte chunk of row r among ROWS rows of 128 channels
// (two halves of 64 channels, swizzled like the tiles).
template <int ROWS>
__device__ __forceinline__ uint32_t q_off(int r, int chunk) {
  return (uint32_t)((chunk >> 3) * (ROWS * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
}

struct TileSrc {
  TileCounts tc;
  int s, b, n_b;      // stream, batch row, drafted tokens
  int slot0;          // ring slot of the window's first token
  size_t draft0;      // first row of the stream in k_draft / v_draft
};

// Raw codes and scales of a thread's share of a tile.
struct RawTile {
  uint2 k[8], v[8];
  uint32_t ks[8], vs[8];
};

// One load per key, without a branch between them: they are all in flight at
// once (a branch per load made each wait for the one before).
template <int BITS>
__device__ __forceinline__ void load_codes(const uint8_t* rows, int pitch, int chunk, uint2 (&c)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint8_t* row = rows + u * pitch;
    if constexpr (BITS == 8) c[u] = __ldg(reinterpret_cast<const uint2*>(row) + chunk);
    else if constexpr (BITS == 4) c[u].x = __ldg(reinterpret_cast<const uint32_t*>(row) + chunk);
    else c[u].x = __ldg(reinterpret_cast<const uint16_t*>(row) + chunk);
  }
}
__device__ __forceinline__ void load_codes(const uint8_t* rows, int bits, int chunk, uint2 (&c)[8]) {
  if (bits == 8) load_codes<8>(rows, 128, chunk, c);
  else if (bits == 4) load_codes<4>(rows, 64, chunk, c);
  else load_codes<2>(rows, 32, chunk, c);
}

// Uniform codes: the thread's loads of quantized tile kt.  Keys past the end
// are not read (Nq is a whole number of groups, so a thread's 8 keys are all
// there or none).
__device__ __forceinline__ void load_keys(const Geometry& G, const LayerPtrs& L, const TileSrc& src, int kt, int tid, RawTile& r) {
  const int cb = tid & 15, f = kt * kTile + (tid >> 4) * 8;
  if (f >= src.tc.Nq) return;
  const size_t tok = (size_t)src.s * G.qcap + f;
  load_codes(L.k_codes + tok * G.krow, G.kb, cb, r.k);
  if (G.gkc) {
    const uint32_t* sc = L.k_scales + tok * 2 + (cb >> 3);
#pragma unroll
    for (int u = 0; u < 8; ++u) r.ks[u] = __ldg(sc + 2 * u);
  } else {
    const uint4* sc = reinterpret_cast<const uint4*>(L.k_scales + ((size_t)src.s * G.gcap + f / kGroupTokens) * kHeadDim + 8 * cb);
    const uint4 a = __ldg(sc), b = __ldg(sc + 1);
    r.ks[0] = a.x, r.ks[1] = a.y, r.ks[2] = a.z, r.ks[3] = a.w;
    r.ks[4] = b.x, r.ks[5] = b.y, r.ks[6] = b.z, r.ks[7] = b.w;
  }
}
__device__ __forceinline__ void load_values(const Geometry& G, const LayerPtrs& L, const TileSrc& src, int kt, int tid, RawTile& r) {
  const int cb = tid & 15, f = kt * kTile + (tid >> 4) * 8;
  if (f >= src.tc.Nq) return;
  const size_t tok = (size_t)src.s * G.qcap + f;
  load_codes(L.v_codes + tok * G.vrow, G.vb, cb, r.v);
  const uint32_t* sc = L.v_scales + tok * G.nvg + 8 * cb / G.gv;
#pragma unroll
  for (int u = 0; u < 8; ++u) r.vs[u] = __ldg(sc + u * G.nvg);
}

// Ask for quantized tile kt in L2 (one thread): codes and scales of its keys
// are contiguous, whole multiples of 16 bytes.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  if (bytes)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(__cvta_generic_to_global(p)), "r"(bytes) : "memory");
}
template <bool V>
__device__ __forceinline__ void prefetch_tile(const Geometry& G, const LayerPtrs& L, const TileSrc& src, int kt) {
  const int f = kt * kTile, n = min(kTile, src.tc.Nq - f);  // whole groups
  if (n <= 0) return;
  const size_t tok = (size_t)src.s * G.qcap + f;
  prefetch_l2(L.k_codes + tok * G.krow, n * G.krow);
  if (G.kb == 3) prefetch_l2(L.k_scales + tok, n * 4);
  else if (G.gkc) prefetch_l2(L.k_scales + tok * G.nkg, n * G.nkg * 4);
  else prefetch_l2(L.k_scales + tok * (kHeadDim / kGroupTokens), n * (kHeadDim / kGroupTokens) * 4);
  if constexpr (V) {
    prefetch_l2(L.v_codes + tok * G.vrow, n * G.vrow);
    prefetch_l2(L.v_scales + tok * (G.vb == 3 ? 1 : G.nvg), n * (G.vb == 3 ? 1 : G.nvg) * 4);
  }
  if (G.kb == 3 && G.nout) {
    prefetch_l2(L.k_col + tok * G.nout, n * G.nout);
    prefetch_l2(L.k_val + tok * G.nout, n * G.nout * 2);
    if constexpr (V) {
      prefetch_l2(L.v_col + tok * G.nout, n * G.nout);
      prefetch_l2(L.v_val + tok * G.nout, n * G.nout * 2);
    }
  }
}

// Channel pair i of a chunk in the operands' order: the index of its first
// and second channel.
template <int BITS>
__device__ __forceinline__ constexpr int pair_a(int i) { return BITS == 8 ? 2 * i : i; }
template <int BITS>
__device__ __forceinline__ constexpr int pair_b(int i) { return BITS == 8 ? 2 * i + 1 : i + 4; }

// Keys of a uniform tile with a scale per channel and group of 32 tokens:
//   k = c' s + (m + 2^(b-1) s),  c' = code - 2^(b-1).
// The product c' s has 19 bits: its fp16 value hi and the rest neg = hi - c' s
// are exact.  The other part is the same for the 32 keys of a group, so it
// reaches the logits as one number per row and group, q . m + 2^(b-1) q . s:
// rows 0..3 of sM hold the tile's groups' m, rows 4..7 their s (8 rows of 128
// channels, q_off<8>).  Half the instructions of an fp32 k split in two.
template <int BITS>
__device__ __forceinline__ void keys_channel(bool have, int tid, const RawTile& r, uint8_t* sK, uint8_t* sN) {
  const int cb = tid & 15, t0 = (tid >> 4) * 8;
  __half2 sc[4];
  bool big = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sc[i] = as_h2(__byte_perm(r.ks[pair_a<BITS>(i)], r.ks[pair_b<BITS>(i)], 0x7632));
    const float2 f = __half22float2(sc[i]);
    big = big || fmaxf(fabsf(f.x), fabsf(f.y)) * (1 << (BITS - 1)) > 65504.0f;  // c' s may pass the fp16 range
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    uint32_t hi[4] = {0, 0, 0, 0}, neg[4] = {0, 0, 0, 0};
    if (have) {
      __half2 c[4];
      code_pairs<BITS, true>(r.k[u], c);
      if (!big) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = __hmul2(c[i], sc[i]);
          hi[i] = as_u32(h);
          neg[i] = as_u32(__hfma2(__hneg2(c[i]), sc[i], h));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = __half22float2(c[i]), b = __half22float2(sc[i]);
          split2(a.x * b.x, a.y * b.y, &hi[i], &neg[i]);
        }
      }
    }
    const uint32_t o = tile_off(t0 + u, cb);
    *reinterpret_cast<uint4*>(sK + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(sN + o) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
  }
}
template <int BITS>
__device__ __forceinline__ void group_rows(bool have, int tid, const RawTile& r, uint8_t* sM) {
  const int cb = tid & 15, tg = tid >> 4;
  if (tg & 3) return;  // the first of the group's four threads of a channel chunk
  uint32_t m[4] = {0, 0, 0, 0}, sc[4] = {0, 0, 0, 0};
  if (have)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = __byte_perm(r.ks[pair_a<BITS>(i)], r.ks[pair_b<BITS>(i)], 0x5410);
      sc[i] = __byte_perm(r.ks[pair_a<BITS>(i)], r.ks[pair_b<BITS>(i)], 0x7632);
    }
  *reinterpret_cast<uint4*>(sM + q_off<8>(tg >> 2, cb)) = make_uint4(m[0], m[1], m[2], m[3]);
  *reinterpret_cast<uint4*>(sM + q_off<8>(4 + (tg >> 2), cb)) = make_uint4(sc[0], sc[1], sc[2], sc[3]);
}

// Keys of a uniform tile with a scale per token and 64 channels (InnerQ):
// k = (min + code * scale) * norm in fp32, split into two fp16 parts.
template <int BITS>
__device__ __forceinline__ void keys_token(const Geometry& G, const LayerPtrs& L, int s, bool have, int tid, const RawTile& r,
                                           uint8_t* sK, uint8_t* sN) {
  const int cb = tid & 15, t0 = (tid >> 4) * 8;
  float norm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) norm[i] = G.knorm ? __ldg(L.k_norm + (size_t)s * kHeadDim + 8 * cb + i) : 1.0f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    uint32_t hi[4] = {0, 0, 0, 0}, neg[4] = {0, 0, 0, 0};
    if (have) {
      __half2 c[4];
      code_pairs<BITS>(r.k[u], c);
      const float2 ms = unpack_min_scale(r.ks[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(c[i]);
        split2(fmaf(f.x, ms.y, ms.x) * norm[pair_a<BITS>(i)], fmaf(f.y, ms.y, ms.x) * norm[pair_b<BITS>(i)], &hi[i], &neg[i]);
      }
    }
    const uint32_t o = tile_off(t0 + u, cb);
    *reinterpret_cast<uint4*>(sK + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(sN + o) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
  }
}

// Values of a uniform tile, rounded to fp16 once.
template <int BITS>
__device__ __forceinline__ void values_uniform(bool have, int tid, const RawTile& r, uint8_t* sV) {
  const int cb = tid & 15, t0 = (tid >> 4) * 8;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    uint32_t v[4] = {0, 0, 0, 0};
    if (have) {
      __half2 c[4];
      code_pairs<BITS>(r.v[u], c);
      const __half2 ms = as_h2(r.vs[u]), mn = __low2half2(ms), sc = __high2half2(ms);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = as_u32(__hfma2(c[i], sc, mn));
      // the largest code's value may pass the fp16 range by the scale's rounding
      if (fabsf(__low2float(ms)) + (float)((1 << BITS) - 1) * fabsf(__high2float(ms)) > 65504.0f) {
        const __half2 top = h2_const(0x7BFF), bottom = h2_const(0xFBFF);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = as_u32(__hmax2_nan(__hmin2_nan(as_h2(v[i]), top), bottom));
      }
    }
    *reinterpret_cast<uint4*>(sV + tile_off(t0 + u, cb)) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

__device__ __forceinline__ void fill_uniform_keys(const Geometry& G, const LayerPtrs& L, const TileSrc& src, int kt, int tid,
                                                  const RawTile& r, uint8_t* sK, uint8_t* sN) {
  const bool have = kt * kTile + (tid >> 4) * 8 < src.tc.Nq;
  if (G.gkc) {
    if (G.kb == 8) keys_token<8>(G, L, src.s, have, tid, r, sK, sN);
    else if (G.kb == 4) keys_token<4>(G, L, src.s, have, tid, r, sK, sN);
    else keys_token<2>(G, L, src.s, have, tid, r, sK, sN);
  } else {
    if (G.kb == 8) keys_channel<8>(have, tid, r, sK, sN);
    else if (G.kb == 4) keys_channel<4>(have, tid, r, sK, sN);
    else keys_channel<2>(have, tid, r, sK, sN);
  }
}
__device__ __forceinline__ void fill_group_rows(const Geometry& G, const TileSrc& src, int kt, int tid, const RawTile& r, uint8_t* sM) {
  const bool have = kt * kTile + (tid >> 4) * 8 < src.tc.Nq;
  if (G.kb == 8) group_rows<8>(have, tid, r, sM);
  else if (G.kb == 4) group_rows<4>(have, tid, r, sM);
  else group_rows<2>(have, tid, r, sM);
}
__device__ __forceinline__ void fill_uniform_values(const Geometry& G, const TileSrc& src, int kt, int tid, const RawTile& r,
                                                    uint8_t* sV) {
  const bool have = kt * kTile + (tid >> 4) * 8 < src.tc.Nq;
  if (G.vb == 8) values_uniform<8>(have, tid, r, sV);
  else if (G.vb == 4) values_uniform<4>(have, tid, r, sV);
  else values_uniform<2>(have, tid, r, sV);
}

// ------------------------------------------- non-uniform codes, RoPE, fp16

// Channels [8 chunk, + 8) of a non-uniform row: 24 bits at bit 24 chunk.
__device__ __forceinline__ uint32_t codes3(const uint8_t* row, int chunk) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
  const int bit = 24 * chunk, i = bit >> 5;
  return __funnelshift_r(__ldg(w + i), __ldg(w + min(i + 1, 11)), bit & 31) & 0xFFFFFFu;
}
__device__ __forceinline__ void values3(uint32_t w, float2 ms, const float* lut, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(ms.y, lut[(w >> (3 * i)) & 7], ms.x);
}

// A thread's share of a general tile: 4 consecutive tokens, the chunks cb and
// cb + 8.  Non-uniform rows: the codes, {min, scale} and (one per lane of the
// 8 that share the tokens) the outliers.  Uniform rows go through k_chunk.
struct RawGeneral {
  uint32_t w[4][2];   // 24 bits each
  uint32_t ms[4];
  uint32_t out[4];    // outlier (tid & 7): column << 16 | value
};
__device__ __forceinline__ void load_general(const uint8_t* codes, const uint32_t* scales, const uint8_t* col, const uint16_t* val,
                                             int nout, size_t tok, int cb, RawGeneral& r) {
  const uint8_t* row = codes + tok * 48;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
#pragma unroll
    for (int h = 0; h < 2; ++h) r.w[u][h] = codes3(row + 48 * u, cb + 8 * h);
    r.ms[u] = __ldg(scales + tok + u);
    r.out[u] = 0xFFFF0000u;  // no channel
    if (cb < nout) {
      const size_t o = (tok + u) * nout + cb;
      r.out[u] = (uint32_t)__ldg(col + o) << 16 | __ldg(val + o);
    }
  }
}
__device__ __forceinline__ void general_values(const RawGeneral& r, int u, const float* lut, int nout, int cb, float (&x)[2][8]) {
  const float2 ms = unpack_min_scale(r.ms[u]);
#pragma unroll
  for (int h = 0; h < 2; ++h) values3(r.w[u][h], ms, lut, x[h]);
  for (int j = 0; j < nout; ++j) {
    const uint32_t o = __shfl_sync(0xffffffffu, r.out[u], j, 8);
    const int c = o >> 16;
    if (((c >> 3) & 7) == cb) {
      const float v = half_bits_to_float((uint16_t)o);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c == 64 * h + 8 * cb + i) x[h][i] = v;
    }
  }
}

__device__ __forceinline__ void store_keys(const float (&x)[8], int t, int chunk, uint8_t* sK, uint8_t* sN) {
  uint32_t hi[4], neg[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(x[2 * i], x[2 * i + 1], &hi[i], &neg[i]);
  const uint32_t o = tile_off(t, chunk);
  *reinterpret_cast<uint4*>(sK + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(sN + o) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
}
__device__ __forceinline__ void zero_chunk(uint8_t* s, int t, int chunk) {
  *reinterpret_cast<uint4*>(s + tile_off(t, chunk)) = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void rotate_pairs(float (&x)[2][8], const float2 (&e)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = x[0][i], c = x[1][i];
    x[0][i] = a * e[i].x - c * e[i].y;
    x[1][i] = c * e[i].x + a * e[i].y;
  }
}

// Keys of a quantized tile with non-uniform codes or RoPE.  The first of the
// thread's 4 consecutive positions has its angles computed, the others
// follow by one complex product each (step: e^{i theta}).
__device__ __forceinline__ void fill_general_keys(const Geometry& G, const LayerPtrs& L, const unsigned long long* freq,
                                                  const float* lut, const TileSrc& src, int kt, int tid, uint8_t* sK, uint8_t* sN) {
  const int cb = tid & 7, t0 = (tid >> 3) * 4, f0 = kt * kTile + t0;
  if (kt * kTile + (t0 & ~31) >= src.tc.Nq) {  // a whole group (and so a whole warp's 16 keys)
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) zero_chunk(sK, t0 + u, cb + 8 * h), zero_chunk(sN, t0 + u, cb + 8 * h);
    return;
  }
  RawGeneral raw;
  if (G.kb == 3)
    load_general(L.k_codes, L.k_scales, L.k_col, L.k_val, G.nout, (size_t)src.s * G.qcap + f0, cb, raw);
  float2 e[8], step[8];
  if (G.pre_rope) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = phasor((uint32_t)(G.pos_offset + G.S + f0), freq[8 * cb + i]);
      step[i] = phasor(1, freq[8 * cb + i]);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float x[2][8];
    if (G.kb == 3) {
      general_values(raw, u, lut, G.nout, cb, x);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) k_chunk(G, L, lut, src.s, f0 + u, cb + 8 * h, x[h]);
    }
    if (G.pre_rope) {
      rotate_pairs(x, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = spec_cmul(e[i], step[i]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) store_keys(x[h], t0 + u, cb + 8 * h, sK, sN);
  }
}
__device__ __forceinline__ void fill_general_values(const Geometry& G, const LayerPtrs& L, const float* lut, const TileSrc& src,
                                                    int kt, int tid, uint8_t* sV) {
  const int cb = tid & 7, t0 = (tid >> 3) * 4, f0 = kt * kTile + t0;
  if (kt * kTile + (t0 & ~31) >= src.tc.Nq) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) zero_chunk(sV, t0 + u, cb + 8 * h);
    return;
  }
  RawGeneral raw;
  if (G.vb == 3)
    load_general(L.v_codes, L.v_scales, L.v_col, L.v_val, G.nout, (size_t)src.s * G.qcap + f0, cb, raw);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float y[2][8];
    if (G.vb == 3) {
      general_values(raw, u, lut, G.nout, cb, y);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) v_chunk(G, L, lut, src.s, f0 + u, cb + 8 * h, y[h]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint4*>(sV + tile_off(t0 + u, cb + 8 * h)) =
          make_uint4(pack_sat(y[h][0], y[h][1]), pack_sat(y[h][2], y[h][3]), pack_sat(y[h][4], y[h][5]), pack_sat(y[h][6], y[h][7]));
  }
}

// Row of fp16 key f: sinks, then the window ring (slot0: the slot of its first
// token), then the drafted tokens; null behind them.
__device__ __forceinline__ const uint16_t* fp16_key(const Geometry& G, const uint16_t* sink, const uint16_t* ring,
                                                    const uint16_t* draft, const TileSrc& src, int f) {
  if (f >= src.tc.k1) return f < src.tc.k1 + src.n_b ? draft + (src.draft0 + f - src.tc.k1) * kHeadDim : nullptr;
  if (f < src.tc.S_eff) return sink + ((size_t)src.s * G.S + f) * kHeadDim;
  int slot = src.slot0 + f - src.tc.S_eff;
  if (slot >= G.ring) slot -= G.ring;  // the window is at most one turn of the ring
  return ring + ((size_t)src.s * G.ring + slot) * kHeadDim;
}
__device__ __forceinline__ int fp16_pos(const TileSrc& src, int S, int f) {  // position of cached fp16 key f
  return f < src.tc.S_eff ? f : S + src.tc.Nq + (f - src.tc.S_eff);
}
// 16 bytes at p (zeros where p is null), as one predicated load.
__device__ __forceinline__ uint4 load16_if(const uint16_t* p, int chunk) {
  uint4 v;
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u64 p, %4, 0;\nmov.u32 %0, 0;\nmov.u32 %1, 0;\nmov.u32 %2, 0;\nmov.u32 %3, 0;\n"
      "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%5];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "l"(p + 8 * chunk));
  return v;
}

// fp16 tile: cached keys (rotated when they were cached before RoPE; then in
// two parts), drafted keys as they are, zeros behind them.
__device__ __forceinline__ void fill_fp16_keys(const Geometry& G, const LayerPtrs& L, const unsigned long long* freq,
                                               const uint16_t* kd, const TileSrc& src, int kt, int tid, uint8_t* sK, uint8_t* sN) {
  if (!G.pre_rope) {
    const int cb = tid & 15;
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = load16_if(fp16_key(G, L.k_sink, L.k_ring, kd, src, kt * kTile + (tid >> 4) + 16 * u), cb);
#pragma unroll
    for (int u = 0; u < 8; ++u) *reinterpret_cast<uint4*>(sK + tile_off((tid >> 4) + 16 * u, cb)) = v[u];
    return;
  }
  const int cb = tid & 7;
#pragma unroll 1
  for (int u = 0; u < 4; ++u) {
    const int t = (tid >> 3) * 4 + u, f = kt * kTile + t;
    const uint16_t* row = fp16_key(G, L.k_sink, L.k_ring, kd, src, f);
    float x[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) unpack8(load16_if(row, cb + 8 * h), x[h]);
    if (f < src.tc.k1) {
      float2 e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = phasor((uint32_t)(G.pos_offset + fp16_pos(src, G.S, f)), freq[8 * cb + i]);
      rotate_pairs(x, e);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) store_keys(x[h], t, cb + 8 * h, sK, sN);
  }
}

// Values of an fp16 tile.  A drafted value that is not finite enters as zero
// (a weight of zero must not meet it); true is returned then, and the merge
// adds it to the rows that see it.
__device__ __forceinline__ bool fill_fp16_values(const Geometry& G, const LayerPtrs& L, const uint16_t* vd, const TileSrc& src,
                                                 int kt, int tid, uint8_t* sV) {
  const int cb = tid & 15;
  bool bad = false;
  uint4 v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] = load16_if(fp16_key(G, L.v_sink, L.v_ring, vd, src, kt * kTile + (tid >> 4) + 16 * u), cb);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int t = (tid >> 4) + 16 * u;
    if (kt * kTile + t >= src.tc.k1 && !finite8(v[u])) {
      bad = true;
      float y[8];
      unpack8(v[u], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = isfinite(y[i]) ? y[i] : 0.0f;
      v[u] = pack8(y);
    }
    *reinterpret_cast<uint4*>(sV + tile_off(t, cb)) = v[u];
  }
  return bad;
}

#endif  // __CUDACC__

}  // namespace kvq
