// kvq_fill.cuh -- dequantization of 96-key tiles into the shared-memory
// operands of the matrix instructions: keys in two fp16 parts (22 bits),
// values as fp16, rows of 128 bytes with the 128-byte swizzle (tile_off).
//
// A tile's stored bytes come to shared memory by asynchronous bulk copies,
// several tiles ahead (load_tiles); 256 threads convert them in short loops,
// whose code stays in the instruction caches (unrolled over registers, the
// fetches cost as much as the work).  Thread (tid & 15) owns 8 channels,
// tid >> 4 the keys 32 j + (tid >> 4) and + 16 of group j; with RoPE or
// non-uniform codes, tid & 7 owns the channel pairs (c, c + 64) of key
// 32 j + (tid >> 3).
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
// 2^-32 turns at every position below 2^31.  The hardware sine and cosine of
// an angle in [-pi, pi] are 5e-7 off at most.
__device__ __forceinline__ float2 phasor(uint32_t pos, unsigned long long f) {
  const uint32_t turns = pos * (uint32_t)(f >> 32) + __umulhi(pos, (uint32_t)f);
  float sn, cs;
  __sincosf((float)(int)turns * 1.4629180792671596e-9f /* 2 pi / 2^32 */, &sn, &cs);
  return make_float2(cs, sn);
}

// Place of channel pair i's frequency in the kernels' table: 8 lanes that read
// the same two pairs of 8 chunks read 128 bytes in a row.
__device__ __forceinline__ int freq_at(int i) { return 2 * (8 * ((i >> 1) & 3) + (i >> 3)) + (i & 1); }

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

// Ask for bytes in L2 (whole multiples of 16).
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(__cvta_generic_to_global(p)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// The copies of a stream's quantized tiles by one thread: sources and sizes
// per tile are set up once per piece, a tile is a few instructions (a lone
// warp pays an instruction fetch for most of what it executes).  The keys of a
// tile are contiguous in every region, and whole groups: sizes and starts are
// multiples of 16 bytes.
template <bool V>
struct TileCopies {
  const uint8_t *k, *ks, *v, *vs;         // the next tile's
  const uint8_t *kcol, *kval, *vcol, *vval;
  uint32_t nk, nks, nv, nvs, no;          // bytes per key; outliers per key
  __device__ __forceinline__ TileCopies(const Geometry& G, const LayerPtrs& L, int s, int kt) {
    const size_t tok = (size_t)s * G.qcap + (size_t)kt * kTile;
    const bool nuq = G.kb == 3;
    nk = G.krow;
    nks = nuq ? 4 : G.gkc ? 4 * G.nkg : kHeadDim * 4 / kGroupTokens;
    nv = V ? G.vrow : 0;
    nvs = V ? (nuq ? 4 : 4 * G.nvg) : 0;
    no = nuq ? G.nout : 0;
    k = L.k_codes + tok * nk;
    ks = reinterpret_cast<const uint8_t*>(L.k_scales) + tok * nks;
    v = L.v_codes + tok * nv;
    vs = reinterpret_cast<const uint8_t*>(L.v_scales) + tok * nvs;
    kcol = L.k_col + tok * no;
    kval = reinterpret_cast<const uint8_t*>(L.k_val) + tok * no * 2;
    vcol = L.v_col + tok * no;
    vval = reinterpret_cast<const uint8_t*>(L.v_val) + tok * no * 2;
  }
  // n keys into the slot at dst; bar expects their bytes.
  __device__ __forceinline__ void next(const RawSlot& R, uint32_t n, uint32_t dst, uint32_t bar) {
    const uint32_t o = no * (V ? 6 : 3);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(n * (nk + nks + nv + nvs + o)) : "memory");
    bulk_copy(dst, k, n * nk, bar);
    bulk_copy(dst + R.ks, ks, n * nks, bar);
    k += kTile * nk;
    ks += kTile * nks;
    if constexpr (V) {
      bulk_copy(dst + R.v, v, n * nv, bar);
      bulk_copy(dst + R.vs, vs, n * nvs, bar);
      v += kTile * nv;
      vs += kTile * nvs;
    }
    if (no) {
      bulk_copy(dst + R.kcol, kcol, n * no, bar);
      bulk_copy(dst + R.kval, kval, n * no * 2, bar);
      kcol += kTile * no;
      kval += kTile * no * 2;
      if constexpr (V) {
        bulk_copy(dst + R.vcol, vcol, n * no, bar);
        bulk_copy(dst + R.vval, vval, n * no * 2, bar);
        vcol += kTile * no;
        vval += kTile * no * 2;
      }
    }
  }
};

template <int BITS>
__device__ __forceinline__ uint2 chunk_word(const uint8_t* rows, int t, int chunk) {
  if constexpr (BITS == 8) return *reinterpret_cast<const uint2*>(rows + t * 128 + chunk * 8);
  else if constexpr (BITS == 4) return make_uint2(*reinterpret_cast<const uint32_t*>(rows + t * 64 + chunk * 4), 0);
  else return make_uint2(*reinterpret_cast<const uint16_t*>(rows + t * 32 + chunk * 2), 0);
}

// Channel pair i of a chunk in the operands' order: the index of its first
// and second channel.
template <int BITS>
__device__ __forceinline__ constexpr int pair_a(int i) { return BITS == 8 ? 2 * i : i; }
template <int BITS>
__device__ __forceinline__ constexpr int pair_b(int i) { return BITS == 8 ? 2 * i + 1 : i + 4; }

__device__ __forceinline__ void store_chunk(uint8_t* s, uint32_t off, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(s + off) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Keys of a uniform tile with a scale per channel and group of 32 tokens:
//   k = c' s + (m + 2^(b-1) s),  c' = code - 2^(b-1).
// The product c' s has 19 bits: its fp16 value hi and the rest neg = hi - c' s
// are exact.  The other part is the same for the 32 keys of a group, so it
// reaches the logits as one number per row and group, q . m + 2^(b-1) q . s:
// rows 0..2 of sM hold the tile's groups' m, rows 4..6 their s (8 rows of 128
// channels, q_off<8>).  Half the instructions of an fp32 k split in two.
//
// Straight-line code without branches, every shared-memory load ahead of the
// arithmetic: with two producer warps per scheduler the tile's time is its
// latency, and branches (rare cases, missing groups) each cost a round trip.
// Scales so large that c' s passes the fp16 range take the second form (SAT):
// fp32 products, hi saturated, and neg holds what exceeds it, up to 288 (8-bit
// codes), 4,400 (4) or 21,856 (2), to half a step of fp16: 1/8, 2 or 8.
template <int BITS, bool SAT>
__device__ __forceinline__ void key_products(const __half2 (&c)[4], const __half2 (&sc)[4], uint32_t (&hi)[4], uint32_t (&neg)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (SAT) {
      const float2 a = __half22float2(c[i]), b = __half22float2(sc[i]);
      split2(a.x * b.x, a.y * b.y, &hi[i], &neg[i]);
    } else {
      const __half2 h = __hmul2(c[i], sc[i]);
      hi[i] = as_u32(h);
      neg[i] = as_u32(__hfma2(__hneg2(c[i]), sc[i], h));
    }
  }
}
template <int BITS>
__device__ __forceinline__ void keys_channel(int groups, int tid, const uint8_t* raw, const uint32_t* scales, const uint32_t* zeros,
                                             uint8_t* sK, uint8_t* sN, uint8_t* sM) {
  constexpr int kG = kTile / 32;
  const int cb = tid & 15, t0 = tid >> 4;
  const uint32_t o0 = tile_off(t0, cb);  // keys 16 apart keep their swizzle
  // a chunk's 8 scale words as two loads; half of the lanes take the second 16
  // bytes first, so that 8 lanes 32 bytes apart cover all banks
  const int swap = (cb >> 2) & 1;
  const uint32_t sel_s = swap ? 0x3276u : 0x7632u, sel_m = swap ? 0x1054u : 0x5410u;
  __half2 most = h2_const(0);
#pragma unroll 1
  for (int j = 0; j < kG; ++j) {
    // a tile's missing groups (stale bytes in the slot): zero scales, so zero keys and rows
    uint32_t sw[8];
    const uint4* p = reinterpret_cast<const uint4*>(j < groups ? scales + j * kHeadDim : zeros) + 2 * cb;
    *reinterpret_cast<uint4*>(&sw[0]) = p[swap];
    *reinterpret_cast<uint4*>(&sw[4]) = p[swap ^ 1];
    uint2 w[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) w[v] = chunk_word<BITS>(raw, t0 + 32 * j + 16 * v, cb);
    __half2 sc[4];
    uint32_t m2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BITS == 8) {  // pairs (2 i, 2 i + 1): swapped lanes hold pairs 2, 3, 0, 1
        const int a = 2 * i, b = 2 * (i ^ 2);
        sc[i] = as_h2(__byte_perm(swap ? sw[b] : sw[a], swap ? sw[b + 1] : sw[a + 1], 0x7632));
        m2[i] = __byte_perm(swap ? sw[b] : sw[a], swap ? sw[b + 1] : sw[a + 1], 0x5410);
      } else {  // pairs (i, i + 4): swapped lanes hold (i + 4, i)
        sc[i] = as_h2(__byte_perm(sw[i], sw[i + 4], sel_s));
        m2[i] = __byte_perm(sw[i], sw[i + 4], sel_m);
      }
      most = __hmax2(most, sc[i]);
    }
    if (t0 == j) {
      const uint32_t s2[4] = {as_u32(sc[0]), as_u32(sc[1]), as_u32(sc[2]), as_u32(sc[3])};
      store_chunk(sM, q_off<8>(j, cb), m2);
      store_chunk(sM, q_off<8>(4 + j, cb), s2);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint32_t o = o0 + (32 * j + 16 * v) * 128;
      __half2 c[4];
      uint32_t hi[4], neg[4];
      code_pairs<BITS, true>(w[v], c);
      key_products<BITS, false>(c, sc, hi, neg);
      store_chunk(sK, o, hi);
      store_chunk(sN, o, neg);
    }
  }
  // c' s past the fp16 range: 2^(b-1) s > 65504, s from 512 (8192, 32768) on
  const float2 top = __half22float2(most);
  if (fmaxf(top.x, top.y) * (1 << (BITS - 1)) > 65504.0f) {
#pragma unroll 1
    for (int v = 0; v < 2 * kG; ++v) {
      __half2 c[4], sc[4];
      uint32_t hi[4], neg[4];
      code_pairs<BITS, true>(chunk_word<BITS>(raw, t0 + 16 * v, cb), c);
      const uint32_t* p = scales + (v >> 1) * kHeadDim + 8 * cb;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sc[i] = (v >> 1) < groups ? as_h2(__byte_perm(p[pair_a<BITS>(i)], p[pair_b<BITS>(i)], 0x7632)) : h2_const(0);
      key_products<BITS, true>(c, sc, hi, neg);
      const uint32_t o = tile_off(t0 + 16 * v, cb);
      store_chunk(sK, o, hi);
      store_chunk(sN, o, neg);
    }
  }
}

// Keys of a uniform tile with a scale per token and 64 channels (InnerQ):
// k = (min + code * scale) * norm in fp32, split into two fp16 parts.
template <int BITS>
__device__ __forceinline__ void keys_token(int groups, int tid, const uint8_t* raw, const uint32_t* scales, const float* norms,
                                           uint8_t* sK, uint8_t* sN) {
  const int cb = tid & 15;
  float norm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) norm[i] = norms ? __ldg(norms + 8 * cb + i) : 1.0f;
#pragma unroll 1
  for (int v = 0; v < kTile / 16; ++v) {
    const int t = (tid >> 4) + 16 * v;
    uint32_t hi[4] = {0, 0, 0, 0}, neg[4] = {0, 0, 0, 0};
    if ((v >> 1) < groups) {
      __half2 c[4];
      code_pairs<BITS>(chunk_word<BITS>(raw, t, cb), c);
      const float2 ms = unpack_min_scale(scales[2 * t + (cb >> 3)]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(c[i]);
        split2(fmaf(f.x, ms.y, ms.x) * norm[pair_a<BITS>(i)], fmaf(f.y, ms.y, ms.x) * norm[pair_b<BITS>(i)], &hi[i], &neg[i]);
      }
    }
    const uint32_t o = tile_off(t, cb);
    store_chunk(sK, o, hi);
    store_chunk(sN, o, neg);
  }
}

// Values of a uniform tile, rounded to fp16 once.
template <int BITS>
__device__ __forceinline__ void values_uniform(int groups, int tid, const uint8_t* raw, const uint32_t* scales, int nvg, int group,
                                               uint8_t* sV) {
  const int cb = tid & 15, t0 = tid >> 4;
  const uint32_t o0 = tile_off(t0, cb);
  __half2 most = h2_const(0);
#pragma unroll 1
  for (int j = 0; j < kTile / 32; ++j) {
    uint2 w[2];
    uint32_t sw[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int t = t0 + 32 * j + 16 * v;
      w[v] = chunk_word<BITS>(raw, t, cb);
      sw[v] = j < groups ? scales[t * nvg + group] : 0;  // missing groups: zeros
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      __half2 c[4];
      uint32_t y[4];
      code_pairs<BITS>(w[v], c);
      const __half2 mn = __low2half2(as_h2(sw[v])), sc = __high2half2(as_h2(sw[v]));
      most = __hmax2(most, __habs2(as_h2(sw[v])));
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = as_u32(__hfma2(c[i], sc, mn));
      store_chunk(sV, o0 + (32 * j + 16 * v) * 128, y);
    }
  }
  // the largest code's value may pass the fp16 range by the scale's rounding: it saturates
  const float2 far = __half22float2(most);
  if (far.x + far.y * ((1 << BITS) - 1) > 65504.0f) {
#pragma unroll 1
    for (int v = 0; v < kTile / 16; ++v) {
      uint4* at = reinterpret_cast<uint4*>(sV + o0 + 16 * v * 128);
      uint32_t y[4];
      *reinterpret_cast<uint4*>(y) = *at;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = as_u32(__hmax2_nan(__hmin2_nan(as_h2(y[i]), h2_const(0x7BFF)), h2_const(0xFBFF)));
      *at = *reinterpret_cast<uint4*>(y);
    }
  }
}

__device__ __forceinline__ int tile_groups(const TileSrc& src, int kt) { return min(kTile / 32, (src.tc.Nq - kt * kTile) / 32); }

__device__ __forceinline__ void fill_uniform_keys(const Geometry& G, const LayerPtrs& L, const RawSlot& R, const TileSrc& src, int kt,
                                                  int tid, const uint8_t* raw, const uint32_t* zeros, uint8_t* sK, uint8_t* sN,
                                                  uint8_t* sM) {
  const int groups = tile_groups(src, kt);
  const uint32_t* sc = reinterpret_cast<const uint32_t*>(raw + R.ks);
  if (G.gkc) {
    const float* norm = G.knorm ? L.k_norm + (size_t)src.s * kHeadDim : nullptr;
    if (G.kb == 8) keys_token<8>(groups, tid, raw, sc, norm, sK, sN);
    else if (G.kb == 4) keys_token<4>(groups, tid, raw, sc, norm, sK, sN);
    else keys_token<2>(groups, tid, raw, sc, norm, sK, sN);
  } else {
    if (G.kb == 8) keys_channel<8>(groups, tid, raw, sc, zeros, sK, sN, sM);
    else if (G.kb == 4) keys_channel<4>(groups, tid, raw, sc, zeros, sK, sN, sM);
    else keys_channel<2>(groups, tid, raw, sc, zeros, sK, sN, sM);
  }
}
__device__ __forceinline__ void fill_uniform_values(const Geometry& G, const RawSlot& R, const TileSrc& src, int kt, int tid,
                                                    const uint8_t* raw, uint8_t* sV) {
  const int groups = tile_groups(src, kt), group = 8 * (tid & 15) / G.gv;
  const uint32_t* sc = reinterpret_cast<const uint32_t*>(raw + R.vs);
  if (G.vb == 8) values_uniform<8>(groups, tid, raw + R.v, sc, G.nvg, group, sV);
  else if (G.vb == 4) values_uniform<4>(groups, tid, raw + R.v, sc, G.nvg, group, sV);
  else values_uniform<2>(groups, tid, raw + R.v, sc, G.nvg, group, sV);
}

// ------------------------------------------- non-uniform codes, RoPE, fp16

// Channels [8 chunk, + 8) of a non-uniform row: 24 bits at bit 24 chunk.
__device__ __forceinline__ uint32_t codes3(const uint8_t* row, int chunk) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
  const int bit = 24 * chunk, i = bit >> 5;
  return __funnelshift_r(w[i], w[min(i + 1, 11)], bit & 31) & 0xFFFFFFu;
}
// Channels of the chunks cb and cb + 8 of key t of a tile, non-uniform codes.
__device__ __forceinline__ void general_row(const uint8_t* codes, const uint32_t* scales, const uint8_t* pairs, int t, int cb,
                                            float (&x)[2][8]) {
  const float2 ms = unpack_min_scale(scales[t]);
  const uint32_t w[2] = {codes3(codes + 48 * t, cb), codes3(codes + 48 * t, cb + 8)};
  const uint32_t copy = (threadIdx.x & 15) * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 128 bytes an entry
      const uint32_t at = lop_and_or(i == 0 ? w[h] << 7 : i == 1 ? w[h] << 1 : w[h] >> (6 * i - 7), 63 << 7, copy);
      const float2 y = *reinterpret_cast<const float2*>(pairs + at);
      x[h][2 * i] = fmaf(ms.y, y.x, ms.x);
      x[h][2 * i + 1] = fmaf(ms.y, y.y, ms.x);
    }
}
// The outliers of the rows that a warp filled, one lane an outlier, over the
// dense values in the tile: f(row, its outlier list, channel, value).
template <class F>
__device__ __forceinline__ void each_outlier(const uint8_t* col, const uint16_t* val, int nout, int groups, int tid, F f) {
  __syncwarp();  // the warp's rows are written
  for (int k = tid & 31; k < 4 * groups * nout; k += 32) {
    const int r = k / nout, t = 32 * (r >> 2) + 4 * (tid >> 5) + (r & 3), at = t * nout + k - r * nout;
    f(t, t * nout, col[at] & 127, half_bits_to_float(val[at]));
  }
}
// The same of a uniform row (keys cached before RoPE: a scale per channel).
__device__ __forceinline__ void uniform_key_row(const uint8_t* codes, int bits, const uint32_t* scales, int t, int cb, float (&x)[2][8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int c[8];
    chunk_codes(codes + t * 16 * bits, bits, cb + 8 * h, c);
    const uint32_t* sc = scales + (t >> 5) * kHeadDim + 8 * cb + 64 * h;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 ms = unpack_min_scale(sc[i]);
      x[h][i] = fmaf((float)c[i], ms.y, ms.x);
    }
  }
}

__device__ __forceinline__ void store_keys(const float (&x)[8], int t, int chunk, uint8_t* sK, uint8_t* sN) {
  uint32_t hi[4], neg[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(x[2 * i], x[2 * i + 1], &hi[i], &neg[i]);
  const uint32_t o = tile_off(t, chunk);
  store_chunk(sK, o, hi);
  store_chunk(sN, o, neg);
}
__device__ __forceinline__ void rotate_pair(float& a, float& b, float2 e) {
  const float x = a, y = b;
  a = x * e.x - y * e.y;
  b = y * e.x + x * e.y;
}

// Keys of a quantized tile with non-uniform codes or RoPE.
__device__ __forceinline__ void fill_general_keys(const Geometry& G, const RawSlot& R, const unsigned long long* freq, const float* lut,
                                                  const uint8_t* pairs, const TileSrc& src, int kt, int tid, const uint8_t* raw, uint8_t* sK, uint8_t* sN) {
  const int cb = tid & 7, groups = tile_groups(src, kt);
#pragma unroll 1
  for (int j = 0; j < kTile / 32; ++j) {
    const int t = 32 * j + (tid >> 3);
    float x[2][8] = {};
    if (j < groups) {
      if (G.kb == 3)
        general_row(raw, reinterpret_cast<const uint32_t*>(raw + R.ks), pairs, t, cb, x);
      else
        uniform_key_row(raw, G.kb, reinterpret_cast<const uint32_t*>(raw + R.ks), t, cb, x);
      if (G.pre_rope) {
        const uint32_t pos = (uint32_t)(G.pos_offset + G.S + kt * kTile + t);
        const ulonglong2* f = reinterpret_cast<const ulonglong2*>(freq) + cb;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const ulonglong2 f2 = f[4 * i];
          rotate_pair(x[0][i], x[1][i], phasor(pos, f2.x));
          rotate_pair(x[0][i + 1], x[1][i + 1], phasor(pos, f2.y));
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) store_keys(x[h], t, cb + 8 * h, sK, sN);
  }
  if (G.nout == 0) return;
  const uint8_t* col = raw + R.kcol;
  const uint16_t* val = reinterpret_cast<const uint16_t*>(raw + R.kval);
  each_outlier(col, val, G.nout, groups, tid, [&](int t, int list, int c, float x) {
    float other = 0.0f;  // the channel that RoPE pairs with c
    const int d = c ^ 64;
    if (G.pre_rope) {
      const float2 ms = unpack_min_scale(reinterpret_cast<const uint32_t*>(raw + R.ks)[t]);
      other = fmaf(ms.y, lut[codes3(raw + 48 * t, d >> 3) >> (3 * (d & 7)) & 7], ms.x);
      for (int j = 0; j < G.nout; ++j)
        if (col[list + j] == d) other = half_bits_to_float(val[list + j]);
      // (a pair of two outliers is written twice, the same)
      const float2 e = phasor((uint32_t)(G.pos_offset + G.S + kt * kTile + t), freq[freq_at(c & 63)]);
      if (c < 64) rotate_pair(x, other, e);
      else rotate_pair(other, x, e);
    }
    uint32_t hi, neg;
    split2(x, other, &hi, &neg);
    const uint32_t o = tile_off(t, c >> 3) + 2 * (c & 7);
    *reinterpret_cast<uint16_t*>(sK + o) = (uint16_t)hi;
    *reinterpret_cast<uint16_t*>(sN + o) = (uint16_t)neg;
    if (G.pre_rope) {
      const uint32_t od = tile_off(t, d >> 3) + 2 * (d & 7);
      *reinterpret_cast<uint16_t*>(sK + od) = (uint16_t)(hi >> 16);
      *reinterpret_cast<uint16_t*>(sN + od) = (uint16_t)(neg >> 16);
    }
  });
}
__device__ __forceinline__ void fill_general_values(const Geometry& G, const RawSlot& R, const uint8_t* pairs, const TileSrc& src,
                                                    int kt, int tid, const uint8_t* raw, uint8_t* sV) {
  const int cb = tid & 7, groups = tile_groups(src, kt);
#pragma unroll 1
  for (int j = 0; j < kTile / 32; ++j) {
    const int t = 32 * j + (tid >> 3);
    float y[2][8] = {};
    if (j < groups)
      general_row(raw + R.v, reinterpret_cast<const uint32_t*>(raw + R.vs), pairs, t, cb, y);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint4*>(sV + tile_off(t, cb + 8 * h)) =
          make_uint4(pack_sat(y[h][0], y[h][1]), pack_sat(y[h][2], y[h][3]), pack_sat(y[h][4], y[h][5]), pack_sat(y[h][6], y[h][7]));
  }
  if (G.nout)
    each_outlier(raw + R.vcol, reinterpret_cast<const uint16_t*>(raw + R.vval), G.nout, groups, tid, [&](int t, int, int c, float y) {
      *reinterpret_cast<uint16_t*>(sV + tile_off(t, c >> 3) + 2 * (c & 7)) = (uint16_t)pack_sat(y, y);
    });
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

// The thread's 16-byte pieces of a tile's fp16 rows.  RUN: a tile that lies in
// one run of the window's slots (nearly all of an unquantized cache) is read
// without an address per row.
template <bool RUN>
__device__ __forceinline__ void load_fp16_rows(const Geometry& G, const uint16_t* sink, const uint16_t* ring, const uint16_t* draft,
                                               const TileSrc& src, int kt, int tid, uint4 (&v)[kTile / 16]) {
  if constexpr (RUN) {
    const int f = kt * kTile;
    int slot = src.slot0 + f - src.tc.S_eff;
    if (slot >= G.ring) slot -= G.ring;
    if (f >= src.tc.S_eff && f + kTile <= src.tc.k1 && slot + kTile <= G.ring) {
      const uint4* at = reinterpret_cast<const uint4*>(ring + ((size_t)src.s * G.ring + slot) * kHeadDim) + tid;
#pragma unroll
      for (int u = 0; u < kTile / 16; ++u) v[u] = __ldg(at + 256 * u);
      return;
    }
  }
#pragma unroll
  for (int u = 0; u < kTile / 16; ++u) v[u] = load16_if(fp16_key(G, sink, ring, draft, src, kt * kTile + (tid >> 4) + 16 * u), tid & 15);
}
__device__ __forceinline__ int fp16_pos(const TileSrc& src, int S, int f) {  // position of cached fp16 key f
  return f < src.tc.S_eff ? f : S + src.tc.Nq + (f - src.tc.S_eff);
}
// fp16 tile: cached keys (rotated when they were cached before RoPE; then in
// two parts), drafted keys as they are, zeros behind them.
template <bool RUN>
__device__ __forceinline__ void fill_fp16_keys(const Geometry& G, const LayerPtrs& L, const unsigned long long* freq,
                                               const uint16_t* kd, const TileSrc& src, int kt, int tid, uint8_t* sK, uint8_t* sN) {
  if (!G.pre_rope) {
    const int cb = tid & 15;
    uint4 v[kTile / 16];
    load_fp16_rows<RUN>(G, L.k_sink, L.k_ring, kd, src, kt, tid, v);
#pragma unroll
    for (int u = 0; u < kTile / 16; ++u) *reinterpret_cast<uint4*>(sK + tile_off((tid >> 4) + 16 * u, cb)) = v[u];
    return;
  }
  const int cb = tid & 7;
#pragma unroll 1
  for (int u = 0; u < kTile / 32; ++u) {
    const int t = 32 * u + (tid >> 3), f = kt * kTile + t;
    const uint16_t* row = fp16_key(G, L.k_sink, L.k_ring, kd, src, f);
    float x[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) unpack8(load16_if(row, cb + 8 * h), x[h]);
    if (f < src.tc.k1) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        rotate_pair(x[0][i], x[1][i], phasor((uint32_t)(G.pos_offset + fp16_pos(src, G.S, f)), freq[freq_at(8 * cb + i)]));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) store_keys(x[h], t, cb + 8 * h, sK, sN);
  }
}

// Values of an fp16 tile.  A drafted value that is not finite enters as zero
// (a weight of zero must not meet it); true is returned then, and the merge
// adds it to the rows that see it.
template <bool RUN>
__device__ __forceinline__ void load_fp16_values(const Geometry& G, const LayerPtrs& L, const uint16_t* vd, const TileSrc& src, int kt,
                                                 int tid, uint4 (&v)[kTile / 16]) {
  load_fp16_rows<RUN>(G, L.v_sink, L.v_ring, vd, src, kt, tid, v);
}
__device__ __forceinline__ bool store_fp16_values(const TileSrc& src, int kt, int tid, uint4 (&v)[kTile / 16], uint8_t* sV) {
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kTile / 16; ++u) {
    const int t = (tid >> 4) + 16 * u;
    if (kt * kTile + t >= src.tc.k1 && !finite8(v[u])) {
      bad = true;
      float y[8];
      unpack8(v[u], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = isfinite(y[i]) ? y[i] : 0.0f;
      v[u] = pack8(y);
    }
    *reinterpret_cast<uint4*>(sV + tile_off(t, tid & 15)) = v[u];
  }
  return bad;
}

#endif  // __CUDACC__

}  // namespace kvq
