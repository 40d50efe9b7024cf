// kvq_pipe.cuh -- what the two tree-attention kernels share: the pieces of a
// CTA's range, barriers with a limit, and the producer warps that keep two
// stages of dequantized tiles full.
#pragma once

#include "kvq_fill.cuh"

namespace kvq {

#ifdef __CUDACC__

constexpr int kProducers = 256;
constexpr uint32_t kTileBytes = kTile * kHeadDim * 2;  // 32 KB
constexpr uint32_t kStageBytes = 3 * kTileBytes;       // K hi, K neg, V
constexpr uint32_t kGroupRowBytes = 8 * kHeadDim * 2;  // the groups' min and scale rows
constexpr int kAhead = 3;                              // tiles asked for in L2 ahead of their loads

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------- barriers
__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// Wait for a phase, with a limit (well over any wait of a running kernel);
// past it the CTA gives up: every role leaves its loop.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t phase, volatile int* gave_up) {
  for (int it = 0; it < (1 << 24); ++it) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    if (ok) return true;
    if ((it & 255) == 255 && *gave_up) return false;
  }
  *gave_up = 1;
  return false;
}

// A piece of the CTA's range: consecutive tiles of one kind of one (b, h, row
// block).
struct Piece {
  TileCounts tc;
  int b, h, s, n_b, r0, nr, k0, cnt, slot;
  bool quant;
};
__device__ __forceinline__ Piece piece_at(const TreeParams& p, int x, int x_end) {
  const Geometry& G = p.geo;
  Piece c;
  c.b = row_of(p.rows.tile0, G.B, x);
  c.n_b = p.rows.nodes[c.b];
  c.tc = tile_counts(G, p.rows.tokens[c.b], p.mask ? c.n_b : 0);
  const int M = G.g * c.n_b, nrb = (M + p.rblk - 1) / p.rblk;
  const int per = c.tc.qt + c.tc.ft, off = x - p.rows.tile0[c.b], pair = off / per, k = off - pair * per;
  c.h = pair / nrb;
  const int rb = pair - c.h * nrb;
  c.s = c.b * G.Hkv + c.h;
  c.quant = k < c.tc.qt;
  c.k0 = c.quant ? k : k - c.tc.qt;
  c.cnt = min((c.quant ? c.tc.qt : c.tc.ft) - c.k0, x_end - x);
  c.slot = blockIdx.x + 2 * (p.rows.pair0[c.b] + pair) + (c.quant ? 0 : 1);
  c.r0 = rb * p.rblk;
  c.nr = min(p.rblk, M - c.r0);
  return c;
}

struct Bars {  // shared-memory addresses; by stage (o_done, done: one)
  uint32_t full_k, full_v, empty_k, empty_v, s_full, p_full, o_done, done;
};

// ------------------------------------------------------------- producers
template <int ROWS>
__device__ __forceinline__ void produce(const TreeParams& p, const Bars& B, uint8_t* sQ, uint8_t* stage0, uint8_t* sM, const float* lut,
                                        volatile int* bad_piece, int x, int x_end, int tid, volatile int* gave_up) {
  const Geometry& G = p.geo;
  const bool general = G.pre_rope || G.kb == 3;
  int i = 0;  // tiles so far
  for (int piece = 0; x < x_end; ++piece) {
    const Piece c = piece_at(p, x, x_end);
    const TileSrc src{c.tc, c.s, c.b, p.mask ? c.n_b : 0, c.tc.Nq % G.ring, in_stream(G, c.s) * p.n};
    RawTile raw;
    const bool uniform = c.quant && !general;
    if (c.quant && tid == 0)
      for (int k = c.k0 + (uniform ? 1 : 0); k < min(c.k0 + kAhead, c.k0 + c.cnt); ++k) prefetch_tile<true>(G, p.L, src, k);
    if (uniform) load_keys(G, p.L, src, c.k0, tid, raw), load_values(G, p.L, src, c.k0, tid, raw);
    // the previous piece's last product has read Q
    if (i && !mbar_wait(B.empty_k + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, gave_up)) return;
    const uint16_t* qb = p.q + ((size_t)c.b * G.Hq_tot + (size_t)layer_head(G, c.h) * G.g) * p.n * kHeadDim;
    const bool paired = uniform && paired_order(G.kb);
#pragma unroll
    for (int u = 0; u < ROWS / 16; ++u) {
      const int r = (tid >> 4) + 16 * u, ch = tid & 15;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < c.nr) {
        const int j = (c.r0 + r) / c.n_b, node = c.r0 + r - j * c.n_b;
        v = __ldg(reinterpret_cast<const uint4*>(qb + ((size_t)j * p.n + node) * kHeadDim) + ch);
        if (paired) v = pair_chunk(v);
      }
      *reinterpret_cast<uint4*>(sQ + q_off<ROWS>(r, ch)) = v;
    }
    bool bad = false;
    for (int k = c.k0; k < c.k0 + c.cnt; ++k, ++i) {
      const int st = i & 1;
      const uint32_t again = ((i >> 1) - 1) & 1;
      uint8_t *sK = stage0 + st * kStageBytes, *sN = sK + kTileBytes, *sV = sN + kTileBytes;
      if (i >= 2 && !mbar_wait(B.empty_k + 8 * st, again, gave_up)) return;
      if (!c.quant) fill_fp16_keys(G, p.L, p.freq, p.kd, src, k, tid, sK, sN);
      else if (general) fill_general_keys(G, p.L, p.freq, lut, src, k, tid, sK, sN);
      else fill_uniform_keys(G, p.L, src, k, tid, raw, sK, sN);
      if (uniform && !G.gkc) {  // (one buffer: the tile before must have been read)
        if (i && !mbar_wait(B.empty_k + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, gave_up)) return;
        fill_group_rows(G, src, k, tid, raw, sM);
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      mbar_arrive(B.full_k + 8 * st);
      const bool more = k + 1 < c.k0 + c.cnt;
      if (uniform && more) load_keys(G, p.L, src, k + 1, tid, raw);  // in flight under the values' conversion
      if (c.quant && tid == 0 && k + kAhead < c.k0 + c.cnt) prefetch_tile<true>(G, p.L, src, k + kAhead);
      if (i >= 2 && !mbar_wait(B.empty_v + 8 * st, again, gave_up)) return;
      if (!c.quant) bad |= fill_fp16_values(G, p.L, p.vd, src, k, tid, sV);
      else if (general) fill_general_values(G, p.L, lut + 8, src, k, tid, sV);
      else fill_uniform_values(G, src, k, tid, raw, sV);
      if (bad) bad_piece[piece & 3] = piece + 1;  // (at most 2 tiles, so 2 pieces, ahead of the reader)
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      mbar_arrive(B.full_v + 8 * st);
      if (uniform && more) load_values(G, p.L, src, k + 1, tid, raw);
    }
    x += c.cnt;
  }
}

// Bit e: the row sees key f0 + e.
__device__ __forceinline__ uint32_t seen(const TreeParams& p, const Piece& c, const uint32_t* mask_row, int f0) {
  if (c.quant) return f0 < c.tc.Nq ? 0xFFFFFFFFu : 0;  // whole groups of 32
  const int d0 = f0 - c.tc.k1;                          // drafted index of key f0
  if (d0 + 32 <= 0) return 0xFFFFFFFFu;
  if (!mask_row || d0 >= c.n_b) return d0 < 0 ? (1u << -d0) - 1 : 0;
  uint32_t m;
  if (d0 <= 0) {
    m = mask_row[0] << -d0;
  } else {
    const int w = d0 >> 5;
    m = __funnelshift_r(mask_row[w], w + 1 < p.words ? mask_row[w + 1] : 0u, d0 & 31);
  }
  if (c.n_b - d0 < 32) m &= (1u << (c.n_b - d0)) - 1;
  return d0 < 0 ? m | ((1u << -d0) - 1) : m;
}

#endif  // __CUDACC__

}  // namespace kvq
