// kvq_pipe.cuh -- what the tile kernels (tree attention, recorded weight) share: the pieces of a
// CTA's range, barriers with a limit, the thread that copies the stored bytes
// of the tiles ahead, and the producer warps that keep two stages of
// dequantized tiles full.
#pragma once

#include "kvq_fill.cuh"

namespace kvq {

#ifdef __CUDACC__

constexpr int kProducers = 256;
constexpr uint32_t kTileBytes = kTile * kHeadDim * 2;  // 24 KB
constexpr uint32_t kStageBytes = 3 * kTileBytes;       // K hi, K neg, V
constexpr uint32_t kKeyStageBytes = 2 * kTileBytes;    // K hi, K neg
constexpr uint32_t kGroupRowBytes = 8 * kHeadDim * 2;  // a stage's groups' min and scale rows

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// ------------------------------------------------------------- barriers
__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// One arrival for a warp, after what every lane did (32 arrivals on one word
// are 32 updates, one after the other).
__device__ __forceinline__ void mbar_arrive_warp(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Wait for a phase, with a limit (well over any wait of a running kernel);
// past it the CTA gives up: every role leaves its loop.  (gave_up null: a wait
// for copies in flight on the way out.)
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t phase, volatile int* gave_up, int tries = 1 << 22) {
#pragma unroll 1
  for (int it = 0; it < tries; ++it) {
    uint32_t ok;
    // asleep for up to 4 us a try: a polling warp takes issue slots from the working ones
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 4000;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    if (ok) return true;
    if ((it & 63) == 63 && gave_up && *gave_up) return false;
  }
  if (gave_up) *gave_up = 1;
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

constexpr uint32_t kTailBytes = 1408;
struct Bars {  // shared-memory addresses; by stage (raw: by slot; o_done, q_full, done: one)
  uint32_t full_k, full_v, empty_k, empty_v, s_full, p_full, raw_full, raw_empty, o_done, q_full, done;
};
constexpr int kBarBytes = (6 * 2 + 2 * kMaxRaw + 3) * 8;
__device__ __forceinline__ Bars bars_at(uint32_t b) {
  return Bars{b, b + 16, b + 32, b + 48, b + 64, b + 80, b + 96, b + 96 + 8 * kMaxRaw, b + 96 + 16 * kMaxRaw, b + 104 + 16 * kMaxRaw,
              b + 112 + 16 * kMaxRaw};
}
// The shared-memory tail of a kernel: barriers, then these words.
struct Tail {
  uint64_t bars[kBarBytes / 8];
  uint32_t tmem;
  int gave_up;
  int bad_piece[4];  // pieces that hold drafted values that are not finite, by number + 1
  float lut[8];      // level offsets of K
  alignas(16) unsigned long long freq[kHeadDim / 2];  // RoPE turns per position
  alignas(16) uint32_t zeros[kHeadDim];  // the scales of groups that a tile lacks
};
static_assert(sizeof(Tail) <= kTailBytes, "tail");

// The tables, by a whole CTA (a barrier follows).
template <bool V>
__device__ __forceinline__ void put_tables(const TreeParams& p, Tail* tail, uint8_t* raw0, int tid) {
  if (tid < 8) tail->lut[tid] = p.k_lut_off[tid];
  if (tid < kHeadDim) tail->zeros[tid] = 0;
  if (tid < kHeadDim / 2) tail->freq[freq_at(tid)] = p.freq[tid];
  if (p.geo.kb != 3) return;
  float2* pairs = reinterpret_cast<float2*>(raw0 + p.raw.pairs);
  for (int i = tid; i < (V ? 2 : 1) * 1024; i += blockDim.x) {
    const float* lut = V && i >= 1024 ? p.v_lut_off : p.k_lut_off;
    pairs[i] = make_float2(lut[(i >> 4) & 7], lut[(i >> 7) & 7]);
  }
}

__device__ __forceinline__ TileSrc tile_src(const TreeParams& p, const Piece& c) {
  return TileSrc{c.tc, c.s, c.b, p.mask ? c.n_b : 0, c.tc.Nq % p.geo.ring, in_stream(p.geo, c.s) * p.n};
}

// ---------------------------------------------------------------- copies
// One thread: the stored bytes of the quantized tiles into the raw slots, as
// many tiles ahead as there are slots; fp16 tiles are asked for in L2.
template <bool V>
__device__ __forceinline__ void load_tiles(const TreeParams& p, const Bars& B, uint32_t raw, int x, int x_end, volatile int* gave_up) {
  const Geometry& G = p.geo;
  int slot = 0, turn = 0;
  bool ok = true;
  while (ok && x < x_end) {
    const Piece c = piece_at(p, x, x_end);
    const TileSrc src = tile_src(p, c);
    if (!c.quant) {
      for (int k = c.k0; k < c.k0 + c.cnt; ++k) {
        // cached rows of the tile from the window's first slot on (the sinks are few)
        const int f0 = max(k * kTile, c.tc.S_eff), f1 = min((k + 1) * kTile, c.tc.k1);
        const int s0 = src.slot0 + f0 - c.tc.S_eff, n = min(f1 - f0, G.ring - s0);
        if (n > 0) {
          const size_t at = ((size_t)c.s * G.ring + s0) * kHeadDim;
          prefetch_l2(p.L.k_ring + at, n * kHeadDim * 2);
          if (V) prefetch_l2(p.L.v_ring + at, n * kHeadDim * 2);
        }
      }
    } else {
      TileCopies<V> copies(G, p.L, c.s, c.k0);
      int left = c.tc.Nq - c.k0 * kTile;
#pragma unroll 1
      for (int t = 0; t < c.cnt; ++t, left -= kTile) {
        if (turn && !(ok = mbar_wait(B.raw_empty + 8 * slot, (turn - 1) & 1, gave_up))) break;
        copies.next(p.raw, min(kTile, left), raw + slot * p.raw.bytes, B.raw_full + 8 * slot);
        if (++slot == p.raw.slots) slot = 0, ++turn;
      }
    }
    x += c.cnt;
  }
  // the copies in flight end before the CTA does, also when another warp gives
  // up after the last of them was started: the last fill of every slot
#pragma unroll 1
  for (int i = 0; i < p.raw.slots; ++i) {
    if (--slot < 0) slot = p.raw.slots - 1, --turn;
    if (turn < 0) break;
    mbar_wait(B.raw_full + 8 * slot, turn & 1, nullptr);
  }
}

// ------------------------------------------------------------- producers
// ROWS > 0: the producers also stage that many query rows of each piece.  V:
// the values too.  (Eight warps one half after the other: with eight more for
// the values side by side, the kernel's loops outgrow the instruction cache and
// it takes longer.)  FP16: every tile is an fp16 one.
template <int ROWS, bool V, bool FP16 = false>
__device__ __forceinline__ void produce(const TreeParams& p, const Bars& B, uint8_t* sQ, uint8_t* stage0, uint8_t* sM, const uint8_t* raw0,
                                        Tail* tail, int x, int x_end, int tid, volatile int* gave_up) {
  const Geometry& G = p.geo;
  const bool general = G.pre_rope || G.kb == 3;
  constexpr bool kAsync = ROWS == 0;  // the tensor core reads the tiles (staged rows: ldmatrix does)
  int i = 0, slot = 0, turn = 0;  // tiles so far, raw slot and its turn
  for (int piece = 0; x < x_end; ++piece) {
    const Piece c = piece_at(p, x, x_end);
    const TileSrc src = tile_src(p, c);
    const bool quant = !FP16 && c.quant;
    if constexpr (ROWS > 0) {
      // the previous piece's last logits are computed
      if (i && !mbar_wait(B.empty_k + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, gave_up)) return;
      const uint16_t* qb = p.q + ((size_t)c.b * G.Hq_tot + (size_t)layer_head(G, c.h) * G.g) * p.n * kHeadDim;
      const bool paired = quant && !general && paired_order(G.kb);
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
    }
    bool bad = false;
#pragma unroll 1
    for (int k = c.k0; k < c.k0 + c.cnt; ++k, ++i) {
      const int st = i & 1;
      const uint32_t again = ((i >> 1) - 1) & 1;
      uint8_t *sK = stage0 + st * (V ? kStageBytes : kKeyStageBytes), *sN = sK + kTileBytes, *sV = sN + kTileBytes;
      const uint8_t* raw = raw0 + slot * p.raw.bytes;
      uint4 held[V ? kTile / 16 : 1];  // an fp16 tile's values, in flight under its keys
      if (quant) {
        if (!mbar_wait(B.raw_full + 8 * slot, turn & 1, gave_up)) return;
      } else if constexpr (V) {
        load_fp16_values<FP16>(G, p.L, p.vd, src, k, tid, held);
      }
      if (i >= 2 && !mbar_wait(B.empty_k + 8 * st, again, gave_up)) return;
      if (!quant) fill_fp16_keys<FP16>(G, p.L, tail->freq, p.kd, src, k, tid, sK, sN);
      else if (general) fill_general_keys(G, p.raw, tail->freq, tail->lut, raw0 + p.raw.pairs, src, k, tid, raw, sK, sN);
      else fill_uniform_keys(G, p.L, p.raw, src, k, tid, raw, tail->zeros, sK, sN, sM + st * kGroupRowBytes);
      if constexpr (kAsync) asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      if constexpr (!V) {
        if (quant) {
          mbar_arrive_warp(B.raw_empty + 8 * slot);
          if (++slot == p.raw.slots) slot = 0, ++turn;
        }
        mbar_arrive_warp(B.full_k + 8 * st);
      } else {
        mbar_arrive_warp(B.full_k + 8 * st);
        if (i >= 2 && !mbar_wait(B.empty_v + 8 * st, again, gave_up)) return;
        if (!quant) bad |= store_fp16_values(src, k, tid, held, sV);
        else if (G.vb == 3) fill_general_values(G, p.raw, raw0 + p.raw.pairs + kLevelPairBytes, src, k, tid, raw, sV);
        else fill_uniform_values(G, p.raw, src, k, tid, raw, sV);
        if (bad) *(volatile int*)&tail->bad_piece[piece & 3] = piece + 1;  // (at most 2 tiles, so 2 pieces, ahead of the reader)
        if constexpr (kAsync) asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        if (quant) {
          mbar_arrive_warp(B.raw_empty + 8 * slot);
          if (++slot == p.raw.slots) slot = 0, ++turn;
        }
        mbar_arrive_warp(B.full_v + 8 * st);
      }
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
