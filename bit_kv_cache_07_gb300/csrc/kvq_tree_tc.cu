// kvq_tree_tc.cu -- the tree attention on the 5th-generation tensor cores, for
// more than 16 query rows per KV head.
//
// One CTA per SM walks its range of 96-key tiles with 128 query rows:
//   1 thread          copies the tiles' stored bytes ahead,
//   8 producer warps  dequantize a tile into shared memory (two stages),
//   1 warp            issues the matrix instructions (one elected lane; run by a
//                     converged warp the operands stay in uniform registers:
//                     alone, a thread took 337 us for the first workload below),
//   4 warps           softmax, one thread per row.
// TMEM: Q as the fp16 operand A of the logits, S = Q K^T in two buffers (the
// next tile's logits are computed under this tile's exponentials), the weights
// P, O += P V.  With Q in TMEM the logits' products read K alone from shared
// memory, whose bandwidth 96 columns would not cover twice.
// P enters in two fp16 parts like the keys: rounded to one, its error adds to
// V's and the output's (1.6 times the output's own rounding instead of 1.3; the
// second product costs 2 to 5 % of the time).
// Quantized keys enter in two exact fp16 parts (two passes of the 128-channel
// product), fp16 keys in one; what the 32 keys of a per-channel group share
// comes from a 16-column product with the groups' min and scale rows.
// A row's reference comes from its first tile's maximum and moves only when a
// tile's weights sum past fp16's range: one pass over the logits per tile, and O
// is rarely rescaled.  It lies 6 octaves below the maximum: fp16 ends at 2^-24,
// so a weight keeps its parts down to 2^-31 of the largest.  With the reference
// at the maximum, weights more than 17 nats below it (all tokens beside an
// attention sink) vanish from the product: of logits spread by 0.4 around 17.9
// nats nine tenths of the sum.  Each octave of that room is one less before a
// row moves: for the first workload below, logits of deviation 1, 2, 4 and 8
// take 293, 306, 353 and 398 us (295, 314, 368 and 410 with 8 octaves).  A move
// takes the whole warp's references along, by their rows' sums of the tile
// (searching the maxima again: 326 and 386 us for 2 and 4 with 8 octaves).
// The roles' loops share the instruction cache: rolled per 32 columns, the
// softmax fits beside the producers (unrolled, four fetches in ten missed and
// the kernel took half as long again).
//
// Measured with the merge, 32 heads on 8: 8 x 32k tokens KV4 and 32 nodes 293 us
// (469 TFLOP/s of the formula's 4 d rows T; the second parts of K and P double
// that on the tensor cores, 48 % of 1969); 28 heads on 4, 16 x up to 8k tokens
// K4V2 rotated, 21 nodes 93 us; 2 x 8191 fp16, 63 nodes 62 us.  What bounds it:
// the producers' conversion (some 3,100 of a tile's 3,900 cycles, 96 keys once
// per 128 rows), at an issue slot in two; DRAM idles (17 % of its rate).
#include "kvq_tc.cuh"
#include "kvq_pipe.cuh"

namespace kvq {
namespace {

constexpr int kSoftThreads = 128;
constexpr int kThreadsTc = kSoftThreads + kProducers + 64;
constexpr float kTopSum = 65504.0f;  // a tile's weights stay within fp16's range
constexpr float kRoom = 6.0f;        // octaves from a row's reference to the maximum (or sum) it was taken from
// The 16-column product reads 8 rows behind the group rows as its columns
// 8..15 (of no use): the first kilobyte of the tail.
constexpr uint32_t kFixedTc = 2 * kStageBytes + 2 * kGroupRowBytes + kTailBytes;
constexpr uint32_t kSmemTc = 227 * 1024;
// TMEM columns: S of stage st; the weights (what is left of them 48 behind);
// O; the groups' products; Q.
constexpr uint32_t kTmemS = 96, kTmemP = 192, kTmemO = 288, kTmemGroup = 416, kTmemQ = 448;

// ---------------------------------------------------------------- issuer
// What the issuer remembers of a tile whose product with the values is due.
struct Due {
  bool first;  // of its piece: O starts anew
  int piece;   // its number
  int slot;    // the last of an fp16 piece: where the piece's flag goes; else -1
};
__device__ __forceinline__ bool issue_pv(uint32_t lead, const TreeParams& p, const Bars& B, uint32_t tmem, uint64_t vd, const Tail* tail, int i,
                                         const Due& due, volatile int* gave_up) {
  auto wait = [&](uint32_t bar, int phase, volatile int* g) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase, g)); };
  const int st = i & 1, ph = (i >> 1) & 1;
  if (!wait(B.p_full + 8 * st, ph, gave_up) || !wait(B.full_v + 8 * st, ph, gave_up)) return false;
  tc_after();
  const uint64_t v = vd + st * (kStageBytes >> 4);
#pragma unroll
  for (int part = 0; part < 2; ++part)
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks)  // 16 keys: 16 rows of both 64-channel halves
      mma_ts(lead, tmem + kTmemO, tmem + kTmemP + kTile / 2 * part + 8 * ks, v + ks * (2048 >> 4), idesc(128) | kRowsB,
             part > 0 || ks > 0 || !due.first);
  // (full_v was waited for at every tile of the piece)
  if (due.slot >= 0 && lead) p.part_flag[due.slot] = *(volatile const int*)&tail->bad_piece[due.piece & 3] == due.piece + 1;
  mma_commit(lead, B.empty_v + 8 * st);
  mma_commit(lead, B.o_done);
  return true;
}
__device__ __forceinline__ void issue(uint32_t lead, const TreeParams& p, const Bars& B, uint32_t tmem, uint32_t stage0, uint32_t rows,
                                      const Tail* tail, int x, int x_end, volatile int* gave_up) {
  auto wait = [&](uint32_t bar, int phase, volatile int* g) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase, g)); };
  // descriptors of stage 0; stages, parts and k-steps add to their addresses
  const uint64_t kd = smem_desc(stage0, 16, 1024), vd = smem_desc(stage0 + 2 * kTileBytes, kTile * 128, 1024), md = smem_desc(rows, 16, 1024);
  int i = 0;
  Due due{};
  for (int piece = 0; x < x_end; ++piece) {
    const Piece c = piece_at(p, x, x_end);
    const int parts = c.quant || p.geo.pre_rope ? 2 : 1;
    const bool grouped = channel_scales(p.geo) && c.quant;
    if (!wait(B.q_full, piece & 1, gave_up)) return;
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      if (!wait(B.full_k + 8 * st, (i >> 1) & 1, gave_up)) return;
      tc_after();
      const uint32_t S = tmem + kTmemS * st;
      const uint64_t k = kd + st * (kStageBytes >> 4);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)  // 16 channels
        mma_ts(lead, S, tmem + kTmemQ + 8 * ks, k + (ks >> 2) * (kTile * 128 >> 4) + (ks & 3) * 2, idesc(kTile), ks > 0);
      if (parts == 2) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts(lead, S, tmem + kTmemQ + 8 * ks, k + (kTileBytes >> 4) + (ks >> 2) * (kTile * 128 >> 4) + (ks & 3) * 2, idesc(kTile) | kNegB, 1);
      }
      if (grouped) {  // q . m and q . s of the tile's groups (columns 8..15 are of no use)
        const uint64_t r = md + st * (kGroupRowBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts(lead, tmem + kTmemGroup + 16 * st, tmem + kTmemQ + 8 * ks, r + (ks >> 2) * (1024 >> 4) + (ks & 3) * 2, idesc(16), ks > 0);
      }
      mma_commit(lead, B.s_full + 8 * st);
      mma_commit(lead, B.empty_k + 8 * st);
      // the product of the tile before, whose weights are computed meanwhile
      if (i && !issue_pv(lead, p, B, tmem, vd, tail, i - 1, due, gave_up)) return;
      due = Due{t == 0, piece, !c.quant && t == c.cnt - 1 ? c.slot : -1};
    }
    x += c.cnt;
  }
  if (i) issue_pv(lead, p, B, tmem, vd, tail, i - 1, due, gave_up);
}

// --------------------------------------------------------------- softmax
// The thread's query row of a piece into TMEM, in the keys' channel order.
__device__ __forceinline__ void put_q(const TreeParams& p, const Bars& B, const Piece& c, uint32_t tmem_lane, int r) {
  const Geometry& G = p.geo;
  const bool paired = c.quant && channel_scales(G) && paired_order(G.kb), paired_iq = c.quant && G.gkc && paired_order(G.kb);
  const uint4* row = nullptr;
  if (r < c.nr) {
    const int j = (c.r0 + r) / c.n_b, node = c.r0 + r - j * c.n_b;
    row = reinterpret_cast<const uint4*>(p.q + (((size_t)c.b * G.Hq_tot + (size_t)layer_head(G, c.h) * G.g + j) * p.n + node) * kHeadDim);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[32];
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row) v = __ldg(row + 8 * h + ch);
      if (paired || paired_iq) v = pair_chunk(v);
      w[4 * ch] = v.x, w[4 * ch + 1] = v.y, w[4 * ch + 2] = v.z, w[4 * ch + 3] = v.w;
    }
    tm_store32(tmem_lane + kTmemQ + 32 * h, w);
  }
  tm_wait_st();
  tc_before();
  mbar_arrive_warp(B.q_full);
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Two logits to two weights: packed multiply-add, two exponentials.
__device__ __forceinline__ float2 weights2(uint32_t s0, uint32_t s1, float2 scale, float2 off) {
  float2 z;
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(z.x), "=f"(z.y)
      : "r"(s0), "r"(s1), "f"(scale.x), "f"(scale.y), "f"(off.x), "f"(off.y));
  return make_float2(ex2(z.x), ex2(z.y));
}
__device__ __forceinline__ void add2(float2& l, float2 a) {
  asm("{\n.reg .b64 a, b;\nmov.b64 a, {%0, %1};\nmov.b64 b, {%2, %3};\nadd.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}\n"
      : "+f"(l.x), "+f"(l.y)
      : "f"(a.x), "f"(a.y));
}

// Two weights as two fp16 parts each (22 bits).
__device__ __forceinline__ void weight_parts(float2 w, uint32_t* hi, uint32_t* rest) {
  *hi = as_u32(__floats2half2_rn(w.x, w.y));
  const float2 h = __half22float2(as_h2(*hi));
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%0, %1};\nmov.b64 b, {%2, %3};\nmov.b64 c, {%4, %4};\nfma.rn.f32x2 d, b, c, a;\nmov.b64 {%0, %1}, d;\n}\n"
      : "+f"(w.x), "+f"(w.y)
      : "f"(h.x), "f"(h.y), "f"(-1.0f));
  *rest = as_u32(__floats2half2_rn(w.x, w.y));
}

__device__ __forceinline__ void softmax(const TreeParams& p, const Bars& B, uint32_t tmem, int x, int x_end, int tid, volatile int* gave_up) {
  // warp-uniform: the TMEM loads are for whole warps
  auto wait = [&](uint32_t bar, int phase) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, gave_up)); };
  constexpr int kCh = kTile / 32;
  const int r = tid;
  const uint32_t lane0 = (uint32_t)(r & ~31) << 16, O = tmem + kTmemO + lane0;
  const float centre = (float)(1 << (p.geo.kb - 1));
  int i = 0;
  Piece c = piece_at(p, x, x_end);
  put_q(p, B, c, tmem + lane0, r);
  while (x < x_end) {
    const bool work = (r & ~31) < c.nr;  // the warp holds rows
    const uint32_t* mask_row =
        p.mask && !c.quant && r < c.nr ? p.mask + ((size_t)c.b * p.n + (c.r0 + r) % c.n_b) * p.words : nullptr;
    const bool grouped = channel_scales(p.geo) && c.quant;
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      const uint32_t S = tmem + kTmemS * st + lane0;
      if (!wait(B.s_full + 8 * st, i >> 1)) return;
      tc_after();
      if (work) {
        const int f0 = (c.k0 + t) * kTile;
        float base[kCh] = {};  // the groups' share of the logits
        if (grouped) {
          uint32_t y[8];
          tm_load8(y, tmem + kTmemGroup + 16 * st + lane0);
#pragma unroll
          for (int ch = 0; ch < kCh; ++ch)
            base[ch] = fmaf(centre, __uint_as_float(y[4 + ch]), __uint_as_float(y[ch])) * p.q_scale;
        }
        auto base_of = [&](int ch) { return ch == 0 ? base[0] : ch == 1 ? base[1] : base[2]; };
        static_assert(kCh == 3, "groups of a tile");
        // 32 logits, those that the row does not see as -inf
        uint32_t v[32];
        auto logits = [&](int ch) {
          tm_load32(v, S + 32 * ch);
          const uint32_t ok = seen(p, c, mask_row, f0 + 32 * ch);
          tm_wait_ld(v);
          if (__any_sync(0xffffffffu, ok != 0xFFFFFFFFu)) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (ok >> e) & 1 ? v[e] : 0xFF800000u;
          }
        };
        float sum = 0.0f;
        bool search = t == 0;  // the row's maximum is to be found
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          if (pass || search || __any_sync(0xffffffffu, m == -INFINITY)) {
            // past the range: the warp's references follow their rows' sums of the tile (then 2^kRoom)
            float to = m + lg2(sum) - kRoom;
            if (!pass || search) {
              float top = -INFINITY;
#pragma unroll 1
              for (int ch = 0; ch < kCh; ++ch) {
                logits(ch);
                float mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(v[e]));
                top = fmaxf(top, fmaf(mx, p.q_scale, base_of(ch)));
              }
              to = top - kRoom;
            }
            const bool move = to > m;
            if (__any_sync(0xffffffffu, move)) {
              const float al = move ? ex2(m - to) : 1.0f;
              if (move) m = to, l *= al;
              if (t > 0) {
                if (!wait(B.o_done, i - 1)) return;  // the products so far
                tc_after();
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                  tm_load32(v, O + 32 * ch);
                  tm_wait_ld(v);
#pragma unroll
                  for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
                  tm_store32(O + 32 * ch, v);
                }
                tm_wait_st();
              }
            }
          }
          const float mu = m == -INFINITY ? 0.0f : m;
          float2 part = make_float2(0.0f, 0.0f);
          const float2 scale = make_float2(p.q_scale, p.q_scale);
#pragma unroll 1
          for (int ch = 0; ch < kCh; ++ch) {
            logits(ch);
            const float o = base_of(ch) - mu;
            uint32_t h[16], rest[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 w = weights2(v[2 * e], v[2 * e + 1], scale, make_float2(o, o));
              add2(part, w);
              weight_parts(w, &h[e], &rest[e]);
            }
            if (ch == 0 && i > 0) {  // the product that reads the weights before is done
              if (!wait(B.o_done, i - 1)) return;
              tc_after();
            }
            tm_store16(tmem + kTmemP + lane0 + 16 * ch, h);
            tm_store16(tmem + kTmemP + kTile / 2 + lane0 + 16 * ch, rest);
          }
          sum = part.x + part.y;
          // past the range: do it again, with the maximum where the sum does not tell it
          if (search || __all_sync(0xffffffffu, sum <= kTopSum)) break;
          search = __any_sync(0xffffffffu, !(sum < INFINITY));
        }
        l += sum;
        tm_wait_st();
      }
      // a wait tells two phases apart, not three: a warp without rows sees them all too
      if (!work && i > 0 && !wait(B.o_done, i - 1)) return;
      tc_before();
      mbar_arrive_warp(B.p_full + 8 * st);
    }
    // the next piece's Q (this piece's logits are all computed), then this piece's partial result
    const Piece d = c;
    x += d.cnt;
    if (x < x_end) {
      c = piece_at(p, x, x_end);
      put_q(p, B, c, tmem + lane0, r);
    }
    if (!wait(B.o_done, i - 1)) return;
    tc_after();
    if (work) {
      const size_t at = (size_t)d.slot * p.rstride + r;
      if (r < d.nr) p.part_ml[at] = make_float2(m, l);
      const bool paired = d.quant && p.geo.vb != 3 && paired_order(p.geo.vb);
      float* acc = p.part_acc + at * kHeadDim;
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t v[32];
        tm_load32(v, O + 32 * ch);
        tm_wait_ld(v);
        if (r < d.nr) {
          uint4* dst = reinterpret_cast<uint4*>(acc + 32 * ch);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t* y = v + 8 * q;
            dst[2 * q] = paired ? make_uint4(y[0], y[2], y[4], y[6]) : make_uint4(y[0], y[1], y[2], y[3]);
            dst[2 * q + 1] = paired ? make_uint4(y[1], y[3], y[5], y[7]) : make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
      }
      tc_before();  // O is read before the next piece's weights are announced
    }
  }
}

// FP16: the unquantized cache, without the quantized tiles' code (63 nodes over
// 2 x 8191 tokens: 71 us with it).
template <bool FP16>
__global__ void __launch_bounds__(kThreadsTc, 1) tree_tc_kernel(const __grid_constant__ TreeParams p) {
  // (the swizzle's 1024-byte alignment: there is no other shared memory to shift the start)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *stage0 = smem, *sM = stage0 + 2 * kStageBytes;
  Tail* tail = reinterpret_cast<Tail*>(sM + 2 * kGroupRowBytes);
  uint8_t* raw0 = sM + 2 * kGroupRowBytes + kTailBytes;
  volatile int* gave_up = &tail->gave_up;
  grid_dep_trigger();  // the merge may be launched; it waits for this grid's end
  const int tid = threadIdx.x, w = tid >> 5;
  const Bars B = bars_at((uint32_t)__cvta_generic_to_shared(tail->bars));
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.full_k + 8 * i, kProducers / 32);
      mbar_init(B.full_v + 8 * i, kProducers / 32);
      mbar_init(B.empty_k + 8 * i, 1);
      mbar_init(B.empty_v + 8 * i, 1);
      mbar_init(B.s_full + 8 * i, 1);
      mbar_init(B.p_full + 8 * i, kSoftThreads / 32);
    }
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(B.raw_full + 8 * i, 1);
      mbar_init(B.raw_empty + 8 * i, kProducers / 32);
    }
    mbar_init(B.o_done, 1);
    mbar_init(B.q_full, kSoftThreads / 32);
    mbar_init(B.done, 1);
    *gave_up = ((uint32_t)__cvta_generic_to_shared(smem) & 1023) != 0;
    for (int i = 0; i < 4; ++i) tail->bad_piece[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  put_tables<true>(p, tail, raw0, tid);
  constexpr int issuer = (kSoftThreads + kProducers) / 32;  // then the copies' warp
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
  } else if (w < kSoftThreads / 32) {
    softmax(p, B, tmem, x, x_end, tid, gave_up);
  } else if (w < issuer) {
    produce<0, true, FP16>(p, B, nullptr, stage0, sM, raw0, tail, x, x_end, tid - kSoftThreads, gave_up);
  } else if (w == issuer) {
    const uint32_t lead = elect_lead();
    issue(lead, p, B, tmem, (uint32_t)__cvta_generic_to_shared(stage0), (uint32_t)__cvta_generic_to_shared(sM), tail, x,
            x_end, gave_up);
    mma_commit(lead, B.done);  // whatever is in flight ends before TMEM is freed
    mbar_wait(B.done, 0, nullptr);
    __syncwarp();
  } else {
    if ((tid & 31) == 0) load_tiles<true>(p, B, (uint32_t)__cvta_generic_to_shared(raw0), x, x_end, gave_up);
    __syncwarp();
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (w == issuer)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  if (*gave_up) {  // a wait ran out: every row of the range becomes NaN
    for (int y = x; y < x_end;) {
      const Piece c = piece_at(p, y, x_end);
      for (int r = tid; r < c.nr; r += kThreadsTc) p.part_ml[(size_t)c.slot * p.rstride + r] = make_float2(NAN, NAN);
      y += c.cnt;
    }
  }
}

}  // namespace

template <bool FP16>
static cudaError_t launch(TreeParams& p, cudaStream_t st) {
  static std::atomic<long long> memo[kMemoDevices];
  const cudaError_t e = ensure_smem_limit(tree_tc_kernel<FP16>, memo, (int)kSmemTc);
  if (e != cudaSuccess) return e;
  tree_tc_kernel<FP16><<<p.ncta, kThreadsTc, kSmemTc, st>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_tree_tc(TreeParams& p, cudaStream_t st) {
  p.raw = raw_slot(p.geo, true, kSmemTc - kFixedTc);
  if (kFixedTc + raw_bytes(p.geo, p.raw, true) > kSmemTc) return cudaErrorInvalidValue;
  return p.geo.fp16_mode ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace kvq
