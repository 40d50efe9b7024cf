// kvq_tree_tc.cu -- the tree attention on the 5th-generation tensor cores, for
// more than 16 query rows per KV head.
//
// One CTA per SM walks its range of 128-key tiles with 128 query rows:
//   8 producer warps  dequantize a tile into shared memory (two stages),
//   1 warp            issues the matrix instructions (one thread),
//   4 warps           softmax, one thread per row.
// S = Q K^T accumulates in TMEM (two buffers of 128 columns: the next tile's
// logits are computed under this tile's exponentials), the weights return
// there as fp16 over the logits they came from, and O += P V reads them from
// TMEM (O in columns 256..383).  Quantized keys enter in two exact fp16 parts
// (two passes of the 128-channel product), fp16 keys in one; what the 32 keys
// of a per-channel group share comes from a 16-column product with the groups'
// min and scale rows (columns 384 + 16 st).
// The maximum moves only when a logit passes it by 2^8 (weights then stay
// below fp16's range), so O is rarely rescaled.
// 13 warps leave every thread 128 registers (17 would leave 96, and spills).
#include "kvq_pipe.cuh"

namespace kvq {
namespace {

constexpr int kSoftThreads = 128;
constexpr int kThreadsTc = kSoftThreads + kProducers + 32;
// The 16-column product reads 8 rows behind the group rows as its columns
// 8..15 (of no use): the kilobyte that holds the barriers.
constexpr uint32_t kSmemTc = kTileBytes + 2 * kStageBytes + kGroupRowBytes + 1024;
static_assert(kSmemTc <= 227 * 1024, "shared memory of one CTA");
constexpr float kLazy = 8.0f;  // log2 units

// ------------------------------------------------- tensor-core operands
// Shared-memory operand with the 128-byte swizzle: start, leading and stride
// offsets in 16-byte units.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
// fp32 accumulator, fp16 operands, M = N = 128.
constexpr uint32_t kIdesc = (1u << 4) | ((128u / 8) << 17) | ((128u / 16) << 24);
constexpr uint32_t kIdesc16 = (1u << 4) | ((16u / 8) << 17) | ((128u / 16) << 24);  // N = 16
constexpr uint32_t kNegB = 1u << 14, kRowsB = 1u << 16;  // B negated; B's keys along its rows

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

#define KVQ_R32(r) \
  r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[11], r[12], r[13], r[14], r[15], r[16], r[17], r[18], \
      r[19], r[20], r[21], r[22], r[23], r[24], r[25], r[26], r[27], r[28], r[29], r[30], r[31]
// 32 columns of the thread's lane.
__device__ __forceinline__ void tm_load32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// The loads' results may be used after this (they are named so that no use moves ahead of it).
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tm_load8(uint32_t (&r)[8], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_store32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// ---------------------------------------------------------------- issuer
__device__ __forceinline__ bool issue_pv(const Bars& B, uint32_t tmem, uint32_t stage0, int i, bool first, volatile int* gave_up) {
  const int st = i & 1, ph = (i >> 1) & 1;
  if (!mbar_wait(B.p_full + 8 * st, ph, gave_up) || !mbar_wait(B.full_v + 8 * st, ph, gave_up)) return false;
  tc_after();
  const uint32_t v = stage0 + st * kStageBytes + 2 * kTileBytes;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)  // 16 keys: 16 rows of both 64-channel halves
    mma_ts(tmem + 256, tmem + 128 * st + 8 * ks, smem_desc(v + ks * 2048, kTile * 128, 1024), kIdesc | kRowsB,
           !(first && ks == 0));
  mma_commit(B.empty_v + 8 * st);
  mma_commit(B.o_done);
  return true;
}
__device__ __forceinline__ void issue(const TreeParams& p, const Bars& B, uint32_t tmem, uint32_t q, uint32_t stage0, uint32_t rows,
                                      int x, int x_end, volatile int* gave_up) {
  int i = 0;
  bool first_prev = false;
  while (x < x_end) {
    const Piece c = piece_at(p, x, x_end);
    const int parts = c.quant || p.geo.pre_rope ? 2 : 1;
    const bool grouped = channel_scales(p.geo) && c.quant;
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      if (!mbar_wait(B.full_k + 8 * st, (i >> 1) & 1, gave_up)) return;
      tc_after();
      for (int part = 0; part < parts; ++part) {
        const uint32_t k = stage0 + st * kStageBytes + part * kTileBytes;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {  // 16 channels
          const uint32_t off = (ks >> 2) * (kTile * 128) + (ks & 3) * 32;
          mma_ss(tmem + 128 * st, smem_desc(q + off, 16, 1024), smem_desc(k + off, 16, 1024), kIdesc | (part ? kNegB : 0),
                 part + ks > 0);
        }
      }
      if (grouped) {  // q . m and q . s of the tile's four groups (columns 8..15 are of no use)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss(tmem + 384 + 16 * st, smem_desc(q + (ks >> 2) * (kTile * 128) + (ks & 3) * 32, 16, 1024),
                 smem_desc(rows + (ks >> 2) * 1024 + (ks & 3) * 32, 16, 1024), kIdesc16, ks > 0);
      }
      mma_commit(B.s_full + 8 * st);
      mma_commit(B.empty_k + 8 * st);
      // the product of the tile before, whose weights are computed meanwhile
      if (i && !issue_pv(B, tmem, stage0, i - 1, first_prev, gave_up)) return;
      first_prev = t == 0;  // a piece's first tile starts O anew
    }
    x += c.cnt;
  }
  if (i) issue_pv(B, tmem, stage0, i - 1, first_prev, gave_up);
}

// --------------------------------------------------------------- softmax
__device__ __forceinline__ void softmax(const TreeParams& p, const Bars& B, uint32_t tmem, volatile int* bad_piece, int x,
                                        int x_end, int tid, volatile int* gave_up) {
  // warp-uniform: the TMEM loads are for whole warps
  auto wait = [&](uint32_t bar, int phase) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, gave_up)); };
  const int r = tid;
  const uint32_t lane0 = (uint32_t)(r & ~31) << 16, O = tmem + 256 + lane0;
  int i = 0;
  for (int piece = 0; x < x_end; ++piece) {
    const Piece c = piece_at(p, x, x_end);
    const bool work = (r & ~31) < c.nr;  // the warp holds rows
    const uint32_t* mask_row =
        p.mask && !c.quant && r < c.nr ? p.mask + ((size_t)c.b * p.n + (c.r0 + r) % c.n_b) * p.words : nullptr;
    const bool grouped = channel_scales(p.geo) && c.quant;
    const float centre = (float)(1 << (p.geo.kb - 1));
    float m = -INFINITY, l = 0.0f;
    for (int t = 0; t < c.cnt; ++t, ++i) {
      const int st = i & 1;
      const uint32_t S = tmem + 128 * st + lane0;
      if (!wait(B.s_full + 8 * st, i >> 1)) return;
      tc_after();
      if (work) {
        const int f0 = (c.k0 + t) * kTile;
        uint32_t ok[4], v[32];
        float top = -INFINITY, base[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // the groups' share of the logits
        if (grouped) {
          uint32_t y[8];
          tm_load8(y, tmem + 384 + 16 * st + lane0);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
            base[ch] = fmaf(centre, __uint_as_float(y[4 + ch]), __uint_as_float(y[ch])) * p.q_scale;
        }
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          ok[ch] = seen(p, c, mask_row, f0 + 32 * ch);
          tm_load32(v, S + 32 * ch);
          tm_wait_ld(v);
          float mx = -INFINITY;
          if (ok[ch] == 0xFFFFFFFFu) {
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(v[e]));
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((ok[ch] >> e) & 1) mx = fmaxf(mx, __uint_as_float(v[e]));
          }
          top = fmaxf(top, fmaf(mx, p.q_scale, base[ch]));
        }
        const bool move = top > m + kLazy;
        if (__any_sync(0xffffffffu, move)) {
          const float al = move ? ex2(m - top) : 1.0f;
          if (move) m = top, l *= al;
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
        const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tm_load32(v, S + 32 * ch);
          tm_wait_ld(v);
          uint32_t h[16];
          const float off = base[ch] - mu;
          if (ok[ch] != 0xFFFFFFFFu) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (ok[ch] >> e) & 1 ? v[e] : 0xFF800000u;  // -inf
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float a = ex2(fmaf(__uint_as_float(v[2 * e]), p.q_scale, off));
            const float b = ex2(fmaf(__uint_as_float(v[2 * e + 1]), p.q_scale, off));
            l += a + b;
            h[e] = as_u32(__floats2half2_rn(a, b));
          }
          tm_store16(S + 16 * ch, h);  // over logits that are read
        }
        tm_wait_st();
      }
      tc_before();
      mbar_arrive(B.p_full + 8 * st);
    }
    // the piece's partial result
    if (!wait(B.o_done, i - 1) || !wait(B.full_v + 8 * ((i - 1) & 1), (i - 1) >> 1)) return;
    if (r == 0 && !c.quant) p.part_flag[c.slot] = bad_piece[piece & 3] == piece + 1;
    tc_after();
    if (work) {
      const size_t at = (size_t)c.slot * p.rstride + r;
      if (r < c.nr) p.part_ml[at] = make_float2(m, l);
      const bool paired = c.quant && !p.geo.pre_rope && p.geo.kb != 3 && paired_order(p.geo.vb);
      float* acc = p.part_acc + at * kHeadDim;
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t v[32];
        tm_load32(v, O + 32 * ch);
        tm_wait_ld(v);
        if (r < c.nr) {
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
    x += c.cnt;
  }
}

__global__ void __launch_bounds__(kThreadsTc, 1) tree_tc_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sQ = smem_raw, *stage0 = sQ + kTileBytes, *sM = stage0 + 2 * kStageBytes, *tail = sM + kGroupRowBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(tail);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 128);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 132);
  float* lut = reinterpret_cast<float*>(tail + 144);  // K levels, V levels
  volatile int* bad_piece = reinterpret_cast<volatile int*>(tail + 208);  // [4] pieces with drafted values that are not finite
  const int tid = threadIdx.x, w = tid >> 5;
  const uint32_t b0 = (uint32_t)__cvta_generic_to_shared(bars);
  const Bars B{b0, b0 + 16, b0 + 32, b0 + 48, b0 + 64, b0 + 80, b0 + 96, b0 + 112};
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.full_k + 8 * i, kProducers);
      mbar_init(B.full_v + 8 * i, kProducers);
      mbar_init(B.empty_k + 8 * i, 1);
      mbar_init(B.empty_v + 8 * i, 1);
      mbar_init(B.s_full + 8 * i, 1);
      mbar_init(B.p_full + 8 * i, kSoftThreads);
    }
    mbar_init(B.o_done, 1);
    mbar_init(B.done, 1);
    // (the swizzle's 1024-byte alignment: there is no other shared memory to shift the start)
    *gave_up = ((uint32_t)__cvta_generic_to_shared(smem_raw) & 1023) != 0;
    for (int i = 0; i < 4; ++i) bad_piece[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid < 16) lut[tid] = tid < 8 ? p.k_lut_off[tid] : p.v_lut_off[tid - 8];
  const int issuer = (kSoftThreads + kProducers) / 32;
  if (w == issuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const int x = cta_first_tile(p.ncta, p.total, blockIdx.x), x_end = cta_first_tile(p.ncta, p.total, blockIdx.x + 1);
  if (*gave_up) {
  } else if (w < kSoftThreads / 32) {
    softmax(p, B, tmem, bad_piece, x, x_end, tid, gave_up);
  } else if (w < issuer) {
    produce<kTile>(p, B, sQ, stage0, sM, lut, bad_piece, x, x_end, tid - kSoftThreads, gave_up);
  } else {
    if ((tid & 31) == 0) {
      issue(p, B, tmem, (uint32_t)__cvta_generic_to_shared(sQ), (uint32_t)__cvta_generic_to_shared(stage0),
            (uint32_t)__cvta_generic_to_shared(sM), x, x_end, gave_up);
      mma_commit(B.done);  // whatever is in flight ends before TMEM is freed
      mbar_wait(B.done, 0, gave_up);
    }
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

cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t st) {
  static std::atomic<long long> memo[kMemoDevices];
  const cudaError_t e = ensure_smem_limit(tree_tc_kernel, memo, (int)kSmemTc);
  if (e != cudaSuccess) return e;
  tree_tc_kernel<<<p.ncta, kThreadsTc, kSmemTc, st>>>(p);
  return cudaGetLastError();
}

}  // namespace kvq
