// kvq_block_attn.cu -- attention of a step's tokens over 8-bit blocks: causal,
// with or without a sliding window and first tokens that stay visible.
//
// Row r = (token i, head j of the KV head's group), key t of a block with the
// scales 2^ek, 2^ev:
//   y_rt = scale log2(e) 2^ek (q_r . c_t) + ev,  w_rt = 2^(y_rt - ref_r),
//   out_r = sum_t w_rt c'_t / l_r,  l_r = sum_t 2^-ev w_rt,
//   lse_r = (ref_r + log2 l_r) ln 2:
// the value scale is a power of two, so it rides in the exponent of the weight
// and costs nothing per element.  The codes are fp16 numbers as they are (e4m3 is
// a subset), so the products on the tensor cores are exact up to fp32 sums.
//
// Bound: the bytes of the visible blocks, each read once for up to 64 rows of a
// KV head.  A 32-token tile of a head is two contiguous runs of 4 KB: one bulk
// copy by one thread, stored in an order that both ldmatrix and the key loads
// read without bank conflicts.  The visible tiles of all (request, head, row
// block) lie end to end, cut into one equal range per SM; lengths come from the
// GPU, so each CTA takes the prefix sums itself.  A CTA's eight warps form teams
// of one warp per 16 rows; teams take a segment's tiles in turn, each with its
// own ring of copies, which runs ahead across segments.  At a segment's end the
// teams join their (ref, l, O) through shared memory, and a (request, head, row
// block) that spans CTAs is joined by the CTA that comes last (nobody waits for
// another CTA).  mma.sync rather than tcgen05: 1 to 64 rows fill an eighth to a
// half of a 128-row tcgen05 tile, and its operands would have to be written back
// to shared memory as fp16 first (4 times the tile's bytes); here the
// conversion happens in the registers that feed the product.
#include "kvq_block.cuh"
#include "kvq_pipe.cuh"

namespace kvq {

namespace {

constexpr int kWarps = kBlockWarps;
constexpr int kThreadsAttn = 32 * kWarps;
constexpr int kStagesPerWarp = 2;    // a tile at work, one on the way: with two on the way (131 KB per SM in
                                     // flight) 16 x 32k tokens take 171 us, with one 160
constexpr int kPairBytes = 2 * kBlockSide;  // a tile: K then V
constexpr int kStages = kWarps * kStagesPerWarp;
constexpr float kRoom = 12.0f;       // weights up to 2^12 at a new reference,
constexpr float kMoveAt = 15.0f;     // up to 2^15 before it moves (fp16 ends at 2^16)

template <typename Walk>
struct AttnSmem {
  uint8_t stage[kStages][kPairBytes];
  float4 join[kWarps][16][32];  // the warps' accumulators, row by row
  uint8_t scale16[kStages][16];
  uint64_t full[kStages], empty[kStages];
  float2 join_ml[kWarps][16];
  int meta[kStages];           // byte of scale16 where the tile's scales are; -1: no such block
  long long warp_sum[kWarps];
  BlockSegment parted[2];
  int last[2], from[2];
  int gave_up;
  Walk first;                  // at the range's begin
};
static_assert(sizeof(AttnSmem<BlockWalk<16>>) <= 227 * 1024, "shared memory");

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void e4m3_halves(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n" : "=r"(lo), "=r"(hi) : "r"(four));
}
// bulk_copy with an L2 policy: blocks that one (head, row block) reads leave L2 first
// (16 x 32k tokens 160.6 to 158.5 us, 256k 84.6 to 82.7), those that several read stay.
__device__ __forceinline__ void stream_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;\n" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar), "l"(policy)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_halves(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
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

// A finished row: lane's four channels of sum w v, the weights' sum, their reference.
__device__ __forceinline__ void put_row(const BlockAttnParams& p, const BlockSegment& s, int r, int lane, float ref, float l, const float (&acc)[4]) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t row = row_at(p, s, r);
  *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 4 * lane) = make_uint2(pack_halves(acc[0] * inv, acc[1] * inv), pack_halves(acc[2] * inv, acc[3] * inv));
  if (p.lse && lane == 0) p.lse[row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
}

// RT: 16-row tiles that read a KV head's blocks together, MT of them by one warp (one
// conversion of keys and values for both; its queries then lie in shared memory)
template <int RT, int MT>
__global__ void __launch_bounds__(kThreadsAttn, 1) block_attn_kernel(const __grid_constant__ BlockAttnParams p) {
  constexpr int ROWS = 16 * RT, WT = RT / MT, TEAMS = kWarps / WT, RING = kStagesPerWarp * WT;  // WT: warps of a team
  extern __shared__ __align__(128) unsigned char smem_raw[];
  AttnSmem<BlockWalk<ROWS>>& sm = *reinterpret_cast<AttnSmem<BlockWalk<ROWS>>*>(smem_raw);
  const BlockGeo& G = p.geo;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, team = w / WT, wt = w % WT;
  const int gq = lane >> 2, tq = lane & 3;
  volatile int* gave_up = &sm.gave_up;
  if (tid < kStages) {
    mbar_init(smem_u32(&sm.full[tid]), 1);
    mbar_init(smem_u32(&sm.empty[tid]), WT);
  }
  if (tid == 0) sm.gave_up = 0;
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  grid_dep_wait();

  // the schedule: the requests' tiles, their sums, the CTA's range and the
  // request that it begins in
  const auto tiles_of = [&](int b) -> long long {
    if (b >= G.B) return 0;
    int nrb, streams, cnt;
    BlockWalk<ROWS>::size(p, request_at(p, b), &nrb, &streams, &cnt);
    return (long long)streams * cnt;
  };
  const int turns = (G.B + kThreadsAttn - 1) / kThreadsAttn;  // consecutive requests per thread
  long long mine[kMaxBlockBatch / kThreadsAttn], run = 0;
#pragma unroll
  for (int i = 0; i < kMaxBlockBatch / kThreadsAttn; ++i) {
    mine[i] = i < turns ? tiles_of(tid * turns + i) : 0;
    run += mine[i];
  }
  long long upto = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sm.warp_sum[w] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) upto += sm.warp_sum[i];
    total += sm.warp_sum[i];
  }
  const long long per = block_range(total, gridDim.x), x0 = per * blockIdx.x, x1 = min(total, x0 + per);
  if (x0 >= x1) return;
  long long at = upto - run;
#pragma unroll
  for (int i = 0; i < kMaxBlockBatch / kThreadsAttn; ++i) {
    if (x0 >= at && x0 < at + mine[i]) sm.first.begin(p, x0, x1, per, tid * turns + i, at);
    at += mine[i];
  }
  __syncthreads();

  grid_dep_trigger();  // the next kernel may come as the CTAs leave

  BlockWalk<ROWS> walk = sm.first, ahead = walk;
  uint8_t* const ring = sm.stage[team * RING];
  // A segment that one team takes goes to the team that has the fewest tiles of such
  // so far, the first of them (lane t of `load`: team t's; every warp keeps the same).
  const auto take = [&](int& load, const BlockSegment& s) {
    const unsigned least = __reduce_min_sync(0xffffffffu, lane < TEAMS ? (unsigned)load << 3 | lane : 0xffffffffu);
    const int t = least & 7;
    if (lane == t) load += s.k1 - s.k0;
    return t;
  };
  // The segment that copies are asked for in, the team's next tile of it, and the
  // block ids of 32 of its tiles, one per lane.
  BlockSegment as = {};
  int ai = 0, step = TEAMS, load_ahead = 0, issued = 0, in_slot = 0, id_at = 0, ids = 0;
  uint32_t in_turn = 0;
  bool have = wt == 0;
  const auto look_up = [&]() {  // by the team's first warp
    const int k = ai + lane * step;
    ids = k < as.k1 ? __ldg(p.t.block_table + (size_t)as.b * G.max_blocks + tile_of(as, k)) : 0;
    id_at = 0;
  };
  const auto find = [&]() {  // the team's next tile, if there is one
    if (ai < as.k1 && id_at < 32) return;
    while (ai >= as.k1) {
      bool solo;
      do {
        if (!(have = ahead.next(p, as))) return;
        solo = as.solo(per, TEAMS);
      } while (solo && take(load_ahead, as) != team);
      step = solo ? 1 : TEAMS;
      ai = as.k0 + (solo ? 0 : team);
    }
    look_up();
  };
  uint64_t leave, keep;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(leave));
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(keep));
  const auto issue = [&]() {  // copies of the next tile
    if (!have) return;
    const int slot = in_slot, st = team * RING + slot;
    if (WT > 1 && in_turn && !mbar_wait(smem_u32(&sm.empty[st]), (in_turn - 1) & 1, gave_up)) {
      have = false;
      return;
    }
    const int id = __shfl_sync(0xffffffffu, ids, id_at);
    if (lane == 0) {
      const bool proper = (unsigned)id < (unsigned)G.n_blocks;
      const size_t place = (size_t)(proper ? id : 0) * G.Hkv + as.h;
      const uint32_t bar = smem_u32(&sm.full[st]);
      sm.meta[st] = proper ? (int)(place * 2 & 15) : -1;
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(kPairBytes + 16) : "memory");
      stream_copy(smem_u32(ring + slot * kPairBytes), p.codes + place * kPairBytes, kPairBytes, bar, ahead.nrb > 1 ? keep : leave);
      bulk_copy(smem_u32(sm.scale16[st]), p.scales + (place * 2 & ~(size_t)15), 16, bar);
    }
    ++issued;
    if (++in_slot == RING) in_slot = 0, ++in_turn;
    ++id_at;
    ai += step;
    find();
  };
  if (wt == 0) {
    find();
    for (int i = 0; i < RING - 1; ++i) issue();
  }

  int out_slot = 0;  // of the tile that the team is at
  uint32_t out_phase = 0;
  int load = 0;
  // Queries of a segment: channel 32 tq + 4 k + {0, 1 | 2, 3} enters step k of the
  // product as its row 2 tq + {0, 1 | 8, 9}.
  uint32_t qa[MT == 1 ? 8 : 1][4];
  uint4* const q_mine = reinterpret_cast<uint4*>(sm.join[w]);  // MT 2: [tile][step][lane], the lane's own words
  const auto load_q = [&](const BlockSegment& s) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint4 v[2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = min((wt * MT + m) * 16 + gq + 8 * hf, s.rows - 1);  // (rows that are not there: the last one again)
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
  };
  // the next segment that the team has a part in (MT 1: its queries are on the way)
  const auto next_segment = [&](BlockSegment& s) {
    do {
      if (!walk.next(p, s)) return false;
    } while (s.solo(per, TEAMS) && take(load, s) != team);
    if (MT == 1) load_q(s);
    return true;
  };
  BlockSegment s;
  bool joined = false;
  int parts = 0;  // 1: the range begins, 2: it ends within a (request, head, row block)
  bool more = next_segment(s);
  if (MT > 1 && more) load_q(s);
  while (more) {
    const bool solo = s.solo(per, TEAMS);
    const int tile_step = solo ? 1 : TEAMS;
    const int row0 = wt * MT * 16, seg_rows = s.rows - row0;  // rows from this warp's first on; may be none
    float O[MT][8][2][4], ref[MT][2], l[MT][2];
    int see[MT][2];  // last position that a row sees
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        ref[m][hf] = -INFINITY;
        l[m][hf] = 0.0f;
        see[m][hf] = s.before + token_at(p, s, min(row0 + 16 * m + gq + 8 * hf, s.rows - 1));
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) O[m][c][e >> 2][e & 3] = 0.0f;
    }
    const bool active = seg_rows > 0;
    const int p_lo = s.before + token_at(p, s, 0), p_hi = s.before + token_at(p, s, s.rows - 1);  // positions of the block's rows

    for (int i = s.k0 + (solo ? 0 : team); i < s.k1; i += tile_step) {
      if (wt == 0) issue();
      const int slot = out_slot, st = team * RING + slot;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.full[st]), out_phase, gave_up));
      if (!ok) {  // the rows become NaN, and nothing more is asked for
#pragma unroll
        for (int m = 0; m < MT; ++m) l[m][0] = l[m][1] = NAN;
        have = false;
      }
      if (ok && active) {
        const uint8_t* K = ring + slot * kPairBytes;
        const uint32_t V = smem_u32(K + kBlockSide);
        const int meta = sm.meta[st], t0 = tile_of(s, i) * kBlockTokens;
        const int kb = meta < 0 ? kScaleNaN : sm.scale16[st][meta & 15], vb = meta < 0 ? kScaleNaN : sm.scale16[st][(meta & 15) + 1];
        const float f = kb == kScaleNaN ? NAN : p.q_scale * __uint_as_float((uint32_t)kb << 23);
        const float ev = vb == kScaleNaN ? NAN : (float)(vb - kScaleBias);
        const float inv_v = __uint_as_float((uint32_t)(254 - min(vb, 254)) << 23);
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
            kc[j] = *reinterpret_cast<const uint4*>(K + (8 * j + gq) * kHeadDim + (((2 * tq + half) ^ gq) << 4));
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
        // ---- logits in log2 units, less the reference (hidden keys: -infinity), weights
        const bool masked = t0 + kBlockTokens - 1 > p_lo || (p.window < kNoWindow && t0 <= p_hi - p.window);
        uint32_t pa[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (16 * m + 8 * hf >= seg_rows) {  // no such rows
            pa[m][0][hf] = pa[m][0][2 + hf] = pa[m][1][hf] = pa[m][1][2 + hf] = 0;
            continue;
          }
          float z[4][2];
          const float base = ev - ref[m][hf];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            z[j][0] = fmaf(S[m][j][2 * hf], f, base);
            z[j][1] = fmaf(S[m][j][2 * hf + 1], f, base);
          }
          if (masked) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int t = t0 + 8 * j + 2 * tq + e;
                if (!(t <= see[m][hf] && (see[m][hf] - t < p.window || t < p.n_first))) z[j][e] = -INFINITY;
              }
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
                if (z[j][e] != -INFINITY) top = fmaxf(top, fmaf(S[m][j][2 * hf + e], f, ev));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
            }
            if (high > kMoveAt) {
              const float to = top - kRoom, a = ex2(ref[m][hf] - to), base_to = ev - to;
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
                  if (z[j][e] != -INFINITY) z[j][e] = fmaf(S[m][j][2 * hf + e], f, base_to);
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
          l[m][hf] = fmaf(sum, inv_v, l[m][hf]);
        }
        // ---- values: a pair of adjacent channels of two tokens per register, sorted by channel
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            uint32_t v[4];
            const int mt = lane >> 3, tok = 16 * kk + 8 * (mt & 1) + (lane & 7);
            ldsm4t(v, V + tok * kHeadDim + (((c + (mt >> 1)) ^ (lane & 7)) << 4));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t e0, o0, e1, o1;
              e4m3_halves(__byte_perm(v[2 * u], 0, 0x3120), e0, o0);
              e4m3_halves(__byte_perm(v[2 * u + 1], 0, 0x3120), e1, o1);
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma16816(O[m][c + u][0], pa[m][kk], e0, e1);
                mma16816(O[m][c + u][1], pa[m][kk], o0, o1);
              }
            }
          }
      }
      if (++out_slot == RING) out_slot = 0, out_phase ^= 1;
      if constexpr (WT > 1) mbar_arrive_warp(smem_u32(&sm.empty[st]));
      else __syncwarp();
    }

    const BlockSegment done = s;
    more = next_segment(s);
    // ---- the teams' parts, joined in a fixed order
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) l[m][hf] += __shfl_xor_sync(0xffffffffu, l[m][hf], o);
    if (solo) {  // (whole)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int r = row0 + 16 * m + gq + 8 * hf;
          if (r >= done.rows) continue;
          const float inv = l[m][hf] == 0.0f ? 0.0f : 1.0f / l[m][hf];
          const size_t row = row_at(p, done, r);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float(&o)[2][4] = O[m][c];
            *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 16 * c + 4 * tq) =
                make_uint2(pack_halves(o[0][2 * hf] * inv, o[1][2 * hf] * inv), pack_halves(o[0][2 * hf + 1] * inv, o[1][2 * hf + 1] * inv));
          }
          if (p.lse && tq == 0) p.lse[row] = l[m][hf] == 0.0f ? -INFINITY : (ref[m][hf] + log2f(l[m][hf])) * 0.6931471805599453f;
        }
      if (MT > 1 && more) load_q(s);
      continue;
    }
    const bool whole = done.whole;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (MT > 1 && 16 * m >= done.rows) break;  // (no team has such rows)
      if (joined) __syncthreads();  // the parts of the time before have been read
      joined = true;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (16 * m + 8 * hf >= seg_rows) break;
        const int r = gq + 8 * hf;
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // (odd rows four places on: no two rows of a store in one bank)
          const float(&o)[2][4] = O[m][c];
          sm.join[w][r][(4 * c + tq) ^ (r & 1) << 2] = make_float4(o[0][2 * hf], o[1][2 * hf], o[0][2 * hf + 1], o[1][2 * hf + 1]);
        }
        if (tq == 0) sm.join_ml[w][r] = make_float2(ref[m][hf], l[m][hf]);
      }
      __syncthreads();
      for (int r = w; r < done.rows; r += kWarps) {
        if (MT > 1 && (r >> 4) % MT != m) continue;
        const int from = (r >> 4) / MT;  // warp of each team
        float2 ml[TEAMS];
        float top = -INFINITY, L = 0.0f, acc[4] = {};
#pragma unroll
        for (int t = 0; t < TEAMS; ++t) {
          ml[t] = sm.join_ml[t * WT + from][r & 15];
          top = fmaxf(top, ml[t].x);
        }
        const float zero = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int t = 0; t < TEAMS; ++t) {
          const float e = ex2(ml[t].x - zero);
          const float4 v = sm.join[t * WT + from][r & 15][lane ^ (r & 1) << 2];
          L = fmaf(e, ml[t].y, L);
          acc[0] = fmaf(e, v.x, acc[0]);
          acc[1] = fmaf(e, v.y, acc[1]);
          acc[2] = fmaf(e, v.z, acc[2]);
          acc[3] = fmaf(e, v.w, acc[3]);
        }
        if (whole) {
          put_row(p, done, r, lane, top, L, acc);
        } else {
          const size_t at_row = (size_t)piece_slot(done.x, per, blockIdx.x) * ROWS + r;
          __stcg(reinterpret_cast<float4*>(p.part_acc + at_row * kHeadDim) + lane, make_float4(acc[0], acc[1], acc[2], acc[3]));
          if (lane == 0) __stcg(reinterpret_cast<float2*>(p.part_ml + at_row * 2), make_float2(top, L));
        }
      }
    }
    if constexpr (MT > 1) {
      __syncthreads();
      joined = false;
      if (more) load_q(s);
    }
    if (!whole) {  // its turn comes at the range's end
      if (tid == 0) sm.parted[done.x >= x0 ? 1 : 0] = done;
      parts |= done.x >= x0 ? 2 : 1;
    }
  }

  // ---- what spans CTAs (the range's first and last segment): the last CTA to come joins the parts
  // (the barrier and the ticket's release order its writes before the ticket; the
  // acquire and the barrier after it, the other CTAs' before the reads)
  if (parts) {
    __syncthreads();
    if (tid < 2 && (parts >> tid & 1)) {
      const BlockSegment& d = sm.parted[tid];
      const int c0 = (int)udiv(d.x, per), c1 = (int)udiv(d.x + d.cnt - 1, per);
      unsigned before;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;\n" : "=r"(before) : "l"(p.counters + c0) : "memory");
      sm.last[tid] = before == (unsigned)(c1 - c0) ? c1 - c0 + 1 : 0;
      sm.from[tid] = c0;
      if (sm.last[tid]) p.counters[c0] = 0;
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
      const int count = parts >> side & 1 ? sm.last[side] : 0;
      if (!count) continue;
      const BlockSegment& d = sm.parted[side];
      const int c0 = sm.from[side];
      const auto piece = [&](int q, int r) { return (size_t)piece_slot(d.x, per, c0 + q) * ROWS + r; };
      for (int r = w; r < d.rows; r += kWarps) {
        const auto ml_at = [&](int q) {
          return q < count ? __ldcg(reinterpret_cast<const float2*>(p.part_ml + piece(q, r) * 2)) : make_float2(-INFINITY, 0.0f);
        };
        constexpr int kAhead = 16;  // accumulators in flight beside the maxima
        const auto acc_at = [&](int q) {
          return q < count ? __ldcg(reinterpret_cast<const float4*>(p.part_acc + piece(q, r) * kHeadDim) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float2 ml = ml_at(lane);
        float4 a[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) a[u] = acc_at(u);
        float top = ml.x;
        for (int q = lane + 32; q < count; q += 32) top = fmaxf(top, ml_at(q).x);
        top = warp_max(top);
        const float zero = top == -INFINITY ? 0.0f : top;
        float L = 0.0f, acc[4] = {};
        for (int q0 = 0; q0 < count; q0 += 32) {
          if (q0) ml = ml_at(q0 + lane);
          const float e = ex2(ml.x - zero);
          L = fmaf(e, ml.y, L);
          for (int q = 0; q < min(32, count - q0); q += kAhead) {
            if (q0 + q)
#pragma unroll
              for (int u = 0; u < kAhead; ++u) a[u] = acc_at(q0 + q + u);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
              const float eq = __shfl_sync(0xffffffffu, e, q + u);
              acc[0] = fmaf(eq, a[u].x, acc[0]);
              acc[1] = fmaf(eq, a[u].y, acc[1]);
              acc[2] = fmaf(eq, a[u].z, acc[2]);
              acc[3] = fmaf(eq, a[u].w, acc[3]);
            }
          }
        }
        L = warp_sum(L);
        put_row(p, d, r, lane, top, L, acc);
      }
    }
  }
  // copies in flight end before the CTA does (all were waited for, unless a wait ran out)
  if (wt == 0 && *gave_up)
    for (int i = max(0, issued - RING); i < issued; ++i) mbar_wait(smem_u32(&sm.full[team * RING + i % RING]), (i / RING) & 1, nullptr);
}

template <int RT, int MT>
cudaError_t launch_rows(const BlockAttnParams& p, int sms, cudaStream_t st) {
  static std::atomic<long long> memo[kMemoDevices];
  const cudaError_t e = ensure_smem_limit(block_attn_kernel<RT, MT>, memo, (int)sizeof(AttnSmem<BlockWalk<16 * RT>>));
  if (e != cudaSuccess) return e;
  return launch_dependent(block_attn_kernel<RT, MT>, dim3(sms), dim3(kThreadsAttn), sizeof(AttnSmem<BlockWalk<16 * RT>>), st, p);
}

}  // namespace

cudaError_t launch_block_attn(const BlockAttnParams& p, int sms, int rows, cudaStream_t st) {
  return rows == 16 ? launch_rows<1, 1>(p, sms, st) : rows == 32 ? launch_rows<2, 2>(p, sms, st) : launch_rows<4, 2>(p, sms, st);
}

}  // namespace kvq
