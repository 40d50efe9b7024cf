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
// KV head (16 x 32k tokens of 32 on 8 heads: 157 to 162 us, 6.6 to 6.8 TB/s).  A
// 32-token tile of a head is one contiguous run of 8 KB: one bulk copy by one thread,
// stored in an order that both ldmatrix and the key loads read without bank conflicts.
// The visible tiles of all (request, head, row block) lie end to end, cut into one equal range per
// SM; lengths come from the GPU, so each CTA takes the prefix sums itself.  A CTA's
// eight warps form teams of one warp per 16 rows (or 8); teams take a segment's tiles
// in turn, each with its own ring of copies, which runs ahead across segments.  At a
// segment's end the teams join their (ref, l, O) through shared memory, and a
// (request, head, row block) that spans CTAs is joined by the CTA that comes last
// (nobody waits for another CTA).  mma.sync rather than tcgen05: 1 to 64 rows fill an
// eighth to a half of a 128-row tcgen05 tile, and its operands would have to be
// written back to shared memory as fp16 first (4 times the tile's bytes); here the
// conversion happens in the registers that feed the product.  Past 16 rows the tiles'
// conversions, done again by every warp of a team, bound it (two warps a scheduler:
// latency; 16 x 8k tokens of 32 on 8 heads: 45 us for 4 rows, 51 for 16, 95 for 32).
#include "kvq_block_tile.cuh"

namespace kvq {

namespace {

using namespace kvq::tile;

constexpr int kWarps = kBlockWarps;
constexpr int kThreadsAttn = 32 * kWarps;
constexpr int kStagesPerWarp = 2;    // a tile at work, one on the way: with two on the way (131 KB per SM in
                                     // flight) 16 x 32k tokens take 171 us, with one 160
constexpr int kPairBytes = 2 * kBlockSide;  // a tile: K then V
constexpr int kStages = kWarps * kStagesPerWarp;

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

// bulk_copy with an L2 policy: blocks that one (head, row block) reads leave L2 first
// (16 x 32k tokens 160.6 to 158.5 us, 256k 84.6 to 82.7), those that several read stay.
__device__ __forceinline__ void stream_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;\n" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar), "l"(policy)
               : "memory");
}
// A finished row: lane's four channels of sum w v, the weights' sum, their reference.
__device__ __forceinline__ void put_row(const BlockAttnParams& p, const BlockSegment& s, int r, int lane, float ref, float l, const float (&acc)[4]) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t row = row_at(p, s, r);
  *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 4 * lane) = make_uint2(pack_halves(acc[0] * inv, acc[1] * inv), pack_halves(acc[2] * inv, acc[3] * inv));
  if (p.lse && lane == 0) p.lse[row] = log_sum(ref, l);
}

// Math: a warp's arithmetic; WT: warps of a team, each with rows of its own
template <typename Math, int WT>
__global__ void __launch_bounds__(kThreadsAttn, 1) block_attn_kernel(const __grid_constant__ BlockAttnParams p) {
  constexpr int ROWS = Math::kRows * WT, TEAMS = kWarps / WT, RING = kStagesPerWarp * WT;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  AttnSmem<BlockWalk<ROWS>>& sm = *reinterpret_cast<AttnSmem<BlockWalk<ROWS>>*>(smem_raw);
  const BlockGeo& G = p.geo;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, team = w / WT, wt = w % WT;
  volatile int* gave_up = &sm.gave_up;
  const auto wait = [&](const uint64_t* bar, uint32_t phase) {  // by a warp: all of its lanes get the same answer
    return (bool)__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), phase, gave_up));
  };
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
  const BlockRange range{x0, x1, per};
  long long at = upto - run;
#pragma unroll
  for (int i = 0; i < kMaxBlockBatch / kThreadsAttn; ++i) {
    if (x0 >= at && x0 < at + mine[i]) sm.first.begin(p, range, tid * turns + i, at);
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
        if (!(have = ahead.next(p, range, as))) return;
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
    // (agreed, as every wait here: lanes whose limits end beside the phase would part ways before the shuffles)
    if (WT > 1 && in_turn && !wait(&sm.empty[st], (in_turn - 1) & 1)) {
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

  // Slot of the tile that the team is at.  -1: a wait ran out; the warp reads and empties no
  // slot any more, and its rows of every further segment become NaN.  (A later tile's phase
  // would look complete where the slot was last filled two turns before, and an arrival
  // without a tile read would let a slot be filled that another warp of the team still reads.)
  int out_slot = 0;
  uint32_t out_phase = 0;
  int load = 0;
  Math math;
  const int row0 = wt * Math::kRows;  // of a block's rows
  // the next segment that the team has a part in; its queries are on the way
  const auto next_segment = [&](BlockSegment& s) {
    do {
      if (!walk.next(p, range, s)) return false;
    } while (s.solo(per, TEAMS) && take(load, s) != team);
    math.load_q(p, s, row0, lane);
    return true;
  };
  BlockSegment s;
  bool joined = false;
  int parts = 0;  // 1: the range begins, 2: it ends within a (request, head, row block)
  bool more = next_segment(s);
  while (more) {
    const bool solo = s.solo(per, TEAMS);
    const int tile_step = solo ? 1 : TEAMS;
    const bool active = s.rows > row0;  // (a team's last warps may have no rows)
    math.begin();
    const int p_lo = s.before + token_at(p, s, 0), p_hi = s.before + token_at(p, s, s.rows - 1);  // positions of the block's rows

    for (int i = out_slot < 0 ? s.k1 : s.k0 + (solo ? 0 : team); i < s.k1; i += tile_step) {
      if (wt == 0) issue();
      const int slot = out_slot, st = team * RING + slot;
      if (!wait(&sm.full[st], out_phase)) {
        out_slot = -1;
        have = false;  // (nothing more is asked for)
        break;
      }
      if (active) {
        const int meta = sm.meta[st];
        const int kb = meta < 0 ? kScaleNaN : sm.scale16[st][meta & 15], vb = meta < 0 ? kScaleNaN : sm.scale16[st][(meta & 15) + 1];
        Tile t;
        t.K = ring + slot * kPairBytes;
        t.V = smem_u32(t.K + kBlockSide);
        t.f = kb == kScaleNaN ? NAN : p.q_scale * __uint_as_float((uint32_t)kb << 23);
        // The weights hold 2^ev and the sum 2^-ev: over 80 octaves of it neither leaves fp32 (a
        // weight that a larger one flushes is below 2^-46 of it).  Smaller scales are as good as
        // the least one, whose values end below 2^-31 (out's least step is 2^-24).
        const int ev = max(vb - kScaleBias, kMinExp);
        t.ev = ev > kMaxExp ? NAN : (float)ev;
        t.inv_v = __uint_as_float((uint32_t)(127 - min(ev, kMaxExp)) << 23);
        t.t0 = tile_of(s, i) * kBlockTokens;
        t.masked = t.t0 + kBlockTokens - 1 > p_lo || (p.window < kNoWindow && t.t0 <= p_hi - p.window);
        math.tile(p, s, t, lane, row0);
      }
      if (++out_slot == RING) out_slot = 0, out_phase ^= 1;
      if constexpr (WT > 1) mbar_arrive_warp(smem_u32(&sm.empty[st]));
      else __syncwarp();
    }

    if (out_slot < 0) math.spoil();
    const BlockSegment done = s;
    more = next_segment(s);
    // ---- the teams' parts, joined in a fixed order
    math.close();
    if (solo) {  // (whole)
      if (active) math.put(p, done, row0, lane);
      continue;
    }
    const bool whole = done.whole;
    if (joined) __syncthreads();  // the parts of the segment before have been read
    joined = true;
    math.dump(sm.join[w], sm.join_ml[w], lane);
    __syncthreads();
    for (int r = w; r < done.rows; r += kWarps) {
      const int from = r / Math::kRows, in = r % Math::kRows;  // warp of each team, its row
      float2 ml[TEAMS];
      float top = -INFINITY, L = 0.0f, acc[4] = {};
#pragma unroll
      for (int t = 0; t < TEAMS; ++t) {
        ml[t] = sm.join_ml[t * WT + from][in];
        top = fmaxf(top, ml[t].x);
      }
      const float zero = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int t = 0; t < TEAMS; ++t) {
        const float e = ex2(ml[t].x - zero);
        const float4 v = sm.join[t * WT + from][in][Math::place(in, lane)];
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
        constexpr int kAhead = 8;  // accumulators in flight beside the maxima (16: code that every call fetches
                                   // once, 0.3 us of 8)
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

template <typename Math, int WT>
cudaError_t launch_rows(const BlockAttnParams& p, int sms, cudaStream_t st) {
  constexpr int smem = (int)sizeof(AttnSmem<BlockWalk<Math::kRows * WT>>);
  static std::atomic<long long> memo[kMemoDevices];
  const cudaError_t e = ensure_smem_limit(block_attn_kernel<Math, WT>, memo, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(block_attn_kernel<Math, WT>, dim3(sms), dim3(kThreadsAttn), smem, st, p);
}

}  // namespace

cudaError_t launch_block_attn(const BlockAttnParams& p, int sms, int rows, cudaStream_t st) {
  switch (rows) {
    case 8: return launch_rows<Rows<1>, 1>(p, sms, st);
    case 16: return launch_rows<Rows<2>, 1>(p, sms, st);
    case 32: return launch_rows<Rows<2>, 2>(p, sms, st);
    default: return launch_rows<Rows<2>, 4>(p, sms, st);
  }
}

}  // namespace kvq
