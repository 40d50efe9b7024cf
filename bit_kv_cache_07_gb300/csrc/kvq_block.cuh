// kvq_block.cuh -- what the calls on the block cache share: sizes, parameters,
// what the device-side tables say of a request, and its visible tiles.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr int kBlockTokens = 32;
constexpr int kMaxBlockBatch = 1024;
constexpr int kBlockSide = kBlockTokens * kHeadDim;  // bytes of a block's keys (or values) of one head
constexpr int kScaleBias = 127;                      // E8M0: 2^(byte - 127)
constexpr int kScaleNaN = 255;
constexpr int kMinExp = -40, kMaxExp = 40;           // exponents that the append gives

struct BlockGeo {
  int B, N, Hq, Hkv, g, n_blocks, max_blocks;
};

// What the tables say of request b.  Anything that the plan would not write
// makes n 0: the request is left out.
struct BlockRequest {
  int n;       // tokens of the step
  int first;   // their first token slot
  int before;  // tokens held before them
};
__host__ __device__ inline BlockRequest block_request(const BlockGeo& G, int len, int start, int end) {
  BlockRequest r;
  r.first = start;
  r.n = 0;
  r.before = len;
  if (start < 0 || end <= start || end > G.N || len < end - start || len > G.max_blocks * kBlockTokens) return r;
  r.n = end - start;
  r.before = len - r.n;
  return r;
}

struct BlockPlanParams {
  BlockGeo geo;
  kvq_block_tables t;
  const int *lens_before, *free_before, *n_new;
  const int* n_back;  // or null
};

struct BlockAppendParams {
  BlockGeo geo;
  kvq_block_tables t;
  uint8_t *codes, *scales;
  const uint16_t *k, *v, *q, *q_weight, *k_weight;
  uint16_t* q_out;
  long long ks, vs, qs;  // elements from a token slot to the next
  int rotate;
  float eps;
  int units, heads_per_cta, kv_chunks, heads_per_warp, q_chunks;
  unsigned long long freq[kHeadDim / 2];  // turns per position, times 2^64
};

struct BlockAttnParams {
  BlockGeo geo;
  kvq_block_tables t;
  const uint8_t *codes, *scales;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  unsigned* counters;  // [CTAs] tickets
  float* part_ml;      // [2 CTAs][rows][2]
  float* part_acc;     // [2 CTAs][rows][128]
  float q_scale;       // softmax_scale * log2(e)
  int window, n_first; // window: kNoWindow or 1..
  unsigned g_inv;      // ceil(2^32 / g), g > 1
};
constexpr int kNoWindow = 1 << 30;
constexpr int kMaxBlockCtas = 256;
constexpr int kMaxBlockRows = 64;  // (token, head) rows that read a KV head's blocks together

// The blocks that rows of tokens i0..i1 of a request see: the first `ns`, then
// those from `lo` on, `cnt` in all.
struct BlockTiles {
  int ns, lo, cnt;
};
__host__ __device__ inline BlockTiles block_tiles(int window, int n_first, int p0, int p1) {
  BlockTiles t;
  const int hi = p1 / kBlockTokens;
  t.ns = 0;
  t.lo = 0;
  if (window < kNoWindow) {
    const int f = n_first > p1 ? p1 + 1 : n_first;
    t.ns = (f + kBlockTokens - 1) / kBlockTokens;
    const int w0 = p0 - window + 1;
    t.lo = w0 > 0 ? w0 / kBlockTokens : 0;
    if (t.lo < t.ns) t.lo = t.ns;
  }
  t.cnt = t.ns + (hi >= t.lo ? hi - t.lo + 1 : 0);
  return t;
}
// The most blocks that any `rows` consecutive (token, head) rows of a request see.
__host__ __device__ inline int block_tiles_max(int window, int n_first, const BlockRequest& r, int g, int rows) {
  if (r.n * g <= rows) return block_tiles(window, n_first, r.before, r.before + r.n - 1).cnt;
  const int all = (r.before + r.n - 1) / kBlockTokens + 1;
  if (window >= kNoWindow) return all;
  const int last = r.before + r.n - 1;
  const int f = n_first > last ? last + 1 : n_first;
  const int span = (rows + g - 1) / g + 1;  // tokens that `rows` rows touch, at most
  const long long wide = ((long long)window + span + kBlockTokens - 3) / kBlockTokens + 1;
  const long long most = (f + kBlockTokens - 1) / kBlockTokens + wide;
  return most < all ? (int)most : all;
}

// ------------------------------------------------- the append's split
constexpr int kRowLanes = 8;  // lanes that hold a token's row of a head
constexpr int kWarpTokens = 32 / kRowLanes;
struct AppendSplit {
  bool few;                     // one warp per CTA, else eight
  int units;                    // touched blocks, at most
  int heads_per_cta, kv_chunks; // heads of a block's CTA, CTAs of a block
  int heads_per_warp, q_chunks; // heads of a query warp, CTAs of its token slots
  long long ctas;
};
inline AppendSplit append_split(const BlockGeo& G, bool queries, int sms) {
  AppendSplit s;
  // no more blocks are touched: each request's tokens start one and end one
  const long long most = (long long)G.N / kBlockTokens + 2ll * G.B;
  s.units = (int)(most < G.N ? most : G.N);
  // eight warps hold a whole block's tokens; up to four tokens per request (drafted
  // chains, single tokens) fill one warp
  s.few = (G.N + G.B - 1) / G.B <= kWarpTokens;
  const int step = kWarpTokens * (s.few ? 1 : 8);
  // heads of a block's CTA: many, since its look-ups and sines are paid once and the
  // next head's rows are read meanwhile.  Up to four as long as the call's rows give
  // each SM its three CTAs (43 prompts of 255 tokens of 4 heads 11.9 us in one CTA, 15.5
  // in four; 51 of 80 tokens of 16 on 8 heads 14.0 in two, 18.5 in eight), more only
  // while a CTA has no more than an eighth of an SM's share (the last CTAs to start are
  // then short beside the call: prompts of 32 on 8 heads 57.4 us with all heads in a
  // CTA, 59.8 in two, 64.2 in four; of 32 heads 105.9 in two, 109.4 in one, 110.3 in
  // four)
  const long long all_rows = (long long)G.N * (2 * G.Hkv + (queries ? G.Hq : 0));
  const long long per_sm = all_rows / (2ll * kBlockTokens * sms);  // CTAs of one head
  const long long up_to_four = per_sm / 3 < 4 ? per_sm / 3 : 4, share = s.few ? 1 : per_sm / 8 > up_to_four ? per_sm / 8 : up_to_four;
  s.heads_per_cta = (int)(share < 1 ? 1 : share > G.Hkv ? G.Hkv : share);
  s.kv_chunks = (G.Hkv + s.heads_per_cta - 1) / s.heads_per_cta;
  s.heads_per_cta = (G.Hkv + s.kv_chunks - 1) / s.kv_chunks;  // (evenly)
  // heads of a query warp: more share a token's sines, fewer spread a small call
  // over the SMs
  const long long rows = (long long)G.N * G.Hq;
  s.heads_per_warp = (int)(rows >= 8ll * 16384 ? 8 : rows >= 16384 ? rows / 16384 : 1);
  s.q_chunks = (G.Hq + s.heads_per_warp - 1) / s.heads_per_warp;
  s.ctas = (long long)s.units * s.kv_chunks + (queries ? (long long)((G.N + step - 1) / step) * s.q_chunks : 0);
  return s;
}

// ------------------------------------------------- the attention's schedule
// The tiles of all (request, head, row block) lie end to end; CTA c takes
// [c per, (c + 1) per).  (Shared with a host check.)
constexpr int kBlockWarps = 8;
// A CTA's range: at least a tile for each of its warps.
__host__ __device__ inline long long block_range(long long total, int ctas) {
  const long long per = udiv(total + ctas - 1, ctas);
  return per < kBlockWarps ? kBlockWarps : per;
}
// Where CTA c leaves its part of what begins at x and spans CTAs: a CTA has at
// most two such parts, the one that its range begins with and the one that it
// ends with.
__host__ __device__ inline int piece_slot(long long x, long long per, int c) { return 2 * c + (x > c * per ? 1 : 0); }

__host__ __device__ inline BlockRequest request_at(const BlockAttnParams& p, int b) {
#ifdef __CUDA_ARCH__
  return block_request(p.geo, __ldg(p.t.lens + b), __ldg(p.t.start + b), __ldg(p.t.start + b + 1));
#else
  return block_request(p.geo, p.t.lens[b], p.t.start[b], p.t.start[b + 1]);
#endif
}

// What a (request, head, row block) costs beyond its tiles, in tiles: the teams'
// parts are joined (64 ragged requests to 8k tokens: 51.7 us where that weighs 8
// tiles, 49.4 with 12, 49.2 with 16, 49.9 with 20; one request of 8k: 12.7, 12.7, 10.4,
// 10.5), or one team takes it alone and the others go on (256 requests of 200 tokens:
// 44.7 us where that ends at 4 tiles, 27.5 at 8 and at 12; the ragged batch 48.2, 49.2,
// 49.1).
constexpr int kSoloTiles = 8;
constexpr int kJoinTiles = 16;
// Short ones are not cut between CTAs, which would have to join them: up to
// kUncutTiles, where ranges that end with whole ones are at most kUncutExtra tiles
// longer (16 requests of 1000 tokens: 15.0 us where that ends at 24 tiles, 10.2 at 48;
// one of 1024 tokens, one head: 8.3 us cut, 9.0 whole, as with an extra of 64).
constexpr int kUncutTiles = 48;
constexpr int kUncutExtra = 16;
__host__ __device__ inline bool block_uncut(int cnt, long long per) {
  if (cnt > kUncutTiles) return false;
  const int range = per < (1 << 30) ? (int)per : 1 << 30;
  return (range / cnt + 1) * (long long)cnt - range <= kUncutExtra;  // (as many begin in a range, at most)
}

// One segment: tiles k0..k1 of a (request, head, row block).
struct BlockSegment {
  int b, h, first, before, n;  // request
  int r0, rows;                // rows of the block
  int k0, k1, ns, lo;          // its visible tiles in the CTA's range (k1 <= the block's own count)
  long long x;                 // where the (request, head, row block) begins
  int cnt;                     // and its own count of tiles
  bool whole;                  // the CTA has all of it

  // Whether one of the CTA's teams takes it by itself, with nothing to join: it is
  // short, and the range holds enough of its like for the other teams.
  __host__ __device__ bool solo(long long per, int teams) const {
    return whole && cnt <= kSoloTiles && (long long)cnt * teams <= 2 * per;
  }
};

// A CTA's range of tiles, of ranges of `per`.
struct BlockRange {
  long long x0, x1, per;
};

template <int ROWS>
struct BlockWalk {
  long long x;      // where it is
  int b, j, k;      // next: request, (head, row block) of it, tile
  int streams, nrb, cnt;  // cnt: tiles of a (head, row block) in the schedule, what it costs beyond them included
  bool uncut;
  BlockRequest r;

  __host__ __device__ inline void load(const BlockAttnParams& p, const BlockRange& g) {
    r = request_at(p, b);
    size(p, r, &nrb, &streams, &cnt);
    uncut = block_uncut(cnt, g.per);
  }
  __host__ __device__ static inline void size(const BlockAttnParams& p, const BlockRequest& r, int* nrb, int* streams, int* cnt) {
    *nrb = (int)(((long long)r.n * p.geo.g + ROWS - 1) / ROWS);
    *streams = *nrb * p.geo.Hkv;
    const int most = r.n ? block_tiles_max(p.window, p.n_first, r, p.geo.g, ROWS) : 0;
    *cnt = most + (most > kSoloTiles ? kJoinTiles : 1);
  }
  // the range g, whose first tile is tile x0 - xb of request b
  __host__ __device__ inline void begin(const BlockAttnParams& p, const BlockRange& g, int b_, long long xb) {
    x = g.x0, b = b_;
    load(p, g);
    const long long at = x - xb;
    j = (int)udiv(at, cnt);
    k = (int)(at - (long long)j * cnt);
  }
  __host__ __device__ inline bool next(const BlockAttnParams& p, const BlockRange& g, BlockSegment& s) {
    const BlockGeo& G = p.geo;
    while (x < g.x1) {
      while (j >= streams) {
        if (++b >= G.B) return false;
        j = 0;
        load(p, g);
      }
      const int M = r.n * G.g;
      int p0 = r.before, p1 = r.before + r.n - 1;
      s.h = j, s.r0 = 0, s.rows = M;
      if (nrb > 1) {
        s.h = j / nrb;
        s.r0 = (j - s.h * nrb) * ROWS;
        s.rows = M - s.r0 < ROWS ? M - s.r0 : ROWS;
        p1 = p0 + (s.r0 + s.rows - 1) / G.g;
        p0 += s.r0 / G.g;
      }
      const BlockTiles t = block_tiles(p.window, p.n_first, p0, p1);
      // (one that is not cut belongs to the range that it begins in)
      const long long left = g.x1 - x;
      const int end = uncut || left >= cnt - k ? cnt : k + (int)left;
      s.b = b, s.first = r.first, s.before = r.before, s.n = r.n;
      s.k0 = k;
      s.k1 = end < t.cnt ? end : t.cnt;
      s.ns = t.ns, s.lo = t.lo;
      s.x = x - k;
      s.cnt = t.cnt;
      s.whole = uncut || (s.x >= g.x0 && s.x + t.cnt <= g.x1);
      const bool here = uncut ? k == 0 : s.k0 < s.k1;  // (or the range begins behind its tiles)
      x += end - k;
      k = 0;
      ++j;
      if (here) return true;
    }
    return false;
  }
};
__host__ __device__ inline int tile_of(const BlockSegment& s, int k) { return k < s.ns ? k : s.lo + (k - s.ns); }

cudaError_t launch_block_plan(const BlockPlanParams& p, cudaStream_t st);
cudaError_t launch_block_append(BlockAppendParams& p, int sms, cudaStream_t st);
cudaError_t launch_block_attn(const BlockAttnParams& p, int sms, int rows, cudaStream_t st);

}  // namespace kvq
