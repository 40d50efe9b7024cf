// Host check of the block append's split (csrc/kvq_block.cuh): over the sizes that the
// configuration allows and GPUs of 1 to 256 SMs, every head of keys, values and
// queries lies in one CTA's share, shares are even, the touched blocks have a CTA
// each; of two GPUs the one with more SMs never gets more heads per CTA, and the
// split follows from rows per SM: twice the SMs and twice the tokens (and requests)
// split a token's heads alike.  Prints "bad <count>".
#include "../bit_kv_cache_07_gb300/csrc/kvq_block.cuh"
#include <cstdio>
using namespace kvq;

static unsigned long long rs = 88172645463325252ull;
static int rnd(int n) { rs ^= rs << 13; rs ^= rs >> 7; rs ^= rs << 17; return (int)(rs % (unsigned)n); }

int main() {
  int bad = 0, several = 0, uneven = 0;
  for (int trial = 0; trial < 200000; ++trial) {
    BlockGeo G = {};
    G.B = 1 + rnd(rnd(2) ? 8 : kMaxBlockBatch);
    G.Hkv = 1 + rnd(rnd(2) ? 12 : 200), G.g = 1 + rnd(8), G.Hq = G.Hkv * G.g;
    G.N = 1 + rnd(rnd(3) ? 20000 : 1 << 19);
    if ((long long)G.N * G.Hq > 1 << 29) continue;
    const bool queries = rnd(3) > 0;
    const int sms = 1 + rnd(rnd(2) ? 256 : 152);
    const AppendSplit s = append_split(G, queries, sms);
    const int last = G.Hkv - (s.kv_chunks - 1) * s.heads_per_cta;
    if (s.heads_per_cta < 1 || last < 1 || last > s.heads_per_cta || s.heads_per_cta - last >= s.kv_chunks) ++bad;
    const int last_q = G.Hq - (s.q_chunks - 1) * s.heads_per_warp;
    if (s.heads_per_warp < 1 || last_q < 1 || last_q > s.heads_per_warp) ++bad;
    const int step = s.few ? kWarpTokens : 8 * kWarpTokens;
    if (s.ctas != (long long)s.units * s.kv_chunks + (queries ? (long long)((G.N + step - 1) / step) * s.q_chunks : 0)) ++bad;
    // the most blocks that N tokens of B requests touch: as many requests as there are pairs of
    // tokens lie over a border, the rest fill blocks
    const int pairs = G.N / 2 < G.B ? G.N / 2 : G.B;
    const int single = G.N - 2 * pairs && pairs < G.B ? 1 : 0;
    if (s.units < 2 * pairs + single || s.units > G.N) ++bad;
    if (append_split(G, queries, sms + 1 + rnd(100)).heads_per_cta > s.heads_per_cta) ++bad;
    BlockGeo two = G;
    two.N *= 2, two.B *= 2;
    if (two.B <= kMaxBlockBatch && append_split(two, queries, 2 * sms).heads_per_cta != s.heads_per_cta) ++bad;
    several += s.heads_per_cta > 1, uneven += last != s.heads_per_cta;
  }
  if (several < 1000 || uneven < 100) ++bad;
  printf("several %d uneven %d bad %d\n", several, uneven, bad);
  return bad != 0;
}
