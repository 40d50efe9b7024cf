// Host check of what the merge of the tree attention makes of partial results
// whose CTA gave up (NaN maxima and sums, flags as the scratch held them): for
// uniform and ragged calls, with and without drafted tokens, the partial
// results of the rows cover every slot once, lie in the scratch, and none
// sends the merge to the drafted tokens.  Prints "bad <count>".
#include "../bit_kv_cache_07_gb300/csrc/kvq_tree.cuh"
#include <cmath>
#include <cstdio>
#include <cstring>
#include <vector>
using namespace kvq;

int main() {
  unsigned long long rs = 88172645463325252ull;
  auto rnd = [&](int n) { rs ^= rs << 13; rs ^= rs >> 7; rs ^= rs << 17; return (int)(rs % n); };
  int bad = 0, reads = 0;
  static TreeParams p;
  for (int trial = 0; trial < 400; ++trial) {
    std::memset(&p, 0, sizeof(p));
    Geometry& G = p.geo;
    G.B = 1 + rnd(5), G.Hkv = 1 + rnd(3), G.g = 1 + rnd(4), G.NS = G.B * G.Hkv;
    G.S = rnd(2) * 4, G.R = rnd(2) * 32, G.fp16_mode = rnd(4) == 0;
    if (G.fp16_mode) G.S = G.R = 0;
    static uint32_t some_mask;
    p.mask = rnd(2) ? &some_mask : nullptr;
    p.n = 1 + rnd(rnd(2) ? 4 : 90);
    const int rows = G.g * p.n;
    p.rblk = rows <= 16 ? 16 : 128, p.sub = rows <= 16 ? 6 : 1;
    p.rstride = rows <= 16 ? 16 : rows < 128 ? (rows + 15) / 16 * 16 : 128;
    long long total = 0, pairs = 0;
    for (int b = 0; b < G.B; ++b) {
      const int nb = rnd(4) ? 1 + rnd(p.n) : 0, T = rnd(3) ? rnd(3000) : 0;
      const TileCounts tc = tile_counts(G, T, p.mask ? nb : 0);
      const long long heads = (long long)G.Hkv * ((G.g * nb + p.rblk - 1) / p.rblk);
      p.rows.tokens[b] = T, p.rows.nodes[b] = nb, p.rows.tile0[b] = (int)total, p.rows.pair0[b] = (int)pairs;
      pairs += heads, total += heads * (tc.qt + tc.ft);
    }
    p.rows.tile0[G.B] = (int)total, p.rows.pair0[G.B] = (int)pairs;
    p.total = (int)total;
    const int most = 1 + rnd(160);
    p.ncta = (int)(total < most ? total : most);
    const size_t slots = kMaxSpecCtas + 2ull * G.NS * ((rows + p.rblk - 1) / p.rblk);
    std::vector<int> readers(slots * p.sub, 0);
    const float2 given_up = {NAN, NAN}, whole = {1.0f, 2.0f};
    if (names_drafted(p, given_up, 0xFFFFFFFFu) || names_drafted(p, whole, 0) || names_drafted(p, whole, 1) != (p.mask != nullptr)) ++bad;
    for (int b = 0; b < G.B; ++b) {
      const int nb = p.rows.nodes[b], M = G.g * nb, nrb = (M + p.rblk - 1) / p.rblk;
      const TileCounts tc = tile_counts(G, p.rows.tokens[b], p.mask ? nb : 0);
      for (int h = 0; h < G.Hkv; ++h)
        for (int rb = 0; rb < nrb; ++rb)
          for (int kind = 0; kind < 2; ++kind) {
            const PartSpan s = part_span(p, tc, b, h * nrb + rb, kind);
            for (size_t i = s.at; i < s.at + s.n; ++i, ++reads)
              if (i >= readers.size() || readers[i]++) ++bad;
          }
    }
  }
  if (reads < 50000) ++bad;
  printf("reads %d bad %d\n", reads, bad);
  return bad != 0;
}
