// Host check of the block attention's schedule (csrc/kvq_block.cuh): for random
// batches, windows, group sizes and CTA counts, every visible block of every
// (request, head, row block) is read by exactly one CTA, none is read that no row
// sees or that lies behind the request's table row, the parts of what spans CTAs
// lie in distinct slots and are as many as the joining CTA expects, and tables
// that the plan would not write leave their requests out.  Prints "bad <count>".
#include <cstdio>
#include <cstring>
#include <map>
#include <set>
#include <tuple>
#include <vector>
#include "../bit_kv_cache_07_gb300/csrc/kvq_block.cuh"
using namespace kvq;

static unsigned long long rs = 88172645463325252ull;
static int rnd(int n) { rs ^= rs << 13; rs ^= rs >> 7; rs ^= rs << 17; return (int)(rs % (unsigned)n); }

template <int ROWS>
static int trial() {
  BlockAttnParams p;
  std::memset(&p, 0, sizeof(p));
  BlockGeo& G = p.geo;
  G.B = 1 + rnd(rnd(3) ? 6 : 200), G.Hkv = 1 + rnd(4), G.g = 1 + rnd(8), G.Hq = G.Hkv * G.g, G.n_blocks = 1000;
  G.max_blocks = 1 + rnd(rnd(2) ? 6 : 90);
  p.window = rnd(2) ? kNoWindow : 1 + rnd(rnd(2) ? 70 : 1500);
  p.n_first = rnd(2) ? 0 : rnd(rnd(2) ? 5 : 200);
  std::vector<int> lens(G.B), start(G.B + 1, 0);
  for (int b = 0; b < G.B; ++b) {
    lens[b] = rnd(32 * G.max_blocks + 1);
    const int n = rnd(4) ? rnd(4) : rnd(120);
    start[b + 1] = start[b] + (n < lens[b] ? n : lens[b]);
  }
  G.N = start[G.B] ? start[G.B] : 1;
  if (rnd(8) == 0) lens[rnd(G.B)] = rnd(2) ? -1 : 32 * G.max_blocks + 1 + rnd(100);  // out of range
  if (rnd(8) == 0 && G.B > 1) start[1 + rnd(G.B - 1)] = rnd(2) ? -3 : G.N + 7;
  p.t.lens = lens.data(), p.t.start = start.data();
  long long total = 0;
  std::vector<long long> first(G.B + 1, 0);
  std::map<std::tuple<int, int, int>, std::set<int>> want, got;
  for (int b = 0; b < G.B; ++b) {
    const BlockRequest r = request_at(p, b);
    int nrb, streams, cnt;
    BlockWalk<ROWS>::size(p, r, &nrb, &streams, &cnt);
    first[b] = total;
    total += (long long)streams * cnt;
    for (int h = 0; h < G.Hkv; ++h)
      for (int row = 0; row < r.n * G.g; ++row) {
        const int pos = r.before + row / G.g;
        auto& set = want[std::make_tuple(b, h, row / ROWS)];
        if (r.n * G.g > 40 && row % 7 && row % ROWS && row % ROWS != ROWS - 1 && row != r.n * G.g - 1) continue;
        for (int t = 0; t <= pos; ++t)
          if (pos - t < p.window || t < p.n_first) set.insert(t / kBlockTokens);
      }
  }
  first[G.B] = total;
  const int ctas = 1 + rnd(rnd(2) ? 152 : kMaxBlockCtas);
  const long long per = block_range(total, ctas);
  int bad = 0;
  std::map<std::tuple<int, int, int>, int> parts;
  std::map<std::tuple<int, int, int>, int> expect;
  std::set<int> slots;
  for (int c = 0; c < ctas; ++c) {
    const long long x0 = per * c, x1 = total < x0 + per ? total : x0 + per;
    if (x0 >= x1) continue;
    int b0 = 0;
    while (!(x0 >= first[b0] && x0 < first[b0 + 1])) ++b0;
    BlockWalk<ROWS> w;
    const BlockRange range{x0, x1, per};
    w.begin(p, range, b0, first[b0]);
    BlockSegment s;
    while (w.next(p, range, s)) {
      const auto key = std::make_tuple(s.b, s.h, s.r0 / ROWS);
      if (s.rows < 1 || s.rows > ROWS || s.first < 0 || s.first + (s.r0 + s.rows - 1) / G.g >= G.N || s.h < 0 || s.h >= G.Hkv) ++bad;
      for (int k = s.k0; k < s.k1; ++k) {
        const int tile = tile_of(s, k);
        if (tile < 0 || tile >= G.max_blocks || !got[key].insert(tile).second) ++bad;
      }
      const bool whole = s.whole;
      const int c0 = (int)(s.x / per), c1 = (int)((s.x + s.cnt - 1) / per);
      if (s.k0 >= s.k1 || c < c0 || c > c1 || (whole ? s.k0 != 0 || s.k1 != s.cnt : c0 == c1)) ++bad;
      if (!whole) {
        ++parts[key];
        expect[key] = c1 - c0 + 1;
        const int slot = piece_slot(s.x, per, c);
        if (slot < 0 || slot >= 2 * kMaxBlockCtas || !slots.insert(slot).second || c0 >= kMaxBlockCtas) ++bad;
      } else {
        parts[key] = expect[key] = 1;
      }
    }
  }
  for (const auto& kv : want) {
    const std::set<int>& g = got[kv.first];
    for (int t : kv.second)
      if (!g.count(t)) ++bad;
    // (a block that only a row between the sampled ones sees lies between theirs)
    if (*g.begin() < *kv.second.begin() || *g.rbegin() > *kv.second.rbegin()) ++bad;
    if (parts[kv.first] != expect[kv.first]) ++bad;
  }
  for (const auto& kv : got)
    if (!want.count(kv.first) && !kv.second.empty()) ++bad;
  return bad;
}

int main() {
  int bad = 0;
  for (int i = 0; i < 400; ++i) bad += trial<8>() + trial<16>() + trial<32>() + trial<64>();
  printf("bad %d\n", bad);
  return bad != 0;
}
