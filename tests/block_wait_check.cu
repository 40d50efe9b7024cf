// The block attention where a bounded wait runs out, on the GPU: the wait of the
// kernels is replaced by one that answers "ran out" at a chosen time to a chosen
// warp (or to one lane of it) of every third CTA, as the limit itself would.  For
// every number of rows the kernel ends, its counters are zero, a call after it on
// the same workspace is right, and a row is NaN as a whole or what it is without.
// Prints "bad <count>".
#include "../bit_kv_cache_07_gb300/csrc/kvq_pipe.cuh"

namespace kvq {
struct Out {  // when a wait answers so: the call-th of a warp's waits (all of them: every), to lane (-1: all)
  int warp, call, lane, every;
};
__device__ Out g_out;
__device__ int g_calls[152][256];
__device__ inline bool mbar_wait_or_out(uint32_t bar, uint32_t phase, volatile int* gave_up) {
  if (gave_up) {  // (null: a wait for copies in flight, never cut short)
    const Out o = g_out;
    const int n = g_calls[blockIdx.x][threadIdx.x]++;
    const bool here = blockIdx.x % 3 == 1 && (int)(threadIdx.x >> 5) == o.warp && (o.lane < 0 || (int)(threadIdx.x & 31) == o.lane);
    if (o.every || (here && n == o.call)) {
      *gave_up = 1;
      return false;
    }
  }
  return mbar_wait(bar, phase, gave_up);
}
}  // namespace kvq
#define mbar_wait mbar_wait_or_out
#include "../bit_kv_cache_07_gb300/csrc/kvq_block_attn.cu"

#include <cmath>
#include <cstdio>
#include <cstring>
#include <vector>
using namespace kvq;

template <typename T>
static T* on_gpu(const std::vector<T>& v) {
  T* d = nullptr;
  cudaMalloc(&d, v.size() * sizeof(T) + 16);
  cudaMemcpy(d, v.data(), v.size() * sizeof(T), cudaMemcpyHostToDevice);
  return d;
}
static bool is_nan(uint16_t h) { return (h & 0x7fff) > 0x7c00; }

int main(int argc, char** argv) {
  const bool later = argc > 1;  // waits after the first, too
  unsigned long long rs = 88172645463325252ull;
  const auto rnd = [&](int n) { rs ^= rs << 13; rs ^= rs >> 7; rs ^= rs << 17; return (int)(rs % n); };
  // long requests, which span CTAs, and short ones, which one team takes
  std::vector<int> lens, start(1, 0), table;
  const int B = 60, most = 400;
  for (int b = 0; b < B; ++b) {
    lens.push_back(b % 6 == 0 ? 6000 + rnd(6000) : 40 + rnd(300));
    start.push_back(start.back() + 1 + rnd(b % 5 ? 1 : 9));
  }
  BlockAttnParams p;
  std::memset(&p, 0, sizeof(p));
  const int g = 4, Hkv = 2, N = start.back();
  int blocks = 0;
  table.assign((size_t)B * most, 0);
  for (int b = 0; b < B; ++b)
    for (int j = 0; j < (lens[b] + 31) / 32; ++j) table[(size_t)b * most + j] = blocks++;
  p.geo = BlockGeo{B, N, g * Hkv, Hkv, g, blocks, most};
  std::vector<uint8_t> codes((size_t)blocks * Hkv * kPairBytes), scales(((size_t)blocks * Hkv * 2 + 15) / 16 * 16);
  for (auto& x : codes) x = (uint8_t)((rnd(2) << 7) | (0x28 + rnd(0x20)));
  for (auto& x : scales) x = (uint8_t)(127 - 4 + rnd(3));
  std::vector<uint16_t> q((size_t)N * g * Hkv * 128), empty(q.size(), 0x1234);
  for (auto& x : q) x = (uint16_t)((rnd(2) << 15) | (0x3000 + rnd(0xC00)));
  p.t.lens = on_gpu(lens), p.t.start = on_gpu(start), p.t.block_table = on_gpu(table);
  p.codes = on_gpu(codes), p.scales = on_gpu(scales), p.q = on_gpu(q), p.out = on_gpu(empty);
  const size_t rows = q.size() / 128;
  p.lse = on_gpu(std::vector<float>(rows));
  p.counters = on_gpu(std::vector<unsigned>(kMaxBlockCtas, 0u));
  p.part_ml = on_gpu(std::vector<float>(2 * kMaxBlockCtas * kMaxBlockRows * 2));
  p.part_acc = on_gpu(std::vector<float>(2 * kMaxBlockCtas * kMaxBlockRows * 128));
  p.q_scale = 0.0883883476f * 1.44269504f;
  p.window = kNoWindow, p.g_inv = (unsigned)(((1ull << 32) + g - 1) / g);

  int bad = 0, spoilt = 0, runs = 0;
  std::vector<uint16_t> want(q.size()), out(q.size());
  std::vector<float> want_lse(rows), lse(rows);
  std::vector<unsigned> counters(kMaxBlockCtas);
  const auto run = [&](int width, Out o, std::vector<uint16_t>& to, std::vector<float>& to_lse) {
    cudaMemcpyToSymbol(g_out, &o, sizeof(o));
    static const int zero[152][256] = {};
    cudaMemcpyToSymbol(g_calls, zero, sizeof(zero));
    cudaMemset(p.out, 0x11, q.size() * 2);
    if (launch_block_attn(p, 152, width, nullptr) != cudaSuccess) return false;
    cudaMemcpy(to.data(), p.out, q.size() * 2, cudaMemcpyDeviceToHost);
    cudaMemcpy(to_lse.data(), p.lse, rows * 4, cudaMemcpyDeviceToHost);
    cudaMemcpy(counters.data(), p.counters, counters.size() * 4, cudaMemcpyDeviceToHost);
    for (unsigned c : counters) bad += c != 0;
    ++runs;
    return cudaGetLastError() == cudaSuccess;
  };
  const Out none = {-1, 0, 0, 0};
  for (const int width : {8, 16, 32, 64}) {
    if (!run(width, none, want, want_lse)) return printf("%s, bad 1\n", cudaGetErrorString(cudaGetLastError())), 1;
    for (size_t r = 0; r < rows; ++r) bad += !std::isfinite(want_lse[r]) || is_nan(want[r * 128]);
    const auto check = [&](Out o, bool all) {
      if (!run(width, o, out, lse)) return ++bad, false;
      for (size_t r = 0; r < rows; ++r) {
        int nans = 0;
        for (int c = 0; c < 128; ++c) nans += is_nan(out[r * 128 + c]);
        const bool gone = nans == 128 && std::isnan(lse[r]);
        spoilt += gone;
        if (gone) continue;
        bad += all || std::memcmp(&out[r * 128], &want[r * 128], 256) || std::memcmp(&lse[r], &want_lse[r], 4);
      }
      return true;
    };
    if (!check({0, 0, -1, 1}, true)) break;  // every wait, at once: every row
    for (int warp = 0; warp < 8; ++warp)
      for (const int call : later ? std::vector<int>{0, 1, 2, 3, 5, 9, 14, 20, 33} : std::vector<int>{})
        for (const int lane : {-1, 7}) check({warp, call, lane, 0}, false);
    if (!run(width, none, out, lse)) return printf("%s, bad 1\n", cudaGetErrorString(cudaGetLastError())), 1;
    bad += out != want || std::memcmp(lse.data(), want_lse.data(), rows * 4);
  }
  bad += spoilt == 0;
  printf("%s, %d runs, %d rows spoilt, bad %d\n", cudaGetErrorString(cudaGetLastError()), runs, spoilt, bad);
  return bad != 0;
}
