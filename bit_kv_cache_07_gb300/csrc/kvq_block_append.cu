// kvq_block_append.cu -- norm, rotation and 8-bit store of a step's keys and
// values, and the queries made ready, in one launch.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (y_i, y_{i+64}) turned by position * f_i
//   e = least exponent with max |y| <= 448 2^e over the block's tokens of a head,
//   code = e4m3(y 2^-e)
//
// Eight lanes hold a token's row of a head: lane l the channels 8l..8l+7 and
// 64+8l..64+8l+7, so that both of a rotated pair are in one lane, loads are two
// 16-byte words and the mean is three shuffles.  A CTA takes one block and several
// heads: keys, then values of each, read once (in registers between the one maximum
// over the CTA and the store) while the next two heads' are on the way to shared
// memory; the sines are the block's.  Calls of few tokens per request run the
// same with one warp per CTA, which walks a longer run of tokens twice.  The
// queries go to CTAs of their own: a warp turns four tokens' rows head after
// head with the same sines.
//
// Angles: position times a 64-bit fraction of a turn, whose top 32 bits are the
// angle.  The fraction is off by less than 2^-54 of a turn (a power in doubles, for a
// base of 1 or more), the angle by position 2^-54 turns, its fp32 radians by 5e-7 at
// most; the hardware sine and cosine in [-pi, pi] add 4.2e-7.  Together the
// absolute error stays below 2^-20 up to position 2^25 and below 2^-19 up to 2^30,
// where q_out's own rounding is 2^-11 and a code's 2^-4: the hardware's functions are
// taken for their speed, and show in neither.
#include "kvq_block.cuh"

namespace kvq {

__device__ __forceinline__ void halves_to_floats(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// Channels 8l..8l+7 in v[0..7], 64+8l.. in v[8..15].
__device__ __forceinline__ void load_row(const uint16_t* row, int l, float (&v)[16]) {
  const uint4* at = reinterpret_cast<const uint4*>(row);
  const uint4 a = __ldg(at + l), b = __ldg(at + kRowLanes + l);
  halves_to_floats(a, v);
  halves_to_floats(b, v + 8);
}
// Where pair i's frequency lies: the eight lanes of a row read side by side.
__device__ __forceinline__ int freq_place(int i) { return (i & 7) * 8 + (i >> 3); }
// What turns a row x into y / r (r: the row's own factor of the norm), weights and
// sines of the token together:
//   y_i = a_i x_i - b_i x_{i+64},  y_{i+64} = c_i x_{i+64} + d_i x_i.
struct Turn {
  float a[8], b[8], c[8], d[8];
};
__device__ __forceinline__ void make_turn(Turn& t, const uint16_t* weight, const unsigned long long* freq, bool rotate, int l, int pos) {
  float w[16];
  if (weight) load_row(weight, l, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.a[i] = weight ? w[i] : 1.0f;
    t.c[i] = weight ? w[8 + i] : 1.0f;
    if (rotate) {
      const int turns = (int)(unsigned)((freq[freq_place(8 * l + i)] * (unsigned long long)pos) >> 32);  // [-1/2, 1/2) turns
      const float x = (float)turns * 1.4629180792671596e-9f;                                 // 2 pi / 2^32
      const float cs = __cosf(x), sn = __sinf(x);
      t.b[i] = t.c[i] * sn;
      t.d[i] = t.a[i] * sn;
      t.a[i] *= cs;
      t.c[i] *= cs;
    }
  }
}
__device__ __forceinline__ void apply_turn(const Turn& t, bool weight, bool rotate, float (&v)[16]) {
  if (rotate) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = v[i], y = v[8 + i];
      v[i] = t.a[i] * x - t.b[i] * y;
      v[8 + i] = t.c[i] * y + t.d[i] * x;
    }
  } else if (weight) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= t.a[i];
      v[8 + i] *= t.c[i];
    }
  }
}
// 1 / sqrt(mean x^2 + eps) of the row
__device__ __forceinline__ float norm_factor(const float (&v)[16], float eps) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return rsqrtf(ss * (1.0f / kHeadDim) + eps);
}
// The largest magnitude of the lane's halves; not below infinity where one is not finite.
__device__ __forceinline__ float halves_max(const uint4 (&raw)[2]) {
  const __half2* h = reinterpret_cast<const __half2*>(raw);
  __half2 m = __habs2(h[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(h[i]));
  const float x = __low2float(m), y = __high2float(m);
  return x <= y || isnan(y) ? y : x;  // (a NaN stays one)
}
// The least e in [kMinExp, kMaxExp] with amax <= 448 2^e (448 = 1.75 2^8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  return min(max(e, kMinExp), kMaxExp);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

// Two values as e4m3, nearest, ties to even, at most 448 (low byte: a).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;\n" : "=h"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A unit's request: the last one whose first unit is not behind it.  By a warp: 32
// requests apart where there are more than 32, then between them, with what the
// request's tokens need read beside (each further read would be a latency that
// nothing hides at a CTA's begin).
struct UnitRequest {
  int b, unit0, len, start, end;
};
__device__ __forceinline__ UnitRequest unit_request(const kvq_block_tables& t, int B, int unit, int lane) {
  const int step = (B + 31) / 32;
  int lo = 0;
  if (step > 1) {
    const int far = lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, far < B && __ldg(t.unit0 + far) <= unit);
    lo = (31 - __clz(below | 1u)) * step;
  }
  const int near = lo + lane, at = min(near, B - 1);  // step <= 32
  const int unit0 = __ldg(t.unit0 + at), len = __ldg(t.lens + at), start = __ldg(t.start + at), end = __ldg(t.start + at + 1);
  const unsigned in = __ballot_sync(0xffffffffu, (step == 1 || lane < step) && near < B && unit0 <= unit);
  const int from = 31 - __clz(in | 1u);
  return {lo + from, __shfl_sync(0xffffffffu, unit0, from), __shfl_sync(0xffffffffu, len, from), __shfl_sync(0xffffffffu, start, from),
          __shfl_sync(0xffffffffu, end, from)};
}

// Rows on the way: each thread copies its own 32 bytes of a row into its own slots of
// shared memory (so that no barrier is needed), kRowsAhead rows ahead, and in flight
// they take no registers (prompts of 32 on 8 heads 64.4 to 57.4 us, of 32 heads 126.1
// to 105.5 us against rows on the way in registers; six rows ahead 58.5 and 106.5; four
// CTAs per SM in place of three, in 64 registers, 57.4 and 110.5).
constexpr int kRowsAhead = 4;
template <int WARPS>
struct RowRing {
  uint4 at[kRowsAhead][2][32 * WARPS];
};
__device__ __forceinline__ void copy_chunk(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? 3 : 16) block_append_kernel(const __grid_constant__ BlockAppendParams p) {
  __shared__ unsigned long long s_freq[kHeadDim / 2];
  __shared__ uint32_t s_top[2][WARPS];
  __shared__ RowRing<WARPS> ring;
  const BlockGeo& G = p.geo;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, l = lane & (kRowLanes - 1), sub = lane / kRowLanes;
  if (p.rotate)
    for (int i = tid; i < kHeadDim / 2; i += 32 * WARPS) s_freq[freq_place(i)] = p.freq[i];
  __syncthreads();
  grid_dep_wait();
  grid_dep_trigger();
  int slot = 0;
  // One group of copies per row, empty past the last: after wait<kRowsAhead - 1> the oldest is there.
  const auto ask = [&](const uint16_t* row, bool any) {
    if (any) {
      copy_chunk(&ring.at[slot][0][tid], row + 8 * l);
      copy_chunk(&ring.at[slot][1][tid], row + kHeadDim / 2 + 8 * l);
    }
    copy_commit();
    slot = (slot + 1) % kRowsAhead;
  };
  const auto take = [&](uint4 (&raw)[2]) {  // the oldest row; its slot is the next to ask for
    copy_wait<kRowsAhead - 1>();
    raw[0] = ring.at[slot][0][tid];
    raw[1] = ring.at[slot][1][tid];
    __syncwarp();
  };
  constexpr int kStep = kWarpTokens * WARPS;  // tokens of a CTA at a time
  const int kv_ctas = p.units * p.kv_chunks;

  if ((int)blockIdx.x >= kv_ctas) {  // queries: kStep token slots, heads_per_warp heads
    const int x = blockIdx.x - kv_ctas, group = x / p.q_chunks, chunk = x - group * p.q_chunks;
    const int i = group * kStep + w * kWarpTokens + sub;
    const int pos = p.rotate ? __ldg(p.t.position + min(i, G.N - 1)) : 0;  // (of a row behind the last: unused)
    const int used = min(max(__ldg(p.t.start + G.B), 0), G.N);
    if (group * kStep + w * kWarpTokens >= used) return;
    const bool live = i < used;
    const int row = live ? i : group * kStep + w * kWarpTokens;
    const int h1 = min(G.Hq, (chunk + 1) * p.heads_per_warp);
    const uint16_t* src = p.q + (long long)row * p.qs;
    uint16_t* dst = p.q_out + (long long)row * G.Hq * kHeadDim;
    const int h0 = chunk * p.heads_per_warp;
    // (q_out may be q: a row is read by its own warp only, and whole before it is written)
    for (int u = 0; u < kRowsAhead; ++u) ask(src + (h0 + u) * kHeadDim, h0 + u < h1);
    Turn turn;  // (made while they come)
    make_turn(turn, p.q_weight, s_freq, p.rotate, l, pos);
    for (int h = h0; h < h1; ++h) {
      uint4 raw[2];
      take(raw);
      ask(src + (h + kRowsAhead) * kHeadDim, h + kRowsAhead < h1);
      float v[16];
      halves_to_floats(raw[0], v);
      halves_to_floats(raw[1], v + 8);
      const float r = p.q_weight ? norm_factor(v, p.eps) : 1.0f;
      apply_turn(turn, p.q_weight, p.rotate, v);
      uint4 o[2];
      uint32_t* ow = reinterpret_cast<uint32_t*>(o);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __half2 two = __floats2half2_rn(v[2 * k] * r, v[2 * k + 1] * r);
        ow[k] = *reinterpret_cast<const uint32_t*>(&two);
      }
      if (live) {
        uint4* at = reinterpret_cast<uint4*>(dst + h * kHeadDim);
        at[l] = o[0];
        at[kRowLanes + l] = o[1];
      }
    }
    return;
  }

  // keys and values: heads_per_cta heads of one touched block
  const int unit = blockIdx.x / p.kv_chunks, chunk = blockIdx.x - unit * p.kv_chunks;
  const int units = __ldg(p.t.unit0 + G.B);
  const UnitRequest u = unit_request(p.t, G.B, unit, lane);
  if (unit >= units) return;
  const BlockRequest r = block_request(G, u.len, u.start, u.end);
  if (r.n == 0) return;
  const int j = r.before / kBlockTokens + (unit - u.unit0);
  if (j < 0 || j >= G.max_blocks) return;
  const int p0 = max(r.before, j * kBlockTokens), p1 = min(r.before + r.n, (j + 1) * kBlockTokens);
  if (p0 >= p1) return;
  const int id = __ldg(p.t.block_table + (size_t)u.b * G.max_blocks + j);
  const int off = p0 - j * kBlockTokens, count = p1 - p0;
  const long long slot0 = r.first + (p0 - r.before);
  const int h0 = chunk * p.heads_per_cta, h1 = min(G.Hkv, h0 + p.heads_per_cta);
  constexpr bool kOnce = kStep >= kBlockTokens;  // no run is longer
  const bool again = !kOnce && count > kStep;    // the run is walked twice
  const int t_first = w * kWarpTokens + sub;

  const uint16_t *k_row = p.k + slot0 * p.ks, *v_row = p.v + slot0 * p.vs;
  const auto fetch = [&](int h, int side, int t, uint4 (&raw)[2]) {  // past the run's end: its first token
    const uint4* at = reinterpret_cast<const uint4*>((side ? v_row + (t < count ? t : 0) * p.vs : k_row + (t < count ? t : 0) * p.ks) + h * kHeadDim);
    raw[0] = __ldg(at + l);
    raw[1] = __ldg(at + kRowLanes + l);
  };
  Turn turn;
  float v[16], r_row = 1.0f;
  bool odd_weight = false;
  const auto turn_to = [&](int t) {
    make_turn(turn, p.k_weight, s_freq, p.rotate, l, p0 + (t < count ? t : 0));
    if (p.k_weight) {
      float zeros = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) zeros += turn.a[i] * 0.0f + turn.c[i] * 0.0f;
      odd_weight = !(zeros == 0.0f);
    }
  };
  const auto make = [&](int side, const uint4 (&raw)[2]) {  // y / r_row in v
    halves_to_floats(raw[0], v);
    halves_to_floats(raw[1], v + 8);
    r_row = 1.0f;
    if (side == 0) {
      if (p.k_weight) r_row = norm_factor(v, p.eps);
      apply_turn(turn, p.k_weight, p.rotate, v);
    }
  };
  const uint16_t *k_at = k_row + (t_first < count ? t_first : 0) * p.ks, *v_at = v_row + (t_first < count ? t_first : 0) * p.vs;
  for (int u = 0; u < kRowsAhead / 2; ++u) {
    ask(k_at + (h0 + u) * kHeadDim, h0 + u < h1);
    ask(v_at + (h0 + u) * kHeadDim, h0 + u < h1);
  }
  if (id < 0 || id >= G.n_blocks) {  // (its read was on the way with the rows)
    copy_wait<0>();
    return;
  }
  turn_to(t_first);
  int flip = 0;
  for (int h = h0; h < h1; ++h) {
    const size_t place = (size_t)id * G.Hkv + h;
    for (int side = 0; side < 2; ++side) {
      const uint8_t was = off ? p.scales[place * 2 + side] : 0;
      uint4 raw[2];
      take(raw);
      ask((side ? v_at : k_at) + (h + kRowsAhead / 2) * kHeadDim, h + kRowsAhead / 2 < h1);
      float amax = 0.0f;
      bool bad = false;
      for (int t0 = 0; t0 < (kOnce ? 1 : count); t0 += kStep) {
        if (t0) {
          turn_to(t0 + t_first);
          fetch(h, side, t0 + t_first, raw);
        }
        make(side, raw);
        float m = halves_max(raw);
        bool odd = !(m < INFINITY);
        if (side == 0) {
          m = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
          m *= r_row;
          odd = odd || odd_weight || !(m < INFINITY);
        }
        if (odd) {  // rare: the largest of the others
          bad = true;
          m = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) m = fabsf(v[i] * r_row) < INFINITY ? fmaxf(m, fabsf(v[i] * r_row)) : m;
        }
        amax = fmaxf(amax, m);
      }
      uint32_t top = __float_as_uint(amax);
      top = __reduce_max_sync(0xffffffffu, top);
      bad = __any_sync(0xffffffffu, bad);
      if constexpr (WARPS > 1) {
        if (lane == 0) s_top[flip][w] = top | (bad ? 0x80000000u : 0u);
        __syncthreads();  // (two sets of maxima: those of the time before are read by now)
        const uint32_t x = lane < WARPS ? s_top[flip][lane] : 0u;
        bad = __any_sync(0xffffffffu, x >> 31);
        top = __reduce_max_sync(0xffffffffu, x & 0x7fffffffu);
        flip ^= 1;
      }
      int e = scale_exponent(__uint_as_float(top));
      const bool spoilt = off && was == kScaleNaN;
      uint8_t* block = p.codes + (place * 2 + side) * kBlockSide;
      if (off && !spoilt) {
        const int e_was = was - kScaleBias;
        if (e_was >= e) {
          e = e_was;
        } else {  // earlier tokens move to the larger scale
          const float f = exp2i(max(e_was - e, -126));
          for (int x = tid; x < off * 32; x += 32 * WARPS) {
            uint32_t* at = reinterpret_cast<uint32_t*>(block) + x;
            const uint32_t u = *at;
            const float2 lo = e4m3x2_floats(u & 0xffffu), hi = e4m3x2_floats(u >> 16);
            *at = e4m3x2(lo.x * f, lo.y * f) | e4m3x2(hi.x * f, hi.y * f) << 16;
          }
        }
      }
      const float f = e >= 127 ? 5.877471754111438e-39f : exp2i(-e);
      for (int t0 = 0; t0 < (kOnce ? 1 : count); t0 += kStep) {
        const int t = t0 + t_first;
        if (again) {
          turn_to(t);
          fetch(h, side, t, raw);
          make(side, raw);
        }
        if (bad)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = fabsf(v[i] * r_row) < INFINITY ? v[i] : 0.0f;
        if (t < count) {
          const float fr = bad && !(fabsf(f * r_row) < INFINITY) ? 0.0f : f * r_row;
          uint32_t code[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            code[i] = e4m3x2(v[4 * i] * fr, v[4 * i + 1] * fr) | e4m3x2(v[4 * i + 2] * fr, v[4 * i + 3] * fr) << 16;
          const int tok = off + t;
          uint8_t* at = block + tok * kHeadDim + (l & 1) * 8;
          *reinterpret_cast<uint2*>(at + (((l >> 1) ^ (tok & 7)) << 4)) = make_uint2(code[0], code[1]);
          *reinterpret_cast<uint2*>(at + (((4 + (l >> 1)) ^ (tok & 7)) << 4)) = make_uint2(code[2], code[3]);
        }
      }
      if (again) turn_to(t_first);
      __syncwarp();  // every lane has read the old scale
      if (tid == 0) p.scales[place * 2 + side] = bad || spoilt ? kScaleNaN : (uint8_t)(e + kScaleBias);
    }
  }
}

cudaError_t launch_block_append(BlockAppendParams& p, int sms, cudaStream_t st) {
  const AppendSplit s = append_split(p.geo, p.q != nullptr, sms);
  p.units = s.units;
  p.heads_per_cta = s.heads_per_cta, p.kv_chunks = s.kv_chunks;
  p.heads_per_warp = s.heads_per_warp, p.q_chunks = s.q_chunks;
  if (s.ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  return s.few ? launch_dependent(block_append_kernel<1>, dim3((unsigned)s.ctas), dim3(32), 0, st, p)
               : launch_dependent(block_append_kernel<8>, dim3((unsigned)s.ctas), dim3(256), 0, st, p);
}

}  // namespace kvq
