// kvq_block_host.cu -- the block cache's entry points: checks, sizes, launches.
#include <cstring>

#include "kvq_block.cuh"

using namespace kvq;

static kvq_status block_geometry(const kvq_block_config* c, BlockGeo* g) {
  if (!c) return KVQ_ERR_INVALID_ARG;
  if (c->batch < 1 || c->n_tokens < 1 || c->n_q_heads < 1 || c->n_kv_heads < 1 || c->n_q_heads % c->n_kv_heads || c->n_blocks < 1 ||
      c->max_blocks < 1 || c->window < 0 || c->n_first < 0)
    return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(c->softmax_scale) || c->softmax_scale < 0.0f || !std::isfinite(c->rope_theta) || c->rope_theta < 0.0f ||
      !std::isfinite(c->norm_eps) || c->norm_eps < 0.0f)
    return KVQ_ERR_INVALID_ARG;
  if (c->head_dim != kHeadDim || c->batch > kMaxBlockBatch || c->n_tokens > (1 << 20) || c->n_kv_heads > 1024 || c->n_q_heads > 1024 * c->n_kv_heads ||
      c->n_blocks > (1 << 26) || c->max_blocks > (1 << 25) || (int64_t)c->n_tokens * c->n_q_heads > (1 << 30))
    return KVQ_ERR_UNSUPPORTED;
  *g = BlockGeo{c->batch, c->n_tokens, c->n_q_heads, c->n_kv_heads, c->n_q_heads / c->n_kv_heads, c->n_blocks, c->max_blocks};
  return KVQ_OK;
}

static kvq_status block_arrays(const kvq_block_tables* t) {
  if (!t) return KVQ_ERR_INVALID_ARG;
  const void* all[] = {t->block_table, t->free_list, t->free_count, t->lens, t->start, t->unit0, t->token_row, t->position, t->slot};
  for (const void* a : all)
    if (!a || (uintptr_t)a % 4) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

// Counters, then (m, l) and accumulators of two partial results per CTA.
static const uint64_t kBlockMl = 4ull * kMaxBlockCtas, kBlockAcc = kBlockMl + 2ull * kMaxBlockCtas * kMaxBlockRows * 8,
                      kBlockScratch = kBlockAcc + 2ull * kMaxBlockCtas * kMaxBlockRows * kHeadDim * 4;

extern "C" {

kvq_status kvq_block_layout_query(const kvq_block_config* cfg, kvq_block_layout* out) {
  BlockGeo g;
  if (!out) return KVQ_ERR_INVALID_ARG;
  const kvq_status st = block_geometry(cfg, &g);
  if (st != KVQ_OK) return st;
  out->codes_bytes = (uint64_t)g.n_blocks * g.Hkv * 2 * kBlockSide;
  out->scales_bytes = ((uint64_t)g.n_blocks * g.Hkv * 2 + 15) / 16 * 16;
  out->workspace_bytes = kBlockScratch;
  return KVQ_OK;
}

kvq_status kvq_block_plan(const kvq_block_config* cfg, const kvq_block_tables* tables, const int32_t* lens_before,
                          const int32_t* free_before, const int32_t* n_new, kvq_stream_t stream) {
  return kvq_block_plan_back(cfg, tables, lens_before, free_before, n_new, nullptr, stream);
}

kvq_status kvq_block_plan_back(const kvq_block_config* cfg, const kvq_block_tables* tables, const int32_t* lens_before,
                               const int32_t* free_before, const int32_t* n_new, const int32_t* n_back, kvq_stream_t stream) {
  BlockPlanParams p;
  kvq_status st = block_geometry(cfg, &p.geo);
  if (st != KVQ_OK) return st;
  if ((st = block_arrays(tables)) != KVQ_OK) return st;
  if (!lens_before || !free_before || !n_new ||
      ((uintptr_t)lens_before | (uintptr_t)free_before | (uintptr_t)n_new | (uintptr_t)n_back) % 4)
    return KVQ_ERR_INVALID_ARG;
  p.t = *tables;
  p.lens_before = lens_before;
  p.free_before = free_before;
  p.n_new = n_new;
  p.n_back = n_back;
  return launch_block_plan(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_block_append(const kvq_block_config* cfg, const kvq_block_tables* tables, uint8_t* codes, uint8_t* scales,
                            const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const uint16_t* q, int64_t q_stride,
                            uint16_t* q_out, const uint16_t* q_weight, const uint16_t* k_weight, kvq_stream_t stream) {
  BlockAppendParams p;
  std::memset(&p, 0, sizeof(p));
  kvq_status st = block_geometry(cfg, &p.geo);
  if (st != KVQ_OK) return st;
  if ((st = block_arrays(tables)) != KVQ_OK) return st;
  const BlockGeo& g = p.geo;
  const int64_t kv_row = (int64_t)g.Hkv * kHeadDim, q_row = (int64_t)g.Hq * kHeadDim, most = 1ll << 40;
  if (!codes || !scales || !k || !v || !q != !q_out || (!q && q_weight)) return KVQ_ERR_INVALID_ARG;
  if (((uintptr_t)codes | (uintptr_t)scales | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q | (uintptr_t)q_out | (uintptr_t)q_weight |
       (uintptr_t)k_weight) % 16)
    return KVQ_ERR_INVALID_ARG;
  if (k_stride < kv_row || v_stride < kv_row || (q && q_stride < q_row) || k_stride % 8 || v_stride % 8 || (q && q_stride % 8) ||
      k_stride > most || v_stride > most || (q && q_stride > most))
    return KVQ_ERR_INVALID_ARG;
  if (q) {  // q_out: q itself, or apart from every input
    const uintptr_t o0 = (uintptr_t)q_out, o1 = o0 + 2ull * g.N * q_row;
    const auto meets = [&](const uint16_t* x, int64_t stride, int64_t row) {
      const uintptr_t x0 = (uintptr_t)x, x1 = x0 + 2ull * ((g.N - 1) * stride + row);
      return x0 < o1 && o0 < x1;
    };
    if (meets(q, q_stride, q_row) && !(q == q_out && q_stride == q_row)) return KVQ_ERR_INVALID_ARG;
    if (meets(k, k_stride, kv_row) || meets(v, v_stride, kv_row)) return KVQ_ERR_INVALID_ARG;
  }
  p.t = *tables;
  p.codes = codes;
  p.scales = scales;
  p.k = k, p.ks = k_stride;
  p.v = v, p.vs = v_stride;
  p.q = q, p.qs = q_stride;
  p.q_out = q_out;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = cfg->norm_eps;
  p.rotate = cfg->rope_theta > 0.0f;
  if (p.rotate) rope_turns(cfg->rope_theta, p.freq);
  int sms = 0;
  if (device_sm_count(&sms) != cudaSuccess) return KVQ_ERR_CUDA;
  return launch_block_append(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_block_attn(const kvq_block_config* cfg, const kvq_block_tables* tables, const uint8_t* codes, const uint8_t* scales,
                          const uint16_t* q, uint16_t* out, float* lse, void* workspace, uint64_t ws_bytes, kvq_stream_t stream) {
  BlockAttnParams p;
  std::memset(&p, 0, sizeof(p));
  kvq_status st = block_geometry(cfg, &p.geo);
  if (st != KVQ_OK) return st;
  if ((st = block_arrays(tables)) != KVQ_OK) return st;
  const BlockGeo& g = p.geo;
  if (!codes || !scales || !q || !out || ((uintptr_t)codes | (uintptr_t)scales | (uintptr_t)q | (uintptr_t)out) % 16 || (uintptr_t)lse % 4)
    return KVQ_ERR_INVALID_ARG;
  const uintptr_t o0 = (uintptr_t)out, q0 = (uintptr_t)q, bytes = 2ull * g.N * g.Hq * kHeadDim;
  if (o0 < q0 + bytes && q0 < o0 + bytes) return KVQ_ERR_INVALID_ARG;  // a row's q is read by several CTAs
  if (!workspace || (uintptr_t)workspace % 16 || ws_bytes < kBlockScratch) return KVQ_ERR_WORKSPACE;
  p.t = *tables;
  p.codes = codes;
  p.scales = scales;
  p.q = q;
  p.out = out;
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.counters = reinterpret_cast<unsigned*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + kBlockMl);
  p.part_acc = reinterpret_cast<float*>(ws + kBlockAcc);
  const double sm = cfg->softmax_scale > 0.0f ? (double)cfg->softmax_scale : 1.0 / std::sqrt((double)kHeadDim);
  p.q_scale = (float)(sm * 1.4426950408889634);
  p.window = cfg->window > 0 && cfg->window < kNoWindow ? cfg->window : kNoWindow;
  p.n_first = cfg->n_first;
  p.g_inv = g.g > 1 ? (unsigned)(((1ull << 32) + g.g - 1) / g.g) : 0;
  int sms = 0;
  if (device_sm_count(&sms) != cudaSuccess) return KVQ_ERR_CUDA;
  if (sms > kMaxBlockCtas) sms = kMaxBlockCtas;
  // rows that read a KV head's blocks together: those of an even share of the token
  // slots (the step's own numbers are on the GPU).  A request of more takes several
  // passes, one of fewer leaves warps without rows: 64 requests of a token each, 100 to 8k
  // tokens, 32 on 8 heads: 84 us with 64 slots, 87 with 256, 330 with 1,024.
  const long long rows = (long long)((g.N + g.B - 1) / g.B) * g.g;
  return launch_block_attn(p, sms, rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

}  // extern "C"
