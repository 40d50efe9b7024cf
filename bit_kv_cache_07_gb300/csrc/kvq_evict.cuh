// kvq_evict.cuh -- parameters of the eviction kernels (kvq_evict.cu).
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

struct EvictParams {
  Geometry geo;
  LayerPtrs L;
  const float* mass;   // [NS][max_tokens]
  float* mass_out;     // may be mass
  int* source;         // [NS][cap] or null
  unsigned long long* keys;  // [NS][cap] order keys of the groups' totals
  int *hole, *mover;   // [NS][cap] freed slots below the new end, groups that fill them
  int* moves;          // [NS] how many
  void* saved;         // [NS][2][save_rows][d] fp16 copies of the window
  int S, R;            // the config's sinks and window (the unquantized cache keeps them too)
  int cap, max_tokens; // group slots per stream, tokens per stream of the record
  int most;            // the most groups any row gives up
  int save_rows;       // window rows copied per stream
  int sum_blocks, save_blocks;
  int tokens[kMaxRaggedRows], evict[kMaxRaggedRows];
};

// Whole 32-token groups between the sinks and the window at T tokens (the
// window rule; for the unquantized cache too).
__host__ __device__ inline int group_count(const EvictParams& p, int T) {
  const int rest = T - p.S - p.R;
  return rest > 0 ? rest / kGroupTokens : 0;
}

cudaError_t launch_evict(EvictParams& p, cudaStream_t st);

}  // namespace kvq
