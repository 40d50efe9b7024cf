// Prints the rotation's frequencies (turns per position as 64-bit fractions) for bases
// given as arguments, one line each, for a comparison in many digits.
#include "../bit_kv_cache_07_gb300/csrc/kvq_internal.cuh"
#include <cstdio>
#include <cstdlib>

int main(int argc, char** argv) {
  for (int a = 1; a < argc; ++a) {
    unsigned long long f[kvq::kHeadDim / 2];
    kvq::rope_turns(strtof(argv[a], nullptr), f);
    for (int i = 0; i < kvq::kHeadDim / 2; ++i) printf("%llu ", f[i]);
    printf("\n");
  }
  return 0;
}
