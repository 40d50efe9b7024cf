// The bounded wait of the tile kernels on the GPU: one that nothing ends runs
// out, says so, and takes the CTA's other waits with it; one whose phase is
// complete returns at once and says nothing.  Prints "bad <count>".
#include "../bit_kv_cache_07_gb300/csrc/kvq_pipe.cuh"
#include <cstdio>
using namespace kvq;

__global__ void waits(int* out) {
  __shared__ uint64_t bars[2];
  __shared__ int flag;
  const uint32_t never = (uint32_t)__cvta_generic_to_shared(&bars[0]), done = (uint32_t)__cvta_generic_to_shared(&bars[1]);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(never, 1);
    mbar_init(done, 1);
    flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    mbar_arrive(done);
  }
  __syncthreads();
  if (lane == 0 && w == 0) out[0] = mbar_wait(done, 0, &flag, 1000);
  if (threadIdx.x == 0) out[1] = flag;
  __syncthreads();
  if (lane == 0) {
    if (w == 0) out[2] = mbar_wait(never, 0, nullptr, 8);          // no flag to set
    if (w == 0) out[3] = *(volatile int*)&flag;
    if (w == 0) out[4] = mbar_wait(never, 0, &flag, 8);            // runs out
    if (w == 1) out[5] = mbar_wait(never, 0, &flag, 1 << 16);      // a quarter of a second of its own: the flag ends it
  }
  __syncthreads();
  if (threadIdx.x == 0) out[6] = flag;
}

int main() {
  int *d = nullptr, h[7] = {};
  cudaEvent_t a, b;
  float ms = 0.0f;
  cudaMalloc(&d, sizeof(h));
  cudaMemset(d, 0xFF, sizeof(h));
  cudaEventCreate(&a);
  cudaEventCreate(&b);
  cudaEventRecord(a);
  waits<<<1, 64>>>(d);
  cudaEventRecord(b);
  const cudaError_t e = cudaMemcpy(h, d, sizeof(h), cudaMemcpyDeviceToHost);
  cudaEventElapsedTime(&ms, a, b);
  const int want[7] = {1, 0, 0, 0, 0, 0, 1};
  int bad = e != cudaSuccess;
  for (int i = 0; i < 7; ++i) bad += h[i] != want[i];
  bad += ms > 100.0f;
  printf("%s, %.3f ms, bad %d\n", cudaGetErrorString(e), ms, bad);
  cudaFree(d);
  return bad != 0;
}
