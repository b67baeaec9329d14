// Waits of a whole warp on an mbarrier (mbar_wait_warp) that are met, that are
// aborted, that run out and that are aborted while the barrier completes. A
// block per case: the second warp acts after `delay` clock cycles, the lanes of
// the first one write what the wait told them. Every wait ends by its limit.
#include "tria_internal.cuh"

namespace {

enum { kMet, kAborted, kRunsOut, kBoth };

__global__ void k_warp_wait(int mode, int limit, int step, int* out) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint32_t abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tria::mbar_init(&bar, 1);
    tria::fence_mbar_init();
    abort_word = 0;
  }
  __syncthreads();
  if (warp == 0) {
    out[blockIdx.x * 32 + lane] = tria::mbar_wait_warp(&bar, 0, &abort_word, limit);
  } else if (lane == 0) {
    const long long t0 = clock64();
    while (clock64() - t0 < (long long)blockIdx.x * step) {
    }
    if (mode == kAborted || mode == kBoth) *(volatile uint32_t*)&abort_word = 1;
    if (mode == kMet || mode == kBoth) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tria::smem_u32(&bar)) : "memory");
  }
}

}  // namespace

extern "C" int warp_wait(int mode, int limit, int step, int blocks, int* out, void* stream) {
  k_warp_wait<<<blocks, 64, 0, (cudaStream_t)stream>>>(mode, limit, step, out);
  return (int)cudaGetLastError();
}
