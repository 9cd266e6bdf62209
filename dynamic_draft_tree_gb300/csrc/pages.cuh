// What the page calls share: sums over requests, the CTA that comes last, the free list's length.
#pragma once

#include "dt_internal.cuh"

namespace dt {
namespace {

constexpr int kPageThreads = 256;
// Up to this many CTAs the last one changes the counts; more of them queue up at the ticket, and a second launch is
// faster. Reserve + release, 64 requests of up to 8000 slots: 13.0 us with two launches each, 15.0 with the ticket;
// 8 requests of 9 slots: 8.2 and 8.3 us on the device, but two launches take 3 us more on the host.
constexpr int kTicketCtas = 64;

#ifdef __CUDACC__
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* smem) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += (int64_t)shfl_xor_u64((uint64_t)v, m);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t t = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += smem[w];
  __syncthreads();
  return t;
}

// True in every thread of the CTA that comes last: what the others read and wrote before is done.
__device__ __forceinline__ bool comes_last(unsigned* ticket, unsigned ctas) {
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicInc(ticket, ctas - 1) == ctas - 1;
    __threadfence();
  }
  __syncthreads();
  return last;
}

__device__ __forceinline__ int free_blocks(const dt_block_pool& p) { return min(max(p.free_count[0], 0), p.n_blocks); }
#endif

inline int shift_of(int page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

}  // namespace
}  // namespace dt
