// How the kernels of paged attention divide a batch among their CTAs: the list of (work
// unit, key block) places is cut into equal runs, by the lengths found on the device. A unit
// cut by a run's end leaves pieces: slot 1 of the CTA where it began, slot 0 of those where
// it went on.
#pragma once
#include <atomic>

#include "fa_launch.cuh"
#include "fa_paged.h"

namespace fa {

// The reference maximum of a running softmax moves when a score exceeds it by more than 2^8
// (scores are in log2 units). With f16 weights it lies 2^7 below the largest score: weights
// reach 2^15, which f16 holds, and the smallest ones keep 7 bits more.
constexpr float kRescale = 8.0f;
constexpr float kF16Lift = 7.0f;

// Sum over the block's threads of x, and the sum of those before this one.
template <int WARPS>
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums,
                                                long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // earlier readers of warp_sums are done
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const long long y = warp_sums[w];
    if (w < warp) before += y;
    all += y;
  }
  *total = all;
  return before + inc - x;
}

// What a CTA leaves for the merge: the unit that its run began and did not end (row0 < 0:
// none), its first token's row, K/V head and query rows; and whether a unit that it did not
// begin ended in its run (or there was none).
struct alignas(16) PieceHeader {
  int row0, h, rows, ended;
};

// The header of CTA c, and the number of CTAs after it that hold further pieces of the unit
// begun there: up to the first one in which it ended (0 if it began none). Called by the whole
// block, which has a thread for every CTA.
__device__ __forceinline__ int pieces_after(const PieceHeader* headers, int c, int ctas, int* shared,
                                            PieceHeader* of_c) {
  const int i = c + 1 + static_cast<int>(threadIdx.x);
  const int ended = i < ctas ? headers[i].ended : 0;
  *of_c = headers[c];
  if (of_c->row0 < 0) return 0;
  if (threadIdx.x == 0) *shared = ctas - 1 - c;
  __syncthreads();
  if (ended != 0) atomicMin(shared, i - c);
  __syncthreads();
  return *shared;
}

// N values of a piece's row, fp32, from p on.
template <int N>
__device__ __forceinline__ void load_part(const float* p, float* v) {
  if constexpr (N == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x;
    v[1] = x.y;
  }
}

}  // namespace fa
