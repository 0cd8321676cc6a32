// rmsnorm.cuh — a row's statistic, shared by the forms of the RMS norm (k_rmsnorm.cu, which has
// the mathematics, and k_rmsnorm_odd.cu).
#pragma once

#include "decode_kernels.h"

namespace awq {

// The form for rows that follow one another at a distance of no whole vectors.
cudaError_t launch_rms_norm_shifted(const NormArgs& a, int num_sms, cudaStream_t s, int* launches);

struct RowStat {
  float ss;
  uint32_t peak;  // bits of max |h w|
};

// A row's fixed cost, this join and the root, is met by every warp for as few as 8 values a lane:
// it takes the fewest instructions that will do (the peak only where there are codes, in one
// instruction over a warp; the reciprocal root of 2 ulp), which took 16384 bf16 rows of 2048 to
// e4m3 from 34.7 to 29.6 us.
//
// Over LANES neighbouring lanes, which come here together.
template <int LANES = 32>
__device__ __forceinline__ RowStat warp_join(RowStat a, bool codes) {
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t mask = LANES == 32 ? ~0u : ((1u << (LANES % 32)) - 1) << (lane / LANES * LANES);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) a.ss = __fadd_rn(a.ss, __shfl_xor_sync(mask, a.ss, o));
  if (codes) {
    if (LANES == 32) {
      a.peak = __reduce_max_sync(mask, a.peak);
    } else {
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) a.peak = max(a.peak, __shfl_xor_sync(mask, a.peak, o));
    }
  }
  return a;
}

// The statistic of a row whose parts the block's threads hold, in every thread. Rows take turns
// between two sets of slots, so that one barrier a row is enough.
__device__ __forceinline__ RowStat block_join(RowStat a, bool codes, RowStat (*shared)[32], int& turn) {
  const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
  a = warp_join(a, codes);
  if (warps == 1) return a;
  RowStat* slots = shared[turn];
  turn ^= 1;
  if (lane == 0) slots[threadIdx.x / 32] = a;
  __syncthreads();
  return warp_join(lane < warps ? slots[lane] : RowStat{0.0f, 0u}, codes);
}

__device__ __forceinline__ float row_factor(float ss, const NormArgs& a) {
  return rsqrtf(__fadd_rn(__fmul_rn(ss, a.inverse_k), a.eps));
}

__device__ __forceinline__ float row_scale(uint32_t peak, float factor) {
  const float scale = __fdiv_rn(__fmul_rn(__uint_as_float(peak), factor), kE4m3Max);
  return scale == 0.0f ? 1.0f : scale;
}

// Value `values` of a tensor of `type`.
__device__ __forceinline__ const void* row_at(const void* p, int64_t values, int type) {
  return static_cast<const uint8_t*>(p) + values * type_bytes(type);
}

}  // namespace awq
