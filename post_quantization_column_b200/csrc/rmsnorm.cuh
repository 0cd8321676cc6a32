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

__device__ __forceinline__ RowStat join(RowStat a, RowStat b) {
  a.ss = __fadd_rn(a.ss, b.ss);
  a.peak = max(a.peak, b.peak);
  return a;
}

__device__ __forceinline__ RowStat warp_join(RowStat a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = join(a, {__shfl_xor_sync(~0u, a.ss, o), __shfl_xor_sync(~0u, a.peak, o)});
  return a;
}

// The statistic of a row whose parts the block's warps hold, in every thread. Rows take turns
// between two sets of slots, so that one barrier a row is enough.
__device__ __forceinline__ RowStat block_join(RowStat a, RowStat (*shared)[32], int& turn) {
  const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
  if (warps == 1) return a;
  RowStat* slots = shared[turn];
  turn ^= 1;
  if (lane == 0) slots[threadIdx.x / 32] = a;
  __syncthreads();
  return warp_join(lane < warps ? slots[lane] : RowStat{0.0f, 0u});
}

__device__ __forceinline__ float row_factor(float ss, int64_t K, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(K)), eps)));
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
