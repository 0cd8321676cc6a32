// k_rmsnorm.cu — RMS norm with the residual's addition, the operation that produces a
// quantized layer's activations: "AWQ：为什么 4-bit 权重量化要先观察 Activation" §6 folds the
// scales s into it, so its weight carries 1 / s and its fp16 output is the W4A16 product's A.
//
//   h = x + r (fp32),  r' = round(h),  y_k = (h_k w_k) / sqrt(mean(h^2) + eps)
//
// rounded once to the output's type, or, as e4m3, to codes e4m3(y / scale) with one scale
// per row, scale = max|y| / 448 (1 where that is zero). Sums and statistics are fp32; the
// norm is of the unrounded h. 1 / sqrt(...) is one positive factor of a row and rounding
// keeps order, so max|y| = fl(max|h w| / sqrt(...)): one reduction of (sum h^2, max|h w|)
// per row serves both forms. The maximum is taken of the bit patterns of |h w|, which
// order as the values do and put NaN above everything: a row that holds a NaN or an
// infinity has a NaN scale.
#include "decode_kernels.h"

#include <algorithm>

namespace awq {
namespace {

struct RowStat {
  float ss;
  uint32_t peak;  // bits of max |h w|
};

__device__ __forceinline__ RowStat join(RowStat a, RowStat b) {
  a.ss = __fadd_rn(a.ss, b.ss);
  a.peak = max(a.peak, b.peak);
  return a;
}

// The statistic of a row whose parts the block's threads hold, in every thread.
__device__ __forceinline__ RowStat block_join(RowStat a, RowStat* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = join(a, {__shfl_xor_sync(~0u, a.ss, o), __shfl_xor_sync(~0u, a.peak, o)});
  const int warps = blockDim.x / 32;
  if (warps == 1) return a;
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = a;
  __syncthreads();
  a = shared[0];
  for (int w = 1; w < warps; ++w) a = join(a, shared[w]);
  __syncthreads();  // the slots are free for the next row
  return a;
}

__device__ __forceinline__ float row_factor(float ss, int64_t K, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(K)), eps)));
}

__device__ __forceinline__ float row_scale(uint32_t peak, float factor) {
  const float scale = __fdiv_rn(__fmul_rn(__uint_as_float(peak), factor), kE4m3Max);
  return scale == 0.0f ? 1.0f : scale;
}

// One row per block and turn, one or more scalars per thread: any K, stride and alignment.
// h stays in shared memory between the two uses of it.
__global__ void __launch_bounds__(1024) norm_any_kernel(NormArgs a) {
  extern __shared__ float h_row[];
  __shared__ RowStat parts[32];
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    RowStat st{0.0f, 0u};
    for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x) {
      float h = load_one(a.X, m * a.x_stride + k, a.x_type);
      if (a.residual) {
        h = __fadd_rn(h, load_one(a.residual, m * a.r_stride + k, a.r_type));
        store_one(a.residual_out, m * a.ro_stride + k, a.r_type, h);
      }
      const float hw = __fmul_rn(h, load_one(a.weight, k, a.w_type));
      h_row[k] = hw;
      st = join(st, {__fmul_rn(h, h), __float_as_uint(hw) & 0x7FFFFFFFu});
    }
    st = block_join(st, parts);
    const float factor = row_factor(st.ss, a.K, a.eps);
    const float scale = a.out_type == kTypeE4m3 ? row_scale(st.peak, factor) : 1.0f;
    if (a.out_type == kTypeE4m3 && threadIdx.x == 0) a.out_scales[m] = scale;
    for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x) {  // each thread's own h
      const float y = __fmul_rn(h_row[k], factor);
      store_one(a.out, m * a.K + k, a.out_type, a.out_type == kTypeE4m3 ? __fdiv_rn(y, scale) : y);
    }
  }
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int threads = static_cast<int>(std::min<int64_t>(1024, ceil_div(a.K, 32) * 32));
  const size_t smem = static_cast<size_t>(a.K) * 4;
  static unsigned long long done = 0;
  cudaError_t e = set_smem_limit_once(norm_any_kernel, static_cast<int>(kNormMaxK * 4), &done);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(a.M, 8 * num_sms));
  norm_any_kernel<<<blocks, threads, smem, s>>>(a);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace awq
