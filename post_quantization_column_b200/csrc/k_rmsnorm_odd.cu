// k_rmsnorm_odd.cu — the RMS norm (k_rmsnorm.cu) of rows whose length is no multiple of 8, one
// after the other in memory.
//
// Row m starts (m K) mod 8 values beyond a whole vector in every tensor, whatever its type, so its
// values still go in whole vectors: at a row's ends the neighbouring rows' values come along,
// and count nothing; they are written value by value, and so is the last window of the last
// row read, behind which memory may end. The weight, which is met at another offset by every
// row, lies in shared memory with a place left free after every eighth value, so that lanes 8
// values apart find theirs in different banks, and zeros around it.
//
// What bounds it: issue slots. A window costs some 250 instructions a warp (its weights come one
// by one, its ends are checked), three times an aligned vector's: 8192 rows of 8191 in bf16 with
// a residual take 114 us (aligned 88; the copy rate 82), to e4m3 without one 87 (47; 31), 100000
// rows of 511 115 (70; 62). The ends' reads and writes in functions of their own, out of the
// loop, took a third longer: the calls wait for the loads before them.
#include "rmsnorm.cuh"

#include <algorithm>

namespace awq {
namespace {

__device__ __forceinline__ int weight_place(int e) { return (e + 8) + ((e + 8) >> 3); }

// The first `valid` values of a window, zeros in place of the others.
template <int TYPE>
__device__ __noinline__ Raw8<TYPE> load_end(const void* row, int first, int valid) {
  Raw8<TYPE> raw;
  uint32_t u[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    u[k] = 0u;
    if (k < valid) u[k] = TYPE == kTypeF32 ? static_cast<const uint32_t*>(row)[first + k] : static_cast<const uint16_t*>(row)[first + k];
  }
  if constexpr (TYPE == kTypeF32) {
    raw.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    raw.w[1] = make_uint4(u[4], u[5], u[6], u[7]);
  } else {
    raw.w[0] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
  }
  return raw;
}

// Values first .. first + 7 of a row, as far as they are its own.
template <int TYPE>
__device__ __forceinline__ void store_window(void* row, int first, int K, const float (&v)[8]) {
  if (first >= 0 && first + 8 <= K) {
    store8_as<TYPE>(row, first, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (first + k >= 0 && first + k < K) store_one(row, first + k, TYPE, v[k]);
  }
}

// Blocks of up to 544 threads: 8192 values and a row's ends in two windows each.
constexpr int threads_of(int lanes) { return lanes ? 256 : 544; }
// of that size an SM
constexpr int blocks_of(int vpt, int lanes, bool wide) {
  return lanes ? (vpt == 1 ? 5 - wide : (vpt == 2 ? 4 - wide : 2)) : (vpt + wide <= 2 ? 2 : 1);
}
template <int TX, int TR, int VPT, int LANES>
__global__ void __launch_bounds__(threads_of(LANES), blocks_of(VPT, LANES, TX == kTypeF32 || TR == kTypeF32)) norm_shifted_kernel(NormArgs a) {
  extern __shared__ float weight[];
  __shared__ RowStat parts[2][32];
  int turn = 0;
  const int tid = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x, width = LANES ? LANES : blockDim.x, K = static_cast<int>(a.K);
  const int rows = LANES ? blockDim.x / width : 1;
  const bool codes = a.out_type == kTypeE4m3;
  wait_for_previous();
  start_next();
  for (int e = static_cast<int>(threadIdx.x) - 8; e < K + 8; e += blockDim.x)
    weight[weight_place(e)] = e >= 0 && e < K ? load_one(a.weight, e, a.w_type) : 0.0f;
  __syncthreads();
  for (int64_t m = static_cast<int64_t>(blockIdx.x) * rows + (LANES ? threadIdx.x / width : 0); m < a.M;
       m += static_cast<int64_t>(gridDim.x) * rows) {
    const int shift = static_cast<int>(m * a.K % 8), vecs = (K + shift + 7) / 8;
    const void* x = row_at(a.X, m * a.x_stride, TX);
    const void* r = row_at(a.residual, m * a.r_stride, TR);
    void* ro = const_cast<void*>(row_at(a.residual_out, m * a.ro_stride, TR));
    void* out = const_cast<void*>(row_at(a.out, m * a.K, a.out_type));
    Raw8<TX> rx[VPT];
    Raw8<TR == kTypeNone ? kTypeF16 : TR> rr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * width, first = 8 * v - shift;
      if (v >= vecs) continue;
      if (m + 1 < a.M || first + 8 <= K) {
        rx[i].load(x, first);
        if constexpr (TR != kTypeNone) rr[i].load(r, first);
      } else {
        rx[i] = load_end<TX>(x, first, K - first);
        if constexpr (TR != kTypeNone) rr[i] = load_end<TR>(r, first, K - first);
      }
    }
    float h[VPT][8];
    RowStat st{0.0f, 0u};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * width, first = 8 * v - shift;
      if (v >= vecs) continue;
      rx[i].to_float(h[i]);
      if constexpr (TR != kTypeNone) {
        float add[8];
        rr[i].to_float(add);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] = __fadd_rn(h[i][k], add[k]);
      }
      if (first < 0 || first + 8 > K) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (first + k < 0 || first + k >= K) h[i][k] = 0.0f;
      }
      if constexpr (TR != kTypeNone) store_window<TR>(ro, first, K, h[i]);
      const float* w = weight + 9 * (v + 1) - shift;  // weight_place of value 8 v - shift
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        st.ss = __fmaf_rn(h[i][k], h[i][k], st.ss);
        h[i][k] = __fmul_rn(h[i][k], w[k < shift ? k - 1 : k]);
      }
      if (codes) {
#pragma unroll
        for (int k = 0; k < 8; ++k) st.peak = max(st.peak, __float_as_uint(h[i][k]) & 0x7FFFFFFFu);
      }
    }
    if (LANES)
      st = warp_join<LANES ? LANES : 32>(st, codes);
    else
      st = block_join(st, codes, parts, turn);
    const float factor = row_factor(st.ss, a);
    const Divisor scale(codes ? row_scale(st.peak, factor) : 1.0f);
    if (codes && tid == 0) a.out_scales[m] = scale.scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * width, first = 8 * v - shift;
      if (v >= vecs) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], factor);
      if (codes) {
        scale.divide(h[i]);
        store_window<kTypeE4m3>(out, first, K, h[i]);
      } else if (a.out_type == kTypeF32) {
        store_window<kTypeF32>(out, first, K, h[i]);
      } else if (a.out_type == kTypeBf16) {
        store_window<kTypeBf16>(out, first, K, h[i]);
      } else {
        store_window<kTypeF16>(out, first, K, h[i]);
      }
    }
  }
}

template <int TX, int TR, int VPT, int LANES>
cudaError_t launch(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int threads = LANES ? 256 : static_cast<int>(ceil_div(ceil_div(a.K / 8 + 2, VPT), 32) * 32);
  const size_t smem = static_cast<size_t>(a.K + 16 + (a.K + 16) / 8 + 1) * 4;
  static unsigned long long done = 0;
  const cudaError_t e = set_smem_limit_once(norm_shifted_kernel<TX, TR, VPT, LANES>, 80 * 1024, &done);
  if (e != cudaSuccess) return e;
  const int64_t resident = std::min<int64_t>(std::min(32, threads_of(LANES) * blocks_of(VPT, LANES, TX == kTypeF32 || TR == kTypeF32) / threads), 220 * 1024 / (smem + 2048));
  const int64_t rows = LANES ? threads / (LANES ? LANES : 1) : 1;
  const unsigned blocks = static_cast<unsigned>(std::min(ceil_div(a.M, rows), resident * num_sms));
  return launch_early(norm_shifted_kernel<TX, TR, VPT, LANES>, dim3(blocks), threads, smem, s, launches, a);
}

template <int TX, int TR>
cudaError_t launch_types(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int64_t vecs = a.K / 8 + 2;
  if (vecs <= 128 && a.M > num_sms) {  // rows of a warp or of half of one
    if (vecs <= 16) return launch<TX, TR, 1, 16>(a, num_sms, s, launches);
    if (vecs <= 32) return launch<TX, TR, 1, 32>(a, num_sms, s, launches);
    if (vecs <= 64) return launch<TX, TR, 2, 32>(a, num_sms, s, launches);
    return launch<TX, TR, 4, 32>(a, num_sms, s, launches);
  }
  // With rows enough, two windows a thread share a warp's fixed cost of a row: 16384 rows of 3333 in
  // fp16 take 81 us so, 97 with one; in fp32, where two leave one block an SM, 10000 of 4099 take 122 and 70.
  const bool many = a.M > 8 * num_sms && TX != kTypeF32 && TR != kTypeF32;
  if (vecs <= threads_of(0) && !many) return launch<TX, TR, 1, 0>(a, num_sms, s, launches);
  if (vecs <= 2 * threads_of(0)) return launch<TX, TR, 2, 0>(a, num_sms, s, launches);
  return launch<TX, TR, 4, 0>(a, num_sms, s, launches);
}

template <int TX>
cudaError_t launch_residual(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  switch (a.residual ? a.r_type : kTypeNone) {
    case kTypeNone: return launch_types<TX, kTypeNone>(a, num_sms, s, launches);
    case kTypeF32: return launch_types<TX, kTypeF32>(a, num_sms, s, launches);
    case kTypeF16: return launch_types<TX, kTypeF16>(a, num_sms, s, launches);
    default: return launch_types<TX, kTypeBf16>(a, num_sms, s, launches);
  }
}

}  // namespace

cudaError_t launch_rms_norm_shifted(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  if (a.x_type == kTypeF32) return launch_residual<kTypeF32>(a, num_sms, s, launches);
  if (a.x_type == kTypeF16) return launch_residual<kTypeF16>(a, num_sms, s, launches);
  return launch_residual<kTypeBf16>(a, num_sms, s, launches);
}

}  // namespace awq
