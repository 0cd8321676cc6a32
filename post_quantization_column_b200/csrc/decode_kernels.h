// decode_kernels.h — the operators of a decode step around the W4A16 products (internal to
// libawqsearch): the RMS norm that feeds a quantized layer, the append to a paged key-value
// cache with the position rotation, and the attention of one new token over that cache.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <utility>

#include "awq_kernels.h"

namespace awq {

// Element types of these operators (AWQ_DTYPE_* of the C ABI).
enum : int { kTypeBf16 = 0, kTypeF32 = 1, kTypeF16 = 2, kTypeE4m3 = 3, kTypeNone = -1 };
__host__ __device__ constexpr int type_bytes(int t) {
  return t == kTypeF32 ? 4 : (t == kTypeE4m3 ? 1 : (t == kTypeNone ? 0 : 2));
}
constexpr float kE4m3Max = 448.0f;  // largest finite e4m3 value

// ---- RMS norm ------------------------------------------------------------------------
constexpr int64_t kNormMaxK = 57344;  // one fp32 row in shared memory
struct NormArgs {
  const void* X;             // [M][K], rows x_stride elements apart
  const void* residual;      // [M][K] or NULL
  void* residual_out;        // [M][K]; may be `residual`
  const void* weight;        // [K]
  void* out;                 // [M][K] contiguous
  float* out_scales;         // [M], e4m3 output only
  int64_t M, K, x_stride, r_stride, ro_stride;
  int x_type, r_type, w_type, out_type;
  float eps, inverse_k;      // inverse_k: 1 / K
};
cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t s, int* launches);

// ---- paged key-value cache -------------------------------------------------------------
// Element (page p, slot s, head h, dim d) of keys and of values lies at
// p * page_stride + s * slot_stride + h * head_stride + d.
struct PagedCache {
  void* k;
  void* v;
  int64_t num_pages, page_stride, slot_stride, head_stride;
  int page_size, heads, head_dim, type;
  const float* k_scale;  // [heads], e4m3 only
  const float* v_scale;
  const int32_t* table;  // [seqs][max_pages], rows table_stride apart
  int64_t seqs, max_pages, table_stride;
};

struct AppendArgs {
  const void* q;  // [T][Hq][D], token and head strides in elements
  const void* k;
  const void* v;
  int64_t q_st, k_st, v_st;
  uint32_t q_head, k_head, v_head;  // the head strides in bytes
  uint32_t cache_head32;            // the cache's in units of 32 bytes
  int64_t T;
  int Hq, in_type, q_type, rot, interleaved;
  const double* freqs;       // [rot / 2] radians per position
  float magnitude;
  const int32_t* positions;  // [T]
  const int32_t* seq;        // [T], NULL: token i belongs to sequence i
  void* q_out;               // [T][Hq][D] contiguous
  int32_t* status;           // may be NULL
  PagedCache c;
};
cudaError_t launch_kv_append(const AppendArgs& a, int num_sms, cudaStream_t s, int* launches);

struct PagedAttnArgs {
  const void* q;  // [B][Hq][D]
  int64_t q_sb, q_sh;
  int64_t B;
  int Hq, q_type;
  const int32_t* lengths;  // [B]
  float scale;
  void* out;         // [B][Hq][D] contiguous, q's type
  void* workspace;   // paged_attn_workspace bytes, 16-byte aligned
  int32_t* status;   // may be NULL
  PagedCache c;
};
int64_t paged_attn_workspace(int Hq, int Hkv, int D, int type);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, int num_sms, cudaStream_t s, int* launches);

// Shared with awq_api.cu: the entry points' error text, device selection and launch count.
int decode_error(int status, const char* msg);
int decode_cuda_error(cudaError_t e, const char* where);
// Makes device *dev current, or for -1 the device that owns `ptr`, and checks it once.
int decode_device(const void* ptr, int* dev, int* num_sms);
bool decode_device_memory(const void* p, int dev);  // memory of device `dev`, or managed memory
bool decode_status_memory(const void* p, int dev);  // the same, or pinned host memory that kernels reach at `p`
void record_launch_count(int launches);

#ifdef __CUDACC__
// Programmatic launches: a kernel is set up while the one before it in the stream still works,
// and waits for that one's end, with all it has written, before it touches memory. Every CTA
// waits, so that a kernel's end implies the end of all before it.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, int* launches,
                         Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

__device__ __forceinline__ float bits_f16(uint32_t h) { return __half2float(__ushort_as_half(static_cast<unsigned short>(h))); }
// The two 16-bit values of a word as floats.
__device__ __forceinline__ float2 unpack16(uint32_t w, int type) {
  if (type == kTypeBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack16(float a, float b, int type) {
  if (type == kTypeBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// v / scale as a product with 1 / scale, where that is finite (within 2^-23 of the quotient, a
// quarter of a millionth of an e4m3 step, for an eighth of a division's instructions).
struct Divisor {
  float scale, inverse;
  bool product;
  __device__ __forceinline__ explicit Divisor(float s) : scale(s), inverse(1.0f / s) {
    product = fabsf(inverse) <= 3.402823466e38f;
  }
  template <int N>
  __device__ __forceinline__ void divide(float (&v)[N]) const {
    if (product) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = __fmul_rn(v[k], inverse);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = __fdiv_rn(v[k], scale);
    }
  }
};
// Two values rounded to e4m3 (finite values beyond +-448 saturate; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float load_one(const void* p, int64_t i, int type) {
  if (type == kTypeF32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const unsigned short*>(p)[i];
  return type == kTypeBf16 ? __uint_as_float(h << 16) : bits_f16(h);
}
__device__ __forceinline__ void store_one(void* p, int64_t i, int type, float v) {
  switch (type) {
    case kTypeF32: static_cast<float*>(p)[i] = v; break;
    case kTypeBf16: static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v); break;
    case kTypeF16: static_cast<__half*>(p)[i] = __float2half_rn(v); break;
    default: static_cast<uint8_t*>(p)[i] = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
  }
}
// Eight consecutive values (16-byte aligned; 8 bytes for e4m3) rounded to `type`.
template <int TYPE>
__device__ __forceinline__ void store8_as(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (TYPE == kTypeF32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else if constexpr (TYPE == kTypeE4m3) {
    const uint32_t lo = pack_e4m3(v[0], v[1]) | (pack_e4m3(v[2], v[3]) << 16);
    const uint32_t hi = pack_e4m3(v[4], v[5]) | (pack_e4m3(v[6], v[7]) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + i) = make_uint2(lo, hi);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack16(v[0], v[1], TYPE), pack16(v[2], v[3], TYPE), pack16(v[4], v[5], TYPE), pack16(v[6], v[7], TYPE));
  }
}
__device__ __forceinline__ void store8(void* p, int64_t i, int type, const float (&v)[8]) {
  switch (type) {
    case kTypeF32: store8_as<kTypeF32>(p, i, v); break;
    case kTypeBf16: store8_as<kTypeBf16>(p, i, v); break;
    case kTypeF16: store8_as<kTypeF16>(p, i, v); break;
    default: store8_as<kTypeE4m3>(p, i, v);
  }
}
// Eight consecutive values (16-byte aligned) in their own form, read once.
template <int TYPE>
struct Raw8 {
  static constexpr int kWords = TYPE == kTypeF32 ? 2 : 1;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * type_bytes(TYPE));
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[k].x), "=r"(w[k].y), "=r"(w[k].z), "=r"(w[k].w)
                   : "l"(s + k));
  }
  __device__ __forceinline__ void to_float(float (&v)[8]) const {
    if constexpr (TYPE == kTypeF32) {
      const uint4 a = w[0], b = w[kWords - 1];
      v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack16(u[k], TYPE);
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      }
    }
  }
};
#endif

}  // namespace awq
