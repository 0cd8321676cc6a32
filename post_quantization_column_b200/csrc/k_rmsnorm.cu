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
// infinity has a NaN scale. The squares are not scaled before they are added: a sum beyond fp32
// divides its row by infinity, and with eps = 0 one that underflows divides it by zero.
//
// What bounds it: the rows' bytes, each read and written once (x, r, r' and y; 1 GB for 16384 x
// 8192 in bf16 with a residual). A row stays in registers between its statistic and its output,
// and the next row's loads are issued before the reduction, so that two blocks an SM keep loads
// on the way while both wait at a barrier: 168 us, 6.4 TB/s of the 6.55 of a copy (12 us more with
// the loads after the output; 22 more with three rows ahead in a shared-memory ring, whose
// traffic costs more than its depth gives). One row of 4096 takes 2.3 us in a captured graph
// (fp32 with a residual), 100000 bf16 rows of 64 5.3 us (18 with a warp a row).
#include "rmsnorm.cuh"

#include <algorithm>

namespace awq {
namespace {

// Vector v of the weight.
__device__ __forceinline__ void load_weight(const NormArgs& a, int v, float (&w)[8]) {
  if (a.w_type == kTypeF32) {
    const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + 8 * v);
    const float4 lo = from[0], hi = from[1];
    w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
    w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + 8 * v);
    const uint32_t words[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack16(words[k], a.w_type);
      w[2 * k] = f.x;
      w[2 * k + 1] = f.y;
    }
  }
}

// The thread's vectors h w of row m, with the row's statistic, to the output.
template <int VPT>
__device__ __forceinline__ void write_row(const NormArgs& a, int64_t m, int lane, int width, int vecs, RowStat st, float (&h)[VPT][8]) {
  const float factor = row_factor(st.ss, a);
  if (a.out_type == kTypeE4m3) {
    const Divisor scale(row_scale(st.peak, factor));
    if (lane == 0) a.out_scales[m] = scale.scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = lane + i * width;
      if (v >= vecs) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], factor);
      scale.divide(h[i]);
      store8_as<kTypeE4m3>(a.out, m * a.K + 8 * v, h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = lane + i * width;
      if (v >= vecs) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], factor);
      store8(a.out, m * a.K + 8 * v, a.out_type, h[i]);
    }
  }
}

// Rows of aligned vectors of 8 values: the whole row lies in the registers of its threads, VPT
// vectors each, between the reduction and the output. A row belongs to 8, 16 or 32 LANES of a warp,
// or to a block (LANES = 0); several blocks an SM load while others reduce, and the weight stays in
// the L1 cache, which the rows themselves pass by.
constexpr int norm_threads(int lanes) { return lanes ? 256 : 512; }  // of a block, at most
constexpr int norm_blocks(int vpt, int lanes) { return (lanes ? 2 : 1) * (vpt <= 2 ? 2 : 1); }  // of that size an SM
template <int TX, int TR, int VPT, int LANES>
__global__ void __launch_bounds__(norm_threads(LANES), norm_blocks(VPT, LANES)) norm_kernel(NormArgs a) {
  __shared__ RowStat parts[2][32];
  int turn = 0;
  const int lane = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x, width = LANES ? LANES : blockDim.x;
  const int rows = LANES ? blockDim.x / width : 1;
  const int vecs = static_cast<int>(a.K / 8);
  const bool codes = a.out_type == kTypeE4m3;
  wait_for_previous();
  start_next();
  Raw8<TX> rx[VPT];
  Raw8<TR == kTypeNone ? kTypeF16 : TR> rr[VPT];
  auto load_row = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = lane + i * width;
      if (v < vecs) {
        rx[i].load(a.X, m * a.x_stride + 8 * v);
        if (TR != kTypeNone) rr[i].load(a.residual, m * a.r_stride + 8 * v);
      }
    }
  };
  int64_t m = static_cast<int64_t>(blockIdx.x) * rows + (LANES ? threadIdx.x / width : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  if (m < a.M) load_row(m);
  for (; m < a.M; m += step) {
    float h[VPT][8];
    RowStat st{0.0f, 0u};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = lane + i * width;
      if (v >= vecs) continue;
      rx[i].to_float(h[i]);
      if constexpr (TR != kTypeNone) {
        float r[8];
        rr[i].to_float(r);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] = __fadd_rn(h[i][k], r[k]);
        store8_as<TR>(a.residual_out, m * a.ro_stride + 8 * v, h[i]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) st.ss = __fmaf_rn(h[i][k], h[i][k], st.ss);
      float w[8];
      load_weight(a, v, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], w[k]);
      if (codes) {
#pragma unroll
        for (int k = 0; k < 8; ++k) st.peak = max(st.peak, __float_as_uint(h[i][k]) & 0x7FFFFFFFu);
      }
    }
    if (m + step < a.M) load_row(m + step);  // on the way during the reduction and the output
    if (LANES)
      st = warp_join<LANES ? LANES : 32>(st, codes);
    else
      st = block_join(st, codes, parts, turn);
    write_row<VPT>(a, m, lane, width, vecs, st, h);
  }
}

// Rows of any length and alignment: E pieces of VEC values per thread and turn, loaded together
// (VEC = 1 for odd rows, 2 for even ones, 8 for aligned rows beyond norm_kernel's). A row of one
// turn stays in registers; of a longer one (LONG) h w waits in shared memory, where each thread
// finds its own again. The types are told apart once per turn and tensor.
template <int TYPE, int VEC, int E>
__device__ __forceinline__ void load_pieces(const void* row, int first, int step, int pieces, float (&v)[E][VEC]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int at = first + i * step;
    if (at >= pieces) continue;
    if constexpr (VEC == 8) {
      Raw8<TYPE> raw;
      raw.load(row, 8 * static_cast<int64_t>(at));
      raw.to_float(v[i]);
    } else if constexpr (TYPE == kTypeF32) {
      if constexpr (VEC == 2) {
        const float2 f = static_cast<const float2*>(row)[at];
        v[i][0] = f.x;
        v[i][1] = f.y;
      } else {
        v[i][0] = static_cast<const float*>(row)[at];
      }
    } else if constexpr (VEC == 2) {
      const float2 f = unpack16(static_cast<const uint32_t*>(row)[at], TYPE);
      v[i][0] = f.x;
      v[i][1] = f.y;
    } else {
      const uint32_t h = static_cast<const uint16_t*>(row)[at];
      v[i][0] = TYPE == kTypeBf16 ? __uint_as_float(h << 16) : bits_f16(h);
    }
  }
}
template <int VEC, int E>
__device__ __forceinline__ void load_pieces(const void* row, int type, int first, int step, int pieces, float (&v)[E][VEC]) {
  if (type == kTypeF32)
    load_pieces<kTypeF32>(row, first, step, pieces, v);
  else if (type == kTypeBf16)
    load_pieces<kTypeBf16>(row, first, step, pieces, v);
  else
    load_pieces<kTypeF16>(row, first, step, pieces, v);
}
template <int TYPE, int VEC, int E>
__device__ __forceinline__ void store_pieces(void* row, int first, int step, int pieces, const float (&v)[E][VEC]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int at = first + i * step;
    if (at >= pieces) continue;
    if constexpr (VEC == 8)
      store8_as<TYPE>(row, 8 * static_cast<int64_t>(at), v[i]);
    else if constexpr (VEC == 1)
      store_one(row, at, TYPE, v[i][0]);
    else if constexpr (TYPE == kTypeF32)
      static_cast<float2*>(row)[at] = make_float2(v[i][0], v[i][1]);
    else if constexpr (TYPE == kTypeE4m3)
      static_cast<uint16_t*>(row)[at] = static_cast<uint16_t>(pack_e4m3(v[i][0], v[i][1]));
    else
      static_cast<uint32_t*>(row)[at] = pack16(v[i][0], v[i][1], TYPE);
  }
}
template <int VEC, int E>
__device__ __forceinline__ void store_pieces(void* row, int type, int first, int step, int pieces, const float (&v)[E][VEC]) {
  switch (type) {
    case kTypeF32: store_pieces<kTypeF32>(row, first, step, pieces, v); break;
    case kTypeBf16: store_pieces<kTypeBf16>(row, first, step, pieces, v); break;
    case kTypeF16: store_pieces<kTypeF16>(row, first, step, pieces, v); break;
    default: store_pieces<kTypeE4m3>(row, first, step, pieces, v);
  }
}

constexpr int any_threads(int e) { return e == 4 ? 128 : 1024; }              // of a block, at most
constexpr int any_blocks(int vec, int e) { return e == 4 ? 12 / vec + 2 * (vec - 1) : 1; }  // of that size an SM
template <int VEC, int E, bool LONG>
__global__ void __launch_bounds__(any_threads(E), any_blocks(VEC, E)) norm_any_kernel(NormArgs a) {
  extern __shared__ float h_row[];  // LONG only
  __shared__ RowStat parts[2][32];
  int turn = 0;
  const int tid = threadIdx.x, step = blockDim.x, pieces = static_cast<int>(a.K / VEC), span = E * step;
  const bool codes = a.out_type == kTypeE4m3;
  wait_for_previous();
  start_next();
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const void* x = row_at(a.X, m * a.x_stride, a.x_type);
    const void* r = row_at(a.residual, m * a.r_stride, a.r_type);
    void* ro = const_cast<void*>(row_at(a.residual_out, m * a.ro_stride, a.r_type));
    void* out = const_cast<void*>(row_at(a.out, m * a.K, a.out_type));
    float h[E][VEC];
    RowStat st{0.0f, 0u};
    for (int base = 0; base < pieces; base += span) {
      const int first = base + tid;
      float w[E][VEC];
      load_pieces(x, a.x_type, first, step, pieces, h);
      if (a.residual) {
        load_pieces(r, a.r_type, first, step, pieces, w);
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
          for (int k = 0; k < VEC; ++k) h[i][k] = __fadd_rn(h[i][k], w[i][k]);
        store_pieces(ro, a.r_type, first, step, pieces, h);
      }
      load_pieces(a.weight, a.w_type, first, step, pieces, w);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (first + i * step >= pieces) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          st.ss = __fmaf_rn(h[i][k], h[i][k], st.ss);
          h[i][k] = __fmul_rn(h[i][k], w[i][k]);
          if (codes) st.peak = max(st.peak, __float_as_uint(h[i][k]) & 0x7FFFFFFFu);
          if (LONG) h_row[((base + i * step) * VEC) + k * step + tid] = h[i][k];
        }
      }
    }
    st = block_join(st, codes, parts, turn);
    const float factor = row_factor(st.ss, a);
    const Divisor scale(codes ? row_scale(st.peak, factor) : 1.0f);
    if (codes && tid == 0) a.out_scales[m] = scale.scale;
    for (int base = 0; base < pieces; base += span) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (base + tid + i * step >= pieces) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          if (LONG) h[i][k] = h_row[((base + i * step) * VEC) + k * step + tid];
          h[i][k] = __fmul_rn(h[i][k], factor);
        }
        if (codes) scale.divide(h[i]);
      }
      store_pieces(out, a.out_type, base + tid, step, pieces, h);
    }
  }
}

}  // namespace

namespace {

template <int TX, int TR, int VPT, int LANES>
cudaError_t launch_norm(const NormArgs& a, int threads, int num_sms, cudaStream_t s, int* launches) {
  const int64_t per = LANES ? threads / LANES : 1;
  const int resident = std::min(32, norm_threads(LANES) * norm_blocks(VPT, LANES) / threads);  // blocks an SM
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(ceil_div(a.M, per), static_cast<int64_t>(resident) * num_sms));
  return launch_early(norm_kernel<TX, TR, VPT, LANES>, dim3(blocks), threads, 0, s, launches, a);
}

template <int TX, int TR>
cudaError_t launch_norm_types(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int64_t vecs = a.K / 8;
  if (vecs <= 128 && a.M > num_sms) {  // rows of a warp or of a part of one
    if (vecs <= 8) return launch_norm<TX, TR, 1, 8>(a, 256, num_sms, s, launches);
    if (vecs <= 16) return launch_norm<TX, TR, 1, 16>(a, 256, num_sms, s, launches);
    if (vecs <= 32) return launch_norm<TX, TR, 1, 32>(a, 256, num_sms, s, launches);
    return launch_norm<TX, TR, 4, 32>(a, 256, num_sms, s, launches);
  }
  // More vectors a thread share a warp's fixed cost of a row, fewer leave more warps to a row. With
  // rows enough for both: without a residual, 16384 rows of 4096 in bf16 take 46 us at two and 56 at one;
  // with one, 16384 rows of 8192 take 168 us at four and 173 at two, but as e4m3, whose output
  // has more instructions, 8192 rows of 7168 take 71 and 66.
  const bool many = a.M > 8 * num_sms;
  const int vpt = vecs <= 512    ? (many && TR == kTypeNone ? 2 : 1)
                  : vecs <= 1024 ? (many && TR != kTypeNone && a.out_type != kTypeE4m3 ? 4 : 2)
                                 : 4;
  const int threads = static_cast<int>(ceil_div(ceil_div(vecs, vpt), 32) * 32);
  if (vpt == 1) return launch_norm<TX, TR, 1, 0>(a, threads, num_sms, s, launches);
  if (vpt == 2) return launch_norm<TX, TR, 2, 0>(a, threads, num_sms, s, launches);
  return launch_norm<TX, TR, 4, 0>(a, threads, num_sms, s, launches);
}

template <int TX>
cudaError_t launch_norm_residual(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  switch (a.residual ? a.r_type : kTypeNone) {
    case kTypeNone: return launch_norm_types<TX, kTypeNone>(a, num_sms, s, launches);
    case kTypeF32: return launch_norm_types<TX, kTypeF32>(a, num_sms, s, launches);
    case kTypeF16: return launch_norm_types<TX, kTypeF16>(a, num_sms, s, launches);
    default: return launch_norm_types<TX, kTypeBf16>(a, num_sms, s, launches);
  }
}

// Whether the rows of every tensor start at whole pieces of `vec` values.
bool rows_aligned(const NormArgs& a, int vec) {
  auto whole = [&](const void* p, int64_t stride, int type) {
    const int64_t bytes = std::min(16, vec * type_bytes(type));  // of a load or store
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (a.M == 1 || stride * type_bytes(type) % bytes == 0);
  };
  return a.K % vec == 0 && whole(a.X, a.x_stride, a.x_type) && whole(a.weight, 0, a.w_type) && whole(a.out, a.K, a.out_type) &&
         (!a.residual || (whole(a.residual, a.r_stride, a.r_type) && whole(a.residual_out, a.ro_stride, a.r_type)));
}

// Whether row m of every tensor starts (m K) mod 8 values beyond a whole vector, and the next row
// behind its end (whose values a row's last window may read).
bool rows_shifted(const NormArgs& a) {
  auto like = [&](const void* p, int64_t stride, int type) {
    return reinterpret_cast<uintptr_t>(p) % std::min(16, 8 * type_bytes(type)) == 0 && (a.M == 1 || (stride >= a.K && (stride - a.K) % 8 == 0));
  };
  return like(a.X, a.x_stride, a.x_type) && like(a.out, a.K, a.out_type) &&
         (!a.residual || (like(a.residual, a.r_stride, a.r_type) && like(a.residual_out, a.ro_stride, a.r_type)));
}

template <int VEC, int E, bool LONG>
cudaError_t launch_any(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int64_t pieces = a.K / VEC;
  const int threads = LONG ? 1024 : static_cast<int>(ceil_div(ceil_div(pieces, E), 32) * 32);
  // of a long row every turn has its own places, the last one's whether or not they are all used
  const size_t smem = LONG ? static_cast<size_t>(ceil_div(pieces, threads) * threads * VEC) * 4 : 0;
  if (LONG) {
    static unsigned long long done = 0;
    const cudaError_t e = set_smem_limit_once(norm_any_kernel<VEC, E, LONG>, static_cast<int>(kNormMaxK * 4), &done);
    if (e != cudaSuccess) return e;
  }
  const int resident = LONG ? 1 : std::min(32, any_threads(E) * any_blocks(VEC, E) / threads);  // blocks an SM
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(a.M, static_cast<int64_t>(resident) * num_sms));
  return launch_early(norm_any_kernel<VEC, E, LONG>, dim3(blocks), threads, smem, s, launches, a);
}

template <int VEC>
cudaError_t launch_any_length(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int64_t pieces = a.K / VEC;
  if constexpr (VEC < 8) {
    if (pieces <= 4 * 128) return launch_any<VEC, 4, false>(a, num_sms, s, launches);
    if (pieces <= (16 / VEC) * 1024) return launch_any<VEC, 16 / VEC, false>(a, num_sms, s, launches);
  }
  return launch_any<VEC, 16 / VEC, true>(a, num_sms, s, launches);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t s, int* launches) {
  if (rows_aligned(a, 8)) {
    if (a.K > 16384) return launch_any_length<8>(a, num_sms, s, launches);
    if (a.x_type == kTypeF32) return launch_norm_residual<kTypeF32>(a, num_sms, s, launches);
    if (a.x_type == kTypeF16) return launch_norm_residual<kTypeF16>(a, num_sms, s, launches);
    return launch_norm_residual<kTypeBf16>(a, num_sms, s, launches);
  }
  if (rows_shifted(a) && a.K >= 64 && a.K < 16384) return launch_rms_norm_shifted(a, num_sms, s, launches);
  if (rows_aligned(a, 2)) return launch_any_length<2>(a, num_sms, s, launches);
  return launch_any_length<1>(a, num_sms, s, launches);
}

}  // namespace awq
