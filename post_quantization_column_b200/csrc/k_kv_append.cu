// k_kv_append.cu — the position rotation of queries and keys and the append of keys and
// values to a paged cache, between the QKV product of a quantized attention block and its
// attention.
//
// Token t at position p: the angle of pair i < rot / 2 is p f_i; a pair (x, y) of a query or
// key head becomes (x c - y s, x s + y c) with c = m cos, s = m sin (m the magnitude of the
// frequency scaling). Pairs are dims (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved;
// dims from rot on stay as they are. The product p f_i is taken in fp64 and reduced to a
// fraction of a turn there, so that a position of a million loses no more than 1e-9 turns;
// the sine and cosine of the fraction are fp32. Results are rounded once to the query's and
// the cache's types (an e4m3 cache holds e4m3(x / scale) of its head's scale).
#include "decode_kernels.h"

#include <algorithm>

namespace awq {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxRot = 256;

// A unit is 16 values of one head: dims 8u .. 8u + 7 and rot/2 + 8u .. of a rotated half
// layout, 16 consecutive dims otherwise. Returns the two vectors' first dims.
__device__ __forceinline__ void unit_dims(int u, int rot, bool half_pairs, int* d0, int* d1) {
  if (half_pairs && 16 * u < rot) {
    *d0 = 8 * u;
    *d1 = rot / 2 + 8 * u;
  } else {
    *d0 = 16 * u;
    *d1 = 16 * u + 8;
  }
}

// One token per blockIdx.x; each of the gridDim.y blocks of the token takes U units per thread
// of its Hq + 2 Hkv heads, and has them on the way before it works out the angles.
template <int XB, int U>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendArgs a) {
  __shared__ float sCos[kMaxRot / 2], sSin[kMaxRot / 2];
  const int64_t t = blockIdx.x;
  const PagedCache& c = a.c;
  const int D = c.head_dim, shift = 31 - __clz(D / 16);  // log2 of a head's units
  const int units = (a.Hq + 2 * c.heads) << shift;
  wait_for_previous();
  start_next();
  Raw8<XB> r0[U], r1[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int w = (blockIdx.y * U + i) * kAppendThreads + threadIdx.x;
    if (w >= units) continue;
    const int head = w >> shift, u = w & ((1 << shift) - 1);
    const bool is_q = head < a.Hq, is_v = head >= a.Hq + c.heads;
    int d0, d1;
    unit_dims(u, a.rot, !is_v && !a.interleaved, &d0, &d1);
    const void* src = is_q ? a.q : (is_v ? a.v : a.k);
    const int64_t at = is_q ? t * a.q_st + head * a.q_sh
                            : (is_v ? t * a.v_st + (head - a.Hq - c.heads) * a.v_sh : t * a.k_st + (head - a.Hq) * a.k_sh);
    r0[i].load(src, at + d0);
    r1[i].load(src, at + d1);
  }
  const int pos = a.positions[t];
  const int64_t seq = a.seq ? a.seq[t] : t;
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < half; i += kAppendThreads) {
    const double turns = static_cast<double>(pos) * a.freqs[i] * 0.15915494309189533577;  // 1 / (2 pi)
    const float frac = static_cast<float>(turns - rint(turns));
    float sn, cs;
    sincospif(2.0f * frac, &sn, &cs);
    sCos[i] = __fmul_rn(a.magnitude, cs);
    sSin[i] = __fmul_rn(a.magnitude, sn);
  }
  // where the token's keys and values go
  int64_t row = -1;
  if (pos >= 0) {
    const int pi = pos / c.page_size;
    if (seq >= 0 && seq < c.seqs && pi < c.max_pages) {
      const int64_t page = c.table[seq * c.table_stride + pi];
      if (page >= 0 && page < c.num_pages)
        row = page * c.page_stride + static_cast<int64_t>(pos - pi * c.page_size) * c.slot_stride;
    }
    if (row < 0 && a.status && threadIdx.x == 0 && blockIdx.y == 0) *a.status = 1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int w = (blockIdx.y * U + i) * kAppendThreads + threadIdx.x;
    if (w >= units) continue;
    const int head = w >> shift, u = w & ((1 << shift) - 1);
    const bool is_q = head < a.Hq, is_v = head >= a.Hq + c.heads;
    if (!is_q && row < 0) continue;
    const int hh = is_q ? head : (is_v ? head - a.Hq - c.heads : head - a.Hq);
    int d0, d1;
    unit_dims(u, a.rot, !is_v && !a.interleaved, &d0, &d1);
    float x[8], y[8];
    r0[i].to_float(x, a.in_type);
    r1[i].to_float(y, a.in_type);
    if (!is_v && 16 * u < a.rot) {
      if (a.interleaved) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float c0 = sCos[8 * u + k], s0 = sSin[8 * u + k], c1 = sCos[8 * u + 4 + k], s1 = sSin[8 * u + 4 + k];
          const float xa = x[2 * k], xb = x[2 * k + 1], ya = y[2 * k], yb = y[2 * k + 1];
          x[2 * k] = xa * c0 - xb * s0;
          x[2 * k + 1] = xa * s0 + xb * c0;
          y[2 * k] = ya * c1 - yb * s1;
          y[2 * k + 1] = ya * s1 + yb * c1;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float cs = sCos[8 * u + k], sn = sSin[8 * u + k], xa = x[k], xb = y[k];
          x[k] = xa * cs - xb * sn;
          y[k] = xa * sn + xb * cs;
        }
      }
    }
    if (is_q) {
      const int64_t to = (t * a.Hq + hh) * D;
      if (pos < 0) {  // a padded row of the batch
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = y[k] = 0.0f;
      }
      store8(a.q_out, to + d0, a.q_type, x);
      store8(a.q_out, to + d1, a.q_type, y);
    } else {
      if (c.type == kTypeE4m3) {
        const float scale = (is_v ? c.v_scale : c.k_scale)[hh];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = __fdiv_rn(x[k], scale);
          y[k] = __fdiv_rn(y[k], scale);
        }
      }
      void* dst = is_v ? c.v : c.k;
      store8(dst, row + hh * c.head_stride + d0, c.type, x);
      store8(dst, row + hh * c.head_stride + d1, c.type, y);
    }
  }
}

template <int XB>
cudaError_t launch(const AppendArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int units = (a.Hq + 2 * a.c.heads) * (a.c.head_dim / 16);
  const int64_t blocks = ceil_div(units, kAppendThreads);  // of a token, at one unit per thread
  // a few tokens are spread over the SMs; of many each block takes what it can keep on the way
  const int per = a.T * blocks < 4 * num_sms || blocks == 1 ? 1 : (blocks == 2 || blocks == 4 ? 2 : 3);
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(ceil_div(blocks, per)));
  auto kernel = per == 1 ? kv_append_kernel<XB, 1> : (per == 2 ? kv_append_kernel<XB, 2> : kv_append_kernel<XB, 3>);
  return launch_early(kernel, grid, kAppendThreads, 0, s, launches, a);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int num_sms, cudaStream_t s, int* launches) {
  return type_bytes(a.in_type) == 4 ? launch<4>(a, num_sms, s, launches) : launch<2>(a, num_sms, s, launches);
}

}  // namespace awq
