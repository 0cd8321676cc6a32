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
//
// What bounds it: the bytes of q, k and v, read and written once. The angles are worked out once
// per block of a token, while its values are on the way; a thread turns 16 values of a head. In
// a captured graph 4096 tokens of 32 + 2 x 32 bf16 heads take 35 us, 5.7 TB/s (address and
// conversion instructions keep the issue slots half busy), 2047 tokens of 64 + 2 x 8 fp32 heads
// 20 us, 6.3 TB/s, one token 1.8 us. A persistent form that loads the next token's values early
// took 50 us for the former: its registers halve the blocks an SM holds.
#include "decode_kernels.h"

#include <algorithm>

namespace awq {
namespace {

constexpr int kAppendThreads = 128;
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
template <int IN, int CACHE, int U>
__global__ void __launch_bounds__(kAppendThreads, 8) kv_append_kernel(AppendArgs a) {
  __shared__ __align__(16) float sCos[kMaxRot / 2], sSin[kMaxRot / 2];
  const int64_t t = blockIdx.x;
  const PagedCache& c = a.c;
  const int D = c.head_dim, shift = 31 - __clz(D / 16);  // log2 of a head's units
  const int units = (a.Hq + 2 * c.heads) << shift;
  wait_for_previous();
  start_next();
  constexpr int B = type_bytes(IN);
  const uint8_t *q = static_cast<const uint8_t*>(a.q) + t * a.q_st * B, *k = static_cast<const uint8_t*>(a.k) + t * a.k_st * B,
                *v = static_cast<const uint8_t*>(a.v) + t * a.v_st * B;
  Raw8<IN> r0[U], r1[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int w = (blockIdx.y * U + i) * kAppendThreads + threadIdx.x;
    if (w >= units) continue;
    const int head = w >> shift, u = w & ((1 << shift) - 1), kh = head - a.Hq, vh = kh - c.heads;
    int d0, d1;
    unit_dims(u, a.rot, vh < 0 && !a.interleaved, &d0, &d1);
    const uint8_t* src = kh < 0 ? q : (vh < 0 ? k : v);
    const uint32_t step = kh < 0 ? a.q_head : (vh < 0 ? a.k_head : a.v_head), hh = kh < 0 ? head : (vh < 0 ? kh : vh);
    src += static_cast<uint64_t>(hh) * step;
    r0[i].load(src, d0);
    r1[i].load(src, d1);
  }
  const int pos = a.positions[t];
  const int64_t seq = a.seq ? a.seq[t] : t;
  const int half = a.rot / 2;
  static_assert(kMaxRot / 2 <= kAppendThreads, "one angle per thread");
  if (threadIdx.x < half) {
    const double turns = static_cast<double>(pos) * a.freqs[threadIdx.x] * 0.15915494309189533577;  // 1 / (2 pi)
    const float frac = static_cast<float>(turns - rint(turns));
    float sn, cs;
    sincospif(2.0f * frac, &sn, &cs);
    sCos[threadIdx.x] = __fmul_rn(a.magnitude, cs);
    sSin[threadIdx.x] = __fmul_rn(a.magnitude, sn);
  }
  // where the token's keys and values go
  int64_t row = -1;  // bytes
  if (pos >= 0) {
    const int pi = pos / c.page_size;
    if (seq >= 0 && seq < c.seqs && pi < c.max_pages) {
      const int64_t page = c.table[seq * c.table_stride + pi];
      if (page >= 0 && page < c.num_pages)
        row = (page * c.page_stride + static_cast<int64_t>(pos - pi * c.page_size) * c.slot_stride) * type_bytes(CACHE);
    }
    if (row < 0 && a.status && threadIdx.x == 0 && blockIdx.y == 0) *a.status = 1;
  }
  uint16_t* q_out = static_cast<uint16_t*>(a.q_out) + t * a.Hq * D;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int w = (blockIdx.y * U + i) * kAppendThreads + threadIdx.x;
    if (w >= units) continue;
    const int head = w >> shift, u = w & ((1 << shift) - 1), kh = head - a.Hq, vh = kh - c.heads;
    int d0, d1;
    unit_dims(u, a.rot, vh < 0 && !a.interleaved, &d0, &d1);
    float x[8], y[8];
    r0[i].to_float(x);
    r1[i].to_float(y);
    if (vh < 0 && 16 * u < a.rot) {
      float cs[8], sn[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<float4*>(cs + 4 * k) = *reinterpret_cast<const float4*>(sCos + 8 * u + 4 * k);
        *reinterpret_cast<float4*>(sn + 4 * k) = *reinterpret_cast<const float4*>(sSin + 8 * u + 4 * k);
      }
      if (a.interleaved) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float xa = x[2 * k], xb = x[2 * k + 1], ya = y[2 * k], yb = y[2 * k + 1];
          x[2 * k] = xa * cs[k] - xb * sn[k];
          x[2 * k + 1] = xa * sn[k] + xb * cs[k];
          y[2 * k] = ya * cs[4 + k] - yb * sn[4 + k];
          y[2 * k + 1] = ya * sn[4 + k] + yb * cs[4 + k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xa = x[k], xb = y[k];
          x[k] = xa * cs[k] - xb * sn[k];
          y[k] = xa * sn[k] + xb * cs[k];
        }
      }
    }
    if (kh < 0) {
      if (pos < 0) {  // a padded row of the batch
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = y[k] = 0.0f;
      }
      uint16_t* to = q_out + head * D;
      if (a.q_type == kTypeBf16) {
        store8_as<kTypeBf16>(to, d0, x);
        store8_as<kTypeBf16>(to, d1, y);
      } else {
        store8_as<kTypeF16>(to, d0, x);
        store8_as<kTypeF16>(to, d1, y);
      }
    } else if (row >= 0) {
      const int hh = vh < 0 ? kh : vh;
      if constexpr (CACHE == kTypeE4m3) {
        const Divisor scale((vh < 0 ? c.k_scale : c.v_scale)[hh]);
        scale.divide(x);
        scale.divide(y);
      }
      uint8_t* dst = static_cast<uint8_t*>(vh < 0 ? c.k : c.v) + row + static_cast<uint64_t>(static_cast<uint32_t>(hh) * a.cache_head32) * 32u;
      store8_as<CACHE>(dst, d0, x);
      store8_as<CACHE>(dst, d1, y);
    }
  }
}

template <int IN, int CACHE>
cudaError_t launch(const AppendArgs& a, int num_sms, cudaStream_t s, int* launches) {
  const int units = (a.Hq + 2 * a.c.heads) * (a.c.head_dim / 16);
  const int64_t blocks = ceil_div(units, kAppendThreads);  // of a token, at one unit per thread
  // a few tokens are spread over the SMs; of many each thread takes two units (4096 tokens of 32 + 2 x
  // 32 heads in bf16: 35.6 us against 41.5 with one; three are 35.1 in 16 bits, but in fp32, where
  // two take 19.9 us for 2047 tokens of 64 + 2 x 8 heads, 22.9)
  const int per = a.T * blocks < 8 * num_sms || blocks == 1 ? 1 : 2;
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(ceil_div(blocks, per)));
  auto kernel = per == 1 ? kv_append_kernel<IN, CACHE, 1> : kv_append_kernel<IN, CACHE, 2>;
  return launch_early(kernel, grid, kAppendThreads, 0, s, launches, a);
}

template <int IN>
cudaError_t launch_cache(const AppendArgs& a, int num_sms, cudaStream_t s, int* launches) {
  switch (a.c.type) {
    case kTypeBf16: return launch<IN, kTypeBf16>(a, num_sms, s, launches);
    case kTypeF16: return launch<IN, kTypeF16>(a, num_sms, s, launches);
    default: return launch<IN, kTypeE4m3>(a, num_sms, s, launches);
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int num_sms, cudaStream_t s, int* launches) {
  switch (a.in_type) {
    case kTypeF32: return launch_cache<kTypeF32>(a, num_sms, s, launches);
    case kTypeF16: return launch_cache<kTypeF16>(a, num_sms, s, launches);
    default: return launch_cache<kTypeBf16>(a, num_sms, s, launches);
  }
}

}  // namespace awq
