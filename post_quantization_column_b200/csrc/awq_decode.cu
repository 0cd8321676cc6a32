// awq_decode.cu — the C ABI of the decode-step operators (declared in include/awq_search.h):
// checks of the arguments, the device of the call, and the launches. All of it is
// asynchronous on the caller's stream, allocates nothing and keeps nothing between calls.
#include "decode_entry.h"
#include "decode_kernels.h"

#include <algorithm>
#include <array>
#include <cmath>
#include <utility>

namespace {

using namespace awq;

static_assert(kTypeBf16 == AWQ_DTYPE_BF16 && kTypeF32 == AWQ_DTYPE_F32 && kTypeF16 == AWQ_DTYPE_F16 &&
                  kTypeE4m3 == AWQ_DTYPE_E4M3,
              "the kernels' types are the ABI's");

constexpr int64_t kIntMax = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_float(int t) { return t == kTypeF32 || t == kTypeF16 || t == kTypeBf16; }

// Whether the rows of a and of b, `wa` and `wb` bytes each and `sa` and `sb` bytes apart, meet; rows at
// one distance may lie between each other (columns of one buffer).
bool ranges_meet(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t rows) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  if (a0 >= b0 + (rows - 1) * sb + wb || b0 >= a0 + (rows - 1) * sa + wa) return false;
  if (sa != sb || sa < wa + wb) return true;
  const int64_t apart = static_cast<int64_t>(b0 - a0) % sa, d = apart < 0 ? apart + sa : apart;  // from a row of a to the next of b
  return d < wa || d + wb > sa;
}

// The bytes from a tensor's first to its last value: `n` rows `stride` bytes apart, of `m` parts `part`
// bytes apart, each `bytes` long.
struct Extent {
  uintptr_t from;
  unsigned __int128 to;
};
Extent extent(const void* p, int64_t n, int64_t stride, int64_t m, int64_t part, int64_t bytes) {
  const uintptr_t from = reinterpret_cast<uintptr_t>(p);
  return {from, from + static_cast<unsigned __int128>(n - 1) * stride + static_cast<unsigned __int128>(m - 1) * part + bytes};
}
Extent extent(const PagedCache& c, const void* p) {
  const int64_t b = type_bytes(c.type);
  return extent(p, c.num_pages, c.page_stride * b, c.page_size, c.slot_stride * b, ((c.heads - 1) * c.head_stride + c.head_dim) * b);
}
bool meet(const Extent& a, const Extent& b) { return a.from < b.to && b.from < a.to; }

// The device of the call is asked of its pointers; else the binding calls, with outputs of its own.
constexpr int kAsk = -1;

// Makes the device of the call current: the caller's, which owns all its pointers (the Python
// binding knows its tensors' device), or that of `first`, where every pointer must lie. A kernel that
// meets a bad page stores to `status` (may be NULL), so an address that it cannot reach is refused here.
int take_device(int device, const void* first, const void* const* ptrs, int n, const int32_t* status, int* num_sms) {
  int dev = device;
  const int st = decode_device(first, &dev, num_sms);
  if (st != AWQ_OK || device != kAsk) return st;
  for (int i = 0; i < n; ++i)
    if (ptrs[i] && !decode_device_memory(ptrs[i], dev))
      return decode_error(AWQ_ERR_INVALID_ARG, "inputs and outputs must be memory of the device the call runs on");
  if (status && !decode_status_memory(status, dev))
    return decode_error(AWQ_ERR_INVALID_ARG, "status must be memory of the device the call runs on, or pinned host memory");
  return AWQ_OK;
}

// The cache's descriptor as the kernels take it.
int take_cache(const awq_paged_cache* in, PagedCache* out) {
  if (!in) return decode_error(AWQ_ERR_INVALID_ARG, "the cache descriptor is NULL");
  if (!in->k || !in->v || !in->block_table) return decode_error(AWQ_ERR_INVALID_ARG, "a required pointer of the cache is NULL");
  if (in->dtype != kTypeBf16 && in->dtype != kTypeF16 && in->dtype != kTypeE4m3)
    return decode_error(AWQ_ERR_INVALID_ARG, "the cache holds AWQ_DTYPE_BF16, AWQ_DTYPE_F16 or AWQ_DTYPE_E4M3");
  if (in->dtype == kTypeE4m3 && (!in->k_scale || !in->v_scale))
    return decode_error(AWQ_ERR_INVALID_ARG, "an e4m3 cache needs k_scale and v_scale");
  if (in->head_dim != 64 && in->head_dim != 128 && in->head_dim != 256)
    return decode_error(AWQ_ERR_SHAPE, "head_dim must be 64, 128 or 256");
  if (in->heads < 1 || in->heads > 65535 || in->page_size < 1 || in->num_pages < 1 || in->n_seqs < 1 ||
      in->max_pages < 1 || in->page_size > kIntMax || in->num_pages > kIntMax || in->n_seqs > kIntMax)
    return decode_error(AWQ_ERR_SHAPE, "heads, page_size, num_pages, n_seqs and max_pages must be positive");
  if (in->max_pages > (kIntMax - 1024) / in->page_size)
    return decode_error(AWQ_ERR_SHAPE, "a block table row names 2^31 tokens or more");
  const int64_t per32 = 32 / type_bytes(static_cast<int>(in->dtype));
  // the stride of a dim of one is never taken
  const int64_t strides[3] = {in->num_pages > 1 ? in->page_stride : 0, in->page_size > 1 ? in->slot_stride : 0,
                              in->heads > 1 ? in->head_stride : 0};
  if (!aligned(in->k, 32) || !aligned(in->v, 32) || strides[0] % per32 || strides[1] % per32 || strides[2] % per32)
    return decode_error(AWQ_ERR_INVALID_ARG, "the cache's rows must be 32-byte aligned");
  if (strides[0] < 0 || strides[1] < 0 || strides[2] < 0 || in->table_stride < 0)
    return decode_error(AWQ_ERR_INVALID_ARG, "strides must not be negative");
  // places within the cache are counted in units of 32 bytes, in 32 bits; a division keeps the
  // check itself from overflowing
  const int64_t room = ((int64_t(1) << 32) - 2) * per32 - in->head_dim, steps[3] = {in->num_pages - 1, in->page_size - 1, in->heads - 1};
  int64_t span = 0;
  for (int i = 0; i < 3; ++i) {
    if (steps[i] > 0 && strides[i] > (room - span) / steps[i])
      return decode_error(AWQ_ERR_SHAPE, "the keys or the values of a cache span 128 GB or more");
    span += steps[i] * strides[i];
  }
  if (!aligned(in->block_table, 4) || !aligned(in->k_scale, 4) || !aligned(in->v_scale, 4))
    return decode_error(AWQ_ERR_INVALID_ARG, "the block table or a scale is misaligned");
  out->k = in->k;
  out->v = in->v;
  out->num_pages = in->num_pages;
  out->page_stride = strides[0];
  out->slot_stride = strides[1];
  out->head_stride = strides[2];
  out->page_size = static_cast<int>(in->page_size);
  out->heads = static_cast<int>(in->heads);
  out->head_dim = static_cast<int>(in->head_dim);
  out->type = static_cast<int>(in->dtype);
  out->k_scale = in->dtype == kTypeE4m3 ? in->k_scale : nullptr;
  out->v_scale = in->dtype == kTypeE4m3 ? in->v_scale : nullptr;
  out->table = in->block_table;
  out->seqs = in->n_seqs;
  out->max_pages = in->max_pages;
  out->table_stride = in->table_stride;
  return AWQ_OK;
}

// Whether no two rows of the cache overlap: each of pages, slots and heads steps over the whole of
// what steps less, as in any order of the three and any part of such a cache.
bool rows_apart(const PagedCache& c) {
  std::array<std::pair<int64_t, int64_t>, 3> dims{{{c.page_stride, c.num_pages - 1}, {c.slot_stride, c.page_size - 1}, {c.head_stride, c.heads - 1}}};
  std::sort(std::begin(dims), std::end(dims));
  int64_t span = c.head_dim;  // the sum is within what take_cache has checked
  for (const auto& [stride, steps] : dims) {
    if (steps > 0 && stride < span) return false;
    span += stride * steps;
  }
  return true;
}

}  // namespace

extern "C" {

int awq_rms_norm_on(int device, const void* X, int x_dtype, int64_t x_stride, const void* residual, int r_dtype, int64_t r_stride,
                 void* residual_out, int64_t ro_stride, const void* weight, int w_dtype, int64_t M, int64_t K,
                 float eps, void* out, int out_dtype, float* out_scales, awq_stream_t stream) {
  decode_error(AWQ_OK, "");
  if (M < 0 || M > kIntMax || K < 1) return decode_error(AWQ_ERR_SHAPE, "M must be in 0 .. 2^31 - 1 and K positive");
  if (K > kNormMaxK) return decode_error(AWQ_ERR_SHAPE, "a row holds at most 57344 values");
  if (!is_float(x_dtype) || !is_float(w_dtype) || (residual && !is_float(r_dtype)))
    return decode_error(AWQ_ERR_INVALID_ARG, "X, residual and weight hold AWQ_DTYPE_F32, AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  if (!is_float(out_dtype) && out_dtype != kTypeE4m3) return decode_error(AWQ_ERR_INVALID_ARG, "unknown output type");
  if (!(eps >= 0.0f) || std::isinf(eps)) return decode_error(AWQ_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (M == 0) return AWQ_OK;
  if (!X || !weight || !out) return decode_error(AWQ_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((residual == nullptr) != (residual_out == nullptr))
    return decode_error(AWQ_ERR_INVALID_ARG, "residual and residual_out come together");
  if (out_dtype == kTypeE4m3 && !out_scales) return decode_error(AWQ_ERR_INVALID_ARG, "an e4m3 output needs out_scales");
  const int xb = type_bytes(x_dtype), wb = type_bytes(w_dtype), rb = residual ? type_bytes(r_dtype) : 1, ob = type_bytes(out_dtype);
  if (!aligned(X, xb) || !aligned(weight, wb) || !aligned(out, ob) || !aligned(out_scales, 4) ||
      !aligned(residual, rb) || !aligned(residual_out, rb))
    return decode_error(AWQ_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (x_stride < 0 || (residual && (r_stride < 0 || ro_stride < K)))
    return decode_error(AWQ_ERR_INVALID_ARG, "row strides must not be negative, and rows of residual_out must not overlap");
  if (residual) {
    const bool same = residual == residual_out && r_stride == ro_stride;
    if ((!same && ranges_meet(residual, r_stride * rb, K * rb, residual_out, ro_stride * rb, K * rb, M)) ||
        ranges_meet(X, x_stride * xb, K * xb, residual_out, ro_stride * rb, K * rb, M) ||
        ranges_meet(weight, 0, K * wb, residual_out, ro_stride * rb, K * rb, M))
      return decode_error(AWQ_ERR_INVALID_ARG, "residual_out may be the residual itself but overlap nothing else");
  }
  if (ranges_meet(X, x_stride * xb, K * xb, out, K * ob, K * ob, M) || ranges_meet(weight, 0, K * wb, out, K * ob, K * ob, M) ||
      (residual && (ranges_meet(residual, r_stride * rb, K * rb, out, K * ob, K * ob, M) ||
                    ranges_meet(residual_out, ro_stride * rb, K * rb, out, K * ob, K * ob, M))))
    return decode_error(AWQ_ERR_INVALID_ARG, "out must not overlap another argument");
  if (out_dtype == kTypeE4m3 && device == kAsk) {
    const Extent to = extent(out_scales, M, 4, 1, 0, 4);
    if (meet(to, extent(X, M, x_stride * xb, 1, 0, K * xb)) || meet(to, extent(weight, 1, 0, 1, 0, K * wb)) ||
        meet(to, extent(out, M, K, 1, 0, K)) ||
        (residual && (meet(to, extent(residual, M, r_stride * rb, 1, 0, K * rb)) || meet(to, extent(residual_out, M, ro_stride * rb, 1, 0, K * rb)))))
      return decode_error(AWQ_ERR_INVALID_ARG, "out_scales must not overlap another argument");
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DeviceRestore restore_device;
  const void* ptrs[] = {X, residual, residual_out, weight, out, out_dtype == kTypeE4m3 ? out_scales : nullptr};
  int num_sms = 0;
  const int st = take_device(device, X, ptrs, 6, nullptr, &num_sms);
  if (st != AWQ_OK) return st;
  NormArgs a;
  a.X = X;
  a.residual = residual;
  a.residual_out = residual_out;
  a.weight = weight;
  a.out = out;
  a.out_scales = out_scales;
  a.M = M;
  a.K = K;
  a.inverse_k = 1.0f / static_cast<float>(K);
  a.x_stride = x_stride;
  a.r_stride = r_stride;
  a.ro_stride = ro_stride;
  a.x_type = x_dtype;
  a.r_type = residual ? r_dtype : kTypeNone;
  a.w_type = w_dtype;
  a.out_type = out_dtype;
  a.eps = eps;
  int launches = 0;
  const cudaError_t e = launch_rms_norm(a, num_sms, s, &launches);
  if (e != cudaSuccess) return decode_cuda_error(e, "RMS norm");
  record_launch_count(launches);
  return AWQ_OK;
}
int awq_rms_norm(const void* X, int x_dtype, int64_t x_stride, const void* residual, int r_dtype, int64_t r_stride,
                 void* residual_out, int64_t ro_stride, const void* weight, int w_dtype, int64_t M, int64_t K,
                 float eps, void* out, int out_dtype, float* out_scales, awq_stream_t stream) {
  return awq_rms_norm_on(kAsk, X, x_dtype, x_stride, residual, r_dtype, r_stride, residual_out, ro_stride, weight, w_dtype, M, K, eps, out, out_dtype, out_scales, stream);
}

int awq_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double original_len, double low,
                         double high, double* out_freqs, double* out_magnitude) {
  decode_error(AWQ_OK, "");
  if (!out_freqs) return decode_error(AWQ_ERR_INVALID_ARG, "a required pointer is NULL");
  if (rotary_dim < 2 || rotary_dim % 2) return decode_error(AWQ_ERR_SHAPE, "rotary_dim must be even and positive");
  if (!(base > 1.0) || std::isinf(base)) return decode_error(AWQ_ERR_INVALID_ARG, "base must be above 1");
  if (scaling < AWQ_ROPE_PLAIN || scaling > AWQ_ROPE_RAMP) return decode_error(AWQ_ERR_INVALID_ARG, "unknown scaling");
  if (scaling != AWQ_ROPE_PLAIN && (!(factor >= 1.0) || std::isinf(factor)))
    return decode_error(AWQ_ERR_INVALID_ARG, "factor must be at least 1");
  const bool banded = scaling == AWQ_ROPE_BANDS || scaling == AWQ_ROPE_RAMP;
  if (banded && (!(original_len >= 1.0) || std::isinf(original_len) || !(low > 0.0) || !(high > low) || std::isinf(high)))
    return decode_error(AWQ_ERR_INVALID_ARG, "original_len must be positive and 0 < low < high");
  if (scaling == AWQ_ROPE_BASE && rotary_dim < 4) return decode_error(AWQ_ERR_SHAPE, "scaling the base needs rotary_dim >= 4");
  const double two_pi = 6.283185307179586476925, R = rotary_dim;
  const double b = scaling == AWQ_ROPE_BASE ? base * std::pow(factor, R / (R - 2.0)) : base;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(b, -2.0 * i / R);
    double kept = 1.0;  // the share of f that stays, against f / factor
    if (scaling == AWQ_ROPE_LINEAR) {
      kept = 0.0;
    } else if (scaling == AWQ_ROPE_BANDS) {
      const double turns = original_len * f / two_pi;  // of this pair over the original length
      kept = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
    } else if (scaling == AWQ_ROPE_RAMP) {
      // the pair index at which a pair turns `high` (the first, kept) and `low` times
      const double first = std::fmax(0.0, std::floor(R * std::log(original_len / (high * two_pi)) / (2.0 * std::log(base))));
      const double end = std::fmin(R - 1.0, std::ceil(R * std::log(original_len / (low * two_pi)) / (2.0 * std::log(base))));
      kept = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - first) / std::fmax(end - first, 1e-3)));
    }
    out_freqs[i] = scaling == AWQ_ROPE_PLAIN || scaling == AWQ_ROPE_BASE ? f : f * kept + f / factor * (1.0 - kept);
  }
  if (out_magnitude) *out_magnitude = scaling == AWQ_ROPE_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return AWQ_OK;
}

int awq_kv_append_on(int device, const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
                  int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride, int in_dtype,
                  int64_t T, int Hq, void* q_out, int q_dtype, const int32_t* positions, const int32_t* seqs,
                  const double* freqs, int rotary_dim, int interleaved, float magnitude, const awq_paged_cache* cache,
                  int32_t* status, awq_stream_t stream) {
  decode_error(AWQ_OK, "");
  AppendArgs a;
  int st = take_cache(cache, &a.c);
  if (st != AWQ_OK) return st;
  if (T < 0 || T > kIntMax || Hq < 0 || Hq > 65535) return decode_error(AWQ_ERR_SHAPE, "T or Hq out of range");
  if (T == 0) return AWQ_OK;
  if (!k || !v || !positions || (Hq > 0 && (!q || !q_out))) return decode_error(AWQ_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!is_float(in_dtype)) return decode_error(AWQ_ERR_INVALID_ARG, "q, k and v hold AWQ_DTYPE_F32, AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  if (Hq > 0 && q_dtype != kTypeF16 && q_dtype != kTypeBf16)
    return decode_error(AWQ_ERR_INVALID_ARG, "q_dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  if (rotary_dim < 0 || rotary_dim > a.c.head_dim || rotary_dim % 16)
    return decode_error(AWQ_ERR_SHAPE, "rotary_dim must be a multiple of 16 of at most head_dim");
  if (rotary_dim > 0 && !freqs) return decode_error(AWQ_ERR_INVALID_ARG, "rotary_dim > 0 needs freqs");
  if (!std::isfinite(magnitude)) return decode_error(AWQ_ERR_INVALID_ARG, "magnitude must be finite");
  if (!seqs && T > a.c.seqs) return decode_error(AWQ_ERR_SHAPE, "more tokens than sequences, and seqs is NULL");
  const int64_t per16 = 16 / type_bytes(in_dtype);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || q_token_stride % per16 ||
      q_head_stride % per16 || k_token_stride % per16 || k_head_stride % per16 || v_token_stride % per16 ||
      v_head_stride % per16)
    return decode_error(AWQ_ERR_INVALID_ARG, "rows of q, k, v and q_out must be 16-byte aligned");
  if (q_token_stride < 0 || q_head_stride < 0 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 ||
      v_head_stride < 0)
    return decode_error(AWQ_ERR_INVALID_ARG, "strides must not be negative");
  if (std::max(q_head_stride, std::max(k_head_stride, v_head_stride)) > kIntMax / 4)
    return decode_error(AWQ_ERR_SHAPE, "the head strides of q, k and v must be below 2^29");
  if (!rows_apart(a.c)) return decode_error(AWQ_ERR_INVALID_ARG, "rows of a cache that is written must not overlap");
  if (!aligned(positions, 4) || !aligned(seqs, 4) || !aligned(freqs, 8) || !aligned(status, 4))
    return decode_error(AWQ_ERR_INVALID_ARG, "positions, seqs, freqs or status is misaligned");
  if (Hq > 0 && device == kAsk) {  // every unit of q is read and written by one thread, so that q_out may be q
    const int64_t D = a.c.head_dim, b = type_bytes(in_dtype);
    const Extent to = extent(q_out, T, Hq * D * 2, Hq, D * 2, D * 2);
    const bool same = q_out == q && in_dtype == q_dtype && (T == 1 || q_token_stride == Hq * D) && (Hq == 1 || q_head_stride == D);
    if ((!same && meet(to, extent(q, T, q_token_stride * b, Hq, q_head_stride * b, D * b))) ||
        meet(to, extent(k, T, k_token_stride * b, a.c.heads, k_head_stride * b, D * b)) ||
        meet(to, extent(v, T, v_token_stride * b, a.c.heads, v_head_stride * b, D * b)) || meet(to, extent(a.c, a.c.k)) ||
        meet(to, extent(a.c, a.c.v)))
      return decode_error(AWQ_ERR_INVALID_ARG, "q_out may be q itself but overlap nothing else");
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DeviceRestore restore_device;
  const void* ptrs[] = {k, v, positions, a.c.k, a.c.v, a.c.table, Hq > 0 ? q : nullptr, Hq > 0 ? q_out : nullptr, seqs,
                        rotary_dim > 0 ? freqs : nullptr, a.c.k_scale, a.c.v_scale};
  int num_sms = 0;
  if ((st = take_device(device, k, ptrs, 12, status, &num_sms)) != AWQ_OK) return st;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_st = q_token_stride;
  a.k_st = k_token_stride;
  a.v_st = v_token_stride;
  a.q_head = static_cast<uint32_t>(q_head_stride * type_bytes(in_dtype));
  a.k_head = static_cast<uint32_t>(k_head_stride * type_bytes(in_dtype));
  a.v_head = static_cast<uint32_t>(v_head_stride * type_bytes(in_dtype));
  a.cache_head32 = static_cast<uint32_t>(a.c.head_stride * type_bytes(a.c.type) / 32);
  a.T = T;
  a.Hq = Hq;
  a.in_type = in_dtype;
  a.q_type = q_dtype;
  a.rot = rotary_dim;
  a.interleaved = interleaved != 0;
  a.freqs = freqs;
  a.magnitude = magnitude;
  a.positions = positions;
  a.seq = seqs;
  a.q_out = q_out;
  a.status = status;
  int launches = 0;
  const cudaError_t e = launch_kv_append(a, num_sms, s, &launches);
  if (e != cudaSuccess) return decode_cuda_error(e, "append to the cache");
  record_launch_count(launches);
  return AWQ_OK;
}
int awq_kv_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
                  int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride, int in_dtype,
                  int64_t T, int Hq, void* q_out, int q_dtype, const int32_t* positions, const int32_t* seqs,
                  const double* freqs, int rotary_dim, int interleaved, float magnitude, const awq_paged_cache* cache,
                  int32_t* status, awq_stream_t stream) {
  return awq_kv_append_on(kAsk, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, in_dtype, T, Hq, q_out, q_dtype, positions, seqs, freqs, rotary_dim, interleaved, magnitude, cache, status, stream);
}

int64_t awq_paged_attention_workspace(int Hq, int Hkv, int head_dim, int cache_dtype) {
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (cache_dtype != kTypeBf16 && cache_dtype != kTypeF16 && cache_dtype != kTypeE4m3))
    return 0;
  return paged_attn_workspace(Hq, Hkv, head_dim, cache_dtype);
}

int awq_paged_attention_on(int device, const void* q, int64_t q_seq_stride, int64_t q_head_stride, int q_dtype, int Hq,
                        const awq_paged_cache* cache, const int32_t* lengths, float scale, void* out, void* workspace,
                        int64_t workspace_bytes, int32_t* status, awq_stream_t stream) {
  decode_error(AWQ_OK, "");
  PagedAttnArgs a;
  int st = take_cache(cache, &a.c);
  if (st != AWQ_OK) return st;
  if (!q || !lengths || !out || !workspace) return decode_error(AWQ_ERR_INVALID_ARG, "a required pointer is NULL");
  if (q_dtype != kTypeF16 && q_dtype != kTypeBf16)
    return decode_error(AWQ_ERR_INVALID_ARG, "q_dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  if (a.c.type != kTypeE4m3 && a.c.type != q_dtype)
    return decode_error(AWQ_ERR_INVALID_ARG, "a 16-bit cache and its queries share a type");
  if (Hq < 1 || Hq > 65535 || Hq % a.c.heads) return decode_error(AWQ_ERR_SHAPE, "the key-value heads must divide the query heads");
  if (a.c.seqs * Hq > kIntMax) return decode_error(AWQ_ERR_SHAPE, "sequences times query heads must be below 2^31");
  if (!std::isfinite(scale)) return decode_error(AWQ_ERR_INVALID_ARG, "scale must be finite");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || q_seq_stride % 8 || q_head_stride % 8)
    return decode_error(AWQ_ERR_INVALID_ARG, "q, out and the work space must be 16-byte aligned");
  if (q_seq_stride < 0 || q_head_stride < 0) return decode_error(AWQ_ERR_INVALID_ARG, "strides must not be negative");
  if (!aligned(lengths, 4) || !aligned(status, 4)) return decode_error(AWQ_ERR_INVALID_ARG, "lengths or status is misaligned");
  const int64_t used = awq_paged_attention_workspace(Hq, a.c.heads, a.c.head_dim, a.c.type);  // of the work space, which may be larger
  if (workspace_bytes < used)
    return decode_error(AWQ_ERR_INVALID_ARG, "the work space is smaller than awq_paged_attention_workspace says");
  if (device == kAsk) {  // a segment's queries are read before any of its outputs are written, so that out may be q
    const int64_t B = a.c.seqs, D = a.c.head_dim;
    const Extent to = extent(out, B, Hq * D * 2, Hq, D * 2, D * 2), from = extent(q, B, q_seq_stride * 2, Hq, q_head_stride * 2, D * 2),
                 ws = extent(workspace, 1, 0, 1, 0, used), ck = extent(a.c, a.c.k), cv = extent(a.c, a.c.v);
    const bool same = out == q && (B == 1 || q_seq_stride == Hq * D) && (Hq == 1 || q_head_stride == D);
    if ((!same && meet(to, from)) || meet(to, ws) || meet(to, ck) || meet(to, cv) || meet(ws, from) || meet(ws, ck) || meet(ws, cv))
      return decode_error(AWQ_ERR_INVALID_ARG, "out may be q itself; it and the work space overlap nothing else");
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DeviceRestore restore_device;
  const void* ptrs[] = {q, a.c.k, a.c.v, a.c.table, lengths, out, workspace, a.c.k_scale, a.c.v_scale};
  int num_sms = 0;
  if ((st = take_device(device, q, ptrs, 9, status, &num_sms)) != AWQ_OK) return st;
  a.q = q;
  a.q_sb = q_seq_stride;
  a.q_sh = q_head_stride;
  a.B = a.c.seqs;
  a.Hq = Hq;
  a.q_type = q_dtype;
  a.lengths = lengths;
  a.scale = scale;
  a.out = out;
  a.workspace = workspace;
  a.status = status;
  int launches = 0;
  const cudaError_t e = launch_paged_attn(a, num_sms, s, &launches);
  if (e != cudaSuccess) return decode_cuda_error(e, "paged attention");
  record_launch_count(launches);
  return AWQ_OK;
}
int awq_paged_attention(const void* q, int64_t q_seq_stride, int64_t q_head_stride, int q_dtype, int Hq,
                        const awq_paged_cache* cache, const int32_t* lengths, float scale, void* out, void* workspace,
                        int64_t workspace_bytes, int32_t* status, awq_stream_t stream) {
  return awq_paged_attention_on(kAsk, q, q_seq_stride, q_head_stride, q_dtype, Hq, cache, lengths, scale, out, workspace, workspace_bytes, status, stream);
}

}  // extern "C"
