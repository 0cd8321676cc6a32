// decode_binding.cpp — CPython binding of the decode-step operators (module _decode).
//
// They run between every two products of every layer of every decode step, where the ctypes
// marshalling of their 20 to 40 arguments took longer (9 to 14 us a call) than the kernels; here a
// call takes what its checks, the output's allocation and the launch take. Arguments are marshalled
// and checked only: all device work is in libawqsearch.so. Each function works on the current
// stream and returns the output tensors, or the library's status as an int when that is not OK. Once
// its Python arguments are taken it runs without the interpreter lock, as ctypes does: an allocation
// or a launch may wait for the device.
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/grad_mode.h>
#include <torch/csrc/autograd/python_variable.h>

#include "decode_entry.h"

namespace {

using at::Tensor;

struct Refusal {  // becomes a Python exception
  PyObject* type;
  const char* text;
};
void value_check(bool ok, const char* text) {
  if (!ok) throw Refusal{PyExc_ValueError, text};
}
void type_check(bool ok, const char* text) {
  if (!ok) throw Refusal{PyExc_TypeError, text};
}

// The AWQ_DTYPE_* code, -1 for other types.
int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return AWQ_DTYPE_BF16;
    case at::kFloat: return AWQ_DTYPE_F32;
    case at::kHalf: return AWQ_DTYPE_F16;
    case at::kFloat8_e4m3fn: return AWQ_DTYPE_E4M3;
    default: return -1;
  }
}
bool plain_float(int code) { return code >= AWQ_DTYPE_BF16 && code <= AWQ_DTYPE_F16; }
bool half_float(int code) { return code == AWQ_DTYPE_BF16 || code == AWQ_DTYPE_F16; }

at::ScalarType dtype_of(PyObject* o) {
  type_check(THPDtype_Check(o), "a dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

const Tensor& tensor(PyObject* o, const char* what) {
  type_check(THPVariable_Check(o), what);
  return THPVariable_Unpack(o);
}
// An optional tensor: undefined for None.
Tensor maybe(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }

// The tensor lies on `device` and carries no gradient, of backward or of forward mode.
void on_device(const Tensor& t, const at::Device& device) {
  if (!t.defined()) return;
  value_check(t.device() == device, "every tensor must be on the device of the first");
  if (t.unsafeGetTensorImpl()->autograd_meta() == nullptr) return;  // as most
  value_check(!(t.requires_grad() && at::GradMode::is_enabled()),
              "the decode-step operators have no backward pass: call them under torch.no_grad()");
  value_check(!(c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined()),
              "the decode-step operators have no forward-mode derivative: pass tensors without tangents");
}

// Tells autograd that `t` has been written, so that a backward pass that saved it is an error.
void written(const Tensor& t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType t, const at::Device& device) {
  return at::detail::empty_cuda(sizes, t, device, std::nullopt);
}

awq_stream_t current_stream(const at::Device& device) {
  return reinterpret_cast<awq_stream_t>(at::cuda::getCurrentCUDAStream(device.index()).stream());
}

bool is_vector(const Tensor& t, at::ScalarType type, int64_t n) {
  return t.dim() == 1 && t.size(0) == n && t.scalar_type() == type && (n <= 1 || t.stride(0) == 1);
}

int32_t* status_word(const Tensor& t, const at::Device& device) {
  if (!t.defined()) return nullptr;
  value_check(t.scalar_type() == at::kInt && t.numel() == 1 && (t.device() == device || (t.device().is_cpu() && t.is_pinned())),
              "status must be one int32 on the device or in pinned host memory");
  return t.data_ptr<int32_t>();
}

// (rows, heads, head_dim) with 16-byte aligned contiguous rows: as it is, or a copy.
Tensor rows16(const Tensor& t, int64_t heads, int64_t head_dim, const char* text) {
  value_check(t.dim() == 3 && (heads < 0 || t.size(1) == heads) && t.size(2) == head_dim, text);
  const int64_t per = 16 / t.element_size();
  if (t.stride(2) == 1 && t.stride(0) % per == 0 && t.stride(1) % per == 0 &&
      reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0)
    return t;
  return t.clone(at::MemoryFormat::Contiguous);
}

// The caches (num_pages, page_size, heads, head_dim), in any memory order with contiguous rows, and
// the block table (sequences, max_pages).
awq_paged_cache cache_of(const Tensor& k, const Tensor& v, const Tensor& table, const Tensor& k_scale, const Tensor& v_scale) {
  value_check(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
              "k_cache and v_cache must be (num_pages, page_size, heads, head_dim) of one dtype");
  value_check(k.stride(3) == 1 && v.strides() == k.strides(), "k_cache and v_cache must have contiguous rows and the same strides");
  awq_paged_cache c;
  c.dtype = dtype_code(k.scalar_type());
  type_check(c.dtype >= 0 && c.dtype != AWQ_DTYPE_F32, "the cache must be float16, bfloat16 or float8_e4m3fn");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.num_pages = k.size(0);
  c.page_size = k.size(1);
  c.heads = k.size(2);
  c.head_dim = k.size(3);
  c.page_stride = k.stride(0);
  c.slot_stride = k.stride(1);
  c.head_stride = k.stride(2);
  c.k_scale = c.v_scale = nullptr;
  if (c.dtype == AWQ_DTYPE_E4M3) {
    value_check(k_scale.defined() && v_scale.defined() && is_vector(k_scale, at::kFloat, c.heads) &&
                    is_vector(v_scale, at::kFloat, c.heads),
                "an e4m3 cache needs k_scale and v_scale, (heads,) contiguous float32");
    c.k_scale = k_scale.data_ptr<float>();
    c.v_scale = v_scale.data_ptr<float>();
  } else {
    value_check(!k_scale.defined() && !v_scale.defined(), "k_scale and v_scale belong to an e4m3 cache");
  }
  value_check(table.scalar_type() == at::kInt && table.dim() == 2 && (table.size(1) <= 1 || table.stride(1) == 1),
              "block_table must be (sequences, max_pages) int32 with contiguous rows");
  c.block_table = table.data_ptr<int32_t>();
  c.n_seqs = table.size(0);
  c.max_pages = table.size(1);
  c.table_stride = table.stride(0);
  return c;
}

// Gives the interpreter lock up while it lives.
class Unlocked {
 public:
  Unlocked() : thread_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(thread_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* thread_;
};

PyObject* result(int status, const Tensor& out) {
  return status == AWQ_OK ? THPVariable_Wrap(out) : PyLong_FromLong(status);
}

// Runs `body`, with its refusals and C++ exceptions as Python's.
template <typename Body>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Body body) {
  HANDLE_TH_ERRORS
  try {
    type_check(given == wanted, "wrong number of arguments");
    return body();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// rms_norm(X, weight, eps, residual, residual_out, out_dtype)
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Tensor X = tensor(args[0], "X must be a tensor"), weight = tensor(args[1], "weight must be a tensor");
    Tensor residual = maybe(args[3], "residual must be a tensor"), into = maybe(args[4], "residual_out must be a tensor");
    const at::ScalarType out_type = dtype_of(args[5]);
    const double eps = PyFloat_AsDouble(args[2]);
    if (PyErr_Occurred()) return nullptr;
    Tensor out, scales;
    const int st = [&] {
      Unlocked unlocked;
      value_check(X.is_cuda(), "rms_norm() takes CUDA tensors");
      const at::Device device = X.device();
      value_check(X.dim() == 2 && weight.dim() == 1 && weight.size(0) == X.size(1), "X must be (M, K) and weight (K,)");
      const int xc = dtype_code(X.scalar_type()), wc = dtype_code(weight.scalar_type()), oc = dtype_code(out_type);
      type_check(plain_float(xc) && plain_float(wc), "X and weight must be float32, float16 or bfloat16");
      type_check(oc >= 0, "out_dtype must be float32, float16, bfloat16 or float8_e4m3fn");
      for (const Tensor* t : std::initializer_list<const Tensor*>{&X, &weight, &residual, &into}) on_device(*t, device);
      const int64_t M = X.size(0), K = X.size(1);
      if (X.stride(1) != 1) X = X.contiguous();
      weight = weight.contiguous();
      int rc = 0;
      int64_t r_stride = K, ro_stride = K;
      if (residual.defined()) {
        if (!into.defined()) into = residual;
        rc = dtype_code(residual.scalar_type());
        value_check(residual.sizes() == X.sizes() && plain_float(rc), "residual must be (M, K) in float32, float16 or bfloat16");
        value_check(into.sizes() == X.sizes() && into.scalar_type() == residual.scalar_type() && (K <= 1 || into.stride(1) == 1),
                    "residual_out must be (M, K) of the residual's dtype with contiguous rows");
        if (residual.stride(1) != 1) residual = residual.contiguous();
        if (M > 1) {
          r_stride = residual.stride(0);
          ro_stride = into.stride(0);
        }
      } else {
        value_check(!into.defined(), "residual_out comes with a residual");
      }
      out = empty({M, K}, out_type, device);
      if (oc == AWQ_DTYPE_E4M3) scales = empty({M}, at::kFloat, device);
      return awq_rms_norm_on(device.index(), X.data_ptr(), xc, X.stride(0), residual.defined() ? residual.data_ptr() : nullptr, rc,
                             r_stride, into.defined() ? into.data_ptr() : nullptr, ro_stride, weight.data_ptr(), wc, M, K,
                             static_cast<float>(eps), out.data_ptr(), oc, scales.defined() ? scales.data_ptr<float>() : nullptr,
                             current_stream(device));
    }();
    if (st == AWQ_OK) written(into);
    if (st != AWQ_OK || !scales.defined()) return result(st, out);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(scales));
  });
}

// kv_append(q, k, v, k_cache, v_cache, block_table, positions, freqs, seqs, interleaved, magnitude,
//           k_scale, v_scale, q_dtype, status)
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    Tensor q = maybe(args[0], "q must be a tensor"), k = tensor(args[1], "k must be a tensor"), v = tensor(args[2], "v must be a tensor");
    const Tensor &k_cache = tensor(args[3], "k_cache must be a tensor"), &v_cache = tensor(args[4], "v_cache must be a tensor");
    const Tensor &table = tensor(args[5], "block_table must be a tensor"), &positions = tensor(args[6], "positions must be a tensor");
    const Tensor freqs = maybe(args[7], "freqs must be a tensor"), seqs = maybe(args[8], "seqs must be a tensor");
    const Tensor k_scale = maybe(args[11], "k_scale must be a tensor"), v_scale = maybe(args[12], "v_scale must be a tensor");
    const Tensor status = maybe(args[14], "status must be a tensor");
    const int interleaved = PyObject_IsTrue(args[9]);
    const double magnitude = PyFloat_AsDouble(args[10]);
    if (PyErr_Occurred()) return nullptr;
    const bool asked = args[13] != Py_None;
    const at::ScalarType asked_type = asked ? dtype_of(args[13]) : at::kHalf;
    Tensor out;
    const int st = [&] {
      Unlocked unlocked;
      value_check(k.is_cuda(), "kv_append() takes CUDA tensors");
      const at::Device device = k.device();
      for (const Tensor* t : std::initializer_list<const Tensor*>{&q, &k, &v, &k_cache, &v_cache, &table, &positions, &freqs, &seqs, &k_scale, &v_scale}) on_device(*t, device);
      const awq_paged_cache cache = cache_of(k_cache, v_cache, table, k_scale, v_scale);
      k = rows16(k, cache.heads, cache.head_dim, "k must be (tokens, heads, head_dim) of the cache's heads");
      v = rows16(v, cache.heads, cache.head_dim, "v must be (tokens, heads, head_dim) of the cache's heads");
      const int64_t T = k.size(0);
      const int in = dtype_code(k.scalar_type());
      const char* same = "q, k and v must share T and a dtype of float32, float16 or bfloat16";
      value_check(v.size(0) == T && v.scalar_type() == k.scalar_type() && plain_float(in), same);
      const at::ScalarType q_type = asked ? asked_type : (cache.dtype == AWQ_DTYPE_E4M3 ? at::kHalf : k_cache.scalar_type());
      type_check(half_float(dtype_code(q_type)), "q_dtype must be float16 or bfloat16");
      int64_t Hq = 0;
      if (q.defined()) {
        q = rows16(q, -1, cache.head_dim, "q must be (T, Hq, head_dim)");
        Hq = q.size(1);
        value_check(q.size(0) == T && q.scalar_type() == k.scalar_type(), same);
        out = empty({T, Hq, cache.head_dim}, q_type, device);
      }
      value_check(is_vector(positions, at::kInt, T) && (!seqs.defined() || is_vector(seqs, at::kInt, T)),
                  "positions and seqs must be (T,) contiguous int32");
      if (freqs.defined())
        value_check(freqs.dim() == 1 && is_vector(freqs, at::kDouble, freqs.size(0)),
                    "freqs must be a contiguous float64 vector (rope_frequencies)");
      const int64_t rot = freqs.defined() ? 2 * freqs.size(0) : 0;
      value_check(rot <= cache.head_dim, "freqs must have at most head_dim / 2 entries");
      if (T == 0) return static_cast<int>(AWQ_OK);  // whose table may be empty too
      return awq_kv_append_on(
          device.index(), Hq ? q.data_ptr() : nullptr, Hq ? q.stride(0) : 0, Hq ? q.stride(1) : 0, k.data_ptr(), k.stride(0), k.stride(1),
          v.data_ptr(), v.stride(0), v.stride(1), in, T, static_cast<int>(Hq), Hq ? out.data_ptr() : nullptr, dtype_code(q_type),
          positions.data_ptr<int32_t>(), seqs.defined() ? seqs.data_ptr<int32_t>() : nullptr,
          rot ? freqs.data_ptr<double>() : nullptr, static_cast<int>(rot), interleaved, static_cast<float>(magnitude), &cache,
          status_word(status, device), current_stream(device));
    }();
    if (st != AWQ_OK) return PyLong_FromLong(st);
    written(k_cache);
    written(v_cache);
    if (!out.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(out);
  });
}

// paged_attention(q, k_cache, v_cache, block_table, lengths, scale or None, k_scale, v_scale, status)
PyObject* paged_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Tensor q = tensor(args[0], "q must be a tensor");
    const Tensor &k_cache = tensor(args[1], "k_cache must be a tensor"), &v_cache = tensor(args[2], "v_cache must be a tensor");
    const Tensor &table = tensor(args[3], "block_table must be a tensor"), &lengths = tensor(args[4], "lengths must be a tensor");
    const Tensor k_scale = maybe(args[6], "k_scale must be a tensor"), v_scale = maybe(args[7], "v_scale must be a tensor");
    const Tensor status = maybe(args[8], "status must be a tensor");
    const bool asked = args[5] != Py_None;
    const double asked_scale = asked ? PyFloat_AsDouble(args[5]) : 0.0;
    if (PyErr_Occurred()) return nullptr;
    Tensor out;
    const int st = [&]() -> int {
      Unlocked unlocked;
      value_check(q.is_cuda(), "paged_attention() takes CUDA tensors");
      const at::Device device = q.device();
      for (const Tensor* t : std::initializer_list<const Tensor*>{&q, &k_cache, &v_cache, &table, &lengths, &k_scale, &v_scale}) on_device(*t, device);
      const int qc = dtype_code(q.scalar_type());
      value_check(q.dim() == 3 && half_float(qc), "q must be (sequences, Hq, head_dim) float16 or bfloat16");
      const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
      const double scale = asked ? asked_scale : 1.0 / std::sqrt(static_cast<double>(std::max<int64_t>(D, 1)));
      out = empty({B, Hq, D}, q.scalar_type(), device);
      if (B == 0) return AWQ_OK;
      const awq_paged_cache cache = cache_of(k_cache, v_cache, table, k_scale, v_scale);
      value_check(cache.n_seqs == B, "block_table needs one row per sequence");
      value_check(D == cache.head_dim && cache.heads > 0 && Hq % cache.heads == 0,
                  "q's head_dim must be the cache's, and the cache's heads must divide q's");
      type_check(cache.dtype == qc || cache.dtype == AWQ_DTYPE_E4M3, "a 16-bit cache and its queries share a dtype");
      value_check(is_vector(lengths, at::kInt, B), "lengths must be (sequences,) contiguous int32");
      q = rows16(q, Hq, D, "q must be (sequences, Hq, head_dim)");
      const int64_t bytes = awq_paged_attention_workspace(static_cast<int>(Hq), static_cast<int>(cache.heads), static_cast<int>(D),
                                                          static_cast<int>(cache.dtype));
      const Tensor workspace = empty({bytes}, at::kByte, device);
      return awq_paged_attention_on(device.index(), q.data_ptr(), q.stride(0), q.stride(1), qc, static_cast<int>(Hq), &cache,
                                    lengths.data_ptr<int32_t>(), static_cast<float>(scale), out.data_ptr(), workspace.data_ptr(),
                                    bytes, status_word(status, device), current_stream(device));
    }();
    return result(st, out);
  });
}

PyMethodDef kMethods[] = {
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rms_norm)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_decode", "Binding of the decode-step operators of libawqsearch.so.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode(void) { return PyModule_Create(&kModule); }
