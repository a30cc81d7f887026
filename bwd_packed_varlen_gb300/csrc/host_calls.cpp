// Host side of the rotary and shared-prefix calls, as a Python extension module.
//
// A decoding step's kernels take 6 to 20 microseconds, and checking the arguments, allocating
// the outputs and marshalling thirty values from Python took 15 to 30 of them before each.
// Here one call does that next to the tensors, and the GPU is what bounds it: rotary positions
// of a step 16 -> 6 us a call, attention of a small step 29 -> 16 us, forward and backward of a
// small batch 77 -> 55 us. The entry points of the C library come in as addresses, so that this
// module serves both its builds.
//
// Returns the outputs, or the library's code if it is not 0. Refusals raise ValueError before
// anything is launched. Outputs that the caller gives are checked and returned as they are. A
// stream other than the current one is made current for the call, so that what is allocated
// here belongs to it.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cstdint>
#include <optional>

#include "te_attn.h"

namespace {

struct Refusal {  // becomes a ValueError
  const char* what;
};

void need(bool ok, const char* what) {
  if (!ok) throw Refusal{what};
}

constexpr const char* kOneDevice = "all tensors must be CUDA tensors on one device (there is no CPU path)";

const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o), "a tensor argument is not a torch tensor");
  return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

int dtype_code(const at::Tensor& t) {
  return t.scalar_type() == at::kHalf ? TE_DTYPE_FP16 : t.scalar_type() == at::kBFloat16 ? TE_DTYPE_BF16 : -1;
}

bool on_device(const at::Tensor& t, c10::DeviceIndex index) { return t.is_cuda() && t.device().index() == index; }

int as_int(int64_t n) {
  need(n <= INT_MAX, "a dimension is 2^31 or more");
  return static_cast<int>(n);
}

// Address of an int32 vector of n values on the device.
const int32_t* lengths(PyObject* o, int64_t n, c10::DeviceIndex index) {
  const at::Tensor& t = tensor(o);
  need(t.scalar_type() == at::kInt && t.dim() == 1 && t.numel() == n && on_device(t, index) && t.is_contiguous(),
       "cu_seqlens, start_positions and prefix_len must be contiguous int32 vectors on q's device, of batch + 1, batch "
       "and one value");
  return t.const_data_ptr<int32_t>();
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

void* address(PyObject* o) {
  void* v = PyLong_AsVoidPtr(o);
  if (!v && PyErr_Occurred()) throw python_error();
  return v;
}

// Makes the device and the caller's stream (None: the device's current one) current.
class Place {
 public:
  Place(c10::DeviceIndex index, PyObject* stream) : device_(index) {
    const auto current = c10::cuda::getCurrentCUDAStream(index);
    stream_ = current.stream();
    if (!given(stream)) return;
    const auto other = static_cast<cudaStream_t>(address(stream));
    if (other == stream_) return;
    guard_.emplace(c10::cuda::getStreamFromExternal(other, index));
    stream_ = other;
  }
  cudaStream_t stream() const { return stream_; }

 private:
  c10::cuda::CUDAGuard device_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
  cudaStream_t stream_;
};

// An output: the caller's after a check, or a new contiguous tensor.
class Output {
 public:
  Output(PyObject* o, c10::IntArrayRef shape, const at::Tensor& like, at::ScalarType type, const char* what) {
    if (given(o)) {
      const at::Tensor& t = tensor(o);
      need(t.sizes() == shape && t.scalar_type() == type && t.device() == like.device() && t.is_contiguous(), what);
      object_ = o;
      at_ = t.mutable_data_ptr();
    } else {
      fresh_ = at::empty(shape, like.options().dtype(type).requires_grad(false).memory_format(std::nullopt));
      at_ = fresh_.mutable_data_ptr();
    }
  }
  void* at() const { return at_; }
  PyObject* result() const {  // a new reference
    if (object_) return Py_NewRef(object_);
    return THPVariable_Wrap(fresh_);
  }

 private:
  PyObject* object_ = nullptr;
  at::Tensor fresh_;
  void* at_ = nullptr;
};

class Workspace {
 public:
  Workspace(PyObject* o, size_t size, const at::Tensor& like) {
    if (given(o)) {
      const at::Tensor& t = tensor(o);
      need(t.device() == like.device() && t.is_contiguous(), "workspace must be contiguous, on q's device");
      at_ = t.mutable_data_ptr();
      bytes_ = static_cast<size_t>(t.nbytes());
    } else {
      bytes_ = size > 0 ? size : 1;
      fresh_ = at::empty({static_cast<int64_t>(bytes_)}, like.options().dtype(at::kByte).requires_grad(false));
      at_ = fresh_.mutable_data_ptr();
    }
  }
  void* at() const { return at_; }
  size_t bytes() const { return bytes_; }

 private:
  at::Tensor fresh_;
  void* at_ = nullptr;
  size_t bytes_ = 0;
};

PyObject* pack(std::initializer_list<const Output*> outputs, bool last_none = false) {
  PyObject* result = PyTuple_New(static_cast<Py_ssize_t>(outputs.size() + (last_none ? 1 : 0)));
  if (!result) throw python_error();
  Py_ssize_t i = 0;
  for (const Output* o : outputs) PyTuple_SET_ITEM(result, i++, o->result());
  if (last_none) PyTuple_SET_ITEM(result, i, Py_NewRef(Py_None));
  return result;
}

// What forward and backward over a shared prefix have in common.
struct Prefix {
  const at::Tensor &q, &k, &v, &kp, &vp;
  c10::DeviceIndex index;
  int code, batch, tq, tk, rows, hq, hkv, d;
  const int32_t* cu[4];
  const int32_t* prefix_len;

  // tensors: q, k, v, k_prefix, v_prefix; lens: the four cu_seqlens, prefix_len
  Prefix(PyObject* const* tensors, PyObject* const* lens)
      : q(tensor(tensors[0])), k(tensor(tensors[1])), v(tensor(tensors[2])), kp(tensor(tensors[3])), vp(tensor(tensors[4])) {
    need(q.is_cuda(), kOneDevice);
    index = q.device().index();
    need(on_device(k, index) && on_device(v, index) && on_device(kp, index) && on_device(vp, index), kOneDevice);
    need(q.is_contiguous() && k.is_contiguous() && v.is_contiguous() && kp.is_contiguous() && vp.is_contiguous(),
         "all tensors must be contiguous");
    code = dtype_code(q);
    const auto type = q.scalar_type();
    need(code >= 0 && k.scalar_type() == type && v.scalar_type() == type && kp.scalar_type() == type &&
             vp.scalar_type() == type,
         "q, k, v, k_prefix, v_prefix must share one dtype, float16 or bfloat16");
    need(q.dim() == 3 && k.dim() == 3 && kp.dim() == 3, "q, k, v, k_prefix, v_prefix must be [rows, heads, d]");
    need(v.sizes() == k.sizes() && vp.sizes() == kp.sizes() && kp.size(1) == k.size(1) && k.size(2) == q.size(2) &&
             kp.size(2) == q.size(2),
         "k, v and k_prefix, v_prefix must share heads and head dim, and d with q");
    tq = as_int(q.size(0));
    tk = as_int(k.size(0));
    rows = as_int(kp.size(0));
    hq = as_int(q.size(1));
    hkv = as_int(k.size(1));
    d = as_int(q.size(2));
    const int64_t n = tensor(lens[0]).numel();
    for (int i = 0; i < 4; ++i) cu[i] = lengths(lens[i], n, index);
    prefix_len = given(lens[4]) ? lengths(lens[4], 1, index) : nullptr;
    batch = as_int(n - 1);
  }
};

constexpr const char* kOutput = "an output must be contiguous, with the shape, dtype and device of its counterpart";
constexpr const char* kLse = "lse must be contiguous float32 [T_q, hq] on q's device";

using SizeFn = size_t (*)(int, int, int, int, int, int, int);

// (entry point, size function, q, k, v, k_prefix, v_prefix, four cu_seqlens, prefix_len, scale, mask, out, lse,
// workspace, stream)
PyObject* prefix_fwd(PyObject* const* a) {
  const auto fn = reinterpret_cast<decltype(&te_attn_prefix_fwd_thd)>(address(a[0]));
  const auto size = reinterpret_cast<SizeFn>(address(a[1]));
  const Prefix p(a + 2, a + 7);
  const float scale = static_cast<float>(number(a[12]));
  const int mask = static_cast<int>(integer(a[13]));
  const Place place(p.index, a[17]);
  const Output out(a[14], p.q.sizes(), p.q, p.q.scalar_type(), kOutput);
  const Output lse(a[15], p.q.sizes().slice(0, 2), p.q, at::kFloat, kLse);
  const Workspace ws(a[16], given(a[16]) ? 0 : size(p.batch, p.tq, p.tk, p.rows, p.hq, p.hkv, p.d), p.q);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fn(p.q.const_data_ptr(), p.k.const_data_ptr(), p.v.const_data_ptr(), p.kp.const_data_ptr(), p.vp.const_data_ptr(),
          out.at(), static_cast<float*>(lse.at()), p.cu[0], p.cu[1], p.cu[2], p.cu[3], p.prefix_len, p.batch, p.tq, p.tk,
          p.rows, p.hq, p.hkv, p.d, scale, mask, p.code, ws.at(), ws.bytes(), place.stream());
  Py_END_ALLOW_THREADS;
  return rc != 0 ? PyLong_FromLong(rc) : pack({&out, &lse});
}

// (entry point, size function, q, k, v, k_prefix, v_prefix, four cu_seqlens, prefix_len, scale, mask, out, dout, lse, dq,
// dk, dv, dk_prefix, dv_prefix, workspace, stream)
PyObject* prefix_bwd(PyObject* const* a) {
  const auto fn = reinterpret_cast<decltype(&te_attn_prefix_bwd_thd)>(address(a[0]));
  const auto size = reinterpret_cast<SizeFn>(address(a[1]));
  const Prefix p(a + 2, a + 7);
  const float scale = static_cast<float>(number(a[12]));
  const int mask = static_cast<int>(integer(a[13]));
  need(given(a[14]) && given(a[15]) && given(a[16]), "the backward needs out, dout and lse");
  const Place place(p.index, a[23]);
  const auto type = p.q.scalar_type();
  const Output out(a[14], p.q.sizes(), p.q, type, kOutput), dout(a[15], p.q.sizes(), p.q, type, kOutput);
  const Output lse(a[16], p.q.sizes().slice(0, 2), p.q, at::kFloat, kLse);
  const Output dq(a[17], p.q.sizes(), p.q, type, kOutput), dk(a[18], p.k.sizes(), p.q, type, kOutput);
  const Output dv(a[19], p.k.sizes(), p.q, type, kOutput), dkp(a[20], p.kp.sizes(), p.q, type, kOutput);
  const Output dvp(a[21], p.kp.sizes(), p.q, type, kOutput);
  const Workspace ws(a[22], given(a[22]) ? 0 : size(p.batch, p.tq, p.tk, p.rows, p.hq, p.hkv, p.d), p.q);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fn(p.q.const_data_ptr(), p.k.const_data_ptr(), p.v.const_data_ptr(), p.kp.const_data_ptr(), p.vp.const_data_ptr(),
          out.at(), dout.at(), static_cast<float*>(lse.at()), dq.at(), dk.at(), dv.at(), dkp.at(), dvp.at(), p.cu[0],
          p.cu[1], p.cu[2], p.cu[3], p.prefix_len, p.batch, p.tq, p.tk, p.rows, p.hq, p.hkv, p.d, scale, mask, p.code,
          ws.at(), ws.bytes(), place.stream());
  Py_END_ALLOW_THREADS;
  return rc != 0 ? PyLong_FromLong(rc) : pack({&dq, &dk, &dv, &dkp, &dvp});
}

// (entry point, q, k or None, inv_freq, cu_seqlens, padded ones or None for the sequence-major layout, start_positions
// or None, interleaved, mscale, inverse, q_out, k_out, stream)
PyObject* rope(PyObject* const* a) {
  const at::Tensor& q = tensor(a[1]);
  const bool with_k = given(a[2]), packed = given(a[5]);
  const at::Tensor& k = with_k ? tensor(a[2]) : q;
  const at::Tensor& w = tensor(a[3]);
  need(q.is_cuda(), kOneDevice);
  const auto index = q.device().index();
  need(on_device(w, index) && on_device(k, index), kOneDevice);
  const int code = dtype_code(q);
  need(code >= 0 && k.scalar_type() == q.scalar_type(), "q and k must share one dtype, float16 or bfloat16");
  const int64_t dims = packed ? 3 : 4;
  for (const at::Tensor* x : {&q, &k})
    need(x->dim() == dims && (x->numel() == 0 || x->stride(dims - 1) == 1),
         packed ? "q and k must have 3 dimensions and adjacent elements in a head"
                : "q and k must have 4 dimensions and adjacent elements in a head");
  need(w.scalar_type() == at::kDouble && w.dim() == 1 && w.is_contiguous(), "inv_freq must be a contiguous float64 vector");
  const int64_t n = tensor(a[4]).numel();
  need(n >= 2, "cu_seqlens must hold batch + 1 values");
  const int32_t* cu = lengths(a[4], n, index);
  const int32_t* start = given(a[6]) ? lengths(a[6], n - 1, index) : nullptr;
  need(k.size(0) == q.size(0) && k.size(dims - 1) == q.size(dims - 1) && (packed || k.size(1) == q.size(1)),
       "q and k must share tokens and head dim");
  need(with_k || !given(a[11]), "k_out without k");
  const int interleaved = PyObject_IsTrue(a[7]), inverse = PyObject_IsTrue(a[9]);
  if (interleaved < 0 || inverse < 0) throw python_error();
  const float mscale = static_cast<float>(number(a[8]));
  const int hq = as_int(q.size(dims - 2)), hkv = with_k ? as_int(k.size(dims - 2)) : 0, d = as_int(q.size(dims - 1));
  const int rows = as_int(q.size(0)), batch = as_int(n - 1), freqs = as_int(w.numel());
  const int32_t* pad = packed ? lengths(a[5], n, index) : nullptr;
  if (!packed) need(q.size(1) == n - 1, "cu_seqlens must hold batch + 1 values");
  // strides (an axis of one element has none: torch lets it be anything)
  auto stride = [](const at::Tensor& x, int64_t dim) { return x.size(dim) > 1 ? x.stride(dim) : 0; };
  auto token_stride = [&](const at::Tensor& x) {
    if (packed || batch == 1) return stride(x, 0);
    need(rows <= 1 || x.stride(0) == batch * x.stride(1), "rows i * batch + b must be evenly spaced");
    return stride(x, 1);
  };
  const int64_t qt = token_stride(q), qh = stride(q, dims - 2), kt = token_stride(k), kh = stride(k, dims - 2);
  const Place place(index, a[12]);
  const Output qo(a[10], q.sizes(), q, q.scalar_type(), "outputs must be contiguous, with the shape, dtype and device of their input");
  std::optional<Output> ko;
  if (with_k)
    ko.emplace(a[11], k.sizes(), k, k.scalar_type(), "outputs must be contiguous, with the shape, dtype and device of their input");
  const void* k_at = with_k ? k.const_data_ptr() : nullptr;
  void* ko_at = with_k ? ko->at() : nullptr;
  int rc;
  void* fn = address(a[0]);
  Py_BEGIN_ALLOW_THREADS;
  if (packed)
    rc = reinterpret_cast<decltype(&te_attn_rope_thd)>(fn)(
        q.const_data_ptr(), k_at, qo.at(), ko_at, w.const_data_ptr<double>(), freqs, cu, pad, start, batch, rows, hq, hkv, d,
        qt, qh, kt, kh, interleaved, mscale, inverse, code, place.stream());
  else
    rc = reinterpret_cast<decltype(&te_attn_rope_sbhd)>(fn)(
        q.const_data_ptr(), k_at, qo.at(), ko_at, w.const_data_ptr<double>(), freqs, cu, start, batch, rows, hq, hkv, d, qt,
        qh, kt, kh, interleaved, mscale, inverse, code, place.stream());
  Py_END_ALLOW_THREADS;
  if (rc != 0) return PyLong_FromLong(rc);
  return with_k ? pack({&qo, &*ko}) : pack({&qo}, true);
}

template <PyObject* (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", kArgs, n);
    return nullptr;
  }
  try {
    return kCall(args);
  } catch (const Refusal& r) {
    PyErr_SetString(PyExc_ValueError, r.what);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"prefix_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<prefix_fwd, 18>)), METH_FASTCALL, nullptr},
    {"prefix_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<prefix_bwd, 24>)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<rope, 13>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_teattn_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__teattn_host() { return PyModule_Create(&module); }
