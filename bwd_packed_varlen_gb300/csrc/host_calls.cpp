// Host side of the rotary, shared-prefix, paged and windowed calls, as a Python extension module.
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

constexpr const char* kCacheForm =
    "k_cache and v_cache must be [pages, hkv, page_size, d] of float16 or bfloat16, or pairs of uint8 codes "
    "[pages, hkv, page_size, d / 2] and steps and least values [pages, hkv, page_size, d / 32, 2], whole pages contiguous";

// A paged cache from (k_cache, v_cache, page_table): tensors of 16 bits, or pairs of codes and
// their steps and least values.
struct Cache {
  te_attn_paged_cache c{};
  const at::Tensor* first;  // of the cache's dtype
  int batch;

  explicit Cache(PyObject* const* o) {
    const bool four = PyTuple_Check(o[0]) || PyList_Check(o[0]);
    const at::Tensor *data[2], *meta[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
      if (four) {
        need((PyTuple_Check(o[i]) || PyList_Check(o[i])) && PySequence_Size(o[i]) == 2, kCacheForm);
        PyObject** two = PySequence_Fast_ITEMS(o[i]);
        data[i] = &tensor(two[0]);
        meta[i] = &tensor(two[1]);
      } else {
        data[i] = &tensor(o[i]);
      }
    }
    first = four ? meta[0] : data[0];
    need(first->is_cuda(), kOneDevice);
    const auto index = first->device().index();
    c.dtype = dtype_code(*first);
    need(c.dtype >= 0 && data[0]->dim() == 4, kCacheForm);
    const int64_t pages = data[0]->size(0), heads = data[0]->size(1), size = data[0]->size(2);
    const int64_t d = four ? 2 * data[0]->size(3) : data[0]->size(3);
    int64_t strides[4] = {0, 0, 0, 0};
    for (int i = 0; i < 2; ++i) {
      need(on_device(*data[i], index) && (!four || on_device(*meta[i], index)), kOneDevice);
      need(data[i]->sizes() == data[0]->sizes() && data[i]->scalar_type() == (four ? at::kByte : first->scalar_type()) &&
               whole(*data[i]),
           kCacheForm);
      strides[i] = page_bytes(*data[i]);
      if (four) {
        const int64_t want[] = {pages, heads, size, d / 32, 2};
        need(d % 32 == 0 && meta[i]->sizes() == at::IntArrayRef(want, 5) && meta[i]->scalar_type() == first->scalar_type() &&
                 whole(*meta[i]),
             kCacheForm);
        strides[2 + i] = page_bytes(*meta[i]);
      }
    }
    const at::Tensor& table = tensor(o[2]);
    need(table.scalar_type() == at::kInt && table.dim() == 2 && on_device(table, index) &&
             (table.size(1) <= 1 || table.stride(1) == 1),
         "page_table must be int32 [batch, pages of a sequence] on the cache's device, its rows contiguous");
    c.k = data[0]->mutable_data_ptr();
    c.v = data[1]->mutable_data_ptr();
    c.k_meta = four ? meta[0]->mutable_data_ptr() : nullptr;
    c.v_meta = four ? meta[1]->mutable_data_ptr() : nullptr;
    c.k_stride = strides[0];
    c.v_stride = strides[1];
    c.k_meta_stride = strides[2];
    c.v_meta_stride = strides[3];
    c.page_table = table.const_data_ptr<int32_t>();
    batch = as_int(table.size(0));
    c.table_stride = batch > 1 ? table.stride(0) : 0;
    c.num_pages = as_int(pages);
    c.page_size = as_int(size);
    c.max_pages = as_int(table.size(1));
    c.hkv = as_int(heads);
    c.d = as_int(d);
  }

 private:
  // everything behind the first axis contiguous (axes of one element have no stride)
  static bool whole(const at::Tensor& t) {
    int64_t n = 1;
    for (int64_t i = t.dim() - 1; i > 0; --i) {
      if (t.size(i) > 1 && t.stride(i) != n) return false;
      n *= t.size(i);
    }
    return true;
  }
  static int64_t page_bytes(const at::Tensor& t) {
    int64_t n = t.element_size();
    if (t.size(0) > 1) return t.stride(0) * n;
    for (int64_t i = 1; i < t.dim(); ++i) n *= t.size(i);
    return (n + 15) / 16 * 16;
  }
};

// One int32 for the call's status bits, or None.
int32_t* status_word(PyObject* o, c10::DeviceIndex index) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o);
  need(t.scalar_type() == at::kInt && t.numel() == 1 && on_device(t, index), "status must be one int32 on the cache's device");
  return t.mutable_data_ptr<int32_t>();
}

// (entry point, k_cache, v_cache, page_table, q or None, k, v, past, cu_seqlens, padded ones, inv_freq or None, interleaved,
// mscale, q_out, status, stream)
PyObject* paged_append(PyObject* const* a) {
  const Cache cache(a + 1);
  const auto index = cache.first->device().index();
  const bool with_q = given(a[4]), turn = given(a[10]);
  const at::Tensor &k = tensor(a[5]), &v = tensor(a[6]);
  const at::Tensor& q = with_q ? tensor(a[4]) : k;
  const auto type = cache.first->scalar_type();
  need(on_device(q, index) && on_device(k, index) && on_device(v, index), kOneDevice);
  for (const at::Tensor* x : {&q, &k, &v})
    need(x->scalar_type() == type && x->dim() == 3 && x->size(0) == k.size(0) && x->size(2) == cache.c.d &&
             (x->numel() == 0 || x->stride(2) == 1),
         "q, k and v must be [T, heads, d] of the cache's dtype, with adjacent elements in a head");
  need(k.size(1) == cache.c.hkv && v.size(1) == cache.c.hkv, "k and v must have the cache's heads");
  need(with_q || !given(a[13]), "q_out without q");
  const at::Tensor* w = turn ? &tensor(a[10]) : nullptr;
  if (turn)
    need(w->scalar_type() == at::kDouble && w->dim() == 1 && w->is_contiguous() && on_device(*w, index),
         "inv_freq must be a contiguous float64 vector");
  const int batch = cache.batch;
  const int32_t* past = lengths(a[7], batch, index);
  const int32_t *cu = lengths(a[8], batch + int64_t{1}, index), *pad = lengths(a[9], batch + int64_t{1}, index);
  const int interleaved = PyObject_IsTrue(a[11]);
  if (interleaved < 0) throw python_error();
  const float mscale = static_cast<float>(number(a[12]));
  int32_t* status = status_word(a[14], index);
  auto stride = [](const at::Tensor& x, int64_t dim) { return x.size(dim) > 1 ? x.stride(dim) : 0; };
  const int hq = with_q ? as_int(q.size(1)) : 0, total = as_int(k.size(0)), freqs = turn ? as_int(w->numel()) : 0;
  const Place place(index, a[15]);
  std::optional<Output> qo;
  if (with_q) qo.emplace(a[13], q.sizes(), q, type, "q_out must be contiguous, with the shape, dtype and device of q");
  const void* q_at = with_q ? q.const_data_ptr() : nullptr;
  void* qo_at = with_q ? qo->at() : nullptr;
  const auto fn = reinterpret_cast<decltype(&te_attn_paged_append)>(address(a[0]));
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fn(&cache.c, q_at, k.const_data_ptr(), v.const_data_ptr(), qo_at, turn ? w->const_data_ptr<double>() : nullptr, freqs,
          cu, pad, past, batch, total, hq, with_q ? stride(q, 0) : 0, with_q ? stride(q, 1) : 0, stride(k, 0), stride(k, 1),
          stride(v, 0), stride(v, 1), interleaved, mscale, status, place.stream());
  Py_END_ALLOW_THREADS;
  if (rc != 0) return PyLong_FromLong(rc);
  return with_q ? qo->result() : Py_NewRef(Py_None);
}

// (entry point, k_cache, v_cache, page_table, start, cu_seqlens, padded ones, total, k, v, status, stream)
PyObject* paged_gather(PyObject* const* a) {
  const Cache cache(a + 1);
  const auto index = cache.first->device().index();
  const int batch = cache.batch;
  const int32_t* start = lengths(a[4], batch, index);
  const int32_t *cu = lengths(a[5], batch + int64_t{1}, index), *pad = lengths(a[6], batch + int64_t{1}, index);
  const long total = integer(a[7]);
  need(total >= 0 && total <= INT_MAX, "total must lie in [0, 2^31)");
  int32_t* status = status_word(a[10], index);
  const Place place(index, a[11]);
  const int64_t shape[] = {total, cache.c.hkv, cache.c.d};
  constexpr const char* what = "k and v must be contiguous [total, hkv, d] of the cache's dtype, on its device";
  const Output k(a[8], at::IntArrayRef(shape, 3), *cache.first, cache.first->scalar_type(), what);
  const Output v(a[9], at::IntArrayRef(shape, 3), *cache.first, cache.first->scalar_type(), what);
  const auto fn = reinterpret_cast<decltype(&te_attn_paged_gather)>(address(a[0]));
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fn(&cache.c, k.at(), v.at(), cu, pad, start, batch, static_cast<int>(total), status, place.stream());
  Py_END_ALLOW_THREADS;
  return rc != 0 ? PyLong_FromLong(rc) : pack({&k, &v});
}

// (entry point, size function, k_cache, v_cache, page_table, q, past, cu_seqlens_q, padded ones, scale, window, sinks, out,
// lse, workspace, stream)
PyObject* paged_fwd(PyObject* const* a) {
  const auto fn = reinterpret_cast<decltype(&te_attn_paged_fwd_thd)>(address(a[0]));
  const auto size = reinterpret_cast<decltype(&te_attn_paged_fwd_workspace_size)>(address(a[1]));
  const Cache cache(a + 2);
  const auto index = cache.first->device().index();
  const at::Tensor& q = tensor(a[5]);
  need(on_device(q, index), kOneDevice);
  need(q.scalar_type() == cache.first->scalar_type() && q.dim() == 3 && q.size(2) == cache.c.d && q.is_contiguous(),
       "q must be contiguous [T_q, hq, d] of the cache's dtype");
  const int batch = cache.batch;
  const int32_t* past = lengths(a[6], batch, index);
  const int32_t *cu = lengths(a[7], batch + int64_t{1}, index), *pad = lengths(a[8], batch + int64_t{1}, index);
  const float scale = static_cast<float>(number(a[9]));
  const int window = static_cast<int>(integer(a[10])), sinks = static_cast<int>(integer(a[11]));
  const int total = as_int(q.size(0)), hq = as_int(q.size(1));
  const Place place(index, a[15]);
  const Output out(a[12], q.sizes(), q, q.scalar_type(), kOutput);
  const Output lse(a[13], q.sizes().slice(0, 2), q, at::kFloat, kLse);
  const Workspace ws(a[14], given(a[14]) ? 0 : size(batch, total, hq, cache.c.hkv, cache.c.d, cache.c.k_meta ? 4 : 16), q);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fn(&cache.c, q.const_data_ptr(), out.at(), static_cast<float*>(lse.at()), cu, pad, past, batch, total, hq, scale, window,
          sinks, ws.at(), ws.bytes(), place.stream());
  Py_END_ALLOW_THREADS;
  return rc != 0 ? PyLong_FromLong(rc) : pack({&out, &lse});
}

// What forward and backward with a sliding window have in common: packed tensors with four
// cu_seqlens, or sequence-major ones with two (the padded ones None).
struct Windowed {
  const at::Tensor &q, &k, &v;
  c10::DeviceIndex index;
  int code, batch, hq, hkv, d;
  bool packed;
  int lq, lk;      // rows, or tokens of a batch entry
  int tq, tk;      // rows
  const int32_t* cu[4];

  Windowed(PyObject* const* tensors, PyObject* const* lens) : q(tensor(tensors[0])), k(tensor(tensors[1])), v(tensor(tensors[2])) {
    need(q.is_cuda(), kOneDevice);
    index = q.device().index();
    need(on_device(k, index) && on_device(v, index), kOneDevice);
    need(q.is_contiguous() && k.is_contiguous() && v.is_contiguous(), "all tensors must be contiguous");
    code = dtype_code(q);
    need(code >= 0 && k.scalar_type() == q.scalar_type() && v.scalar_type() == q.scalar_type(),
         "q, k, v must share one dtype, float16 or bfloat16");
    packed = given(lens[2]);
    const int64_t dims = packed ? 3 : 4;
    need(q.dim() == dims && k.dim() == dims && v.sizes() == k.sizes() && k.size(dims - 1) == q.size(dims - 1),
         packed ? "q, k and v must be [rows, heads, d], v shaped like k" : "q, k and v must be [S, B, heads, d], v shaped like k");
    const int64_t n = tensor(lens[0]).numel();
    need(n >= 2, "cu_seqlens must hold batch + 1 values");
    batch = as_int(n - 1);
    for (int i = 0; i < (packed ? 4 : 2); ++i) cu[i] = lengths(lens[i], n, index);
    need(packed || (q.size(1) == batch && k.size(1) == batch), "q, k and v must have one batch entry per sequence");
    hq = as_int(q.size(dims - 2));
    hkv = as_int(k.size(dims - 2));
    d = as_int(q.size(dims - 1));
    lq = as_int(q.size(0));
    lk = as_int(k.size(0));
    tq = packed ? lq : as_int(static_cast<int64_t>(lq) * batch);
    tk = packed ? lk : as_int(static_cast<int64_t>(lk) * batch);
  }
};

constexpr const char* kWindowLse = "lse must be contiguous float32, one value per row and head of q, on q's device";
using WindowSizeFn = size_t (*)(int, int, int, int, int, int);

// (entry point, size function, q, k, v, cu_seqlens_q, cu_seqlens_kv, padded ones or None, scale, mask, window, sinks, out,
// lse, workspace, stream)
PyObject* window_fwd(PyObject* const* a) {
  const auto size = reinterpret_cast<WindowSizeFn>(address(a[1]));
  const Windowed p(a + 2, a + 5);
  const float scale = static_cast<float>(number(a[9]));
  const int mask = static_cast<int>(integer(a[10])), window = static_cast<int>(integer(a[11])), sinks = static_cast<int>(integer(a[12]));
  const Place place(p.index, a[16]);
  const Output out(a[13], p.q.sizes(), p.q, p.q.scalar_type(), kOutput);
  const Output lse(a[14], p.q.sizes().slice(0, p.q.dim() - 1), p.q, at::kFloat, kWindowLse);
  const Workspace ws(a[15], given(a[15]) ? 0 : size(p.batch, p.tq, p.tk, p.hq, p.hkv, p.d), p.q);
  void* fn = address(a[0]);
  const void *q = p.q.const_data_ptr(), *k = p.k.const_data_ptr(), *v = p.v.const_data_ptr();
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  if (p.packed)
    rc = reinterpret_cast<decltype(&te_attn_window_fwd_thd)>(fn)(
        q, k, v, out.at(), static_cast<float*>(lse.at()), p.cu[0], p.cu[1], p.cu[2], p.cu[3], p.batch, p.lq, p.lk, p.hq, p.hkv, p.d,
        scale, mask, window, sinks, p.code, ws.at(), ws.bytes(), place.stream());
  else
    rc = reinterpret_cast<decltype(&te_attn_window_fwd_sbhd)>(fn)(
        q, k, v, out.at(), static_cast<float*>(lse.at()), p.cu[0], p.cu[1], p.batch, p.lq, p.lk, p.hq, p.hkv, p.d, scale, mask, window,
        sinks, p.code, ws.at(), ws.bytes(), place.stream());
  Py_END_ALLOW_THREADS;
  return rc != 0 ? PyLong_FromLong(rc) : pack({&out, &lse});
}

// (entry point, size function, q, k, v, cu_seqlens_q, cu_seqlens_kv, padded ones or None, scale, mask, window, sinks, out,
// dout, lse, dq, dk, dv, workspace, stream)
PyObject* window_bwd(PyObject* const* a) {
  const auto size = reinterpret_cast<decltype(&te_attn_window_bwd_workspace_size)>(address(a[1]));
  const Windowed p(a + 2, a + 5);
  const float scale = static_cast<float>(number(a[9]));
  const int mask = static_cast<int>(integer(a[10])), window = static_cast<int>(integer(a[11])), sinks = static_cast<int>(integer(a[12]));
  need(given(a[13]) && given(a[14]) && given(a[15]), "the backward needs out, dout and lse");
  const Place place(p.index, a[20]);
  const auto type = p.q.scalar_type();
  const Output out(a[13], p.q.sizes(), p.q, type, kOutput), dout(a[14], p.q.sizes(), p.q, type, kOutput);
  const Output lse(a[15], p.q.sizes().slice(0, p.q.dim() - 1), p.q, at::kFloat, kWindowLse);
  const Output dq(a[16], p.q.sizes(), p.q, type, kOutput), dk(a[17], p.k.sizes(), p.q, type, kOutput);
  const Output dv(a[18], p.k.sizes(), p.q, type, kOutput);
  const Workspace ws(a[19], given(a[19]) ? 0 : size(p.batch, p.tq, p.tk, p.hq, p.hkv, p.d, window, sinks), p.q);
  void* fn = address(a[0]);
  const void *q = p.q.const_data_ptr(), *k = p.k.const_data_ptr(), *v = p.v.const_data_ptr();
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  if (p.packed)
    rc = reinterpret_cast<decltype(&te_attn_window_bwd_thd)>(fn)(
        q, k, v, out.at(), dout.at(), static_cast<float*>(lse.at()), dq.at(), dk.at(), dv.at(), p.cu[0], p.cu[1], p.cu[2], p.cu[3],
        p.batch, p.lq, p.lk, p.hq, p.hkv, p.d, scale, mask, window, sinks, p.code, ws.at(), ws.bytes(), place.stream());
  else
    rc = reinterpret_cast<decltype(&te_attn_window_bwd_sbhd)>(fn)(
        q, k, v, out.at(), dout.at(), static_cast<float*>(lse.at()), dq.at(), dk.at(), dv.at(), p.cu[0], p.cu[1], p.batch, p.lq, p.lk,
        p.hq, p.hkv, p.d, scale, mask, window, sinks, p.code, ws.at(), ws.bytes(), place.stream());
  Py_END_ALLOW_THREADS;
  return rc != 0 ? PyLong_FromLong(rc) : pack({&dq, &dk, &dv});
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
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<paged_append, 16>)), METH_FASTCALL, nullptr},
    {"paged_gather", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<paged_gather, 12>)), METH_FASTCALL, nullptr},
    {"paged_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<paged_fwd, 16>)), METH_FASTCALL, nullptr},
    {"window_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<window_fwd, 17>)), METH_FASTCALL, nullptr},
    {"window_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<window_bwd, 21>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_teattn_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__teattn_host() { return PyModule_Create(&module); }
