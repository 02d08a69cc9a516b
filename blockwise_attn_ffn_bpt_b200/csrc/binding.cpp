// The part of the Python binding that a token-by-token loop calls: argument
// checks, outputs and workspaces of the rotary and 4-bit cache entry points in
// C++, because the same through ctypes takes two to three times as long as the
// kernels of a small call. Each function takes its arguments by place, runs on
// torch's current stream of the tensors' device, and returns its outputs, or the
// library's status as an int where that is not BPT_OK; a bad argument raises.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <climits>
#include <string>

#include "bpt.h"

namespace {

// A bad argument: raises `type` with the message.
struct Refused {};
template <typename... Parts>
[[noreturn]] void refuse(PyObject* type, const Parts&... parts) {
  const std::string text = c10::str(parts...);
  PyErr_SetString(type, text.c_str());
  throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a tensor");
  return THPVariable_Unpack(o);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

int small(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT_MIN || v > INT_MAX) refuse(PyExc_ValueError, name, " = ", v, " is out of range");
  return (int)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

// Token rows [b, s, width] of a CUDA tensor, each contiguous.
struct Rows {
  void* p = nullptr;
  long long bs = 0, ld = 0;
};

Rows rows_of(const at::Tensor& t, const char* name, int64_t width, const at::Tensor* like = nullptr) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, name, " must be a CUDA tensor");
  if (t.dim() != 3 || t.size(2) != width)
    refuse(PyExc_ValueError, name, " has shape ", t.sizes(), ", expected [b, s, ", width, "]");
  if (like != nullptr && (t.size(0) != like->size(0) || t.size(1) != like->size(1) ||
                          t.scalar_type() != like->scalar_type() || t.device() != like->device()))
    refuse(PyExc_ValueError, name, " must have the tokens, dtype and device of the first tensor");
  if (t.stride(2) != 1) refuse(PyExc_ValueError, name, "'s rows must be contiguous");
  return Rows{t.data_ptr(), t.stride(0), t.stride(1)};
}

int count_of(int64_t n, const char* name) {
  if (n > INT_MAX) refuse(PyExc_ValueError, name, " = ", n, " is out of range");
  return (int)n;
}

at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) {
  return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);  // at::empty without the dispatcher
}

Rows new_rows(const at::Tensor& t) { return Rows{t.data_ptr(), t.stride(0), t.stride(1)}; }

PyObject* answer(std::initializer_list<at::Tensor> out) {
  PyObject* r = PyTuple_New((Py_ssize_t)out.size());
  if (r == nullptr) throw Refused{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : out) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// A 4-bit cache: its tensor [b, kv_heads, capacity / 64, block bytes] and dh.
struct Cache {
  const at::Tensor* data;
  int b, kv_heads, capacity, dh;
  Cache(PyObject* o, PyObject* dim, const char* name) : data(&tensor(o, name)), dh(small(dim, "dh")) {
    const at::Tensor& t = *data;
    if (!t.is_cuda() || t.scalar_type() != at::kByte || t.dim() != 4 || !t.is_contiguous())
      refuse(PyExc_ValueError, name, " must be a contiguous uint8 CUDA tensor of 4 dimensions");
    if ((dh != 64 && dh != 128) || t.size(3) != 72 * dh)
      refuse(PyExc_ValueError, name, "'s blocks are ", t.size(3), " bytes, which is not 72 dh for dh = ", dh);
    b = count_of(t.size(0), "b");
    kv_heads = count_of(t.size(1), "kv_heads");
    capacity = count_of(t.size(2) * 64, "capacity");
  }
  int64_t width() const { return (int64_t)kv_heads * dh; }
  int* ints(PyObject* o, const char* name) const {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || t.device() != data->device() || t.dim() != 1 || t.size(0) != b || !t.is_contiguous())
      refuse(PyExc_ValueError, name, " must be a contiguous int32 tensor [", b, "] on the cache's device");
    return t.data_ptr<int>();
  }
  float* floats(const at::Tensor& t, const char* name) const {
    if (t.scalar_type() != at::kFloat || t.device() != data->device() || t.dim() != 3 || t.size(0) != b ||
        t.size(1) != kv_heads || t.size(2) != capacity || !t.is_contiguous())
      refuse(PyExc_ValueError, name, " must be a contiguous fp32 tensor [", b, ", ", kv_heads, ", ", capacity,
             "] on the cache's device");
    return t.data_ptr<float>();
  }
};

// While outputs are allocated and kernels launched, either of which may wait for
// the GPU, other Python threads run. Nothing in its scope raises through Python.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject* status(int r) { return PyLong_FromLong(r); }

void* stream_of(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

// rotary(q, k, heads, kv_heads, inv_freq, positions, offset, interleaved, magnitude, inverse, q_out, k_out)
PyObject* rotary(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [b, s, heads * dh]");
  const int heads = small(a[2], "heads");
  if (heads <= 0 || q.size(2) % heads)
    refuse(PyExc_ValueError, "q's last dimension ", q.size(2), " does not hold ", heads, " heads");
  const int dh = count_of(q.size(2) / heads, "dh"), b = count_of(q.size(0), "b"), s = count_of(q.size(1), "s");
  const Rows rq = rows_of(q, "q", q.size(2));
  if (q.scalar_type() != at::kBFloat16 && q.scalar_type() != at::kFloat)
    refuse(PyExc_TypeError, "q has dtype ", q.scalar_type());
  const bool keys = a[1] != Py_None;
  const int kv_heads = keys ? small(a[3], "kv_heads") : 0;
  const int64_t k_width = (int64_t)kv_heads * dh;
  const Rows rk = keys ? rows_of(tensor(a[1], "k"), "k", k_width, &q) : Rows{};
  const at::Tensor& freq = tensor(a[4], "inv_freq");
  if (freq.scalar_type() != at::kDouble || !freq.device().is_cpu() || freq.dim() != 1 || !freq.is_contiguous())
    refuse(PyExc_TypeError, "inv_freq must be a contiguous fp64 vector in host memory");
  const void* at = nullptr;
  int size = 8;
  long long step = 0;
  if (a[5] != Py_None) {
    const at::Tensor& p = tensor(a[5], "positions");
    if ((p.scalar_type() != at::kInt && p.scalar_type() != at::kLong) || p.device() != q.device())
      refuse(PyExc_TypeError, "positions must be int32 or int64 on q's device");
    const bool two = p.dim() == 2;
    if (!(two && p.size(0) == b && p.size(1) == s) && !(p.dim() == 1 && p.size(0) == s))
      refuse(PyExc_ValueError, "positions has shape ", p.sizes(), ", expected [", b, ", ", s, "] or [", s, "]");
    if (s > 1 && p.stride(-1) != 1) refuse(PyExc_ValueError, "positions must be contiguous along the sequence");
    at = p.data_ptr();
    size = (int)p.element_size();
    step = two ? p.stride(0) : 0;
  }
  const double magnitude = PyFloat_AsDouble(a[8]);
  if (magnitude == -1.0 && PyErr_Occurred()) throw Refused{};
  const int rot = count_of(2 * freq.numel(), "rot"), interleaved = truth(a[7]), inverse = truth(a[9]);
  const long long offset = integer(a[6]);
  at::Tensor q_out, k_out;
  Rows rqo, rko;
  const bool own_q = a[10] == Py_None, own_k = keys && a[11] == Py_None;
  if (!own_q) rqo = rows_of(tensor(a[10], "q_out"), "q_out", q.size(2), &q);
  if (keys && !own_k) rko = rows_of(tensor(a[11], "k_out"), "k_out", k_width, &q);
  int r;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(q.device());
    if (own_q) {
      q_out = new_tensor(q.sizes(), q.scalar_type(), q);
      rqo = new_rows(q_out);
    }
    if (own_k) {
      k_out = new_tensor({b, s, k_width}, q.scalar_type(), q);
      rko = new_rows(k_out);
    }
    r = bpt_rotary(q.scalar_type() == at::kFloat ? BPT_DTYPE_F32 : BPT_DTYPE_BF16, rq.p, rq.bs, rq.ld, rk.p, rk.bs, rk.ld,
                   b, s, heads, kv_heads, dh, rot, interleaved, freq.data_ptr<double>(), (float)magnitude, at, size, step,
                   offset, inverse, rqo.p, rqo.bs, rqo.ld, rko.p, rko.bs, rko.ld, stream_of(q));
  }
  if (r != BPT_OK) return status(r);
  PyObject* first = own_q ? THPVariable_Wrap(q_out) : Py_NewRef(a[10]);
  PyObject* second = own_k ? THPVariable_Wrap(k_out) : Py_NewRef(keys ? a[11] : Py_None);
  PyObject* both = PyTuple_Pack(2, first, second);
  Py_XDECREF(first);
  Py_XDECREF(second);
  return both;
}

// kv4_store(data, dh, k, v, start, counts)
PyObject* kv4_store(PyObject* const* a) {
  const Cache c(a[0], a[1], "the cache");
  const at::Tensor& k = tensor(a[2], "k");
  const at::Tensor& v = tensor(a[3], "v");
  const Rows rk = rows_of(k, "k", c.width()), rv = rows_of(v, "v", c.width(), &k);
  if (k.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "k has dtype ", k.scalar_type());
  if (k.size(0) != c.b || k.device() != c.data->device())
    refuse(PyExc_ValueError, "k must hold ", c.b, " sequences on the cache's device");
  const int* start = c.ints(a[4], "start");
  const int* counts = a[5] == Py_None ? nullptr : c.ints(a[5], "counts");
  const int n = count_of(k.size(1), "n");
  int r;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(k.device());
    r = bpt_kv4_store(c.data->data_ptr(), c.b, c.kv_heads, c.capacity, c.dh, rk.p, rk.bs, rk.ld, rv.p, rv.bs, rv.ld, n,
                      start, counts, stream_of(k));
  }
  return status(r);
}

// kv4_load(data, dh, lens, n, start)
PyObject* kv4_load(PyObject* const* a) {
  const Cache c(a[0], a[1], "the cache");
  const int* lens = c.ints(a[2], "lens");
  const int n = small(a[3], "n");
  if (n < 0) refuse(PyExc_ValueError, "n = ", n, " is negative");
  const int* start = a[4] == Py_None ? nullptr : c.ints(a[4], "start");
  at::Tensor k, v;
  int r;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(c.data->device());
    k = new_tensor({c.b, n, c.width()}, at::kBFloat16, *c.data);
    v = new_tensor({c.b, n, c.width()}, at::kBFloat16, *c.data);
    r = bpt_kv4_load(c.data->data_ptr(), c.b, c.kv_heads, c.capacity, c.dh, start, lens, n, k.data_ptr(), v.data_ptr(),
                     stream_of(*c.data));
  }
  return r != BPT_OK ? status(r) : answer({k, v});
}

// kv4_attention(q, data, dh, lens, heads, causal, weights, return_lse)
PyObject* kv4_attention(PyObject* const* a) {
  const Cache c(a[1], a[2], "the cache");
  const at::Tensor& q = tensor(a[0], "q");
  const int heads = small(a[4], "heads");
  const Rows rq = rows_of(q, "q", (int64_t)heads * c.dh);
  if (q.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "q has dtype ", q.scalar_type());
  if (q.size(0) != c.b || q.device() != c.data->device())
    refuse(PyExc_ValueError, "q must hold ", c.b, " sequences on the cache's device");
  const int* lens = c.ints(a[3], "lens");
  float* weights = a[6] == Py_None ? nullptr : c.floats(tensor(a[6], "weights"), "weights");
  const bool lse = truth(a[7]), causal = truth(a[5]);
  const int n = count_of(q.size(1), "n");
  at::Tensor o, lse2, ws;
  int r;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(q.device());
    o = new_tensor(q.sizes(), at::kBFloat16, q);
    if (lse) lse2 = new_tensor({c.b, heads, n}, at::kFloat, q);
    const size_t bytes =
        bpt_kv4_attention_workspace_bytes(c.b, n, heads, c.kv_heads, c.capacity, c.dh, weights != nullptr);
    if (bytes) ws = new_tensor({(int64_t)bytes}, at::kByte, q);
    r = bpt_kv4_attention(rq.p, rq.bs, rq.ld, c.data->data_ptr(), lens, c.b, n, heads, c.kv_heads, c.capacity, c.dh, causal,
                          o.data_ptr(), lse ? lse2.data_ptr<float>() : nullptr, weights, bytes ? ws.data_ptr() : nullptr,
                          bytes, stream_of(q));
  }
  if (r != BPT_OK) return status(r);
  return lse ? answer({o, lse2}) : THPVariable_Wrap(o);
}

// kv4_evict(data, dh, weights, lens, keep, recent, out data, out dh)
PyObject* kv4_evict(PyObject* const* a) {
  const Cache c(a[0], a[1], "the cache"), out(a[6], a[7], "out");
  if (out.b != c.b || out.kv_heads != c.kv_heads || out.dh != c.dh || out.data->device() != c.data->device())
    refuse(PyExc_ValueError, "out must have the sequences, heads and device of the cache");
  const float* weights = c.floats(tensor(a[2], "weights"), "weights");
  const int* lens = c.ints(a[3], "lens");
  const int keep = small(a[4], "keep"), recent = small(a[5], "recent");
  at::Tensor kept, new_lens, new_weights;
  int r;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(c.data->device());
    kept = new_tensor({c.b, c.kv_heads, std::min(std::max(keep, 0), out.capacity)}, at::kInt, *c.data);
    new_lens = new_tensor({c.b}, at::kInt, *c.data);
    new_weights = new_tensor({c.b, c.kv_heads, out.capacity}, at::kFloat, *c.data);
    r = bpt_kv4_evict(c.data->data_ptr(), weights, lens, c.b, c.kv_heads, c.capacity, c.dh, keep, recent,
                      out.data->data_ptr(), out.capacity, new_weights.data_ptr<float>(), new_lens.data_ptr<int>(),
                      kept.data_ptr<int>(), stream_of(*c.data));
  }
  return r != BPT_OK ? status(r) : answer({kept, new_lens, new_weights});
}

// No C++ exception leaves a call: torch's become its Python ones.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
constexpr PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>));
}

PyMethodDef methods[] = {{"rotary", method<rotary, 12>(), METH_FASTCALL, nullptr},
                         {"kv4_store", method<kv4_store, 6>(), METH_FASTCALL, nullptr},
                         {"kv4_load", method<kv4_load, 5>(), METH_FASTCALL, nullptr},
                         {"kv4_attention", method<kv4_attention, 8>(), METH_FASTCALL, nullptr},
                         {"kv4_evict", method<kv4_evict, 8>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
