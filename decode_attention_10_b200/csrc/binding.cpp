// The two chunk calls of mfa.py for torch tensors, from C++: checks of the arguments, the
// current stream, and the C entry point (include/mfa.h), whose address mfa.py hands over from
// the library it has loaded. A serving loop makes these calls per layer and step, and reading
// the tensors' attributes from Python took longer (5 us) than the launch itself (2.7 us).
//
// Each function returns the mfa_status of the call, or -1 - i if its i-th tensor argument is
// not what the call takes, or kOtherDevice (the caller then finds the words).
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mfa.h"

namespace {

using at::Tensor;

decltype(&mfa_rope_append) f_rope_append = nullptr;
decltype(&mfa_chunk_attn) f_chunk_attn = nullptr;

// bind(address of mfa_rope_append, address of mfa_chunk_attn)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  void* f[2] = {nullptr, nullptr};
  for (Py_ssize_t i = 0; i < 2 && n_args == 2; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  if (f[0] == nullptr || f[1] == nullptr) {
    PyErr_SetString(PyExc_TypeError, "bind takes two addresses");
    return nullptr;
  }
  f_rope_append = reinterpret_cast<decltype(f_rope_append)>(f[0]);
  f_chunk_attn = reinterpret_cast<decltype(f_chunk_attn)>(f[1]);
  Py_RETURN_NONE;
}

bool ready(Py_ssize_t n_args, Py_ssize_t takes) {
  if (n_args == takes && f_chunk_attn != nullptr) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or no library bound");
  return false;
}

// The current device; -1 without one (no tensor of a device is there then).
int current_device() {
  c10::DeviceIndex dev = 0;
  return c10::cuda::GetDevice(&dev) == cudaSuccess ? dev : -1;
}

// What the cache, the workspace and the rotation's table have their memory on (`o`, a device's
// index) is not the current device.
constexpr long kOtherDevice = -100;
bool elsewhere(PyObject* o, int dev) { return PyLong_AsLong(o) != dev; }

// A tensor argument; false if it is none.
bool tensor(PyObject* o, const Tensor** t) {
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return true;
}

bool on(const Tensor& t, int dev, at::ScalarType type) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == dev;
}

// Dense bf16 [n, 64, 256].
bool queries(const Tensor& t, int dev, int64_t n) {
  return on(t, dev, at::kBFloat16) && t.dim() == 3 && t.size(0) == n && t.size(1) == MFA_N_HEADS &&
         t.size(2) == MFA_HEAD_DIM && t.is_contiguous();
}

// bf16 [n, 256] with dense rows.
bool rows(const Tensor& t, int dev, int64_t n) {
  return on(t, dev, at::kBFloat16) && t.dim() == 2 && t.size(0) == n && t.size(1) == MFA_HEAD_DIM &&
         t.stride(1) == 1;
}

// Dense int32 [n].
bool ints(const Tensor& t, int dev, int64_t n) {
  return on(t, dev, at::kInt) && t.dim() == 1 && t.size(0) == n && t.is_contiguous();
}

void* stream_of(PyObject* o, int dev) {
  return o == Py_None ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev).stream())
                      : PyLong_AsVoidPtr(o);
}

PyObject* refused(int i) { return PyLong_FromLong(-1 - i); }

// rope_append(q|None, k, v, cache, batch, q_start, seq_lens, rope, axes, positions|None,
//             q_out|None, ws, ws_bytes, stream|None, device)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!ready(n_args, 15)) return nullptr;
  try {
    const int dev = current_device();
    const Tensor *q = nullptr, *k, *v, *q_start, *seq_lens, *pos = nullptr, *q_out = nullptr;
    if (!tensor(a[1], &k) || k->dim() != 2) return refused(0);
    const int64_t n = k->size(0), batch = PyLong_AsLongLong(a[4]), axes = PyLong_AsLongLong(a[8]);
    if (!rows(*k, dev, n) || n > MFA_MAX_ROWS) return refused(0);
    if (!tensor(a[2], &v) || !rows(*v, dev, n)) return refused(1);
    if (!tensor(a[5], &q_start) || !ints(*q_start, dev, batch + 1)) return refused(2);
    if (!tensor(a[6], &seq_lens) || !ints(*seq_lens, dev, batch)) return refused(3);
    if (a[0] != Py_None) {
      if (!tensor(a[0], &q) || !queries(*q, dev, n)) return refused(4);
      if (!tensor(a[10], &q_out) || !queries(*q_out, dev, n)) return refused(5);
    }
    if (a[9] != Py_None) {
      if (!tensor(a[9], &pos) || !on(*pos, dev, at::kInt) || !pos->is_contiguous() ||
          pos->numel() != axes * n || pos->size(-1) != n || pos->dim() > 2)
        return refused(6);
    }
    // (the row stride of a single row says nothing)
    const int64_t k_ld = n > 1 ? k->stride(0) : MFA_HEAD_DIM, v_ld = n > 1 ? v->stride(0) : MFA_HEAD_DIM;
    if (k_ld > INT32_MAX) return refused(0);
    if (v_ld > INT32_MAX) return refused(1);
    auto* kv = static_cast<const mfa_kv_cache*>(PyLong_AsVoidPtr(a[3]));
    auto* rope = static_cast<const mfa_rope*>(PyLong_AsVoidPtr(a[7]));
    void* ws = PyLong_AsVoidPtr(a[11]);
    const size_t ws_bytes = PyLong_AsSize_t(a[12]);
    void* stream = stream_of(a[13], dev);
    if (elsewhere(a[14], dev) && !PyErr_Occurred()) return PyLong_FromLong(kOtherDevice);
    if (PyErr_Occurred()) return nullptr;
    return PyLong_FromLong(f_rope_append(
        q ? q->data_ptr() : nullptr, k->data_ptr(), static_cast<int32_t>(k_ld), v->data_ptr(),
        static_cast<int32_t>(v_ld), rope, pos ? static_cast<const int32_t*>(pos->data_ptr()) : nullptr,
        kv, static_cast<const int32_t*>(q_start->data_ptr()),
        static_cast<const int32_t*>(seq_lens->data_ptr()), static_cast<int32_t>(n),
        q_out ? q_out->data_ptr() : nullptr, ws, ws_bytes, stream));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// chunk_attn(q, cache, batch, q_start, seq_lens, scale, out, ws, ws_bytes, stream|None, device)
PyObject* chunk_attn(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!ready(n_args, 11)) return nullptr;
  try {
    const int dev = current_device();
    const Tensor *q, *q_start, *seq_lens, *out;
    if (!tensor(a[0], &q) || q->dim() != 3) return refused(0);
    const int64_t n = q->size(0), batch = PyLong_AsLongLong(a[2]);
    if (!queries(*q, dev, n) || n > MFA_MAX_ROWS) return refused(0);
    if (!tensor(a[3], &q_start) || !ints(*q_start, dev, batch + 1)) return refused(1);
    if (!tensor(a[4], &seq_lens) || !ints(*seq_lens, dev, batch)) return refused(2);
    if (!tensor(a[6], &out) || !queries(*out, dev, n)) return refused(3);
    auto* kv = static_cast<const mfa_kv_cache*>(PyLong_AsVoidPtr(a[1]));
    const double scale = PyFloat_AsDouble(a[5]);
    void* ws = PyLong_AsVoidPtr(a[7]);
    const size_t ws_bytes = PyLong_AsSize_t(a[8]);
    void* stream = stream_of(a[9], dev);
    if (elsewhere(a[10], dev) && !PyErr_Occurred()) return PyLong_FromLong(kOtherDevice);
    if (PyErr_Occurred()) return nullptr;
    return PyLong_FromLong(f_chunk_attn(
        q->data_ptr(), kv, static_cast<const int32_t*>(q_start->data_ptr()),
        static_cast<const int32_t*>(seq_lens->data_ptr()), static_cast<int32_t>(n),
        static_cast<float>(scale), out->data_ptr(), ws, ws_bytes, stream));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_append)),
     METH_FASTCALL, nullptr},
    {"chunk_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(chunk_attn)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "mfa_torch", nullptr, -1, methods,
                      nullptr,              nullptr,     nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mfa_torch(void) { return PyModule_Create(&module); }
