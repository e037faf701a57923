// The gate and block-scaled operators as Python calls on torch tensors.
//
// A decode step makes these calls for one token, where the kernels take 3 to 5
// us: checks and marshalling in Python (3 to 5 us a call) would be what such a
// call costs, here they take some 0.3 us.  Each function checks what the library
// takes for granted about its tensors (dtype, shape, strides, memory of the
// current GPU, a stream of it) and calls the entry point of the same name; it returns the status, or None if
// a tensor is not as it should be (the Python side then says which).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <climits>
#include <initializer_list>

#include "moe.h"

namespace {

// The current device, which the library launches on: asked for once a call, and
// only if there is a tensor of a GPU.  -1: not asked yet.
thread_local int current = -1;
int current_device() {
  if (current < 0) current = c10::hip::current_device();
  return current;
}

// A tensor in the current GPU's memory, or null.
const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda()) return nullptr;
  return t.get_device() == current_device() ? &t : nullptr;
}

bool is_codes(at::ScalarType t) { return t == at::kFloat8_e4m3fn || t == at::kByte; }

// Sizes past int32 are past every limit of the library, which then says so.
int32_t narrow(int64_t n) { return n > INT_MAX ? INT_MAX : (int32_t)n; }

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// The whole tensor: this dtype (kByte: codes) and shape, no gaps.
bool whole(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, void** p) {
  const at::Tensor* t = tensor(o);
  if (!t || t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous()) return false;
  const at::ScalarType have = t->scalar_type();
  if (have != type && !(type == at::kByte && is_codes(have))) return false;
  *p = t->data_ptr();
  return true;
}

// A matrix whose rows have no gaps.
struct Rows {
  void* p;
  int64_t rows, cols, ld;
  at::ScalarType type;
};
bool rows_of(PyObject* o, Rows* r) {
  const at::Tensor* t = tensor(o);
  if (!t || t->dim() != 2) return false;
  r->rows = t->size(0);
  r->cols = t->size(1);
  if (t->stride(1) != 1 && r->cols > 1) return false;
  r->ld = r->rows > 1 ? t->stride(0) : r->cols;  // (a single row's stride is free)
  r->type = t->scalar_type();
  r->p = t->data_ptr();
  return true;
}
// MOE_F32 or MOE_BF16, -1 for another type.
int32_t float_type(at::ScalarType t) { return t == at::kFloat ? MOE_F32 : t == at::kBFloat16 ? MOE_BF16 : -1; }

bool shape_of(PyObject* o, int64_t dim, at::IntArrayRef* shape) {
  const at::Tensor* t = tensor(o);
  if (!t || t->dim() != dim) return false;
  *shape = t->sizes();
  return true;
}

// None (no workspace) or any contiguous tensor.
bool workspace_of(PyObject* o, void** p, size_t* bytes) {
  *p = nullptr;
  *bytes = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  *bytes = t->nbytes();
  return true;
}

// The value of attribute `name`, or null (no error) where there is none.
PyObject* attribute(PyObject* o, const char* name) {
  PyObject* v = PyObject_GetAttrString(o, name);
  if (!v) PyErr_Clear();
  return v;
}

// Not a stream of another device (an object that names no device is taken).
bool stream_here(PyObject* o) {
  if (o == Py_None) return true;
  PyObject* v = attribute(o, "device_index");
  if (!v) return true;
  const long index = PyLong_Check(v) ? PyLong_AsLong(v) : current_device();
  Py_DECREF(v);
  return index == current_device();
}

// A gate's bias, which the description holds by address, is of this device (a
// description that gate() did not make keeps no tensor to look at).
bool bias_here(PyObject* gate) {
  PyObject* v = attribute(gate, "bias_tensor");
  if (!v) return true;
  const bool here = v == Py_None || tensor(v);
  Py_DECREF(v);
  return here;
}

// None: torch's current stream; else an object with torch.cuda.Stream's handle.
bool stream_of(PyObject* o, void** s) {
  if (o == Py_None) {
    *s = (void*)c10::hip::getCurrentHIPStream().stream();
    return true;
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) return false;
  *s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return !PyErr_Occurred();
}

template <class F>
PyObject* call(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

// A function of N objects; C++ exceptions become Python ones.
template <int N, PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments needed, not %zd", N, n);
    return nullptr;
  }
  current = -1;
  try {
    return F(a);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// gate (a moe_gate's bytes), z, idx, wt, stream
PyObject* gate_topk(PyObject* const* a) {
  Py_buffer view;
  if (PyObject_GetBuffer(a[0], &view, PyBUF_SIMPLE)) return nullptr;
  const bool sized = view.len == (Py_ssize_t)sizeof(moe_gate);
  moe_gate g;
  if (sized) memcpy(&g, view.buf, sizeof g);
  PyBuffer_Release(&view);
  Rows z;
  void *idx, *wt, *s;
  if (!sized || !rows_of(a[1], &z) || float_type(z.type) < 0 || z.cols != g.n_experts ||
      !whole(a[2], at::kInt, {z.rows, g.top_k}, &idx) || !whole(a[3], at::kFloat, {z.rows, g.top_k}, &wt) ||
      (g.bias && !bias_here(a[0])) || !stream_here(a[4]))
    Py_RETURN_NONE;
  if (!stream_of(a[4], &s)) return nullptr;
  return call([&] {
    return moe_gate_topk(&g, z.p, float_type(z.type), z.ld, narrow(z.rows), (int32_t*)idx, (float*)wt, s);
  });
}

// x, q, s, stream
PyObject* quantize(PyObject* const* a) {
  Rows x, q;
  void *sc, *s;
  if (!rows_of(a[0], &x) || float_type(x.type) < 0 || !rows_of(a[1], &q) || !is_codes(q.type) || q.rows != x.rows ||
      q.cols != x.cols || !whole(a[2], at::kFloat, {x.rows, blocks(x.cols)}, &sc) || !stream_here(a[3]))
    Py_RETURN_NONE;
  if (!stream_of(a[3], &s)) return nullptr;
  return call([&] {
    return moe_blockscale_quantize(x.p, float_type(x.type), x.ld, narrow(x.rows), narrow(x.cols), (uint8_t*)q.p, q.ld,
                                   (float*)sc, s);
  });
}

// xq, xs, wq, ws, y, workspace, stream
PyObject* matmul(PyObject* const* a) {
  Rows x, y;
  at::IntArrayRef w;
  void *xs, *wq, *ws, *work, *s;
  size_t work_bytes;
  if (!rows_of(a[0], &x) || !is_codes(x.type) || !rows_of(a[4], &y) || float_type(y.type) < 0 ||
      !shape_of(a[2], 2, &w) || y.rows != x.rows || y.cols != w[0])
    Py_RETURN_NONE;
  const int64_t N = w[0], K = x.cols;
  if (!whole(a[1], at::kFloat, {x.rows, blocks(K)}, &xs) || !whole(a[2], at::kByte, {N, K}, &wq) ||
      !whole(a[3], at::kFloat, {blocks(N), blocks(K)}, &ws) || !workspace_of(a[5], &work, &work_bytes) ||
      !stream_here(a[6]))
    Py_RETURN_NONE;
  if (!stream_of(a[6], &s)) return nullptr;
  return call([&] {
    return moe_blockscale_matmul((const uint8_t*)x.p, x.ld, (const float*)xs, narrow(x.rows), (const uint8_t*)wq,
                                 (const float*)ws, narrow(N), narrow(K), y.p, float_type(y.type), y.ld, work,
                                 work_bytes, s);
  });
}

// xq, xs, k, offsets, perm, w_gate, s_gate, w_up, s_up, hq, hs, stream
PyObject* gateup(PyObject* const* a) {
  const int64_t k = PyLong_AsLongLong(a[2]);
  if (k == -1 && PyErr_Occurred()) return nullptr;
  at::IntArrayRef x, w;
  if (!shape_of(a[0], 2, &x) || !shape_of(a[5], 3, &w) || k < 0 || k > INT_MAX || x[0] > INT_MAX) Py_RETURN_NONE;
  const int64_t T = x[0], d = x[1], E = w[0], f = w[1], R = T * k, DB = blocks(d), FB = blocks(f);
  void *xq, *xs, *offsets, *perm, *wg, *sg, *wu, *su, *hq, *hs, *s;
  if (!whole(a[0], at::kByte, {T, d}, &xq) || !whole(a[1], at::kFloat, {T, DB}, &xs) ||
      !whole(a[3], at::kInt, {E + 1}, &offsets) || !whole(a[4], at::kInt, {R}, &perm) ||
      !whole(a[5], at::kByte, {E, f, d}, &wg) || !whole(a[6], at::kFloat, {E, FB, DB}, &sg) ||
      !whole(a[7], at::kByte, {E, f, d}, &wu) || !whole(a[8], at::kFloat, {E, FB, DB}, &su) ||
      !whole(a[9], at::kByte, {R, f}, &hq) || !whole(a[10], at::kFloat, {R, FB}, &hs) ||
      !stream_here(a[11]))
    Py_RETURN_NONE;
  if (!stream_of(a[11], &s)) return nullptr;
  return call([&] {
    return moe_blockscale_gateup((const uint8_t*)xq, (const float*)xs, narrow(T), narrow(k), (const int32_t*)offsets,
                                 (const int32_t*)perm, narrow(E), (const uint8_t*)wg, (const float*)sg,
                                 (const uint8_t*)wu, (const float*)su, narrow(f), narrow(d), (uint8_t*)hq, (float*)hs,
                                 s);
  });
}

// hq, hs, wt, offsets, pos, w_down, s_down, y, workspace, add, stream
PyObject* down(PyObject* const* a) {
  at::IntArrayRef r, w;
  if (!shape_of(a[2], 2, &r) || !shape_of(a[5], 3, &w) || r[0] > INT_MAX || r[1] > INT_MAX) Py_RETURN_NONE;
  const int64_t T = r[0], k = r[1], E = w[0], d = w[1], f = w[2], R = T * k, DB = blocks(d), FB = blocks(f);
  void *hq, *hs, *wt, *offsets, *pos, *wd, *sd, *y, *work, *add = nullptr, *s;
  size_t work_bytes;
  if (!whole(a[0], at::kByte, {R, f}, &hq) || !whole(a[1], at::kFloat, {R, FB}, &hs) ||
      !whole(a[2], at::kFloat, {T, k}, &wt) || !whole(a[3], at::kInt, {E + 1}, &offsets) ||
      !whole(a[4], at::kInt, {R}, &pos) || !whole(a[5], at::kByte, {E, d, f}, &wd) ||
      !whole(a[6], at::kFloat, {E, DB, FB}, &sd) || !whole(a[7], at::kFloat, {T, d}, &y) ||
      !workspace_of(a[8], &work, &work_bytes) || (a[9] != Py_None && !whole(a[9], at::kFloat, {T, d}, &add)) ||
      !stream_here(a[10]))
    Py_RETURN_NONE;
  if (!stream_of(a[10], &s)) return nullptr;
  return call([&] {
    return moe_blockscale_down((const uint8_t*)hq, (const float*)hs, narrow(T), narrow(k), (const float*)wt,
                               (const int32_t*)offsets, (const int32_t*)pos, narrow(E), (const uint8_t*)wd,
                               (const float*)sd, narrow(d), narrow(f), (const float*)add, (float*)y, work, work_bytes,
                               s);
  });
}

#define ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<n, name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(gate_topk, 5), ENTRY(quantize, 4), ENTRY(matmul, 7), ENTRY(gateup, 12),
                         ENTRY(down, 11), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
