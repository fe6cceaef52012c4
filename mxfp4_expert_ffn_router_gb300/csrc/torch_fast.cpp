// torch_fast.cpp -- the binding's short way into the decoder layer's calls.
//
// A decode step makes these calls back to back with kernels of 2 to 4 us, so the host's
// time per call is what a small batch waits for: checking the tensors attribute by attribute
// from Python and going through ctypes took 5.7 us of an RMS norm call whose launch
// itself takes 1.8 (GB300's host).  Each function here takes the Python arguments by
// position, checks the same things (dtype, shape, device, packing) on the tensors directly
// and calls the C ABI; it returns the status, or None when an argument is not acceptable:
// the Python function then says which and why.  No exception leaves it.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/k3moe.h"

namespace {

using RmsnormFn = decltype(&k3moe_rmsnorm);
using WriteFn = decltype(&k3moe_kv_write);
using ReadFn = decltype(&k3moe_kv_read);
using AttnFn = decltype(&k3moe_attn_decode);
using AppendFn = decltype(&k3moe_kv_append);
using ExtendFn = decltype(&k3moe_attn_extend);
using TreeFn = decltype(&k3moe_attn_tree);
RmsnormFn g_rmsnorm;
WriteFn g_write;
ReadFn g_read;
AttnFn g_attn;
AppendFn g_append;
ExtendFn g_extend;
TreeFn g_tree;

enum Kind { kBf16, kCodes, kScales, kI32, kI64, kF32, kAny };

bool is_kind(const at::Tensor &t, Kind k) {
  const auto s = t.scalar_type();
  switch (k) {
    case kBf16: return s == at::kBFloat16 || s == at::kShort;
    case kCodes: return s == at::kByte || s == at::kFloat8_e4m3fn;
    case kScales: return s == at::kByte || s == at::kFloat8_e8m0fnu;
    case kI32: return s == at::kInt;
    case kI64: return s == at::kLong;
    case kF32: return s == at::kFloat;
    default: return true;
  }
}

// A packed CUDA tensor (or None) of the kind and, unless null, the shape; its pointer, null if empty.
bool packed(PyObject *o, Kind k, const at::IntArrayRef *shape, void **p) {
  *p = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda() || !is_kind(t, k) || !t.is_contiguous() || (shape && t.sizes() != *shape)) return false;
  if (t.numel()) *p = t.data_ptr();
  return true;
}

// Tokens' vectors [n, heads, dim], packed but for the first axis.
bool rows(PyObject *o, const at::IntArrayRef &shape, void **p, int64_t *stride) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda() || !is_kind(t, kBf16) || t.sizes() != shape) return false;
  *p = nullptr;
  *stride = shape[1] * shape[2];
  if (shape[0] == 0) return true;
  if (t.stride(2) != 1 || (shape[1] > 1 && t.stride(1) != shape[2])) return false;
  *p = t.data_ptr();
  if (shape[0] > 1) *stride = t.stride(0);
  return true;
}

const at::Tensor *tensor(PyObject *o, int64_t dim) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor &t = THPVariable_Unpack(o);
  return t.dim() == dim ? &t : nullptr;
}

// None: the current stream; a number: a stream's handle.
bool stream_of(PyObject *o, k3moe_stream_t *s) {
  if (o == Py_None) {
    *s = reinterpret_cast<k3moe_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    return true;
  }
  *s = static_cast<k3moe_stream_t>(PyLong_AsVoidPtr(o));
  return !PyErr_Occurred();
}

bool small(int64_t v) { return v >= 0 && v <= INT32_MAX; }

template <class F>
PyObject *guarded(F f) {
  try {
    int rc = 0;
    if (f(rc)) return PyLong_FromLong(rc);
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

uint16_t *u16(void *p) { return static_cast<uint16_t *>(p); }

// x, weight, eps, residual, residual_out, y, codes, scales, stream
PyObject *fast_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&](int &rc) {
    if (n != 9) return false;
    const at::Tensor *x = tensor(a[0], 2);
    if (!x || !small(x->size(0)) || !small(x->size(1))) return false;
    const at::IntArrayRef shape = x->sizes();
    const int64_t T = shape[0], H = shape[1], sc[2] = {T, H / 32};
    const at::IntArrayRef wshape(&H, 1), sshape(sc, 2);
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) return false;
    void *px, *pw, *pr, *po, *py, *pc, *ps;
    k3moe_stream_t st;
    if (!packed(a[0], kBf16, &shape, &px) || !packed(a[1], kBf16, &wshape, &pw) || !packed(a[3], kBf16, &shape, &pr) ||
        !packed(a[4], kBf16, &shape, &po) || !packed(a[5], kBf16, &shape, &py) || !packed(a[6], kCodes, &shape, &pc) ||
        !packed(a[7], kScales, &sshape, &ps) || !stream_of(a[8], &st))
      return false;
    rc = g_rmsnorm(static_cast<int32_t>(T), static_cast<int32_t>(H), u16(px), u16(pr), u16(pw), static_cast<float>(eps),
                   u16(po), u16(py), static_cast<uint8_t *>(pc), static_cast<uint8_t *>(ps), st);
    return true;
  });
}

// cache address, k, v, slots, dev_status, stream
PyObject *fast_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&](int &rc) {
    if (n != 6) return false;
    const auto *c = static_cast<const k3moe_kv_cache *>(PyLong_AsVoidPtr(a[0]));
    const at::Tensor *s = tensor(a[3], 1);
    if (!c || !s || !small(s->size(0))) return false;
    const int64_t sh[3] = {s->size(0), c->heads, c->dim};
    const at::IntArrayRef shape(sh, 3);
    void *pk, *pv, *ps, *pd;
    int64_t ks, vs;
    k3moe_stream_t st;
    if (!rows(a[1], shape, &pk, &ks) || !rows(a[2], shape, &pv, &vs) || !packed(a[3], kI32, nullptr, &ps) ||
        !packed(a[4], kI32, nullptr, &pd) || !stream_of(a[5], &st))
      return false;
    rc = g_write(c, static_cast<int32_t>(sh[0]), u16(pk), u16(pv), ks, vs, static_cast<int32_t *>(ps),
                 static_cast<int32_t *>(pd), st);
    return true;
  });
}

// cache address, slots, k, v, dev_status, stream
PyObject *fast_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&](int &rc) {
    if (n != 6) return false;
    const auto *c = static_cast<const k3moe_kv_cache *>(PyLong_AsVoidPtr(a[0]));
    const at::Tensor *s = tensor(a[1], 1);
    if (!c || !s || !small(s->size(0))) return false;
    const int64_t sh[3] = {s->size(0), c->heads, c->dim};
    const at::IntArrayRef shape(sh, 3);
    void *pk, *pv, *ps, *pd;
    k3moe_stream_t st;
    if (!packed(a[1], kI32, nullptr, &ps) || !packed(a[2], kBf16, &shape, &pk) || !packed(a[3], kBf16, &shape, &pv) ||
        !packed(a[4], kI32, nullptr, &pd) || !stream_of(a[5], &st) || a[2] == Py_None || a[3] == Py_None)
      return false;
    rc = g_read(c, static_cast<int32_t>(sh[0]), static_cast<int32_t *>(ps), u16(pk), u16(pv), static_cast<int32_t *>(pd),
                st);
    return true;
  });
}

// cache address, q, block_table, seq_lens, out, lse, scale, window, ws, dev_status, stream
PyObject *fast_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&](int &rc) {
    if (n != 11) return false;
    const auto *c = static_cast<const k3moe_kv_cache *>(PyLong_AsVoidPtr(a[0]));
    const at::Tensor *q = tensor(a[1], 3), *table = tensor(a[2], 2);
    if (!c || !q || !table || !small(q->size(0)) || !small(q->size(1)) || !small(table->size(1))) return false;
    const int64_t B = q->size(0), Hq = q->size(1), sh[3] = {B, Hq, c->dim}, ts[2] = {B, table->size(1)};
    const at::IntArrayRef shape(sh, 3), tshape(ts, 2), bshape(sh, 1), lshape(sh, 2);
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) return false;
    const long window = PyLong_AsLong(a[7]);
    if ((window == -1 && PyErr_Occurred()) || window > INT32_MAX || window < INT32_MIN) return false;
    void *pq, *pt, *pl, *po, *pe, *pw, *pd;
    int64_t qs;
    k3moe_stream_t st;
    if (!rows(a[1], shape, &pq, &qs) || !packed(a[2], kI32, &tshape, &pt) || !packed(a[3], kI32, &bshape, &pl) ||
        !packed(a[4], kBf16, &shape, &po) || !packed(a[5], kF32, &lshape, &pe) || !packed(a[8], kAny, nullptr, &pw) ||
        !packed(a[9], kI32, nullptr, &pd) || !stream_of(a[10], &st))
      return false;
    const size_t bytes = pw ? THPVariable_Unpack(a[8]).nbytes() : 0;
    rc = g_attn(c, static_cast<int32_t>(B), static_cast<int32_t>(Hq), u16(pq), qs, static_cast<int32_t *>(pt),
                static_cast<int32_t>(ts[1]), static_cast<int32_t *>(pl), static_cast<int32_t>(window),
                static_cast<float>(scale), u16(po), static_cast<float *>(pe), pw, bytes, static_cast<int32_t *>(pd), st);
    return true;
  });
}

// A count that Python holds, cut to what the library can tell apart: no place is larger, and none below 0 is allowed.
bool count_of(PyObject *o, int32_t *v) {
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &over);
  if (x == -1 && !over && PyErr_Occurred()) return false;
  *v = over > 0 || x > INT32_MAX ? INT32_MAX : over < 0 || x < -1 ? -1 : static_cast<int32_t>(x);
  return true;
}

// cache address, k, v, slots, positions, rotation address, q, q_out, dev_status, stream
PyObject *fast_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&](int &rc) {
    if (n != 10) return false;
    const auto *c = static_cast<const k3moe_kv_cache *>(PyLong_AsVoidPtr(a[0]));
    const auto *r = static_cast<const k3moe_rotation *>(PyLong_AsVoidPtr(a[5]));
    const at::Tensor *s = tensor(a[3], 1);
    if (!c || !r || !s || !small(s->size(0))) return false;
    const int64_t sh[3] = {s->size(0), c->heads, c->dim};
    const at::IntArrayRef shape(sh, 3), one(sh, 1);
    void *pk, *pv, *ps, *pp, *pd, *pq = nullptr, *po = nullptr;
    int64_t ks, vs, qs = 0, os = 0, qsh[3] = {sh[0], 0, c->dim};
    k3moe_stream_t st;
    if (!rows(a[1], shape, &pk, &ks) || !rows(a[2], shape, &pv, &vs) || !packed(a[3], kI32, nullptr, &ps) ||
        a[4] == Py_None || !packed(a[4], kI32, &one, &pp) || !packed(a[8], kI32, nullptr, &pd) || !stream_of(a[9], &st))
      return false;
    if (a[6] != Py_None || a[7] != Py_None) {
      const at::Tensor *q = tensor(a[6], 3);
      if (!q || !small(q->size(1))) return false;
      qsh[1] = q->size(1);
      const at::IntArrayRef qshape(qsh, 3);
      if (!rows(a[6], qshape, &pq, &qs) || !rows(a[7], qshape, &po, &os)) return false;
    }
    rc = g_append(c, static_cast<int32_t>(sh[0]), static_cast<int32_t>(qsh[1]), u16(pq), u16(pk), u16(pv), qs, ks, vs,
                  static_cast<int32_t *>(ps), static_cast<int32_t *>(pp), r, u16(po), os, static_cast<int32_t *>(pd), st);
    return true;
  });
}

// cache address, q, q_offsets, masks (or None), block_table, seq_lens, out, lse, scale, window, sinks, max_new (or None), ws,
// dev_status, stream
PyObject *fast_extend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&](int &rc) {
    if (n != 15) return false;
    const auto *c = static_cast<const k3moe_kv_cache *>(PyLong_AsVoidPtr(a[0]));
    const at::Tensor *q = tensor(a[1], 3), *table = tensor(a[4], 2);
    if (!c || !q || !table || !small(q->size(0)) || !small(q->size(1)) || !small(table->size(0)) || !small(table->size(1)))
      return false;
    const int64_t B = table->size(0), sh[3] = {q->size(0), q->size(1), c->dim}, osz = B + 1;
    const at::IntArrayRef shape(sh, 3), lshape(sh, 2), tshape = table->sizes(), bshape(&B, 1), oshape(&osz, 1);
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) return false;
    int32_t window, sinks, most = static_cast<int32_t>(sh[0]);
    if (!count_of(a[9], &window) || !count_of(a[10], &sinks) || (a[11] != Py_None && !count_of(a[11], &most))) return false;
    void *pq, *pf, *pm = nullptr, *pt, *pl, *po, *pe, *pw, *pd;
    int64_t qs, msh[2] = {sh[0], 0};
    k3moe_stream_t st;
    if (!rows(a[1], shape, &pq, &qs) || a[2] == Py_None || !packed(a[2], kI32, &oshape, &pf) ||
        !packed(a[4], kI32, &tshape, &pt) || a[5] == Py_None || !packed(a[5], kI32, &bshape, &pl) || a[6] == Py_None ||
        !packed(a[6], kBf16, &shape, &po) || !packed(a[7], kF32, &lshape, &pe) || !packed(a[12], kAny, nullptr, &pw) ||
        !packed(a[13], kI32, nullptr, &pd) || !stream_of(a[14], &st))
      return false;
    const size_t bytes = pw ? THPVariable_Unpack(a[12]).nbytes() : 0;
    const auto i32 = [](void *p) { return static_cast<int32_t *>(p); };
    if (a[3] != Py_None) {
      const at::Tensor *m = tensor(a[3], 2);
      if (!m || !small(m->size(1))) return false;
      msh[1] = m->size(1);
      const at::IntArrayRef mshape(msh, 2);
      if (!packed(a[3], kI64, &mshape, &pm)) return false;
      rc = g_tree(c, static_cast<int32_t>(B), static_cast<int32_t>(sh[0]), static_cast<int32_t>(sh[1]), u16(pq), qs, i32(pf),
                  static_cast<int64_t *>(pm), static_cast<int32_t>(msh[1]), i32(pt), static_cast<int32_t>(tshape[1]), i32(pl),
                  window, sinks, static_cast<float>(scale), u16(po), static_cast<float *>(pe), pw, bytes, i32(pd), st);
    } else {
      rc = g_extend(c, static_cast<int32_t>(B), static_cast<int32_t>(sh[0]), static_cast<int32_t>(sh[1]), u16(pq), qs,
                    i32(pf), most, i32(pt), static_cast<int32_t>(tshape[1]), i32(pl), window, sinks,
                    static_cast<float>(scale), u16(po), static_cast<float *>(pe), pw, bytes, i32(pd), st);
    }
    return true;
  });
}

// Addresses of the library's k3moe_rmsnorm, k3moe_kv_write, k3moe_kv_read, k3moe_attn_decode, k3moe_kv_append,
// k3moe_attn_extend, k3moe_attn_tree.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind: seven addresses");
    return nullptr;
  }
  void *p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_rmsnorm = reinterpret_cast<RmsnormFn>(p[0]);
  g_write = reinterpret_cast<WriteFn>(p[1]);
  g_read = reinterpret_cast<ReadFn>(p[2]);
  g_attn = reinterpret_cast<AttnFn>(p[3]);
  g_append = reinterpret_cast<AppendFn>(p[4]);
  g_extend = reinterpret_cast<ExtendFn>(p[5]);
  g_tree = reinterpret_cast<TreeFn>(p[6]);
  Py_RETURN_NONE;
}

#define K3_DEF(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {K3_DEF("bind", bind), K3_DEF("rmsnorm", fast_rmsnorm), K3_DEF("kv_write", fast_write),
                           K3_DEF("kv_read", fast_read), K3_DEF("attn_decode", fast_attn),
                           K3_DEF("kv_append", fast_append), K3_DEF("attn_extend", fast_extend),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_k3torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__k3torch() { return PyModule_Create(&g_module); }
