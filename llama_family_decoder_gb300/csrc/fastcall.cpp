// The packed calls' short way from Python: the checks, outputs and structs that binding.py
// makes for them, in compiled code. Calls on a few tokens take the GPU 2 to 8 us, so what the
// host does for them is what they cost: through binding.py a call in a row of such calls took
// 13 to 16 us, here 4.3 (norm and rotary of 64 tokens: 1.5 the launch, 2 the two outputs); a store
// with a load 23, here 6.5; decode attention 14, here 3.2 beside 8 on the GPU. Each function
// returns its outputs, or None for whatever is not a plain call that succeeds: then binding.py
// makes the call itself and says what is wrong with it. The kernels and their checks are those
// of the C ABI (blk.h) either way.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/blk.h"

namespace {

struct Block {
  blk_handle* h;
  int64_t H, Hkv, d;
  at::ScalarType type;
  int dev;
  bool qk_norm, no_rope;
};

// What a call borrows from its arguments; ok turns false at the first thing that is not plain.
struct Call {
  const Block* b = nullptr;
  bool ok = false;
  void* stream = nullptr;

  explicit Call(PyObject* capsule) {
    b = static_cast<const Block*>(PyCapsule_GetPointer(capsule, nullptr));
    if (!b) {
      PyErr_Clear();
      return;
    }
    ok = c10::cuda::current_device() == b->dev;
    if (ok) stream = c10::cuda::getCurrentCUDAStream(b->dev).stream();
  }
  const at::Tensor* tensor(PyObject* o, at::ScalarType type) {
    if (!ok || !THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.scalar_type() == type && t.is_cuda() && t.get_device() == b->dev && t.layout() == at::kStrided ? &t : fail();
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  // [n, heads, d]; n < 0: any, and set
  blk_head_rows rows(PyObject* o, int64_t& n, int64_t heads) {
    const at::Tensor* t = tensor(o, b ? b->type : at::kFloat);
    if (!t || t->dim() != 3 || (n >= 0 && t->size(0) != n) || t->size(1) != heads || t->size(2) != b->d || t->stride(2) != 1) {
      ok = false;
      return {};
    }
    n = t->size(0);
    ok = n <= INT32_MAX;
    return {t->data_ptr(), t->stride(0), t->stride(1)};
  }
  const void* contiguous(PyObject* o, at::ScalarType type, int64_t n) {  // [n]
    const at::Tensor* t = tensor(o, type);
    if (!t || t->dim() != 1 || !t->is_contiguous() || t->size(0) != n) return fail();
    return t->data_ptr();
  }
  const int* ints(PyObject* o, int64_t n) {  // None: null
    return o == Py_None ? nullptr : static_cast<const int*>(contiguous(o, at::kInt, n));
  }
  // torch.empty without its dispatch
  at::Tensor fresh(at::IntArrayRef size, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, static_cast<at::DeviceIndex>(b->dev)), std::nullopt));
  }
  at::Tensor make(int64_t n, int64_t heads) const {
    return fresh({n, heads, b->d}, b->type);
  }
  // an output: the given tensor, or a new one (kept in `made`)
  blk_head_rows out(PyObject* o, int64_t n, int64_t heads, at::Tensor& made) {
    if (!ok) return {};
    if (o != Py_None) return rows(o, n, heads);
    made = make(n, heads);
    return {made.data_ptr(), heads * b->d, b->d};
  }
  at::Tensor scratch(size_t bytes) const {
    return fresh({static_cast<int64_t>(bytes)}, at::kByte);
  }
  blk_kv4_cache cache(PyObject* o, int64_t& batch) {
    blk_kv4_cache c{};
    if (!ok || !PyDict_Check(o)) {
      ok = false;
      return c;
    }
    static const char* const names[5] = {"k", "k_scale", "v", "v_scale", "lens"};
    void** const to[4] = {&c.k, &c.k_scale, &c.v, &c.v_scale};
    int64_t cap = -1;
    batch = -1;
    for (int i = 0; i < 4 && ok; ++i) {
      PyObject* x = PyDict_GetItemString(o, names[i]);
      const at::Tensor* t = x ? tensor(x, i % 2 ? at::kBFloat16 : at::kByte) : fail();
      if (!t) return c;
      ok = t->dim() == 4 && t->is_contiguous() && (batch < 0 || t->size(0) == batch) && t->size(1) == b->Hkv &&
           (cap < 0 || t->size(2) == cap) && t->size(3) == (i % 2 ? 8 : 64);
      if (!ok) return c;
      batch = t->size(0);
      cap = t->size(2);
      *to[i] = t->data_ptr();
    }
    PyObject* x = PyDict_GetItemString(o, names[4]);
    const at::Tensor* t = x ? tensor(x, at::kInt) : fail();
    if (!t) return c;
    ok = t->dim() == 1 && t->size(0) == batch && t->is_contiguous() && cap <= INT32_MAX && batch <= INT32_MAX;
    c.lens = ok ? static_cast<int*>(t->data_ptr()) : nullptr;
    c.capacity = static_cast<int>(cap);
    return c;
  }
};

PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// A launch waits when the GPU's queue is full: other threads have the interpreter meanwhile. It is
// taken back before anything here goes on, also when the call throws (a message that finds no memory).
struct WithoutInterpreter {
  PyThreadState* const t = PyEval_SaveThread();
  ~WithoutInterpreter() { PyEval_RestoreThread(t); }
};
template <class F>
bool launched(F call) {
  const WithoutInterpreter scope;
  return call() == BLK_OK;
}

PyObject* given(PyObject* o, const at::Tensor& made) {
  if (o == Py_None) return THPVariable_Wrap(made);
  Py_INCREF(o);
  return o;
}

PyObject* pair(PyObject* a, const at::Tensor& ta, PyObject* b, const at::Tensor& tb) {
  PyObject *x = given(a, ta), *y = x ? given(b, tb) : nullptr;
  PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// block(handle, n_heads, n_kv_heads, head_dim, bf16, device, qk_norm, no_rope)
PyObject* block(PyObject*, PyObject* args) {
  unsigned long long h;
  int H, Hkv, d, bf16, dev, qk_norm, no_rope;
  if (!PyArg_ParseTuple(args, "Kiiiiiii", &h, &H, &Hkv, &d, &bf16, &dev, &qk_norm, &no_rope)) return nullptr;
  Block* b = new Block{reinterpret_cast<blk_handle*>(static_cast<uintptr_t>(h)), H, Hkv, d, bf16 ? at::kBFloat16 : at::kFloat,
                       dev, qk_norm != 0, no_rope != 0};
  return PyCapsule_New(b, nullptr, [](PyObject* c) { delete static_cast<Block*>(PyCapsule_GetPointer(c, nullptr)); });
}

// qk_norm_rope(block, q, k, positions, q_gain, k_gain, sections, interleaved, q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 10) return none();
  try {
    Call c(a[0]);
    int64_t n = -1;
    const blk_head_rows q = c.rows(a[1], n, c.b ? c.b->H : 0), k = c.rows(a[2], n, c.b ? c.b->Hkv : 0);
    if (!c.ok) return none();
    blk_rope_axes axes{};
    const int* pos = nullptr;
    const bool with_axes = !c.b->no_rope && a[6] != Py_None;
    if (!c.b->no_rope) {
      axes.n_axes = 1;
      if (with_axes) {
        if (!PyList_Check(a[6]) && !PyTuple_Check(a[6])) return none();
        axes.n_axes = static_cast<int>(PySequence_Fast_GET_SIZE(a[6]));
        if (axes.n_axes < 1 || axes.n_axes > 4) return none();
        for (int i = 0; i < axes.n_axes; ++i) {
          const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(a[6], i));
          if (PyErr_Occurred()) PyErr_Clear();  // then x is -1, and refused
          if (x < 0 || x > INT32_MAX) return none();
          axes.sections[i] = static_cast<int>(x);
        }
        const int inter = PyObject_IsTrue(a[7]);
        if (inter < 0) return none();
        axes.interleaved = inter;
      }
      const at::Tensor* t = c.tensor(a[3], at::kInt);
      if (!t || !t->is_contiguous() || !(t->dim() == 2 ? t->size(0) == axes.n_axes && t->size(1) == n
                                                       : t->dim() == 1 && axes.n_axes == 1 && t->size(0) == n))
        return none();
      pos = static_cast<const int*>(t->data_ptr());
    }
    const void *gq = nullptr, *gk = nullptr;
    if (c.b->qk_norm) {
      gq = c.contiguous(a[4], c.b->type, c.b->d);
      gk = c.contiguous(a[5], c.b->type, c.b->d);
    }
    at::Tensor tq, tk;
    const blk_head_rows qo = c.out(a[8], n, c.b->H, tq), ko = c.out(a[9], n, c.b->Hkv, tk);
    if (!c.ok || !launched([&] {
          return blk_qk_norm_rope(c.b->h, &q, &k, static_cast<int>(n), pos, with_axes ? &axes : nullptr, gq, gk, &qo, &ko,
                                  c.stream);
        }))
      return none();
    return pair(a[8], tq, a[9], tk);
  } catch (...) {
    return none();
  }
}

// attn_packed(block, q, k, v, cu_seqlens, out)
PyObject* attn_packed(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 6) return none();
  try {
    Call c(a[0]);
    int64_t n = -1;
    const blk_head_rows q = c.rows(a[1], n, c.b ? c.b->H : 0);
    const blk_head_rows k = c.rows(a[2], n, c.b ? c.b->Hkv : 0), v = c.rows(a[3], n, c.b ? c.b->Hkv : 0);
    const at::Tensor* cu = c.tensor(a[4], at::kInt);
    if (!c.ok || cu->dim() != 1 || !cu->is_contiguous() || cu->numel() < 1 || cu->numel() > INT32_MAX) return none();
    const int batch = static_cast<int>(cu->numel() - 1);
    at::Tensor to, ws;
    const blk_head_rows o = c.out(a[5], n, c.b->H, to);
    if (!c.ok) return none();
    const size_t bytes = blk_attn_packed_workspace_bytes(c.b->h, static_cast<int>(n), batch);
    if (bytes) ws = c.scratch(bytes);
    if (!launched([&] {
          return blk_attn_packed(c.b->h, &q, &k, &v, static_cast<int>(n), static_cast<const int*>(cu->data_ptr()), batch, &o,
                                 bytes ? ws.data_ptr() : nullptr, bytes, c.stream);
        }))
      return none();
    return given(a[5], to);
  } catch (...) {
    return none();
  }
}

// kv4_store(block, cache, k, v, cu_seqlens, starts, host_lens_max): True, or None
PyObject* kv4_store(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 7) return none();
  try {
    Call c(a[0]);
    int64_t batch = -1, n = -1;
    const blk_kv4_cache cache = c.cache(a[1], batch);
    const blk_head_rows k = c.rows(a[2], n, c.b ? c.b->Hkv : 0), v = c.rows(a[3], n, c.b ? c.b->Hkv : 0);
    const int* cu = c.ints(a[4], batch + 1);
    const int* starts = c.ints(a[5], batch);
    const long most = PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) return none();
    if (!c.ok || most > INT32_MAX || most < INT32_MIN || !launched([&] {
          return blk_kv4_store(c.b->h, &k, &v, static_cast<int>(n), cu, starts, static_cast<int>(batch), &cache,
                               static_cast<int>(most), c.stream);
        }))
      return none();
    Py_RETURN_TRUE;
  } catch (...) {
    return none();
  }
}

// kv4_load(block, cache, cu_seqlens, rows, starts, k_out, v_out)
PyObject* kv4_load(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 7) return none();
  try {
    Call c(a[0]);
    int64_t batch = -1;
    const blk_kv4_cache cache = c.cache(a[1], batch);
    const int* cu = c.ints(a[2], batch + 1);
    const int* starts = c.ints(a[4], batch);
    int64_t n = batch;
    if (a[3] == Py_None) {
      if (a[2] != Py_None) return none();  // packed rows, but how many?
    } else {
      n = PyLong_AsLong(a[3]);
      if (PyErr_Occurred()) PyErr_Clear();  // then n is -1, and refused
    }
    if (!c.ok || n < 0 || n > INT32_MAX) return none();
    at::Tensor tk, tv;
    const blk_head_rows k = c.out(a[5], n, c.b->Hkv, tk), v = c.out(a[6], n, c.b->Hkv, tv);
    if (!c.ok || !launched([&] {
          return blk_kv4_load(c.b->h, &cache, cu, starts, static_cast<int>(batch), static_cast<int>(n), &k, &v, c.stream);
        }))
      return none();
    return pair(a[5], tk, a[6], tv);
  } catch (...) {
    return none();
  }
}

// attn_decode_kv4(block, q, cache, out)
PyObject* attn_decode_kv4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 4) return none();
  try {
    Call c(a[0]);
    int64_t batch = -1;
    const blk_kv4_cache cache = c.cache(a[2], batch);
    const blk_head_rows q = c.rows(a[1], batch, c.b ? c.b->H : 0);
    at::Tensor to, ws;
    if (!c.ok) return none();
    const blk_head_rows o = c.out(a[3], batch, c.b->H, to);
    if (!c.ok) return none();
    const size_t bytes = blk_attn_decode_kv4_workspace_bytes(c.b->h, static_cast<int>(batch), cache.capacity);
    if (bytes) ws = c.scratch(bytes);
    if (!launched([&] {
          return blk_attn_decode_kv4(c.b->h, &q, &cache, static_cast<int>(batch), &o, bytes ? ws.data_ptr() : nullptr, bytes,
                                     c.stream);
        }))
      return none();
    return given(a[3], to);
  } catch (...) {
    return none();
  }
}

typedef PyObject* (*Fast)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef fast(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {{"block", block, METH_VARARGS, nullptr},
                         fast("qk_norm_rope", qk_norm_rope),
                         fast("attn_packed", attn_packed),
                         fast("kv4_store", kv4_store),
                         fast("kv4_load", kv4_load),
                         fast("attn_decode_kv4", attn_decode_kv4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
