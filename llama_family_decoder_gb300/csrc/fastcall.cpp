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

// the keys of a paged cache, made once (PyDict_GetItemString makes a string each time)
PyObject *key_k, *key_v, *key_pages, *key_lens;

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
  // like: a cache whose page table and lens were looked at already, or null
  blk_paged_cache paged(PyObject* o, int64_t& batch, PyObject* like = nullptr, const blk_paged_cache* its = nullptr) {
    blk_paged_cache c{};
    if (!ok || !PyDict_Check(o)) {
      ok = false;
      return c;
    }
    void** const to[2] = {&c.k, &c.v};
    int64_t n_pages = -1, size = -1;
    for (int i = 0; i < 2; ++i) {
      PyObject* x = PyDict_GetItem(o, i ? key_v : key_k);
      const at::Tensor* t = x ? tensor(x, b->type) : fail();
      if (!t) return c;
      ok = t->dim() == 4 && t->is_contiguous() && (n_pages < 0 || t->size(0) == n_pages) && t->size(1) == b->Hkv &&
           (size < 0 || t->size(2) == size) && t->size(3) == b->d;
      if (!ok) return c;
      n_pages = t->size(0);
      size = t->size(2);
      *to[i] = t->data_ptr();
    }
    PyObject *x = PyDict_GetItem(o, key_pages), *y = PyDict_GetItem(o, key_lens);
    ok = n_pages <= INT32_MAX && size <= INT32_MAX;
    c.n_pages = static_cast<int>(n_pages);
    c.page_size = static_cast<int>(size);
    if (like && x && y && x == PyDict_GetItem(like, key_pages) && y == PyDict_GetItem(like, key_lens)) {
      c.pages = its->pages;
      c.lens = its->lens;
      c.max_pages = its->max_pages;
      return c;
    }
    const at::Tensor *p = x ? tensor(x, at::kInt) : fail(), *l = y ? tensor(y, at::kInt) : fail();
    if (!p || !l) return c;
    ok = p->dim() == 2 && p->is_contiguous() && l->dim() == 1 && l->is_contiguous() && l->size(0) == p->size(0) &&
         p->size(0) <= INT32_MAX && p->size(1) <= INT32_MAX;
    if (!ok) return c;
    batch = p->size(0);
    c.pages = static_cast<const int*>(p->data_ptr());
    c.lens = static_cast<int*>(l->data_ptr());
    c.max_pages = static_cast<int>(p->size(1));
    return c;
  }
  const float* probs(PyObject* o, int64_t& n, int64_t& vocab, int64_t& stride) {  // [n, vocab]; below 0: any, and set
    const at::Tensor* t = tensor(o, at::kFloat);
    if (!t || t->dim() != 2 || (n >= 0 && t->size(0) != n) || (vocab >= 0 && t->size(1) != vocab) ||
        (t->stride(1) != 1 && t->size(1) > 1)) {
      ok = false;
      return nullptr;
    }
    n = t->size(0);
    vocab = t->size(1);
    stride = t->stride(0);
    ok = n <= INT32_MAX && vocab <= INT32_MAX;
    return static_cast<const float*>(t->data_ptr());
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

// paged_append(block, cache, q, k, v, cu_seqlens, depths, q_gain, k_gain, rope_table, interleaved, q_out, host_lens_max)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 13) return none();
  try {
    Call c(a[0]);
    int64_t batch = -1, n = -1;
    const blk_paged_cache cache = c.paged(a[1], batch);
    const blk_head_rows q = c.rows(a[2], n, c.b ? c.b->H : 0);
    const blk_head_rows k = c.rows(a[3], n, c.b ? c.b->Hkv : 0), v = c.rows(a[4], n, c.b ? c.b->Hkv : 0);
    if (!c.ok) return none();
    const int *cu = c.ints(a[5], batch + 1), *depths = c.ints(a[6], n);
    const void *gq = nullptr, *gk = nullptr;
    if (c.b->qk_norm) {
      gq = c.contiguous(a[7], c.b->type, c.b->d);
      gk = c.contiguous(a[8], c.b->type, c.b->d);
    }
    const int inter = PyObject_IsTrue(a[10]);
    const long most = PyLong_AsLong(a[12]);
    if (inter < 0 || PyErr_Occurred()) return none();
    blk_rope_layout layout{nullptr, static_cast<int>(c.b->d), 0, inter};
    if (a[9] != Py_None) {
      const at::Tensor* t = c.tensor(a[9], at::kFloat);
      if (!t || t->dim() != 3 || !t->is_contiguous() || t->size(0) > INT32_MAX || t->size(1) > c.b->d || t->size(2) != 2)
        return none();
      layout = {t->data_ptr(), 2 * static_cast<int>(t->size(1)), static_cast<int>(t->size(0)), inter};
    }
    const bool plain = c.b->no_rope || (a[9] == Py_None && !inter);
    at::Tensor to;
    const blk_head_rows qo = c.out(a[11], n, c.b->H, to);
    if (!c.ok || most > INT32_MAX || most < INT32_MIN || !launched([&] {
          return blk_paged_append(c.b->h, &q, &k, &v, static_cast<int>(n), cu, depths, static_cast<int>(batch), &cache,
                                  plain ? nullptr : &layout, gq, gk, &qo, static_cast<int>(most), c.stream);
        }))
      return none();
    return given(a[11], to);
  } catch (...) {
    return none();
  }
}

// attn_paged(block, q, cache, cu_seqlens, parents, out)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 6) return none();
  try {
    Call c(a[0]);
    int64_t batch = -1, n = -1;
    const blk_paged_cache cache = c.paged(a[2], batch);
    const blk_head_rows q = c.rows(a[1], n, c.b ? c.b->H : 0);
    if (!c.ok) return none();
    const int *cu = c.ints(a[3], batch + 1), *parents = c.ints(a[4], n);
    at::Tensor to, ws;
    const blk_head_rows o = c.out(a[5], n, c.b->H, to);
    if (!c.ok) return none();
    const size_t bytes = blk_attn_paged_workspace_bytes(c.b->h, static_cast<int>(n), cu != nullptr, parents != nullptr,
                                                        static_cast<int>(batch), &cache);
    if (bytes) ws = c.scratch(bytes);
    if (!launched([&] {
          return blk_attn_paged(c.b->h, &q, static_cast<int>(n), cu, parents, static_cast<int>(batch), &cache, &o,
                                bytes ? ws.data_ptr() : nullptr, bytes, c.stream);
        }))
      return none();
    return given(a[5], to);
  } catch (...) {
    return none();
  }
}

// verify_drafts(block, target, tokens, u, u_next, cu_seqlens, parents, draft)
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 8) return none();
  try {
    Call c(a[0]);
    int64_t n = -1, vocab = -1, t_row = 0, d_row = 0;
    const float* target = c.probs(a[1], n, vocab, t_row);
    const float* draft = a[7] == Py_None ? nullptr : c.probs(a[7], n, vocab, d_row);
    const at::Tensor* last = c.tensor(a[4], at::kFloat);
    if (!c.ok || last->dim() != 1 || !last->is_contiguous() || last->numel() > INT32_MAX) return none();
    const int64_t batch = last->numel();
    const int* tokens = static_cast<const int*>(c.contiguous(a[2], at::kInt, n));
    const float* u = static_cast<const float*>(c.contiguous(a[3], at::kFloat, n));
    const int *cu = c.ints(a[5], batch + 1), *parents = c.ints(a[6], n);
    if (!c.ok) return none();
    const at::Tensor counts = c.fresh({batch}, at::kInt), path = c.fresh({n}, at::kInt), next = c.fresh({batch}, at::kInt);
    if (!launched([&] {
          return blk_verify_drafts(c.b->h, target, t_row, draft, d_row, static_cast<int>(n), static_cast<int>(vocab), tokens,
                                   parents, cu, u, static_cast<const float*>(last->data_ptr()), static_cast<int>(batch),
                                   static_cast<int*>(counts.data_ptr()), static_cast<int*>(path.data_ptr()),
                                   static_cast<int*>(next.data_ptr()), c.stream);
        }))
      return none();
    PyObject *x = THPVariable_Wrap(counts), *y = THPVariable_Wrap(path), *z = THPVariable_Wrap(next);
    PyObject* r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
  } catch (...) {
    return none();
  }
}

// paged_keep(block, caches, counts, path, cu_seqlens, starts): True, or None
PyObject* paged_keep(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 6) return none();
  try {
    Call c(a[0]);
    if (!c.ok || !PyList_Check(a[1]) || PyList_GET_SIZE(a[1]) < 1 || PyList_GET_SIZE(a[1]) > 256) return none();
    blk_paged_cache caches[256];
    const int n_caches = static_cast<int>(PyList_GET_SIZE(a[1]));
    int64_t batch = -1, n = 0;
    for (int i = 0; i < n_caches; ++i) {
      int64_t its = batch;
      caches[i] = i ? c.paged(PyList_GET_ITEM(a[1], i), its, PyList_GET_ITEM(a[1], 0), caches)
                    : c.paged(PyList_GET_ITEM(a[1], 0), its);
      if (!c.ok || (i && its != batch)) return none();
      batch = its;
    }
    const int* path = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor* t = c.tensor(a[3], at::kInt);
      if (!t || t->dim() != 1 || !t->is_contiguous() || t->numel() > INT32_MAX) return none();
      n = t->numel();
      path = static_cast<const int*>(t->data_ptr());
    }
    const int* counts = a[2] == Py_None ? nullptr : c.ints(a[2], batch);
    const int *cu = c.ints(a[4], batch + 1), *starts = c.ints(a[5], batch);
    if (!c.ok || !counts || !launched([&] {
          return blk_paged_keep(c.b->h, caches, n_caches, counts, path, cu, starts, static_cast<int>(batch),
                                static_cast<int>(n), c.stream);
        }))
      return none();
    Py_RETURN_TRUE;
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
                         fast("paged_append", paged_append),
                         fast("attn_paged", attn_paged),
                         fast("verify_drafts", verify_drafts),
                         fast("paged_keep", paged_keep),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
  key_k = PyUnicode_InternFromString("k");
  key_v = PyUnicode_InternFromString("v");
  key_pages = PyUnicode_InternFromString("pages");
  key_lens = PyUnicode_InternFromString("lens");
  return key_k && key_v && key_pages && key_lens ? PyModule_Create(&module) : nullptr;
}
