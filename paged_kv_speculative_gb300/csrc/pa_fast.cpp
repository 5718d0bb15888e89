// The binding's short way into the prompt-side calls of the C ABI: checks the tensors and makes the call in one step.
//
// These calls take few microseconds on the device, and reading some fifty attributes of a dozen tensors from Python takes
// longer. A function here returns what its Python counterpart in pa_verify.py returns; None when anything is not as the
// plain case has it (types, shapes, strides, devices), and the Python code then says what, or goes its longer way (another
// current device); or a negative status of the C ABI. Nothing is decided here that the Python code does not decide alike.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <memory>
#include <vector>

#include "../../include/pa_verify.h"

namespace {

// Addresses of the C ABI's functions, handed over by init: this module does not link the library.
struct Api {
  decltype(&pa_rope_write) rope;
  decltype(&pa_chunk_attention) chunk;
  decltype(&pa_pages_fork) fork;
  decltype(&pa_pages_resize) resize;
  decltype(&pa_pages_compact) compact;
  decltype(&pa_pages_copy) copy;
};
Api api{};

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }
bool plain(const at::Tensor& t, int dev, at::ScalarType type) { return t.scalar_type() == type && on(t, dev) && t.is_contiguous(); }
bool vec(const at::Tensor* t, int dev, at::ScalarType type, int64_t n) {
  return t && t->dim() == 1 && t->size(0) == n && plain(*t, dev, type);
}

// Elements between the tokens of a [T, heads, D] bf16 tensor whose heads are contiguous and whose tokens do not overlap; -1: it is none.
int64_t rows(const at::Tensor* t) {
  if (!t || t->dim() != 3 || t->scalar_type() != at::kBFloat16 || !t->is_cuda()) return -1;
  if (t->stride(2) != 1 || (t->size(1) > 1 && t->stride(1) != t->size(2))) return -1;
  const int64_t row = t->size(1) * t->size(2);
  if (t->size(0) <= 1) return row;
  return t->stride(0) >= row ? t->stride(0) : -1;  // an expanded tensor's 0 would mean contiguous
}

struct Caches {
  void *k, *v;
  float *ks, *vs;
  int64_t pages;
};
bool caches(PyObject* k_, PyObject* v_, PyObject* ks_, PyObject* vs_, int dev, bool fp8, int64_t hkv, int64_t d, Caches* c) {
  const at::Tensor *k = tensor(k_), *v = tensor(v_);
  if (!k || !v || k->dim() != 4 || v->sizes() != k->sizes()) return false;
  auto typed = [&](const at::Tensor& t) {
    return fp8 ? t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn : t.scalar_type() == at::kBFloat16;
  };
  if (k->size(1) != hkv || k->size(2) != 16 || k->size(3) != d || !typed(*k) || !typed(*v)) return false;
  if (!on(*k, dev) || !on(*v, dev) || !k->is_contiguous() || !v->is_contiguous()) return false;
  *c = Caches{k->data_ptr(), v->data_ptr(), nullptr, nullptr, k->size(0)};
  if (!fp8) return true;
  const at::Tensor *ks = tensor(ks_), *vs = tensor(vs_);
  const int64_t n = c->pages * hkv * 16;
  if (!ks || !vs || !plain(*ks, dev, at::kFloat) || !plain(*vs, dev, at::kFloat) || ks->numel() != n || vs->numel() != n) return false;
  c->ks = static_cast<float*>(ks->data_ptr());
  c->vs = static_cast<float*>(vs->data_ptr());
  return true;
}

template <typename T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
pa_stream_t stream_of(int dev) { return reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream()); }
bool current(int dev) { return c10::cuda::current_device() == dev; }
at::Tensor ints(at::IntArrayRef shape, const at::Tensor& like) { return at::empty(shape, like.options().dtype(at::kInt)); }

// body() returns a new reference; C++ exceptions become the Python ones that torch makes of them (OutOfMemoryError, ...)
template <typename F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  return body();
  END_HANDLE_TH_ERRORS
}
PyObject* none() { Py_RETURN_NONE; }

PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "init takes six addresses");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  api = Api{reinterpret_cast<decltype(api.rope)>(p[0]),   reinterpret_cast<decltype(api.chunk)>(p[1]),
            reinterpret_cast<decltype(api.fork)>(p[2]),   reinterpret_cast<decltype(api.resize)>(p[3]),
            reinterpret_cast<decltype(api.compact)>(p[4]), reinterpret_cast<decltype(api.copy)>(p[5])};
  return none();
}

// q, k, v, positions, inv_freq, pair_axis, slots, k_cache, v_cache, k_scale, v_scale, kv_dtype, q_out, pairs, error_flags
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 15) return none();
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *pos = tensor(a[3]), *freq = tensor(a[4]), *axis = tensor(a[5]),
                     *slots = tensor(a[6]);
    const int64_t qs = rows(q), ks = rows(k), vs = rows(v);
    if (qs < 0 || ks < 0 || vs < 0 || !pos || !freq || !axis || !slots) return none();
    const int dev = q->get_device();
    const int64_t t = q->size(0), hq = q->size(1), d = q->size(2), hkv = k->size(1), half = freq->numel();
    if (!current(dev) || !on(*k, dev) || !on(*v, dev) || k->size(0) != t || k->size(2) != d || v->sizes() != k->sizes()) return none();
    if (pos->dim() != 2 || pos->size(1) != t || !plain(*pos, dev, at::kInt) || !vec(freq, dev, at::kDouble, half) ||
        !vec(axis, dev, at::kInt, half) || !vec(slots, dev, at::kLong, t))
      return none();
    const long kv = PyLong_AsLong(a[11]), pairs = PyLong_AsLong(a[13]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    Caches c;
    if (!caches(a[7], a[8], a[9], a[10], dev, kv == PA_KV_FP8_E4M3, hkv, d, &c)) return none();
    uint32_t* flags = nullptr;
    if (a[14] != Py_None) {
      const at::Tensor* e = tensor(a[14]);
      if (!e || !on(*e, dev) || e->element_size() != 4) return none();
      flags = ptr<uint32_t>(*e);
    }
    at::Tensor made;
    const at::Tensor* out = nullptr;
    if (a[12] != Py_None) {
      out = tensor(a[12]);
      if (!out || !on(*out, dev) || out->sizes() != q->sizes()) return none();
    } else {
      made = at::empty(q->sizes(), q->options());
      out = &made;
    }
    const int64_t os = rows(out);
    if (os < 0) return none();
    const pa_rope_desc desc{static_cast<int32_t>(t), static_cast<int32_t>(hq), static_cast<int32_t>(hkv), static_cast<int32_t>(d),
                            static_cast<int32_t>(2 * half), static_cast<int32_t>(pos->size(0)), static_cast<int32_t>(pairs),
                            static_cast<int32_t>(kv), static_cast<int32_t>(c.pages), qs, ks, vs, os};
    const int rc = api.rope(&desc, q->data_ptr(), k->data_ptr(), v->data_ptr(), ptr<int32_t>(*pos), ptr<double>(*freq), ptr<int32_t>(*axis),
                            ptr<int64_t>(*slots), out->data_ptr(), c.k, c.v, c.ks, c.vs, flags, stream_of(dev));
    if (rc != PA_OK) return PyLong_FromLong(rc);
    if (a[12] != Py_None) {
      Py_INCREF(a[12]);
      return a[12];
    }
    return THPVariable_Wrap(std::move(made));
  });
}

// (hq, hkv, d, kv_dtype, num_pages, table stride, max_seqs, sm_count, workspace, its bytes, device), q, k_cache, v_cache, k_scale,
// v_scale, block_table, context_lens, query_lens, softmax_scale, out
PyObject* chunk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 11) return none();
    long long f[11];
    for (int i = 0; i < 11; ++i) f[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a[0], i));
    const double scale = PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    const int dev = static_cast<int>(f[10]);
    const at::Tensor *q = tensor(a[1]), *table = tensor(a[6]), *ctx = tensor(a[7]), *ql = tensor(a[8]);
    const int64_t qs = rows(q);
    if (qs < 0 || !table || !ctx || !ql || !current(dev) || !on(*q, dev) || q->size(1) != f[0] || q->size(2) != f[2]) return none();
    const int64_t t = q->size(0), b = ctx->numel();
    if (b > f[6] || !vec(ctx, dev, at::kInt, b) || !vec(ql, dev, at::kInt, b)) return none();
    if (table->dim() != 2 || table->size(0) != b || table->size(1) != f[5] || !plain(*table, dev, at::kInt)) return none();
    Caches c;
    if (!caches(a[2], a[3], a[4], a[5], dev, f[3] == PA_KV_FP8_E4M3, f[1], f[2], &c) || c.pages != f[4]) return none();
    at::Tensor made;
    const at::Tensor* out = nullptr;
    if (a[10] != Py_None) {
      out = tensor(a[10]);
      if (!out || out->sizes() != q->sizes() || !plain(*out, dev, at::kBFloat16)) return none();
    } else {
      made = at::empty(q->sizes(), q->options());
      out = &made;
    }
    const pa_chunk_desc desc{static_cast<int32_t>(b), static_cast<int32_t>(t), static_cast<int32_t>(f[0]), static_cast<int32_t>(f[1]),
                             static_cast<int32_t>(f[2]), 16, static_cast<int32_t>(f[3]), static_cast<int32_t>(f[4]),
                             static_cast<int32_t>(f[5]), static_cast<int32_t>(f[7]), qs};
    const int rc = api.chunk(&desc, q->data_ptr(), c.k, c.v, c.ks, c.vs, ptr<int32_t>(*table), ptr<int32_t>(*ctx), ptr<int32_t>(*ql),
                             static_cast<float>(scale), out->data_ptr(), reinterpret_cast<void*>(f[8]), static_cast<size_t>(f[9]), stream_of(dev));
    if (rc != PA_OK) return PyLong_FromLong(rc);
    if (a[10] != Py_None) {
      Py_INCREF(a[10]);
      return a[10];
    }
    return THPVariable_Wrap(std::move(made));
  });
}

struct Pool {
  pa_pool_desc desc;
  int dev;
  uint32_t* errors;
  void* workspace;
  size_t bytes;
  std::vector<void*> data[4];  // K, V, their scales: one a layer
};
const char kPoolName[] = "pa_fast.pool";
void drop_pool(PyObject* o) { delete static_cast<Pool*>(PyCapsule_GetPointer(o, kPoolName)); }

// num_pages, hkv, d, kv_dtype, device, errors, workspace, its bytes, [K], [V], [K scales], [V scales] (lists of addresses)
PyObject* pool_new(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) return none();
    auto p = std::make_unique<Pool>();
    long long f[8];
    for (int i = 0; i < 8; ++i) f[i] = PyLong_AsLongLong(a[i]);
    for (int g = 0; g < 4; ++g) {
      if (!PyList_Check(a[8 + g])) return none();
      for (Py_ssize_t i = 0; i < PyList_GET_SIZE(a[8 + g]); ++i) p->data[g].push_back(PyLong_AsVoidPtr(PyList_GET_ITEM(a[8 + g], i)));
    }
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    p->desc = pa_pool_desc{static_cast<int32_t>(f[0]), static_cast<int32_t>(f[1]), static_cast<int32_t>(f[2]), static_cast<int32_t>(f[3]),
                           static_cast<int32_t>(p->data[0].size())};
    p->dev = static_cast<int>(f[4]);
    p->errors = reinterpret_cast<uint32_t*>(f[5]);
    p->workspace = reinterpret_cast<void*>(f[6]);
    p->bytes = static_cast<size_t>(f[7]);
    return PyCapsule_New(p.release(), kPoolName, drop_pool);
  });
}

struct Tables {
  Pool* pool;
  const at::Tensor *table, *lens, *ref;
  pa_pages_desc desc;
};
// capsule, block_table, context_lens, ref_counts
bool tables(PyObject* const* a, Tables* t) {
  t->pool = static_cast<Pool*>(PyCapsule_GetPointer(a[0], kPoolName));
  if (!t->pool) {
    PyErr_Clear();
    return false;
  }
  t->table = tensor(a[1]);
  t->lens = tensor(a[2]);
  t->ref = tensor(a[3]);
  const int dev = t->pool->dev;
  if (!current(dev) || !t->table || t->table->dim() != 2 || !plain(*t->table, dev, at::kInt) ||
      !vec(t->lens, dev, at::kInt, t->table->size(0)) || !vec(t->ref, dev, at::kInt, t->pool->desc.num_pages))
    return false;
  t->desc = pa_pages_desc{static_cast<int32_t>(t->table->size(0)), static_cast<int32_t>(t->table->size(1)), t->pool->desc.num_pages};
  return true;
}

// pool, block_table, context_lens, ref_counts, parents, children -> True
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tables t;
    if (n != 6 || !tables(a, &t)) return none();
    const at::Tensor *from = tensor(a[4]), *to = tensor(a[5]);
    const int dev = t.pool->dev;
    if (!from || !vec(from, dev, at::kInt, from->numel()) || !vec(to, dev, at::kInt, from->numel())) return none();
    const int rc = api.fork(&t.desc, ptr<int32_t>(*t.table), ptr<int32_t>(*t.lens), ptr<int32_t>(*t.ref), ptr<int32_t>(*from),
                            ptr<int32_t>(*to), static_cast<int32_t>(from->numel()), t.pool->errors, stream_of(dev));
    if (rc != PA_OK) return PyLong_FromLong(rc);
    Py_RETURN_TRUE;
  });
}

// pool, block_table, context_lens, ref_counts, new_lens -> (copy_src, copy_dst)
PyObject* resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tables t;
    if (n != 5 || !tables(a, &t)) return none();
    const at::Tensor* to = tensor(a[4]);
    const int dev = t.pool->dev;
    if (!vec(to, dev, at::kInt, t.desc.num_seqs)) return none();
    at::Tensor src = ints({t.desc.num_seqs}, *to), dst = ints({t.desc.num_seqs}, *to);
    const int rc = api.resize(&t.desc, ptr<int32_t>(*t.table), ptr<int32_t>(*t.lens), ptr<int32_t>(*t.ref), ptr<int32_t>(*to),
                              ptr<int32_t>(src), ptr<int32_t>(dst), t.pool->errors, t.pool->workspace, t.pool->bytes, stream_of(dev));
    if (rc != PA_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(src)), THPVariable_Wrap(std::move(dst)));
  });
}

// pool, block_table, context_lens, ref_counts, in_place -> (block_table, ref_counts, copy_src, copy_dst, num_moves)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tables t;
    if (n != 5 || !tables(a, &t)) return none();
    const bool in_place = a[4] == Py_True;
    if (!in_place && a[4] != Py_False) return none();
    const int64_t half = t.desc.num_pages / 2;
    at::Tensor table = in_place ? *t.table : ints(t.table->sizes(), *t.ref), ref = in_place ? *t.ref : ints({t.desc.num_pages}, *t.ref);
    at::Tensor src = ints({half}, *t.ref), dst = ints({half}, *t.ref), moves = ints({1}, *t.ref);
    const int rc = api.compact(&t.desc, ptr<int32_t>(*t.table), ptr<int32_t>(*t.lens), ptr<int32_t>(*t.ref), ptr<int32_t>(table),
                               ptr<int32_t>(ref), ptr<int32_t>(src), ptr<int32_t>(dst), ptr<int32_t>(moves), t.pool->errors,
                               t.pool->workspace, t.pool->bytes, stream_of(t.pool->dev));
    if (rc != PA_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("(NNNNN)", THPVariable_Wrap(std::move(table)), THPVariable_Wrap(std::move(ref)), THPVariable_Wrap(std::move(src)),
                         THPVariable_Wrap(std::move(dst)), THPVariable_Wrap(std::move(moves)));
  });
}

// pool, copy_src, copy_dst, num_pairs -> True
PyObject* copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) return none();
    Pool* p = static_cast<Pool*>(PyCapsule_GetPointer(a[0], kPoolName));
    if (!p) {
      PyErr_Clear();
      return none();
    }
    const at::Tensor *src = tensor(a[1]), *dst = tensor(a[2]);
    if (!src || !current(p->dev) || !vec(src, p->dev, at::kInt, src->numel()) || !vec(dst, p->dev, at::kInt, src->numel())) return none();
    const int32_t* count = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor* c = tensor(a[3]);
      if (!vec(c, p->dev, at::kInt, 1)) return none();
      count = ptr<int32_t>(*c);
    }
    const bool fp8 = p->desc.kv_dtype == PA_KV_FP8_E4M3;
    const int rc = api.copy(&p->desc, ptr<int32_t>(*src), ptr<int32_t>(*dst), static_cast<int32_t>(src->numel()), count, p->data[0].data(),
                            p->data[1].data(), fp8 ? reinterpret_cast<float* const*>(p->data[2].data()) : nullptr,
                            fp8 ? reinterpret_cast<float* const*>(p->data[3].data()) : nullptr, p->errors, stream_of(p->dev));
    if (rc != PA_OK) return PyLong_FromLong(rc);
    Py_RETURN_TRUE;
  });
}

#define PA_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_FAST(init),   PA_FAST(rope),    PA_FAST(chunk), PA_FAST(pool_new), PA_FAST(fork),
                         PA_FAST(resize), PA_FAST(compact), PA_FAST(copy),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_fast() { return PyModule_Create(&module); }
