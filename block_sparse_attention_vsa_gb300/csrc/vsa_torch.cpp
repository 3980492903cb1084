// vsa_torch.cpp -- the short way from torch tensors to the library's calls that run for
// microseconds (block means, the choice of blocks, the 8-bit cache): argument checks,
// output allocation and the call in one step of C++.
//
// Every function returns its result, or the library's status as an int where that is not
// VSA_OK, or None where an argument is not what the short way takes (another device than
// the current one, a wrong type or shape, an unusual object).  The caller then goes the
// long way, which serves the call or says what is wrong with it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <initializer_list>

#include "../../include/vsa.h"

namespace {

// The library's entry points, from the handle that the binding has opened.
struct Entry {
  decltype(&vsa_block_mean) block_mean;
  decltype(&vsa_select_blocks) select_blocks;
  decltype(&vsa_cache_select) cache_select;
  decltype(&vsa_cache_write) cache_write;
  decltype(&vsa_fwd_cache) fwd_cache;
  decltype(&vsa_cache_evict) cache_evict;
} lib;

// Thrown where the long way has to be taken.
struct LongWay {};

using Shape = std::initializer_list<int64_t>;

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw LongWay();
  return THPVariable_Unpack(o);
}

// What a call goes by: the device of its first tensor, which has to be the current one.
struct Device {
  int index;
  explicit Device(const at::Tensor& t) : index(t.is_cuda() ? t.get_device() : -1) {
    if (index < 0 || c10::cuda::current_device() != index) throw LongWay();
  }
  vsa_stream_t stream() const {
    return reinterpret_cast<vsa_stream_t>(c10::cuda::getCurrentCUDAStream(index).stream());
  }
};

// A contiguous tensor of this type and number of dimensions on the call's device.
const at::Tensor& lead(PyObject* o, at::ScalarType type, int64_t dims) {
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != type || t.dim() != dims || !t.is_cuda() || !t.is_contiguous())
    throw LongWay();
  return t;
}
template <typename T>
T* need(PyObject* o, at::ScalarType type, Shape shape, const Device& dev) {
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_cuda() ||
      t.get_device() != dev.index || !t.is_contiguous())
    throw LongWay();
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* maybe(PyObject* o, at::ScalarType type, Shape shape, const Device& dev) {
  return o == Py_None ? nullptr : need<T>(o, type, shape, dev);
}
template <typename T>
T* address(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
at::Tensor empty(const at::Tensor& like, at::ScalarType type, Shape shape) {
  return at::detail::empty_cuda(at::IntArrayRef(shape), type, like.device(), std::nullopt);
}
// Consecutive parts of one allocation of int32.
struct Parts {
  at::Tensor all;
  int64_t at = 0;
  Parts(const at::Tensor& like, int64_t n) : all(empty(like, at::kInt, {n})) {}
  at::Tensor part(Shape shape) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()),
                                                            all.key_set(), all.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(shape));
    at += t.numel();
    return t;
  }
};
int to_int(int64_t v) {
  if (v < INT_MIN || v > INT_MAX) throw LongWay();
  return (int)v;
}
int whole(PyObject* o) {
  const long v = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
  if (!PyLong_Check(o) || PyErr_Occurred()) {
    PyErr_Clear();
    throw LongWay();
  }
  return to_int(v);
}
float real(PyObject* o) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) throw LongWay();
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw LongWay();
  }
  return (float)v;
}
bool truth(PyObject* o) {
  if (o != Py_True && o != Py_False) throw LongWay();
  return o == Py_True;
}

// A list of new references, as a tuple.
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t != nullptr)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_XDECREF(o);
  }
  return t;
}
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// Runs f, which returns a new reference; what it throws sends the caller the long way.
template <typename F>
PyObject* run(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) Py_RETURN_NONE;
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}
template <typename C>
vsa_status unlocked(C call) {
  vsa_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  return st;
}

constexpr at::ScalarType kBf16 = at::kBFloat16, kI32 = at::kInt, kF32 = at::kFloat,
                         kE4m3 = at::kFloat8_e4m3fn;

// (x, sizes, block, out)
PyObject* block_mean(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 4, [&]() -> PyObject* {
    const at::Tensor& x = lead(a[0], kBf16, 4);
    const Device dev(x);
    const int block = whole(a[2]);
    if (block < 1) throw LongWay();
    const int64_t B = x.size(0), H = x.size(1), S = x.size(2), D = x.size(3);
    const int64_t nb = (S + block - 1) / block;
    const int32_t* sizes = maybe<int32_t>(a[1], kI32, {nb}, dev);
    at::Tensor made;
    vsa_bf16* out;
    if (a[3] == Py_None) {
      made = empty(x, kBf16, {B, H, nb, D});
      out = address<vsa_bf16>(made);
    } else {
      out = need<vsa_bf16>(a[3], kBf16, {B, H, nb, D}, dev);
    }
    const vsa_bf16* xp = address<vsa_bf16>(x);
    const int b = to_int(B), h = to_int(H), s = to_int(S), d = to_int(D);
    const vsa_stream_t stream = dev.stream();
    const vsa_status st =
        unlocked([&] { return lib.block_mean(xp, sizes, b, h, s, d, block, out, stream); });
    if (st != VSA_OK) return PyLong_FromLong(st);
    return tuple({a[3] == Py_None ? THPVariable_Wrap(made) : same(a[3])});
  });
}

// (q_mean, k_mean, topk, sizes, causal, n_first, n_near)
PyObject* select_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 7, [&]() -> PyObject* {
    const at::Tensor &q = lead(a[0], kBf16, 4), &k = lead(a[1], kBf16, 4);
    const Device dev(q);
    const int topk = whole(a[2]), n_first = whole(a[5]), n_near = whole(a[6]);
    const bool causal = truth(a[4]);
    const int64_t B = q.size(0), Hq = q.size(1), nq = q.size(2), D = q.size(3);
    const int64_t Hkv = k.size(1), nk = k.size(2);
    if (topk < 1) throw LongWay();
    const vsa_bf16* kp = need<vsa_bf16>(a[1], kBf16, {B, Hkv, nk, D}, dev);
    const int32_t* sizes = maybe<int32_t>(a[3], kI32, {nk}, dev);
    const at::Tensor idx = empty(q, kI32, {B, Hq, nq, topk}), num = empty(q, kI32, {B, Hq, nq});
    const vsa_bf16* qp = address<vsa_bf16>(q);
    int32_t *ip = address<int32_t>(idx), *np = address<int32_t>(num);
    const int v[6] = {to_int(B), to_int(Hq), to_int(Hkv), to_int(nq), to_int(nk), to_int(D)};
    const vsa_stream_t stream = dev.stream();
    const vsa_status st = unlocked([&] {
      return lib.select_blocks(qp, kp, sizes, v[0], v[1], v[2], v[3], v[4], v[5], topk, causal,
                               n_first, n_near, ip, np, stream);
    });
    if (st != VSA_OK) return PyLong_FromLong(st);
    return tuple({THPVariable_Wrap(idx), THPVariable_Wrap(num)});
  });
}

// (q, k_mean, table, lens, topk, block, n_first, n_near)
PyObject* cache_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 8, [&]() -> PyObject* {
    const at::Tensor &q = lead(a[0], kBf16, 4), &mean = lead(a[1], kBf16, 2);
    const at::Tensor& table = lead(a[2], kI32, 3);
    const Device dev(q);
    const int topk = whole(a[4]), block = whole(a[5]), n_first = whole(a[6]), n_near = whole(a[7]);
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(3), pages = mean.size(0);
    const int64_t Hkv = table.size(1), blocks = table.size(2);
    if (q.size(2) != 1 || topk < 1) throw LongWay();
    const vsa_bf16* mp = need<vsa_bf16>(a[1], kBf16, {pages, D}, dev);
    const int32_t* tp = need<int32_t>(a[2], kI32, {B, Hkv, blocks}, dev);
    const int32_t* lens = need<int32_t>(a[3], kI32, {B}, dev);
    const at::Tensor idx = empty(q, kI32, {B, Hkv, topk}), num = empty(q, kI32, {B, Hkv});
    const vsa_bf16* qp = address<vsa_bf16>(q);
    int32_t *ip = address<int32_t>(idx), *np = address<int32_t>(num);
    const int v[6] = {to_int(B), to_int(Hq), to_int(Hkv), to_int(D), to_int(pages), to_int(blocks)};
    const vsa_stream_t stream = dev.stream();
    const vsa_status st = unlocked([&] {
      return lib.cache_select(qp, mp, tp, lens, v[0], v[1], v[2], v[3], v[4], v[5], block, topk,
                              n_first, n_near, ip, np, stream);
    });
    if (st != VSA_OK) return PyLong_FromLong(st);
    return tuple({THPVariable_Wrap(idx), THPVariable_Wrap(num)});
  });
}

// The tensors of a Cache8, checked against one another.
struct Cache {
  int64_t pages, block;
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  PyObject* k_mean;
  Cache(PyObject* o, const Device& dev) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) throw LongWay();
    const at::Tensor& first = lead(PyTuple_GET_ITEM(o, 0), kE4m3, 3);
    pages = first.size(0);
    block = first.size(1);
    k = need<uint8_t>(PyTuple_GET_ITEM(o, 0), kE4m3, {pages, block, VSA_HEAD_DIM}, dev);
    v = need<uint8_t>(PyTuple_GET_ITEM(o, 1), kE4m3, {pages, block, VSA_HEAD_DIM}, dev);
    k_scale = need<float>(PyTuple_GET_ITEM(o, 2), kF32, {pages}, dev);
    v_scale = need<float>(PyTuple_GET_ITEM(o, 3), kF32, {pages}, dev);
    k_mean = PyTuple_GET_ITEM(o, 4);
  }
};

// (cache, k, v, table, lens, n_new)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 6, [&]() -> PyObject* {
    const at::Tensor &k = lead(a[1], kBf16, 4), &table = lead(a[3], kI32, 3);
    const Device dev(k);
    const int64_t B = k.size(0), Hkv = k.size(1), T = k.size(2), D = k.size(3);
    const int64_t blocks = table.size(2);
    const Cache c(a[0], dev);
    const vsa_bf16* vp = need<vsa_bf16>(a[2], kBf16, {B, Hkv, T, D}, dev);
    vsa_bf16* mean = maybe<vsa_bf16>(c.k_mean, kBf16, {c.pages, VSA_HEAD_DIM}, dev);
    const int32_t* tp = need<int32_t>(a[3], kI32, {B, Hkv, blocks}, dev);
    const int32_t* lens = need<int32_t>(a[4], kI32, {B}, dev);
    const int32_t* n_new = maybe<int32_t>(a[5], kI32, {B}, dev);
    const vsa_bf16* kp = address<vsa_bf16>(k);
    const int v[7] = {to_int(B),       to_int(Hkv),    to_int(T),      to_int(D),
                      to_int(c.pages), to_int(blocks), to_int(c.block)};
    const vsa_stream_t stream = dev.stream();
    const vsa_status st = unlocked([&] {
      return lib.cache_write(kp, vp, tp, lens, n_new, v[0], v[1], v[2], v[3], v[4], v[5], v[6], c.k,
                             c.v, c.k_scale, c.v_scale, mean, stream);
    });
    if (st != VSA_OK) return PyLong_FromLong(st);
    return tuple({});
  });
}

// (q, cache, table, lens, idx, num, scale, out, lse, weight, keep, workspace)
PyObject* fwd_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 12, [&]() -> PyObject* {
    const at::Tensor &q = lead(a[0], kBf16, 4), &table = lead(a[2], kI32, 3);
    const Device dev(q);
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(3);
    const int64_t Hkv = table.size(1), blocks = table.size(2);
    if (q.size(2) != 1) throw LongWay();
    const Cache c(a[1], dev);
    const int32_t* tp = need<int32_t>(a[2], kI32, {B, Hkv, blocks}, dev);
    const int32_t* lens = need<int32_t>(a[3], kI32, {B}, dev);
    const int32_t *idx = nullptr, *num = nullptr;
    int64_t width = 0;
    if (a[4] != Py_None) {
      width = lead(a[4], kI32, 3).size(2);
      if (width < 1) throw LongWay();  // an empty tensor has no address: not "all blocks"
      idx = need<int32_t>(a[4], kI32, {B, Hkv, width}, dev);
      num = need<int32_t>(a[5], kI32, {B, Hkv}, dev);
    } else if (a[5] != Py_None) {
      throw LongWay();
    }
    const float scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : real(a[6]);
    float* weight = maybe<float>(a[9], kF32, {B, Hkv, blocks}, dev);
    const float keep = real(a[10]);
    const at::Tensor& ws = tensor(a[11]);
    if (!ws.is_cuda() || ws.get_device() != dev.index || !ws.is_contiguous()) throw LongWay();
    at::Tensor out, lse;
    vsa_bf16* op;
    if (a[7] == Py_None) {
      out = empty(q, kBf16, {B, Hq, 1, D});
      op = address<vsa_bf16>(out);
    } else {
      op = need<vsa_bf16>(a[7], kBf16, {B, Hq, 1, D}, dev);
    }
    float* lp = nullptr;
    PyObject* lse_given = nullptr;
    if (a[8] == Py_True) {
      lse = empty(q, kF32, {B, Hq, 1});
      lp = address<float>(lse);
    } else if (a[8] == Py_None || a[8] == Py_False) {
      lse_given = Py_None;
    } else {
      lp = need<float>(a[8], kF32, {B, Hq, 1}, dev);
      lse_given = a[8];
    }
    const vsa_bf16* qp = address<vsa_bf16>(q);
    void* wp = ws.data_ptr();
    const size_t bytes = ws.nbytes();
    const int v[8] = {to_int(width), to_int(B),       to_int(Hq),     to_int(Hkv),
                      to_int(D),     to_int(c.pages), to_int(blocks), to_int(c.block)};
    const vsa_stream_t stream = dev.stream();
    const vsa_status st = unlocked([&] {
      return lib.fwd_cache(qp, c.k, c.v, c.k_scale, c.v_scale, tp, lens, idx, num, v[0], v[1], v[2],
                           v[3], v[4], v[5], v[6], v[7], scale, keep, op, lp, weight, wp, bytes,
                           stream);
    });
    if (st != VSA_OK) return PyLong_FromLong(st);
    return tuple({a[7] == Py_None ? THPVariable_Wrap(out) : same(a[7]),
                  lse_given != nullptr ? same(lse_given) : THPVariable_Wrap(lse)});
  });
}

// (weight, table, lens, budget, block, n_first, n_last)
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 7, [&]() -> PyObject* {
    const at::Tensor &weight = lead(a[0], kF32, 3), &table = lead(a[1], kI32, 3);
    const Device dev(weight);
    const int budget = whole(a[3]), block = whole(a[4]), n_first = whole(a[5]), n_last = whole(a[6]);
    const int64_t B = weight.size(0), Hkv = weight.size(1), blocks = weight.size(2);
    const int32_t* tp = need<int32_t>(a[1], kI32, {B, Hkv, blocks}, dev);
    const int32_t* lens = need<int32_t>(a[2], kI32, {B}, dev);
    // An allocation for what a server goes on with together (the table and the lengths), one
    // for what it lets go, one for the weights: one for all takes 1.5 us of host time less, but
    // tensors of two types over one storage cannot be saved together, and what is kept would
    // hold the memory of what is not.
    Parts kept(table, B * Hkv * blocks + B), gone(table, B * Hkv * blocks + B);
    const at::Tensor table_out = kept.part({B, Hkv, blocks}), lens_out = kept.part({B}),
                     weight_out = empty(table, kF32, {B, Hkv, blocks}),
                     freed = gone.part({B, Hkv, blocks}), n_freed = gone.part({B});
    const float* wp = address<float>(weight);
    float* wo = address<float>(weight_out);
    int32_t *to = address<int32_t>(table_out), *lo = address<int32_t>(lens_out);
    int32_t *fo = address<int32_t>(freed), *no = address<int32_t>(n_freed);
    const int b = to_int(B), h = to_int(Hkv), mb = to_int(blocks);
    const vsa_stream_t stream = dev.stream();
    const vsa_status st = unlocked([&] {
      return lib.cache_evict(wp, tp, lens, b, h, mb, block, budget, n_first, n_last, to, wo, lo, fo,
                             no, stream);
    });
    if (st != VSA_OK) return PyLong_FromLong(st);
    return tuple({THPVariable_Wrap(table_out), THPVariable_Wrap(weight_out),
                  THPVariable_Wrap(lens_out), THPVariable_Wrap(freed), THPVariable_Wrap(n_freed)});
  });
}

// bind(handle): takes the entry points from an open handle of the library.
PyObject* bind(PyObject*, PyObject* arg) {
  void* h = PyLong_AsVoidPtr(arg);
  if (PyErr_Occurred()) return nullptr;
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    return f != nullptr;
  };
  if (!find(lib.block_mean, "vsa_block_mean") || !find(lib.select_blocks, "vsa_select_blocks") ||
      !find(lib.cache_select, "vsa_cache_select") || !find(lib.cache_write, "vsa_cache_write") ||
      !find(lib.fwd_cache, "vsa_fwd_cache") || !find(lib.cache_evict, "vsa_cache_evict")) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point");
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define VSA_FAST(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {VSA_FAST(block_mean),
                         VSA_FAST(select_blocks),
                         VSA_FAST(cache_select),
                         VSA_FAST(cache_write),
                         VSA_FAST(fwd_cache),
                         VSA_FAST(cache_evict),
                         {"bind", bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vsa_torch", nullptr, -1, methods,
                      nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vsa_torch() { return PyModule_Create(&module); }
