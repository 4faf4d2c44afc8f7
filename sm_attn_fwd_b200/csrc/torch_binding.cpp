// Native part of the Python binding for the calls a serving loop makes every step
// (cache append and read-back, 8-bit and shared-prefix decode): checks the tensors,
// allocates what the caller did not give and calls the C ABI.  Host time of a
// call here and through ctypes with the checks in Python: an append 3.9 and 10.6 us, a
// small 8-bit decode 9.3 and 20.9, a shared-prefix decode 12.2 and 24.6; the kernels of
// such calls take 2, 9 and 17 us.
//
// Each function takes its arguments by position (the wrappers in __init__.py fill in
// the optional ones), raises ValueError for a tensor that does not fit, and returns
// the library's status where that is not ATTN_OK, else its result.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <stdexcept>
#include <string>

#include "attn.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// Argument `name` as a tensor on a CUDA device.
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
  return t;
}

// ... contiguous, of this type and shape, on CUDA device `dev`.
const Tensor& tensor(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape,
                     int dev) {
  const Tensor& t = tensor(o, name);
  if (t.get_device() != dev)
    throw Refused(std::string(name) + " must be on cuda:" + std::to_string(dev));
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
    throw Refused(std::string(name) + " must be a contiguous " + at::toString(type) +
                  " tensor of shape " + shape_text(shape) + ", got " +
                  at::toString(t.scalar_type()) + " " + shape_text(t.sizes()));
  return t;
}

int to_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused(std::string(name) + " must be an integer");
  if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " is out of range");
  return (int)v;
}

int dim(int64_t v, const char* name) {
  if (v > INT32_MAX) throw Refused(std::string(name) + " has a dimension out of range");
  return (int)v;
}

// A K/V cache: contiguous [B, Hkv, Lk, d], or pages [num_pages, Hkv, page, d] with a
// block table [B, pages_per_seq].
struct Cache {
  const void *k, *v;
  const int32_t *table, *lens;
  int dev, B, Hkv, Lk, d, page, per_seq, num_pages;
  int64_t rows;  // Lk, or pages_per_seq * page
};

Cache parse_cache(PyObject* ok, PyObject* ov, PyObject* otable, PyObject* olens,
                  at::ScalarType type) {
  Cache c = {};
  const Tensor& k = tensor(ok, "k_cache");
  if (k.dim() != 4)
    throw Refused(
        "the cache must have 4 dimensions: [B, Hkv, Lk_max, d], or [num_pages, Hkv, page_size, "
        "d] for pages");
  c.dev = k.get_device();
  tensor(ok, "k_cache", type, k.sizes(), c.dev);
  c.k = k.data_ptr();
  c.v = tensor(ov, "v_cache", type, k.sizes(), c.dev).data_ptr();
  c.Hkv = dim(k.size(1), "k_cache");
  c.d = dim(k.size(3), "k_cache");
  if (otable == Py_None) {
    c.B = dim(k.size(0), "k_cache");
    c.Lk = dim(k.size(2), "k_cache");
    c.rows = c.Lk;
  } else {
    const Tensor& t = tensor(otable, "block_table");
    if (t.dim() != 2) throw Refused("block_table must be an int32 CUDA tensor [B, pages_per_seq]");
    tensor(otable, "block_table", at::kInt, t.sizes(), c.dev);
    c.table = t.const_data_ptr<int32_t>();
    c.B = dim(t.size(0), "block_table");
    c.per_seq = dim(t.size(1), "block_table");
    c.page = dim(k.size(2), "k_pages");
    c.num_pages = dim(k.size(0), "k_pages");
    c.rows = (int64_t)c.per_seq * c.page;
    c.Lk = c.rows > INT32_MAX ? INT32_MAX : (int)c.rows;  // the library refuses such a table
  }
  c.lens = tensor(olens, "kv_lens", at::kInt, {c.B}, c.dev).const_data_ptr<int32_t>();
  return c;
}

uint8_t* scale_bytes(PyObject* o, const char* name, PyObject* ocache, const Cache& c) {
  const Tensor& k = THPVariable_Unpack(ocache);
  return tensor(o, name, at::kByte, k.sizes().slice(0, 3), c.dev).data_ptr<uint8_t>();
}

// The library launches on the current device, so the cache's device is made that one; the
// stream is the given handle or that device's current stream.
struct On {
  c10::cuda::CUDAGuard guard;
  int dev;
  cudaStream_t stream, current;
  On(int dev_, PyObject* ostream) : guard((c10::DeviceIndex)dev_), dev(dev_) {
    stream = current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    if (ostream != Py_None) {
      stream = (cudaStream_t)PyLong_AsVoidPtr(ostream);
      if (!stream && PyErr_Occurred()) throw Refused("stream must be a stream handle");
    }
  }
  // A tensor allocated here belongs to the current stream: one that another stream uses
  // must not be handed out again before that stream is done with it.
  void uses(const Tensor& t) const {
    if (stream != current && t.nbytes())
      c10::cuda::CUDACachingAllocator::recordStream(
          t.storage().data_ptr(),
          c10::cuda::getStreamFromExternal(stream, (c10::DeviceIndex)dev));
  }
};

// A call into the library: a launch may wait for room in the stream's queue, and other
// Python threads run meanwhile.
template <typename F>
attn_status_t launch(F f) {
  PyThreadState* state = PyEval_SaveThread();
  const attn_status_t st = f();
  PyEval_RestoreThread(state);
  return st;
}

// Queries and outputs of a decode (outputs allocated where None).
struct Decode {
  const void* q;
  int Hq, Lq;
  float scale;
  Tensor o, lse;
};

Decode parse_decode(PyObject* oq, const Cache& c, PyObject* oscale, PyObject* oo, PyObject* olse,
                    const On& on) {
  Decode x;
  const Tensor& q = tensor(oq, "q");
  if (q.dim() != 4) throw Refused("q must be a [B, Hq, Lq, d] CUDA tensor");
  tensor(oq, "q", at::kBFloat16, {c.B, q.size(1), q.size(2), c.d}, c.dev);
  x.q = q.data_ptr();
  x.Hq = dim(q.size(1), "q");
  x.Lq = dim(q.size(2), "q");
  if (oscale == Py_None) {
    x.scale = (float)(1.0 / std::sqrt((double)c.d));
  } else {
    const double s = PyFloat_AsDouble(oscale);
    if (s == -1.0 && PyErr_Occurred()) throw Refused("scale must be a number");
    x.scale = (float)s;
  }
  x.o = oo == Py_None ? at::empty_like(q) : tensor(oo, "o", at::kBFloat16, q.sizes(), c.dev);
  x.lse = olse == Py_None ? at::empty({c.B, x.Hq, x.Lq}, q.options().dtype(at::kFloat))
                          : tensor(olse, "lse", at::kFloat, {c.B, x.Hq, x.Lq}, c.dev);
  if (oo == Py_None) on.uses(x.o);
  if (olse == Py_None) on.uses(x.lse);
  return x;
}

// The caller's workspace, or a new one of `need` bytes.
Tensor workspace(PyObject* o, size_t need, const Tensor& like, const On& on) {
  if (o == Py_None) {
    Tensor t = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
    on.uses(t);
    return t;
  }
  const Tensor& t = tensor(o, "workspace");
  if (t.get_device() != like.get_device() || !t.is_contiguous())
    throw Refused("workspace must be a contiguous CUDA tensor on the cache's device");
  return t;
}

PyObject* status(attn_status_t st) { return PyLong_FromLong((long)st); }

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

// (k, v, k_cache, v_cache, k_exp, v_exp, block_table, kv_lens, new_lens, stream) -> None
PyObject* cache_append(PyObject* const* a) {
  const Cache c = parse_cache(a[2], a[3], a[6], a[7], at::kFloat8_e4m3fn);
  uint8_t* ke = scale_bytes(a[4], "k_exp", a[2], c);
  uint8_t* ve = scale_bytes(a[5], "v_exp", a[2], c);
  const Tensor& k = tensor(a[0], "k");
  if (k.dim() != 4) throw Refused("k must be a [B, Hkv, Ln, d] CUDA tensor");
  const int64_t shape[4] = {c.B, c.Hkv, k.size(2), c.d};
  tensor(a[0], "k", at::kBFloat16, shape, c.dev);
  const Tensor& v = tensor(a[1], "v", at::kBFloat16, shape, c.dev);
  const int Ln = dim(k.size(2), "k");
  const int32_t* n = nullptr;
  if (a[8] != Py_None)
    n = tensor(a[8], "new_lens", at::kInt, {c.B}, c.dev).const_data_ptr<int32_t>();
  On on(c.dev, a[9]);
  void *kc = const_cast<void*>(c.k), *vc = const_cast<void*>(c.v);
  const attn_status_t st = launch([&] {
    return c.table ? attn_cache_append_paged_q8(k.data_ptr(), v.data_ptr(), kc, vc, ke, ve, c.table,
                                           c.lens, n, c.B, c.Hkv, Ln, c.page, c.per_seq,
                                           c.num_pages, c.d, on.stream)
              : attn_cache_append_q8(k.data_ptr(), v.data_ptr(), kc, vc, ke, ve, c.lens, n, c.B,
                                     c.Hkv, Ln, c.Lk, c.d, on.stream);
  });
  if (st != ATTN_OK) return status(st);
  Py_RETURN_NONE;
}

// (k_cache, v_cache, k_exp, v_exp, block_table, kv_lens, k, v, stream) -> (k, v)
PyObject* cache_read(PyObject* const* a) {
  const Cache c = parse_cache(a[0], a[1], a[4], a[5], at::kFloat8_e4m3fn);
  const uint8_t* ke = scale_bytes(a[2], "k_exp", a[0], c);
  const uint8_t* ve = scale_bytes(a[3], "v_exp", a[0], c);
  const int64_t shape[4] = {c.B, c.Hkv, c.rows, c.d};
  const auto options = THPVariable_Unpack(a[0]).options().dtype(at::kBFloat16);
  On on(c.dev, a[8]);
  const Tensor k = a[6] == Py_None ? at::empty(shape, options)
                                   : tensor(a[6], "k", at::kBFloat16, shape, c.dev);
  const Tensor v = a[7] == Py_None ? at::empty(shape, options)
                                   : tensor(a[7], "v", at::kBFloat16, shape, c.dev);
  if (a[6] == Py_None) on.uses(k);
  if (a[7] == Py_None) on.uses(v);
  const attn_status_t st = launch([&] {
    return c.table ? attn_cache_read_paged_q8(c.k, c.v, ke, ve, c.table, c.lens, k.data_ptr(),
                                         v.data_ptr(), c.B, c.Hkv, c.page, c.per_seq, c.num_pages,
                                         c.d, on.stream)
              : attn_cache_read_q8(c.k, c.v, ke, ve, c.lens, k.data_ptr(), v.data_ptr(), c.B,
                                   c.Hkv, c.Lk, c.d, on.stream);
  });
  return st == ATTN_OK ? pair(k, v) : status(st);
}

// (q, k_cache, v_cache, k_exp, v_exp, block_table, kv_lens, scale, num_ctas, workspace, o, lse,
// stream) -> (o, lse)
PyObject* decode_q8(PyObject* const* a) {
  const Cache c = parse_cache(a[1], a[2], a[5], a[6], at::kFloat8_e4m3fn);
  const uint8_t* ke = scale_bytes(a[3], "k_exp", a[1], c);
  const uint8_t* ve = scale_bytes(a[4], "v_exp", a[1], c);
  const int ctas = to_int(a[8], "num_ctas");
  On on(c.dev, a[12]);
  const Decode x = parse_decode(a[0], c, a[7], a[10], a[11], on);
  const size_t need =
      a[9] == Py_None ? attn_decode_q8_workspace_size(x.Hq, c.Hkv, x.Lq, c.d, ctas) : 0;
  if (a[9] == Py_None && need == 0) return status(ATTN_ERR_INVALID_ARG);
  const Tensor ws = workspace(a[9], need, x.o, on);
  const attn_status_t st = launch([&] {
    return c.table ? attn_decode_paged_q8(x.q, c.k, c.v, ke, ve, c.table, x.o.data_ptr(),
                                     x.lse.data_ptr<float>(), c.lens, c.B, x.Hq, c.Hkv, x.Lq,
                                     c.page, c.per_seq, c.num_pages, c.d, x.scale, ctas,
                                     ws.data_ptr(), ws.nbytes(), on.stream)
              : attn_decode_splitkv_q8(x.q, c.k, c.v, ke, ve, x.o.data_ptr(),
                                       x.lse.data_ptr<float>(), c.lens, c.B, x.Hq, c.Hkv, x.Lq,
                                       c.Lk, c.d, x.scale, ctas, ws.data_ptr(), ws.nbytes(),
                                       on.stream);
  });
  return st == ATTN_OK ? pair(x.o, x.lse) : status(st);
}

// (q, k_prefix, v_prefix, prefix_table, prefix_len, k_cache, v_cache, block_table, kv_lens,
// scale, num_splits, workspace, o, lse, stream) -> (o, lse); contiguous: prefix_table and
// block_table None; paged: k_prefix and v_prefix None
PyObject* shared_prefix(PyObject* const* a) {
  const Cache c = parse_cache(a[5], a[6], a[7], a[8], at::kBFloat16);
  const void *kp = nullptr, *vp = nullptr;
  const int32_t* table = nullptr;
  int Lp = 0;
  if (c.table) {
    Lp = to_int(a[4], "prefix_len");
    const int64_t n = c.page > 0 && Lp > 0 ? ((int64_t)Lp + c.page - 1) / c.page : 0;
    table = tensor(a[3], "prefix_table", at::kInt, {n}, c.dev).const_data_ptr<int32_t>();
  } else {
    const Tensor& k = tensor(a[1], "k_prefix");
    if (k.dim() != 3) throw Refused("k_prefix must be a [Hkv, Lp, d] CUDA tensor");
    const int64_t shape[3] = {c.Hkv, k.size(1), c.d};
    tensor(a[1], "k_prefix", at::kBFloat16, shape, c.dev);
    kp = k.data_ptr();
    vp = tensor(a[2], "v_prefix", at::kBFloat16, shape, c.dev).data_ptr();
    Lp = dim(k.size(1), "k_prefix");
  }
  const int splits = to_int(a[10], "num_splits");
  On on(c.dev, a[14]);
  const Decode x = parse_decode(a[0], c, a[9], a[12], a[13], on);
  const size_t need = a[11] == Py_None
                          ? attn_decode_shared_prefix_workspace_size(c.B, x.Hq, c.Hkv, x.Lq, Lp,
                                                                     c.Lk, c.d, splits)
                          : 0;
  if (a[11] == Py_None && need == 0) return status(ATTN_ERR_INVALID_ARG);
  const Tensor ws = workspace(a[11], need, x.o, on);
  const attn_status_t st = launch([&] {
    return c.table ? attn_decode_shared_prefix_paged(x.q, c.k, c.v, table, c.table, x.o.data_ptr(),
                                                x.lse.data_ptr<float>(), c.lens, c.B, x.Hq, c.Hkv,
                                                x.Lq, Lp, c.page, c.per_seq, c.num_pages, c.d,
                                                x.scale, splits, ws.data_ptr(), ws.nbytes(),
                                                on.stream)
              : attn_decode_shared_prefix(x.q, kp, vp, c.k, c.v, x.o.data_ptr(),
                                          x.lse.data_ptr<float>(), c.lens, c.B, x.Hq, c.Hkv, x.Lq,
                                          Lp, c.Lk, c.d, x.scale, splits, ws.data_ptr(),
                                          ws.nbytes(), on.stream);
  });
  return st == ATTN_OK ? pair(x.o, x.lse) : status(st);
}

template <PyObject* (*fn)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return fn(args);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*fn)(PyObject* const*), Py_ssize_t kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<fn, kArgs>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<cache_append, 10>("cache_append"), method<cache_read, 9>("cache_read"),
    method<decode_q8, 13>("decode_q8"),       method<shared_prefix, 15>("shared_prefix"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "attn_torch", nullptr, -1, g_methods};

}  // namespace

// Which interpreter, torch and C ABI this object is built for; looked up before it is loaded.
extern "C" __attribute__((used, visibility("default"))) const char attn_torch_mark[] =
    ATTN_TORCH_MARK;

PyMODINIT_FUNC PyInit_attn_torch() { return PyModule_Create(&g_module); }
