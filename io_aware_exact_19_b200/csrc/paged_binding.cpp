// Python binding of the paged-cache entry points.
//
// A serving step on a small batch keeps the GPU busy for a few microseconds, and reading ten
// tensors' types, devices, strides and addresses from Python takes longer than that. This module
// reads them from the tensors themselves, checks them and calls the C ABI (whose addresses the
// Python side passes in once, from the library it has loaded). Each function returns the status
// code; mismatched tensors raise ValueError or TypeError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "fa.h"

namespace {

struct Refused : std::exception {};  // a Python error is set

[[noreturn]] void refuse(PyObject* type, const std::string& why) {
  PyErr_SetString(type, why.c_str());
  throw Refused();
}

std::string text(const at::Tensor& t) {
  std::string s = std::string(c10::toString(t.scalar_type())) + " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "] on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

// A size that the C ABI takes as an int (one beyond it is refused there).
int size(long long v) {
  return v > 0x7FFFFFFFll ? 0x7FFFFFFF : (v < -0x7FFFFFFFll ? -0x7FFFFFFF : static_cast<int>(v));
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v;
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + ": expected a CUDA tensor, got " + text(t));
  return t.get_device();
}

// Address of a contiguous tensor of one type on device `dev`.
template <typename T>
T* plain(PyObject* o, const char* name, at::ScalarType type, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + ": expected a contiguous " + c10::toString(type) + " tensor on cuda:" +
                                 std::to_string(dev) + ", got " + text(t));
  return static_cast<T*>(t.data_ptr());
}

int32_t* ints(PyObject* o, const char* name, int dev) { return plain<int32_t>(o, name, at::kInt, dev); }

void expect(bool ok, const char* what) {
  if (!ok) refuse(PyExc_ValueError, what);
}

fa_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kHalf) return FA_FP16;
  if (t.scalar_type() == at::kBFloat16) return FA_BF16;
  refuse(PyExc_TypeError, "unsupported dtype; expected float16 or bfloat16");
}

// Element stride of dimension i (a dimension of size 1 has none of its own: the row's length).
long long stride_of(const at::Tensor& t, int64_t i) { return t.size(i) == 1 ? t.size(t.dim() - 1) : t.stride(i); }

void rows_contiguous(const at::Tensor& t) {
  const int64_t last = t.dim() - 1;
  if (t.size(last) > 1 && t.stride(last) != 1) refuse(PyExc_ValueError, "the head dimension must be contiguous");
}

// Two caches [pages, H_kv, page_size, d].
struct Cache {
  fa_kv_cache c;
  at::ScalarType type;
  int dev;
  Cache(PyObject* ko, PyObject* vo) {
    const at::Tensor &k = tensor(ko, "cache_k"), &v = tensor(vo, "cache_v");
    expect(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() && v.device() == k.device(),
           "expected two caches of one type, shape [pages, H_kv, page_size, d] and device");
    dev = device_of(k, "cache_k");
    type = k.scalar_type();
    c.dtype = dtype_of(k);
    rows_contiguous(k);
    rows_contiguous(v);
    for (int i = 0; i < 3; ++i)
      expect(stride_of(k, i) == stride_of(v, i), "the caches of K and V must have the same strides");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.num_pages = size(k.size(0));
    c.H_kv = size(k.size(1));
    c.page_size = size(k.size(2));
    c.d = size(k.size(3));
    c.page_stride = stride_of(k, 0);
    c.head_stride = stride_of(k, 1);
    c.row_stride = stride_of(k, 2);
  }
};

// Packed rows [T, heads, d] of the cache's type (heads < 0: any).
fa_rows rows_of(PyObject* o, const char* name, const Cache& cache, long long T, long long heads) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 3 || t.size(0) != T || (heads >= 0 && t.size(1) != heads) || t.size(2) != cache.c.d ||
      t.scalar_type() != cache.type || !t.is_cuda() || t.get_device() != cache.dev)
    refuse(PyExc_ValueError, std::string(name) + ": expected packed rows [" + std::to_string(T) + ", heads, " +
                                 std::to_string(cache.c.d) + "] of the cache's type and device, got " + text(t));
  rows_contiguous(t);
  return fa_rows{t.data_ptr(), stride_of(t, 0), stride_of(t, 1)};
}

cudaStream_t stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  return reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(integer(o)));
}

// The C ABI, from the library that the Python side has loaded.
decltype(&::fa_cache_plan) call_plan = nullptr;
decltype(&::fa_rope) call_rope = nullptr;
decltype(&::fa_rope_append) call_append = nullptr;
decltype(&::fa_tree_fwd) call_tree = nullptr;
decltype(&::fa_tree_fwd_workspace_size) call_tree_workspace = nullptr;
decltype(&::fa_cache_commit) call_commit = nullptr;

PyObject* bind(PyObject* const* a) {
  auto at = [&](int i) { return static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(a[i])); };
  call_plan = reinterpret_cast<decltype(call_plan)>(at(0));
  call_rope = reinterpret_cast<decltype(call_rope)>(at(1));
  call_append = reinterpret_cast<decltype(call_append)>(at(2));
  call_tree = reinterpret_cast<decltype(call_tree)>(at(3));
  call_tree_workspace = reinterpret_cast<decltype(call_tree_workspace)>(at(4));
  call_commit = reinterpret_cast<decltype(call_commit)>(at(5));
  if (PyErr_Occurred()) throw Refused();
  return PyLong_FromLong(0);
}

// ctx_len, cu_new, block_table, n_pages, free_list, free_count, seq_len, slot, position, page_size,
// max_new, parent, tree_mask, stream
PyObject* plan(PyObject* const* a) {
  const at::Tensor &ctx = tensor(a[0], "ctx_len"), &table = tensor(a[2], "block_table"), &slot = tensor(a[7], "slot");
  const int dev = device_of(ctx, "ctx_len");
  const long long B = ctx.numel(), rows = slot.numel(), max_new = integer(a[10]);
  expect(table.dim() == 2 && table.size(0) == B && tensor(a[1], "cu_new").numel() == B + 1 &&
             tensor(a[3], "n_pages").numel() == B && tensor(a[6], "seq_len").numel() == B &&
             tensor(a[8], "position").numel() == rows && tensor(a[5], "free_count").numel() == 1,
         "lengths do not fit: cu_new [B+1]; block_table [B, max_pages]; n_pages, seq_len [B]; free_count [1]; position "
         "like slot");
  expect((a[11] == Py_None) == (a[12] == Py_None), "parent and tree_mask go together");
  int32_t* parent = nullptr;
  int64_t* mask = nullptr;
  if (a[11] != Py_None) {
    const at::Tensor& m = tensor(a[12], "tree_mask");
    expect(tensor(a[11], "parent").numel() == rows && m.dim() == 2 && m.size(0) == rows &&
               m.size(1) == (max_new + 63) / 64,
           "expected parent [rows] and tree_mask [rows, ceil(max_new/64)]");
    parent = ints(a[11], "parent", dev);
    mask = plain<int64_t>(a[12], "tree_mask", at::kLong, dev);
  }
  int32_t *c = ints(a[0], "ctx_len", dev), *cu = ints(a[1], "cu_new", dev), *tb = ints(a[2], "block_table", dev),
          *held = ints(a[3], "n_pages", dev), *free = ints(a[4], "free_list", dev), *count = ints(a[5], "free_count", dev),
          *seq = ints(a[6], "seq_len", dev), *sl = ints(a[7], "slot", dev), *pos = ints(a[8], "position", dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  return PyLong_FromLong(call_plan(size(B), size(rows), size(max_new), size(integer(a[9])),
                                   size(tensor(a[4], "free_list").numel()), size(table.size(1)), c, cu, parent, tb, held,
                                   free, count, seq, sl, pos, reinterpret_cast<uint64_t*>(mask), stream_of(a[13], dev)));
}

struct Tables {
  const int32_t* positions = nullptr;
  const float* inv_freq = nullptr;
  const uint8_t* axis = nullptr;
  long long axis_stride = 0;
  int axes = 0, rot = 0;
  Tables() = default;
  Tables(PyObject* po, PyObject* fo, PyObject* ao, int dev) {
    const at::Tensor &p = tensor(po, "positions"), &f = tensor(fo, "inv_freq"), &x = tensor(ao, "axis");
    const int64_t last = p.dim() - 1;
    expect(p.scalar_type() == at::kInt && p.is_cuda() && p.get_device() == dev && last >= 1 &&
               (p.size(last) <= 1 || p.stride(last) == 1),
           "positions: expected int32 on the same device, contiguous along the tokens");
    expect(f.numel() == x.numel(), "inv_freq and axis hold one entry for each rotated pair");
    positions = static_cast<const int32_t*>(p.data_ptr());
    inv_freq = plain<float>(fo, "inv_freq", at::kFloat, dev);
    axis = plain<uint8_t>(ao, "axis", at::kByte, dev);
    axis_stride = p.stride(0);
    axes = size(p.size(0));
    rot = size(2 * f.numel());
  }
};

// x, out, positions, inv_freq, axis, inverse, pairs, stream
PyObject* rope(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &out = tensor(a[1], "out"), &pos = tensor(a[2], "positions");
  const int dev = device_of(x, "x");
  expect(x.dim() == 4 && out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type() && out.device() == x.device(),
         "x and out must be CUDA tensors [B, H, N, d] of one shape and type");
  const fa_dtype dtype = dtype_of(x);
  rows_contiguous(x);
  rows_contiguous(out);
  const int64_t B = x.size(0), N = x.size(2);
  const bool shared = pos.dim() == 2;
  expect((shared && pos.size(1) == N) || (pos.dim() == 3 && pos.size(1) == B && pos.size(2) == N),
         "expected positions [axes, B, N] or [axes, N]");
  const Tables t(a[2], a[3], a[4], dev);
  long long xs[3], os[3];
  for (int i = 0; i < 3; ++i) {
    xs[i] = stride_of(x, i);
    os[i] = stride_of(out, i);
  }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  return PyLong_FromLong(call_rope(dtype, x.data_ptr(), out.data_ptr(), size(B), size(x.size(1)), size(N), size(x.size(3)),
                                   xs, os, t.positions, t.axis_stride, shared ? 0 : pos.stride(1), t.axes, t.inv_freq,
                                   t.axis, t.rot, truth(a[5]), truth(a[6]), stream_of(a[7], dev)));
}

// q, k, v, q_out, cache_k, cache_v, slot, positions, inv_freq, axis, pairs, stream
PyObject* append(PyObject* const* a) {
  const Cache cache(a[4], a[5]);
  const int dev = cache.dev;
  const long long T = tensor(a[1], "k").dim() ? tensor(a[1], "k").size(0) : 0;
  const fa_rows k = rows_of(a[1], "k", cache, T, cache.c.H_kv), v = rows_of(a[2], "v", cache, T, cache.c.H_kv);
  expect((a[0] == Py_None) == (a[3] == Py_None), "q and q_out go together");
  expect(tensor(a[6], "slot").numel() == T, "slot and k hold the same rows");
  fa_rows q{}, q_out{};
  int heads = 0;
  const bool with_q = a[0] != Py_None;
  if (with_q) {
    q = rows_of(a[0], "q", cache, T, -1);
    heads = size(tensor(a[0], "q").size(1));
    q_out = rows_of(a[3], "q_out", cache, T, heads);
  }
  Tables t;
  if (a[7] != Py_None) {
    const at::Tensor& pos = tensor(a[7], "positions");
    expect(pos.dim() == 2 && pos.size(1) == T, "expected positions [axes, T]");
    t = Tables(a[7], a[8], a[9], dev);
  }
  const int32_t* slot = ints(a[6], "slot", dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  return PyLong_FromLong(call_append(&cache.c, size(T), heads, with_q ? &q : nullptr, &k, &v, with_q ? &q_out : nullptr, slot,
                                     t.positions, t.axis_stride, t.axes, t.inv_freq, t.axis, t.rot, truth(a[10]),
                                     stream_of(a[11], dev)));
}

// q, cache_k, cache_v, block_table, seq_len, cu_q, o, lse, workspace, max_q, tree_mask, scale, stream
PyObject* tree(PyObject* const* a) {
  const Cache cache(a[1], a[2]);
  const int dev = cache.dev;
  const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "block_table"), &lse = tensor(a[7], "lse"),
                   &ws = tensor(a[8], "workspace");
  expect(q.dim() == 3, "expected q [T, Hq, d]");
  const long long T = q.size(0), Hq = q.size(1), B = tensor(a[4], "seq_len").numel(), max_q = integer(a[9]);
  const fa_rows qr = rows_of(a[0], "q", cache, T, Hq), orows = rows_of(a[6], "o", cache, T, Hq);
  expect(table.dim() == 2 && table.size(0) == B && tensor(a[5], "cu_q").numel() == B + 1,
         "expected block_table [B, max_pages], seq_len [B], cu_q [B+1]");
  expect(lse.dim() == 2 && lse.size(0) == T && lse.size(1) == Hq, "expected lse [T, Hq]");
  expect(ws.is_contiguous() && ws.is_cuda() && ws.get_device() == dev, "expected a contiguous workspace on the same device");
  expect(ws.nbytes() >= call_tree_workspace(size(B), size(T), size(max_q), size(Hq), cache.c.H_kv, cache.c.d),
         "workspace is smaller than fa_tree_fwd_workspace_size");
  int64_t* mask = nullptr;
  if (a[10] != Py_None) {
    const at::Tensor& m = tensor(a[10], "tree_mask");
    expect(m.dim() == 2 && m.size(0) == T && m.size(1) == (max_q + 63) / 64, "expected tree_mask [T, ceil(max_q/64)]");
    mask = plain<int64_t>(a[10], "tree_mask", at::kLong, dev);
  }
  const int32_t *tb = ints(a[3], "block_table", dev), *len = ints(a[4], "seq_len", dev), *cu = ints(a[5], "cu_q", dev);
  float* out = plain<float>(a[7], "lse", at::kFloat, dev);
  const float scale = static_cast<float>(real(a[11]));
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  return PyLong_FromLong(call_tree(&cache.c, &qr, &orows, out, size(B), size(T), size(max_q), size(Hq), size(table.size(1)),
                                   tb, cu, len, reinterpret_cast<const uint64_t*>(mask), scale, ws.data_ptr(),
                                   stream_of(a[12], dev)));
}

// cache_k, cache_v, block_table, ctx_len, accepted, n_accepted, new_len, stream
PyObject* commit(PyObject* const* a) {
  const Cache cache(a[0], a[1]);
  const int dev = cache.dev;
  const at::Tensor &table = tensor(a[2], "block_table"), &acc = tensor(a[4], "accepted");
  const long long B = tensor(a[3], "ctx_len").numel();
  expect(table.dim() == 2 && acc.dim() == 2 && table.size(0) == B && acc.size(0) == B &&
             tensor(a[5], "n_accepted").numel() == B && tensor(a[6], "new_len").numel() == B,
         "expected block_table [B, max_pages], accepted [B, max_accept], n_accepted and new_len [B]");
  const int32_t *tb = ints(a[2], "block_table", dev), *ctx = ints(a[3], "ctx_len", dev), *ac = ints(a[4], "accepted", dev),
                *n = ints(a[5], "n_accepted", dev);
  int32_t* out = ints(a[6], "new_len", dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  return PyLong_FromLong(call_commit(&cache.c, size(B), size(table.size(1)), size(acc.size(1)), tb, ctx, ac, n, out,
                                     stream_of(a[7], dev)));
}

// Counts the arguments and keeps C++ exceptions on this side.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 6>("bind"), method<plan, 14>("plan"),     method<rope, 8>("rope"),
                         method<append, 12>("append"), method<tree, 13>("tree"), method<commit, 8>("commit"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() {
  PyObject* m = PyModule_Create(&module);
  // The interpreter and torch that it was compiled against (the build passes them in).
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", FA_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
