// The Python face of the calls over a cache in 8 bits and of the pages' call: checks tensors, marshals them and calls the C ABI
// on the current stream.  These calls take 3 to 10 us on the GPU for a small batch; their checks and ctypes arguments took as long
// from Python (settling one tree: 11.3 us a call, 4.6 from here).  Arguments come by position from the functions of the package,
// None for one that is not given.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/sdv.h"

namespace {

// A Python error that is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* what) {
  PyErr_SetString(type, what);
  throw Raised{};
}
[[noreturn]] void value_error(const char* what) { raise(PyExc_ValueError, what); }

PyObject* sdv_error = nullptr;  // the package's SdvError
void check_status(int rc, const char* what) {
  if (rc == SDV_OK) return;
  if (PyObject* e = PyObject_CallFunction(sdv_error, "is", rc, what)) {
    PyErr_SetObject(sdv_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

using Tensor = at::Tensor;
const Tensor* tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
    throw Raised{};
  }
  return &THPVariable_Unpack(o);
}
const Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : tensor(o, what); }

int index_of(const Tensor& t) { return t.is_cuda() ? (int)t.get_device() : -1; }

// The address of a contiguous vector of n values on device `index`.
template <class T>
T* vector(const Tensor& t, at::ScalarType type, int64_t n, int index, const char* what, const char* type_name) {
  if (t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && index_of(t) == index && t.is_contiguous())
    return static_cast<T*>(t.data_ptr());
  PyErr_Format(PyExc_ValueError, "%s must be a contiguous torch.%s vector of %lld values on the call's device", what, type_name,
               (long long)n);
  throw Raised{};
}
int32_t* ints(const Tensor& t, int64_t n, int index, const char* what) {
  return vector<int32_t>(t, at::kInt, n, index, what, "int32");
}

// A Python number for a 32-bit argument; what lies beyond becomes the nearest.
int32_t int32_of(PyObject* o) {
  int over = 0;
  const long long n = PyLong_AsLongLongAndOverflow(o, &over);
  if (n == -1 && !over && PyErr_Occurred()) throw Raised{};
  if (over > 0 || n > INT32_MAX) return INT32_MAX;
  return over < 0 || n < -INT32_MAX ? -INT32_MAX : (int32_t)n;
}

int dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return SDV_BF16;
  if (t.scalar_type() == at::kFloat) return SDV_FP32;
  raise(PyExc_TypeError, "rows over a cache in 8 bits must be bfloat16 or float32");
}

struct Call {
  sdv_cache8 c;
  int index;
  int32_t B;
  const int32_t* offsets;
};

// One layer's cache, or with `layers` [L, ...] of them.
Call cache_of(const Tensor& keys, const Tensor& values, const Tensor& table, const Tensor& len, const Tensor& offsets,
              const Tensor& key_scales, const Tensor& value_scales, int dtype, bool layers) {
  Call call;
  if (keys.scalar_type() != at::kFloat8_e4m3fn) raise(PyExc_TypeError, "a cache with scales must be float8_e4m3fn");
  call.index = index_of(keys);
  if (call.index < 0) value_error("the cache must be on the GPU");
  const int64_t dim = keys.dim();
  if ((dim != 4 && !(layers && dim == 5)) || !keys.is_contiguous())
    value_error("key_cache must be a contiguous [n_pages, n_kv_heads, page_size, head_dim] tensor");
  const auto shape = keys.sizes();
  if (values.scalar_type() != keys.scalar_type() || index_of(values) != call.index || values.sizes() != shape ||
      !values.is_contiguous())
    value_error("value_cache must be like key_cache");
  if (offsets.dim() != 1 || offsets.size(0) < 2 || offsets.size(0) > INT32_MAX)
    value_error("offsets must be a vector of B + 1 values");
  call.B = (int32_t)(offsets.size(0) - 1);
  call.offsets = ints(offsets, (int64_t)call.B + 1, call.index, "offsets");
  sdv_cache& c = call.c.cache;
  c.cache_len = ints(len, call.B, call.index, "cache_len");
  if (table.scalar_type() != at::kInt || index_of(table) != call.index || table.dim() != 2 || table.size(0) != call.B ||
      !table.is_contiguous())
    value_error("page_table must be a contiguous int32 [B, max_pages] tensor on the cache's device");
  const int64_t max_pages = table.size(1), heads = shape[dim - 3], page_size = shape[dim - 2], head_dim = shape[dim - 1];
  if (max_pages > INT32_MAX || heads > INT32_MAX || page_size > INT32_MAX || head_dim > INT32_MAX)
    value_error("sizes of the cache beyond 32 bits");
  const int64_t blocks = key_scales.dim() == dim - 1 ? key_scales.size(dim - 2) : 0;
  for (const Tensor* t : {&key_scales, &value_scales}) {
    bool ok = (t->scalar_type() == at::kByte || t->scalar_type() == at::kFloat8_e8m0fnu) && index_of(*t) == call.index &&
              blocks > 0 && page_size % blocks == 0 && t->dim() == dim - 1 && t->is_contiguous();
    for (int64_t d = 0; ok && d < dim - 1; ++d) ok = t->size(d) == (d < dim - 2 ? shape[d] : blocks);
    if (!ok)
      value_error("key_scales and value_scales must be contiguous uint8 or float8_e8m0fnu tensors "
                  "[n_pages, n_kv_heads, page_size / block] on the cache's device");
  }
  c.keys = keys.data_ptr();
  c.values = values.data_ptr();
  c.page_table = static_cast<const int32_t*>(table.data_ptr());
  c.n_pages = shape[dim - 4];
  c.max_pages = (int32_t)max_pages;
  c.page_size = (int32_t)page_size;
  c.n_kv_heads = (int32_t)heads;
  c.head_dim = (int32_t)head_dim;
  c.dtype = dtype;
  call.c.key_scales = static_cast<uint8_t*>(key_scales.data_ptr());
  call.c.value_scales = static_cast<uint8_t*>(value_scales.data_ptr());
  call.c.block = (int32_t)(page_size / blocks);
  return call;
}

// The row stride of a [rows, heads, head_dim] tensor whose heads lie next to each other (heads -1: any number).
int64_t rows_of(const Tensor& t, const char* what, int64_t rows, int64_t heads, const Call& call, at::ScalarType type) {
  const int64_t head_dim = call.c.cache.head_dim;
  if (t.scalar_type() == type && index_of(t) == call.index && t.dim() == 3 && t.size(0) == rows &&
      (heads < 0 || t.size(1) == heads) && t.size(2) == head_dim && t.stride(2) == 1 &&
      (t.stride(1) == head_dim || t.size(1) == 1) && t.size(1) <= INT32_MAX)
    return rows > 1 ? t.stride(0) : t.size(1) * head_dim;
  PyErr_Format(PyExc_ValueError,
               "%s must be a [n_draft_rows + B, heads, head_dim] tensor of the rows' dtype on the cache's device, each row "
               "contiguous",
               what);
  throw Raised{};
}

// `launch(stream)` with device `index` current, on its current stream.
template <class F>
int on(int index, F launch) {
  const int current = c10::hip::current_device();
  if (current != index) c10::hip::set_device(index);
  int rc = SDV_ERR_HIP;
  try {
    rc = launch(static_cast<void*>(c10::hip::getCurrentHIPStream(index).stream()));
  } catch (...) {
    if (current != index) c10::hip::set_device(current);
    throw;
  }
  if (current != index) c10::hip::set_device(current);
  return rc;
}

// The call's workspace: the one given, or the package's of this stream and thread.
struct Workspace {
  Tensor held;
  void* at = nullptr;
  size_t bytes = 0;
  void take(PyObject* given, PyObject* scratch, size_t need, PyObject* device, int index, void* stream) {
    if (given != Py_None) {
      held = *tensor(given, "workspace");
      if (index_of(held) != index || !held.is_contiguous())
        value_error("workspace must be a contiguous tensor on the call's device");
    } else if (need > 0) {
      PyObject* got = PyObject_CallFunction(scratch, "KOiK", (unsigned long long)need, device, index,
                                            (unsigned long long)reinterpret_cast<uintptr_t>(stream));
      if (!got) throw Raised{};
      const bool is_tensor = THPVariable_Check(got);
      if (is_tensor) held = THPVariable_Unpack(got);
      Py_DECREF(got);
      if (!is_tensor) raise(PyExc_TypeError, "workspace must be a tensor");
    } else {
      return;
    }
    at = held.data_ptr();
    bytes = held.nbytes();
  }
};

// f's result, with every C++ exception as the Python error that torch makes of it.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  HANDLE_TH_ERRORS
  try {
    if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
    return f();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// keys, values, key_cache, value_cache, page_table, cache_len, offsets, key_scales, value_scales, parents, inv_freq, interleaved,
// queries, queries_out
PyObject* kv_append8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Tensor &keys = *tensor(a[0], "keys"), &values = *tensor(a[1], "values");
    const int dtype = dtype_of(keys);
    const Call call = cache_of(*tensor(a[2], "key_cache"), *tensor(a[3], "value_cache"), *tensor(a[4], "page_table"),
                               *tensor(a[5], "cache_len"), *tensor(a[6], "offsets"), *tensor(a[7], "key_scales"),
                               *tensor(a[8], "value_scales"), dtype, false);
    const int64_t rows = keys.dim() > 0 ? keys.size(0) : 0, heads = call.c.cache.n_kv_heads;
    const auto type = keys.scalar_type();
    if (rows < call.B) value_error("keys must have n_draft_rows + B rows");
    const int64_t ks = rows_of(keys, "keys", rows, heads, call, type), vs = rows_of(values, "values", rows, heads, call, type);
    const Tensor *parents = maybe(a[9], "parents"), *freq = maybe(a[10], "inv_freq"), *queries = maybe(a[12], "queries"),
                 *given = maybe(a[13], "queries_out");
    const int32_t* p_parents = parents ? ints(*parents, rows - call.B, call.index, "parents") : nullptr;
    const int64_t pairs = freq ? freq->numel() : 0;
    const float* p_freq = freq ? vector<float>(*freq, at::kFloat, pairs, call.index, "inv_freq", "float32") : nullptr;
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) throw Raised{};
    int64_t qs = 0, n_q = 0;
    Tensor out;
    if (queries) {
      qs = rows_of(*queries, "queries", rows, -1, call, type);
      n_q = queries->size(1);
      if (!given)
        out = at::empty(queries->sizes(), keys.options());
      else if (given->scalar_type() != type || index_of(*given) != call.index || given->sizes() != queries->sizes() ||
               !given->is_contiguous())
        value_error("queries_out must be a contiguous tensor like queries");
      else
        out = *given;
    } else if (given) {
      value_error("queries_out without queries");
    }
    const int rc = on(call.index, [&](void* stream) {
      return sdv_kv_append8(&call.c, call.B, rows - call.B, call.offsets, p_parents, keys.data_ptr(), ks, values.data_ptr(), vs,
                            p_freq, (int32_t)(pairs > INT32_MAX / 2 ? INT32_MAX : 2 * pairs), interleaved,
                            queries ? queries->data_ptr() : nullptr, qs, (int32_t)n_q, queries ? out.data_ptr() : nullptr,
                            stream);
    });
    check_status(rc, "sdv_kv_append8");
    if (!queries) Py_RETURN_NONE;
    if (given) {
      Py_INCREF(a[13]);
      return a[13];
    }
    return THPVariable_Wrap(out);
  });
}

// queries, key_cache, value_cache, page_table, cache_len, offsets, key_scales, value_scales, parents, scale, window, sinks, out,
// workspace, the package's scratch, the cache's device
PyObject* attend8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const Tensor& queries = *tensor(a[0], "queries");
    const Call call = cache_of(*tensor(a[1], "key_cache"), *tensor(a[2], "value_cache"), *tensor(a[3], "page_table"),
                               *tensor(a[4], "cache_len"), *tensor(a[5], "offsets"), *tensor(a[6], "key_scales"),
                               *tensor(a[7], "value_scales"), dtype_of(queries), false);
    const int64_t rows = queries.dim() > 0 ? queries.size(0) : 0;
    const auto type = queries.scalar_type();
    const int64_t qs = rows_of(queries, "queries", rows, -1, call, type);
    if (rows < call.B) value_error("queries must have n_draft_rows + B rows");
    const int64_t n_q = queries.size(1), n_k = call.c.cache.n_kv_heads;
    if (n_q < 1 || n_k < 1 || n_q % n_k) value_error("the number of query heads must be a multiple of the cache's heads");
    const Tensor *parents = maybe(a[8], "parents"), *given = maybe(a[12], "out");
    const int32_t* p_parents = parents ? ints(*parents, rows - call.B, call.index, "parents") : nullptr;
    double scale = 1.0 / std::sqrt((double)call.c.cache.head_dim);
    if (a[9] != Py_None) {
      scale = PyFloat_AsDouble(a[9]);
      if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    }
    const int32_t window = int32_of(a[10]), sinks = int32_of(a[11]);  // slots are numbered below 2^31: what is larger sees no more
    if (given && (given->scalar_type() != type || index_of(*given) != call.index || given->sizes() != queries.sizes() ||
                  !given->is_contiguous()))
      value_error("out must be a contiguous tensor like queries");
    const Tensor out = given ? *given : at::empty(queries.sizes(), queries.options());
    const int rc = on(call.index, [&](void* stream) {
      Workspace ws;
      ws.take(a[13], a[14], sdv_attend8_workspace_bytes(&call.c, call.B, rows - call.B, (int32_t)n_q, window, sinks), a[15],
              call.index, stream);
      return sdv_attend8(&call.c, call.B, rows - call.B, call.offsets, p_parents, queries.data_ptr(), qs, (int32_t)n_q,
                         (float)scale, window, sinks, out.data_ptr(), ws.at, ws.bytes, stream);
    });
    check_status(rc, "sdv_attend8");
    if (given) {
      Py_INCREF(a[12]);
      return a[12];
    }
    return THPVariable_Wrap(out);
  });
}

// key_cache, value_cache, page_table, cache_len, offsets, accepted_len, accepted_nodes, key_scales, value_scales
PyObject* kv_settle8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensor &keys = *tensor(a[0], "key_cache"), &len = *tensor(a[3], "cache_len");
    const Call call = cache_of(keys, *tensor(a[1], "value_cache"), *tensor(a[2], "page_table"), len, *tensor(a[4], "offsets"),
                               *tensor(a[7], "key_scales"), *tensor(a[8], "value_scales"), SDV_BF16, true);
    const Tensor &accepted = *tensor(a[5], "accepted_len"), &nodes = *tensor(a[6], "accepted_nodes");
    const int64_t n_d = nodes.numel(), layers = keys.dim() == 5 ? keys.size(0) : 1;
    const int32_t* p_accepted = ints(accepted, call.B, call.index, "accepted_len");
    const int32_t* p_nodes = ints(nodes, n_d, call.index, "accepted_nodes");
    if (layers > INT32_MAX) value_error("sizes of the cache beyond 32 bits");
    const Tensor out = at::empty(len.sizes(), len.options());
    const int rc = on(call.index, [&](void* stream) {
      return sdv_kv_settle8(&call.c, (int32_t)layers, call.B, n_d, call.offsets, p_accepted, n_d ? p_nodes : nullptr,
                            static_cast<int32_t*>(out.data_ptr()), stream);
    });
    check_status(rc, "sdv_kv_settle8");
    return THPVariable_Wrap(out);
  });
}

// page_table, cache_len, offsets, n_draft_rows, free_pages, free_state, page_size, window, sinks, slots, placed, workspace, the
// package's scratch, the table's device
PyObject* kv_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Tensor &table = *tensor(a[0], "page_table"), &len = *tensor(a[1], "cache_len"), &offsets = *tensor(a[2], "offsets"),
                 &ring = *tensor(a[4], "free_pages"), &state = *tensor(a[5], "free_state");
    const int index = index_of(table);
    if (index < 0) value_error("page_table must be on the GPU");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || !table.is_contiguous())
      value_error("page_table must be a contiguous int32 [B, max_pages] tensor");
    const int64_t B = table.size(0), max_pages = table.size(1), n_pages = ring.numel();
    int over = 0;
    const long long n_d = PyLong_AsLongLongAndOverflow(a[3], &over);
    if (n_d == -1 && !over && PyErr_Occurred()) throw Raised{};
    if (B < 1 || over < 0 || n_d < 0) value_error("B >= 1 requests and n_draft_rows >= 0 rows are needed");
    if (over > 0 || B > INT32_MAX || max_pages > INT32_MAX || n_pages > INT32_MAX || n_d > INT32_MAX - B)
      value_error("sizes beyond 32 bits");
    const int32_t* p_len = ints(len, B, index, "cache_len");
    const int32_t* p_offsets = ints(offsets, B + 1, index, "offsets");
    int32_t* p_ring = ints(ring, n_pages, index, "free_pages");
    int32_t* p_state = ints(state, 2, index, "free_state");
    const Tensor *slots = maybe(a[9], "slots"), *placed = maybe(a[10], "placed");
    const Tensor to_slots = slots ? *slots : at::empty({n_d + B}, table.options().dtype(at::kLong));
    const Tensor to_placed = placed ? *placed : at::empty({B}, table.options());
    int64_t* p_slots = vector<int64_t>(to_slots, at::kLong, n_d + B, index, "slots", "int64");
    int32_t* p_placed = ints(to_placed, B, index, "placed");
    const int32_t page_size = int32_of(a[6]), window = int32_of(a[7]), sinks = int32_of(a[8]);
    const int rc = on(index, [&](void* stream) {
      Workspace ws;
      ws.take(a[11], a[12], sdv_kv_pages_workspace_bytes((int32_t)B, (int32_t)max_pages), a[13], index, stream);
      return sdv_kv_pages(static_cast<int32_t*>(table.data_ptr()), (int32_t)B, (int32_t)max_pages, page_size, p_len, n_d, p_offsets,
                          n_pages, p_ring, p_state, window, sinks, p_placed, p_slots, ws.at, ws.bytes, stream);
    });
    check_status(rc, "sdv_kv_pages");
    return Py_BuildValue("(NN)", THPVariable_Wrap(to_placed), THPVariable_Wrap(to_slots));
  });
}

// The package's error.
PyObject* bind(PyObject*, PyObject* error) {
  Py_XDECREF(sdv_error);
  Py_INCREF(error);
  sdv_error = error;
  Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"kv_append8", fast<kv_append8>(), METH_FASTCALL, nullptr},
                         {"attend8", fast<attend8>(), METH_FASTCALL, nullptr},
                         {"kv_settle8", fast<kv_settle8>(), METH_FASTCALL, nullptr},
                         {"kv_pages", fast<kv_pages>(), METH_FASTCALL, nullptr},
                         {"bind", bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
