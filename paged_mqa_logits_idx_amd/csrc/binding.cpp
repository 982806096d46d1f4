// binding.cpp -- the Python side of include/kv_cache.h: checks tensors, takes their
// addresses, sizes and strides and calls the library's entry points.  A call on a few
// tokens takes the GPU a few microseconds and the host not much less for the launch;
// the same checks in Python took another five to ten.
//
// The module is the package's own and its functions take positional arguments; the
// package binds them to the library's entry points by address when it is imported.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "kv_cache.h"

namespace {

// The library's functions, in the order in which bind() takes their addresses.
struct Library {
  decltype(&idx_plan_batch) plan_batch;
  decltype(&idx_store_kv_fp8) store_kv_fp8;
  decltype(&idx_store_kv_bf16) store_kv_bf16;
  decltype(&idx_page_bounds_fp8) page_bounds_fp8;
  decltype(&idx_page_bounds_bf16) page_bounds_bf16;
  decltype(&idx_page_scores) page_scores;
  decltype(&idx_kv_attention_fp8) kv_attention_fp8;
  decltype(&idx_kv_attention_bf16) kv_attention_bf16;
  decltype(&idx_kv_attention_workspace) kv_attention_workspace;
} lib;
constexpr int kFunctions = 9;
static_assert(sizeof(Library) == kFunctions * sizeof(void*));

PyObject* make_workspace = nullptr;  // (bytes, stream) -> tensor, for streams that are not the current one

struct Refused {};  // a Python error is set

template <class... T>
[[noreturn]] void refuse(const char* text, T... args) {
  PyErr_Format(PyExc_ValueError, text, args...);
  throw Refused();
}

std::string text_of(at::IntArrayRef shape) {
  std::string s = "[";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "]";
}

const char* text_of(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return at::toString(t);
  }
}

const at::Tensor& tensor(const char* name, PyObject* x) {
  if (!THPVariable_Check(x)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(x);
}

void typed(const char* name, const at::Tensor& x, at::ScalarType type) {
  if (x.scalar_type() != type) refuse("%s must be %s, got %s", name, text_of(type), text_of(x.scalar_type()));
}

// All arguments are on the device of the first.
struct Place {
  at::Device device;
  explicit Place(const at::Tensor& x) : device(x.device()) {}
  void check(const char* name, const at::Tensor& x) const {
    if (x.device() != device)
      refuse("%s is on %s, the arguments before it on %s", name, x.device().str().c_str(), device.str().c_str());
  }
};

// Address of a contiguous tensor of this type and n elements.
template <class T = void>
T* flat(const char* name, PyObject* object, at::ScalarType type, int64_t n, const Place& place) {
  const at::Tensor& x = tensor(name, object);
  typed(name, x, type);
  if (x.numel() != n) refuse("%s must be of %lld elements, got %s", name, (long long)n, text_of(x.sizes()).c_str());
  if (!x.is_contiguous()) refuse("%s must be contiguous", name);
  place.check(name, x);
  return static_cast<T*>(x.data_ptr());
}

template <class T = void>
T* optional(const char* name, PyObject* object, at::ScalarType type, int64_t n, const Place& place) {
  return object == Py_None ? nullptr : flat<T>(name, object, type, n, place);
}

struct Grid {
  int32_t* at;
  int64_t rows, width, step;
};

// An int32 table.
Grid grid(const char* name, PyObject* object, const Place& place) {
  const at::Tensor& x = tensor(name, object);
  typed(name, x, at::kInt);
  if (x.dim() != 2) refuse("%s must have two dims", name);
  if (x.size(1) > 1 && x.stride(1) != 1) refuse("%s must be unit-stride along its last dim", name);
  place.check(name, x);
  return {static_cast<int32_t*>(x.data_ptr()), x.size(0), x.size(1), x.stride(0)};
}

struct Table {
  int32_t *at, *row_table;
  int64_t tables, width, step;
};

Table table(PyObject* page_table, PyObject* row_table, int64_t rows, const Place& place) {
  const Grid g = grid("page_table", page_table, place);
  Table t = {g.at, nullptr, 0, g.width, g.step};
  if (row_table != Py_None) {
    t.row_table = flat<int32_t>("row_table", row_table, at::kInt, rows, place);
    t.tables = g.rows;
  } else if (g.rows == 1) {
    t.step = 0;
  } else if (g.rows < rows) {
    refuse("page_table holds %lld tables for %lld rows", (long long)g.rows, (long long)rows);
  }
  return t;
}

// Bytes between pages and heads of a pool of blocks: [pages, heads, *block], dense
// behind its first two dims.
struct Pool {
  void* at;
  int64_t pages, heads, page, head;
};

Pool pool(const char* name, PyObject* object, bool typed_so, const char* types, std::initializer_list<int64_t> block,
          const Place& place) {
  const at::Tensor& x = tensor(name, object);
  if (!typed_so) refuse("%s must be %s, got %s", name, types, text_of(x.scalar_type()));
  const at::IntArrayRef shape = x.sizes(), step = x.strides();
  bool fits = shape.size() == 2 + block.size(), dense = true;
  int64_t values = 1;
  for (size_t i = block.size(); fits && i-- > 0;) {
    fits = shape[2 + i] == block.begin()[i];
    dense = dense && step[2 + i] == values;
    values *= block.begin()[i];
  }
  if (!fits) {
    const std::string want = text_of(at::IntArrayRef(block.begin(), block.size()));
    refuse("%s must be [pages, kv_heads, %s, got %s", name, want.c_str() + 1, text_of(shape).c_str());
  }
  if (!dense) refuse("%s must be dense behind its first two dims", name);
  place.check(name, x);
  const int64_t size = x.element_size(), page = shape[0] > 1 || step[0] > values ? step[0] : values;
  return {x.data_ptr(), shape[0], shape[1], page * size, step[1] * size};
}

// Address of a pool of the type, shape and strides of the one before it.
void* alike(const char* name, PyObject* object, const at::Tensor& first, const Place& place) {
  const at::Tensor& x = tensor(name, object);
  if (x.scalar_type() != first.scalar_type() || x.sizes() != first.sizes())
    refuse("%s must be %s %s, as the one before it", name, text_of(first.scalar_type()), text_of(first.sizes()).c_str());
  if (x.strides() != first.strides()) refuse("%s must have the strides of the one before it", name);
  place.check(name, x);
  return x.data_ptr();
}

struct Pools {
  void *keys, *values;
  float *kscale, *vscale;
  int64_t pages, heads, page, head, scale_page, scale_head;
};

// values == nullptr: keys alone.
Pools pools(bool fp8, PyObject* keys, PyObject* values, PyObject* kscale, PyObject* vscale, int64_t dim, const Place& place) {
  const at::Tensor& k = tensor("k_pages", keys);
  const at::ScalarType type = k.scalar_type();
  const Pool kv = fp8 ? pool("k_pages", keys, type == at::kByte || type == at::kFloat8_e4m3fn, "torch.uint8 or torch.float8_e4m3fn",
                             {IDX_PAGE_POSITIONS, dim}, place)
                      : pool("k_pages", keys, type == at::kBFloat16, "torch.bfloat16", {IDX_PAGE_POSITIONS, dim}, place);
  Pools p = {kv.at, nullptr, nullptr, nullptr, kv.pages, kv.heads, kv.page, kv.head, 0, 0};
  if (values) p.values = alike("v_pages", values, k, place);
  if (!fp8) return p;
  const at::Tensor& scale = tensor("kscale", kscale);
  const Pool ks = pool("kscale", kscale, scale.scalar_type() == at::kFloat, "torch.float32", {IDX_PAGE_POSITIONS}, place);
  if (ks.pages != kv.pages || ks.heads != kv.heads) refuse("kscale must be of the keys' pages and heads");
  p.kscale = static_cast<float*>(ks.at);
  p.scale_page = ks.page;
  p.scale_head = ks.head;
  if (values) p.vscale = static_cast<float*>(alike("vscale", vscale, scale, place));
  return p;
}

int64_t integer(PyObject* x) {
  const int64_t v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

// A whole number that the library takes in 32 bits; what does not fit it refuses too.
int32_t integer32(PyObject* x) {
  const int64_t v = integer(x);
  return v < INT32_MIN || v > INT32_MAX ? -1 : (int32_t)v;
}
int32_t size32(int64_t v) { return v > INT32_MAX ? -1 : (int32_t)v; }

// Pages of a pool, of which a call may take the first num_pages.
int64_t pages_taken(PyObject* num_pages, int64_t pages) {
  if (num_pages == Py_None) return pages;
  const int64_t n = integer(num_pages);
  if (n > pages) refuse("the pool holds %lld pages, not %lld", (long long)pages, (long long)n);
  return n;
}

// The handle of a torch stream, which must be of the arguments' device, or of a number.
hipStream_t handle_of(PyObject* stream, const Place& place) {
  PyObject* number = nullptr;
  if (PyObject_HasAttrString(stream, "cuda_stream")) {
    PyObject* index = PyObject_GetAttrString(stream, "device_index");
    if (!index) throw Refused();
    const int64_t device = PyLong_AsLongLong(index);
    Py_DECREF(index);
    if (device == -1 && PyErr_Occurred()) throw Refused();
    if (device != place.device.index()) refuse("stream is on cuda:%lld, the tensors on %s", (long long)device, place.device.str().c_str());
    number = PyObject_GetAttrString(stream, "cuda_stream");
  } else {
    number = PyNumber_Long(stream);
  }
  if (!number) throw Refused();
  void* handle = PyLong_AsVoidPtr(number);
  Py_DECREF(number);
  if (PyErr_Occurred()) throw Refused();
  return static_cast<hipStream_t>(handle);
}

// Calls f(stream) on the arguments' device, whatever the current one is.
template <class F>
PyObject* launch(const Place& place, PyObject* stream, F f) {
  if (!place.device.is_cuda()) refuse("tensors passed to the indexer library must be device tensors");
  const c10::DeviceGuard guard(place.device);
  const hipStream_t handle = stream == Py_None ? c10::hip::getCurrentHIPStream(place.device.index()).stream() : handle_of(stream, place);
  return PyLong_FromLong(f(handle));
}

template <class F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F f) {
  HANDLE_TH_ERRORS
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, have);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* plan_batch(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& first = tensor("cached", x[0]);
    const Place place(first);
    const int64_t requests = first.numel();
    const int32_t* cached = flat<int32_t>("cached", x[0], at::kInt, requests, place);
    const int32_t* added = flat<int32_t>("added", x[1], at::kInt, requests, place);
    const int64_t num_free = tensor("free_pages", x[2]).numel();
    const int32_t* free_pages = flat<int32_t>("free_pages", x[2], at::kInt, num_free, place);
    const Grid t = grid("page_table", x[3], place);
    if (t.rows != requests) refuse("page_table holds %lld tables for %lld requests", (long long)t.rows, (long long)requests);
    int64_t rows = 0;
    for (int i = 7; i >= 4; --i)
      if (x[i] != Py_None) rows = tensor("slots, positions, row_table and seqlens", x[i]).numel();
    int64_t* slots = optional<int64_t>("slots", x[4], at::kLong, rows, place);
    int64_t* positions = optional<int64_t>("positions", x[5], at::kLong, rows, place);
    int32_t* row_table = optional<int32_t>("row_table", x[6], at::kInt, rows, place);
    int32_t* seqlens = optional<int32_t>("seqlens", x[7], at::kInt, rows, place);
    int64_t* starts = optional<int64_t>("starts", x[8], at::kLong, requests + 1, place);
    int64_t* taken = optional<int64_t>("taken", x[9], at::kLong, 1, place);
    return launch(place, x[10], [&](hipStream_t stream) {
      return lib.plan_batch(cached, added, size32(requests), free_pages, num_free, t.at, size32(t.width),
                            requests > 1 ? t.step : t.width, rows, slots, positions, row_table, seqlens, starts, taken, stream);
    });
  });
}

// Elements between the tokens of [n, heads, D], dense behind its first dim.
int64_t tokens(const char* name, const at::Tensor& x) {
  typed(name, x, at::kBFloat16);
  if (x.dim() != 3) refuse("%s must have 3 dims, got %s", name, text_of(x.sizes()).c_str());
  const int64_t heads = x.size(1), dim = x.size(2);
  if ((dim > 1 && x.stride(2) != 1) || (heads > 1 && x.stride(1) != dim)) refuse("%s must be dense behind its first dim", name);
  return x.size(0) > 1 ? x.stride(0) : heads * dim;
}

PyObject* store_kv(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const bool fp8 = x[0] == Py_True;
    const at::Tensor &keys = tensor("keys", x[1]), &values = tensor("values", x[2]);
    const Place place(keys);
    const int64_t k_step = tokens("keys", keys), v_step = tokens("values", values);
    if (values.sizes() != keys.sizes()) refuse("values must be %s, got %s", text_of(keys.sizes()).c_str(), text_of(values.sizes()).c_str());
    place.check("values", values);
    const int64_t count = keys.size(0), heads = keys.size(1), dim = keys.size(2);
    const int64_t* slots = flat<int64_t>("slots", x[3], at::kLong, count, place);
    const Pools p = pools(fp8, x[4], x[5], x[6], x[7], dim, place);
    if (p.heads != heads) refuse("k_pages must have %lld heads, got %lld", (long long)heads, (long long)p.heads);
    const int64_t pages = pages_taken(x[8], p.pages);
    return launch(place, x[9], [&](hipStream_t stream) {
      return fp8 ? lib.store_kv_fp8(keys.data_ptr(), values.data_ptr(), slots, count, size32(heads), size32(dim), k_step, v_step,
                                    p.keys, p.values, p.kscale, p.vscale, pages, p.page, p.head, p.scale_page, p.scale_head, stream)
                 : lib.store_kv_bf16(keys.data_ptr(), values.data_ptr(), slots, count, size32(heads), size32(dim), k_step, v_step,
                                     p.keys, p.values, pages, p.page, p.head, stream);
    });
  });
}

PyObject* page_bounds(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const bool fp8 = x[0] == Py_True;
    const at::Tensor &keys = tensor("k_pages", x[1]), &lengths = tensor("seqlens", x[4]), &bounds = tensor("bounds", x[5]);
    const Place place(lengths);
    const int64_t rows = lengths.numel(), dim = keys.dim() > 0 ? keys.size(-1) : 0;
    const int32_t* seqlens = flat<int32_t>("seqlens", x[4], at::kInt, rows, place);
    const Table t = table(x[3], x[7], rows, place);
    const Pools p = pools(fp8, x[1], nullptr, x[2], nullptr, dim, place);
    const int64_t pages = pages_taken(x[8], p.pages);
    if (bounds.dim() != 4 || bounds.size(0) < pages || bounds.size(1) != p.heads || bounds.size(2) != 2 || bounds.size(3) != dim)
      refuse("bounds must be [%lld, %lld, 2, %lld], got %s", (long long)pages, (long long)p.heads, (long long)dim,
             text_of(bounds.sizes()).c_str());
    void* out = flat("bounds", x[5], at::kBFloat16, bounds.numel(), place);
    const int32_t* first = optional<int32_t>("first", x[6], at::kInt, rows, place);
    return launch(place, x[9], [&](hipStream_t stream) {
      return fp8 ? lib.page_bounds_fp8(p.keys, p.kscale, t.at, t.row_table, size32(t.tables), first, seqlens, out, size32(rows),
                                       size32(p.heads), size32(dim), size32(t.width), pages, p.page, p.head, p.scale_page,
                                       p.scale_head, t.step, stream)
                 : lib.page_bounds_bf16(p.keys, t.at, t.row_table, size32(t.tables), first, seqlens, out, size32(rows),
                                        size32(p.heads), size32(dim), size32(t.width), pages, p.page, p.head, t.step, stream);
    });
  });
}

PyObject* page_scores(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor &q = tensor("q", x[0]), &bounds = tensor("bounds", x[1]), &scores = tensor("scores", x[4]);
    if (q.dim() != 3 || bounds.dim() != 4 || bounds.size(2) != 2 || bounds.size(3) != q.size(2))
      refuse("q must be [rows, heads, D] and bounds [pages, kv_heads, 2, D], got %s and %s", text_of(q.sizes()).c_str(),
             text_of(bounds.sizes()).c_str());
    const Place place(q);
    const int64_t rows = q.size(0), heads = q.size(1), dim = q.size(2), pages = bounds.size(0), kv_heads = bounds.size(1);
    const void* from_q = flat("q", x[0], at::kBFloat16, q.numel(), place);
    const void* near = flat("bounds", x[1], at::kBFloat16, bounds.numel(), place);
    const int32_t* seqlens = flat<int32_t>("seqlens", x[3], at::kInt, rows, place);
    const Table t = table(x[2], x[8], rows, place);
    typed("scores", scores, at::kFloat);
    if (scores.dim() != 3 || scores.size(0) != rows || scores.size(1) != kv_heads || scores.size(2) != t.width)
      refuse("scores must be [%lld, %lld, %lld], got %s", (long long)rows, (long long)kv_heads, (long long)t.width,
             text_of(scores.sizes()).c_str());
    place.check("scores", scores);
    const int64_t apart = kv_heads > 1 ? scores.stride(1) : rows > 1 ? scores.stride(0) : t.width;
    if ((t.width > 1 && scores.stride(2) != 1) || (rows > 1 && kv_heads > 1 && scores.stride(0) != kv_heads * scores.stride(1)))
      refuse("scores must be unit-stride along its last dim, its rows evenly apart");
    int32_t* counts = optional<int32_t>("page_counts", x[5], at::kInt, rows * kv_heads, place);
    const int32_t first = integer32(x[6]), last = integer32(x[7]);
    return launch(place, x[9], [&](hipStream_t stream) {
      return lib.page_scores(from_q, near, t.at, t.row_table, size32(t.tables), seqlens, static_cast<float*>(scores.data_ptr()),
                             counts, size32(rows), size32(heads), size32(kv_heads), size32(dim), size32(t.width), pages, t.step,
                             apart, first, last, stream);
    });
  });
}

PyObject* kv_attention(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    const bool fp8 = x[0] == Py_True;
    const at::Tensor &q = tensor("q", x[1]), &out = tensor("out", x[9]);
    if (q.dim() != 3 || out.sizes() != q.sizes())
      refuse("q and out must be [rows, heads, D], got %s and %s", text_of(q.sizes()).c_str(), text_of(out.sizes()).c_str());
    const Place place(q);
    const int64_t rows = q.size(0), heads = q.size(1), dim = q.size(2);
    const void* from_q = flat("q", x[1], at::kBFloat16, q.numel(), place);
    void* to = flat("out", x[9], at::kBFloat16, q.numel(), place);
    const Pools p = pools(fp8, x[2], x[3], x[4], x[5], dim, place);
    const Table t = table(x[6], x[13], rows, place);
    const int32_t* seqlens = flat<int32_t>("seqlens", x[8], at::kInt, rows, place);
    int64_t k = -1;
    const int32_t* page_idx = nullptr;
    if (x[7] != Py_None) {
      const at::Tensor& listed = tensor("page_idx", x[7]);
      k = listed.dim() > 0 ? listed.size(-1) : 0;
      page_idx = flat<int32_t>("page_idx", x[7], at::kInt, rows * p.heads * k, place);
    }
    const float* sinks = optional<float>("sinks", x[12], at::kFloat, heads, place);
    float* lse = optional<float>("lse", x[10], at::kFloat, rows * heads, place);
    const int64_t pages = pages_taken(x[15], p.pages);
    const double scale = PyFloat_AsDouble(x[11]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused();
    at::Tensor workspace;
    if (x[14] != Py_None) {
      workspace = tensor("workspace", x[14]);
      if (!workspace.is_contiguous()) refuse("workspace must be contiguous");
      place.check("workspace", workspace);
    }
    return launch(place, x[16], [&](hipStream_t stream) {
      if (!workspace.defined()) {
        const int64_t need = lib.kv_attention_workspace(size32(rows), size32(heads), size32(p.heads), size32(dim), size32(t.width),
                                                        size32(k));
        if (need > 0 && x[16] == Py_None) {
          workspace = at::empty({need}, at::TensorOptions(at::kByte).device(place.device));
        } else if (need > 0) {
          PyObject* made = PyObject_CallFunction(make_workspace, "LO", (long long)need, x[16]);
          if (!made) throw Refused();
          workspace = THPVariable_Unpack(made);
          Py_DECREF(made);
        }
      }
      void* space = workspace.defined() && workspace.nbytes() > 0 ? workspace.data_ptr() : nullptr;
      const int64_t bytes = workspace.defined() ? (int64_t)workspace.nbytes() : 0;
      return fp8 ? lib.kv_attention_fp8(from_q, p.keys, p.values, p.kscale, p.vscale, t.at, t.row_table, size32(t.tables), page_idx,
                                        seqlens, sinks, to, lse, size32(rows), size32(heads), size32(p.heads), size32(dim),
                                        size32(t.width), pages, p.page, p.head, p.scale_page, p.scale_head, t.step, size32(k),
                                        (float)scale, space, bytes, stream)
                 : lib.kv_attention_bf16(from_q, p.keys, p.values, t.at, t.row_table, size32(t.tables), page_idx, seqlens, sinks,
                                         to, lse, size32(rows), size32(heads), size32(p.heads), size32(dim), size32(t.width), pages,
                                         p.page, p.head, t.step, size32(k), (float)scale, space, bytes, stream);
    });
  });
}

// bind(make_workspace, address of each function)
PyObject* bind(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 1 + kFunctions, [&]() -> PyObject* {
    Py_INCREF(x[0]);
    Py_XDECREF(make_workspace);
    make_workspace = x[0];
    void** to = reinterpret_cast<void**>(&lib);
    for (int i = 0; i < kFunctions; ++i) to[i] = PyLong_AsVoidPtr(x[1 + i]);
    if (PyErr_Occurred()) throw Refused();
    Py_RETURN_NONE;
  });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(plan_batch), METHOD(store_kv), METHOD(page_bounds), METHOD(page_scores), METHOD(kv_attention),
                         METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
