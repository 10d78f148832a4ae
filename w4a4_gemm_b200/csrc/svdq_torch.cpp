// svdq_torch.cpp -- the cache operators' calls from Python, as a CPython module.
//
// These calls run once per layer and decode step, where the launch itself takes
// a few microseconds: the module reads torch's tensors directly, checks them, makes
// the outputs and calls the C entry points of libsvdq.so (include/svdq.h).  The
// functions take positional arguments only; the package's functions of the same
// names have the signatures, the defaults and the documentation.  A status other
// than SVDQ_OK comes back as an int, which the package turns into an SvdqError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/svdq.h"

namespace {

struct Refused {
  PyObject* type;
  std::string what;
};

[[noreturn]] void bad_type(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void bad_value(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, at::ScalarType dtype, const char* name, int dev) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) bad_type(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != dtype)
    bad_type(std::string(name) + " must be torch." + (dtype == at::kBFloat16 ? "bfloat16" : dtype == at::kInt ? "int32" : dtype == at::kLong ? "int64" : dtype == at::kFloat ? "float32" : "uint8"));
  if (t.get_device() != dev)
    bad_value(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the current device is cuda:" + std::to_string(dev));
  return t;
}

// A contiguous vector, of n elements unless n < 0.
const at::Tensor& array(PyObject* o, at::ScalarType dtype, const char* name, int dev, int64_t n = -1) {
  const at::Tensor& t = tensor(o, dtype, name, dev);
  if (t.dim() != 1 || (n >= 0 && t.size(0) != n))
    bad_value(std::string(name) + " must have shape (" + (n < 0 ? "n" : std::to_string(n)) + ",), got " + shape_text(t.sizes()));
  if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
  if (t.numel() > 0x7fffffffLL) bad_value(std::string(name) + " has too many elements");
  return t;
}

struct Rows {
  void* p;
  int64_t stride;
};

// rows x heads x dim bf16 whose heads are contiguous in a row.  Rows that are written must not overlap.
Rows check_rows(const at::Tensor& t, const char* name, int64_t rows, int64_t heads, int64_t dim, bool written = false) {
  if (t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != dim)
    bad_value(std::string(name) + " must have shape " + shape_text({rows, heads, dim}) + ", got " + shape_text(t.sizes()));
  if ((t.stride(2) != 1 && dim > 1) || (t.stride(1) != dim && heads > 1)) bad_value(std::string(name) + ": the heads of a row must be contiguous");
  const int64_t s = rows > 1 ? t.stride(0) : heads * dim;
  char* p = static_cast<char*>(t.data_ptr());
  if (s % 8 != 0 || reinterpret_cast<uintptr_t>(p) % 16 != 0) bad_value(std::string(name) + ": rows must start on 16-byte boundaries");
  if (written && rows > 1 && s < heads * dim) bad_value(std::string(name) + ": rows that are written must not overlap");
  return {p, s};
}
Rows rows_of(PyObject* o, const char* name, int dev, int64_t rows, int64_t heads, int64_t dim, bool written = false) {
  return check_rows(tensor(o, at::kBFloat16, name, dev), name, rows, heads, dim, written);
}

struct Table {
  int* p;
  int64_t stride, batch, width;
  at::Device device;
};

Table table_of(PyObject* o, int dev) {
  const at::Tensor& t = tensor(o, at::kInt, "block_table", dev);
  if (t.dim() != 2) bad_value("block_table must be batch x pages");
  const int64_t b = t.size(0), w = t.size(1);
  if (b > 0 && ((w > 1 && t.stride(1) != 1) || (b > 1 && t.stride(0) < w)))
    bad_value("block_table: the pages of a request must be contiguous, and its rows must not overlap");
  if (b > 0x7fffffffLL || w > 0x7fffffffLL) bad_value("block_table is too large");
  return {static_cast<int*>(t.data_ptr()), b > 1 ? t.stride(0) : w, b, w, t.device()};
}

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad_type(std::string(name) + " must be an integer");
  }
  return v;
}
int small(PyObject* o, const char* name) {
  const long long v = integer(o, name);
  if (v < -0x7fffffffLL || v > 0x7fffffffLL) bad_value(std::string(name) + " is out of range");
  return static_cast<int>(v);
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad_type(std::string(name) + " must be a number");
  }
  return v;
}
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    bad_type(std::string(name) + " must be a truth value");
  }
  return v == 1;
}

// The stream that the call runs on: the caller's (a cudaStream_t as an int; outputs are then allocated for
// it) or the current one.
struct Launch {
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  void* stream;
  Launch(PyObject* o, int dev) {
    if (o != Py_None) {
      cudaStream_t s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
      if (PyErr_Occurred()) {
        PyErr_Clear();
        bad_type("stream must be a torch.cuda.Stream");
      }
      guard.emplace(c10::cuda::getStreamFromExternal(s, static_cast<c10::DeviceIndex>(dev)));
      stream = s;
    } else {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    }
  }
};

int here() { return c10::cuda::current_device(); }

at::Tensor make(at::IntArrayRef shape, at::ScalarType dtype, at::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
}

// A cache description is a bytes object that holds an svdq_kv_cache, and the device of its pool.
struct Cache {
  svdq_kv_cache c;
  int device;
};
const Cache& cache_of(PyObject* o, int dev) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != sizeof(Cache)) bad_type("cache must be a KVCache");
  const Cache& c = *reinterpret_cast<const Cache*>(PyBytes_AS_STRING(o));
  if (c.device != dev)
    bad_value("the cache is on cuda:" + std::to_string(c.device) + ", the current device is cuda:" + std::to_string(dev));
  return c;
}

void need(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) bad_type("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

// (fmt, kv_heads, head_dim, page_size, pool) -> (description, bytes of a page); pool None: the bytes alone
PyObject* cache(PyObject* const* a, Py_ssize_t n) {
  need(n, 5);
  Cache c{};
  c.c = {small(a[0], "fmt"), small(a[1], "kv_heads"), small(a[2], "head_dim"), small(a[3], "page_size"), 0, nullptr};
  size_t bytes = 0;
  const int rc = svdq_kv_page_bytes(&c.c, &bytes);
  if (rc) return PyLong_FromLong(rc);
  if (a[4] == Py_None) return Py_BuildValue("On", Py_None, static_cast<Py_ssize_t>(bytes));
  if (!THPVariable_Check(a[4])) bad_type("pool must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(a[4]);
  if (!t.is_cuda()) bad_type("pool must be a CUDA tensor");
  if (t.scalar_type() != at::kByte) bad_type("pool must be torch.uint8");
  const int64_t block = static_cast<int64_t>(bytes) / c.c.kv_heads;
  if (t.dim() != 3 || t.size(1) != c.c.kv_heads || t.size(2) != block || !t.is_contiguous())
    bad_value("pool must be contiguous, [pages, " + std::to_string(c.c.kv_heads) + ", " + std::to_string(block) + "], got " + shape_text(t.sizes()));
  if (t.size(0) > 0x7fffffffLL) bad_value("pool has too many pages");
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0) bad_value("pool must start on a 16-byte boundary");
  c.c.num_pages = t.size(0);
  c.c.pool = t.data_ptr();
  c.device = t.get_device();
  return Py_BuildValue("y#n", reinterpret_cast<const char*>(&c), static_cast<Py_ssize_t>(sizeof c), static_cast<Py_ssize_t>(bytes));
}

// (q_lens, kv_lens, block_table, free_pages, rows, page_size, stream)
PyObject* kv_plan(PyObject* const* a, Py_ssize_t n) {
  need(n, 7);
  const int dev = here();
  const Table tb = table_of(a[2], dev);
  const at::Tensor& ql = array(a[0], at::kInt, "q_lens", dev, tb.batch);
  const at::Tensor& kl = array(a[1], at::kInt, "kv_lens", dev, tb.batch);
  const at::Tensor& free = array(a[3], at::kInt, "free_pages", dev);
  const int rows = small(a[4], "rows"), page = small(a[5], "page_size"), batch = static_cast<int>(tb.batch);
  if (rows < 0) bad_value("rows must not be negative");
  Launch on(a[6], dev);
  at::Tensor cu = make({batch + 1}, at::kInt, tb.device), total = make({batch}, at::kInt, tb.device);
  at::Tensor pos = make({rows}, at::kInt, tb.device), slots = make({rows}, at::kLong, tb.device), used = make({1}, at::kInt, tb.device);
  svdq_kv_plan_desc d{};
  d.q_lens = static_cast<const int*>(ql.data_ptr());
  d.kv_lens = static_cast<const int*>(kl.data_ptr());
  d.block_table = tb.p;
  d.table_stride = tb.stride;
  d.table_width = static_cast<int>(tb.width);
  d.free_pages = static_cast<const int*>(free.data_ptr());
  d.free_count = static_cast<int>(free.size(0));
  d.batch = batch;
  d.rows = rows;
  d.page_size = page;
  d.cu_q = static_cast<int*>(cu.data_ptr());
  d.total_lens = static_cast<int*>(total.data_ptr());
  d.positions = static_cast<int*>(pos.data_ptr());
  d.slots = static_cast<int64_t*>(slots.data_ptr());
  d.used = static_cast<int*>(used.data_ptr());
  const int rc = svdq_kv_plan(&d, on.stream);
  if (rc) return PyLong_FromLong(rc);
  return Py_BuildValue("NNNNN", THPVariable_Wrap(cu), THPVariable_Wrap(total), THPVariable_Wrap(pos), THPVariable_Wrap(slots), THPVariable_Wrap(used));
}

// (q, k, table, positions, q_weight, k_weight, eps, norm, interleaved, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject* const* a, Py_ssize_t n) {
  need(n, 12);
  const int dev = here();
  const at::Tensor& q = tensor(a[0], at::kBFloat16, "q", dev);
  const at::Tensor& k = tensor(a[1], at::kBFloat16, "k", dev);
  if (q.dim() != 3 || k.dim() != 3) bad_type("q and k must be rows x heads x dim tensors");
  const int64_t rows = q.size(0), hq = q.size(1), dim = q.size(2), hk = k.size(1);
  if (rows > 0x7fffffffLL || hq > 0x7fffffffLL || hk > 0x7fffffffLL || dim > 0x7fffffffLL) bad_value("q or k is too large");
  svdq_qk_norm_rope_desc d{};
  Rows r = check_rows(q, "q", rows, hq, dim);
  d.q = r.p, d.q_stride = r.stride;
  r = check_rows(k, "k", rows, hk, dim);
  d.k = r.p, d.k_stride = r.stride;
  if (a[2] != Py_None) {
    const at::Tensor& t = tensor(a[2], at::kFloat, "table", dev);
    if (t.dim() != 2 || !t.is_contiguous()) bad_value("table must be a contiguous positions x rot_dim tensor");
    if (t.size(0) > 0x7fffffffLL || t.size(1) > 0x7fffffffLL) bad_value("table is too large");
    d.table = static_cast<const float*>(t.data_ptr());
    d.table_rows = static_cast<int>(t.size(0));
    d.rot_dim = static_cast<int>(t.size(1));
  }
  if (a[3] != Py_None) d.positions = static_cast<const int*>(array(a[3], at::kInt, "positions", dev, rows).data_ptr());
  if (a[4] != Py_None) d.q_weight = array(a[4], at::kBFloat16, "q_weight", dev, dim).data_ptr();
  if (a[5] != Py_None) d.k_weight = array(a[5], at::kBFloat16, "k_weight", dev, dim).data_ptr();
  d.eps = static_cast<float>(number(a[6], "eps"));
  d.norm = truth(a[7], "norm");
  d.interleaved = truth(a[8], "interleaved");
  d.rows = static_cast<int>(rows);
  d.q_heads = static_cast<int>(hq);
  d.k_heads = static_cast<int>(hk);
  d.head_dim = static_cast<int>(dim);
  Launch on(a[11], dev);
  at::Tensor qo = a[9] == Py_None ? make({rows, hq, dim}, at::kBFloat16, q.device()) : tensor(a[9], at::kBFloat16, "q_out", dev);
  at::Tensor ko = a[10] == Py_None ? make({rows, hk, dim}, at::kBFloat16, q.device()) : tensor(a[10], at::kBFloat16, "k_out", dev);
  r = check_rows(qo, "q_out", rows, hq, dim, true);
  d.q_out = r.p, d.q_out_stride = r.stride;
  r = check_rows(ko, "k_out", rows, hk, dim, true);
  d.k_out = r.p, d.k_out_stride = r.stride;
  const int rc = svdq_qk_norm_rope(&d, on.stream);
  if (rc) return PyLong_FromLong(rc);
  return Py_BuildValue("NN", THPVariable_Wrap(qo), THPVariable_Wrap(ko));
}

// (cache, k, v, slots, stream)
PyObject* kv_append(PyObject* const* a, Py_ssize_t n) {
  need(n, 5);
  const int dev = here();
  const Cache& c = cache_of(a[0], dev);
  const at::Tensor& slots = array(a[3], at::kLong, "slots", dev);
  const int64_t rows = slots.size(0);
  const Rows k = rows_of(a[1], "k", dev, rows, c.c.kv_heads, c.c.head_dim), v = rows_of(a[2], "v", dev, rows, c.c.kv_heads, c.c.head_dim);
  Launch on(a[4], dev);
  const int rc = svdq_kv_append(&c.c, k.p, v.p, k.stride, v.stride, static_cast<const int64_t*>(slots.data_ptr()), static_cast<int>(rows), on.stream);
  if (rc) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
}

// (cache, slots, fp32, stream)
PyObject* kv_read(PyObject* const* a, Py_ssize_t n) {
  need(n, 4);
  const int dev = here();
  const Cache& c = cache_of(a[0], dev);
  const at::Tensor& slots = array(a[1], at::kLong, "slots", dev);
  const bool fp32 = truth(a[2], "fp32");
  Launch on(a[3], dev);
  const at::ScalarType dtype = fp32 ? at::kFloat : at::kBFloat16;
  at::Tensor k = make({slots.size(0), c.c.kv_heads, c.c.head_dim}, dtype, slots.device());
  at::Tensor v = make({slots.size(0), c.c.kv_heads, c.c.head_dim}, dtype, slots.device());
  const int rc = svdq_kv_read(&c.c, static_cast<const int64_t*>(slots.data_ptr()), static_cast<int>(slots.size(0)), fp32, k.data_ptr(), v.data_ptr(), on.stream);
  if (rc) return PyLong_FromLong(rc);
  return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
}

// (cache, q_heads, rows, batch) -> bytes
PyObject* kv_attention_workspace_bytes(PyObject* const* a, Py_ssize_t n) {
  need(n, 4);
  if (!PyBytes_Check(a[0]) || PyBytes_GET_SIZE(a[0]) != sizeof(Cache)) bad_type("cache must be a KVCache");
  svdq_kv_attention_desc d{};
  d.cache = reinterpret_cast<const Cache*>(PyBytes_AS_STRING(a[0]))->c;
  d.q_heads = small(a[1], "q_heads");
  d.rows = small(a[2], "rows");
  d.batch = small(a[3], "batch");
  size_t bytes = 0;
  const int rc = svdq_kv_attention_workspace_bytes(&d, &bytes);
  if (rc) return Py_BuildValue("(i)", rc);
  return PyLong_FromSize_t(bytes);
}

// (cache, q, cu_q, kv_lens, block_table, scale, causal, window, out, return_lse, workspace, stream)
PyObject* kv_attention(PyObject* const* a, Py_ssize_t n) {
  need(n, 12);
  const int dev = here();
  const Cache& c = cache_of(a[0], dev);
  const at::Tensor& q = tensor(a[1], at::kBFloat16, "q", dev);
  if (q.dim() != 3) bad_type("q must be a rows x heads x dim tensor");
  const int64_t rows = q.size(0), heads = q.size(1), dim = q.size(2);
  if (dim != c.c.head_dim) bad_value("q has head_dim " + std::to_string(dim) + ", the cache has " + std::to_string(c.c.head_dim));
  if (rows > 0x7fffffffLL || heads > 0x7fffffffLL) bad_value("q is too large");
  svdq_kv_attention_desc d{};
  d.cache = c.c;
  Rows r = check_rows(q, "q", rows, heads, dim);
  d.q = r.p, d.q_stride = r.stride;
  const Table tb = table_of(a[4], dev);
  d.cu_q = static_cast<const int*>(array(a[2], at::kInt, "cu_q", dev, tb.batch + 1).data_ptr());
  d.kv_lens = static_cast<const int*>(array(a[3], at::kInt, "kv_lens", dev, tb.batch).data_ptr());
  d.block_table = tb.p;
  d.table_stride = tb.stride;
  d.table_width = static_cast<int>(tb.width);
  d.batch = static_cast<int>(tb.batch);
  d.rows = static_cast<int>(rows);
  d.q_heads = static_cast<int>(heads);
  d.scale = a[5] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim))) : static_cast<float>(number(a[5], "scale"));
  d.causal = truth(a[6], "causal");
  d.window = small(a[7], "window");
  Launch on(a[11], dev);
  at::Tensor out = a[8] == Py_None ? make({rows, heads, dim}, at::kBFloat16, q.device()) : tensor(a[8], at::kBFloat16, "out", dev);
  r = check_rows(out, "out", rows, heads, dim, true);
  d.out = r.p, d.out_stride = r.stride;
  at::Tensor lse;
  if (truth(a[9], "return_lse")) {
    lse = make({rows, heads}, at::kFloat, q.device());
    d.lse = static_cast<float*>(lse.data_ptr());
  }
  size_t bytes = 0;
  int rc = svdq_kv_attention_workspace_bytes(&d, &bytes);
  if (rc) return PyLong_FromLong(rc);
  at::Tensor ws;
  if (a[10] == Py_None) {
    ws = make({static_cast<int64_t>(bytes)}, at::kByte, q.device());
  } else {
    ws = tensor(a[10], at::kByte, "workspace", dev);
    if (ws.dim() != 1 || !ws.is_contiguous()) bad_value("workspace must be a contiguous vector");
    if (ws.numel() < static_cast<int64_t>(bytes)) bad_value("workspace too small");
  }
  d.workspace = ws.data_ptr();
  rc = svdq_kv_attention(&d, on.stream);
  if (rc) return PyLong_FromLong(rc);
  if (lse.defined()) return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
  return THPVariable_Wrap(out);
}

// No C++ exception leaves a call.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

#define SVDQ_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SVDQ_METHOD(cache),         SVDQ_METHOD(kv_plan),  SVDQ_METHOD(qk_norm_rope), SVDQ_METHOD(kv_append),
                         SVDQ_METHOD(kv_read),       SVDQ_METHOD(kv_attention_workspace_bytes), SVDQ_METHOD(kv_attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "svdq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_svdq_torch(void) { return PyModule_Create(&module); }
