// Python calls of the serving entry points (rotation, paged cache, candidates
// against it), as a CPython extension.
//
// A decode step is a few microseconds on the GPU, and a call through ctypes
// with its checks in Python took 13 us; here the same checks, the outputs'
// allocation and the launch take 4 to 5 us. The functions take the tensors as
// they are, check what the C ABI cannot see (types, shapes, strides, devices),
// and call the entry points of the library that binding.py has loaded; they
// compute nothing. binding.py holds the documented wrappers.
//
// A status other than HSTU_OK is returned as an integer and raised there.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/hstu_attn.h"

namespace {

// Entry points of the loaded library, set by bind().
decltype(&hstu_attn_rope) g_rope = nullptr;
decltype(&hstu_attn_cache_write) g_cache_write = nullptr;
decltype(&hstu_attn_cache_read) g_cache_read = nullptr;
decltype(&hstu_attn_cache_read) g_cache_read_zeroed = nullptr;
decltype(&hstu_attn_paged_workspace_size) g_paged_size = nullptr;
decltype(&hstu_attn_fwd_paged) g_fwd_paged = nullptr;

// A refusal, raised as ValueError.
struct Refused {
  std::string what;
};

std::string shape_text(at::IntArrayRef sizes) {
  std::string s = "(";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + (sizes.size() == 1 ? ",)" : ")");
}
std::string shape_text(std::initializer_list<int64_t> sizes) {
  return shape_text(at::IntArrayRef(sizes.begin(), sizes.size()));
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_none(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

void check_device(const at::Tensor& t, int index, const char* name) {
  if (!t.is_cuda()) throw Refused{std::string(name) + " must be a CUDA tensor"};
  if (t.get_device() != index)
    throw Refused{std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", not on cuda:" +
                  std::to_string(index)};
}

// The library launches on the current device.
void check_current(int index, const char* name) {
  if (index < 0) throw Refused{std::string(name) + " must be a CUDA tensor"};
  const int current = c10::cuda::current_device();
  if (index != current)
    throw Refused{std::string(name) + " is on cuda:" + std::to_string(index) + ", the current device is cuda:" +
                  std::to_string(current)};
}

at::ScalarType element(int dtype) { return dtype == HSTU_DTYPE_F16 ? at::kHalf : at::kBFloat16; }

void check_dtype(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    throw Refused{std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type())};
}

// A (rows, heads, width) tensor whose rows may lie apart (a slice of a wider
// projection); returns the distance between rows in elements.
int64_t check_rows(const at::Tensor& t, at::ScalarType type, int64_t heads, int64_t width, int index,
                   const char* name) {
  check_device(t, index, name);
  check_dtype(t, type, name);
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != width)
    throw Refused{std::string(name) + " must be (rows, " + std::to_string(heads) + ", " + std::to_string(width) +
                  "), got " + shape_text(t.sizes())};
  if (t.stride(2) != 1 || (t.stride(1) != width && heads > 1))
    throw Refused{std::string(name) + ": heads and columns of a row must be contiguous"};
  if (t.size(0) <= 1) return heads * width;
  if (t.stride(0) < heads * width) throw Refused{std::string(name) + ": rows overlap"};
  return t.stride(0);
}

const int32_t* check_ints(const at::Tensor& t, std::initializer_list<int64_t> shape, int index, const char* name) {
  check_device(t, index, name);
  check_dtype(t, at::kInt, name);
  if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
    throw Refused{std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes())};
  if (!t.is_contiguous()) throw Refused{std::string(name) + " must be contiguous"};
  return static_cast<const int32_t*>(t.data_ptr());
}

const int32_t* check_pages(const at::Tensor& t, int64_t batch, int index) {
  if (t.dim() != 2 || t.size(0) != batch || t.size(1) < 1)
    throw Refused{"page_table must be (batch = " + std::to_string(batch) + ", pages), got " + shape_text(t.sizes())};
  if (batch > INT32_MAX || t.size(1) > INT32_MAX) throw Refused{"page_table is too large"};
  return check_ints(t, {batch, t.size(1)}, index, "page_table");
}

// An output given by the caller: contiguous (rows, heads, width).
void check_output(const at::Tensor& t, at::ScalarType type, int64_t rows, int64_t heads, int64_t width, int index,
                  const char* name) {
  check_rows(t, type, heads, width, index, name);
  if (t.size(0) != rows || !t.is_contiguous())
    throw Refused{std::string(name) + " must be contiguous and have " + std::to_string(rows) + " rows"};
}

struct Workspace {
  void* ptr = nullptr;
  size_t bytes = 0;
};
Workspace check_ws(const at::Tensor* t, int index) {
  if (!t) return {};
  check_device(*t, index, "ws");
  if (!t->is_contiguous()) throw Refused{"ws must be contiguous"};
  if (t->nbytes() == 0) throw Refused{"ws is empty"};  // its address is null, as if none had been given
  return {t->data_ptr(), static_cast<size_t>(t->nbytes())};
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return p;
}

// The stream to launch on, whose memory the outputs are allocated from.
void* current_stream(int index) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
}

at::Tensor new_rows(int64_t rows, int64_t heads, int64_t width, at::ScalarType type, int index) {
  return at::empty({rows, heads, width},
                   at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
}

PyObject* pair(const at::Tensor& a, const std::optional<at::Tensor>& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = b ? THPVariable_Wrap(*b) : Py_NewRef(Py_None);
  PyObject* r = x && y ? PyTuple_New(2) : nullptr;
  if (!r) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    throw python_error();
  }
  PyTuple_SET_ITEM(r, 0, x);
  PyTuple_SET_ITEM(r, 1, y);
  return r;
}

// Calls an entry point without the interpreter's lock: a launch waits while the
// stream's queue is full.
template <typename F>
hstu_status_t without_lock(F&& call) {
  hstu_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return st;
}

void need_args(Py_ssize_t got, Py_ssize_t want) {
  if (got != want || !g_rope) throw Refused{"called by the wrappers of binding.py only"};
}

// rope(q, k, positions, table, table_device, backward, q_out, k_out)
PyObject* rope(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 8);
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor* k = tensor_or_none(a[1], "k");
  const at::ScalarType type = q.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf)
    throw Refused{std::string("q must be one of (torch.bfloat16, torch.float16), got ") + c10::toString(type)};
  const int index = q.is_cuda() ? q.get_device() : -1;
  check_current(index, "q");
  if (q.dim() != 3) throw Refused{"q must be (rows, heads, width), got " + shape_text(q.sizes())};
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
  const int64_t qs = check_rows(q, type, H, D, index, "q");
  int64_t ks = 0;
  if (k) {
    ks = check_rows(*k, type, H, D, index, "k");
    if (k->size(0) != T) throw Refused{"k must have q's shape " + shape_text(q.sizes()) + ", got " + shape_text(k->sizes())};
  }
  const int32_t* positions = check_ints(tensor(a[2], "positions"), {T}, index, "positions");
  const auto* table = static_cast<const hstu_rope_t*>(address(a[3]));
  if (integer(a[4]) != index) throw Refused{"table is on another device"};
  const at::Tensor* q_given = tensor_or_none(a[6], "outs[0]");
  const at::Tensor* k_given = tensor_or_none(a[7], "outs[1]");
  at::Tensor qo;
  std::optional<at::Tensor> ko;
  int64_t qos = H * D, kos = H * D;
  if (q_given || k_given) {
    if (!q_given || (k_given == nullptr) != (k == nullptr)) throw Refused{"outs must match q and k"};
    qo = *q_given;
    qos = check_rows(qo, type, H, D, index, "outs[0]");
    if (k) {
      ko = *k_given;
      kos = check_rows(*ko, type, H, D, index, "outs[1]");
    }
    if (qo.size(0) != T || (ko && ko->size(0) != T)) throw Refused{"outs must match q and k"};
  } else {
    qo = new_rows(T, H, D, type, index);
    if (k) ko = new_rows(T, H, D, type, index);
  }
  void* stream = current_stream(index);
  const int backward = a[5] == Py_True;
  const hstu_status_t st = without_lock([&] {
    return g_rope(q.data_ptr(), qs, k ? k->data_ptr() : nullptr, ks, qo.data_ptr(), qos, ko ? ko->data_ptr() : nullptr,
                  kos, positions, T, static_cast<int32_t>(H), static_cast<int32_t>(D),
                  type == at::kHalf ? HSTU_DTYPE_F16 : HSTU_DTYPE_BF16, table, backward, stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  return pair(qo, ko);
}

// cache_write(cache, cache_device, k, v, seq_offsets, cache_lens, page_table,
//             rope, rope_device, positions, ws)
PyObject* cache_write(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 11);
  const auto* cache = static_cast<const hstu_cache_t*>(address(a[0]));
  const int index = static_cast<int>(integer(a[1]));
  check_current(index, "cache");
  const at::ScalarType type = element(cache->dtype);
  const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  const int64_t ks = check_rows(k, type, cache->num_heads, cache->head_dim, index, "k");
  const int64_t vs = check_rows(v, type, cache->num_heads, cache->head_dim_v, index, "v");
  const int64_t T = k.size(0);
  if (v.size(0) != T)
    throw Refused{"k has " + std::to_string(T) + " rows, v " + std::to_string(v.size(0))};
  const at::Tensor &offsets = tensor(a[4], "seq_offsets"), &table = tensor(a[6], "page_table");
  const int64_t B = offsets.numel() - 1;
  const int32_t* off = check_ints(offsets, {B + 1}, index, "seq_offsets");
  const int32_t* lens = check_ints(tensor(a[5], "cache_lens"), {B}, index, "cache_lens");
  const int32_t* pages = check_pages(table, B, index);
  const auto* rope = static_cast<const hstu_rope_t*>(address(a[7]));
  if (rope && integer(a[8]) != index) throw Refused{"rope is on another device"};
  const at::Tensor* positions = tensor_or_none(a[9], "positions");
  const int32_t* pos = positions ? check_ints(*positions, {T}, index, "positions") : nullptr;
  const Workspace ws = check_ws(tensor_or_none(a[10], "ws"), index);
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    return g_cache_write(cache, k.data_ptr(), ks, v.data_ptr(), vs, off, static_cast<int32_t>(B), T, lens, pages,
                         static_cast<int32_t>(table.size(1)), rope, pos, ws.ptr, ws.bytes, stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  Py_RETURN_NONE;
}

// cache_read(cache, cache_device, seq_offsets, rows, page_table, starts, k_out,
//            v_out, ws)
PyObject* cache_read(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  const auto* cache = static_cast<const hstu_cache_t*>(address(a[0]));
  const int index = static_cast<int>(integer(a[1]));
  check_current(index, "cache");
  const at::ScalarType type = element(cache->dtype);
  const at::Tensor &offsets = tensor(a[2], "seq_offsets"), &table = tensor(a[4], "page_table");
  const int64_t B = offsets.numel() - 1, rows = integer(a[3]), H = cache->num_heads;
  if (rows < 0) throw Refused{"rows must not be negative"};
  const int32_t* off = check_ints(offsets, {B + 1}, index, "seq_offsets");
  const int32_t* pages = check_pages(table, B, index);
  const at::Tensor* starts = tensor_or_none(a[5], "starts");
  const int32_t* first = starts ? check_ints(*starts, {B}, index, "starts") : nullptr;
  const at::Tensor* k_given = tensor_or_none(a[6], "outs[0]");
  const at::Tensor* v_given = tensor_or_none(a[7], "outs[1]");
  at::Tensor k, v;
  const bool given = k_given || v_given;
  if (given) {
    if (!k_given || !v_given) throw Refused{"outs must hold k and v"};
    check_output(*k_given, type, rows, H, cache->head_dim, index, "outs[0]");
    check_output(*v_given, type, rows, H, cache->head_dim_v, index, "outs[1]");
    k = *k_given;
    v = *v_given;
  } else {
    k = new_rows(rows, H, cache->head_dim, type, index);
    v = new_rows(rows, H, cache->head_dim_v, type, index);
  }
  const Workspace ws = check_ws(tensor_or_none(a[8], "ws"), index);
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    // Rows that are skipped hold zeros in new memory, not what was there before.
    return (given ? g_cache_read : g_cache_read_zeroed)(cache, k.data_ptr(), v.data_ptr(), off, static_cast<int32_t>(B), rows, first, pages,
                        static_cast<int32_t>(table.size(1)), ws.ptr, ws.bytes, stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  return pair(k, v);
}

// fwd_paged(cache, cache_device, q_c, cache_lens, page_table, max_seqlen, alpha,
//           cand_offsets, func_c, ws, out)
PyObject* fwd_paged(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 11);
  const auto* cache = static_cast<const hstu_cache_t*>(address(a[0]));
  const int index = static_cast<int>(integer(a[1]));
  check_current(index, "cache");
  const at::ScalarType type = element(cache->dtype);
  const at::Tensor &q = tensor(a[2], "q_c"), &lens = tensor(a[3], "cache_lens"), &table = tensor(a[4], "page_table");
  const int64_t H = cache->num_heads;
  const int64_t qs = check_rows(q, type, H, cache->head_dim, index, "q_c");
  const int64_t C = q.size(0), B = lens.numel();
  const int32_t* len = check_ints(lens, {B}, index, "cache_lens");
  const int32_t* pages = check_pages(table, B, index);
  const int64_t max_seqlen = integer(a[5]);
  if (max_seqlen < INT32_MIN || max_seqlen > INT32_MAX) throw Refused{"max_seqlen is out of range"};
  const double alpha = PyFloat_AsDouble(a[6]);
  if (alpha == -1.0 && PyErr_Occurred()) throw python_error();
  const at::Tensor* offsets = tensor_or_none(a[7], "cand_offsets");
  const int32_t* cand = offsets ? check_ints(*offsets, {B + 1}, index, "cand_offsets") : nullptr;
  const at::Tensor* func = tensor_or_none(a[8], "func_c");
  const int64_t nfunc = func && func->dim() > 0 ? func->size(0) : 0;
  const int32_t* intervals = func ? check_ints(*func, {nfunc, C}, index, "func_c") : nullptr;
  const at::Tensor* given = tensor_or_none(a[10], "out");
  at::Tensor out;
  uint32_t flags = 0;
  if (given) {
    check_output(*given, type, C, H, cache->head_dim_v, index, "out");
    out = *given;
  } else {
    out = new_rows(C, H, cache->head_dim_v, type, index);
    flags |= HSTU_FLAG_ZERO_SKIPPED;  // not what the memory held before
  }
  Workspace ws = check_ws(tensor_or_none(a[9], "ws"), index);
  at::Tensor own;  // freed on return, for the allocator to reuse behind this call on its stream
  if (!ws.ptr) {
    flags |= HSTU_FLAG_NO_STATUS;  // nobody could read the error word
    const size_t bytes = g_paged_size(cache, static_cast<int32_t>(B), C, static_cast<int32_t>(max_seqlen));
    if (bytes > 256) {  // sums of splits; without them nothing but the error word
      own = at::empty({static_cast<int64_t>(bytes)},
                      at::TensorOptions().dtype(at::kByte).device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
      ws = {own.data_ptr(), bytes};
    }
  }
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    return g_fwd_paged(q.data_ptr(), qs, out.data_ptr(), cache, len, static_cast<int32_t>(B), pages,
                       static_cast<int32_t>(table.size(1)), cand, C, intervals, static_cast<int32_t>(nfunc),
                       static_cast<int32_t>(max_seqlen), static_cast<float>(alpha), ws.ptr, ws.bytes, flags, stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  PyObject* r = THPVariable_Wrap(out);
  if (!r) throw python_error();
  return r;
}

// bind(rope, cache_write, cache_read, paged_workspace_size, fwd_paged,
// cache_read_zeroed): addresses of the entry points.
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  if (n != 6) throw Refused{"six addresses"};
  g_rope = reinterpret_cast<decltype(g_rope)>(address(a[0]));
  g_cache_write = reinterpret_cast<decltype(g_cache_write)>(address(a[1]));
  g_cache_read = reinterpret_cast<decltype(g_cache_read)>(address(a[2]));
  g_paged_size = reinterpret_cast<decltype(g_paged_size)>(address(a[3]));
  g_fwd_paged = reinterpret_cast<decltype(g_fwd_paged)>(address(a[4]));
  g_cache_read_zeroed = reinterpret_cast<decltype(g_cache_read_zeroed)>(address(a[5]));
  Py_RETURN_NONE;
}

// No C++ exception reaches the interpreter: refusals become ValueError, the
// rest (out of memory among it) what torch makes of them.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<bind>("bind"),
    method<rope>("rope"),
    method<cache_write>("cache_write"),
    method<cache_read>("cache_read"),
    method<fwd_paged>("fwd_paged"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
