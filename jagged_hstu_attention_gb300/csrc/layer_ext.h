// The layer's row operators as Python calls; a part of serving_ext.cpp, inside its
// unnamed namespace.

namespace layer {

// Entry points of the loaded library, set by bind_layer().
decltype(&hstu_attn_embed) g_embed = nullptr;
decltype(&hstu_attn_embed_workspace_size) g_embed_size = nullptr;
decltype(&hstu_attn_embed_bwd) g_embed_bwd = nullptr;
decltype(&hstu_attn_rms_norm) g_norm = nullptr;
decltype(&hstu_attn_quantise_rows) g_quantise = nullptr;
decltype(&hstu_attn_rms_norm_workspace_size) g_norm_size = nullptr;
decltype(&hstu_attn_rms_norm_bwd) g_norm_bwd = nullptr;
decltype(&hstu_attn_linear) g_linear = nullptr;
decltype(&hstu_attn_linear_workspace_size) g_linear_size = nullptr;
decltype(&hstu_attn_linear_bwd) g_linear_bwd = nullptr;

void need(Py_ssize_t got, Py_ssize_t want) {
  if (got != want || !g_embed) throw Refused{"called by the wrappers of binding.py only"};
}

at::ScalarType wide(int dtype) { return dtype == HSTU_DTYPE_F32 ? at::kFloat : element(dtype); }
int code(at::ScalarType t, const char* name) {
  if (t == at::kBFloat16) return HSTU_DTYPE_BF16;
  if (t == at::kHalf) return HSTU_DTYPE_F16;
  throw Refused{std::string(name) + " must be one of (torch.bfloat16, torch.float16), got " + c10::toString(t)};
}

// New memory of the current stream on the current device, which check_current() has
// compared with the tensors': what at::empty() does, without its dispatch (1.3 us a
// tensor on this GPU's host; a norm has up to four outputs).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, int) {
  return at::Tensor(at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(),
                                              c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
}

// Codes (T, D) and their rows' scales (T) in one piece of memory: the two live and die
// together, and a piece less to ask for is half a microsecond.
std::pair<at::Tensor, at::Tensor> fresh_codes(int64_t T, int64_t D, int index) {
  const int64_t body = (T * D + 255) / 256 * 256;
  const at::Tensor codes = fresh({body + T}, at::kByte, index);
  auto scale = c10::make_intrusive<c10::TensorImpl>(c10::Storage(codes.storage()), codes.key_set(), codes.dtype());
  scale->set_storage_offset(body);
  scale->set_sizes_contiguous({T});
  codes.unsafeGetTensorImpl()->set_sizes_contiguous({T, D});
  return {codes, at::Tensor(std::move(scale))};
}

// A (rows, width) matrix whose rows may lie apart; returns the distance between
// rows in elements. `rows` < 0: any number.
int64_t check_matrix(const at::Tensor& t, at::ScalarType type, int64_t rows, int64_t width, int index,
                     const char* name) {
  check_device(t, index, name);
  check_dtype(t, type, name);
  if (t.dim() != 2 || t.size(1) != width || (rows >= 0 && t.size(0) != rows))
    throw Refused{std::string(name) + " must be (" + (rows >= 0 ? std::to_string(rows) : "rows") + ", " +
                  std::to_string(width) + "), got " + shape_text(t.sizes())};
  if (width > 1 && t.stride(1) != 1) throw Refused{std::string(name) + ": the columns of a row must be contiguous"};
  if (t.size(0) <= 1) return width;
  if (t.stride(0) < width) throw Refused{std::string(name) + ": rows overlap"};
  return t.stride(0);
}
void check_whole(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, int index,
                 const char* name) {
  check_device(t, index, name);
  check_dtype(t, type, name);
  if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
    throw Refused{std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes())};
  if (!t.is_contiguous()) throw Refused{std::string(name) + " must be contiguous"};
}
int index_of(const at::Tensor& t, const char* name) {
  const int index = t.is_cuda() ? t.get_device() : -1;
  check_current(index, name);
  return index;
}
void check_2d(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) throw Refused{std::string(name) + " must be (rows, width), got " + shape_text(t.sizes())};
}
int32_t width32(int64_t v, const char* name) {
  if (v > INT32_MAX) throw Refused{std::string(name) + " is too wide"};
  return static_cast<int32_t>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
void* data(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* data(const std::optional<at::Tensor>& t) { return t ? t->data_ptr() : nullptr; }

PyObject* wrap(const std::optional<at::Tensor>& t) { return t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None); }
template <size_t N>
PyObject* tuple(const std::optional<at::Tensor> (&ts)[N]) {
  PyObject* r = PyTuple_New(N);
  if (!r) throw python_error();
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = wrap(ts[i]);
    if (!o) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// The caller's workspace, or one of the size needed, freed on return for the
// allocator to reuse behind this call on its stream.
Workspace workspace(PyObject* given, size_t bytes, int index, at::Tensor& own) {
  Workspace ws = check_ws(tensor_or_none(given, "ws"), index);
  if (!ws.ptr && bytes > 0) {
    own = fresh({static_cast<int64_t>(bytes)}, at::kByte, index);
    ws = {own.data_ptr(), bytes};
  }
  return ws;
}

int id_bytes(const at::Tensor& ids, int index) {
  check_device(ids, index, "ids");
  const bool wide_ids = ids.scalar_type() == at::kLong;
  if (!wide_ids) check_dtype(ids, at::kInt, "ids");
  if (ids.dim() != 1) throw Refused{"ids must be (tokens,), got " + shape_text(ids.sizes())};
  if (!ids.is_contiguous()) throw Refused{"ids must be contiguous"};
  return wide_ids ? 8 : 4;
}

// embed(table, ids, scale, dtype, out, ws)
PyObject* embed(PyObject* const* a, Py_ssize_t n) {
  need(n, 6);
  const at::Tensor &table = tensor(a[0], "table"), &ids = tensor(a[1], "ids");
  const int index = index_of(table, "table");
  check_2d(table, "table");
  const int64_t V = table.size(0), D = table.size(1), T = ids.numel();
  const bool f32 = table.scalar_type() == at::kFloat;
  const int dtype = static_cast<int>(integer(a[3]));
  if (!f32) {
    code(table.scalar_type(), "table");
    check_dtype(table, element(dtype), "table");
  }
  check_whole(table, table.scalar_type(), {V, D}, index, "table");
  const int bytes = id_bytes(ids, index);
  const float scale = static_cast<float>(number(a[2]));
  const at::Tensor* given = tensor_or_none(a[4], "out");
  if (given) check_whole(*given, element(dtype), {T, D}, index, "out");
  const at::Tensor out = given ? *given : fresh({T, D}, element(dtype), index);
  const Workspace ws = check_ws(tensor_or_none(a[5], "ws"), index);
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    return g_embed(table.data_ptr(), f32 ? HSTU_DTYPE_F32 : dtype, V, width32(D, "table"), ids.data_ptr(), bytes, T,
                   scale, out.data_ptr(), dtype, ws.ptr, ws.bytes, stream);
  });
  return st != HSTU_OK ? PyLong_FromLong(st) : wrap(out);
}

// embed_bwd(dy, ids, vocab, scale, grad dtype, out, accumulate, ws)
PyObject* embed_bwd(PyObject* const* a, Py_ssize_t n) {
  need(n, 8);
  const at::Tensor &dy = tensor(a[0], "dy"), &ids = tensor(a[1], "ids");
  const int index = index_of(dy, "dy");
  check_2d(dy, "dy");
  const int dtype = code(dy.scalar_type(), "dy"), bytes = id_bytes(ids, index);
  const int64_t T = ids.numel(), D = dy.size(1), V = integer(a[2]);
  const int64_t stride = check_matrix(dy, dy.scalar_type(), T, D, index, "dy");
  const int grad = static_cast<int>(integer(a[4]));
  const float scale = static_cast<float>(number(a[3]));
  const at::Tensor* given = tensor_or_none(a[5], "out");
  const bool accumulate = a[6] == Py_True;
  if (accumulate && !given) throw Refused{"accumulate adds to an out that is given"};
  if (V < 1 || D < 1) throw Refused{"the table must have rows and columns"};
  if (given) check_whole(*given, wide(grad), {V, D}, index, "out");
  const size_t size = g_embed_size(T, V, width32(D, "dy"));
  if (size == 0) return PyLong_FromLong(HSTU_ERR_UNSUPPORTED);
  const at::Tensor out = given ? *given : fresh({V, D}, wide(grad), index);
  at::Tensor own;
  const Workspace ws = workspace(a[7], size, index, own);
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    return g_embed_bwd(dy.data_ptr(), stride, dtype, ids.data_ptr(), bytes, T, scale, out.data_ptr(), grad, V,
                       static_cast<int32_t>(D), accumulate, ws.ptr, ws.bytes, stream);
  });
  return st != HSTU_OK ? PyLong_FromLong(st) : wrap(out);
}

// rms_norm(x, weight, residual, gate, eps, quantise, want_rstd, y, y_scale, h)
PyObject* rms_norm(PyObject* const* a, Py_ssize_t n) {
  need(n, 10);
  const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
  const int index = index_of(x, "x");
  check_2d(x, "x");
  const at::ScalarType type = x.scalar_type();
  const int dtype = code(type, "x");
  const int64_t T = x.size(0), D = x.size(1), xs = check_matrix(x, type, T, D, index, "x");
  check_whole(weight, type, {D}, index, "weight");
  const at::Tensor *residual = tensor_or_none(a[2], "residual"), *gate = tensor_or_none(a[3], "gate");
  const int64_t rs = residual ? check_matrix(*residual, type, T, D, index, "residual") : 0;
  const int64_t gs = gate ? check_matrix(*gate, type, T, D, index, "gate") : 0;
  const float eps = static_cast<float>(number(a[4]));
  const bool codes = a[5] == Py_True;
  const at::Tensor *y_given = tensor_or_none(a[7], "outs[0]"), *s_given = tensor_or_none(a[8], "outs[0]'s scales"),
                   *h_given = tensor_or_none(a[9], "outs[1]");
  const at::ScalarType y_type = codes ? at::kByte : type;
  if (y_given) check_whole(*y_given, y_type, {T, D}, index, "outs[0]");
  if (s_given) check_whole(*s_given, at::kByte, {T}, index, "outs[0]'s scales");
  if (y_given && codes != (s_given != nullptr)) throw Refused{"outs[0] must be of the output's kind"};
  if (h_given) {
    if (!residual) throw Refused{"outs[1] is written where there is a residual"};
    check_whole(*h_given, type, {T, D}, index, "outs[1]");
  }
  at::Tensor y;
  std::optional<at::Tensor> scale, h, rstd;
  if (codes && !y_given) {
    std::tie(y, scale) = fresh_codes(T, D, index);
  } else {
    y = y_given ? *y_given : fresh({T, D}, type, index);
    if (codes) scale = *s_given;
  }
  if (residual) h = h_given ? *h_given : fresh({T, D}, type, index);
  if (a[6] == Py_True) rstd = fresh({T}, at::kFloat, index);
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    return g_norm(x.data_ptr(), xs, data(residual), rs, data(gate), gs, weight.data_ptr(), T, width32(D, "x"), dtype,
                  eps, y.data_ptr(), static_cast<uint8_t*>(data(scale)), data(h), static_cast<float*>(data(rstd)),
                  stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  return tuple<4>({y, scale, h, rstd});
}

// quantise_rows(x)
PyObject* quantise_rows(PyObject* const* a, Py_ssize_t n) {
  need(n, 1);
  const at::Tensor& x = tensor(a[0], "x");
  const int index = index_of(x, "x");
  check_2d(x, "x");
  const int dtype = code(x.scalar_type(), "x");
  const int64_t T = x.size(0), D = x.size(1), xs = check_matrix(x, x.scalar_type(), T, D, index, "x");
  const auto [codes, scale] = fresh_codes(T, D, index);
  void *stream = current_stream(index), *to = codes.data_ptr(), *to_scale = scale.data_ptr();
  const hstu_status_t st = without_lock([&] {
    return g_quantise(x.data_ptr(), xs, T, width32(D, "x"), dtype, static_cast<uint8_t*>(to),
                      static_cast<uint8_t*>(to_scale), stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  return tuple<2>({codes, scale});
}

// rms_norm_bwd(dy, h, rstd, weight, gate, dh, ws)
PyObject* rms_norm_bwd(PyObject* const* a, Py_ssize_t n) {
  need(n, 7);
  const at::Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h"), &rstd = tensor(a[2], "rstd"),
                   &weight = tensor(a[3], "weight");
  const int index = index_of(dy, "dy");
  check_2d(dy, "dy");
  const at::ScalarType type = dy.scalar_type();
  const int dtype = code(type, "dy");
  const int64_t T = dy.size(0), D = dy.size(1), ds = check_matrix(dy, type, T, D, index, "dy");
  const int64_t hs = check_matrix(h, type, T, D, index, "h");
  check_whole(rstd, at::kFloat, {T}, index, "rstd");
  check_whole(weight, type, {D}, index, "weight");
  const at::Tensor *gate = tensor_or_none(a[4], "gate"), *dh = tensor_or_none(a[5], "dh");
  const int64_t gs = gate ? check_matrix(*gate, type, T, D, index, "gate") : 0;
  const int64_t es = dh ? check_matrix(*dh, type, T, D, index, "dh") : 0;
  const size_t size = g_norm_size(T, width32(D, "dy"));
  if (size == 0) return PyLong_FromLong(D < 1 ? HSTU_ERR_INVALID_ARG : HSTU_ERR_UNSUPPORTED);
  const at::Tensor dx = fresh({T, D}, type, index), dw = fresh({D}, type, index);
  std::optional<at::Tensor> dgate;
  if (gate) dgate = fresh({T, D}, type, index);
  at::Tensor own;
  const Workspace ws = workspace(a[6], size, index, own);
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    return g_norm_bwd(dy.data_ptr(), ds, h.data_ptr(), hs, static_cast<const float*>(rstd.data_ptr()),
                      weight.data_ptr(), data(gate), gs, data(dh), es, T, static_cast<int32_t>(D), dtype,
                      dx.data_ptr(), dw.data_ptr(), data(dgate), ws.ptr, ws.bytes, stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  return tuple<3>({dx, dw, dgate});
}

// linear(x, x_scale, w, w_scale, bias, act, residual, dtype, want_z, out, ws)
PyObject* linear(PyObject* const* a, Py_ssize_t n) {
  need(n, 11);
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[2], "w");
  const at::Tensor *xsc = tensor_or_none(a[1], "x's scales"), *wsc = tensor_or_none(a[3], "w's scales");
  if ((xsc != nullptr) != (wsc != nullptr)) throw Refused{"x and w must both be quantised rows, or neither"};
  const int index = index_of(x, "x");
  check_2d(x, "x");
  check_2d(w, "w");
  const bool codes = xsc != nullptr;
  const int dtype = static_cast<int>(integer(a[7]));
  const at::ScalarType type = element(dtype), in_type = codes ? at::kByte : type;
  const int64_t T = x.size(0), K = x.size(1), N = w.size(0), xs = check_matrix(x, in_type, T, K, index, "x");
  check_whole(w, in_type, {N, K}, index, "w");
  if (codes) {
    check_whole(*xsc, at::kByte, {T}, index, "x's scales");
    check_whole(*wsc, at::kByte, {N}, index, "w's scales");
  }
  const at::Tensor *bias = tensor_or_none(a[4], "bias"), *residual = tensor_or_none(a[6], "residual");
  if (bias) check_whole(*bias, type, {N}, index, "bias");
  const int64_t rs = residual ? check_matrix(*residual, type, T, N, index, "residual") : 0;
  const at::Tensor* given = tensor_or_none(a[9], "out");
  if (given) check_whole(*given, type, {T, N}, index, "out");
  const at::Tensor y = given ? *given : fresh({T, N}, type, index);
  std::optional<at::Tensor> z;
  if (a[8] == Py_True) z = fresh({T, N}, type, index);
  const Workspace ws = check_ws(tensor_or_none(a[10], "ws"), index);
  void* stream = current_stream(index);
  const int act = static_cast<int>(integer(a[5]));
  const hstu_status_t st = without_lock([&] {
    return g_linear(x.data_ptr(), xs, static_cast<const uint8_t*>(data(xsc)), w.data_ptr(),
                    static_cast<const uint8_t*>(data(wsc)), data(bias), data(residual), rs, T, width32(K, "x"),
                    width32(N, "w"), dtype, act, y.data_ptr(), data(z), ws.ptr, ws.bytes, stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  return pair(y, z);
}

// linear_bwd(dy, z, x, w, act, want_dbias, ws)
PyObject* linear_bwd(PyObject* const* a, Py_ssize_t n) {
  need(n, 7);
  const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[2], "x"), &w = tensor(a[3], "w");
  const at::Tensor* z = tensor_or_none(a[1], "z");
  const int index = index_of(dy, "dy");
  check_2d(dy, "dy");
  check_2d(w, "w");
  const at::ScalarType type = dy.scalar_type();
  const int dtype = code(type, "dy"), act = static_cast<int>(integer(a[4]));
  const int64_t T = dy.size(0), N = w.size(0), K = w.size(1), ds = check_matrix(dy, type, T, N, index, "dy");
  const int64_t xs = check_matrix(x, type, T, K, index, "x");
  check_whole(w, type, {N, K}, index, "w");
  if (act != HSTU_ACT_NONE) {
    if (!z) throw Refused{"z is needed where there is an activation"};
    check_whole(*z, type, {T, N}, index, "z");
  }
  const size_t size = g_linear_size(T, width32(K, "x"), width32(N, "w"), act);
  if (size == 0) return PyLong_FromLong(K < 1 || N < 1 ? HSTU_ERR_INVALID_ARG : HSTU_ERR_UNSUPPORTED);
  const at::Tensor dx = fresh({T, K}, type, index), dw = fresh({N, K}, type, index);
  std::optional<at::Tensor> db;
  if (a[5] == Py_True) db = fresh({N}, type, index);
  at::Tensor own;
  const Workspace ws = workspace(a[6], size, index, own);
  void* stream = current_stream(index);
  const hstu_status_t st = without_lock([&] {
    return g_linear_bwd(dy.data_ptr(), ds, act != HSTU_ACT_NONE ? data(z) : nullptr, x.data_ptr(), xs, w.data_ptr(), T,
                        static_cast<int32_t>(K), static_cast<int32_t>(N), dtype, act, dx.data_ptr(), dw.data_ptr(),
                        data(db), ws.ptr, ws.bytes, stream);
  });
  if (st != HSTU_OK) return PyLong_FromLong(st);
  return tuple<3>({dx, dw, db});
}

// bind_layer(addresses of the entry points, in the order of their declarations above)
PyObject* bind_layer(PyObject* const* a, Py_ssize_t n) {
  if (n != 10) throw Refused{"ten addresses"};
  g_embed = reinterpret_cast<decltype(g_embed)>(address(a[0]));
  g_embed_size = reinterpret_cast<decltype(g_embed_size)>(address(a[1]));
  g_embed_bwd = reinterpret_cast<decltype(g_embed_bwd)>(address(a[2]));
  g_norm = reinterpret_cast<decltype(g_norm)>(address(a[3]));
  g_quantise = reinterpret_cast<decltype(g_quantise)>(address(a[4]));
  g_norm_size = reinterpret_cast<decltype(g_norm_size)>(address(a[5]));
  g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(address(a[6]));
  g_linear = reinterpret_cast<decltype(g_linear)>(address(a[7]));
  g_linear_size = reinterpret_cast<decltype(g_linear_size)>(address(a[8]));
  g_linear_bwd = reinterpret_cast<decltype(g_linear_bwd)>(address(a[9]));
  Py_RETURN_NONE;
}

}  // namespace layer
