// The paged calls' part of the compiled marshalling (see fp8_calls.cpp, whose
// helpers it uses): rotary positions, and the paged cache's append, read and
// attention.  Each returns a tuple where it made the call, None where it did
// not take it.
#pragma once

decltype(&quarot_rope) g_rope = nullptr;
decltype(&quarot_paged_append) g_append = nullptr;
decltype(&quarot_paged_read) g_read = nullptr;
decltype(&quarot_paged_workspace_bytes) g_workspace = nullptr;
decltype(&quarot_paged_attn) g_attn = nullptr;

// A CUDA tensor (exactly a tensor or parameter) of this many dimensions on the device; or null.
const Tensor* tensor(PyObject* o, int dev, int64_t dims) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.get_device() == dev && t.dim() == dims && t.layout() == at::kStrided ? &t : nullptr;
}
const Tensor* dense(PyObject* o, int dev, int64_t dims, ScalarType type) {
  const Tensor* t = tensor(o, dev, dims);
  return t != nullptr && t->scalar_type() == type && t->is_contiguous() ? t : nullptr;
}

// [N, H, d] of 16-bit elements, heads one after the other.
struct HeadsArg {
  const Tensor* t = nullptr;
  int64_t N = 0, H = 0, d = 0, ld = 0;
  bool set(PyObject* o, int dev) {
    t = tensor(o, dev, 3);
    if (t == nullptr || dtype_of(*t) < 0) return false;
    N = t->size(0), H = t->size(1), d = t->size(2);
    if (H < 1 || d < 2 || t->stride(2) != 1 || (H > 1 && t->stride(1) != d)) return false;
    ld = N > 1 ? t->stride(0) : H * d;
    return ld >= H * d;
  }
};
// An output like `like`: the given tensor, or a new one.
bool heads_output(PyObject* given, const HeadsArg& like, int dev, Tensor& out, int64_t& ld) {
  if (given == Py_None) {
    out = at::detail::empty_cuda({like.N, like.H, like.d}, like.t->scalar_type(),
                                 at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
    ld = like.H * like.d;
    return true;
  }
  HeadsArg h;
  if (!h.set(given, dev) || h.N != like.N || h.H != like.H || h.d != like.d || h.t->scalar_type() != like.t->scalar_type())
    return false;
  out = *h.t;
  ld = h.ld;
  return true;
}
bool rotation(PyObject* inv_freq, PyObject* scale, int dev, const double*& f, int64_t& rot, float& s) {
  f = nullptr, rot = 0, s = 1.0f;
  if (inv_freq == Py_None) return true;
  const Tensor* t = dense(inv_freq, dev, 1, ScalarType::Double);
  if (t == nullptr || !PyFloat_CheckExact(scale)) return false;
  f = static_cast<const double*>(t->data_ptr()), rot = 2 * t->size(0), s = float(PyFloat_AS_DOUBLE(scale));
  return true;
}
struct CacheArg {
  uint8_t *k_q, *v_q;
  void *k_s, *v_s;
  int64_t pages, ps, H, d;
  bool set(PyObject* const* o, int dev) {
    const Tensor *kq = dense(o[0], dev, 4, ScalarType::Byte), *ks = dense(o[1], dev, 3, ScalarType::Half);
    const Tensor *vq = dense(o[2], dev, 4, ScalarType::Byte), *vs = dense(o[3], dev, 3, ScalarType::Half);
    if (kq == nullptr || ks == nullptr || vq == nullptr || vs == nullptr || kq->sizes() != vq->sizes() ||
        ks->sizes() != vs->sizes() || kq->sizes().slice(0, 3) != ks->sizes())
      return false;
    k_q = u8(*kq), v_q = u8(*vq), k_s = ks->data_ptr(), v_s = vs->data_ptr();
    pages = kq->size(0), H = kq->size(1), ps = kq->size(2), d = 2 * kq->size(3);
    return true;
  }
};
struct BatchArg {
  const int32_t *table, *lengths, *cu = nullptr;
  int64_t B, pages;
  bool set(PyObject* const* o, int dev) {
    const Tensor *t = dense(o[0], dev, 2, ScalarType::Int), *l = dense(o[1], dev, 1, ScalarType::Int);
    if (t == nullptr || l == nullptr || l->size(0) != t->size(0)) return false;
    B = t->size(0), pages = t->size(1);
    table = static_cast<const int32_t*>(t->data_ptr()), lengths = static_cast<const int32_t*>(l->data_ptr());
    if (o[2] == Py_None) return true;
    const Tensor* c = dense(o[2], dev, 1, ScalarType::Int);
    if (c == nullptr || c->size(0) != B + 1) return false;
    cu = static_cast<const int32_t*>(c->data_ptr());
    return true;
  }
};

// rope(q, k, positions, inv_freq, interleaved, scale, q_out, k_out) -> (q, k)
PyObject* rope(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8 || g_rope == nullptr) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  HeadsArg q, k;
  if (dev < 0 || !q.set(args[0], dev)) Py_RETURN_NONE;
  const bool has_k = args[1] != Py_None;
  if (has_k ? !k.set(args[1], dev) || k.N != q.N || k.d != q.d || k.t->scalar_type() != q.t->scalar_type() : args[7] != Py_None)
    Py_RETURN_NONE;
  const Tensor* pos = dense(args[2], dev, 1, ScalarType::Int);
  const double* f;
  int64_t rot, ld_q, ld_k = 0;
  float scale;
  Tensor qo, ko;
  if (pos == nullptr || pos->size(0) != q.N || !rotation(args[3], args[5], dev, f, rot, scale) ||
      !heads_output(args[6], q, dev, qo, ld_q) || (has_k && !heads_output(args[7], k, dev, ko, ld_k)))
    Py_RETURN_NONE;
  const int st = g_rope(q.t->data_ptr(), q.H, q.ld, qo.data_ptr(), ld_q, has_k ? k.t->data_ptr() : nullptr, k.H, k.ld,
                        has_k ? ko.data_ptr() : nullptr, ld_k, dtype_of(*q.t), q.N, q.d,
                        static_cast<const int32_t*>(pos->data_ptr()), f, rot, PyObject_IsTrue(args[4]), scale, stream(dev));
  if (st != QUAROT_OK) return refused(module, st, "quarot_rope");
  PyObject* none = Py_None;
  if (!has_k) Py_INCREF(none);
  return tuple_of({back(args[6], qo), has_k ? back(args[7], ko) : none});
  END_HANDLE_TH_ERRORS
}

// append(k, v, cache x 4, table, lengths, cu_q, q, inv_freq, interleaved, scale, q_out) -> (q or None,)
PyObject* append(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14 || g_append == nullptr) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  HeadsArg k, v, q;
  CacheArg c;
  BatchArg b;
  if (dev < 0 || !k.set(args[0], dev) || !v.set(args[1], dev) || !c.set(args + 2, dev) || !b.set(args + 6, dev)) Py_RETURN_NONE;
  if (k.H != c.H || k.d != c.d || v.N != k.N || v.H != c.H || v.d != c.d || v.t->scalar_type() != k.t->scalar_type()) Py_RETURN_NONE;
  const bool has_q = args[9] != Py_None;
  if (has_q ? !q.set(args[9], dev) || q.N != k.N || q.d != k.d || q.t->scalar_type() != k.t->scalar_type() : args[13] != Py_None)
    Py_RETURN_NONE;
  const double* f;
  int64_t rot, ld = 0;
  float scale;
  Tensor qo;
  if (!rotation(args[10], args[12], dev, f, rot, scale) || (has_q && !heads_output(args[13], q, dev, qo, ld))) Py_RETURN_NONE;
  const int st = g_append(k.t->data_ptr(), k.ld, v.t->data_ptr(), v.ld, has_q ? q.t->data_ptr() : nullptr, q.H, q.ld,
                          has_q ? qo.data_ptr() : nullptr, ld, dtype_of(*k.t), k.N, c.H, c.d, f, rot, PyObject_IsTrue(args[11]),
                          scale, c.k_q, c.k_s, c.v_q, c.v_s, c.pages, c.ps, b.table, b.B, b.pages, b.lengths, b.cu, stream(dev));
  if (st != QUAROT_OK) return refused(module, st, "quarot_paged_append");
  PyObject* none = Py_None;
  if (!has_q) Py_INCREF(none);
  return tuple_of({has_q ? back(args[13], qo) : none});
  END_HANDLE_TH_ERRORS
}

// read(cache x 4, table, lengths, cu_q, n, unrotate, dtype, k_out, v_out) -> (k, v)
PyObject* read(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12 || g_read == nullptr || !PyLong_CheckExact(args[9])) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  CacheArg c;
  BatchArg b;
  if (dev < 0 || !c.set(args, dev) || !b.set(args + 4, dev)) Py_RETURN_NONE;
  if (args[7] == Py_None ? b.cu != nullptr : !PyLong_CheckExact(args[7])) Py_RETURN_NONE;
  const int64_t N = args[7] == Py_None ? b.B : PyLong_AsLongLong(args[7]);
  const long dt = PyLong_AsLong(args[9]);
  if (PyErr_Occurred() != nullptr) return nullptr;
  if (N < 0 || N > (int64_t(1) << 24) || (dt != QUAROT_FP16 && dt != QUAROT_BF16)) Py_RETURN_NONE;
  const ScalarType type = dt == QUAROT_FP16 ? ScalarType::Half : ScalarType::BFloat16;
  Tensor out[2];
  for (int i = 0; i < 2; ++i) {
    if (args[10 + i] == Py_None) {
      out[i] = at::detail::empty_cuda({N, c.H, c.d}, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
    } else {
      const Tensor* t = dense(args[10 + i], dev, 3, type);
      if (t == nullptr || t->size(0) != N || t->size(1) != c.H || t->size(2) != c.d) Py_RETURN_NONE;
      out[i] = *t;
    }
  }
  const int st = g_read(c.k_q, c.k_s, c.v_q, c.v_s, c.pages, c.ps, c.H, c.d, b.table, b.B, b.pages, b.lengths, b.cu, N,
                        PyObject_IsTrue(args[8]), out[0].data_ptr(), out[1].data_ptr(), int(dt), stream(dev));
  if (st != QUAROT_OK) return refused(module, st, "quarot_paged_read");
  return tuple_of({back(args[10], out[0]), back(args[11], out[1])});
  END_HANDLE_TH_ERRORS
}

// attn(q, cache x 4, table, lengths, cu_q, max_q, shared_len, sm_scale, unrotate, out, workspace) -> (out,)
PyObject* attn(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14 || g_attn == nullptr || !PyLong_CheckExact(args[9]) || !PyFloat_CheckExact(args[10])) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  HeadsArg q;
  CacheArg c;
  BatchArg b;
  if (dev < 0 || !q.set(args[0], dev) || !c.set(args + 1, dev) || !b.set(args + 5, dev) || q.d != c.d) Py_RETURN_NONE;
  if (args[8] != Py_None && !PyLong_CheckExact(args[8])) Py_RETURN_NONE;
  const int64_t max_q = args[8] != Py_None ? PyLong_AsLongLong(args[8]) : b.cu == nullptr || q.N < 1 ? 1 : q.N;
  const int64_t shared = PyLong_AsLongLong(args[9]);
  if (PyErr_Occurred() != nullptr) return nullptr;
  const size_t bytes = g_workspace(q.N, b.B, q.H, c.H, c.d, max_q, shared);
  Tensor out, ws;
  int64_t ld;
  if (args[13] == Py_None) {
    ws = at::detail::empty_cuda({int64_t(bytes < 256 ? 256 : bytes)}, ScalarType::Byte,
                                at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
  } else {
    if (!THPVariable_CheckExact(args[13])) Py_RETURN_NONE;
    ws = THPVariable_Unpack(args[13]);
    if (!ws.defined() || !ws.is_cuda() || ws.get_device() != dev || ws.layout() != at::kStrided || !ws.is_contiguous()) Py_RETURN_NONE;
  }
  if (!heads_output(args[12], q, dev, out, ld)) Py_RETURN_NONE;
  const int st = g_attn(q.t->data_ptr(), q.ld, dtype_of(*q.t), q.N, q.H, c.H, c.d, c.k_q, c.k_s, c.v_q, c.v_s, c.pages, c.ps, b.table,
                        b.B, b.pages, b.lengths, b.cu, max_q, shared, float(PyFloat_AS_DOUBLE(args[10])), PyObject_IsTrue(args[11]),
                        out.data_ptr(), ld, ws.data_ptr(), ws.nbytes(), stream(dev));
  if (st != QUAROT_OK) return refused(module, st, "quarot_paged_attn");
  return tuple_of({back(args[12], out)});
  END_HANDLE_TH_ERRORS
}

// bind_paged(rope, append, read, workspace_bytes, attn): the entry points' addresses
PyObject* bind_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[5];
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind_paged takes five addresses");
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred() != nullptr) return nullptr;
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_read = reinterpret_cast<decltype(g_read)>(p[2]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[3]);
  g_attn = reinterpret_cast<decltype(g_attn)>(p[4]);
  Py_RETURN_NONE;
}
