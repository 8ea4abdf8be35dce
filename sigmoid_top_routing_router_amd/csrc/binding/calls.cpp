// The Python binding's short way to the small calls, a CPython extension beside
// the ctypes binding: on ordinary arguments (contiguous tensors of the expected
// types and shapes on the current device, its current stream) a function here
// allocates the outputs and calls the C ABI; on anything else, an error included,
// it returns None, and the Python code runs with its checks and messages.  Every
// condition here is one that the Python code checks as well.
//
// A call through ctypes takes 7 to 9 us on the host, 3 of them the launch: 4 are
// attributes of tensors, the arguments' conversion and the interpreter.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../../include/moe_mi355x.h"

namespace {

// The library's entry points, as the ctypes binding has loaded them.
struct Abi {
  decltype(&moe_group_workspace_bytes) group_workspace_bytes;
  decltype(&moe_group) group;
  decltype(&moe_permute) permute;
  decltype(&moe_permute_backward) permute_backward;
  decltype(&moe_unpermute) unpermute;
  decltype(&moe_unpermute_backward) unpermute_backward;
  decltype(&moe_int8_quantize_rows) int8_quantize_rows;
  decltype(&moe_int8_matmul) int8_matmul;
} abi;
bool bound = false;

struct NotOrdinary {};
void need(bool ok) {
  if (!ok) throw NotOrdinary{};
}

using Sizes = at::IntArrayRef;

int32_t narrow(int64_t v) {
  need(v >= 0 && v <= INT32_MAX);
  return (int32_t)v;
}

// A tensor argument; absent: None, where that is allowed.
struct Arg {
  const at::Tensor* t = nullptr;
  Arg(PyObject* o, bool optional = false) {
    if (optional && o == Py_None) return;
    need(THPVariable_CheckExact(o));
    t = &THPVariable_Unpack(o);
    need(t->is_cuda() && t->layout() == at::kStrided && t->is_contiguous());
  }
  explicit operator bool() const { return t != nullptr; }
  const at::Tensor* operator->() const { return t; }
  template <class T = void>
  T* data() const {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
  }
  at::ScalarType type() const { return t->scalar_type(); }
  // of this type and shape, on this device, if it is there
  void is(at::ScalarType s, Sizes sizes, const Arg& first) const {
    if (!t) return;
    need(t->scalar_type() == s && t->sizes() == sizes && t->device() == first->device());
  }
};

bool bf16_bits(at::ScalarType s) {
  return s == at::kBFloat16 || s == at::kUInt16 || s == at::kShort;
}
bool row_type(at::ScalarType s) { return bf16_bits(s) || s == at::kFloat; }
uint32_t rows_flag(const Arg& a) { return a.type() == at::kFloat ? MOE_ROWS_F32 : 0u; }

// The current stream of the first tensor's device, which has to be the current one.
void* stream_of(const Arg& first) {
  const auto device = first->device().index();
  need(bound && device == c10::hip::current_device());
  return c10::hip::getCurrentHIPStream(device).stream();
}

at::Tensor empty(const Arg& like, at::ScalarType type, Sizes sizes) {
  return at::empty(sizes, like->options().dtype(type));
}

// The C call, without the interpreter's lock.
template <class F>
void call(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const moe_status_t status = f();
  PyEval_RestoreThread(s);
  need(status == MOE_OK);
}

PyObject* wrap(const at::Tensor& t) {
  PyObject* r = THPVariable_Wrap(t);
  need(r != nullptr);
  return r;
}
PyObject* wrap_or_none(const at::Tensor& t) {
  if (t.defined()) return wrap(t);
  Py_RETURN_NONE;
}
template <class... P>
PyObject* tuple(P... p) {
  PyObject* r = PyTuple_New(sizeof...(P));
  need(r != nullptr);
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, p), ...);
  return r;
}

// Runs a call with n arguments; None where it is not an ordinary one.
template <class F>
PyObject* ordinary(Py_ssize_t have, Py_ssize_t n, F&& f) {
  if (have == n) {
    try {
      return f();
    } catch (...) {  // not ordinary, out of memory, ...: the Python code says what
      PyErr_Clear();
    }
  }
  Py_RETURN_NONE;
}

// The scales of n rows of d codes.  Below 128 columns they would be empty, and the C
// entry tells codes from rows of 16 bits by the scales' address.
void are_scales(const Arg& s, int64_t n, int64_t d, const Arg& first) {
  if (!s) return;
  need(d % 128 == 0);
  s.is(at::kFloat, {n, d / 128}, first);
}

struct Places {
  Arg pos;
  int64_t N, K;
  Places(PyObject* o) : pos(o) {
    need(pos.type() == at::kInt && pos->dim() == 2 && pos->size(1) <= MOE_MAX_K);
    N = pos->size(0);
    K = pos->size(1);
  }
};

// n int32 elements of buf from `from` on, as a tensor of its own.
at::Tensor part(const at::Tensor& buf, int64_t from, Sizes sizes) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(buf.storage()), buf.key_set(), buf.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(from);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}

// group(topk_ids, E) -> counts, offsets, sorted_src, src_pos
PyObject* group(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 2, [&] {
    const Arg ids(a[0]);
    need(ids.type() == at::kInt && ids->dim() == 2 && PyLong_CheckExact(a[1]));
    const int64_t E = PyLong_AsLong(a[1]), N = ids->size(0), K = ids->size(1), P = N * K;
    void* stream = stream_of(ids);
    need(E > 0 && E <= MOE_MAX_E && K > 0 && K <= MOE_MAX_K);
    const int64_t bytes = (int64_t)abi.group_workspace_bytes(N, (int32_t)E, (int32_t)K);
    need(bytes > 0);
    const int64_t w = (bytes + 255) / 256 * 64;
    const at::Tensor buf = empty(ids, at::kInt, {w + 2 * E + 1 + 2 * P});
    int32_t* p = static_cast<int32_t*>(buf.data_ptr());
    call([&] {
      return abi.group(ids.data<int32_t>(), N, (int32_t)E, (int32_t)K, p + w, p + w + E,
                       p + w + 2 * E + 1, p + w + 2 * E + 1 + P, p, (size_t)w * 4, stream);
    });
    return tuple(wrap(part(buf, w, {E})), wrap(part(buf, w + E, {E + 1})),
                 wrap(part(buf, w + 2 * E + 1, {P})), wrap(part(buf, w + 2 * E + 1 + P, {N, K})));
  });
}

// permute(x, x_scales or None, src_pos, out or None) -> rows
PyObject* permute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 4, [&] {
    const Arg x(a[0]), xs(a[1], true), out(a[3], true);
    const Places at(a[2]);
    need(x->dim() == 2 && x->size(0) == at.N);
    const int64_t d = x->size(1);
    at.pos.is(at::kInt, at.pos->sizes(), x);
    at::ScalarType type = x.type();
    if (xs) {
      need(type == at::kByte);
      are_scales(xs, at.N, d, x);
      type = out ? out.type() : at::kBFloat16;
      need(bf16_bits(type));
    } else {
      need(row_type(type));
    }
    out.is(type, {at.N * at.K, d}, x);
    void* stream = stream_of(x);
    const at::Tensor rows = out ? *out.t : empty(x, type, {at.N * at.K, d});
    call([&] {
      return abi.permute(x.data(), xs.data<float>(), at.pos.data<int32_t>(), at.N, narrow(d),
                         (int32_t)at.K, xs ? 0u : rows_flag(x), rows.data_ptr(), stream);
    });
    return wrap(rows);
  });
}

// permute_backward(grad_rows, src_pos) -> grad_x
PyObject* permute_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 2, [&] {
    const Arg g(a[0]);
    const Places at(a[1]);
    need(row_type(g.type()) && g->dim() == 2 && g->size(0) == at.N * at.K);
    at.pos.is(at::kInt, at.pos->sizes(), g);
    const int64_t d = g->size(1);
    void* stream = stream_of(g);
    const at::Tensor x = empty(g, g.type(), {at.N, d});
    call([&] {
      return abi.permute_backward(g.data(), at.pos.data<int32_t>(), at.N, narrow(d),
                                  (int32_t)at.K, rows_flag(g), x.data_ptr(), stream);
    });
    return wrap(x);
  });
}

// unpermute(rows, src_pos, weights or None, base or None, checkpoint)
//   -> y, codes or None, scales or None
PyObject* unpermute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 5, [&] {
    const Arg rows(a[0]), w(a[2], true), base(a[3], true);
    const Places at(a[1]);
    need(row_type(rows.type()) && rows->dim() == 2 && rows->size(0) == at.N * at.K);
    need(a[4] == Py_True || a[4] == Py_False);
    at.pos.is(at::kInt, at.pos->sizes(), rows);
    const int64_t d = rows->size(1);
    w.is(at::kFloat, {at.N, at.K}, rows);
    base.is(rows.type(), {at.N, d}, rows);
    void* stream = stream_of(rows);
    const at::Tensor y = empty(rows, rows.type(), {at.N, d});
    at::Tensor codes, scales;
    if (a[4] == Py_True) {
      codes = empty(rows, at::kByte, {at.N * at.K, d});
      scales = empty(rows, at::kFloat, {at.N * at.K, d / 128});
    }
    call([&] {
      return abi.unpermute(rows.data(), at.pos.data<int32_t>(), w.data<float>(), base.data(), at.N,
                           narrow(d), (int32_t)at.K, rows_flag(rows), y.data_ptr(),
                           codes.defined() ? static_cast<uint8_t*>(codes.data_ptr()) : nullptr,
                           scales.defined() ? static_cast<float*>(scales.data_ptr()) : nullptr,
                           stream);
    });
    return tuple(wrap(y), wrap_or_none(codes), wrap_or_none(scales));
  });
}

// unpermute_backward(grad_y, src_pos, weights or None, rows or None, row_scales or
// None, out or None) -> grad_rows, grad_weights or None
PyObject* unpermute_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 6, [&] {
    const Arg g(a[0]), w(a[2], true), rows(a[3], true), rs(a[4], true), out(a[5], true);
    const Places at(a[1]);
    need(row_type(g.type()) && g->dim() == 2 && g->size(0) == at.N && (rows || !rs));
    at.pos.is(at::kInt, at.pos->sizes(), g);
    const int64_t d = g->size(1), P = at.N * at.K;
    w.is(at::kFloat, {at.N, at.K}, g);
    rows.is(rs ? at::kByte : g.type(), {P, d}, g);
    are_scales(rs, P, d, g);
    out.is(g.type(), {P, d}, g);
    void* stream = stream_of(g);
    const at::Tensor dr = out ? *out.t : empty(g, g.type(), {P, d});
    at::Tensor dw;
    if (rows) dw = empty(g, at::kFloat, {at.N, at.K});
    call([&] {
      return abi.unpermute_backward(g.data(), rows.data(), rs.data<float>(), at.pos.data<int32_t>(),
                                    w.data<float>(), at.N, narrow(d), (int32_t)at.K, rows_flag(g),
                                    dr.data_ptr(),
                                    dw.defined() ? static_cast<float*>(dw.data_ptr()) : nullptr,
                                    stream);
    });
    return tuple(wrap(dr), wrap_or_none(dw));
  });
}

// int8_quantize_rows(x) -> codes, scales
PyObject* int8_quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 1, [&] {
    const Arg x(a[0]);
    need(bf16_bits(x.type()) && x->dim() >= 2);
    const Sizes s = x->sizes(), per_row = s.slice(0, s.size() - 1);
    int64_t rows = 1;
    for (const int64_t i : per_row) rows *= i;
    void* stream = stream_of(x);
    const at::Tensor codes = empty(x, at::kChar, s), scales = empty(x, at::kFloat, per_row);
    call([&] {
      return abi.int8_quantize_rows(x.data<uint16_t>(), rows, narrow(s.back()),
                                    static_cast<int8_t*>(codes.data_ptr()),
                                    static_cast<float*>(scales.data_ptr()), stream);
    });
    return tuple(wrap(codes), wrap(scales));
  });
}

// int8_matmul(x codes, x scales, w codes, w scales, w_up codes or None, w_up scales
// or None, offsets or None, sorted_src or None (no gather), src_pos or None, out or
// None) -> out.  offsets and src_pos: of the grouping, both or neither.
PyObject* int8_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary(n, 10, [&] {
    const Arg x(a[0]), xs(a[1]), w(a[2]), ws(a[3]), u(a[4], true), us(a[5], true);
    const Arg offsets(a[6], true), src(a[7], true), out(a[9], true);
    need(x.type() == at::kChar && x->dim() == 2 && (u || !us) && (us || !u));
    const int64_t m = x->size(0), k = x->size(1);
    xs.is(at::kFloat, {m}, x);
    const bool grouped = (bool)offsets;
    need(w->dim() == (grouped ? 3 : 2) && w->size(-1) == k && grouped == (a[8] != Py_None) &&
         (grouped || !src));
    const Sizes shape = w->sizes(), channels = shape.slice(0, shape.size() - 1);
    w.is(at::kChar, shape, x);
    ws.is(at::kFloat, channels, x);
    u.is(at::kChar, shape, x);
    us.is(at::kFloat, channels, x);
    const int64_t E = grouped ? w->size(0) : 1, cols = w->size(-2);
    int64_t rows = m, K = 1;
    if (grouped) {
      const Places at(a[8]);
      K = at.K;
      rows = at.N * at.K;
      offsets.is(at::kInt, {E + 1}, x);
      src.is(at::kInt, {rows}, x);
      need(m == (src ? at.N : rows));
    }
    if (out) need(bf16_bits(out.type()));
    out.is(out ? out.type() : at::kBFloat16, {rows, cols}, x);
    void* stream = stream_of(x);
    const at::Tensor y = out ? *out.t : empty(x, at::kBFloat16, {rows, cols});
    moe_int8_matmul_t p{};
    p.a_rows = m;
    p.rows = rows;
    p.k = narrow(k);
    p.cols = narrow(cols);
    p.E = narrow(E);
    p.K = narrow(K);
    p.a = x.data<int8_t>();
    p.a_scales = xs.data<float>();
    p.w = w.data<int8_t>();
    p.w_scales = ws.data<float>();
    p.w_up = u.data<int8_t>();
    p.w_up_scales = us.data<float>();
    p.offsets = offsets.data<int32_t>();
    p.sorted_src = src.data<int32_t>();
    call([&] { return abi.int8_matmul(&p, static_cast<uint16_t*>(y.data_ptr()), stream); });
    return wrap(y);
  });
}

// bind(address of each entry of Abi, in its order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[8];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  }
  static_assert(sizeof(Abi) == sizeof(p), "eight entries");
  abi = Abi{(decltype(abi.group_workspace_bytes))p[0], (decltype(abi.group))p[1],
            (decltype(abi.permute))p[2], (decltype(abi.permute_backward))p[3],
            (decltype(abi.unpermute))p[4], (decltype(abi.unpermute_backward))p[5],
            (decltype(abi.int8_quantize_rows))p[6], (decltype(abi.int8_matmul))p[7]};
  bound = true;
  Py_RETURN_NONE;
}

#define MOE_METHOD(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD(bind),
                         MOE_METHOD(group),
                         MOE_METHOD(permute),
                         MOE_METHOD(permute_backward),
                         MOE_METHOD(unpermute),
                         MOE_METHOD(unpermute_backward),
                         MOE_METHOD(int8_quantize_rows),
                         MOE_METHOD(int8_matmul),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Short calls of the binding", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for and abi_version: what the binding compares with its own before it uses the
// module, whose inlined code knows torch's tensors and the C entries by their layout.
PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && (PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) < 0 ||
            PyModule_AddIntConstant(m, "abi_version", MOE_ABI_VERSION) < 0))
    Py_CLEAR(m);
  return m;
}
