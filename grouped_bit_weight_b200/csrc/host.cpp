// host.cpp -- the Python module _host: argument checks, output allocation and
// the C ABI call of the routing, combine, whole-layer and MXFP4-activation
// entry points.  Their kernels take a few microseconds; done in Python, the
// checks, six allocations and the call took 20 (a routing call 27).
//
// Every function takes its arguments by position (the public functions in
// __init__.py carry the signatures and documentation), raises TypeError or
// ValueError for arguments the library cannot see through bare pointers, and
// GbwError (set by __init__.py) for a status of the library.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/gbw.h"

namespace {

PyObject* g_error = nullptr;  // GbwError(status, where)

struct Raise {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& s) { throw Raise{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Raise{PyExc_ValueError, s}; }

std::string str(int64_t v) { return std::to_string(v); }

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return "another dtype";
  }
}

// A tensor argument of one type, contiguous.
const at::Tensor& need(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType type) {
  const at::Tensor& t = need(o, name);
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + dtype_name(type) + ", got " +
               dtype_name(t.scalar_type()));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t;
}
const at::Tensor* optional(PyObject* o, const char* name, at::ScalarType type) {
  return o == Py_None ? nullptr : &need(o, name, type);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

bool is_shape(const at::Tensor& t, std::initializer_list<int64_t> s) {
  return t.sizes() == at::IntArrayRef(s.begin(), s.size());
}
void numel(const at::Tensor& t, const char* name, int64_t n, const std::string& where) {
  if (t.numel() != n)
    value_error(where + ": " + name + " has " + str(t.numel()) + " elements, needs " + str(n));
}

// The device of a call's tensors: one CUDA device.
struct Device {
  std::string where;
  int index = -1;
  void add(const char* name, const at::Tensor& t) {
    if (!t.is_cuda()) value_error(where + ": " + name + " must be a CUDA tensor");
    const int i = t.get_device();
    if (index < 0)
      index = i;
    else if (i != index)
      value_error(where + ": " + name + " is on cuda:" + str(i) + ", expected cuda:" + str(index));
  }
  void add(const char* name, const at::Tensor* t) {
    if (t) add(name, *t);
  }
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, index));
  }
};

// A tensor over part of another's memory, from its element `first` on (counted in
// `type`): much cheaper to make than an allocation or a view.
at::Tensor part(const at::Tensor& whole, at::ScalarType type, int64_t first, at::IntArrayRef sizes) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(whole.storage()), whole.key_set(), at::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(first);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}

template <typename T = void>
T* at_(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* at_(const at::Tensor* t) {
  return t ? at_<T>(*t) : nullptr;
}

// f(stream) with the device current; raises on a status.
template <typename F>
void call(const Device& d, F f) {
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (at::DeviceIndex)d.index));
  const gbw_status st = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(d.index).stream()));
  if (st == GBW_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, d.where.c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

// An output the caller gave (returned as that object) or one made here.
PyObject* given_or(PyObject* given, at::Tensor&& made) {
  if (given == Py_None) return wrap(std::move(made));
  Py_INCREF(given);
  return given;
}

int32_t logits_type(const at::Tensor& t, const std::string& where) {
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    type_error(std::string("logits must be torch.bfloat16 or torch.float32, got ") +
               dtype_name(t.scalar_type()));
  if (!t.is_contiguous()) value_error("logits must be contiguous");
  if (t.dim() != 2 || t.size(1) > INT32_MAX) value_error(where + ": logits must be [T, E]");
  return t.scalar_type() == at::kFloat ? GBW_LOGITS_FP32 : GBW_LOGITS_BF16;
}

// route(logits, k, renormalize) -> the six tensors of a Routing
PyObject* route(PyObject* const* a) {
  Device d{"gmoe_route"};
  const at::Tensor& l = need(a[0], "logits");
  const int32_t type = logits_type(l, d.where);
  const int64_t T = l.size(0), E = l.size(1), k = integer(a[1]);
  if (k < 1 || k > std::min<int64_t>(E, 32))
    value_error(d.where + ": k=" + str(k) + " must be in 1 .. min(E=" + str(E) + ", 32)");
  if (T * k > INT32_MAX) value_error(d.where + ": T * k must be below 2^31");
  d.add("logits", l);
  // the integer results and the workspace in one allocation; the weights in
  // their own (torch.save refuses one storage under two types)
  const int64_t n = T * k, bytes = gmoe_route_workspace(T, (int32_t)E);
  const at::Tensor all = d.empty({4 * n + E + 1 + bytes / 4}, at::kInt);
  const at::Tensor w = d.empty({T, k}, at::kFloat);
  const at::Tensor ids = part(all, at::kInt, 0, {T, k}), r2t = part(all, at::kInt, n, {n}),
                   ros = part(all, at::kInt, 2 * n, {T, k}), sor = part(all, at::kInt, 3 * n, {n}),
                   off = part(all, at::kInt, 4 * n, {E + 1});
  int32_t* ws = at_<int32_t>(all) + 4 * n + E + 1;
  const bool renorm = truth(a[2]);
  call(d, [&](void* s) {
    return gmoe_route(l.data_ptr(), type, T, (int32_t)E, (int32_t)k, renorm, at_<int32_t>(ids),
                      at_<float>(w), at_<int32_t>(off), at_<int32_t>(r2t), at_<int32_t>(ros),
                      at_<int32_t>(sor), bytes ? ws : nullptr, bytes, s);
  });
  return Py_BuildValue("NNNNNN", wrap(ids), wrap(w), wrap(off), wrap(r2t), wrap(ros), wrap(sor));
}

// route_bwd(logits, topk_ids, topk_weights, dweights, renormalize) -> dlogits
PyObject* route_bwd(PyObject* const* a) {
  Device d{"gmoe_route_bwd"};
  const at::Tensor& l = need(a[0], "logits");
  const int32_t type = logits_type(l, d.where);
  const at::Tensor &ids = need(a[1], "topk_ids", at::kInt), &w = need(a[2], "topk_weights", at::kFloat),
                   &dw = need(a[3], "dweights", at::kFloat);
  const int64_t T = l.size(0), E = l.size(1), k = ids.dim() == 2 ? ids.size(1) : 0;
  const bool fits = k >= 1 && k <= std::min<int64_t>(E, 32);
  auto check = [&](const char* name, const at::Tensor& t) {
    if (!fits || !is_shape(t, {T, k}))
      value_error(d.where + ": " + name + " must be [T=" + str(T) + ", k], k in 1 .. min(E, 32)");
  };
  check("topk_ids", ids);
  check("topk_weights", w);
  check("dweights", dw);
  d.add("logits", l);
  d.add("topk_ids", ids);
  d.add("topk_weights", w);
  d.add("dweights", dw);
  const at::Tensor out = d.empty({T, E}, l.scalar_type());
  const bool renorm = truth(a[4]);
  call(d, [&](void* s) {
    return gmoe_route_bwd(l.data_ptr(), type, T, (int32_t)E, (int32_t)k, renorm, at_<int32_t>(ids),
                          at_<float>(w), at_<float>(dw), out.data_ptr(), s);
  });
  return wrap(out);
}

struct Slots {
  int64_t P, H, T, k;
};
Slots slots(const std::string& where, const at::Tensor& y, const at::Tensor& rows,
            const at::Tensor* w) {
  if (y.dim() != 2 || rows.dim() != 2)
    value_error(where + ": y must be [P, H] and row_of_slot [T, k]");
  const Slots s{y.size(0), y.size(1), rows.size(0), rows.size(1)};
  if (w && !is_shape(*w, {s.T, s.k}))
    value_error(where + ": weights must be [" + str(s.T) + ", " + str(s.k) + "]");
  return s;
}

// combine(y, row_of_slot, weights, out) -> out
PyObject* combine(PyObject* const* a) {
  Device d{"gmoe_combine"};
  const at::Tensor &y = need(a[0], "y", at::kBFloat16), &rows = need(a[1], "row_of_slot", at::kInt);
  const at::Tensor* w = optional(a[2], "weights", at::kFloat);
  const Slots s = slots(d.where, y, rows, w);
  const at::Tensor* given = optional(a[3], "out", at::kBFloat16);
  if (given && !is_shape(*given, {s.T, s.H}))
    value_error(d.where + ": out must be [" + str(s.T) + ", " + str(s.H) + "]");
  d.add("y", y);
  d.add("row_of_slot", rows);
  d.add("weights", w);
  d.add("out", given);
  at::Tensor out = given ? *given : d.empty({s.T, s.H}, at::kBFloat16);
  call(d, [&](void* st) {
    return gmoe_combine(at_<uint16_t>(y), s.P, s.H, at_<int32_t>(rows), at_<float>(w), s.T,
                        (int32_t)s.k, at_<uint16_t>(out), st);
  });
  return given_or(a[3], std::move(out));
}

// combine_bwd(dout, y, row_of_slot, slot_of_row, weights, dy) -> (dy, dweights)
PyObject* combine_bwd(PyObject* const* a) {
  Device d{"gmoe_combine_bwd"};
  const at::Tensor &y = need(a[1], "y", at::kBFloat16), &rows = need(a[2], "row_of_slot", at::kInt);
  if (a[4] == Py_None) value_error(d.where + ": weights are needed");
  const at::Tensor& w = need(a[4], "weights", at::kFloat);
  const Slots s = slots(d.where, y, rows, &w);
  const at::Tensor &dout = need(a[0], "dout", at::kBFloat16), &inv = need(a[3], "slot_of_row", at::kInt);
  if (!is_shape(dout, {s.T, s.H}))
    value_error(d.where + ": dout must be [" + str(s.T) + ", " + str(s.H) + "]");
  numel(inv, "slot_of_row", s.P, d.where);
  const at::Tensor* given = optional(a[5], "dy", at::kBFloat16);
  if (given && !is_shape(*given, {s.P, s.H}))
    value_error(d.where + ": dy must be [" + str(s.P) + ", " + str(s.H) + "]");
  d.add("dout", dout);
  d.add("y", y);
  d.add("row_of_slot", rows);
  d.add("slot_of_row", inv);
  d.add("weights", w);
  d.add("dy", given);
  at::Tensor dy = given ? *given : d.empty({s.P, s.H}, at::kBFloat16);
  if (!given && s.P > s.T * s.k) dy.zero_();
  const at::Tensor dw = d.empty({s.T, s.k}, at::kFloat);
  call(d, [&](void* st) {
    return gmoe_combine_bwd(at_<uint16_t>(dout), at_<uint16_t>(y), s.P, s.H, at_<int32_t>(rows),
                            at_<int32_t>(inv), at_<float>(w), s.T, (int32_t)s.k, at_<uint16_t>(dy),
                            at_<float>(dw), st);
  });
  return Py_BuildValue("NN", given_or(a[5], std::move(dy)), wrap(dw));
}

// quantize_rows(x, row_to_token, swiglu) -> (codes, scales)
PyObject* quantize_rows(PyObject* const* a) {
  Device d{"gmxfp4_quantize_rows"};
  const at::Tensor& x = need(a[0], "x", at::kBFloat16);
  const bool glu = truth(a[2]);
  if (x.dim() != 2 || (glu && x.size(1) % 2))
    value_error(d.where + ": x must be [T, " + (glu ? "2K" : "K") + "]");
  const int64_t T = x.size(0), K = x.size(1) / (glu ? 2 : 1);
  if (K <= 0 || K % 32) value_error(d.where + ": K=" + str(K) + " must be a positive multiple of 32");
  const at::Tensor* r2t = optional(a[1], "row_to_token", at::kInt);
  const int64_t P = r2t ? r2t->numel() : T;
  if (P && !T) value_error(d.where + ": x has no rows");
  d.add("x", x);
  d.add("row_to_token", r2t);
  const int64_t KA = (K + 127) / 128;
  const at::Tensor all = d.empty({P * (K / 2 + KA * 4)}, at::kByte);
  const at::Tensor codes = part(all, at::kByte, 0, {P, K / 32, 16}),
                   scales = part(all, at::kByte, P * (K / 2), {KA, P, 4});
  call(d, [&](void* s) {
    return gmxfp4_quantize_rows(at_<uint16_t>(x), T, K, at_<int32_t>(r2t), P, glu,
                                at_<uint8_t>(codes), at_<uint8_t>(scales), s);
  });
  return Py_BuildValue("NN", wrap(codes), wrap(scales));
}

// grouped_gemm_a4(x_codes, x_scales, blocks, scales, expert_offsets, out) -> out
PyObject* grouped_gemm_a4(PyObject* const* a) {
  Device d{"gmxfp4_grouped_gemm_a4"};
  const at::Tensor &xc = need(a[0], "x_codes", at::kByte), &xs = need(a[1], "x_scales", at::kByte),
                   &w = need(a[2], "packed weights", at::kByte), &ws = need(a[3], "scales", at::kByte),
                   &off = need(a[4], "expert_offsets", at::kInt);
  if (xc.dim() != 3 || xc.size(2) != 16 || w.dim() < 3)
    value_error(d.where + ": x_codes must be [P, K/32, 16] and the weights [E, N, ...]");
  const int64_t P = xc.size(0), K = xc.size(1) * 32, E = w.size(0), N = w.size(1);
  if (K == 0 || !is_shape(xs, {(K + 127) / 128, P, 4}))
    value_error(d.where + ": x_scales must be [" + str((K + 127) / 128) + ", " + str(P) + ", 4]");
  numel(w, "packed weights", E * N * (K / 2), d.where);
  numel(ws, "scales", E * N * (K / 32), d.where);
  numel(off, "expert_offsets", E + 1, d.where);
  const at::Tensor* given = optional(a[5], "out", at::kBFloat16);
  if (given && !is_shape(*given, {P, N}))
    value_error(d.where + ": out must be [" + str(P) + ", " + str(N) + "]");
  d.add("x_codes", xc);
  d.add("x_scales", xs);
  d.add("blocks", w);
  d.add("scales", ws);
  d.add("expert_offsets", off);
  d.add("out", given);
  at::Tensor out = given ? *given : d.empty({P, N}, at::kBFloat16);
  call(d, [&](void* s) {
    return gmxfp4_grouped_gemm_a4(at_<uint8_t>(xc), at_<uint8_t>(xs), P, K, at_<uint8_t>(w),
                                  at_<uint8_t>(ws), (int32_t)E, N, at_<int32_t>(off),
                                  at_<uint16_t>(out), s);
  });
  return given_or(a[5], std::move(out));
}

// moe_layer(nf4, x, router_w, gu, gu_scale, dn, dn_scale, k, renormalize,
//           router_bias, out, workspace) -> out
PyObject* moe_layer(PyObject* const* a) {
  const bool nf4 = truth(a[0]);
  Device d{nf4 ? "gnf4_moe_layer" : "gmxfp4_moe_layer"};
  const at::ScalarType st = nf4 ? at::kFloat : at::kByte;
  const int64_t sdiv = nf4 ? 64 : 32;
  const at::Tensor &x = need(a[1], "x", at::kBFloat16), &rw = need(a[2], "router_w", at::kBFloat16),
                   &gu = need(a[3], "gate_up weights", at::kByte),
                   &gs = need(a[4], "gate_up scales", st),
                   &dn = need(a[5], "down weights", at::kByte), &ds = need(a[6], "down scales", st);
  if (x.dim() != 2 || rw.dim() != 2 || gu.dim() < 3 || dn.dim() < 3)
    value_error(d.where + ": x must be [T, H], router_w [E, H] and the weights [E, rows, ...]");
  const int64_t T = x.size(0), H = x.size(1), E = gu.size(0), I2 = gu.size(1), I = I2 / 2,
                k = integer(a[7]);
  if (T > 32)
    value_error(d.where + ": T=" + str(T) + ": the whole layer takes at most 32 tokens; use "
                "gmoe_route, the fused expert pass and gmoe_combine");
  if (I2 % 2 || dn.size(0) != E || dn.size(1) != H)
    value_error(d.where + ": gate_up must be [E, 2I, ...] and down [E, H=" + str(H) + ", ...]");
  if (!is_shape(rw, {E, H}))
    value_error(d.where + ": router_w must be [" + str(E) + ", " + str(H) + "]");
  if (k < 1 || k > std::min<int64_t>(E, 16))
    value_error(d.where + ": k=" + str(k) + " must be in 1 .. min(E=" + str(E) + ", 16)");
  if (!H || !I || H % 64 || I % 64)
    value_error(d.where + ": H=" + str(H) + " and I=" + str(I) + " must be positive multiples of 64");
  numel(gu, "gate_up weights", E * I2 * (H / 2), d.where);
  numel(gs, "gate_up scales", E * I2 * (H / sdiv), d.where);
  numel(dn, "down weights", E * H * (I / 2), d.where);
  numel(ds, "down scales", E * H * (I / sdiv), d.where);
  const at::Tensor* rb = optional(a[9], "router_bias", at::kFloat);
  if (rb) numel(*rb, "router_bias", E, d.where);
  const at::Tensor* given = optional(a[10], "out", at::kBFloat16);
  if (given && !is_shape(*given, {T, H}))
    value_error(d.where + ": out must be [" + str(T) + ", " + str(H) + "]");
  const int64_t bytes = gmoe_layer_workspace(T, (int32_t)E, (int32_t)k, H, I);
  const at::Tensor* own = optional(a[11], "workspace", at::kByte);
  if (own && own->numel() < bytes)
    value_error(d.where + ": workspace has " + str(own->numel()) + " bytes, needs " + str(bytes));
  d.add("x", x);
  d.add("router_w", rw);
  d.add("gu", gu);
  d.add("gu_scale", gs);
  d.add("dn", dn);
  d.add("dn_scale", ds);
  d.add("router_bias", rb);
  d.add("out", given);
  d.add("workspace", own);
  at::Tensor out = given ? *given : d.empty({T, H}, at::kBFloat16);
  const at::Tensor ws = own ? *own : d.empty({bytes}, at::kByte);
  const bool renorm = truth(a[8]);
  call(d, [&](void* s) {
    return nf4 ? gnf4_moe_layer(at_<uint16_t>(x), T, H, at_<uint16_t>(rw), at_<float>(rb),
                                at_<uint8_t>(gu), at_<float>(gs), at_<uint8_t>(dn), at_<float>(ds),
                                (int32_t)E, I, (int32_t)k, renorm, at_<uint16_t>(out), ws.data_ptr(),
                                ws.numel(), s)
               : gmxfp4_moe_layer(at_<uint16_t>(x), T, H, at_<uint16_t>(rw), at_<float>(rb),
                                  at_<uint8_t>(gu), at_<uint8_t>(gs), at_<uint8_t>(dn),
                                  at_<uint8_t>(ds), (int32_t)E, I, (int32_t)k, renorm,
                                  at_<uint16_t>(out), ws.data_ptr(), ws.numel(), s);
  });
  return given_or(a[10], std::move(out));
}

// A function of n positional arguments as a CPython one.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t n>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != n) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", n, nargs);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raise& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

#define GBW_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GBW_ENTRY(route, 3),
                         GBW_ENTRY(route_bwd, 5),
                         GBW_ENTRY(combine, 4),
                         GBW_ENTRY(combine_bwd, 6),
                         GBW_ENTRY(quantize_rows, 3),
                         GBW_ENTRY(grouped_gemm_a4, 6),
                         GBW_ENTRY(moe_layer, 12),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&module); }
