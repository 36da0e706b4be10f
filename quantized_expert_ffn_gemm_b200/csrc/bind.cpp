// The block operators of moe_ffn.h for torch tensors: argument checks, outputs from torch's allocator, one call of
// the C ABI. A decode step calls these operators with a microsecond or two of work for the GPU, and the same
// marshalling in Python with ctypes cost 9 to 15 us a call, most of it outputs allocated one by one. The
// functions take their arguments by position; block.py is the documented interface over them.
//
// A tensor of another type, shape, layout or device than the call takes raises ValueError, a status of the
// library raises the package's MoeError. The call runs on its tensors' device and that device's current stream.
//
// No call records a gradient (the gradients are entry points of their own). Where torch records and an input requires one,
// the results require one too, of a node that raises when a backward pass comes to it: as constants they would leave
// their share out of it unseen.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/VariableTypeUtils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/moe_ffn.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *g_moe_error = nullptr, *g_oom_error = nullptr;  // the package's MoeError, torch's out-of-memory error

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Status {
  const char *fn;
  moe_status code;
};

int type_code(ScalarType t) {
  return t == at::kFloat ? MOE_F32 : t == at::kHalf ? MOE_F16 : t == at::kBFloat16 ? MOE_BF16 : -1;
}

std::string sizes_of(const Tensor &t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

enum Types { kFloats, kF32Only, kI32Only, kU8Only };
const char *names_of(Types k) {
  return k == kFloats ? "float32, float16 or bfloat16" : k == kF32Only ? "float32" : k == kI32Only ? "int32" : "uint8";
}
bool type_in(ScalarType t, Types k) {
  return k == kFloats ? type_code(t) >= 0 : k == kF32Only ? t == at::kFloat : k == kI32Only ? t == at::kInt : t == at::kByte;
}

// The device of a call and its guard: set by the first tensor. And the inputs that require gradients.
struct Call {
  int device = -1;
  std::optional<c10::cuda::CUDAGuard> guard;
  std::vector<Tensor> grads;  // empty where torch does not record

  // a tensor argument, checked; nullptr for None where that is allowed
  const Tensor *tensor(const char *name, PyObject *o, Types types, int dim, bool optional = false) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": a tensor, got " + Py_TYPE(o)->tp_name);
    const Tensor &t = THPVariable_Unpack(o);
    if (!type_in(t.scalar_type(), types))
      throw Refused(std::string(name) + ": type " + c10::toString(t.scalar_type()) + ", takes " + names_of(types));
    if (dim >= 0 && t.dim() != dim)
      throw Refused(std::string(name) + ": shape " + sizes_of(t) + ", takes " + std::to_string(dim) + " dimensions");
    if (!t.is_cuda()) throw Refused(std::string(name) + ": not a CUDA tensor");
    if (device < 0) {
      device = t.get_device();
      if (device != c10::cuda::current_device()) guard.emplace(device);
    } else if (t.get_device() != device) {
      throw Refused(std::string(name) + ": on cuda:" + std::to_string(t.get_device()) + ", the call's other tensors on cuda:" +
                    std::to_string(device));
    }
    if (!t.is_contiguous()) throw Refused(std::string(name) + ": not contiguous");
    if (t.requires_grad() && c10::GradMode::is_enabled()) grads.push_back(t);
    return &t;
  }
  const Tensor *vector(const char *name, PyObject *o, Types types, int64_t n, bool optional = false) {
    const Tensor *t = tensor(name, o, types, 1, optional);
    if (t && t->size(0) != n)
      throw Refused(std::string(name) + ": shape " + sizes_of(*t) + ", takes (" + std::to_string(n) + ")");
    return t;
  }
  const Tensor *matrix(const char *name, PyObject *o, Types types, int64_t n, int64_t m, bool optional = false) {
    const Tensor *t = tensor(name, o, types, 2, optional);
    if (t && (t->size(0) != n || t->size(1) != m))
      throw Refused(std::string(name) + ": shape " + sizes_of(*t) + ", takes (" + std::to_string(n) + ", " +
                    std::to_string(m) + ")");
    return t;
  }
  // before a launch that writes a caller's buffer, all inputs read: torch's own rules for such a tensor
  void may_write(const char *name, const Tensor &buffer) const {
    if (!grads.empty() && buffer.is_inference()) throw Refused(std::string(name) + ": an inference tensor, with inputs that require gradients");
    torch::autograd::check_inplace(buffer, !grads.empty());
  }
  // Behind a launch that wrote it: whoever saved it for a backward pass is told by its version. (Inference tensors
  // have none.)
  void written(const char *call, const char *says, const Tensor &buffer) const {
    if (!buffer.is_inference()) torch::autograd::increment_version(buffer);
    if (!grads.empty()) torch::autograd::rebase_history(buffer, no_graph(call, says));
  }
  void results(const char *call, const char *says, std::initializer_list<const Tensor *> outs) const {
    if (grads.empty()) return;
    for (const Tensor *t : outs)
      if (t->defined()) torch::autograd::set_history(*t, no_graph(call, says));
  }
  std::shared_ptr<torch::autograd::Node> no_graph(const char *call, const char *says) const {
    return {new torch::autograd::Error(std::string(call) + " records no graph: " + says, torch::autograd::collect_next_edges(grads)),
            torch::autograd::deleteNode};
  }
  void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
};

void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
template <class T>
T *ptr_as(const Tensor *t) {
  return static_cast<T *>(ptr(t));
}
int32_t size32(int64_t n) {
  if (n > INT32_MAX) throw Refused("a size beyond 2^31 - 1");
  return (int32_t)n;
}
Tensor fresh(at::IntArrayRef sizes, const Tensor &like, ScalarType t) {
  return Tensor(at::detail::empty_cuda(sizes, t, like.device(), std::nullopt));
}
// Small outputs of one call in one allocation: tensors over parts of a buffer, each starting on 32 bytes.
struct Parts {
  const Tensor buf;
  int64_t at = 0;
  Parts(int64_t n, const Tensor &like, ScalarType t) : buf(fresh({n}, like, t)) {}
  static int64_t round(int64_t n) { return (n + 7) / 8 * 8; }  // of four bytes each
  Tensor take(at::IntArrayRef sizes) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(buf.storage()), buf.key_set(),
                                                     buf.dtype());
    impl->set_storage_offset(at);
    impl->set_sizes_contiguous(sizes);
    at += round(impl->numel());
    return Tensor(std::move(impl));
  }
};
void done(const char *fn, moe_status code) {
  if (code != MOE_OK) throw Status{fn, code};
}

// A Workspace: its buffer's address and size
struct Space {
  void *p;
  size_t n;
};
Space workspace(Call &c, PyObject *ws) {
  if (ws == Py_None) throw Refused("ws: this call needs a Workspace");
  static PyObject *const kBuf = PyUnicode_InternFromString("buf"), *const kBytes = PyUnicode_InternFromString("nbytes");
  PyObject *buf = PyObject_GetAttr(ws, kBuf), *n = buf ? PyObject_GetAttr(ws, kBytes) : nullptr;
  if (!buf || !n) {
    Py_XDECREF(buf);
    PyErr_Clear();
    throw Refused("ws: not a Workspace");
  }
  // the Workspace keeps its buffer: borrowed from here on
  Py_DECREF(buf);
  const long long bytes = PyLong_AsLongLong(n);
  Py_DECREF(n);
  const Tensor *t = c.tensor("ws", buf, kU8Only, 1);
  if (bytes < 0 || bytes > t->numel()) throw Refused("ws: not a Workspace");
  return {t->data_ptr(), (size_t)bytes};
}

bool flag(PyObject *o) {
  const int b = PyObject_IsTrue(o);
  if (b < 0) {
    PyErr_Clear();
    throw Refused("a truth value is needed");
  }
  return b;
}
float number(const char *name, PyObject *o) {
  const double d = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + ": takes a number");
  }
  return (float)d;
}
ScalarType dtype(const char *name, PyObject *o) {
  if (THPDtype_Check(o)) {
    const ScalarType t = reinterpret_cast<THPDtype *>(o)->scalar_type;
    if (type_code(t) >= 0) return t;
  }
  throw Refused(std::string(name) + ": takes torch.float32, torch.float16 or torch.bfloat16");
}

PyObject *wrap(const Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
template <class... T>
PyObject *tuple_of(const T &...t) {
  PyObject *items[] = {wrap(t)...};
  PyObject *out = PyTuple_New(sizeof...(t));
  for (size_t i = 0; i < sizeof...(t); ++i) PyTuple_SET_ITEM(out, (Py_ssize_t)i, items[i]);
  return out;
}

// runs f with the argument count checked and C++ failures turned into Python ones
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, const F &f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "takes %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Status &s) {
    if (PyObject *e = PyObject_CallFunction(g_moe_error, "si", s.fn, (int)s.code)) {
      PyErr_SetObject(g_moe_error, e);
      Py_DECREF(e);
    }
  } catch (const c10::OutOfMemoryError &e) {
    PyErr_SetString(g_oom_error, e.what_without_backtrace());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ----------------------------------------------------------------------------- the norms around a block
int gate_mode(Call &c, PyObject *o, int64_t T, int64_t H, const Tensor *&gate) {
  gate = nullptr;
  if (o == Py_None) return MOE_GATE_NONE;
  if (THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 2) {
    gate = c.matrix("gate", o, kF32Only, T, 1);
    return MOE_GATE_TOKEN;
  }
  gate = c.vector("gate", o, kF32Only, H);
  return MOE_GATE_CHANNEL;
}

// (r, y, post_gain, gate, res_scale, pre_gain, eps, post_norm, pre_norm, u_dtype, r_out)
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    Call c;
    const Tensor &r = *c.tensor("r", a[0], kFloats, 2);
    const int64_t T = r.size(0), H = r.size(1);
    const Tensor *y = c.matrix("y", a[1], kFloats, T, H, true), *post = c.vector("post_gain", a[2], kF32Only, H, true);
    const Tensor *pre = c.vector("pre_gain", a[5], kF32Only, H, true), *gate;
    const int mode = gate_mode(c, a[3], T, H, gate);
    const bool post_norm = flag(a[7]), pre_norm = flag(a[8]);
    const ScalarType ut = pre_norm ? dtype("u_dtype", a[9]) : at::kFloat;
    Tensor r_out;
    if (a[10] == Py_None) {
      r_out = fresh({T, H}, r, r.scalar_type());
    } else {
      r_out = *c.matrix("r_out", a[10], kFloats, T, H);
      if (r_out.scalar_type() != r.scalar_type()) throw Refused("r_out: another type than r");
      c.may_write("r_out", r_out);
    }
    Tensor u, rstd_y, rstd_u;
    const bool close = y && post_norm;
    if (pre_norm) u = fresh({T, H}, r, ut);
    if (pre_norm || close) {
      Parts parts((pre_norm + close) * Parts::round(T), r, at::kFloat);
      if (pre_norm) rstd_u = parts.take({T});
      if (close) rstd_y = parts.take({T});
    }
    done("moe_block_norm",
         moe_block_norm(r.data_ptr(), type_code(r.scalar_type()), ptr(y), y ? type_code(y->scalar_type()) : MOE_F32,
                        size32(T), size32(H), post_norm, ptr_as<float>(post), ptr_as<float>(gate), mode,
                        number("res_scale", a[4]), number("eps", a[6]), ptr_as<float>(pre), r_out.data_ptr(),
                        u.defined() ? u.data_ptr() : nullptr, type_code(ut),
                        rstd_y.defined() ? rstd_y.data_ptr<float>() : nullptr,
                        rstd_u.defined() ? rstd_u.data_ptr<float>() : nullptr, c.stream()));
    constexpr const char *kSays = "its gradient is block_norm_backward, for a torch.autograd.Function";
    if (a[10] != Py_None) c.written("block_norm", kSays, r_out);
    else c.results("block_norm", kSays, {&r_out});
    c.results("block_norm", kSays, {&u, &rstd_y, &rstd_u});
    return tuple_of(r_out, u, rstd_y, rstd_u);
  });
}

// (dr_out, du, r_out, rstd_u, y, rstd_y, post_gain, gate, res_scale, pre_gain, post_norm, ws)
PyObject *block_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Call c;
    const Tensor &r = *c.tensor("r_out", a[2], kFloats, 2);
    const int64_t T = r.size(0), H = r.size(1);
    const bool post_norm = flag(a[10]);
    const Tensor *dr_out = c.matrix("dr_out", a[0], kFloats, T, H, true), *du = c.matrix("du", a[1], kFloats, T, H, true);
    if (dr_out && dr_out->scalar_type() != r.scalar_type()) throw Refused("dr_out: another type than r_out");
    const Tensor *rstd_u = du ? c.vector("rstd_u", a[3], kF32Only, T) : nullptr;
    const Tensor *y = c.matrix("y", a[4], kFloats, T, H, true);
    const Tensor *rstd_y = y && post_norm ? c.vector("rstd_y", a[5], kF32Only, T) : nullptr;
    const Tensor *post = c.vector("post_gain", a[6], kF32Only, H, true), *gate;
    const Tensor *pre = c.vector("pre_gain", a[9], kF32Only, H, true);
    const int mode = gate_mode(c, a[7], T, H, gate);
    const Space ws = workspace(c, a[11]);
    Tensor dr = fresh({T, H}, r, r.scalar_type()), dy, d_post, d_gate, d_pre;
    if (y) dy = fresh({T, H}, r, y->scalar_type());
    if (post || gate || pre) {
      Parts parts(((post != nullptr) + (pre != nullptr)) * Parts::round(H) + (gate ? Parts::round(gate->numel()) : 0), r,
                  at::kFloat);
      if (post) d_post = parts.take({H});
      if (gate) d_gate = parts.take(gate->sizes());
      if (pre) d_pre = parts.take({H});
    }
    auto p32 = [](const Tensor &t) { return t.defined() ? t.data_ptr<float>() : nullptr; };
    done("moe_block_norm_backward",
         moe_block_norm_backward(ptr(dr_out), ptr(du), du ? type_code(du->scalar_type()) : MOE_F32, r.data_ptr(),
                                 type_code(r.scalar_type()), ptr_as<float>(rstd_u), ptr(y),
                                 y ? type_code(y->scalar_type()) : MOE_F32, ptr_as<float>(rstd_y), size32(T), size32(H),
                                 post_norm, ptr_as<float>(post), ptr_as<float>(gate), mode, number("res_scale", a[8]),
                                 du ? ptr_as<float>(pre) : nullptr, dr.data_ptr(), y ? dy.data_ptr() : nullptr, p32(d_post),
                                 p32(d_gate), du ? p32(d_pre) : nullptr, ws.p, ws.n, c.stream()));
    if (pre && !du) d_pre.zero_();  // nothing reaches u: the library takes pre_gain with du alone
    c.results("block_norm_backward", "second derivatives are not offered", {&dr, &dy, &d_post, &d_gate, &d_pre});
    return tuple_of(dr, dy, d_post, d_gate, d_pre);
  });
}

// ----------------------------------------------------------------------------- pairs sorted by expert
// (idx, E, ws)
PyObject *sort_pairs(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    Call c;
    const Tensor &idx = *c.tensor("idx", a[0], kI32Only, 2);
    const long long E = PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred() || E < 0 || E > INT32_MAX) {
      PyErr_Clear();
      throw Refused("E: takes a number of experts");
    }
    const Space ws = workspace(c, a[2]);
    const int64_t T = idx.size(0), k = idx.size(1);
    // what the library will refuse takes no memory: E alone, no tensor's size, says how much that would be
    if (!moe_block_workspace_bytes(size32(T), size32(k), (int32_t)E, 64)) throw Status{"moe_sort_pairs", MOE_ERR_INVALID_ARG};
    Parts parts(Parts::round(E) + Parts::round(E + 1) + 2 * Parts::round(T * k), idx, at::kInt);
    Tensor counts = parts.take({E}), offsets = parts.take({E + 1}), row_of = parts.take({T, k}), src = parts.take({T * k});
    done("moe_sort_pairs", moe_sort_pairs(idx.data_ptr<int32_t>(), size32(T), size32(k), (int32_t)E,
                                          counts.data_ptr<int32_t>(), offsets.data_ptr<int32_t>(),
                                          row_of.data_ptr<int32_t>(), src.data_ptr<int32_t>(), ws.p, ws.n, c.stream()));
    return tuple_of(counts, offsets, row_of, src);
  });
}

// device pointer to the kept pairs' number, the last offset
const int32_t *kept_of(Call &c, PyObject *o) {
  const Tensor *t = c.tensor("offsets", o, kI32Only, 1, true);
  if (!t) return nullptr;
  if (t->size(0) < 2) throw Refused("offsets: takes E + 1 entries");
  return t->data_ptr<int32_t>() + (t->size(0) - 1);
}

const Tensor &rows_of(Call &c, PyObject *o, PyObject *row_of, const Tensor *&pairs) {
  pairs = c.tensor("row_of", row_of, kI32Only, 2);
  const Tensor &rows = *c.tensor("rows", o, kFloats, 2);
  if (rows.size(0) != pairs->size(0) * pairs->size(1))
    throw Refused("rows: shape " + sizes_of(rows) + ", takes a row for each of row_of " + sizes_of(*pairs));
  return rows;
}

// (x, row_of, offsets, rows)
PyObject *dispatch(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    Call c;
    const Tensor &x = *c.tensor("x", a[0], kFloats, 2);
    const Tensor &row_of = *c.tensor("row_of", a[1], kI32Only, 2);
    const int64_t T = x.size(0), H = x.size(1), k = row_of.size(1);
    if (row_of.size(0) != T) throw Refused("row_of: shape " + sizes_of(row_of) + ", x has " + std::to_string(T) + " tokens");
    const int32_t *kept = kept_of(c, a[2]);
    Tensor rows;
    if (a[3] == Py_None) {
      rows = fresh({T * k, H}, x, x.scalar_type());
    } else {
      rows = *c.matrix("rows", a[3], kFloats, T * k, H);
      if (rows.scalar_type() != x.scalar_type()) throw Refused("rows: another type than x");
      c.may_write("rows", rows);
    }
    done("moe_dispatch", moe_dispatch(x.data_ptr(), type_code(x.scalar_type()), size32(T), size32(k), size32(H),
                                      row_of.data_ptr<int32_t>(), kept, rows.data_ptr(), c.stream()));
    constexpr const char *kSays = "its gradient is collect without weights, for a torch.autograd.Function";
    if (a[3] != Py_None) c.written("dispatch", kSays, rows);
    else c.results("dispatch", kSays, {&rows});
    return wrap(rows);
  });
}

// (rows, row_of, w, residual, dtype)
PyObject *collect(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    Call c;
    const Tensor *row_of, &rows = rows_of(c, a[0], a[1], row_of);
    const int64_t T = row_of->size(0), k = row_of->size(1), H = rows.size(1);
    const Tensor *w = c.matrix("w", a[2], kF32Only, T, k, true), *res = c.matrix("residual", a[3], kF32Only, T, H, true);
    const ScalarType yt = dtype("dtype", a[4]);
    Tensor y = fresh({T, H}, rows, yt);
    done("moe_collect", moe_collect(rows.data_ptr(), type_code(rows.scalar_type()), size32(T), size32(k), size32(H),
                                    row_of->data_ptr<int32_t>(), ptr_as<float>(w), ptr_as<float>(res), y.data_ptr(),
                                    type_code(yt), c.stream()));
    c.results("collect", "its gradient is collect_backward, for a torch.autograd.Function", {&y});
    return wrap(y);
  });
}

// (dy, rows, row_of, w, offsets)
PyObject *collect_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    Call c;
    const Tensor *row_of, &rows = rows_of(c, a[1], a[2], row_of);
    const int64_t T = row_of->size(0), k = row_of->size(1), H = rows.size(1);
    const Tensor &dy = *c.matrix("dy", a[0], kFloats, T, H);
    const Tensor *w = c.matrix("w", a[3], kF32Only, T, k, true);
    const int32_t *kept = kept_of(c, a[4]);
    Tensor d_rows = fresh(rows.sizes(), rows, rows.scalar_type()), d_w;
    if (w) d_w = fresh({T, k}, rows, at::kFloat);
    done("moe_collect_backward",
         moe_collect_backward(dy.data_ptr(), type_code(dy.scalar_type()), rows.data_ptr(), type_code(rows.scalar_type()),
                              size32(T), size32(k), size32(H), row_of->data_ptr<int32_t>(), ptr_as<float>(w), kept,
                              d_rows.data_ptr(), w ? d_w.data_ptr<float>() : nullptr, c.stream()));
    c.results("collect_backward", "second derivatives are not offered", {&d_rows, &d_w});
    return tuple_of(d_rows, d_w);
  });
}

// ----------------------------------------------------------------------------- MXFP4
// (x, row_of, offsets)
PyObject *mx4_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    Call c;
    const bool sorted = a[1] != Py_None;
    if (!sorted && a[2] != Py_None) throw Refused("offsets: goes with row_of");
    const Tensor &x = *c.tensor("x", a[0], kFloats, sorted ? 2 : -1);
    if (x.dim() < 1) throw Refused("x: takes a tensor [..., K]");
    const int64_t K = x.size(x.dim() - 1);
    int64_t T = 1, k = 1;
    const int32_t *kept = nullptr;
    const Tensor *row_of = nullptr;
    at::DimVector codes_size(x.sizes().begin(), x.sizes().end()), scales_size;
    for (int64_t i = 0; i + 1 < x.dim(); ++i) T *= x.size(i);
    if (sorted) {
      row_of = c.tensor("row_of", a[1], kI32Only, 2);
      if (row_of->size(0) != T) throw Refused("row_of: shape " + sizes_of(*row_of) + ", x has " + std::to_string(T) + " tokens");
      k = row_of->size(1);
      kept = kept_of(c, a[2]);
      codes_size[0] = T * k;
    }
    scales_size = codes_size;
    codes_size.back() = K / 2;
    scales_size.back() = K / 32;
    Tensor codes = fresh(codes_size, x, at::kByte), scales = fresh(scales_size, x, at::kByte);
    done("moe_mx4_quantize",
         moe_mx4_quantize(x.data_ptr(), type_code(x.scalar_type()), size32(T), size32(K), ptr_as<int32_t>(row_of),
                          size32(k), kept, codes.data_ptr<uint8_t>(), scales.data_ptr<uint8_t>(), c.stream()));
    return tuple_of(codes, scales);
  });
}

// MXFP4 rows (codes, scales), checked against one another: K
int64_t mx4(Call &c, const char *name, PyObject *o, const Tensor *&codes, const Tensor *&scales) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) throw Refused(std::string(name) + ": takes Mx4 rows");
  const std::string n = name;
  codes = c.tensor((n + ".codes").c_str(), PyTuple_GET_ITEM(o, 0), kU8Only, -1);
  scales = c.tensor((n + ".scales").c_str(), PyTuple_GET_ITEM(o, 1), kU8Only, -1);
  const int64_t d = codes->dim();
  if (d < 1 || codes->size(d - 1) % 16) throw Refused(n + ".codes: shape " + sizes_of(*codes) + ", takes [..., K/2], K % 32 = 0");
  bool same = scales->dim() == d && scales->size(d - 1) * 16 == codes->size(d - 1);
  for (int64_t i = 0; same && i + 1 < d; ++i) same = scales->size(i) == codes->size(i);
  if (!same) throw Refused(n + ".scales: shape " + sizes_of(*scales) + ", codes have " + sizes_of(*codes));
  return 2 * codes->size(d - 1);
}

// (q, dtype)
PyObject *mx4_dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 2, [&] {
    Call c;
    const Tensor *codes, *scales;
    const int64_t K = mx4(c, "q", a[0], codes, scales);
    const ScalarType t = dtype("dtype", a[1]);
    at::DimVector size(codes->sizes().begin(), codes->sizes().end());
    size.back() = K;
    int64_t rows = 1;
    for (size_t i = 0; i + 1 < size.size(); ++i) rows *= size[i];
    Tensor out = fresh(size, *codes, t);
    done("moe_mx4_dequantize", moe_mx4_dequantize(codes->data_ptr<uint8_t>(), scales->data_ptr<uint8_t>(), size32(rows),
                                                  size32(K), out.data_ptr(), type_code(t), c.stream()));
    return wrap(out);
  });
}

// (a, w, offsets, up, dtype, ws)
PyObject *mx4_product(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    Call c;
    const Tensor *ac, *as, *wc, *wsc, *uc = nullptr, *us = nullptr;
    const int64_t K = mx4(c, "a", a[0], ac, as);
    if (ac->dim() != 2) throw Refused("a: takes rows [rows, K]");
    if (mx4(c, "w", a[1], wc, wsc) != K || wc->dim() != 3)
      throw Refused("w: codes " + sizes_of(*wc) + ", takes [E, N, K/2] with a's K = " + std::to_string(K));
    if (a[3] != Py_None) {
      mx4(c, "up", a[3], uc, us);
      if (uc->sizes() != wc->sizes()) throw Refused("up: codes " + sizes_of(*uc) + ", w has " + sizes_of(*wc));
    }
    const int64_t rows = ac->size(0), E = wc->size(0), N = wc->size(1);
    const Tensor *offsets = c.vector("offsets", a[2], kI32Only, E + 1, true);
    const ScalarType t = dtype("dtype", a[4]);
    const Space ws = workspace(c, a[5]);
    const moe_mx4_mat w{size32(E), size32(N), size32(K), wc->data_ptr<uint8_t>(), wsc->data_ptr<uint8_t>()};
    moe_mx4_mat up = w;
    if (uc) {
      up.codes = uc->data_ptr<uint8_t>();
      up.scales = us->data_ptr<uint8_t>();
    }
    Tensor out = fresh({rows, N}, *ac, t);
    done("moe_mx4_product",
         moe_mx4_product(ac->data_ptr<uint8_t>(), as->data_ptr<uint8_t>(), size32(rows), ptr_as<int32_t>(offsets), w.n_experts,
                         &w, uc ? &up : nullptr, out.data_ptr(), type_code(t), ws.p, ws.n, c.stream()));
    return wrap(out);
  });
}

PyObject *init_errors(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 2, [&] {
    g_moe_error = Py_NewRef(a[0]);
    g_oom_error = Py_NewRef(a[1]);
    return Py_NewRef(Py_None);
  });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(block_norm),
                           FAST(block_norm_backward),
                           FAST(sort_pairs),
                           FAST(dispatch),
                           FAST(collect),
                           FAST(collect_backward),
                           FAST(mx4_quantize),
                           FAST(mx4_dequantize),
                           FAST(mx4_product),
                           FAST(init_errors),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
  PyObject *m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
