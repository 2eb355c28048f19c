// marshal.cpp -- the part of the Python binding whose calls are too short for
// interpreted marshalling: the low-rank adapters (a decode step's call takes a
// few microseconds on the GPU) and gradient clipping (hundreds of tensors a
// call).  Checks the tensors, allocates outputs and workspace on the current
// stream and calls libspops; it computes nothing.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "spops.h"

namespace {

struct BadArgument {
  std::string what;
};
struct BadStatus {
  const char* fn;
  int code;
};
struct PythonError {};

void need(bool ok, const char* name, const char* what) {
  if (!ok) throw BadArgument{std::string(name) + " " + what};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  need(THPVariable_Check(o), name, "must be a torch.Tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o && o != Py_None; }

spops_dtype dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return SPOPS_F32;
    case at::kHalf: return SPOPS_F16;
    case at::kBFloat16: return SPOPS_BF16;
    default: throw BadArgument{std::string(name) + " must be float32, float16 or bfloat16"};
  }
}

void status(const char* fn, int code) {
  if (code != SPOPS_OK) throw BadStatus{fn, code};
}

// Rows of unit stride; the distance between rows.
int64_t leading(const at::Tensor& t, const char* name) {
  need(t.layout() == at::kStrided, name, "must be a dense tensor");
  need(t.dim() == 2, name, "must be a matrix");
  need(t.size(1) <= 1 || t.stride(1) == 1, name, "must have unit stride along its rows");
  if (t.size(0) <= 1) return t.size(1) > 1 ? t.size(1) : 1;
  need(t.stride(0) >= t.size(1) && t.stride(0) >= 1, name, "must have rows that do not overlap");
  return t.stride(0);
}

// Whether two matrices with unit stride along their rows may share memory.
bool spans_meet(const at::Tensor& a, int64_t lda, const at::Tensor& b, int64_t ldb) {
  if (a.numel() == 0 || b.numel() == 0) return false;
  const auto end = [](const at::Tensor& t, int64_t ld) {
    return (const char*)t.data_ptr() + ((t.size(0) - 1) * ld + t.size(1)) * t.element_size();
  };
  return (const char*)a.data_ptr() < end(b, ldb) && (const char*)b.data_ptr() < end(a, lda);
}

void contiguous(const at::Tensor& t, const char* name) {
  need(t.layout() == at::kStrided && t.is_contiguous(), name, "must be contiguous");
}

void same_device(const at::Tensor& t, const char* name, c10::Device d) {
  need(t.is_cuda(), name, "must be a GPU tensor");
  need(t.device() == d, name, "must be on the device of the other tensors");
}

void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void* stream_of(c10::Device d) {
  return (void*)c10::hip::getCurrentHIPStream(d.index()).stream();
}

// Runs f and turns what it throws into Python errors.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const BadStatus& e) {
    PyObject* m = PyImport_ImportModule("unstructured_sparse_linear_amd.spops");
    if (m) {
      Py_XDECREF(PyObject_CallMethod(m, "_check", "si", e.fn, e.code));
      Py_DECREF(m);
      if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed with status %d", e.fn, e.code);
    }
  } catch (const PythonError&) {
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool count_args(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return false;
}

// ----------------------------------------------------- low-rank adapters --

// Arguments shared by the three calls: first (yt, dyt or W), xt, A, B,
// offsets, adapter, scale, ranks.
struct LowRank {
  const at::Tensor &first, &xt, &A, &B, &offsets, &adapter;
  spops_low_rank d{};
  int64_t ldx, ldf;
  PyObject* const* v;

  LowRank(PyObject* const* args, const char* first_name)
      : first(tensor(args[0], first_name)), xt(tensor(args[1], "xt")), A(tensor(args[2], "A")),
        B(tensor(args[3], "B")), offsets(tensor(args[4], "offsets")),
        adapter(tensor(args[5], "adapter")), v(args) {
    d.dtype = dtype_of(xt, "xt");
    ldx = leading(xt, "xt");
    ldf = leading(first, first_name);
    need(first.scalar_type() == xt.scalar_type(), first_name, "must have xt's dtype");
    need(A.scalar_type() == xt.scalar_type(), "A", "must have xt's dtype");
    need(B.scalar_type() == xt.scalar_type(), "B", "must have xt's dtype");
    need(A.dim() == 3, "A", "must be adapters x rank x in_features");
    need(B.dim() == 3, "B", "must be adapters x out_features x rank");
    contiguous(A, "A");
    contiguous(B, "B");
    d.tokens = xt.size(1);
    d.in_features = xt.size(0);
    d.adapters = A.size(0);
    d.rank = A.size(1);
    d.out_features = B.size(1);
    need(A.size(2) == d.in_features, "A", "must be adapters x rank x in_features");
    need(B.size(0) == d.adapters && B.size(2) == d.rank, "B",
         "must be adapters x out_features x rank");
    need(offsets.scalar_type() == at::kInt && offsets.dim() == 1, "offsets",
         "must be a vector of int32");
    need(adapter.scalar_type() == at::kInt && adapter.dim() == 1, "adapter",
         "must be a vector of int32");
    contiguous(offsets, "offsets");
    contiguous(adapter, "adapter");
    d.requests = adapter.numel();
    need(offsets.numel() == d.requests + 1, "offsets", "must have one entry more than adapter");
    d.A = A.data_ptr();
    d.B = B.data_ptr();
    d.offsets = (const int32_t*)offsets.data_ptr();
    d.adapter = (const int32_t*)adapter.data_ptr();
    if (given(args[6])) {
      const at::Tensor& t = tensor(args[6], "scale");
      need(t.scalar_type() == at::kFloat && t.dim() == 1 && t.numel() == d.adapters, "scale",
           "must be float32, one per adapter");
      contiguous(t, "scale");
      d.scale = (const float*)t.data_ptr();
    }
    if (given(args[7])) {
      const at::Tensor& t = tensor(args[7], "ranks");
      need(t.scalar_type() == at::kInt && t.dim() == 1 && t.numel() == d.adapters, "ranks",
           "must be int32, one per adapter");
      contiguous(t, "ranks");
      d.ranks = (const int32_t*)t.data_ptr();
    }
  }
  void devices(const char* first_name) const {
    const c10::Device dev = xt.device();
    same_device(xt, "xt", dev);
    same_device(first, first_name, dev);
    same_device(A, "A", dev);
    same_device(B, "B", dev);
    same_device(offsets, "offsets", dev);
    same_device(adapter, "adapter", dev);
    if (d.scale) same_device(THPVariable_Unpack(v[6]), "scale", dev);
    if (d.ranks) same_device(THPVariable_Unpack(v[7]), "ranks", dev);
  }
  at::Tensor workspace(int op, size_t& bytes) const {
    status("spops_low_rank_workspace_size",
           spops_low_rank_workspace_size(&d, (spops_low_rank_op)op, &bytes));
    return bytes ? at::empty({(int64_t)bytes}, xt.options().dtype(at::kByte)) : at::Tensor();
  }
};

PyObject* low_rank_forward(PyObject* const* args, Py_ssize_t n, bool project) {
  if (!count_args(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* name = project ? "W" : "yt";
    const LowRank L(args, name);
    if (project)
      need(L.first.size(0) == L.d.out_features && L.first.size(1) == L.d.in_features, name,
           "must be out_features x in_features");
    else
      need(L.first.size(0) == L.d.out_features && L.first.size(1) == L.d.tokens, name,
           "must be out_features x tokens");
    const bool into = given(args[8]);
    if (into) {
      const at::Tensor& o = tensor(args[8], "out");
      need(o.scalar_type() == L.xt.scalar_type(), "out", "must have xt's dtype");
      leading(o, "out");
      need(o.size(0) == L.d.out_features && o.size(1) == L.d.tokens, "out",
           "must be out_features x tokens");
    }
    L.devices(name);
    if (into) same_device(THPVariable_Unpack(args[8]), "out", L.xt.device());
    const c10::DeviceGuard guard(L.xt.device());
    at::Tensor out = into ? THPVariable_Unpack(args[8])
                          : at::empty({L.d.out_features, L.d.tokens}, L.xt.options());
    const int64_t ldo = leading(out, "out");
    const bool over_x = into && spans_meet(out, ldo, L.xt, L.ldx);
    size_t bytes = 0;
    const at::Tensor ws = L.workspace((project ? SPOPS_LOW_RANK_PROJECT : SPOPS_LOW_RANK_ADD) |
                                          (over_x ? SPOPS_LOW_RANK_OVER_X : 0),
                                      bytes);
    const auto call = project ? spops_low_rank_project : spops_low_rank_add;
    status(project ? "spops_low_rank_project" : "spops_low_rank_add",
           call(&L.d, L.first.data_ptr(), L.ldf, L.xt.data_ptr(), L.ldx, out.data_ptr(),
                ldo, ws.defined() ? ws.data_ptr() : nullptr, bytes, stream_of(L.xt.device())));
    if (into) {
      written(out);
      Py_INCREF(args[8]);
      return args[8];
    }
    return THPVariable_Wrap(out);
  });
}

PyObject* low_rank_add(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return low_rank_forward(args, n, false);
}
PyObject* low_rank_project(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return low_rank_forward(args, n, true);
}

PyObject* low_rank_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_args(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const LowRank L(args, "dyt");
    need(L.first.size(0) == L.d.out_features && L.first.size(1) == L.d.tokens, "dyt",
         "must be out_features x tokens");
    L.devices("dyt");
    const c10::DeviceGuard guard(L.xt.device());
    size_t bytes = 0;
    const at::Tensor ws = L.workspace(SPOPS_LOW_RANK_BACKWARD, bytes);
    const at::Tensor dx = at::empty({L.d.in_features, L.d.tokens}, L.xt.options());
    const at::Tensor dA = at::empty(L.A.sizes(), L.xt.options());
    const at::Tensor dB = at::empty(L.B.sizes(), L.xt.options());
    status("spops_low_rank_backward",
           spops_low_rank_backward(&L.d, L.first.data_ptr(), L.ldf, L.xt.data_ptr(), L.ldx,
                                   dx.data_ptr(), leading(dx, "dxt"), dA.data_ptr(), dB.data_ptr(),
                                   ws.defined() ? ws.data_ptr() : nullptr, bytes, stream_of(L.xt.device())));
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dx), THPVariable_Wrap(dA),
                         THPVariable_Wrap(dB));
  });
}

// ------------------------------------------- gradient norm and clipping --

// A borrowed view of a list or tuple.
struct Sequence {
  PyObject* seq;
  Sequence(PyObject* o, const char* what) : seq(PySequence_Fast(o, what)) {
    if (!seq) throw PythonError{};
  }
  ~Sequence() { Py_DECREF(seq); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// Whether no output starts where another one or another tensor's gradient does: the
// same tensor twice, a buffer beside its first slice, outputs in another order.  An
// open table of the outputs' addresses, under a microsecond for 200 tensors.
bool apart(const std::vector<spops_clip_tensor>& ts) {
  size_t size = 16;
  while (size < 2 * ts.size()) size *= 2;
  std::vector<int32_t> table(size, -1);
  const auto slot = [&](const void* p) {
    size_t at = ((uint64_t)(uintptr_t)p * 0x9e3779b97f4a7c15ull >> 20) & (size - 1);
    while (table[at] >= 0 && ts[(size_t)table[at]].out != p) at = (at + 1) & (size - 1);
    return &table[at];
  };
  for (size_t i = 0; i < ts.size(); ++i) {
    if (ts[i].numel == 0) continue;
    int32_t* s = slot(ts[i].out);
    if (*s >= 0) return false;
    *s = (int32_t)i;
  }
  for (size_t i = 0; i < ts.size(); ++i) {
    if (ts[i].numel == 0 || ts[i].grad == ts[i].out) continue;
    if (*slot(ts[i].grad) >= 0) return false;
  }
  return true;
}

PyObject* clip_grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!count_args(n, 3)) return nullptr;
  return guarded([&]() -> PyObject* {
    const double max_norm = PyFloat_AsDouble(args[1]);
    if (max_norm == -1.0 && PyErr_Occurred()) throw PythonError{};
    const Sequence grads(args[0], "grads must be a sequence of tensors");
    const bool into = given(args[2]);
    // one pass over grads: an iterator has no second
    const Sequence outs(into ? args[2] : grads.seq, "out must be a sequence of tensors");
    const Py_ssize_t count = grads.size();
    need(count > 0, "grads", "must hold at least one tensor");
    need(outs.size() == count, "out", "must have one tensor per gradient");
    std::vector<spops_clip_tensor> ts((size_t)count);
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor& g = tensor(grads[i], "every gradient");
      spops_clip_tensor& t = ts[(size_t)i];
      t.dtype = dtype_of(g, "every gradient");
      contiguous(g, "every gradient");
      t.numel = g.numel();
      t.grad = t.out = t.numel ? g.data_ptr() : nullptr;
      if (into) {
        const at::Tensor& o = tensor(outs[i], "every out");
        need(o.scalar_type() == g.scalar_type() && o.numel() == t.numel, "every out",
             "must have its gradient's dtype and size");
        contiguous(o, "every out");
        t.out = t.numel ? o.data_ptr() : nullptr;
      }
    }
    need(apart(ts), into ? "every out" : "every gradient",
         "must be a tensor of its own, given once");
    const at::Tensor& g0 = THPVariable_Unpack(grads[0]);
    const c10::Device dev = g0.device();
    for (Py_ssize_t i = 0; i < count; ++i) {
      same_device(THPVariable_Unpack(grads[i]), "every gradient", dev);
      if (into) same_device(THPVariable_Unpack(outs[i]), "every out", dev);
    }
    const c10::DeviceGuard guard(dev);
    size_t bytes = 0;
    status("spops_clip_grad_norm_workspace_size",
           spops_clip_grad_norm_workspace_size(count, &bytes));
    const at::Tensor ws = at::empty({(int64_t)bytes}, g0.options().dtype(at::kByte));
    const at::Tensor norm = at::empty({}, g0.options().dtype(at::kFloat));
    status("spops_clip_grad_norm",
           spops_clip_grad_norm(ts.data(), count, max_norm, (float*)norm.data_ptr(),
                                ws.data_ptr(), bytes, stream_of(dev)));
    for (Py_ssize_t i = 0; i < count; ++i) written(THPVariable_Unpack(outs[i]));
    return THPVariable_Wrap(norm);
  });
}

PyMethodDef methods[] = {
    {"low_rank_add", (PyCFunction)(void*)low_rank_add, METH_FASTCALL, nullptr},
    {"low_rank_project", (PyCFunction)(void*)low_rank_project, METH_FASTCALL, nullptr},
    {"low_rank_backward", (PyCFunction)(void*)low_rank_backward, METH_FASTCALL, nullptr},
    {"clip_grad_norm", (PyCFunction)(void*)clip_grad_norm, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
