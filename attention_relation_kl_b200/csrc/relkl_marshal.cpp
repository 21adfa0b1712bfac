// Marshalling of tensors into the C ABI's records, for the calls whose time on
// the host is the marshalling: a step over many small tensors, a rotation or a
// product of a single token.  Checks, packing, and where a call has outputs or
// scratch of its own also those and the call.  What took 2.4 us a tensor in
// Python takes 0.1 us; a product of one row, 11.7 us in all, takes 6.4, of 77
// rows 9.2 instead of 16.4, and a rotation with two outputs 7.5 instead of 13.2.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <map>
#include <unordered_set>
#include <utility>
#include <vector>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <ATen/Functions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include "../../include/relkl.h"
#include "relkl_ranges.h"

namespace {

// A Python error that has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be tensors", what);
    throw Raised{};
  }
  return THPVariable_Unpack(o);
}

// A list or tuple (or what becomes one), held for the time of a call.
struct Items {
  PyObject* fast;
  Items(PyObject* o, const char* text) : fast(PySequence_Fast(o, text)) {
    if (!fast) throw Raised{};
  }
  ~Items() { Py_DECREF(fast); }
  Items(const Items&) = delete;
  Items& operator=(const Items&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  PyObject* operator[](Py_ssize_t k) const { return PySequence_Fast_GET_ITEM(fast, k); }
};

int32_t element(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return RELKL_BF16;
  if (t.scalar_type() == at::kFloat) return RELKL_FP32;
  PyErr_Format(PyExc_TypeError, "%s must be bfloat16 or float32", what);
  throw Raised{};
}

void on_device(const at::Tensor& t, int index) {
  if (!t.is_cuda() || t.get_device() != index)
    raise(PyExc_ValueError, "all tensors must be CUDA tensors on one device (there is no CPU path)");
}

void array_on_device(const at::Tensor& t, int index) {
  on_device(t, index);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "tensors must be contiguous");
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "marshalling failed");
  }
  return nullptr;
}

template <typename T>
PyObject* bytes_of(const std::vector<T>& v) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()),
                                   static_cast<Py_ssize_t>(v.size() * sizeof(T)));
}

// The library's entry points (bind).
struct Library {
  decltype(&relkl_rotary) rotary;
  decltype(&relkl_linear_i8) linear_i8;
  decltype(&relkl_linear_i8_bytes) linear_i8_bytes;
  decltype(&relkl_grad_norm) grad_norm;
  decltype(&relkl_grad_norm_bytes) grad_norm_bytes;
} library = {};

// bind(relkl_rotary, relkl_linear_i8, relkl_linear_i8_bytes, relkl_grad_norm,
//      relkl_grad_norm_bytes): their addresses
PyObject* bind(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    unsigned long long a, b, c, d, e;
    if (!PyArg_ParseTuple(args, "KKKKK", &a, &b, &c, &d, &e)) throw Raised{};
    library.rotary = reinterpret_cast<decltype(library.rotary)>(static_cast<uintptr_t>(a));
    library.linear_i8 = reinterpret_cast<decltype(library.linear_i8)>(static_cast<uintptr_t>(b));
    library.linear_i8_bytes = reinterpret_cast<decltype(library.linear_i8_bytes)>(static_cast<uintptr_t>(c));
    library.grad_norm = reinterpret_cast<decltype(library.grad_norm)>(static_cast<uintptr_t>(d));
    library.grad_norm_bytes = reinterpret_cast<decltype(library.grad_norm_bytes)>(static_cast<uintptr_t>(e));
    Py_RETURN_NONE;
  });
}

// Other threads run while device memory is had or a launch waits for its turn.
struct Released {
  PyThreadState* state;
  Released() : state(PyEval_SaveThread()) {}
  ~Released() { PyEval_RestoreThread(state); }
  Released(const Released&) = delete;
  Released& operator=(const Released&) = delete;
};

at::ScalarType output_type(PyObject* o) {
  if (THPDtype_Check(o)) {
    const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
    if (t == at::kBFloat16 || t == at::kFloat) return t;
  }
  PyErr_Format(PyExc_TypeError, "unsupported output dtype %R", o);
  throw Raised{};
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}

long long whole(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}

// adamw(params, grads, states, copies, weight_decay, step) ->
//   (device index, [(state bits, step, count, relkl_adamw_tensor records), ...]): tensors of
// one kind of states and one step number make a group, float32 states first, then by number
PyObject* adamw(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject *ps, *gs, *ss, *cs, *ds, *ns;
    if (!PyArg_ParseTuple(args, "OOOOOO", &ps, &gs, &ss, &cs, &ds, &ns)) throw Raised{};
    const Items params(ps, "params must be a sequence"), grads(gs, "grads must be a sequence");
    const Items states(ss, "states must be a sequence");
    const Items copies(cs == Py_None ? ps : cs, "copies must be a sequence");
    const Py_ssize_t n = params.size();
    if (grads.size() != n || states.size() != n || copies.size() != n)
      raise(PyExc_ValueError, "params, grads, states and copies need one entry for each tensor");
    const bool one_decay = PyFloat_Check(ds) || PyLong_Check(ds);
    const double decay = one_decay ? number(ds) : 0.0;
    const Items decays(one_decay ? ps : ds, "weight_decay must be a number or a sequence");
    if (decays.size() != n)
      raise(PyExc_ValueError, "weight_decay needs one number, or one for each tensor");
    const bool one_step = PyIndex_Check(ns) && !PySequence_Check(ns);
    const long long step = one_step ? whole(ns) : 0;
    const Items steps(one_step ? ps : ns, "step must be a number or a sequence");
    if (steps.size() != n) raise(PyExc_ValueError, "step needs one number, or one for each tensor");
    int index = -1;
    using Key = std::pair<bool, long long>;      // 8 bits, step
    std::map<Key, std::vector<relkl_adamw_tensor>> groups;
    std::vector<relkl_adamw_tensor>* group = nullptr;   // that of the last tensor, whose key is
    Key last;
    for (Py_ssize_t k = 0; k < n; ++k) {
      const at::Tensor& p = tensor(params[k], "params");
      const at::Tensor& g = tensor(grads[k], "gradients");
      if (k == 0) {
        if (!p.is_cuda()) raise(PyExc_ValueError, "params must be CUDA tensors (there is no CPU path)");
        index = static_cast<int>(p.get_device());
      }
      PyObject* s = states[k];
      if (!PyTuple_Check(s) || PyTuple_GET_SIZE(s) != 4)
        raise(PyExc_TypeError, "states must be AdamWState");
      const at::Tensor& m = tensor(PyTuple_GET_ITEM(s, 0), "states");
      const at::Tensor& v = tensor(PyTuple_GET_ITEM(s, 1), "states");
      PyObject *mo = PyTuple_GET_ITEM(s, 2), *vo = PyTuple_GET_ITEM(s, 3);
      const bool bits8 = m.scalar_type() == at::kFloat8_e4m3fn;
      if ((!bits8 && m.scalar_type() != at::kFloat) || v.scalar_type() != m.scalar_type())
        raise(PyExc_TypeError, "m and v must both be float32, or both float8_e4m3fn");
      relkl_adamw_tensor r = {};
      r.grad_dtype = element(g, "gradients");
      r.param_dtype = element(p, "parameters");
      const at::IntArrayRef shape = p.sizes();
      if (g.sizes() != shape || m.sizes() != shape || v.sizes() != shape)
        raise(PyExc_ValueError, "a parameter's gradient, states and copy must have its shape");
      array_on_device(p, index);
      array_on_device(g, index);
      array_on_device(m, index);
      array_on_device(v, index);
      r.grad = g.const_data_ptr();
      r.param = p.data_ptr();
      r.m = m.data_ptr();
      r.v = v.data_ptr();
      r.n = p.numel();
      if (cs != Py_None) {
        const at::Tensor& c = tensor(copies[k], "copies");
        if (c.scalar_type() != at::kBFloat16) raise(PyExc_TypeError, "copies must be bfloat16");
        if (c.sizes() != shape)
          raise(PyExc_ValueError, "a parameter's gradient, states and copy must have its shape");
        array_on_device(c, index);
        r.copy = c.data_ptr();
      }
      if (bits8) {
        if (mo == Py_None || vo == Py_None) raise(PyExc_ValueError, "8-bit states need their scales");
        const at::Tensor &a = tensor(mo, "states"), &b = tensor(vo, "states");
        const int64_t blocks = (r.n + 255) / 256;
        if (a.scalar_type() != at::kFloat || b.scalar_type() != at::kFloat || a.numel() != blocks ||
            b.numel() != blocks)
          raise(PyExc_ValueError, "8-bit states need a float32 scale for each 256 elements");
        array_on_device(a, index);
        array_on_device(b, index);
        r.m_scale = static_cast<float*>(a.data_ptr());
        r.v_scale = static_cast<float*>(b.data_ptr());
      } else if (mo != Py_None || vo != Py_None) {
        raise(PyExc_ValueError, "float32 states have no scales");
      }
      r.weight_decay = static_cast<float>(one_decay ? decay : number(decays[k]));
      const Key key{bits8, one_step ? step : whole(steps[k])};
      if (!group || key != last) {
        group = &groups[key];
        last = key;
        if (groups.size() == 1) group->reserve(static_cast<size_t>(n));
      }
      group->push_back(r);
    }
    if (groups.size() > 1) {   // as many calls, each of which looks at its own arrays
      std::vector<relkl::Range> ranges(relkl::kAdamwRanges * static_cast<size_t>(n));
      int64_t count = 0;
      for (const auto& [key, group] : groups)
        for (const relkl_adamw_tensor& t : group)
          count += relkl::adamw_ranges(t, key.first, ranges.data() + count);
      if (relkl::overlaps(ranges.data(), count))
        raise(PyExc_RuntimeError, "relkl_adamw: a tensor that is written overlaps another one of the call");
    }
    PyObject* list = PyList_New(0);
    if (!list) throw Raised{};
    for (const auto& [key, group] : groups) {
      PyObject* one = Py_BuildValue("(iLnN)", key.first ? 8 : 32, key.second,
                                    static_cast<Py_ssize_t>(group.size()), bytes_of(group));
      if (!one || PyList_Append(list, one) != 0) {
        Py_XDECREF(one);
        Py_DECREF(list);
        throw Raised{};
      }
      Py_DECREF(one);
    }
    return Py_BuildValue("(iN)", index, list);
  });
}

// written(tensors): what autograd saved of their old values is no longer valid
PyObject* written(PyObject*, PyObject* arg) {
  return guarded([&]() -> PyObject* {
    const Items items(arg, "expected a sequence");
    for (Py_ssize_t k = 0; k < items.size(); ++k) {
      const at::Tensor& t = tensor(items[k], "items");
      if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    }
    Py_RETURN_NONE;
  });
}

// graph_elsewhere(x) -> whether a node that x's gradient would reach belongs to another stream
// of x's device than the current one
PyObject* graph_elsewhere(PyObject*, PyObject* arg) {
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(arg, "x");
    if (!x.is_cuda() || !x.requires_grad()) Py_RETURN_FALSE;
    const c10::Stream here = c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getStream(x.device());
    std::unordered_set<torch::autograd::Node*> seen;
    const auto edge = torch::autograd::impl::gradient_edge(x);
    std::vector<torch::autograd::Node*> next{edge.function.get()};
    while (!next.empty()) {
      torch::autograd::Node* node = next.back();
      next.pop_back();
      if (!node || !seen.insert(node).second) continue;
      const auto stream = node->stream();
      if (stream && stream->device() == here.device() && *stream != here) Py_RETURN_TRUE;
      for (const auto& e : node->next_edges()) next.push_back(e.function.get());
    }
    Py_RETURN_FALSE;
  });
}

// norm(grads) -> (device index, relkl_norm_tensor records)
PyObject* norm(PyObject*, PyObject* arg) {
  return guarded([&]() -> PyObject* {
    const Items grads(arg, "grads must be a sequence");
    if (grads.size() == 0) raise(PyExc_ValueError, "no gradients");
    std::vector<relkl_norm_tensor> out(static_cast<size_t>(grads.size()));
    int index = -1;
    for (Py_ssize_t k = 0; k < grads.size(); ++k) {
      const at::Tensor& g = tensor(grads[k], "gradients");
      if (k == 0) {
        if (!g.is_cuda()) raise(PyExc_ValueError, "gradients must be CUDA tensors (there is no CPU path)");
        index = static_cast<int>(g.get_device());
      }
      array_on_device(g, index);
      out[k] = relkl_norm_tensor{g.const_data_ptr(), g.numel(), element(g, "gradients"), 0};
    }
    return Py_BuildValue("(iN)", index, bytes_of(out));
  });
}

// grad_norm(a gradient, records of norm, max_norm, out, stream) -> (status, out); out None: a
// tensor on the gradient's device
PyObject* grad_norm(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject *go, *yo;
    const char* records;
    Py_ssize_t bytes;
    double max_norm;
    unsigned long long stream;
    if (!PyArg_ParseTuple(args, "Oy#dOK", &go, &records, &bytes, &max_norm, &yo, &stream)) throw Raised{};
    if (!library.grad_norm) raise(PyExc_RuntimeError, "no library");
    const at::Tensor& g = tensor(go, "gradients");
    at::Tensor out;
    if (yo != Py_None) out = tensor(yo, "out");
    const int32_t n = static_cast<int32_t>(bytes / static_cast<Py_ssize_t>(sizeof(relkl_norm_tensor)));
    relkl_status status;
    {
      const Released released;
      if (yo == Py_None) out = at::empty({2}, g.options().dtype(at::kFloat));
      const size_t need = library.grad_norm_bytes(n);
      const at::Tensor scratch = at::empty({static_cast<int64_t>(need)}, g.options().dtype(at::kByte));
      status = library.grad_norm(n, reinterpret_cast<const relkl_norm_tensor*>(records),
                                 static_cast<float>(max_norm), static_cast<float*>(out.data_ptr()),
                                 scratch.data_ptr(), need, reinterpret_cast<void*>(stream));
    }
    return Py_BuildValue("(iN)", static_cast<int>(status), THPVariable_Wrap(out));
  });
}

// A [B, H, N, d] tensor's rows are contiguous (a dimension of one element has any stride).
bool rows_contiguous(const at::Tensor& t) { return t.size(3) <= 1 || t.stride(3) == 1; }

// rotary_inputs(xs, inv_freq) -> device index; checks what a call is given
PyObject* rotary_inputs(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject *xo, *fo;
    if (!PyArg_ParseTuple(args, "OO", &xo, &fo)) throw Raised{};
    const Items xs(xo, "expected a sequence of tensors");
    const Py_ssize_t n = xs.size();
    if (n < 1 || n > 3) raise(PyExc_ValueError, "1 to 3 tensors per call");
    const at::Tensor &x0 = tensor(xs[0], "xs"), &f = tensor(fo, "inv_freq");
    if (!x0.is_cuda()) raise(PyExc_ValueError, "x must be a CUDA tensor (there is no CPU path)");
    if (x0.dim() != 4) raise(PyExc_ValueError, "expected [B, H, N, d] tensors");
    element(x0, "inputs");
    const int index = static_cast<int>(x0.get_device());
    if (f.scalar_type() != at::kDouble || f.dim() != 1 || !f.is_contiguous() || !f.is_cuda() ||
        f.get_device() != index)
      raise(PyExc_ValueError, "inv_freq must be a contiguous float64 vector on the inputs' device");
    if (2 * f.numel() > x0.size(3))
      raise(PyExc_ValueError, "inv_freq has more pairs than a head holds");
    for (Py_ssize_t k = 0; k < n; ++k) {
      const at::Tensor& x = tensor(xs[k], "xs");
      if (x.dim() != 4 || x.scalar_type() != x0.scalar_type() || !x.is_cuda() || x.get_device() != index ||
          x.size(0) != x0.size(0) || x.size(2) != x0.size(2) || x.size(3) != x0.size(3))
        raise(PyExc_ValueError, "all tensors must share device, dtype, B, N and d");
      if (!rows_contiguous(x)) raise(PyExc_ValueError, "the last dimension must be contiguous");
      for (int i = 0; i < 4; ++i)
        if (x.size(i) > 0x7fffffff) raise(PyExc_ValueError, "a dimension exceeds 2^31 - 1");
    }
    return PyLong_FromLong(index);
  });
}

// rotary(xs, outs, output type, apply, inv_freq, positions, interleaved, inverse, mscale,
//        pos_scale, pos_offset, stream) -> (status, outputs), of inputs that rotary_inputs has
// accepted; outs None: contiguous tensors of the output type
PyObject* rotary(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject *xo, *yo, *to, *ao, *fo, *po;
    int interleaved, inverse;
    double mscale, pos_scale, pos_offset;
    unsigned long long stream;
    if (!PyArg_ParseTuple(args, "OOOOOOppdddK", &xo, &yo, &to, &ao, &fo, &po, &interleaved, &inverse,
                          &mscale, &pos_scale, &pos_offset, &stream))
      throw Raised{};
    if (!library.rotary) raise(PyExc_RuntimeError, "no library");
    const Items xs(xo, "expected a sequence of tensors");
    const Py_ssize_t n = xs.size();
    // held by references of their own: another thread may change the lists meanwhile
    std::vector<at::Tensor> inputs, outputs;
    for (Py_ssize_t k = 0; k < n; ++k) inputs.push_back(tensor(xs[k], "xs"));
    if (yo == Py_None) {
      const at::ScalarType type = output_type(to);
      const Released released;
      for (const at::Tensor& x : inputs) outputs.push_back(at::empty(x.sizes(), x.options().dtype(type)));
    } else {
      const Items ys(yo, "out must be a sequence of tensors");
      for (Py_ssize_t k = 0; k < ys.size(); ++k) outputs.push_back(tensor(ys[k], "out"));
    }
    if (n == 0 || static_cast<Py_ssize_t>(outputs.size()) != n)
      raise(PyExc_ValueError, "apply and out need one entry for each tensor");
    const Items apply(ao == Py_None ? xo : ao, "apply must be a sequence");
    if (apply.size() != n) raise(PyExc_ValueError, "apply and out need one entry for each tensor");
    const at::Tensor &x0 = inputs[0], &y0 = outputs[0], &f = tensor(fo, "inv_freq");
    const int index = static_cast<int>(x0.get_device());
    relkl_rotary_plan plan = {};
    plan.B = static_cast<int32_t>(x0.size(0));
    plan.N = static_cast<int32_t>(x0.size(2));
    plan.d = static_cast<int32_t>(x0.size(3));
    plan.rot = static_cast<int32_t>(2 * f.numel());
    plan.x_dtype = element(x0, "inputs");
    plan.y_dtype = element(y0, "outputs");
    plan.interleaved = interleaved;
    plan.inverse = inverse;
    plan.mscale = static_cast<float>(mscale);
    plan.pos_scale = pos_scale;
    plan.pos_offset = pos_offset;
    plan.inv_freq = static_cast<const double*>(f.const_data_ptr());
    if (po != Py_None) {
      const at::Tensor& p = tensor(po, "positions");
      if ((p.scalar_type() != at::kInt && p.scalar_type() != at::kLong) || !p.is_cuda() || p.get_device() != index)
        raise(PyExc_ValueError, "positions must be an int32 or int64 tensor on the inputs' device");
      const bool shared = p.dim() == 1 && p.size(0) == plan.N;
      if (!shared && !(p.dim() == 2 && p.size(0) == plan.B && p.size(1) == plan.N))
        raise(PyExc_ValueError, "positions must have shape (B, N) or (N,)");
      plan.positions = p.const_data_ptr();
      if (plan.positions) {      // else there is no token, and nothing to read
        plan.pos_bytes = static_cast<int32_t>(p.element_size());
        plan.pos_stride[0] = shared ? 0 : p.stride(0);
        plan.pos_stride[1] = p.stride(shared ? 0 : 1);
      }
    }
    std::vector<relkl_rotary_tensor> out(static_cast<size_t>(n));
    for (Py_ssize_t k = 0; k < n; ++k) {
      const at::Tensor &x = inputs[k], &y = outputs[k];
      if (y.sizes() != x.sizes() || y.scalar_type() != y0.scalar_type() || !y.is_cuda() ||
          y.get_device() != index || !rows_contiguous(y))
        raise(PyExc_ValueError,
              "out must be tensors of the inputs' shapes, of one type and on their device, whose last "
              "dimension is contiguous");
      relkl_rotary_tensor& t = out[k];
      t.x = x.const_data_ptr();
      t.y = y.data_ptr();
      for (int i = 0; i < 3; ++i) {
        t.x_stride[i] = x.stride(i);
        t.y_stride[i] = y.stride(i);
      }
      t.H = static_cast<int32_t>(x.size(1));
      const int turns = ao == Py_None ? 1 : PyObject_IsTrue(apply[k]);
      if (turns < 0) throw Raised{};
      t.apply = turns;
    }
    relkl_status status;
    {
      const Released released;
      status = library.rotary(static_cast<int32_t>(n), out.data(), &plan, reinterpret_cast<void*>(stream));
    }
    PyObject* list = PyList_New(n);
    if (!list) throw Raised{};
    for (Py_ssize_t k = 0; k < n; ++k) PyList_SET_ITEM(list, k, THPVariable_Wrap(outputs[k]));
    return Py_BuildValue("(iN)", static_cast<int>(status), list);
  });
}

[[noreturn]] void raise_about(PyObject* type, const char* what, const char* text) {
  PyErr_Format(type, "%s %s", what, text);
  throw Raised{};
}

struct Matrix {
  int64_t rows, K, stride;
  uintptr_t at;
  int32_t type;
};

// The rows of x [..., K], which must follow one another evenly.
Matrix matrix_of(const at::Tensor& x, const char* what) {
  if (!x.is_cuda()) raise_about(PyExc_ValueError, what, "must be a CUDA tensor (there is no CPU path)");
  const int32_t type = element(x, what);
  const int64_t dims = x.dim();
  if (dims < 1) raise_about(PyExc_ValueError, what, "must have at least one dimension");
  const int64_t K = x.size(dims - 1);
  if (K > 1 && x.stride(dims - 1) != 1)
    raise_about(PyExc_ValueError, what, "must have a contiguous last dimension");
  if (K > 0x7fffffff) raise_about(PyExc_ValueError, what, "has rows of more than 2^31 - 1 elements");
  int64_t rows = 1, stride = K, next = -1;   // next: the stride of a dimension around those seen
  for (int64_t i = dims - 2; i >= 0; --i) {
    const int64_t n = x.size(i);
    rows *= n;
    if (n <= 1) continue;
    if (next < 0)
      stride = x.stride(i);
    else if (x.stride(i) != next)
      raise_about(PyExc_ValueError, what, "must have rows that follow one another at one stride");
    next = x.stride(i) * n;
  }
  return Matrix{rows, K, stride, reinterpret_cast<uintptr_t>(x.const_data_ptr()), type};
}

// An int8 matrix laid out as relkl_quantize_rows lays it out; index -1: on any device.
Matrix codes_of(const at::Tensor& q, const char* what, int index) {
  if (!q.is_cuda() || (index >= 0 && q.get_device() != index))
    raise_about(PyExc_ValueError, what, "must be a CUDA tensor on the inputs' device (there is no CPU path)");
  if (q.scalar_type() != at::kChar || q.dim() != 2)
    raise_about(PyExc_ValueError, what, "must be an int8 matrix");
  const int64_t rows = q.size(0), K = q.size(1);
  int64_t stride = q.stride(0);
  if (rows <= 1) stride = (K + 15) / 16 * 16;   // one row has no stride
  const uintptr_t at = reinterpret_cast<uintptr_t>(q.const_data_ptr());
  if ((K > 1 && q.stride(1) != 1) || stride % 16 || stride < K || at % 16)
    raise_about(PyExc_ValueError, what,
                "must have contiguous rows that start at 16-byte boundaries, as relkl_quantize_rows "
                "lays them out");
  return Matrix{rows, K, stride, at, 0};
}

// A float32 vector of n, or None.
const float* vector_of(PyObject* o, long long n, const char* what, int index) {
  if (o == Py_None) return nullptr;
  const at::Tensor& v = tensor(o, what);
  if (v.scalar_type() != at::kFloat || v.dim() != 1 || v.numel() != n || !v.is_contiguous() || !v.is_cuda() ||
      v.get_device() != index) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous float32 vector of %lld on the inputs' device",
                 what, n);
    throw Raised{};
  }
  return static_cast<const float*>(v.const_data_ptr());
}

// matrix(x, what) -> (rows, K, row stride, address, relkl_dtype, device index)
PyObject* matrix(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject* o;
    const char* what;
    if (!PyArg_ParseTuple(args, "Os", &o, &what)) throw Raised{};
    const at::Tensor& x = tensor(o, what);
    const Matrix m = matrix_of(x, what);
    return Py_BuildValue("(LLLKii)", static_cast<long long>(m.rows), static_cast<long long>(m.K),
                         static_cast<long long>(m.stride), static_cast<unsigned long long>(m.at),
                         static_cast<int>(m.type), static_cast<int>(x.get_device()));
  });
}

// codes(q, what, device index) -> (rows, K, row stride, address)
PyObject* codes(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject* o;
    const char* what;
    int index;
    if (!PyArg_ParseTuple(args, "Osi", &o, &what, &index)) throw Raised{};
    const Matrix m = codes_of(tensor(o, what), what, index);
    return Py_BuildValue("(LLLK)", static_cast<long long>(m.rows), static_cast<long long>(m.K),
                         static_cast<long long>(m.stride), static_cast<unsigned long long>(m.at));
  });
}

// vector(v, n, what, device index) -> address of a float32 vector of n, 0 for None
PyObject* vector(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject* o;
    const char* what;
    long long n;
    int index;
    if (!PyArg_ParseTuple(args, "OLsi", &o, &n, &what, &index)) throw Raised{};
    return PyLong_FromVoidPtr(const_cast<float*>(vector_of(o, n, what, index)));
  });
}

// linear_i8(x, w, w_scale, bias, output type, out, ws, stream) -> (status, y); out None: a
// contiguous tensor, else one of the right shape and type on x's device that meets no input
PyObject* linear_i8(PyObject*, PyObject* args) {
  return guarded([&]() -> PyObject* {
    PyObject *xo, *wo, *so, *bo, *to, *yo, *ro;
    unsigned long long stream;
    if (!PyArg_ParseTuple(args, "OOOOOOOK", &xo, &wo, &so, &bo, &to, &yo, &ro, &stream)) throw Raised{};
    if (!library.linear_i8) raise(PyExc_RuntimeError, "no library");
    const at::Tensor &xt = tensor(xo, "x"), &wt = tensor(wo, "w"), &record = tensor(ro, "ws");
    const Matrix x = matrix_of(xt, "x");
    const int index = static_cast<int>(xt.get_device());
    const Matrix w = codes_of(wt, "w", index);
    if (w.K != x.K) {
      PyErr_Format(PyExc_ValueError, "x has rows of %lld elements, w of %lld", static_cast<long long>(x.K),
                   static_cast<long long>(w.K));
      throw Raised{};
    }
    if (w.rows > 0x7fffffff) raise(PyExc_ValueError, "w has more than 2^31 - 1 channels");
    if (so == Py_None) raise(PyExc_ValueError, "w_scale must be a float32 vector");
    const float* scale = vector_of(so, w.rows, "w_scale", index);
    const float* bias = vector_of(bo, w.rows, "bias", index);
    const int32_t K = static_cast<int32_t>(x.K);
    const at::ScalarType type = output_type(to);
    at::Tensor out, scratch;
    if (yo != Py_None) out = tensor(yo, "out");
    const size_t bytes = library.linear_i8_bytes(x.rows, K);
    {
      const Released released;
      if (yo == Py_None) {
        c10::SmallVector<int64_t, 5> shape(xt.sizes().begin(), xt.sizes().end());
        shape.back() = w.rows;
        out = at::empty(shape, xt.options().dtype(type));
      }
      if (bytes) scratch = at::empty({static_cast<int64_t>(bytes)}, xt.options().dtype(at::kByte));
    }
    const Matrix y = matrix_of(out, "out");
    relkl_status status;
    {
      const Released released;
      status = library.linear_i8(x.rows, static_cast<int32_t>(w.rows), K, reinterpret_cast<const void*>(x.at),
                                 x.type, x.stride, reinterpret_cast<const int8_t*>(w.at), w.stride, scale, bias,
                                 reinterpret_cast<void*>(y.at), y.type, y.stride,
                                 bytes ? scratch.data_ptr() : nullptr, bytes, record.data_ptr(),
                                 static_cast<size_t>(record.numel()), reinterpret_cast<void*>(stream));
    }
    return Py_BuildValue("(iN)", static_cast<int>(status), THPVariable_Wrap(out));
  });
}

PyMethodDef methods[] = {
    {"adamw", adamw, METH_VARARGS, "records of relkl_adamw"},
    {"written", written, METH_O, "marks tensors as changed in place"},
    {"graph_elsewhere", graph_elsewhere, METH_O, "whether a gradient would leave the current stream"},
    {"norm", norm, METH_O, "records of relkl_grad_norm"},
    {"grad_norm", grad_norm, METH_VARARGS, "relkl_grad_norm"},
    {"rotary_inputs", rotary_inputs, METH_VARARGS, "checks of relkl_rotary's inputs"},
    {"bind", bind, METH_VARARGS, "gives the library's entry points"},
    {"rotary", rotary, METH_VARARGS, "relkl_rotary"},
    {"linear_i8", linear_i8, METH_VARARGS, "relkl_linear_i8"},
    {"matrix", matrix, METH_VARARGS, "layout of a matrix of rows"},
    {"codes", codes, METH_VARARGS, "layout of a matrix of codes"},
    {"vector", vector, METH_VARARGS, "address of a float32 vector"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
