// pkv_tensors.cpp -- torch tensors checked and handed to the rotary, append and
// verification calls of include/pkv.h, as a CPython module.
//
// These calls run a few microseconds on the device, so the host's share is what a
// decode step waits for.  Reading a tensor's device, type, sizes, strides and
// pointer through Python attributes and filling ctypes structures cost 20-23 us a
// call on the Grace host; here the same checks read the tensors directly.
// Every function returns the library's status code and raises ValueError for
// tensors that do not fit.  No computation happens here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "pkv.h"

namespace {

// A tensor or argument that does not fit: raised as ValueError.
struct Bad : std::invalid_argument {
  using std::invalid_argument::invalid_argument;
};

std::string shape_text(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}

// The tensors of one call: all on one CUDA device, none recording a gradient or
// carrying a tangent (both would end here unnoticed).
class Call {
 public:
  // The tensor behind `o`; nullptr for None where that is allowed.
  const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (o == Py_None) {
      if (optional) return nullptr;
      throw Bad(std::string(name) + ": a tensor is needed");
    }
    if (!THPVariable_Check(o)) throw Bad(std::string(name) + ": a tensor is needed");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.is_neg() ||
        (device_ >= 0 && t.get_device() != device_))
      throw Bad(std::string(name) + " on " + t.device().str() +
                ": plain tensors on one CUDA device are needed");
    device_ = t.get_device();
    // (tangents: of floating types only; asking costs 10 ns a tensor)
    if ((grad_ && t.requires_grad()) ||
        (tangents_ && at::isFloatingType(t.scalar_type()) && t._fw_grad(0).defined()))
      throw Bad(std::string(name) + ": this call records no gradient, detach its tensors "
                "(rope_apply with backward is the gradient of rope_apply)");
    return &t;
  }

  // A tensor that the call writes.
  const at::Tensor* output(PyObject* o, const char* name, bool optional = false) {
    const at::Tensor* t = tensor(o, name, optional);
    if (t) written_[num_written_++] = t;
    return t;
  }

  // Rows [tokens, heads, dim] with unit stride along dim.
  pkv_rows rows(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads, int64_t dim,
                at::ScalarType type) const {
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim ||
        t.scalar_type() != type || (t.numel() > 0 && dim > 1 && t.stride(2) != 1))
      fail(t, name, shape_text({tokens, heads, dim}), type);
    return {t.data_ptr(), t.stride(0), t.stride(1)};
  }

  pkv_probs probs(const at::Tensor& t, const char* name, int64_t b, int64_t rows, int64_t vocab,
                  at::ScalarType type) const {
    if (t.dim() != 3 || t.size(0) != b || t.size(1) != rows || t.size(2) != vocab ||
        t.scalar_type() != type || (t.numel() > 0 && vocab > 1 && t.stride(2) != 1))
      fail(t, name, shape_text({b, rows, vocab}), type);
    return {t.data_ptr(), t.stride(0), t.stride(1)};
  }

  // Contiguous values of `type`, [a] or (b >= 0) [a, b].
  template <typename T>
  T* flat(const at::Tensor* t, const char* name, at::ScalarType type, int64_t a,
          int64_t b = -1) const {
    if (!t) return nullptr;
    if (t->dim() != (b < 0 ? 1 : 2) || t->size(0) != a || (b >= 0 && t->size(1) != b) ||
        t->scalar_type() != type || !t->is_contiguous())
      throw Bad(std::string(name) + ": contiguous " + c10::toString(type) + " " +
                (b < 0 ? shape_text({a}) : shape_text({a, b})) + " is needed, got " +
                c10::toString(t->scalar_type()) + " " + shape_text(t->sizes()));
    return static_cast<T*>(t->data_ptr());
  }

  // Run `f(stream)` with the tensors' device current, on the given stream or the
  // device's current one; the interpreter is free meanwhile.  The outputs' version
  // counters go up, so that a graph which saved one raises instead of using it.
  template <typename F>
  PyObject* run(PyObject* stream, F f) const {
    cudaStream_t s;
    if (stream == Py_None) {
      s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
    } else {
      PyObject* p = PyObject_GetAttrString(stream, "cuda_stream");
      if (!p) return nullptr;
      s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(p));
      Py_DECREF(p);
      if (!s && PyErr_Occurred()) return nullptr;
    }
    for (int i = 0; i < num_written_; ++i)
      if (!written_[i]->is_inference()) written_[i]->unsafeGetTensorImpl()->bump_version();
    const int before = c10::cuda::current_device();
    if (before != device_) c10::cuda::set_device(static_cast<c10::DeviceIndex>(device_));
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f(s);
    Py_END_ALLOW_THREADS
    if (before != device_) c10::cuda::set_device(static_cast<c10::DeviceIndex>(before));
    return PyLong_FromLong(rc);
  }

 private:
  [[noreturn]] static void fail(const at::Tensor& t, const char* name, const std::string& shape,
                                at::ScalarType type) {
    throw Bad(std::string(name) + ": " + shape + " of " + c10::toString(type) +
              " with unit stride along the last dimension is needed, got " +
              shape_text(t.sizes()) + " of " + c10::toString(t.scalar_type()) + ", strides " +
              shape_text(t.strides()));
  }
  int64_t device_ = -1;
  const at::Tensor* written_[3];   // at most: verify_drafts has three outputs
  int num_written_ = 0;
  const bool grad_ = c10::GradMode::is_enabled();
  const bool tangents_ = c10::AutogradState::get_tls_state().get_fw_grad_mode();
};

pkv_dtype act_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return PKV_F32;
    case at::kHalf: return PKV_F16;
    case at::kBFloat16: return PKV_BF16;
    default: throw Bad(std::string("dtype ") + c10::toString(t) +
                       ": float32, float16 or bfloat16 is needed");
  }
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad(std::string(name) + ": an integer is needed");
  }
  return v;
}

int small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) throw Bad(std::string(name) + ": out of range");
  return static_cast<int>(v);
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad(std::string(name) + ": a number is needed");
  }
  return static_cast<float>(v);
}

template <typename T>
T* address(PyObject* o, const char* name) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p) {
    PyErr_Clear();
    throw Bad(std::string(name) + ": not open");
  }
  return static_cast<T*>(p);
}

// A rotation from its table [rotary_dim / 2], rotary_dim, interleaved and attn_scale,
// as they are at the call.
pkv_rope rotation(Call& c, PyObject* const* a) {
  const at::Tensor* freqs = c.tensor(a[0], "rope.freqs");
  const int rotary = small(a[1], "rope.rotary_dim");
  return {reinterpret_cast<const uint64_t*>(
              c.flat<int64_t>(freqs, "rope.freqs", at::kLong, rotary / 2)),
          rotary, small(a[2], "rope.interleaved"), number(a[3], "rope.attn_scale")};
}

// No C++ exception leaves a function of the module.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return f();
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// rope_apply(q_out, q, positions, freqs, rotary_dim, interleaved, attn_scale, k_out, k,
//            backward, stream)
PyObject* rope_apply_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    if ((a[7] == Py_None) != (a[8] == Py_None))
      throw Bad("rope_apply takes k and k_out together");
    Call c;
    const at::Tensor& q = *c.tensor(a[1], "q");
    const at::Tensor& qo = *c.output(a[0], "q_out");
    const at::Tensor* pos = c.tensor(a[2], "positions");
    const pkv_rope rope = rotation(c, a + 3);
    const at::Tensor* ko = c.output(a[7], "k_out", true);
    const at::Tensor* k = c.tensor(a[8], "k", true);
    const pkv_dtype dt = act_code(q.scalar_type());
    if (q.dim() != 3) throw Bad("q: [tokens, heads, head_dim] is needed, got " +
                                shape_text(q.sizes()));
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    if (H > INT32_MAX || D > INT32_MAX) throw Bad("q: out of range");
    const pkv_rows rq = c.rows(q, "q", T, H, D, q.scalar_type());
    const pkv_rows rqo = c.rows(qo, "q_out", T, H, D, q.scalar_type());
    pkv_rows rk{}, rko{};
    int64_t Hk = 0;
    if (k) {
      if (k->dim() != 3 || k->size(1) > INT32_MAX)
        throw Bad("k: [tokens, heads, head_dim] is needed, got " + shape_text(k->sizes()));
      Hk = k->size(1);
      rk = c.rows(*k, "k", T, Hk, D, q.scalar_type());
      rko = c.rows(*ko, "k_out", T, Hk, D, q.scalar_type());
    }
    const int32_t* p = c.flat<int32_t>(pos, "positions", at::kInt, T);
    const int backward = small(a[9], "backward");
    return c.run(a[10], [&](cudaStream_t s) {
      return rope_apply(&rqo, &rq, static_cast<int>(H), &rko, &rk, static_cast<int>(Hk), dt,
                        static_cast<int>(D), p, T, &rope, backward, s);
    });
  });
}

// append_rope(pool handle, pool storage, layer, q_out, q, k, v, freqs, rotary_dim,
//             interleaved, attn_scale, tables, positions, seq_ids, k_scale, v_scale, stream)
PyObject* append_rope_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    if ((a[3] == Py_None) != (a[4] == Py_None))
      throw Bad("append_rope takes q and q_out together");
    pkv_pool* pool = address<pkv_pool>(a[0], "pool");
    Call c;
    c.output(a[1], "pool");
    const int layer = small(a[2], "layer");
    const at::Tensor* qo = c.output(a[3], "q_out", true);
    const at::Tensor* q = c.tensor(a[4], "q", true);
    const at::Tensor& k = *c.tensor(a[5], "k");
    const at::Tensor& v = *c.tensor(a[6], "v");
    const pkv_rope rope = rotation(c, a + 7);
    const at::Tensor* tables = c.tensor(a[11], "tables");
    const at::Tensor* positions = c.tensor(a[12], "positions");
    const at::Tensor* seq = c.tensor(a[13], "seq_ids", true);
    pkv_geometry g;
    if (kv_pool_geometry(pool, &g) != PKV_OK) throw Bad("pool: not open");
    const at::ScalarType type = k.scalar_type();
    const pkv_dtype dt = act_code(type);
    const int64_t T = k.dim() ? k.size(0) : 0;
    const pkv_rows rk = c.rows(k, "k", T, g.num_kv_heads, g.head_dim, type);
    const pkv_rows rv = c.rows(v, "v", T, g.num_kv_heads, g.head_dim, type);
    pkv_rows rq{}, rqo{};
    if (q) {
      rq = c.rows(*q, "q", T, g.num_q_heads, g.head_dim, type);
      rqo = c.rows(*qo, "q_out", T, g.num_q_heads, g.head_dim, type);
    }
    if (tables->dim() != 2 || tables->size(0) > INT32_MAX || tables->size(1) > INT32_MAX ||
        (!seq && tables->size(0) < T))
      throw Bad("tables: one row [max_blocks] for each sequence is needed, got " +
                shape_text(tables->sizes()));
    const int B = static_cast<int>(tables->size(0)), W = static_cast<int>(tables->size(1));
    const int32_t* tab = c.flat<int32_t>(tables, "tables", at::kInt, B, W);
    const int32_t* pos = c.flat<int32_t>(positions, "positions", at::kInt, T);
    const int32_t* ids = c.flat<int32_t>(seq, "seq_ids", at::kInt, T);
    const float ks = number(a[14], "k_scale"), vs = number(a[15], "v_scale");
    return c.run(a[16], [&](cudaStream_t s) {
      return kv_append_rope(pool, layer, q ? &rqo : nullptr, q ? &rq : nullptr, &rk, &rv, dt,
                            &rope, tab, W, B, ids, pos, T, ks, vs, s);
    });
  });
}

// verify_drafts(tokens, num_accepted, target, draft, drafts, u_accept, u_sample,
//               num_drafts, status, stream)
PyObject* verify_drafts_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    Call c;
    const at::Tensor* tokens = c.output(a[0], "tokens");
    const at::Tensor* accepted = c.output(a[1], "num_accepted");
    const at::Tensor& target = *c.tensor(a[2], "target");
    const at::Tensor* draft = c.tensor(a[3], "draft", true);
    const at::Tensor* drafts = c.tensor(a[4], "drafts");
    const at::Tensor* ua = c.tensor(a[5], "u_accept");
    const at::Tensor* us = c.tensor(a[6], "u_sample");
    const at::Tensor* num = c.tensor(a[7], "num_drafts", true);
    const at::Tensor* status = c.output(a[8], "status", true);
    const pkv_dtype dt = act_code(target.scalar_type());
    if (drafts->dim() != 2 || target.dim() != 3 || drafts->size(0) > INT32_MAX ||
        drafts->size(1) >= INT32_MAX || target.size(2) > INT32_MAX)
      throw Bad("drafts [batch, max_drafts] and target [batch, max_drafts + 1, vocab] are needed, "
                "got " + shape_text(drafts->sizes()) + " and " + shape_text(target.sizes()));
    const int64_t B = drafts->size(0), K = drafts->size(1), V = target.size(2);
    const pkv_probs t = c.probs(target, "target", B, K + 1, V, target.scalar_type());
    pkv_probs d{};
    if (draft) d = c.probs(*draft, "draft", B, K, V, target.scalar_type());
    if (status && (status->scalar_type() != at::kInt || status->numel() < 1))
      throw Bad("status: an int32 tensor is needed");
    int32_t* out = c.flat<int32_t>(tokens, "tokens", at::kInt, B, K + 1);
    int32_t* acc = c.flat<int32_t>(accepted, "num_accepted", at::kInt, B);
    const int32_t* x = c.flat<int32_t>(drafts, "drafts", at::kInt, B, K);
    const int32_t* m = c.flat<int32_t>(num, "num_drafts", at::kInt, B);
    const float* u = c.flat<float>(ua, "u_accept", at::kFloat, B, K);
    const float* w = c.flat<float>(us, "u_sample", at::kFloat, B);
    int32_t* st = status ? static_cast<int32_t*>(status->data_ptr()) : nullptr;
    return c.run(a[9], [&](cudaStream_t s) {
      return verify_drafts(out, acc, &t, draft ? &d : nullptr, dt, x, m, u, w,
                           static_cast<int>(B), static_cast<int>(K), static_cast<int>(V), st, s);
    });
  });
}

#define PKV_METHOD(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PKV_METHOD("rope_apply", rope_apply_py),
    PKV_METHOD("append_rope", append_rope_py),
    PKV_METHOD("verify_drafts", verify_drafts_py),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pkv_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pkv_tensors() { return PyModule_Create(&module); }
