// bind.cpp -- the Python side of the latent calls (include/fp8idx.h): checks
// torch tensors, makes the outputs and the workspace, and calls the C ABI on
// the current stream.  These calls are made once a layer and token, and their
// kernels take a few microseconds, so the checks are compiled: the same ones
// in Python took 20 microseconds a call.
//
// Every function returns the library's code (an int, to be raised by the
// caller) or its results; arguments are positional, as __init__.py gives them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/fp8idx.h"

namespace {

constexpr int64_t kLatent = 512, kRope = 64, kPage = 64;

// The entry points of the loaded library.
decltype(&fp8idx_latent_store) f_store;
decltype(&fp8idx_sparse_latent_attention) f_sparse;
decltype(&fp8idx_sparse_latent_attention_workspace) f_sparse_ws;
decltype(&fp8idx_paged_latent_attention) f_paged;
decltype(&fp8idx_paged_latent_attention_workspace) f_paged_ws;

struct TypeError : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct ValueError : std::runtime_error {
  using std::runtime_error::runtime_error;
};

std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

// A CUDA tensor of one type; `o` may be None only where `optional`.
at::Tensor tensor(PyObject* o, const char* name, at::ScalarType type, bool optional = false) {
  if (optional && o == Py_None) return {};
  if (!THPVariable_Check(o)) throw TypeError(std::string(name) + " must be a CUDA tensor");
  at::Tensor t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw TypeError(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type)
    throw TypeError(std::string(name) + " must be torch." + (type == at::kBFloat16 ? "bfloat16" : type == at::kFloat ? "float32" : type == at::kInt ? "int32" : type == at::kLong ? "int64" : "uint8") +
                    ", got " + c10::toString(t.scalar_type()));
  return t;
}

const at::Tensor& dense(const at::Tensor& t, const char* name) {
  if (t.defined() && !t.is_contiguous()) throw ValueError(std::string(name) + " must be contiguous");
  return t;
}

// [..., width] whose last dimension is dense (outer strides are free).
const at::Tensor& rows(const at::Tensor& t, const char* name, int64_t width, int64_t dim) {
  if (t.dim() != dim || t.size(dim - 1) != width)
    throw ValueError(std::string(name) + " must have " + std::to_string(dim) + " dimensions, the last of " +
                     std::to_string(width) + ", got " + shape_of(t));
  if (t.stride(dim - 1) != 1) throw ValueError(std::string(name) + " must have unit stride in its last dimension");
  return t;
}

void same_device(const at::Tensor& ref, const at::Tensor& t, const char* name) {
  if (t.defined() && t.device() != ref.device())
    throw ValueError(std::string(name) + " is on " + t.device().str() + ", expected " + ref.device().str());
}

struct Pool {
  at::Tensor kv, s, pe;
  int64_t pages = 0, page = 0;
};

Pool pool(PyObject* kv, PyObject* s, PyObject* pe) {
  Pool p;
  if ((s == Py_None) != (pe == Py_None))
    throw ValueError("an fp8 pool has both s_pages and pe_pages, a bf16 pool neither");
  const bool fp8 = s != Py_None;
  if (fp8 && THPVariable_Check(kv) && THPVariable_Unpack(kv).scalar_type() == at::kFloat8_e4m3fn)
    p.kv = tensor(kv, "kv_pages", at::kFloat8_e4m3fn);
  else
    p.kv = tensor(kv, "kv_pages", fp8 ? at::kByte : at::kBFloat16);
  dense(p.kv, "kv_pages");
  const int64_t width = fp8 ? kLatent : kLatent + kRope;
  if (p.kv.dim() != 3 || p.kv.size(2) != width)
    throw ValueError("kv_pages must be [pages, 64, " + std::to_string(width) + "], got " + shape_of(p.kv));
  p.pages = p.kv.size(0);
  p.page = p.kv.size(1);
  if (fp8) {
    p.s = dense(tensor(s, "s_pages", at::kFloat), "s_pages");
    p.pe = dense(tensor(pe, "pe_pages", at::kBFloat16), "pe_pages");
    if (p.s.numel() != p.pages * p.page || p.pe.dim() != 3 || p.pe.size(0) != p.pages || p.pe.size(1) != p.page ||
        p.pe.size(2) != kRope)
      throw ValueError("kv_pages, s_pages and pe_pages disagree");
    same_device(p.kv, p.s, "s_pages");
    same_device(p.kv, p.pe, "pe_pages");
  }
  return p;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <class T>
T* as(const at::Tensor& t) {
  return static_cast<T*>(ptr(t));
}

// Makes the call's device current, and its stream, if the caller names one (a
// pointer as an int): the outputs and the workspace that the call makes are
// then that stream's, as under torch.cuda.stream, and the allocator does not
// hand the workspace to another stream while the call still uses it.
struct OnStream {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  void* stream;
  OnStream(PyObject* o, const at::Tensor& t) : device(t.device()) {
    if (o != Py_None)
      guard.reset_stream(
          c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(PyLong_AsVoidPtr(o)), t.device().index()));
    stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  }
};

// The stride of a dimension; one of size 1 has none that matters.
int64_t row_stride(const at::Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

// The calls have no backward pass and carry no tangents: neither must be lost
// in silence.  Every floating-point tensor of a call is looked at, those that
// it writes among them.
void no_grad(const at::Tensor& t, const char* name) {
  if (!t.defined()) return;
  if (t.requires_grad() && c10::GradMode::is_enabled())
    throw ValueError(std::string(name) + " requires grad, and this call has no backward: detach it or call under torch.no_grad()");
  if (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
    throw ValueError(std::string(name) + " has a tangent, and this call has no forward-mode derivative: detach it");
}
void no_grad(const Pool& p) {
  no_grad(p.kv, "kv_pages");
  no_grad(p.s, "s_pages");
  no_grad(p.pe, "pe_pages");
}

struct Outputs {
  at::Tensor out, lse;
};

Outputs outputs(const at::Tensor& q, PyObject* out, PyObject* lse, bool want_lse) {
  Outputs r;
  const int64_t n = q.size(0), h = q.size(1);
  r.out = dense(tensor(out, "out", at::kBFloat16, true), "out");
  if (!r.out.defined()) r.out = at::empty({n, h, kLatent}, q.options());
  else if (r.out.dim() != 3 || r.out.size(0) != n || r.out.size(1) != h || r.out.size(2) != kLatent)
    throw ValueError("out must be [" + std::to_string(n) + ", " + std::to_string(h) + ", 512]");
  r.lse = dense(tensor(lse, "lse", at::kFloat, true), "lse");
  if (!r.lse.defined()) {
    if (want_lse) r.lse = at::empty({n, h}, q.options().dtype(at::kFloat));
  } else if (r.lse.dim() != 2 || r.lse.size(0) != n || r.lse.size(1) != h) {
    throw ValueError("lse must be [" + std::to_string(n) + ", " + std::to_string(h) + "]");
  }
  same_device(q, r.out, "out");
  same_device(q, r.lse, "lse");
  no_grad(r.out, "out");
  no_grad(r.lse, "lse");
  return r;
}

at::Tensor workspace_of(const at::Tensor& q, PyObject* ws, size_t need) {
  if (ws == Py_None)
    return at::empty({static_cast<int64_t>(need < 256 ? 256 : need)}, q.options().dtype(at::kByte));
  at::Tensor t = dense(tensor(ws, "workspace", at::kByte), "workspace");
  same_device(q, t, "workspace");
  return t;
}

PyObject* results(int rc, const Outputs& o, bool want_lse) {
  if (rc != FP8IDX_OK) return PyLong_FromLong(rc);
  if (!want_lse) return THPVariable_Wrap(o.out);
  return Py_BuildValue("(NN)", THPVariable_Wrap(o.out), THPVariable_Wrap(o.lse));
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    PyObject* r = f();
    if (PyErr_Occurred()) {
      Py_XDECREF(r);
      return nullptr;
    }
    return r;
  } catch (const TypeError& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* kind = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (kind) PyErr_SetString(kind, e.what_without_backtrace());
    Py_XDECREF(kind);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// c, k_pe, positions, cos_sin, slot_mapping, kv_pages, s_pages, pe_pages, q_pe, q_out, interleaved, stream
PyObject* latent_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Pool p = pool(a[5], a[6], a[7]);
    if (p.page != kPage) throw ValueError("page size must be 64, got " + std::to_string(p.page));
    const at::Tensor c = rows(tensor(a[0], "c", at::kBFloat16), "c", kLatent, 2);
    const at::Tensor k_pe = rows(tensor(a[1], "k_pe", at::kBFloat16), "k_pe", kRope, 2);
    const at::Tensor pos = dense(tensor(a[2], "positions", at::kLong), "positions");
    const at::Tensor cs = dense(tensor(a[3], "cos_sin", at::kFloat), "cos_sin");
    const at::Tensor slot = dense(tensor(a[4], "slot_mapping", at::kLong), "slot_mapping");
    same_device(p.kv, c, "c");
    same_device(p.kv, k_pe, "k_pe");
    same_device(p.kv, pos, "positions");
    same_device(p.kv, cs, "cos_sin");
    same_device(p.kv, slot, "slot_mapping");
    const int64_t T = c.size(0);
    if (k_pe.size(0) != T || pos.numel() != T || slot.numel() != T)
      throw ValueError("c, k_pe, positions and slot_mapping must have one entry per token");
    if (cs.dim() != 2 || cs.size(1) != kRope) throw ValueError("cos_sin must be [max_pos, 64]");
    if ((a[8] == Py_None) != (a[9] == Py_None)) throw ValueError("q_pe and q_out go together");
    at::Tensor qi, qo;
    int64_t s[4] = {0, 0, 0, 0}, H = 1;
    if (a[8] != Py_None) {
      qi = rows(tensor(a[8], "q_pe", at::kBFloat16), "q_pe", kRope, 3);
      qo = rows(tensor(a[9], "q_out", at::kBFloat16), "q_out", kRope, 3);
      if (qi.sizes() != qo.sizes() || qi.size(0) != T) throw ValueError("q_pe and q_out must be [T, H, 64]");
      same_device(p.kv, qi, "q_pe");
      same_device(p.kv, qo, "q_out");
      s[0] = row_stride(qi, 0), s[1] = row_stride(qi, 1), s[2] = row_stride(qo, 0), s[3] = row_stride(qo, 1);
      no_grad(qi, "q_pe");
      no_grad(qo, "q_out");
      H = qi.size(1);
    }
    const int interleaved = PyObject_IsTrue(a[10]);
    no_grad(c, "c");
    no_grad(k_pe, "k_pe");
    no_grad(cs, "cos_sin");
    no_grad(p);
    const OnStream on(a[11], p.kv);
    return PyLong_FromLong(f_store(as<uint16_t>(c), row_stride(c, 0), as<uint16_t>(k_pe), row_stride(k_pe, 0), T, as<int64_t>(pos),
                                   as<float>(cs), cs.size(0), interleaved, as<int64_t>(slot), p.pages * kPage,
                                   ptr(p.kv), as<float>(p.s), as<uint16_t>(p.pe), as<uint16_t>(qi), s[0], s[1],
                                   as<uint16_t>(qo), s[2], s[3], static_cast<int>(H), on.stream));
  });
}

// q, kv_pages, slots, scale, s_pages, pe_pages, out, lse, workspace, return_lse, stream
PyObject* sparse_latent_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor q = rows(tensor(a[0], "q", at::kBFloat16), "q", kLatent + kRope, 3);
    const Pool p = pool(a[1], a[4], a[5]);
    const at::Tensor slots = tensor(a[2], "slots", at::kInt);
    const int64_t nr = q.size(0), H = q.size(1);
    if (slots.dim() != 2 || slots.size(0) != nr) throw ValueError("slots must be [rows, topk]");
    const int64_t topk = slots.size(1);
    if (topk > 1 && slots.stride(1) != 1) throw ValueError("slots must have unit column stride");
    if (topk > INT32_MAX || H > INT32_MAX) throw ValueError("size too large");
    same_device(q, p.kv, "kv_pages");
    same_device(q, slots, "slots");
    const double scale = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) return nullptr;
    const bool want_lse = PyObject_IsTrue(a[9]);
    no_grad(q, "q");
    no_grad(p);
    const OnStream on(a[10], q);
    const Outputs o = outputs(q, a[6], a[7], want_lse);
    const at::Tensor ws = workspace_of(q, a[8], f_sparse_ws(nr, static_cast<int>(H), static_cast<int>(topk)));
    const int64_t ld = nr <= 1 || topk == 0 ? topk : slots.stride(0);
    return results(f_sparse(as<uint16_t>(q), row_stride(q, 0), row_stride(q, 1), ptr(p.kv), as<float>(p.s), as<uint16_t>(p.pe),
                            p.pages * p.page, as<int32_t>(slots), ld, nr, static_cast<int>(topk), static_cast<int>(H),
                            kLatent, kRope, static_cast<float>(scale), as<uint16_t>(o.out), as<float>(o.lse), ptr(ws),
                            ws.numel(), on.stream),
                   o, want_lse);
  });
}

// q, kv_pages, block_table, seq_lens, R, scale, s_pages, pe_pages, out, lse, workspace, return_lse, stream
PyObject* paged_latent_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor q = rows(tensor(a[0], "q", at::kBFloat16), "q", kLatent + kRope, 3);
    const Pool p = pool(a[1], a[6], a[7]);
    const at::Tensor bt = dense(tensor(a[2], "block_table", at::kInt), "block_table");
    const at::Tensor sl = dense(tensor(a[3], "seq_lens", at::kInt), "seq_lens");
    if (bt.dim() != 2 || sl.numel() != bt.size(0)) throw ValueError("block_table must be [B, max_blocks] and seq_lens [B]");
    const int64_t B = bt.size(0), mb = bt.size(1), H = q.size(1);
    const int64_t R = PyLong_AsLongLong(a[4]);
    const double scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) return nullptr;
    if (R < INT32_MIN || R > INT32_MAX || H > INT32_MAX || mb > INT32_MAX) throw ValueError("size too large");
    if (q.size(0) != B * R)
      throw ValueError("q has " + std::to_string(q.size(0)) + " rows, expected B*R = " + std::to_string(B * R));
    same_device(q, p.kv, "kv_pages");
    same_device(q, bt, "block_table");
    same_device(q, sl, "seq_lens");
    const bool want_lse = PyObject_IsTrue(a[11]);
    no_grad(q, "q");
    no_grad(p);
    const OnStream on(a[12], q);
    const Outputs o = outputs(q, a[8], a[9], want_lse);
    const at::Tensor ws = workspace_of(
        q, a[10], f_paged_ws(B, static_cast<int>(R), static_cast<int>(mb), static_cast<int>(H)));
    return results(f_paged(as<uint16_t>(q), row_stride(q, 0), row_stride(q, 1), ptr(p.kv), as<float>(p.s), as<uint16_t>(p.pe),
                           as<int32_t>(bt), as<int32_t>(sl), B, static_cast<int>(R), static_cast<int>(mb), p.pages,
                           static_cast<int>(p.page), static_cast<int>(H), kLatent, kRope, static_cast<float>(scale),
                           as<uint16_t>(o.out), as<float>(o.lse), ptr(ws), ws.numel(), on.stream),
                   o, want_lse);
  });
}

// Takes the entry points from the library at `path` (already loaded or not).
PyObject* attach(PyObject*, PyObject* path) {
  const char* s = PyUnicode_AsUTF8(path);
  if (!s) return nullptr;
  void* h = dlopen(s, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  auto take = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    return f != nullptr;
  };
  if (!take(f_store, "fp8idx_latent_store") || !take(f_sparse, "fp8idx_sparse_latent_attention") ||
      !take(f_sparse_ws, "fp8idx_sparse_latent_attention_workspace") ||
      !take(f_paged, "fp8idx_paged_latent_attention") ||
      !take(f_paged_ws, "fp8idx_paged_latent_attention_workspace")) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks a latent entry point");
    return nullptr;
  }
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef kMethods[] = {
    {"attach", attach, METH_O, nullptr},
    {"latent_store", fast<latent_store>(), METH_FASTCALL, nullptr},
    {"sparse_latent_attention", fast<sparse_latent_attention>(), METH_FASTCALL, nullptr},
    {"paged_latent_attention", fast<paged_latent_attention>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&kModule); }
