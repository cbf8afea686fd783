// Python binding of the paged append and 8-bit cache entry points: tensors in, the C ABI (axr.h) out.
//
// The same marshalling as the ctypes front end (argument checks, current stream, output and workspace allocation),
// compiled: a call with fourteen tensors takes a few microseconds of host time here and about thirty through ctypes,
// more than these kernels themselves run on small batches.  No arithmetic happens here; there is no CPU path.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "axr.h"

namespace {

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(PyObject* type, const char* fmt, const char* a = "", const char* b = "") {
  PyErr_Format(type, fmt, a, b);
  throw Refused();
}

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kByte: return "torch.uint8";
    case at::kChar: return "torch.int8";
    case at::kInt: return "torch.int32";
    default: return c10::toString(t);
  }
}

// A tensor argument; None where it may be absent.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return &THPVariable_Unpack(o);
}

void need_cuda(const at::Tensor& t, const char* name, at::ScalarType dtype) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor (libaxr has no CPU path)", name);
  if (t.scalar_type() != dtype) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, dtype_name(dtype), dtype_name(t.scalar_type()));
    throw Refused();
  }
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
}

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? AXR_F32 : t == at::kHalf ? AXR_F16 : t == at::kBFloat16 ? AXR_BF16 : -1;
}

// Element stride between the tokens of t [n_tok, H, d], whose heads are contiguous (a slice of a fused projection row,
// or a contiguous tensor).
int64_t token_rows(const at::Tensor& t, const char* name, std::optional<at::ScalarType> dtype = std::nullopt) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor (libaxr has no CPU path)", name);
  if (dtype_code(t.scalar_type()) < 0 || (dtype && t.scalar_type() != *dtype)) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name,
                 dtype ? dtype_name(*dtype) : "float32, float16 or bfloat16", dtype_name(t.scalar_type()));
    throw Refused();
  }
  if (t.dim() != 3) refuse(PyExc_ValueError, "%s must be [n_tok, heads, d]", name);
  const int64_t n = t.size(0), H = t.size(1), d = t.size(2);
  if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && H > 1))
    refuse(PyExc_ValueError, "%s: the heads of a token must be contiguous", name);
  return n > 1 ? t.stride(0) : H * d;
}

void same_device(const at::Tensor& ref, std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    if (t && t->device() != ref.device())
      refuse(PyExc_ValueError, "tensors on %s and %s: one device expected", t->device().str().c_str(),
             ref.device().str().c_str());
}

const void* ptr(const at::Tensor* t) { return t ? t->const_data_ptr() : nullptr; }
void* mut(const at::Tensor* t) { return t ? t->mutable_data_ptr() : nullptr; }

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}

// axr statuses become the package's AxrError.
void check(axr_status st, const char* what) {
  if (st == AXR_OK) return;
  PyObject* m = PyImport_ImportModule("kv_cache_quantized_b200._abi");
  PyObject* r = m ? PyObject_CallMethod(m, "check", "is", static_cast<int>(st), what) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(m);
  throw Refused();
}

// What the two append calls share.
struct NewTokens {
  const at::Tensor *k, *v, *table, *lens, *cu, *q, *rope, *pos;
  at::Tensor q_out;
  PyObject* q_out_obj = nullptr;  // borrowed, when the caller passed it
  int64_t ks, vs, qs = 0, n, Hkv, Hq = 0, d, B, max_pos = 0, rot = 0;

  NewTokens(PyObject* k_, PyObject* v_, PyObject* table_, PyObject* lens_, PyObject* cu_, PyObject* q_,
            PyObject* rope_, PyObject* pos_, PyObject* out_, bool out_fp32) {
    k = tensor(k_, "k_new");
    v = tensor(v_, "v_new");
    ks = token_rows(*k, "k_new");
    vs = token_rows(*v, "v_new", k->scalar_type());
    n = k->size(0);
    Hkv = k->size(1);
    d = k->size(2);
    if (v->sizes() != k->sizes()) refuse(PyExc_ValueError, "k_new and v_new must have one shape");
    table = tensor(table_, "block_table");
    lens = tensor(lens_, "seq_lens");
    need_cuda(*table, "block_table", at::kInt);
    need_cuda(*lens, "seq_lens", at::kInt);
    if (table->dim() != 2 || lens->numel() != table->size(0))
      refuse(PyExc_ValueError, "block_table [B, max_blocks] and seq_lens [B] expected");
    B = table->size(0);
    cu = tensor(cu_, "cu_new", true);
    if (cu) {
      need_cuda(*cu, "cu_new", at::kInt);
      if (cu->numel() != B + 1) refuse(PyExc_ValueError, "cu_new must have B + 1 entries");
    } else if (n != B) {
      refuse(PyExc_ValueError, "without cu_new there is one new token per sequence");
    }
    pos = tensor(pos_, "positions", true);
    if (pos) {
      need_cuda(*pos, "positions", at::kInt);
      if (pos->numel() != n) refuse(PyExc_ValueError, "positions must have one entry per new token");
    }
    rope = tensor(rope_, "cos_sin", true);
    if (rope) {
      need_cuda(*rope, "cos_sin", at::kFloat);
      if (rope->dim() != 2) refuse(PyExc_ValueError, "cos_sin must be [max_pos, rot]");
      max_pos = rope->size(0);
      rot = rope->size(1);
    }
    q = tensor(q_, "q", true);
    if (q) {
      if (!rope) refuse(PyExc_ValueError, "q is taken to be rotated: pass cos_sin");
      qs = token_rows(*q, "q", k->scalar_type());
      if (q->size(0) != n || q->size(2) != d) refuse(PyExc_ValueError, "q must be [n_tok, Hq, d]");
      Hq = q->size(1);
      const auto dt = out_fp32 ? at::kFloat : k->scalar_type();
      if (out_ == Py_None) {
        q_out = at::empty({n, Hq, d}, q->options().dtype(dt));
      } else {
        q_out_obj = out_;
        q_out = *tensor(out_, "q_out");
        need_cuda(q_out, "q_out", dt);
        if (q_out.sizes() != q->sizes()) refuse(PyExc_ValueError, "q_out must have q's shape");
      }
    } else if (out_ != Py_None) {
      refuse(PyExc_ValueError, "q_out without q");
    }
    same_device(*k, {v, table, lens, cu, q, rope, pos, q ? &q_out : nullptr});
  }

  axr_dtype dtype() const { return static_cast<axr_dtype>(dtype_code(k->scalar_type())); }

  PyObject* result() const {
    if (!q) Py_RETURN_NONE;
    if (q_out_obj) {
      Py_INCREF(q_out_obj);
      return q_out_obj;
    }
    return THPVariable_Wrap(q_out);
  }
};

PyObject* wrong_count(const char* name, Py_ssize_t want, Py_ssize_t got) {
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
  return nullptr;
}

// k_new, v_new, kcodes, knorms, signs, bits, block_table, seq_lens, cu_new, q, cos_sin, positions, interleaved, v,
// vcodes, vnorms, q_out
PyObject* append_paged(PyObject*, PyObject* const* a, Py_ssize_t na) {
  if (na != 17) return wrong_count("append_paged", 17, na);
  HANDLE_TH_ERRORS
  try {
    NewTokens nt(a[0], a[1], a[6], a[7], a[8], a[9], a[10], a[11], a[16], true);
    const at::Tensor &kc = *tensor(a[2], "kcodes"), &kn = *tensor(a[3], "knorms"), &sg = *tensor(a[4], "signs");
    const int64_t bits = integer(a[5]);
    const int interleaved = truth(a[12]) ? 1 : 0;
    need_cuda(kc, "kcodes", at::kByte);
    need_cuda(kn, "knorms", at::kHalf);
    need_cuda(sg, "signs", at::kChar);
    if (kc.dim() != 4 || kc.size(1) != nt.Hkv || kc.size(3) != nt.d * bits / 8 || kn.dim() != 3 ||
        kn.sizes() != kc.sizes().slice(0, 3) || sg.numel() != nt.d)
      refuse(PyExc_ValueError, "kcodes [blocks, Hkv, bt, d*bits/8], knorms [blocks, Hkv, bt], signs [d] expected");
    const at::Tensor *v = tensor(a[13], "v", true), *vc = tensor(a[14], "vcodes", true),
                     *vn = tensor(a[15], "vnorms", true);
    if ((v == nullptr) == (vc == nullptr)) refuse(PyExc_ValueError, "pass exactly one of v or vcodes");
    if (v) {
      need_cuda(*v, "v", at::kHalf);
      if (v->dim() != 4 || v->sizes().slice(0, 3) != kc.sizes().slice(0, 3) || v->size(3) != nt.d)
        refuse(PyExc_ValueError, "v must be [blocks, Hkv, bt, d]");
      vn = nullptr;
    } else {
      need_cuda(*vc, "vcodes", at::kByte);
      if (!vn) refuse(PyExc_TypeError, "vnorms must be a torch.Tensor");
      need_cuda(*vn, "vnorms", at::kHalf);
      if (vc->sizes() != kc.sizes() || vn->sizes() != kn.sizes())
        refuse(PyExc_ValueError, "vcodes / vnorms must have the key pools' shapes");
    }
    same_device(*nt.k, {&kc, &kn, &sg, v, vc, vn});
    const c10::cuda::CUDAGuard guard(nt.k->device());
    check(axr_append_paged(
              ptr(nt.q), ptr(nt.k), ptr(nt.v), nt.dtype(), nt.qs, nt.ks, nt.vs,
              static_cast<const float*>(ptr(nt.rope)), nt.max_pos, static_cast<int>(nt.rot),
              interleaved, static_cast<const int32_t*>(ptr(nt.pos)),
              static_cast<const int32_t*>(ptr(nt.cu)), static_cast<const int32_t*>(ptr(nt.lens)), nt.n,
              static_cast<int>(nt.B), static_cast<int>(nt.Hq), static_cast<int>(nt.Hkv), static_cast<int>(nt.d),
              static_cast<int>(bits), static_cast<const int8_t*>(ptr(&sg)), static_cast<uint8_t*>(mut(&kc)),
              static_cast<uint16_t*>(mut(&kn)), v ? AXR_V_F16 : AXR_V_QUANT, v ? mut(v) : mut(vc),
              static_cast<uint16_t*>(mut(vn)), static_cast<const int32_t*>(ptr(nt.table)),
              static_cast<int>(nt.table->size(1)), static_cast<int>(kc.size(2)), static_cast<int>(kc.size(0)),
              nt.q ? static_cast<float*>(nt.q_out.mutable_data_ptr()) : nullptr,
              c10::cuda::getCurrentCUDAStream().stream()),
          "axr_append_paged");
    return nt.result();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

struct Pools8 {
  const at::Tensor *kc, *ks, *vc, *vs;
  int64_t nb, Hkv, bt, d;
  Pools8(PyObject* const* a) {
    kc = tensor(a[0], "kcodes");
    ks = tensor(a[1], "kscales");
    vc = tensor(a[2], "vcodes");
    vs = tensor(a[3], "vscales");
    one(*kc, *ks, "kcodes", "kscales");
    one(*vc, *vs, "vcodes", "vscales");
    if (vc->sizes() != kc->sizes()) refuse(PyExc_ValueError, "vcodes must have kcodes' shape");
    nb = kc->size(0);
    Hkv = kc->size(1);
    bt = kc->size(2);
    d = kc->size(3);
  }
  static void one(const at::Tensor& c, const at::Tensor& s, const char* cn, const char* sn) {
    need_cuda(c, cn, at::kByte);
    need_cuda(s, sn, at::kFloat);
    if (c.dim() != 4 || s.dim() != 3 || c.size(2) % 16 || s.size(0) != c.size(0) || s.size(1) != c.size(1) ||
        s.size(2) != c.size(2) / 16)
      refuse(PyExc_ValueError, "%s [blocks, Hkv, bt, d], %s [blocks, Hkv, bt/16] expected", cn, sn);
  }
};

// k_new, v_new, kcodes, kscales, vcodes, vscales, block_table, seq_lens, kind, cu_new, q, cos_sin, positions,
// interleaved, q_out
PyObject* q8_append_paged(PyObject*, PyObject* const* a, Py_ssize_t na) {
  if (na != 15) return wrong_count("q8_append_paged", 15, na);
  HANDLE_TH_ERRORS
  try {
    NewTokens nt(a[0], a[1], a[6], a[7], a[9], a[10], a[11], a[12], a[14], false);
    const Pools8 p(a + 2);
    const int interleaved = truth(a[13]) ? 1 : 0;
    if (p.Hkv != nt.Hkv || p.d != nt.d) refuse(PyExc_ValueError, "the pools do not match the new tokens' heads");
    same_device(*nt.k, {p.kc, p.ks, p.vc, p.vs});
    const c10::cuda::CUDAGuard guard(nt.k->device());
    check(axr_q8_append_paged(
              ptr(nt.q), ptr(nt.k), ptr(nt.v), nt.dtype(), nt.qs, nt.ks, nt.vs,
              static_cast<const float*>(ptr(nt.rope)), nt.max_pos, static_cast<int>(nt.rot),
              interleaved, static_cast<const int32_t*>(ptr(nt.pos)),
              static_cast<const int32_t*>(ptr(nt.cu)), static_cast<const int32_t*>(ptr(nt.lens)), nt.n,
              static_cast<int>(nt.B), static_cast<int>(nt.Hq), static_cast<int>(nt.Hkv), static_cast<int>(nt.d),
              static_cast<int>(integer(a[8])), static_cast<uint8_t*>(mut(p.kc)), static_cast<float*>(mut(p.ks)),
              static_cast<uint8_t*>(mut(p.vc)), static_cast<float*>(mut(p.vs)),
              static_cast<const int32_t*>(ptr(nt.table)), static_cast<int>(nt.table->size(1)),
              static_cast<int>(p.bt), static_cast<int>(p.nb), nt.q ? nt.q_out.mutable_data_ptr() : nullptr,
              c10::cuda::getCurrentCUDAStream().stream()),
          "axr_q8_append_paged");
    return nt.result();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// q, kcodes, kscales, vcodes, vscales, block_table, seq_lens, kind, cu_q, max_q, T, scale, out, workspace
PyObject* q8_attend_paged(PyObject*, PyObject* const* a, Py_ssize_t na) {
  if (na != 14) return wrong_count("q8_attend_paged", 14, na);
  HANDLE_TH_ERRORS
  try {
    const at::Tensor& q = *tensor(a[0], "q");
    const int64_t qs = token_rows(q, "q"), n = q.size(0), Hq = q.size(1), d = q.size(2);
    const Pools8 p(a + 1);
    if (p.d != d) refuse(PyExc_ValueError, "the pools do not match q's head dimension");
    const at::Tensor& table = *tensor(a[5], "block_table");
    need_cuda(table, "block_table", at::kInt);
    if (table.dim() != 2) refuse(PyExc_ValueError, "block_table must be [B, max_blocks]");
    const int64_t B = table.size(0), mb = table.size(1);
    const at::Tensor *lens = tensor(a[6], "seq_lens", true), *cu = tensor(a[8], "cu_q", true);
    if (lens) {
      need_cuda(*lens, "seq_lens", at::kInt);
      if (lens->numel() != B) refuse(PyExc_ValueError, "seq_lens must have B entries");
    }
    int64_t max_q = 1;
    if (cu) {
      need_cuda(*cu, "cu_q", at::kInt);
      if (cu->numel() != B + 1) refuse(PyExc_ValueError, "cu_q must have B + 1 entries");
      max_q = a[9] == Py_None ? 0 : integer(a[9]);
    } else if (n != B) {
      refuse(PyExc_ValueError, "without cu_q there is one query token per sequence");
    }
    const int64_t T = a[10] == Py_None ? mb * p.bt : integer(a[10]);
    double scale = 1.0 / std::sqrt(static_cast<double>(d));
    if (a[11] != Py_None) {
      scale = PyFloat_AsDouble(a[11]);
      if (scale == -1.0 && PyErr_Occurred()) throw Refused();
    }
    if (T < 0 || T > 0x7fffffff || max_q < 0 || max_q > 0x7fffffff)
      refuse(PyExc_ValueError, "T and max_q must be non-negative and below 2^31");
    at::Tensor out;
    if (a[12] == Py_None) {
      out = at::empty({n, Hq, d}, q.options());
    } else {
      out = *tensor(a[12], "out");
      need_cuda(out, "out", q.scalar_type());
      if (out.sizes() != q.sizes()) refuse(PyExc_ValueError, "out must be [n_tok, Hq, d]");
    }
    const at::Tensor* ws = tensor(a[13], "workspace", true);
    if (ws) need_cuda(*ws, "workspace", at::kByte);
    same_device(q, {p.kc, p.ks, p.vc, p.vs, &table, lens, cu, &out, ws});
    const size_t need = axr_q8_attend_workspace_bytes(n, static_cast<int>(max_q), static_cast<int>(B),
                                                      static_cast<int>(Hq), static_cast<int>(p.Hkv),
                                                      static_cast<int>(T), static_cast<int>(d));
    at::Tensor own;
    if (!ws && need) {
      own = at::empty({static_cast<int64_t>(need)}, q.options().dtype(at::kByte));
      ws = &own;
    }
    const c10::cuda::CUDAGuard guard(q.device());
    check(axr_q8_attend_paged(
              ptr(&q), static_cast<axr_dtype>(dtype_code(q.scalar_type())), qs, static_cast<const uint8_t*>(ptr(p.kc)),
              static_cast<const float*>(ptr(p.ks)), static_cast<const uint8_t*>(ptr(p.vc)),
              static_cast<const float*>(ptr(p.vs)), static_cast<int>(integer(a[7])),
              static_cast<const int32_t*>(ptr(&table)), static_cast<int>(mb), static_cast<int>(p.bt),
              static_cast<int>(p.nb), static_cast<const int32_t*>(ptr(cu)), static_cast<const int32_t*>(ptr(lens)), n,
              static_cast<int>(max_q), static_cast<int>(B), static_cast<int>(Hq), static_cast<int>(p.Hkv),
              static_cast<int>(T), static_cast<int>(d), static_cast<float>(scale), mut(&out), mut(ws),
              ws ? static_cast<size_t>(ws->numel()) : 0, c10::cuda::getCurrentCUDAStream().stream()),
          "axr_q8_attend_paged");
    if (a[12] != Py_None) {
      Py_INCREF(a[12]);
      return a[12];
    }
    return THPVariable_Wrap(out);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append_paged)), METH_FASTCALL, nullptr},
    {"q8_append_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(q8_append_paged)), METH_FASTCALL, nullptr},
    {"q8_attend_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(q8_attend_paged)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_axr_torch", "Compiled front end of libaxr's paged entry points.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__axr_torch(void) { return PyModule_Create(&module); }
