// binding.cpp -- the calls of a serving step (rotary positions, writes to pages, paged attention) from
// Python without the cost of ctypes.
//
// A step of one token takes a few microseconds on the GPU and several such calls per layer; checking a
// dozen tensors and packing them into C structures took 12 to 17 microseconds per call in Python.  This
// module does the same for the same C ABI (include/cowa.h): it checks its arguments, allocates what was
// not given, and calls the library that cowa.py has loaded, whose entry points it looks up in `use`.
// Each function returns (status, outputs ...); cowa.py turns a status into an exception.  It computes
// nothing itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/cowa.h"

namespace {

struct {
  decltype(&cowa_rope) rope, rope_bwd;
  decltype(&cowa_paged_append) append;
  decltype(&cowa_paged_append_fp8) append_fp8;
  decltype(&cowa_decode_paged) decode;
  decltype(&cowa_decode_paged_fp8) decode_fp8;
  decltype(&cowa_decode_paged_workspace_size) decode_size, decode_fp8_size;
  decltype(&cowa_fwd_paged) fwd;
  decltype(&cowa_fwd_paged_workspace_size) fwd_size;
} lib;

// A refused argument: a Python exception's type and text.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void bad_value(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
[[noreturn]] void bad_type(const std::string& s) { throw Refused{PyExc_TypeError, s}; }

const at::Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (!t) bad_type(std::string(name) + " must be a tensor");
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}

void of_type(const at::Tensor& t, const char* name, at::ScalarType type, const char* what) {
  if (!t.is_cuda() || t.scalar_type() != type) bad_type(std::string(name) + " must be a CUDA " + what + " tensor");
}
void bf16(const at::Tensor& t, const char* name) { of_type(t, name, at::kBFloat16, "bfloat16"); }
void of_shape(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) {
    std::string s = std::string(name) + " has shape [";
    for (auto v : t.sizes()) s += std::to_string(v) + ", ";
    s += "], expected [";
    for (auto v : shape) s += std::to_string(v) + ", ";
    bad_value(s + "]");
  }
}
// int32 values, contiguous along the last dimension
const int32_t* int32(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  of_type(t, name, at::kInt, "int32");
  of_shape(t, name, shape);
  if (shape.back() > 1 && t.stride(-1) != 1) bad_value(std::string(name) + " must be contiguous along its last dimension");
  return static_cast<const int32_t*>(t.data_ptr());
}
// every tensor of a call is on x's device
void same_device(const at::Tensor& x, std::initializer_list<const at::Tensor*> others) {
  for (const at::Tensor* y : others)
    if (y && y->device() != x.device())
      bad_value("tensors are on different devices: " + x.device().str() + " and " + y->device().str());
}
// The stride of dimension i; that of a dimension of one element, which may be anything, as d: the library wants
// every stride to be a positive multiple of 16 bytes
int64_t stride(const at::Tensor& t, int i) { return t.size(i) > 1 ? t.stride(i) : t.size(-1); }
// [B, N, H, d] or packed [total, H, d] (d contiguous) as a cowa_tensor
cowa_tensor rows(const at::Tensor& t, const char* name) {
  if (t.stride(-1) != 1) bad_value(std::string("the last dimension of ") + name + " must be contiguous");
  if (t.dim() == 3) return {t.data_ptr(), stride(t, 0) * std::max<int64_t>(1, t.size(0)), stride(t, 0), stride(t, 1)};
  return {t.data_ptr(), stride(t, 0), stride(t, 1), stride(t, 2)};
}
int to_int(int64_t v) {
  if (v > 0x7fffffff) bad_value("a dimension is larger than 2^31 - 1");
  return (int)v;
}

// Pools [n_pages, page_size, H, d] ("bthd") or [n_pages, H, page_size, d] ("bhtd") with a table
// [n_seq, max_pages], H = H_kv, or [n_seq, H_kv, max_pages], H = 1.
struct Pages {
  cowa_tensor k, v;
  cowa_page_table table;
  int n_seq, Hkv;
};
Pages pages(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, PyObject* layout, int64_t d,
            bool codes) {
  of_type(k, "k_pages", codes ? at::kByte : at::kBFloat16, codes ? "uint8 (E4M3 codes)" : "bfloat16");
  of_type(v, "v_pages", codes ? at::kByte : at::kBFloat16, codes ? "uint8 (E4M3 codes)" : "bfloat16");
  of_type(table, "page_table", at::kInt, "int32");
  const char* l = PyUnicode_Check(layout) ? PyUnicode_AsUTF8(layout) : nullptr;
  const bool bthd = l && std::string(l) == "bthd";
  if (!bthd && !(l && std::string(l) == "bhtd")) bad_value("layout must be 'bhtd' or 'bthd'");
  const int t = bthd ? 1 : 2, h = bthd ? 2 : 1;
  const int64_t dims = table.dim();
  if ((dims != 2 && dims != 3) || (table.size(-1) > 1 && table.stride(-1) != 1))
    bad_value("page_table is [n_seq, max_pages] or [n_seq, H_kv, max_pages], contiguous along the last dimension");
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.size(3) != d)
    bad_value("k_pages and v_pages must be 4-D pools of the same shape and head dimension");
  if (dims == 3 && k.size(h) != 1) bad_value("with a page table per KV head a page holds one head");
  if (k.stride(3) != 1 || v.stride(3) != 1) bad_value("the last dimension of the pools must be contiguous");
  Pages p;
  p.k = {k.data_ptr(), stride(k, 0), stride(k, t), stride(k, h)};
  p.v = {v.data_ptr(), stride(v, 0), stride(v, t), stride(v, h)};
  p.Hkv = to_int(dims == 3 ? table.size(1) : k.size(h));
  p.n_seq = to_int(table.size(0));
  p.table = {static_cast<const int32_t*>(table.data_ptr()), stride(table, 0), dims == 3 ? stride(table, 1) : 0,
             to_int(table.size(-1)), to_int(k.size(t)), to_int(k.size(0)), dims == 3};
  return p;
}

cowa_pattern pattern(PyObject* o) {
  static PyObject* names[7] = {};
  if (!names[0]) {
    const char* s[7] = {"S", "L", "T", "D", "kv_head_base", "h_kv_global", "softmax_scale"};
    for (int i = 6; i >= 0; --i) names[i] = PyUnicode_InternFromString(s[i]);
  }
  long v[6];
  for (int i = 0; i < 7; ++i) {
    PyObject* x = PyObject_GetAttr(o, names[i]);
    if (!x) throw Refused{nullptr, ""};
    if (i < 6) v[i] = PyLong_AsLong(x);
    const double f = i == 6 ? PyFloat_AsDouble(x) : 0.0;
    Py_DECREF(x);
    if (PyErr_Occurred()) throw Refused{nullptr, ""};
    if (i == 6) {
      for (long w : v)
        if (w > 0x7fffffffL || w < -0x80000000L) bad_value("a pattern parameter does not fit 32 bits");
      return {(int32_t)v[0], (int32_t)v[1], (int32_t)v[2], (int32_t)v[3], (int32_t)v[4], (int32_t)v[5], (float)f};
    }
  }
  return {};
}

// A cowa_rotary that cowa.py keeps: its address and the tensor of its frequencies; None for no rotation.
struct Rotary {
  const cowa_rotary* c = nullptr;
  const at::Tensor* freq = nullptr;
  int axes = 0;
};
Rotary rotary(PyObject* address, PyObject* freq) {
  Rotary r;
  if (address == Py_None) return r;
  r.c = reinterpret_cast<const cowa_rotary*>(PyLong_AsVoidPtr(address));
  if (!r.c) throw Refused{PyErr_Occurred() ? nullptr : PyExc_ValueError, "rope"};
  r.freq = &tensor(freq, "inv_freq");
  r.axes = r.c->n_axes;
  return r;
}

// A contiguous tensor on x's device, past the dispatcher (0.7 us less than at::empty_like)
at::Tensor fresh(const at::Tensor& x, at::IntArrayRef shape, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(shape, type, x.device(), std::nullopt));
}
at::Tensor fresh_like(const at::Tensor& x) { return fresh(x, x.sizes(), x.scalar_type()); }

void* stream_of(const at::Tensor& x) { return c10::cuda::getCurrentCUDAStream(x.get_device()).stream(); }

// (status, object, ...): the object given, or the tensor made in its place
PyObject* given_or(PyObject* given, const at::Tensor& made) {
  if (given != Py_None || !made.defined()) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(made);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) bad_type("wrong number of arguments");
    return f();
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    // torch.OutOfMemoryError, whose C++ symbol libtorch_python does not export
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// use(handle of the loaded library)
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    void* h = PyLong_AsVoidPtr(a[0]);
    auto get = [&](const char* name) {
      void* f = dlsym(h, name);
      if (!f) throw Refused{PyExc_RuntimeError, std::string(name) + " is not in the library"};
      return f;
    };
#define COWA_GET(field, name) lib.field = reinterpret_cast<decltype(lib.field)>(get(#name))
    COWA_GET(rope, cowa_rope);
    COWA_GET(rope_bwd, cowa_rope_bwd);
    COWA_GET(append, cowa_paged_append);
    COWA_GET(append_fp8, cowa_paged_append_fp8);
    COWA_GET(decode, cowa_decode_paged);
    COWA_GET(decode_fp8, cowa_decode_paged_fp8);
    COWA_GET(decode_size, cowa_decode_paged_workspace_size);
    COWA_GET(decode_fp8_size, cowa_decode_paged_fp8_workspace_size);
    COWA_GET(fwd, cowa_fwd_paged);
    COWA_GET(fwd_size, cowa_fwd_paged_workspace_size);
    Py_RETURN_NONE;
  });
}

// rope(backward, q, k, rotary, inv_freq, positions, q_out, k_out) -> (status, q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor *q = tensor_or_none(a[1], "q"), *k = tensor_or_none(a[2], "k");
    if (!q && !k) bad_value("q or k is needed");
    const at::Tensor& x = q ? *q : *k;
    for (const at::Tensor* t : {q, k})
      if (t) {
        bf16(*t, t == q ? "q" : "k");
        if (t->dim() != 4 || t->size(0) != x.size(0) || t->size(1) != x.size(1) || t->size(3) != x.size(3))
          bad_value("q and k are [B, N, H, d] with the same B, N and d");
      }
    const Rotary r = rotary(a[3], a[4]);
    if (!r.c) bad_type("a Rope is needed");
    const at::Tensor *pos = tensor_or_none(a[5], "positions"), *qo = tensor_or_none(a[6], "q_out"),
                     *ko = tensor_or_none(a[7], "k_out");
    if ((qo && !q) || (ko && !k)) bad_value("an output without its input");
    if (qo) { bf16(*qo, "q_out"); of_shape(*qo, "q_out", q->sizes()); }
    if (ko) { bf16(*ko, "k_out"); of_shape(*ko, "k_out", k->sizes()); }
    const int64_t B = x.size(0), N = x.size(1);
    const int32_t* p = nullptr;
    int64_t sa = 0, sb = 0;
    if (pos) {
      if (pos->dim() == 2 && r.axes == 1) {
        p = int32(*pos, "positions", {B, N});
        sb = pos->stride(0);
      } else {
        p = int32(*pos, "positions", {r.axes, B, N});
        sa = pos->stride(0);
        sb = pos->stride(1);
      }
    }
    same_device(x, {k, pos, qo, ko, r.freq});
    const c10::cuda::CUDAGuard guard(x.device());
    at::Tensor mq, mk;
    if (q && !qo) qo = &(mq = fresh_like(*q));
    if (k && !ko) ko = &(mk = fresh_like(*k));
    const cowa_tensor none{nullptr, 0, 0, 0};
    const int status = (PyObject_IsTrue(a[0]) ? lib.rope_bwd : lib.rope)(
        r.c, to_int(B), to_int(N), q ? to_int(q->size(2)) : 0, k ? to_int(k->size(2)) : 0, to_int(x.size(3)),
        q ? rows(*q, "q") : none, k ? rows(*k, "k") : none, qo ? rows(*qo, "q_out") : none, ko ? rows(*ko, "k_out") : none,
        p, sa, sb, stream_of(x));
    return Py_BuildValue("(iNN)", status, given_or(a[6], mq), given_or(a[7], mk));
  });
}

// append(q, k, v, pos, k_pages, v_pages, page_table, rotary, inv_freq, seq, rope_pos, q_out, layout, scales)
// -> (status, q_out); scales: None, or (k_scale, v_scale) of E4M3 pages
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor* q = tensor_or_none(a[0], "q");
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &pos = tensor(a[3], "pos");
    const at::Tensor &kp = tensor(a[4], "k_pages"), &vp = tensor(a[5], "v_pages"), &tab = tensor(a[6], "page_table");
    bf16(k, "k");
    bf16(v, "v");
    if (k.dim() != 3) bad_value("k and v are [total, H_kv, d]");
    of_shape(v, "v", k.sizes());
    const int64_t total = k.size(0), Hkv = k.size(1), d = k.size(2);
    if (q) {
      bf16(*q, "q");
      if (q->dim() != 3 || q->size(0) != total || q->size(2) != d) bad_value("q is [total, H_q, d]");
    }
    const Rotary r = rotary(a[7], a[8]);
    const at::Tensor *seq = tensor_or_none(a[9], "seq"), *rp = tensor_or_none(a[10], "rope_pos"),
                     *qo = tensor_or_none(a[11], "q_out");
    if (qo) {
      if (!q) bad_value("q_out without q");
      bf16(*qo, "q_out");
      of_shape(*qo, "q_out", q->sizes());
    }
    const int32_t* pos_p = int32(pos, "pos", {total});
    const int32_t* seq_p = seq ? int32(*seq, "seq", {total}) : nullptr;
    const int32_t* rp_p = nullptr;
    int64_t rs = 0;
    if (rp) {
      if (!r.c) bad_value("rope_pos without rope");
      if (rp->dim() == 1 && r.axes == 1) {
        rp_p = int32(*rp, "rope_pos", {total});
      } else {
        rp_p = int32(*rp, "rope_pos", {r.axes, total});
        rs = rp->stride(0);
      }
    }
    const bool codes = a[13] != Py_None;
    const Pages p = pages(kp, vp, tab, a[12], d, codes);
    if (p.Hkv != Hkv) bad_value("the pages do not hold the KV heads of k");
    same_device(k, {q, &v, &pos, seq, rp, qo, &kp, &vp, &tab, r.freq});
    const c10::cuda::CUDAGuard guard(k.device());
    at::Tensor made;
    if (q && !qo) qo = &(made = fresh_like(*q));
    const cowa_tensor none{nullptr, 0, 0, 0}, qt = q ? rows(*q, "q") : none, qot = qo ? rows(*qo, "q_out") : none;
    const int Hq = q ? to_int(q->size(1)) : 0;
    int status;
    if (codes)
      status = lib.append_fp8(r.c, to_int(total), p.n_seq, Hq, p.Hkv, to_int(d), qt, rows(k, "k"), rows(v, "v"), qot, pos_p,
                              seq_p, rp_p, rs, p.k, p.v, (float)number(PyTuple_GetItem(a[13], 0)),
                              (float)number(PyTuple_GetItem(a[13], 1)), p.table, stream_of(k));
    else
      status = lib.append(r.c, to_int(total), p.n_seq, Hq, p.Hkv, to_int(d), qt, rows(k, "k"), rows(v, "v"), qot, pos_p,
                          seq_p, rp_p, rs, p.k, p.v, p.table, stream_of(k));
    return Py_BuildValue("(iN)", status, given_or(a[11], made));
  });
}

// The caller's lse, or none; float32 and contiguous
void check_lse(const at::Tensor* lse, at::IntArrayRef shape) {
  if (!lse) return;
  if (lse->scalar_type() != at::kFloat || lse->sizes() != shape || !lse->is_contiguous())
    bad_value("lse must be a contiguous float32 tensor of the shape of the rows");
}

// The caller's workspace, or none: one piece of memory, so that its size is what the kernels may use
void check_workspace(const at::Tensor* ws) {
  if (ws && !ws->is_contiguous()) bad_value("workspace must be a contiguous tensor");
}

// decode(q_t, k_pages, v_pages, page_table, pos, pattern, scales, layout, out, lse, workspace, want_lse)
// -> (status, out, lse)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q_t"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
    const at::Tensor &tab = tensor(a[3], "page_table"), &pos = tensor(a[4], "pos");
    bf16(q, "q_t");
    if (q.dim() != 3 || !q.is_contiguous()) bad_value("q_t must be contiguous [B, H_q, d]");
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2);
    const bool codes = a[6] != Py_None;
    const Pages p = pages(kp, vp, tab, a[7], d, codes);
    if (p.n_seq != B) bad_value("page_table must have one row per sequence");
    const int32_t* pos_p = int32(pos, "pos", {B});
    const cowa_pattern pat = pattern(a[5]);
    const at::Tensor *out = tensor_or_none(a[8], "out"), *lse = tensor_or_none(a[9], "lse"),
                     *ws = tensor_or_none(a[10], "workspace");
    if (out) {
      bf16(*out, "out");
      if (out->sizes() != q.sizes() || !out->is_contiguous()) bad_value("out must be contiguous [B, H_q, d]");
    }
    check_lse(lse, {B, Hq});
    check_workspace(ws);
    same_device(q, {&kp, &vp, &tab, &pos, out, lse, ws});
    const c10::cuda::CUDAGuard guard(q.device());
    at::Tensor mo, ml, mw;
    if (!out) out = &(mo = fresh_like(q));
    if (!lse && PyObject_IsTrue(a[11])) lse = &(ml = fresh(q, {B, Hq}, at::kFloat));
    const int b = to_int(B), hq = to_int(Hq), di = to_int(d);
    if (!ws) {
      const size_t bytes = (codes ? lib.decode_fp8_size : lib.decode_size)(&pat, b, hq, p.Hkv, di, p.table.max_pages,
                                                                          p.table.page_size);
      ws = &(mw = at::zeros({(int64_t)std::max<size_t>(256, bytes)}, q.options().dtype(at::kByte)));
    }
    float* lse_p = lse ? static_cast<float*>(lse->data_ptr()) : nullptr;
    int status;
    if (codes)
      status = lib.decode_fp8(&pat, b, hq, p.Hkv, di, q.data_ptr(), p.k, p.v, (float)number(PyTuple_GetItem(a[6], 0)),
                              (float)number(PyTuple_GetItem(a[6], 1)), p.table, pos_p, out->data_ptr(), lse_p,
                              ws->data_ptr(), ws->nbytes(), stream_of(q));
    else
      status = lib.decode(&pat, b, hq, p.Hkv, di, q.data_ptr(), p.k, p.v, p.table, pos_p, out->data_ptr(), lse_p,
                          ws->data_ptr(), ws->nbytes(), stream_of(q));
    return Py_BuildValue("(iNN)", status, given_or(a[8], mo), given_or(a[9], ml));
  });
}

// fwd(q, k_pages, v_pages, page_table, cu_seqlens, q_start, pattern, layout, out, lse, workspace)
// -> (status, out, lse)
PyObject* fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
    const at::Tensor &tab = tensor(a[3], "page_table"), &cu = tensor(a[4], "cu_seqlens"), &start = tensor(a[5], "q_start");
    bf16(q, "q");
    if (q.dim() != 3) bad_value("q is [total, H_q, d]");
    const int64_t total = q.size(0), Hq = q.size(1), d = q.size(2);
    const Pages p = pages(kp, vp, tab, a[7], d, false);
    const int32_t *cu_p = int32(cu, "cu_seqlens", {p.n_seq + 1L}), *start_p = int32(start, "q_start", {p.n_seq});
    const cowa_pattern pat = pattern(a[6]);
    const at::Tensor *out = tensor_or_none(a[8], "out"), *lse = tensor_or_none(a[9], "lse"),
                     *ws = tensor_or_none(a[10], "workspace");
    if (out) { bf16(*out, "out"); of_shape(*out, "out", q.sizes()); }
    check_lse(lse, {Hq, total});
    check_workspace(ws);
    same_device(q, {&kp, &vp, &tab, &cu, &start, out, lse, ws});
    const c10::cuda::CUDAGuard guard(q.device());
    at::Tensor mo, ml, mw;
    if (!out) out = &(mo = fresh_like(q));
    if (!lse) lse = &(ml = fresh(q, {Hq, total}, at::kFloat));
    const int t = to_int(total), hq = to_int(Hq), di = to_int(d);
    if (!ws) {
      const size_t bytes = lib.fwd_size(&pat, p.n_seq, t, hq, p.Hkv, di, p.table.max_pages, p.table.page_size);
      ws = &(mw = at::zeros({(int64_t)std::max<size_t>(256, bytes)}, q.options().dtype(at::kByte)));
    }
    const int status = lib.fwd(&pat, p.n_seq, t, hq, p.Hkv, di, cu_p, start_p, rows(q, "q"), p.k, p.v, p.table,
                               rows(*out, "out"), static_cast<float*>(lse->data_ptr()), ws->data_ptr(), ws->nbytes(),
                               stream_of(q));
    return Py_BuildValue("(iNN)", status, given_or(a[8], mo), given_or(a[9], ml));
  });
}

#define COWA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {COWA_METHOD(use),    COWA_METHOD(rope), COWA_METHOD(append),
                         COWA_METHOD(decode), COWA_METHOD(fwd),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
