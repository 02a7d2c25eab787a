// Python binding of the calls that are made once per layer and step: cb_rope_append,
// cb_shared_prefix_attention, cb_rope_append_attention, cb_scored_attention and the calls on the
// quantised cache, on torch tensors.
//
// It checks the tensors, makes the outputs and the workspace that the caller left out, and calls the
// C ABI on the current stream.  A call on a few tokens is a few microseconds of GPU work, and through
// ctypes its checks alone took longer: cb_rope_append on one token 17.7 us of host time in all, here
// 4.2 us (a GB300's Grace host).  Arguments that fail a check come back as
// NotImplemented, a refusal of the library as its status; the Python side makes the errors.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "../../include/cb.h"

namespace {

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// Contiguous, of the type and number of dimensions, on CUDA device dev.
bool plain(const at::Tensor* t, at::ScalarType type, int64_t dim, int dev) {
  return t != nullptr && t->scalar_type() == type && t->dim() == dim && t->is_cuda() &&
         t->get_device() == dev && t->is_contiguous();
}

// bf16 [T, H, D] with contiguous token rows (a view of a wider projection's output, for instance)
// that do not overlap (as a broadcast row's would).
bool rows(const at::Tensor* t, int dev) {
  if (t == nullptr || t->scalar_type() != at::kBFloat16 || t->dim() != 3 || !t->is_cuda() ||
      t->get_device() != dev)
    return false;
  return t->size(0) == 0 ||
         (t->stride(2) == 1 && (t->stride(1) == t->size(2) || t->size(1) == 1) &&
          (t->size(0) == 1 || t->stride(0) >= t->size(1) * t->size(2)));
}

// The row stride that the library is given: 0 (contiguous) for one token, whatever its stride says.
int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : 0; }

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (at::DeviceIndex)dev), std::nullopt);
}

bool fits(int64_t x) { return x <= INT_MAX; }

// An integer (Python's, numpy's, ...) that fits 32 bits; no error is left pending where it is none.
bool read_int(PyObject* o, int32_t* x) {
  long v = -1;
  if (PyLong_Check(o)) {
    v = PyLong_AsLong(o);
  } else if (PyObject* i = PyNumber_Index(o)) {
    v = PyLong_AsLong(i);
    Py_DECREF(i);
  }
  if (v == -1 && PyErr_Occurred()) {  // no integer, or beyond a long
    PyErr_Clear();
    return false;
  }
  *x = (int32_t)v;
  return v == *x;
}

struct Step {
  cb_dims dims;
  int dev;
  int32_t block_size;
  const at::Tensor *k_pages, *v_pages, *block_table, *cu, *kv;
};

// Pools and metadata (args: k_pages, v_pages, block_table, cu_seqlens_q, kv_lens, block_size).
bool read_step(PyObject* const* args, int dev, Step* s, at::ScalarType type = at::kBFloat16) {
  const at::Tensor* t[5];
  for (int i = 0; i < 5; ++i) t[i] = tensor(args[i]);
  if (dev != c10::cuda::current_device() || !plain(t[0], type, 4, dev) ||
      !plain(t[1], type, 4, dev) || !plain(t[2], at::kInt, 2, dev) ||
      !plain(t[3], at::kInt, t[3] ? t[3]->dim() : 0, dev) ||
      !plain(t[4], at::kInt, t[4] ? t[4]->dim() : 0, dev) || !read_int(args[5], &s->block_size))
    return false;
  const int64_t S = t[4]->numel();
  if (t[3]->numel() != S + 1 || t[2]->size(0) != S || t[0]->sizes() != t[1]->sizes() ||
      t[0]->size(1) != s->block_size || !fits(S) || !fits(t[0]->size(0)) || !fits(t[2]->size(1)))
    return false;
  s->dev = dev;
  s->k_pages = t[0];
  s->v_pages = t[1];
  s->block_table = t[2];
  s->cu = t[3];
  s->kv = t[4];
  s->dims.num_seqs = (int32_t)S;
  s->dims.num_kv_heads = (int32_t)t[0]->size(2);
  s->dims.head_dim = (int32_t)t[0]->size(3);
  s->dims.num_pages = (int32_t)t[0]->size(0);
  s->dims.max_blocks_per_seq = (int32_t)t[2]->size(1);
  return true;
}

// The rotary append's inputs (q may be nullptr) and cb_rope; completes s->dims.  optional: cos_sin may
// be None (nothing is rotated).
bool read_rope(const at::Tensor* q, const at::Tensor* k, const at::Tensor* v, PyObject* cos_sin,
               PyObject* interleaved, Step* s, cb_rope* r, bool optional = false) {
  const at::Tensor* cs = tensor(cos_sin);
  const bool rotates = !optional || cos_sin != Py_None;
  if (!rows(k, s->dev) || !rows(v, s->dev) || (rotates && !plain(cs, at::kFloat, 2, s->dev)) ||
      k->sizes() != v->sizes() || k->size(1) != s->dims.num_kv_heads ||
      k->size(2) != s->dims.head_dim || !fits(k->size(0)) ||
      (rotates && (!fits(cs->size(0)) || !fits(cs->size(1)))))
    return false;
  s->dims.num_tokens = (int32_t)k->size(0);
  s->dims.num_q_heads = s->dims.num_kv_heads;
  if (q != nullptr) {
    if (!rows(q, s->dev) || q->size(0) != k->size(0) || q->size(2) != k->size(2) || !fits(q->size(1)))
      return false;
    s->dims.num_q_heads = (int32_t)q->size(1);
  }
  const int on = PyObject_IsTrue(interleaved);
  if (on < 0) {
    PyErr_Clear();
    return false;
  }
  *r = cb_rope{};
  if (rotates) {
    r->cos_sin = static_cast<const float*>(cs->data_ptr());
    r->max_positions = (int32_t)cs->size(0);
    r->rot_dim = (int32_t)cs->size(1);
    r->interleaved = on;
  }
  r->q_stride = q != nullptr ? row_stride(*q) : 0;
  r->k_stride = row_stride(*k);
  r->v_stride = row_stride(*v);
  return true;
}

// A bf16 output of `shape`: the caller's, or a new one.
bool output(PyObject* o, at::IntArrayRef shape, int dev, at::Tensor* out) {
  if (o == Py_None) {
    *out = empty(shape, at::kBFloat16, dev);
    return true;
  }
  const at::Tensor* t = tensor(o);
  if (!plain(t, at::kBFloat16, (int64_t)shape.size(), dev) || t->sizes() != shape) return false;
  *out = *t;
  return true;
}

int32_t* i32(const at::Tensor* t) { return static_cast<int32_t*>(t->data_ptr()); }

PyObject* status(cb_status st) { return PyLong_FromLong((long)st); }

PyObject* not_implemented() { Py_RETURN_NOTIMPLEMENTED; }

// rope_append(k_pages, v_pages, block_table, cu_seqlens_q, kv_lens, block_size, q, k_new, v_new,
//             cos_sin, interleaved, q_out) -> q_out (None without q), status or NotImplemented
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) return not_implemented();
  const at::Tensor *q = tensor(args[6]), *k = tensor(args[7]), *v = tensor(args[8]);
  if ((q == nullptr && args[6] != Py_None) || k == nullptr || !k->is_cuda()) return not_implemented();
  Step s;
  cb_rope r;
  at::Tensor out;
  if (!read_step(args, k->get_device(), &s) || !read_rope(q, k, v, args[9], args[10], &s, &r))
    return not_implemented();
  if (q != nullptr ? !output(args[11], q->sizes(), s.dev, &out) : args[11] != Py_None)
    return not_implemented();
  const cb_status st = cb_rope_append(
      q != nullptr ? q->data_ptr() : nullptr, k->data_ptr(), v->data_ptr(),
      q != nullptr ? out.data_ptr() : nullptr, s.k_pages->data_ptr(), s.v_pages->data_ptr(),
      i32(s.block_table), i32(s.cu), i32(s.kv), s.block_size, &r, &s.dims,
      c10::cuda::getCurrentCUDAStream().stream());
  if (st != CB_OK) return status(st);
  if (q == nullptr) Py_RETURN_NONE;
  if (args[11] != Py_None) return Py_NewRef(args[11]);
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// What the attention calls take beside their inputs (args: prefix_group, prefix_lens, out, lse,
// workspace, decode_ctas, serial, window, phase_events).
struct Tail {
  cb_prefix prefix = {};
  bool grouped = false;
  at::Tensor out, lse, ws;
  cb_options options = {};
  void* events[CB_NUM_PHASE_EVENTS];
};

bool read_tail(PyObject* const* args, const at::Tensor& q, const Step& s, Tail* t) {
  const int dev = s.dev;
  t->grouped = args[0] != Py_None || args[1] != Py_None;
  if (t->grouped) {
    const at::Tensor *g = tensor(args[0]), *l = tensor(args[1]);
    if (!plain(g, at::kInt, g ? g->dim() : 0, dev) || !plain(l, at::kInt, l ? l->dim() : 0, dev) ||
        g->numel() != s.dims.num_seqs || !fits(l->numel()))
      return false;
    t->prefix.prefix_group = i32(g);
    t->prefix.prefix_lens = i32(l);
    t->prefix.num_groups = (int32_t)l->numel();
  }
  if (!output(args[2], q.sizes(), dev, &t->out)) return false;
  if (args[3] == Py_True) {
    t->lse = empty(q.sizes().slice(0, 2), at::kFloat, dev);
  } else if (args[3] != Py_None && args[3] != Py_False) {
    const at::Tensor* l = tensor(args[3]);
    if (!plain(l, at::kFloat, 2, dev) || l->sizes() != q.sizes().slice(0, 2)) return false;
    t->lse = *l;
  }
  if (args[4] == Py_None) {
    const int64_t need = (int64_t)cb_prefix_workspace_size(&s.dims, t->prefix.num_groups);
    t->ws = empty({need > 256 ? need : 256}, at::kByte, dev);
  } else {
    const at::Tensor* w = tensor(args[4]);
    if (!plain(w, at::kByte, w ? w->dim() : 0, dev)) return false;
    t->ws = *w;
  }
  if (!read_int(args[5], &t->options.decode_ctas) || !read_int(args[7], &t->options.window)) return false;
  const int serial = PyObject_IsTrue(args[6]);
  if (serial < 0) {
    PyErr_Clear();
    return false;
  }
  t->options.flags = serial ? CB_OPT_SERIAL : 0;
  if (args[8] != Py_None) {  // a tuple of event handles, made by the Python side
    if (!PyTuple_Check(args[8]) || PyTuple_GET_SIZE(args[8]) != CB_NUM_PHASE_EVENTS) return false;
    for (int i = 0; i < CB_NUM_PHASE_EVENTS; ++i)
      t->events[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[8], i));
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    t->options.phase_events = t->events;
  }
  return true;
}

// out, or (out, lse): the caller's objects where given.
PyObject* result(PyObject* const* args, Tail& t) {
  PyObject* out = args[2] != Py_None ? Py_NewRef(args[2]) : THPVariable_Wrap(std::move(t.out));
  if (out == nullptr || args[3] == Py_None || args[3] == Py_False) return out;
  PyObject* lse = args[3] != Py_True ? Py_NewRef(args[3]) : THPVariable_Wrap(std::move(t.lse));
  if (lse == nullptr) {
    Py_DECREF(out);
    return nullptr;
  }
  PyObject* both = PyTuple_Pack(2, out, lse);
  Py_DECREF(out);
  Py_DECREF(lse);
  return both;
}

// shared_prefix_attention(k_pages, v_pages, block_table, cu_seqlens_q, kv_lens, block_size, q, scale,
//                         <Tail's arguments>) -> out or (out, lse), status or NotImplemented
PyObject* shared_prefix_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 17) return not_implemented();
  const at::Tensor* q = tensor(args[6]);
  if (q == nullptr || !q->is_cuda()) return not_implemented();
  Step s;
  if (!read_step(args, q->get_device(), &s) || !plain(q, at::kBFloat16, 3, s.dev) ||
      q->size(2) != s.dims.head_dim || !fits(q->size(0)) || !fits(q->size(1)))
    return not_implemented();
  s.dims.num_tokens = (int32_t)q->size(0);
  s.dims.num_q_heads = (int32_t)q->size(1);
  const double scale = PyFloat_AsDouble(args[7]);
  if (PyErr_Occurred()) return nullptr;
  Tail t;
  if (!read_tail(args + 8, *q, s, &t) || !t.grouped) return not_implemented();
  const cb_status st = cb_shared_prefix_attention(
      q->data_ptr(), s.k_pages->data_ptr(), s.v_pages->data_ptr(), i32(s.block_table), i32(s.cu),
      i32(s.kv), s.block_size, (float)scale, &t.prefix, t.out.data_ptr(),
      t.lse.defined() ? static_cast<float*>(t.lse.data_ptr()) : nullptr, t.ws.data_ptr(),
      (size_t)t.ws.numel(), &s.dims, &t.options, c10::cuda::getCurrentCUDAStream().stream());
  return st != CB_OK ? status(st) : result(args + 8, t);
  END_HANDLE_TH_ERRORS
}

// rope_append_attention(k_pages, v_pages, block_table, cu_seqlens_q, kv_lens, block_size, q, k_new,
//                       v_new, cos_sin, interleaved, q_out, scale, <Tail's arguments>)
PyObject* rope_append_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 22) return not_implemented();
  const at::Tensor *q = tensor(args[6]), *k = tensor(args[7]), *v = tensor(args[8]);
  if (q == nullptr || k == nullptr || !k->is_cuda()) return not_implemented();
  Step s;
  cb_rope r;
  at::Tensor q_out;
  if (!read_step(args, k->get_device(), &s) || !read_rope(q, k, v, args[9], args[10], &s, &r) ||
      !output(args[11], q->sizes(), s.dev, &q_out))
    return not_implemented();
  const double scale = PyFloat_AsDouble(args[12]);
  if (PyErr_Occurred()) return nullptr;
  Tail t;
  if (!read_tail(args + 13, q_out, s, &t)) return not_implemented();
  const cb_status st = cb_rope_append_attention(
      q->data_ptr(), k->data_ptr(), v->data_ptr(), q_out.data_ptr(), s.k_pages->data_ptr(),
      s.v_pages->data_ptr(), i32(s.block_table), i32(s.cu), i32(s.kv), s.block_size, (float)scale, &r,
      t.grouped ? &t.prefix : nullptr, t.out.data_ptr(),
      t.lse.defined() ? static_cast<float*>(t.lse.data_ptr()) : nullptr, t.ws.data_ptr(),
      (size_t)t.ws.numel(), &s.dims, &t.options, c10::cuda::getCurrentCUDAStream().stream());
  return st != CB_OK ? status(st) : result(args + 13, t);
  END_HANDLE_TH_ERRORS
}

// The quantised cache's scales, [P, block_size, Hkv, 2].
bool read_scales(PyObject* o, const Step& s, const at::Tensor** out) {
  const at::Tensor* t = tensor(o);
  if (!plain(t, at::kByte, 4, s.dev) || t->sizes().slice(0, 3) != s.k_pages->sizes().slice(0, 3) ||
      t->size(3) != 2)
    return false;
  *out = t;
  return true;
}

// quant_append(k_pages, v_pages, block_table, cu_seqlens_q, kv_lens, block_size, kv_scales, q, k_new,
//              v_new, cos_sin, interleaved, q_out) -> q_out (None without q), status or NotImplemented
PyObject* quant_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13) return not_implemented();
  const at::Tensor *q = tensor(args[7]), *k = tensor(args[8]), *v = tensor(args[9]), *sc;
  if ((q == nullptr && args[7] != Py_None) || k == nullptr || !k->is_cuda()) return not_implemented();
  Step s;
  cb_rope r;
  at::Tensor out;
  if (!read_step(args, k->get_device(), &s, at::kFloat8_e4m3fn) || !read_scales(args[6], s, &sc) ||
      !read_rope(q, k, v, args[10], args[11], &s, &r, true))
    return not_implemented();
  if (q != nullptr ? !output(args[12], q->sizes(), s.dev, &out) : args[12] != Py_None)
    return not_implemented();
  const cb_status st = cb_quant_append(
      q != nullptr ? q->data_ptr() : nullptr, k->data_ptr(), v->data_ptr(),
      q != nullptr ? out.data_ptr() : nullptr, s.k_pages->data_ptr(), s.v_pages->data_ptr(),
      sc->data_ptr(), i32(s.block_table), i32(s.cu), i32(s.kv), s.block_size, &r, &s.dims,
      c10::cuda::getCurrentCUDAStream().stream());
  if (st != CB_OK) return status(st);
  if (q == nullptr) Py_RETURN_NONE;
  if (args[12] != Py_None) return Py_NewRef(args[12]);
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// quant_gather(k_pages, v_pages, block_table, cu_seqlens_k, block_size, kv_scales, key_starts, num_rows,
//              k_out, v_out) -> (k_out, v_out), status or NotImplemented
PyObject* quant_gather(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) return not_implemented();
  const at::Tensor *k = tensor(args[0]), *table = tensor(args[2]), *sc;
  if (k == nullptr || !k->is_cuda() || table == nullptr || table->dim() != 2) return not_implemented();
  const int dev = k->get_device();
  Step s;
  const at::Tensor *v = tensor(args[1]), *cu = tensor(args[3]), *starts = tensor(args[6]);
  int32_t rows;
  if (dev != c10::cuda::current_device() || !plain(k, at::kFloat8_e4m3fn, 4, dev) ||
      !plain(v, at::kFloat8_e4m3fn, 4, dev) || !plain(table, at::kInt, 2, dev) ||
      !plain(cu, at::kInt, cu ? cu->dim() : 0, dev) || k->sizes() != v->sizes() ||
      !read_int(args[4], &s.block_size) || !read_int(args[7], &rows) || rows < 0)
    return not_implemented();
  const int64_t S = table->size(0);
  if (cu->numel() != S + 1 || k->size(1) != s.block_size || !fits(S) || !fits(k->size(0)) ||
      !fits(table->size(1)))
    return not_implemented();
  if (args[6] != Py_None && (!plain(starts, at::kInt, starts ? starts->dim() : 0, dev) || starts->numel() != S))
    return not_implemented();
  s.dev = dev;
  s.k_pages = k;
  s.dims = cb_dims{(int32_t)S, rows, (int32_t)k->size(2), (int32_t)k->size(2), (int32_t)k->size(3),
                   (int32_t)k->size(0), (int32_t)table->size(1)};
  at::Tensor ko, vo;
  const int64_t shape[3] = {rows, k->size(2), k->size(3)};
  if (!read_scales(args[5], s, &sc) || !output(args[8], shape, dev, &ko) || !output(args[9], shape, dev, &vo))
    return not_implemented();
  const cb_status st = cb_quant_gather(
      k->data_ptr(), v->data_ptr(), sc->data_ptr(), i32(table), i32(cu),
      args[6] != Py_None ? i32(starts) : nullptr, s.block_size, ko.data_ptr(), vo.data_ptr(), &s.dims,
      c10::cuda::getCurrentCUDAStream().stream());
  if (st != CB_OK) return status(st);
  PyObject* a = args[8] != Py_None ? Py_NewRef(args[8]) : THPVariable_Wrap(std::move(ko));
  PyObject* b = args[9] != Py_None ? Py_NewRef(args[9]) : THPVariable_Wrap(std::move(vo));
  PyObject* both = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return both;
  END_HANDLE_TH_ERRORS
}

// Changed scores (args: softcap, slopes, visible_lens).
bool read_score(PyObject* const* args, const Step& s, cb_score* out) {
  *out = cb_score{};
  const double cap = PyFloat_AsDouble(args[0]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  out->softcap = (float)cap;
  if (cap != 0 && out->softcap == 0.f) return false;  // (0 is no cap)
  if (args[1] != Py_None) {
    const at::Tensor* t = tensor(args[1]);
    if (!plain(t, at::kFloat, 1, s.dev) || t->numel() != s.dims.num_q_heads) return false;
    out->slopes = static_cast<const float*>(t->data_ptr());
  }
  if (args[2] != Py_None) {
    const at::Tensor* t = tensor(args[2]);
    if (!plain(t, at::kInt, 1, s.dev) || t->numel() != s.dims.num_seqs) return false;
    out->visible_lens = i32(t);
  }
  return true;
}

// scored_attention(k_pages, v_pages, block_table, cu_seqlens_q, kv_lens, block_size, kv_scales, q, scale,
//                  softcap, slopes, visible_lens, <Tail's arguments>) -> out or (out, lse), status or
// NotImplemented.  kv_scales: those of a quantised cache, or None (a bf16 cache).
PyObject* scored_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 21) return not_implemented();
  const at::Tensor *q = tensor(args[7]), *sc = nullptr;
  if (q == nullptr || !q->is_cuda()) return not_implemented();
  Step s;
  const bool quant = args[6] != Py_None;
  if (!read_step(args, q->get_device(), &s, quant ? at::kFloat8_e4m3fn : at::kBFloat16) ||
      (quant && !read_scales(args[6], s, &sc)) || !plain(q, at::kBFloat16, 3, s.dev) ||
      q->size(2) != s.dims.head_dim || !fits(q->size(0)) || !fits(q->size(1)))
    return not_implemented();
  s.dims.num_tokens = (int32_t)q->size(0);
  s.dims.num_q_heads = (int32_t)q->size(1);
  const double scale = PyFloat_AsDouble(args[8]);
  if (PyErr_Occurred()) return nullptr;
  cb_score score;
  Tail t;
  if (!read_score(args + 9, s, &score) || !read_tail(args + 12, *q, s, &t) || t.grouped)
    return not_implemented();
  float* lse = t.lse.defined() ? static_cast<float*>(t.lse.data_ptr()) : nullptr;
  void* stream = c10::cuda::getCurrentCUDAStream().stream();
  const cb_status st =
      quant ? cb_quant_attention(q->data_ptr(), s.k_pages->data_ptr(), s.v_pages->data_ptr(),
                                 sc->data_ptr(), i32(s.block_table), i32(s.cu), i32(s.kv), s.block_size,
                                 (float)scale, &score, t.out.data_ptr(), lse, t.ws.data_ptr(),
                                 (size_t)t.ws.numel(), &s.dims, &t.options, stream)
            : cb_scored_attention(q->data_ptr(), s.k_pages->data_ptr(), s.v_pages->data_ptr(),
                                  i32(s.block_table), i32(s.cu), i32(s.kv), s.block_size, (float)scale,
                                  &score, t.out.data_ptr(), lse, t.ws.data_ptr(), (size_t)t.ws.numel(),
                                  &s.dims, &t.options, stream);
  return st != CB_OK ? status(st) : result(args + 12, t);
  END_HANDLE_TH_ERRORS
}

// quant_append_attention(k_pages, v_pages, block_table, cu_seqlens_q, kv_lens, block_size, kv_scales, q,
//                        k_new, v_new, cos_sin, interleaved, q_out, scale, softcap, slopes, visible_lens,
//                        <Tail's arguments>)
PyObject* quant_append_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 26) return not_implemented();
  const at::Tensor *q = tensor(args[7]), *k = tensor(args[8]), *v = tensor(args[9]), *sc;
  if (q == nullptr || k == nullptr || !k->is_cuda()) return not_implemented();
  Step s;
  cb_rope r;
  at::Tensor q_out;
  const bool rotates = args[10] != Py_None;
  if (!read_step(args, k->get_device(), &s, at::kFloat8_e4m3fn) || !read_scales(args[6], s, &sc) ||
      !read_rope(q, k, v, args[10], args[11], &s, &r, true) ||
      (rotates ? !output(args[12], q->sizes(), s.dev, &q_out)
               : args[12] != Py_None || !q->is_contiguous()))
    return not_implemented();
  if (!rotates) r.q_stride = 0;
  const double scale = PyFloat_AsDouble(args[13]);
  if (PyErr_Occurred()) return nullptr;
  cb_score score;
  Tail t;
  if (!read_score(args + 14, s, &score) || !read_tail(args + 17, *q, s, &t) || t.grouped)
    return not_implemented();
  const cb_status st = cb_quant_append_attention(
      q->data_ptr(), k->data_ptr(), v->data_ptr(), rotates ? q_out.data_ptr() : nullptr,
      s.k_pages->data_ptr(), s.v_pages->data_ptr(), sc->data_ptr(), i32(s.block_table), i32(s.cu),
      i32(s.kv), s.block_size, (float)scale, &r, &score, t.out.data_ptr(),
      t.lse.defined() ? static_cast<float*>(t.lse.data_ptr()) : nullptr, t.ws.data_ptr(),
      (size_t)t.ws.numel(), &s.dims, &t.options, c10::cuda::getCurrentCUDAStream().stream());
  return st != CB_OK ? status(st) : result(args + 17, t);
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rope_append", (PyCFunction)(void (*)())rope_append, METH_FASTCALL, nullptr},
    {"shared_prefix_attention", (PyCFunction)(void (*)())shared_prefix_attention, METH_FASTCALL,
     nullptr},
    {"rope_append_attention", (PyCFunction)(void (*)())rope_append_attention, METH_FASTCALL, nullptr},
    {"quant_append", (PyCFunction)(void (*)())quant_append, METH_FASTCALL, nullptr},
    {"quant_gather", (PyCFunction)(void (*)())quant_gather, METH_FASTCALL, nullptr},
    {"scored_attention", (PyCFunction)(void (*)())scored_attention, METH_FASTCALL, nullptr},
    {"quant_append_attention", (PyCFunction)(void (*)())quant_append_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cb_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__cb_torch() { return PyModule_Create(&module); }
