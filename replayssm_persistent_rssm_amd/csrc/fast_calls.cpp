// fast_calls.cpp -- argument marshalling of the prompt-side operators for the
// common case, as a CPython extension of the binding.
//
// At their smallest these operators are a few microseconds of GPU work, as long as
// Python needs to read the attributes of their tensors.  Each function here
// takes the binding's arguments, checks that every tensor is contiguous, on the
// given device and of the expected dtype and shape, and makes the C call.  It returns True when the
// call was enqueued; on anything else (strided views, wrong arguments, a library error) it returns
// False, and the binding's Python code handles the call or names the error.  Nothing has been enqueued
// then, unless a later launch of a call that has several failed: the binding's call then starts over, and only
// the last launch of each writes what the caller sees.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "rssm_block_norm.h"
#include "rssm_linear_attention.h"
#include "rssm_paged_attention.h"

namespace {

struct NotCommon {};   // leaves a function towards `return False`

void need(bool ok) {
  if (!ok) throw NotCommon();
}

const at::Tensor& tensor(PyObject* o, int dev) {
  need(THPVariable_Check(o));
  const at::Tensor& t = THPVariable_Unpack(o);
  need(t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.is_contiguous());
  return t;
}

// Address of a contiguous tensor of this dtype and shape.
void* addr(PyObject* o, int dev, at::ScalarType st, std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, dev);
  need(t.scalar_type() == st && t.sizes() == at::IntArrayRef(shape));
  return t.data_ptr();
}

void* opt(PyObject* o, int dev, at::ScalarType st, std::initializer_list<int64_t> shape) {
  return o == Py_None ? nullptr : addr(o, dev, st, shape);
}

int32_t code_of(at::ScalarType st) {
  switch (st) {
    case at::kFloat: return RSSM_F32;
    case at::kBFloat16: return RSSM_BF16;
    case at::kHalf: return RSSM_F16;
    default: throw NotCommon();
  }
}

int64_t integer(PyObject* o) {
  need(PyLong_Check(o));
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotCommon();
  }
  return v;
}

int32_t i32(int64_t v) {
  need(v >= INT32_MIN && v <= INT32_MAX);
  return static_cast<int32_t>(v);
}

int32_t i32(PyObject* o) { return i32(integer(o)); }

float real(PyObject* o) {
  need(PyFloat_Check(o) || PyLong_Check(o));
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotCommon();
  }
  return static_cast<float>(v);
}

void* stream(PyObject* o) { return reinterpret_cast<void*>(static_cast<intptr_t>(integer(o))); }

// The caller's workspace, or a new one from torch's allocator, in the order of the current stream.
at::Tensor workspace(PyObject* given, int64_t bytes, int dev) {
  if (given != Py_None) return tensor(given, dev);
  if (bytes == 0) return at::Tensor();
  return at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(at::Device(at::kCUDA, dev)));
}

// Whether every tensor among the arguments is contiguous and on device a[0].  Asked first, so that views, the
// other ordinary case, do not pay for an exception (1 to 3 us) before the binding's Python code takes them.
bool plain(PyObject* const* a, Py_ssize_t n) {
  if (n < 2 || !PyLong_Check(a[0])) return false;
  int over = 0;
  const long dev = PyLong_AsLongAndOverflow(a[0], &over);
  for (Py_ssize_t i = 2; i < n; ++i) {
    if (!THPVariable_Check(a[i])) continue;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) return false;
  }
  return true;
}

template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, F f) {
  bool done = false;
  try {
    done = plain(a, n) && f();
  } catch (...) {
    if (PyErr_Occurred()) PyErr_Clear();
    done = false;
  }
  return PyBool_FromLong(done);
}

// (device, stream, step, state, A, x, B, C, dt, y, slots, seq_start, max_seq_len, load_state, D, dt_bias, z,
//  dt_softplus, pad_slot_id, workspace)
PyObject* linear_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 20);
    const int dev = i32(a[0]);
    const bool step = a[2] == Py_True;
    const at::Tensor &state = tensor(a[3], dev), &x = tensor(a[5], dev), &B = tensor(a[6], dev), &slots = tensor(a[10], dev);
    need(state.dim() == 4 && x.dim() == 3 && B.dim() == 3 && slots.dim() == 1);
    const int64_t S = state.size(0), H = state.size(1), dim = state.size(2), dstate = state.size(3);
    const int64_t N = x.size(0), G = B.size(1), R = slots.size(0);
    need(G >= 1 && H % G == 0);
    const at::ScalarType it = x.scalar_type();
    rssm_linear_attention_desc d{};
    d.num_seqs = i32(R);
    d.num_tokens = i32(N);
    d.num_heads = i32(H);
    d.heads_per_group = i32(H / G);
    d.dim = i32(dim);
    d.dstate = i32(dstate);
    d.num_slots = i32(S);
    d.pad_slot_id = i32(a[18]);
    d.max_seq_len = i32(a[12]);
    d.state_dtype = code_of(state.scalar_type());
    d.input_dtype = code_of(it);
    d.dt_softplus = a[8] != Py_None && PyObject_IsTrue(a[17]) == 1;
    d.state_slot_stride = H * dim * dstate;
    d.x_token_stride = d.z_token_stride = d.y_token_stride = H * dim;
    d.B_token_stride = d.C_token_stride = G * dstate;
    d.dt_token_stride = H;
    rssm_linear_attention_tables t{};
    t.state = state.data_ptr();
    t.A = static_cast<const float*>(addr(a[4], dev, at::kFloat, {H}));
    t.x = addr(a[5], dev, it, {N, H, dim});
    t.B = addr(a[6], dev, it, {N, G, dstate});
    t.C = addr(a[7], dev, it, {N, G, dstate});
    t.dt = static_cast<const float*>(opt(a[8], dev, at::kFloat, {N, H}));
    t.y = addr(a[9], dev, it, {N, H, dim});
    t.slots = static_cast<const int32_t*>(addr(a[10], dev, at::kInt, {R}));
    t.D = static_cast<const float*>(opt(a[14], dev, at::kFloat, {H}));
    t.dt_bias = static_cast<const float*>(opt(a[15], dev, at::kFloat, {H}));
    t.z = opt(a[16], dev, it, {N, H, dim});
    if (step) return rssm_linear_attention_step(&d, &t, stream(a[1])) == RSSM_OK;
    t.seq_start = static_cast<const int32_t*>(addr(a[11], dev, at::kInt, {R + 1}));
    t.load_state = static_cast<const int32_t*>(opt(a[13], dev, at::kInt, {R}));
    int64_t bytes = 0;
    need(rssm_linear_attention_workspace(&d, &bytes) == RSSM_OK);
    const at::Tensor ws = workspace(a[19], bytes, dev);
    if (ws.defined()) {
      t.workspace = ws.data_ptr();
      d.workspace_bytes = static_cast<int64_t>(ws.nbytes());
    }
    return rssm_linear_attention(&d, &t, stream(a[1])) == RSSM_OK;
  });
}

void caches(PyObject* k, PyObject* v, PyObject* table, PyObject* seq_start, PyObject* kv_len, int dev,
            rssm_paged_attention_desc* d, rssm_paged_attention_tables* t, at::ScalarType* st) {
  const at::Tensor& kc = tensor(k, dev);
  const at::Tensor& pt = tensor(table, dev);
  need(kc.dim() == 4 && pt.dim() == 2 && pt.scalar_type() == at::kInt);
  const int64_t P = kc.size(0), ps = kc.size(1), Hkv = kc.size(2), D = kc.size(3), S = pt.size(0), M = pt.size(1);
  *st = kc.scalar_type();
  d->num_seqs = i32(S);
  d->num_kv_heads = i32(Hkv);
  d->head_dim = i32(D);
  d->page_size = i32(ps);
  d->num_pages = i32(P);
  d->max_pages = i32(M);
  d->dtype = code_of(*st);
  d->page_stride = ps * Hkv * D;
  d->row_stride = Hkv * D;
  d->head_stride = D;
  d->table_stride = M;
  t->k_cache = kc.data_ptr();
  t->v_cache = addr(v, dev, *st, {P, ps, Hkv, D});
  t->page_table = static_cast<const int32_t*>(pt.data_ptr());
  t->seq_start = static_cast<const int32_t*>(addr(seq_start, dev, at::kInt, {S + 1}));
  t->kv_len = static_cast<const int32_t*>(addr(kv_len, dev, at::kInt, {S}));
}

// (device, stream, k_cache, v_cache, k_new, v_new, page_table, seq_start, kv_len)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 9);
    const int dev = i32(a[0]);
    rssm_paged_attention_desc d{};
    rssm_paged_attention_tables t{};
    at::ScalarType st;
    caches(a[2], a[3], a[6], a[7], a[8], dev, &d, &t, &st);
    const int64_t N = tensor(a[4], dev).size(0);
    t.k_new = addr(a[4], dev, st, {N, d.num_kv_heads, d.head_dim});
    t.v_new = addr(a[5], dev, st, {N, d.num_kv_heads, d.head_dim});
    d.num_tokens = i32(N);
    d.new_token_stride = static_cast<int64_t>(d.num_kv_heads) * d.head_dim;
    return rssm_paged_append(&d, &t, stream(a[1])) == RSSM_OK;
  });
}

// (device, stream, q, k_cache, v_cache, page_table, seq_start, kv_len, out, max_seq_len, max_kv_len, scale, window,
//  sinks, lse, workspace)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 16);
    const int dev = i32(a[0]);
    rssm_paged_attention_desc d{};
    rssm_paged_attention_tables t{};
    at::ScalarType st;
    caches(a[3], a[4], a[5], a[6], a[7], dev, &d, &t, &st);
    const at::Tensor& q = tensor(a[2], dev);
    need(q.dim() == 3);
    const int64_t N = q.size(0), Hq = q.size(1), D = d.head_dim;
    t.q = addr(a[2], dev, st, {N, Hq, D});
    t.out = addr(a[8], dev, st, {N, Hq, D});
    t.lse = static_cast<float*>(opt(a[14], dev, at::kFloat, {N, Hq}));
    d.num_tokens = i32(N);
    d.num_q_heads = i32(Hq);
    d.q_token_stride = d.out_token_stride = Hq * D;
    d.max_seq_len = i32(a[9]);
    d.max_kv_len = i32(a[10]);
    d.scale = a[11] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : real(a[11]);
    d.window = i32(a[12]);
    d.sinks = i32(a[13]);
    int64_t bytes = 0;
    need(rssm_paged_attention_workspace(&d, &bytes) == RSSM_OK);
    const at::Tensor ws = workspace(a[15], bytes, dev);
    if (ws.defined()) {
      t.workspace = ws.data_ptr();
      d.workspace_bytes = static_cast<int64_t>(ws.nbytes());
    }
    return rssm_paged_attention(&d, &t, stream(a[1])) == RSSM_OK;
  });
}

// (device, stream, y, residual, residual_out, normed, z, post_weight, pre_weight, channel_scale, residual_scale,
//  groups, eps)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 13);
    const int dev = i32(a[0]);
    const at::Tensor &y = tensor(a[2], dev), &r = tensor(a[3], dev);
    need(y.dim() == 2);
    const int64_t R = y.size(0), C = y.size(1);
    const at::ScalarType it = y.scalar_type(), rt = r.scalar_type();
    rssm_block_norm_desc d{};
    rssm_block_norm_tables t{};
    d.rows = i32(R);
    d.channels = i32(C);
    d.groups = i32(a[11]);
    d.input_dtype = code_of(it);
    d.residual_dtype = code_of(rt);
    d.eps = real(a[12]);
    d.residual_scale = real(a[10]);
    d.y_row_stride = d.z_row_stride = d.residual_row_stride = d.residual_out_row_stride = d.normed_row_stride = C;
    t.y = y.data_ptr();
    t.residual = addr(a[3], dev, rt, {R, C});
    t.residual_out = addr(a[4], dev, rt, {R, C});
    t.normed = opt(a[5], dev, it, {R, C});
    t.z = opt(a[6], dev, it, {R, C});
    t.post_weight = static_cast<const float*>(opt(a[7], dev, at::kFloat, {C}));
    t.pre_weight = static_cast<const float*>(opt(a[8], dev, at::kFloat, {C}));
    t.channel_scale = static_cast<const float*>(opt(a[9], dev, at::kFloat, {C}));
    return rssm_block_norm(&d, &t, stream(a[1])) == RSSM_OK;
  });
}

PyMethodDef methods[] = {
    {"linear_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear_attention)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_attention)), METH_FASTCALL, nullptr},
    {"block_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(block_norm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_calls() { return PyModule_Create(&module); }
