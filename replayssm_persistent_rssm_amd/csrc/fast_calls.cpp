// fast_calls.cpp -- argument marshalling of the prompt-side operators for the
// common case, as a CPython extension of the binding.
//
// At their smallest these operators are a few microseconds of GPU work, as long as
// Python needs to read the attributes of their tensors.  Each function here
// takes the binding's arguments, checks that every tensor is contiguous (the convolution, selective scan and
// rotary calls also take rows of wider ones, as a packed projection gives them), on the
// given device and of the expected dtype and shape, and makes the C call.  It returns True when the
// call was enqueued; on anything else (strided views, wrong arguments, a library error) it returns
// False, and the binding's Python code handles the call or names the error.  Nothing has been enqueued
// then, unless a later launch of a call that has several failed: the binding's call then starts over, and only
// the last launch of each writes what the caller sees.  (A page fork and a compaction change the tables with their
// first launch: where one fails they return the library's status, which the binding raises, and are not repeated.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "rssm_block_norm.h"
#include "rssm_causal_conv.h"
#include "rssm_linear_attention.h"
#include "rssm_paged_attention.h"
#include "rssm_pages.h"
#include "rssm_rotary.h"
#include "rssm_selective_scan.h"

namespace {

struct NotCommon {};   // leaves a function towards `return False`
struct Failed { rssm_status status; };   // leaves a function towards `return status`

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

// A tensor on the device, of any strides.
const at::Tensor& look(PyObject* o, int dev) {
  need(THPVariable_Check(o));
  const at::Tensor& t = THPVariable_Unpack(o);
  need(t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev);
  return t;
}

// Address and row stride of a tensor of this dtype and shape whose rows are dense inside; the stride of a single row says
// nothing.
void* rows(PyObject* o, int dev, at::ScalarType st, std::initializer_list<int64_t> shape, int64_t* stride) {
  const at::Tensor& t = look(o, dev);
  need(t.scalar_type() == st && t.sizes() == at::IntArrayRef(shape));
  int64_t dense = 1;
  for (int64_t i = t.dim() - 1; i > 0; --i) {
    need(t.size(i) == 1 || t.stride(i) == dense);
    dense *= t.size(i);
  }
  *stride = t.size(0) > 1 ? t.stride(0) : dense;
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

// Whether every tensor among the arguments is on device a[0], and contiguous unless views are taken.  Asked first, so that views, the
// other ordinary case, do not pay for an exception (1 to 3 us) before the binding's Python code takes them.
bool plain(PyObject* const* a, Py_ssize_t n, bool views) {
  if (n < 2 || !PyLong_Check(a[0])) return false;
  int over = 0;
  const long dev = PyLong_AsLongAndOverflow(a[0], &over);
  for (Py_ssize_t i = 2; i < n; ++i) {
    if (!THPVariable_Check(a[i])) continue;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev || (!views && !t.is_contiguous())) return false;
  }
  return true;
}

template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, F f, bool views = false) {
  bool done = false;
  try {
    done = plain(a, n, views) && f();
  } catch (const Failed& e) {
    return PyLong_FromLong(e.status);
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

// (device, stream, step, x, weight, y, state, slots, seq_start, bias, load_state, silu, pad_slot_id)
PyObject* causal_conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 13);
    const int dev = i32(a[0]);
    const bool step = a[2] == Py_True;
    const at::Tensor &x = look(a[3], dev), &w = tensor(a[4], dev), &state = look(a[6], dev), &slots = tensor(a[7], dev);
    need(x.dim() == 2 && w.dim() == 2 && state.dim() == 3 && slots.dim() == 1);
    const int64_t N = x.size(0), C = x.size(1), W = w.size(0), S = state.size(0), R = slots.size(0);
    const at::ScalarType it = x.scalar_type();
    rssm_causal_conv_desc d{};
    d.num_seqs = i32(R);
    d.num_tokens = i32(N);
    d.channels = i32(C);
    d.width = i32(W);
    d.num_slots = i32(S);
    d.pad_slot_id = i32(a[12]);
    d.dtype = code_of(it);
    d.silu = PyObject_IsTrue(a[11]) == 1;
    rssm_causal_conv_tables t{};
    t.x = rows(a[3], dev, it, {N, C}, &d.x_token_stride);
    t.weight = static_cast<const float*>(addr(a[4], dev, at::kFloat, {W, C}));
    t.bias = static_cast<const float*>(opt(a[9], dev, at::kFloat, {C}));
    t.y = rows(a[5], dev, it, {N, C}, &d.y_token_stride);
    t.state = rows(a[6], dev, it, {S, W - 1, C}, &d.state_slot_stride);
    t.slots = static_cast<const int32_t*>(addr(a[7], dev, at::kInt, {R}));
    if (step) return rssm_causal_conv_step(&d, &t, stream(a[1])) == RSSM_OK;
    t.seq_start = static_cast<const int32_t*>(addr(a[8], dev, at::kInt, {R + 1}));
    t.load_state = static_cast<const int32_t*>(opt(a[10], dev, at::kInt, {R}));
    return rssm_causal_conv(&d, &t, stream(a[1])) == RSSM_OK;
  }, true);
}

// (device, stream, step, state, A, x, B, C, dt, y, slots, seq_start, max_seq_len, load_state, D, dt_bias, z,
//  dt_softplus, pad_slot_id, workspace)
PyObject* selective_scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 20);
    const int dev = i32(a[0]);
    const bool step = a[2] == Py_True;
    const at::Tensor &state = look(a[3], dev), &x = look(a[5], dev), &B = look(a[6], dev), &slots = tensor(a[10], dev);
    need(state.dim() == 3 && x.dim() == 2 && B.dim() == 3 && slots.dim() == 1);
    const int64_t S = state.size(0), Ch = state.size(1), ds = state.size(2), N = x.size(0), G = B.size(1), R = slots.size(0);
    const at::ScalarType it = x.scalar_type();
    rssm_selective_scan_desc d{};
    d.num_seqs = i32(R);
    d.num_tokens = i32(N);
    d.channels = i32(Ch);
    d.groups = i32(G);
    d.dstate = i32(ds);
    d.num_slots = i32(S);
    d.pad_slot_id = i32(a[18]);
    d.max_seq_len = i32(a[12]);
    d.state_dtype = code_of(state.scalar_type());
    d.input_dtype = code_of(it);
    d.dt_softplus = PyObject_IsTrue(a[17]) == 1;
    rssm_selective_scan_tables t{};
    t.state = rows(a[3], dev, state.scalar_type(), {S, Ch, ds}, &d.state_slot_stride);
    t.A = static_cast<const float*>(addr(a[4], dev, at::kFloat, {Ch, ds}));
    t.D = static_cast<const float*>(opt(a[14], dev, at::kFloat, {Ch}));
    t.dt_bias = static_cast<const float*>(opt(a[15], dev, at::kFloat, {Ch}));
    t.x = rows(a[5], dev, it, {N, Ch}, &d.x_token_stride);
    t.B = rows(a[6], dev, it, {N, G, ds}, &d.B_token_stride);
    t.C = rows(a[7], dev, it, {N, G, ds}, &d.C_token_stride);
    t.dt = rows(a[8], dev, it, {N, Ch}, &d.dt_token_stride);
    t.y = rows(a[9], dev, it, {N, Ch}, &d.y_token_stride);
    d.z_token_stride = d.x_token_stride;
    if (a[16] != Py_None) t.z = rows(a[16], dev, it, {N, Ch}, &d.z_token_stride);
    t.slots = static_cast<const int32_t*>(addr(a[10], dev, at::kInt, {R}));
    if (step) return rssm_selective_scan_step(&d, &t, stream(a[1])) == RSSM_OK;
    t.seq_start = static_cast<const int32_t*>(addr(a[11], dev, at::kInt, {R + 1}));
    t.load_state = static_cast<const int32_t*>(opt(a[13], dev, at::kInt, {R}));
    int64_t bytes = 0;
    need(rssm_selective_scan_workspace(&d, &bytes) == RSSM_OK);
    const at::Tensor ws = workspace(a[19], bytes, dev);
    if (ws.defined()) {
      t.workspace = ws.data_ptr();
      d.workspace_bytes = static_cast<int64_t>(ws.nbytes());
    }
    return rssm_selective_scan(&d, &t, stream(a[1])) == RSSM_OK;
  }, true);
}

// (device, stream, q, q_out, k_cache, v_cache, k_new, v_new, page_table, seq_start, kv_len, inv_freq, interleaved,
//  factor, positions): queries, keys and values all there
PyObject* rotary_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 15);
    const int dev = i32(a[0]);
    rssm_paged_attention_desc p{};
    rssm_paged_attention_tables pt{};
    at::ScalarType st;
    caches(a[4], a[5], a[8], a[9], a[10], dev, &p, &pt, &st);
    const at::Tensor &q = look(a[2], dev), &f = tensor(a[11], dev);
    need(q.dim() == 3 && f.dim() == 1);
    const int64_t N = q.size(0), Hq = q.size(1), D = p.head_dim, Hkv = p.num_kv_heads;
    rssm_rotary_desc d{};
    rssm_rotary_tables t{};
    d.num_seqs = p.num_seqs;
    d.num_tokens = i32(N);
    d.num_q_heads = i32(Hq);
    d.num_kv_heads = p.num_kv_heads;
    d.head_dim = p.head_dim;
    d.rot_dim = i32(2 * f.size(0));
    d.interleaved = PyObject_IsTrue(a[12]) == 1;
    d.page_size = p.page_size;
    d.num_pages = p.num_pages;
    d.max_pages = p.max_pages;
    d.dtype = p.dtype;
    d.factor = real(a[13]);
    d.page_stride = p.page_stride;
    d.row_stride = p.row_stride;
    d.head_stride = p.head_stride;
    d.table_stride = p.table_stride;
    t.q = rows(a[2], dev, st, {N, Hq, D}, &d.q_token_stride);
    t.q_out = rows(a[3], dev, st, {N, Hq, D}, &d.q_out_token_stride);
    t.k_new = rows(a[6], dev, st, {N, Hkv, D}, &d.k_token_stride);
    t.v_new = rows(a[7], dev, st, {N, Hkv, D}, &d.v_token_stride);
    t.k_cache = pt.k_cache;
    t.v_cache = pt.v_cache;
    t.page_table = pt.page_table;
    t.seq_start = pt.seq_start;
    t.kv_len = pt.kv_len;
    t.positions = static_cast<const int32_t*>(opt(a[14], dev, at::kInt, {N}));
    t.inv_freq = static_cast<const float*>(addr(a[11], dev, at::kFloat, {f.size(0)}));
    return rssm_rotary_append(&d, &t, stream(a[1])) == RSSM_OK;
  }, true);
}

// The page pool's fields: page_table, kv_len, page_ref and page_size.
void pool(PyObject* table, PyObject* kv_len, PyObject* ref, PyObject* page_size, int dev, rssm_pages_desc* d,
          rssm_pages_tables* t) {
  const at::Tensor &pt = tensor(table, dev), &pr = tensor(ref, dev);
  need(pt.dim() == 2 && pt.scalar_type() == at::kInt && pr.dim() == 1 && pr.scalar_type() == at::kInt);
  d->num_rows = i32(pt.size(0));
  d->max_pages = i32(pt.size(1));
  d->num_pages = i32(pr.size(0));
  d->page_size = i32(page_size);
  d->table_stride = pt.size(1);
  t->page_table = static_cast<int32_t*>(pt.data_ptr());
  t->kv_len = static_cast<int32_t*>(addr(kv_len, dev, at::kInt, {pt.size(0)}));
  t->page_ref = static_cast<int32_t*>(pr.data_ptr());
}

int64_t items(PyObject* dst, int dev, rssm_pages_desc* d, rssm_pages_tables* t) {
  const at::Tensor& r = tensor(dst, dev);
  need(r.dim() == 1 && r.scalar_type() == at::kInt);
  d->num_items = i32(r.size(0));
  t->dst = static_cast<const int32_t*>(r.data_ptr());
  return r.size(0);
}

int32_t* ints(PyObject* o, int dev, int64_t n) { return static_cast<int32_t*>(opt(o, dev, at::kInt, {n})); }

void pool_caches(PyObject* ptrs, PyObject* page_bytes, PyObject* page_stride, int dev, rssm_pages_desc* d,
                 rssm_pages_tables* t) {
  const at::Tensor& p = tensor(ptrs, dev);
  need(p.dim() == 1 && p.scalar_type() == at::kLong);
  d->num_caches = i32(p.size(0));
  d->page_bytes = integer(page_bytes);
  d->page_stride = integer(page_stride);
  t->cache_ptrs = p.data_ptr<int64_t>();
}

at::Tensor pool_workspace(PyObject* given, int dev, rssm_pages_desc* d, rssm_pages_tables* t) {
  int64_t bytes = 0;
  need(rssm_pages_workspace(d, &bytes) == RSSM_OK);
  const at::Tensor ws = workspace(given, bytes, dev);
  t->workspace = ws.data_ptr();
  d->workspace_bytes = static_cast<int64_t>(ws.nbytes());
  return ws;
}

// Whether a call of two launches, the first of which changes the tables, was enqueued.
bool enqueued(rssm_status st) {
  if (st == RSSM_ERR_HIP) throw Failed{st};
  return st == RSSM_OK;
}

// (device, stream, page_table, kv_len, page_ref, rows, add, status, page_size, workspace)
PyObject* page_extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 10);
    const int dev = i32(a[0]);
    rssm_pages_desc d{};
    rssm_pages_tables t{};
    pool(a[2], a[3], a[4], a[8], dev, &d, &t);
    const int64_t k = items(a[5], dev, &d, &t);
    t.lengths = ints(a[6], dev, k);
    t.status = ints(a[7], dev, k);
    const at::Tensor ws = pool_workspace(a[9], dev, &d, &t);
    return rssm_page_extend(&d, &t, stream(a[1])) == RSSM_OK;
  });
}

// (device, stream, cache_ptrs, page_table, kv_len, page_ref, src, dst, status, page_size, page_bytes, page_stride,
//  token_bytes, lengths, workspace)
PyObject* page_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 15);
    const int dev = i32(a[0]);
    rssm_pages_desc d{};
    rssm_pages_tables t{};
    pool(a[3], a[4], a[5], a[9], dev, &d, &t);
    const int64_t k = items(a[7], dev, &d, &t);
    t.src = ints(a[6], dev, k);
    t.status = ints(a[8], dev, k);
    t.lengths = ints(a[13], dev, k);
    pool_caches(a[2], a[10], a[11], dev, &d, &t);
    d.token_bytes = integer(a[12]);
    const at::Tensor ws = pool_workspace(a[14], dev, &d, &t);
    return enqueued(rssm_page_fork(&d, &t, stream(a[1])));
  });
}

// (device, stream, page_table, kv_len, page_ref, rows, page_size, lengths)
PyObject* page_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 8);
    const int dev = i32(a[0]);
    rssm_pages_desc d{};
    rssm_pages_tables t{};
    pool(a[2], a[3], a[4], a[6], dev, &d, &t);
    const int64_t k = items(a[5], dev, &d, &t);
    t.lengths = ints(a[7], dev, k);
    return rssm_page_release(&d, &t, stream(a[1])) == RSSM_OK;
  });
}

// (device, stream, cache_ptrs, page_table, kv_len, page_ref, live, page_size, page_bytes, page_stride, workspace)
PyObject* page_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, [&] {
    need(n == 11);
    const int dev = i32(a[0]);
    rssm_pages_desc d{};
    rssm_pages_tables t{};
    pool(a[3], a[4], a[5], a[7], dev, &d, &t);
    pool_caches(a[2], a[8], a[9], dev, &d, &t);
    t.live = static_cast<int32_t*>(addr(a[6], dev, at::kInt, {1}));
    const at::Tensor ws = pool_workspace(a[10], dev, &d, &t);
    return enqueued(rssm_page_compact(&d, &t, stream(a[1])));
  });
}

PyMethodDef methods[] = {
    {"linear_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear_attention)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_attention)), METH_FASTCALL, nullptr},
    {"block_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(block_norm)), METH_FASTCALL, nullptr},
    {"causal_conv", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(causal_conv)), METH_FASTCALL, nullptr},
    {"selective_scan", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(selective_scan)), METH_FASTCALL, nullptr},
    {"rotary_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rotary_append)), METH_FASTCALL, nullptr},
    {"page_extend", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_extend)), METH_FASTCALL, nullptr},
    {"page_fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_fork)), METH_FASTCALL, nullptr},
    {"page_release", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_release)), METH_FASTCALL, nullptr},
    {"page_compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_compact)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_calls() { return PyModule_Create(&module); }
