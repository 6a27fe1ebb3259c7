// rssm_linear_attention.hip -- host side of rssm_linear_attention.h: argument
// checks, the split of the token axis, launches on the caller's stream.
#include "rssm_linear_attention.h"

#include <algorithm>
#include <cstdio>

#include "linattn_inst.h"
#include "rssm_host.h"

namespace rssm {
const void* linattn_f32_for(int which, int state_dtype, int dstate);
const void* linattn_bf16_for(int which, int state_dtype, int dstate);
const void* linattn_f16_for(int which, int state_dtype, int dstate);
}  // namespace rssm

namespace {

using namespace rssm;

const void* kernel_for(int which, const rssm_linear_attention_desc* d) {
  switch (d->input_dtype) {
    case RSSM_F32: return linattn_f32_for(which, d->state_dtype, d->dstate);
    case RSSM_BF16: return linattn_bf16_for(which, d->state_dtype, d->dstate);
    default: return linattn_f16_for(which, d->state_dtype, d->dstate);
  }
}

int elem_bytes(int dt) { return dt == RSSM_F32 ? 4 : 2; }

rssm_status check_desc(const rssm_linear_attention_desc* d, bool step) {
  if (d == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->num_seqs < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_seqs must be >= 0 (got %d)", d->num_seqs);
  if (d->num_tokens < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_tokens must be >= 0 (got %d)", d->num_tokens);
  if (step && d->num_tokens != d->num_seqs)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "the single-token form takes one row per request (num_tokens %d, num_seqs %d)",
                d->num_tokens, d->num_seqs);
  if (d->num_heads < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_heads must be >= 1 (got %d)", d->num_heads);
  if (d->heads_per_group < 1 || d->num_heads % d->heads_per_group != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "heads_per_group (%d) must be >= 1 and divide num_heads (%d)",
                d->heads_per_group, d->num_heads);
  if (d->num_slots < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_slots must be >= 1 (got %d)", d->num_slots);
  if (d->max_seq_len < 0 || d->max_seq_len > (1 << 30))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "max_seq_len must be in [0, 2^30] (got %d)", d->max_seq_len);
  if (d->dt_softplus != 0 && d->dt_softplus != 1)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "dt_softplus must be 0 or 1 (got %d)", d->dt_softplus);
  for (int dt : {d->state_dtype, d->input_dtype})
    if (dt < RSSM_F32 || dt > RSSM_F8E4M3) return fail(RSSM_ERR_INVALID_ARGUMENT, "unknown dtype %d", dt);
  if (d->state_dtype > RSSM_F16 || d->input_dtype > RSSM_F16)
    return fail(RSSM_ERR_UNSUPPORTED, "state and input dtypes must be f32, bf16 or f16 (got %s, %s)",
                dtype_name(d->state_dtype), dtype_name(d->input_dtype));
  if ((d->dim != 64 && d->dim != 128) || (d->dstate != 64 && d->dstate != 128))
    return fail(RSSM_ERR_UNSUPPORTED, "no compiled instance for dim=%d dstate=%d (64 or 128 each)", d->dim, d->dstate);
  const int64_t H = d->num_heads, G = H / d->heads_per_group;
  const int64_t sb = elem_bytes(d->state_dtype), ib = elem_bytes(d->input_dtype);
  if (H > (int64_t(1) << 20)) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_heads exceeds 2^20");
  if (d->state_slot_stride < H * d->dim * d->dstate)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "state_slot_stride is below the dense per-slot size");
  if ((d->state_slot_stride * sb) % 16 != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "state_slot_stride must be a multiple of 16 bytes");
  if (d->state_slot_stride > (int64_t(1) << 46) / d->num_slots)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_slots*state_slot_stride exceeds 2^46 elements");
  struct T { int64_t v, least; const char* n; };
  const T strides[] = {{d->x_token_stride, H * d->dim, "x_token_stride"}, {d->B_token_stride, G * d->dstate, "B_token_stride"},
                       {d->C_token_stride, G * d->dstate, "C_token_stride"}, {d->z_token_stride, H * d->dim, "z_token_stride"},
                       {d->y_token_stride, H * d->dim, "y_token_stride"}};
  for (const T& t : strides) {
    if (t.v < t.least) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is below the dense row", t.n);
    if ((t.v * ib) % 16 != 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s must be a multiple of 16 bytes", t.n);
    // 32-bit byte offsets inside a chunk of 64 rows
    if (t.v > (int64_t(1) << 22)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s exceeds 2^22 elements", t.n);
  }
  if (d->dt_token_stride < H || d->dt_token_stride > (int64_t(1) << 22))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "dt_token_stride must be in [num_heads, 2^22]");
  if (d->workspace_bytes < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "workspace_bytes must be >= 0");
  return RSSM_OK;
}

rssm_status check_tables(const rssm_linear_attention_desc* d, const rssm_linear_attention_tables* t, bool step) {
  struct P { const void* p; const char* n; size_t align; };
  const P need[] = {{t->state, "state", 16}, {t->A, "A", 4}, {t->slots, "slots", 4}};
  for (const P& e : need) {
    if (e.p == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
    if (!aligned(e.p, e.align)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  }
  if (!step && t->seq_start == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "seq_start is NULL");
  if (d->num_tokens > 0) {   // empty tensors may have NULL addresses
    const P rows[] = {{t->x, "x", 16}, {t->B, "B", 16}, {t->C, "C", 16}, {t->y, "y", 16}};
    for (const P& e : rows) {
      if (e.p == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
      if (!aligned(e.p, e.align)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
    }
  }
  const P opt[] = {{t->D, "D", 4}, {t->dt_bias, "dt_bias", 4}, {t->dt, "dt", 4}, {t->z, "z", 16},
                   {t->seq_start, "seq_start", 4}, {t->load_state, "load_state", 4}, {t->workspace, "workspace", 16}};
  for (const P& e : opt)
    if (e.p != nullptr && !aligned(e.p, e.align))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  if (t->dt == nullptr && d->num_tokens > 0 && (t->dt_bias != nullptr || d->dt_softplus != 0))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "without dt there is no dt_bias and dt_softplus is 0");
  return RSSM_OK;
}

struct Split { int nseg, seg_len; };

// Stretches of the token axis.  Every stretch but the last is folded twice (its
// state, then its outputs), so the axis is split only when the (sequence, head)
// tiles leave compute units without a workgroup (5 prompts of 1,500 tokens, 64 heads, 320 tiles: 103 us
// whole, 125 in two stretches).  Then as many stretches as give each two (8 ragged prompts up to
// 2,500, 24 heads: 90 us with three, 117 with two; one prompt of 16,384 tokens and 64 heads: 228 us with 8
// stretches, 234 with 16, 253 with 24), at most one a chunk (7 prompts up to 605 tokens of 2 heads:
// 18.6 us, 28.2 with four chunks a stretch) and 64, because the scan is serial (one prompt of
// 16,384 tokens and one head: 34.5 us with 64, 52.4 with 256).
Split split_of(const rssm_linear_attention_desc* d) {
  const int64_t items = static_cast<int64_t>(d->num_seqs) * d->num_heads * (d->dim / kLinP);
  const int64_t chunks = (static_cast<int64_t>(d->max_seq_len) + kLinQ - 1) / kLinQ;
  constexpr int64_t kFill = 512, kMaxStretches = 64;
  if (items == 0 || items > kFill / 2 || chunks < 3) return {1, static_cast<int>(std::max<int64_t>(chunks, 1) * kLinQ)};
  const int64_t want = std::min(std::min((kFill + items - 1) / items, chunks), kMaxStretches);
  if (want <= 1) return {1, static_cast<int>(chunks * kLinQ)};
  const int64_t per = (chunks + want - 1) / want;
  return {static_cast<int>((chunks + per - 1) / per), static_cast<int>(per * kLinQ)};
}

int64_t state_bytes(const rssm_linear_attention_desc* d, const Split& s) {
  return static_cast<int64_t>(d->num_seqs) * s.nseg * d->num_heads * d->dim * d->dstate * 4;
}

int64_t workspace_of(const rssm_linear_attention_desc* d, const Split& s) {
  if (s.nseg == 1) return 0;
  return state_bytes(d, s) + static_cast<int64_t>(d->num_seqs) * s.nseg * d->num_heads * 4;
}

void fill_args(LinArgs* a, const rssm_linear_attention_desc* d, const rssm_linear_attention_tables* t) {
  a->state = static_cast<char*>(t->state);
  a->A = t->A;
  a->D = t->D;
  a->dt_bias = t->dt_bias;
  a->x = static_cast<const char*>(t->x);
  a->B = static_cast<const char*>(t->B);
  a->C = static_cast<const char*>(t->C);
  a->dt = t->dt;
  a->z = static_cast<const char*>(t->z);
  a->y = static_cast<char*>(t->y);
  a->slots = t->slots;
  a->seq_start = t->seq_start;
  a->load_state = t->load_state;
  a->ws_state = nullptr;
  a->ws_decay = nullptr;
  a->state_stride = d->state_slot_stride;
  a->x_stride = d->x_token_stride;
  a->B_stride = d->B_token_stride;
  a->C_stride = d->C_token_stride;
  a->dt_stride = d->dt_token_stride;
  a->z_stride = d->z_token_stride;
  a->y_stride = d->y_token_stride;
  a->num_seqs = d->num_seqs;
  a->num_tokens = d->num_tokens;
  a->H = d->num_heads;
  a->hpg = d->heads_per_group;
  a->dim = d->dim;
  a->num_slots = d->num_slots;
  a->pad = d->pad_slot_id;
  a->max_seq_len = d->max_seq_len;
  a->dt_softplus = d->dt_softplus;
  a->nseg = 1;
  a->seg_len = 0;
}

rssm_status launch(const void* fn, dim3 grid, LinArgs* args, int* elems, hipStream_t stream, const char* name) {
  void* params[] = {args, elems};
  hipError_t e = hipLaunchKernel(fn, grid, dim3(kLinBlock), params, 0, stream);
  if (e != hipSuccess) return fail(RSSM_ERR_HIP, "launch of %s failed: %s", name, hipGetErrorString(e));
  return RSSM_OK;
}

}  // namespace

extern "C" {

rssm_status rssm_linear_attention_workspace(const rssm_linear_attention_desc* d, int64_t* bytes) {
  clear_error();
  rssm_status st = check_desc(d, false);
  if (st != RSSM_OK) return st;
  if (bytes == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = workspace_of(d, split_of(d));
  return RSSM_OK;
}

rssm_status rssm_linear_attention(const rssm_linear_attention_desc* d, const rssm_linear_attention_tables* t,
                                  void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, false);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_seqs == 0) return RSSM_OK;
  st = check_tables(d, t, false);
  if (st != RSSM_OK) return st;
  const Split sp = split_of(d);
  const int64_t need = workspace_of(d, sp);
  if (need > 0 && (t->workspace == nullptr || d->workspace_bytes < need))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "workspace of %lld bytes is needed (got %lld)", static_cast<long long>(need),
                static_cast<long long>(t->workspace == nullptr ? 0 : d->workspace_bytes));
  const int64_t items = static_cast<int64_t>(d->num_seqs) * sp.nseg * d->num_heads * (d->dim / kLinP);
  if (items > kMaxWorkgroups)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_seqs*num_heads*dim/64 must be below 2^24 (got %lld)", static_cast<long long>(items));
  LinArgs a;
  fill_args(&a, d, t);
  a.nseg = sp.nseg;
  a.seg_len = sp.seg_len;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (verbose())
    std::fprintf(stderr, "[rssm_linear_attention] %s/%s seqs=%d heads=%d %dx%d stretches=%d of %d\n",
                 dtype_name(d->state_dtype), dtype_name(d->input_dtype), d->num_seqs, d->num_heads, d->dim, d->dstate,
                 sp.nseg, sp.seg_len);
  if (sp.nseg > 1) {
    a.ws_state = static_cast<float*>(t->workspace);
    a.ws_decay = reinterpret_cast<float*>(static_cast<char*>(t->workspace) + state_bytes(d, sp));
    st = launch(kernel_for(kLinFold, d), dim3(static_cast<unsigned>(items)), &a, nullptr, stream, "linattn_fold");
    if (st != RSSM_OK) return st;
    int elems = d->dim * d->dstate;
    const void* scan = d->state_dtype == RSSM_F32 ? reinterpret_cast<const void*>(&linattn_scan_kernel<kF32>)
                       : d->state_dtype == RSSM_BF16 ? reinterpret_cast<const void*>(&linattn_scan_kernel<kBF16>)
                                                     : reinterpret_cast<const void*>(&linattn_scan_kernel<kF16>);
    st = launch(scan, dim3((elems / 4 + kLinBlock - 1) / kLinBlock, d->num_heads, d->num_seqs), &a, &elems, stream,
                "linattn_scan");
    if (st != RSSM_OK) return st;
  }
  return launch(kernel_for(kLinChunk, d), dim3(static_cast<unsigned>(items)), &a, nullptr, stream, "linattn_chunk");
}

rssm_status rssm_linear_attention_step(const rssm_linear_attention_desc* d, const rssm_linear_attention_tables* t,
                                       void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, true);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_seqs == 0) return RSSM_OK;
  st = check_tables(d, t, true);
  if (st != RSSM_OK) return st;
  const int64_t items = static_cast<int64_t>(d->num_seqs) * d->num_heads * (d->dim / kLinP);
  if (items > kMaxWorkgroups)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_seqs*num_heads*dim/64 must be below 2^24 (got %lld)", static_cast<long long>(items));
  LinArgs a;
  fill_args(&a, d, t);
  if (verbose())
    std::fprintf(stderr, "[rssm_linear_attention_step] %s/%s requests=%d heads=%d %dx%d\n", dtype_name(d->state_dtype),
                 dtype_name(d->input_dtype), d->num_seqs, d->num_heads, d->dim, d->dstate);
  return launch(kernel_for(kLinStep, d), dim3(static_cast<unsigned>(items)), &a, nullptr,
                static_cast<hipStream_t>(hip_stream), "linattn_step");
}

}  // extern "C"
