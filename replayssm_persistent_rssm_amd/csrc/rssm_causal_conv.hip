// rssm_causal_conv.hip -- host side of rssm_causal_conv.h: argument checks and
// launches on the caller's stream.
#include "rssm_causal_conv.h"

#include <cstdio>

#include "conv_kernel.h"
#include "rssm_host.h"

namespace {

using namespace rssm;

rssm_status check_desc(const rssm_causal_conv_desc* d, bool step) {
  if (d == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->num_seqs < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_seqs must be >= 0 (got %d)", d->num_seqs);
  if (d->num_tokens < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_tokens must be >= 0 (got %d)", d->num_tokens);
  if (step && d->num_tokens != d->num_seqs)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "the single-token form takes one row per request (num_tokens %d, num_seqs %d)",
                d->num_tokens, d->num_seqs);
  if (d->channels < 8 || d->channels > (1 << 20) || d->channels % 8 != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "channels must be a multiple of 8 in [8, 2^20] (got %d)", d->channels);
  if (d->width < 2 || d->width > 4) return fail(RSSM_ERR_UNSUPPORTED, "no compiled instance for width=%d (2, 3, 4)", d->width);
  if (d->num_slots < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_slots must be >= 1 (got %d)", d->num_slots);
  if (d->dtype < RSSM_F32 || d->dtype > RSSM_F8E4M3) return fail(RSSM_ERR_INVALID_ARGUMENT, "unknown dtype %d", d->dtype);
  if (d->dtype > RSSM_F16)
    return fail(RSSM_ERR_UNSUPPORTED, "dtype must be f32, bf16 or f16 (got %s)", dtype_name(d->dtype));
  if (d->silu != 0 && d->silu != 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "silu must be 0 or 1 (got %d)", d->silu);
  const int64_t es = d->dtype == RSSM_F32 ? 4 : 2;
  struct S { int64_t v, least; const char* n; };
  const S strides[] = {{d->state_slot_stride, static_cast<int64_t>(d->width - 1) * d->channels, "state_slot_stride"},
                       {d->x_token_stride, d->channels, "x_token_stride"}, {d->y_token_stride, d->channels, "y_token_stride"}};
  for (const S& s : strides) {
    if (s.v < s.least) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is below the dense size", s.n);
    if (s.v > (int64_t(1) << 31)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s exceeds 2^31 elements", s.n);
    if ((s.v * es) % 16 != 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s must be a multiple of 16 bytes", s.n);
  }
  return RSSM_OK;
}

rssm_status check_tables(const rssm_causal_conv_desc* d, const rssm_causal_conv_tables* t, bool step) {
  struct P { const void* p; const char* n; size_t align; };
  const P need[] = {{t->weight, "weight", 16}, {t->state, "state", 16}, {t->slots, "slots", 4}};
  for (const P& e : need) {
    if (e.p == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
    if (!aligned(e.p, e.align)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  }
  if (!step && t->seq_start == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "seq_start is NULL");
  if (d->num_tokens > 0) {   // empty tensors may have NULL addresses
    const P rows[] = {{t->x, "x", 16}, {t->y, "y", 16}};
    for (const P& e : rows) {
      if (e.p == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
      if (!aligned(e.p, e.align)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
    }
    if (!step && t->x == t->y) return fail(RSSM_ERR_INVALID_ARGUMENT, "y may not be x in the prompt form");
  }
  const P opt[] = {{t->bias, "bias", 16}, {t->seq_start, "seq_start", 4}, {t->load_state, "load_state", 4}};
  for (const P& e : opt)
    if (e.p != nullptr && !aligned(e.p, e.align))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  return RSSM_OK;
}

void fill_args(ConvArgs* a, const rssm_causal_conv_desc* d, const rssm_causal_conv_tables* t) {
  a->x = static_cast<const char*>(t->x);
  a->weight = t->weight;
  a->bias = t->bias;
  a->y = static_cast<char*>(t->y);
  a->state = static_cast<char*>(t->state);
  a->slots = t->slots;
  a->seq_start = t->seq_start;
  a->load_state = t->load_state;
  a->state_stride = d->state_slot_stride;
  a->x_stride = d->x_token_stride;
  a->y_stride = d->y_token_stride;
  a->num_seqs = d->num_seqs;
  a->num_tokens = d->num_tokens;
  a->channels = d->channels;
  a->num_slots = d->num_slots;
  a->pad = d->pad_slot_id;
  a->silu = d->silu;
  a->blocks = (d->channels + kConvLanes - 1) / kConvLanes;
}

template <int DT, int W>
const void* instance(bool step, int size) {
  if (step)
    return size > 1 ? reinterpret_cast<const void*>(&conv_step_kernel<DT, W, 4>)
                    : reinterpret_cast<const void*>(&conv_step_kernel<DT, W, 1>);
  return size > 4 ? reinterpret_cast<const void*>(&conv_prompt_kernel<DT, W, 8>)
                  : reinterpret_cast<const void*>(&conv_prompt_kernel<DT, W, 4>);
}

template <int DT>
const void* of_width(int width, bool step, int size) {
  return width == 2 ? instance<DT, 2>(step, size) : width == 3 ? instance<DT, 3>(step, size) : instance<DT, 4>(step, size);
}

const void* kernel_for(const rssm_causal_conv_desc* d, bool step, int size) {
  return d->dtype == RSSM_F32 ? of_width<kF32>(d->width, step, size)
         : d->dtype == RSSM_BF16 ? of_width<kBF16>(d->width, step, size) : of_width<kF16>(d->width, step, size);
}

rssm_status launch(ConvArgs* a, const rssm_causal_conv_desc* d, bool step, int size, int64_t items, void* stream) {
  const char* name = step ? "causal_conv_step" : "causal_conv";
  const int64_t units = items * a->blocks;
  const int64_t grid = (units + kConvBlock / 64 - 1) / (kConvBlock / 64);
  if (grid > kMaxWorkgroups)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "%s needs %lld workgroups, more than one launch takes (2^24 - 1)", name,
                static_cast<long long>(grid));
  a->units = static_cast<int32_t>(units);
  if (verbose())
    std::fprintf(stderr, "[rssm_%s] %s seqs=%d tokens=%d channels=%d width=%d size=%d\n", name, dtype_name(d->dtype),
                 d->num_seqs, d->num_tokens, d->channels, d->width, size);
  void* params[] = {a};
  hipError_t e = hipLaunchKernel(kernel_for(d, step, size), dim3(static_cast<unsigned>(grid)), dim3(kConvBlock), params, 0,
                                 static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(RSSM_ERR_HIP, "launch of %s failed: %s", name, hipGetErrorString(e));
  return RSSM_OK;
}

}  // namespace

extern "C" {

rssm_status rssm_causal_conv(const rssm_causal_conv_desc* d, const rssm_causal_conv_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, false);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_seqs == 0) return RSSM_OK;
  st = check_tables(d, t, false);
  if (st != RSSM_OK) return st;
  ConvArgs a;
  fill_args(&a, d, t);
  // tiles of 8 tokens; of 4 where those would be at most 8,192 wavefronts and a tile's latency counts (us with 4 and 8: 97 tokens,
  // 1,024 channels 3.6, 4.5; 300 tokens, 18,432 channels 7.0, 8.2; 1,000 tokens 14.7, 15.4; 4,000 tokens, 18,000
  // wavefronts, 66, 60).  Longer tiles read fewer rows twice and gain nothing by it (16,384 tokens, 18,432 channels: 221 with 8,
  // 226 with 16, 228 with 32, 243 with 64)
  const int64_t tiles = d->num_tokens / 8 + static_cast<int64_t>(d->num_seqs);
  const int size = tiles * a.blocks > 8192 ? 8 : 4;
  return launch(&a, d, false, size, d->num_tokens / size + static_cast<int64_t>(d->num_seqs), hip_stream);
}

rssm_status rssm_causal_conv_step(const rssm_causal_conv_desc* d, const rssm_causal_conv_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, true);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_seqs == 0) return RSSM_OK;
  st = check_tables(d, t, true);
  if (st != RSSM_OK) return st;
  ConvArgs a;
  fill_args(&a, d, t);
  const int size = static_cast<int64_t>(d->num_seqs) * a.blocks >= 4096 ? 4 : 1;
  return launch(&a, d, true, size, (d->num_seqs + static_cast<int64_t>(size) - 1) / size, hip_stream);
}

}  // extern "C"
