// rssm_selective_scan.hip -- host side of rssm_selective_scan.h: argument
// checks, the split of the token axis, launches on the caller's stream.
#include "rssm_selective_scan.h"

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "rssm_host.h"
#include "scan_inst.h"

namespace rssm {
const void* scan_f32_for(int which, int state_dtype, int dstate);
const void* scan_bf16_for(int which, int state_dtype, int dstate);
const void* scan_f16_for(int which, int state_dtype, int dstate);
}  // namespace rssm

namespace {

using namespace rssm;

const void* kernel_for(int which, const rssm_selective_scan_desc* d) {
  switch (d->input_dtype) {
    case RSSM_F32: return scan_f32_for(which, d->state_dtype, d->dstate);
    case RSSM_BF16: return scan_bf16_for(which, d->state_dtype, d->dstate);
    default: return scan_f16_for(which, d->state_dtype, d->dstate);
  }
}

rssm_status check_desc(const rssm_selective_scan_desc* d, bool step) {
  if (d == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->num_seqs < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_seqs must be >= 0 (got %d)", d->num_seqs);
  if (d->num_tokens < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_tokens must be >= 0 (got %d)", d->num_tokens);
  if (step && d->num_tokens != d->num_seqs)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "the single-token form takes one row per request (num_tokens %d, num_seqs %d)",
                d->num_tokens, d->num_seqs);
  if (d->channels < 8 || d->channels > (1 << 20) || d->channels % 8 != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "channels must be a multiple of 8 in [8, 2^20] (got %d)", d->channels);
  if (d->groups < 1 || d->channels % d->groups != 0 || (d->groups > 1 && (d->channels / d->groups) % 16 != 0))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "groups (%d) must be >= 1 and split channels (%d) into multiples of 16",
                d->groups, d->channels);
  if (d->num_slots < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_slots must be >= 1 (got %d)", d->num_slots);
  if (d->max_seq_len < 0 || d->max_seq_len > (1 << 30))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "max_seq_len must be in [0, 2^30] (got %d)", d->max_seq_len);
  if (d->dt_softplus != 0 && d->dt_softplus != 1)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "dt_softplus must be 0 or 1 (got %d)", d->dt_softplus);
  if (d->reserved != 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "reserved must be 0");
  for (int dt : {d->state_dtype, d->input_dtype})
    if (dt < RSSM_F32 || dt > RSSM_F8E4M3) return fail(RSSM_ERR_INVALID_ARGUMENT, "unknown dtype %d", dt);
  if (d->state_dtype > RSSM_F16 || d->input_dtype > RSSM_F16)
    return fail(RSSM_ERR_UNSUPPORTED, "state and input dtypes must be f32, bf16 or f16 (got %s, %s)",
                dtype_name(d->state_dtype), dtype_name(d->input_dtype));
  if (d->dstate != 16 && d->dstate != 32 && d->dstate != 64)
    return fail(RSSM_ERR_UNSUPPORTED, "no compiled instance for dstate=%d (16, 32, 64)", d->dstate);
  const int64_t ib = d->input_dtype == RSSM_F32 ? 4 : 2, sb = d->state_dtype == RSSM_F32 ? 4 : 2;
  const int64_t C = d->channels, GN = static_cast<int64_t>(d->groups) * d->dstate;
  if (d->state_slot_stride < C * d->dstate)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "state_slot_stride is below the dense per-slot size");
  if ((d->state_slot_stride * sb) % 16 != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "state_slot_stride must be a multiple of 16 bytes");
  if (d->state_slot_stride > (int64_t(1) << 46) / d->num_slots)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_slots*state_slot_stride exceeds 2^46 elements");
  struct T { int64_t v, least; const char* n; };
  const T strides[] = {{d->x_token_stride, C, "x_token_stride"}, {d->dt_token_stride, C, "dt_token_stride"},
                       {d->B_token_stride, GN, "B_token_stride"}, {d->C_token_stride, GN, "C_token_stride"},
                       {d->z_token_stride, C, "z_token_stride"}, {d->y_token_stride, C, "y_token_stride"}};
  for (const T& t : strides) {
    if (t.v < t.least) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is below the dense row", t.n);
    if ((t.v * ib) % 16 != 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s must be a multiple of 16 bytes", t.n);
    // 32-bit byte offsets inside a tile of 16 rows
    if (t.v > (int64_t(1) << 24)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s exceeds 2^24 elements", t.n);
  }
  if (d->workspace_bytes < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "workspace_bytes must be >= 0");
  return RSSM_OK;
}

rssm_status check_tables(const rssm_selective_scan_desc* d, const rssm_selective_scan_tables* t, bool step) {
  struct P { const void* p; const char* n; size_t align; };
  const P need[] = {{t->state, "state", 16}, {t->A, "A", 16}, {t->slots, "slots", 4}};
  for (const P& e : need) {
    if (e.p == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
    if (!aligned(e.p, e.align)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  }
  if (!step && t->seq_start == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "seq_start is NULL");
  if (d->num_tokens > 0) {   // empty tensors may have NULL addresses
    const P rows[] = {{t->x, "x", 16}, {t->dt, "dt", 16}, {t->B, "B", 16}, {t->C, "C", 16}, {t->y, "y", 16}};
    for (const P& e : rows) {
      if (e.p == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
      if (!aligned(e.p, e.align)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
    }
  }
  const P opt[] = {{t->D, "D", 16}, {t->dt_bias, "dt_bias", 16}, {t->z, "z", 16}, {t->seq_start, "seq_start", 4},
                   {t->load_state, "load_state", 4}, {t->workspace, "workspace", 16}};
  for (const P& e : opt)
    if (e.p != nullptr && !aligned(e.p, e.align))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  return RSSM_OK;
}

struct Split { int nseg, seg_len; };

int64_t main_blocks(const rssm_selective_scan_desc* d) { return (d->channels + kScanChannels - 1) / kScanChannels; }

// Few channels and short sequences go to scan_short_kernel: up to 4,096 wavefronts of it (four a SIMD) and 512 tokens
// (us with it and without: 12 prompts of 200, 1,024 channels: 24.4, 33.6; one of 200, 8,192 channels: 17.5, 21.6; of 400,
// 4,096 channels: 19.2, 21.6; of 1,000: 41.3, 43.7 and with 8,192 channels 67.4, 63.6), 320 tokens where stretches would have
// most of the device to themselves (1,024 channels: 14.3, 14.9 for 300 tokens, 17.9, 15.2 for 400).  More states a channel
// make the other form's tiles longer and this one's sums cheaper: with 32 and 64 of them up to 2,048 tokens while there are at
// most 2,048 wavefronts (2,000 tokens, 4,096 channels: 107, 113 and 174, 206; 8,192: 179, 195 and 327, 367; 8 of 1,000,
// 2,048 channels, 4,096 wavefronts: 190, 184).
bool is_short(const rssm_selective_scan_desc* d) {
  const int64_t waves = static_cast<int64_t>(d->num_seqs) * ((d->channels + 3) / 4);
  const int longest = waves <= 512 ? 320 : d->dstate > 16 && waves <= 2048 ? 2048 : 512;
  return waves <= 4096 && d->max_seq_len <= longest;
}

// Stretches of the token axis.  All but the last are folded once more than they are computed (70 % of a
// stretch's time), so the axis is split only when the sequences' channel blocks (of 64) leave compute units without a
// workgroup (one prompt of 8,000 tokens, 8,192 channels, 128 blocks: 401 us, 573 with two stretches; three of
// them, 384 blocks: 1,016 us whole, 1,090 in four).  Then as many stretches as give each unit six
// workgroups (one of 16,384 tokens, 4,096 channels: 413 us, 453 with two a unit), of at least two tiles, at most
// sqrt(8 tiles) of them because each reads the ends of those before it (2,048 tokens, 1,024 channels: 27 us with 32, 35
// with 64), and none below 8 tiles, where the second launch costs as much as it saves.
Split split_of(const rssm_selective_scan_desc* d) {
  const int64_t items = d->num_seqs * main_blocks(d);
  const int64_t tiles = (static_cast<int64_t>(d->max_seq_len) + kScanTile - 1) / kScanTile;
  constexpr int64_t kSplit = 256, kFill = 1536, kMost = 64;
  if (items == 0 || items > kSplit || tiles < 8 || is_short(d)) return {1, static_cast<int>(std::max<int64_t>(tiles, 1) * kScanTile)};
  const int64_t reads = static_cast<int64_t>(std::sqrt(8.0 * static_cast<double>(tiles)));
  const int64_t want = std::min(std::min(kFill / items, tiles / 2), std::min(reads, kMost));
  const int64_t per = (tiles + want - 1) / want;
  return {static_cast<int>((tiles + per - 1) / per), static_cast<int>(per * kScanTile)};
}

int64_t workspace_of(const rssm_selective_scan_desc* d, const Split& s) {
  if (s.nseg == 1) return 0;
  return static_cast<int64_t>(d->num_seqs) * s.nseg * d->channels * (d->dstate + 1) * 4;
}

void fill_args(ScanArgs* a, const rssm_selective_scan_desc* d, const rssm_selective_scan_tables* t) {
  a->state = static_cast<char*>(t->state);
  a->A = t->A;
  a->D = t->D;
  a->dt_bias = t->dt_bias;
  a->x = static_cast<const char*>(t->x);
  a->dt = static_cast<const char*>(t->dt);
  a->B = static_cast<const char*>(t->B);
  a->C = static_cast<const char*>(t->C);
  a->z = static_cast<const char*>(t->z);
  a->y = static_cast<char*>(t->y);
  a->slots = t->slots;
  a->seq_start = t->seq_start;
  a->load_state = t->load_state;
  a->ws_h = nullptr;
  a->ws_d = nullptr;
  a->state_stride = d->state_slot_stride;
  a->x_stride = d->x_token_stride;
  a->dt_stride = d->dt_token_stride;
  a->B_stride = d->B_token_stride;
  a->C_stride = d->C_token_stride;
  a->z_stride = d->z_token_stride;
  a->y_stride = d->y_token_stride;
  a->num_seqs = d->num_seqs;
  a->num_tokens = d->num_tokens;
  a->channels = d->channels;
  a->groups = d->groups;
  a->per_group = d->channels / d->groups;
  a->num_slots = d->num_slots;
  a->pad = d->pad_slot_id;
  a->max_seq_len = d->max_seq_len;
  a->dt_softplus = d->dt_softplus;
  a->state_dtype = d->state_dtype;
  a->nseg = 1;
  a->seg_len = 1 << 30;
  a->blocks = 1;
}

rssm_status launch(const void* fn, int64_t grid, ScanArgs* args, void* stream, const char* name) {
  if (grid > kMaxWorkgroups)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "%s needs %lld workgroups, more than one launch takes (2^24 - 1)", name,
                static_cast<long long>(grid));
  void* params[] = {args};
  hipError_t e = hipLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kScanBlock), params, 0,
                                 static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(RSSM_ERR_HIP, "launch of %s failed: %s", name, hipGetErrorString(e));
  return RSSM_OK;
}

}  // namespace

extern "C" {

rssm_status rssm_selective_scan_workspace(const rssm_selective_scan_desc* d, int64_t* bytes) {
  clear_error();
  rssm_status st = check_desc(d, false);
  if (st != RSSM_OK) return st;
  if (bytes == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = workspace_of(d, split_of(d));
  return RSSM_OK;
}

rssm_status rssm_selective_scan(const rssm_selective_scan_desc* d, const rssm_selective_scan_tables* t, void* hip_stream) {
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
  ScanArgs a;
  fill_args(&a, d, t);
  a.nseg = sp.nseg;
  a.seg_len = sp.seg_len;
  a.blocks = static_cast<int32_t>(main_blocks(d));
  if (verbose())
    std::fprintf(stderr, "[rssm_selective_scan] %s/%s seqs=%d channels=%d dstate=%d stretches=%d of %d\n",
                 dtype_name(d->state_dtype), dtype_name(d->input_dtype), d->num_seqs, d->channels, d->dstate, sp.nseg, sp.seg_len);
  if (is_short(d)) {
    a.blocks = (d->channels + kScanShortChannels - 1) / kScanShortChannels;
    return launch(kernel_for(kScanShort, d), static_cast<int64_t>(d->num_seqs) * a.blocks, &a, hip_stream, "selective_scan_short");
  }
  const int64_t grid = static_cast<int64_t>(d->num_seqs) * sp.nseg * a.blocks;
  if (sp.nseg > 1) {
    a.ws_h = static_cast<float*>(t->workspace);
    a.ws_d = a.ws_h + static_cast<int64_t>(d->num_seqs) * sp.nseg * d->channels * d->dstate;
    st = launch(kernel_for(kScanFold, d), grid, &a, hip_stream, "selective_scan_fold");
    if (st != RSSM_OK) return st;
  }
  return launch(kernel_for(kScanMain, d), grid, &a, hip_stream, "selective_scan");
}

rssm_status rssm_selective_scan_step(const rssm_selective_scan_desc* d, const rssm_selective_scan_tables* t,
                                     void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, true);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_seqs == 0) return RSSM_OK;
  st = check_tables(d, t, true);
  if (st != RSSM_OK) return st;
  ScanArgs a;
  fill_args(&a, d, t);
  const int lanes = d->dstate * (d->state_dtype == RSSM_F32 ? 4 : 2) / 16;   // a channel
  const int per = kScanBlock / lanes * (lanes < 4 ? 2 : 4);                  // channels a workgroup
  a.blocks = (d->channels + per - 1) / per;
  const int Q = static_cast<int64_t>(d->num_seqs) * a.blocks >= 2048 ? 2 : 1;
  if (verbose())
    std::fprintf(stderr, "[rssm_selective_scan_step] %s/%s requests=%d channels=%d dstate=%d\n", dtype_name(d->state_dtype),
                 dtype_name(d->input_dtype), d->num_seqs, d->channels, d->dstate);
  return launch(kernel_for(Q == 2 ? kScanStepTwo : kScanStepOne, d), (d->num_seqs + static_cast<int64_t>(Q) - 1) / Q * a.blocks,
                &a, hip_stream, "selective_scan_step");
}

}  // extern "C"
