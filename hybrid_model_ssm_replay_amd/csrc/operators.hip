// Host side of the operators around the recurrence declared in
// include/replayssm.h: argument checks and launches.
#include "internal.h"
#include "ops.h"

using namespace rssm;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool dtype_ok(int d) { return d == REPLAY_DT_F32 || d == REPLAY_DT_BF16; }
size_t elem_size(int d) { return d == REPLAY_DT_BF16 ? 2 : 4; }
bool elem_aligned(const void *p, int d) { return ((uintptr_t)p & (elem_size(d) - 1)) == 0; }
constexpr int kMost = 1 << 30;  // tokens, sequences, channels, vocabulary: indexes a little past them still fit 32 bits
constexpr int kMostRow = 1 << 23;  // values of a token's x, and of its B or C
int hip_status(int e) { return e == 0 ? REPLAY_OK : e == kTooLarge ? REPLAY_EINVAL : REPLAY_EHIP; }

bool prompt_ok(const replay_prompt *p, int batch) {
  return p && p->tokens >= 0 && p->tokens <= kMost && p->sequences >= 1 && p->sequences <= batch &&
         p->sequences <= kMost && p->seq_start;
}

Packed packed_of(const replay_prompt &p, int batch) {
  return Packed{p.tokens, p.sequences, batch, p.seq_start, p.rows, p.resume, p.status};
}

bool conv_ok(const replay_short_conv *c) {
  if (!c || c->channels < 1 || c->taps < 2 || c->taps > 4 || c->batch < 1 || !dtype_ok(c->dtype) || c->reserved)
    return false;
  if (c->silu != 0 && c->silu != 1) return false;
  if (c->channels > kMost || c->batch > kMost || c->slots < c->taps - 1) return false;
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (c->width[i] < 0) return false;
    sum += c->width[i];
  }
  return sum == c->channels && c->weight && c->ring && aligned16(c->weight) && aligned16(c->bias) &&
         elem_aligned(c->ring, c->dtype);
}

// The arguments both convolution calls share; false if an output is missing.
bool conv_args(ShortConvArgs *a, const replay_short_conv &c, const void *x, void *o0, void *o1, void *o2) {
  *a = ShortConvArgs{};
  a->C = c.channels, a->K = c.taps, a->slots = c.slots, a->batch = c.batch, a->dtype = c.dtype, a->silu = c.silu;
  a->weight = c.weight, a->bias = c.bias, a->ring = c.ring, a->pos = c.pos, a->status = c.status;
  a->x = x;
  void *const out[3] = {o0, o1, o2};
  for (int i = 0; i < 3; ++i) {
    a->w[i] = c.width[i], a->out[i] = out[i];
    if (c.width[i] && (!out[i] || !elem_aligned(out[i], c.dtype))) return false;
  }
  return x && elem_aligned(x, c.dtype);
}

bool scan_cfg_ok(const replay_config *c) {
  if (!c || c->kind != REPLAY_KIND_MAMBA2) return false;
  if (c->batch < 1 || c->heads < 1 || c->groups < 1 || c->heads % c->groups) return false;
  if (c->head_dim < 16 || c->head_dim > 128 || c->head_dim % 16) return false;
  if (c->state_dim != 16 && c->state_dim != 32 && c->state_dim != 64 && c->state_dim != 128) return false;
  // The kernel addresses a chunk's 64 rows of up to 4 bytes a value by 32 bits.
  if ((int64_t)c->heads * c->head_dim >= kMostRow || (int64_t)c->groups * c->state_dim >= kMostRow) return false;
  return (int64_t)c->batch * c->heads <= 0x7fffffffLL;
}

bool scan_size_ok(const replay_config *c, int tokens, int sequences) {
  return scan_cfg_ok(c) && tokens >= 0 && tokens <= kMost && sequences >= 1 && sequences <= c->batch && sequences <= kMost;
}

ScanArgs scan_args(const replay_config &c, int tokens, int sequences) {
  ScanArgs a{};
  a.H = c.heads, a.G = c.groups, a.P = c.head_dim, a.N = c.state_dim;
  a.bf16 = (c.flags & REPLAY_FLAG_BF16_RECORDS) ? 1 : 0;
  a.p.tokens = tokens, a.p.n = sequences, a.p.batch = c.batch;
  return a;
}

}  // namespace

extern "C" {

int replay_short_conv_step(const replay_short_conv *conv, const void *x, int64_t seq_stride, int64_t row_stride,
                           int32_t T, void *out0, void *out1, void *out2, void *stream) {
  ShortConvArgs a;
  if (!conv_ok(conv) || !conv->pos || !conv_args(&a, *conv, x, out0, out1, out2)) return REPLAY_EINVAL;
  if (T < 1 || conv->slots - (conv->taps - 1) < T) return REPLAY_EINVAL;
  if (row_stride < 0 || seq_stride < 0) return REPLAY_EINVAL;
  a.seq_stride = seq_stride, a.row_stride = row_stride, a.T = T;
  return hip_status(launch_short_conv_step(a, (hipStream_t)stream));
}

int replay_short_conv_prompt(const replay_short_conv *conv, const replay_prompt *prompt, const void *x,
                             int64_t row_stride, void *out0, void *out1, void *out2, void *stream) {
  ShortConvArgs a;
  if (!conv_ok(conv) || !prompt_ok(prompt, conv->batch)) return REPLAY_EINVAL;
  if (!conv_args(&a, *conv, x, out0, out1, out2) && prompt->tokens > 0) return REPLAY_EINVAL;
  if (row_stride < 0) return REPLAY_EINVAL;
  a.row_stride = row_stride;
  a.p = packed_of(*prompt, conv->batch);
  return hip_status(launch_short_conv_prompt(a, (hipStream_t)stream));
}

size_t replay_scan_workspace_bytes(const replay_config *cfg, int32_t tokens, int32_t sequences) {
  return scan_size_ok(cfg, tokens, sequences) ? scan_workspace(scan_args(*cfg, tokens, sequences)) : 0;
}

int replay_scan_plan(const replay_config *cfg, int32_t tokens, int32_t sequences, replay_scan_layout *layout) {
  if (!scan_size_ok(cfg, tokens, sequences) || !layout) return REPLAY_EINVAL;
  int32_t plan[4];
  scan_plan(scan_args(*cfg, tokens, sequences), plan);
  *layout = replay_scan_layout{plan[0], plan[1], plan[2], plan[3]};
  return REPLAY_OK;
}

int replay_scan_prompt(const replay_config *cfg, const replay_prompt *prompt, const replay_record *rec,
                       const float *A, const float *D, const float *initial, float *state, void *y, int32_t y_dtype,
                       void *workspace, void *stream) {
  if (!scan_cfg_ok(cfg) || !prompt_ok(prompt, cfg->batch)) return REPLAY_EINVAL;
  if (!A || !D || !state || !aligned16(state) || !aligned16(initial) || !dtype_ok(y_dtype)) return REPLAY_EINVAL;
  ScanArgs a = scan_args(*cfg, prompt->tokens, prompt->sequences);
  if (y_dtype == REPLAY_DT_BF16 && !a.bf16) return REPLAY_ENOTSUP;
  if (prompt->tokens > 0) {
    if (!rec || !rec->f0 || !rec->f1 || !rec->f2 || !rec->f3 || !y) return REPLAY_EINVAL;
    if (!aligned16(rec->f0) || !aligned16(rec->f1) || !aligned16(rec->f2) || !aligned16(y)) return REPLAY_EINVAL;
  }
  if (scan_workspace(a) && (!workspace || ((uintptr_t)workspace & 255u))) return REPLAY_EINVAL;
  a.y_bf16 = y_dtype == REPLAY_DT_BF16;
  a.p = packed_of(*prompt, cfg->batch);
  if (rec) a.x = rec->f0, a.Bm = rec->f1, a.Cm = rec->f2, a.dt = rec->f3;
  a.A = A, a.D = D, a.initial = initial, a.state = state, a.y = y, a.workspace = workspace;
  return hip_status(launch_scan(a, (hipStream_t)stream));
}

int replay_gated_norm(const replay_gated_norm_args *a, void *stream) {
  if (!a || a->tokens < 0 || a->tokens > kMost || a->channels < 1 || a->channels > kMost || a->group < 1 ||
      a->channels % a->group || a->reserved)
    return REPLAY_EINVAL;
  if (a->weight_len != a->channels && a->weight_len != a->group) return REPLAY_EINVAL;
  if (!dtype_ok(a->y_dtype) || !dtype_ok(a->z_dtype) || !dtype_ok(a->out_dtype)) return REPLAY_EINVAL;
  if ((a->norm_first != 0 && a->norm_first != 1) || !(a->eps >= 0.f)) return REPLAY_EINVAL;
  if (a->tokens == 0) return REPLAY_OK;
  if (!a->y || !a->z || !a->weight || !a->out) return REPLAY_EINVAL;
  if (!elem_aligned(a->y, a->y_dtype) || !elem_aligned(a->z, a->z_dtype) || !elem_aligned(a->out, a->out_dtype) ||
      !elem_aligned(a->weight, REPLAY_DT_F32))
    return REPLAY_EINVAL;
  if (a->y_stride < 0 || a->z_stride < 0 || (a->tokens > 1 && a->out_stride < a->channels)) return REPLAY_EINVAL;
  return hip_status(launch_gated_norm(*a, (hipStream_t)stream));
}

size_t replay_accept_workspace_bytes(int32_t batch, int32_t vocab) {
  return batch < 1 || vocab < 1 || vocab > kMost ? 0 : accept_workspace(batch, vocab);
}

int replay_accept_drafts(const replay_accept_args *a, void *workspace, void *stream) {
  if (!a || a->batch < 1 || a->vocab < 1 || a->vocab > kMost || a->drafts < 0 || a->drafts > (1 << 20) || a->reserved) return REPLAY_EINVAL;
  if (!dtype_ok(a->target_dtype) || !a->target || !elem_aligned(a->target, a->target_dtype)) return REPLAY_EINVAL;
  if (a->draft && (!dtype_ok(a->draft_dtype) || !elem_aligned(a->draft, a->draft_dtype))) return REPLAY_EINVAL;
  if ((a->drafts && !a->tokens) || !a->uniforms || !a->accepted || !a->next) return REPLAY_EINVAL;
  if (!workspace || !aligned16(workspace)) return REPLAY_EINVAL;
  if (a->target_row_stride < 0 || a->target_seq_stride < 0) return REPLAY_EINVAL;
  if (a->draft && (a->draft_row_stride < 0 || a->draft_seq_stride < 0)) return REPLAY_EINVAL;
  return hip_status(launch_accept(*a, workspace, (hipStream_t)stream));
}

}  // extern "C"
