// Entry points of the operators around the chunked one (include/kda.h):
// validation on the host, then the launches.
#include <cmath>

#include "../kda_host.h"
#include "../kda_internal.h"
#include "kda.h"
#include "kda_checks.h"
#include "kda_layer.h"

using namespace kda;

namespace {

// Largest |L| as for the chunked operator, so that every state it returns
// can be decoded from with the same problem and none it refuses can.
constexpr float kMaxGateBound = 5.9f;

int check_recurrent(const kda_recurrent_problem* p, bool g2, bool has_cu, bool has_idx) {
  if (!p) return KDA_ERR_INVALID;
  if (p->n_seqs < 0 || p->total_tokens < 0 || p->total_tokens > 0x7fffffffLL || p->H < 1 ||
      p->K < 1 || p->V < 1 || p->n_slots < 0 || p->n_slots > 0x7fffffffLL)
    return KDA_ERR_INVALID;
  if (!has_cu && p->total_tokens != p->n_seqs) return KDA_ERR_INVALID;
  if (!has_idx && p->n_slots < p->n_seqs) return KDA_ERR_INVALID;
  if (!(p->gate_lower_bound < 0.f) || !std::isfinite(p->gate_lower_bound)) return KDA_ERR_INVALID;
  if (!(p->l2_eps >= 0.f) || !std::isfinite(p->l2_eps) || !std::isfinite(p->scale))
    return KDA_ERR_INVALID;
  if (!known_dtype(p->dtype)) return KDA_ERR_UNSUPPORTED;
  if (p->gate_lower_bound < -kMaxGateBound) return KDA_ERR_UNSUPPORTED;
  const int gmap = p->gate_mode & ~KDA_GATE_PER_HEAD;
  if (gmap != KDA_GATE_SIGMOID_BOUND && gmap != KDA_GATE_SOFTPLUS_CLAMP) return KDA_ERR_UNSUPPORTED;
  const bool ph = (p->gate_mode & KDA_GATE_PER_HEAD) != 0;
  if (g2 && ph) return KDA_ERR_UNSUPPORTED;
  if (p->K != p->V || (p->K != 64 && p->K != 128)) return KDA_ERR_UNSUPPORTED;
  const int64_t T = p->total_tokens, HK = static_cast<int64_t>(p->H) * p->K;
  if (!stride_ok(p->q_stride, HK, p->dtype, T, true) || !stride_ok(p->k_stride, HK, p->dtype, T, true) ||
      !stride_ok(p->v_stride, HK, p->dtype, T, true) ||
      !stride_ok(p->g_stride, ph ? p->H : HK, p->dtype, T, !ph))
    return KDA_ERR_INVALID;
  if (g2 ? (!stride_ok(p->b_stride, HK, p->dtype, T, true) || !stride_ok(p->w_stride, HK, p->dtype, T, true))
         : !stride_ok(p->beta_stride, p->H, p->dtype, T, false))
    return KDA_ERR_INVALID;
  // one block of 256 threads per (sequence, head), below 2^32 threads
  // in all, at least one of them for the rows that belong to no sequence
  if (static_cast<int64_t>(p->n_seqs) * p->H + (p->zero_rest && has_cu) >= (int64_t{1} << 24))
    return KDA_ERR_UNSUPPORTED;
  if (has_idx && p->n_seqs > kMaxIndexed) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

int recurrent_common(bool g2, const kda_recurrent_problem* p, const void* q, const void* k,
                     const void* v, const void* raw_g, const void* raw_beta, const void* raw_b,
                     const void* raw_w, const float* A_log, const float* dt_bias,
                     const int32_t* cu_seqlens, const int32_t* state_indices, float* state,
                     void* o, void* stream) {
  const int st = check_recurrent(p, g2, cu_seqlens != nullptr, state_indices != nullptr);
  if (st != KDA_OK) return st;
  if (p->n_seqs == 0 || p->total_tokens == 0) return KDA_OK;
  if (!q || !k || !v || !raw_g || !A_log || !dt_bias || !state || !o) return KDA_ERR_INVALID;
  if (g2 ? (!raw_b || !raw_w) : !raw_beta) return KDA_ERR_INVALID;
  const int64_t HK = static_cast<int64_t>(p->H) * p->K;
  RecurrentArgs a{};
  a.N = p->n_seqs;
  a.H = p->H;
  a.T = p->total_tokens;
  a.n_slots = p->n_slots;
  a.scale = p->scale;
  a.lb = p->gate_lower_bound;
  a.eps = p->l2_eps;
  a.gate_mode = p->gate_mode & ~KDA_GATE_PER_HEAD;
  a.gate_head = (p->gate_mode & KDA_GATE_PER_HEAD) ? 1 : 0;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = raw_g;
  a.beta = raw_beta;
  a.bk = raw_b;
  a.wv = raw_w;
  a.qs = stride_of(p->q_stride, HK);
  a.ks = stride_of(p->k_stride, HK);
  a.vs = stride_of(p->v_stride, HK);
  a.gs = stride_of(p->g_stride, a.gate_head ? p->H : HK);
  a.bes = stride_of(p->beta_stride, p->H);
  a.bks = stride_of(p->b_stride, HK);
  a.wvs = stride_of(p->w_stride, HK);
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.cu = cu_seqlens;
  a.idx = state_indices;
  a.state = state;
  a.o = o;
  a.zero_rest = p->zero_rest != 0 && cu_seqlens;
  const size_t e = p->dtype == KDA_F32 ? 4 : 2;
  const int64_t gw = a.gate_head ? p->H : HK;
  const Range others[] = {
      rows_of(q, a.T, a.qs, HK, e),      rows_of(k, a.T, a.ks, HK, e),
      rows_of(v, a.T, a.vs, HK, e),      rows_of(raw_g, a.T, a.gs, gw, e),
      rows_of(raw_beta, a.T, a.bes, p->H, e), rows_of(raw_b, a.T, a.bks, HK, e),
      rows_of(raw_w, a.T, a.wvs, HK, e), dense(A_log, p->H, 1, 4),
      dense(dt_bias, gw, 1, 4),          dense(cu_seqlens, int64_t{a.N} + 1, 1, 4),
      dense(state_indices, a.N, 1, 4),   rows_of(o, a.T, HK, HK, e)};
  if (over_any(dense(state, a.n_slots, HK * p->V, 4), others, sizeof others / sizeof *others))
    return KDA_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_RECURRENT, a.T * a.H, launch_recurrent(p->dtype, p->K, g2, a, s));
  return KDA_OK;
}

int check_gated_norm(const kda_gated_norm_problem* p) {
  if (!p || p->rows < 0 || p->V < 1 || bad_eps(p->eps)) return KDA_ERR_INVALID;
  if (p->rows > (int64_t{1} << 40)) return KDA_ERR_UNSUPPORTED;
  if (!known_dtype(p->dtype) || (p->V != 64 && p->V != 128 && p->V != 256)) return KDA_ERR_UNSUPPORTED;
  if (p->activation != KDA_ACT_SIGMOID && p->activation != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

size_t gated_norm_ws(const kda_gated_norm_problem* p) {
  return static_cast<size_t>(gated_norm_blocks(p->dtype, p->V, p->rows)) * p->V * sizeof(float);
}

int check_block_norm(const kda_block_norm_problem* p) {
  if (!p || p->tokens < 0 || p->D < 1 || bad_eps(p->eps) || !std::isfinite(p->residual_scale))
    return KDA_ERR_INVALID;
  if (p->tokens > (int64_t{1} << 31)) return KDA_ERR_UNSUPPORTED;
  if (!known_dtype(p->dtype) || p->D % 8 != 0 || p->D > 8192) return KDA_ERR_UNSUPPORTED;
  if (p->gate != KDA_BLOCK_GATE_NONE && p->gate != KDA_BLOCK_GATE_TOKEN &&
      p->gate != KDA_BLOCK_GATE_CHANNEL)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// Room for both weights' partial sums, whether or not w_post is given.
size_t block_norm_ws(const kda_block_norm_problem* p) {
  return static_cast<size_t>(block_norm_blocks(p->dtype, p->D, p->tokens)) * 2 * p->D * sizeof(float);
}

int check_short_conv(const kda_short_conv_problem* p) {
  if (!p || p->n_seqs < 0 || p->total_tokens < 0 || p->total_tokens > 0x7fffffffLL || p->C < 1 ||
      p->W < 1)
    return KDA_ERR_INVALID;
  if (!known_dtype(p->dtype) || p->C % 8 != 0 || p->C > (1 << 20) || p->W < 2 || p->W > 4)
    return KDA_ERR_UNSUPPORTED;
  if (p->activation != KDA_ACT_NONE && p->activation != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(p->x_stride, p->C, p->dtype, p->total_tokens, true)) return KDA_ERR_INVALID;
  // token numbers in 32 bits with room for the tokens loaded ahead, and launches
  // below 2^32 threads: a thread per four channels of a state row, 2^30 of them,
  // and a wave per 256 channels of a run; runs of such sizes are of 160 tokens
  // (cover_of), so T * (C / 256 + 1) < 2^32 + 2^31 makes 0.4 * 2^32.6 threads
  if (p->total_tokens > 0x7fffff00LL ||
      static_cast<int64_t>(p->n_seqs) * (p->W - 1) * p->C >= (int64_t{1} << 32) ||
      p->total_tokens * p->C >= (int64_t{1} << 40))
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

size_t short_conv_ws(const kda_short_conv_problem* p) {
  return static_cast<size_t>(short_conv_blocks(p->C, p->total_tokens)) * p->C *
         (p->W + 1) * sizeof(float);
}

ShortConvArgs short_conv_args(const kda_short_conv_problem* p, const void* x, const float* weight,
                              const float* bias, const int32_t* cu) {
  ShortConvArgs a{};
  a.N = p->n_seqs;
  a.C = p->C;
  a.T = p->total_tokens;
  a.xs = stride_of(p->x_stride, p->C);
  a.n_slots = p->n_slots;
  a.act = p->activation;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.cu = cu;
  return a;
}

}  // namespace

extern "C" {

int kda_recurrent(const kda_recurrent_problem* p, const void* q, const void* k, const void* v,
                  const void* raw_g, const void* raw_beta, const float* A_log,
                  const float* dt_bias, const int32_t* cu_seqlens, const int32_t* state_indices,
                  float* state, void* o, void* stream) {
  return recurrent_common(false, p, q, k, v, raw_g, raw_beta, nullptr, nullptr, A_log, dt_bias,
                          cu_seqlens, state_indices, state, o, stream);
}

int kda_gdn2_recurrent(const kda_recurrent_problem* p, const void* q, const void* k,
                       const void* v, const void* raw_g, const void* raw_b, const void* raw_w,
                       const float* A_log, const float* dt_bias, const int32_t* cu_seqlens,
                       const int32_t* state_indices, float* state, void* o, void* stream) {
  return recurrent_common(true, p, q, k, v, raw_g, nullptr, raw_b, raw_w, A_log, dt_bias,
                          cu_seqlens, state_indices, state, o, stream);
}

int kda_gated_norm_fwd(const kda_gated_norm_problem* p, const void* o, const void* gate,
                       const float* weight, void* y, void* stream) {
  const int st = check_gated_norm(p);
  if (st != KDA_OK) return st;
  if (p->rows == 0) return KDA_OK;
  if (!o || !gate || !weight || !y) return KDA_ERR_INVALID;
  GatedNormArgs a{};
  a.rows = p->rows;
  a.act = p->activation;
  a.eps = p->eps;
  a.o = o;
  a.gate = gate;
  a.weight = weight;
  a.y = y;
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_GATED_NORM, p->rows, launch_gated_norm_fwd(p->dtype, p->V, a, s));
  return KDA_OK;
}

size_t kda_gated_norm_bwd_workspace_bytes(const kda_gated_norm_problem* p) {
  return check_gated_norm(p) == KDA_OK ? gated_norm_ws(p) : 0;
}

int kda_gated_norm_bwd(const kda_gated_norm_problem* p, const void* o, const void* gate,
                       const float* weight, const void* dy, void* d_o, void* dgate,
                       float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_gated_norm(p);
  if (st != KDA_OK) return st;
  if (!dweight) return KDA_ERR_INVALID;
  if (p->rows > 0 && (!o || !gate || !weight || !dy || !d_o || !dgate || !workspace))
    return KDA_ERR_INVALID;
  if (workspace_bytes < gated_norm_ws(p)) return KDA_ERR_WORKSPACE;
  GatedNormArgs a{};
  a.rows = p->rows;
  a.act = p->activation;
  a.eps = p->eps;
  a.o = o;
  a.gate = gate;
  a.weight = weight;
  a.dy = dy;
  a.d_o = d_o;
  a.dgate = dgate;
  a.partials = static_cast<float*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p->rows > 0)
    KDA_TRY(KDA_KERNEL_GATED_NORM_BWD, p->rows, launch_gated_norm_bwd(p->dtype, p->V, a, s));
  const ParamReduceArgs r{a.partials, gated_norm_blocks(p->dtype, p->V, p->rows), p->V, 0, dweight,
                          nullptr};
  KDA_TRY(KDA_KERNEL_PARAM_REDUCE, 0, launch_param_reduce(r, s));
  return KDA_OK;
}

int kda_block_norm_fwd(const kda_block_norm_problem* p, const void* x, const void* y,
                       const void* raw_gate, const float* w_post, const float* w_pre,
                       void* x_out, void* h, void* stream) {
  const int st = check_block_norm(p);
  if (st != KDA_OK) return st;
  if (p->tokens == 0) return KDA_OK;
  if (!x || !y || !w_pre || !x_out || !h) return KDA_ERR_INVALID;
  if ((p->gate == KDA_BLOCK_GATE_NONE) != (raw_gate == nullptr)) return KDA_ERR_INVALID;
  BlockNormArgs a{};
  a.T = p->tokens;
  a.D = p->D;
  a.scale = p->residual_scale;
  a.eps = p->eps;
  a.x = x;
  a.y = y;
  a.gate = raw_gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.x_out = x_out;
  a.h = h;
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_BLOCK_NORM, p->tokens, launch_block_norm_fwd(p->dtype, p->gate, a, s));
  return KDA_OK;
}

size_t kda_block_norm_bwd_workspace_bytes(const kda_block_norm_problem* p) {
  return check_block_norm(p) == KDA_OK ? block_norm_ws(p) : 0;
}

int kda_block_norm_bwd(const kda_block_norm_problem* p, const void* x, const void* y,
                       const void* raw_gate, const float* w_post, const float* w_pre,
                       const void* dx_out, const void* dh, void* dx, void* dy, void* dgate,
                       float* dw_post, float* dw_pre, void* workspace, size_t workspace_bytes,
                       void* stream) {
  const int st = check_block_norm(p);
  if (st != KDA_OK) return st;
  if (!dw_pre || (w_post != nullptr && !dw_post)) return KDA_ERR_INVALID;
  if (p->tokens > 0) {
    if (!x || !y || !w_pre || !dx || !dy || !workspace) return KDA_ERR_INVALID;
    if ((p->gate == KDA_BLOCK_GATE_NONE) != (raw_gate == nullptr)) return KDA_ERR_INVALID;
    if (p->gate != KDA_BLOCK_GATE_NONE && !dgate) return KDA_ERR_INVALID;
  }
  if (workspace_bytes < block_norm_ws(p)) return KDA_ERR_WORKSPACE;
  BlockNormArgs a{};
  a.T = p->tokens;
  a.D = p->D;
  a.scale = p->residual_scale;
  a.eps = p->eps;
  a.x = x;
  a.y = y;
  a.gate = raw_gate;
  a.dx_out = dx_out;
  a.dh = dh;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.partials = static_cast<float*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p->tokens > 0)
    KDA_TRY(KDA_KERNEL_BLOCK_NORM_BWD, p->tokens, launch_block_norm_bwd(p->dtype, p->gate, a, s));
  const ParamReduceArgs r = w_post
      ? ParamReduceArgs{a.partials, block_norm_blocks(p->dtype, p->D, p->tokens), p->D, p->D, dw_post, dw_pre}
      : ParamReduceArgs{a.partials, block_norm_blocks(p->dtype, p->D, p->tokens), p->D, 0, dw_pre, nullptr};
  KDA_TRY(KDA_KERNEL_PARAM_REDUCE, 0, launch_param_reduce(r, s));
  return KDA_OK;
}

int kda_short_conv_fwd(const kda_short_conv_problem* p, const void* x, const float* weight,
                       const float* bias, const int32_t* cu_seqlens, const void* initial_state,
                       void* y, void* final_state, void* stream) {
  const int st = check_short_conv(p);
  if (st != KDA_OK) return st;
  if (!cu_seqlens && p->n_seqs != 1) return KDA_ERR_INVALID;
  if (p->total_tokens > 0 && (!x || !weight || !y)) return KDA_ERR_INVALID;
  if (p->total_tokens == 0 && (p->n_seqs == 0 || !final_state)) return KDA_OK;
  ShortConvArgs a = short_conv_args(p, x, weight, bias, cu_seqlens);
  a.init = initial_state;
  a.y = y;
  a.final_state = final_state;
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_SHORT_CONV, a.T, launch_short_conv_fwd(p->dtype, p->W, a, s));
  return KDA_OK;
}

size_t kda_short_conv_bwd_workspace_bytes(const kda_short_conv_problem* p) {
  return check_short_conv(p) == KDA_OK ? short_conv_ws(p) : 0;
}

int kda_short_conv_bwd(const kda_short_conv_problem* p, const void* x, const float* weight,
                       const float* bias, const int32_t* cu_seqlens, const void* initial_state,
                       const void* dy, const void* d_final_state, void* dx, float* dweight,
                       float* dbias, void* d_initial_state, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const int st = check_short_conv(p);
  if (st != KDA_OK) return st;
  if (!cu_seqlens && p->n_seqs != 1) return KDA_ERR_INVALID;
  if (!dweight) return KDA_ERR_INVALID;
  if (p->total_tokens > 0 && (!x || !weight || !dy || !dx || !workspace)) return KDA_ERR_INVALID;
  if (workspace_bytes < short_conv_ws(p)) return KDA_ERR_WORKSPACE;
  ShortConvArgs a = short_conv_args(p, x, weight, bias, cu_seqlens);
  a.init = initial_state;
  a.dy = dy;
  a.dfinal = d_final_state;
  a.dx = dx;
  a.dinit = d_initial_state;
  a.partials = static_cast<float*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.T > 0 || (a.N > 0 && a.dinit))
    KDA_TRY(KDA_KERNEL_SHORT_CONV_BWD, a.T, launch_short_conv_bwd(p->dtype, p->W, a, s));
  const ParamReduceArgs r{a.partials, short_conv_blocks(p->C, a.T), p->C * p->W, p->C,
                          dweight, dbias};
  KDA_TRY(KDA_KERNEL_PARAM_REDUCE, 0, launch_param_reduce(r, s));
  return KDA_OK;
}

int kda_short_conv_update(const kda_short_conv_problem* p, const void* x, const float* weight,
                          const float* bias, const int32_t* cu_seqlens,
                          const int32_t* state_indices, void* state, void* y, void* stream) {
  const int st = check_short_conv(p);
  if (st != KDA_OK) return st;
  if (p->n_slots < 0 || p->n_slots > 0x7fffffffLL) return KDA_ERR_INVALID;
  // a block of 256 threads per sequence and 1024 channels, below 2^32 threads
  // in all, at least one of them for the rows that belong to no sequence
  if (static_cast<int64_t>(p->n_seqs) * ((p->C + 1023) / 1024) + (p->zero_rest && cu_seqlens) >=
      (int64_t{1} << 24))
    return KDA_ERR_UNSUPPORTED;
  if (state_indices && p->n_seqs > kMaxIndexed) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens && p->total_tokens != p->n_seqs) return KDA_ERR_INVALID;
  if (!state_indices && p->n_slots < p->n_seqs) return KDA_ERR_INVALID;
  if (p->n_seqs == 0 || p->total_tokens == 0) return KDA_OK;
  if (!x || !weight || !state || !y) return KDA_ERR_INVALID;
  ShortConvArgs a = short_conv_args(p, x, weight, bias, cu_seqlens);
  a.idx = state_indices;
  a.state = state;
  a.y = y;
  a.zero_rest = p->zero_rest != 0 && cu_seqlens;
  const size_t e = p->dtype == KDA_F32 ? 4 : 2;
  const Range others[] = {rows_of(x, a.T, a.xs, a.C, e),     dense(weight, a.C, p->W, 4),
                          dense(bias, a.C, 1, 4),            dense(cu_seqlens, int64_t{a.N} + 1, 1, 4),
                          dense(state_indices, a.N, 1, 4),   rows_of(y, a.T, a.C, a.C, e)};
  if (over_any(dense(state, a.n_slots, int64_t{a.C} * (p->W - 1), e), others,
               sizeof others / sizeof *others))
    return KDA_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_SHORT_CONV_UPDATE, p->n_seqs, launch_short_conv_update(p->dtype, p->W, a, s));
  return KDA_OK;
}

}  // extern "C"
