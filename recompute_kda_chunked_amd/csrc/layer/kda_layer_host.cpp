// Entry points of the operators around the chunked one (include/kda.h):
// validation on the host, then the launches.
#include <cmath>

#include "../kda_host.h"
#include "../kda_internal.h"
#include "kda.h"
#include "kda_layer.h"

using namespace kda;

namespace {

// Largest |L| as for the chunked operator, so that every state it returns
// can be decoded from with the same problem and none it refuses can.
constexpr float kMaxGateBound = 5.9f;

bool known_dtype(int dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }

// A token stride in elements: `row` when 0; otherwise at least a row and,
// with `vec`, a multiple of 16 bytes. A single token's stride is not used.
bool stride_ok(int64_t st, int64_t row, int dtype, int64_t T, bool vec) {
  if (st == 0 || T <= 1) return st >= 0;
  if (st < row) return false;
  return !vec || st % (dtype == KDA_F32 ? 4 : 8) == 0;
}
int64_t stride_of(int64_t st, int64_t row) { return st ? st : row; }

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
  if (static_cast<int64_t>(p->n_seqs) * p->H >= (int64_t{1} << 24)) return KDA_ERR_UNSUPPORTED;
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
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_RECURRENT, a.T * a.H, launch_recurrent(p->dtype, p->K, g2, a, s));
  return KDA_OK;
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

}  // extern "C"
