// Entry points of a state-space layer's operators (include/kda.h): validation
// on the host, then the launches.
#include <cmath>

#include "../kda_host.h"
#include "kda.h"
#include "kda_checks.h"
#include "kda_layer.h"
#include "kda_ssm.h"

using namespace kda;

namespace {

int check_ssm(const kda_ssm_problem* p) {
  if (!p || p->n_seqs < 0 || p->total_tokens < 0 || p->total_tokens > 0x7fffffffLL || p->H < 1 ||
      p->G < 1 || p->N < 1 || p->P < 1 || p->H % p->G != 0)
    return KDA_ERR_INVALID;
  if (!(p->dt_min >= 0.f) || !(p->dt_max >= p->dt_min) || !std::isfinite(p->dt_min)) return KDA_ERR_INVALID;
  if (!known_dtype(p->dtype) || (p->N != 64 && p->N != 128) || (p->P != 64 && p->P != 128))
    return KDA_ERR_UNSUPPORTED;
  const int64_t T = p->total_tokens, HP = static_cast<int64_t>(p->H) * p->P, GN = static_cast<int64_t>(p->G) * p->N;
  if (!stride_ok(p->x_stride, HP, p->dtype, T, true) || !stride_ok(p->dt_stride, p->H, p->dtype, T, false) ||
      !stride_ok(p->B_stride, GN, p->dtype, T, true) || !stride_ok(p->C_stride, GN, p->dtype, T, true))
    return KDA_ERR_INVALID;
  return KDA_OK;
}

// The scan's launches and its workspace, in parts that start at multiples of 256
// bytes.
struct ScanPlan {
  int Q, sets = 1, seg = 0;
  int64_t slots, whole, seg_slots = 0, long_from;
  size_t steps, state, dstate = 0, local, seg_log, sums = 0, before = 0, ends = 0, cross = 0, partial = 0, param = 0;
  ScanPlan(const kda_ssm_problem* p, bool bwd) {
    Q = ssm_chunk(p->dtype);
    const int64_t T = p->total_tokens, HP = static_cast<int64_t>(p->H) * p->P;
    slots = T / Q + p->n_seqs;
    // A block takes the heads of a group in turn, as many rounds of blocks as fill
    // the chip; the chunks and groups left over are divided by heads, into as many
    // blocks as cost least: rounds times a block's heads and a part of one for its
    // start, and backward the partial sums of dB and dC. Microseconds forward and
    // backward, bf16, N 128, P 64, against a block a unit (both sides in turn, within
    // 1%):
    //   8192 tokens in 1, 48 heads of 1 group   (65 units)   126 / 256   337 / 608
    //   8192 tokens in 3, 48 heads of 1 group   (67 units)   174 / 304   331 / 602
    //   8192 tokens in 1, 64 heads of 8 groups  (520 units)  141 / 141   380 / 376
    //   8192 tokens in 3, 64 heads of 8 groups  (536 units)  154 / 176   364 / 418
    //   4099 tokens in 9, 48 heads of 1 group   (41 units)    64 / 213   168 / 517
    //   1531 tokens in 6, 12 heads of 2 groups  (34 units)    31 / 48     58 / 94
    const int per = p->H / p->G;
    const int64_t units = slots * p->G, round = bwd ? 256 : 512;
    whole = units / round * round;
    double best = 0.0;
    for (int k = 1; k <= per; ++k) {
      const int64_t blocks = (units - whole) * k;
      const double cost = static_cast<double>((blocks + round - 1) / round) * ((per + k - 1) / k + 0.5) +
                          (bwd && k > 1 ? 0.004 * blocks : 0.0);
      if (k == 1 || cost < best) {
        best = cost;
        sets = k;
      }
    }
    // The states of a long sequence in segments, which costs them twice over: where
    // its chunks in turn take longer than that work of the whole launch, 512 blocks
    // at a time, and a launch's start (7 chunks). Measured with N 128, P 64, bf16,
    // forward, one sequence or 4 alike, without and with segments: 8192 tokens x 64
    // heads 293 / 166 us and 142 / 182, x 8 heads 230 / 67 and 78 / 59. The lengths
    // are known on the device, which decides, and every sequence has a slot for a
    // segment: with more than a sequence for four chunks their room would come near
    // the states', and no sequence is divided, also not a long one among short ones,
    // which then takes its chunks in turn. Forward and backward, 8 heads: one of 7500
    // tokens with 15 others (692 tokens) 63 and 103 us, with 16 208 and 250; one of
    // 30000 with 63 others (2768) 125 and 255, with 64 770 and 911.
    const int dirs = bwd ? 2 : 1;
    const int64_t chunks = (T + Q - 1) / Q, chain = dirs * (HP / 64);
    const int64_t want = 512 / chain < 32 ? 512 / chain : 32;
    long_from = chain > 512 ? T : (2 * chunks * chain / 512 + 7) * Q;
    if (T > long_from && 4 * int64_t{p->n_seqs} <= chunks) {
      seg = static_cast<int>((chunks + want - 1) / want);
      if (seg < 4) seg = 4;
      seg_slots = T / (static_cast<int64_t>(seg) * Q) + p->n_seqs;
    }
    auto part = [](int64_t n, size_t size) { return (static_cast<size_t>(n) * size + 255) / 256 * 256; };
    steps = part(slots * p->H * Q, 16);
    state = part(slots * HP * p->N, bwd || p->dtype == KDA_F32 ? 4 : 2);
    local = part(dirs * seg_slots * HP * p->N, 4);
    seg_log = part(dirs * seg_slots * p->H, 4);
    if (bwd) {
      dstate = state;
      sums = steps;
      before = part(slots * p->H * Q, 4);
      ends = part(slots * p->H * 2, 4);
      cross = part(slots * p->H * (Q / 16) * (Q / 16), 4);
      partial = sets > 1 ? part((units - whole) * sets * Q * p->N, 4) : 0;
      param = part(slots * p->H * 3, 4);
    }
  }
  size_t bytes() const {
    return steps + state + dstate + local + seg_log + sums + before + ends + cross + 2 * partial + param;
  }
};

// What the scan's launches can hold: blocks of 512 threads (256 of a state pass),
// below 2^32 threads, some of them for the rows of no sequence; elements of a
// workspace part below 2^40.
int check_scan(const kda_ssm_problem* p, bool has_cu) {
  const int st = check_ssm(p);
  if (st != KDA_OK) return st;
  if (!has_cu && p->n_seqs != 1) return KDA_ERR_INVALID;
  const int64_t T = p->total_tokens, slots = T / 64 + p->n_seqs, H = p->H;
  // rows of a chunk in 32 bits
  constexpr int64_t most = 1 << 22;
  if (H * p->P >= most || int64_t{p->G} * p->N >= most) return KDA_ERR_UNSUPPORTED;
  if (T > 1 && (p->x_stride >= most || p->B_stride >= most || p->C_stride >= most)) return KDA_ERR_UNSUPPORTED;
  if (H > (1 << 20) || slots * H >= (int64_t{1} << 26) || slots * H * p->N * p->P >= (int64_t{1} << 40))
    return KDA_ERR_UNSUPPORTED;
  if (slots * H >= (1 << 23) - 1024 || slots * ((H + 3) / 4) >= (1 << 24) ||
      2 * (slots + 8) * H * (p->P / 64) >= (1 << 24))
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

SsmArgs scan_args(const kda_ssm_problem* p, const ScanPlan& plan, const void* x, const void* raw_dt,
                  const float* A_log, const void* B, const void* C, const float* D,
                  const float* dt_bias, const int32_t* cu, const float* init, void* workspace) {
  SsmArgs a{};
  a.n_seqs = p->n_seqs;
  a.H = p->H;
  a.G = p->G;
  a.P = p->P;
  a.T = p->total_tokens;
  a.slots = plan.slots;
  a.dt_min = p->dt_min;
  a.dt_max = p->dt_max;
  a.x = x;
  a.dt = raw_dt;
  a.B = B;
  a.C = C;
  a.xs = stride_of(p->x_stride, static_cast<int64_t>(p->H) * p->P);
  a.dts = stride_of(p->dt_stride, p->H);
  a.Bs = stride_of(p->B_stride, static_cast<int64_t>(p->G) * p->N);
  a.Cs = stride_of(p->C_stride, static_cast<int64_t>(p->G) * p->N);
  a.A_log = A_log;
  a.D = D;
  a.dt_bias = dt_bias;
  a.cu = cu;
  a.init = init;
  char* w = static_cast<char*>(workspace);
  auto take = [&w](size_t bytes) {
    char* at = w;
    w += bytes;
    return at;
  };
  a.steps = reinterpret_cast<float*>(take(plan.steps));
  a.S = take(plan.state);
  a.dS = take(plan.dstate);
  a.S_full = plan.dstate > 0;
  a.local = reinterpret_cast<float*>(take(plan.local));
  a.seg_log = reinterpret_cast<float*>(take(plan.seg_log));
  a.sums = reinterpret_cast<float*>(take(plan.sums));
  a.before = reinterpret_cast<float*>(take(plan.before));
  a.ends = reinterpret_cast<float*>(take(plan.ends));
  a.cross = reinterpret_cast<float*>(take(plan.cross));
  a.pB = reinterpret_cast<float*>(take(plan.partial));
  a.pC = reinterpret_cast<float*>(take(plan.partial));
  a.param = reinterpret_cast<float*>(take(plan.param));
  a.seg = plan.seg;
  a.long_from = plan.long_from;
  a.seg_slots = plan.seg_slots;
  a.whole = static_cast<unsigned>(plan.whole);
  a.sets = plan.sets;
  return a;
}

int check_group_norm(const kda_group_norm_problem* p) {
  if (!p || p->rows < 0 || p->C < 1 || p->groups < 1 || p->C % p->groups != 0 || bad_eps(p->eps))
    return KDA_ERR_INVALID;
  if (p->rows > (int64_t{1} << 31) || p->C > (1 << 20)) return KDA_ERR_UNSUPPORTED;
  const int W = p->C / p->groups;
  if (!known_dtype(p->dtype) || W % 8 != 0 || W > 8192) return KDA_ERR_UNSUPPORTED;
  if (p->gate != KDA_GROUP_GATE_NONE && p->gate != KDA_GROUP_GATE_AFTER && p->gate != KDA_GROUP_GATE_FIRST)
    return KDA_ERR_UNSUPPORTED;
  if (p->activation != KDA_ACT_SIGMOID && p->activation != KDA_ACT_SILU &&
      !(p->activation == KDA_ACT_NONE && p->gate == KDA_GROUP_GATE_NONE))
    return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(p->x_stride, p->C, p->dtype, p->rows, true) ||
      !stride_ok(p->gate_stride, p->C, p->dtype, p->rows, true))
    return KDA_ERR_INVALID;
  return KDA_OK;
}

// Room for both parameters' partial sums, whether or not the bias's are wanted.
size_t group_norm_ws(const kda_group_norm_problem* p) {
  return static_cast<size_t>(group_norm_partials(p->dtype, p->C, p->groups, p->rows)) * 2 * p->C * sizeof(float);
}

GroupNormArgs group_norm_args(const kda_group_norm_problem* p, const void* x, const void* gate,
                              const float* weight, const float* bias) {
  GroupNormArgs a{};
  a.rows = p->rows;
  a.xs = stride_of(p->x_stride, p->C);
  a.gs = stride_of(p->gate_stride, p->C);
  a.C = p->C;
  a.groups = p->groups;
  a.W = p->C / p->groups;
  a.act = p->activation;
  a.center = p->center != 0;
  a.eps = p->eps;
  a.x = x;
  a.gate = gate;
  a.weight = weight;
  a.bias = bias;
  return a;
}

}  // namespace

extern "C" {

size_t kda_ssm_fwd_workspace_bytes(const kda_ssm_problem* p) {
  return check_scan(p, true) == KDA_OK ? ScanPlan(p, false).bytes() : 0;
}

int kda_ssm_fwd(const kda_ssm_problem* p, const void* x, const void* raw_dt, const float* A_log,
                const void* B, const void* C, const float* D, const float* dt_bias,
                const int32_t* cu_seqlens, const float* initial_state, void* y,
                float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_scan(p, cu_seqlens != nullptr);
  if (st != KDA_OK) return st;
  if (p->total_tokens > 0 && (!x || !raw_dt || !A_log || !B || !C || !y)) return KDA_ERR_INVALID;
  const ScanPlan plan(p, false);
  if (plan.bytes() > 0 && !workspace) return KDA_ERR_INVALID;
  if (workspace_bytes < plan.bytes()) return KDA_ERR_WORKSPACE;
  SsmArgs a = scan_args(p, plan, x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, initial_state, workspace);
  a.y = y;
  a.final_state = final_state;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t units = a.T * a.H;
  if (a.T > 0 && a.n_seqs > 0) KDA_TRY(KDA_KERNEL_SSM_STEPS, units, launch_ssm_steps(p->dtype, a, s));
  if (a.n_seqs > 0 && (a.T > 0 || final_state))
    KDA_TRY(KDA_KERNEL_SSM_STATE, units, launch_ssm_state(p->dtype, p->N, 1, 0, a, s));
  if (a.T > 0) KDA_TRY(KDA_KERNEL_SSM_OUT, units, launch_ssm_out(p->dtype, p->N, a, s));
  return KDA_OK;
}

size_t kda_ssm_bwd_workspace_bytes(const kda_ssm_problem* p) {
  return check_scan(p, true) == KDA_OK ? ScanPlan(p, true).bytes() : 0;
}

int kda_ssm_bwd(const kda_ssm_problem* p, const void* x, const void* raw_dt, const float* A_log,
                const void* B, const void* C, const float* D, const float* dt_bias,
                const int32_t* cu_seqlens, const float* initial_state, const void* dy,
                const float* d_final_state, void* dx, void* draw_dt, float* dA_log, void* dB,
                void* dC, float* dD, float* ddt_bias, float* d_initial_state, void* workspace,
                size_t workspace_bytes, void* stream) {
  const int st = check_scan(p, cu_seqlens != nullptr);
  if (st != KDA_OK) return st;
  if (!dA_log) return KDA_ERR_INVALID;
  if (p->total_tokens > 0 && (!x || !raw_dt || !A_log || !B || !C || !dy || !dx || !draw_dt || !dB || !dC))
    return KDA_ERR_INVALID;
  const ScanPlan plan(p, true);
  if (plan.bytes() > 0 && !workspace) return KDA_ERR_INVALID;
  if (workspace_bytes < plan.bytes()) return KDA_ERR_WORKSPACE;
  SsmArgs a = scan_args(p, plan, x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, initial_state, workspace);
  a.dy = dy;
  a.dfinal = d_final_state;
  a.dx = dx;
  a.ddt = draw_dt;
  a.dB = dB;
  a.dC = dC;
  a.dinit = d_initial_state;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t units = a.T * a.H;
  if (a.T > 0 && a.n_seqs > 0) {
    KDA_TRY(KDA_KERNEL_SSM_STEPS, units, launch_ssm_steps(p->dtype, a, s));
    KDA_TRY(KDA_KERNEL_SSM_STATE, units, launch_ssm_state(p->dtype, p->N, 2, 0, a, s));
  } else if (a.n_seqs > 0 && d_initial_state) {  // empty sequences only
    KDA_TRY(KDA_KERNEL_SSM_STATE, units, launch_ssm_state(p->dtype, p->N, 1, 1, a, s));
  }
  if (a.T > 0) {
    KDA_TRY(KDA_KERNEL_SSM_GRAD, units, launch_ssm_grad(p->dtype, p->N, a, s));
    // no sequences and less than a chunk of tokens: no slot
    if (a.slots > 0) KDA_TRY(KDA_KERNEL_SSM_GRAD, units, launch_ssm_scalars(p->dtype, a, s));
    if (a.sets > 1 && plan.whole < a.slots * a.G)
      KDA_TRY(KDA_KERNEL_SSM_REDUCE, a.T, launch_ssm_reduce(p->dtype, p->N, a, s));
  }
  // without tokens the sums are empty
  const int64_t nb = a.T > 0 ? a.slots : 0;
  const ParamReduceArgs r{a.param, nb, p->H, p->H, dA_log, ddt_bias, p->H, dD};
  KDA_TRY(KDA_KERNEL_PARAM_REDUCE, 0, launch_param_reduce(r, s));
  return KDA_OK;
}

int kda_ssm_recurrent(const kda_ssm_problem* p, const void* x, const void* raw_dt,
                      const float* A_log, const void* B, const void* C, const float* D,
                      const float* dt_bias, const int32_t* cu_seqlens,
                      const int32_t* state_indices, float* state, void* y, void* stream) {
  const int st = check_ssm(p);
  if (st != KDA_OK) return st;
  if (p->n_slots < 0 || p->n_slots > 0x7fffffffLL) return KDA_ERR_INVALID;
  if (!cu_seqlens && p->total_tokens != p->n_seqs) return KDA_ERR_INVALID;
  if (!state_indices && p->n_slots < p->n_seqs) return KDA_ERR_INVALID;
  // one block of 256 threads per (sequence, head), below 2^32 threads
  // in all, at least one of them for the rows that belong to no sequence
  if (static_cast<int64_t>(p->n_seqs) * p->H + (p->zero_rest && cu_seqlens) >= (int64_t{1} << 24))
    return KDA_ERR_UNSUPPORTED;
  if (state_indices && p->n_seqs > kMaxIndexed) return KDA_ERR_UNSUPPORTED;
  if (p->n_seqs == 0 || p->total_tokens == 0) return KDA_OK;
  if (!x || !raw_dt || !A_log || !B || !C || !state || !y) return KDA_ERR_INVALID;
  const int64_t HP = static_cast<int64_t>(p->H) * p->P, GN = static_cast<int64_t>(p->G) * p->N;
  SsmStepArgs a{};
  a.n_seqs = p->n_seqs;
  a.H = p->H;
  a.G = p->G;
  a.T = p->total_tokens;
  a.n_slots = p->n_slots;
  a.dt_min = p->dt_min;
  a.dt_max = p->dt_max;
  a.x = x;
  a.dt = raw_dt;
  a.B = B;
  a.C = C;
  a.xs = stride_of(p->x_stride, HP);
  a.dts = stride_of(p->dt_stride, p->H);
  a.Bs = stride_of(p->B_stride, GN);
  a.Cs = stride_of(p->C_stride, GN);
  a.A_log = A_log;
  a.D = D;
  a.dt_bias = dt_bias;
  a.cu = cu_seqlens;
  a.idx = state_indices;
  a.state = state;
  a.y = y;
  a.zero_rest = p->zero_rest != 0 && cu_seqlens;
  const size_t e = p->dtype == KDA_F32 ? 4 : 2;
  const Range others[] = {
      rows_of(x, a.T, a.xs, HP, e),        rows_of(raw_dt, a.T, a.dts, p->H, e),
      rows_of(B, a.T, a.Bs, GN, e),        rows_of(C, a.T, a.Cs, GN, e),
      dense(A_log, p->H, 1, 4),            dense(D, p->H, 1, 4),
      dense(dt_bias, p->H, 1, 4),          dense(cu_seqlens, int64_t{a.n_seqs} + 1, 1, 4),
      dense(state_indices, a.n_seqs, 1, 4), rows_of(y, a.T, HP, HP, e)};
  if (over_any(dense(state, a.n_slots, HP * p->N, 4), others, sizeof others / sizeof *others))
    return KDA_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_SSM_RECURRENT, a.T * a.H, launch_ssm_recurrent(p->dtype, p->N, p->P, a, s));
  return KDA_OK;
}

int kda_group_norm_fwd(const kda_group_norm_problem* p, const void* x, const void* gate,
                       const float* weight, const float* bias, void* y, void* stream) {
  const int st = check_group_norm(p);
  if (st != KDA_OK) return st;
  if (p->rows == 0) return KDA_OK;
  if (!x || !weight || !y) return KDA_ERR_INVALID;
  if ((p->gate == KDA_GROUP_GATE_NONE) != (gate == nullptr)) return KDA_ERR_INVALID;
  GroupNormArgs a = group_norm_args(p, x, gate, weight, bias);
  a.y = y;
  hipStream_t s = static_cast<hipStream_t>(stream);
  KDA_TRY(KDA_KERNEL_GROUP_NORM, p->rows, launch_group_norm_fwd(p->dtype, p->gate, a, s));
  return KDA_OK;
}

size_t kda_group_norm_bwd_workspace_bytes(const kda_group_norm_problem* p) {
  return check_group_norm(p) == KDA_OK ? group_norm_ws(p) : 0;
}

int kda_group_norm_bwd(const kda_group_norm_problem* p, const void* x, const void* gate,
                       const float* weight, const float* bias, const void* dy, void* dx,
                       void* dgate, float* dweight, float* dbias, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const int st = check_group_norm(p);
  if (st != KDA_OK) return st;
  if (!dweight) return KDA_ERR_INVALID;
  if (p->rows > 0) {
    if (!x || !weight || !dy || !dx || !workspace) return KDA_ERR_INVALID;
    if ((p->gate == KDA_GROUP_GATE_NONE) != (gate == nullptr)) return KDA_ERR_INVALID;
    if (gate && !dgate) return KDA_ERR_INVALID;
  }
  if (workspace_bytes < group_norm_ws(p)) return KDA_ERR_WORKSPACE;
  GroupNormArgs a = group_norm_args(p, x, gate, weight, bias);
  a.dy = dy;
  a.dx = dx;
  a.dgate = dgate;
  a.dbias = dbias != nullptr;
  a.partials = static_cast<float*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p->rows > 0)
    KDA_TRY(KDA_KERNEL_GROUP_NORM_BWD, p->rows, launch_group_norm_bwd(p->dtype, p->gate, a, s));
  const int64_t nb = group_norm_partials(p->dtype, p->C, p->groups, p->rows);
  const ParamReduceArgs r{a.partials, nb, p->C, dbias ? p->C : 0, dweight, dbias};
  KDA_TRY(KDA_KERNEL_PARAM_REDUCE, 0, launch_param_reduce(r, s));
  return KDA_OK;
}

}  // extern "C"
