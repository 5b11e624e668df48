// engram_layers_api.cpp -- the C entry points of the layers around the gate
// (linear, qk_norm_rope, decay_attn): argument validation on the host, then
// kernel launches on the caller's stream.  Nothing here allocates, copies or
// synchronises.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "engram.h"
#include "engram_check.h"
#include "engram_launch.h"

using engram::aligned16;
using engram::any_overlap;
using engram::flat;
using engram::launched;
using engram::Rows;

namespace {

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

bool ld_in_range(int64_t ld, int64_t width) { return ld >= width && ld <= ENGRAM_LD_MAX; }

bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

// ---- linear ----

bool linear_sizes_ok(int64_t N, int64_t K, int64_t M) {
  return in(N, 1, ENGRAM_LINEAR_ROWS_MAX) && in(K, 8, ENGRAM_LINEAR_WIDTH_MAX) && in(M, 8, ENGRAM_LINEAR_WIDTH_MAX);
}
bool linear_kind_ok(int dtype, int act) {
  return (dtype == ENGRAM_BF16 || dtype == ENGRAM_FP16) && act >= ENGRAM_ACT_NONE && act <= ENGRAM_ACT_GELU;
}

// ---- query/key norm ----

bool qk_sizes_ok(int64_t N, int64_t Hq, int64_t Hk, int64_t D) {
  return in(N, 1, ENGRAM_QK_ROWS_MAX) && in(Hq, 1, ENGRAM_QK_HEADS_MAX) && in(Hk, 1, ENGRAM_QK_HEADS_MAX) &&
         in(D, 8, ENGRAM_QK_D_MAX);
}
int64_t bytes_of(int dtype) { return dtype == ENGRAM_FP32 ? 4 : 2; }

// ---- decay attention ----

bool decay_sizes_ok(int64_t N, int64_t B, int64_t H, int64_t Dk, int64_t Dv) {
  return in(N, 1, ENGRAM_DECAY_ROWS_MAX) && in(H, 1, ENGRAM_DECAY_HEADS_MAX) &&
         in(B, 1, ENGRAM_DECAY_STATES_MAX / H) && in(Dk, 8, ENGRAM_DECAY_D_MAX) && in(Dv, 8, ENGRAM_DECAY_D_MAX);
}
bool decay_dims_ok(int64_t Dk, int64_t Dv) { return Dk % 8 == 0 && Dv % 8 == 0; }

Rows heads(const void* p, int64_t rows, int64_t ld, int64_t H, int64_t D) { return Rows{p, rows, ld * 2, H * D * 2}; }

}  // namespace

extern "C" {

size_t engram_linear_fwd_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  if (!linear_sizes_ok(N, K, M) || K % 8 || M % 8) return 0;
  return engram::linear_fwd_workspace(N, K, M);
}

size_t engram_linear_bwd_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  if (!linear_sizes_ok(N, K, M) || K % 8 || M % 8) return 0;
  return engram::linear_bwd_workspace(N, K, M);
}

engram_status engram_linear_fwd(const void* x, const void* w, const float* bias, const void* residual, void* y, void* z,
                                void* workspace, int64_t N, int64_t K, int64_t M, int64_t ldx, int64_t ldr, int64_t ldy,
                                int64_t ldz, int dtype, int act, void* stream) {
  if (!x || !w || !y) return ENGRAM_ERR_NULL;
  if (!linear_kind_ok(dtype, act)) return ENGRAM_ERR_KIND;
  if (!residual) ldr = M;
  if (!z) ldz = M;
  if (!linear_sizes_ok(N, K, M) || !ld_in_range(ldx, K) || !ld_in_range(ldr, M) || !ld_in_range(ldy, M) ||
      !ld_in_range(ldz, M))
    return ENGRAM_ERR_N_RANGE;
  if ((K | M | ldx | ldr | ldy | ldz) % 8) return ENGRAM_ERR_ALIGN;
  const size_t ws = engram::linear_fwd_workspace(N, K, M);
  if (ws && !workspace) return ENGRAM_ERR_NULL;
  const void* ptrs[] = {x, w, bias, residual, y, z, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const Rows ins[] = {Rows{x, N, ldx * 2, K * 2}, flat(w, M * K * 2), flat(bias, M * 4), Rows{residual, N, ldr * 2, M * 2}};
  const Rows outs[] = {Rows{y, N, ldy * 2, M * 2}, Rows{z, N, ldz * 2, M * 2}, flat(workspace, (int64_t)ws)};
  if (any_overlap(ins, 4, outs, 3)) return ENGRAM_ERR_OVERLAP;
  engram::LinearCall l{};
  l.x = x; l.w = w; l.bias = bias; l.residual = residual; l.y = y; l.z = z; l.workspace = workspace;
  l.N = N; l.K = K; l.M = M; l.ldx = ldx; l.ldr = ldr; l.ldy = ldy; l.ldz = ldz;
  l.dtype = dtype; l.act = act;
  return launched(engram::launch_linear_fwd(l, (hipStream_t)stream));
}

engram_status engram_linear_bwd(const void* grad_y, const void* x, const void* w, const void* z, void* grad_x,
                                void* grad_w, float* grad_bias, void* workspace, int64_t N, int64_t K, int64_t M,
                                int64_t ldgy, int64_t ldx, int64_t ldz, int64_t ldgx, int dtype, int act, void* stream) {
  if (!grad_y || !x || !w || !workspace || (!grad_x && !grad_w && !grad_bias)) return ENGRAM_ERR_NULL;
  if (!linear_kind_ok(dtype, act)) return ENGRAM_ERR_KIND;
  if (act == ENGRAM_ACT_NONE) z = nullptr;
  else if (!z) return ENGRAM_ERR_NULL;
  if (!z) ldz = M;
  if (!grad_x) ldgx = K;
  if (!linear_sizes_ok(N, K, M) || !ld_in_range(ldgy, M) || !ld_in_range(ldx, K) || !ld_in_range(ldz, M) ||
      !ld_in_range(ldgx, K))
    return ENGRAM_ERR_N_RANGE;
  if ((K | M | ldgy | ldx | ldz | ldgx) % 8) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {grad_y, x, w, z, grad_x, grad_w, grad_bias, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const Rows ins[] = {Rows{grad_y, N, ldgy * 2, M * 2}, Rows{x, N, ldx * 2, K * 2}, flat(w, M * K * 2),
                      Rows{z, N, ldz * 2, M * 2}};
  const Rows outs[] = {Rows{grad_x, N, ldgx * 2, K * 2}, flat(grad_w, M * K * 2), flat(grad_bias, M * 4),
                       flat(workspace, (int64_t)engram::linear_bwd_workspace(N, K, M))};
  if (any_overlap(ins, 4, outs, 4)) return ENGRAM_ERR_OVERLAP;
  engram::LinearCall l{};
  l.grad_y = grad_y; l.x = x; l.w = w; l.z_in = z; l.grad_x = grad_x; l.grad_w = grad_w; l.grad_bias = grad_bias;
  l.workspace = workspace;
  l.N = N; l.K = K; l.M = M; l.ldgy = ldgy; l.ldx = ldx; l.ldz = ldz; l.ldgx = ldgx;
  l.dtype = dtype; l.act = act;
  return launched(engram::launch_linear_bwd(l, (hipStream_t)stream));
}

size_t engram_qk_norm_rope_bwd_workspace_bytes(int64_t N, int64_t Hq, int64_t Hk, int64_t D) {
  if (!qk_sizes_ok(N, Hq, Hk, D) || D % 8) return 0;
  return engram::qk_norm_rope_bwd_workspace(D);
}

// What the forward and the backward check alike; R's arrays only where R is not 0.
static engram_status qk_check(const int64_t* positions, const int64_t* freqs, int64_t N, int64_t Hq, int64_t Hk,
                              int64_t D, int64_t R, const int64_t* ldq, int nq, const int64_t* ldk, int nk, float eps,
                              int dtype) {
  if (R != 0 && (!positions || !freqs)) return ENGRAM_ERR_NULL;
  if (dtype < ENGRAM_BF16 || dtype > ENGRAM_FP32) return ENGRAM_ERR_KIND;
  if (!qk_sizes_ok(N, Hq, Hk, D) || !in(R, 0, D) || !(eps >= 0.0f) || eps > 1.0f) return ENGRAM_ERR_N_RANGE;
  for (int i = 0; i < nq; ++i)
    if (!ld_in_range(ldq[i], Hq * D)) return ENGRAM_ERR_N_RANGE;
  for (int i = 0; i < nk; ++i)
    if (!ld_in_range(ldk[i], Hk * D)) return ENGRAM_ERR_N_RANGE;
  if (D % 8 || R % 16) return ENGRAM_ERR_ALIGN;
  for (int i = 0; i < nq; ++i)
    if (ldq[i] % 8) return ENGRAM_ERR_ALIGN;
  for (int i = 0; i < nk; ++i)
    if (ldk[i] % 8) return ENGRAM_ERR_ALIGN;
  if (R != 0 && (!aligned8(positions) || !aligned8(freqs))) return ENGRAM_ERR_ALIGN;
  return ENGRAM_OK;
}

engram_status engram_qk_norm_rope_fwd(const void* q, const void* k, const float* wq, const float* wk,
                                      const int64_t* positions, const int64_t* freqs, void* q_out, void* k_out, int64_t N,
                                      int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t ldq, int64_t ldk,
                                      int64_t ldq_out, int64_t ldk_out, float eps, int interleaved, int dtype,
                                      void* stream) {
  if (!q || !k || !wq || !wk || !q_out || !k_out) return ENGRAM_ERR_NULL;
  const int64_t lq[] = {ldq, ldq_out}, lk[] = {ldk, ldk_out};
  const engram_status st = qk_check(positions, freqs, N, Hq, Hk, D, R, lq, 2, lk, 2, eps, dtype);
  if (st != ENGRAM_OK) return st;
  const void* ptrs[] = {q, k, wq, wk, q_out, k_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t e = bytes_of(dtype), wide_q = Hq * D * e, wide_k = Hk * D * e;
  const Rows ins[] = {Rows{q, N, ldq * e, wide_q}, Rows{k, N, ldk * e, wide_k}, flat(wq, D * 4), flat(wk, D * 4),
                      flat(R ? positions : nullptr, N * 8), flat(R ? freqs : nullptr, R / 2 * 8)};
  const Rows outs[] = {Rows{q_out, N, ldq_out * e, wide_q}, Rows{k_out, N, ldk_out * e, wide_k}};
  if (any_overlap(ins, 6, outs, 2)) return ENGRAM_ERR_OVERLAP;
  engram::QkCall c{};
  c.q = q; c.k = k; c.wq = wq; c.wk = wk; c.positions = positions; c.freqs = freqs; c.q_out = q_out; c.k_out = k_out;
  c.N = N; c.Hq = Hq; c.Hk = Hk; c.D = D; c.R = R;
  c.ldq = ldq; c.ldk = ldk; c.ldq_out = ldq_out; c.ldk_out = ldk_out;
  c.eps = eps; c.interleaved = interleaved != 0; c.dtype = dtype;
  return launched(engram::launch_qk_norm_rope_fwd(c, (hipStream_t)stream));
}

engram_status engram_qk_norm_rope_bwd(const void* grad_q_out, const void* grad_k_out, const void* q, const void* k,
                                      const float* wq, const float* wk, const int64_t* positions, const int64_t* freqs,
                                      void* grad_q, void* grad_k, float* grad_wq, float* grad_wk, void* workspace,
                                      int64_t N, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t ldgq_out,
                                      int64_t ldgk_out, int64_t ldq, int64_t ldk, int64_t ldgq, int64_t ldgk, float eps,
                                      int interleaved, int dtype, void* stream) {
  if (!grad_q_out || !grad_k_out || !q || !k || !wq || !wk || !grad_q || !grad_k || !grad_wq || !grad_wk || !workspace)
    return ENGRAM_ERR_NULL;
  const int64_t lq[] = {ldgq_out, ldq, ldgq}, lk[] = {ldgk_out, ldk, ldgk};
  const engram_status st = qk_check(positions, freqs, N, Hq, Hk, D, R, lq, 3, lk, 3, eps, dtype);
  if (st != ENGRAM_OK) return st;
  const void* ptrs[] = {grad_q_out, grad_k_out, q, k, wq, wk, grad_q, grad_k, grad_wq, grad_wk, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t e = bytes_of(dtype), wide_q = Hq * D * e, wide_k = Hk * D * e;
  const Rows ins[] = {Rows{grad_q_out, N, ldgq_out * e, wide_q}, Rows{grad_k_out, N, ldgk_out * e, wide_k},
                      Rows{q, N, ldq * e, wide_q}, Rows{k, N, ldk * e, wide_k}, flat(wq, D * 4), flat(wk, D * 4),
                      flat(R ? positions : nullptr, N * 8), flat(R ? freqs : nullptr, R / 2 * 8)};
  const Rows outs[] = {Rows{grad_q, N, ldgq * e, wide_q}, Rows{grad_k, N, ldgk * e, wide_k}, flat(grad_wq, D * 4),
                       flat(grad_wk, D * 4), flat(workspace, (int64_t)engram::qk_norm_rope_bwd_workspace(D))};
  if (any_overlap(ins, 8, outs, 5)) return ENGRAM_ERR_OVERLAP;
  engram::QkCall c{};
  c.q = q; c.k = k; c.grad_q_out = grad_q_out; c.grad_k_out = grad_k_out; c.wq = wq; c.wk = wk;
  c.positions = positions; c.freqs = freqs; c.q_out = grad_q; c.k_out = grad_k; c.grad_wq = grad_wq; c.grad_wk = grad_wk;
  c.workspace = workspace;
  c.N = N; c.Hq = Hq; c.Hk = Hk; c.D = D; c.R = R;
  c.ldq = ldq; c.ldk = ldk; c.ldgq = ldgq_out; c.ldgk = ldgk_out; c.ldq_out = ldgq; c.ldk_out = ldgk;
  c.eps = eps; c.interleaved = interleaved != 0; c.dtype = dtype;
  return launched(engram::launch_qk_norm_rope_bwd(c, (hipStream_t)stream));
}

engram_status engram_rope_freqs(double theta, int64_t R, int64_t* freqs) {
  if (!freqs) return ENGRAM_ERR_NULL;
  if (!in(R, 16, ENGRAM_QK_D_MAX) || !(theta > 0.0) || !isfinite(theta)) return ENGRAM_ERR_N_RANGE;
  if (R % 16) return ENGRAM_ERR_ALIGN;
  const long double turn = 2.0L * acosl(-1.0L);
  for (int64_t i = 0; i < R / 2; ++i) {
    // whole turns per position do not matter (theta below 1 makes some)
    const long double f = powl((long double)theta, -2.0L * (long double)i / (long double)R) / turn;
    const long double scaled = rintl((f - floorl(f)) * 18446744073709551616.0L);
    freqs[i] = (int64_t)(scaled >= 18446744073709551616.0L ? 0 : (uint64_t)scaled);
  }
  return ENGRAM_OK;
}

size_t engram_decay_attn_fwd_workspace_bytes(int64_t N, int64_t B, int64_t H, int64_t Dk, int64_t Dv) {
  if (!decay_sizes_ok(N, B, H, Dk, Dv) || !decay_dims_ok(Dk, Dv)) return 0;
  return engram::decay_fwd_workspace(N, H, Dk, Dv);
}

size_t engram_decay_attn_bwd_workspace_bytes(int64_t N, int64_t B, int64_t H, int64_t Dk, int64_t Dv) {
  if (!decay_sizes_ok(N, B, H, Dk, Dv) || !decay_dims_ok(Dk, Dv)) return 0;
  return engram::decay_bwd_workspace(N, H, Dk, Dv);
}

engram_status engram_decay_attn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                                    const int64_t* cu_seqlens, const float* state_in, void* o, float* state_out,
                                    void* workspace, int64_t N, int64_t B, int64_t H, int64_t Dk, int64_t Dv, int64_t ldq,
                                    int64_t ldk, int64_t ldv, int64_t ldo, float scale, void* stream) {
  if (!q || !k || !v || !log_decay || !cu_seqlens || !o || !workspace) return ENGRAM_ERR_NULL;
  if (!decay_sizes_ok(N, B, H, Dk, Dv) || !ld_in_range(ldq, H * Dk) || !ld_in_range(ldk, H * Dk) ||
      !ld_in_range(ldv, H * Dv) || !ld_in_range(ldo, H * Dv) || !isfinite(scale))
    return ENGRAM_ERR_N_RANGE;
  if (!decay_dims_ok(Dk, Dv) || (ldq | ldk | ldv | ldo) % 8 || !aligned8(cu_seqlens)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {q, k, v, log_decay, state_in, o, state_out, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t states = B * H * Dk * Dv * 4;
  const Rows ins[] = {heads(q, N, ldq, H, Dk), heads(k, N, ldk, H, Dk),      heads(v, N, ldv, H, Dv),
                      flat(log_decay, H * 4),  flat(cu_seqlens, (B + 1) * 8), flat(state_in, states)};
  const Rows outs[] = {heads(o, N, ldo, H, Dv), flat(state_out, states),
                       flat(workspace, (int64_t)engram::decay_fwd_workspace(N, H, Dk, Dv))};
  if (any_overlap(ins, 6, outs, 3)) return ENGRAM_ERR_OVERLAP;
  engram::DecayCall d{};
  d.q = static_cast<const uint16_t*>(q); d.k = static_cast<const uint16_t*>(k); d.v = static_cast<const uint16_t*>(v);
  d.log_decay = log_decay; d.cu = cu_seqlens; d.state_in = state_in; d.state_out = state_out;
  d.o = static_cast<uint16_t*>(o); d.workspace = workspace;
  d.N = N; d.B = B; d.H = H; d.Dk = Dk; d.Dv = Dv; d.ldq = ldq; d.ldk = ldk; d.ldv = ldv; d.ldo = ldo; d.scale = scale;
  return launched(engram::launch_decay_fwd(d, (hipStream_t)stream));
}

engram_status engram_decay_attn_bwd(const void* grad_o, const void* q, const void* k, const void* v,
                                    const float* log_decay, const int64_t* cu_seqlens, const float* state_in,
                                    const float* grad_state_out, void* grad_q, void* grad_k, void* grad_v,
                                    float* grad_state_in, void* workspace, int64_t N, int64_t B, int64_t H, int64_t Dk,
                                    int64_t Dv, int64_t ldgo, int64_t ldq, int64_t ldk, int64_t ldv, int64_t ldgq,
                                    int64_t ldgk, int64_t ldgv, float scale, void* stream) {
  if (!grad_o || !q || !k || !v || !log_decay || !cu_seqlens || !grad_q || !grad_k || !grad_v || !workspace)
    return ENGRAM_ERR_NULL;
  if (!decay_sizes_ok(N, B, H, Dk, Dv) || !ld_in_range(ldgo, H * Dv) || !ld_in_range(ldq, H * Dk) ||
      !ld_in_range(ldk, H * Dk) || !ld_in_range(ldv, H * Dv) || !ld_in_range(ldgq, H * Dk) ||
      !ld_in_range(ldgk, H * Dk) || !ld_in_range(ldgv, H * Dv) || !isfinite(scale))
    return ENGRAM_ERR_N_RANGE;
  if (!decay_dims_ok(Dk, Dv) || (ldgo | ldq | ldk | ldv | ldgq | ldgk | ldgv) % 8 || !aligned8(cu_seqlens))
    return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {grad_o, q, k, v, log_decay, state_in, grad_state_out, grad_q, grad_k, grad_v, grad_state_in,
                        workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t states = B * H * Dk * Dv * 4;
  const Rows ins[] = {heads(grad_o, N, ldgo, H, Dv), heads(q, N, ldq, H, Dk), heads(k, N, ldk, H, Dk),
                      heads(v, N, ldv, H, Dv), flat(log_decay, H * 4), flat(cu_seqlens, (B + 1) * 8),
                      flat(state_in, states), flat(grad_state_out, states)};
  const Rows outs[] = {heads(grad_q, N, ldgq, H, Dk), heads(grad_k, N, ldgk, H, Dk), heads(grad_v, N, ldgv, H, Dv),
                       flat(grad_state_in, states),
                       flat(workspace, (int64_t)engram::decay_bwd_workspace(N, H, Dk, Dv))};
  if (any_overlap(ins, 8, outs, 5)) return ENGRAM_ERR_OVERLAP;
  engram::DecayCall d{};
  d.grad_o = static_cast<const uint16_t*>(grad_o);
  d.q = static_cast<const uint16_t*>(q); d.k = static_cast<const uint16_t*>(k); d.v = static_cast<const uint16_t*>(v);
  d.log_decay = log_decay; d.cu = cu_seqlens; d.state_in = state_in; d.grad_state_out = grad_state_out;
  d.grad_q = static_cast<uint16_t*>(grad_q); d.grad_k = static_cast<uint16_t*>(grad_k);
  d.grad_v = static_cast<uint16_t*>(grad_v); d.grad_state_in = grad_state_in; d.workspace = workspace;
  d.N = N; d.B = B; d.H = H; d.Dk = Dk; d.Dv = Dv;
  d.ldgo = ldgo; d.ldq = ldq; d.ldk = ldk; d.ldv = ldv; d.ldgq = ldgq; d.ldgk = ldgk; d.ldgv = ldgv; d.scale = scale;
  return launched(engram::launch_decay_bwd(d, (hipStream_t)stream));
}

engram_status engram_decay_attn_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                                     const int64_t* slots, void* o, int64_t B, int64_t H, int64_t Dk, int64_t Dv,
                                     int64_t slots_total, int64_t ldq, int64_t ldk, int64_t ldv, int64_t ldo, float scale,
                                     void* stream) {
  if (!q || !k || !v || !log_decay || !state || !slots || !o) return ENGRAM_ERR_NULL;
  if (!decay_sizes_ok(1, 1, H, Dk, Dv) || !in(B, 1, ENGRAM_DECAY_STEP_ROWS_MAX) ||
      !in(slots_total, 1, INT64_MAX / (H * Dk * Dv * 4)) || !ld_in_range(ldq, H * Dk) || !ld_in_range(ldk, H * Dk) ||
      !ld_in_range(ldv, H * Dv) || !ld_in_range(ldo, H * Dv) || !isfinite(scale))
    return ENGRAM_ERR_N_RANGE;
  if (!decay_dims_ok(Dk, Dv) || (ldq | ldk | ldv | ldo) % 8 || !aligned8(slots)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {q, k, v, log_decay, state, o};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const Rows ins[] = {heads(q, B, ldq, H, Dk), heads(k, B, ldk, H, Dk), heads(v, B, ldv, H, Dv), flat(log_decay, H * 4),
                      flat(slots, B * 8)};
  const Rows outs[] = {heads(o, B, ldo, H, Dv), flat(state, slots_total * H * Dk * Dv * 4)};
  if (any_overlap(ins, 5, outs, 2)) return ENGRAM_ERR_OVERLAP;
  engram::DecayCall d{};
  d.q = static_cast<const uint16_t*>(q); d.k = static_cast<const uint16_t*>(k); d.v = static_cast<const uint16_t*>(v);
  d.log_decay = log_decay; d.pool = state; d.slots = slots; d.n_slots = slots_total; d.o = static_cast<uint16_t*>(o);
  d.B = B; d.H = H; d.Dk = Dk; d.Dv = Dv; d.ldq = ldq; d.ldk = ldk; d.ldv = ldv; d.ldo = ldo; d.scale = scale;
  return launched(engram::launch_decay_step(d, (hipStream_t)stream));
}

}  // extern "C"
