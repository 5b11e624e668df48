// engram_block_api.cpp -- the C entry points of the rest of a block around the
// gate (layer_norm, window_attn, gated_scan): argument validation on the host, then kernel
// launches on the caller's stream.  Nothing here allocates, copies or
// synchronises.
#include <hip/hip_runtime.h>

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

bool float_kind_ok(int dtype) { return dtype >= ENGRAM_BF16 && dtype <= ENGRAM_FP32; }
int64_t bytes_of(int dtype) { return dtype == ENGRAM_FP32 ? 4 : 2; }

bool norm_sizes_ok(int64_t N, int64_t D) { return in(N, 1, ENGRAM_NORM_ROWS_MAX) && in(D, 8, ENGRAM_NORM_D_MAX); }

bool half_kind_ok(int dtype) { return dtype == ENGRAM_BF16 || dtype == ENGRAM_FP16; }

bool window_sizes_ok(int64_t N, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t window, int64_t sinks) {
  return in(N, 1, ENGRAM_WINDOW_ROWS_MAX) && in(Hq, 1, ENGRAM_WINDOW_HEADS_MAX) && in(Hk, 1, Hq) && Hq % Hk == 0 &&
         N <= ENGRAM_WINDOW_HEAD_ROWS_MAX / Hq && in(B, 1, ENGRAM_WINDOW_SEQ_HEADS_MAX / Hk) &&
         in(D, 8, ENGRAM_WINDOW_D_MAX) && window >= 1 && in(sinks, 0, ENGRAM_WINDOW_SINKS_MAX);
}
bool step_sizes_ok(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t capacity) {
  return window_sizes_ok(1, 1, Hq, Hk, D, 1, 0) && in(B, 1, ENGRAM_WINDOW_STEP_ROWS_MAX) &&
         in(capacity, 1, ENGRAM_WINDOW_CAPACITY_MAX);
}
// (the kernels' exponents are of 2: with scale log2(e) infinite a score of 0 would be NaN)
bool scale_ok(float scale) { return scale > 0.0f && scale <= 0x1p126f; }

Rows heads(const void* p, int64_t rows, int64_t ld, int64_t H, int64_t D) { return Rows{p, rows, ld * 2, H * D * 2}; }

bool scan_sizes_ok(int64_t N, int64_t B, int64_t D) {
  return in(N, 1, ENGRAM_SCAN_ROWS_MAX) && in(B, 1, ENGRAM_SCAN_STATES_MAX) && in(D, 8, ENGRAM_SCAN_D_MAX) &&
         N <= ENGRAM_SCAN_VALUES_MAX / D;
}
size_t scan_workspace_bytes(int64_t N, int64_t B, int64_t D) {
  return scan_sizes_ok(N, B, D) && D % 8 == 0 ? engram::scan_workspace(N, D) : 0;
}

}  // namespace

extern "C" {

size_t engram_layer_norm_bwd_workspace_bytes(int64_t N, int64_t D) {
  if (!norm_sizes_ok(N, D) || D % 8) return 0;
  return engram::layer_norm_bwd_workspace(N, D);
}

engram_status engram_layer_norm_fwd(const void* x, const float* w, const float* b, void* y, float* saved, int64_t N,
                                    int64_t D, int64_t ldx, int64_t ldy, float eps, int dtype, void* stream) {
  if (!x || !w || !y) return ENGRAM_ERR_NULL;
  if (!float_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!norm_sizes_ok(N, D) || !ld_in_range(ldx, D) || !ld_in_range(ldy, D) || !(eps >= 0.0f) || eps > 1.0f)
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldx | ldy) % 8) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {x, w, b, y, saved};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t e = bytes_of(dtype);
  const Rows ins[] = {Rows{x, N, ldx * e, D * e}, flat(w, D * 4), flat(b, D * 4)};
  const Rows outs[] = {Rows{y, N, ldy * e, D * e}, flat(saved, N * 8)};
  if (any_overlap(ins, 3, outs, 2)) return ENGRAM_ERR_OVERLAP;
  engram::NormCall c{};
  c.x = x; c.w = w; c.b = b; c.y = y; c.saved = saved;
  c.N = N; c.D = D; c.ldx = ldx; c.ldy = ldy; c.eps = eps; c.dtype = dtype;
  return launched(engram::launch_layer_norm_fwd(c, (hipStream_t)stream));
}

engram_status engram_layer_norm_bwd(const void* grad_y, const void* x, const float* w, const float* saved,
                                    const void* grad_residual, void* grad_x, float* grad_w, float* grad_b,
                                    void* workspace, int64_t N, int64_t D, int64_t ldgy, int64_t ldx, int64_t ldgr,
                                    int64_t ldgx, int dtype, void* stream) {
  if (!grad_y || !x || !w || !saved || !grad_x || !workspace) return ENGRAM_ERR_NULL;
  if (!float_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!grad_residual) ldgr = D;
  if (!norm_sizes_ok(N, D) || !ld_in_range(ldgy, D) || !ld_in_range(ldx, D) || !ld_in_range(ldgr, D) ||
      !ld_in_range(ldgx, D))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldgy | ldx | ldgr | ldgx) % 8) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {grad_y, x, w, saved, grad_residual, grad_x, grad_w, grad_b, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t e = bytes_of(dtype);
  const Rows ins[] = {Rows{grad_y, N, ldgy * e, D * e}, Rows{x, N, ldx * e, D * e}, flat(w, D * 4), flat(saved, N * 8),
                      Rows{grad_residual, N, ldgr * e, D * e}};
  const Rows outs[] = {Rows{grad_x, N, ldgx * e, D * e}, flat(grad_w, D * 4), flat(grad_b, D * 4),
                       flat(workspace, (int64_t)engram::layer_norm_bwd_workspace(N, D))};
  if (any_overlap(ins, 5, outs, 4)) return ENGRAM_ERR_OVERLAP;
  engram::NormCall c{};
  c.grad_y = grad_y; c.x = x; c.w = w; c.saved = const_cast<float*>(saved); c.grad_residual = grad_residual;
  c.grad_x = grad_x; c.grad_w = grad_w; c.grad_b = grad_b; c.workspace = workspace;
  c.N = N; c.D = D; c.ldgy = ldgy; c.ldx = ldx; c.ldgr = ldgr; c.ldgx = ldgx; c.dtype = dtype;
  return launched(engram::launch_layer_norm_bwd(c, (hipStream_t)stream));
}

size_t engram_window_attn_bwd_workspace_bytes(int64_t N, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t window,
                                              int64_t sinks) {
  if (!window_sizes_ok(N, B, Hq, Hk, D, window, sinks) || D % 8) return 0;
  return engram::window_bwd_workspace(N, B, Hq, Hk, D, window, sinks);
}

engram_status engram_window_attn_fwd(const void* q, const void* k, const void* v, const int64_t* cu_seqlens, void* o,
                                     float* lse, int64_t N, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t window,
                                     int64_t sinks, int64_t ldq, int64_t ldk, int64_t ldv, int64_t ldo, float scale,
                                     int dtype, void* stream) {
  if (!q || !k || !v || !cu_seqlens || !o) return ENGRAM_ERR_NULL;
  if (!half_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!window_sizes_ok(N, B, Hq, Hk, D, window, sinks) || !ld_in_range(ldq, Hq * D) || !ld_in_range(ldk, Hk * D) ||
      !ld_in_range(ldv, Hk * D) || !ld_in_range(ldo, Hq * D) || !scale_ok(scale))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldq | ldk | ldv | ldo) % 8 || !aligned8(cu_seqlens)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {q, k, v, o, lse};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const Rows ins[] = {heads(q, N, ldq, Hq, D), heads(k, N, ldk, Hk, D), heads(v, N, ldv, Hk, D),
                      flat(cu_seqlens, (B + 1) * 8)};
  const Rows outs[] = {heads(o, N, ldo, Hq, D), flat(lse, N * Hq * 4)};
  if (any_overlap(ins, 4, outs, 2)) return ENGRAM_ERR_OVERLAP;
  engram::WindowCall w{};
  w.q = static_cast<const uint16_t*>(q); w.k = static_cast<const uint16_t*>(k); w.v = static_cast<const uint16_t*>(v);
  w.cu = cu_seqlens; w.o = static_cast<uint16_t*>(o); w.lse = lse;
  w.N = N; w.B = B; w.Hq = Hq; w.Hk = Hk; w.D = D; w.window = window; w.sinks = sinks;
  w.ldq = ldq; w.ldk = ldk; w.ldv = ldv; w.ldo = ldo; w.scale = scale; w.dtype = dtype;
  return launched(engram::launch_window_fwd(w, (hipStream_t)stream));
}

engram_status engram_window_attn_bwd(const void* grad_o, const void* q, const void* k, const void* v, const void* o,
                                     const float* lse, const int64_t* cu_seqlens, void* grad_q, void* grad_k,
                                     void* grad_v, void* workspace, int64_t N, int64_t B, int64_t Hq, int64_t Hk,
                                     int64_t D, int64_t window, int64_t sinks, int64_t ldgo, int64_t ldq, int64_t ldk,
                                     int64_t ldv, int64_t ldo, int64_t ldgq, int64_t ldgk, int64_t ldgv, float scale,
                                     int dtype, void* stream) {
  if (!grad_o || !q || !k || !v || !o || !lse || !cu_seqlens || !grad_q || !grad_k || !grad_v || !workspace)
    return ENGRAM_ERR_NULL;
  if (!half_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!window_sizes_ok(N, B, Hq, Hk, D, window, sinks) || !ld_in_range(ldgo, Hq * D) || !ld_in_range(ldq, Hq * D) ||
      !ld_in_range(ldk, Hk * D) || !ld_in_range(ldv, Hk * D) || !ld_in_range(ldo, Hq * D) || !ld_in_range(ldgq, Hq * D) ||
      !ld_in_range(ldgk, Hk * D) || !ld_in_range(ldgv, Hk * D) || !scale_ok(scale))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldgo | ldq | ldk | ldv | ldo | ldgq | ldgk | ldgv) % 8 || !aligned8(cu_seqlens)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {grad_o, q, k, v, o, lse, grad_q, grad_k, grad_v, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const Rows ins[] = {heads(grad_o, N, ldgo, Hq, D), heads(q, N, ldq, Hq, D), heads(k, N, ldk, Hk, D),
                      heads(v, N, ldv, Hk, D), heads(o, N, ldo, Hq, D), flat(lse, N * Hq * 4),
                      flat(cu_seqlens, (B + 1) * 8)};
  const Rows outs[] = {heads(grad_q, N, ldgq, Hq, D), heads(grad_k, N, ldgk, Hk, D), heads(grad_v, N, ldgv, Hk, D),
                       flat(workspace, (int64_t)engram::window_bwd_workspace(N, B, Hq, Hk, D, window, sinks))};
  if (any_overlap(ins, 7, outs, 4)) return ENGRAM_ERR_OVERLAP;
  engram::WindowCall w{};
  w.grad_o = static_cast<const uint16_t*>(grad_o); w.q = static_cast<const uint16_t*>(q);
  w.k = static_cast<const uint16_t*>(k); w.v = static_cast<const uint16_t*>(v); w.o_in = static_cast<const uint16_t*>(o);
  w.lse_in = lse; w.cu = cu_seqlens; w.grad_q = static_cast<uint16_t*>(grad_q);
  w.grad_k = static_cast<uint16_t*>(grad_k); w.grad_v = static_cast<uint16_t*>(grad_v); w.workspace = workspace;
  w.N = N; w.B = B; w.Hq = Hq; w.Hk = Hk; w.D = D; w.window = window; w.sinks = sinks;
  w.ldgo = ldgo; w.ldq = ldq; w.ldk = ldk; w.ldv = ldv; w.ldo = ldo; w.ldgq = ldgq; w.ldgk = ldgk; w.ldgv = ldgv;
  w.scale = scale; w.dtype = dtype;
  return launched(engram::launch_window_bwd(w, (hipStream_t)stream));
}

size_t engram_window_attn_step_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t capacity) {
  if (!step_sizes_ok(B, Hq, Hk, D, capacity) || D % 8) return 0;
  return engram::window_step_workspace(B, Hq, Hk, D, capacity);
}

engram_status engram_window_attn_step(const void* q, const void* k, const void* v, void* cache_k, void* cache_v,
                                      const int64_t* slots, const int64_t* positions, void* o, void* workspace, int64_t B,
                                      int64_t Hq, int64_t Hk, int64_t D, int64_t slots_total, int64_t capacity,
                                      int64_t window, int64_t sinks, int64_t ldq, int64_t ldk, int64_t ldv, int64_t ldo,
                                      float scale, int dtype, void* stream) {
  if (!q || !k || !v || !cache_k || !cache_v || !slots || !positions || !o) return ENGRAM_ERR_NULL;
  if (!half_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!step_sizes_ok(B, Hq, Hk, D, capacity) || !in(sinks, 0, ENGRAM_WINDOW_SINKS_MAX) || !in(window, 1, capacity - sinks) ||
      !in(slots_total, 1, INT64_MAX / (Hk * capacity * D * 2)) || !ld_in_range(ldq, Hq * D) || !ld_in_range(ldk, Hk * D) ||
      !ld_in_range(ldv, Hk * D) || !ld_in_range(ldo, Hq * D) || !scale_ok(scale))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldq | ldk | ldv | ldo) % 8 || !aligned8(slots) || !aligned8(positions)) return ENGRAM_ERR_ALIGN;
  const size_t ws = engram::window_step_workspace(B, Hq, Hk, D, capacity);
  if (ws && !workspace) return ENGRAM_ERR_NULL;
  const void* ptrs[] = {q, k, v, cache_k, cache_v, o, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t pool = slots_total * Hk * capacity * D * 2;
  const Rows ins[] = {heads(q, B, ldq, Hq, D), heads(k, B, ldk, Hk, D), heads(v, B, ldv, Hk, D), flat(slots, B * 8),
                      flat(positions, B * 8)};
  const Rows outs[] = {flat(cache_k, pool), flat(cache_v, pool), heads(o, B, ldo, Hq, D), flat(workspace, (int64_t)ws)};
  if (any_overlap(ins, 5, outs, 4)) return ENGRAM_ERR_OVERLAP;
  engram::WindowStepCall w{};
  w.q = static_cast<const uint16_t*>(q); w.k = static_cast<const uint16_t*>(k); w.v = static_cast<const uint16_t*>(v);
  w.cache_k = static_cast<uint16_t*>(cache_k); w.cache_v = static_cast<uint16_t*>(cache_v);
  w.slots = slots; w.positions = positions; w.o = static_cast<uint16_t*>(o); w.workspace = workspace;
  w.B = B; w.Hq = Hq; w.Hk = Hk; w.D = D; w.n_slots = slots_total; w.capacity = capacity; w.window = window; w.sinks = sinks;
  w.ldq = ldq; w.ldk = ldk; w.ldv = ldv; w.ldo = ldo; w.scale = scale; w.dtype = dtype;
  return launched(engram::launch_window_step(w, (hipStream_t)stream));
}

engram_status engram_window_cache_fill(const void* k, const void* v, const int64_t* cu_seqlens, const int64_t* slots,
                                       void* cache_k, void* cache_v, int64_t N, int64_t B, int64_t Hk, int64_t D,
                                       int64_t slots_total, int64_t capacity, int64_t sinks, int64_t ldk, int64_t ldv,
                                       int dtype, void* stream) {
  if (!k || !v || !cu_seqlens || !slots || !cache_k || !cache_v) return ENGRAM_ERR_NULL;
  if (!half_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!in(N, 1, ENGRAM_WINDOW_ROWS_MAX) || !step_sizes_ok(B, Hk, Hk, D, capacity) || !in(sinks, 0, ENGRAM_WINDOW_SINKS_MAX) ||
      sinks >= capacity || !in(slots_total, 1, INT64_MAX / (Hk * capacity * D * 2)) || !ld_in_range(ldk, Hk * D) ||
      !ld_in_range(ldv, Hk * D))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldk | ldv) % 8 || !aligned8(cu_seqlens) || !aligned8(slots)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {k, v, cache_k, cache_v};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t pool = slots_total * Hk * capacity * D * 2;
  const Rows ins[] = {heads(k, N, ldk, Hk, D), heads(v, N, ldv, Hk, D), flat(cu_seqlens, (B + 1) * 8), flat(slots, B * 8)};
  const Rows outs[] = {flat(cache_k, pool), flat(cache_v, pool)};
  if (any_overlap(ins, 4, outs, 2)) return ENGRAM_ERR_OVERLAP;
  engram::WindowStepCall w{};
  w.k = static_cast<const uint16_t*>(k); w.v = static_cast<const uint16_t*>(v); w.cu = cu_seqlens; w.slots = slots;
  w.cache_k = static_cast<uint16_t*>(cache_k); w.cache_v = static_cast<uint16_t*>(cache_v);
  w.N = N; w.B = B; w.Hk = Hk; w.D = D; w.n_slots = slots_total; w.capacity = capacity; w.sinks = sinks;
  w.ldk = ldk; w.ldv = ldv; w.dtype = dtype;
  return launched(engram::launch_window_fill(w, (hipStream_t)stream));
}

size_t engram_gated_scan_fwd_workspace_bytes(int64_t N, int64_t B, int64_t D) { return scan_workspace_bytes(N, B, D); }

size_t engram_gated_scan_bwd_workspace_bytes(int64_t N, int64_t B, int64_t D) { return scan_workspace_bytes(N, B, D); }

engram_status engram_gated_scan_fwd(const void* gate, const void* u, const int64_t* cu_seqlens, const float* state_in,
                                    void* h, float* state_out, void* workspace, int64_t N, int64_t B, int64_t D,
                                    int64_t ldg, int64_t ldu, int64_t ldh, int dtype, void* stream) {
  if (!gate || !u || !cu_seqlens || !h || !workspace) return ENGRAM_ERR_NULL;
  if (!float_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!scan_sizes_ok(N, B, D) || !ld_in_range(ldg, D) || !ld_in_range(ldu, D) || !ld_in_range(ldh, D))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldg | ldu | ldh) % 8 || !aligned8(cu_seqlens)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {gate, u, state_in, h, state_out, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t e = bytes_of(dtype);
  const Rows ins[] = {Rows{gate, N, ldg * e, D * e}, Rows{u, N, ldu * e, D * e}, flat(cu_seqlens, (B + 1) * 8),
                      flat(state_in, B * D * 4)};
  const Rows outs[] = {Rows{h, N, ldh * e, D * e}, flat(state_out, B * D * 4),
                       flat(workspace, (int64_t)engram::scan_workspace(N, D))};
  if (any_overlap(ins, 4, outs, 3)) return ENGRAM_ERR_OVERLAP;
  engram::ScanCall c{};
  c.gate = gate; c.u = u; c.cu = cu_seqlens; c.state_in = state_in; c.h = h; c.state_out = state_out;
  c.workspace = workspace;
  c.N = N; c.B = B; c.D = D; c.ldg = ldg; c.ldu = ldu; c.ldh = ldh; c.dtype = dtype;
  return launched(engram::launch_scan_fwd(c, (hipStream_t)stream));
}

engram_status engram_gated_scan_bwd(const void* grad_h, const void* gate, const void* u, const void* h,
                                    const int64_t* cu_seqlens, const float* state_in, const float* grad_state_out,
                                    void* grad_gate, void* grad_u, float* grad_state_in, void* workspace, int64_t N,
                                    int64_t B, int64_t D, int64_t ldgh, int64_t ldg, int64_t ldu, int64_t ldh,
                                    int64_t ldgg, int64_t ldgu, int dtype, void* stream) {
  if (!grad_h || !gate || !u || !h || !cu_seqlens || !grad_gate || !grad_u || !workspace) return ENGRAM_ERR_NULL;
  if (!float_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!scan_sizes_ok(N, B, D) || !ld_in_range(ldgh, D) || !ld_in_range(ldg, D) || !ld_in_range(ldu, D) ||
      !ld_in_range(ldh, D) || !ld_in_range(ldgg, D) || !ld_in_range(ldgu, D))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldgh | ldg | ldu | ldh | ldgg | ldgu) % 8 || !aligned8(cu_seqlens)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {grad_h, gate, u, h, state_in, grad_state_out, grad_gate, grad_u, grad_state_in, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t e = bytes_of(dtype);
  const Rows ins[] = {Rows{grad_h, N, ldgh * e, D * e}, Rows{gate, N, ldg * e, D * e}, Rows{u, N, ldu * e, D * e},
                      Rows{h, N, ldh * e, D * e}, flat(cu_seqlens, (B + 1) * 8), flat(state_in, B * D * 4),
                      flat(grad_state_out, B * D * 4)};
  const Rows outs[] = {Rows{grad_gate, N, ldgg * e, D * e}, Rows{grad_u, N, ldgu * e, D * e},
                       flat(grad_state_in, B * D * 4), flat(workspace, (int64_t)engram::scan_workspace(N, D))};
  if (any_overlap(ins, 7, outs, 4)) return ENGRAM_ERR_OVERLAP;
  engram::ScanCall c{};
  c.grad_h = grad_h; c.gate = gate; c.u = u; c.h_in = h; c.cu = cu_seqlens; c.state_in = state_in;
  c.grad_state_out = grad_state_out; c.grad_gate = grad_gate; c.grad_u = grad_u; c.grad_state_in = grad_state_in;
  c.workspace = workspace;
  c.N = N; c.B = B; c.D = D; c.ldgh = ldgh; c.ldg = ldg; c.ldu = ldu; c.ldh = ldh; c.ldgg = ldgg; c.ldgu = ldgu;
  c.dtype = dtype;
  return launched(engram::launch_scan_bwd(c, (hipStream_t)stream));
}

engram_status engram_gated_scan_step(const void* gate, const void* u, float* state, const int64_t* slots, void* h,
                                     int64_t B, int64_t D, int64_t slots_total, int64_t ldg, int64_t ldu, int64_t ldh,
                                     int dtype, void* stream) {
  if (!gate || !u || !state || !slots || !h) return ENGRAM_ERR_NULL;
  if (!float_kind_ok(dtype)) return ENGRAM_ERR_KIND;
  if (!scan_sizes_ok(1, 1, D) || !in(B, 1, ENGRAM_SCAN_STEP_ROWS_MAX) || !in(slots_total, 1, INT64_MAX / (D * 4)) ||
      !ld_in_range(ldg, D) || !ld_in_range(ldu, D) || !ld_in_range(ldh, D))
    return ENGRAM_ERR_N_RANGE;
  if ((D | ldg | ldu | ldh) % 8 || !aligned8(slots)) return ENGRAM_ERR_ALIGN;
  const void* ptrs[] = {gate, u, state, h};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ENGRAM_ERR_ALIGN;
  const int64_t e = bytes_of(dtype);
  const Rows ins[] = {Rows{gate, B, ldg * e, D * e}, Rows{u, B, ldu * e, D * e}, flat(slots, B * 8)};
  const Rows outs[] = {Rows{h, B, ldh * e, D * e}, flat(state, slots_total * D * 4)};
  if (any_overlap(ins, 3, outs, 2)) return ENGRAM_ERR_OVERLAP;
  engram::ScanCall c{};
  c.gate = gate; c.u = u; c.pool = state; c.slots = slots; c.n_slots = slots_total; c.h = h;
  c.B = B; c.D = D; c.ldg = ldg; c.ldu = ldu; c.ldh = ldh; c.dtype = dtype;
  return launched(engram::launch_scan_step(c, (hipStream_t)stream));
}

}  // extern "C"
