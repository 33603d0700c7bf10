// C ABI of the operators around the layer (moe_ext.h): argument checks,
// workspace layout and launch order. Every check runs on the host before
// anything is enqueued.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <initializer_list>

#include "../../include/moe_ext.h"
#include "api_common.h"
#include "internal.h"

using namespace moe;

namespace {

// A caller's buffer: NULL means it was left out.
struct Buf {
  const void* ptr;
  size_t bytes;
  bool out;
};

inline Buf in(const void* p, size_t n) { return {p, n, false}; }
inline Buf out(const void* p, size_t n) { return {p, n, true}; }

// Alignment of every buffer, and no output overlapping another buffer.
bool buffers_ok(std::initializer_list<Buf> bufs) {
  for (const Buf& a : bufs) {
    if (!a.ptr) continue;
    if (!aligned16(a.ptr)) return false;
    const uintptr_t a0 = (uintptr_t)a.ptr;
    if (a.bytes > UINTPTR_MAX - a0) return false;
    if (!a.out) continue;
    for (const Buf& b : bufs) {
      if (&a == &b || !b.ptr) continue;
      const uintptr_t b0 = (uintptr_t)b.ptr;
      if (a0 < b0 + b.bytes && b0 < a0 + a.bytes) return false;
    }
  }
  return true;
}

// The gradient's factor coef E has to stay finite: masked rows multiply it by 0.
bool coef_ok(const moe_problem_t& p, float coef) { return std::isfinite(coef * (float)p.E); }

// Codes of x8, of one expert's weight and of a tile's 256 rows (bf16 rows of
// the result included) are reached with 32-bit byte offsets. (Those of x8 only
// through a permutation: without one the limit is the interface's, the same for both.)
// The second product's pieces fit where the first's rows do: T k d_model < 2^31 * 256.
bool fp8_supported(const moe_problem_t& p, bool gathered) {
  const int64_t rows = gathered ? p.T : p.T * p.k;
  const int64_t lim = INT32_MAX, cd = (int64_t)moex_code_pitch(p.d_model), ce = (int64_t)moex_code_pitch(p.d_expert);
  return p.dtype == MOE_DTYPE_BF16 && rows * cd < lim && p.d_expert * cd < lim && p.d_model * ce < lim &&
         512 * cd < lim && 512 * ce < lim && gemm_fp8_fits(p.T * p.k, p.d_expert, p.E);
}

struct FfnWs {
  uint8_t *h, *hs;  // 8-bit rows of the hidden activations
  float* partials;  // of the second product's cut tiles
};

FfnWs carve_ffn(Carver& c, const moe_problem_t& p) {
  const size_t R = (size_t)p.T * p.k;
  FfnWs w;
  w.h = c.take<uint8_t>(R * moex_code_pitch(p.d_expert));
  w.hs = c.take<uint8_t>(R * moex_scale_pitch(p.d_expert));
  w.partials = c.take<float>(gemm_fp8_partials_bytes((int64_t)R, p.d_expert, p.d_model, p.E) / sizeof(float));
  return w;
}

struct ForwardWs {
  int32_t *idx, *counts, *offsets, *perm, *inv;
  float *gate, *route_part;
  PermuteWs pw;
  uint8_t *x8, *xs;
  FfnWs fw;
  void* y_perm;
};

ForwardWs carve_forward(Carver& c, const moe_problem_t& p) {
  const size_t R = (size_t)p.T * p.k;
  ForwardWs w;
  w.idx = c.take<int32_t>(R);
  w.gate = c.take<float>(R);
  w.counts = c.take<int32_t>(p.E);
  w.offsets = c.take<int32_t>(p.E + 1);
  w.perm = c.take<int32_t>(R);
  w.inv = c.take<int32_t>(R);
  w.pw = carve_permute(c, p);
  w.route_part = carve_route(c, p);
  w.x8 = c.take<uint8_t>((size_t)p.T * moex_code_pitch(p.d_model));
  w.xs = c.take<uint8_t>((size_t)p.T * moex_scale_pitch(p.d_model));
  w.fw = carve_ffn(c, p);
  w.y_perm = c.take<uint16_t>(R * p.d_model);
  return w;
}

size_t stage_bytes(const moe_problem_t& p, int32_t stage) {
  Carver c(nullptr);
  switch (stage) {
    case MOEX_STAGE_NORM_BACKWARD:
      c.take<float>((size_t)norm_bwd_blocks(p.T, p.d_model) * p.d_model);
      break;
    case MOEX_STAGE_BALANCE:
      c.take<int32_t>(balance_ws_ints(p));
      break;
    case MOEX_STAGE_FFN_FP8:
      carve_ffn(c, p);
      break;
    case MOEX_STAGE_FORWARD_FP8:
      carve_forward(c, p);
      break;
    default:  // the training workspace, then the balance loss's
      return train_ws_bytes(p) + kAlign + balance_ws_ints(p) * sizeof(int32_t) + kAlign;
  }
  return c.off + kAlign;  // slack so a 16-byte aligned base can be rounded up to kAlign
}

hipError_t run_ffn(const moe_problem_t& p, const void* x8, const void* xs, const int32_t* perm, const int32_t* offsets,
                   const void* W1q, const void* W1s, const void* W2q, const void* W2s, void* y_perm, const FfnWs& w,
                   hipStream_t s) {
  const int64_t R = p.T * p.k;
  hipError_t e = launch_gemm_fp8(x8, xs, perm, perm ? p.T : R, offsets, W1q, W1s, w.h, w.hs, R, p.d_model, p.d_expert,
                                 p.E, true, nullptr, s);
  if (e == hipSuccess)
    e = launch_gemm_fp8(w.h, w.hs, nullptr, R, offsets, W2q, W2s, y_perm, nullptr, R, p.d_expert, p.d_model, p.E, false,
                        w.partials, s);
  return e;
}

}  // namespace

MOE_API moe_status_t moex_workspace_size(const moe_problem_t* p, int32_t stage, size_t* bytes) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!bytes || stage < MOEX_STAGE_NORM_BACKWARD || stage > MOEX_STAGE_TRAIN_BALANCED) return MOE_ERR_INVALID_ARGUMENT;
  *bytes = stage_bytes(*p, stage);
  return MOE_OK;
}

MOE_API moe_status_t moex_add_rmsnorm(const moe_problem_t* p, const void* x, const void* residual, const void* gain,
                                      float eps, void* h, void* y, void* y8, void* y_scale, float* rstd,
                                      void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!x || !gain || !!residual != !!h || !!y8 != !!y_scale || (!y && !y8 && !rstd)) return MOE_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(eps) || eps < 0.0f) return MOE_ERR_INVALID_ARGUMENT;
  const size_t rows = (size_t)p->T * p->d_model * elem_size(p->dtype);
  if (!buffers_ok({in(x, rows), in(residual, rows), in(gain, p->d_model * elem_size(p->dtype)), out(h, rows),
                   out(y, rows), out(y8, p->T * moex_code_pitch(p->d_model)),
                   out(y_scale, p->T * moex_scale_pitch(p->d_model)), out(rstd, p->T * sizeof(float))}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->d_model > kNormMaxWidth) return MOE_ERR_UNSUPPORTED;
  return hip_status(launch_add_rmsnorm(*p, x, residual, gain, eps, h, y, y8, y_scale, rstd, (hipStream_t)stream));
}

MOE_API moe_status_t moex_add_rmsnorm_backward(const moe_problem_t* p, const void* h, const void* gain,
                                               const float* rstd, const void* dy, const void* dh, void* dx,
                                               float* dgain, void* ws, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!h || !gain || !rstd || !dy || !dx || !dgain || !ws) return MOE_ERR_INVALID_ARGUMENT;
  const size_t rows = (size_t)p->T * p->d_model * elem_size(p->dtype), need = stage_bytes(*p, MOEX_STAGE_NORM_BACKWARD);
  if (!buffers_ok({in(h, rows), in(gain, p->d_model * elem_size(p->dtype)), in(rstd, p->T * sizeof(float)),
                   in(dy, rows), in(dh, rows), out(dx, rows), out(dgain, p->d_model * sizeof(float)),
                   out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->d_model > kNormMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return hip_status(launch_rmsnorm_backward(*p, h, gain, rstd, dy, dh, dx, dgain, (float*)align_ws(ws),
                                            (hipStream_t)stream));
}

MOE_API moe_status_t moex_quantize_rows(const moe_problem_t* p, const void* x, void* x8, void* x_scale, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!x || !x8 || !x_scale) return MOE_ERR_INVALID_ARGUMENT;
  if (!buffers_ok({in(x, (size_t)p->T * p->d_model * elem_size(p->dtype)),
                   out(x8, p->T * moex_code_pitch(p->d_model)), out(x_scale, p->T * moex_scale_pitch(p->d_model))}))
    return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_quantize_rows(*p, x, x8, x_scale, (hipStream_t)stream));
}

MOE_API moe_status_t moex_balance_loss(const moe_problem_t* p, const float* logits, const int32_t* topk_idx,
                                       const uint8_t* token_mask, float coef, float* loss, int32_t* counts,
                                       float* mean_prob, float* dlogits, void* ws, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!logits || !topk_idx || !loss || !counts || !mean_prob || !ws || !coef_ok(*p, coef))
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t te = (size_t)p->T * p->E * sizeof(float), need = stage_bytes(*p, MOEX_STAGE_BALANCE);
  if (!buffers_ok({in(logits, te), in(topk_idx, (size_t)p->T * p->k * sizeof(int32_t)), in(token_mask, (size_t)p->T),
                   out(loss, sizeof(float)), out(counts, p->E * sizeof(int32_t)), out(mean_prob, p->E * sizeof(float)),
                   out(dlogits, te), out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return hip_status(launch_balance(*p, logits, topk_idx, token_mask, coef, loss, counts, mean_prob, dlogits,
                                   (int32_t*)align_ws(ws), (hipStream_t)stream));
}

MOE_API moe_status_t moex_backward_balanced(const moe_problem_t* p, const void* x, const void* w_router,
                                            const void* W1, const void* W2, const void* dy, const uint8_t* token_mask,
                                            float coef, void* dx, void* dw_router, float* dbias, void* dW1, void* dW2,
                                            float* loss, int32_t* counts, float* mean_prob, void* ws, size_t ws_bytes,
                                            void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!x || !w_router || !W1 || !W2 || !dy || !dx || !dw_router || !dW1 || !dW2 || !loss || !ws ||
      !coef_ok(*p, coef))
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t td = (size_t)p->T * p->d_model * 2, de = (size_t)p->d_model * p->E * 2,
               w = (size_t)p->E * p->d_model * p->d_expert * 2, E = (size_t)p->E * 4;
  if (!backward_supported(*p)) return MOE_ERR_UNSUPPORTED;
  const size_t need = stage_bytes(*p, MOEX_STAGE_TRAIN_BALANCED);
  if (!buffers_ok({in(x, td), in(w_router, de), in(W1, w), in(W2, w), in(dy, td), in(token_mask, (size_t)p->T),
                   out(dx, td), out(dw_router, de), out(dbias, E), out(dW1, w), out(dW2, w), out(loss, sizeof(float)),
                   out(counts, E), out(mean_prob, E), out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const BalanceTerm bal = {token_mask, coef, loss, counts, mean_prob,
                           (int32_t*)align_ws((char*)ws + train_ws_bytes(*p))};
  return hip_status(run_backward(*p, x, w_router, W1, W2, dy, dx, dw_router, dbias, dW1, dW2, nullptr, nullptr, ws,
                                 &bal, (hipStream_t)stream));
}

MOE_API moe_status_t moex_quantize_experts(const moe_problem_t* p, const void* W1, const void* W2, void* W1q,
                                           void* W1s, void* W2q, void* W2s, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!W1 || !W2 || !W1q || !W1s || !W2q || !W2s) return MOE_ERR_INVALID_ARGUMENT;
  const int E = p->E, d = p->d_model, de = p->d_expert;
  const size_t w = (size_t)E * d * de * 2;
  if (!buffers_ok({in(W1, w), in(W2, w), out(W1q, moex_weight_bytes(E, d, de)),
                   out(W1s, moex_weight_scale_bytes(E, d, de)), out(W2q, moex_weight_bytes(E, de, d)),
                   out(W2s, moex_weight_scale_bytes(E, de, d))}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->dtype != MOE_DTYPE_BF16 || !quantize_weights_fits(d, de) || !quantize_weights_fits(de, d))
    return MOE_ERR_UNSUPPORTED;
  hipError_t e = launch_quantize_weights(W1, W1q, W1s, E, d, de, (hipStream_t)stream);
  if (e == hipSuccess) e = launch_quantize_weights(W2, W2q, W2s, E, de, d, (hipStream_t)stream);
  return hip_status(e);
}

MOE_API moe_status_t moex_grouped_ffn_fp8(const moe_problem_t* p, const void* x8, const void* x_scale,
                                          const int32_t* perm, const int32_t* offsets, const void* W1q,
                                          const void* W1s, const void* W2q, const void* W2s, void* y_perm, void* ws,
                                          size_t ws_bytes, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!x8 || !x_scale || !offsets || !W1q || !W1s || !W2q || !W2s || !y_perm || !ws) return MOE_ERR_INVALID_ARGUMENT;
  const int E = p->E, d = p->d_model, de = p->d_expert;
  const size_t R = (size_t)p->T * p->k, xr = perm ? (size_t)p->T : R, need = stage_bytes(*p, MOEX_STAGE_FFN_FP8);
  if (!buffers_ok({in(x8, xr * moex_code_pitch(d)), in(x_scale, xr * moex_scale_pitch(d)), in(perm, R * 4),
                   in(offsets, (E + 1) * sizeof(int32_t)), in(W1q, moex_weight_bytes(E, d, de)),
                   in(W1s, moex_weight_scale_bytes(E, d, de)), in(W2q, moex_weight_bytes(E, de, d)),
                   in(W2s, moex_weight_scale_bytes(E, de, d)), out(y_perm, R * d * 2), out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!fp8_supported(*p, perm != nullptr)) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  Carver c(align_ws(ws));
  const FfnWs fw = carve_ffn(c, *p);
  return hip_status(run_ffn(*p, x8, x_scale, perm, offsets, W1q, W1s, W2q, W2s, y_perm, fw, (hipStream_t)stream));
}

MOE_API moe_status_t moex_forward_fp8(const moe_problem_t* p, const void* x, const void* x8, const void* x_scale,
                                      const void* w_router, const float* router_bias, const void* W1q,
                                      const void* W1s, const void* W2q, const void* W2s, void* y, void* ws,
                                      size_t ws_bytes, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!x || !!x8 != !!x_scale || !w_router || !W1q || !W1s || !W2q || !W2s || !y || !ws)
    return MOE_ERR_INVALID_ARGUMENT;
  const int E = p->E, d = p->d_model, de = p->d_expert;
  const size_t T = (size_t)p->T, need = stage_bytes(*p, MOEX_STAGE_FORWARD_FP8);
  if (!buffers_ok({in(x, T * d * 2), in(x8, T * moex_code_pitch(d)), in(x_scale, T * moex_scale_pitch(d)),
                   in(w_router, (size_t)d * E * 2), in(router_bias, E * sizeof(float)),
                   in(W1q, moex_weight_bytes(E, d, de)), in(W1s, moex_weight_scale_bytes(E, d, de)),
                   in(W2q, moex_weight_bytes(E, de, d)), in(W2s, moex_weight_scale_bytes(E, de, d)), out(y, T * d * 2),
                   out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!fp8_supported(*p, true)) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t s = (hipStream_t)stream;
  Carver c(align_ws(ws));
  const ForwardWs w = carve_forward(c, *p);
  hipError_t e;
  if (route_permute_fused(*p)) {
    e = launch_route_partials(*p, x, w_router, w.route_part, s);
    if (e == hipSuccess)
      e = launch_finalize_permute_small(*p, w.route_part, route_splits(*p), router_bias, w.idx, w.gate, w.counts,
                                        w.offsets, w.perm, w.inv, s);
  } else {
    e = launch_route(*p, x, w_router, router_bias, nullptr, w.idx, w.gate, w.route_part, s);
    if (e == hipSuccess)
      e = launch_permute_index(*p, w.idx, w.counts, w.offsets, w.perm, w.inv, w.pw.blockcounts, w.pw.blockbase, s);
  }
  if (e == hipSuccess && !x8) e = launch_quantize_rows(*p, x, w.x8, w.xs, s);
  if (e == hipSuccess)
    e = run_ffn(*p, x8 ? x8 : w.x8, x8 ? x_scale : w.xs, w.perm, w.offsets, W1q, W1s, W2q, W2s, w.y_perm, w.fw, s);
  if (e == hipSuccess) e = launch_combine(*p, w.y_perm, w.inv, w.gate, y, s);
  return hip_status(e);
}
