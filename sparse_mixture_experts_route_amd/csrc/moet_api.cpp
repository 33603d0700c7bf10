// C ABI of what trains the layer's surroundings (moe_train.h): argument checks,
// workspace layout and launch order. Every check runs on the host before
// anything is enqueued.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "../../include/moe_train.h"
#include "api_common.h"
#include "internal.h"
#include "linear.h"
#include "optim.h"

using namespace moe;

namespace {

float* carve_partials(Carver& c, size_t bytes) { return bytes ? c.take<float>(bytes / sizeof(float)) : nullptr; }

struct LinearBwdWs {
  uint16_t* du;
  float *sums, *partials;  // the products follow each other: they share their partial sums
};

LinearBwdWs carve_linear_backward(Carver& c, const moe_problem_t& p) {
  LinearBwdWs w;
  w.du = c.take<uint16_t>((size_t)p.T * p.d_expert);
  w.sums = c.take<float>((size_t)slope_parts(p.T, p.d_expert) * p.d_expert);
  w.partials = carve_partials(c, std::max(dense_partials_bytes(DENSE_NT, p.T, p.d_model, p.d_expert),
                                          dense_partials_bytes(DENSE_TN, p.d_model, p.d_expert, p.T)));
  return w;
}

size_t stage_bytes(const moe_problem_t& p, int32_t stage) {
  Carver c(nullptr);
  switch (stage) {
    case MOET_STAGE_DISPATCH:
      carve_permute(c, p);
      break;
    case MOET_STAGE_LINEAR:
      carve_partials(c, dense_partials_bytes(DENSE_NN, p.T, p.d_expert, p.d_model));
      break;
    default:
      carve_linear_backward(c, p);
      break;
  }
  return c.off + kAlign;  // slack so a 16-byte aligned base can be rounded up to kAlign
}

inline size_t row_bytes(const moe_problem_t& p) { return (size_t)p.d_model * elem_size(p.dtype); }

}  // namespace

MOE_API moe_status_t moet_workspace_size(const moe_problem_t* p, int32_t stage, size_t* bytes) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!bytes || stage < MOET_STAGE_DISPATCH || stage > MOET_STAGE_LINEAR_BACKWARD) return MOE_ERR_INVALID_ARGUMENT;
  *bytes = stage_bytes(*p, stage);
  return MOE_OK;
}

// ---- rows sorted by expert and back

MOE_API moe_status_t moet_dispatch(const moe_problem_t* p, const int32_t* topk_idx, const float* weight, const void* x,
                                   int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* x_perm,
                                   void* ws, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!topk_idx || !x || !counts || !offsets || !perm || !inv || !x_perm || !ws) return MOE_ERR_INVALID_ARGUMENT;
  const size_t T = (size_t)p->T, R = T * p->k, row = row_bytes(*p), need = stage_bytes(*p, MOET_STAGE_DISPATCH);
  if (!buffers_ok({in(topk_idx, R * 4), in(weight, R * 4), in(x, T * row), out(counts, (size_t)p->E * 4),
                   out(offsets, ((size_t)p->E + 1) * 4), out(perm, R * 4), out(inv, R * 4), out(x_perm, R * row),
                   out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t s = (hipStream_t)stream;
  if (dispatch_small(*p))
    return hip_status(launch_dispatch_small(*p, topk_idx, weight, x, counts, offsets, perm, inv, x_perm, s));
  Carver c(align_ws(ws));
  const PermuteWs w = carve_permute(c, *p);
  hipError_t e = launch_permute_index(*p, topk_idx, counts, offsets, perm, inv, w.blockcounts, w.blockbase, s, nullptr, 0,
                                      true);
  if (e == hipSuccess) e = launch_to_rows(*p, x, inv, weight, nullptr, x_perm, nullptr, s);
  return hip_status(e);
}

MOE_API moe_status_t moet_dispatch_backward(const moe_problem_t* p, const void* dx_perm, const int32_t* inv,
                                            const void* x, const float* weight, const void* residual, void* dx,
                                            float* dweight, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!dx_perm || !inv || !dx || !!x != !!dweight) return MOE_ERR_INVALID_ARGUMENT;
  const size_t T = (size_t)p->T, R = T * p->k, row = row_bytes(*p);
  if (!buffers_ok({in(dx_perm, R * row), in(inv, R * 4), in(x, T * row), in(weight, R * 4), in(residual, T * row),
                   out(dx, T * row), out(dweight, R * 4)}))
    return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_from_rows(*p, dx_perm, inv, weight, residual, x, dx, dweight, (hipStream_t)stream));
}

MOE_API moe_status_t moet_combine(const moe_problem_t* p, const void* y_perm, const int32_t* inv, const float* gate,
                                  const void* residual, void* y, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!y_perm || !inv || !y) return MOE_ERR_INVALID_ARGUMENT;
  const size_t T = (size_t)p->T, R = T * p->k, row = row_bytes(*p);
  if (!buffers_ok({in(y_perm, R * row), in(inv, R * 4), in(gate, R * 4), in(residual, T * row), out(y, T * row)}))
    return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_from_rows(*p, y_perm, inv, gate, residual, nullptr, y, nullptr, (hipStream_t)stream));
}

MOE_API moe_status_t moet_combine_backward(const moe_problem_t* p, const void* dy, const int32_t* inv,
                                           const void* y_perm, const float* gate, void* dy_perm, float* dgate,
                                           void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!dy || !inv || !dy_perm || !!y_perm != !!dgate) return MOE_ERR_INVALID_ARGUMENT;
  const size_t T = (size_t)p->T, R = T * p->k, row = row_bytes(*p);
  if (!buffers_ok({in(dy, T * row), in(inv, R * 4), in(y_perm, R * row), in(gate, R * 4), out(dy_perm, R * row),
                   out(dgate, R * 4)}))
    return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_to_rows(*p, dy, inv, gate, y_perm, dy_perm, dgate, (hipStream_t)stream));
}

MOE_API moe_status_t moet_gate_backward(const moe_problem_t* p, const float* logits, const int32_t* topk_idx,
                                        const float* dgate, const float* add, float* dlogits, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!logits || !topk_idx || !dgate || !dlogits) return MOE_ERR_INVALID_ARGUMENT;
  const size_t R = (size_t)p->T * p->k * 4, te = (size_t)p->T * p->E * 4;
  if (!buffers_ok({in(logits, te), in(topk_idx, R), in(dgate, R), in(add, te), out(dlogits, te)}))
    return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_gate_backward(*p, logits, topk_idx, dgate, add, dlogits, (hipStream_t)stream));
}

// ---- a dense projection

namespace {

// Operands are reached with 32-bit byte offsets, in whole tiles of up to 256 rows.
bool linear_supported(const moe_problem_t& p) {
  const int64_t K = p.d_model, N = p.d_expert, lim = (int64_t)1 << 30;  // of 2 bytes each
  return p.dtype == MOE_DTYPE_BF16 && p.T * K < lim && p.T * N < lim && K * N < lim && 256 * K < lim && 256 * N < lim;
}

bool act_ok(int32_t act) { return act >= MOET_ACT_NONE && act <= MOET_ACT_RELU; }

}  // namespace

MOE_API moe_status_t moet_linear(const moe_problem_t* p, const void* x, const void* W, const void* bias, int32_t act,
                                 const void* residual, void* u, void* y, void* ws, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!x || !W || !y || !ws || !act_ok(act)) return MOE_ERR_INVALID_ARGUMENT;
  if (!linear_supported(*p)) return MOE_ERR_UNSUPPORTED;
  const size_t T = (size_t)p->T, K = p->d_model, N = p->d_expert, need = stage_bytes(*p, MOET_STAGE_LINEAR);
  if (!buffers_ok({in(x, T * K * 2), in(W, K * N * 2), in(bias, N * 2), in(residual, T * N * 2), out(u, T * N * 2),
                   out(y, T * N * 2), out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  Carver c(align_ws(ws));
  float* part = carve_partials(c, dense_partials_bytes(DENSE_NN, p->T, p->d_expert, p->d_model));
  return hip_status(launch_dense(DENSE_NN, x, W, p->T, p->d_expert, p->d_model, bias, act, residual, u, y, part,
                                 (hipStream_t)stream));
}

MOE_API moe_status_t moet_linear_backward(const moe_problem_t* p, const void* x, const void* W, const void* u,
                                          int32_t act, const void* dy, void* dx, void* dW, void* dbias, void* ws,
                                          size_t ws_bytes, void* stream) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!act_ok(act) || (!u && act != MOET_ACT_NONE) || !dy || !ws || (!dx && !dW && !dbias) || (dx && !W) || (dW && !x))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!linear_supported(*p)) return MOE_ERR_UNSUPPORTED;
  const size_t T = (size_t)p->T, K = p->d_model, N = p->d_expert, need = stage_bytes(*p, MOET_STAGE_LINEAR_BACKWARD);
  if (!buffers_ok({in(x, T * K * 2), in(W, K * N * 2), in(u, T * N * 2), in(dy, T * N * 2), out(dx, T * K * 2),
                   out(dW, K * N * 2), out(dbias, N * 2), out(ws, need)}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t s = (hipStream_t)stream;
  Carver c(align_ws(ws));
  const LinearBwdWs w = carve_linear_backward(c, *p);
  const void* du = act == MOET_ACT_NONE ? dy : w.du;
  hipError_t e = hipSuccess;
  if (act != MOET_ACT_NONE || dbias)
    e = launch_slope(dy, u, act, act != MOET_ACT_NONE && (dx || dW) ? w.du : nullptr, dbias, w.sums, p->T, p->d_expert, s);
  if (e == hipSuccess && dx)
    e = launch_dense(DENSE_NT, du, W, p->T, p->d_model, p->d_expert, nullptr, MOET_ACT_NONE, nullptr, nullptr, dx,
                     w.partials, s);
  if (e == hipSuccess && dW)
    e = launch_dense(DENSE_TN, x, du, p->d_model, p->d_expert, p->T, nullptr, MOET_ACT_NONE, nullptr, nullptr, dW,
                     w.partials, s);
  return hip_status(e);
}

// ---- the optimizer's step

namespace {

// A caller's buffer of a list, and the check that no output overlaps another buffer.
struct Span {
  uintptr_t lo, hi;
  bool out;
};

// (Those of a long list on the heap: they are 24 bytes each, up to seven a tensor, and
// a thread's stack may be small.)
struct Spans {
  static constexpr int kFew = 16 * 7 + 8;
  Span few[kFew];
  Span* s = few;
  int n = 0;
  Spans() = default;
  Spans(const Spans&) = delete;
  Spans& operator=(const Spans&) = delete;
  ~Spans() {
    if (s != few) delete[] s;
  }
  // Room for a list's tensors and what goes with them; false: no memory
  bool reserve(int32_t tensors) {
    if (tensors * 7 + 8 > kFew) {
      Span* const many = new (std::nothrow) Span[tensors * 7 + 8];
      if (!many) return false;
      s = many;
    }
    return true;
  }
  bool add(const void* p, size_t bytes, bool out) {
    const uintptr_t a = (uintptr_t)p;
    if (!p || !aligned16(p) || bytes > UINTPTR_MAX - a) return false;
    s[n++] = {a, a + bytes, out};
    return true;
  }
  bool apart() {
    std::sort(s, s + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t all = 0, outs = 0;  // ends of what began before
    for (int i = 0; i < n; ++i) {
      if (s[i].lo < (s[i].out ? all : outs)) return false;
      all = std::max(all, s[i].hi);
      if (s[i].out) outs = std::max(outs, s[i].hi);
    }
    return true;
  }
};

bool dtype_ok(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16; }

constexpr int64_t kMostValues = (int64_t)1 << 41;  // chunks are counted in 31 bits

// Types and sizes of a list, and the number of values (-1: refused, -2: too many)
int64_t list_values(const moet_tensor_t* t, int32_t count) {
  if (count < 0 || count > MOET_MAX_TENSORS || (count && !t)) return -1;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].n < 0 || !dtype_ok(t[i].grad_dtype)) return -1;
    if (t[i].n >= kMostValues) return -2;
    total += (t[i].n + kOptChunk - 1) / kOptChunk * kOptChunk;
  }
  return total >= kMostValues ? -2 : total;
}

}  // namespace

namespace {

// The checks of a step, spans of its tensors included
moe_status_t check_step(const moet_tensor_t* tensors, int32_t count, const moet_adamw_t* opt, const int32_t* counter,
                        const float* lr_scale, Spans& spans) {
  if (!opt || !counter) return MOE_ERR_INVALID_ARGUMENT;
  const double b1 = opt->beta1, b2 = opt->beta2;
  if (!std::isfinite(opt->lr) || opt->lr < 0 || !(b1 >= 0 && b1 < 1) || !(b2 >= 0 && b2 < 1) ||
      !std::isfinite(opt->eps) || opt->eps < 1e-15 || opt->eps > 1e15)
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t total = list_values(tensors, count);
  if (total == -1) return MOE_ERR_INVALID_ARGUMENT;
  if (total == -2) return MOE_ERR_UNSUPPORTED;
  if (!spans.reserve(count)) return MOE_ERR_HIP;
  bool ok = spans.add(counter, 8, true) && (!lr_scale || spans.add(lr_scale, 4, false));
  for (int i = 0; ok && i < count; ++i) {
    const moet_tensor_t& t = tensors[i];
    if (!t.n) continue;
    if (!dtype_ok(t.param_dtype) || !std::isfinite(t.lr_factor) || t.lr_factor < 0 || !std::isfinite(t.weight_decay) ||
        t.weight_decay < 0 || (t.param_dtype == MOE_DTYPE_BF16) != !!t.master || !!t.m_scale != !!t.v_scale)
      return MOE_ERR_INVALID_ARGUMENT;
    const size_t n = (size_t)t.n, blocks = (n + 127) / 128, mb = t.m_scale ? n : 4 * n;
    ok = spans.add(t.param, n * elem_size(t.param_dtype), true) && spans.add(t.grad, n * elem_size(t.grad_dtype), false) &&
         (!t.master || spans.add(t.master, 4 * n, true)) && spans.add(t.m, mb, true) && spans.add(t.v, mb, true) &&
         (!t.m_scale || (spans.add(t.m_scale, blocks, true) && spans.add(t.v_scale, blocks, true)));
  }
  return ok ? MOE_OK : MOE_ERR_INVALID_ARGUMENT;
}

moe_status_t run_step(const moet_tensor_t* tensors, int32_t count, const moet_adamw_t* opt, int32_t* counter,
                      const float* lr_scale, const GradScale& gs, hipStream_t s) {
  const OptHyper h = {opt->lr, opt->beta1, opt->beta2, std::log(opt->beta1), std::log(opt->beta2), (float)opt->eps, opt->seed};
  int64_t values = 0, grads = 0;
  for (int j = 0; j < count; ++j) {
    values += tensors[j].n;
    grads += tensors[j].n * (int64_t)elem_size(tensors[j].grad_dtype);
  }
  const bool past_caches = values >= (int64_t)8 << 20 && grads <= (int64_t)192 << 20;  // see optim.hip
  OptList l;
  int i = 0;
  do {
    l.count = 0;
    l.chunks = 0;
    l.base = i;
    for (; i < count && l.count < kOptTensors; ++i) {
      const moet_tensor_t& t = tensors[i];
      l.t[l.count++] = {t.param, t.grad, t.master, t.m, t.v, (uint8_t*)t.m_scale, (uint8_t*)t.v_scale, t.n,
                        (float)t.lr_factor, (float)t.weight_decay,
                        (t.grad_dtype == MOE_DTYPE_BF16 ? kGrad16 : 0u) | (t.master ? kParam16 : 0u) |
                            (t.m_scale ? kMoments8 : 0u),
                        l.chunks};
      l.chunks += (int32_t)((t.n + kOptChunk - 1) / kOptChunk);
    }
    l.last = i >= count;
    if (launch_adamw(l, h, counter, lr_scale, gs, past_caches, s) != hipSuccess) return MOE_ERR_HIP;
  } while (i < count);
  return MOE_OK;
}

// Sums of squares of a list's gradients, to slots in ws
moe_status_t run_squares(const moet_tensor_t* tensors, int32_t count, double* slots, hipStream_t s) {
  NormList l;
  int i = 0;
  do {
    l.count = 0;
    l.chunks = 0;
    l.add = i > 0;
    for (; i < count && l.count < kNormTensors; ++i) {
      const moet_tensor_t& t = tensors[i];
      l.t[l.count++] = {t.grad, t.n, l.chunks, t.grad_dtype == MOE_DTYPE_BF16 ? 1u : 0u};
      l.chunks += (int32_t)((t.n + kOptChunk - 1) / kOptChunk);
    }
    if (launch_square_sums(l, slots, s) != hipSuccess) return MOE_ERR_HIP;
  } while (i < count);
  return MOE_OK;
}

static_assert(kNormSlots * sizeof(double) + kAlign <= MOET_GRAD_NORM_WS_BYTES, "partial sums");

}  // namespace

MOE_API moe_status_t moet_adamw(const moet_tensor_t* tensors, int32_t count, const moet_adamw_t* opt, int32_t* counter,
                                const float* lr_scale, const float* grad_scale, void* stream) {
  Spans spans;
  const moe_status_t st = check_step(tensors, count, opt, counter, lr_scale, spans);
  if (st != MOE_OK) return st;
  if ((grad_scale && !spans.add(grad_scale, 4, false)) || !spans.apart()) return MOE_ERR_INVALID_ARGUMENT;
  return run_step(tensors, count, opt, counter, lr_scale, {grad_scale, nullptr, 0.0, nullptr, nullptr}, (hipStream_t)stream);
}

MOE_API moe_status_t moet_grad_norm(const moet_tensor_t* tensors, int32_t count, double max_norm, float* norm,
                                    float* scale, void* ws, size_t ws_bytes, void* stream) {
  if (!norm || !ws || !(max_norm > 0)) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t total = list_values(tensors, count);
  if (total == -1) return MOE_ERR_INVALID_ARGUMENT;
  if (total == -2) return MOE_ERR_UNSUPPORTED;
  Spans spans;
  if (!spans.reserve(count)) return MOE_ERR_HIP;
  bool ok = spans.add(norm, 4, true) && (!scale || spans.add(scale, 4, true)) &&
            spans.add(ws, MOET_GRAD_NORM_WS_BYTES, true);
  for (int i = 0; ok && i < count; ++i)
    ok = !tensors[i].n || spans.add(tensors[i].grad, (size_t)tensors[i].n * elem_size(tensors[i].grad_dtype), false);
  if (!ok || !spans.apart()) return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < MOET_GRAD_NORM_WS_BYTES) return MOE_ERR_WORKSPACE_TOO_SMALL;
  double* slots = (double*)align_ws(ws);
  const moe_status_t st = run_squares(tensors, count, slots, (hipStream_t)stream);
  if (st != MOE_OK) return st;
  return hip_status(launch_norm_scale(slots, max_norm, norm, scale, (hipStream_t)stream));
}

MOE_API moe_status_t moet_adamw_clipped(const moet_tensor_t* tensors, int32_t count, const moet_adamw_t* opt,
                                        int32_t* counter, const float* lr_scale, double max_norm, float* norm,
                                        float* scale, void* ws, size_t ws_bytes, void* stream) {
  if (!norm || !ws || !(max_norm > 0)) return MOE_ERR_INVALID_ARGUMENT;
  Spans spans;
  moe_status_t st = check_step(tensors, count, opt, counter, lr_scale, spans);
  if (st != MOE_OK) return st;
  if (!spans.add(norm, 4, true) || (scale && !spans.add(scale, 4, true)) ||
      !spans.add(ws, MOET_GRAD_NORM_WS_BYTES, true) || !spans.apart())
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < MOET_GRAD_NORM_WS_BYTES) return MOE_ERR_WORKSPACE_TOO_SMALL;
  double* slots = (double*)align_ws(ws);
  st = run_squares(tensors, count, slots, (hipStream_t)stream);
  if (st != MOE_OK) return st;
  return run_step(tensors, count, opt, counter, lr_scale, {nullptr, slots, max_norm, norm, scale}, (hipStream_t)stream);
}
