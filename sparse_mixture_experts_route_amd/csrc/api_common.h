// Argument checks and workspace carving shared by the C ABI's entry points
// (host only). Every check runs before anything is enqueued.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "internal.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {

constexpr size_t kAlign = 256;

inline bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15u) == 0; }

inline size_t elem_size(int32_t dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }

inline moe_status_t check_problem(const moe_problem_t* p) {
  if (!p) return MOE_ERR_INVALID_ARGUMENT;
  if (p->dtype != MOE_DTYPE_F32 && p->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (p->T < 1 || p->E < 1 || p->k < 1 || p->k > p->E || p->d_model < 1 || p->d_expert < 1)
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->E > 256) return MOE_ERR_UNSUPPORTED;
  if (p->T > (int64_t)INT32_MAX / p->k) return MOE_ERR_UNSUPPORTED;
  if (p->d_model % 64 != 0 || p->d_expert % 64 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A caller's buffer: NULL means it was left out.
struct Buf {
  const void* ptr;
  size_t bytes;
  bool out;
};

inline Buf in(const void* p, size_t n) { return {p, n, false}; }
inline Buf out(const void* p, size_t n) { return {p, n, true}; }

// Alignment of every buffer, and no output overlapping another buffer.
inline bool buffers_ok(std::initializer_list<Buf> bufs) {
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

// Sequential sub-allocation of a caller-provided workspace (or size counting when base is null).
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base((char*)b) {}
  template <typename T>
  T* take(size_t n) {
    off = (off + kAlign - 1) / kAlign * kAlign;
    T* ptr = base ? (T*)(base + off) : nullptr;
    off += n * sizeof(T);
    return ptr;
  }
};

struct PermuteWs {
  int32_t* blockcounts;
  int32_t* blockbase;
};

inline PermuteWs carve_permute(Carver& c, const moe_problem_t& p) {
  const size_t n = (size_t)moe::permute_blocks(p.T) * (size_t)p.E;
  PermuteWs w;
  w.blockcounts = c.take<int32_t>(n);
  w.blockbase = c.take<int32_t>(n);
  return w;
}

// float32 partial logits of a router split over d_model (none when unsplit)
inline float* carve_route(Carver& c, const moe_problem_t& p) {
  const size_t n = moe::route_partials_bytes(p) / sizeof(float);
  return n ? c.take<float>(n) : nullptr;
}

inline char* align_ws(void* ws) { return (char*)(((uintptr_t)ws + kAlign - 1) / kAlign * kAlign); }

inline moe_status_t hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// moe_forward_train's and moe_backward's workspace, in bytes
size_t train_ws_bytes(const moe_problem_t& p);
// Whether the training forward takes problem p, and whether the backward does
bool train_supported(const moe_problem_t& p);
bool backward_supported(const moe_problem_t& p);

// The balance loss that a backward pass adds to the layer's loss (moe_ext.h);
// ws: balance_ws_ints(p) int32
struct BalanceTerm {
  const uint8_t* mask;
  float coef;
  float* loss;
  int32_t* counts;
  float* mean_prob;
  int32_t* ws;
};

// Enqueues moe_backward's kernels (arguments already checked); `bal` may be NULL.
hipError_t run_backward(const moe_problem_t& p, const void* x, const void* w_router, const void* W1, const void* W2,
                        const void* dy, void* dx, void* dw_router, float* dbias, void* dW1, void* dW2,
                        float* load_frac, float* mean_prob, void* ws, const BalanceTerm* bal, hipStream_t s);

}  // namespace moe
