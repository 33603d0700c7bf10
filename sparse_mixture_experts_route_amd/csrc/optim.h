// What the optimizer's launches take: a list of tensors in the kernel's own
// arguments, so that a captured step needs no memory besides the tensors.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kOptThreads = 256;
constexpr int kOptChunk = 2048;      // values that a workgroup takes at once, 8 a thread
constexpr int kNormTensors = 128;    // of one launch of the norm
constexpr int kNormSlots = 1024;     // workgroups, and partial sums, of the norm

enum : uint32_t { kGrad16 = 1, kParam16 = 2, kMoments8 = 4 };

struct OptTensor {
  void* param;
  const void* grad;
  float* master;
  void *m, *v;
  uint8_t *m_scale, *v_scale;
  int64_t n;
  float lr_factor, weight_decay;
  uint32_t flags;
  int32_t first;  // first chunk of the launch
};

constexpr int kOptTensors = 48;  // of one launch: with the other arguments 4 KB

struct OptList {
  OptTensor t[kOptTensors];
  int32_t count;
  int32_t chunks;
  int32_t base;  // number of the first tensor in the caller's list
  int32_t last;  // 1: the call's last launch, which advances the counter
};

struct OptHyper {
  double lr, beta1, beta2, log_beta1, log_beta2;
  float eps;
  uint32_t seed;
};

struct NormTensor {
  const void* grad;
  int64_t n;
  int32_t first;
  uint32_t flags;
};

struct NormList {
  NormTensor t[kNormTensors];
  int32_t count;
  int32_t chunks;
  int32_t add;  // 1: onto the partial sums of the launch before
};

// Where the gradients' factor comes from: `scale` (may be null: 1), or, with `slots`, the
// sums of squares of launch_square_sums, from which norm and scale are written too
struct GradScale {
  const float* scale;
  const double* slots;
  double max_norm;
  float *norm_out, *scale_out;
};

static_assert(sizeof(OptList) + sizeof(OptHyper) + sizeof(GradScale) + 16 <= 4096 && sizeof(NormList) + 64 <= 4096, "kernel arguments");

// past_caches: for master copies and moments
hipError_t launch_adamw(const OptList& l, const OptHyper& h, int32_t* counter, const float* lr_scale,
                        const GradScale& gs, bool past_caches, hipStream_t s);
// One launch over a list; the partial sums in `slots` [kNormSlots]
hipError_t launch_square_sums(const NormList& l, double* slots, hipStream_t s);
hipError_t launch_norm_scale(const double* slots, double max_norm, float* norm, float* scale, hipStream_t s);

}  // namespace moe
