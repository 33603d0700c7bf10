// Load-balancing loss of the router, per-expert counts and the gradient.
//
// "Distributed training part 4" (jesamkim's AI tech blog), section 3, has the
// router choose k of E experts per token; nothing in the layer keeps the choice
// even. With n valid tokens, p_t = softmax(logits_t), counts_e the selections of
// expert e, f_e = counts_e / (n k) and P_e the mean of p_te over them:
//   loss = coef E sum_e f_e P_e
//   dlogits_te = (coef E / n) p_te (f_e - sum_e' f_e' p_te')
// The last bracket is a small difference of shares. It does not change when all
// f move by the same amount, so f is taken from the row's most probable expert
// m: f'_e = (counts_e - counts_m) / (n k), an exact integer difference, and the
// large term p_m f'_m is zero.
//
// The gradient needs every count and the loss every p, so two launches: the
// selections of 32 token ranges are counted in LDS (integers: any order gives
// the same), then every workgroup adds the 32 counts, reads its logits once and
// writes their gradient. The last workgroup to finish (a ticket) adds the
// workgroups' probability sums in a fixed order. No float atomics. A batch of up
// to four rounds of one workgroup counts for itself: one launch.
//
// Statistics are float32 within a row and 64-bit across rows, so that the means'
// error does not grow with the batch; what a workgroup sends to the last one is
// rounded to float32 once, half a unit of its sum, as the mean itself is.
//
// Measured: 64 tokens of 8 experts 5.2 us of GPU time, 8192 of 64 3 + 9, 16384 of
// 256 with a mask 5.7 + 22 (34 MB, 7 us at the rate of a copy: the rows' arithmetic
// takes about 9, the counts before it and the ticket after it the rest).
#include "common.h"
#include "e4m3.h"
#include "internal.h"
#include "lds_dma.h"

namespace moe {

namespace {

constexpr int kCountBlocks = 32;    // token ranges counted side by side
constexpr int kBalThreads = 1024;
constexpr int kBalBlocks = 256;     // most workgroups of the second launch
constexpr int kBalBlocksFew = 128;  // and while that leaves each at most four rounds

// s_c[0 .. E) += selections per expert of tokens [t0, t1), s_c[E] += their valid ones
__device__ __forceinline__ void count_tokens(const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
                                             int64_t t0, int64_t t1, int k, int E, int* s_c) {
  int nv = 0;
  const uint32_t n = t1 > t0 ? (uint32_t)((t1 - t0) * k) : 0u;  // T k fits in 31 bits
  const int32_t* const p = idx + t0 * k;
#pragma unroll 4
  for (uint32_t i = threadIdx.x; i < n; i += kBalThreads) {
    const int e = p[i];
    const bool valid = !mask || mask[t0 + i / (uint32_t)k];  // loaded beside e, not behind it
    if (valid && e >= 0 && e < E) atomicAdd(&s_c[e], 1);
  }
  if (mask) {
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kBalThreads) nv += mask[t] ? 1 : 0;
  } else if (threadIdx.x == 0) {
    nv = (int)max(t1 - t0, (int64_t)0);
  }
  if (nv) atomicAdd(&s_c[E], nv);
}

// part[block][0 .. E) = selections per expert of the block's tokens, part[block][E] = its valid tokens
__global__ __launch_bounds__(kBalThreads) void balance_count_kernel(const int32_t* __restrict__ idx,
                                                                    const uint8_t* __restrict__ mask,
                                                                    int32_t* __restrict__ part,
                                                                    int32_t* __restrict__ ticket, int64_t T, int k,
                                                                    int E, int64_t per) {
  __shared__ int s_c[257];
  if (threadIdx.x <= E) s_c[threadIdx.x] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * per;
  count_tokens(idx, mask, t0, min(T, t0 + per), k, E, s_c);
  __syncthreads();
  if (threadIdx.x <= E) part[blockIdx.x * (E + 1) + threadIdx.x] = s_c[threadIdx.x];
}

// Sum and maximum over the G lanes of a group; inside a DPP row by rotations
// (every lane of the row is active)
template <int G, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  if constexpr (G >= 2) v = op(v, dpp<0xB1>(v));         // quad_perm 1, 0, 3, 2
  if constexpr (G >= 4) v = op(v, dpp<0x4E>(v));         // quad_perm 2, 3, 0, 1
  if constexpr (G >= 8) v = op(v, dpp<0x141>(v));        // row_half_mirror
  if constexpr (G >= 16) v = op(v, dpp<0x140>(v));       // row_mirror
  if constexpr (G >= 32) v = op(v, __shfl_xor(v, 16, kWave));
  if constexpr (G >= 64) v = op(v, __shfl_xor(v, 32, kWave));
  return v;
}

// G lanes per token, four experts per lane: 4 l .. 4 l + 3 (VEC, E a multiple
// of 4, 16-byte accesses) or l, l + G, l + 2 G, l + 3 G. ALONE: one workgroup
// that counts for itself.
template <int G, bool VEC, bool ALONE>
__global__ __launch_bounds__(kBalThreads) void balance_main_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ part, int nparts, float coef, float* __restrict__ loss, int32_t* __restrict__ counts,
    float* __restrict__ mean_prob, float* __restrict__ dlogits, float* __restrict__ psum, int32_t* __restrict__ ticket,
    int64_t T, int k, int E) {
  constexpr int TPB = kBalThreads / G;  // tokens side by side
  __shared__ int s_c[257];
  __shared__ __attribute__((aligned(16))) double s_p[TPB * 4 * G];
  __shared__ double s_d[16 * 4 * G > kBalThreads ? 16 * 4 * G : kBalThreads];
  __shared__ int s_last;
  const int tid = threadIdx.x;
  if (tid <= E) s_c[tid] = 0;
  __syncthreads();
  if constexpr (ALONE) {
    count_tokens(idx, mask, 0, T, k, E, s_c);
  } else {
    const int step = kBalThreads % (E + 1);
    int col = tid % (E + 1);
#pragma unroll 4
    for (int i = tid; i < nparts * (E + 1); i += kBalThreads) {
      const int c = part[i];
      if (c) atomicAdd(&s_c[col], c);
      col += step;
      if (col > E) col -= E + 1;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && counts && tid < E) counts[tid] = s_c[tid];
  const int l = tid % G, grp = tid / G;
  const int n = s_c[E];
  const float w = n > 0 ? (float)((double)coef * E / n) : 0.0f;
  const float per = n > 0 ? (float)(1.0 / ((double)n * k)) : 0.0f;
  int cnt[4];
  bool has[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = VEC ? 4 * l + i : l + i * G;
    has[i] = e < E;
    cnt[i] = has[i] ? s_c[e] : 0;
  }
  const auto vmax = [](float a, float b) { return fmaxf(a, b); };
  const auto vadd = [](float a, float b) { return a + b; };
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  // a token's logits and mask, loaded a round ahead (those of masked tokens are dropped)
  struct Row {
    float v[4];
    bool live;
  };
  auto load = [&](int64_t t) {
    Row r;
    r.live = t < T;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = -INFINITY;
    if (r.live) {
      if (mask) r.live = mask[t] != 0;
      if constexpr (VEC) {
        if (has[0]) {
          const f32x4 q = *(const f32x4*)(logits + t * E + 4 * l);
#pragma unroll
          for (int i = 0; i < 4; ++i) r.v[i] = q[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (has[i]) r.v[i] = logits[t * E + l + i * G];
      }
    }
    return r;
  };
  const int64_t stride = (int64_t)gridDim.x * TPB;
  Row next = load((int64_t)blockIdx.x * TPB + grp);
  for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < T; t0 += stride) {
    const int64_t t = t0 + grp;
    const Row row = next;
    next = load(t + stride);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = row.live ? row.v[i] : -INFINITY;
    const float m = group_reduce<G>(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), vmax);
    int cm = -1;  // the count of the most probable expert (the largest of several)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (has[i] && v[i] == m) cm = max(cm, cnt[i]);
    cm = __float_as_int(group_reduce<G>(__int_as_float(cm), [](float a, float b) {
      return __int_as_float(max(__float_as_int(a), __float_as_int(b)));
    }));
    // m is -infinity for a row without any probability (and for one that is not live)
    float p[4], f[4], s = 0.0f, sf = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = m == -INFINITY && !isnan(v[i]) ? 0.0f : expf(v[i] - m);
      f[i] = (float)(cnt[i] - cm) * per;
      s += p[i];
    }
    s = group_reduce<G>(s, vadd);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = has[i] ? p[i] * inv : 0.0f;
      acc[i] += p[i];
      sf = fmaf(p[i], f[i], sf);
    }
    if (dlogits) {
      sf = group_reduce<G>(sf, vadd);
      if (t < T) {
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = w * p[i] * (f[i] - sf);
        if constexpr (VEC) {
          if (has[0]) *(f32x4*)(dlogits + t * E + 4 * l) = f32x4{d[0], d[1], d[2], d[3]};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (has[i]) dlogits[t * E + l + i * G] = d[i];
        }
      }
    }
  }
  // the workgroup's probability sums: slices of its token groups, then the slices in order
#pragma unroll
  for (int i = 0; i < 4; ++i) s_p[grp * 4 * G + (VEC ? 4 * l + i : l + i * G)] = acc[i];
  __syncthreads();
  constexpr int EW = 4 * G, SL = kBalThreads / EW;  // experts side by side, slices
  const int e = tid % EW, sl = tid / EW;
  double a = 0.0;
#pragma unroll 8
  for (int g = sl; g < TPB; g += SL) a += s_p[g * EW + e];
  s_d[tid] = a;
  __syncthreads();
  double P = 0.0;  // threads below EW: the expert's sum (0 past E)
  if (tid < EW)
#pragma unroll
    for (int i = 0; i < SL; ++i) P += s_d[i * EW + tid];
  if constexpr (!ALONE) {
    // Ticket: a workgroup's sums go past the L2 of its XCD (atomic stores of device
    // scope) and are acknowledged before it counts itself in; the last one reads
    // them the same way. A release fence instead would write the
    // whole L2 back, with the gradients in it, once per workgroup (2 to 3 us).
    if (tid < EW)
      __hip_atomic_store(psum + (int64_t)blockIdx.x * EW + tid, (float)P, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    wait_vmem<0>();
    __syncthreads();
    if (tid == 0)
      s_last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    // slices of the workgroups side by side, two experts a load, then the slices in order
    constexpr int FS = EW / 2 * 16 <= kBalThreads ? 16 : 8;
    const int pair = tid % (EW / 2), fs = tid / (EW / 2);
    if (fs < FS) {
      double q0 = 0.0, q1 = 0.0;
      for (int b0 = fs; b0 < (int)gridDim.x; b0 += kBalBlocksFew)
#pragma unroll
        for (int i = 0; i < kBalBlocksFew / FS; ++i) {
          const int b = b0 + i * FS;
          uint64_t u = 0;
          if (b < (int)gridDim.x)
            u = __hip_atomic_load((const uint64_t*)(psum + (int64_t)b * EW) + pair, __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_AGENT);
          q0 += __uint_as_float((uint32_t)u);
          q1 += __uint_as_float((uint32_t)(u >> 32));
        }
      s_d[fs * EW + 2 * pair] = q0;
      s_d[fs * EW + 2 * pair + 1] = q1;
    }
    __syncthreads();
    P = 0.0;
    if (tid < E)
#pragma unroll
      for (int i = 0; i < FS; ++i) P += s_d[i * EW + tid];
    __syncthreads();
  }
  P = n > 0 ? P / n : 0.0;
  if (tid < E && mean_prob) mean_prob[tid] = (float)P;
  // sum of counts times means over the experts: wave by wave, then the waves in order
  double c = tid < E ? P * s_c[tid] : 0.0;
  for (int o = 32; o > 0; o >>= 1) c += __shfl_xor(c, o, kWave);
  __syncthreads();
  if (tid % kWave == 0) s_d[tid / kWave] = c;
  __syncthreads();
  if (tid == 0) {
    c = 0.0;
    for (int i = 0; i < (E + kWave - 1) / kWave; ++i) c += s_d[i];
    *loss = n > 0 ? (float)((double)coef * E * c / ((double)n * k)) : 0.0f;
  }
}

// lanes of four experts each
int lanes_per_token(int E) {
  int g = 1;
  while (4 * g < E) g <<= 1;
  return g;
}

// the selections of every token range, up to a multiple of 16 bytes
size_t count_ints(int E) { return ((size_t)kCountBlocks * (E + 1) + 3) / 4 * 4; }

}  // namespace

size_t balance_ws_ints(const moe_problem_t& p) {
  // ticket; selections; probability sums of up to 256 padded experts
  return 64 + count_ints(p.E) + (size_t)kBalBlocks * 4 * lanes_per_token(p.E);
}

hipError_t launch_balance(const moe_problem_t& p, const float* logits, const int32_t* idx, const uint8_t* mask,
                          float coef, float* loss, int32_t* counts, float* mean_prob, float* dlogits, int32_t* ws,
                          hipStream_t s) {
  int32_t* const ticket = ws;
  int32_t* const part = ws + 64;
  float* const psum = (float*)(part + count_ints(p.E));
  const bool vec = p.E % 4 == 0;
  const int g = lanes_per_token(p.E);
  // Up to four rounds of one workgroup need no second one. Measured in graphs at 64
  // experts, top-8 (64 tokens a round), in one launch against two: 2 rounds 6.0
  // against 8.2 us, 4 rounds 8.5 and 8.5 (where a launch less is worth its 4 us on
  // the host), 8 rounds 13.5 against 8.5.
  const bool alone = p.T <= (int64_t)4 * (kBalThreads / g);
  // The last workgroup reads every other one's sums: 128 instead of 256 workgroups
  // take 16.1 instead of 18.6 us at 4096 tokens of 256 experts, 19.3 instead of 20.5
  // at 8192, 25.8 instead of 24.6 at 16384 (8 rounds; graph replays of both launches).
  const int64_t most = p.T <= (int64_t)4 * kBalBlocksFew * (kBalThreads / g) ? kBalBlocksFew : kBalBlocks;
  // at least 64 tokens a range: small batches need few partial counts
  const int64_t per = max(ceil_div(p.T, kCountBlocks), (int64_t)64);
  const int nparts = (int)ceil_div(p.T, per);
  if (!alone) {
    hipLaunchKernelGGL(balance_count_kernel, dim3((unsigned)nparts), dim3(kBalThreads), 0, s, idx, mask, part, ticket,
                       p.T, p.k, p.E, per);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#define MOE_BALANCE_LAUNCH(G, VEC, ALONE)                                                                         \
  hipLaunchKernelGGL((balance_main_kernel<G, VEC, ALONE>), dim3(ALONE ? 1u : blocks), dim3(kBalThreads), 0, s,    \
                     logits, idx, mask, (const int32_t*)part, nparts, coef, loss, counts, mean_prob, dlogits,     \
                     psum, ticket, p.T, p.k, p.E)
#define MOE_BALANCE(G)                                                                                            \
  case G: {                                                                                                       \
    const unsigned blocks = (unsigned)min(ceil_div(p.T, kBalThreads / G), most);                   \
    if (alone && vec) MOE_BALANCE_LAUNCH(G, true, true);                                                          \
    else if (alone) MOE_BALANCE_LAUNCH(G, false, true);                                                           \
    else if (vec) MOE_BALANCE_LAUNCH(G, true, false);                                                             \
    else MOE_BALANCE_LAUNCH(G, false, false);                                                                     \
    break;                                                                                                        \
  }
  switch (g) {
    MOE_BALANCE(1)
    MOE_BALANCE(2)
    MOE_BALANCE(4)
    MOE_BALANCE(8)
    MOE_BALANCE(16)
    MOE_BALANCE(32)
    MOE_BALANCE(64)
    default:
      return hipErrorInvalidValue;
  }
#undef MOE_BALANCE
#undef MOE_BALANCE_LAUNCH
  return hipGetLastError();
}

}  // namespace moe
