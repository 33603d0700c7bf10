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
// selections of 64 token ranges are counted in LDS (integers: any order gives
// the same), then every workgroup adds the 64 counts, reads its logits once and
// writes their gradient. The last workgroup to finish (a ticket) adds the
// workgroups' probability sums in workgroup order. No float atomics.
#include "common.h"
#include "internal.h"
#include "lds_dma.h"

namespace moe {

namespace {

constexpr int kCountBlocks = 64;   // token ranges counted side by side
constexpr int kBalThreads = 256;
constexpr int kBalBlocks = 256;    // most workgroups of the second launch

// part[block][0 .. E) = selections per expert of the block's tokens, part[block][E] = its valid tokens
__global__ __launch_bounds__(kBalThreads) void balance_count_kernel(const int32_t* __restrict__ idx,
                                                                    const uint8_t* __restrict__ mask,
                                                                    int32_t* __restrict__ part,
                                                                    int32_t* __restrict__ ticket, int64_t T, int k,
                                                                    int E, int64_t per) {
  __shared__ int s_c[257];
  for (int e = threadIdx.x; e <= E; e += kBalThreads) s_c[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * per, t1 = min(T, t0 + per);
  for (int64_t i = t0 * k + threadIdx.x; i < t1 * k; i += kBalThreads) {
    const int e = idx[i];
    if (e >= 0 && e < E && (!mask || mask[i / k])) atomicAdd(&s_c[e], 1);
  }
  int nv = 0;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kBalThreads) nv += !mask || mask[t] ? 1 : 0;
  if (nv) atomicAdd(&s_c[E], nv);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kBalThreads) part[blockIdx.x * (E + 1) + e] = s_c[e];
}

// G lanes per token, four experts per lane: 4 l .. 4 l + 3 (VEC, E a multiple
// of 4, 16-byte accesses) or l, l + G, l + 2 G, l + 3 G.
template <int G, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_main_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ mask, const int32_t* __restrict__ part, int nparts,
    float coef, float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ mean_prob,
    float* __restrict__ dlogits, float* __restrict__ psum, int32_t* __restrict__ ticket, int64_t T, int k, int E) {
  constexpr int TPB = kBalThreads / G;  // tokens side by side
  __shared__ int s_c[257];
  __shared__ float s_p[TPB][4 * G];
  __shared__ int s_last;
  for (int e = threadIdx.x; e <= E; e += kBalThreads) {
    int c = 0;
#pragma unroll 8
    for (int b = 0; b < nparts; ++b) c += part[b * (E + 1) + e];
    s_c[e] = c;
    if (blockIdx.x == 0 && counts && e < E) counts[e] = c;
  }
  __syncthreads();
  const int l = threadIdx.x % G, grp = threadIdx.x / G;
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
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < T; t0 += (int64_t)gridDim.x * TPB) {
    const int64_t t = t0 + grp;
    const bool live = t < T && (!mask || mask[t] != 0);
    float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (live) {
      if constexpr (VEC) {
        if (has[0]) {
          const f32x4 q = *(const f32x4*)(logits + t * E + 4 * l);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = q[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (has[i]) v[i] = logits[t * E + l + i * G];
      }
    }
    float m = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    int cm = -1;  // the count of the most probable expert (the largest of several)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (has[i] && v[i] == m) cm = max(cm, cnt[i]);
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) cm = max(cm, __shfl_xor(cm, o, kWave));
    // m is -infinity for a row without any probability (and for one that is not live)
    float p[4], f[4], s = 0.0f, sf = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = m == -INFINITY && !isnan(v[i]) ? 0.0f : expf(v[i] - m);
      f[i] = (float)(cnt[i] - cm) * per;
      s += p[i];
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = has[i] ? p[i] * inv : 0.0f;
      acc[i] += p[i];
      sf = fmaf(p[i], f[i], sf);
    }
    if (dlogits) {
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) sf += __shfl_xor(sf, o, kWave);
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
  // the workgroup's probability sums, its token groups in order
#pragma unroll
  for (int i = 0; i < 4; ++i) s_p[grp][VEC ? 4 * l + i : l + i * G] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    float a = 0.0f;
    for (int g = 0; g < TPB; ++g) a += s_p[g][e];
    psum[(int64_t)blockIdx.x * E + e] = a;
  }
  // ticket: this workgroup's sums are visible to the device before it counts
  // itself in (every wave's stores acknowledged, then one release by wave 0);
  // the last one sees all of them
  wait_vmem<0>();
  __syncthreads();
  if (threadIdx.x == 0) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    s_last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  double part_loss = 0.0;
  __shared__ double s_l[kBalThreads];
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    double a = 0.0;
#pragma unroll 8
    for (unsigned b = 0; b < gridDim.x; ++b) a += psum[(int64_t)b * E + e];
    const double P = n > 0 ? a / n : 0.0;
    if (mean_prob) mean_prob[e] = (float)P;
    part_loss += P * s_c[e];
  }
  s_l[threadIdx.x] = part_loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = 0.0;
    for (int i = 0; i < min(E, kBalThreads); ++i) a += s_l[i];
    *loss = n > 0 ? (float)((double)coef * E * a / ((double)n * k)) : 0.0f;
  }
}

}  // namespace

size_t balance_ws_ints(const moe_problem_t& p) {
  return 64 + (size_t)kCountBlocks * (p.E + 1) + (size_t)kBalBlocks * p.E;
}

hipError_t launch_balance(const moe_problem_t& p, const float* logits, const int32_t* idx, const uint8_t* mask,
                          float coef, float* loss, int32_t* counts, float* mean_prob, float* dlogits, int32_t* ws,
                          hipStream_t s) {
  int32_t* const ticket = ws;
  int32_t* const part = ws + 64;
  float* const psum = (float*)(part + (size_t)kCountBlocks * (p.E + 1));
  // at least 64 tokens a range: small batches need few partial counts
  const int64_t per = max(ceil_div(p.T, kCountBlocks), (int64_t)64);
  const int nparts = (int)ceil_div(p.T, per);
  hipLaunchKernelGGL(balance_count_kernel, dim3((unsigned)nparts), dim3(kBalThreads), 0, s, idx, mask, part, ticket,
                     p.T, p.k, p.E, per);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool vec = p.E % 4 == 0;
  int g = 1;
  while (4 * g < p.E) g <<= 1;
#define MOE_BALANCE(G)                                                                                            \
  case G: {                                                                                                       \
    const unsigned blocks = (unsigned)min(ceil_div(p.T, kBalThreads / G), (int64_t)kBalBlocks);                   \
    if (vec)                                                                                                      \
      hipLaunchKernelGGL((balance_main_kernel<G, true>), dim3(blocks), dim3(kBalThreads), 0, s, logits, mask,     \
                         (const int32_t*)part, nparts, coef, loss, counts, mean_prob, dlogits, psum, ticket, p.T, \
                         p.k, p.E);                                                                               \
    else                                                                                                          \
      hipLaunchKernelGGL((balance_main_kernel<G, false>), dim3(blocks), dim3(kBalThreads), 0, s, logits, mask,    \
                         (const int32_t*)part, nparts, coef, loss, counts, mean_prob, dlogits, psum, ticket, p.T, \
                         p.k, p.E);                                                                               \
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
  return hipGetLastError();
}

}  // namespace moe
