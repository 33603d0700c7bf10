// AdamW over a list of tensors, moments in 32 or 8 bits, and the gradients' norm.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p -= lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay p)
//
// Every value is read and written once: HBM is the bound (28 bytes a value for
// bfloat16 parameters with a master copy and moments in 32 bits, 16 with moments
// in 8). A thread has 8 consecutive values, so 16 neighbouring lanes (a DPP row)
// have the 128 that share a scale. Workgroups take chunks of the whole list in
// turn; the list is in the kernel's arguments.
//
// The moments are updated in 64 bits, where a CU multiplies as fast as in
// 32: their codes then do not depend on how the two products are rounded.
//
// Measured in a graph: 67 million values, moments in 32 bits 361 us (5.2 TB/s), in 8 bits
// 209 us (5.1 TB/s), with their norm 386 and 233; 525 thousand values in 5 tensors 6.8 us,
// with their norm 11. (Traced one by one, behind other kernels: 368 and 228, the norm 35 to
// 40 and at best 27, its 134 MB at 5 TB/s.)
#include "common.h"
#include "e4m3.h"
#include "internal.h"
#include "optim.h"

namespace moe {

namespace {

constexpr int kVals = 8;

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// NT: master copies and moments pass by the last-level cache (256 MB), so that the
// gradients that the norm has just read stay there: a list of 8 million values or more
// whose gradients are at most 192 MB. Step with norm, NT / through the caches, 32-bit
// moments and 8-bit ones: 4 M values (through) 34 and 26 us, 8 M 54 / 58 and 39 / 43, 67 M
// 404 / 409 and 247 / 259, 134 M 850 / 817 and 511 / 512, 268 M 1720 / 1631 and 1031 / 1031.
// The step alone, whose gradients a kernel has just written (with that kernel): 8 M 54 / 59 and
// 37 / 42, 16 M 110 / 109 and 72 / 75, 67 M 438 / 430 and 272 / 278; not just written: 8 M 48 /
// 52 and 32 / 34, 16 M 92 / 98 and 58 / 62, 67 M 402 / 380 and 231 / 227.
template <bool NT, typename V>
__device__ __forceinline__ V load(const V* p) {
  return NT ? __builtin_nontemporal_load(p) : *p;
}

template <bool NT, typename V>
__device__ __forceinline__ void store(V* p, const V& v) {
  if (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// 8 values of a float32 or bfloat16 array from value i0 on; those at or past n are 0
template <bool B16, bool NT = false>
__device__ __forceinline__ void load_vals(const void* base, int64_t i0, int64_t n, bool whole, float* f) {
  if (whole) {
    if constexpr (B16) {
      const u32x4 q = *(const u32x4*)((const bf16_bits*)base + i0);
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        f[i] = (i & 1) ? __uint_as_float(q[i / 2] & 0xFFFF0000u) : __uint_as_float(q[i / 2] << 16);
    } else {
      const f32x4* p = (const f32x4*)((const float*)base + i0);
      const f32x4 a = load<NT>(p), b = load<NT>(p + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    f[i] = 0.0f;
    if (i0 + i < n) f[i] = B16 ? bf16_to_f32(((const bf16_bits*)base)[i0 + i]) : ((const float*)base)[i0 + i];
  }
}

template <bool B16, bool NT = false>
__device__ __forceinline__ void store_vals(void* base, int64_t i0, int64_t n, bool whole, const float* f) {
  if (whole) {
    if constexpr (B16) {
      u32x4 q;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      *(u32x4*)((bf16_bits*)base + i0) = q;
    } else {
      f32x4* p = (f32x4*)((float*)base + i0);
      store<NT>(p, f32x4{f[0], f[1], f[2], f[3]});
      store<NT>(p + 1, f32x4{f[4], f[5], f[6], f[7]});
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    if (i0 + i >= n) continue;
    if constexpr (B16) ((bf16_bits*)base)[i0 + i] = (bf16_bits)(pack_bf16x2(f[i], 0.0f) & 0xFFFFu);
    else ((float*)base)[i0 + i] = f[i];
  }
}

// 8 bytes of codes from i0 on
template <bool NT>
__device__ __forceinline__ u32x2 load_codes(const void* base, int64_t i0, int64_t n, bool whole) {
  const uint8_t* p = (const uint8_t*)base + i0;
  if (whole) return load<NT>((const u32x2*)p);
  u32x2 q = {0u, 0u};
#pragma unroll
  for (int i = 0; i < kVals; ++i)
    if (i0 + i < n) q[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  return q;
}

template <bool NT>
__device__ __forceinline__ void store_codes(void* base, int64_t i0, int64_t n, bool whole, const u32x2& q) {
  uint8_t* p = (uint8_t*)base + i0;
  if (whole) {
    store<NT>((u32x2*)p, q);
    return;
  }
#pragma unroll
  for (int i = 0; i < kVals; ++i)
    if (i0 + i < n) p[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
}

// e4m3 (E5 false) or e5m2 codes as float32 values
template <bool E5>
__device__ __forceinline__ void decode8(const u32x2& q, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 a = E5 ? __builtin_amdgcn_cvt_pk_f32_bf8(q[i], false) : __builtin_amdgcn_cvt_pk_f32_fp8(q[i], false);
    const f32x2 b = E5 ? __builtin_amdgcn_cvt_pk_f32_bf8(q[i], true) : __builtin_amdgcn_cvt_pk_f32_fp8(q[i], true);
    f[4 * i] = a[0];
    f[4 * i + 1] = a[1];
    f[4 * i + 2] = b[0];
    f[4 * i + 3] = b[1];
  }
}

// 2^e in 64 bits
__device__ __forceinline__ double pow2(int e) { return __longlong_as_double((long long)(1023 + e) << 52); }

// The smallest float32 that is not below x >= 0
__device__ __forceinline__ float up32(double x) {
  const float f = (float)x;
  return (double)f < x && f < INFINITY ? __uint_as_float(__float_as_uint(f) + 1u) : f;
}

// Exponent of the scale of a block whose largest second moment is x >= 0: the smallest e
// with x <= 1.75 2^(15 + e), in [-120, 120]. From the upper half of the double, a unit up
// where the lower one is not 0: float32 ends at 2^128, the codes 2^8 further on.
__device__ __forceinline__ int scale_exp_v(double x) {
  uint32_t hi = (uint32_t)__double2hiint(x) + (__double2loint(x) != 0 ? 1u : 0u);
  auto turn = [&](auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)hi, decltype(ctrl)::value, 0xF, 0xF, true);
  };
  // over the lanes of a DPP row, which have the 128 values of a scale
  hi = max(hi, turn(IntC<0x128>{}));
  hi = max(hi, turn(IntC<0x124>{}));
  hi = max(hi, turn(IntC<0x122>{}));
  hi = max(hi, turn(IntC<0x121>{}));
  // what is above 1.75 carries into the exponent's field
  return min(max((int)((hi + 0x3FFFFu) >> 20) - (1023 + 15), -120), 120);
}

// Code of x / 2^e with random number r < 2^16: e4m3 (3 bits of mantissa, bias 7) or
// e5m2 (2 bits, bias 15). x is sig 2^(exp - 20) with 21 bits of sig from the double's
// upper half; shifted to units of 2^-16 spacings, below the smallest normal those of
// that one, floor(|x| / s + r / 2^16) is an integer sum. The lower half of the
// double lies below those units and cannot change the floor.
template <bool E5>
__device__ __forceinline__ uint32_t encode(double x, int e, uint32_t r) {
  constexpr int M = E5 ? 2 : 3, BIAS = E5 ? 15 : 7;
  constexpr uint32_t TOP = E5 ? 0x40EC0000u : 0x407C0000u;  // upper halves of 57344.0 and 448.0
  const uint32_t full = (uint32_t)__double2hiint(x), hi = full & 0x7FFFFFFFu;
  const int up = (int)(hi >> 20) - (1024 - BIAS + e);  // exponent above that of the smallest normal
  const uint32_t sig = (hi & 0xFFFFFu) | 0x100000u;
  uint32_t c = ((sig >> min(4 - M + max(-up, 0), 31)) + r) >> 16;
  c += (uint32_t)max(up, 0) << M;
  if (E5) c = x > 0.0 ? max(c, 1u) : c;  // a second moment that is not 0
  if (hi > TOP + (uint32_t)(e << 20)) c = 0x7Fu;
  return E5 ? c : c | ((full >> 24) & 0x80u);
}

// b m + c d, products and sum rounded one by one: the same bits wherever they are computed.
// (A fused one is a step off in 64 bits; where the sum lies on a border of two codes, as
// one in five does for short factors, that would show.)
__device__ __forceinline__ double moment(double b, double m, double c, double d) {
#pragma clang fp contract(off)
  return b * m + c * d;
}

struct Hyper {
  double b1, b2, gs;
  float step, root, decay, eps;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), lr weight_decay
  uint32_t key;
};

// WHOLE: the workgroup's chunk ends inside the tensor. All loads then go out together; with
// the tail's branches between them the first was waited for before the second left.
template <bool G16, bool P16, bool S8, bool WHOLE, bool NT>
__device__ __forceinline__ void update_chunk(const OptTensor& T, const Hyper& h, int64_t i0) {
  const int64_t n = T.n;
  const bool whole = WHOLE || i0 + kVals <= n;
  float g[kVals], p[kVals], mf[kVals], vf[kVals];
  double m[kVals], v[kVals];
  load_vals<G16>(T.grad, i0, n, whole, g);
  load_vals<false, NT>(P16 ? T.master : (const float*)T.param, i0, n, whole, p);
  const int64_t block = i0 / kQBlock;
  const bool inside = WHOLE || i0 < n;
  if constexpr (S8) {
    const u32x2 mq = load_codes<NT>(T.m, i0, n, whole), vq = load_codes<NT>(T.v, i0, n, whole);
    const double ms = pow2(inside ? (int)T.m_scale[block] - 127 : 0), vs = pow2(inside ? (int)T.v_scale[block] - 127 : 0);
    decode8<false>(mq, mf);
    decode8<true>(vq, vf);
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      m[i] = (double)mf[i] * ms;
      v[i] = (double)vf[i] * vs;
    }
  } else {
    load_vals<false, NT>(T.m, i0, n, whole, mf);
    load_vals<false, NT>(T.v, i0, n, whole, vf);
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      m[i] = mf[i];
      v[i] = vf[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const double d = (double)g[i] * h.gs;
    m[i] = moment(h.b1, m[i], 1.0 - h.b1, d);
    v[i] = moment(h.b2, v[i], (1.0 - h.b2) * d, d);
    mf[i] = (float)m[i];
    vf[i] = (float)v[i];
    // the hardware's root and reciprocal, each within a unit in the last place: the move is
    // a small part of p (with eps >= 1e-15 a root that it takes for 0 does not count)
    const float move = h.step * mf[i] * __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_sqrtf(vf[i]), h.root, h.eps));
    p[i] = p[i] - fmaf(h.decay, p[i], move);
  }
  store_vals<false, NT>(P16 ? (void*)T.master : T.param, i0, n, whole, p);
  if constexpr (P16) store_vals<true>(T.param, i0, n, whole, p);
  if constexpr (S8) {
    double mt = 0.0, vt = 0.0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {  // values past the end are 0; NaN is left out
      mt = fmax(mt, fabs(m[i]));
      vt = fmax(vt, v[i]);
    }
    // (a first moment past float32 has the largest scale: 448 2^119 is within it)
    const int me = scale_byte(row16_max(up32(mt))) - 127, ve = scale_exp_v(vt);
    u32x2 mq = {0u, 0u}, vq = {0u, 0u};
    const uint32_t high = (uint32_t)((uint64_t)i0 >> 32) * 0x9E3779B9u;  // a chunk does not cross 2^32
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const uint32_t r = mix32(((uint32_t)(i0 + i) + h.key) ^ high);
      mq[i / 4] |= encode<false>(m[i], me, r & 0xFFFFu) << (8 * (i % 4));
      vq[i / 4] |= encode<true>(v[i], ve, r >> 16) << (8 * (i % 4));
    }
    store_codes<NT>(T.m, i0, n, whole, mq);
    store_codes<NT>(T.v, i0, n, whole, vq);
    if (inside && i0 % kQBlock == 0) {
      T.m_scale[block] = (uint8_t)(me + 127);
      T.v_scale[block] = (uint8_t)(ve + 127);
    }
  } else {
    store_vals<false, NT>(T.m, i0, n, whole, mf);
    store_vals<false, NT>(T.v, i0, n, whole, vf);
  }
}

template <bool G16, bool P16, bool S8, bool NT>
__device__ __forceinline__ void update(const OptTensor& T, const Hyper& h, int64_t first) {
  const int64_t i0 = first + threadIdx.x % kOptThreads * kVals;
  if (first + kOptChunk <= T.n) update_chunk<G16, P16, S8, true, NT>(T, h, i0);
  else update_chunk<G16, P16, S8, false, NT>(T, h, i0);
}

// First chunks of a list's tensors, one or two a lane, loaded together; the tensor of chunk
// c is the last whose first chunk is not above it. (A search through the arguments would
// wait for each of its steps.)
template <typename L, int N>
struct Finder {
  int first[(N + kWave - 1) / kWave];
  __device__ __forceinline__ explicit Finder(const L& l) {
#pragma unroll
    for (int i = 0; i * kWave < N; ++i) {
      const int j = i * kWave + threadIdx.x % kWave;
      first[i] = j < l.count ? l.t[j].first : INT32_MAX;
    }
  }
  __device__ __forceinline__ int tensor(int c) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i * kWave < N; ++i) n += __popcll(__ballot(first[i] <= c));
    return n - 1;
  }
};

// Sum over a workgroup of N threads, the same order and the same bits in each of them
template <int N>
__device__ __forceinline__ double block_sum(double v, double* slots) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  if (threadIdx.x % kWave == 0) slots[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < N / kWave; ++i) v += slots[i];
  return v;
}

// The factor that clips gradients of norm n, NaN when it is not finite (an infinite
// max_norm is not below an infinite n)
__device__ __forceinline__ float clip_scale(double n, double max_norm) {
  return !(n < INFINITY) ? NAN : n <= max_norm ? 1.0f : (float)(max_norm / n);
}

// Four chunks a workgroup side by side: each workgroup takes part in the count at the end,
// one after another (259 of them 2.7 us, 65 0.8).
constexpr int kAdamSide = 4;
template <bool NT>
__global__ __launch_bounds__(kAdamSide * kOptThreads) void adamw_kernel(const OptList l, const OptHyper o,
                                                            int32_t* __restrict__ counter,
                                                            const float* __restrict__ lr_scale, const GradScale g) {
  const int32_t before = __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  float gs = g.scale ? *g.scale : 1.0f;
  const float ls = lr_scale ? *lr_scale : 1.0f;
  const Finder<OptList, kOptTensors> find(l);
  if (g.slots) {  // every workgroup adds them for itself: a launch and its wait less
    static_assert(kNormSlots == kAdamSide * kOptThreads, "a sum for each thread");
    __shared__ double s_v[kAdamSide * kOptThreads / kWave];
    const double n = sqrt(block_sum<kAdamSide * kOptThreads>(g.slots[threadIdx.x], s_v));
    gs = clip_scale(n, g.max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      g.norm_out[0] = (float)n;
      if (g.scale_out) g.scale_out[0] = gs;
    }
  }
  const bool skip = gs != gs;
  if (!skip) {
    // 1 - b^t, good for float32 for every b below 1: 1 - b is a multiple of 2^-53 and so is, to first
    // order, 1 - b^t, which the difference of a rounded b^t therefore has exactly; the second order
    // is off by half of t (1 - b) of it where it is lost, below 2^-27 (5.3e-9 the most of 2^24 pairs)
    const double t = (double)(before + 1);
    const float c1 = (float)(1.0 - exp(t * o.log_beta1)), c2 = (float)(1.0 - exp(t * o.log_beta2));
    const float lr = (float)(o.lr * (double)ls);
    const uint32_t draw = (uint32_t)(before + 1) * 0x9E3779B9u;
    Hyper h;
    h.b1 = o.beta1;
    h.b2 = o.beta2;
    h.gs = gs;
    h.root = __builtin_amdgcn_rsqf(c2);
    h.eps = o.eps;
    // Workgroups side by side take neighbouring chunks: ranges of their own, all at the
    // same place of the memory channels' period at a time, took 28% longer for the norm.
    for (int c = __builtin_amdgcn_readfirstlane(blockIdx.x * kAdamSide + threadIdx.x / kOptThreads); c < l.chunks;
         c += gridDim.x * kAdamSide) {
      const int j = __builtin_amdgcn_readfirstlane(find.tensor(c));
      const OptTensor& T = l.t[j];
      const float f = lr * T.lr_factor;
      h.step = f / c1;
      h.decay = f * T.weight_decay;
      h.key = mix32(o.seed + mix32(draw + (uint32_t)(l.base + j)));
      const int64_t i0 = (int64_t)(c - T.first) * kOptChunk;
      switch (T.flags) {  // the same for the chunk's waves
        case 0: update<false, false, false, NT>(T, h, i0); break;
        case kGrad16: update<true, false, false, NT>(T, h, i0); break;
        case kParam16: update<false, true, false, NT>(T, h, i0); break;
        case kGrad16 | kParam16: update<true, true, false, NT>(T, h, i0); break;
        case kMoments8: update<false, false, true, NT>(T, h, i0); break;
        case kGrad16 | kMoments8: update<true, false, true, NT>(T, h, i0); break;
        case kParam16 | kMoments8: update<false, true, true, NT>(T, h, i0); break;
        default: update<true, true, true, NT>(T, h, i0); break;
      }
    }
  }
  if (!l.last) return;
  // The last workgroup to come here advances the counter: by then a wave that had a chunk has
  // made its updates from `before`, and one that had none does not need it. Nothing else
  // is passed on, so no fence: one of the device's scope writes the L2 back.
  __syncthreads();
  if (threadIdx.x == 0) {
    const int32_t n = __hip_atomic_fetch_add(counter + 1, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (n == (int32_t)gridDim.x - 1) {
      __hip_atomic_store(counter + 1, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (!skip) __hip_atomic_store(counter, before + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

__global__ __launch_bounds__(kOptThreads) void square_sums_kernel(const NormList l, double* __restrict__ slots) {
  __shared__ double s_v[kOptThreads / kWave];
  double sum = 0.0;
  constexpr int U = 4;  // chunks under way together
  const Finder<NormList, kNormTensors> find(l);
  for (int c0 = blockIdx.x; c0 < l.chunks; c0 += gridDim.x * U) {
    u32x4 q[U][2];
    uint32_t b16[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * (int)gridDim.x;
      b16[u] = 0;
      q[u][0] = q[u][1] = u32x4{0u, 0u, 0u, 0u};
      if (c >= l.chunks) continue;
      const NormTensor& T = l.t[__builtin_amdgcn_readfirstlane(find.tensor(c))];
      const int64_t first = (int64_t)(c - T.first) * kOptChunk, i = first + threadIdx.x * kVals;
      b16[u] = T.flags;
      if (first + kOptChunk <= T.n) {
        if (T.flags) {
          q[u][0] = *(const u32x4*)((const bf16_bits*)T.grad + i);
        } else {
          const u32x4* p = (const u32x4*)((const float*)T.grad + i);
          q[u][0] = p[0];
          q[u][1] = p[1];
        }
      } else {
        b16[u] = 0;
        float g[kVals];
        if (T.flags) load_vals<true>(T.grad, i, T.n, i + kVals <= T.n, g);
        else load_vals<false>(T.grad, i, T.n, i + kVals <= T.n, g);
#pragma unroll
        for (int v = 0; v < kVals; ++v) q[u][v / 4][v % 4] = __float_as_uint(g[v]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        const double g = __uint_as_float(!b16[u] ? q[u][i / 4][i % 4] : (i & 1) ? q[u][0][i / 2] & 0xFFFF0000u : q[u][0][i / 2] << 16);
        sum = fma(g, g, sum);
      }
    }
  }
  sum = block_sum<kOptThreads>(sum, s_v);
  if (threadIdx.x == 0) slots[blockIdx.x] = l.add ? slots[blockIdx.x] + sum : sum;
}

// The sums are added as moet_adamw_clipped's workgroups add them: the same bits
__global__ __launch_bounds__(kNormSlots) void norm_scale_kernel(const double* __restrict__ slots, double max_norm,
                                                                float* __restrict__ norm, float* __restrict__ scale) {
  __shared__ double s_v[kNormSlots / kWave];
  const double v = slots[threadIdx.x];
  const double n = sqrt(block_sum<kNormSlots>(v, s_v));
  if (threadIdx.x == 0) {
    norm[0] = (float)n;
    if (scale) scale[0] = clip_scale(n, max_norm);
  }
}

}  // namespace

hipError_t launch_adamw(const OptList& l, const OptHyper& h, int32_t* counter, const float* lr_scale,
                        const GradScale& gs, bool past_caches, hipStream_t s) {
  // a workgroup's 16 waves of up to 128 registers fill a CU
  const unsigned grid = (unsigned)max(1, min((l.chunks + kAdamSide - 1) / kAdamSide, device_cus()));
  hipLaunchKernelGGL(past_caches ? adamw_kernel<true> : adamw_kernel<false>, dim3(grid), dim3(kAdamSide * kOptThreads), 0, s, l, h, counter, lr_scale, gs);
  return hipGetLastError();
}

hipError_t launch_square_sums(const NormList& l, double* slots, hipStream_t s) {
  hipLaunchKernelGGL(square_sums_kernel, dim3(kNormSlots), dim3(kOptThreads), 0, s, l, slots);
  return hipGetLastError();
}

hipError_t launch_norm_scale(const double* slots, double max_norm, float* norm, float* scale, hipStream_t s) {
  hipLaunchKernelGGL(norm_scale_kernel, dim3(1), dim3(kNormSlots), 0, s, slots, max_norm, norm, scale);
  return hipGetLastError();
}

}  // namespace moe
