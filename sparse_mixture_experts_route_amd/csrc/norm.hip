// Root-mean-square norm in front of the layer, with the residual's addition
// and 8-bit rows, and its backward pass.
//
//   h = x + residual (rounded), r = 1 / sqrt(mean(h^2) + eps), y = h r gain
//   z = h r, a = dy gain: dx = r (a - z mean(a z)) + dh, dgain = sum over tokens of dy z
//
// Both directions touch every row once and are bound by HBM. A row stays in
// the registers of the TPR threads that share it (VPT pieces of 8 values each):
// it is read once, its sum of squares is reduced, and y, its 8-bit form and h
// leave from the same registers. 16 neighbouring lanes hold the 128 values of
// one 8-bit block, so a block's largest magnitude is a reduction within a DPP
// row. The mean square and r are taken in 64 bits (hidden behind the memory
// traffic), everything else in float32, but where a code depends on more. Codes
// round y to e4m3 (half a step, 2^-4), h and y are rounded to the rows' type.
//
// Measured: 16384 rows of 7168 bf16 with residual, y and 8-bit y 181 us, 5.8 TB/s;
// forward and backward of 8192 rows of 2048 51 us, 5.3 TB/s of 268 MB, which the
// last-level cache holds in part (61 us on inputs that change from call to call);
// 8 rows of 7168 3.1 us, a chain of latencies; 8-bit rows alone of 16384 rows of 7168
// 66 us, 5.4 TB/s.
// dgain's partial sums, a row per workgroup of the backward launch, are added by
// a second launch; up to 1024 rows its columns have workgroups of their own.
#include "common.h"
#include "e4m3.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

// 8 consecutive values of a row: one 16-byte piece of bfloat16, two of float32
template <bool BF16>
struct Piece8 {
  u32x4 v[BF16 ? 1 : 2];
};

template <bool BF16, bool NT = false>
__device__ __forceinline__ Piece8<BF16> load8(const void* base, int64_t piece) {
  Piece8<BF16> r;
  const u32x4* p = (const u32x4*)base + piece * (BF16 ? 1 : 2);
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.v[i] = NT ? __builtin_nontemporal_load(p + i) : p[i];
  return r;
}

template <bool BF16>
__device__ __forceinline__ void widen8(const Piece8<BF16>& q, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = BF16 ? ((i & 1) ? __uint_as_float(q.v[0][i / 2] & 0xFFFF0000u) : __uint_as_float(q.v[0][i / 2] << 16))
                : __uint_as_float(q.v[BF16 ? 0 : i / 4][i % 4]);
}

// rounds 8 values to the row's type and stores them
template <bool BF16>
__device__ __forceinline__ Piece8<BF16> narrow8(const float* f) {
  Piece8<BF16> r;
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[0][i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i / 4][i % 4] = __float_as_uint(f[i]);
  }
  return r;
}

template <bool BF16, bool NT = false>
__device__ __forceinline__ void store8(void* base, int64_t piece, const Piece8<BF16>& q) {
  u32x4* p = (u32x4*)base + piece * (BF16 ? 1 : 2);
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
    if (NT) __builtin_nontemporal_store(q.v[i], p + i);
    else p[i] = q.v[i];
  }
}

// dpp of a float or a double
template <int CTRL, typename S>
__device__ __forceinline__ S dpp_any(S v) {
  if constexpr (sizeof(S) == 4) {
    return dpp<CTRL>(v);
  } else {
    u32x2 u = __builtin_bit_cast(u32x2, v);
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u[i], CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(S, u);
  }
}

// v + lo, |lo| at most half a step of v, to float32 by rounding to odd: a further
// rounding to fewer bits then gives what v + lo itself would (v alone may sit on a
// tie that v + lo is beside). 0, infinities and NaN stay.
__device__ __forceinline__ float to_odd(float v, float lo) {
  const int b = (int)__float_as_uint(v), differ = (b ^ (int)__float_as_uint(lo)) >> 31;  // -1: lo points to 0
  return lo != 0.0f && fabsf(lo) < fabsf(v) ? __uint_as_float((uint32_t)((b + differ) | 1)) : v;
}

// 1 / sqrt(v), v >= 0: the hardware's estimate and one Newton step (which 0 and
// infinity, whose estimates are exact, skip)
__device__ __forceinline__ double rsqrt64(double v) {
  const double r = __builtin_amdgcn_rsq(v);
  const double n = r * fma(-0.5 * v * r, r, 1.5);
  return v > 0.0 && v < INFINITY ? n : r;
}

// Sum over the TPR threads of a row, the same bits in each of them. `slots`
// holds one value per wave; a barrier separates two uses.
template <int TPR, typename S>
__device__ __forceinline__ S row_sum(S v, S* slots) {
  v += dpp_any<0xB1>(v);   // quad_perm 1, 0, 3, 2
  v += dpp_any<0x4E>(v);   // quad_perm 2, 3, 0, 1
  v += dpp_any<0x141>(v);  // row_half_mirror
  v += dpp_any<0x140>(v);  // row_mirror
  v += __shfl_xor(v, 16, kWave);
  v += __shfl_xor(v, 32, kWave);
  if constexpr (TPR > kWave) {
    const int wave = threadIdx.x / kWave, first = threadIdx.x / TPR * (TPR / kWave);
    if (threadIdx.x % kWave == 0) slots[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < TPR / kWave; ++i) v += slots[first + i];
  }
  return v;
}

// NT: the rows pass by the caches (see launch_add_rmsnorm)
template <bool BF16, int TPR, int VPT, bool NT>
__global__ __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads) void add_rmsnorm_kernel(
    const void* __restrict__ x, const void* __restrict__ residual, const void* __restrict__ gain, float eps,
    void* __restrict__ h, void* __restrict__ y, uint8_t* __restrict__ y8, uint8_t* __restrict__ y_scale,
    float* __restrict__ rstd, int64_t T, int nvec, double inv_d) {
  constexpr int THREADS = TPR > kNormThreads ? TPR : kNormThreads;
  __shared__ double s_sum[THREADS / kWave];
  const int j = threadIdx.x % TPR;  // place in the row
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (THREADS / TPR) + threadIdx.x / TPR;
  const bool live = t < T;
  if (TPR <= kWave && !live) return;  // a whole wave: no barrier below
  const int64_t row = (live ? t : T - 1) * nvec;
  constexpr bool EARLY = VPT <= 2;  // gain's load does not wait for the sum; more pieces would cost registers
  Piece8<BF16> in[VPT], res[VPT], gn[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * TPR + j;
    if (c < nvec) {
      if (EARLY) gn[i] = load8<BF16>(gain, c);
      in[i] = load8<BF16, NT>(x, row + c);
      if (residual) res[i] = load8<BF16, NT>(residual, row + c);
    }
  }
  float v[VPT][8];
  double ss = 0.0;  // one rounding of r: its error would be every value's of the row
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * TPR + j;
    if (c < nvec) {
      widen8<BF16>(in[i], v[i]);
      if (residual) {
        float b[8];
        widen8<BF16>(res[i], b);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[i][q] += b[q];
        in[i] = narrow8<BF16>(v[i]);
        if (live) store8<BF16, NT>(h, row + c, in[i]);
        widen8<BF16>(in[i], v[i]);  // the norm is taken of the stored h
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fma((double)v[i][q], (double)v[i][q], ss);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[i][q] = 0.0f;
    }
  }
  ss = row_sum<TPR>(ss, s_sum);
  const double r64 = rsqrt64(ss * inv_d + (double)eps);
  const float r = (float)r64, r_lo = (float)(r64 - (double)r);
  if (rstd && live && j == 0) rstd[t] = r;
  if (!y && !y8) return;  // the same for every thread
  const int64_t cp = code_pitch((int64_t)nvec * 8), sp = scale_pitch((int64_t)nvec * 8);
  const int kb = (int)(cp / kQBlock);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * TPR + j;
    if (c < nvec) {
      float g[8], h8[8];
      widen8<BF16>(EARLY ? gn[i] : load8<BF16>(gain, c), g);
      uint32_t near = ~0u;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        h8[q] = v[i][q];
        v[i][q] = v[i][q] * r * g[q];
        near = min(near, (__float_as_uint(v[i][q]) + 4u) << 13);
      }
      if (y && live) store8<BF16, NT>(y, row + c, narrow8<BF16>(v[i]));
      // Codes and scales go by y in more bits than float32 has. That changes them
      // where y is within 3 of its own steps (three roundings) of a value whose low
      // 19 bits are 0, as all ties of e4m3 and steps of the scale are: one wave in
      // 100 does this for random values (8 rows of 7168 3.0 -> 3.1 us, 4096 of 4096 22.6 -> 23.8;
      // correcting every value 3.6 and 24.9). Without it one code in 10^6 is a step off.
      if (y8 && __any(near <= 8u << 13)) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float z = h8[q] * r, z_lo = fmaf(h8[q], r_lo, fmaf(h8[q], r, -z));
          const float c_lo = z_lo * g[q], w = fmaf(z, g[q], c_lo);
          if (fabsf(v[i][q]) < INFINITY) v[i][q] = to_odd(w, fmaf(z, g[q], -w) + c_lo);
        }
      }
    }
    if (y8) {
      float m = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(v[i][q]));
      const int byte = scale_byte(row16_max(m));  // the lanes of a block: pieces 16 b .. 16 b + 15
      const float inv = inv_scale(byte);
      u32x2 o;
      o[0] = encode4(v[i][0], v[i][1], v[i][2], v[i][3], inv);
      o[1] = encode4(v[i][4], v[i][5], v[i][6], v[i][7], inv);
      if (live && c < kb * 16) {  // a last half block ends in zero codes
        if (NT) __builtin_nontemporal_store(o, (u32x2*)(y8 + t * cp + (int64_t)c * 8));
        else *(u32x2*)(y8 + t * cp + (int64_t)c * 8) = o;
        if (c % 16 == 0) y_scale[t * sp + c / 16] = (uint8_t)byte;
      }
    }
  }
  if (y8 && live && kb + j < sp) y_scale[t * sp + kb + j] = 0;
}

// 8-bit rows of x alone: one thread per piece of 8 values
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ x, uint8_t* __restrict__ x8,
                                                            uint8_t* __restrict__ x_scale, int64_t T, int nvec) {
  const int64_t cp = code_pitch((int64_t)nvec * 8), sp = scale_pitch((int64_t)nvec * 8);
  const int pv = (int)(cp / 8);  // pieces per padded row, a multiple of 16
  const int64_t n = T * pv;
  for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < n; i0 += (int64_t)gridDim.x * 256) {
    const int64_t i = i0 + threadIdx.x, t = min(i, n - 1) / pv;
    const int c = (int)(i - t * pv);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < n && c < nvec) widen8<BF16>(load8<BF16>(x, t * nvec + c), v);
    float m = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(v[q]));
    const int byte = scale_byte(row16_max(m));
    const float inv = inv_scale(byte);
    u32x2 o;
    o[0] = encode4(v[0], v[1], v[2], v[3], inv);
    o[1] = encode4(v[4], v[5], v[6], v[7], inv);
    if (i < n) {
      *(u32x2*)(x8 + i * 8) = o;
      if (c % 16 == 0) x_scale[t * sp + c / 16] = (uint8_t)byte;
      // the bytes past the last block, written by the row's first pieces
      for (int q = pv / 16 + c; c < 16 && q < sp; q += 16) x_scale[t * sp + q] = 0;
    }
  }
}

// Few rows: dgain in the same launch. It needs r, which the call is given, and no
// sum over a row, so workgroups of their own add 32 columns over all rows: 128 rows
// side by side, 8 columns a thread. Rows are shared out as without it: dx has the
// same bits.
constexpr int kFewThreads = 512, kFewCols = 32;
template <bool BF16>
__device__ __forceinline__ void dgain_columns(const void* __restrict__ h, const float* __restrict__ rstd,
                                              const void* __restrict__ dy, float* __restrict__ dgain, int64_t T,
                                              int nvec, int col0, float (*s_w)[kFewCols]) {
  constexpr int CT = kFewCols / 8;  // threads side by side in a row
  const int c = threadIdx.x % CT, wave = threadIdx.x / kWave;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t t = threadIdx.x / CT; t < T; t += kFewThreads / CT) {
    float z[8], d[8];
    widen8<BF16>(load8<BF16>(h, t * nvec + col0 / 8 + c), z);
    widen8<BF16>(load8<BF16>(dy, t * nvec + col0 / 8 + c), d);
    const float r = rstd[t];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = fmaf(d[q], z[q] * r, acc[q]);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
#pragma unroll
    for (int o = CT; o < kWave; o <<= 1) acc[q] += __shfl_xor(acc[q], o, kWave);
    if (threadIdx.x % kWave < CT) s_w[wave][c * 8 + q] = acc[q];
  }
  __syncthreads();
  if (threadIdx.x < kFewCols) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewThreads / kWave; ++w) v += s_w[w][threadIdx.x];
    dgain[col0 + threadIdx.x] = v;
  }
}

// A block takes rows blockIdx, blockIdx + gridDim, ... of its row groups and
// keeps its share of dgain in registers; the row groups of the block are then
// added through LDS and leave as one float32 row of `part`. 1024 threads of a row
// wider than 16384 have 128 registers each, too few for h, dy, dh and the sums: 25
// spill in bf16 and 68 in float32, and 4096 rows of 32768 take 325 and 603 us (3.3 and
// 3.6 TB/s) where 16384 take 128 and 234 (4.2 and 4.6). FEW: workgroups from
// `row_blocks` on add dgain by columns, the others leave it out.
template <bool BF16, int TPR, int VPT, bool FEW>
__global__ __launch_bounds__(FEW ? kFewThreads : TPR > kNormThreads ? TPR : kNormThreads) void rmsnorm_backward_kernel(
    const void* __restrict__ h, const void* __restrict__ gain, const float* __restrict__ rstd,
    const void* __restrict__ dy, const void* __restrict__ dh, void* __restrict__ dx, float* __restrict__ part,
    int64_t T, int nvec, float inv_d, int row_blocks) {
  constexpr int THREADS = FEW ? kFewThreads : TPR > kNormThreads ? TPR : kNormThreads;
  constexpr int RPB = THREADS / TPR;
  __shared__ float s_sum[2][THREADS / kWave];
  __shared__ float s_acc[RPB > 1 && !FEW ? TPR * VPT * 8 : 1];
  if constexpr (FEW) {  // `part` is dgain
    __shared__ float s_w[kFewThreads / kWave][kFewCols];
    if ((int)blockIdx.x >= row_blocks) {
      dgain_columns<BF16>(h, rstd, dy, part, T, nvec, ((int)blockIdx.x - row_blocks) * kFewCols, s_w);
      return;
    }
  }
  const int j = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float acc[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.0f;
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * RPB; t0 < T; t0 += (int64_t)row_blocks * RPB, turn ^= 1) {
    const int64_t t = t0 + grp;
    const bool live = t < T;  // a row group past the end adds zeros and stores nothing
    const int64_t row = t * nvec;
    const float r = live ? rstd[t] : 0.0f;
    Piece8<BF16> ph[VPT], pd[VPT], pr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * TPR + j;
      ph[i] = Piece8<BF16>{};
      pd[i] = Piece8<BF16>{};
      pr[i] = Piece8<BF16>{};
      if (live && c < nvec) {
        ph[i] = load8<BF16>(h, row + c);
        pd[i] = load8<BF16>(dy, row + c);
        if (dh) pr[i] = load8<BF16>(dh, row + c);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * TPR + j;
      if (c < nvec) {
        float z[8], d[8], g[8];
        widen8<BF16>(ph[i], z);
        widen8<BF16>(pd[i], d);
        widen8<BF16>(load8<BF16>(gain, c), g);
        float p = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float zz = z[q] * r;
          if (!FEW) acc[i][q] = fmaf(d[q], zz, acc[i][q]);
          p = fmaf(d[q] * g[q], zz, p);
        }
        s += p;
      }
    }
    // two sets of slots in turn: a wave may be one row ahead of the slowest reader
    s = row_sum<TPR>(s, s_sum[turn]) * inv_d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * TPR + j;
      if (live && c < nvec) {
        float z[8], d[8], g[8], o[8];
        widen8<BF16>(ph[i], z);
        widen8<BF16>(pd[i], d);
        widen8<BF16>(load8<BF16>(gain, c), g);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = r * (d[q] * g[q] - z[q] * r * s);
        if (dh) {
          float e[8];
          widen8<BF16>(pr[i], e);
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] += e[q];
        }
        store8<BF16>(dx, row + c, narrow8<BF16>(o));
      }
    }
  }
  if constexpr (FEW) return;
  // the block's row groups in order
  if constexpr (RPB > 1) {
    for (int u = 1; u < RPB; ++u) {
      __syncthreads();
      if (grp == u)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int q = 0; q < 8; ++q) s_acc[(i * 8 + q) * TPR + j] = acc[i][q];
      __syncthreads();
      if (grp == 0)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[i][q] += s_acc[(i * 8 + q) * TPR + j];
    }
  }
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * TPR + j;
      if (c < nvec) {
        f32x4* p = (f32x4*)(part + ((int64_t)blockIdx.x * nvec + c) * 8);
        p[0] = f32x4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
        p[1] = f32x4{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
      }
    }
  }
}

// dgain: 16 columns per block, 64 slices of the partial rows added side by side,
// then 16 by 16 and the four sums, in slice order. (64 columns and 16 slices, a
// quarter of the workgroups: 4.8 us against 4.6 for 512 partial rows of 2048.)
constexpr int kDgCols = 16, kDgSlices = 64;
__global__ __launch_bounds__(kDgCols * kDgSlices) void dgain_kernel(const float* __restrict__ part,
                                                                    float* __restrict__ dgain, int rows, int d) {
  __shared__ float s_v[kDgSlices][kDgCols], s_w[4][kDgCols];
  const int c = threadIdx.x % kDgCols, sl = threadIdx.x / kDgCols;
  const int col = blockIdx.x * kDgCols + c;  // d is a multiple of 64
  float a = 0.0f;
#pragma unroll 8
  for (int i = sl; i < rows; i += kDgSlices) a += part[(int64_t)i * d + col];
  s_v[sl][c] = a;
  __syncthreads();
  if (sl < 4) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kDgSlices / 4; ++i) v += s_v[sl * (kDgSlices / 4) + i][c];
    s_w[sl][c] = v;
  }
  __syncthreads();
  if (sl == 0) dgain[col] = (s_w[0][c] + s_w[1][c]) + (s_w[2][c] + s_w[3][c]);
}

// Threads per row and pieces per thread by row width (pieces of 8 values). Four
// pieces per thread keep the reductions' share small where HBM is the bound.
#define MOE_NORM_SHAPES_256(F)                                                                          \
  if (nvec <= 64) { F(64, 1); }                                                                         \
  else if (nvec <= 128) { F(64, 2); }                                                                   \
  else if (nvec <= 256) { F(64, 4); }                                                                   \
  else if (nvec <= 512) { F(128, 4); }                                                                  \
  else { F(256, 4); }
#define MOE_NORM_SHAPES(F)                                                                              \
  if (nvec <= 1024) { MOE_NORM_SHAPES_256(F) }                                                          \
  else if (nvec <= 2048) { F(512, 4); }                                                                 \
  else { F(1024, 4); }

// The same for few rows, where the bound is the chain of one row: loads, 64-bit
// sums, the reduction, the stores. One piece per thread against four, with the
// gain loaded behind the sum in both: 8 rows of 7168 bf16 3.5 and 4.2 us. Against
// four as they are: 512 rows 6.6 and 7.1 us, 1024 rows 12.9 and 11.6 (of 2048
// 4.6 and 5.4; 4096 rows 13.2 and 12.8).
#define MOE_NORM_SHAPES_FEW(F)                                                                          \
  if (nvec <= 64) { F(64, 1); }                                                                         \
  else if (nvec <= 128) { F(128, 1); }                                                                  \
  else if (nvec <= 256) { F(256, 1); }                                                                  \
  else if (nvec <= 512) { F(512, 1); }                                                                  \
  else if (nvec <= 1024) { F(1024, 1); }                                                                \
  else if (nvec <= 2048) { F(1024, 2); }                                                                \
  else { F(1024, 4); }

constexpr int64_t kNormFewRows = 512;

// dgain in the launch of dx (h and dy are read twice, from the caches) or by partial
// sums and a second launch, us in a graph: 1 row of 7168 bf16 3.5 / 6.3, 512 of 2048
// 4.2 / 7.9, 1024 of 7168 22.0 / 22.0, 777 of 320 float32 5.6 / 5.5 (and a launch less
// on the host); 2048 of 2048 bf16 15.0 / 12.4, 4096 of 320 17.0 / 6.3.
bool norm_bwd_few(const moe_problem_t& p) { return p.T <= 1024 && p.d_model <= 8192; }

int rows_per_block_few(int nvec) { return nvec <= 64 ? 4 : nvec <= 128 ? 2 : 1; }
int rows_per_block(int nvec) { return nvec <= 256 ? 4 : nvec <= 512 ? 2 : 1; }

}  // namespace

// Blocks of the backward launch, and rows of partial sums
int64_t norm_bwd_blocks(int64_t T, int d) {
  return min(ceil_div(T, rows_per_block(d / 8)), (int64_t)512);
}

hipError_t launch_add_rmsnorm(const moe_problem_t& p, const void* x, const void* residual, const void* gain, float eps,
                              void* h, void* y, void* y8, void* y_scale, float* rstd, hipStream_t s) {
  const int nvec = p.d_model / 8;
  const bool few = p.T <= kNormFewRows;
  const int64_t blocks = ceil_div(p.T, few ? rows_per_block_few(nvec) : rows_per_block(nvec));
  const double inv_d = 1.0 / p.d_model;
  if (p.d_model > kNormMaxWidth) return hipErrorInvalidValue;
  // A launch takes less than 2^32 threads along x (2^26 rows of up to 2048 values):
  // at most 2^21 workgroups there, the others along y.
  const int64_t gy = ceil_div(blocks, (int64_t)1 << 21), gx = ceil_div(blocks, gy);
  // Arrays of 128 MB or more are gone from the last-level cache before the next
  // operator reads them: past the caches, 16384 rows of 7168 bf16 with residual
  // and both outputs take 181 instead of 192 us (5.8 TB/s), while at 8192 rows of
  // 2048 (32 MB arrays) a forward and backward pass take 58 instead of 52 us.
  const bool nt = (double)p.T * p.d_model * (p.dtype == MOE_DTYPE_BF16 ? 2 : 4) >= (double)(128 << 20);
#define MOE_NORM_LAUNCH(BF16, TPR, VPT, NT)                                                                      \
  hipLaunchKernelGGL((add_rmsnorm_kernel<BF16, TPR, VPT, NT>), dim3((unsigned)gx, (unsigned)gy),                 \
                     dim3(TPR > kNormThreads ? TPR : kNormThreads), 0, s, x, residual, gain, eps, h, y,          \
                     (uint8_t*)y8, (uint8_t*)y_scale, rstd, p.T, nvec, inv_d)
#define MOE_NORM(TPR, VPT)                                       \
  do {                                                           \
    if (p.dtype == MOE_DTYPE_BF16) {                             \
      if (nt) MOE_NORM_LAUNCH(true, TPR, VPT, true);             \
      else MOE_NORM_LAUNCH(true, TPR, VPT, false);               \
    } else {                                                     \
      if (nt) MOE_NORM_LAUNCH(false, TPR, VPT, true);            \
      else MOE_NORM_LAUNCH(false, TPR, VPT, false);              \
    }                                                            \
  } while (0)
#define MOE_NORM_FEW(TPR, VPT)                                            \
  do {                                                                    \
    if (p.dtype == MOE_DTYPE_BF16) MOE_NORM_LAUNCH(true, TPR, VPT, false); \
    else MOE_NORM_LAUNCH(false, TPR, VPT, false);                         \
  } while (0)
  if (few) {  // 64 MB at most: never past the caches
    static_assert(kNormFewRows * kNormMaxWidth * 4 < (128 << 20), "few rows take the plain form alone");
    MOE_NORM_SHAPES_FEW(MOE_NORM_FEW)
  } else {
    MOE_NORM_SHAPES(MOE_NORM)
  }
#undef MOE_NORM_FEW
#undef MOE_NORM
#undef MOE_NORM_LAUNCH
  return hipGetLastError();
}

hipError_t launch_rmsnorm_backward(const moe_problem_t& p, const void* h, const void* gain, const float* rstd,
                                   const void* dy, const void* dh, void* dx, float* dgain, float* part,
                                   hipStream_t s) {
  const int nvec = p.d_model / 8;
  if (p.d_model > kNormMaxWidth) return hipErrorInvalidValue;
  const float inv_d = 1.0f / (float)p.d_model;
#define MOE_NORM_LAUNCH(BF16, TPR, VPT, FEW, GRID, THREADS, OUT)                                                  \
  hipLaunchKernelGGL((rmsnorm_backward_kernel<BF16, TPR, VPT, FEW>), dim3((unsigned)(GRID)), dim3(THREADS), 0, s, h, \
                     gain, rstd, dy, dh, dx, OUT, p.T, nvec, inv_d, (int)blocks)
  if (norm_bwd_few(p)) {
    const int64_t blocks = ceil_div(p.T, kFewThreads / kNormThreads * rows_per_block(nvec));
#define MOE_NORM(TPR, VPT)                                                                                    \
  do {                                                                                                        \
    if (p.dtype == MOE_DTYPE_BF16)                                                                            \
      MOE_NORM_LAUNCH(true, TPR, VPT, true, blocks + p.d_model / kFewCols, kFewThreads, dgain);                     \
    else                                                                                                      \
      MOE_NORM_LAUNCH(false, TPR, VPT, true, blocks + p.d_model / kFewCols, kFewThreads, dgain);                    \
  } while (0)
    MOE_NORM_SHAPES_256(MOE_NORM)
#undef MOE_NORM
    return hipGetLastError();
  }
  const int64_t blocks = norm_bwd_blocks(p.T, p.d_model);
#define MOE_NORM(TPR, VPT)                                                                                       \
  do {                                                                                                           \
    constexpr int threads = TPR > kNormThreads ? TPR : kNormThreads;                                             \
    if (p.dtype == MOE_DTYPE_BF16) MOE_NORM_LAUNCH(true, TPR, VPT, false, blocks, threads, part);                \
    else MOE_NORM_LAUNCH(false, TPR, VPT, false, blocks, threads, part);                                         \
  } while (0)
  MOE_NORM_SHAPES(MOE_NORM)
#undef MOE_NORM
#undef MOE_NORM_LAUNCH
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(dgain_kernel, dim3((unsigned)(p.d_model / kDgCols)), dim3(kDgCols * kDgSlices), 0, s, (const float*)part,
                     dgain, (int)blocks, p.d_model);
  return hipGetLastError();
}

hipError_t launch_quantize_rows(const moe_problem_t& p, const void* x, void* x8, void* x_scale, hipStream_t s) {
  const int64_t n = p.T * (code_pitch(p.d_model) / 8);
  const int64_t blocks = min(ceil_div(n, 256), (int64_t)65536);
  if (p.dtype == MOE_DTYPE_BF16)
    hipLaunchKernelGGL(quantize_rows_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, s, x, (uint8_t*)x8,
                       (uint8_t*)x_scale, p.T, p.d_model / 8);
  else
    hipLaunchKernelGGL(quantize_rows_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, x, (uint8_t*)x8,
                       (uint8_t*)x_scale, p.T, p.d_model / 8);
  return hipGetLastError();
}

}  // namespace moe
