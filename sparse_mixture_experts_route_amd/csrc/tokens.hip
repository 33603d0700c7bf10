// Rows sorted by expert and back, with weights, and the gradients.
//
// With r(t, j) the row of selection j of token t (-1: dropped):
//   to rows    dst[r(t, j)] = w[t, j] src[t],  dw[t, j] = <src[t], rows[r(t, j)]>
//   from rows  dst[t] = add[t] + sum over j of w[t, j] rows[r(t, j)],  dw[t, j] = <x[t], rows[r(t, j)]>
// Dispatch is the first without dw, the gradient of combine the first with it;
// combine is the second without, the gradient of dispatch the second with it.
// Each pass moves every row once: HBM is the bound. A wave takes a token, or a
// part of its row, so a token's own row is read once for all its selections,
// sums stay inside a wave and no atomics are needed.
//
// Measured, bfloat16, inputs that change from call to call: 8192 tokens of 8
// selections, rows of 2048: to rows 54 us (302 MB, 5.6 TB/s), from rows with a
// residual 59 us (335 MB, 5.7 TB/s), to rows with dw 120 us (570 MB, 4.8 TB/s: reads and
// writes in equal parts, one or two pieces a lane under way alike), gradient of 64 logits 5.5 us;
// 16384 tokens of 8 selections, rows of 7168: to rows 430 us (2.1 GB), from rows 418 us
// (2.35 GB), 4.9 and 5.6 TB/s. A copy reaches 5.1.
#include "common.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int kWaves = 4;     // waves of a workgroup
constexpr int kThreads = kWaves * kWave;
constexpr int kGroup = 8;     // selections of a token handled together
constexpr int kPieces = 2;    // 16-byte pieces of a row per lane and step
constexpr int kStep = kWave * kPieces;

template <bool BF16>
constexpr int kVals = BF16 ? 8 : 4;  // values of a 16-byte piece

template <bool BF16>
__device__ __forceinline__ void widen(const u32x4& q, float* f) {
#pragma unroll
  for (int i = 0; i < kVals<BF16>; ++i)
    f[i] = BF16 ? ((i & 1) ? __uint_as_float(q[i / 2] & 0xFFFF0000u) : __uint_as_float(q[i / 2] << 16))
                : __uint_as_float(q[i % 4]);
}

template <bool BF16>
__device__ __forceinline__ u32x4 narrow(const float* f) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = BF16 ? pack_bf16x2(f[2 * i % 8], f[(2 * i + 1) % 8]) : __float_as_uint(f[i]);
  return q;
}

template <bool NT>
__device__ __forceinline__ u32x4 load(const u32x4* p) {
  return NT ? __builtin_nontemporal_load(p) : *p;
}

template <bool NT>
__device__ __forceinline__ void store(u32x4* p, const u32x4& v) {
  if (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// Which token and which pieces of its row a wave has. Without dot products a row
// may be cut over waves of any workgroup (`parts`), with them over those of one.
struct Share {
  int64_t t;
  int64_t lo, hi;
};

__device__ __forceinline__ Share share_of(int64_t w, int parts, int64_t row_vecs) {
  const int64_t t = w / parts, cut = (row_vecs + parts - 1) / parts;
  Share s;
  s.t = t;
  s.lo = (w - t * parts) * cut;
  s.hi = min(row_vecs, s.lo + cut);
  return s;
}

// Rows (as piece offsets, -1: dropped) and weights of selections j0 .. j0 + 7
__device__ __forceinline__ void selections(const int32_t* __restrict__ inv, const float* __restrict__ w, int64_t t,
                                           int j0, int k, int64_t rows, int64_t row_vecs, int64_t* at, float* wt) {
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    const int32_t r = j0 + j < k ? inv[t * k + j0 + j] : -1;
    const bool ok = r >= 0 && r < rows;
    at[j] = ok ? (int64_t)r * row_vecs : -1;
    wt[j] = ok && w ? w[t * k + j0 + j] : 1.0f;
  }
}

// A value (int or float) of another lane of the DPP row, and of a given lane
template <int CTRL, typename V>
__device__ __forceinline__ V dpp_row(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Sum over the wave: within rows of 16 lanes by DPP, then the four rows' by scalar reads
template <typename V>
__device__ __forceinline__ V wave_total(V v) {
  v += dpp_row<0xB1>(v);   // quad_perm 1, 0, 3, 2
  v += dpp_row<0x4E>(v);   // quad_perm 2, 3, 0, 1
  v += dpp_row<0x141>(v);  // row_half_mirror
  v += dpp_row<0x140>(v);  // row_mirror
  auto row = [&](int l) { return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// Adds the waves' sums of one token and stores them. `slots` [waves][8]; every
// wave of the workgroup comes here.
template <int WPT>
__device__ __forceinline__ void store_dots(float* dot, float* __restrict__ dw, int64_t t, int64_t T, int j0, int k,
                                           float (*slots)[kGroup]) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
  for (int j = 0; j < kGroup; ++j) dot[j] = wave_total(dot[j]);
  if constexpr (WPT > 1) {
    __syncthreads();  // the slots' last readers are through
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (lane == j) slots[wave][j] = dot[j];
    __syncthreads();
    if (wave % WPT == 0 && lane < kGroup) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < WPT; ++i) v += slots[wave + i][lane];
      if (t < T && j0 + lane < k) dw[t * k + j0 + lane] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (lane == j && t < T && j0 + j < k) dw[t * k + j0 + j] = dot[j];
  }
}

// DOT: dw is written too, and the WPT waves of a token are in one workgroup
template <bool BF16, bool NT, bool DOT, int WPT>
__global__ __launch_bounds__(kThreads) void to_rows_kernel(const u32x4* __restrict__ src,
                                                           const int32_t* __restrict__ inv,
                                                           const float* __restrict__ w,
                                                           const u32x4* __restrict__ rows, u32x4* __restrict__ dst,
                                                           float* __restrict__ dw, int64_t T, int k, int64_t row_vecs,
                                                           int parts) {
  constexpr int V = kVals<BF16>;
  __shared__ float slots[DOT && WPT > 1 ? kWaves : 1][kGroup];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);  // rows and weights by scalar loads
  const int64_t total = T * parts, R = T * k;
  for (int64_t w0 = (int64_t)blockIdx.x * kWaves; w0 < total; w0 += (int64_t)gridDim.x * kWaves) {
    Share s = share_of(w0 + wave, parts, row_vecs);
    if (s.t >= T) {  // past the end: only the barriers are left
      if (!DOT || WPT == 1) return;
      s.hi = s.lo;
    }
    for (int j0 = 0; j0 < k; j0 += kGroup) {
      int64_t at[kGroup];
      float wt[kGroup], dot[kGroup];
      if (s.t < T) selections(inv, w, s.t, j0, k, R, row_vecs, at, wt);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) dot[j] = 0.0f;
      for (int64_t c0 = s.lo + lane; c0 < s.hi; c0 += kStep) {
        u32x4 v[kPieces], b[DOT ? kGroup : 1][kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          const int64_t c = c0 + u * kWave;
          if (c >= s.hi) continue;
          v[u] = src[s.t * row_vecs + c];
          if constexpr (DOT) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
              if (at[j] >= 0) b[j][u] = load<NT>(rows + at[j] + c);
          }
        }
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          const int64_t c = c0 + u * kWave;
          if (c >= s.hi) continue;
          float a[V];
          widen<BF16>(v[u], a);
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            if (at[j] < 0) continue;
            if constexpr (DOT) {
              float y[V];
              widen<BF16>(b[j][u], y);
#pragma unroll
              for (int i = 0; i < V; ++i) dot[j] = fmaf(a[i], y[i], dot[j]);
            }
            u32x4 o = v[u];
            if (w) {
              float z[V];
#pragma unroll
              for (int i = 0; i < V; ++i) z[i] = a[i] * wt[j];
              o = narrow<BF16>(z);
            }
            store<NT>(dst + at[j] + c, o);
          }
        }
      }
      if constexpr (DOT) store_dots<WPT>(dot, dw, s.t, T, j0, k, slots);
    }
  }
}

// FEW: k <= 8, so that the selections' rows and weights stay in registers and a
// row is read once; else a second pass over the rows takes the dot products.
template <bool BF16, bool NT, bool DOT, int WPT, bool FEW>
__global__ __launch_bounds__(kThreads) void from_rows_kernel(const u32x4* __restrict__ rows,
                                                             const int32_t* __restrict__ inv,
                                                             const float* __restrict__ w,
                                                             const u32x4* __restrict__ add,
                                                             const u32x4* __restrict__ x, u32x4* __restrict__ dst,
                                                             float* __restrict__ dw, int64_t T, int k,
                                                             int64_t row_vecs, int parts) {
  constexpr int V = kVals<BF16>;
  __shared__ float slots[DOT && WPT > 1 ? kWaves : 1][kGroup];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);  // rows and weights by scalar loads
  const int64_t total = T * parts, R = T * k;
  for (int64_t w0 = (int64_t)blockIdx.x * kWaves; w0 < total; w0 += (int64_t)gridDim.x * kWaves) {
    Share s = share_of(w0 + wave, parts, row_vecs);
    if (s.t >= T) {
      if (!DOT || WPT == 1) return;
      s.hi = s.lo;
    }
    int64_t at[kGroup];
    float wt[kGroup], dot[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) dot[j] = 0.0f;
    if (FEW && s.t < T) selections(inv, w, s.t, 0, k, R, row_vecs, at, wt);
    for (int64_t c0 = s.lo + lane; c0 < s.hi; c0 += kStep) {
      float acc[kPieces][V];
      u32x4 extra[kPieces], own[kPieces];
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int64_t c = c0 + u * kWave;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[u][i] = 0.0f;
        if (c >= s.hi) continue;
        if (add) extra[u] = load<NT>(add + s.t * row_vecs + c);
        if (DOT && FEW) own[u] = load<NT>(x + s.t * row_vecs + c);
      }
      for (int j0 = 0; j0 < (FEW ? 1 : k); j0 += kGroup) {
        if (!FEW) selections(inv, w, s.t, j0, k, R, row_vecs, at, wt);
        u32x4 v[kGroup][kPieces];
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
#pragma unroll
          for (int u = 0; u < kPieces; ++u)
            if (at[j] >= 0 && c0 + u * kWave < s.hi) v[j][u] = load<NT>(rows + at[j] + c0 + u * kWave);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          if (c0 + u * kWave >= s.hi) continue;
          float a[V];
          if (DOT && FEW) widen<BF16>(own[u], a);
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            if (at[j] < 0) continue;
            float f[V];
            widen<BF16>(v[j][u], f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              acc[u][i] = fmaf(wt[j], f[i], acc[u][i]);
              if (DOT && FEW) dot[j] = fmaf(a[i], f[i], dot[j]);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int64_t c = c0 + u * kWave;
        if (c >= s.hi) continue;
        if (add) {
          float f[V];
          widen<BF16>(extra[u], f);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[u][i] += f[i];
        }
        store<NT>(dst + s.t * row_vecs + c, narrow<BF16>(acc[u]));
      }
    }
    if constexpr (DOT) {
      if constexpr (FEW) {
        store_dots<WPT>(dot, dw, s.t, T, 0, k, slots);
      } else {
        for (int j0 = 0; j0 < k; j0 += kGroup) {
          if (s.t < T) selections(inv, w, s.t, j0, k, R, row_vecs, at, wt);
#pragma unroll
          for (int j = 0; j < kGroup; ++j) dot[j] = 0.0f;
          for (int64_t c = s.lo + lane; c < s.hi; c += kWave) {
            float a[V];
            widen<BF16>(x[s.t * row_vecs + c], a);
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
              if (at[j] < 0) continue;
              float f[V];
              widen<BF16>(rows[at[j] + c], f);
#pragma unroll
              for (int i = 0; i < V; ++i) dot[j] = fmaf(a[i], f[i], dot[j]);
            }
          }
          store_dots<WPT>(dot, dw, s.t, T, j0, k, slots);
        }
      }
    }
  }
}

// Index and rows of a few selections in one launch: workgroup (t, part) counts the
// selections before its token's own ones in the order of the rows, P compares for
// each, and writes its part of their rows; one more workgroup counts the experts. The
// compares are made for every part of a row, so their number is T^2 k times the parts.
// Against histograms, ranks and rows in three launches, us in a graph, rows of one part
// (bfloat16 of 2048): 32 tokens of 8 selections 4.5 / 10.9, 128 of 8 6.4 / 11.6, 777 of 3
// 11.1 / 11.9, 1024 of 2 9.8 / 11.5, 512 of 8 15.1 / 15.0; of two (bfloat16 of 7168): 128 of 8
// 8.0 / 13.2, 1024 of 1 12.3 / 15.5, 777 of 3 20.4 / 16.9, 512 of 8 22.8 / 21.7; of four
// (float32 of 7168): 128 of 8 11.1 / 16.4, 1024 of 1 19.4 / 20.2, 777 of 3 30.1 / 23.1, 512
// of 8 40.6 / 31.5.
constexpr int kSmallPart = 2 * kThreads;  // 16-byte pieces of a row per workgroup

template <bool BF16>
__global__ __launch_bounds__(kThreads) void dispatch_small_kernel(const int32_t* __restrict__ idx,
                                                                  const float* __restrict__ w,
                                                                  const u32x4* __restrict__ x,
                                                                  int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ perm,
                                                                  int32_t* __restrict__ inv,
                                                                  u32x4* __restrict__ x_perm, int T, int k, int E,
                                                                  int row_vecs) {
  constexpr int V = kVals<BF16>;
  __shared__ int s_n[256];
  __shared__ int s_row[kWaves][kGroup];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, t = blockIdx.x, P = T * k;
  if (t == T) {  // the experts' counts and their prefix sums
    if (blockIdx.y) return;
    s_n[tid] = 0;
    __syncthreads();
    for (int i = tid; i < P; i += kThreads) {
      const int e = idx[i];
      if ((unsigned)e < (unsigned)E) atomicAdd(&s_n[e], 1);
    }
    __syncthreads();
    const int c = s_n[tid];
    int incl = c;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == kWave - 1) s_n[wave] = incl;
    __syncthreads();
    for (int i = 0; i < wave; ++i) incl += s_n[i];
    if (tid < E) {
      counts[tid] = c;
      offsets[tid] = incl - c;
      if (tid == E - 1) offsets[E] = incl;
    }
    return;
  }
  const int c0 = blockIdx.y * kSmallPart + tid;
  u32x4 v[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (c0 + u * kThreads < row_vecs) v[u] = x[(int64_t)t * row_vecs + c0 + u * kThreads];
  for (int j0 = 0; j0 < k; j0 += kGroup) {
    int e[kGroup], n[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      e[j] = j0 + j < k ? idx[t * k + j0 + j] : -1;
      n[j] = 0;
    }
    for (int i0 = 0; i0 < P; i0 += kThreads) {
      const int i = i0 + tid, f = i < P ? idx[i] : -1;
      const bool named = (unsigned)f < (unsigned)E;
#pragma unroll
      for (int j = 0; j < kGroup; ++j) n[j] += named && (f < e[j] || (f == e[j] && i < t * k + j0 + j));
    }
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      n[j] = wave_total(n[j]);
      if (lane == 0) s_row[wave][j] = n[j];
    }
    __syncthreads();
    int row[kGroup];
    float wt[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      row[j] = -1;
      wt[j] = 1.0f;
      if ((unsigned)e[j] >= (unsigned)E) continue;
      row[j] = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) row[j] += s_row[i][j];
      if (w) wt[j] = w[t * k + j0 + j];
    }
    __syncthreads();  // read before the next group's
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      if (blockIdx.y == 0 && tid == j && j0 + j < k) {
        inv[t * k + j0 + j] = row[j];
        if (row[j] >= 0) perm[row[j]] = t;
      }
      if (row[j] < 0) continue;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = c0 + u * kThreads;
        if (c >= row_vecs) continue;
        u32x4 o = v[u];
        if (w) {
          float a[V];
          widen<BF16>(o, a);
#pragma unroll
          for (int i = 0; i < V; ++i) a[i] *= wt[j];
          o = narrow<BF16>(a);
        }
        x_perm[(int64_t)row[j] * row_vecs + c] = o;
      }
    }
  }
}

// Gradient of the gates: LPT lanes have a token's E logits, VPT each (LPT VPT >= E)
template <int LPT, int VPT>
__global__ __launch_bounds__(kThreads) void gate_backward_kernel(const float* __restrict__ logits,
                                                                 const int32_t* __restrict__ idx,
                                                                 const float* __restrict__ dgate,
                                                                 const float* __restrict__ add,
                                                                 float* __restrict__ dlogits, int64_t T, int k, int E) {
  constexpr int TPW = kWave / LPT;  // tokens of a wave
  const int lane = threadIdx.x % kWave, l = lane % LPT;
  const int64_t first = ((int64_t)blockIdx.x * kWaves + threadIdx.x / kWave) * TPW + lane / LPT;
  for (int64_t t0 = first; t0 - lane / LPT < T; t0 += (int64_t)gridDim.x * kWaves * TPW) {
    const bool live = t0 < T;
    const int64_t t = live ? t0 : T - 1;
    float v[VPT], dp[VPT];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = i * LPT + l;
      v[i] = e < E ? logits[t * E + e] : -INFINITY;
      top = fmaxf(top, v[i]);
      dp[i] = 0.0f;
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
    // a row of -infinity alone: exp(-infinity - 0) = 0 everywhere
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      v[i] = expf(v[i] - base);
      sum += v[i];
    }
    for (int j = 0; j < k; ++j) {
      const int e = idx[t * k + j];
      if ((unsigned)e < (unsigned)E) {
        const float g = dgate[t * k + j];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (e == i * LPT + l) dp[i] += g;
      }
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) sum += __shfl_xor(sum, o, kWave);
    const float inv = sum > 0.0f ? 1.0f / sum : sum;  // 0 for an empty row; NaN stays
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      v[i] *= inv;
      if (v[i] != 0.0f) mean = fmaf(v[i], dp[i], mean);
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) mean += __shfl_xor(mean, o, kWave);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = i * LPT + l;
      if (live && e < E) {
        const float d = v[i] != 0.0f ? v[i] * (dp[i] - mean) : 0.0f;
        dlogits[t * E + e] = add ? d + add[t * E + e] : d;
      }
    }
  }
}

constexpr int64_t kMostBlocks = 1 << 22;  // the rest by strides: a launch holds less than 2^32 threads

// Arrays of 128 MB or more pass by the caches. By / through, us in a graph, arrays that change
// from call to call, 8 selections, bfloat16 rows of 2048: 4096 tokens (134 MB) dispatch 37 / 38,
// combine 27 / 30, combine's gradient with dots 63 / 69, dispatch's 33 / 36; 7000 tokens 57 / 64,
// 46 / 50, 100 / 108, 54 / 60; 12000 tokens 88 / 101, 77 / 89, 160 / 174, 88 / 100; below, 2048
// tokens (67 MB, one array for all results) 25 / 24, 15 / 15, 39 / 31. (Combine right behind the dispatch of the same rows
// would want them through: 64 / 62 and 102 / 95, from 10000 tokens on 139 / 175; the experts'
// products come between.)
bool streams(const moe_problem_t& p) {
  return (double)p.T * p.k * p.d_model * (p.dtype == MOE_DTYPE_BF16 ? 2 : 4) >= (double)(128 << 20);
}

// Waves of a token whose dot products are wanted: one where the tokens fill the chip or
// a row is one step of a wave. One / four, us in a graph, gradient of combine and of dispatch,
// 8 selections of bfloat16 rows of 2048: 64 tokens 8.1 / 5.6 and 7.1 / 5.5, 512 11.6 / 10.1 and
// 9.2 / 8.0, 1024 16.3 / 14.2 and 11.8 / 13.4, 2048 28.9 / 27.7 and 16.7 / 21.3, 3000 42 / 40
// and 27 / 31; rows of 7168: 512 29 / 24 and 21 / 16, 4000 187 / 186 and 111 / 103; 2 selections
// of rows of 1024 (one step): 1024 tokens 5.5 / 7.5 and 4.9 / 9.3.
int dot_waves(const moe_problem_t& p, int64_t row_vecs) { return p.T >= 2048 || row_vecs <= kStep ? 1 : kWaves; }

unsigned grid_of(int64_t waves) { return (unsigned)min(ceil_div(waves, (int64_t)kWaves), kMostBlocks); }

}  // namespace

// (Rows of up to 2^24 values: their parts lie along the grid's second dimension.)
bool dispatch_small(const moe_problem_t& p) {
  const int64_t parts = ceil_div(p.d_model / (p.dtype == MOE_DTYPE_BF16 ? 8 : 4), kSmallPart);
  return p.T <= 1024 && p.T * p.T * p.k * parts <= (int64_t)1 << 21 && p.d_model <= 1 << 24;
}

hipError_t launch_dispatch_small(const moe_problem_t& p, const int32_t* idx, const float* w, const void* x,
                                 int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* x_perm,
                                 hipStream_t s) {
  const bool bf16 = p.dtype == MOE_DTYPE_BF16;
  const int row_vecs = p.d_model / (bf16 ? 8 : 4);
  const dim3 grid((unsigned)p.T + 1, (unsigned)ceil_div(row_vecs, kSmallPart));
  hipLaunchKernelGGL(bf16 ? dispatch_small_kernel<true> : dispatch_small_kernel<false>, grid, dim3(kThreads), 0, s, idx, w,
                     (const u32x4*)x, counts, offsets, perm, inv, (u32x4*)x_perm, (int)p.T, p.k, p.E, row_vecs);
  return hipGetLastError();
}

hipError_t launch_to_rows(const moe_problem_t& p, const void* src, const int32_t* inv, const float* w, const void* rows,
                          void* dst, float* dw, hipStream_t s) {
  const int64_t row_vecs = p.d_model / (p.dtype == MOE_DTYPE_BF16 ? 8 : 4);
  const int wpt = dw ? dot_waves(p, row_vecs) : 1;
  const int parts = dw ? wpt : (int)ceil_div(row_vecs, (int64_t)kStep);
  const bool nt = streams(p);
#define MOE_TO_ROWS(BF16, NT, DOT, WPT)                                                                             \
  hipLaunchKernelGGL((to_rows_kernel<BF16, NT, DOT, WPT>), dim3(grid_of(p.T * parts)), dim3(kThreads), 0, s,        \
                     (const u32x4*)src, inv, w, (const u32x4*)rows, (u32x4*)dst, dw, p.T, p.k, row_vecs, parts)
#define MOE_TO_ROWS_T(BF16, NT)                            \
  do {                                                     \
    if (!dw) MOE_TO_ROWS(BF16, NT, false, 1);              \
    else if (wpt == 1) MOE_TO_ROWS(BF16, NT, true, 1);     \
    else MOE_TO_ROWS(BF16, NT, true, kWaves);              \
  } while (0)
  if (p.dtype == MOE_DTYPE_BF16) {
    if (nt) MOE_TO_ROWS_T(true, true);
    else MOE_TO_ROWS_T(true, false);
  } else {
    if (nt) MOE_TO_ROWS_T(false, true);
    else MOE_TO_ROWS_T(false, false);
  }
#undef MOE_TO_ROWS_T
#undef MOE_TO_ROWS
  return hipGetLastError();
}

hipError_t launch_from_rows(const moe_problem_t& p, const void* rows, const int32_t* inv, const float* w, const void* add,
                            const void* x, void* dst, float* dw, hipStream_t s) {
  const int64_t row_vecs = p.d_model / (p.dtype == MOE_DTYPE_BF16 ? 8 : 4);
  const int wpt = dw ? dot_waves(p, row_vecs) : 1;
  const int parts = dw ? wpt : (int)ceil_div(row_vecs, (int64_t)kStep);
  const bool nt = streams(p);
#define MOE_FROM_ROWS(BF16, NT, DOT, WPT, FEW)                                                                       \
  hipLaunchKernelGGL((from_rows_kernel<BF16, NT, DOT, WPT, FEW>), dim3(grid_of(p.T * parts)), dim3(kThreads), 0, s,  \
                     (const u32x4*)rows, inv, w, (const u32x4*)add, (const u32x4*)x, (u32x4*)dst, dw, p.T, p.k,      \
                     row_vecs, parts)
#define MOE_FROM_ROWS_T(BF16, NT, FEW)                          \
  do {                                                          \
    if (!dw) MOE_FROM_ROWS(BF16, NT, false, 1, FEW);            \
    else if (wpt == 1) MOE_FROM_ROWS(BF16, NT, true, 1, FEW);   \
    else MOE_FROM_ROWS(BF16, NT, true, kWaves, FEW);            \
  } while (0)
#define MOE_FROM_ROWS_K(BF16, NT)                    \
  do {                                               \
    if (p.k <= kGroup) MOE_FROM_ROWS_T(BF16, NT, true); \
    else MOE_FROM_ROWS_T(BF16, NT, false);           \
  } while (0)
  if (p.dtype == MOE_DTYPE_BF16) {
    if (nt) MOE_FROM_ROWS_K(true, true);
    else MOE_FROM_ROWS_K(true, false);
  } else {
    if (nt) MOE_FROM_ROWS_K(false, true);
    else MOE_FROM_ROWS_K(false, false);
  }
#undef MOE_FROM_ROWS_K
#undef MOE_FROM_ROWS_T
#undef MOE_FROM_ROWS
  return hipGetLastError();
}

hipError_t launch_gate_backward(const moe_problem_t& p, const float* logits, const int32_t* idx, const float* dgate,
                                const float* add, float* dlogits, hipStream_t s) {
#define MOE_GATE(LPT, VPT)                                                                                          \
  hipLaunchKernelGGL((gate_backward_kernel<LPT, VPT>), dim3(grid_of(ceil_div(p.T, (int64_t)(kWave / LPT)))),        \
                     dim3(kThreads), 0, s, logits, idx, dgate, add, dlogits, p.T, p.k, p.E)
  if (p.E <= 8) MOE_GATE(8, 1);
  else if (p.E <= 16) MOE_GATE(16, 1);
  else if (p.E <= 32) MOE_GATE(32, 1);
  else if (p.E <= 64) MOE_GATE(64, 1);
  else if (p.E <= 128) MOE_GATE(64, 2);
  else MOE_GATE(64, 4);
#undef MOE_GATE
  return hipGetLastError();
}

}  // namespace moe
