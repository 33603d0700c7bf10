// Expert FFN products with 8-bit operands over ragged per-expert row groups.
//
// "Distributed training part 4" (jesamkim's AI tech blog), section 3: the
// experts are independent FFNs. For every expert e with rows [offsets[e],
// offsets[e+1]): C[rows] = A[rows] B[e], both operands e4m3 codes with a scale
// 2^e per block of 128 positions along the contraction (moe_ext.h).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 rows by 32 columns over 64
// positions at twice the bf16 rate and applies one power-of-two scale per lane
// of each operand while it multiplies. A lane holds 32 bytes of one row (lane
// & 31); the two lanes of a row hold different halves of the 64 positions, and
// since the operands only have to agree on which position sits where, a lane
// half h takes the 16-byte pieces 2 q + h of the 128-byte block. Both halves
// share the block's scale. Operands are passed as (B, A), so a lane's 16
// accumulators are columns 8 (v / 4) + 4 (lane >> 5) + v % 4 of row lane & 31.
//
// The first product's epilogue applies GELU_tanh in float32 and writes 8-bit
// rows: a workgroup owns whole blocks of 128 columns, so a block's largest
// magnitude is at hand and the hidden activations never exist in more bits.
#include <stdlib.h>

#include "common.h"
#include "e4m3.h"
#include "internal.h"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 join8(const u32x4& a, const u32x4& b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Expert and rows of m-tile `m_tile` of BM rows (expert by expert): info =
// {expert or -1, first row, end row}. Wave 0; ends with a barrier.
template <int BM>
__device__ __forceinline__ void find_rows(const int32_t* __restrict__ offsets, int E, int64_t R, int m_tile,
                                          int* info) {
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    if (lane == 0) info[0] = -1;
    int lo[4], hi[4], cnt[4], local = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane * 4 + i;
      lo[i] = hi[i] = cnt[i] = 0;
      if (e < E) {
        lo[i] = max(offsets[e], 0);
        hi[i] = (int)min((int64_t)offsets[e + 1], R);
        cnt[i] = hi[i] > lo[i] ? (int)ceil_div(hi[i] - lo[i], BM) : 0;
      }
      local += cnt[i];
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    int run = incl - local;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (m_tile >= run && m_tile < run + cnt[i]) {
        info[0] = lane * 4 + i;
        info[1] = lo[i] + (m_tile - run) * BM;
        info[2] = hi[i];
      }
      run += cnt[i];
    }
  }
  __syncthreads();
}

// A workgroup multiplies 32 TM rows by 32 NG columns; wave (g, ks) takes column
// group g and every KS-th block of 128 positions, straight from memory into
// registers, and the KS sums of a group are added in order through LDS.
template <int TM, int NG, int KS, bool ACT>
__global__ __launch_bounds__(NG * KS * kWave) void gemm_fp8_small_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const int32_t* __restrict__ perm, int64_t a_rows,
    const int32_t* __restrict__ offsets, const uint8_t* __restrict__ B, const uint8_t* __restrict__ Bs,
    void* __restrict__ C, uint8_t* __restrict__ Cs, int64_t R, int K, int N, int E, int n_tiles) {
  static_assert(!ACT || NG == 4, "an 8-bit output block spans 128 columns");
  constexpr int BM = 32 * TM;
  __shared__ int s_info[3];
  __shared__ float s_acc[KS > 1 ? (KS - 1) * NG * TM * 16 * kWave : 1];
  __shared__ float s_max[ACT ? NG * BM : 1];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int g = wave % NG, ks = wave / NG;
  find_rows<BM>(offsets, E, R, blockIdx.x / n_tiles, s_info);
  const int e = s_info[0];
  if (e < 0) return;  // the whole workgroup
  const int64_t row0 = s_info[1], row_end = s_info[2];
  const int ng = (blockIdx.x % n_tiles) * NG + g;  // column group
  const bool cols = ng * 32 < N;
  const int KB = (int)(code_pitch(K) / kQBlock);
  const int64_t cp = code_pitch(K), sp = scale_pitch(K);
  const int half = lane >> 5;
  const u32x4* pa[TM];
  const uint8_t* ps[TM];
#pragma unroll
  for (int mi = 0; mi < TM; ++mi) {
    const int64_t r = min(row0 + mi * 32 + (lane & 31), row_end - 1);  // rows past the end repeat the last
    int64_t src = r;
    if (perm) {
      src = perm[r];
      if (src < 0 || src >= a_rows) src = 0;
    }
    pa[mi] = (const u32x4*)(A + src * cp) + half;
    ps[mi] = As + src * sp;
  }
  const int64_t slab = (int64_t)e * (N / 32) + (cols ? ng : 0);
  const u32x4* pb = (const u32x4*)(B + slab * KB * 4096) + half * 32 + (lane & 31);
  const uint8_t* pbs = Bs + slab * KB * 32 + (lane & 31);
  f32x16 acc[TM];
#pragma unroll
  for (int mi = 0; mi < TM; ++mi)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[mi][v] = 0.0f;
  if (cols) {
#pragma unroll 2
    for (int kb = ks; kb < KB; kb += KS) {
      u32x4 b[4], a[TM][4];
      int sb = pbs[kb * 32], sa[TM];
#pragma unroll
      for (int q = 0; q < 4; ++q) b[q] = pb[(int64_t)kb * 256 + q * 64];
#pragma unroll
      for (int mi = 0; mi < TM; ++mi) {
        sa[mi] = ps[mi][kb];
#pragma unroll
        for (int q = 0; q < 4; ++q) a[mi][q] = pa[mi][kb * 8 + q * 2];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int mi = 0; mi < TM; ++mi)
          acc[mi] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join8(b[2 * j], b[2 * j + 1]),
                                                                    join8(a[mi][2 * j], a[mi][2 * j + 1]), acc[mi], 0,
                                                                    0, 0, sb, 0, sa[mi]);
    }
  }
  if constexpr (KS > 1) {
    if (ks > 0)
#pragma unroll
      for (int mi = 0; mi < TM; ++mi)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          s_acc[((((ks - 1) * NG + g) * TM + mi) * 16 + v) * kWave + lane] = acc[mi][v];
    __syncthreads();
    if (ks == 0)
#pragma unroll
      for (int u = 0; u < KS - 1; ++u)
#pragma unroll
        for (int mi = 0; mi < TM; ++mi)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[mi][v] += s_acc[(((u * NG + g) * TM + mi) * 16 + v) * kWave + lane];
  }
  if constexpr (ACT) {
    if (ks == 0)
#pragma unroll
      for (int mi = 0; mi < TM; ++mi) {
        float m = 0.0f;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          acc[mi][v] = gelu_tanh(acc[mi][v]);  // 0 stays 0: columns past N
          m = fmaxf(m, fabsf(acc[mi][v]));
        }
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        s_max[g * BM + mi * 32 + (lane & 31)] = m;
      }
    __syncthreads();
    if (ks > 0) return;
    const int64_t hp = code_pitch(N), hs = scale_pitch(N);
    const int cb = blockIdx.x % n_tiles;  // block of 128 columns
#pragma unroll
    for (int mi = 0; mi < TM; ++mi) {
      const int rl = mi * 32 + (lane & 31);
      float m = 0.0f;
#pragma unroll
      for (int u = 0; u < NG; ++u) m = fmaxf(m, s_max[u * BM + rl]);
      const int byte = scale_byte(m);
      const float inv = inv_scale(byte);
      const int64_t r = row0 + rl;
      if (r >= row_end) continue;
      uint8_t* out = (uint8_t*)C + r * hp + (int64_t)ng * 32 + 4 * half;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *(uint32_t*)(out + 8 * v) = encode4(acc[mi][4 * v], acc[mi][4 * v + 1], acc[mi][4 * v + 2],
                                            acc[mi][4 * v + 3], inv);
      if (g == 0 && half == 0) Cs[r * hs + cb] = (uint8_t)byte;
    }
  } else {
    if (ks > 0 || !cols) return;
#pragma unroll
    for (int mi = 0; mi < TM; ++mi) {
      const int64_t r = row0 + mi * 32 + (lane & 31);
      if (r >= row_end) continue;
      bf16_bits* out = (bf16_bits*)C + r * N + ng * 32 + 4 * half;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        u32x2 o;
        o[0] = pack_bf16x2(acc[mi][4 * v], acc[mi][4 * v + 1]);
        o[1] = pack_bf16x2(acc[mi][4 * v + 2], acc[mi][4 * v + 3]);
        *(u32x2*)(out + 8 * v) = o;
      }
    }
  }
}

// Weights [K, N] of one expert to codes and scales. A workgroup takes 128
// positions of 64 columns: rows of 64 bf16 are read whole, transposed through
// LDS, and 16 codes of a column leave as one 16-byte piece.
__global__ __launch_bounds__(256) void quantize_weights_kernel(const bf16_bits* __restrict__ w, uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ qs, int K, int N, int KB) {
  __shared__ float s_w[kQBlock][65];
  const int kb = blockIdx.x % KB, n0 = blockIdx.x / KB * 64;
  const int64_t e = blockIdx.y;
  const bf16_bits* src = w + e * K * N;
  for (int i = threadIdx.x; i < kQBlock * 64; i += 256) {
    const int k = kb * kQBlock + i / 64, c = i % 64;
    s_w[i / 64][c] = k < K ? bf16_to_f32(src[(int64_t)k * N + n0 + c]) : 0.0f;
  }
  __syncthreads();
  const int c = threadIdx.x / 4, part = threadIdx.x % 4;  // column, its positions 32 part .. + 31
  float m = 0.0f;
  for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(s_w[part * 32 + i][c]));
  m = fmaxf(m, __shfl_xor(m, 1, kWave));
  m = fmaxf(m, __shfl_xor(m, 2, kWave));
  const int byte = scale_byte(m);
  const float inv = inv_scale(byte);
  const int64_t grp = (e * (N / 32) + (n0 + c) / 32) * KB + kb;
  for (int h = 0; h < 2; ++h) {
    u32x4 o;
    for (int v = 0; v < 4; ++v) {
      const int k = part * 32 + h * 16 + v * 4;
      o[v] = encode4(s_w[k][c], s_w[k + 1][c], s_w[k + 2][c], s_w[k + 3][c], inv);
    }
    *(u32x4*)(q + grp * 4096 + ((part * 2 + h) * 32 + c % 32) * 16) = o;
  }
  if (part == 0) qs[grp * 32 + c % 32] = (uint8_t)byte;
}

// m-tiles of BM rows over E groups of R rows in all, at most
int64_t m_tiles_bound(int64_t R, int E, int bm) { return min(R, (R + (int64_t)E * (bm - 1)) / bm); }

template <int TM, int NG, int KS, bool ACT>
hipError_t launch_small(const void* A, const void* As, const int32_t* perm, int64_t a_rows, const int32_t* offsets,
                        const void* B, const void* Bs, void* C, void* Cs, int64_t R, int K, int N, int E,
                        hipStream_t s) {
  const int n_tiles = (int)ceil_div(N, 32 * NG);
  const int64_t grid = m_tiles_bound(R, E, 32 * TM) * n_tiles;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_fp8_small_kernel<TM, NG, KS, ACT>), dim3((unsigned)grid), dim3(NG * KS * kWave), 0, s,
                     (const uint8_t*)A, (const uint8_t*)As, perm, a_rows, offsets, (const uint8_t*)B,
                     (const uint8_t*)Bs, C, (uint8_t*)Cs, R, K, N, E, n_tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_fp8(const void* A, const void* As, const int32_t* perm, int64_t a_rows, const int32_t* offsets,
                           const void* B, const void* Bs, void* C, void* Cs, int64_t R, int K, int N, int E, bool act,
                           hipStream_t s) {
  if (act) return launch_small<1, 4, 4, true>(A, As, perm, a_rows, offsets, B, Bs, C, Cs, R, K, N, E, s);
  return launch_small<1, 2, 4, false>(A, As, perm, a_rows, offsets, B, Bs, C, Cs, R, K, N, E, s);
}

hipError_t launch_quantize_weights(const void* w, void* q, void* qs, int E, int K, int N, hipStream_t s) {
  const int KB = (int)(code_pitch(K) / kQBlock);
  const int64_t grid = (int64_t)KB * (N / 64);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(quantize_weights_kernel, dim3((unsigned)grid, (unsigned)E), dim3(256), 0, s, (const bf16_bits*)w,
                     (uint8_t*)q, (uint8_t*)qs, K, N, KB);
  return hipGetLastError();
}

}  // namespace moe
