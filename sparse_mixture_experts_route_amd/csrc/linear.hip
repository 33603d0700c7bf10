// A dense projection with bias, activation and residual, and its gradients.
//
//   u = x W + bias, y = residual + act(u);  dU = dy act'(u)
//   dx = dU W^T, dW = x^T dU, dbias = sum over rows of dU
//
// Three products C [M, N] = A B over K with bfloat16 operands and float32 sums:
//   x W      A rows with K contiguous, B [K, N]
//   dU W^T   A rows with K contiguous, B rows with K contiguous ([N, K])
//   x^T dU   A [K, M], B [K, N]: the contraction goes along the tokens
// One kernel takes them, by two ways of an operand through LDS:
//   * K contiguous: a tile of rows x 64, 16-byte chunks XOR-ed with (row >> 1) & 7;
//     a lane's 8 values of an MFMA operand are one ds_read_b128;
//   * K outermost: a tile of 64 x columns, chunks XOR-ed with 4 (k & 3); the 8
//     values are two transposing reads (ds_read_b64_tr_b16).
// Both are conflict-free (the LDS has 64 banks of 4 bytes) and filled by loads
// that go from memory to LDS directly.
//
// v_mfma_f32_32x32x16_bf16, operands passed as (B, A): a lane's sums are 4
// neighbouring columns of a row. Steps of 64 along K through a ring of LDS
// stages, one barrier a step; reads of the next fragments and the loads of a
// later stage are issued between the matrix instructions. Workgroups are
// persistent: while a tile's results leave, the first stages of the next come in, and
// its first step waits for neither (waiting for the stores there: 8192 x 2048 -> 8192
// 331 us with u, 287 and 269 for the gradients, then 291, 234 and 235; now 271 to 285, 225 and
// 230: 964 to 1222 TFLOP/s where torch's products alone reach 1215, 1153 and 943; traced
// between other kernels 307, 227 and 229. Other places of the barrier, of the reads and of
// the loads among the matrix instructions, and priorities, make no difference).
// The results go through LDS of their own as float32 rows, so that bias, activation and
// residual are applied in 16-byte pieces of the row and rounded once.
//
// Few tiles are cut along K over the workgroups; their float32 sums meet in a
// second launch, in an order that depends on the sizes alone.
#include <stdlib.h>

#include "common.h"
#include "gemm_lanes.h"
#include "internal.h"
#include "lds_dma.h"
#include "linear.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr int kBK = 64;
constexpr int kKS = kBK / 16;

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

// act(u), and act'(u). GELU: with s = sigmoid(2 z), z = sqrt(2/pi) (u + 0.044715 u^3),
// the value is u s and the slope s + 2 u s (1 - s) z'.
template <int ACT>
__device__ __forceinline__ float act_one(float u) {
  if constexpr (ACT == MOET_ACT_GELU) return gelu_tanh(u);
  if constexpr (ACT == MOET_ACT_SILU) return u * sigmoid(u);
  if constexpr (ACT == MOET_ACT_RELU) return u > 0.0f ? u : u != u ? u : 0.0f;
  return u;
}

template <int ACT>
__device__ __forceinline__ float slope_one(float u) {
  if constexpr (ACT == MOET_ACT_GELU) {
    const float c = 2.0f * 0.7978845608028654f, u2 = u * u;
    const float s = sigmoid(c * u * fmaf(0.044715f, u2, 1.0f)), t = s * (1.0f - s);
    return t > 0.0f ? fmaf(u * t, c * fmaf(3.0f * 0.044715f, u2, 1.0f), s) : s;  // else it has saturated
  }
  if constexpr (ACT == MOET_ACT_SILU) {
    const float s = sigmoid(u), t = s * (1.0f - s);
    return t > 0.0f ? fmaf(u, t, s) : s;
  }
  if constexpr (ACT == MOET_ACT_RELU) return u > 0.0f ? 1.0f : u != u ? u : 0.0f;
  return 1.0f;
}

// N values by one branch
template <int N>
__device__ __forceinline__ void act_all(float* f, int act) {
  if (act == MOET_ACT_GELU) {
#pragma unroll
    for (int v = 0; v < N; ++v) f[v] = act_one<MOET_ACT_GELU>(f[v]);
  } else if (act == MOET_ACT_SILU) {
#pragma unroll
    for (int v = 0; v < N; ++v) f[v] = act_one<MOET_ACT_SILU>(f[v]);
  } else if (act == MOET_ACT_RELU) {
#pragma unroll
    for (int v = 0; v < N; ++v) f[v] = act_one<MOET_ACT_RELU>(f[v]);
  }
}

__device__ __forceinline__ void widen8(const u32x4& q, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = (i & 1) ? __uint_as_float(q[i / 2] & 0xFFFF0000u) : __uint_as_float(q[i / 2] << 16);
}

__device__ __forceinline__ u32x4 narrow8(const float* f) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return q;
}

// What becomes of 8 neighbouring sums
struct Epilogue {
  const bf16_bits *bias, *residual;
  bf16_bits *u, *y;
  int act;
};

struct DenseArgs {
  const bf16_bits *A, *B;
  int lda, ldb;  // values from one row to the next, as stored
  int M, N, K;
  int nk;        // steps along K
  int m_tiles, n_tiles, splits, gm;
  Epilogue ep;
  float* partials;  // [splits][M][N] when splits > 1
};

// One 16-byte piece of an operand's stage: `row` along M or N and `k`, both within the tile
struct Slot {
  int row, k;
};

template <bool MN, int ROWS>
__device__ __forceinline__ Slot slot_of(int p) {
  if constexpr (MN) {
    const int k = p / (ROWS / 8);
    return {((p % (ROWS / 8)) ^ (ROWS >= 128 ? 4 * (k & 3) : 0)) * 8, k};
  } else {
    const int row = p / 8;
    return {row, ((p % 8) ^ ((row >> 1) & 7)) * 8};
  }
}

template <bool A_MN, bool B_MN, int BM, int BN, int WM, int WN, int S, int OCC>
__global__ __launch_bounds__(WM * WN * 64, OCC * WM * WN / 4) void dense_kernel(DenseArgs args) {
  constexpr int NW = WM * WN, TPB = NW * kWave;
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  constexpr int A_STAGE = BM * kBK * 2, B_STAGE = BN * kBK * 2, STAGE = A_STAGE + B_STAGE;
  constexpr int A_LD = A_STAGE / 1024 / NW, B_LD = B_STAGE / 1024 / NW, NL = A_LD + B_LD;
  constexpr int A_RB = BM * 2, B_RB = BN * 2;  // bytes of a k row (K outermost)
  static_assert(A_LD * 1024 * NW == A_STAGE && B_LD * 1024 * NW == B_STAGE, "whole loads");
  constexpr int EP = 32 * 32 * 4;  // a wave's 32 x 32 results
  __shared__ __attribute__((aligned(1024))) char smem[S * STAGE + NW * EP];

  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm0 = (wave / WN) * WTM, wn0 = (wave % WN) * WTN;
  lds_char* const lds = (lds_char*)smem;
  const uint32_t lds_base = lds_addr(smem);

  // fragments' places in a stage
  const int q = lane & 15, g = lane >> 4, kr = q >> 2;
  auto mn_rd = [&](int col0, int rb) {
    const int col = col0 + (g & 1) * 16 + (q & 3) * 4;
    return ((g >> 1) * 8 + kr) * rb + (((col >> 3) ^ (4 * kr)) << 4) + (col & 7) * 2;
  };
  int kc_x[kKS];
#pragma unroll
  for (int ks = 0; ks < kKS; ++ks) kc_x[ks] = ((ks * 2 + (lane >> 5)) ^ (((lane & 31) >> 1) & 7)) << 4;
  int a_rd[TM], b_rd[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) a_rd[i] = A_MN ? mn_rd(wm0 + i * 32, A_RB) : (wm0 + i * 32 + (lane & 31)) * (kBK * 2);
#pragma unroll
  for (int i = 0; i < TN; ++i)
    b_rd[i] = A_STAGE + (B_MN ? mn_rd(wn0 + i * 32, B_RB) : (wn0 + i * 32 + (lane & 31)) * (kBK * 2));

  bf16x8 fa[2][TM], fb[2][TN];
  constexpr int A_RD = A_MN ? 2 : 1, B_RD = B_MN ? 2 : 1;  // reads of a fragment
  constexpr int NR = TM * A_RD + TN * B_RD;
  auto read_mn = [&](bf16x8& f, const lds_char* p, int half, int rb) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + half * 4 * rb));
    s16x8 w = __builtin_bit_cast(s16x8, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[half * 4 + i] = v[i];
    f = __builtin_bit_cast(bf16x8, w);
  };
  // read r of the fragments of sub-step ks of a buffer
  auto read_one = [&](int buf, int ks, int set, int r) {
    const lds_char* const st = lds + buf * STAGE;
    if (r < TM * A_RD) {
      const int i = r / A_RD;
      if constexpr (A_MN) read_mn(fa[set][i], st + a_rd[i] + ks * 16 * A_RB, r % A_RD, A_RB);
      else fa[set][i] = *(const lds_bf16x8*)(st + a_rd[i] + kc_x[ks]);
    } else {
      const int i = (r - TM * A_RD) / B_RD;
      if constexpr (B_MN) read_mn(fb[set][i], st + b_rd[i] + ks * 16 * B_RB, (r - TM * A_RD) % B_RD, B_RB);
      else fb[set][i] = *(const lds_bf16x8*)(st + b_rd[i] + kc_x[ks]);
    }
  };

  // An item: a tile and its steps [kb, kb + kn). The tiles of a split lie together;
  // the list is cut into 8 ranges, one for each XCD (workgroups are dealt to them in turn).
  struct Item {
    int m0, n0, split, kb, kn;
    i32x4 rsA, rsB;
    uint32_t a_off[A_LD], b_off[B_LD];
  };
  const int tiles = args.m_tiles * args.n_tiles, total = tiles * args.splits;
  const int xcd = blockIdx.x % 8, nb = gridDim.x / 8;
  const int lo = (int)((int64_t)total * xcd / 8), hi = (int)((int64_t)total * (xcd + 1) / 8);
  auto make = [&](int i) {
    Item it;
    const int t = i % tiles;
    it.split = i / tiles;
    int nt, mt;
    tile_coords(t, args.m_tiles, args.n_tiles, args.gm, nt, mt);
    it.m0 = __builtin_amdgcn_readfirstlane(mt * BM);
    it.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
    it.kb = __builtin_amdgcn_readfirstlane((int)((int64_t)args.nk * it.split / args.splits));
    it.kn = __builtin_amdgcn_readfirstlane((int)((int64_t)args.nk * (it.split + 1) / args.splits)) - it.kb;
    // what lies past an operand's end reads as zero; past its columns, as what follows there: not stored
    if constexpr (A_MN) it.rsA = buffer_rsrc(args.A, (uint32_t)((int64_t)args.K * args.lda * 2));
    else it.rsA = buffer_rsrc(args.A + (int64_t)it.m0 * args.lda, (uint32_t)((int64_t)min(args.M - it.m0, BM) * args.lda * 2));
    if constexpr (B_MN) it.rsB = buffer_rsrc(args.B, (uint32_t)((int64_t)args.K * args.ldb * 2));
    else it.rsB = buffer_rsrc(args.B + (int64_t)it.n0 * args.ldb, (uint32_t)((int64_t)min(args.N - it.n0, BN) * args.ldb * 2));
#pragma unroll
    for (int l = 0; l < A_LD; ++l) {
      const Slot s = slot_of<A_MN, BM>((wave * A_LD + l) * kWave + lane);
      it.a_off[l] = A_MN ? (uint32_t)(s.k * args.lda + it.m0 + s.row) * 2u : (uint32_t)(s.row * args.lda + s.k) * 2u;
    }
#pragma unroll
    for (int l = 0; l < B_LD; ++l) {
      const Slot s = slot_of<B_MN, BN>((wave * B_LD + l) * kWave + lane);
      it.b_off[l] = B_MN ? (uint32_t)(s.k * args.ldb + it.n0 + s.row) * 2u : (uint32_t)(s.row * args.ldb + s.k) * 2u;
    }
    return it;
  };
  auto issue_one = [&](const Item& it, int step, int buf, int l) {
    const uint32_t st = lds_base + buf * STAGE, kt = (uint32_t)(it.kb + step) * kBK;
    if (l < A_LD)
      buffer_load_lds16(it.rsA, it.a_off[l], kt * (A_MN ? (uint32_t)args.lda * 2u : 2u), st + (wave * A_LD + l) * 1024);
    else
      buffer_load_lds16(it.rsB, it.b_off[l - A_LD], kt * (B_MN ? (uint32_t)args.ldb * 2u : 2u),
                        st + A_STAGE + (wave * B_LD + l - A_LD) * 1024);
  };
  auto fill = [&](const Item& it) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s < it.kn)
#pragma unroll
        for (int l = 0; l < NL; ++l) issue_one(it, s, s, l);
  };

  f32x16 acc[TM][TN];
  auto mfma_one = [&](int set, int i) {
    acc[i / TN][i % TN] =
        __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[set][i % TN], fa[set][i / TN], acc[i / TN][i % TN], 0, 0, 0);
  };
  constexpr int NM = TM * TN, H = NM / 2;  // matrix instructions of a sub-step, and before the step's barrier
  constexpr int RPM = (NR + (NM + 1) / 2 - 1) / ((NM + 1) / 2);  // a set's reads go out in the first half
  constexpr int STORES = TM * TN * 2;  // 16-byte stores of a tile's results

  int i = lo + (int)blockIdx.x / 8;
  if (i >= hi) return;
  Item it = make(i);
  fill(it);
  bool first = true;
  while (true) {
    const int kn = it.kn;
    // the stages that were asked for before the last results left; their stores may still be under way
    if (first || args.splits > 1) wait_vmem<0>();
    else if (args.ep.u) wait_vmem<(2 * STORES < 63 ? 2 * STORES : 63)>();
    else wait_vmem<(STORES < 63 ? STORES : 63)>();
    first = false;
    __syncthreads();
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;

#pragma unroll
    for (int r = 0; r < NR; ++r) read_one(0, 0, 0, r);
    int buf = 0;
    for (int kt = 0; kt < kn; ++kt) {
#pragma unroll
      for (int ks = 0; ks < kKS - 1; ++ks) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          mfma_one(ks & 1, m);
#pragma unroll
          for (int u = 0; u < RPM; ++u)
            if (m * RPM + u < NR) read_one(buf, ks + 1, (ks + 1) & 1, m * RPM + u);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      constexpr int LAST = (kKS - 1) & 1;
#pragma unroll
      for (int m = 0; m < H; ++m) {
        mfma_one(LAST, m);
        __builtin_amdgcn_sched_barrier(0);
      }
      const bool more = kt + 1 < kn, refill = kt + S < kn;
      const int nbuf = buf + 1 == S ? 0 : buf + 1;
      if (more) {
        // stage kt + 1 has landed (the item began with its first S); kt + 2 .. kt + S - 1 may be under way
        if (kt + 1 >= S) {
          if (kt + S - 1 < kn) wait_vmem<NL * (S - 2)>();
          else wait_vmem<0>();
        }
        __syncthreads();  // every wave's part of it; and all have read `buf`
      }
      constexpr int PER = (NL + NR + (NM - H) - 1) / (NM - H);
#pragma unroll
      for (int m = 0; m < NM - H; ++m) {
        mfma_one(LAST, H + m);
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          const int op = m * PER + u;  // the next fragments first, then the loads
          if (op < NR) {
            if (more) read_one(nbuf, 0, 0, op);
          } else if (op < NR + NL) {
            if (refill) issue_one(it, kt + S, buf, op - NR);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      buf = nbuf;
    }
    __syncthreads();  // every wave is through with the stages

    const Item done = it;
    i += nb;
    const bool next = i < hi;
    if (next) {
      it = make(i);
      fill(it);
    }

    if (args.splits > 1) {
      float* const dst = args.partials + (int64_t)done.split * args.M * args.N;
#pragma unroll
      for (int a = 0; a < TM; ++a) {
        const int row = done.m0 + wm0 + a * 32 + (lane & 31);
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int col = done.n0 + wn0 + b * 32 + 8 * v + 4 * (lane >> 5);
            if (row < args.M && col < args.N)
              *(f32x4*)(dst + (int64_t)row * args.N + col) =
                  f32x4{acc[a][b][4 * v], acc[a][b][4 * v + 1], acc[a][b][4 * v + 2], acc[a][b][4 * v + 3]};
          }
      }
    } else {
      lds_char* const ep = lds + S * STAGE + wave * EP;
      const int rows = min(args.M - done.m0, BM);
      const int64_t base = (int64_t)done.m0 * args.N;
      const Epilogue& E = args.ep;
      const __amdgpu_buffer_rsrc_t rsY =
          __builtin_amdgcn_make_buffer_rsrc((void*)(E.y + base), (short)0, rows * args.N * 2, kBufferFlags);
      const __amdgpu_buffer_rsrc_t rsU = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((E.u ? E.u : E.y) + base), (short)0, rows * args.N * 2, kBufferFlags);
#pragma unroll
      for (int b = 0; b < TN; ++b) {
        const int col = done.n0 + wn0 + b * 32 + (lane % 4) * 8;  // this lane's 8 columns
        float bias[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) bias[v] = 0.0f;
        if (E.bias && col < args.N) widen8(*(const u32x4*)(E.bias + col), bias);
#pragma unroll
        for (int a = 0; a < TM; ++a) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int row = lane & 31, ch = v * 2 + (lane >> 5);
            *(__attribute__((address_space(3))) f32x4*)(ep + row * 128 + ((ch ^ ((row >> 1) & 7)) << 4)) =
                f32x4{acc[a][b][4 * v], acc[a][b][4 * v + 1], acc[a][b][4 * v + 2], acc[a][b][4 * v + 3]};
          }
          // a wave's LDS operations are done in their order
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = h * 16 + lane / 4, row = wm0 + a * 32 + r;
            const int64_t off = (int64_t)row * args.N + col;
            const bool inside = row < rows && col < args.N;
            u32x4 res = {0u, 0u, 0u, 0u};
            if (E.residual && inside) res = *(const u32x4*)(E.residual + base + off);
            float f[8];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const f32x4 w = *(__attribute__((address_space(3))) f32x4*)(
                  ep + r * 128 + ((((lane % 4) * 2 + v) ^ ((r >> 1) & 7)) << 4));
#pragma unroll
              for (int z = 0; z < 4; ++z) f[4 * v + z] = w[z] + bias[4 * v + z];
            }
            const int at = inside ? (int)(off * 2) : 0x7FFFFFF0;
            // u passes by the caches: the backward pass reads it, later than they keep it. By / through,
            // forward with u, and with the gradients right after: 512 x 2048 -> 2048 (2 MB) 23 / 23 and
            // 59 / 59 us, 2048 x 2048 -> 4096 (17 MB) 40 / 41 and 139 / 139, 4096 x 2048 -> 8192 (67 MB)
            // 132 / 134 and 448 / 448, 8192 x 2048 -> 8192 (134 MB) 274 / 293 and 809 / 818
            if (E.u) __builtin_amdgcn_raw_buffer_store_b128(narrow8(f), rsU, at, 0, 2);
            act_all<8>(f, E.act);
            if (E.residual) {
              float w[8];
              widen8(res, w);
#pragma unroll
              for (int v = 0; v < 8; ++v) f[v] += w[v];
            }
            __builtin_amdgcn_raw_buffer_store_b128(narrow8(f), rsY, at, 0, 0);
          }
        }
      }
    }
    if (!next) break;
  }
}

// Few rows, or few tiles: 32 x 32 results a workgroup, whose 8 waves share the steps
// along K. Each wave has a ring of its own in LDS and waits for nobody, so up to 128 KB
// are under way on a CU; the waves' sums meet in LDS in their order, and where the
// steps need no further cut the results leave in the same launch. (Tiles of 32 x 128 with
// barriers, always cut, and a second launch: 1 row of 2048 to 8192 12.9 us a call.)
// A tile of 32 columns with K outermost has rows of 64 bytes: 4 of them are one
// period of the banks, and a transposing read takes 4 rows as they are.
constexpr int kThin = 32, kThinWaves = 8, kThinStages = 2;

template <bool A_MN, bool B_MN>
__global__ __launch_bounds__(kThinWaves * kWave) void thin_kernel(DenseArgs args) {
  constexpr int OP = kThin * kBK * 2, STAGE = 2 * OP, RING = kThinStages * STAGE, LD = OP / 1024;
  __shared__ __attribute__((aligned(1024))) char smem[kThinWaves * RING];
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  lds_char* const ring = (lds_char*)smem + wave * RING;
  const uint32_t ring_addr = lds_addr(smem) + wave * RING;

  // neighbouring tiles along N on one XCD: two of them share a cache line of W
  const int tiles = args.m_tiles * args.n_tiles, total = tiles * args.splits;
  const int xcd = blockIdx.x % 8, lo = (int)((int64_t)total * xcd / 8), hi = (int)((int64_t)total * (xcd + 1) / 8);
  const int item = lo + (int)blockIdx.x / 8;
  if (item >= hi) return;
  const int split = item / tiles, t = item - split * tiles, mt = t / args.n_tiles;
  const int m0 = mt * kThin, n0 = (t - mt * args.n_tiles) * kThin;
  const int s0 = (int)((int64_t)args.nk * split / args.splits), s1 = (int)((int64_t)args.nk * (split + 1) / args.splits);
  const int kb = s0 + (s1 - s0) * wave / kThinWaves, kn = s0 + (s1 - s0) * (wave + 1) / kThinWaves - kb;

  i32x4 rsA, rsB;
  if constexpr (A_MN) rsA = buffer_rsrc(args.A, (uint32_t)((int64_t)args.K * args.lda * 2));
  else rsA = buffer_rsrc(args.A + (int64_t)m0 * args.lda, (uint32_t)((int64_t)min(args.M - m0, kThin) * args.lda * 2));
  if constexpr (B_MN) rsB = buffer_rsrc(args.B, (uint32_t)((int64_t)args.K * args.ldb * 2));
  else rsB = buffer_rsrc(args.B + (int64_t)n0 * args.ldb, (uint32_t)((int64_t)kThin * args.ldb * 2));
  uint32_t a_off[LD], b_off[LD];
#pragma unroll
  for (int l = 0; l < LD; ++l) {
    const Slot a = slot_of<A_MN, kThin>(l * kWave + lane), b = slot_of<B_MN, kThin>(l * kWave + lane);
    a_off[l] = A_MN ? (uint32_t)(a.k * args.lda + m0 + a.row) * 2u : (uint32_t)(a.row * args.lda + a.k) * 2u;
    b_off[l] = B_MN ? (uint32_t)(b.k * args.ldb + n0 + b.row) * 2u : (uint32_t)(b.row * args.ldb + b.k) * 2u;
  }
  auto issue = [&](int step) {
    const uint32_t st = ring_addr + (step % kThinStages) * STAGE, k = (uint32_t)(kb + step) * kBK;
#pragma unroll
    for (int l = 0; l < LD; ++l) buffer_load_lds16(rsB, b_off[l], k * (B_MN ? (uint32_t)args.ldb * 2u : 2u), st + OP + l * 1024);
#pragma unroll
    for (int l = 0; l < LD; ++l) buffer_load_lds16(rsA, a_off[l], k * (A_MN ? (uint32_t)args.lda * 2u : 2u), st + l * 1024);
  };
  const int q = lane & 15, g = lane >> 4;
  const int mn_rd = ((g >> 1) * 8 + (q >> 2)) * (kThin * 2) + ((g & 1) * 16 + (q & 3) * 4) * 2;
  auto fragment = [&](const lds_char* op, bool mn, int ks) {
    if (mn) {
      const lds_char* const p = op + ks * 16 * (kThin * 2) + mn_rd;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (kThin * 2)));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    const int row = lane & 31;
    return *(const lds_bf16x8*)(op + row * (kBK * 2) + (((ks * 2 + (lane >> 5)) ^ ((row >> 1) & 7)) << 4));
  };

  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
#pragma unroll
  for (int s = 0; s < kThinStages; ++s)
    if (s < kn) issue(s);
  for (int kt = 0; kt < kn; ++kt) {
    if (kt + 1 < kn) wait_vmem<2 * LD>();  // the next step's loads alone may be under way
    else wait_vmem<0>();
    const lds_char* const st = ring + (kt % kThinStages) * STAGE;
    bf16x8 a[kKS], b[kKS];
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      a[ks] = fragment(st, A_MN, ks);
      b[ks] = fragment(st + OP, B_MN, ks);
    }
    if (kt + kThinStages < kn) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads are through
      issue(kt + kThinStages);
    }
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[ks], a[ks], acc, 0, 0, 0);
  }
  // a lane's sums: row lane & 31, columns 8 v + 4 (lane >> 5) .. + 3
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int row = lane & 31, ch = v * 2 + (lane >> 5);
    *(__attribute__((address_space(3))) f32x4*)(ring + row * 128 + ((ch ^ (row & 7)) << 4)) =
        f32x4{acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3]};
  }
  __syncthreads();
  const int row = tid / 8, ch = tid % 8;  // 4 columns a thread
  if (row >= kThin || m0 + row >= args.M) return;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kThinWaves; ++w)
    sum += *(__attribute__((address_space(3))) f32x4*)((lds_char*)smem + w * RING + row * 128 + ((ch ^ (row & 7)) << 4));
  const int col = n0 + ch * 4;
  const int64_t off = (int64_t)(m0 + row) * args.N + col;
  if (args.splits > 1) {
    *(f32x4*)(args.partials + (int64_t)split * args.M * args.N + off) = sum;
    return;
  }
  const Epilogue& E = args.ep;
  auto widen4 = [](const bf16_bits* p, float* f) {
    const u32x2 v = *(const u32x2*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = bf16_to_f32(i & 1 ? v[i / 2] >> 16 : v[i / 2] & 0xFFFFu);
  };
  float f[4], w[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) f[v] = sum[v];
  if (E.bias) {
    widen4(E.bias + col, w);
#pragma unroll
    for (int v = 0; v < 4; ++v) f[v] += w[v];
  }
  if (E.u) *(u32x2*)(E.u + off) = u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
  act_all<4>(f, E.act);
  if (E.residual) {
    widen4(E.residual + off, w);
#pragma unroll
    for (int v = 0; v < 4; ++v) f[v] += w[v];
  }
  *(u32x2*)(E.y + off) = u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
}

// The cut tiles' sums in split order, 8 columns a thread
__global__ __launch_bounds__(256) void dense_join_kernel(const float* __restrict__ partials, Epilogue E, int64_t M, int N,
                                                         int splits) {
  const int64_t n = M * (N / 8);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t off = i * 8;
    const int col = (int)(off % N);
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const f32x4* p = (const f32x4*)(partials + s * M * N + off);
      const f32x4 a = p[0], b = p[1];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        f[v] += a[v];
        f[4 + v] += b[v];
      }
    }
    if (E.bias) {
      float b[8];
      widen8(*(const u32x4*)(E.bias + col), b);
#pragma unroll
      for (int v = 0; v < 8; ++v) f[v] += b[v];
    }
    if (E.u) *(u32x4*)(E.u + off) = narrow8(f);
    act_all<8>(f, E.act);
    if (E.residual) {
      float w[8];
      widen8(*(const u32x4*)(E.residual + off), w);
#pragma unroll
      for (int v = 0; v < 8; ++v) f[v] += w[v];
    }
    *(u32x4*)(E.y + off) = narrow8(f);
  }
}

// dU = dy act'(u), and sums of its columns: 256 columns by `rows` rows a workgroup, 8
// columns a thread and 8 rows beside each other. 8192 x 8192: 85 us for 403 MB, 4.7 TB/s
// (when it was 102, 2048 columns a workgroup, 4 KB of a row at a time, took 106). dy and u
// are loaded past the caches, which leaves dU there for the products: 8192 x 1024 -> 4096 with
// gradients 276 us, through them 295; 8192 x 2048 -> 8192 809 and 825; up to 34 MB of u equal.
// dU is rounded to bfloat16, as the products' operands are (two bfloat16 parts of it would
// make each product twice): dx and dW are then off by 0.0023 of themselves in the norm, the
// rounding of dU and their own being 0.0017 each. The sums of its columns are of dU before.
constexpr int kSlopeCols = 256;
template <int ACT>
__global__ __launch_bounds__(256) void slope_kernel(const bf16_bits* __restrict__ dy, const bf16_bits* __restrict__ u,
                                                    bf16_bits* __restrict__ du, float* __restrict__ sums, int64_t T, int N,
                                                    int64_t rows) {
  __shared__ float s_v[8][kSlopeCols];
  const int c = threadIdx.x % 32, r0 = threadIdx.x / 32, col = blockIdx.x * kSlopeCols + c * 8;
  const int64_t t0 = (int64_t)blockIdx.y * rows, t1 = min(T, t0 + rows);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (col < N) {
#pragma unroll 4
    for (int64_t t = t0 + r0; t < t1; t += 8) {
      float g[8];
      widen8(__builtin_nontemporal_load((const u32x4*)(dy + t * N + col)), g);
      if constexpr (ACT != MOET_ACT_NONE) {
        float z[8];
        widen8(__builtin_nontemporal_load((const u32x4*)(u + t * N + col)), z);
#pragma unroll
        for (int v = 0; v < 8; ++v) g[v] *= slope_one<ACT>(z[v]);
      }
      if (du) *(u32x4*)(du + t * N + col) = narrow8(g);
#pragma unroll
      for (int v = 0; v < 8; ++v) sum[v] += g[v];
    }
  }
  if (!sums) return;
#pragma unroll
  for (int v = 0; v < 8; ++v) s_v[r0][c * 8 + v] = sum[v];
  __syncthreads();
  const int n = blockIdx.x * kSlopeCols + threadIdx.x;
  if (n < N) {
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) v += s_v[r][threadIdx.x];
    sums[(int64_t)blockIdx.y * N + n] = v;
  }
}

// dbias: the workgroups' sums in their order, 16 columns and 16 slices of them a workgroup
__global__ __launch_bounds__(256) void dbias_kernel(const float* __restrict__ sums, bf16_bits* __restrict__ dbias, int parts,
                                                    int N) {
  __shared__ float s_v[16][16];
  const int c = threadIdx.x % 16, sl = threadIdx.x / 16, col = blockIdx.x * 16 + c;  // N is a multiple of 64
  float v = 0.0f;
#pragma unroll 4
  for (int i = sl; i < parts; i += 16) v += sums[(int64_t)i * N + col];
  s_v[sl][c] = v;
  __syncthreads();
  if (sl == 0) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += s_v[i][c];
    dbias[col] = (bf16_bits)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  }
}

}  // namespace

// The tile and the cut along K by estimated time, us, fitted to 17 shapes in three forms
// (rows 1 to 8192, widths 512 to 8192); what it takes is within 10% of the best of each.
// Measured in a graph on inputs that change, best cut of tile 0 / 1 / 2, x W with bias and
// GELU: 32 rows of 2048 to 8192 18.5 / 16.4 / 12.6, 256 of 2048 to 2048 26.9 / 16.7 / 18.1,
// 512 of 2048 to 2048 29.4 / 22.2 / 31.2, 2048 of 2048 to 2048 45.3 / 36.5 / -, 8192 of 2048 to
// 8192 255 / 276 / -.
DensePlan dense_plan(DenseForm form, int64_t M, int64_t N, int64_t K) {
  static const int edge[3] = {256, 128, kThin};
  const int cus = device_cus() / 8 * 8;
  const int64_t nk = ceil_div(K, (int64_t)kBK);
  // MOE_LINEAR_TILE=0|1|2 and MOE_LINEAR_SPLITS=<power of two> force the choice where it is possible
  const char *ft = getenv("MOE_LINEAR_TILE"), *fs = getenv("MOE_LINEAR_SPLITS");
  const int64_t most = max((int64_t)1, nk / 4);  // at least four steps of a cut tile
  DensePlan best{};
  double best_us = 1e30;
  for (int i = 0; i < 6 && (i < 3 || best.grid == 0); ++i) {
    const int tile = i % 3;  // all of them again only where a forced one is not possible
    if (i < 3 && ft && ft[0] && atoi(ft) != tile) continue;
    const int64_t mt = ceil_div(M, (int64_t)edge[tile]), nt = ceil_div(N, (int64_t)edge[tile]);
    for (int64_t splits = 1; splits <= 32 && splits <= most; splits *= 2) {
      const int64_t items = mt * nt * splits, steps = ceil_div(nk, splits);
      if (items >= (int64_t)1 << 22) continue;  // less than 2^32 threads, 8 for each a multiple
      if (fs && fs[0] && splits > 1 && splits > atoi(fs)) continue;
      double us, base;
      if (tile == 0) base = 5.0, us = ceil_div(items, (int64_t)cus) * steps * 1.8;
      else if (tile == 1)
        base = 4.0, us = steps * (items <= cus ? 0.7 + 0.25 * items / cus : ceil_div(items, (int64_t)2 * cus) * 1.2);
      else
        base = 3.0, us = max(1.0, (double)items / cus) * steps * (form == DENSE_NN ? 0.22 : form == DENSE_NT ? 0.18 : 0.25);
      us = base + max(us, 2.0 * (M * K + K * N) / 4.2e6);  // the operands have to come in
      if (splits > 1) us += (tile == 2 ? 3.5 : 3.0) + 8.0 * M * N * splits / 5.5e6;  // partial sums out and in, and their launch
      if (fs && fs[0]) us = -(double)splits;
      if (us < best_us) {
        best_us = us;
        best = {tile, (int)splits, (int)mt, (int)nt, (int)nk,
                (int)((tile == 0 ? min(items, (int64_t)cus) : tile == 1 ? min(items, (int64_t)2 * cus) : items) + 7) / 8 * 8};
      }
    }
  }
  return best;
}

size_t dense_partials_bytes(DenseForm form, int64_t M, int64_t N, int64_t K) {
  const DensePlan p = dense_plan(form, M, N, K);
  return p.splits > 1 ? (size_t)p.splits * M * N * sizeof(float) : 0;
}

hipError_t launch_dense(DenseForm form, const void* A, const void* B, int64_t M, int64_t N, int64_t K, const void* bias,
                        int act, const void* residual, void* u, void* y, float* partials, hipStream_t s) {
  const DensePlan p = dense_plan(form, M, N, K);
  DenseArgs a{};
  a.A = (const bf16_bits*)A;
  a.B = (const bf16_bits*)B;
  a.lda = (int)(form == DENSE_TN ? M : K);
  a.ldb = (int)(form == DENSE_NT ? K : N);
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.nk = p.nk;
  a.m_tiles = p.m_tiles;
  a.n_tiles = p.n_tiles;
  a.splits = p.splits;
  a.gm = group_m();
  a.ep = {(const bf16_bits*)bias, (const bf16_bits*)residual, (bf16_bits*)u, (bf16_bits*)y, act};
  a.partials = partials;
#define MOE_DENSE(AM, BM_, BM, BN, WM, WN, S, OCC)                                                                   \
  hipLaunchKernelGGL((dense_kernel<AM, BM_, BM, BN, WM, WN, S, OCC>), dim3((unsigned)p.grid), dim3(WM * WN * kWave), 0, \
                     s, a)
#define MOE_DENSE_FORM(BM, BN, WM, WN, S, OCC)                        \
  do {                                                                \
    if (form == DENSE_NN) MOE_DENSE(false, true, BM, BN, WM, WN, S, OCC);  \
    else MOE_DENSE(false, false, BM, BN, WM, WN, S, OCC);             \
  } while (0)
  if (p.tile == 2) {
    hipLaunchKernelGGL((form == DENSE_NN   ? thin_kernel<false, true>
                        : form == DENSE_NT ? thin_kernel<false, false>
                                           : thin_kernel<true, true>),
                       dim3((unsigned)p.grid), dim3(kThinWaves * kWave), 0, s, a);
  } else if (form == DENSE_TN) {
    if (p.tile == 0) MOE_DENSE(true, true, 256, 256, 2, 4, 2, 1);
    else MOE_DENSE(true, true, 128, 128, 2, 2, 2, 2);
  } else if (p.tile == 0) {
    MOE_DENSE_FORM(256, 256, 2, 4, 2, 1);
  } else {
    MOE_DENSE_FORM(128, 128, 2, 2, 2, 2);
  }
#undef MOE_DENSE_FORM
#undef MOE_DENSE
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t blocks = min(ceil_div(M * (N / 8), (int64_t)256), (int64_t)4096);
  hipLaunchKernelGGL(dense_join_kernel, dim3((unsigned)blocks), dim3(256), 0, s, (const float*)partials, a.ep, M, (int)N,
                     p.splits);
  return hipGetLastError();
}

// Workgroups along the rows: 8 rows each at least, about 2048 of them with those along the
// columns, and at most 256 sums of a column
int64_t slope_parts(int64_t T, int N) {
  return max((int64_t)1, min(min(ceil_div(T, (int64_t)8), (int64_t)256), ceil_div((int64_t)2048, ceil_div(N, (int64_t)kSlopeCols))));
}

hipError_t launch_slope(const void* dy, const void* u, int act, void* du, void* dbias, float* sums, int64_t T, int N,
                        hipStream_t s) {
  const int64_t parts = slope_parts(T, N), rows = ceil_div(ceil_div(T, parts), (int64_t)8) * 8;
  const int used = (int)ceil_div(T, rows);
  hipLaunchKernelGGL((act == MOET_ACT_GELU   ? slope_kernel<MOET_ACT_GELU>
                      : act == MOET_ACT_SILU ? slope_kernel<MOET_ACT_SILU>
                      : act == MOET_ACT_RELU ? slope_kernel<MOET_ACT_RELU>
                                             : slope_kernel<MOET_ACT_NONE>),
                     dim3((unsigned)ceil_div(N, kSlopeCols), (unsigned)used), dim3(256), 0, s, (const bf16_bits*)dy,
                     (const bf16_bits*)u, (bf16_bits*)du, dbias ? sums : nullptr, T, N, rows);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dbias) return e;
  hipLaunchKernelGGL(dbias_kernel, dim3((unsigned)(N / 16)), dim3(256), 0, s, (const float*)sums, (bf16_bits*)dbias, used, N);
  return hipGetLastError();
}

}  // namespace moe
