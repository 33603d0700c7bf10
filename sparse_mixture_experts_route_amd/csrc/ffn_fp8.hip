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
//
// Roundings: rows, weights and hidden activations to e4m3 (half a step, 2^-4), the
// result to bf16. Sums are float32; the instruction cuts the products it adds at
// once some 2^-12 below the largest (1.6e-5 of a dot product of normal data in the
// root mean square), less than the 2^-8 of the result's bf16. Hidden values that this
// carries over the border of two codes take the result from 0.0017 of it, the rounding
// to bf16 alone, to 0.0018 .. 0.0020.
//
// Measured on MI355X, where a large 8-bit library product reaches 2.9 PFLOP/s and
// a large copy 5.0 TB/s, both products together, on weights that change from call
// to call: 1 token, 64 experts of 2048 x 1024, top-8 14.7 us; 32 tokens, 8 experts of
// 2048 x 8192 58 us (4.7 TB/s of weights; 51 us on the same weights again, which the
// last-level cache holds in part); 8192 tokens of the fine experts 344 to 351 us (1.6
// PFLOP/s), 4096 tokens of the coarse ones 294 to 308 us (1.8 to 1.9).
#include <stdlib.h>

#include "common.h"
#include "e4m3.h"
#include "gemm_lanes.h"
#include "internal.h"
#include "lds_dma.h"
#include "tiles.h"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 join8(u32x4 a, u32x4 b) {
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

// A workgroup multiplies 32 rows by 32 NG columns; wave (g, ks) takes column
// group g and every KS-th block of 128 positions, straight from memory into
// registers, and the KS sums of a group are added in order through LDS.
// Bound by the weights' bytes (8 tokens of 64 experts of 7168 x 2048, top-8: 210 us,
// 5.5 TB/s), for few of them by the chain offsets, row numbers, rows, sums (one
// token of 2048 x 1024 10 + 5 us: the first product's 128 columns, those of a scale
// block, leave it 64 workgroups for 256 CUs, the second one has 256). 1, 2 or 4
// waves along the contraction are within 4% of each other at 1 to 777 tokens but for
// wide experts' second product (8192: 1 wave 64 us, 4 waves 50); loading the next
// weights ahead in registers costs the second workgroup of a CU (one token 13.5 ->
// 18.1 us).
template <int NG, int KS, bool ACT>
__global__ __launch_bounds__(NG * KS * kWave) void gemm_fp8_small_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const int32_t* __restrict__ perm, int64_t a_rows,
    const int32_t* __restrict__ offsets, const uint8_t* __restrict__ B, const uint8_t* __restrict__ Bs,
    void* __restrict__ C, uint8_t* __restrict__ Cs, int64_t R, int K, int N, int E, int n_tiles) {
  static_assert(!ACT || NG == 4, "an 8-bit output block spans 128 columns");
  constexpr int BM = 32;
  __shared__ int s_info[3];
  __shared__ float s_acc[KS > 1 ? (KS - 1) * NG * 16 * kWave : 1];
  __shared__ float s_max[ACT ? NG * BM : 1];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int g = wave % NG, ks = wave / NG;
  const uint32_t tile = blockIdx.y * gridDim.x + blockIdx.x, m_tile = tile / (uint32_t)n_tiles;
  const int n_tile = (int)(tile - m_tile * (uint32_t)n_tiles);
  find_rows<BM>(offsets, E, R, (int)m_tile, s_info);
  const int e = s_info[0];
  if (e < 0) return;  // the whole workgroup
  const int64_t row0 = s_info[1], row_end = s_info[2];
  const int ng = n_tile * NG + g;  // column group
  const bool cols = ng * 32 < N;
  const int KB = (int)(code_pitch(K) / kQBlock);
  const int64_t cp = code_pitch(K), sp = scale_pitch(K);
  const int half = lane >> 5;
  const int64_t row = row0 + (lane & 31);
  int64_t src = min(row, row_end - 1);  // rows past the end repeat the last
  if (perm) {
    src = perm[src];
    if (src < 0 || src >= a_rows) src = 0;
  }
  const u32x4* pa = (const u32x4*)(A + src * cp) + half;
  const uint8_t* ps = As + src * sp;
  const int64_t slab = (int64_t)e * (N / 32) + (cols ? ng : 0);
  const u32x4* pb = (const u32x4*)(B + slab * KB * 4096) + half * 32 + (lane & 31);
  const uint8_t* pbs = Bs + slab * KB * 32 + (lane & 31);
  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
  if (cols) {
#pragma unroll 2
    for (int kb = ks; kb < KB; kb += KS) {
      u32x4 a[4], b[4];
      const int sa = ps[kb], sb = pbs[kb * 32];
#pragma unroll
      for (int q = 0; q < 4; ++q) b[q] = pb[(int64_t)kb * 256 + q * 64];
#pragma unroll
      for (int q = 0; q < 4; ++q) a[q] = pa[kb * 8 + q * 2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join8(b[2 * j], b[2 * j + 1]),
                                                              join8(a[2 * j], a[2 * j + 1]), acc, 0, 0, 0, sb, 0, sa);
    }
  }
  if constexpr (KS > 1) {
    if (ks > 0)
#pragma unroll
      for (int v = 0; v < 16; ++v) s_acc[(((ks - 1) * NG + g) * 16 + v) * kWave + lane] = acc[v];
    __syncthreads();
    if (ks == 0)
#pragma unroll
      for (int u = 0; u < KS - 1; ++u)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[v] += s_acc[((u * NG + g) * 16 + v) * kWave + lane];
  }
  if constexpr (ACT) {
    if (ks == 0) {
      float m = 0.0f;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        acc[v] = gelu_tanh(acc[v]);  // 0 stays 0: columns past N
        m = fmaxf(m, fabsf(acc[v]));
      }
      s_max[g * BM + (lane & 31)] = fmaxf(m, __shfl_xor(m, 32, kWave));
    }
    __syncthreads();
    if (ks > 0) return;
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < NG; ++u) m = fmaxf(m, s_max[u * BM + (lane & 31)]);
    if (row >= row_end) return;
    const int byte = scale_byte(m);
    const float inv = inv_scale(byte);
    uint8_t* out = (uint8_t*)C + row * code_pitch(N) + (int64_t)ng * 32 + 4 * half;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *(uint32_t*)(out + 8 * v) = encode4(acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3], inv);
    if (g == 0 && half == 0) Cs[row * scale_pitch(N) + n_tile] = (uint8_t)byte;
  } else {
    if (ks > 0 || !cols || row >= row_end) return;
    bf16_bits* out = (bf16_bits*)C + row * N + ng * 32 + 4 * half;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      u32x2 o;
      o[0] = pack_bf16x2(acc[4 * v], acc[4 * v + 1]);
      o[1] = pack_bf16x2(acc[4 * v + 2], acc[4 * v + 3]);
      *(u32x2*)(out + 8 * v) = o;
    }
  }
}

// ---- 256 x 256 tiles of large groups
//
// Eight waves of 64 x 128 (two per SIMD: one multiplies while the other issues
// loads), a step of 128 positions, two LDS stages of 64 KB filled by direct
// loads, persistent workgroups over a tile list made on the device. A sits
// row-major in LDS with the 16-byte piece index XOR-ed by (row >> 1) & 7, so
// the 16 lanes served together touch every bank once; a stage of B is a
// straight copy of the weight layout, in which a wave's fragment read is 1 KB
// in lane order. The scales of four steps, a dword a row, are one load per wave
// and come in two windows used in turn. A fragment of B is read again as soon
// as the two instructions that use it are issued, so only A needs two register
// sets: 192 of the 256 registers that two waves per SIMD leave hold operands
// and sums.
//
// The ring runs on across tiles: a tile's last two steps already load the next
// tile's first two stages, and the epilogue works in 2 KB of LDS per wave of
// its own while they arrive. Tiles are short (8 to 64 steps), so a ring that
// drained between them cost a third of the time.
//
// Measured: 1.75 us a step with all CUs busy (1.48 would be the library product's
// rate; 1.33 without the stage loads: matrix instructions and fragment reads, 256 KB
// of LDS traffic a step; 1.25 to 1.66 the loads alone, by how many of them miss the
// L2). The GELU epilogue is 6 to 8 us of a tile, its exponential and reciprocal at a
// quarter of the vector rate. Without GELU the stores cost nearly as much: the second
// product of 8192 tokens of the fine experts, 9 rounds of tiles of 8 steps and 268 MB
// of result, takes 187 us, with its stores dropped 151 (126 of steps, 3 a round
// around them). Four waves of 128 x 128, half stages in a ring of
// four, wave groups a phase apart and prefetching the weights into the L2 all ended
// at the same step or above it.
constexpr int L_BM = 256, L_BN = 256, L_NW = 8, L_WN = 2, L_TM = 2, L_TN = 4;
constexpr int L_A = L_BM * kQBlock, L_B = L_BN * kQBlock, L_STAGE = L_A + L_B;
constexpr int L_WIN = 2048;       // four steps' scales of 256 rows, then of 256 columns
constexpr int L_EP = 2048;        // epilogue staging per wave
constexpr int L_NL = L_STAGE / 1024 / L_NW;  // loads per wave and stage
constexpr int L_ALD = L_NL / 2;

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 4 bytes per lane into LDS when `now` is 0 (wave-uniform). The branch stays
// inside the block: in the source it would end the basic block, and the matrix
// instructions before it would sink behind it.
__device__ __forceinline__ void buffer_load_lds4_if0(int now, i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile(
      "s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lmoe_win%=\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
      "buffer_load_dword %2, %3, %4 offen lds\n.Lmoe_win%=:"
      :
      : "s"(now), "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// At most N of this wave's vector-memory operations outstanding, none when `all` is 0 (wave-uniform).
template <int N>
__device__ __forceinline__ void wait_vmem_all_if0(int all) {
  asm volatile(
      "s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lmoe_wait%=\n\ts_waitcnt vmcnt(0)\n.Lmoe_wait%=:\n\ts_waitcnt vmcnt(%1)"
      :
      : "s"(all), "n"(N)
      : "memory", "scc");
}

// Tiles of an expert: ceil(rows / 256) m-tiles of n_tiles each. A last m-tile of
// at most 128 rows costs less than a whole one; those come after all others, so
// that a last, partly filled round of tiles is a cheap one.
struct TileList {
  int start[257], tail[257];  // first tile of each expert among either, and their numbers
  int lo[256], hi[256];       // its rows
};

// m-tiles of a group of `rows` rows that are not a tail of at most half a tile
__device__ __forceinline__ int full_m_tiles(int rows) { return rows / L_BM + (rows % L_BM > L_BM / 2 ? 1 : 0); }

// Wave 0 builds the list; ends with a barrier.
__device__ __forceinline__ void build_list(const int32_t* __restrict__ offsets, int E, int64_t R, int n_tiles,
                                           TileList& list) {
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    int cnt[4], tail[4], local = 0, tlocal = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane * 4 + i;
      int rows = 0;
      if (e < E) {
        const int lo = max(offsets[e], 0), hi = (int)min((int64_t)offsets[e + 1], R);
        list.lo[e] = lo;
        list.hi[e] = hi;
        rows = max(hi - lo, 0);
      }
      cnt[i] = full_m_tiles(rows) * n_tiles;
      tail[i] = rows % L_BM > 0 && rows % L_BM <= L_BM / 2 ? n_tiles : 0;
      local += cnt[i];
      tlocal += tail[i];
    }
    int incl = local, tincl = tlocal;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave), w = __shfl_up(tincl, o, kWave);
      if (lane >= o) {
        incl += v;
        tincl += w;
      }
    }
    int run = incl - local, trun = tincl - tlocal;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (lane * 4 + i < E) {
        list.start[lane * 4 + i] = run;
        list.tail[lane * 4 + i] = trun;
      }
      run += cnt[i];
      trun += tail[i];
    }
    if (lane == kWave - 1) {
      list.start[E] = incl;
      list.tail[E] = tincl;
    }
  }
  __syncthreads();
}

// An XCD's contiguous share of either list (workgroups are dealt to the 8 XCDs
// in turn): n_full tiles from `lo`, then tails from `tlo`, n_all together.
struct XcdShare {
  int lo, n_full, tlo, n_all;
};
__device__ __forceinline__ XcdShare xcd_share(const TileList& list, int E, int xcd) {
  const int total = __builtin_amdgcn_readfirstlane(list.start[E]), tails = __builtin_amdgcn_readfirstlane(list.tail[E]);
  XcdShare s;
  s.lo = (int)((int64_t)total * xcd / 8);
  s.n_full = (int)((int64_t)total * (xcd + 1) / 8) - s.lo;
  s.tlo = (int)((int64_t)tails * xcd / 8);
  s.n_all = s.n_full + (int)((int64_t)tails * (xcd + 1) / 8) - s.tlo;
  return s;
}

// Tile `i` of an XCD's share; every lane of the wave takes part.
struct TilePlace {
  int e, n_tile, row0, rows;
};
__device__ __forceinline__ TilePlace find_tile(const TileList& list, const XcdShare& share, int E, int i, int n_tiles,
                                               int gm) {
  const int lane = threadIdx.x % kWave;
  const bool is_tail = i >= share.n_full;
  const int t = is_tail ? share.tlo + i - share.n_full : share.lo + i;
  const int* const start = is_tail ? list.tail : list.start;
  int e = 0;  // experts after the first that start at or before t
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4) {
    const int q = 1 + q4 * kWave + lane;
    e += __popcll(__ballot(q < E && start[q < E ? q : 0] <= t));
  }
  TilePlace p;
  p.e = __builtin_amdgcn_readfirstlane(e);
  const int first = __builtin_amdgcn_readfirstlane(list.lo[p.e]), end = __builtin_amdgcn_readfirstlane(list.hi[p.e]);
  const int mt = full_m_tiles(end - first), local = t - __builtin_amdgcn_readfirstlane(start[p.e]);
  int m_idx = mt;
  p.n_tile = local;
  if (!is_tail) tile_coords(local, mt, n_tiles, gm, p.n_tile, m_idx);
  p.row0 = first + m_idx * L_BM;
  p.rows = min(end - p.row0, L_BM);
  return p;
}

// Tiles of a last round are cut where that saves at least so many pairs of steps:
// 21 us at the 1.75 us of a step, against 10 us of the launch that joins the parts
// (4096x2048, 8 experts of 8192: second product 166 us whole, 131 + 10 us cut)
constexpr int kFp8SplitPairs = 6;

template <bool ACT, bool GATHER>
__global__ __launch_bounds__(L_NW * kWave, 1) void gemm_fp8_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const int32_t* __restrict__ perm, int64_t a_rows,
    const int32_t* __restrict__ offsets, const uint8_t* __restrict__ B, const uint8_t* __restrict__ Bs,
    void* __restrict__ C, uint8_t* __restrict__ Cs, int64_t R, int K, int N, int E, int n_tiles, int gm,
    float* __restrict__ partials, int max_rem) {
  __shared__ __attribute__((aligned(1024))) char smem[2 * L_STAGE + 2 * L_WIN + L_NW * L_EP];
  __shared__ TileList list;
  const int tid = threadIdx.x, lane = tid % kWave, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  build_list(offsets, E, R, n_tiles, list);
  const int xcd = blockIdx.x % 8, nb = gridDim.x / 8, j = blockIdx.x / 8;
  const XcdShare share = xcd_share(list, E, xcd);
  // whole tiles, then, of products with a long contraction, at most two parts of
  // the tiles of a last round, cut between pairs of steps
  const int pairs = (int)(code_pitch(K) / kQBlock) >> 1;
  const SplitK sk = split_k(share.n_all, nb, j, pairs, kFp8SplitPairs, max_rem);
  const int n_items = sk.n_items;
  if (n_items == 0) return;
  const int cp = (int)code_pitch(K), sp = (int)scale_pitch(K), KB = cp / kQBlock;  // KB >= 2
  lds_char* const lds = (lds_char*)smem;
  const uint32_t lds_base = lds_addr(smem);
  const int wm0 = (wave / L_WN) * (L_TM * 32), wn0 = (wave % L_WN) * (L_TN * 32);

  struct Tile {
    int e, n0, row0, rows;  // rows of the group from row0 on, at most L_BM
    int kb, kn, slot;       // first step and steps; slot of its partial sums (-1: the tile is whole)
  };
  struct Loads {
    i32x4 rsA, rsB, rsS;
    uint32_t ga[L_ALD], gs, gb;  // this lane's byte offsets of the A, scale and B loads
  };
  // the rows of this lane's A pieces and scale load (waves 0 .. 3 load the rows' scales, 4 .. 7 the columns')
  int a_row[L_ALD], a_c16[L_ALD];
#pragma unroll
  for (int i = 0; i < L_ALD; ++i) {
    const lanes::Piece pc = lanes::a_piece<64>((wave * L_ALD + i) * 64 + lane);  // 128-byte rows
    a_row[i] = pc.row;
    a_c16[i] = pc.c * 16;
  }
  const int s_row = (wave & 3) * 64 + lane;
  // tile t; past the workgroup's last item: no rows and no columns
  auto locate = [&](int item) {
    Tile tl = {0, 0, 0, 0, 0, KB, -1};
    if (item >= n_items) return tl;
    int i0 = j + item * nb;
    if (item >= sk.full && sk.rem > 0) {
      const int r = sk.r_first + item - sk.full;
      i0 = sk.full * nb + r;
      const int first = (int)max(sk.s0 - (int64_t)r * pairs, (int64_t)0), last = (int)min(sk.s1 - (int64_t)r * pairs, (int64_t)pairs);
      tl.kb = 2 * first;
      tl.kn = (last == pairs ? KB : 2 * last) - tl.kb;
      if (tl.kn < KB) tl.slot = (int)blockIdx.x * 2 + item - sk.full;
    }
    const TilePlace pl = find_tile(list, share, E, i0, n_tiles, gm);
    tl.e = pl.e;
    tl.row0 = pl.row0;
    tl.rows = pl.rows;
    tl.n0 = pl.n_tile * L_BN;
    return tl;
  };
  auto load_perm = [&](const Tile& t_, int (&pv)[L_ALD + 1]) {
#pragma unroll
    for (int i = 0; i <= L_ALD; ++i) {
      const int r = i < L_ALD ? a_row[i < L_ALD ? i : 0] : s_row;
      pv[i] = r < t_.rows ? perm[t_.row0 + r] : -1;
    }
  };
  auto bind = [&](const Tile& t_, const int (&pv)[L_ALD + 1]) {
    Loads l;
    const bool some = t_.rows > 0;
    l.rsA = GATHER ? buffer_rsrc(A, some ? (uint32_t)(a_rows * cp) : 0u)
                   : buffer_rsrc(A + (int64_t)t_.row0 * cp, (uint32_t)(t_.rows * cp));
    l.rsB = buffer_rsrc(B + (int64_t)t_.e * N * cp, some ? (uint32_t)((int64_t)N * cp) : 0u);
    if (wave < 4)
      l.rsS = GATHER ? buffer_rsrc(As, some ? (uint32_t)(a_rows * sp) : 0u)
                     : buffer_rsrc(As + (int64_t)t_.row0 * sp, (uint32_t)(t_.rows * sp));
    else
      l.rsS = buffer_rsrc(Bs + (int64_t)t_.e * N * KB, some ? (uint32_t)((int64_t)N * KB) : 0u);
#pragma unroll
    for (int i = 0; i <= L_ALD; ++i) {
      const int row = i < L_ALD ? a_row[i < L_ALD ? i : 0] : s_row;
      const int src = GATHER ? pv[i] : row;  // past the group's end: -1, or past the descriptor's range
      const bool ok = src >= 0 && (!GATHER || src < a_rows);
      if (i < L_ALD)
        l.ga[i] = ok ? (uint32_t)src * (uint32_t)cp + a_c16[i < L_ALD ? i : 0] : lanes::kOutOfRange;
      else
        l.gs = ok ? (uint32_t)src * (uint32_t)sp : lanes::kOutOfRange;
    }
    const int g = t_.n0 / 32 + wave;  // this wave's column group of the stage
    l.gb = g * 32 < N ? (uint32_t)g * (uint32_t)(KB * 4096) + lane * 16 : lanes::kOutOfRange;
    if (wave >= 4) {
      const int sg = t_.n0 / 32 + (wave - 4) * 2 + half;
      l.gs = sg * 32 < N ? (uint32_t)sg * (uint32_t)(KB * 32) + (lane & 31) * 4 : lanes::kOutOfRange;
    }
    return l;
  };
  // Load `i` of step kt's stage into ring buffer `buf`. Windows: that of steps
  // 4 w .. goes out before the first of them, into the buffer of window w - 2,
  // whose last scales were read two steps ago.
  auto issue_one = [&](const Loads& l, int kt, int buf, int i) {
    if (i < L_ALD)
      buffer_load_lds16(l.rsA, l.ga[i], (uint32_t)kt * kQBlock, lds_base + buf * L_A + (wave * L_ALD + i) * 1024);
    else
      buffer_load_lds16(l.rsB, l.gb, (uint32_t)kt * 4096u + (i - L_ALD) * 1024u,
                        lds_base + 2 * L_A + buf * L_B + wave * 4096 + (i - L_ALD) * 1024);
  };
  auto issue_window = [&](const Loads& l, int kt, int wbuf, int now) {
    buffer_load_lds4_if0(now, l.rsS, l.gs, (uint32_t)(kt >> 2) * (wave < 4 ? 4u : 128u),
                         lds_base + 2 * L_STAGE + wbuf * L_WIN + wave * 256);
  };

  i32x8 fa[2][L_TM], fb[L_TN];
  int sa = 0, sb = 0, sa_n[L_TM], sb_n[L_TN];  // the scale bytes of a step, one per byte
  f32x16 acc[L_TM][L_TN];
  typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  typedef __attribute__((address_space(3))) uint32_t lds_u32;
  typedef __attribute__((address_space(3))) uint8_t lds_u8;
  // LDS addresses of this lane's fragment pieces in the buffer being read: both
  // operands' buffers are L_A apart, so a step moves them all by +-L_A
  static_assert(L_A == L_B, "one distance moves both operands' addresses");
  uint32_t ra[4], rb;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    ra[q] = lds_base + (wm0 + (lane & 31)) * kQBlock + (((2 * q + half) ^ (((lane & 31) >> 1) & 7)) << 4);
  rb = lds_base + 2 * L_A + wn0 * kQBlock + lane * 16;
  auto move_addresses = [&](int buf) {  // to ring buffer `buf` from the other one
    const uint32_t d = buf ? (uint32_t)L_A : (uint32_t)-L_A;
#pragma unroll
    for (int q = 0; q < 4; ++q) asm("v_add_u32 %0, %0, %1" : "+v"(ra[q]) : "s"(d));
    asm("v_add_u32 %0, %0, %1" : "+v"(rb) : "s"(d));
  };
  auto read_a = [&](int js, int mi) {
    fa[js][mi] = join8(*(lds_u32x4*)(uintptr_t)(ra[2 * js] + mi * (32 * kQBlock)),
                       *(lds_u32x4*)(uintptr_t)(ra[2 * js + 1] + mi * (32 * kQBlock)));
  };
  auto read_b = [&](int js, int ni) {
    fb[ni] = join8(*(lds_u32x4*)(uintptr_t)(rb + ni * 4096 + js * 2048),
                   *(lds_u32x4*)(uintptr_t)(rb + ni * 4096 + js * 2048 + 1024));
  };
  auto read_scales = [&](int kt, int wbuf) {
    lds_char* const w = lds + 2 * L_STAGE + wbuf * L_WIN;
#pragma unroll
    for (int mi = 0; mi < L_TM; ++mi) sa_n[mi] = *(lds_u8*)(w + (kt & 3) + (wm0 + (lane & 31)) * 4 + mi * 128);
#pragma unroll
    for (int ni = 0; ni < L_TN; ++ni)
      sb_n[ni] = *(lds_u8*)(w + 1024 + (kt & 3) * 32 + wn0 * 4 + (lane & 31) + ni * 128);
  };
  auto take_scales = [&]() {
    sa = sa_n[0] | sa_n[1] << 8;
    sb = sb_n[0] | sb_n[1] << 8 | sb_n[2] << 16 | sb_n[3] << 24;
  };
  auto mfma = [&](int js, auto mi_c, auto ni_c) {
    constexpr int mi = decltype(mi_c)::value, ni = decltype(ni_c)::value;
    acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[ni], fa[js][mi], acc[mi][ni], 0, 0, ni, sb, mi, sa);
  };
  auto mfma_pair = [&](int js, int ni, auto after) {
    auto two = [&](auto ni_c) {
      mfma(js, IntC<0>{}, ni_c);
      after(0);
      __builtin_amdgcn_sched_barrier(0);
      mfma(js, IntC<1>{}, ni_c);
      after(1);
      __builtin_amdgcn_sched_barrier(0);
    };
    if (ni == 0) two(IntC<0>{});
    else if (ni == 1) two(IntC<1>{});
    else if (ni == 2) two(IntC<2>{});
    else two(IntC<3>{});
  };
  // stores of an epilogue, each issued whatever its lanes hold
  constexpr int EP_ST = ACT ? 8 + L_TM : 16;
  // One step of 128 positions from ring buffer `buf`. After the barrier in its
  // middle that buffer is free: step `fill` of `l` is loaded into it, its window
  // (when it starts one) into `fwin`. LAST (of a tile): the next step's stage is
  // waited for after the epilogue. Else the next step kt + 1 has to have landed
  // (its scales in window `nwin`) and its first fragments are read here; `stores`
  // is not 0 where an epilogue's stores came after the loads waited for.
  auto step = [&](const Loads& l, int kt, int buf, int nwin, int fill, int fwin, int fnow, int stores, auto last_c) {
    constexpr bool LAST = decltype(last_c)::value;
#pragma unroll
    for (int ni = 0; ni < L_TN; ++ni)
      mfma_pair(0, ni, [&](int mi) {
        if (ni == 0) read_a(1, mi);
        if (mi == 1) read_b(1, ni);
      });
#pragma unroll
    for (int ni = 0; ni < L_TN / 2; ++ni) mfma_pair(1, ni, [](int) {});
    if constexpr (!LAST) wait_vmem_all_if0<EP_ST>(stores);
    __syncthreads();  // step kt + 1 is in for every wave, and every wave is done reading this buffer
    if constexpr (!LAST) {
      move_addresses(buf ^ 1);
      read_scales(kt + 1, nwin);
#pragma unroll
      for (int mi = 0; mi < L_TM; ++mi) read_a(0, mi);
#pragma unroll
      for (int ni = 0; ni < L_TN / 2; ++ni) read_b(0, ni);
    }
    issue_window(l, fill, fwin, fnow);
#pragma unroll
    for (int ni = L_TN / 2; ni < L_TN; ++ni)
      mfma_pair(1, ni, [&](int mi) {
        if (!LAST && mi == 1) read_b(0, ni);
        const int at = (ni - L_TN / 2) * L_TM + mi;  // 0 .. 3: two loads each
        issue_one(l, fill, buf, 2 * at);
        issue_one(l, fill, buf, 2 * at + 1);
      });
    if constexpr (!LAST) take_scales();
  };
  auto idle_step = [&](const Loads& l, int buf, int fill, int fwin, int fnow, int stores, bool last) {
    if (!last) wait_vmem_all_if0<EP_ST>(stores);
    __syncthreads();
    issue_window(l, fill, fwin, fnow);
#pragma unroll
    for (int i = 0; i < L_NL; ++i) issue_one(l, fill, buf, i);
  };

  Tile tl = locate(0), nxt;
  Loads ld;
  int npv[L_ALD + 1];
  if constexpr (GATHER) load_perm(tl, npv);
  ld = bind(tl, npv);
  issue_window(ld, tl.kb, 0, 0);
#pragma unroll
  for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
    for (int i = 0; i < L_NL; ++i) issue_one(ld, tl.kb + s2, s2, i);
  int buf = 0, win = 0;  // ring buffer and window of the item's first step

  for (int item = 0; item < n_items; ++item) {
    // the tile's first stage: its second one, and the last tile's stores, were issued after it
    if (item == 0) wait_vmem<L_NL>();
    else wait_vmem<L_NL + EP_ST>();
    __syncthreads();
    nxt = locate(item + 1);
    if constexpr (GATHER) load_perm(nxt, npv);
#pragma unroll
    for (int mi = 0; mi < L_TM; ++mi)
#pragma unroll
      for (int ni = 0; ni < L_TN; ++ni)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[mi][ni][v] = 0.0f;
    // window of block kb: win + kb / 4 - tl.kb / 4; the next item's first one: win + nwins.
    // (Items start at even blocks, so a second block never starts a window.)
    const int end = tl.kb + tl.kn, w0 = win - (tl.kb >> 2), nwins = ((end - 1) >> 2) - (tl.kb >> 2) + 1;
    const int b0 = buf - tl.kb;  // ring buffer of block kb: (b0 + kb) & 1
    if (tl.rows > wm0) {
      read_scales(tl.kb, win & 1);
      take_scales();
#pragma unroll
      for (int mi = 0; mi < L_TM; ++mi) read_a(0, mi);
#pragma unroll
      for (int ni = 0; ni < L_TN; ++ni) read_b(0, ni);
      for (int kb = tl.kb; kb < end - 2; ++kb)
        step(ld, kb, (b0 + kb) & 1, (w0 + ((kb + 1) >> 2)) & 1, kb + 2, (w0 + ((kb + 2) >> 2)) & 1, (kb + 2) & 3,
             kb == tl.kb ? item : 0, BoolC<false>{});
      ld = bind(nxt, npv);
      step(ld, end - 2, (b0 + end) & 1, (w0 + ((end - 1) >> 2)) & 1, nxt.kb, (win + nwins) & 1, 0,
           tl.kn == 2 ? item : 0, BoolC<false>{});
      step(ld, end - 1, (b0 + end + 1) & 1, 0, nxt.kb + 1, 0, 1, 0, BoolC<true>{});
      move_addresses((b0 + end) & 1);
    } else {
      // all of this wave's rows lie past the group's end: its share of the loads alone
      for (int kb = tl.kb; kb < end - 2; ++kb)
        idle_step(ld, (b0 + kb) & 1, kb + 2, (w0 + ((kb + 2) >> 2)) & 1, (kb + 2) & 3, kb == tl.kb ? item : 0, false);
      ld = bind(nxt, npv);
      idle_step(ld, (b0 + end) & 1, nxt.kb, (win + nwins) & 1, 0, tl.kn == 2 ? item : 0, false);
      idle_step(ld, (b0 + end + 1) & 1, nxt.kb + 1, 0, 1, 0, true);
      if (tl.kn & 1) move_addresses((buf + 1) & 1);
    }
    if (tl.rows <= wm0) {
      // nothing to store, but the waits below count stores: leave nothing for them to wait for
      wait_vmem<0>();
    } else if (!ACT && tl.slot >= 0) {
      // part of a tile: its sums in the accumulators' layout, 16 bytes per lane and
      // register group (more stores than the waits below allow for: only stricter)
      float* const dst = partials + (int64_t)tl.slot * (L_BM * L_BN) + tid * 4;
#pragma unroll
      for (int mi = 0; mi < L_TM; ++mi)
#pragma unroll
        for (int ni = 0; ni < L_TN; ++ni)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *(f32x4*)(dst + ((mi * L_TN + ni) * 4 + v) * (L_NW * kWave * 4)) =
                f32x4{acc[mi][ni][4 * v], acc[mi][ni][4 * v + 1], acc[mi][ni][4 * v + 2], acc[mi][ni][4 * v + 3]};
    } else {
    lds_char* const ep = lds + 2 * L_STAGE + 2 * L_WIN + wave * L_EP;
    // 32 rows of 64 bytes at a time: pieces of 16 bytes, XOR-ed by the row
    auto ep_at = [&](int row, int ch) { return ep + row * 64 + ((ch ^ ((row >> 2) & 3)) << 4); };
    if constexpr (ACT) {
      const int hp = (int)code_pitch(N), hs = (int)scale_pitch(N);
      const __amdgpu_buffer_rsrc_t rsC = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((uint8_t*)C + (int64_t)tl.row0 * hp), (short)0, tl.rows * hp, kBufferFlags);
      const __amdgpu_buffer_rsrc_t rsCs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(Cs + (int64_t)tl.row0 * hs), (short)0, tl.rows * hs, kBufferFlags);
      const int col = tl.n0 + wn0;
      const bool cols = col < hp;
#pragma unroll
      for (int mi = 0; mi < L_TM; ++mi) {
        float m = 0.0f;
#pragma unroll
        for (int ni = 0; ni < L_TN; ++ni)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            acc[mi][ni][v] = gelu_tanh(acc[mi][ni][v]);
            m = fmaxf(m, fabsf(acc[mi][ni][v]));
          }
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        const int byte = scale_byte(m);
        const float inv = inv_scale(byte);
        const int row = lane & 31;
#pragma unroll
        for (int np = 0; np < 2; ++np) {  // 64 columns at a time
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const int ni = np * 2 + v / 4, q = v % 4;
            *(lds_u32*)(ep_at(row, v / 2) + (v & 1) * 8 + half * 4) =
                encode4(acc[mi][ni][4 * q], acc[mi][ni][4 * q + 1], acc[mi][ni][4 * q + 2], acc[mi][ni][4 * q + 3], inv);
          }
          // a wave's LDS operations complete in order: no barrier before its own reads
#pragma unroll
          for (int it = 0; it < 2; ++it) {
            const int r = it * 16 + lane / 4, ch = lane % 4;
            const u32x4 v = *(lds_u32x4*)ep_at(r, ch);
            __builtin_amdgcn_raw_buffer_store_b128(
                v, rsC, cols ? (wm0 + mi * 32 + r) * hp + col + np * 64 + ch * 16 : 0x7FFFFFF0, 0, 0);
          }
        }
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)byte, rsCs,
                                             cols && half == 0 ? (wm0 + mi * 32 + row) * hs + col / kQBlock : 0x7FFFFFF0,
                                             0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      const __amdgpu_buffer_rsrc_t rsC = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((bf16_bits*)C + (int64_t)tl.row0 * N), (short)0, tl.rows * N * 2, kBufferFlags);
#pragma unroll
      for (int mi = 0; mi < L_TM; ++mi)
#pragma unroll
        for (int ni = 0; ni < L_TN; ++ni) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            u32x2 o;
            o[0] = pack_bf16x2(acc[mi][ni][4 * v], acc[mi][ni][4 * v + 1]);
            o[1] = pack_bf16x2(acc[mi][ni][4 * v + 2], acc[mi][ni][4 * v + 3]);
            *(lds_u32x2*)(ep_at(lane & 31, v) + half * 8) = o;
          }
#pragma unroll
          for (int it = 0; it < 2; ++it) {
            const int r = it * 16 + lane / 4, ch = lane % 4;
            const u32x4 v = *(lds_u32x4*)ep_at(r, ch);
            const int n = tl.n0 + wn0 + ni * 32 + ch * 8;
            __builtin_amdgcn_raw_buffer_store_b128(v, rsC, lanes::c_store_off(wm0 + mi * 32 + r, n, N), 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    }
    tl = nxt;
    buf = (b0 + end) & 1;
    win += nwins;
  }
  wait_vmem<0>();  // the loads past the last tile (of no bytes) have ended before the LDS is given back
}

// The tiles that were cut: workgroup (x, sub, r0) adds the parts of 32 rows and 128
// columns of the last round's tiles r0, r0 + gridDim.z, ... of XCD x in the order
// of their steps, rounds once and stores.
__global__ __launch_bounds__(4 * kWave) void gemm_fp8_join_kernel(const int32_t* __restrict__ offsets,
                                                                  const float* __restrict__ partials,
                                                                  bf16_bits* __restrict__ C, int64_t R, int N, int E,
                                                                  int n_tiles, int gm, int nb, int pairs,
                                                                  int max_rem) {
  __shared__ TileList list;
  build_list(offsets, E, R, n_tiles, list);
  const int xcd = blockIdx.x, part = blockIdx.y, lane = threadIdx.x % kWave, ni = threadIdx.x / kWave;
  const XcdShare share = xcd_share(list, E, xcd);
  const int full = share.n_all / nb, rem = share.n_all - full * nb;
  if (!split_leftover(rem, nb, pairs, kFp8SplitPairs, max_rem)) return;
  const int64_t W = (int64_t)rem * pairs;
  const int wave = part / L_TM, mi = part % L_TM;  // the GEMM's wave and row group
  const int wm = wave / L_WN * (L_TM * 32) + mi * 32, wn = wave % L_WN * (L_TN * 32);
  for (int r = blockIdx.z; r < rem; r += gridDim.z) {
    const TilePlace pl = find_tile(list, share, E, full * nb + r, n_tiles, gm);
    const int n = pl.n_tile * L_BN + wn + ni * 32;
    if (pl.rows <= wm || n >= N) continue;
    // workgroups j whose pairs [W j / nb, W (j + 1) / nb) meet the tile's [r pairs, (r + 1) pairs)
    const int64_t u0 = (int64_t)r * pairs, u1 = u0 + pairs;
    int j0 = (int)(u0 * nb / W), j1 = (int)min((u1 * nb + W - 1) / W, (int64_t)nb);
    while (W * (j0 + 1) / nb <= u0) ++j0;
    if (W * j0 / nb <= u0 && W * (j0 + 1) / nb >= u1) continue;  // one workgroup did it all and has stored it
    const float* const src = partials + (int64_t)(mi * L_TN + ni) * 4 * (L_NW * kWave * 4) + (wave * kWave + lane) * 4;
    f32x4 acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j = j0; j < j1; j += 4) {  // four parts' loads in flight
      f32x4 u[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t s0 = W * (j + q) / nb, s1 = W * (j + q + 1) / nb;
        const bool has = j + q < j1 && s1 > s0 && s0 < u1;
        const int slot = ((j + q) * 8 + xcd) * 2 + r - (int)(s0 / pairs);
        const f32x4* const p = (const f32x4*)(src + (has ? (int64_t)slot * (L_BM * L_BN) : 0));
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          u[q][v] = p[v * (L_NW * kWave)];  // of slot 0 when there is no part: dropped
          if (!has) u[q][v] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] += u[q][v];
    }
    const int row = wm + (lane & 31);
    if (row >= pl.rows) continue;
    bf16_bits* const out = C + (int64_t)(pl.row0 + row) * N + n + 4 * (lane >> 5);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      u32x2 o;
      o[0] = pack_bf16x2(acc[v][0], acc[v][1]);
      o[1] = pack_bf16x2(acc[v][2], acc[v][3]);
      *(u32x2*)(out + 8 * v) = o;
    }
  }
}

// Weights [K, N] of one expert to codes and scales. A workgroup takes 128
// positions of 64 columns: rows of 64 bf16 are read whole, transposed through
// LDS, and 16 codes of a column leave as one 16-byte piece. Called once per set of
// weights: 1.3 TB/s (64 experts of 2048 x 1024 0.62 ms, 256 of 7168 x 2048 16.7 ms), 2
// bytes a lane and load.
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

// Whether a product takes the 256 x 256 tiles rather than workgroups of 32 rows
// that read the weights straight into registers. The tiles do a matrix
// instruction's work with an eighth of the weight reads, the small form has no
// pipeline to fill and eight times the workgroups. Both estimates in us, from
// times on MI355X over 1 .. 6000 tokens of five layer shapes (three below): a
// workgroup of the small form costs about 0.7 us per block of 128 positions and 128
// columns, four blocks' worth of it before the first; a tile 1.5 us a block and 6 us
// around them, per round of tiles. Both products of a layer, us, small form / tiles:
// 8192-wide coarse experts at 8 rows an expert 50 / 102, at 128 220 / 125;
// 64 fine experts of 2048 x 1024 at 4 rows 50 / 56, at 64 132 / 63; 12 experts of
// 320 x 448 at 194 rows 17 / 26, at 1500 65 / 31. (Workgroups of 64 and 128 rows
// were behind one of the two at every size.)
// MOE_FP8_TILES=0|1 forces the choice where both are possible.
bool fp8_tiles(int64_t R, int K, int N, int E) {
  if (K <= kQBlock) return false;  // the tiles' pipeline needs two steps
  const char* force = getenv("MOE_FP8_TILES");
  if (force && force[0]) return atoi(force) != 0;
  const double kb = (double)(code_pitch(K) / kQBlock), cus = device_cus(), busy = (double)min(R, (int64_t)E);
  const double m_small = max(busy, R / 32.0 + 0.5 * E), m_large = max(busy, (double)R / L_BM + 0.5 * E);
  const double small = m_small * N / 128.0 * (kb + 4.0) * 0.7 / cus;
  const double rounds = m_large * ceil_div(N, L_BN) / cus;
  const double large = (double)(int64_t)(rounds + 0.999) * (1.5 * kb + 6.0);
  return large < small;
}

template <int NG, int KS, bool ACT>
hipError_t launch_small(const void* A, const void* As, const int32_t* perm, int64_t a_rows, const int32_t* offsets,
                        const void* B, const void* Bs, void* C, void* Cs, int64_t R, int K, int N, int E,
                        hipStream_t s) {
  const int n_tiles = (int)ceil_div(N, 32 * NG);
  const int64_t grid = m_tiles_bound(R, E, 32) * n_tiles;
  // a launch takes less than 2^32 threads along x: the other workgroups go along y
  const int64_t gy = ceil_div(grid, (int64_t)1 << 21), gx = ceil_div(grid, gy);
  hipLaunchKernelGGL((gemm_fp8_small_kernel<NG, KS, ACT>), dim3((unsigned)gx, (unsigned)gy), dim3(NG * KS * kWave), 0,
                     s, (const uint8_t*)A, (const uint8_t*)As, perm, a_rows, offsets, (const uint8_t*)B,
                     (const uint8_t*)Bs, C, (uint8_t*)Cs, R, K, N, E, n_tiles);
  return hipGetLastError();
}

// persistent workgroups of the tiles: one per CU, as many on every XCD
unsigned fp8_grid(int64_t R, int N, int E) {
  const int64_t tiles = m_tiles_bound(R, E, L_BM) * ceil_div(N, L_BN);
  return (unsigned)max((int64_t)8, min(ceil_div(tiles, 8) * 8, (int64_t)device_cus() / 8 * 8));
}

// Whether a contraction is long enough for a last round's tiles to be cut.
bool fp8_splits(int K) { return code_pitch(K) / kQBlock / 2 > kFp8SplitPairs; }

}  // namespace

bool gemm_fp8_fits(int64_t R, int N, int E) { return m_tiles_bound(R, E, 32) * ceil_div(N, 64) <= INT32_MAX; }

size_t gemm_fp8_partials_bytes(int64_t R, int K, int N, int E) {
  if (!fp8_tiles(R, K, N, E) || !fp8_splits(K)) return 0;
  return (size_t)fp8_grid(R, N, E) * 2 * L_BM * L_BN * sizeof(float);  // two parts per workgroup at most
}

hipError_t launch_gemm_fp8(const void* A, const void* As, const int32_t* perm, int64_t a_rows, const int32_t* offsets,
                           const void* B, const void* Bs, void* C, void* Cs, int64_t R, int K, int N, int E, bool act,
                           float* partials, hipStream_t s) {
  if (!gemm_fp8_fits(R, N, E)) return hipErrorInvalidValue;
  if (fp8_tiles(R, K, N, E)) {
    const int n_tiles = (int)ceil_div(N, L_BN);
    const unsigned grid = fp8_grid(R, N, E);
    const int nb = (int)grid / 8, pairs = (int)(code_pitch(K) / kQBlock) / 2;
    const int max_rem = !act && partials && fp8_splits(K) ? nb - 1 : 0;
#define MOE_LAUNCH(ACT_, GATHER_)                                                                                \
  hipLaunchKernelGGL((gemm_fp8_kernel<ACT_, GATHER_>), dim3(grid), dim3(L_NW * kWave), 0, s, (const uint8_t*)A,  \
                     (const uint8_t*)As, perm, a_rows, offsets, (const uint8_t*)B, (const uint8_t*)Bs, C,        \
                     (uint8_t*)Cs, R, K, N, E, n_tiles, group_m(), partials, max_rem)
    if (act && perm) MOE_LAUNCH(true, true);
    else if (act) MOE_LAUNCH(true, false);
    else MOE_LAUNCH(false, false);
#undef MOE_LAUNCH
    if (max_rem > 0)
      hipLaunchKernelGGL(gemm_fp8_join_kernel, dim3(8, L_NW * L_TM, 4), dim3(4 * kWave), 0, s, offsets,
                         (const float*)partials, (bf16_bits*)C, R, N, E, n_tiles, group_m(), nb, pairs, max_rem);
    return hipGetLastError();
  }
  if (act) return launch_small<4, 4, true>(A, As, perm, a_rows, offsets, B, Bs, C, Cs, R, K, N, E, s);
  return launch_small<2, 4, false>(A, As, perm, a_rows, offsets, B, Bs, C, Cs, R, K, N, E, s);
}

// less than 2^32 threads along x
bool quantize_weights_fits(int K, int N) { return code_pitch(K) / kQBlock * (N / 64) < (int64_t)1 << 24; }

hipError_t launch_quantize_weights(const void* w, void* q, void* qs, int E, int K, int N, hipStream_t s) {
  if (!quantize_weights_fits(K, N)) return hipErrorInvalidValue;
  const int KB = (int)(code_pitch(K) / kQBlock);
  const int64_t grid = (int64_t)KB * (N / 64);
  hipLaunchKernelGGL(quantize_weights_kernel, dim3((unsigned)grid, (unsigned)E), dim3(256), 0, s, (const bf16_bits*)w,
                     (uint8_t*)q, (uint8_t*)qs, K, N, KB);
  return hipGetLastError();
}

}  // namespace moe
