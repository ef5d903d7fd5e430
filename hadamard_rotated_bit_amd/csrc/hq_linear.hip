// Dense linear layer of libhq (the layers that stay in 16 or 32 bits beside
// the low-bit ones): Y = R + g phi(X W^T + b) with X [M, K], W [N, K] (the
// nn.Linear layout: both operands K-contiguous, no transposition anywhere) in
// bf16 or fp32, fp32 accumulation, and the epilogue of hq_epilogue.h.
//
// Kernels, chosen by shape (linear_plan):
//  linear_rows_kernel   M <= 4: one pass over W on the vector ALU.
//  linear_few_kernel    16 x 16 tiles for products of few tiles.
//  linear_tile_kernel   MFMA tiles of 32 x 64 to 128 x 192; few tiles share
//                       their k-steps among groups of waves and are split over K
//                       (partial sums in the workspace, added in split order by
//                       linear_reduce_kernel, which then runs the epilogue).
//  linear_pp_kernel     bf16 tiles of 256 x 192 and 256 x 256.
#include "hq_epilogue.h"
#include "hq_gemm6_kernel.h"
#include "hq_internal.h"

#include <algorithm>

namespace hq {

// ---- few rows ------------------------------------------------------------------
//
// One wave owns NC output columns and all TT rows; its lanes split K in
// pieces of 8 elements, U pieces of 512 per wave and pass, all of W's and X's
// loads of a pass in flight before the first is used. The wave's sums meet in a
// fixed lane tree. Bound by reading W once (N K elements); X is read by every
// wave from L2. 2 x 1152 -> 6912 bf16: 5.8 us, 2.7 TB/s (16 MB fill the chip for
// too short a time to reach a copy's rate); 1 x 256 -> 1152: 2.9 us, latency.
template <typename TE, int TT, int NC>
__global__ __launch_bounds__(256) void linear_rows_kernel(const TE* __restrict__ X, int M,
                                                          const TE* __restrict__ W, int64_t N,
                                                          int K, LinEpi ep) {
  constexpr int U = TT <= 2 ? 4 : 3;   // bounded by the registers of the X pieces
  const int lane = threadIdx.x & 63;
  const int64_t n0 = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6)) * NC;
  if (n0 >= N) return;
  const TE* wp[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) wp[c] = W + (n0 + c < N ? n0 + c : N - 1) * K;
  const TE* xp[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) xp[t] = X + int64_t(t < M ? t : M - 1) * K;
  float acc[TT][NC];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[t][c] = 0.0f;
  for (int kb = lane * 8; kb < K; kb += 512 * U) {
    Raw8<TE> w[U][NC], x[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + 512 * u < K) {
#pragma unroll
        for (int c = 0; c < NC; ++c) w[u][c] = raw_load(wp[c] + kb + 512 * u);
#pragma unroll
        for (int t = 0; t < TT; ++t) x[u][t] = raw_load(xp[t] + kb + 512 * u);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + 512 * u < K) {
        float wf[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) raw_get(w[u][c], wf[c]);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          float xf[8];
          raw_get(x[u][t], xf);
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[t][c] = fmaf(xf[e], wf[c][e], acc[t][c]);
        }
      }
    }
  }
  // every lane ends with every sum; lane t NC + c finishes output (t, n0 + c)
  float v = 0.0f;
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float s = group_sum<64>(acc[t][c]);
      if (lane == t * NC + c) v = s;
    }
  const int m = lane / NC;
  const int64_t n = n0 + lane % NC;
  if (lane < TT * NC && m < M && n < N) finish1(v, m, n, N, ep);
}

// ---- MFMA tiles -----------------------------------------------------------------
//
// Fragments: for a 32 x 128-byte piece of an operand, lane l holds row l % 32,
// 16-byte chunk 2 s + l / 32 of substep s = 0 .. 3. In bf16 a chunk is the 8
// consecutive k of one v_mfma_f32_32x32x16_bf16. The weight fragment is the
// first operand: lane l's accumulator r belongs to row l % 32 and column
// 8 (r / 4) + 4 (l / 32) + r % 4.
//
// fp32 operands run on the bf16 matrix units too: x = h + m + l with h the
// upper 16 bits of x (a bf16 by truncation), m those of x - h and l = x - h - m,
// which has 8 bits left, all three exact (|x| >= 2^-110: below, l is cut at 2^-133, the
// smallest bf16; the matrix unit keeps subnormals). The product keeps
//   x w = h h + (h m + m h) + (h l + m m + l h)
// and leaves m l and l m, each at most 2^-22 of |x w| (with |x| in [2^e, 2^(e+1)):
// m < 2^(e-7), l < 2^(e-15)), and l l below 2^-29; sums stay in fp32. Six MFMAs of 32
// cycles per 16 k instead of eight v_mfma_f32_32x32x2_f32 of 64 cycles. With m
// rounded to nearest the two are half as large, but every size took 2 to 4 % longer.
// (The split of an infinity is inf, NaN, NaN: an infinite operand gives NaN.)
// The 8 values per lane are two chunks, substeps 2 t and 2 t + 1: any pairing
// of k is the same sum, as both operands use the same one.
struct Split {
  v8bf h, m, l;
};
__device__ __forceinline__ Split split8(const v4i& c0, const v4i& c1) {
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x0 = uint32_t(i < 2 ? c0[2 * i] : c1[2 * i - 4]);
    const uint32_t x1 = uint32_t(i < 2 ? c0[2 * i + 1] : c1[2 * i - 3]);
    const float r0 = __uint_as_float(x0) - __uint_as_float(x0 & 0xFFFF0000u);
    const float r1 = __uint_as_float(x1) - __uint_as_float(x1 & 0xFFFF0000u);
    const uint32_t b0 = __float_as_uint(r0), b1 = __float_as_uint(r1);
    const float l0 = r0 - __uint_as_float(b0 & 0xFFFF0000u);
    const float l1 = r1 - __uint_as_float(b1 & 0xFFFF0000u);
    h[i] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);   // the upper halves of a pair
    m[i] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
    l[i] = __builtin_amdgcn_perm(__float_as_uint(l1), __float_as_uint(l0), 0x07060302u);
  }
  Split s;
  s.h = __builtin_bit_cast(v8bf, make_uint4(h[0], h[1], h[2], h[3]));
  s.m = __builtin_bit_cast(v8bf, make_uint4(m[0], m[1], m[2], m[3]));
  s.l = __builtin_bit_cast(v8bf, make_uint4(l[0], l[1], l[2], l[3]));
  return s;
}

__device__ __forceinline__ v16f mfma_bf16(const v8bf& w, const v8bf& x, const v16f& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x, c, 0, 0, 0);
}

// The bias as accumulators: register r of strip j belongs to column n + 32 j +
// 8 (r / 4) + r % 4 (the same for every row), zero without a bias. bf16 products
// start from it; an fp32 one would round all six of its terms at the bias's size, so
// it is added to their sum.
template <int TN>
__device__ __forceinline__ void bias_strips(v16f (&b)[TN], const float* __restrict__ bias, int64_t n,
                                            int64_t N) {
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int64_t c = n + 32 * j + 8 * g;
      const float4 v = bias && c < N ? *reinterpret_cast<const float4*>(bias + c)
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      b[j][4 * g] = v.x;
      b[j][4 * g + 1] = v.y;
      b[j][4 * g + 2] = v.z;
      b[j][4 * g + 3] = v.w;
    }
}

// A wave's staged 32 rows as raw sums into part [M, N].
template <int LPR>
__device__ __forceinline__ void store_part(const float* stg, int pitch, int lane, int64_t m0,
                                           int64_t n0, int64_t M, int64_t N, float* part) {
#pragma unroll
  for (int q = 0; q < 32 * LPR / 64; ++q) {
    const int i = lane + 64 * q, r = i / LPR, c = 8 * (i - r * LPR);
    float v[8];
    load8(stg + r * pitch + c, v);
    if (m0 + r < M && n0 + c < N) store8(part + (m0 + r) * N + n0 + c, v);
  }
}

// Instruction order: NM MFMAs with NV vector instructions spread between them.
template <int I, int NM, int NV>
__device__ __forceinline__ void mfma_valu_interleave() {
  if constexpr (I < NM) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr int v = (I + 1) * NV / NM - I * NV / NM;
    __builtin_amdgcn_sched_group_barrier(0x002, v, 0);
    mfma_valu_interleave<I + 1, NM, NV>();
  }
}

// The products of one k-step.
template <typename TE, int TM, int TN>
__device__ __forceinline__ void lin_kstep(v16f (&acc)[TM][TN], const v4i (&a)[TM][4],
                                          const v4i (&b)[TN][4]) {
  if constexpr (sizeof(TE) == 2) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = mfma_bf16(__builtin_bit_cast(v8bf, b[j][s]), __builtin_bit_cast(v8bf, a[i][s]),
                                acc[i][j]);
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      Split x[TM], w[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) x[i] = split8(a[i][2 * t], a[i][2 * t + 1]);
#pragma unroll
      for (int j = 0; j < TN; ++j) w[j] = split8(b[j][2 * t], b[j][2 * t + 1]);
      // the small terms first, each over all tiles before the next
#define HL_TERM(W_, X_)                                                     \
  _Pragma("unroll") for (int i = 0; i < TM; ++i)                            \
      _Pragma("unroll") for (int j = 0; j < TN; ++j) acc[i][j] = mfma_bf16(w[j].W_, x[i].X_, acc[i][j])
      HL_TERM(l, h);
      HL_TERM(m, m);
      HL_TERM(h, l);
      HL_TERM(m, h);
      HL_TERM(h, m);
      HL_TERM(h, h);
#undef HL_TERM
    }
    // the second half's split runs between the first half's MFMAs
    constexpr int NM = 6 * TM * TN, NV = 44 * (TM + TN);
    __builtin_amdgcn_sched_group_barrier(0x002, NV, 0);
    mfma_valu_interleave<0, NM, NV>();
    __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
  }
}

// LDS fragment reads are inline asm that waits for its own results: written as
// ordinary loads, the compiler would wait for every stage load in flight (it
// cannot tell that they fill other buffers). All fragments of a k-step are read
// at once (one LDS latency per k-step): p[s], q[s] are the addresses of substep
// s of the wave's rows of A and of B; a second 32-row block is 4096 bytes on.
__device__ __forceinline__ void lds_kstep(v4i (&a)[1][4], v4i (&b)[1][4], const uint32_t (&p)[4],
                                          const uint32_t (&q)[4]) {
  asm volatile(
      "ds_read_b128 %0, %8\n ds_read_b128 %4, %12\n ds_read_b128 %1, %9\n ds_read_b128 %5, %13\n"
      "ds_read_b128 %2, %10\n ds_read_b128 %6, %14\n ds_read_b128 %3, %11\n ds_read_b128 %7, %15\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(b[0][0]),
        "=&v"(b[0][1]), "=&v"(b[0][2]), "=&v"(b[0][3])
      : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3])
      : "memory");
}
__device__ __forceinline__ void lds_kstep(v4i (&a)[2][4], v4i (&b)[1][4], const uint32_t (&p)[4],
                                          const uint32_t (&q)[4]) {
  asm volatile(
      "ds_read_b128 %0, %12\n ds_read_b128 %4, %12 offset:4096\n ds_read_b128 %8, %16\n"
      "ds_read_b128 %1, %13\n ds_read_b128 %5, %13 offset:4096\n ds_read_b128 %9, %17\n"
      "ds_read_b128 %2, %14\n ds_read_b128 %6, %14 offset:4096\n ds_read_b128 %10, %18\n"
      "ds_read_b128 %3, %15\n ds_read_b128 %7, %15 offset:4096\n ds_read_b128 %11, %19\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(a[1][0]),
        "=&v"(a[1][1]), "=&v"(a[1][2]), "=&v"(a[1][3]), "=&v"(b[0][0]), "=&v"(b[0][1]),
        "=&v"(b[0][2]), "=&v"(b[0][3])
      : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3])
      : "memory");
}
__device__ __forceinline__ void lds_kstep(v4i (&a)[2][4], v4i (&b)[2][4], const uint32_t (&p)[4],
                                          const uint32_t (&q)[4]) {
  asm volatile(
      "ds_read_b128 %0, %16\n ds_read_b128 %4, %16 offset:4096\n"
      "ds_read_b128 %8, %20\n ds_read_b128 %12, %20 offset:4096\n"
      "ds_read_b128 %1, %17\n ds_read_b128 %5, %17 offset:4096\n"
      "ds_read_b128 %9, %21\n ds_read_b128 %13, %21 offset:4096\n"
      "ds_read_b128 %2, %18\n ds_read_b128 %6, %18 offset:4096\n"
      "ds_read_b128 %10, %22\n ds_read_b128 %14, %22 offset:4096\n"
      "ds_read_b128 %3, %19\n ds_read_b128 %7, %19 offset:4096\n"
      "ds_read_b128 %11, %23\n ds_read_b128 %15, %23 offset:4096\n s_waitcnt lgkmcnt(0)"
      : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(a[1][0]),
        "=&v"(a[1][1]), "=&v"(a[1][2]), "=&v"(a[1][3]), "=&v"(b[0][0]), "=&v"(b[0][1]),
        "=&v"(b[0][2]), "=&v"(b[0][3]), "=&v"(b[1][0]), "=&v"(b[1][1]), "=&v"(b[1][2]),
        "=&v"(b[1][3])
      : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3])
      : "memory");
}

__device__ __forceinline__ void lds_kstep(v4i (&a)[2][4], v4i (&b)[3][4], const uint32_t (&p)[4],
                                          const uint32_t (&q)[4]) {
  asm volatile(
      "ds_read_b128 %0, %20\n ds_read_b128 %4, %20 offset:4096\n ds_read_b128 %8, %24\n"
      "ds_read_b128 %12, %24 offset:4096\n ds_read_b128 %16, %24 offset:8192\n"
      "ds_read_b128 %1, %21\n ds_read_b128 %5, %21 offset:4096\n ds_read_b128 %9, %25\n"
      "ds_read_b128 %13, %25 offset:4096\n ds_read_b128 %17, %25 offset:8192\n"
      "ds_read_b128 %2, %22\n ds_read_b128 %6, %22 offset:4096\n ds_read_b128 %10, %26\n"
      "ds_read_b128 %14, %26 offset:4096\n ds_read_b128 %18, %26 offset:8192\n"
      "ds_read_b128 %3, %23\n ds_read_b128 %7, %23 offset:4096\n ds_read_b128 %11, %27\n"
      "ds_read_b128 %15, %27 offset:4096\n ds_read_b128 %19, %27 offset:8192\n s_waitcnt lgkmcnt(0)"
      : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(a[1][0]),
        "=&v"(a[1][1]), "=&v"(a[1][2]), "=&v"(a[1][3]), "=&v"(b[0][0]), "=&v"(b[0][1]),
        "=&v"(b[0][2]), "=&v"(b[0][3]), "=&v"(b[1][0]), "=&v"(b[1][1]), "=&v"(b[1][2]),
        "=&v"(b[1][3]), "=&v"(b[2][0]), "=&v"(b[2][1]), "=&v"(b[2][2]), "=&v"(b[2][3])
      : "v"(p[0]), "v"(p[1]), "v"(p[2]), "v"(p[3]), "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3])
      : "memory");
}

// f6_tile_origin gives the blocks of one XCD (block b runs on XCD b mod 8) a
// contiguous range of tiles where the count n is a multiple of 8; this does it
// for other counts of no more than one tile per CU (the first n mod 8 XCDs have
// one tile more): a weight row is then fetched by one or two XCDs instead of
// all (300 x 4096 -> 1152 bf16, 180 tiles of two groups: 13.8 us against 15.6; 367 x
// 3808 -> 6896, 162 tiles of 128 x 128: 33.6 against 36.3). With several
// tiles per CU the plain order, in which an XCD keeps to one tile row, is as good
// or better (1037 x 1160 -> 2312 in 323 tiles of 64 x 128: 18.8 us against 20.3).
__device__ __forceinline__ int xcd_tile(int tile, int n) {
  const int odd = n & 7, x = tile & 7;
  if (odd == 0 || n > 256) return tile;
  return x * (n >> 3) + (x < odd ? x : odd) + (tile >> 3);
}

// BM x BN tile, waves of WM x WN (32 or 64 rows and columns), S stage buffers of 128
// bytes per row (64 bf16 or 32 fp32 values of K), filled by buffer loads
// straight into LDS, S - 1 stages ahead. Rows past M or N and chunks past K
// lie outside the tile's buffer descriptor: they arrive as zeros and move no
// memory, so any M, N and any K of whole chunks takes the same loop. Chunk c
// of row r sits in slot c ^ ((r / 2) mod 8): the 16 lanes of one read phase
// hit 16 distinct 16-byte positions of the 64 banks.
// blockIdx.y is the split: k-steps [kper y, kper (y + 1)); with more than one
// split the raw sums go to part [splits, M, N]. G groups of waves hold the whole
// tile each and share the k-steps of a block among them (group g takes steps g,
// g + G, ...; one barrier per G steps), for products with too few tiles to fill
// the CUs: their sums meet in LDS, in group order.
// Few tiles are bound by the latency of their k-steps (300 x 4096 -> 1152 bf16:
// 12.0 us; 1037 x 1160 -> 2312: 16.8 us, where rows of 2320 bytes straddle the
// 128-byte lines), fp32 by the vector instructions of the splits beside the MFMAs
// (8192 x 4096 -> 4096: 1.38 ms, 199 TFLOP/s; 12288 x 256 -> 256: 17.7 us).
template <typename TE, int BM, int BN, int WM, int WN, int G, int S, int OCC>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64 * G)
__attribute__((amdgpu_waves_per_eu(OCC))) void linear_tile_kernel(
    const TE* __restrict__ X, int64_t M, const TE* __restrict__ W, int64_t N, int K, int kper,
    float* __restrict__ part, LinEpi ep) {
  constexpr int NW = (BM / WM) * (BN / WN), WAVES_N = BN / WN;
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW, L = LA + LB;
  constexpr int STAGE = 128 * (BM + BN);
  constexpr int SPITCH = 4 * WN + 16;            // staging row: WN floats and one 16-byte pad
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN && NW % 2 == 0, "whole 1-KB units per wave");
  static_assert(TM <= 2 && TN <= TM + 1, "waves of 32 x 32 or 64 x 32, 64 or 96");
  static_assert(G * NW * 32 * SPITCH <= S * G * STAGE, "epilogue staging fits in the stage buffers");
  static_assert((S - 1) * L <= 63, "outstanding loads fit vmcnt");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * G * STAGE];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int grp = wave / NW, wv = wave % NW;     // k group, wave of the tile
  int64_t m0, n0;
  f6_tile_origin<BM, BN, 8>(xcd_tile(int(blockIdx.x), int(gridDim.x)), M, N, &m0, &n0);
  const int wm0 = (wv / WAVES_N) * WM, wn0 = (wv % WAVES_N) * WN;
  const int ldb = K * int(sizeof(TE));
  const int ksteps = (ldb + 127) / 128;
  const int kt0 = int(blockIdx.y) * kper;
  const int KT = (ksteps - kt0) < kper ? (ksteps - kt0) : kper;

  const int64_t rows_a = (M - m0) < BM ? (M - m0) : BM;
  const int64_t rows_b = (N - n0) < BN ? (N - n0) : BN;
  const uint8_t* const abase = reinterpret_cast<const uint8_t*>(X) + m0 * ldb;
  const uint8_t* const bbase = reinterpret_cast<const uint8_t*>(W) + n0 * ldb;
  const int nrec_a = int(rows_a * ldb), nrec_b = int(rows_b * ldb);
  // Unit u (1 KB of LDS) holds 8 rows: lane l fetches the chunk that belongs
  // in slot l % 8 of row 8 u + l / 8. u = q NW + wv has wv's parity, so the
  // chunk is the same for all of a wave's units.
  const int chunk = (lane & 7) ^ (((wv & 1) * 4 + (lane >> 4)) & 7);
  const uint32_t voff = uint32_t((8 * wv + (lane >> 3)) * ldb + 16 * chunk);
#define HL_ISSUE(KT_)                                                                        \
  do {                                                                                       \
    const int kt_ = (KT_);                                                                   \
    uint8_t* base_ = smem + ((kt_ % S) * G + grp) * STAGE;                                   \
    const bool ok_ = kt_ * G + grp < KT;                                                     \
    const int kb_ = (kt0 + kt_ * G + grp) * 128;                                             \
    const __amdgpu_buffer_rsrc_t ra_ = make_rsrc(abase, ok_ ? nrec_a : 0);                   \
    const __amdgpu_buffer_rsrc_t rb_ = make_rsrc(bbase, ok_ ? nrec_b : 0);                   \
    const bool in_ = kb_ + 16 * chunk < ldb;                                                 \
    _Pragma("unroll") for (int q = 0; q < LA; ++q)                                           \
        lds_dma16_buf(ra_, in_ ? voff + uint32_t(8 * q * NW * ldb + kb_) : 0x80000000u, 0u,  \
                      base_ + (q * NW + wv) * 1024);                                         \
    _Pragma("unroll") for (int q = 0; q < LB; ++q)                                           \
        lds_dma16_buf(rb_, in_ ? voff + uint32_t(8 * q * NW * ldb + kb_) : 0x80000000u, 0u,  \
                      base_ + 128 * BM + (q * NW + wv) * 1024);                              \
  } while (0)

  const int lrow = lane & 31, lhalf = lane >> 5;
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(smem));
  uint32_t pa[4], pb[4];   // substep s of the wave's first rows of A and B in buffer 0
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t co = lds0 + uint32_t(grp * STAGE) + uint32_t(((2 * s + lhalf) ^ ((lrow >> 1) & 7)) * 16);
    pa[s] = co + uint32_t((wm0 + lrow) * 128);
    pb[s] = co + uint32_t((BM + wn0 + lrow) * 128);
  }

  v16f acc[TM][TN], bias[TN];
  bias_strips<TN>(bias, part || grp ? nullptr : ep.bias, n0 + wn0 + 4 * lhalf, N);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if constexpr (sizeof(TE) == 2) acc[i][j] = bias[j];
      else acc[i][j] = v16f{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    }
#pragma unroll
  for (int p = 0; p < S - 1; ++p) HL_ISSUE(p);
  int buf = 0;
  for (int kt = 0; kt * G < KT; ++kt) {
    // stage kt has landed in every wave; every wave is done with stage kt - 1
    wait_vm_lgkm0<(S - 2) * L>();
    __builtin_amdgcn_s_barrier();
    HL_ISSUE(kt + S - 1);
    const uint32_t o = uint32_t(buf * (G * STAGE));
    buf = buf == S - 1 ? 0 : buf + 1;
    v4i af[TM][4], bf[TN][4];
    const uint32_t qa[4] = {pa[0] + o, pa[1] + o, pa[2] + o, pa[3] + o};
    const uint32_t qb[4] = {pb[0] + o, pb[1] + o, pb[2] + o, pb[3] + o};
    lds_kstep(af, bf, qa, qb);
    __builtin_amdgcn_sched_barrier(0);
    lin_kstep<TE, TM, TN>(acc, af, bf);
    __builtin_amdgcn_sched_barrier(0);
  }
#undef HL_ISSUE
  wait_vm_lgkm0<0>();  // no LDS write may land in the staging area (or after the block ends)
  __builtin_amdgcn_s_barrier();

  if constexpr (sizeof(TE) == 4) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] += bias[j];
  }

  // Each wave stages its 32-row slices in its own part of the LDS and takes
  // them back as rows, eight consecutive columns per lane: whole row segments
  // per store, and one epilogue for every kernel. With groups, the G copies of a
  // slice are added on the way and their waves share its rows.
  constexpr int SLOT = 32 * SPITCH;
  float* const stg = reinterpret_cast<float*>(smem + wave * SLOT);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(stg + lrow * (SPITCH / 4) + j * 32 + 8 * g + 4 * lhalf) =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                        acc[i][j][4 * g + 3]);
    const int64_t mr = m0 + wm0 + 32 * i, nc = n0 + wn0;
    float* const mine = part ? part + int64_t(blockIdx.y) * M * N : nullptr;
    if constexpr (G == 1) {
      __builtin_amdgcn_wave_barrier();
      if (part)
        store_part<WN / 8>(stg, SPITCH / 4, lane, mr, nc, M, N, mine);
      else
        finish_rows<WN / 8, WN == 32 ? 2 : WN == 96 ? 3 : 4>(stg, SPITCH / 4, lane, mr, nc, M, N, ep);
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();
      const float* const all = reinterpret_cast<const float*>(smem + wv * SLOT);
      constexpr int LPR = WN / 8;
      for (int q = lane + 64 * grp; q < 32 * LPR; q += 64 * G) {
        const int r = q / LPR, c = 8 * (q - r * LPR);
        float v[8] = {};
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float a[8];
          load8(all + g * (NW * SLOT / 4) + r * (SPITCH / 4) + c, a);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += a[e];
        }
        const int64_t m = mr + r, n = nc + c;
        if (m >= M || n >= N) continue;
        if (mine) store8(mine + m * N + n, v);
        else finish_piece(v, m, n, N, ep);
      }
      __syncthreads();
    }
  }
}

// ---- large bf16 products --------------------------------------------------------
//
// 256 x (64 NP) tile, eight waves of 64 x (32 NP) (4 x 2), 128 bytes of K per
// stage, two stage buffers. Waves w and w + 4 share a SIMD; the second half of
// the block runs one barrier interval behind the first, so on every SIMD one
// wave reads LDS and issues stage loads while the other's MFMAs run (and has
// priority for them). A k-step is NP phases, one 32-column strip of B each:
//   L_p  issue this phase's stage loads, read strip p of B and a share of the
//        next k-step's A (into the register set that the MFMAs do not use),
//        wait, barrier
//   M_p  16 MFMAs (64 rows x 32 columns x 64 k), barrier
// The L parts are kept even (2 or 3 loads, 6 or 8 fragment reads), since an
// interval lasts as long as the longer of the two halves' parts.
// A piece of a buffer is refilled once its last reader has passed a barrier:
// strip p of stage kt + 2 in phase p + 1 (the last strip in the next k-step's
// first phase); A of stage kt + 1 is read during k-step kt, its first 32-row half
// in phases 0 and 1 (then refilled with stage kt + 3), its second half after
// that (refilled in the next k-step's phases 0 and 1). The waits count the
// newer loads (they retire in order), the same sequence in every k-step;
// stages past the end are issued against an empty descriptor and move nothing.
// Bound by the MFMAs under the chip's power limit: 8192 x 4096 -> 4096 with GELU
// 201 us, 1.37 PFLOP/s, in a long run (241 us in the first thirty calls after idle);
// 8192 x 4608 -> 1152 gated 86 us (95), 1.0 PFLOP/s, as its 192 tiles leave a quarter
// of the CUs idle.
// LDS rows and their swizzle are those of linear_tile_kernel; the rows of A
// are stored half by half (rows 64 r + 32 i + .. of half i together), those of
// B strip by strip, so that each piece is one contiguous range.

// The MFMA is v_mfma_f32_16x16x32_bf16: under the chip's power limit, with every
// CU busy, it sustains 1.87 PFLOP/s on random operands against 1.61 for 32x32x16
// (registers only), and square4k-sized products run into that limit. A
// fragment is 16 rows of 32 k: lane l holds chunk l / 16 + 4 s of row l % 16;
// fragment 2 rb + s of a 32-row piece is row block rb, k half s. The weight
// fragment is the first operand: lane l's accumulator r belongs to row l % 16
// and column 4 (l / 16) + r of its 16 x 16 block.

// Fragments of a piece from the addresses p of its k halves (OFF: the piece; the
// second row block is 2048 bytes on), all four or a strip of B's four and one
// row block of A's or all of them, and the wait for all of them.
template <int OFF>
__device__ __forceinline__ void lds_frag4(v4i (&f)[4], const uint32_t (&p)[2]) {
  asm volatile(
      "ds_read_b128 %0, %4 offset:%6\n ds_read_b128 %1, %5 offset:%6\n"
      "ds_read_b128 %2, %4 offset:%7\n ds_read_b128 %3, %5 offset:%7\n s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
      : "v"(p[0]), "v"(p[1]), "n"(OFF), "n"(OFF + 2048)
      : "memory");
}
template <int OFFB, int OFFA>
__device__ __forceinline__ void lds_frag6(v4i (&f)[4], const uint32_t (&p)[2], v4i& g0, v4i& g1,
                                          const uint32_t (&q)[2]) {
  asm volatile(
      "ds_read_b128 %0, %6 offset:%10\n ds_read_b128 %1, %7 offset:%10\n"
      "ds_read_b128 %2, %6 offset:%11\n ds_read_b128 %3, %7 offset:%11\n"
      "ds_read_b128 %4, %8 offset:%12\n ds_read_b128 %5, %9 offset:%12\n s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(g0), "=&v"(g1)
      : "v"(p[0]), "v"(p[1]), "v"(q[0]), "v"(q[1]), "n"(OFFB), "n"(OFFB + 2048), "n"(OFFA)
      : "memory");
}
template <int OFFB, int OFFA>
__device__ __forceinline__ void lds_frag8(v4i (&f)[4], const uint32_t (&p)[2], v4i (&g)[4],
                                          const uint32_t (&q)[2]) {
  asm volatile(
      "ds_read_b128 %0, %8 offset:%12\n ds_read_b128 %1, %9 offset:%12\n"
      "ds_read_b128 %2, %8 offset:%13\n ds_read_b128 %3, %9 offset:%13\n"
      "ds_read_b128 %4, %10 offset:%14\n ds_read_b128 %5, %11 offset:%14\n"
      "ds_read_b128 %6, %10 offset:%15\n ds_read_b128 %7, %11 offset:%15\n s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(g[0]), "=&v"(g[1]), "=&v"(g[2]),
        "=&v"(g[3])
      : "v"(p[0]), "v"(p[1]), "v"(q[0]), "v"(q[1]), "n"(OFFB), "n"(OFFB + 2048), "n"(OFFA),
        "n"(OFFA + 2048)
      : "memory");
}

// Loads that may still be in flight when phase p ends, for what phase p + 1
// reads to have landed. Issue order of a k-step (u: unit of a half of A):
//   NP = 4: B3 A1u0 | B0 A1u1 | B1 A0u0 | B2 A0u1     (8 loads)
//   NP = 3: B2 A1u0 | B0 A1u1 | B1 A0u0 A0u1          (7 loads)
// Next phase 0 reads A half 0, last issued two k-steps back (one k-step newer);
// phase 1 reads B1, phase 2 (NP = 3: the last) A half 1, phase 3 B3.
template <int NP>
constexpr int pp_wait(int p) {
  if (NP == 4) return p == 0 || p == 2 ? 13 : 8;
  return p == 0 ? 11 : 7;
}

template <int NP>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void linear_pp_kernel(
    const uint16_t* __restrict__ X, int64_t M, const uint16_t* __restrict__ W, int64_t N, int K,
    LinEpi ep) {
  static_assert(NP == 3 || NP == 4, "waits are counted for 3 and 4 strips");
  constexpr int BM = 256, WN = 32 * NP, BN = 2 * WN;
  constexpr int ASZ = 128 * BM, STAGE = 65536;   // a power of two: buffers toggle by one xor
  constexpr int SPITCH = 4 * WN + 16;
  constexpr int LDSN = STAGE + ASZ + 128 * BN, LDSE = 8 * 32 * SPITCH;
  constexpr int LDSB = LDSN > LDSE ? LDSN : LDSE;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDSB];

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  int64_t m0, n0;
  f6_tile_origin<BM, BN, 4>(int(blockIdx.x), M, N, &m0, &n0);
  const int wm = wv >> 1, wn = wv & 1;
  const int ldb = 2 * K;
  const int KT = (ldb + 127) / 128;
  const int64_t rows_a = (M - m0) < BM ? (M - m0) : BM;
  const int64_t rows_b = (N - n0) < BN ? (N - n0) : BN;
  const uint8_t* const abase = reinterpret_cast<const uint8_t*>(X) + m0 * ldb;
  const uint8_t* const bbase = reinterpret_cast<const uint8_t*>(W) + n0 * ldb;
  const int nrec_a = int(rows_a * ldb), nrec_b = int(rows_b * ldb);

  const int chunk = (lane & 7) ^ (((wv & 1) * 4 + (lane >> 4)) & 7);
  const uint32_t sub = uint32_t((wv & 3) * 8 + (lane >> 3));
  const uint32_t va = (uint32_t(wv >> 2) * 64 + sub) * uint32_t(ldb) + 16 * chunk;
  const uint32_t vb = (uint32_t(wv >> 2) * WN + sub) * uint32_t(ldb) + 16 * chunk;
  // One unit of a half of A / the wave's unit of a strip of B. FAST: a whole
  // stage inside K (the row in the vector offset, so that rows past the end
  // stay out of range, the stage in the scalar one); otherwise stages past K
  // take an empty descriptor and chunks past K an offset out of range.
  auto issue = [&](auto fastc, const uint8_t* base, int nrec, uint32_t v, int row, int kt, int lds) {
    const int kb = kt * 128;
    uint8_t* const dst = smem + (kt & 1) * STAGE + lds + wv * 1024;
    if constexpr (decltype(fastc)::value) {
      lds_dma16_buf(make_rsrc(base, nrec), v + uint32_t(row * ldb), uint32_t(kb), dst);
    } else {
      const bool in = kb + 16 * chunk < ldb;
      lds_dma16_buf(make_rsrc(base, kt < KT ? nrec : 0), in ? v + uint32_t(row * ldb + kb) : 0x80000000u,
                    0u, dst);
    }
  };
  auto issue_a = [&](auto fastc, int i, int q, int kt) {
    issue(fastc, abase, nrec_a, va, q * 128 + i * 32, kt, i * (ASZ / 2) + q * 8192);
  };
  auto issue_b = [&](auto fastc, int j, int kt) {
    issue(fastc, bbase, nrec_b, vb, 32 * j, kt, ASZ + j * 8192);
  };
  constexpr std::false_type slow{};
  constexpr std::true_type fast{};

  const int lrow = lane & 15, lquad = lane >> 4;
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(smem));
  uint32_t pa[2], pb[2];   // k half s of the wave's first rows in this stage's buffer
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint32_t co = lds0 + uint32_t(((lquad + 4 * s) ^ (lrow >> 1)) * 16);
    pa[s] = co + uint32_t((wm * 32 + lrow) * 128);
    pb[s] = co + uint32_t((wn * 32 + lrow) * 128);
  }

  // accumulators of 16 x 16 block (row block i, column block j), from the bias
  v4f acc[4][2 * NP];
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j) {
    const int64_t n = n0 + wn * WN + 16 * j + 4 * lquad;
    const v4f b = ep.bias && n < N ? *reinterpret_cast<const v4f*>(ep.bias + n) : v4f{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][j] = b;
  }
  v4i af[2][2][4], bf[4];

  // the order of steady k-steps -3, -2 and -1
  issue_a(slow, 0, 0, 0);
  issue_a(slow, 0, 1, 0);
  issue_a(slow, 1, 0, 0);
  issue_b(slow, 0, 0);
  issue_a(slow, 1, 1, 0);
  issue_b(slow, 1, 0);
  issue_a(slow, 0, 0, 1);
  if constexpr (NP == 4) issue_b(slow, 2, 0);
  issue_a(slow, 0, 1, 1);
  issue_b(slow, NP - 1, 0);
  issue_a(slow, 1, 0, 1);
  issue_b(slow, 0, 1);
  issue_a(slow, 1, 1, 1);
  wait_vm_lgkm0<NP + 4>();   // all of A of stage 0
  __builtin_amdgcn_s_barrier();
  lds_frag4<0>(af[0][0], pa);
  lds_frag4<ASZ / 2>(af[0][1], pa);
  __builtin_amdgcn_s_barrier();
  issue_b(slow, 1, 1);
  issue_a(slow, 0, 0, 2);
  if constexpr (NP == 4) issue_b(slow, 2, 1);
  issue_a(slow, 0, 1, 2);
  wait_vm_lgkm0<pp_wait<NP>(NP - 1)>();
  __builtin_amdgcn_s_barrier();
  if (wv >= 4) __builtin_amdgcn_s_barrier();

  auto phase = [&](auto pc, auto setc, auto fc, int kt) {
    constexpr int P = decltype(pc)::value, SET = decltype(setc)::value;
    if constexpr (P == 0) issue_b(fc, NP - 1, kt + 1);
    else issue_b(fc, P - 1, kt + 2);
    if constexpr (P < 2) issue_a(fc, 1, P, kt + 2);
    if constexpr (P == 2) issue_a(fc, 0, 0, kt + 3);
    if constexpr (P == NP - 1) issue_a(fc, 0, 1, kt + 3);
    // pa, pb: this stage's buffer
    const uint32_t pn[2] = {pa[0] ^ STAGE, pa[1] ^ STAGE};
    if constexpr (NP == 3 && P == 2) {
      lds_frag8<ASZ + P * 8192, ASZ / 2>(bf, pb, af[1 - SET][1], pn);
    } else {
      constexpr int I = P / 2, RB = P % 2;
      lds_frag6<ASZ + P * 8192, I * (ASZ / 2) + RB * 2048>(bf, pb, af[1 - SET][I][2 * RB],
                                                           af[1 - SET][I][2 * RB + 1], pn);
    }
    if constexpr (P == NP - 1) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        pa[s] ^= STAGE;
        pb[s] ^= STAGE;
      }
    }
    wait_vm_lgkm0<pp_wait<NP>(P)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][2 * P + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(v8bf, bf[2 * j + s]),
              __builtin_bit_cast(v8bf, af[SET][i / 2][2 * (i % 2) + s]), acc[i][2 * P + j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
  };
  auto kstep = [&](auto setc, auto fc, int kt) {
    phase(std::integral_constant<int, 0>{}, setc, fc, kt);
    phase(std::integral_constant<int, 1>{}, setc, fc, kt);
    phase(std::integral_constant<int, 2>{}, setc, fc, kt);
    if constexpr (NP == 4) phase(std::integral_constant<int, 3>{}, setc, fc, kt);
  };
  constexpr std::integral_constant<int, 0> set0{};
  constexpr std::integral_constant<int, 1> set1{};
  const int KF = ldb / 128;      // stages of whole chunks
  int kt = 0;
  for (; kt + 4 < KF; kt += 2) {
    kstep(set0, fast, kt);
    kstep(set1, fast, kt + 1);
  }
  for (; kt + 1 < KT; kt += 2) {
    kstep(set0, slow, kt);
    kstep(set1, slow, kt + 1);
  }
  if (kt < KT) kstep(set0, slow, kt);
  if (wv < 4) __builtin_amdgcn_s_barrier();
  wait_vm_lgkm0<0>();
  __builtin_amdgcn_s_barrier();

  float* const stg = reinterpret_cast<float*>(smem + wv * 32 * SPITCH);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int j = 0; j < 2 * NP; ++j)
        *reinterpret_cast<v4f*>(stg + (16 * rb + lrow) * (SPITCH / 4) + 16 * j + 4 * lquad) =
            acc[2 * i + rb][j];
    __builtin_amdgcn_wave_barrier();
    finish_rows<WN / 8, NP == 4 ? 4 : 3>(stg, SPITCH / 4, lane, m0 + wm * 64 + 32 * i, n0 + wn * WN, M,
                                         N, ep);
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- a few rows -----------------------------------------------------------------
//
// Tiles of 16 x 16 outputs for products of few tiles: the eight waves of a block
// take the k-steps (128 bytes of a row) in turn, fragments go from memory straight
// into registers, U k-steps in flight, no barrier until the waves' sums meet in LDS,
// in wave order. Lane l holds bytes 32 (l / 16) .. + 31 of row l % 16 (bf16: two chunks
// for two v_mfma_f32_16x16x32_bf16; fp32: the eight values of one split), the same k
// for both operands. Rows past the end repeat the last one and are not stored; chunks
// past K are zeros. Bound by latency (16 x 256 -> 1152 bf16: 2.9 us) or by what each
// block reads, its 16 rows of X and of W: many tiles with a long K take wider ones.
template <typename TE>
__global__ __launch_bounds__(512) void linear_few_kernel(const TE* __restrict__ X, int64_t M,
                                                         const TE* __restrict__ W, int64_t N, int K,
                                                         LinEpi ep) {
  constexpr int NW = 8, U = 4, PITCH = 20, SLOT = 16 * PITCH;
  __shared__ __attribute__((aligned(16))) float smem[NW * SLOT];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int lrow = lane & 15, q = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * 16, m0 = int64_t(blockIdx.y) * 16;
  const int ldb = K * int(sizeof(TE)), KT = (ldb + 127) / 128;
  const int64_t ma = m0 + lrow < M ? m0 + lrow : M - 1, nb = n0 + lrow < N ? n0 + lrow : N - 1;
  const uint8_t* const px = reinterpret_cast<const uint8_t*>(X) + ma * ldb;
  const uint8_t* const pw = reinterpret_cast<const uint8_t*>(W) + nb * ldb;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = wv; s0 < KT; s0 += NW * U) {
    v4i x[U][2], w[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {   // both chunks of an operand in a row: they share its lines
      const int o = (s0 + NW * u) * 128 + 32 * q;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        x[u][c] = o + 16 * c < ldb ? *reinterpret_cast<const v4i*>(px + o + 16 * c) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 2; ++c)
        w[u][c] = o + 16 * c < ldb ? *reinterpret_cast<const v4i*>(pw + o + 16 * c) : v4i{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + NW * u >= KT) break;
#define HL_FEW(W_, X_) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(W_, X_, acc, 0, 0, 0)
      if constexpr (sizeof(TE) == 2) {
        HL_FEW(__builtin_bit_cast(v8bf, w[u][0]), __builtin_bit_cast(v8bf, x[u][0]));
        HL_FEW(__builtin_bit_cast(v8bf, w[u][1]), __builtin_bit_cast(v8bf, x[u][1]));
      } else {
        const Split a = split8(x[u][0], x[u][1]), b = split8(w[u][0], w[u][1]);
        HL_FEW(b.l, a.h);
        HL_FEW(b.m, a.m);
        HL_FEW(b.h, a.l);
        HL_FEW(b.m, a.h);
        HL_FEW(b.h, a.m);
        HL_FEW(b.h, a.h);
      }
#undef HL_FEW
    }
  }
  *reinterpret_cast<v4f*>(smem + wv * SLOT + lrow * PITCH + 4 * q) = acc;
  __syncthreads();
  const int r = int(threadIdx.x) / 2, c = 8 * (int(threadIdx.x) % 2);
  const int64_t m = m0 + r, n = n0 + c;
  if (r >= 16 || m >= M || n >= N) return;
  float v[8] = {}, b[8] = {};
  if (ep.bias) load8(ep.bias + n, b);
#pragma unroll
  for (int g = 0; g < NW; ++g) {
    float a[8];
    load8(smem + g * SLOT + r * PITCH + c, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += a[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += b[e];
  finish_piece(v, m, n, N, ep);
}

// Y from the splits' partial sums [splits, M, N], added in split order; one
// lane per 8 columns. Bound by reading the partial sums (L2 / Infinity Cache).
__global__ __launch_bounds__(256) void linear_reduce_kernel(const float* __restrict__ part,
                                                            int splits, int64_t M, int64_t N,
                                                            LinEpi ep) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t npr = N / 8;
  if (i >= M * npr) return;
  const int64_t m = i / npr, n = (i - m * npr) * 8;
  const float* p = part + m * N + n;
  float v[8] = {}, b[8] = {};
  if (ep.bias) load8(ep.bias + n, b);
  for (int s = 0; s < splits; ++s) {
    float a[8];
    load8(p + int64_t(s) * M * N, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += a[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += b[e];
  finish_piece(v, m, n, N, ep);
}

// ---- host side --------------------------------------------------------------------

// Kernel and split count of a product.
//  up to 4 rows: the vector kernel (4096 -> 16384 bf16: 25 us at one row, 30 at four;
//    at eight it would take 43).
//  16 x 16 tiles, waves sharing the k-steps, up to one tile per CU and 48 k-steps (16 x
//    1152 -> 1152 bf16: 4.4 us against 5.6 for 32 x 64 tiles, fp32 6.7 against 9.2;
//    912 x 576 -> 24 fp32: 4.7 against 8.6; at 72 k-steps 10.6 against 8.9), up to two
//    per CU and 24 k-steps in fp32 (64 x 768 -> 1152: 8.2 us against 9.3, at 36 the other
//    way, 10.8 against 9.9) or 4 in bf16 (8 x 1152 -> 4608 still 5.8 against 6.0 at 18,
//    as half the rows are not there; 64 x 768 -> 1152 the other way, 5.0 against 4.8),
//    and for 3 or 4 bf16 rows of many outputs (4 x 4096 -> 16384: 26.1 us against 30.1
//    for the vector kernel).
//  bf16:
//    More than 128 tiles of 256 x 192: the wide tiles, 192 or 256 columns, whichever's
//    rounds of one tile per CU cost less; except that 128 x 128 tiles of eight waves,
//    two blocks per CU, take up to 32 k-steps where all of them run at once (12288 x
//    512 -> 512: 14.3 us against 18.5; 6000 x 1000 -> 1000: 23.9 against 26.3; 6000 x
//    4096 -> 1024, 64 k-steps: no better, 60.8 against 61.5).
//    Otherwise the tile shrinks until there is about one per CU:
//    more than one 128 x 128 per CU: 128 x 192 with two groups of waves on a tile's
//    k-steps (1024 x 4608 -> 4608: 52 us against 67 for 256 x 192 and 59 for 128 x
//    128; 4096 x 4608 -> 1152: 53 against 66 and 59);
//    more than one for two CUs: 128 x 128, eight waves and three stages (1037 x 1160
//    -> 2312: 17.2 us against 19.6 for 64 x 128; 367 x 3808 -> 6896: 33.7 against 64),
//    or two groups of four where most CUs have one and K is long (1024 x 4096 -> 4096:
//    40.0 us against 42.6);
//    more 64 x 64 than CUs: 64 x 128 with two groups of eight waves (512 x 4096 ->
//    4096: 24.5 us against 30.7 for one group of four, 1024 x 1152 -> 1152: 9.4 against
//    10.0 for 64 x 64);
//    fewer: 64 x 64 with two groups (512 x 4096 -> 1152: 15.3 us against 15.7 for one
//    group split in three over blocks; 256 x 4096 -> 4096: 15.8 us against 20.2 for 64
//    x 128), and 32 x 64 tiles where those are no more than the CUs (300 x 1152 ->
//    1152: 6.2 us against 6.7), with four groups from 32 k-steps on where a split would
//    not leave each block as many (300 x 4096 -> 1152: 11.9 us against 13.6 with two;
//    77 x 2048 -> 1280: 7.6 against 8.3 with two and a split; 128 x 4096 -> 1152, 72
//    tiles, the other way, 10.9 against 10.4).
//    What still leaves CUs idle is split over K, at 16 k-steps a block or more (64
//    x 4096 -> 4096: 11.9 us in two against 13.2 whole and 12.7 in four; 32 x 1152
//    -> 4608: 5.6 us whole against 7.3): a split costs a second launch and the
//    partial sums.
//  fp32 computes six times as much per byte and pays for its fragments' splits by
//  the rows and columns of a wave:
//    128 x 128 tiles for more than 64 rows and outputs (6724 x 2344 -> 64: 41 us, with
//    64 x 64 in four 26) where they, split over K at 12 k-steps a block or more, come
//    to 200 blocks (512 x 4096 -> 1152: 42 us in six against 46 for 64 x 64 in three;
//    2048 x 1152 -> 1152: 45.6 us in three against 50.5; 1024 x 4096 -> 4096: 188 us
//    in two against 200 whole and 236 for 64 x 64);
//    32 x 64 tiles for one tile row or up to 128 of them (9 x 4096 -> 4096: 18.4 us
//    against 22.1), split at 12 k-steps (16 x 1152 -> 4608: 10.0 us in three against
//    11.2 in four) into two blocks per CU, or one for a single tile row, which
//    streams W (16 x 8192 -> 4096: 34 us in four against 45 in eight; 128 x 4096 ->
//    1152 the other way, 19.1 in six against 21 in four), or where K is too short to
//    split (2048 x 256 -> 256: 6.2 us against 7.2);
//    64 x 64 tiles otherwise: with two groups of waves, split at 12 k-steps (300 x
//    4096 -> 1152: 33 us in five against 36 in six; 64 x 1152 -> 4608: 14.0 us in
//    three against 20 whole), where they are half the CUs at 40 (8192 x 1152 -> 128,
//    256 tiles: 21.4 us whole against 25.6 in two), or more than 512 of them with one group and a third
//    block per CU (4096 x 640 -> 640: 31.9 us against 33.6).
LinPlan linear_plan(int64_t M, int64_t N, int K, int esize) {
  LinPlan p = {LIN_ROWS, 1, (K * esize + 127) / 128};
  const bool bf16 = esize == 2;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  const int64_t t16 = tiles(16, 16);
  const int most = M <= 4 ? 8 : M <= 8 ? 64 : 48;   // k-steps, where every tile has a CU
  const bool few = (t16 <= 256 && p.kper <= most) ||
                   (t16 <= 512 && p.kper <= (!bf16 ? 24 : M <= 4 ? 8 : M <= 8 ? 18 : 4)) ||
                   (M <= 4 && N >= 4096);
  if (few && M > (bf16 ? 2 : 4)) {
    p.kind = LIN_FEW;
    return p;
  }
  if (M <= 4) return p;
  const int64_t t = tiles(64, 64), t32 = tiles(32, 64), t128 = tiles(128, 128);
  const int ksteps = p.kper;
  if (bf16 && t128 > 256 && t128 <= 512 && ksteps <= 32) {
    p.kind = LIN_T128W8;
    return p;
  }
  if (bf16 && tiles(256, 192) > 128) {
    const int64_t r3 = (tiles(256, 192) + 255) / 256 * 3, r4 = (tiles(256, 256) + 255) / 256 * 4;
    p.kind = r3 < r4 ? LIN_PP3 : LIN_PP4;
    return p;
  }
  // splits of n tiles: `blocks` in all, `least` k-steps each, at most `most`
  auto split = [&](int64_t blocks, int64_t n, int least, int64_t most) {
    return std::max<int64_t>(1, std::min({blocks / n, int64_t(ksteps / least), most}));
  };
  const int64_t split128 = split(512, t128, 12, 6);
  int64_t want = 1;
  if (bf16 && t128 > 128) {
    p.kind = t128 > 256 ? LIN_T128X192 : t128 > 192 && ksteps >= 48 ? LIN_T128X2 : LIN_T128;
  } else if (bf16 && t32 > 256) {
    p.kind = t > 256 ? LIN_T64X128 : LIN_T64X2;
  } else if (bf16) {
    const bool four = ksteps >= 32 && split(256, t32, 32, 4) == 1;
    p.kind = four ? LIN_T32X4 : LIN_T32;
    want = four ? 1 : split(256, t32, 16, 4);
  } else if (M > 64 && N > 64 && t128 * split128 >= 200) {
    p.kind = LIN_T128;
    want = split128;
  } else if (M <= 32 || t32 <= 128 || (t32 <= 256 && ksteps < 24)) {
    p.kind = LIN_T32;
    want = split(M <= 32 ? 256 : 512, t32, 12, 8);
  } else if (t <= 512) {
    p.kind = LIN_T64X2;
    want = split(512, t, t > 128 ? 40 : 12, 8);
  } else {
    p.kind = LIN_T64;
  }
  if (want > 1) {
    p.kper = int((ksteps + want - 1) / want);
    p.splits = (ksteps + p.kper - 1) / p.kper;
  }
  return p;
}

namespace {

template <typename TE, int TT>
void launch_rows_nc(const TE* X, int M, const TE* W, int64_t N, int K, const LinEpi& ep,
                    hipStream_t s) {
  // columns per wave: more reuse of X per load of W where there are waves enough (3
  // and 4 bf16 rows of as many outputs take linear_few_kernel)
  if constexpr (sizeof(TE) == 4 || TT <= 2) {
    if (N >= 4096) {
      hipLaunchKernelGGL((linear_rows_kernel<TE, TT, 2>), dim3(unsigned((N + 7) / 8)), dim3(256), 0,
                         s, X, M, W, N, K, ep);
      return;
    }
  }
  hipLaunchKernelGGL((linear_rows_kernel<TE, TT, 1>), dim3(unsigned((N + 3) / 4)), dim3(256), 0, s,
                     X, M, W, N, K, ep);
}

template <typename TE, int BM, int BN, int WM, int WN, int G, int S, int OCC>
void launch_tile(const TE* X, int64_t M, const TE* W, int64_t N, int K, const LinPlan& p,
                 float* part, const LinEpi& ep, hipStream_t s) {
  const int64_t ntiles = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  hipLaunchKernelGGL((linear_tile_kernel<TE, BM, BN, WM, WN, G, S, OCC>),
                     dim3(unsigned(ntiles), unsigned(p.splits)),
                     dim3((BM / WM) * (BN / WN) * 64 * G), 0, s, X, M, W, N, K, p.kper,
                     p.splits > 1 ? part : nullptr, ep);
}

template <typename TE>
hipError_t launch_typed(const TE* X, int64_t M, const TE* W, int64_t N, int K, float* part,
                        const LinEpi& ep, hipStream_t s) {
  const LinPlan p = linear_plan(M, N, K, int(sizeof(TE)));
  switch (p.kind) {
    case LIN_ROWS:
      if (M == 1) launch_rows_nc<TE, 1>(X, int(M), W, N, K, ep, s);
      else if (M == 2) launch_rows_nc<TE, 2>(X, int(M), W, N, K, ep, s);
      else launch_rows_nc<TE, 4>(X, int(M), W, N, K, ep, s);
      break;
    case LIN_FEW:
      hipLaunchKernelGGL((linear_few_kernel<TE>), dim3(unsigned((N + 15) / 16), unsigned((M + 15) / 16)),
                         dim3(512), 0, s, X, M, W, N, K, ep);
      break;
    case LIN_PP3:
    case LIN_PP4:
      if constexpr (sizeof(TE) == 2) {
        const int bn = p.kind == LIN_PP3 ? 192 : 256;
        const dim3 grid(unsigned(((M + 255) / 256) * ((N + bn - 1) / bn)));
        if (p.kind == LIN_PP3)
          hipLaunchKernelGGL(linear_pp_kernel<3>, grid, dim3(512), 0, s, X, M, W, N, K, ep);
        else
          hipLaunchKernelGGL(linear_pp_kernel<4>, grid, dim3(512), 0, s, X, M, W, N, K, ep);
      }
      break;
    case LIN_T32: launch_tile<TE, 32, 64, 32, 32, 2, 3, 2>(X, M, W, N, K, p, part, ep, s); break;
    case LIN_T32X4:
      if constexpr (sizeof(TE) == 2)
        launch_tile<TE, 32, 64, 32, 32, 4, 3, 1>(X, M, W, N, K, p, part, ep, s);
      break;
    case LIN_T64X2:
      if constexpr (sizeof(TE) == 2)
        launch_tile<TE, 64, 64, 32, 32, 2, 3, 1>(X, M, W, N, K, p, part, ep, s);
      else
        launch_tile<TE, 64, 64, 32, 32, 2, 2, 2>(X, M, W, N, K, p, part, ep, s);
      break;
    case LIN_T64:
      if constexpr (sizeof(TE) == 4)
        launch_tile<TE, 64, 64, 32, 32, 1, 3, 2>(X, M, W, N, K, p, part, ep, s);
      break;
    case LIN_T64X128:
      if constexpr (sizeof(TE) == 2)
        launch_tile<TE, 64, 128, 32, 32, 2, 3, 1>(X, M, W, N, K, p, part, ep, s);
      break;
    case LIN_T128:
      if constexpr (sizeof(TE) == 2)
        launch_tile<TE, 128, 128, 64, 32, 1, 3, 1>(X, M, W, N, K, p, part, ep, s);
      else
        launch_tile<TE, 128, 128, 64, 64, 1, 2, 2>(X, M, W, N, K, p, part, ep, s);
      break;
    case LIN_T128X2:
      if constexpr (sizeof(TE) == 2)
        launch_tile<TE, 128, 128, 64, 64, 2, 2, 2>(X, M, W, N, K, p, part, ep, s);
      break;
    case LIN_T128W8:
      if constexpr (sizeof(TE) == 2)
        launch_tile<TE, 128, 128, 64, 32, 1, 2, 2>(X, M, W, N, K, p, part, ep, s);
      break;
    case LIN_T128X192:
      if constexpr (sizeof(TE) == 2)
        launch_tile<TE, 128, 192, 64, 96, 2, 2, 2>(X, M, W, N, K, p, part, ep, s);
      break;
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.splits > 1) {
    const int64_t n8 = M * (N / 8);
    hipLaunchKernelGGL(linear_reduce_kernel, dim3(unsigned((n8 + 255) / 256)), dim3(256), 0, s,
                       part, p.splits, M, N, ep);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

size_t linear_part_bytes(int64_t M, int64_t N, int K, int esize) {
  const LinPlan p = linear_plan(M, N, K, esize);
  return p.splits > 1 ? size_t(p.splits) * size_t(M) * size_t(N) * 4 : 0;
}

hipError_t launch_linear(const void* X, int bf16, int64_t M, const void* W, int64_t N, int K,
                         void* part, const LinEpi& ep, hipStream_t s) {
  if (M <= 0) return hipSuccess;
  if (bf16)
    return launch_typed(static_cast<const uint16_t*>(X), M, static_cast<const uint16_t*>(W), N, K,
                        static_cast<float*>(part), ep, s);
  return launch_typed(static_cast<const float*>(X), M, static_cast<const float*>(W), N, K,
                      static_cast<float*>(part), ep, s);
}

// GELU (bf16 results): degree-6 weighted least-maximum fit of -log2(Phi(x) / Phi(-x)) / x in
// x^2 on |x| <= 5; the other two are exact forms.
ActCoef act_coef(int act) {
  ActCoef a = {};
  a.act = act;
  constexpr float log2e = 1.4426950408889634f;
  if (act == ACT_SILU) {
    a.c[0] = -log2e;
  } else if (act == ACT_GELU_TANH) {
    a.c[0] = -1.5957691216057308f * log2e;
    a.c[1] = -1.5957691216057308f * 0.044715f * log2e;
  } else if (act == ACT_GELU) {
    a.tmax = 25.0f;
    const float c[7] = {-2.3017581959277815f,   -0.10552445421016707f,   0.0003938443860880515f,
                        0.0001041246928390452f, -6.513520962607899e-06f, 1.7551338906125295e-07f,
                        -1.842194984814521e-09f};
    for (int k = 0; k < 7; ++k) a.c[k] = c[k];
  }
  return a;
}

}  // namespace hq
