// Dense linear layer of libhq (the layers that stay in 16 or 32 bits beside
// the low-bit ones): Y = R + g phi(X W^T + b) with X [M, K], W [N, K] (the
// nn.Linear layout: both operands K-contiguous, no transposition anywhere) in
// bf16 or fp32, fp32 accumulation, and the epilogue of hq_epilogue.h.
//
// Three kernels, chosen by shape (linear_plan):
//  linear_rows_kernel  M <= 8: one pass over W on the vector ALU.
//  linear_tile_kernel  MFMA tiles; few tiles are split over K (partial sums
//                      in the workspace, added in split order by
//                      linear_reduce_kernel, which then runs the epilogue).
#include "hq_epilogue.h"
#include "hq_gemm6_kernel.h"
#include "hq_internal.h"

namespace hq {

// ---- few rows ------------------------------------------------------------------
//
// One wave owns NC output columns and all TT rows; its lanes split K in
// 16-byte (bf16) or 32-byte (fp32) pieces, U pieces of 512 elements loaded
// before the first is used. The wave's sums meet in a fixed lane tree. Bound
// by reading W once (N K elements); X is read by every wave from L2.
template <typename TE, int TT, int NC>
__global__ __launch_bounds__(256) void linear_rows_kernel(const TE* __restrict__ X, int M,
                                                          const TE* __restrict__ W, int64_t N,
                                                          int K, LinEpi ep) {
  constexpr int U = 4;
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
    float w[U][NC][8];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (kb + 512 * u < K) {
          load8(wp[c] + kb + 512 * u, w[u][c]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[u][c][e] = 0.0f;
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + 512 * u >= K) break;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        float x[8];
        load8(xp[t] + kb + 512 * u, x);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[t][c] = fmaf(x[e], w[u][c][e], acc[t][c]);
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
// 16-byte chunk 2 s + l / 32 of substep s. In bf16 a chunk is the 8
// consecutive k of one v_mfma_f32_32x32x16_bf16; in fp32 its 4 values enter
// four v_mfma_f32_32x32x2_f32, whose k pairs are (chunk 2s, chunk 2s + 1)
// value by value (the same map for both operands, so any pairing is the same
// sum). The weight fragment is the first operand: lane l's accumulator r
// belongs to row l % 32 and column 8 (r / 4) + 4 (l / 32) + r % 4.
template <typename TE>
__device__ __forceinline__ v16f lin_mfma(const v4i& w, const v4i& x, v16f c) {
  if constexpr (sizeof(TE) == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w),
                                                   __builtin_bit_cast(v8bf, x), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__int_as_float(w[e]), __int_as_float(x[e]), c, 0, 0, 0);
    return c;
  }
}

// LDS fragment reads as inline asm that waits for its own results: written as
// ordinary loads, the compiler would wait for every stage load in flight (it
// cannot tell that they fill other buffers).
__device__ __forceinline__ void lds_read2(v4i& a, v4i& b, uint32_t pa, uint32_t pb) {
  asm volatile("ds_read_b128 %0, %2\n ds_read_b128 %1, %3\n s_waitcnt lgkmcnt(0)"
               : "=&v"(a), "=&v"(b)
               : "v"(pa), "v"(pb)
               : "memory");
}
__device__ __forceinline__ void lds_read4(v4i& a, v4i& b, v4i& c, v4i& d, uint32_t pa, uint32_t pb) {
  asm volatile(
      "ds_read_b128 %0, %4\n ds_read_b128 %1, %4 offset:4096\n"
      "ds_read_b128 %2, %5\n ds_read_b128 %3, %5 offset:4096\n s_waitcnt lgkmcnt(0)"
      : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
      : "v"(pa), "v"(pb)
      : "memory");
}

// BM x BN tile, waves of WM x WN (32 x 32 or 64 x 64), S stage buffers of 128
// bytes per row (64 bf16 or 32 fp32 values of K), filled by buffer loads
// straight into LDS, S - 1 stages ahead. Rows past M or N and chunks past K
// lie outside the tile's buffer descriptor: they arrive as zeros and move no
// memory, so any M, N and any K of whole chunks takes the same loop. Chunk c
// of row r sits in slot c ^ ((r / 2) mod 8): the 16 lanes of one read phase
// hit 16 distinct 16-byte positions of the 64 banks.
// blockIdx.y is the split: k-steps [kper y, kper (y + 1)); with more than one
// split the raw sums go to part [splits, M, N].
template <typename TE, int BM, int BN, int WM, int WN, int S, int OCC>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64)
__attribute__((amdgpu_waves_per_eu(OCC))) void linear_tile_kernel(
    const TE* __restrict__ X, int64_t M, const TE* __restrict__ W, int64_t N, int K, int kper,
    float* __restrict__ part, LinEpi ep) {
  constexpr int NW = (BM / WM) * (BN / WN), WAVES_N = BN / WN;
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW, L = LA + LB;
  constexpr int STAGE = 128 * (BM + BN);
  constexpr int SPITCH = 4 * WN + 16;            // staging row: WN floats and one 16-byte pad
  static_assert(LA * NW * 8 == BM && LB * NW * 8 == BN && NW % 2 == 0, "whole 1-KB units per wave");
  static_assert(TM == TN && (TM == 1 || TM == 2), "32 x 32 or 64 x 64 waves");
  static_assert(NW * 32 * SPITCH <= S * STAGE, "epilogue staging fits in the stage buffers");
  static_assert((S - 1) * L <= 63, "outstanding loads fit vmcnt");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE];

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  int64_t m0, n0;
  f6_tile_origin<BM, BN, 8>(int(blockIdx.x), M, N, &m0, &n0);
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
    uint8_t* base_ = smem + (kt_ % S) * STAGE;                                               \
    const bool ok_ = kt_ < KT;                                                               \
    const int kb_ = (kt0 + kt_) * 128;                                                       \
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
  uint32_t co[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) co[s] = uint32_t(((2 * s + lhalf) ^ ((lrow >> 1) & 7)) * 16);
  const uint32_t arow = lds0 + uint32_t((wm0 + lrow) * 128);
  const uint32_t brow = lds0 + uint32_t((BM + wn0 + lrow) * 128);

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
      acc[i][j] = v16f{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  v4i af[2][TM], bf[2][TN];
#define HL_READ(SET_, BUF_, S_)                                                              \
  do {                                                                                       \
    const uint32_t o_ = uint32_t((BUF_) * STAGE) + co[S_];                                   \
    if constexpr (TM == 2)                                                                   \
      lds_read4(af[SET_][0], af[SET_][TM - 1], bf[SET_][0], bf[SET_][TN - 1], arow + o_, brow + o_); \
    else                                                                                     \
      lds_read2(af[SET_][0], bf[SET_][0], arow + o_, brow + o_);                             \
  } while (0)

#pragma unroll
  for (int p = 0; p < S - 1; ++p) HL_ISSUE(p);
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt has landed in every wave; every wave is done with stage kt - 1
    wait_vm_lgkm0<(S - 2) * L>();
    __builtin_amdgcn_s_barrier();
    HL_ISSUE(kt + S - 1);
    const int buf = kt % S;
    HL_READ(0, buf, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) HL_READ((s + 1) & 1, buf, s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = lin_mfma<TE>(bf[s & 1][j], af[s & 1][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#undef HL_READ
#undef HL_ISSUE
  wait_vm_lgkm0<0>();  // no LDS write may land in the staging area (or after the block ends)
  __builtin_amdgcn_s_barrier();

  // Each wave stages its 32-row slices in its own part of the LDS and takes
  // them back as rows, eight consecutive columns per lane: whole row segments
  // per store, and one epilogue for every kernel.
  float* const stg = reinterpret_cast<float*>(smem + wv * 32 * SPITCH);
  constexpr int LPR = WN / 8;                    // lanes per row
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(stg + lrow * (SPITCH / 4) + j * 32 + 8 * g + 4 * lhalf) =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                        acc[i][j][4 * g + 3]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < 32 * LPR / 64; ++q) {
      const int r = (lane + 64 * q) / LPR, c = 8 * ((lane + 64 * q) % LPR);
      const int64_t m = m0 + wm0 + 32 * i + r, n = n0 + wn0 + c;
      float v[8];
      load8(stg + r * (SPITCH / 4) + c, v);
      if (m < M && n < N) {
        if (part)
          store8(part + (int64_t(blockIdx.y) * M + m) * N + n, v);
        else
          finish8(v, m, n, N, ep);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- large bf16 products --------------------------------------------------------
//
// 256 x (64 NP) tile, eight waves of 64 x (32 NP) (4 x 2), 128 bytes of K per
// stage, two stage buffers. Waves w and w + 4 share a SIMD; the second half of
// the block runs one barrier interval behind the first, so on every SIMD one
// wave reads LDS and issues stage loads while the other's MFMAs run (and has
// priority for them). A k-step is NP phases, one 32-column strip of B each:
//   L_p  issue this phase's stage loads, read strip p of B (and in the last
//        two phases one half of the next k-step's A, which replaces the set
//        the MFMAs use by a second one), wait, barrier
//   M_p  8 MFMAs (64 rows x 32 columns x 64 k), barrier
// A piece of a buffer is refilled as soon as its last reader has passed a
// barrier: strip p of stage kt + 2 in phase p + 1 (the last strip in the first
// phase of the next k-step), the two 32-row halves of A in phases 0 and 1. Every load thus
// has 2 NP - 1 (B) or NP + 2 (A) phases to land; the waits count the newer
// loads (they retire in order), the same sequence in every k-step (stages past
// the end are issued against an empty descriptor and move nothing).
// LDS rows and their swizzle are those of linear_tile_kernel; the rows of A
// are stored half by half (rows 64 r + 32 i + .. of half i together), those of
// B strip by strip, so that each piece is one contiguous range.
template <int OFF>
__device__ __forceinline__ void lds_frag4(v4i (&f)[4], const uint32_t (&p)[4], uint32_t base) {
  asm volatile(
      "ds_read_b128 %0, %4 offset:%8\n ds_read_b128 %1, %5 offset:%8\n"
      "ds_read_b128 %2, %6 offset:%8\n ds_read_b128 %3, %7 offset:%8\n s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
      : "v"(p[0] + base), "v"(p[1] + base), "v"(p[2] + base), "v"(p[3] + base), "n"(OFF)
      : "memory");
}
template <int OFFA, int OFFB>
__device__ __forceinline__ void lds_frag8(v4i (&f)[4], const uint32_t (&p)[4], uint32_t base_a,
                                          v4i (&g)[4], const uint32_t (&q)[4], uint32_t base_b) {
  asm volatile(
      "ds_read_b128 %0, %8 offset:%16\n ds_read_b128 %1, %9 offset:%16\n"
      "ds_read_b128 %2, %10 offset:%16\n ds_read_b128 %3, %11 offset:%16\n"
      "ds_read_b128 %4, %12 offset:%17\n ds_read_b128 %5, %13 offset:%17\n"
      "ds_read_b128 %6, %14 offset:%17\n ds_read_b128 %7, %15 offset:%17\n s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(g[0]), "=&v"(g[1]), "=&v"(g[2]),
        "=&v"(g[3])
      : "v"(p[0] + base_a), "v"(p[1] + base_a), "v"(p[2] + base_a), "v"(p[3] + base_a),
        "v"(q[0] + base_b), "v"(q[1] + base_b), "v"(q[2] + base_b), "v"(q[3] + base_b),
        "n"(OFFA), "n"(OFFB)
      : "memory");
}

// Loads that may still be in flight when phase p ends, for what phase p + 1
// reads to have landed (1 per B strip, 2 per half of A; see the order above).
template <int NP>
constexpr int pp_wait(int p) {
  if (p == NP - 1) return 2 * NP + 4;      // strip 0 of the next k-step
  if (p == NP - 2) return NP == 4 ? 9 : 7;   // half 1 of the next A
  if (p == NP - 3) return NP == 4 ? 11 : 7;  // half 0 of the next A
  return 12;                               // NP = 4, p = 0: strip 1
}

template <int NP>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void linear_pp_kernel(
    const uint16_t* __restrict__ X, int64_t M, const uint16_t* __restrict__ W, int64_t N, int K,
    LinEpi ep) {
  static_assert(NP == 3 || NP == 4, "waits are counted for 3 and 4 strips");
  constexpr int BM = 256, WN = 32 * NP, BN = 2 * WN;
  constexpr int ASZ = 128 * BM, STAGE = ASZ + 128 * BN;
  constexpr int SPITCH = 4 * WN + 16;
  constexpr int LDSB = 2 * STAGE > 8 * 32 * SPITCH ? 2 * STAGE : 8 * 32 * SPITCH;
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
  auto issue_a = [&](int i, int kt) {
    const int kb = kt * 128;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(abase, kt < KT ? nrec_a : 0);
    const bool in = kb + 16 * chunk < ldb;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      lds_dma16_buf(r, in ? va + uint32_t((q * 128 + i * 32) * ldb + kb) : 0x80000000u, 0u,
                    smem + (kt & 1) * STAGE + i * (ASZ / 2) + (q * 8 + wv) * 1024);
  };
  auto issue_b = [&](int j, int kt) {
    const int kb = kt * 128;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(bbase, kt < KT ? nrec_b : 0);
    const bool in = kb + 16 * chunk < ldb;
    lds_dma16_buf(r, in ? vb + uint32_t(32 * j * ldb + kb) : 0x80000000u, 0u,
                  smem + (kt & 1) * STAGE + ASZ + j * 8192 + wv * 1024);
  };

  const int lrow = lane & 31, lhalf = lane >> 5;
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(smem));
  uint32_t pa[4], pb[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t co = lds0 + uint32_t(((2 * s + lhalf) ^ ((lrow >> 1) & 7)) * 16);
    pa[s] = co + uint32_t((wm * 32 + lrow) * 128);
    pb[s] = co + uint32_t((wn * 32 + lrow) * 128);
  }

  v16f acc[2][NP];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j)
      acc[i][j] = v16f{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  v4i af[2][2][4], bf[4];

  // the order of a steady k-step, from stage 0 on
  issue_a(0, 0);
  issue_b(0, 0);
  issue_a(1, 0);
#pragma unroll
  for (int j = 1; j < NP; ++j) issue_b(j, 0);
  issue_a(0, 1);
  issue_b(0, 1);
  issue_a(1, 1);
#pragma unroll
  for (int j = 1; j < NP - 1; ++j) issue_b(j, 1);
  wait_vm_lgkm0<2 * NP + 2>();   // both halves of A and strip 0 of stage 0
  __builtin_amdgcn_s_barrier();
  lds_frag4<0>(af[0][0], pa, 0u);
  lds_frag4<ASZ / 2>(af[0][1], pa, 0u);
  __builtin_amdgcn_s_barrier();
  if (wv >= 4) __builtin_amdgcn_s_barrier();

  auto phase = [&](auto pc, auto setc, int kt) {
    constexpr int P = decltype(pc)::value, SET = decltype(setc)::value;
    if constexpr (P == 0) {
      issue_b(NP - 1, kt + 1);
      issue_a(0, kt + 2);
    } else {
      issue_b(P - 1, kt + 2);
      if constexpr (P == 1) issue_a(1, kt + 2);
    }
    const uint32_t cur = uint32_t(kt & 1) * STAGE, nxt = uint32_t(STAGE) - cur;
    if constexpr (P >= NP - 2) {
      constexpr int I = P - (NP - 2);
      lds_frag8<ASZ + P * 8192, I * (ASZ / 2)>(bf, pb, cur, af[1 - SET][I], pa, nxt);
    } else {
      lds_frag4<ASZ + P * 8192>(bf, pb, cur);
    }
    wait_vm_lgkm0<pp_wait<NP>(P)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i][P] = lin_mfma<uint16_t>(bf[s], af[SET][i][s], acc[i][P]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
  };
  auto kstep = [&](auto setc, int kt) {
    phase(std::integral_constant<int, 0>{}, setc, kt);
    phase(std::integral_constant<int, 1>{}, setc, kt);
    phase(std::integral_constant<int, 2>{}, setc, kt);
    if constexpr (NP == 4) phase(std::integral_constant<int, 3>{}, setc, kt);
  };
  int kt = 0;
  for (; kt + 1 < KT; kt += 2) {
    kstep(std::integral_constant<int, 0>{}, kt);
    kstep(std::integral_constant<int, 1>{}, kt + 1);
  }
  if (kt < KT) kstep(std::integral_constant<int, 0>{}, kt);
  if (wv < 4) __builtin_amdgcn_s_barrier();
  wait_vm_lgkm0<0>();
  __builtin_amdgcn_s_barrier();

  float* const stg = reinterpret_cast<float*>(smem + wv * 32 * SPITCH);
  constexpr int LPR = WN / 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(stg + lrow * (SPITCH / 4) + j * 32 + 8 * g + 4 * lhalf) =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                        acc[i][j][4 * g + 3]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll 4
    for (int q = 0; q < 32 * LPR / 64; ++q) {
      const int r = (lane + 64 * q) / LPR, c = 8 * ((lane + 64 * q) % LPR);
      const int64_t m = m0 + wm * 64 + 32 * i + r, n = n0 + wn * WN + c;
      float v[8];
      load8(stg + r * (SPITCH / 4) + c, v);
      if (m < M && n < N) finish8(v, m, n, N, ep);
    }
    __builtin_amdgcn_wave_barrier();
  }
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
  float v[8];
  load8(p, v);
  for (int s = 1; s < splits; ++s) {
    float a[8];
    load8(p + int64_t(s) * M * N, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += a[e];
  }
  finish8(v, m, n, N, ep);
}

// ---- host side --------------------------------------------------------------------

namespace {

enum LinKind { LIN_ROWS, LIN_T32, LIN_T64, LIN_T128, LIN_PP3, LIN_PP4 };

// Kernel and split count of a product. Rows up to 8 take the vector kernel.
// Otherwise the tile shrinks until the tiles cover the 256 CUs, and a product
// that still leaves CUs idle is split over K, at least 4 k-steps per split.
struct LinPlan {
  LinKind kind;
  int splits, kper;
};
LinPlan linear_plan(int64_t M, int64_t N, int K, int esize) {
  LinPlan p = {LIN_ROWS, 1, (K * esize + 127) / 128};
  if (M <= 8) return p;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  int64_t t = tiles(128, 128);
  p.kind = LIN_T128;
  if (t < 256) {
    p.kind = M <= 32 ? LIN_T32 : LIN_T64;
    t = M <= 32 ? tiles(32, 128) : tiles(64, 64);
  }
  if (esize == 2 && tiles(256, 192) >= 128) {
    // the wide tiles whose rounds of one per CU cost less
    const int64_t r3 = (tiles(256, 192) + 255) / 256 * 3, r4 = (tiles(256, 256) + 255) / 256 * 4;
    p.kind = r3 < r4 ? LIN_PP3 : LIN_PP4;
    return p;
  }
  const int ksteps = p.kper;
  if (t < 256) {
    int64_t want = 512 / t;
    if (want > ksteps / 4) want = ksteps / 4;
    if (want > 16) want = 16;
    if (want > 1) {
      p.kper = int((ksteps + want - 1) / want);
      p.splits = (ksteps + p.kper - 1) / p.kper;
    }
  }
  return p;
}

template <typename TE, int TT>
void launch_rows_nc(const TE* X, int M, const TE* W, int64_t N, int K, const LinEpi& ep,
                    hipStream_t s) {
  // columns per wave: more reuse of X per load of W where there are waves enough
  if (N >= 4096)
    hipLaunchKernelGGL((linear_rows_kernel<TE, TT, 2>), dim3(unsigned((N + 7) / 8)), dim3(256), 0, s,
                       X, M, W, N, K, ep);
  else
    hipLaunchKernelGGL((linear_rows_kernel<TE, TT, 1>), dim3(unsigned((N + 3) / 4)), dim3(256), 0, s,
                       X, M, W, N, K, ep);
}

template <typename TE, int BM, int BN, int WM, int WN, int S, int OCC>
void launch_tile(const TE* X, int64_t M, const TE* W, int64_t N, int K, const LinPlan& p,
                 float* part, const LinEpi& ep, hipStream_t s) {
  const int64_t ntiles = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  hipLaunchKernelGGL((linear_tile_kernel<TE, BM, BN, WM, WN, S, OCC>),
                     dim3(unsigned(ntiles), unsigned(p.splits)),
                     dim3((BM / WM) * (BN / WN) * 64), 0, s, X, M, W, N, K, p.kper,
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
      else if (M <= 4) launch_rows_nc<TE, 4>(X, int(M), W, N, K, ep, s);
      else launch_rows_nc<TE, 8>(X, int(M), W, N, K, ep, s);
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
    case LIN_T32: launch_tile<TE, 32, 128, 32, 32, 3, 2>(X, M, W, N, K, p, part, ep, s); break;
    case LIN_T64: launch_tile<TE, 64, 64, 32, 32, 3, 2>(X, M, W, N, K, p, part, ep, s); break;
    case LIN_T128: launch_tile<TE, 128, 128, 64, 64, 2, 2>(X, M, W, N, K, p, part, ep, s); break;
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

// GELU (bf16 results): degree-6 weighted least-maximum fit of log2(Phi(x) / Phi(-x)) / x in
// x^2 on |x| <= 5; the other two are exact forms.
ActCoef act_coef(int act) {
  ActCoef a = {};
  a.act = act;
  constexpr float log2e = 1.4426950408889634f;
  if (act == ACT_SILU) {
    a.tmax = 0.0f;
    a.c[0] = log2e;
  } else if (act == ACT_GELU_TANH) {
    a.tmax = 1e6f;   // 2^(-x P) is 0 or infinite long before; keeps x^2 finite
    a.c[0] = 1.5957691216057308f * log2e;
    a.c[1] = 1.5957691216057308f * 0.044715f * log2e;
  } else if (act == ACT_GELU) {
    a.tmax = 25.0f;
    const float c[7] = {2.3017581959277815f,     0.10552445421016707f,   -0.0003938443860880515f,
                        -0.0001041246928390452f, 6.513520962607899e-06f, -1.7551338906125295e-07f,
                        1.842194984814521e-09f};
    for (int k = 0; k < 7; ++k) a.c[k] = c[k];
  }
  return a;
}

}  // namespace hq
