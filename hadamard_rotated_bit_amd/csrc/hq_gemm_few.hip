// The low-bit product with the extended epilogue for few tokens (HaTQ Sec.
// III-B Eq. (4), then hq_epilogue.h): where a tile of rows is all there is, the
// tiled GEMMs walk their stages one after another on a handful of CUs.
//
// Here a block of eight waves owns 32 tokens x 32 channels, and the waves take
// the 128-code stages in turn: fragments go straight from memory into registers
// (a wave's 32 rows of a stage are whole 384-byte groups of the E2M3 layout or
// whole 128-byte lines of int8 codes), several stages in flight, no barrier until
// the waves' sums meet in LDS. Integer sums are exact in any order (fp32 below
// 2^24 on the FP6 engine, int32 on the int8 one), so the results are those of the
// tiled kernels; with group-wise scales the waves' fp32 sums are joined in wave
// order. Bound by latency: one or two rounds of loads, one join. A call (two
// launches) of one token, 4608 -> 1152: 10.4 us against 17.8 with the tiled FP6
// kernel, 12.6 against 22.9 with the int8 one, 17.3 against 55.3 with group-wise
// scales; 1152 -> 4608: 7.7 against 10.7, 7.8 against 11.1, 12.5 against 23.8.
#include "hq_epilogue.h"
#include "hq_gemm6_kernel.h"
#include "hq_internal.h"

namespace hq {

namespace {

// Group-wise scales (EngF6G): s_x [group, ldx], s_w [group, ldw].
struct GroupScales {
  const float* sx;
  int64_t ldx;
  const float* sw;
  int64_t ldw;
};

// A wave's operand of one stage: lane l holds row l % 32, half l / 32; its
// scales of a stage, where there are any, are of token row l % 32 and of the
// accumulators' channels.
struct NoScales {
  __device__ __forceinline__ void load(const GroupScales&, int, int64_t, int64_t, int64_t, int) {}
};
struct EngF6 {
  static constexpr int U = 3;   // stages in flight per wave
  typedef NoScales Scales;
  typedef v16f Acc;
  typedef Frag6 Frag;
  static __device__ __forceinline__ const uint8_t* row(const uint8_t* p, int64_t r, int half, int K) {
    return p + (r / F6_GROUP) * F6_GROUP * f6_row_bytes(K) + (r % F6_GROUP) * 96 + 48 * half;
  }
  static constexpr int STEP = 96 * F6_GROUP;   // bytes from a stage to the next
  static __device__ __forceinline__ void load(Frag& f, const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < 3; ++i) f.c[i] = *reinterpret_cast<const v4i*>(p + 16 * i);
  }
  static __device__ __forceinline__ void mfma(Acc& c, const Frag& w, const Frag& x, const Scales&) {
    c = mfma_f6(f6_op0(w), f6_op0(x), c);
    c = mfma_f6(f6_op1(w), f6_op1(x), c);
  }
};
// 64-channel groups: each half of a stage is a group with scales of its own, the
// lane's two 24-byte operands are the halves of one group each.
struct EngF6G {
  static constexpr int U = 2;
  struct Scales {
    float x[2];
    v4f w[2][4];
    __device__ __forceinline__ void load(const GroupScales& g, int stage, int64_t m, int64_t n0,
                                         int64_t N, int lhalf) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = g.sx[(2 * int64_t(stage) + i) * g.ldx + m];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t n = n0 + 8 * q + 4 * lhalf;
          w[i][q] = *reinterpret_cast<const v4f*>(g.sw + (2 * int64_t(stage) + i) * g.ldw + (n < N ? n : 0));
        }
      }
    }
  };
  typedef v16f Acc;
  struct Frag {
    v2i c[6];
  };
  static __device__ __forceinline__ const uint8_t* row(const uint8_t* p, int64_t r, int half, int K) {
    return p + (r / F6_GROUP) * F6_GROUP * f6_row_bytes(K) + (r % F6_GROUP) * 96 + 24 * half;
  }
  static constexpr int STEP = 96 * F6_GROUP;
  static __device__ __forceinline__ void load(Frag& f, const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < 6; ++i) f.c[i] = *reinterpret_cast<const v2i*>(p + (i < 3 ? 0 : 24) + 8 * i);
  }
  static __device__ __forceinline__ v8i op(const Frag& f, int g) {
    return v8i{f.c[3 * g][0], f.c[3 * g][1], f.c[3 * g + 1][0], f.c[3 * g + 1][1],
               f.c[3 * g + 2][0], f.c[3 * g + 2][1], 0, 0};
  }
  static __device__ __forceinline__ void mfma(Acc& c, const Frag& w, const Frag& x, const Scales& s) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const Acc t = mfma_f6(op(w, g), op(x, g), Acc{});
#pragma unroll
      for (int r = 0; r < 16; ++r) c[r] = fmaf(t[r], s.x[g] * s.w[g][r / 4][r % 4], c[r]);
    }
  }
};
struct EngI8 {
  static constexpr int U = 3;
  typedef NoScales Scales;
  typedef v16i Acc;
  struct Frag {
    v4i c[4];
  };
  static __device__ __forceinline__ const uint8_t* row(const uint8_t* p, int64_t r, int half, int K) {
    return p + r * K + 64 * half;
  }
  static constexpr int STEP = 128;
  static __device__ __forceinline__ void load(Frag& f, const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.c[i] = *reinterpret_cast<const v4i*>(p + 16 * i);
  }
  static __device__ __forceinline__ void mfma(Acc& c, const Frag& w, const Frag& x, const Scales&) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_i32_32x32x32_i8(w.c[i], x.c[i], c, 0, 0, 0);
  }
};

constexpr int FEW_NW = 8;

template <typename E>
__global__ __launch_bounds__(64 * FEW_NW) void gemm_few_kernel(const uint8_t* __restrict__ A, int64_t M,
                                                               const uint8_t* __restrict__ B, int64_t N,
                                                               int K, GemmEpi ep, GroupScales gs) {
  constexpr int U = E::U;
  constexpr int PITCH = 36;   // words: 32 and one 16-byte pad
  constexpr int SLOT = 32 * PITCH;
  __shared__ __attribute__((aligned(16))) uint32_t smem[(FEW_NW + 1) * SLOT];
  typedef decltype(typename E::Acc{}[0] + 0) T;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int lrow = lane & 31, lhalf = lane >> 5;
  const int64_t n0 = int64_t(blockIdx.x) * 32, m0 = int64_t(blockIdx.y) * 32;
  const int KT = K / 128;
  // rows past the end repeat the last one; nothing of them is stored
  const int64_t ma = m0 + lrow < M ? m0 + lrow : M - 1, nb = n0 + lrow < N ? n0 + lrow : N - 1;
  const uint8_t* const pa = E::row(A, ma, lhalf, K);
  const uint8_t* const pb = E::row(B, nb, lhalf, K);

  typename E::Acc acc = {};
  for (int s0 = wv; s0 < KT; s0 += FEW_NW * U) {
    typename E::Frag a[U], b[U];
    typename E::Scales sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + FEW_NW * u < KT) {
        E::load(a[u], pa + int64_t(s0 + FEW_NW * u) * E::STEP);
        E::load(b[u], pb + int64_t(s0 + FEW_NW * u) * E::STEP);
        sc[u].load(gs, s0 + FEW_NW * u, ma, n0, N, lhalf);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s0 + FEW_NW * u < KT) E::mfma(acc, b[u], a[u], sc[u]);
  }
  uint32_t* const mine = smem + wv * SLOT + lrow * PITCH + 4 * lhalf;
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const T v = acc[4 * g + e];
      mine[8 * g + e] = __builtin_bit_cast(uint32_t, v);
    }
  if (ep.rank && wv == FEW_NW - 1) {   // the low-rank product, the last slot
    v16f lr = {};
    for (int k0 = 0; k0 < ep.rank; k0 += 16) {
      float f[8];
      load8(ep.U + ma * ep.rank + k0 + 8 * lhalf, f);
      const v8bf uh = pack_bf16x8(f, false), ul = pack_bf16x8(f, true);
      const int64_t off = nb * ep.rank + k0 + 8 * lhalf;
      const v8bf wh = *reinterpret_cast<const v8bf*>(ep.l2_hi + off);
      lr = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wh, uh, lr, 0, 0, 0);
      if (!ep.l2_lo_zero) {
        const v8bf wl = *reinterpret_cast<const v8bf*>(ep.l2_lo + off);
        lr = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wl, uh, lr, 0, 0, 0);
      }
      lr = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wh, ul, lr, 0, 0, 0);
    }
    uint32_t* const l = smem + FEW_NW * SLOT + lrow * PITCH + 4 * lhalf;
#pragma unroll
    for (int r = 0; r < 16; ++r) l[8 * (r / 4) + r % 4] = __float_as_uint(lr[r]);
  }
  // one lane per 8 channels of a token
  const int r = int(threadIdx.x) / 4, c = 8 * (int(threadIdx.x) % 4);
  const int64_t m = m0 + r, n = n0 + c;
  const bool live = threadIdx.x < 128 && m < M && n < N;
  float sx = 0.0f, mu = 0.0f, sw[8], cb[8], bb[8];
  if (live) {
    mu = ep.mu[m];
    if (!ep.prescaled) {
      sx = ep.s_x[m];
      load8(ep.s_w + n, sw);
    }
    load8(ep.c + n, cb);
    load8(ep.bias + n, bb);
  }
  __syncthreads();
  if (!live) return;
  T sum[8] = {};
  const uint32_t* const s = smem + r * PITCH + c;
#pragma unroll
  for (int w = 0; w < FEW_NW; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += __builtin_bit_cast(T, s[w * SLOT + e]);
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // the tiled kernels' expressions, term by term (the same bits)
    y[e] = fmaf(mu, cb[e], bb[e]);
    y[e] = ep.prescaled ? float(sum[e]) + y[e] : fmaf(float(sum[e]), sx * sw[e], y[e]);
    if (ep.rank) y[e] += __uint_as_float(s[FEW_NW * SLOT + e]);
  }
  finish_piece(y, m, n, N, ep.lin);
}

}  // namespace

// Four tiles per CU on the FP6 engine (a call of 160 x 1152 -> 4608, 720 tiles: 10.6
// us against 12.4 with the tiled kernel; 256 x 4096 -> 4096, 1024 tiles: 18.2 against
// 20.0; 300 x 4096 -> 4096, 1280 tiles, the other way, 21.0 against 20.2), also with
// group-wise scales (1024 tiles: 38 against 55; 512 x 1152 -> 4608, 2304 tiles, the
// other way, 38.6 against 27.0); three for two CUs with int8 codes (96 x 4096 ->
// 4096, 384 tiles: 22.6 against 23.2; 128 x 1152 -> 4608, 576 tiles, the other way,
// 13.6 against 12.8).
bool gemm_few_fits(int engine, int64_t M, int64_t N) {
  return ((M + 31) / 32) * ((N + 31) / 32) <= (engine == GEMM_FEW_I8 ? 384 : 1024);
}

hipError_t launch_gemm_few(int engine, const void* A, int64_t M, const void* B, int64_t N, int K,
                           const GemmEpi& ep, hipStream_t s, const float* s_xg, int64_t ld_sx,
                           const float* s_wg, int64_t ld_sw) {
  if (K % 128) return hipErrorInvalidValue;
  const dim3 grid(unsigned((N + 31) / 32), unsigned((M + 31) / 32)), block(64 * FEW_NW);
  const uint8_t *a = static_cast<const uint8_t*>(A), *b = static_cast<const uint8_t*>(B);
  const GroupScales gs = {s_xg, ld_sx, s_wg, ld_sw};
  if (engine == GEMM_FEW_F6G)
    hipLaunchKernelGGL(gemm_few_kernel<EngF6G>, grid, block, 0, s, a, M, b, N, K, ep, gs);
  else if (engine == GEMM_FEW_F6)
    hipLaunchKernelGGL(gemm_few_kernel<EngF6>, grid, block, 0, s, a, M, b, N, K, ep, gs);
  else
    hipLaunchKernelGGL(gemm_few_kernel<EngI8>, grid, block, 0, s, a, M, b, N, K, ep, gs);
  return hipGetLastError();
}

}  // namespace hq
