// Root-mean-square norm of the residual stream, with the residual's addition
// before it and, where asked for, its result as the 8-bit codes of a low-bit
// layer:
//
//   h = x + r,   y = h rstd gamma,   rstd = 1 / sqrt(mean(h^2) + eps),
//   code_c = rint(y_c / s),   s = max_c |y_c| / 127   (one scale per row).
//
// rstd is one factor per row, so the codes do not depend on it: code_c =
// rint(127 v_c / max |v|) with v = h gamma, and s = rstd max |v| / 127. The sum of
// squares and max |v| are taken in one pass over the row in registers; bound by
// memory: x and r are read once, h, y and the codes written once.
//
// A code is decided as if v and the quotient were exact. In fp32, q = v rcp(max) 127
// carries two roundings of 2^-24 in v, two in the maximum, and 2^-23 + 2^-24 in 127
// rcp(max): an error below 127 x 7 x 2^-24 = 5.3e-5. Where q is further
// than 1e-4 from a half-integer its rounding is the exact one; the values nearer to one
// (2 in 10^4) are decided again from v and the row's maximum in fp64, which needs only
// the values within 2^-21 of the fp32 maximum in fp64. Ties are common where gamma is absent
// (half of the largest value is 63.5 of the scale) and a rounded quotient misses them for 15
// of the 128 bf16 mantissas, so products are compared (code_of). A row with a v that is not
// a finite float has codes 0 and a NaN scale.
#include "hq_epilogue.h"
#include "hq_internal.h"

#include <algorithm>

namespace hq {

namespace {

constexpr float kBorder = 0.5f - 1e-4f;
// Rows whose maximum is below 2^-100 lose bits of v in fp32 to the smallest floats (all of
// them where no v is as large as half of one), and above 2^125 the reciprocal does: all their
// codes and their scale are made in fp64.
constexpr float kTiny = 0x1p-100f, kHuge = 0x1p125f;
// Of the others, a value that can be the row's largest in fp64 is at least this part of the
// fp32 maximum: each of the two carries 2^-23 of itself.
constexpr float kNear = 1.0f - 0x1p-21f;
// The norm is v rstd: what v loses to the smallest floats (half of one, 2^-150) is below
// 2^-126 of the norm up to this rstd. Beyond, gamma comes last.
constexpr float kSteep = 0x1p24f;

// 127 v / top rounded half to even, without the rounding of a quotient: the products that
// decide between two codes are compared with what their roundings leave out.
__device__ __forceinline__ int code_of(double v, double top) {
  const double a = fabs(v), n = floor(127.0 * a / top), c = 2.0 * n + 1.0;
  const double p = 254.0 * a, q = c * top;
  const double over = (p - q) + (fma(254.0, a, -p) - fma(c, top, -q));   // of 254 |v| over c top
  const int code = int(n) + (over > 0.0 || (over == 0.0 && (int(n) & 1)) ? 1 : 0);
  return v < 0.0 ? -code : code;
}

// Maximum over the wave of a non-negative double that few lanes have.
__device__ __forceinline__ double few_max(double v, bool mine) {
  uint64_t left = __ballot(mine);
  double m = 0.0;
  while (left) {
    const int l = __builtin_ctzll(left);
    left &= left - 1;
    const uint64_t bits = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(bits), l);
    const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(bits >> 32), l);
    m = fmax(m, __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo));
  }
  return m;
}

// Maximum over aligned groups of L lanes of the bits of non-negative floats: as
// integers NaN is above infinity and infinity above every number.
template <int L>
__device__ __forceinline__ uint32_t bits_max(uint32_t v) {
  auto other = [](uint32_t a, float b) { return max(a, __float_as_uint(b)); };
  if constexpr (L >= 2) v = other(v, lane_xor<1>(__uint_as_float(v)));
  if constexpr (L >= 4) v = other(v, lane_xor<2>(__uint_as_float(v)));
  if constexpr (L >= 8) v = other(v, lane_xor<4>(__uint_as_float(v)));
  if constexpr (L >= 16) v = other(v, lane_xor<8>(__uint_as_float(v)));
  if constexpr (L >= 32) { float lo, hi; lane_pair<16>(__uint_as_float(v), &lo, &hi); v = other(__float_as_uint(lo), hi); }
  if constexpr (L >= 64) { float lo, hi; lane_pair<32>(__uint_as_float(v), &lo, &hi); v = other(__float_as_uint(lo), hi); }
  return v;
}
constexpr uint32_t kInf = 0x7f800000u;

// Is any of eight values as loaded other than +-0?
template <typename TE>
__device__ __forceinline__ bool not_zero(const Raw8<TE>& r) {
  uint32_t b = 0;
#pragma unroll
  for (unsigned i = 0; i < sizeof(TE) / 2; ++i) b |= r.q[i].x | r.q[i].y | r.q[i].z | r.q[i].w;
  return (b & (sizeof(TE) == 2 ? 0x7fff7fffu : 0x7fffffffu)) != 0;
}

}  // namespace

// L lanes per row (64 / L rows per wave) and W waves per row (W > 1: L = 64, a block
// per row), R pieces of 8 channels per lane. Q: codes are wanted. Rows of up to 2048
// channels take a wave or part of one, which needs no barrier; longer ones a block, which
// keeps them in registers. 8192 x 4096 bf16, residual, sum, norm and codes: 54 to 59 us, 5.1
// to 5.6 TB/s; 8192 x 1152, sum and codes: 16.6 us, 4.0 TB/s (a quarter of the lanes' third
// pieces have channels; deciding codes again costs a tenth). fp32, norm and codes: 12288 x 256
// 9.4 us, 8192 x 1024 16.1 (4.7 TB/s), 4096 x 2048 18.1, 2048 x 8192 35.4 (4.3); one row of
// 4096: 2.6 us, all of it latency.
// The least waves per SIMD keep the registers of the codes' rare path down (12288 x 256
// fp32 9.9 -> 9.6 us, 8192 x 4096 bf16 61.6 -> 59.5; one more wave spills: 13.1, 70.9).
// fp32 takes one wave less where it would spill: with codes at two pieces (8192 x 1024: 5
// waves 19.9 us, 4 waves 16.0) and at four (2048 x 8192 norm and codes: 4 waves 45.7, 3 waves
// 35.3; 4096 x 2048: 23.0, 18.1).
constexpr int rms_waves(bool f32, int R, bool Q) {
  return R == 1 ? 6 : R == 2 ? (f32 && Q ? 4 : 5) : R == 4 && f32 ? 3 : 4;
}
template <typename TE, int L, int W, int R, bool Q>
__global__ __launch_bounds__(256, rms_waves(sizeof(TE) == 4, R, Q)) void rms_kernel(RmsArgs k) {
  static_assert(W == 1 || (W == 4 && L == 64), "a block per row or whole rows per wave");
  __shared__ float part[2][W], part_z[W];   // of rows in turn: one barrier for each
  __shared__ uint32_t part_bits[2][W];
  __shared__ double part_top[W];
  int turn = 0;
  constexpr int RPB = 256 / (L * W);   // rows per block
  const int VR = k.C / 8;
  const int sub = W > 1 ? int(threadIdx.x) : int(threadIdx.x) & (L - 1);
  constexpr int STEP = L * W;          // pieces between a lane's pieces
  for (int64_t r0 = int64_t(blockIdx.x) * RPB; r0 < k.T; r0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = W > 1 ? r0 : r0 + int(threadIdx.x) / L;
    const int nv = row < k.T ? VR : 0;
    const int64_t base = row * k.C + 8 * sub;
    Raw8<TE> x[R], r[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (sub + STEP * i < nv) x[i] = raw_load(static_cast<const TE*>(k.x) + base + 8 * STEP * i);
    if (k.r) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (sub + STEP * i < nv) r[i] = raw_load(static_cast<const TE*>(k.r) + base + 8 * STEP * i);
    }
    // h of piece i, in fp32: x and r stay as they were loaded, beside v = h gamma
    auto sum_of = [&](int i, float (&h)[8]) {
      raw_get(x[i], h);
      if (k.r) {
        float t[8];
        raw_get(r[i], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += t[e];
      }
    };
    // h gamma of value n = 8 i + e of the lane in fp64, from memory (nothing of the row is
    // written before the codes are decided; few values come here, and indexes that are not
    // known beforehand keep registers free)
    auto exact = [&](int n) {
      const int64_t c = 8 * (sub + STEP * (n >> 3)) + (n & 7);
      auto at = [&](const void* p) {
        if constexpr (sizeof(TE) == 2) return double(bf16_to_f32(static_cast<const uint16_t*>(p)[row * k.C + c]));
        else return double(static_cast<const float*>(p)[row * k.C + c]);
      };
      const double h = k.r ? at(k.x) + at(k.r) : at(k.x);
      return k.gamma ? h * double(k.gamma[c]) : h;
    };
    float v[R][8];
    float s2 = 0.0f;
    uint32_t tb = 0;   // bits of max |h gamma|
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (sub + STEP * i < nv) {
        float h[8], g[8];
        if (k.gamma) load8(k.gamma + 8 * (sub + STEP * i), g);
        sum_of(i, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s2 = fmaf(h[e], h[e], s2);
          v[i][e] = k.gamma ? h[e] * g[e] : h[e];
          if constexpr (Q) tb = max(tb, __float_as_uint(v[i][e]) & 0x7fffffffu);
        }
      }
    }
    s2 = group_sum<L>(s2);
    const float mine = __uint_as_float(tb);   // the lane's largest |h gamma|
    double top64 = 0.0;
    if constexpr (Q) tb = bits_max<L>(tb);
    // The largest of the lanes' values `which` in fp64, for every lane: of the wave's part of
    // a row (W > 1) or of each row of the wave.
    auto max64 = [&](uint32_t which) {
      double m = 0.0;
      const bool any = which != 0;
      for (; which; which &= which - 1) m = fmax(m, fabs(exact(__builtin_ctz(which))));
      if constexpr (L == 64) {
        m = few_max(m, any);
      } else {
#pragma unroll
        for (int d = 1; d < L; d <<= 1) m = fmax(m, __shfl_xor(m, d, 64));
      }
      return m;
    };
    if constexpr (W > 1) {
      const int w = int(threadIdx.x) >> 6;
      if ((threadIdx.x & 63) == 0) {
        part[turn][w] = s2;
        if constexpr (Q) part_bits[turn][w] = tb;
      }
      __syncthreads();
      const float* const p = part[turn];
      s2 = (p[0] + p[1]) + (p[2] + p[3]);
      if constexpr (Q) {
        const uint32_t* const b = part_bits[turn];
        tb = max(max(b[0], b[1]), max(b[2], b[3]));
      }
      turn ^= 1;
    }
    // rsq is off by one unit; eps keeps it from the smallest floats, which it does not take
    const float ms = fmaf(s2, k.inv_c, k.eps);
    float rstd = __builtin_amdgcn_rsqf(ms);
    if (__any(ms == INFINITY)) {
      // squares past the largest float, or with eps: once more, of h 2^-80 (the same branch
      // for a whole block where a block has one row)
      float z2 = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (sub + STEP * i >= nv) continue;
        float h[8];
        sum_of(i, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = h[e] * 0x1p-80f;
          z2 = fmaf(z, z, z2);
        }
      }
      z2 = group_sum<L>(z2);
      if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part_z[int(threadIdx.x) >> 6] = z2;
        __syncthreads();
        z2 = (part_z[0] + part_z[1]) + (part_z[2] + part_z[3]);
      }
      if (ms == INFINITY) rstd = 0x1p-80f / sqrtf(z2 * k.inv_c + k.eps * 0x1p-80f * 0x1p-80f);
    }
    if constexpr (Q) {
      const bool finite = tb < kInf;
      const float top = __uint_as_float(tb);
      const bool plain = top >= kTiny && top <= kHuge;
      const float rcp = plain ? 127.0f * __builtin_amdgcn_rcpf(top) : 0.0f;
      const float border = plain || !finite || top == 0.0f ? kBorder : -1.0f;
      uint32_t again = 0;   // values next to a half-integer; all of a row that is not plain
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (sub + STEP * i >= nv) continue;
        uint32_t d[2] = {};
        float far = -0.5f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = rintf(v[i][e] * rcp);
          far = fmaxf(far, fabsf(fmaf(v[i][e], rcp, -n)));
          d[e >> 2] |= (uint32_t(int(n)) & 255u) << (8 * (e & 3));
        }
        if (far > border) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            again |= fabsf(fmaf(v[i][e], rcp, -rintf(v[i][e] * rcp))) > border ? 1u << (8 * i + e) : 0u;
        }
        // zeros, or products that are none but round to it
        if (top == 0.0f && k.gamma && (not_zero(x[i]) || (k.r && not_zero(r[i]))) &&
            not_zero(raw_load(k.gamma + 8 * (sub + STEP * i))))
          again |= 255u << (8 * i);
        *reinterpret_cast<uint2*>(k.codes + base + 8 * STEP * i) =
            finite ? make_uint2(d[0], d[1]) : make_uint2(0, 0);
      }
      auto largest = [&] {   // the lane's values among which the row's fp64 maximum is
        uint32_t which = plain ? 0u : again;
        if (plain && mine >= top * kNear) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            if (sub + STEP * i >= nv) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) which |= fabsf(v[i][e]) >= top * kNear ? 1u << (8 * i + e) : 0u;
          }
        }
        return which;
      };
      // every wave of the row has to help where one needs the fp64 maximum
      if constexpr (W == 1) {
        if (__any(again)) top64 = max64(largest());
      } else if (__syncthreads_or(again != 0)) {
        top64 = max64(largest());
        if ((threadIdx.x & 63) == 0) part_top[int(threadIdx.x) >> 6] = top64;
        __syncthreads();
        top64 = fmax(fmax(part_top[0], part_top[1]), fmax(part_top[2], part_top[3]));
      }
      for (; again; again &= again - 1) {
        const int n = __builtin_ctz(again);
        k.codes[base + 8 * STEP * (n >> 3) + (n & 7)] = uint8_t(top64 > 0.0 ? code_of(exact(n), top64) : 0);
      }
      if (sub == 0 && row < k.T)
        k.scales[row] = !finite ? __uint_as_float(0x7fc00000u)
                        : plain ? top * (1.0f / 127.0f) * rstd
                                : float(top64 * double(rstd) * (1.0 / 127.0));
    }
    if (k.h) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (sub + STEP * i >= nv) continue;
        float h[8];
        sum_of(i, h);
        store8(static_cast<TE*>(k.h) + base + 8 * STEP * i, h);
      }
    }
    if (k.y) {
      const bool steep = k.gamma && rstd > kSteep;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (sub + STEP * i >= nv) continue;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[i][e] * rstd;
        if (steep) {
          float h[8], g[8];
          load8(k.gamma + 8 * (sub + STEP * i), g);
          sum_of(i, h);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = h[e] * rstd * g[e];
        }
        if (k.y_bf16) store8(static_cast<uint16_t*>(k.y) + base + 8 * STEP * i, y);
        else store8(static_cast<float*>(k.y) + base + 8 * STEP * i, y);
      }
    }
  }
}

namespace {

template <typename TE, int L, int W, int R>
hipError_t launch_rms_form(const RmsArgs& a, hipStream_t s) {
  constexpr int RPB = 256 / (L * W);
  const int64_t blocks = std::min<int64_t>((a.T + RPB - 1) / RPB, 1 << 20);
  if (a.codes)
    hipLaunchKernelGGL((rms_kernel<TE, L, W, R, true>), dim3(unsigned(blocks)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((rms_kernel<TE, L, W, R, false>), dim3(unsigned(blocks)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename TE>
hipError_t launch_rms_typed(const RmsArgs& a, hipStream_t s) {
  const int v = a.C / 8;
  if (v <= 8) return launch_rms_form<TE, 8, 1, 1>(a, s);
  if (v <= 16) return launch_rms_form<TE, 16, 1, 1>(a, s);
  if (v <= 32) return launch_rms_form<TE, 32, 1, 1>(a, s);
  if (v <= 64) return launch_rms_form<TE, 64, 1, 1>(a, s);
  if (v <= 128) return launch_rms_form<TE, 64, 1, 2>(a, s);
  if (v <= 192) return launch_rms_form<TE, 64, 1, 3>(a, s);
  if (v <= 256) return launch_rms_form<TE, 64, 1, 4>(a, s);
  if (v <= 512) return launch_rms_form<TE, 64, 4, 2>(a, s);
  if (v <= 768) return launch_rms_form<TE, 64, 4, 3>(a, s);
  return launch_rms_form<TE, 64, 4, 4>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const RmsArgs& a, hipStream_t s) {
  return a.x_bf16 ? launch_rms_typed<uint16_t>(a, s) : launch_rms_typed<float>(a, s);
}

}  // namespace hq
