// Rotary positions with several axes (time, height, width) on the q and k heads of a
// packed projection, behind an RMS norm of each head where the model has one:
//
//   n = x / sqrt(mean(x^2) + eps) gamma          (per head; absent: n = x)
//   (a', b') = (a cos t - b sin t, b cos t + a sin t),   t = pos[token, axis(i)] freq_i,
//
// for pair i of a head; pairs are neighbours (2i, 2i + 1) or halves (i, i + P) of its
// first 2 P channels, P the pairs of all axes; the channels behind them pass. The
// inverse takes -t. Bound by memory: q and k are read once and written once.
//
// Angles. pos freq can be many turns, so it is reduced in fp64: u = pos (freq / 2 pi)
// less its nearest integer, then less the nearest quarter, and only what remains (at
// most an eighth of a turn) goes to fp32, where sin and cos are their Taylor series
// (first term left out below 2^-28). cos and sin are off by at most 2.2e-7 plus
// |pos freq| 2^-51.
// One lane evaluates each pair of a token and shares it with the heads through LDS.
#include "hq_epilogue.h"
#include "hq_internal.h"

#include <algorithm>

namespace hq {

namespace {

__device__ __forceinline__ void turn_sincos(double pos, double freq, float* s, float* c) {
  double u = pos * (freq * 0.15915494309189533577);
  u -= rint(u);
  u *= 4.0;
  const double k = rint(u);
  const float x = float(u - k) * 1.57079632679489662f, z = x * x;
  float a = 1.0f / 362880.0f;
  a = fmaf(a, z, -1.0f / 5040.0f);
  a = fmaf(a, z, 1.0f / 120.0f);
  a = fmaf(a, z, -1.0f / 6.0f);
  a = fmaf(a * z, x, x);
  float b = -1.0f / 3628800.0f;
  b = fmaf(b, z, 1.0f / 40320.0f);
  b = fmaf(b, z, -1.0f / 720.0f);
  b = fmaf(b, z, 1.0f / 24.0f);
  b = fmaf(b, z, -0.5f);
  b = fmaf(b, z, 1.0f);
  const int q = int(k);                    // -2 .. 2 quarter turns
  const float sn = (q & 1) ? b : a, cs = (q & 1) ? a : b;
  *s = (q & 2) ? -sn : sn;                 // quarters 2 and 3 (= -2, -1)
  *c = ((q + 1) & 2) ? -cs : cs;           // quarters 1 and 2
}

// Four consecutive elements.
__device__ __forceinline__ void load4(const float* p, float v[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float v[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float v[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float v[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// Sum over the n lanes from `first` (n uniform, up to 32; lanes of other runs do the
// same): every lane gets the sum, in one fixed order.
__device__ __forceinline__ float run_sum(float v, int first, int n, int pos) {
  for (int d = 32; d >= 1; d >>= 1) {
    if (d >= n) continue;
    const float o = __shfl(v, first + pos + d, 64);
    if (pos + d < n && pos < d) v += o;
  }
  return __shfl(v, first, 64);
}

}  // namespace

// A wave per token and part of its heads (parts per token: `split`); a head's D / 8
// units of 8 channels go to D / 8 lanes, 64 / (D / 8) heads at a time.
template <typename TE, typename TY, bool HALVES>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs k) {
  __shared__ float cs[4][2][ROPE_MAX_PAIRS];
  const int lane = int(threadIdx.x) & 63, w = int(threadIdx.x) >> 6;
  const int U = k.D / 8, slots = 64 / U;
  const int slot = lane / U, u = lane - slot * U;
  const int P = k.pairs;
  // no barrier below: waves are on their own
  for (int64_t job = int64_t(blockIdx.x) * 4 + w; job < k.T * k.split; job += int64_t(gridDim.x) * 4) {
  const int64_t tok = job / k.split;
  const int part = int(job - tok * k.split);
  for (int i = lane; i < P; i += 64) {
    int ax = 0;
    while (ax < k.axes - 1 && i >= k.end[ax]) ++ax;
    const double pos = k.pos_f32 ? double(static_cast<const float*>(k.pos)[tok * k.axes + ax])
                                 : double(static_cast<const int32_t*>(k.pos)[tok * k.axes + ax]);
    float s, c;
    turn_sincos(pos, k.freqs[i], &s, &c);
    cs[w][0][i] = c;
    cs[w][1][i] = k.inverse ? -s : s;
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  // the unit's channels: 8 neighbours, or 4 of each half and, behind them, 8 that pass
  const int NU = P / 4;               // units with pairs
  const bool turns = u < NU;
  const int o0 = HALVES && turns ? 4 * u : 8 * u;
  const int o1 = HALVES && turns ? P + 4 * u : 8 * u + 4;
  float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (turns) {
    load4(&cs[w][0][4 * u], c);
    load4(&cs[w][1][4 * u], s);
  }
  const int heads = k.Hq + k.Hk;
  const int per = (heads + slots * k.split - 1) / (slots * k.split);   // turns of each part
  const TE* const x = static_cast<const TE*>(k.x) + tok * k.ldx;
  TY* const y = static_cast<TY*>(k.y) + tok * k.ldy;
  const float inv = 1.0f / float(k.D);
  for (int it = 0; it < per; ++it) {
    const int head = (part * per + it) * slots + slot;
    const bool live = slot < slots && head < heads;
    float v[8] = {};
    if (live) {
      load4(x + head * k.D + o0, v);
      load4(x + head * k.D + o1, v + 4);
    }
    if (k.norm) {
      float q = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(v[e], v[e], q);
      q = run_sum(q, slot * U, U, u);
      const float rstd = 1.0f / sqrtf(q * inv + k.eps);
      if (live) {
        const float* const ga = head < k.Hq ? k.gamma_q : k.gamma_k;
        float g[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        if (ga) {
          load4(ga + o0, g);
          load4(ga + o1, g + 4);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * g[e];
      }
    }
    if (!live) continue;
    if (turns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ia = HALVES ? e : 2 * e, ib = HALVES ? 4 + e : 2 * e + 1;
        const float a = v[ia], b = v[ib];
        v[ia] = a * c[e] - b * s[e];
        v[ib] = b * c[e] + a * s[e];
      }
    }
    store4(y + head * k.D + o0, v);
    store4(y + head * k.D + o1, v + 4);
  }
  }
}

namespace {

template <typename TE, typename TY>
hipError_t launch_rope_typed(RopeArgs a, hipStream_t s) {
  // few tokens: their heads are shared among up to 8 waves
  const int turns = (a.Hq + a.Hk + 64 / (a.D / 8) - 1) / (64 / (a.D / 8));
  a.split = int(std::max<int64_t>(1, std::min<int64_t>(std::min(turns, 8), 2048 / a.T)));
  const int64_t waves = a.T * a.split;
  const dim3 grid(unsigned(std::min<int64_t>((waves + 3) / 4, 1 << 20)));
  if (a.halves) hipLaunchKernelGGL((rope_kernel<TE, TY, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((rope_kernel<TE, TY, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  if (a.x_bf16) return a.y_bf16 ? launch_rope_typed<uint16_t, uint16_t>(a, s)
                                : launch_rope_typed<uint16_t, float>(a, s);
  return a.y_bf16 ? launch_rope_typed<float, uint16_t>(a, s) : launch_rope_typed<float, float>(a, s);
}

}  // namespace hq
