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

// Sum over the runs of n lanes (n uniform, up to 32) that a wave's heads take, in one
// fixed order; pos is the lane's place in its run, first the run's first lane.
__device__ __forceinline__ float run_sum(float v, int first, int n, int pos) {
  switch (n) {
    case 1: return v;
    case 2: return group_sum<2>(v);
    case 4: return group_sum<4>(v);
    case 8: return group_sum<8>(v);
    case 16: return group_sum<16>(v);
    case 32: return group_sum<32>(v);
  }
  for (int d = 16; d >= 1; d >>= 1) {
    if (d >= n) continue;
    const float o = __shfl(v, first + pos + d, 64);
    if (pos + d < n && pos < d) v += o;
  }
  return __shfl(v, first, 64);
}

// A unit's eight channels as loaded: neighbours, or four of each half.
template <typename TE, bool SPLIT>
__device__ __forceinline__ Raw8<TE> unit_load(const TE* p, uint32_t o0, uint32_t o1) {
  if constexpr (!SPLIT) {
    return raw_load(p + o0);
  } else if constexpr (sizeof(TE) == 2) {
    const uint2 a = *reinterpret_cast<const uint2*>(p + o0), b = *reinterpret_cast<const uint2*>(p + o1);
    Raw8<TE> r;
    r.q[0] = make_uint4(a.x, a.y, b.x, b.y);
    return r;
  } else {
    Raw8<TE> r;
    r.q[0] = *reinterpret_cast<const uint4*>(p + o0);
    r.q[1] = *reinterpret_cast<const uint4*>(p + o1);
    return r;
  }
}

}  // namespace

// A wave per token and part of its heads (`split` parts per token); a head's D / 8 units
// of 8 channels go to D / 8 lanes, 64 / (D / 8) heads at a time, the next ones' loads in
// flight meanwhile (and the first ones' during the angles). 24576 tokens of 32 heads of 128
// bf16: 79 us, 5.1 TB/s; 8192 of 32 heads of 72, normed: 15.8 us, 4.8 TB/s (nine lanes a
// head, whose sums pass through LDS); three tokens of 40 heads: 4.2 us.
template <typename TE, typename TY, bool HALVES, bool NORM>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs k) {
  __shared__ __attribute__((aligned(16))) float cs[4][2][ROPE_MAX_PAIRS];
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int U = k.D / 8, slots = 64 / U;
  const int slot = lane / U, u = lane - slot * U;
  const int P = k.pairs;
  const int NU = P / 4;               // units with pairs
  const bool turns = u < NU;
  // the unit's channels: 8 neighbours, or 4 of each half and, behind them, 8 that pass
  const int o0 = HALVES && turns ? 4 * u : 8 * u;
  const int o1 = HALVES && turns ? P + 4 * u : 8 * u + 4;
  const int heads = k.Hq + k.Hk;
  const int per = (heads + slots * k.split - 1) / (slots * k.split);   // turns of each part
  const float inv = 1.0f / float(k.D);
  float gq[8], gk[8];
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < 8; ++e) gq[e] = gk[e] = 1.0f;
    if (k.gamma_q && slot < slots) {
      load4(k.gamma_q + o0, gq);
      load4(k.gamma_q + o1, gq + 4);
    }
    if (k.gamma_k && slot < slots) {
      load4(k.gamma_k + o0, gk);
      load4(k.gamma_k + o1, gk + 4);
    }
  }
  // no barrier: waves are on their own
  for (int64_t job = int64_t(blockIdx.x) * 4 + w; job < k.T * k.split; job += int64_t(gridDim.x) * 4) {
    const int64_t tok = k.split == 1 ? job : job / k.split;
    const int h0 = int(job - tok * k.split) * per * slots, h1 = min(h0 + per * slots, heads);
    const TE* const x = static_cast<const TE*>(k.x) + tok * k.ldx;
    TY* const y = static_cast<TY*>(k.y) + tok * k.ldy;
    Raw8<TE> next = {};
    int head = slot < slots ? h0 + slot : h1;
    if (head < h1) next = unit_load<TE, HALVES>(x + head * k.D, o0, o1);
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
    wave_lds_sync();
    float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (turns) {
      load4(&cs[w][0][4 * u], c);
      load4(&cs[w][1][4 * u], s);
    }
    wave_lds_sync();   // the next token's take their place
#pragma unroll 1
    for (int it = h0; it < h1; it += slots, head += slots) {
      float v[8];
      raw_get(next, v);
      if (head + slots < h1) next = unit_load<TE, HALVES>(x + (head + slots) * k.D, o0, o1);
      if constexpr (NORM) {
        float q = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(v[e], v[e], q);
        q = run_sum(q, slot * U, U, u);
        const float ms = fmaf(q, inv, k.eps);
        const bool large = ms == INFINITY;
        // rsq is off by one unit; eps keeps it from the smallest floats, which it does not take
        float rstd = __builtin_amdgcn_rsqf(ms);
        if (__any(large)) {   // squares past the largest float, or with eps: once more, of x 2^-80
          float z = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float t = v[e] * 0x1p-80f;
            z = fmaf(t, t, z);
            v[e] = large ? t : v[e];
          }
          z = run_sum(z, slot * U, U, u);
          if (large) rstd = 1.0f / sqrtf(fmaf(z, inv, k.eps * 0x1p-80f * 0x1p-80f));
        }
        const bool isq = head < k.Hq;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * (isq ? gq[e] : gk[e]);
      }
      if (head >= h1) continue;
      if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ia = HALVES ? e : 2 * e, ib = HALVES ? 4 + e : 2 * e + 1;
          const float a = v[ia], b = v[ib];
          v[ia] = a * c[e] - b * s[e];
          v[ib] = b * c[e] + a * s[e];
        }
      }
      TY* const out = y + head * k.D;
      if constexpr (HALVES) {
        store4(out + o0, v);
        store4(out + o1, v + 4);
      } else {
        store8(out + o0, v);
      }
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
  if (a.halves) {
    if (a.norm) hipLaunchKernelGGL((rope_kernel<TE, TY, true, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((rope_kernel<TE, TY, true, false>), grid, dim3(256), 0, s, a);
  } else {
    if (a.norm) hipLaunchKernelGGL((rope_kernel<TE, TY, false, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((rope_kernel<TE, TY, false, false>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  if (a.x_bf16) return a.y_bf16 ? launch_rope_typed<uint16_t, uint16_t>(a, s)
                                : launch_rope_typed<uint16_t, float>(a, s);
  return a.y_bf16 ? launch_rope_typed<float, uint16_t>(a, s) : launch_rope_typed<float, float>(a, s);
}

}  // namespace hq
