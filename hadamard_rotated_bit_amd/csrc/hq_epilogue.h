// Epilogue of a linear layer beyond its bias: y = r + g phi(v), shared by the
// dense and the quantised products and (phi alone) by the group norm.
//   v  the product with its bias, in fp32
//   phi identity, ReLU max(x, 0), SiLU x / (1 + e^-x), GELU x Phi(x) (Gaussian
//      CDF) or its tanh form x / (1 + e^-2u), u = sqrt(2/pi) (x + 0.044715 x^3)
//   g  one row of [*, N] per gate_rows rows of the output (absent: 1)
//   r  the residual [M, N] (absent: 0)
// Everything is computed in fp32 and rounded once, when y is stored.
#pragma once

#include "hq_device.h"
#include "hq_gemm_types.h"

namespace hq {

__device__ __forceinline__ float relu_f32(float x) { return x < 0.0f ? 0.0f : x; }  // keeps NaN

// SiLU, GELU and its tanh form are all x / (1 + 2^(x P(x^2))): P is the
// constant -log2(e) for SiLU (DEG 0) and linear for the tanh form (DEG 1), and
// for GELU with a bf16 result (DEG 6) the fit of -log2(Phi(x) / Phi(-x)) / x on
// |x| <= 5 (relative error of phi at most 1.1e-4 there: 1/37 to 1/18 of a bf16
// half step, which is 2^-8 to 2^-9 of the value; beyond, x^2 is held at 25 and phi
// differs from x or 0 by less than 1.5e-5 in absolute value). The exponent x P
// carries about two (DEG 0) to five (DEG 1) fp32 roundings, each |x P| 2^-24 ln 2 of
// the result where x < 0. One exp2 and one reciprocal per value;
// the degree is fixed per loop, as the exponent's terms are what the vector
// ALU spends on it.
template <int DEG>
__device__ __forceinline__ float act_sigmoid(float x, const ActCoef& a) {
  float p = a.c[DEG];
  if constexpr (DEG == 1) p = fmaf(p, x * x, a.c[0]);   // an infinite square saturates as it should
  if constexpr (DEG > 1) {
    const float t = fminf(x * x, a.tmax);
#pragma unroll
    for (int k = DEG - 1; k >= 0; --k) p = fmaf(p, t, a.c[k]);
  }
  return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * p));
}

// GELU for an fp32 result: max(x, 0) - |x| h(|x|), h(a) = Phi(-a) =
// e^(-a^2/2) times a degree-10 fit in t = 1 / (1 + 0.4 a) (relative error
// 1.4e-8); no difference of near-equal numbers for any x. a^2 / 2 carries three
// roundings, each a^2 / 2 x 2^-24 of h. a is held at 40,
// where h is 0 in fp32, so that +-inf give inf and 0.
__device__ __forceinline__ float gelu_full(float x) {
  const float a = fminf(fabsf(x), 40.0f);
  const float d = fmaf(0.4f, a, 1.0f);
  float t = __builtin_amdgcn_rcpf(d);
  t = fmaf(t, fmaf(-d, t, 1.0f), t);
  float p = 0.031375720731075134f;
  p = fmaf(p, t, -0.17226340215955868f);
  p = fmaf(p, t, 0.3716291512061377f);
  p = fmaf(p, t, -0.3598523486270329f);
  p = fmaf(p, t, 0.1077760623043252f);
  p = fmaf(p, t, -0.020622834591990737f);
  p = fmaf(p, t, 0.08922175130220084f);
  p = fmaf(p, t, 0.133581291732006f);
  p = fmaf(p, t, 0.15957620720558505f);
  p = fmaf(p, t, 0.15957840770412896f);
  const float h = p * t * __builtin_amdgcn_exp2f(-0.72134752044448170f * a * a);
  return fmaf(-a, h, relu_f32(x));
}

// phi on N values; FULL: fp32 result. `act` is uniform over the launch.
template <int N, bool FULL>
__device__ __forceinline__ void apply_act(float (&v)[N], const ActCoef& a) {
  if (a.act == ACT_NONE) return;
  if (a.act == ACT_RELU) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = relu_f32(v[k]);
    return;
  }
  if (a.act == ACT_SILU) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = act_sigmoid<0>(v[k], a);
  } else if (a.act == ACT_GELU_TANH) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = act_sigmoid<1>(v[k], a);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = FULL ? gelu_full(v[k]) : act_sigmoid<6>(v[k], a);
  }
}

// Eight consecutive elements as loaded.
template <typename TE>
struct Raw8 {
  uint4 q[sizeof(TE) / 2];
};
template <typename TE>
__device__ __forceinline__ Raw8<TE> raw_load(const TE* p) {
  Raw8<TE> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(TE) / 2; ++i) r.q[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void raw_get(const Raw8<uint16_t>& r, float v[8]) {
  load8(reinterpret_cast<const uint16_t*>(&r.q[0]), v);
}
__device__ __forceinline__ void raw_get(const Raw8<float>& r, float v[8]) {
  load8(reinterpret_cast<const float*>(&r.q[0]), v);
}

__device__ __forceinline__ void store8(float* __restrict__ p, const float v[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* __restrict__ p, const float v[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Q pieces of eight consecutive outputs each (columns n[q] .. n[q] + 7, n a
// multiple of 8, of row m[q]; ok[q]: inside the output) from v, the product with
// its bias: phi, gate, residual, one rounding, one 16- or 32-byte store. All
// loads come before the first store: Y may be the residual's own buffer, so the
// compiler cannot move a later piece's loads above an earlier one's store, and
// each piece would wait for its own residual. Every element is read by the lane
// that writes it.
template <typename TY, int Q>
__device__ __forceinline__ void finish8(float (&v)[Q][8], const int64_t (&m)[Q],
                                        const int64_t (&n)[Q], const bool (&ok)[Q], int64_t N,
                                        const LinEpi& ep) {
  Raw8<TY> r[Q], g[Q];
  if (ep.residual) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (ok[q]) r[q] = raw_load(static_cast<const TY*>(ep.residual) + m[q] * N + n[q]);
  }
  if (ep.gate) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (ok[q])
        g[q] = raw_load(static_cast<const TY*>(ep.gate) +
                        int64_t(uint32_t(m[q]) / uint32_t(ep.gate_rows)) * ep.gate_ld + n[q]);
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (!ok[q]) continue;
    float t[8];
    apply_act<8, sizeof(TY) == 4>(v[q], ep.act);
    if (ep.gate) {
      raw_get(g[q], t);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[q][k] *= t[k];
    }
    if (ep.residual) {
      raw_get(r[q], t);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[q][k] += t[k];
    }
    store8(static_cast<TY*>(ep.Y) + m[q] * N + n[q], v[q]);
  }
}

// One piece: eight consecutive outputs n .. n+7 of row m.
__device__ __forceinline__ void finish_piece(const float (&v)[8], int64_t m, int64_t n, int64_t N,
                                             const LinEpi& ep) {
  float a[1][8];
#pragma unroll
  for (int k = 0; k < 8; ++k) a[0][k] = v[k];
  const int64_t am[1] = {m}, an[1] = {n};
  const bool ok[1] = {true};
  if (ep.y_bf16) finish8<uint16_t, 1>(a, am, an, ok, N, ep);
  else finish8<float, 1>(a, am, an, ok, N, ep);
}

// A wave's 32 rows x (8 LPR) columns, staged as fp32 rows of `pitch` floats, as
// rows again: eight consecutive columns per lane, whole row segments per store,
// Q pieces at a time. Rows from m0, columns from n0.
template <typename TY, int LPR, int Q>
__device__ __forceinline__ void finish_rows_as(const float* stg, int pitch, int lane, int64_t m0,
                                               int64_t n0, int64_t M, int64_t N, const LinEpi& ep) {
  constexpr int NQ = 32 * LPR / 64;             // pieces per lane
  static_assert(NQ % Q == 0, "whole groups");
#pragma unroll 1
  for (int q0 = 0; q0 < NQ; q0 += Q) {
    float v[Q][8];
    int64_t m[Q], n[Q];
    bool ok[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = lane + 64 * (q0 + q), r = i / LPR, c = 8 * (i - r * LPR);
      m[q] = m0 + r;
      n[q] = n0 + c;
      ok[q] = m[q] < M && n[q] < N;
      load8(stg + r * pitch + c, v[q]);
    }
    finish8<TY, Q>(v, m, n, ok, N, ep);
  }
}
// Q: pieces at a time for bf16 results, what the kernel's registers leave room
// for; fp32 ones take half as many.
template <int LPR, int Q>
__device__ __forceinline__ void finish_rows(const float* stg, int pitch, int lane, int64_t m0,
                                            int64_t n0, int64_t M, int64_t N, const LinEpi& ep) {
  if (ep.y_bf16)
    finish_rows_as<uint16_t, LPR, Q>(stg, pitch, lane, m0, n0, M, N, ep);
  else
    finish_rows_as<float, LPR, Q % 2 ? 1 : Q / 2>(stg, pitch, lane, m0, n0, M, N, ep);
}

// One output, the same steps.
template <typename TY>
__device__ __forceinline__ void finish1_as(float v, int64_t m, int64_t n, int64_t N,
                                           const LinEpi& ep) {
  auto val = [](const void* p, int64_t i) -> float {
    if constexpr (sizeof(TY) == 4) return static_cast<const float*>(p)[i];
    else return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  };
  float a[1] = {v + (ep.bias ? ep.bias[n] : 0.0f)};
  apply_act<1, sizeof(TY) == 4>(a, ep.act);
  if (ep.gate) a[0] *= val(ep.gate, (m / ep.gate_rows) * ep.gate_ld + n);
  if (ep.residual) a[0] += val(ep.residual, m * N + n);
  if constexpr (sizeof(TY) == 4) static_cast<float*>(ep.Y)[m * N + n] = a[0];
  else static_cast<uint16_t*>(ep.Y)[m * N + n] = f32_to_bf16(a[0]);
}
__device__ __forceinline__ void finish1(float v, int64_t m, int64_t n, int64_t N, const LinEpi& ep) {
  if (ep.y_bf16) finish1_as<uint16_t>(v, m, n, N, ep);
  else finish1_as<float>(v, m, n, N, ep);
}

}  // namespace hq
