// Group norm over channels-last data [S samples, P positions, C channels], with
// an activation behind it (an unquantised layer between the low-bit ones):
//
//   y = phi(gamma_c (x - mean_sg) / sqrt(var_sg + eps) + beta_c),
//
// mean and (biased) variance over the P positions and the C / G channels of
// group g of sample s. Bound by memory: x has to be read once and y written
// once; the statistics need all of a group before its first output.
//
// Statistics never subtract large sums. A lane owns 8 consecutive channels
// (one 16- or 32-byte load per row) and takes, per channel, the mean of the
// rows in its registers and then the squares about that mean; batches, lanes
// and chunks are joined in a fixed tree by
//   mean = m_a + d n_b / n,   M2 = M2_a + M2_b + d^2 n_a n_b / n,   d = m_b - m_a,
// and the channels of a group by mean_g = avg m_c, M2_g = sum M2_c + n (m_c -
// mean_g)^2. Everything is fp32; groups need not be multiples of 8 channels
// wide, since channels meet only in the last step.
//
// Two forms (norm_plan):
//  norm_block_kernel   a block holds all positions of one sample's slab of
//                      whole groups in registers: one launch, x read once.
//  norm_stats_kernel + norm_apply_kernel
//                      chunks of positions; partial statistics in the
//                      workspace; the second pass finds x in the Infinity
//                      Cache where it fits.
#include "hq_epilogue.h"
#include "hq_internal.h"

namespace hq {

struct NormKArgs {
  const void* x;
  void* y;
  const float* gamma;   // [C] or NULL (ones)
  const float* beta;    // [C] or NULL (zeros)
  int64_t P;
  int C, G;
  float eps;
  int y_bf16;
  ActCoef act;
  float2* part;         // [S, G, chunks] (mean, M2)
  int chunks;
  int64_t rpc;          // rows per chunk
  int slab;             // channels per block (norm_block_kernel)
};

// Eight channels as loaded.
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

// Running statistics of 8 channels over n rows.
struct Stat8 {
  float n, mean[8], m2[8];
};
__device__ __forceinline__ void stat_merge(Stat8& a, float nb, const float mb[8], const float m2b[8]) {
  if (nb == 0.0f) return;
  const float nt = a.n + nb, r = nb / nt, w = a.n * r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = mb[e] - a.mean[e];
    a.mean[e] = fmaf(d, r, a.mean[e]);
    a.m2[e] += fmaf(d * d, w, m2b[e]);
  }
  a.n = nt;
}

// The statistics of the first `n` of the R rows in `x` (n uniform in nothing:
// each lane its own), merged into `a`.
template <typename TE, int R>
__device__ __forceinline__ void stat_rows(Stat8& a, const Raw8<TE> (&x)[R], int n) {
  if (n <= 0) return;
  float m[8] = {0, 0, 0, 0, 0, 0, 0, 0}, q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float v[8];
      raw_get(x[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] += v[e];
    }
  }
  const float inv = 1.0f / float(n);
#pragma unroll
  for (int e = 0; e < 8; ++e) m[e] *= inv;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float v[8];
      raw_get(x[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = v[e] - m[e];
        q[e] = fmaf(d, d, q[e]);
      }
    }
  }
  stat_merge(a, float(n), m, q);
}

// Joins the statistics of the block's RY row lanes (ty) for each of the VR
// channel vectors (tx): halves the lanes until lane 0 has all, the upper part
// of each step through LDS. sm: NT 17-float slots. Leaves the per-channel
// means in sm[0 .. 8 VR) and M2 in sm[8 VR .. 16 VR) (after a barrier).
template <int NT>
__device__ __forceinline__ void stat_tree(Stat8& a, float* sm, int tx, int ty, int VR, int RY,
                                          bool live) {
  float* const slot = sm + (ty * VR + tx) * 17;   // odd pitch: lanes hit distinct banks
  int n = RY;
  while (n > 1) {
    const int h = (n + 1) >> 1;
    if (live && ty >= h && ty < n) {
      slot[16] = a.n;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        slot[e] = a.mean[e];
        slot[8 + e] = a.m2[e];
      }
    }
    __syncthreads();
    if (live && ty < n - h) {
      const float* o = slot + h * VR * 17;
      float mb[8], qb[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mb[e] = o[e];
        qb[e] = o[8 + e];
      }
      stat_merge(a, o[16], mb, qb);
    }
    n = h;
  }
  __syncthreads();
  if (live && ty == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sm[8 * tx + e] = a.mean[e];
      sm[8 * VR + 8 * tx + e] = a.m2[e];
    }
  }
  __syncthreads();
}

// Sum over aligned runs of `lanes` (a power of two up to 64) lanes.
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ int pow2_at_least(int n, int most) {
  int l = 1;
  while (l < n && l < most) l <<= 1;
  return l;
}

// Group statistics from per-channel ones (cm, cq: channel means and M2 over n
// rows each): calls out(g, mean, M2) once per group.
template <int NT, typename F>
__device__ __forceinline__ void group_stats(const float* cm, const float* cq, int groups, int cg,
                                            float n, F out) {
  const int lg = pow2_at_least(cg, 64);
  const int l = threadIdx.x & (lg - 1);
  const float inv = 1.0f / float(cg);
  for (int g = threadIdx.x / lg; g < groups; g += NT / lg) {
    float s = 0.0f;
    for (int c = l; c < cg; c += lg) s += cm[g * cg + c];
    const float mean = lanes_sum(s, lg) * inv;
    float q = 0.0f;
    for (int c = l; c < cg; c += lg) {
      const float d = cm[g * cg + c] - mean;
      q += fmaf(n * d, d, cq[g * cg + c]);
    }
    q = lanes_sum(q, lg);
    if (l == 0) out(g, mean, q);
  }
}

// y of one row's 8 channels: (x - mean) a + b, phi, one rounding.
__device__ __forceinline__ void norm_store(const float v[8], const float mean[8], const float a[8],
                                           const float b[8], const NormKArgs& k, int64_t off) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fmaf(v[e] - mean[e], a[e], b[e]);
  if (k.y_bf16) {
    apply_act<8, false>(y, k.act);
    store8(static_cast<uint16_t*>(k.y) + off, y);
  } else {
    apply_act<8, true>(y, k.act);
    store8(static_cast<float*>(k.y) + off, y);
  }
}

// Per-lane coefficients of channels c0 .. c0+7 (c0 counted from the block's
// first channel cb): mean, gamma rstd, beta. gm / gr: the groups' means and
// 1 / sqrt(var + eps), from the block's first group.
__device__ __forceinline__ void norm_coef(const NormKArgs& k, int cb, int c0, int cg,
                                          const float* gm, const float* gr, float mean[8],
                                          float a[8], float b[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int g = (c0 + e) / cg;
    mean[e] = gm[g];
    a[e] = gr[g] * (k.gamma ? k.gamma[cb + c0 + e] : 1.0f);
    b[e] = k.beta ? k.beta[cb + c0 + e] : 0.0f;
  }
}

// ---- one launch -------------------------------------------------------------------

constexpr int NORM_BLOCK_GROUPS = 512;   // groups per slab at most

// Block (slab, sample): R rows per lane in registers.
template <typename TE, int NT, int R>
__global__ __launch_bounds__(NT) void norm_block_kernel(NormKArgs k) {
  __shared__ float sm[NT * 17];
  __shared__ float gm[NORM_BLOCK_GROUPS], gr[NORM_BLOCK_GROUPS];
  const int nslab = (k.C + k.slab - 1) / k.slab;
  const int64_t s = blockIdx.x / nslab;
  const int cb = int(blockIdx.x - s * nslab) * k.slab;
  const int nc = (k.C - cb) < k.slab ? (k.C - cb) : k.slab;
  const int VR = nc / 8, RY = NT / VR, cg = k.C / k.G;
  const int ty = int(threadIdx.x) / VR, tx = int(threadIdx.x) - ty * VR;
  const bool live = ty < RY;
  const int64_t base = s * k.P * k.C + cb + 8 * tx;
  const TE* const x = static_cast<const TE*>(k.x);
  Raw8<TE> v[R];
  int n = 0;   // rows ty, ty + RY, ... of this lane
  if (live && ty < k.P) n = int((k.P - ty + RY - 1) / RY);
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < n) v[i] = raw_load(x + base + int64_t(ty + i * RY) * k.C);
  Stat8 a = {};
  stat_rows<TE, R>(a, v, n);
  stat_tree<NT>(a, sm, tx, ty, VR, RY, live);
  const float inv = 1.0f / (float(k.P) * float(cg));
  group_stats<NT>(sm, sm + 8 * VR, nc / cg, cg, float(k.P), [&](int g, float mean, float m2) {
    gm[g] = mean;
    gr[g] = 1.0f / sqrtf(fmaf(m2, inv, k.eps));
  });
  __syncthreads();
  if (!live) return;
  float mean[8], ca[8], cbeta[8];
  norm_coef(k, cb, 8 * tx, cg, gm, gr, mean, ca, cbeta);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float f[8];
      raw_get(v[i], f);
      norm_store(f, mean, ca, cbeta, k, base + int64_t(ty + i * RY) * k.C);
    }
  }
}

// ---- two launches -----------------------------------------------------------------

// Partial statistics of chunk c of sample s (block s chunks + c).
template <typename TE, int NT>
__global__ __launch_bounds__(NT) void norm_stats_kernel(NormKArgs k) {
  constexpr int R = 8;
  __shared__ float sm[NT * 17];
  const int64_t s = blockIdx.x / k.chunks;
  const int c = int(blockIdx.x - s * k.chunks);
  const int64_t r0 = int64_t(c) * k.rpc;
  const int rows = int((k.P - r0) < k.rpc ? (k.P - r0) : k.rpc);
  const int VR = k.C / 8, RY = NT / VR, cg = k.C / k.G;
  const int ty = int(threadIdx.x) / VR, tx = int(threadIdx.x) - ty * VR;
  const bool live = ty < RY;
  const TE* const x = static_cast<const TE*>(k.x) + (s * k.P + r0) * k.C + 8 * tx;
  Stat8 a = {};
  if (live) {
    for (int r = ty; r < rows; r += R * RY) {
      Raw8<TE> v[R];
      const int n = (rows - r + RY - 1) / RY;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) v[i] = raw_load(x + int64_t(r + i * RY) * k.C);
      stat_rows<TE, R>(a, v, n < R ? n : R);
    }
  }
  stat_tree<NT>(a, sm, tx, ty, VR, RY, live);
  group_stats<NT>(sm, sm + 8 * VR, k.G, cg, float(rows), [&](int g, float mean, float m2) {
    k.part[(s * k.G + g) * k.chunks + c] = make_float2(mean, m2);
  });
}

// Joins the chunks' statistics (every block for its sample), then normalises
// rows [rpb b, rpb (b + 1)) of the sample.
template <typename TE, int NT>
__global__ __launch_bounds__(NT) void norm_apply_kernel(NormKArgs k, int bps, int64_t rpb) {
  constexpr int R = 4;
  constexpr int MAXG = NT == 256 ? 2048 : NORM_MAX_C;   // G <= C, C <= 2048 with 256 threads
  __shared__ float gm[MAXG], gr[MAXG];
  const int64_t s = blockIdx.x / bps;
  const int64_t r0 = int64_t(int(blockIdx.x - s * bps)) * rpb;
  const int rows = int((k.P - r0) < rpb ? (k.P - r0) : rpb);
  const int cg = k.C / k.G;
  const int lq = pow2_at_least(k.chunks, 64);
  const int l = threadIdx.x & (lq - 1);
  const float inv = 1.0f / (float(k.P) * float(cg));
  for (int g = threadIdx.x / lq; g < k.G; g += NT / lq) {
    const float2* p = k.part + (s * k.G + g) * k.chunks;
    float sum = 0.0f;
    for (int c = l; c < k.chunks; c += lq) {
      const int64_t left = k.P - int64_t(c) * k.rpc;
      sum = fmaf(p[c].x, float(left < k.rpc ? left : k.rpc), sum);
    }
    const float mean = lanes_sum(sum, lq) / float(k.P);
    float q = 0.0f;
    for (int c = l; c < k.chunks; c += lq) {
      const int64_t left = k.P - int64_t(c) * k.rpc;
      const float2 v = p[c];
      const float d = v.x - mean;
      q += fmaf(d * d, float(left < k.rpc ? left : k.rpc) * float(cg), v.y);
    }
    q = lanes_sum(q, lq);
    if (l == 0) {
      gm[g] = mean;
      gr[g] = 1.0f / sqrtf(fmaf(q, inv, k.eps));
    }
  }
  __syncthreads();
  const int VR = k.C / 8, RY = NT / VR;
  const int ty = int(threadIdx.x) / VR, tx = int(threadIdx.x) - ty * VR;
  if (ty >= RY) return;
  float mean[8], ca[8], cbeta[8];
  norm_coef(k, 0, 8 * tx, cg, gm, gr, mean, ca, cbeta);
  const int64_t base = (s * k.P + r0) * k.C + 8 * tx;
  const TE* const x = static_cast<const TE*>(k.x) + base;
  for (int r = ty; r < rows; r += R * RY) {
    Raw8<TE> v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (r + i * RY < rows) v[i] = raw_load(x + int64_t(r + i * RY) * k.C);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r + i * RY < rows) {
        float f[8];
        raw_get(v[i], f);
        norm_store(f, mean, ca, cbeta, k, base + int64_t(r + i * RY) * k.C);
      }
    }
  }
}

// ---- host side ----------------------------------------------------------------------

namespace {

struct NormPlan {
  int block;         // 1: norm_block_kernel
  int nt, r, slab;   // its threads, rows per lane and channels per block
  int chunks;        // two launches: chunks per sample and their rows
  int64_t rpc;
  int bps;           // apply blocks per sample and their rows
  int64_t rpb;
};

int gcd_i(int a, int b) { return b ? gcd_i(b, a % b) : a; }

// Slabs are whole groups and whole 8-channel vectors: multiples of `unit` =
// lcm(C / G, 8) channels, taken until a row's piece is a 128-byte line, then
// doubled while all positions still are one pass of 256 lanes.
NormPlan norm_plan(int64_t S, int64_t P, int C, int G, int esize) {
  NormPlan p = {};
  const int cg = C / G, unit = cg / gcd_i(cg, 8) * 8;
  int slab = unit;
  while (slab * esize < 128 && slab < C) slab += unit;
  while (slab < C && P * slab / 4 <= 256 && 2 * slab / cg <= NORM_BLOCK_GROUPS) slab *= 2;
  if (slab > C) slab = C;
  for (int nt : {256, 1024}) {
    const int VR = slab / 8;
    if (VR > nt || slab / cg > NORM_BLOCK_GROUPS) continue;
    const int RY = nt / VR;
    const int64_t need = (P + RY - 1) / RY;
    if (need <= 8) {
      p.block = 1;
      p.nt = nt;
      p.slab = slab;
      p.r = need <= 2 ? 2 : 8;
      return p;
    }
  }
  p.nt = C <= 2048 ? 256 : 1024;
  if (S * P * C >= int64_t(1) << 22) p.nt = 1024;
  const int RY = p.nt / (C / 8);
  int64_t want = (512 + S - 1) / S;                       // about two blocks per CU
  const int64_t most = (P + RY * 8 - 1) / (RY * 8);       // at least 8 rows per lane
  if (want > most) want = most;
  if (want > 256) want = 256;
  if (want < 1) want = 1;
  p.rpc = (P + want - 1) / want;
  p.chunks = int((P + p.rpc - 1) / p.rpc);
  p.rpb = p.rpc;
  p.bps = p.chunks;
  return p;
}

template <typename TE>
hipError_t launch_norm_typed(const NormPlan& p, const NormKArgs& k, int64_t S, hipStream_t s) {
  if (p.block) {
    const dim3 grid(unsigned(S * ((k.C + p.slab - 1) / p.slab)));
    if (p.nt == 256 && p.r == 2)
      hipLaunchKernelGGL((norm_block_kernel<TE, 256, 2>), grid, dim3(256), 0, s, k);
    else if (p.nt == 256)
      hipLaunchKernelGGL((norm_block_kernel<TE, 256, 8>), grid, dim3(256), 0, s, k);
    else if (p.r == 2)
      hipLaunchKernelGGL((norm_block_kernel<TE, 1024, 2>), grid, dim3(1024), 0, s, k);
    else
      hipLaunchKernelGGL((norm_block_kernel<TE, 1024, 8>), grid, dim3(1024), 0, s, k);
    return hipGetLastError();
  }
  const dim3 g1(unsigned(S * p.chunks)), g2(unsigned(S * p.bps));
  if (p.nt == 256) {
    hipLaunchKernelGGL((norm_stats_kernel<TE, 256>), g1, dim3(256), 0, s, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((norm_apply_kernel<TE, 256>), g2, dim3(256), 0, s, k, p.bps, p.rpb);
  } else {
    hipLaunchKernelGGL((norm_stats_kernel<TE, 1024>), g1, dim3(1024), 0, s, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((norm_apply_kernel<TE, 1024>), g2, dim3(1024), 0, s, k, p.bps, p.rpb);
  }
  return hipGetLastError();
}

}  // namespace

size_t norm_part_bytes(int64_t S, int64_t P, int C, int G, int esize) {
  if (S <= 0 || P <= 0) return 0;
  const NormPlan p = norm_plan(S, P, C, G, esize);
  return p.block ? 0 : sizeof(float2) * size_t(S) * size_t(G) * size_t(p.chunks);
}

hipError_t launch_group_norm(const NormArgs& a, int64_t S, hipStream_t s) {
  const NormPlan p = norm_plan(S, a.P, a.C, a.G, a.x_bf16 ? 2 : 4);
  NormKArgs k = {};
  k.x = a.x;
  k.y = a.y;
  k.gamma = a.gamma;
  k.beta = a.beta;
  k.P = a.P;
  k.C = a.C;
  k.G = a.G;
  k.eps = a.eps;
  k.y_bf16 = a.y_bf16;
  k.act = a.act;
  k.part = static_cast<float2*>(a.part);
  k.chunks = p.chunks;
  k.rpc = p.rpc;
  k.slab = p.slab;
  return a.x_bf16 ? launch_norm_typed<uint16_t>(p, k, S, s) : launch_norm_typed<float>(p, k, S, s);
}

}  // namespace hq
