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
// (one 16- or 32-byte load per row) and takes, per unit of channels that share
// a group, the mean of the rows in its registers and then the squares about
// that mean; batches and lanes are joined in a fixed tree by
//   mean = m_a + d n_b / n,   M2 = M2_a + M2_b + d^2 n_a n_b / n,   d = m_b - m_a,
// and the units of a group, and its chunks, by mean_g = avg m_u, M2_g = sum M2_u +
// n (m_u - mean_g)^2. An average rounds, by several units in sums of many values, so
// each one, m', is followed by the sum s1 of the n differences from it beside that of
// their squares: mean = m' + s1 / n, M2 = s2 - s1^2 / n. A group of equal values then
// has exactly their value as its mean. Everything is fp32; groups may have any width.
//
// Forms (norm_plan):
//  norm_rows_kernel    one position, groups of whole 8-channel pieces: a wave or
//                      a part of one holds a group (8192 rows of 1152 bf16: 10.0
//                      us, 3.8 TB/s, fp32 15.1 us, 5.0 TB/s, against 21.9 and 21.8
//                      with a block per row; 8192 x 18 groups of 64: 9.9 us
//                      against 21.1).
//  norm_block_kernel   a block holds all positions of one sample's slab of
//                      whole groups in registers: one launch, x read once.
//  norm_stats_kernel (+ norm_join_kernel) + norm_apply_kernel
//                      chunks of positions; partial statistics in the
//                      workspace; the second pass finds x in the caches
//                      where it fits.
#include "hq_epilogue.h"
#include "hq_internal.h"

#include <algorithm>

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
  float2* part;         // [S, G, chunks] (mean, M2), then [S, G] joined
  int chunks;
  int64_t rpc;          // rows per chunk
  int slab;             // channels per block (norm_block_kernel)
};

// A lane's 8 channels are taken in units of U = gcd(C / G, 8) channels: a unit
// lies within one group, so its channels share one mean and one M2 (NS = 8 / U
// of them per lane: 1 where the group width is a multiple of 8, 4 at 10).
// Running statistics of a lane's units over n values each.
template <int NS>
struct Stat {
  float n, mean[NS], m2[NS];
};
template <int NS>
__device__ __forceinline__ void stat_merge(Stat<NS>& a, float nb, const float (&mb)[NS],
                                           const float (&m2b)[NS]) {
  if (nb == 0.0f) return;
  const float nt = a.n + nb, r = nb / nt, w = a.n * r;
#pragma unroll
  for (int e = 0; e < NS; ++e) {
    const float d = mb[e] - a.mean[e];
    a.mean[e] = fmaf(d, r, a.mean[e]);
    a.m2[e] += fmaf(d * w, d, m2b[e]);   // in this order 0 where w is, also for a d^2 past the floats
  }
  a.n = nt;
}

// s2 - c, the sum of squares about a rounded mean less its correction c = s1^2 / n
// (no larger than s2 but for roundings). An s2 past the largest float stays infinite.
__device__ __forceinline__ float about_mean(float s2, float c) {
  return c < s2 ? s2 - c : s2 < INFINITY ? 0.0f : s2;   // NaN stays
}

// The statistics of the first `n` of the R rows in `x` (each lane its own n),
// merged into `a`.
template <typename TE, int U, int R>
__device__ __forceinline__ void stat_rows(Stat<8 / U>& a, Raw8<TE> (&x)[R], int n) {
  constexpr int NS = 8 / U;
  if (n <= 0) return;
  float m[NS] = {}, s[NS] = {}, q[NS] = {};
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float v[8];
      raw_get(x[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e / U] += v[e];
    }
  }
  const float nv = float(n * U), inv = 1.0f / nv;
#pragma unroll
  for (int e = 0; e < NS; ++e) m[e] *= inv;
  // the rows stay packed between the two passes (their floats, kept, would
  // take twice the registers of a batch)
  if constexpr (sizeof(TE) == 2) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      asm volatile("" : "+v"(x[i].q[0].x), "+v"(x[i].q[0].y), "+v"(x[i].q[0].z), "+v"(x[i].q[0].w));
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      float v[8];
      raw_get(x[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = v[e] - m[e / U];
        s[e / U] += d;
        q[e / U] = fmaf(d, d, q[e / U]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < NS; ++e) {
    const float c = s[e] * inv;
    m[e] += c;
    q[e] = about_mean(q[e], c * s[e]);
  }
  stat_merge<NS>(a, nv, m, q);
}

// Joins the statistics of the block's RY row lanes (ty) for each of the VR
// channel vectors (tx): halves the lanes until lane 0 has all, the upper part
// of each step through LDS (slots of an odd number of floats: lanes hit
// distinct banks). Leaves the units' means in sm[0 .. NS VR) and their M2
// behind them, after a barrier. sm: NT (2 NS + 1) floats.
template <int NS>
__device__ __forceinline__ void stat_tree(Stat<NS>& a, float* sm, int tx, int ty, int VR, int RY,
                                          bool live) {
  constexpr int PITCH = 2 * NS + 1;
  float* const slot = sm + (ty * VR + tx) * PITCH;
  int n = RY;
  while (n > 1) {
    const int h = (n + 1) >> 1;
    if (live && ty >= h && ty < n) {
      slot[2 * NS] = a.n;
#pragma unroll
      for (int e = 0; e < NS; ++e) {
        slot[e] = a.mean[e];
        slot[NS + e] = a.m2[e];
      }
    }
    __syncthreads();
    if (live && ty < n - h) {
      const float* o = slot + h * VR * PITCH;
      float mb[NS], qb[NS];
#pragma unroll
      for (int e = 0; e < NS; ++e) {
        mb[e] = o[e];
        qb[e] = o[NS + e];
      }
      stat_merge<NS>(a, o[2 * NS], mb, qb);
    }
    n = h;
  }
  __syncthreads();
  if (live && ty == 0) {
#pragma unroll
    for (int e = 0; e < NS; ++e) {
      sm[NS * tx + e] = a.mean[e];
      sm[NS * VR + NS * tx + e] = a.m2[e];
    }
  }
  __syncthreads();
}

// Sum over aligned runs of `lanes` (a power of two up to 64) lanes, on the
// VALU; `lanes` is uniform.
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  switch (lanes) {
    case 2: return group_sum<2>(v);
    case 4: return group_sum<4>(v);
    case 8: return group_sum<8>(v);
    case 16: return group_sum<16>(v);
    case 32: return group_sum<32>(v);
    case 64: return group_sum<64>(v);
    default: return v;
  }
}
__device__ __forceinline__ int pow2_at_least(int n, int most) {
  int l = 1;
  while (l < n && l < most) l <<= 1;
  return l;
}

// Group statistics from the units' (cm, cq: means and M2 over n values each;
// cu units per group): calls out(g, mean, M2) once per group.
template <int NT, typename F>
__device__ __forceinline__ void group_stats(const float* cm, const float* cq, int groups, int cu,
                                            float n, F out) {
  const int lg = pow2_at_least(cu, 64), sh = __builtin_ctz(lg);
  const int l = threadIdx.x & (lg - 1);
  const float inv = 1.0f / float(cu);
  for (int g = threadIdx.x >> sh; g < groups; g += NT >> sh) {
    float s = 0.0f;
    for (int c = l; c < cu; c += lg) s += cm[g * cu + c];
    const float mean = lanes_sum(s, lg) * inv;
    float s1 = 0.0f, q = 0.0f;
    for (int c = l; c < cu; c += lg) {
      const float d = cm[g * cu + c] - mean;
      s1 += d;
      q += fmaf(n * d, d, cq[g * cu + c]);
    }
    s1 = lanes_sum(s1, lg);
    q = lanes_sum(q, lg);
    if (l == 0) out(g, fmaf(s1, inv, mean), about_mean(q, n * (s1 * inv) * s1));
  }
}

__device__ __forceinline__ float rstd_of(float m2, const NormKArgs& k) {
  return 1.0f / sqrtf(m2 / (float(k.P) * float(k.C / k.G)) + k.eps);
}

// gamma and beta of channels c .. c+7.
__device__ __forceinline__ void load_affine(const NormKArgs& k, int c, float a[8], float b[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = 1.0f;
    b[e] = 0.0f;
  }
  if (k.gamma) load8(k.gamma + c, a);
  if (k.beta) load8(k.beta + c, b);
}

// A lane's coefficients, y = (x - mean) a + b with a = gamma rstd. The mean is
// not folded into b: a constant group (rstd = 1 / sqrt(eps)) then gives b
// exactly instead of a rounding of mean a.
struct Coef {
  float mean[8], a[8], b[8];
};
// c0: the lane's first channel counted from the first of gm / gr (the groups'
// means and reciprocal deviations); c.a, c.b hold gamma and beta.
__device__ __forceinline__ void coef_finish(Coef& c, int c0, int cg, const float* gm,
                                            const float* gr) {
  int g = c0 / cg, r = c0 - g * cg;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c.mean[e] = gm[g];
    c.a[e] *= gr[g];
    if (++r == cg) {
      r = 0;
      ++g;
    }
  }
}

// y of one row's 8 channels: phi, one rounding.
template <typename TE>
__device__ __forceinline__ void norm_store(const Raw8<TE>& x, const Coef& c, const NormKArgs& k,
                                           int64_t off) {
  float y[8];
  raw_get(x, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e] - c.mean[e], c.a[e], c.b[e]);
  if (k.y_bf16) {
    apply_act<8, false>(y, k.act);
    store8(static_cast<uint16_t*>(k.y) + off, y);
  } else {
    apply_act<8, true>(y, k.act);
    store8(static_cast<float*>(k.y) + off, y);
  }
}

// ---- one position -----------------------------------------------------------------

// One position per sample and groups of whole 8-channel pieces (G = 1 is layer
// norm, G heads a norm of each head): `rows` = S G rows of w = C / G channels, L
// lanes per row (64, or fewer for short rows: several rows per wave), R pieces of
// 8 channels per lane in registers, no LDS. The first sum gives a mean m', the
// second pass sums x - m' and its square and corrects both: mean = m' + s1 / w,
// M2 = s2 - s1^2 / w, so a rounded m' (or a constant row) leaves no trace. HOLD
// (G = 1): gamma and beta stay in registers over a wave's rows.
template <typename TE, int R, bool HOLD>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormKArgs k, int64_t rows, int L) {
  const int w = k.C / k.G, VR = w / 8;
  const int sub = int(threadIdx.x) & (L - 1), rpb = 256 / L;
  const float inv = 1.0f / float(w);
  auto sum = [&](float v) {   // rows of more than one piece per lane take whole waves
    if constexpr (R > 1) return group_sum<64>(v);
    else return lanes_sum(v, L);
  };
  Coef c[HOLD ? R : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (sub + 64 * i < VR) load_affine(k, 8 * (sub + 64 * i), c[i].a, c[i].b);
  }
  // the same number of turns for every lane of a wave: sums run over all lanes
  for (int64_t r0 = int64_t(blockIdx.x) * rpb; r0 < rows; r0 += int64_t(gridDim.x) * rpb) {
    const int64_t row = r0 + int(threadIdx.x) / L;
    const int nv = row < rows ? VR : 0;   // pieces of the lane's row
    const int64_t base = row * w + 8 * sub;
    const TE* const x = static_cast<const TE*>(k.x) + base;
    Raw8<TE> v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (sub + 64 * i < nv) v[i] = raw_load(x + 512 * i);
    float s0 = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (sub + 64 * i < nv) {
        float f[8];
        raw_get(v[i], f);
        s0 += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
      }
    }
    const float m0 = sum(s0) * inv;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (sub + 64 * i < nv) {
        float f[8];
        raw_get(v[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = f[e] - m0;
          s1 += d;
          s2 = fmaf(d, d, s2);
        }
      }
    }
    s1 = sum(s1);
    s2 = sum(s2);
    const float mean = fmaf(s1, inv, m0);
    const float rstd = rstd_of(fmaxf(fmaf(-s1 * inv, s1, s2), 0.0f), k);
    const int c0 = HOLD ? 0 : int(row % k.G) * w;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (sub + 64 * i >= nv) continue;
      Coef d;
      if constexpr (HOLD) d = c[i];
      else load_affine(k, c0 + 8 * (sub + 64 * i), d.a, d.b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d.mean[e] = mean;
        d.a[e] *= rstd;
      }
      norm_store<TE>(v[i], d, k, base + 512 * i);
    }
  }
}

// ---- one launch -------------------------------------------------------------------

constexpr int NORM_BLOCK_GROUPS = 512;   // groups per slab at most

// Block (slab, sample): R rows per lane in registers. Bound by the one read and
// write of its slab by as many CUs as there are slabs (8 x 1536 x 256 fp32, 128
// blocks: 13.9 us, 1.8 TB/s) and by the barriers of the tree (3 x 77 x 320: 6.4 us).
template <typename TE, int U, int NT, int R>
__global__ __launch_bounds__(NT) void norm_block_kernel(NormKArgs k) {
  constexpr int NS = 8 / U;
  __shared__ float sm[NT * (2 * NS + 1)];
  __shared__ float gm[NORM_BLOCK_GROUPS], gr[NORM_BLOCK_GROUPS];
  // slabs of a sample share its lines: on one XCD (block b runs on XCD b mod 8)
  // where the samples are a multiple of 8
  const uint32_t nslab = uint32_t(k.C + k.slab - 1) / uint32_t(k.slab);
  const uint32_t samples = gridDim.x / nslab;
  const bool by_xcd = samples % 8 == 0;
  const uint32_t major = blockIdx.x / (by_xcd ? samples : nslab);
  const uint32_t minor = blockIdx.x - major * (by_xcd ? samples : nslab);
  const uint32_t smp = by_xcd ? minor : major;
  const int cb = int(by_xcd ? major : minor) * k.slab;
  const int nc = (k.C - cb) < k.slab ? (k.C - cb) : k.slab;
  const int VR = nc / 8, RY = NT / VR, cg = k.C / k.G;
  const int ty = int(threadIdx.x) / VR, tx = int(threadIdx.x) - ty * VR;
  const bool live = ty < RY;
  const int P = int(k.P);
  const int64_t base = int64_t(smp) * k.P * k.C + cb + 8 * tx;
  const TE* const x = static_cast<const TE*>(k.x) + base;
  Raw8<TE> v[R];
  int n = 0;   // rows ty, ty + RY, ... of this lane
  if (live && ty < P) n = (P - ty + RY - 1) / RY;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < n) v[i] = raw_load(x + int64_t(ty + i * RY) * k.C);
  Coef c = {};
  if (live) load_affine(k, cb + 8 * tx, c.a, c.b);
  Stat<NS> a = {};
  stat_rows<TE, U, R>(a, v, n);
  stat_tree<NS>(a, sm, tx, ty, VR, RY, live);
  group_stats<NT>(sm, sm + NS * VR, nc / cg, cg / U, float(P) * float(U),
                  [&](int g, float mean, float m2) {
                    gm[g] = mean;
                    gr[g] = rstd_of(m2, k);
                  });
  __syncthreads();
  if (!live) return;
  coef_finish(c, 8 * tx, cg, gm, gr);
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i < n) norm_store<TE>(v[i], c, k, base + int64_t(ty + i * RY) * k.C);
}

// ---- two or three launches ----------------------------------------------------------

// Partial statistics of chunk c of sample s (block s chunks + c). A batch of
// rows is loaded before the one in registers is summed. 512 x 512 x 128 bf16
// (one sample of 2^18 positions): 16.8 us, 4.0 TB/s; norm_apply_kernel on the
// same: 20.4 us, 6.6 TB/s of reads and writes.
template <typename TE, int U, int NT>
__global__ __launch_bounds__(NT) void norm_stats_kernel(NormKArgs k) {
  constexpr int NS = 8 / U;
  constexpr int R = 16 / sizeof(TE);   // 8 or 4 rows: 32 registers
  __shared__ float sm[NT * (2 * NS + 1)];
  const uint32_t s = blockIdx.x / uint32_t(k.chunks);
  const int c = int(blockIdx.x - s * uint32_t(k.chunks));
  const int64_t r0 = int64_t(c) * k.rpc;
  const int rows = int((k.P - r0) < k.rpc ? (k.P - r0) : k.rpc);
  const int VR = k.C / 8, RY = NT / VR, cg = k.C / k.G;
  const int ty = int(threadIdx.x) / VR, tx = int(threadIdx.x) - ty * VR;
  const bool live = ty < RY;
  const TE* const x = static_cast<const TE*>(k.x) + (int64_t(s) * k.P + r0) * k.C + 8 * tx;
  Stat<NS> a = {};
  if (live) {
    Raw8<TE> v[2][R];
    auto fetch = [&](Raw8<TE> (&d)[R], int r) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (r + i * RY < rows) d[i] = raw_load(x + int64_t(r + i * RY) * k.C);
    };
    auto sum = [&](Raw8<TE> (&d)[R], int r) {
      const int n = (rows - r + RY - 1) / RY;
      stat_rows<TE, U, R>(a, d, n < R ? n : R);
    };
    fetch(v[0], ty);
    for (int r = ty; r < rows; r += 2 * R * RY) {
      fetch(v[1], r + R * RY);
      sum(v[0], r);
      if (r + R * RY < rows) {
        fetch(v[0], r + 2 * R * RY);
        sum(v[1], r + R * RY);
      }
    }
  }
  stat_tree<NS>(a, sm, tx, ty, VR, RY, live);
  group_stats<NT>(sm, sm + NS * VR, k.G, cg / U, float(rows) * float(U),
                  [&](int g, float mean, float m2) {
                    k.part[(int64_t(s) * k.G + g) * k.chunks + c] = make_float2(mean, m2);
                  });
}

__device__ __forceinline__ float chunk_rows(const NormKArgs& k, int c) {
  const int64_t left = k.P - int64_t(c) * k.rpc;
  return float(left < k.rpc ? left : k.rpc);
}

// (mean, M2) of a group's chunks from their average, the rows' sum s1 of differences
// from it and the squares s2 about it over all the group's channels.
__device__ __forceinline__ float2 joined(const NormKArgs& k, float mean, float s1, float s2) {
  const float c = s1 / float(k.P);
  return make_float2(mean + c, about_mean(s2, float(k.C / k.G) * c * s1));
}

// The chunks (up to 1024) of each (sample, group) joined into one: a block
// each, the partial results in registers, mean first, then the squares about it.
__global__ __launch_bounds__(256) void norm_join_kernel(NormKArgs k, float2* __restrict__ out) {
  __shared__ float red[3][4];
  const float2* p = k.part + int64_t(blockIdx.x) * k.chunks;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float2 v[4];
  float w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = int(threadIdx.x) + 256 * i;
    v[i] = c < k.chunks ? p[c] : make_float2(0.0f, 0.0f);
    w[i] = c < k.chunks ? chunk_rows(k, c) : 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(v[i].x, w[i], s);
  s = group_sum<64>(s);
  if (lane == 0) red[0][wave] = s;
  __syncthreads();
  const float mean = ((red[0][0] + red[0][1]) + (red[0][2] + red[0][3])) / float(k.P);
  const float cg = float(k.C / k.G);
  float s1 = 0.0f, q = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float d = v[i].x - mean;
    s1 += w[i] > 0.0f ? d * w[i] : 0.0f;
    q += w[i] > 0.0f ? fmaf(d * d, w[i] * cg, v[i].y) : 0.0f;
  }
  s1 = group_sum<64>(s1);
  q = group_sum<64>(q);
  if (lane == 0) {
    red[1][wave] = s1;
    red[2][wave] = q;
  }
  __syncthreads();
  if (threadIdx.x == 0)
    out[blockIdx.x] = joined(k, mean, (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]),
                             (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]));
}

// Normalises rows of sample s. Chunk c of the first pass is cut into `subs`
// parts, and block s subs chunks + sub chunks + c takes part sub (from the
// chunk's end): blocks b and b mod chunks share an XCD where chunks is a
// multiple of 8, and the rows that its L2 still holds from the first pass, the
// last ones of each chunk, come first. Statistics: join_n partial results per
// group (1 after norm_join_kernel), joined by every block.
template <typename TE, int NT>
__global__ __launch_bounds__(NT) void norm_apply_kernel(NormKArgs k, const float2* __restrict__ stats,
                                                        int join_n, int subs, int64_t rps) {
  constexpr int R = 8 / sizeof(TE);    // 4 or 2 rows
  constexpr int MAXG = NT == 256 ? 2048 : NORM_MAX_C;   // G <= C, C <= 2048 with 256 threads
  __shared__ float gm[MAXG], gr[MAXG];
  const uint32_t per = uint32_t(subs) * uint32_t(k.chunks);
  const uint32_t s = blockIdx.x / per, rest = blockIdx.x - s * per;
  const int sub = int(rest / uint32_t(k.chunks)), c = int(rest - uint32_t(sub) * uint32_t(k.chunks));
  const int64_t c0 = int64_t(c) * k.rpc, c1 = c0 + k.rpc < k.P ? c0 + k.rpc : k.P;
  const int64_t r1 = c1 - sub * rps;
  const int64_t r0 = r1 - rps > c0 ? r1 - rps : c0;
  const int rows = int(r1 - r0);       // <= 0 for parts past a short last chunk
  const int VR = k.C / 8, RY = NT / VR, cg = k.C / k.G;
  const int ty = int(threadIdx.x) / VR, tx = int(threadIdx.x) - ty * VR;
  const bool live = ty < RY;
  const int64_t base = (int64_t(s) * k.P + r0) * k.C + 8 * tx;
  const TE* const x = static_cast<const TE*>(k.x) + base;   // rows <= 0: no row is touched
  Raw8<TE> v[2][R];
  auto fetch = [&](Raw8<TE> (&d)[R], int r) {   // rows r, r - RY, ...
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (r - i * RY >= 0) d[i] = raw_load(x + int64_t(r - i * RY) * k.C);
  };
  const int last = live ? rows - 1 - ty : -1;
  fetch(v[0], last);
  Coef cf = {};
  if (live) load_affine(k, 8 * tx, cf.a, cf.b);

  const float2* const ps = stats + int64_t(s) * k.G * join_n;
  if (join_n == 1) {
    for (int g = threadIdx.x; g < k.G; g += NT) {
      const float2 r = ps[g];
      gm[g] = r.x;
      gr[g] = rstd_of(r.y, k);
    }
  } else {
    const int lq = pow2_at_least(join_n, 32), sh = __builtin_ctz(lq);
    const int l = threadIdx.x & (lq - 1);
    for (int g = threadIdx.x >> sh; g < k.G; g += NT >> sh) {
      const float2 r = l < join_n ? ps[int64_t(g) * join_n + l] : make_float2(0.0f, 0.0f);
      const float w = l < join_n ? chunk_rows(k, l) : 0.0f;
      const float mean = lanes_sum(r.x * w, lq) / float(k.P);
      const float d = r.x - mean;
      const float s1 = lanes_sum(w > 0.0f ? d * w : 0.0f, lq);
      const float2 j = joined(k, mean, s1, lanes_sum(w > 0.0f ? fmaf(d * d, w * float(cg), r.y) : 0.0f, lq));
      if (l == 0) {
        gm[g] = j.x;
        gr[g] = rstd_of(j.y, k);
      }
    }
  }
  __syncthreads();
  if (!live) return;
  coef_finish(cf, 8 * tx, cg, gm, gr);
  auto emit = [&](const Raw8<TE> (&d)[R], int r) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (r - i * RY >= 0) norm_store<TE>(d[i], cf, k, base + int64_t(r - i * RY) * k.C);
  };
  for (int r = last; r >= 0; r -= 2 * R * RY) {
    fetch(v[1], r - R * RY);
    emit(v[0], r);
    if (r - R * RY >= 0) {
      fetch(v[0], r - 2 * R * RY);
      emit(v[1], r - R * RY);
    }
  }
}

// ---- host side ----------------------------------------------------------------------

namespace {

struct NormPlan {
  int block;         // 1: one launch without a workspace,
  int rows;          // 1: norm_rows_kernel, otherwise norm_block_kernel:
  int nt, r, slab;   // threads; its rows per lane and channels per block
  int chunks;        // otherwise: chunks per sample and their rows,
  int64_t rpc;
  int subs;          // parts of a chunk in the second pass and their rows,
  int64_t rps;
  int join;          // 1: norm_join_kernel between the passes
  int64_t slice;     // samples per launch
  int64_t grid;      // threads of the call's largest launch
};

int gcd_i(int a, int b) { return b ? gcd_i(b, a % b) : a; }

// Slabs are whole groups and whole 8-channel vectors: multiples of `unit` =
// lcm(C / G, 8) channels, taken until a row's piece is 64 bytes (8 x 1536 x
// 256 fp32: 13.3 us against 14.0 with 32 bytes and 14.3 with 128), or 32 bytes
// where a sample's slabs share an XCD's L2 and wider ones would leave CUs idle
// (the same in bf16: 9.7 us against 11.8); where all positions are less than
// one pass of 256 lanes, they are doubled. Up to 8 rows per lane a block keeps
// its slab in registers (1 x 1024 x 512 fp32: 8.4 us against 9.6 for two
// launches); longer ones, and those that would be less than 48 blocks of 1024
// threads (2 x 1024 x 640 bf16, 32 blocks: 11.2 us against 12.6; 50 x 3000 x 8, 50
// blocks, the other way, 9.2 against 10.0), take the chunked form, which spreads a
// sample over every CU, at 4 rows per lane or more (1 x 4096 x 320 bf16: 11.7 us
// against 13.1 with 8, 1 x 65536 x 16 fp32: 11.0 against 13.3).
NormPlan norm_form(int64_t S, int64_t P, int C, int G, int esize) {
  NormPlan p = {};
  if (P == 1 && C / G % 8 == 0) {
    p.block = p.rows = 1;
    return p;
  }
  const int cg = C / G, unit = cg / gcd_i(cg, 8) * 8;
  const int piece = esize == 2 && S % 8 == 0 && S * (C / 16) <= 256 ? 32 : 64;
  int slab = unit;
  while (slab * esize < piece && slab < C) slab += unit;
  while (slab < C && P * slab / 4 <= 256 && 2 * slab / cg <= NORM_BLOCK_GROUPS) slab *= 2;
  if (slab > C) slab = C;
  for (int nt : {256, 1024}) {
    const int VR = slab / 8;
    if (VR > nt || slab / cg > NORM_BLOCK_GROUPS) continue;
    if (nt == 1024 && S * ((C + slab - 1) / slab) < 48) continue;
    const int64_t need = (P + nt / VR - 1) / (nt / VR);   // rows per lane
    if (need <= 8) {
      p.block = 1;
      p.nt = nt;
      p.slab = slab;
      p.r = need <= 2 && nt == 256 ? 2 : 8;
      return p;
    }
  }
  p.nt = C <= 2048 ? 256 : 1024;
  const int RY = p.nt / (C / 8);
  int64_t want = (1024 + S - 1) / S;                      // about four blocks per CU
  const int64_t most = (P + RY * 4 - 1) / (RY * 4);       // at least 4 rows per lane
  if (want > most) want = most;
  p.rpc = (P + want - 1) / want;
  p.chunks = int((P + p.rpc - 1) / p.rpc);
  // parts of at most 16 rows per lane
  p.subs = int((p.rpc + RY * 16 - 1) / (RY * 16));
  p.rps = (p.rpc + p.subs - 1) / p.subs;
  // many chunks: every block of the second pass would read them all
  p.join = p.chunks > 32;
  return p;
}

// norm_rows_kernel: lanes per row of w channels, pieces of 8 channels per lane (one
// up to 512 channels, at most 8: C <= NORM_MAX_C), and blocks, no more than the CUs
// hold at once.
int norm_rows_lanes(int w) {
  int L = 1;
  while (L < 64 && L * 8 < w) L <<= 1;
  return L;
}
int norm_rows_pieces(int C, int G) {
  const int r = (C / G + 511) / 512;
  if (r == 1) return 1;
  return G > 1 ? 4 : r <= 4 ? r : 8;
}
int64_t norm_rows_blocks(int64_t rows, int L, int R) {
  return std::min<int64_t>((rows * L + 255) / 256, R == 1 ? 2048 : 1280);
}

// The form, and how many samples one launch takes: a grid holds less than 2^32
// threads (kept to half of that here), and a sample may be hundreds of blocks. Slices
// are whole eights where they can be (norm_block_kernel's order of slabs).
NormPlan norm_plan(int64_t S, int64_t P, int C, int G, int esize) {
  NormPlan p = norm_form(S, P, C, G, esize);
  p.slice = S;
  if (p.rows) {
    const int R = norm_rows_pieces(C, G);
    p.grid = 256 * norm_rows_blocks(S * G, norm_rows_lanes(C / G), R);
    return p;
  }
  // blocks per sample of the first and the second pass (join: 256 threads for a group)
  const int64_t blocks = p.block ? (C + p.slab - 1) / p.slab : int64_t(p.chunks) * p.subs;
  const int64_t threads = std::max<int64_t>(blocks * p.nt, p.join ? int64_t(G) * 256 : 0);
  const int64_t most = (int64_t(1) << 31) / threads;
  if (S > most) p.slice = most >= 8 ? most & ~int64_t(7) : most;
  p.grid = p.slice * threads;
  return p;
}

template <typename TE, int U>
void launch_norm_first(const NormPlan& p, const NormKArgs& k, dim3 grid, hipStream_t s) {
  if (!p.block && p.nt == 256)
    hipLaunchKernelGGL((norm_stats_kernel<TE, U, 256>), grid, dim3(256), 0, s, k);
  else if (!p.block)
    hipLaunchKernelGGL((norm_stats_kernel<TE, U, 1024>), grid, dim3(1024), 0, s, k);
  else if (p.nt == 256 && p.r == 2)
    hipLaunchKernelGGL((norm_block_kernel<TE, U, 256, 2>), grid, dim3(256), 0, s, k);
  else if (p.nt == 256)
    hipLaunchKernelGGL((norm_block_kernel<TE, U, 256, 8>), grid, dim3(256), 0, s, k);
  else
    hipLaunchKernelGGL((norm_block_kernel<TE, U, 1024, 8>), grid, dim3(1024), 0, s, k);
}

template <typename TE, int R, bool HOLD>
hipError_t launch_norm_rows(const NormKArgs& k, int64_t S, hipStream_t s) {
  const int64_t rows = S * k.G;
  const int L = norm_rows_lanes(k.C / k.G);
  const int64_t blocks = norm_rows_blocks(rows, L, R);
  hipLaunchKernelGGL((norm_rows_kernel<TE, R, HOLD>), dim3(unsigned(blocks)), dim3(256), 0, s, k, rows,
                     L);
  return hipGetLastError();
}

template <typename TE>
hipError_t launch_norm_typed(const NormPlan& p, const NormKArgs& k, int64_t S, hipStream_t s) {
  if (p.rows) {
    const int r = norm_rows_pieces(k.C, k.G);
    if (k.G > 1)
      return r == 1 ? launch_norm_rows<TE, 1, false>(k, S, s) : launch_norm_rows<TE, 4, false>(k, S, s);
    switch (r) {
      case 1: return launch_norm_rows<TE, 1, true>(k, S, s);
      case 2: return launch_norm_rows<TE, 2, true>(k, S, s);
      case 3: return launch_norm_rows<TE, 3, true>(k, S, s);
      case 4: return launch_norm_rows<TE, 4, true>(k, S, s);
      default: return launch_norm_rows<TE, 8, false>(k, S, s);
    }
  }
  const dim3 g1(unsigned(S * (p.block ? (k.C + p.slab - 1) / p.slab : p.chunks)));
  switch (gcd_i(k.C / k.G, 8)) {
    case 8: launch_norm_first<TE, 8>(p, k, g1, s); break;
    case 4: launch_norm_first<TE, 4>(p, k, g1, s); break;
    case 2: launch_norm_first<TE, 2>(p, k, g1, s); break;
    default: launch_norm_first<TE, 1>(p, k, g1, s); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.block) return e;
  const dim3 g2(unsigned(S * p.chunks * p.subs));
  const float2* stats = k.part;
  int join_n = p.chunks;
  if (p.join) {
    float2* joined = k.part + S * k.G * p.chunks;
    hipLaunchKernelGGL(norm_join_kernel, dim3(unsigned(S * k.G)), dim3(256), 0, s, k, joined);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    stats = joined;
    join_n = 1;
  }
  if (p.nt == 256)
    hipLaunchKernelGGL((norm_apply_kernel<TE, 256>), g2, dim3(256), 0, s, k, stats, join_n, p.subs,
                       p.rps);
  else
    hipLaunchKernelGGL((norm_apply_kernel<TE, 1024>), g2, dim3(1024), 0, s, k, stats, join_n,
                       p.subs, p.rps);
  return hipGetLastError();
}

}  // namespace

size_t norm_part_bytes(int64_t S, int64_t P, int C, int G, int esize) {
  if (S <= 0 || P <= 0) return 0;
  const NormPlan p = norm_plan(S, P, C, G, esize);
  return p.block ? 0 : sizeof(float2) * size_t(S) * size_t(G) * size_t(p.chunks + p.join);
}

NormPlanInfo norm_plan_info(int64_t S, int64_t P, int C, int G, int esize) {
  NormPlanInfo i = {};
  if (S <= 0 || P <= 0) return i;
  const NormPlan p = norm_plan(S, P, C, G, esize);
  i.kernel = p.rows ? NORM_ROWS : p.block ? NORM_BLOCK : p.join ? NORM_CHUNKS_JOINED : NORM_CHUNKS;
  i.slices = int((S + p.slice - 1) / p.slice);
  i.grid = p.grid;
  return i;
}

hipError_t launch_group_norm(const NormArgs& a, int64_t S, hipStream_t s) {
  const NormPlan p = norm_plan(S, a.P, a.C, a.G, a.x_bf16 ? 2 : 4);
  NormKArgs k = {};
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
  for (int64_t s0 = 0; s0 < S; s0 += p.slice) {
    const int64_t n = std::min(S - s0, p.slice), off = s0 * a.P * a.C;
    k.x = static_cast<const char*>(a.x) + off * (a.x_bf16 ? 2 : 4);
    k.y = static_cast<char*>(a.y) + off * (a.y_bf16 ? 2 : 4);
    const hipError_t e = a.x_bf16 ? launch_norm_typed<uint16_t>(p, k, n, s)
                                  : launch_norm_typed<float>(p, k, n, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace hq
