// Low-rank adapters of many requests beside a projection that they share:
//
//   Y[t] = R[t] + g[t / gate_rows] phi(base[t] + s_a B_a (A_a x[t])),   a = ids[t],
//
// A_a [rank, K], B_a [N, rank]; a row whose id names no adapter has base alone, and its
// x is not read. Sums are fp32; u = s_a A_a x stays in fp32 between the two products.
// Bound by memory: base is read and Y written once, x once, each adapter once per row or
// tile that uses it (from the caches).
#include "hq_epilogue.h"
#include "hq_internal.h"

#include <algorithm>

namespace hq {

// ---- row by row ---------------------------------------------------------------

// u[t, j] = s_a sum_k x[t, k] A_a[j, k]: a wave per row and rank index.
template <typename TE>
__global__ __launch_bounds__(256) void adapt_down_kernel(AdaptArgs k) {
  const int lane = int(threadIdx.x) & 63;
  for (int64_t job = int64_t(blockIdx.x) * 4 + (int(threadIdx.x) >> 6); job < k.T * k.rank;
       job += int64_t(gridDim.x) * 4) {
  const int64_t t = job / k.rank;
  const int j = int(job - t * k.rank);
  const int id = k.ids[t];
  if (uint32_t(id) >= uint32_t(k.count)) continue;
  const TE* const x = static_cast<const TE*>(k.x) + t * k.K;
  const TE* const a = static_cast<const TE*>(k.a) + (int64_t(id) * k.rank + j) * k.K;
  float s = 0.0f;
  for (int c = 8 * lane; c < k.K; c += 512) {
    float p[8], q[8];
    load8(x + c, p);
    load8(a + c, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(p[e], q[e], s);
  }
  s = group_sum<64>(s);
  if (lane == 0) k.u[t * k.rank + j] = k.scales ? s * k.scales[id] : s;
  }
}

// Y[t, n .. n + 7] from base and u: a lane per 8 columns of a row.
template <typename TE>
__global__ __launch_bounds__(256) void adapt_up_kernel(AdaptArgs k) {
  const int per = k.N / 8;
  for (int64_t job = int64_t(blockIdx.x) * 256 + threadIdx.x; job < k.T * per;
       job += int64_t(gridDim.x) * 256) {
  const int64_t t = job / per;
  const int n = 8 * int(job - t * per);
  float v[8] = {};
  if (k.base) {
    if (k.ep.y_bf16) load8(static_cast<const uint16_t*>(k.base) + t * k.N + n, v);
    else load8(static_cast<const float*>(k.base) + t * k.N + n, v);
  }
  const int id = k.ids[t];
  if (uint32_t(id) < uint32_t(k.count)) {
    const TE* const b = static_cast<const TE*>(k.b) + (int64_t(id) * k.N + n) * k.rank;
    const float* const u = k.u + t * k.rank;
    float d[8] = {};
    for (int j = 0; j < k.rank; j += 8) {
      float p[8];
      load8(u + j, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float q[8];
        load8(b + e * k.rank + j, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[e] = fmaf(p[i], q[i], d[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += d[e];
  }
  finish_piece(v, t, n, k.N, k.ep);
  }
}

// ---- tiles of rows -------------------------------------------------------------

namespace {

__device__ __forceinline__ v4f mfma16(v8bf a, v8bf b, v4f c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
  return c;
#endif
}
__device__ __forceinline__ v4f mfma16(float a, float b, v4f c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
#else
  return c;
#endif
}

// A lane's 16 bytes of a k-step's operand, and the products of a step: 32 k of bf16 in
// one MFMA, 16 k of fp32 in four (lane group g holds k 4 g .. 4 g + 3; MFMA q takes the
// q-th of each, the same k on both sides).
template <typename TE>
struct Frag;
template <>
struct Frag<uint16_t> {
  static constexpr int KS = 32, PER = 8;
  uint4 q;
  __device__ __forceinline__ v8bf get() const { return __builtin_bit_cast(v8bf, q); }
};
template <>
struct Frag<float> {
  static constexpr int KS = 16, PER = 4;
  uint4 q;
};
template <typename TE>
__device__ __forceinline__ v4f frag_mfma(const Frag<TE>& a, const Frag<TE>& b, v4f c) {
  if constexpr (sizeof(TE) == 2) {
    return mfma16(a.get(), b.get(), c);
  } else {
    c = mfma16(__uint_as_float(a.q.x), __uint_as_float(b.q.x), c);
    c = mfma16(__uint_as_float(a.q.y), __uint_as_float(b.q.y), c);
    c = mfma16(__uint_as_float(a.q.z), __uint_as_float(b.q.z), c);
    return mfma16(__uint_as_float(a.q.w), __uint_as_float(b.q.w), c);
  }
}
template <typename TE>
__device__ __forceinline__ Frag<TE> frag_load(const TE* p, bool ok) {
  Frag<TE> f;
  f.q = ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  return f;
}

// The adapter of lane (lane % rows) of a tile from row r0, -1 where it has none.
__device__ __forceinline__ int tile_id(const AdaptArgs& k, int64_t r0, int r) {
  const int id = r0 + r < k.T ? k.ids[r0 + r] : -1;
  return uint32_t(id) < uint32_t(k.count) ? id : -1;
}

}  // namespace

// u of 16 MT rows: NW waves take the 64-k chunks of the rows and of A_a in turn, for each
// adapter that the rows have; their sums are joined in LDS in wave order. RT: tiles of 16
// rank indexes (RT 16 >= rank).
template <typename TE, int MT, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void adapt_down_tile_kernel(AdaptArgs k) {
  using F = Frag<TE>;
  constexpr int ROWS = 16 * MT, STEPS = 64 / F::KS;
  constexpr int RJ = RT < 2 ? RT : 2;   // tiles joined at a time
  __shared__ float red[NW][ROWS][16 * RJ + 1];
  const int lane = int(threadIdx.x) & 63, w = int(threadIdx.x) >> 6;
  const int i = lane & 15, g = lane >> 4;
  for (int64_t r0 = int64_t(blockIdx.x) * ROWS; r0 < k.T; r0 += int64_t(gridDim.x) * ROWS) {
  const int id = lane < ROWS ? tile_id(k, r0, lane) : -1;
  uint64_t left = __ballot(id >= 0);
  while (left) {   // the same for every wave
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t match = __ballot(id == a);
    left &= ~match;
    const TE* x[MT];
    const TE* ar[RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      x[m] = static_cast<const TE*>(k.x) + min(r0 + 16 * m + i, k.T - 1) * k.K + F::PER * g;
#pragma unroll
    for (int t = 0; t < RT; ++t)
      ar[t] = static_cast<const TE*>(k.a) + (int64_t(a) * k.rank + min(16 * t + i, k.rank - 1)) * k.K +
              F::PER * g;
    v4f acc[MT][RT] = {};
    for (int c = 64 * w; c < k.K; c += 64 * NW) {
      F fx[STEPS][MT], fa[STEPS][RT];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int kk = c + F::KS * s;
        const bool ok = kk + F::PER * g < k.K;
#pragma unroll
        for (int m = 0; m < MT; ++m) fx[s][m] = frag_load<TE>(x[m] + kk, ok);
#pragma unroll
        for (int t = 0; t < RT; ++t) fa[s][t] = frag_load<TE>(ar[t] + kk, ok);
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[m][t] = frag_mfma<TE>(fx[s][m], fa[s][t], acc[m][t]);
    }
    const float scale = k.scales ? k.scales[a] : 1.0f;
#pragma unroll
    for (int t0 = 0; t0 < RT; t0 += RJ) {
      __syncthreads();   // the last sums are read
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < RJ; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) red[w][16 * m + 4 * g + e][16 * t + i] = acc[m][t0 + t][e];
      __syncthreads();
      for (int o = int(threadIdx.x); o < ROWS * 16 * RJ; o += 64 * NW) {
        const int row = o / (16 * RJ), j = o - row * (16 * RJ);
        float s = red[0][row][j];
#pragma unroll
        for (int n = 1; n < NW; ++n) s += red[n][row][j];
        if (((match >> row) & 1) && 16 * t0 + j < k.rank)
          k.u[(r0 + row) * k.rank + 16 * t0 + j] = s * scale;
      }
    }
  }
  }
}

// Y of 16 MT rows x 256 columns, 64 columns a wave. B_a's rows are the MFMA's rows, so a
// lane ends with columns n .. n + 7 and n + 32 .. n + 39 of one row: MFMAs 2 p and 2 p + 1
// take the columns 32 p + 8 (i / 4) + i % 4 and the four behind each. u enters a bf16
// product as three bf16 parts (24 bits).
template <typename TE, typename TY, int MT>
__global__ __launch_bounds__(256) void adapt_up_tile_kernel(AdaptArgs k) {
  using F = Frag<TE>;
  constexpr int ROWS = 16 * MT, NP = sizeof(TE) == 2 ? 3 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = int(threadIdx.x) & 63, w = int(threadIdx.x) >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int nb = (k.N + 255) / 256;
  const int steps = (k.rank + F::KS - 1) / F::KS;
  const int pitch = steps * F::KS + F::PER;   // elements; 16 bytes past a row
  TE* const us = reinterpret_cast<TE*>(smem);
  for (int64_t tile = blockIdx.x; tile < (k.T + ROWS - 1) / ROWS * nb; tile += gridDim.x) {
  const int64_t r0 = tile / nb * ROWS;
  const int n0 = int(tile % nb) * 256 + 64 * w;
  const int id = lane < ROWS ? tile_id(k, r0, lane) : -1;
  uint64_t left = __ballot(id >= 0);
  __syncthreads();   // the last tile's u is read
  if (left) {
    const int octs = steps * F::KS / 4;
    for (int o = int(threadIdx.x); o < ROWS * octs; o += 256) {
      const int row = o / octs, j = 4 * (o - row * octs);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r0 + row < k.T && j < k.rank)
        v = *reinterpret_cast<const float4*>(k.u + (r0 + row) * k.rank + j);
      if constexpr (NP == 1) {
        *reinterpret_cast<float4*>(us + row * pitch + j) = v;
      } else {
        float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const uint32_t a = pack_bf16x2(f[0], f[1]), b = pack_bf16x2(f[2], f[3]);
          *reinterpret_cast<uint2*>(us + (p * ROWS + row) * pitch + j) = make_uint2(a, b);
          f[0] -= __uint_as_float(a << 16);
          f[1] -= __uint_as_float(a & 0xFFFF0000u);
          f[2] -= __uint_as_float(b << 16);
          f[3] -= __uint_as_float(b & 0xFFFF0000u);
        }
      }
    }
  }
  __syncthreads();
  if (n0 >= k.N) continue;
  // rows without an adapter first, then adapter by adapter
  uint64_t match = __ballot(id < 0) & ((uint64_t(1) << (ROWS - 1) << 1) - 1);
  int a = -1;
  for (;;) {
    if (match) {
      v4f acc[MT][4] = {};
      if (a >= 0) {
        const TE* br[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          br[t] = static_cast<const TE*>(k.b) +
                  (int64_t(a) * k.N + min(n0 + 32 * (t >> 1) + 8 * (i >> 2) + 4 * (t & 1) + (i & 3), k.N - 1)) * k.rank +
                  F::PER * g;
        for (int s = 0; s < steps; ++s) {
          const bool ok = F::KS * s + F::PER * g < k.rank;
          F fb[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) fb[t] = frag_load<TE>(br[t] + F::KS * s, ok);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              F fu;
              fu.q = *reinterpret_cast<const uint4*>(us + (p * ROWS + 16 * m + i) * pitch + F::KS * s +
                                                     F::PER * g);
#pragma unroll
              for (int t = 0; t < 4; ++t) acc[m][t] = frag_mfma<TE>(fb[t], fu, acc[m][t]);
            }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bool mine = (match >> (16 * m + i)) & 1;
        const int64_t row = r0 + 16 * m + i;
        float v[2][8];
        int64_t mm[2], nn[2];
        bool ok[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          mm[p] = row;
          nn[p] = n0 + 32 * p + 8 * g;
          ok[p] = mine && row < k.T && nn[p] < k.N;
          float b[8] = {};
          if (k.base && ok[p]) load8(static_cast<const TY*>(k.base) + row * k.N + nn[p], b);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[p][e] = b[e] + acc[m][2 * p + (e >> 2)][e & 3];
        }
        finish8<TY, 2>(v, mm, nn, ok, k.N, k.ep);
      }
    }
    if (!left) break;
    a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    match = __ballot(id == a);
    left &= ~match;
  }
  }
}

namespace {

template <typename TE, int RT>
hipError_t launch_down_tiles(const AdaptArgs& a, hipStream_t s) {
  constexpr int MT = 2, NW = 8;
  const dim3 grid(unsigned(std::min<int64_t>((a.T + 16 * MT - 1) / (16 * MT), 1 << 20)));
  hipLaunchKernelGGL((adapt_down_tile_kernel<TE, MT, RT, NW>), grid, dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}
template <typename TE, typename TY>
hipError_t launch_up_tiles(const AdaptArgs& a, hipStream_t s) {
  constexpr int MT = 4, NP = sizeof(TE) == 2 ? 3 : 1;
  const int64_t nb = (a.N + 255) / 256, tiles = (a.T + 16 * MT - 1) / (16 * MT);
  const int steps = (a.rank + Frag<TE>::KS - 1) / Frag<TE>::KS;
  const size_t lds = size_t(NP) * 16 * MT * size_t(steps * Frag<TE>::KS + Frag<TE>::PER) * sizeof(TE);
  hipLaunchKernelGGL((adapt_up_tile_kernel<TE, TY, MT>), dim3(unsigned(std::min<int64_t>(nb * tiles, 1 << 20))), dim3(256), lds, s, a);
  return hipGetLastError();
}
template <typename TE>
hipError_t launch_tiles(const AdaptArgs& a, hipStream_t s) {
  const int rt = (a.rank + 15) / 16;
  const hipError_t e = rt <= 1   ? launch_down_tiles<TE, 1>(a, s)
                       : rt <= 2 ? launch_down_tiles<TE, 2>(a, s)
                       : rt <= 4 ? launch_down_tiles<TE, 4>(a, s)
                                 : launch_down_tiles<TE, 8>(a, s);
  if (e != hipSuccess) return e;
  return a.ep.y_bf16 ? launch_up_tiles<TE, uint16_t>(a, s) : launch_up_tiles<TE, float>(a, s);
}

template <typename TE>
hipError_t launch_adapters_typed(const AdaptArgs& a, hipStream_t s) {
  const int64_t down = std::min<int64_t>((a.T * a.rank + 3) / 4, 1 << 20);
  const int64_t up = std::min<int64_t>((a.T * (a.N / 8) + 255) / 256, 1 << 20);
  hipLaunchKernelGGL(adapt_down_kernel<TE>, dim3(unsigned(down)), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(adapt_up_kernel<TE>, dim3(unsigned(up)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t adapters_part_bytes(int64_t T, int rank) { return size_t(T) * size_t(rank) * 4; }

hipError_t launch_adapters(const AdaptArgs& a, hipStream_t s) {
  if (a.T > 64) return a.bf16 ? launch_tiles<uint16_t>(a, s) : launch_tiles<float>(a, s);
  return a.bf16 ? launch_adapters_typed<uint16_t>(a, s) : launch_adapters_typed<float>(a, s);
}

}  // namespace hq
