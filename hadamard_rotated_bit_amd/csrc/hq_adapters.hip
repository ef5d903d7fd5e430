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

namespace {

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
  return a.bf16 ? launch_adapters_typed<uint16_t>(a, s) : launch_adapters_typed<float>(a, s);
}

}  // namespace hq
