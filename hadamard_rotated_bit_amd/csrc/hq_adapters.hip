// Low-rank adapters of many requests beside a projection that they share:
//
//   Y[t] = R[t] + g[t / gate_rows] phi(base[t] + s_a B_a (A_a x[t])),   a = ids[t],
//
// A_a [rank, K], B_a [N, rank]; a row whose id names no adapter has base alone. Sums are
// fp32; u = s_a A_a x keeps 24 bits between the two products. Bound by memory: base is
// read and Y written once, x once, each adapter once per row or tile that uses it (from
// the caches). Few rows take one launch, a block per row (adapt_rows_kernel); many take
// tiles of rows on the matrix units, a launch for each product.
#include "hq_epilogue.h"
#include "hq_gemm_kernel.h"
#include "hq_internal.h"

#include <algorithm>

namespace hq {

namespace {

// 16 bytes at a uniform base and a lane's 32-bit offset (one address register).
__device__ __forceinline__ uint4 load16(const void* base, uint32_t off) {
  return *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + off);
}
template <typename TE>
__device__ __forceinline__ Raw8<TE> raw_at(const void* base, uint32_t off) {
  Raw8<TE> r;
#pragma unroll
  for (unsigned i = 0; i < sizeof(TE) / 2; ++i) r.q[i] = load16(base, off + 16 * i);
  return r;
}

// The elements of 16 bytes as floats.
template <typename TE>
__device__ __forceinline__ void get16(const uint4& q, float* v) {
  if constexpr (sizeof(TE) == 2) {
    load8(reinterpret_cast<const uint16_t*>(&q), v);
  } else {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
}

}  // namespace

// ---- row by row ---------------------------------------------------------------

// Y of one row (block x) and a part of its columns (block y; each part takes the row's u
// for itself: one launch). Eight waves share the rank indexes of u, JW each, all their
// loads of U strips of K in flight; then 64 columns a wave at a time: B_a's rows pass
// through the wave's own LDS, read in whole lines, so that each lane has a column. Bound
// by the chain of a launch, the id, A_a and x, B_a and the store for few rows (24 rows of
// 4096 -> 4096 rank 16: 6.0 us). Many rows take several rounds of blocks, each with that
// chain: 1037 of 1160 -> 2312 rank 8 fp32, 18.7 us, two rounds of 768 blocks, the vector ALU
// busy half of the time, waves waiting 48 % of theirs. Two or four rows a block that share
// what they fetch are no faster (700 rows of 1024 -> 1024 rank 8: 7.7, 7.8, 8.7).
template <typename TE, int JW, int U>
__global__ __launch_bounds__(512) void adapt_rows_kernel(AdaptArgs k) {
  constexpr int PER = 16 / sizeof(TE);             // elements of 16 bytes
  constexpr int SP = JW * int(sizeof(TE)) / 2 < 8 ? JW * int(sizeof(TE)) / 2 : 8;
  constexpr int PITCH = 16 * SP + 16;              // SP pieces of a column's row in LDS
  __shared__ __attribute__((aligned(16))) float u[8 * JW];
  __shared__ __attribute__((aligned(16))) uint8_t bs[8][64 * PITCH];
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int64_t t = blockIdx.x;
  const int id = __builtin_amdgcn_readfirstlane(k.ids[t]);
  const bool has = uint32_t(id) < uint32_t(k.count);
  // the wave's first columns are on their way while u is made, the next ones while they are
  // multiplied
  const uint32_t brow = uint32_t(k.rank) * sizeof(TE), ppr = brow / 16;
  const int units = (k.N + 63) / 64;
  const int u1 = int(int64_t(units) * (blockIdx.y + 1) / gridDim.y);
  int n0 = int(int64_t(units) * blockIdx.y / gridDim.y) + w;
  uint4 q[SP];
  auto load_b = [&](int unit, uint32_t z0) {   // SP pieces from z0 of 64 columns' rows
    const uint8_t* const B = static_cast<const uint8_t*>(k.b) + (int64_t(id) * k.N + 64 * unit) * brow;
    const uint32_t sp = min(ppr - z0, uint32_t(SP)), most = uint32_t(min(64, k.N - 64 * unit)) * sp;
#pragma unroll
    for (int z = 0; z < SP; ++z) {
      const uint32_t o = lane + 64 * z, r = o / sp;
      if (o < most) q[z] = load16(B, r * brow + 16 * (z0 + o - r * sp));
    }
  };
  auto load_base = [&](int unit) {
    const int n = 64 * unit + lane;
    if (!k.base || n >= k.N) return 0.0f;
    return k.ep.y_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(k.base)[t * k.N + n])
                       : static_cast<const float*>(k.base)[t * k.N + n];
  };
  float base = 0.0f;
  if (n0 < u1) {
    base = load_base(n0);
    if (has) load_b(n0, 0);
  }
  if (has) {
    const TE* const x = static_cast<const TE*>(k.x) + t * k.K;
    const TE* const A = static_cast<const TE*>(k.a) + int64_t(id) * k.rank * k.K;
    float s[JW] = {};
    uint32_t row[JW];   // rank indexes w, w + 8, ...; past the last one it again
#pragma unroll
    for (int j = 0; j < JW; ++j) row[j] = uint32_t(min(w + 8 * j, k.rank - 1)) * uint32_t(k.K);
#pragma unroll 1
    for (int c = PER * lane; c < k.K; c += 64 * PER * U) {
      uint4 xq[U], aq[U][JW];
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int cc = c + 64 * PER * n;
        if (cc >= k.K) continue;
        xq[n] = load16(x, uint32_t(cc) * sizeof(TE));
#pragma unroll
        for (int j = 0; j < JW; ++j) aq[n][j] = load16(A, (row[j] + cc) * uint32_t(sizeof(TE)));
      }
#pragma unroll
      for (int n = 0; n < U; ++n) {
        if (c + 64 * PER * n >= k.K) continue;
        float p[PER], q[PER];
        get16<TE>(xq[n], p);
#pragma unroll
        for (int j = 0; j < JW; ++j) {
          get16<TE>(aq[n][j], q);
#pragma unroll
          for (int e = 0; e < PER; ++e) s[j] = fmaf(p[e], q[e], s[j]);
        }
      }
    }
    const float scale = k.scales ? k.scales[id] : 1.0f;
#pragma unroll
    for (int j = 0; j < JW; ++j) {
      const float v = group_sum<64>(s[j]) * scale;
      if (lane == 0 && w + 8 * j < k.rank) u[w + 8 * j] = v;
    }
  }
  __syncthreads();
  for (; n0 < u1; n0 += 8) {
    const int n = 64 * n0 + lane;
    const float b0 = base;
    float d = 0.0f;
    if (n0 + 8 < u1) base = load_base(n0 + 8);
    if (has) {
#pragma unroll 1
      for (uint32_t z0 = 0; z0 < ppr; z0 += SP) {
        const uint32_t sp = min(ppr - z0, uint32_t(SP));
#pragma unroll
        for (int z = 0; z < SP; ++z) {
          const uint32_t o = lane + 64 * z, r = o / sp;
          if (o < 64 * sp) *reinterpret_cast<uint4*>(bs[w] + r * PITCH + 16 * (o - r * sp)) = q[z];
        }
        wave_lds_sync();   // the pieces are those of other lanes
        if (z0 + SP < ppr) load_b(n0, z0 + SP);
        else if (n0 + 8 < u1) load_b(n0 + 8, 0);
        for (uint32_t z = 0; z < sp; ++z) {
          float b[PER];
          get16<TE>(*reinterpret_cast<const uint4*>(bs[w] + lane * PITCH + 16 * z), b);
#pragma unroll
          for (int e = 0; e < PER; ++e) d = fmaf(b[e], u[PER * (z0 + z) + e], d);
        }
        wave_lds_sync();   // the next ones take their place
      }
    }
    if (n < k.N) finish1(b0 + d, t, n, k.N, k.ep);
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
constexpr uint32_t kOutside = 0x80000000u;   // an offset outside every descriptor here
__device__ __forceinline__ uint4 buf_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, int(off), 0, 0));
#else
  return make_uint4(0, 0, 0, 0);
#endif
}
__device__ __forceinline__ void buf_store16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint4 v) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v), r, int(off), 0, 0);
#endif
}

// A barrier that waits for LDS alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The row tile of block x: block b runs on XCD b mod 8, and the tiles of one XCD are
// neighbours, which share an adapter where rows come in runs (grid: a multiple of 8).
__device__ __forceinline__ int64_t tile_of_block() {
  return int64_t(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
}

// The adapter of row r of a tile from row r0, -1 where it has none.
__device__ __forceinline__ int tile_id(const AdaptArgs& k, int64_t r0, int r) {
  const int id = r0 + r < k.T ? k.ids[r0 + r] : -1;
  return uint32_t(id) < uint32_t(k.count) ? id : -1;
}

}  // namespace

// A_a x of 16 MT rows over one of `splits` parts of K, for each adapter that the rows
// have, into u [splits, T, rank]. The part's chunks of 128 bytes a row go to NW waves in
// turn. A wave loads a chunk of its rows of x and of A_a eight lanes a row (a fragment's
// own order, 16 rows in consecutive lanes, costs the address unit four times as much),
// passes it through its own part of the LDS (slot c ^ (r / 2) mod 8 of row r: 16 lanes
// read 16 distinct positions of the 64 banks) and has the next chunk's loads in flight
// meanwhile. The waves' sums are joined in LDS in wave order. 8192 x 4096 rank 64: 27 us,
// 7.3 TB/s of x and A_a through the L2s (2.5 TB/s of x from memory); with tiles of 64 rows,
// which halve A_a's part and make two of u, both products take 58.6 us against 59.5, at 2500
// rows 29.2 against 27.3; two chunks in flight no gain.
template <typename TE, int MT, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void adapt_down_tile_kernel(AdaptArgs k) {
  using F = Frag<TE>;
  constexpr int ROWS = 16 * MT, LROWS = 16 * (MT + RT), UNITS = LROWS / 8;
  constexpr int CK = 128 / sizeof(TE);   // k of a chunk
  constexpr int RJ = RT < 2 ? RT : 2;    // rank tiles joined at a time
  constexpr int RP = 16 * RJ + 1;
  static_assert(NW * ROWS * RP * 4 <= NW * LROWS * 128, "the sums fit in the chunks' place");
  __shared__ __attribute__((aligned(16))) uint8_t smem[NW * LROWS * 128];
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int chunks = (k.K + CK - 1) / CK;
  const uint32_t ldb = uint32_t(k.K) * sizeof(TE);
  uint8_t* const mine = smem + w * LROWS * 128;
  const int urow = lane >> 3, piece = lane & 7;
  const int64_t r0 = tile_of_block() * ROWS;
  if (r0 >= k.T) return;
  const int split = int(blockIdx.y);
  const int c1 = int(int64_t(chunks) * (split + 1) / k.splits);
  const int rows = int(min(k.T - r0, int64_t(ROWS)));
  const uint8_t* const x = static_cast<const uint8_t*>(k.x) + r0 * ldb;
  uint32_t off[UNITS];   // of the lane's rows of x and of A_a
#pragma unroll
  for (int n = 0; n < UNITS; ++n) {
    const int r = 8 * n + urow;
    off[n] = uint32_t(r < ROWS ? min(r, rows - 1) : min(r - ROWS, k.rank - 1)) * ldb + 16 * piece;
  }
  const int id = lane < ROWS ? tile_id(k, r0, lane) : -1;
  for (uint64_t left = __ballot(id >= 0); left;) {   // the same for every wave
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t match = __ballot(id == a);
    left &= ~match;
    const uint8_t* const A = static_cast<const uint8_t*>(k.a) + int64_t(a) * k.rank * ldb;
    uint4 st[UNITS];
    auto load = [&](int c) {   // zeros past the end of a row
      if (uint32_t(c + 1) * 128 <= ldb) {
#pragma unroll
        for (int n = 0; n < UNITS; ++n) st[n] = load16((n < 2 * MT ? x : A) + c * 128, off[n]);
      } else {
        const bool ok = uint32_t(c) * 128 + 16 * piece < ldb;
#pragma unroll
        for (int n = 0; n < UNITS; ++n)
          st[n] = ok ? load16((n < 2 * MT ? x : A) + c * 128, off[n]) : make_uint4(0, 0, 0, 0);
      }
    };
    v4f acc[MT][RT] = {};
    const int c0 = int(int64_t(chunks) * split / k.splits) + w;
    const int nc = c0 < c1 ? (c1 - c0 + NW - 1) / NW : 0;
    int jc = nc ? int(blockIdx.x % unsigned(nc)) : 0;   // row tiles start apart
    if (nc) load(c0 + NW * jc);
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      jc = jc + 1 < nc ? jc + 1 : 0;
#pragma unroll
      for (int n = 0; n < UNITS; ++n) {
        const int r = 8 * n + urow;
        *reinterpret_cast<uint4*>(mine + r * 128 + 16 * (piece ^ ((r >> 1) & 7))) = st[n];
      }
      wave_lds_sync();   // rows are read by other lanes
      if (c + 1 < nc) load(c0 + NW * jc);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        F fx[MT], fa[RT];
        const int slot = 16 * ((4 * s + g) ^ ((i >> 1) & 7));
#pragma unroll
        for (int m = 0; m < MT; ++m)
          fx[m].q = *reinterpret_cast<const uint4*>(mine + (16 * m + i) * 128 + slot);
#pragma unroll
        for (int t = 0; t < RT; ++t)
          fa[t].q = *reinterpret_cast<const uint4*>(mine + (ROWS + 16 * t + i) * 128 + slot);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[m][t] = frag_mfma<TE>(fx[m], fa[t], acc[m][t]);
      }
      wave_lds_sync();   // the next chunk takes their place
    }
    float* const red = reinterpret_cast<float*>(smem);   // [NW][ROWS][RP]
    float* const u = k.u + int64_t(split) * k.T * k.rank;
#pragma unroll
    for (int t0 = 0; t0 < RT; t0 += RJ) {
      lds_barrier();   // the chunks and the last sums are read
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < RJ; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            red[(w * ROWS + 16 * m + 4 * g + e) * RP + 16 * t + i] = acc[m][t0 + t][e];
      lds_barrier();
#pragma unroll 1
      for (int o = int(threadIdx.x); o < ROWS * 16 * RJ; o += 64 * NW) {
        const int row = o / (16 * RJ), j = o - row * (16 * RJ);
        float s = red[row * RP + j];
#pragma unroll
        for (int n = 1; n < NW; ++n) s += red[(n * ROWS + row) * RP + j];
        if (((match >> row) & 1) && 16 * t0 + j < k.rank) u[(r0 + row) * k.rank + 16 * t0 + j] = s;
      }
    }
    lds_barrier();   // the sums are read
  }
}

constexpr int EXT_NONE = -1, EXT_ANY = 100;

// Y of 64 rows (block x) and every gridDim.y-th slab of 128 columns, 16 rows a wave. A wave
// keeps its rows' u in registers, added over its parts and scaled (for bf16 products as
// three bf16 parts, 24 bits). B_a goes slab by slab through registers and two buffers in
// LDS, its loads in flight during the slab before. MFMA t has the columns 8 j + t on its
// lanes j, so that a lane ends with eight consecutive columns of four rows, and 16 lanes
// with 256 bytes of a bf16 row: base, residual and Y move in whole lines. 8192 x 4096 rank
// 64: 33 us, 4.1 TB/s of base and Y, waves waiting 43 % of their time; 8192 x 4608 rank 32
// with a tanh GELU: 38 us, the vector ALU busy three quarters of it. SU: k-steps of the
// product. EXT: EXT_NONE (no activation, gate or residual), an activation known here, or
// EXT_ANY: a short launch has to fetch its code first, and the first kind is a third of the
// last. As EXT_ANY and by themselves: 1500 x 1152 -> 2304 rank 16, nothing 8.1 and 6.7 us, SiLU
// 8.8 and 8.2, tanh GELU 9.0 and 8.4; both products of 8192 x 4096 -> 4096 rank 64, nothing
// 61.7 and 59.5, of 8192 x 1152 -> 4608 rank 32, SiLU 38.7 and 37.9, tanh GELU 39.2 and 38.5.
// ReLU (8.5 and 37.1) and GELU (41.2), gates and residuals have no kernel of their own.
template <typename TE, typename TY, int SU, int EXT>
__global__ __launch_bounds__(256, SU > 2 ? 1 : 3) void adapt_up_tile_kernel(AdaptArgs k) {
  using F = Frag<TE>;
  constexpr int NP = sizeof(TE) == 2 ? 3 : 1;
  constexpr uint32_t ES = sizeof(TE), EY = sizeof(TY);
  constexpr uint32_t PITCH = SU * 64 + 16;   // bytes of a row in LDS
  constexpr int NB = 2 * SU;                 // 16-byte pieces of a slab per thread
  __shared__ __attribute__((aligned(16))) uint8_t bs[2][128 * PITCH];
  const int lane = int(threadIdx.x) & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int64_t r0 = tile_of_block() * 64;
  if (r0 >= k.T) return;
  const int s0 = int(blockIdx.y), s1 = (k.N + 127) / 128, sd = int(gridDim.y);
  const uint32_t brow = uint32_t(k.rank) * ES;   // bytes of a row of B
  const uint32_t ppr = brow / 16, npiece = 128 * ppr;
  const int id = tile_id(k, r0, lane);
  const uint64_t all = __ballot(id >= 0);
  // Memory is reached through buffer descriptors: what lies outside reads as zero and is
  // not written, without a branch, so the waits count the loads and stores that follow.
  // (slab, left): the next product; left has the tile's rows whose adapters are to come
  auto next_of = [&](int& slab, uint64_t& left) {
    left &= ~__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(left)));
    if (!left) {
      left = all;
      slab += sd;
    }
  };
  uint4 bq[NB];
  auto load_b = [&](int slab, uint64_t left) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const __amdgpu_buffer_rsrc_t B = make_rsrc(static_cast<const uint8_t*>(k.b) + int64_t(a) * k.N * brow,
                                               slab < s1 ? int(k.N * brow) : 0);
#pragma unroll
    for (int z = 0; z < NB; ++z) {
      const uint32_t q = threadIdx.x + 256 * z;
      bq[z] = buf_load16(B, q < npiece ? 128 * slab * brow + 16 * q : kOutside);
    }
  };
  // the lane's rows are 4 g + e of the wave's 16
  const int64_t w0 = r0 + 16 * w;
  const int wrows = int(max(min(k.T - w0, int64_t(16)), int64_t(0)));
  const uint32_t inside = (1u << wrows) - 1;
  const uint32_t rowb = uint32_t(k.N) * EY, at0 = 4 * g * rowb + 8 * i * EY;
  const int span = int(wrows * rowb);
  const __amdgpu_buffer_rsrc_t base = make_rsrc(static_cast<const uint8_t*>(k.base) + w0 * k.N * EY, k.base ? span : 0);
  const __amdgpu_buffer_rsrc_t Y = make_rsrc(static_cast<const uint8_t*>(k.ep.Y) + w0 * k.N * EY, span);
  constexpr int H = EY / 2;   // 16-byte halves of eight values
  uint4 bb[4][H];
  auto load_base = [&](int slab) {
    const uint32_t at = 128 * slab + 8 * i < k.N ? at0 + 128 * slab * EY : kOutside;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int h = 0; h < H; ++h) bb[e][h] = buf_load16(base, at + e * rowb + 16 * h);
  };
  // The wave's u goes through its part of the second buffer: read in whole lines, PARTS
  // parts of K at a time, and added in their order (read as the products take it, a part
  // after the other, 256 rows of 2776 -> 4448 rank 128 fp32 take 96 us, 68 so).
  constexpr uint32_t UP = F::KS * SU * 4 + 32;   // bytes of a row there
  constexpr int NU = SU * F::KS / 16;            // 16-byte pieces of a part per lane
  constexpr int PARTS = NU > 4 ? 1 : SU > 1 ? 2 : 4;
  static_assert(4 * 16 * UP <= sizeof(bs[1]), "u of four waves");
  uint8_t* const us = bs[1] + w * 16 * UP;
  float4 uq[PARTS][NU];
  auto load_u = [&](int n) {
#pragma unroll
    for (int j = 0; j < PARTS; ++j) {
      const __amdgpu_buffer_rsrc_t U = make_rsrc(reinterpret_cast<const uint8_t*>(k.u + ((n + j) * k.T + w0) * k.rank),
                                                 n + j < k.splits ? wrows * k.rank * 4 : 0);
#pragma unroll
      for (int z = 0; z < NU; ++z) uq[j][z] = __builtin_bit_cast(float4, buf_load16(U, 16 * (lane + 64 * z)));
    }
  };
  load_u(0);
  if (all) load_b(s0, all);
  load_base(s0);
  // row n of a slab is row (n mod 8) 16 + n / 8 in LDS: the 16 lanes of MFMA t read neighbours
  uint32_t to[NB];
#pragma unroll
  for (int z = 0; z < NB; ++z) {
    const uint32_t q = threadIdx.x + 256 * z, n = q / ppr;
    to[z] = ((n & 7) * 16 + (n >> 3)) * PITCH + 16 * (q - n * ppr);
  }
  F fu[SU][NP] = {};   // row i's u, rank indexes KS s + PER g ..
  {
    const int a = __shfl(id, 16 * w + i, 64);
    const float scale = a >= 0 && k.scales ? k.scales[a] : 1.0f;
    float4 sum[NU] = {};
#pragma unroll 1
    for (int n = 0;;) {
#pragma unroll
      for (int j = 0; j < PARTS; ++j)
#pragma unroll
        for (int z = 0; z < NU; ++z) {
          sum[z].x += uq[j][z].x; sum[z].y += uq[j][z].y; sum[z].z += uq[j][z].z; sum[z].w += uq[j][z].w;
        }
      n += PARTS;
      if (n >= k.splits) break;
      load_u(n);
    }
#pragma unroll
    for (int z = 0; z < NU; ++z) {
      const uint32_t q = 4 * (lane + 64 * z), r = q / uint32_t(k.rank);
      if (r < 16) *reinterpret_cast<float4*>(us + r * UP + 4 * (q - r * k.rank)) = sum[z];
    }
    wave_lds_sync();
#pragma unroll
    for (int s = 0; s < SU; ++s) {
      float f[F::PER];
      const bool has = a >= 0 && F::KS * s + F::PER * g < k.rank;
#pragma unroll
      for (int h = 0; h < F::PER / 4; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(us + i * UP + 4 * (F::KS * s + F::PER * g + 4 * h));
        f[4 * h] = has ? q.x * scale : 0.0f;
        f[4 * h + 1] = has ? q.y * scale : 0.0f;
        f[4 * h + 2] = has ? q.z * scale : 0.0f;
        f[4 * h + 3] = has ? q.w * scale : 0.0f;
      }
      if constexpr (NP == 1) {
        fu[s][0].q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      } else {
#pragma unroll
        for (int p3 = 0; p3 < NP; ++p3) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
            f[2 * e] -= __uint_as_float(h[e] << 16);
            f[2 * e + 1] -= __uint_as_float(h[e] & 0xFFFF0000u);
          }
          fu[s][p3].q = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
  }
  if (brow < SU * 64) {   // rank indexes past the last one
    lds_barrier();        // every wave has its u
    for (uint32_t o = threadIdx.x; o < 2 * 128 * PITCH / 16; o += 256)
      reinterpret_cast<uint4*>(bs)[o] = make_uint4(0, 0, 0, 0);
  }
  // Y of row 4 g + e of the wave in a slab, from v = base + what the adapter adds, where ok
  auto finish = [&](float (&v)[8], int e, int slab, bool ok) {
    uint32_t at = at0;
    asm volatile("" : "+v"(at));   // addresses made here, not kept over the slabs
    at += e * rowb + 128 * slab * EY;
    ok = ok && 128 * slab + 8 * i < k.N;
    if constexpr (EXT != EXT_NONE) {
      float t[8];
      ActCoef act = k.ep.act;
      if constexpr (EXT != EXT_ANY) act.act = EXT;
      apply_act<8, EY == 4>(v, act);
      if (k.ep.gate) {
        if (ok) raw_get(raw_load(static_cast<const TY*>(k.ep.gate) + 128 * slab + 8 * i +
                                 int64_t(uint32_t(w0 + 4 * g + e) / uint32_t(k.ep.gate_rows)) * k.ep.gate_ld), t);
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] *= t[x];
      }
      if (k.ep.residual) {
        if (ok) raw_get(raw_at<TY>(static_cast<const uint8_t*>(k.ep.residual) + w0 * k.N * EY, at), t);
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] += t[x];
      }
    }
    if (!ok) at = kOutside;
    if constexpr (EY == 2) {
      buf_store16(Y, at, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        buf_store16(Y, at + 16 * h, make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])));
    }
  };
  auto base_of = [&](int e, float (&v)[8]) {
    Raw8<TY> r;
#pragma unroll
    for (int h = 0; h < H; ++h) r.q[h] = bb[e][h];
    raw_get(r, v);
  };
  const uint32_t none = uint32_t(~all >> (16 * w)) & inside;   // rows without an adapter
  if (none) {
#pragma unroll 1
    for (int slab = s0; slab < s1; slab += sd) {
      float v[4][8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        base_of(e, v[e]);
#pragma unroll
        for (int x = 0; x < 8; ++x) asm volatile("" : "+v"(v[e][x]));   // bb is free
      }
      load_base(slab + sd);   // past the last slab nothing is read
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        finish(v[e], e, slab, (none >> (4 * g + e)) & 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (all) load_base(s0);
  }
  if (!all) return;
  auto store_b = [&](int buf) {
#pragma unroll
    for (int z = 0; z < NB; ++z)
      if (threadIdx.x + 256 * z < npiece) *reinterpret_cast<uint4*>(bs[buf] + to[z]) = bq[z];
  };
  if (brow < SU * 64) lds_barrier();
  store_b(0);
  int slab = s0, bslab = s0, buf = 0;
  uint64_t left = all, bleft = all;   // the product that is computed, the one that is loaded
  next_of(bslab, bleft);
  load_b(bslab, bleft);
  lds_barrier();
#pragma unroll 1
  while (slab < s1) {
    store_b(buf ^ 1);
    next_of(bslab, bleft);
    load_b(bslab, bleft);
    const uint64_t match = __ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(left)));
    const uint32_t here = uint32_t(match >> (16 * w)) & inside;   // the wave's rows that have it
    v4f d[8] = {};
    // fp32 products take the matrix units long enough to leave them to waves that have rows of
    // this adapter (5783 x 312 -> 3512 rank 32, runs of 88 rows: 66 -> 61 us; bf16 no gain)
    if (sizeof(TE) == 2 || here) {
#pragma unroll
      for (int s = 0; s < SU; ++s) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          F fb;
          fb.q = *reinterpret_cast<const uint4*>(bs[buf] + (16 * t + i) * PITCH + 64 * s + 16 * g);
#pragma unroll
          for (int p = 0; p < NP; ++p) d[t] = frag_mfma<TE>(fu[s][p], fb, d[t]);
          if ((t & 3) == 3) __builtin_amdgcn_sched_barrier(0);   // four reads ahead, no more registers
        }
      }
    }
    float v[4][8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      base_of(e, v[e]);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        v[e][x] += d[x][e];
        asm volatile("" : "+v"(v[e][x]));   // single registers from here, not the MFMA's fours
      }
    }
    const int was = slab;
    next_of(slab, left);
    load_base(slab);   // past the last slab nothing is read
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      finish(v[e], e, was, (here >> (4 * g + e)) & 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    lds_barrier();   // this product is read, the next one written
    buf ^= 1;
  }
}

namespace {

int down_splits(int64_t T, int K, int es) {
  const int64_t tiles = (T + 31) / 32, chunks = (int64_t(K) * es + 127) / 128;
  return int(std::max<int64_t>(1, std::min(256 / tiles, (chunks + 7) / 8)));
}

template <typename TE, int MT, int RT, int NW>
hipError_t launch_down(const AdaptArgs& a, hipStream_t s) {
  const dim3 grid(unsigned((a.T + 16 * MT - 1) / (16 * MT) + 7) / 8 * 8, unsigned(a.splits));
  hipLaunchKernelGGL((adapt_down_tile_kernel<TE, MT, RT, NW>), grid, dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}
template <typename TE, typename TY, int SU>
hipError_t launch_up(AdaptArgs a, hipStream_t s) {
  const int64_t tiles = (a.T + 63) / 64, slabs = (a.N + 127) / 128;
  // column groups: up to 12 per row tile, more where that leaves CUs without a block, whole
  // slabs each (both products, 8192 rows: 36 slabs rank 32, 4 groups 37.6 us, 8 36.8, 12 38.4,
  // 36 40.8; 32 slabs rank 64, 4 63.4, 8 60.8, 12 59.5, 16 60.7, 32 63.4; this one, 1000 rows,
  // 19 slabs: 8 8.9, 12 7.2, 19 6.6)
  const int64_t groups = std::max<int64_t>(12, 512 / tiles);
  a.slabs = int((slabs + groups - 1) / groups);
  const dim3 grid(unsigned(tiles + 7) / 8 * 8, unsigned((slabs + a.slabs - 1) / a.slabs));
  const int act = a.ep.act.act;
  if (act == ACT_NONE && !a.ep.gate && !a.ep.residual)
    hipLaunchKernelGGL((adapt_up_tile_kernel<TE, TY, SU, EXT_NONE>), grid, dim3(256), 0, s, a);
  else if (act == ACT_SILU)
    hipLaunchKernelGGL((adapt_up_tile_kernel<TE, TY, SU, ACT_SILU>), grid, dim3(256), 0, s, a);
  else if (act == ACT_GELU_TANH)
    hipLaunchKernelGGL((adapt_up_tile_kernel<TE, TY, SU, ACT_GELU_TANH>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((adapt_up_tile_kernel<TE, TY, SU, EXT_ANY>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}
template <typename TE, typename TY>
hipError_t launch_up_typed(const AdaptArgs& a, hipStream_t s) {
  const int steps = (a.rank + Frag<TE>::KS - 1) / Frag<TE>::KS;
  if (steps <= 1) return launch_up<TE, TY, 1>(a, s);
  if (steps <= 2) return launch_up<TE, TY, 2>(a, s);
  if (steps <= 4) return launch_up<TE, TY, 4>(a, s);
  if constexpr (sizeof(TE) == 4) return launch_up<TE, TY, 8>(a, s);
  return hipErrorInvalidValue;
}
template <typename TE>
hipError_t launch_tiles(AdaptArgs a, hipStream_t s) {
  a.splits = down_splits(a.T, a.K, int(sizeof(TE)));
  const hipError_t e = a.rank <= 16   ? launch_down<TE, 2, 1, 8>(a, s)
                       : a.rank <= 32 ? launch_down<TE, 2, 2, 8>(a, s)
                       : a.rank <= 64 ? launch_down<TE, 2, 4, 8>(a, s)
                                      : launch_down<TE, 2, 8, 4>(a, s);
  if (e != hipSuccess) return e;
  return a.ep.y_bf16 ? launch_up_typed<TE, uint16_t>(a, s) : launch_up_typed<TE, float>(a, s);
}

template <typename TE, int JW, int U>
hipError_t launch_rows(const AdaptArgs& a, hipStream_t s) {
  // parts of the columns: a unit of 64 per wave at best, and no more blocks than run at
  // once, two to a CU up to rank 32 (24 rows of 4096 -> 4096 rank 16: 1 part 12.2 us, 2 8.6,
  // 4 6.8, 8 5.9; 64 rows, rank 64: 2 parts 19.9, 4 15.6, 6 24)
  const int64_t most = (JW > 4 ? 256 : 512) / a.T;
  const int64_t parts = std::min<int64_t>((a.N + 511) / 512, std::max<int64_t>(1, most));
  hipLaunchKernelGGL((adapt_rows_kernel<TE, JW, U>), dim3(unsigned(a.T), unsigned(parts)), dim3(512), 0, s, a);
  return hipGetLastError();
}
template <typename TE>
hipError_t launch_rows(const AdaptArgs& a, hipStream_t s) {
  if (a.rank <= 8) return launch_rows<TE, 1, 8>(a, s);
  if (a.rank <= 16) return launch_rows<TE, 2, 4>(a, s);
  if (a.rank <= 32) return launch_rows<TE, 4, 2>(a, s);
  if (a.rank <= 64) return launch_rows<TE, 8, 2>(a, s);
  return launch_rows<TE, 16, 1>(a, s);
}

// One row after the other or tiles of rows? Row by row each row fetches its adapter's
// factors (from the caches), in tiles each adapter of a tile is fetched once, but there
// are two launches and a chain of waits in each. The ids are on the device, so the rule counts
// products alone, and batches of a decoding step's size count as mixed up to 2^27 products, 256
// rows of 4096 -> 4096 rank 64. Rows / tiles, a call among others, and the kernels alone (us,
// no epilogue, bf16 but for the third):
//   700 rows of 1024 -> 1024 rank 8, 11 million       9.0 / 13.3    7.8 / 10.0
//   600 of 2048 -> 2048 rank 16, 39 million          11.4 / 13.1   12.0 / 9.8
//   1037 of 2160 -> 2312 rank 8 fp32, 37 million     20.4 / 18.0   20.8 / 18.0
//   300 of 4096 -> 1152 rank 32, 50 million          12.9 / 13.1   13.5 / 9.9
//   1000 of 1160 -> 2312 rank 32, 111 million        24.1 / 13.1   25.0 / 12.5
//   4000 of 256 -> 512 rank 16, 49 million                         21.6 / 9.9
//   512 of 2048 -> 2048 rank 32, one adapter         13.6 / 13.0   14.7 / 8.7
//   256 of 2048 -> 2048 rank 32, 64 adapters mixed   13.4 / 73     13.6 / 73
//   512 of 2048 -> 2048 rank 32, 128 adapters mixed  21.3 / 94
//   256 of 4096 -> 4096 rank 64, 64 adapters mixed   40.7 / 113; one adapter 27.0 / 12.8
// Mixed rows past the limit take the tiles' passes: 128 rows of 4096 -> 14336 rank 64 with 32
// adapters 146 us (row by row 50).
bool by_rows(int64_t T, int K, int N, int rank) {
  const double products = double(T) * rank * (double(K) + N);
  return T <= 4 || (T <= 512 && products <= 0x1p27) || (T <= 2048 && products <= 40e6);
}

}  // namespace

size_t adapters_part_bytes(int64_t T, int K, int N, int rank, int esize) {
  if (by_rows(T, K, N, rank)) return 0;
  return size_t(down_splits(T, K, esize)) * size_t(T) * size_t(rank) * 4;
}

hipError_t launch_adapters(const AdaptArgs& a, hipStream_t s) {
  if (by_rows(a.T, a.K, a.N, a.rank))
    return a.bf16 ? launch_rows<uint16_t>(a, s) : launch_rows<float>(a, s);
  return a.bf16 ? launch_tiles<uint16_t>(a, s) : launch_tiles<float>(a, s);
}

}  // namespace hq
