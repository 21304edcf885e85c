// The down products of rows of many adapters: U_i = X_i A_a^T with a the
// adapter of row i, as fp32 partial sums over slices of K (the tile kernels
// add the slices where they take U).
//
// Bound by reading X and the adapters once.  A workgroup owns 64 rows and one
// slice of K.  The adapters that its rows have, taken from their indices,
// make a list of units of 16 adapter rows each; the workgroup multiplies all
// its rows with up to four units at a time (MFMA 16x16x32, operands straight
// from memory in fragment layout: each is used once) and keeps, of every
// unit, the rows that have its adapter.  So a unit is read once per 64 rows
// whatever the order of the rows, and rows in runs (prompts) meet one or two
// adapters.  The products with other rows' adapters are thrown away: at 64
// rows of 64 adapters 63 of 64, still far below the time that reading the
// adapters takes.  The four waves split the slice and add up in LDS.
#include "kernels.hpp"

namespace qn {
namespace {

constexpr int kRows = 64;    // rows per workgroup
constexpr int kUnits = 4;    // units of 16 adapter rows at a time
constexpr int kRedLd = 20;   // LDS row stride: the four row quarters of a wave in different banks

struct DownArgs {
  const uint16_t* X;
  int64_t M, K;
  const uint16_t* A;    // [adapters][r][K]
  int r, adapters;
  const int32_t* index;
  float* part;          // [slices][M][ldp]
  int64_t ldp, slice;   // ceil(r / 8) * 8; columns per slice
  int slices, groups;   // workgroups that share a tile's units
};

// The products of the tile's rows with `NU` units, of which unit u has the
// adapter rows at arow[u] (this lane's).
template <int NU>
__device__ __forceinline__ void products(f32x4 (&acc)[4][kUnits], const uint16_t* const (&xrow)[4],
                                         const uint16_t* const (&arow)[kUnits], int64_t k0,
                                         int64_t k1) {
  constexpr int kDepth = 2;  // steps whose loads are in flight together
  int64_t k = k0;
  for (; k + 32 * kDepth <= k1; k += 32 * kDepth) {
    u32x4 x[kDepth][4], a[kDepth][NU];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[d][i] = *reinterpret_cast<const u32x4*>(xrow[i] + k + 32 * d);
#pragma unroll
      for (int u = 0; u < NU; ++u) a[d][u] = *reinterpret_cast<const u32x4*>(arow[u] + k + 32 * d);
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < NU; ++u)
          acc[i][u] = mfma16(as_bf16x8(x[d][i]), as_bf16x8(a[d][u]), acc[i][u]);
  }
  for (; k < k1; k += 32)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(xrow[i] + k);
#pragma unroll
      for (int u = 0; u < NU; ++u)
        acc[i][u] = mfma16(as_bf16x8(x), as_bf16x8(*reinterpret_cast<const u32x4*>(arow[u] + k)),
                           acc[i][u]);
    }
}

__global__ __launch_bounds__(256) void k_multi_down(DownArgs p) {
  __shared__ int row_a[kRows];
  __shared__ int list[kRows];
  __shared__ int found;
  __shared__ __attribute__((aligned(16))) float red[4][kRows * kRedLd];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t id = blockIdx.x;
  const int group = (int)(id % p.groups);
  id /= p.groups;
  const int s = (int)(id % p.slices);
  const int64_t m0 = id / p.slices * kRows;
  if (wave == 0) {
    int a = m0 + lane < p.M ? p.index[m0 + lane] : -1;
    if ((unsigned)a >= (unsigned)p.adapters) a = -1;
    bool first = a >= 0;
#pragma unroll 8
    for (int t = 0; t < 63; ++t)
      if (__builtin_amdgcn_readlane(a, t) == a && t < lane) first = false;
    const uint64_t mask = __builtin_amdgcn_ballot_w64(first);
    row_a[lane] = a;
    if (first) list[__builtin_popcountll(mask & (((uint64_t)1 << lane) - 1))] = a;
    if (lane == 0) found = __builtin_popcountll(mask);
  }
  __syncthreads();
  const int per = (p.r + 15) >> 4;  // units of an adapter
  const int total = found * per;
  const int64_t c0 = s * p.slice, c1 = c0 + p.slice < p.K ? c0 + p.slice : p.K;
  // this wave's columns (multiples of 32)
  const int64_t steps = (c1 - c0) >> 5;
  const int64_t k0 = c0 + 32 * (steps * wave >> 2), k1 = c0 + 32 * (steps * (wave + 1) >> 2);
  const int i16 = lane & 15, q = lane >> 4;
  const uint16_t* xrow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int64_t m = m0 + 16 * i + i16;
    if (m >= p.M) m = p.M - 1;  // computed and dropped
    xrow[i] = p.X + m * p.K + 8 * q;
  }
  for (int u0 = group * kUnits; u0 < total; u0 += p.groups * kUnits) {
    const int nu = total - u0 < kUnits ? total - u0 : kUnits;
    const uint16_t* arow[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int v = u < nu ? u0 + u : u0, ai = v / per;
      int j = 16 * (v - ai * per) + i16;
      if (j >= p.r) j = p.r - 1;  // computed and dropped
      arow[u] = p.A + ((int64_t)list[ai] * p.r + j) * p.K + 8 * q;
    }
    f32x4 acc[4][kUnits];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) acc[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (nu > 2) products<4>(acc, xrow, arow, k0, k1);
    else if (nu == 2) products<2>(acc, xrow, arow, k0, k1);
    else products<1>(acc, xrow, arow, k0, k1);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (u >= nu) break;  // uniform
      __syncthreads();     // the last unit's sums have been read
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[wave][(16 * i + 4 * q + v) * kRedLd + i16] = acc[i][u][v];
      __syncthreads();
      const int row = tid >> 2, c = 4 * (tid & 3);
      const int ai = (u0 + u) / per, j = 16 * (u0 + u - ai * per) + c;
      if (row_a[row] == list[ai] && j < p.ldp) {
        f32x4 sum = *reinterpret_cast<const f32x4*>(&red[0][row * kRedLd + c]);
#pragma unroll
        for (int w = 1; w < 4; ++w) sum += *reinterpret_cast<const f32x4*>(&red[w][row * kRedLd + c]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e >= p.r) sum[e] = 0.0f;
        *reinterpret_cast<f32x4*>(p.part + (s * p.M + m0 + row) * p.ldp + j) = sum;
      }
    }
  }
}

}  // namespace

// Slices of at least 512 columns, as many as give the chip about two
// workgroups per compute unit, 8 at most (the tile kernels add them up).
int multi_down_slices(int64_t M, int64_t K) {
  const int64_t tiles = (M + kRows - 1) / kRows;
  int64_t s = (512 + tiles - 1) / tiles;
  if (s > K / 512) s = K / 512;
  if (s > 8) s = 8;
  if (s < 1) s = 1;
  // no slice is empty
  const int64_t len = ((K + s - 1) / s + 31) / 32 * 32;
  return (int)((K + len - 1) / len);
}

size_t multi_down_bytes(int64_t M, int64_t K, int32_t r) {
  return (size_t)multi_down_slices(M, K) * M * ((r + 7) / 8 * 8) * sizeof(float);
}

hipError_t launch_multi_down(const uint16_t* X, int64_t M, int64_t K, const uint16_t* A, int32_t r,
                             int adapters, const int32_t* index, float* part, hipStream_t stream) {
  DownArgs a{X, M, K, A, r, adapters, index, part, (r + 7) / 8 * 8, 0, multi_down_slices(M, K), 1};
  a.slice = ((K + a.slices - 1) / a.slices + 31) / 32 * 32;
  // Up to 64 adapters per tile: the units are shared by as many workgroups as
  // there can be sets of four, while the chip is not full.
  const int64_t tiles = (M + kRows - 1) / kRows;
  const int64_t most = ((M < kRows ? M : kRows) < adapters ? (M < kRows ? M : kRows) : adapters) *
                       ((r + 15) / 16);
  int64_t groups = (most + kUnits - 1) / kUnits;
  const int64_t fill = (2048 + tiles * a.slices - 1) / (tiles * a.slices);
  if (groups > fill) groups = fill;
  a.groups = (int)(groups < 1 ? 1 : groups);
  const int64_t wgs = tiles * a.slices * a.groups;
  if (wgs >= (int64_t)1 << 24) return hipErrorInvalidValue;  // (M is checked before)
  k_multi_down<<<dim3((unsigned)wgs), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace qn
