// The down products of rows of many adapters: U_i = X_i A_a^T with a the
// adapter of row i, times the adapter's scale, as fp32 partial sums over
// slices of K (the kernels that take U add the slices).
//
// Bound by reading X and the adapters once.  A workgroup owns 64 rows and one
// slice of K.  The adapters that its rows have, taken from their indices,
// make a list of units of 16 adapter rows each; the workgroup multiplies all
// its rows with up to four units at a time and keeps, of every unit, the rows
// that have its adapter.  So a unit is read once per 64 rows whatever the
// order of the rows, and rows in runs (prompts) meet one or two adapters.
// The products with other rows' adapters are thrown away: at 64 rows of 64
// adapters 63 of 64, still far below the time that reading the adapters takes.
//
// The four waves split the slice, each with its own piece of LDS, so nothing
// but the final sum over the waves needs a barrier.  A wave moves 64 columns
// at a time as whole lines (8 lanes per row) into LDS and reads the MFMA
// fragments there; loads in fragment layout, whose neighbouring lanes lie in
// different rows, cost the memory pipe a cycle per lane (4096 rows of K =
// 4096, rank 64, 5 adapters: 54 us against 21; 61 rows of K = 8192, rank 32, 24
// adapters, 13 MB of them: 13 us).
//
// Before the tile kernels the rows are put in order first (k_multi_order): the
// rows of each window of 4096 by adapter, so that a tile meets few of them
// (4096 rows that take 64 adapters of rank 64 in turn: 64 contraction steps
// more per tile, 1685 us, against 457).
//
// For the kernel of qrows.hip the X fragments are also written out in its
// order, 1 KB per 16 rows and 32 columns.
#include "kernels.hpp"

namespace qn {
namespace {

constexpr int kRows = 64;    // rows per workgroup
constexpr int kUnits = 4;    // units of 16 adapter rows at a time
constexpr int kLd = 72;      // LDS row stride of a 64-column tile
constexpr int kTile = 64 * kLd;
constexpr int kRedLd = 68;   // floats: the four row quarters of a wave in different banks

// order[w + rank of row w + i] = w + i for the rows of window w .. w +
// kMultiWindow - 1, ranked by adapter (rows without one last), rows of one
// adapter in their order.  A workgroup ranks 16 rows by counting, over all of
// the window, the rows that come before each: 16 lanes share a row (sorting a
// window in one workgroup took 37 us for 4096 rows, this 8).
constexpr int kOrderRows = 16, kOrderParts = 16;

struct __attribute__((packed, aligned(4))) Loose4 {
  u32x4 v;
};

__global__ __launch_bounds__(256) void k_multi_order(const int32_t* index, int64_t M, int adapters,
                                                     int32_t* order) {
  __shared__ __attribute__((aligned(16))) uint32_t key[kMultiWindow];
  __shared__ int before[kOrderParts][kOrderRows];
  const int64_t first = (int64_t)blockIdx.x * kOrderRows, w0 = first / kMultiWindow * kMultiWindow;
  const int n = (int)(M - w0 < kMultiWindow ? M - w0 : kMultiWindow);
  const int tid = threadIdx.x;
  const auto key_of = [&](uint32_t a) { return a < (uint32_t)adapters ? a : 0x80000000u; };
  constexpr int kLoads = kMultiWindow / 4 / 256;
  u32x4 v[kLoads];
#pragma unroll
  for (int l = 0; l < kLoads; ++l) {
    const int j = 4 * (tid + 256 * l);
    v[l] = u32x4{~0u, ~0u, ~0u, ~0u};
    if (j + 4 <= n) {
      v[l] = reinterpret_cast<const Loose4*>(index + w0 + j)->v;
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (j + e < n) v[l][e] = (uint32_t)index[w0 + j + e];
    }
  }
#pragma unroll
  for (int l = 0; l < kLoads; ++l) {
    const int j = 4 * (tid + 256 * l);
    if (j < n) {
      u32x4 k;  // past the last row: after everything
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = j + e < n ? key_of(v[l][e]) : ~0u;
      *reinterpret_cast<u32x4*>(key + j) = k;
    }
  }
  __syncthreads();
  const int i = (int)(first - w0) + tid % kOrderRows, part = tid / kOrderRows;
  const uint32_t mine = i < n ? key[i] : 0u;
  const int quads = (n + 3) >> 2;
  int count = 0;
#pragma unroll 4
  for (int q = part; q < quads; q += kOrderParts) {
    const u32x4 k = *reinterpret_cast<const u32x4*>(key + 4 * q);
#pragma unroll
    for (int e = 0; e < 4; ++e) count += k[e] < mine + (4 * q + e < i ? 1u : 0u);
  }
  before[part][tid % kOrderRows] = count;
  __syncthreads();
  if (tid < kOrderRows && i < n) {
    int rank = 0;
#pragma unroll
    for (int w = 0; w < kOrderParts; ++w) rank += before[w][tid];
    order[w0 + rank] = (int32_t)(w0 + i);
  }
}

struct DownArgs {
  const uint16_t* X;
  int64_t M, K;
  const uint16_t* A;    // [adapters][r][K]
  int r, adapters;
  const float* scales;
  const int32_t* index;
  float* part;          // [slices][M][ldp], times the adapter's scale
  int64_t ldp, slice;   // ceil(r / 8) * 8; columns per slice (a multiple of 64)
  int slices, groups;   // `groups` workgroups share a tile's units ...
  int take;             // ... `take` at a time (1 .. kUnits)
  uint32_t wgs;         // workgroups of a group
  const int32_t* order; // [M]: the rows in the order of the tiles, or null
  uint16_t* xfrag;      // [ceil(M / 16)][K / 64][2][64 lanes][8], or null
};

struct Tiles {
  const DownArgs& p;
  uint16_t* xs;         // this wave's [64][kLd]
  uint16_t* as;
  __amdgpu_buffer_rsrc_t xrs;
  int lane;
  int xoff[8];          // byte offsets of this lane's rows and chunk in X
  int aoff;             // ... and in a unit, rows of 8 apart
  int rows8;            // bytes of 8 rows (K at most 2^22)
  int64_t m0;
};

// 64 columns from column k on of the tile's rows.
__device__ __forceinline__ void load_x(u32x4 (&x)[8], const Tiles& t, int64_t k) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = __builtin_amdgcn_raw_buffer_load_b128(t.xrs, t.xoff[i], (int)(2 * k), 0);
}

// The products of the tile's rows with NU units (rows of a unit through
// ars[u]) over the columns [k0, k1), and the X fragments written out.  x holds
// the first columns.  Two steps are in flight: the loads of the next but one
// go out as soon as the registers are free.
template <int NU>
__device__ __forceinline__ void products(const Tiles& t, u32x4 (&x0)[8], f32x4 (&acc)[4][kUnits],
                                         const __amdgpu_buffer_rsrc_t (&ars)[kUnits], int64_t k0,
                                         int64_t k1, bool write_x) {
  constexpr int NA = NU > 0 ? 2 * NU : 1;
  const int lane = t.lane, i16 = lane & 15, q = lane >> 4;
  u32x4 a0[NA], x1[8], a1[NA];
  auto load_a = [&](u32x4 (&a)[NA], int64_t k) {
#pragma unroll
    for (int i = 0; i < 2 * NU; ++i)
      a[i] = __builtin_amdgcn_raw_buffer_load_b128(ars[i >> 1], t.aoff + (i & 1) * t.rows8,
                                                   (int)(2 * k), 0);
  };
  const int at = (lane >> 3) * kLd + (lane & 7) * 8;
  const int xo = 32 * (q & 1) + 16 * (q >> 1);  // the column order of qrows.hip
  // (a wave's LDS accesses complete in order; this keeps them in order)
  auto ordered = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  auto step = [&](u32x4 (&x)[8], u32x4 (&a)[NA], int64_t k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<u32x4*>(t.xs + at + 8 * i * kLd) = x[i];
#pragma unroll
    for (int i = 0; i < 2 * NU; ++i) *reinterpret_cast<u32x4*>(t.as + at + 8 * i * kLd) = a[i];
    if (k + 128 < k1) {
      load_x(x, t, k + 128);
      load_a(a, k + 128);
    }
    ordered();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x4 xf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xf[i] = *reinterpret_cast<const u32x4*>(t.xs + (16 * i + i16) * kLd + xo + 8 * j);
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const bf16x8 af =
            as_bf16x8(*reinterpret_cast<const u32x4*>(t.as + (16 * u + i16) * kLd + xo + 8 * j));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][u] = mfma16(as_bf16x8(xf[i]), af, acc[i][u]);
      }
      if (write_x) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t.m0 + 16 * i < t.p.M)  // uniform
            *reinterpret_cast<u32x4*>(
                t.p.xfrag + (((t.m0 >> 4) + i) * (t.p.K >> 5) + (k >> 5) + j) * 512 + lane * 8) = xf[i];
      }
    }
    ordered();
  };
  if (k0 >= k1) return;
  load_a(a0, k0);
  if (k0 + 64 < k1) {
    load_x(x1, t, k0 + 64);
    load_a(a1, k0 + 64);
  }
  for (int64_t k = k0; k < k1; k += 128) {
    step(x0, a0, k);
    if (k + 64 < k1) step(x1, a1, k + 64);
  }
}

__global__ __launch_bounds__(256, 2) void k_multi_down(DownArgs p) {
  __shared__ int row_a[kRows];
  __shared__ int list[kRows];
  __shared__ int found;
  __shared__ __attribute__((aligned(16))) uint16_t tiles[4][2][kTile];
  float* red = reinterpret_cast<float*>(tiles);  // [4][kRows][kRedLd], after the products
  static_assert(4 * kRows * kRedLd * 4 <= sizeof(tiles), "sums over the waves");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // groups outermost: those without units end at once, and neighbouring
  // workgroups go to different XCDs
  const int64_t id = blockIdx.x % p.wgs;
  const int group = (int)(blockIdx.x / p.wgs);
  const int s = (int)(id % p.slices);
  const int64_t m0 = id / p.slices * kRows;
  // this wave's columns
  const int64_t c0 = s * p.slice, c1 = c0 + p.slice < p.K ? c0 + p.slice : p.K;
  const int64_t steps = (c1 - c0) >> 6;
  const int64_t k0 = c0 + 64 * (steps * wave >> 2), k1 = c0 + 64 * (steps * (wave + 1) >> 2);
  // Rows past M and past the adapter's rank lie past the ends of the buffer
  // resources and read 0.
  const int64_t base = p.order ? m0 / kMultiWindow * kMultiWindow : m0;
  const int64_t span = p.order ? kMultiWindow : kRows;
  const int64_t left = p.M - base < span ? p.M - base : span;
  Tiles t{p, tiles[wave][0], tiles[wave][1], bytes_rsrc(p.X + base * p.K, left * p.K * 2), lane,
          {}, (int)((lane >> 3) * p.K * 2) + (lane & 7) * 16, (int)(p.K * 16), m0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = m0 + 8 * i + (lane >> 3);
    if (!p.order) t.xoff[i] = (int)((m - m0) * p.K * 2) + (lane & 7) * 16;
    else t.xoff[i] = m < p.M ? (int)((p.order[m] - base) * p.K * 2) + (lane & 7) * 16 : INT32_MIN;
  }
  u32x4 x[8];
  if (k0 < k1) load_x(x, t, k0);  // under the search for the adapters
  if (wave == 0) {
    int a = -1;
    if (m0 + lane < p.M) a = p.index[p.order ? p.order[m0 + lane] : m0 + lane];
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
  const int total = __builtin_amdgcn_readfirstlane(found) * per;
  const bool write_x = p.xfrag && group == 0;
  if (group * p.take >= total && !write_x) return;
  bool first_pass = true;
  for (int u0 = group * p.take; u0 < total || (first_pass && write_x); u0 += p.groups * p.take) {
    const int nu = total - u0 < p.take ? (total > u0 ? total - u0 : 0) : p.take;
    __amdgpu_buffer_rsrc_t ars[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int v = u < nu ? u0 + u : u0, ai = v / per, j = 16 * (v - ai * per);
      const int64_t a = nu ? __builtin_amdgcn_readfirstlane(list[ai]) : 0;
      const int64_t rows = p.r - j < 16 ? p.r - j : 16;
      ars[u] = bytes_rsrc(p.A + (a * p.r + (nu ? j : 0)) * p.K, nu ? rows * p.K * 2 : 0);
    }
    f32x4 acc[4][kUnits];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) acc[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool wx = write_x && first_pass;
    if (!first_pass && k0 < k1) load_x(x, t, k0);
    if (nu > 2) products<4>(t, x, acc, ars, k0, k1, wx);
    else if (nu == 2) products<2>(t, x, acc, ars, k0, k1, wx);
    else if (nu == 1) products<1>(t, x, acc, ars, k0, k1, wx);
    else products<0>(t, x, acc, ars, k0, k1, wx);
    first_pass = false;
    // the waves' sums, all units at once
    __syncthreads();  // the tiles have been read
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (u >= nu) break;  // uniform
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[(wave * kRows + 16 * i + 4 * (lane >> 4) + v) * kRedLd + 16 * u + (lane & 15)] =
              acc[i][u][v];
    }
    __syncthreads();
    const int row = tid >> 2, c = 4 * (tid & 3);
    for (int u = 0; u < nu; ++u) {
      const int ai = (u0 + u) / per, j = 16 * (u0 + u - ai * per) + c;
      if (row_a[row] == list[ai] && j < p.ldp) {
        f32x4 sum = *reinterpret_cast<const f32x4*>(&red[row * kRedLd + 16 * u + c]);
#pragma unroll
        for (int w = 1; w < 4; ++w)
          sum += *reinterpret_cast<const f32x4*>(&red[(w * kRows + row) * kRedLd + 16 * u + c]);
        const float sc = p.scales[list[ai]];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = j + e < p.r ? sum[e] * sc : 0.0f;
        *reinterpret_cast<f32x4*>(p.part + (s * p.M + m0 + row) * p.ldp + j) = sum;
      }
    }
    __syncthreads();  // the sums have been read before the next pass's tiles
  }
}

int64_t slice_len(int64_t K, int64_t s) { return ((K + s - 1) / s + 63) / 64 * 64; }

}  // namespace

// Slices of at least 512 columns, as many as give the chip about one
// workgroup per compute unit, 8 at most (the kernels that take U add them up).
int multi_down_slices(int64_t M, int64_t K) {
  const int64_t tiles = (M + kRows - 1) / kRows;
  int64_t s = (256 + tiles - 1) / tiles;
  if (s > K / 512) s = K / 512;
  if (s > 8) s = 8;
  if (s < 1) s = 1;
  const int64_t len = slice_len(K, s);  // no slice is empty
  return (int)((K + len - 1) / len);
}

size_t multi_down_bytes(int64_t M, int64_t K, int32_t r) {
  return (size_t)multi_down_slices(M, K) * M * ((r + 7) / 8 * 8) * sizeof(float);
}

size_t multi_xfrag_bytes(int64_t M, int64_t K) { return (size_t)((M + 15) / 16 * 16) * K * 2; }

// A window's rows are addressed with 32-bit offsets.
bool multi_order_takes(int64_t K) { return kMultiWindow * K * 2 < (int64_t)1 << 31; }

hipError_t launch_multi_order(const int32_t* index, int64_t M, int adapters, int32_t* order,
                              hipStream_t stream) {
  static_assert(kMultiWindow % kOrderRows == 0, "a workgroup's rows are in one window");
  k_multi_order<<<dim3((unsigned)((M + kOrderRows - 1) / kOrderRows)), dim3(256), 0, stream>>>(index, M, adapters, order);
  return hipGetLastError();
}

hipError_t launch_multi_down(const uint16_t* X, int64_t M, int64_t K, const uint16_t* A, int32_t r,
                             const float* scales, int adapters, const int32_t* index,
                             const int32_t* order, float* part, uint16_t* xfrag,
                             hipStream_t stream) {
  DownArgs a{};
  a.X = X;
  a.M = M;
  a.K = K;
  a.A = A;
  a.r = r;
  a.adapters = adapters;
  a.scales = scales;
  a.index = index;
  a.order = order;
  a.part = part;
  a.xfrag = xfrag;
  a.ldp = (r + 7) / 8 * 8;
  a.slices = multi_down_slices(M, K);
  a.slice = slice_len(K, a.slices);
  // Up to 64 adapters per tile: the units are shared by as many workgroups as
  // there can be sets of `take`, while the chip is not full; sets of fewer
  // than four where that leaves compute units idle.
  const int64_t wgs = (M + kRows - 1) / kRows * a.slices;
  const int64_t rows = M < kRows ? M : kRows;
  const int64_t most = (rows < adapters ? rows : adapters) * ((r + 15) / 16);
  a.take = kUnits;
  while (a.take > 1 && wgs * ((most + a.take - 1) / a.take) < 256) a.take /= 2;
  int64_t groups = (most + a.take - 1) / a.take;
  const int64_t fill = (1024 + wgs - 1) / wgs;
  if (groups > fill) groups = fill;
  a.groups = (int)(groups < 1 ? 1 : groups);
  a.wgs = (uint32_t)wgs;
  if (wgs * a.groups >= (int64_t)1 << 24) return hipErrorInvalidValue;  // (M is checked before)
  k_multi_down<<<dim3((unsigned)(wgs * a.groups)), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace qn
