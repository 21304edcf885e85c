// The global 2-norm of many gradient tensors, and their scaling by
// min(1, max_norm / (norm + 1e-6)).
//
//   norm = sqrt(sum over tensors, elements of g^2)
//
// Two passes over the data, both bound by HBM: the sum of squares (read
// once), then the scaling (read and written once; nothing is read or written
// when the factor is 1 and the gradients stay where they are).  Squares are
// exact products in fp64 and add up in fp64, so that neither gradients near
// the fp32 limit overflow nor small ones vanish; a workgroup's sum goes to
// its own slot and every workgroup of the second pass adds all slots in the
// same order, so the result is deterministic and needs no third launch.
//
// The tensors' addresses and sizes travel by value in the launch arguments
// (at most kClipTable of them per launch, under the 4 KB of arguments a
// launch takes): no table in device memory has to be filled or kept, and a
// captured launch replays with the addresses it was captured with.
//
// Measured (448 tensors, 320 MB of bf16, into another buffer): 57 us for the
// sums (5.6 TB/s) and 128 us for the scaling (5.0 TB/s), 188 us for the call;
// 14 tensors of one block at rank 8: 19 us, most of it the call's own time.
#include "kernels.hpp"

namespace qn {
namespace {

constexpr int64_t kChunk = 10240;  // elements per unit of work: 20 KB of bf16, 40 KB of fp32
constexpr int kUnroll = 5;         // vectors in flight per thread; a chunk is 5 or 10 per thread
constexpr int kNT = 256;

struct NormTable {
  const void* g[kClipNormTable];
  uint32_t end[kClipNormTable];   // chunks of the tensors up to and including this one
  uint32_t tail[kClipNormTable];  // elements of its last chunk (1 .. kChunk) | fp32 << 31
  int32_t n;
};
struct ScaleTable {
  const void* g[kClipScaleTable];
  void* out[kClipScaleTable];
  uint32_t end[kClipScaleTable];
  uint32_t tail[kClipScaleTable];
  int32_t n;
};
static_assert(sizeof(NormTable) + 64 <= 4096 && sizeof(ScaleTable) + 64 <= 4096,
              "launch arguments");

template <class E>
struct __attribute__((packed, aligned(sizeof(E)))) Loose16 {
  u32x4 v;
};

// Calls f(tensor, first element, elements, fp32?) for the chunks of workgroup
// blockIdx.x: an equal, contiguous share of the table's chunks, so that the
// search for the first one's tensor is done once.
template <class Table, class F>
__device__ __forceinline__ void for_chunks(const Table& tb, F&& f) {
  const uint32_t total = tb.end[tb.n - 1];
  uint32_t c = (uint32_t)((uint64_t)total * blockIdx.x / gridDim.x);
  const uint32_t ce = (uint32_t)((uint64_t)total * (blockIdx.x + 1) / gridDim.x);
  if (c >= ce) return;
  int lo = 0, hi = tb.n - 1;  // the first tensor with end > c
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (tb.end[m] > c) hi = m;
    else lo = m + 1;
  }
  for (; c < ce; ++c) {
    while (tb.end[lo] <= c) ++lo;
    const uint32_t first = lo ? tb.end[lo - 1] : 0u;
    const uint32_t tail = tb.tail[lo];
    const int count = c + 1 == tb.end[lo] ? (int)(tail & 0x7fffffffu) : (int)kChunk;
    f(lo, (int64_t)(c - first) * kChunk, count, (tail >> 31) != 0);
  }
}

__device__ __forceinline__ void add_squares(double& a, const u32x4& v, bool f32) {
  if (f32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double d = word_to_f32(v[e]);
      a = fma(d, d, a);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double l = bf16_lo_to_f32(v[e]), h = bf16_hi_to_f32(v[e]);
      a = fma(l, l, a);
      a = fma(h, h, a);
    }
  }
}

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kNT / 64; ++w) v += s[w];
  __syncthreads();
  return v;
}

template <class E>
__device__ __forceinline__ void chunk_squares(double (&a)[kUnroll], const E* p, int count, bool f32) {
  constexpr int VEC = 16 / (int)sizeof(E);
  const int nv = count / VEC;
  int i = threadIdx.x;
  for (; i + (kUnroll - 1) * kNT < nv; i += kUnroll * kNT) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      v[u] = reinterpret_cast<const Loose16<E>*>(p + (int64_t)(i + u * kNT) * VEC)->v;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add_squares(a[u], v[u], f32);
  }
  for (; i < nv; i += kNT)
    add_squares(a[0], reinterpret_cast<const Loose16<E>*>(p + (int64_t)i * VEC)->v, f32);
  const int j = nv * VEC + threadIdx.x;
  if (j < count) {
    double d;
    if constexpr (sizeof(E) == 4) d = p[j];
    else d = bf16_to_f32(p[j]);
    a[1] = fma(d, d, a[1]);
  }
}

__global__ __launch_bounds__(kNT) void k_grad_squares(NormTable tb, double* __restrict__ part) {
  __shared__ double s[kNT / 64];
  double a[kUnroll] = {};
  for_chunks(tb, [&](int t, int64_t first, int count, bool f32) {
    if (f32) chunk_squares(a, (const float*)tb.g[t] + first, count, true);
    else chunk_squares(a, (const uint16_t*)tb.g[t] + first, count, false);
  });
  double sum = 0.0;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) sum += a[u];
  const double v = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// The norm from all slots, in the same order in every workgroup.
__device__ __forceinline__ double total_norm(const double* part, int slots, double* s) {
  double v = 0.0;
  for (int i = threadIdx.x; i < slots; i += kNT) v += part[i];
  return sqrt(block_sum(v, s));
}

__device__ __forceinline__ u32x4 scale_vec(const u32x4& v, float c, bool f32) {
  u32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    r[e] = f32 ? __builtin_bit_cast(uint32_t, word_to_f32(v[e]) * c)
               : pack_bf16x2(bf16_lo_to_f32(v[e]) * c, bf16_hi_to_f32(v[e]) * c);
  return r;
}

template <class E>
__device__ __forceinline__ void chunk_scale(E* out, const E* p, int count, float c) {
  constexpr int VEC = 16 / (int)sizeof(E);
  constexpr bool f32 = sizeof(E) == 4;
  const int nv = count / VEC;
  int i = threadIdx.x;
  for (; i + (kUnroll - 1) * kNT < nv; i += kUnroll * kNT) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      v[u] = reinterpret_cast<const Loose16<E>*>(p + (int64_t)(i + u * kNT) * VEC)->v;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      // Nontemporal: written through instead of left dirty in the Infinity
      // Cache, whose write-back would share HBM with the next pass's reads
      // (448 tensors, 320 MB: 198 -> 185 us for the whole call).
      __builtin_nontemporal_store(
          scale_vec(v[u], c, f32),
          &reinterpret_cast<Loose16<E>*>(out + (int64_t)(i + u * kNT) * VEC)->v);
  }
  for (; i < nv; i += kNT)
    reinterpret_cast<Loose16<E>*>(out + (int64_t)i * VEC)->v =
        scale_vec(reinterpret_cast<const Loose16<E>*>(p + (int64_t)i * VEC)->v, c, f32);
  const int j = nv * VEC + threadIdx.x;
  if (j < count) {
    if constexpr (f32) out[j] = p[j] * c;
    else out[j] = f32_to_bf16(bf16_to_f32(p[j]) * c);
  }
}

// in_place: out[t] == g[t] for every tensor, which a factor of 1 leaves alone.
__global__ __launch_bounds__(kNT) void k_grad_scale(ScaleTable tb, const double* __restrict__ part,
                                                    int slots, float max_norm, bool in_place,
                                                    float* norm_out) {
  __shared__ double s[kNT / 64];
  const double norm = total_norm(part, slots, s);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // a norm that is NaN gives a factor of NaN, an infinite one a factor of 0, but
  // 1 without a limit (inf / inf)
  const double f = (double)max_norm / (norm + 1e-6);
  const double inf = __builtin_inf();
  const float c = f >= 1.0 || (max_norm == inf && norm == inf) ? 1.0f : (float)f;
  if (in_place && c == 1.0f) return;
  for_chunks(tb, [&](int t, int64_t first, int count, bool f32) {
    if (f32) chunk_scale((float*)tb.out[t] + first, (const float*)tb.g[t] + first, count, c);
    else chunk_scale((uint16_t*)tb.out[t] + first, (const uint16_t*)tb.g[t] + first, count, c);
  });
}

__global__ __launch_bounds__(kNT) void k_grad_norm(const double* __restrict__ part, int slots,
                                                   float* norm_out) {
  __shared__ double s[kNT / 64];
  const double norm = total_norm(part, slots, s);
  if (threadIdx.x == 0) *norm_out = (float)norm;
}

// Fills a launch's table with the tensors from i on towards n (upwards or
// downwards; empty ones are left out) and returns the first that is not in it.
template <class Table, class Add>
int64_t fill(Table& tb, int cap, int64_t i, int64_t n, const int64_t* sizes, const int32_t* types,
             Add&& add) {
  uint32_t end = 0;
  tb.n = 0;
  const int64_t dir = n < i ? -1 : 1;
  for (; i != n && tb.n < cap; i += dir) {
    if (sizes[i] == 0) continue;
    const int64_t chunks = (sizes[i] + kChunk - 1) / kChunk;
    if (end + (uint64_t)chunks > 0x7fffffffu) break;  // the next launch takes it
    end += (uint32_t)chunks;
    tb.end[tb.n] = end;
    tb.tail[tb.n] = (uint32_t)(sizes[i] - (chunks - 1) * kChunk) |
                    (types[i] == kNormF32 ? 0x80000000u : 0u);
    add(tb.n++, i);
  }
  return i;
}

inline int grid_of(uint32_t chunks) {
  return (int)(chunks < (uint32_t)kClipGrid ? chunks : (uint32_t)kClipGrid);
}

}  // namespace

hipError_t launch_clip(const ClipArgs& a, hipStream_t stream) {
  int slots = 0;
  for (int64_t i = 0; i < a.n;) {
    NormTable tb;
    i = fill(tb, kClipNormTable, i, a.n, a.sizes, a.types,
             [&](int k, int64_t t) { tb.g[k] = a.grads[t]; });
    if (tb.n == 0) break;
    const int grid = grid_of(tb.end[tb.n - 1]);
    k_grad_squares<<<grid, kNT, 0, stream>>>(tb, a.part + slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    slots += grid;
  }
  float* norm_out = a.norm;
  if (a.scale) {
    // From the last tensor to the first: what the sum read last is still in the
    // 256 MB Infinity Cache.
    for (int64_t i = a.n - 1; i >= 0;) {
      ScaleTable tb;
      bool in_place = true;
      i = fill(tb, kClipScaleTable, i, -1, a.sizes, a.types, [&](int k, int64_t t) {
        tb.g[k] = a.grads[t];
        tb.out[k] = a.out ? a.out[t] : const_cast<void*>(a.grads[t]);
        in_place = in_place && tb.out[k] == tb.g[k];
      });
      if (tb.n == 0) break;
      k_grad_scale<<<grid_of(tb.end[tb.n - 1]), kNT, 0, stream>>>(tb, a.part, slots, a.max_norm,
                                                                  in_place, norm_out);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      norm_out = nullptr;  // the first launch writes it
    }
  }
  if (norm_out) {  // no scaling, or nothing to scale
    k_grad_norm<<<1, kNT, 0, stream>>>(a.part, slots, norm_out);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace qn
