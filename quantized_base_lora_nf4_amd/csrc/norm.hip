// Layer norm and root-mean-square norm over the rows of a [rows, width]
// matrix, forward and backward, bf16 or fp32.
//
//   forward   mu = sum(x) / width            (0 in the root-mean-square form)
//             rstd = 1 / sqrt(sum((x - mu)^2) / width + eps)
//             y = (x - mu) rstd w + b
//   backward  z = (x - mu) rstd,  g = dy w
//             dx = rstd (g - z mean(g z) - mean(g))   (the last term only with mu)
//             dw = sum over rows of dy z,  db = sum over rows of dy
//
// Both directions are bound by HBM: every element of x (and dy) is read
// once, held in registers as loaded, and the output is written once.  All
// statistics and sums are fp32; the only roundings to bf16 are the outputs'.
//
// A row belongs to TPR consecutive threads, each holding NV 16-byte vectors
// of it (vector i of thread t covers elements (i TPR + t) VEC ...).  Rows of
// a width that is not a whole number of vectors start unaligned; gfx950
// loads and stores 16 bytes at any element address, so those rows take the
// same path, with the one partial vector at the end element by element.
#include <type_traits>

#include "kernels.hpp"

namespace qn {
namespace {

struct F32T {
  using elem = float;
  static constexpr int VEC = 4;
};
struct BF16T {
  using elem = uint16_t;
  static constexpr int VEC = 8;
};

// 16 bytes at an address aligned to the element only.
template <class E>
struct __attribute__((packed, aligned(sizeof(E)))) Loose16 {
  u32x4 v;
};

template <class T>
__device__ __forceinline__ float elem_f32(typename T::elem e) {
  if constexpr (std::is_same<T, F32T>::value) return e;
  else return bf16_to_f32(e);
}
template <class T>
__device__ __forceinline__ typename T::elem f32_elem(float f) {
  if constexpr (std::is_same<T, F32T>::value) return f;
  else return f32_to_bf16(f);
}

// Element e of a held vector.
template <class T>
__device__ __forceinline__ float vec_get(const u32x4& v, int e) {
  if constexpr (std::is_same<T, F32T>::value) return word_to_f32(v[e]);
  else return (e & 1) ? bf16_hi_to_f32(v[e >> 1]) : bf16_lo_to_f32(v[e >> 1]);
}
template <class T>
__device__ __forceinline__ u32x4 vec_pack(const float* f) {
  if constexpr (std::is_same<T, F32T>::value) {
    return u32x4{__builtin_bit_cast(uint32_t, f[0]), __builtin_bit_cast(uint32_t, f[1]),
                 __builtin_bit_cast(uint32_t, f[2]), __builtin_bit_cast(uint32_t, f[3])};
  } else {
    return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                 pack_bf16x2(f[6], f[7])};
  }
}

// The vector at p[col ..], zeros past `width`.
template <class T>
__device__ __forceinline__ u32x4 load_vec(const typename T::elem* p, int col, int width) {
  using E = typename T::elem;
  if (col + T::VEC <= width) return reinterpret_cast<const Loose16<E>*>(p + col)->v;
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < T::VEC; ++e) {
    if (col + e < width) {
      if constexpr (std::is_same<T, F32T>::value)
        v[e] = __builtin_bit_cast(uint32_t, p[col + e]);
      else
        v[e >> 1] |= (uint32_t)p[col + e] << (16 * (e & 1));
    }
  }
  return v;
}

template <class T>
__device__ __forceinline__ void store_vec(typename T::elem* p, int col, int width, const float* f) {
  using E = typename T::elem;
  if (col + T::VEC <= width) {
    reinterpret_cast<Loose16<E>*>(p + col)->v = vec_pack<T>(f);
    return;
  }
#pragma unroll
  for (int e = 0; e < T::VEC; ++e)
    if (col + e < width) p[col + e] = f32_elem<T>(f[e]);
}

// VEC consecutive parameters (weight or bias) at p[col ..] as fp32, 0 past
// `width`; their type PT need not be the row type's.
template <class PT, int VEC>
__device__ __forceinline__ void load_params(float* f, const typename PT::elem* p, int col,
                                            int width) {
  if (col + VEC <= width) {
#pragma unroll
    for (int h = 0; h < VEC; h += 4) {
      if constexpr (std::is_same<PT, F32T>::value) {
        const u32x4 v = reinterpret_cast<const Loose16<float>*>(p + col + h)->v;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[h + e] = word_to_f32(v[e]);
      } else {
        struct __attribute__((packed, aligned(2))) Loose8 {
          u32x2 v;
        };
        const u32x2 v = reinterpret_cast<const Loose8*>(p + col + h)->v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[h + e] = (e & 1) ? bf16_hi_to_f32(v[e >> 1]) : bf16_lo_to_f32(v[e >> 1]);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = col + e < width ? elem_f32<PT>(p[col + e]) : 0.0f;
}

// Sum over the TPR threads of a row, the same bits in each of them.
// red: 2 * TPR / 64 floats per row of LDS when a row spans several waves
// (used alternately, so that one barrier per sum is enough).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red, int& flip) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* r = red + flip * W;
    flip ^= 1;
    if ((threadIdx.x & 63) == 0) r[(threadIdx.x >> 6) & (W - 1)] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += r[w];
  }
  return v;
}

template <int TPR>
constexpr int block_threads() {
  return TPR < 256 ? 256 : TPR;
}

// One row per TPR threads; the row stays in registers between the mean, the
// variance and the output (two passes over registers, so the variance is of
// differences and does not cancel).
template <class T, class PT, int TPR, int NV, bool kRms>
__global__ __launch_bounds__(block_threads<TPR>()) void k_norm_fwd(
    const typename T::elem* __restrict__ x, int64_t rows, int width,
    const typename PT::elem* __restrict__ w, const typename PT::elem* __restrict__ b, float eps,
    typename T::elem* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int VEC = T::VEC;
  constexpr int RPB = block_threads<TPR>() / TPR;
  __shared__ float red[TPR > 64 ? 2 * TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= rows) return;  // whole waves (TPR 64) or never (one row per workgroup)
  const typename T::elem* xr = x + row * width;
  const float inv_n = 1.0f / (float)width;
  int flip = 0;

  u32x4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + t) * VEC;
    v[i] = col < width ? load_vec<T>(xr, col, width) : u32x4{0u, 0u, 0u, 0u};
  }
  float mu = 0.0f;
  if constexpr (!kRms) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += vec_get<T>(v[i], e);
    mu = row_sum<TPR>(s, red, flip) * inv_n;
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = vec_get<T>(v[i], e) - mu;
      // without a mean, the zeros past the width add nothing by themselves
      if (kRms || col + e < width) q += d * d;
    }
  }
  const float rs = 1.0f / sqrtf(row_sum<TPR>(q, red, flip) * inv_n + eps);
  if (t == 0) {
    if constexpr (!kRms) mean[row] = mu;
    rstd[row] = rs;
  }
  typename T::elem* yr = y + row * width;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + t) * VEC;
    if (col >= width) break;
    float wv[VEC], f[VEC];
    load_params<PT, VEC>(wv, w, col, width);
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = (vec_get<T>(v[i], e) - mu) * rs * wv[e];
    if (b) {
      load_params<PT, VEC>(wv, b, col, width);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] += wv[e];
    }
    store_vec<T>(yr, col, width, f);
  }
}

// Backward: workgroup `blockIdx.x` of G takes rows blockIdx.x, + G, ...; a
// thread owns the same columns of every row, so its share of dw and db adds
// up in registers, and each workgroup writes one row of partial sums
// part[2][G][width] (dw, then db if kBias).  k_norm_bwd_params adds the
// G partial rows in a fixed order.
template <class T, class PT, int TPR, int NV, bool kRms, bool kBias>
__global__ __launch_bounds__(TPR) void k_norm_bwd(
    const typename T::elem* __restrict__ dy, const typename T::elem* __restrict__ x, int64_t rows,
    int width, const typename PT::elem* __restrict__ w, const float* __restrict__ mean,
    const float* __restrict__ rstd, typename T::elem* __restrict__ dx, float* __restrict__ part) {
  constexpr int VEC = T::VEC;
  __shared__ float red[TPR > 64 ? 4 * TPR / 64 : 1];
  const int t = threadIdx.x;
  const float inv_n = 1.0f / (float)width;
  float aw[NV][VEC], ab[kBias ? NV : 1][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      aw[i][e] = 0.0f;
      if constexpr (kBias) ab[i][e] = 0.0f;
    }
  float wv[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + t) * VEC;
    load_params<PT, VEC>(wv[i], w, col < width ? col : 0, col < width ? width : 0);
  }
  int flip = 0;
  u32x4 nx[NV], ny[NV];
  float nmu = 0.0f, nrs = 0.0f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * VEC;
      const bool in = col < width;
      nx[i] = in ? load_vec<T>(x + row * width, col, width) : u32x4{0u, 0u, 0u, 0u};
      ny[i] = in ? load_vec<T>(dy + row * width, col, width) : u32x4{0u, 0u, 0u, 0u};
    }
    if constexpr (!kRms) nmu = mean[row];
    nrs = rstd[row];
  };
  int64_t row = blockIdx.x;
  if (row < rows) fetch(row);
  for (; row < rows; row += gridDim.x) {
    u32x4 vx[NV], vy[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      vx[i] = nx[i];
      vy[i] = ny[i];
    }
    const float mu = nmu, rs = nrs;
    if (row + gridDim.x < rows) fetch(row + gridDim.x);  // the next row, in flight meanwhile
    float sg = 0.0f, sz = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        // past the width: dy = 0 and w = 0, so nothing is added
        const float z = (vec_get<T>(vx[i], e) - mu) * rs;
        const float d = vec_get<T>(vy[i], e);
        const float g = d * wv[i][e];
        sg += g;
        sz += g * z;
        aw[i][e] += d * z;
        if constexpr (kBias) ab[i][e] += d;
      }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      sz += __shfl_xor(sz, o, 64);
      if constexpr (!kRms) sg += __shfl_xor(sg, o, 64);
    }
    if constexpr (TPR > 64) {
      constexpr int W = TPR / 64;
      float* r = red + flip * 2 * W;
      flip ^= 1;
      if ((t & 63) == 0) {
        r[2 * (t >> 6)] = sz;
        r[2 * (t >> 6) + 1] = sg;
      }
      __syncthreads();
      sz = sg = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        sz += r[2 * k];
        sg += r[2 * k + 1];
      }
    }
    const float cz = sz * inv_n, cg = kRms ? 0.0f : sg * inv_n;
    if (dx) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * VEC;
        if (col < width) {
          float f[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float z = (vec_get<T>(vx[i], e) - mu) * rs;
            f[e] = rs * (vec_get<T>(vy[i], e) * wv[i][e] - z * cz - cg);
          }
          store_vec<T>(dx + row * width, col, width, f);
        }
      }
    }
  }
  if (!part) return;
  float* pw = part + (int64_t)blockIdx.x * width;
  float* pb = pw + (int64_t)gridDim.x * width;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + t) * VEC;
    if (col < width) {
#pragma unroll
      for (int h = 0; h < VEC; h += 4) {
        store_vec<F32T>(pw, col + h, width, &aw[i][h]);
        if constexpr (kBias) store_vec<F32T>(pb, col + h, width, &ab[i][h]);
      }
    }
  }
}

// dw (and db) from the G partial rows: 64 columns per workgroup of 16
// waves, each wave adding every 16th row; then the 16 sums in wave order.
constexpr int kPW = 16;
template <class PT>
__global__ __launch_bounds__(64 * kPW) void k_norm_bwd_params(const float* __restrict__ part,
                                                              int G, int width,
                                                              typename PT::elem* dw,
                                                              typename PT::elem* db) {
  __shared__ float s[kPW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  typename PT::elem* out = blockIdx.y ? db : dw;
  const float* p = part + (blockIdx.y ? (int64_t)G * width : 0);
  float a = 0.0f;
  if (col < width) {
    int g = wave;
    for (; g + 3 * kPW < G; g += 4 * kPW) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = p[(int64_t)(g + u * kPW) * width + col];
#pragma unroll
      for (int u = 0; u < 4; ++u) a += v[u];
    }
    for (; g < G; g += kPW) a += p[(int64_t)g * width + col];
  }
  s[wave][lane] = a;
  __syncthreads();
  if (wave == 0 && col < width && out) {
    a = 0.0f;
#pragma unroll
    for (int k = 0; k < kPW; ++k) a += s[k][lane];
    out[col] = f32_elem<PT>(a);
  }
}

// ---- launch shapes ----

template <class F>
auto with_norm_type(int t, F&& f) {
  return t == kNormF32 ? f(F32T{}) : f(BF16T{});
}

// Vectors of a row.
inline int64_t row_vecs(int64_t width, int type) {
  const int vec = type == kNormF32 ? F32T::VEC : BF16T::VEC;
  return (width + vec - 1) / vec;
}

template <int V>
using IntC = std::integral_constant<int, V>;

// Forward: threads per row and vectors per thread.  A wave per row has no
// barriers and is taken while there are rows enough to fill the chip;
// otherwise a row is spread over more threads.
template <class F>
hipError_t with_fwd_shape(int64_t rows, int64_t nv, F&& f) {
  const bool many = rows >= 2048;
  if (nv <= 64) return f(IntC<64>{}, IntC<1>{});
  if (nv <= 128 && many) return f(IntC<64>{}, IntC<2>{});
  if (nv <= 256 && many) return f(IntC<64>{}, IntC<4>{});
  if (nv <= 512 && many) return f(IntC<64>{}, IntC<8>{});
  if (nv <= 256) return f(IntC<256>{}, IntC<1>{});
  if (nv <= 512) return f(IntC<256>{}, IntC<2>{});
  if (nv <= 1024) return f(IntC<256>{}, IntC<4>{});
  if (nv <= 2048) return f(IntC<256>{}, IntC<8>{});
  if (nv <= 4096) return f(IntC<1024>{}, IntC<4>{});
  return f(IntC<1024>{}, IntC<8>{});
}

// Backward: as many threads as cover the row with one vector each, up to
// 512; wider rows take several vectors per thread.
template <class F>
auto with_bwd_shape(int64_t nv, F&& f) {
  if (nv <= 64) return f(IntC<64>{}, IntC<1>{});
  if (nv <= 128) return f(IntC<128>{}, IntC<1>{});
  if (nv <= 256) return f(IntC<256>{}, IntC<1>{});
  if (nv <= 512) return f(IntC<512>{}, IntC<1>{});
  if (nv <= 1024) return f(IntC<512>{}, IntC<2>{});
  if (nv <= 2048) return f(IntC<512>{}, IntC<4>{});
  if (nv <= 4096) return f(IntC<1024>{}, IntC<4>{});
  return f(IntC<1024>{}, IntC<8>{});
}

}  // namespace

int64_t norm_max_width(int type) {
  return 8192 * (int64_t)(type == kNormF32 ? F32T::VEC : BF16T::VEC);
}

int norm_bwd_groups(int64_t rows, int64_t width, int type) {
  const int tpr = with_bwd_shape(row_vecs(width, type),
                                 [](auto tp, auto) { return (int)decltype(tp)::value; });
  const int64_t g = 256 * 1024 / tpr;  // about 16 waves per CU
  return (int)(rows < g ? rows : g);
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return with_norm_type(a.x_type, [&](auto t) {
    return with_norm_type(a.w_type, [&](auto pt) {
      return with_fwd_shape(a.rows, row_vecs(a.width, a.x_type), [&](auto tp, auto nv) {
        using T = decltype(t);
        using PT = decltype(pt);
        constexpr int TPR = decltype(tp)::value, NV = decltype(nv)::value;
        constexpr int NT = block_threads<TPR>();
        const unsigned grid = (unsigned)((a.rows + NT / TPR - 1) / (NT / TPR));
        auto go = [&](auto kern) {
          kern<<<grid, NT, 0, stream>>>((const typename T::elem*)a.x, a.rows, (int)a.width,
                                        (const typename PT::elem*)a.w,
                                        (const typename PT::elem*)a.b, a.eps,
                                        (typename T::elem*)a.y, a.mean, a.rstd);
          return hipGetLastError();
        };
        return a.rms ? go(k_norm_fwd<T, PT, TPR, NV, true>)
                     : go(k_norm_fwd<T, PT, TPR, NV, false>);
      });
    });
  });
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream) {
  if (!a.dx && !a.dw && !a.db) return hipSuccess;
  const int G = norm_bwd_groups(a.rows, a.width, a.x_type);
  if (G > 0) {
    const hipError_t e = with_norm_type(a.x_type, [&](auto t) {
      return with_norm_type(a.w_type, [&](auto pt) {
        return with_bwd_shape(row_vecs(a.width, a.x_type), [&](auto tp, auto nv) {
          using T = decltype(t);
          using PT = decltype(pt);
          constexpr int TPR = decltype(tp)::value, NV = decltype(nv)::value;
          auto go = [&](auto kern) {
            kern<<<G, TPR, 0, stream>>>((const typename T::elem*)a.dy,
                                        (const typename T::elem*)a.x, a.rows, (int)a.width,
                                        (const typename PT::elem*)a.w, a.mean, a.rstd,
                                        (typename T::elem*)a.dx, a.dw || a.db ? a.part : nullptr);
            return hipGetLastError();
          };
          if (a.rms)
            return a.db ? go(k_norm_bwd<T, PT, TPR, NV, true, true>)
                        : go(k_norm_bwd<T, PT, TPR, NV, true, false>);
          return a.db ? go(k_norm_bwd<T, PT, TPR, NV, false, true>)
                      : go(k_norm_bwd<T, PT, TPR, NV, false, false>);
        });
      });
    });
    if (e != hipSuccess) return e;
  }
  if (!a.dw && !a.db) return hipSuccess;
  return with_norm_type(a.w_type, [&](auto pt) {
    using PT = decltype(pt);
    const dim3 grid((unsigned)((a.width + 63) / 64), a.db ? 2 : 1);
    k_norm_bwd_params<PT><<<grid, 64 * kPW, 0, stream>>>(a.part, G, (int)a.width,
                                                         (typename PT::elem*)a.dw,
                                                         (typename PT::elem*)a.db);
    return hipGetLastError();
  });
}

}  // namespace qn
