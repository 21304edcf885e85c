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
//
// The backward pass of rows of more than 2048 bf16 or 4096 fp32 vectors does
// not fit the registers: its workgroups of 1024 threads have 128 each, and 56 to
// 105 (four bf16 vectors per thread), 365 to 640 (eight) or 96 to 141 (eight fp32
// vectors) are kept in scratch memory and move with every row (512 x 32768 bf16
// rms 47 us where the bytes take 20, 512 x 65536 328 where they take 39).
//
// Measured: forward 4096 x 4096 bf16 13.8 us (4.9 TB/s, a large copy reaches
// 5.1 to 5.2); backward 8192 x 8192 bf16 (rms) 76 us (5.3 TB/s), 2047 x 5120
// fp32 31 us, of which 24 are the main kernel's (5.3 TB/s) and 4 the parameters'.
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

// Backward: a workgroup holds RG = NT / TPR row groups of TPR threads.  Group
// k of workgroup b takes rows b RG + k, + gridDim.x RG, ...; a thread owns the
// same columns of every row, so its share of dw and db adds up in registers.
// At the end the groups' shares are added pairwise through LDS, and the
// workgroup writes one row of partial sums part[2][G][width] (dw, then db if
// kBias), which k_norm_bwd_params adds in a fixed order; a single workgroup
// (few rows) writes dw and db itself.  The next row's loads run during the
// current one.
//
// Few, large workgroups keep the partial rows few: 256 of them, written once
// and read once, add 4 % to the pass's bytes at 8192 x 8192 (bf16, dw alone) and
// 17 % at 4096 x 1024 (dw and db).
template <class T, class PT, int NT, int TPR, int NV, bool kRms, bool kBias>
__global__ __launch_bounds__(NT) void k_norm_bwd(
    const typename T::elem* __restrict__ dy, const typename T::elem* __restrict__ x, int64_t rows,
    int width, const typename PT::elem* __restrict__ w, const float* __restrict__ mean,
    const float* __restrict__ rstd, typename T::elem* __restrict__ dx, float* __restrict__ part,
    typename PT::elem* __restrict__ dw, typename PT::elem* __restrict__ db) {
  constexpr int VEC = T::VEC, RG = NT / TPR, W = TPR / 64;
  constexpr int kSums = W > 1 ? 4 * (NT / 64) : 1;            // floats for the row sums
  constexpr int kShare = RG > 1 ? RG / 2 * TPR * NV * VEC : 1;  // and for half of the groups' shares
  __shared__ __attribute__((aligned(16))) float red[kSums];
  __shared__ __attribute__((aligned(16))) float share[kShare];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const float inv_n = 1.0f / (float)width;
  // Up to two vectors per thread, the weight stays in registers and the next
  // row is fetched ahead; with more there are not enough of them.
  constexpr bool kHold = NV <= 2;
  float aw[NV][VEC] = {}, ab[kBias ? NV : 1][VEC] = {};
  float wv[NV][VEC];
  auto load_w = [&](int i) {
    const int col = (i * TPR + t) * VEC;
    load_params<PT, VEC>(wv[i], w, col < width ? col : 0, col < width ? width : 0);
  };
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NV; ++i) load_w(i);
  }
  int flip = 0;
  u32x4 nx[NV], ny[NV];
  float nmu = 0.0f, nrs = 0.0f;
  // A row past the end has dy = 0 and adds nothing.
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + t) * VEC;
      const bool in = col < width && row < rows;
      nx[i] = in ? load_vec<T>(x + row * width, col, width) : u32x4{0u, 0u, 0u, 0u};
      ny[i] = in ? load_vec<T>(dy + row * width, col, width) : u32x4{0u, 0u, 0u, 0u};
    }
    nmu = !kRms && row < rows ? mean[row] : 0.0f;
    nrs = row < rows ? rstd[row] : 0.0f;
  };
  const int64_t stride = (int64_t)gridDim.x * RG;
  int64_t row = (int64_t)blockIdx.x * RG + group;
  if constexpr (kHold) fetch(row);
  // the same number of turns in every group: there is a barrier in each
  for (int64_t base = (int64_t)blockIdx.x * RG; base < rows; base += stride, row += stride) {
    u32x4 vx[NV], vy[NV];
    if constexpr (!kHold) fetch(row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      vx[i] = nx[i];
      vy[i] = ny[i];
    }
    const float mu = nmu, rs = nrs;
    if constexpr (kHold) {
      if (base + stride < rows) fetch(row + stride);
    }
    float sg = 0.0f, sz = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (!kHold) load_w(i);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        // past the width: dy = 0 and w = 0, so nothing is added
        const float z = (vec_get<T>(vx[i], e) - mu) * rs;
        const float d = vec_get<T>(vy[i], e);
        const float g = d * wv[i][e];
        if constexpr (!kRms) sg += g;
        sz += g * z;
        aw[i][e] += d * z;
        if constexpr (kBias) ab[i][e] += d;
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      sz += __shfl_xor(sz, o, 64);
      if constexpr (!kRms) sg += __shfl_xor(sg, o, 64);
    }
    if constexpr (W > 1) {
      float* r = red + flip * 2 * (NT / 64);
      flip ^= 1;
      if ((threadIdx.x & 63) == 0) {
        r[2 * (threadIdx.x >> 6)] = sz;
        r[2 * (threadIdx.x >> 6) + 1] = sg;
      }
      __syncthreads();
      sz = sg = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        sz += r[2 * (group * W + k)];
        if constexpr (!kRms) sg += r[2 * (group * W + k) + 1];
      }
    }
    const float cz = sz * inv_n, cg = kRms ? 0.0f : sg * inv_n;
    if (dx && row < rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + t) * VEC;
        if (col < width) {
          if constexpr (!kHold) load_w(i);
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
  // upper half of the groups -> LDS -> lower half, until one group has it all
  auto gather = [&](float (&a)[NV][VEC]) {
#pragma unroll
    for (int half = RG / 2; half > 0; half /= 2) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int h = 0; h < VEC; h += 4) {
          f32x4* p = reinterpret_cast<f32x4*>(
              share + ((((group & (half - 1)) * NV + i) * (VEC / 4) + h / 4) * TPR + t) * 4);
          if (group >= half && group < 2 * half)
            *p = f32x4{a[i][h], a[i][h + 1], a[i][h + 2], a[i][h + 3]};
        }
      __syncthreads();
      if (group < half) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int h = 0; h < VEC; h += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(
                share + (((group * NV + i) * (VEC / 4) + h / 4) * TPR + t) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[i][h + e] += v[e];
          }
      }
    }
  };
  if constexpr (RG > 1) {
    gather(aw);
    if constexpr (kBias) gather(ab);
    if (group > 0) return;
  }
  if (gridDim.x == 1) {  // the only partial sums are the sums
    auto store = [&](typename PT::elem* out, const float (&a)[NV][VEC]) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int col = (i * TPR + t) * VEC + e;
          if (out && col < width) out[col] = f32_elem<PT>(a[i][e]);
        }
    };
    store(dw, aw);
    if constexpr (kBias) store(db, ab);
    return;
  }
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
// waves, each wave adding every 16th row (at most 16 of them, all loaded at
// once); then the 16 sums in wave order.
constexpr int kPW = 16;
constexpr int kMaxGroups = 256;  // one workgroup per CU
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
    float v[kMaxGroups / kPW];
#pragma unroll
    for (int u = 0; u < kMaxGroups / kPW; ++u) {
      const int g = wave + u * kPW;
      v[u] = g < G ? p[(int64_t)g * width + col] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kMaxGroups / kPW; ++u) a += v[u];
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

// Workgroups of a forward launch; more rows take further launches.  HIP takes
// fewer than 2^32 threads along a dimension of the grid (2^26 + 5 rows in one
// launch of four rows per 256 threads: most rows were never written, and no
// error came back), which is 2^22 workgroups of 1024.  At a quarter of that a
// launch lasts far longer than the next one's start takes.
constexpr int64_t kMaxGrid = 1 << 20;

// Forward: threads per row and vectors per thread.  A wave per row has no
// barriers and is taken for up to 256 vectors while there are rows enough to
// fill the chip (16384 x 1024 bf16: 14.1 us against 21.9 with 256 threads);
// with more vectors a wave's row takes the registers that would keep more
// loads in flight (4096 x 4096 bf16: 20.1 us against 14.6), and with few rows
// one wave's latency counts: there a row is spread over more threads.
template <class F>
hipError_t with_fwd_shape(int64_t rows, int64_t nv, F&& f) {
  const bool many = rows >= 2048;
  if (nv <= 64) return f(IntC<64>{}, IntC<1>{});
  if (nv <= 128 && many) return f(IntC<64>{}, IntC<2>{});
  if (nv <= 256 && many) return f(IntC<64>{}, IntC<4>{});
  if (nv <= 256) return f(IntC<256>{}, IntC<1>{});
  if (nv <= 512) return f(IntC<256>{}, IntC<2>{});
  if (nv <= 1024) return f(IntC<256>{}, IntC<4>{});
  if (nv <= 2048) return f(IntC<256>{}, IntC<8>{});
  if (nv <= 4096) return f(IntC<1024>{}, IntC<4>{});
  return f(IntC<1024>{}, IntC<8>{});
}

// Backward: threads per workgroup and row, and vectors per thread: a wave per
// row up to two vectors per lane (no barriers), otherwise as many threads as
// give each one vector.  Sums of dw and db take 16 registers per bf16 vector
// and 8 per fp32 vector, and 1024 threads have 128 each, 512 threads 256:
// two or more bf16 vectors per thread run faster in the smaller workgroup
// (16384 x 1024: 32.9 -> 21.5 us; 2000 x 16384: 62 -> 49 us), two fp32
// vectors in the larger one (2048 x 5120: 24.4 us against 28.0).
template <class T, class F>
auto with_bwd_shape(int64_t nv, F&& f) {
  if (nv <= 64) return f(IntC<1024>{}, IntC<64>{}, IntC<1>{});
  if (nv <= 128) return f(IntC<512>{}, IntC<64>{}, IntC<2>{});
  if (nv <= 256) return f(IntC<1024>{}, IntC<256>{}, IntC<1>{});
  if (nv <= 512) return f(IntC<1024>{}, IntC<512>{}, IntC<1>{});
  if (nv <= 1024) return f(IntC<1024>{}, IntC<1024>{}, IntC<1>{});
  if (nv <= 2048) {
    if constexpr (std::is_same<T, F32T>::value) return f(IntC<1024>{}, IntC<1024>{}, IntC<2>{});
    else return f(IntC<512>{}, IntC<512>{}, IntC<4>{});
  }
  if (nv <= 4096) return f(IntC<1024>{}, IntC<1024>{}, IntC<4>{});
  return f(IntC<1024>{}, IntC<1024>{}, IntC<8>{});
}

}  // namespace

int64_t norm_max_width(int type) {
  return 8192 * (int64_t)(type == kNormF32 ? F32T::VEC : BF16T::VEC);
}

int norm_bwd_groups(int64_t rows, int64_t width, int type) {
  const int rg = with_norm_type(type, [&](auto t) {
    return with_bwd_shape<decltype(t)>(row_vecs(width, type), [](auto nt, auto tp, auto) {
      return (int)decltype(nt)::value / (int)decltype(tp)::value;
    });
  });
  const int64_t g = (rows + rg - 1) / rg;
  return (int)(g < kMaxGroups ? g : kMaxGroups);
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return with_norm_type(a.x_type, [&](auto t) {
    return with_norm_type(a.w_type, [&](auto pt) {
      return with_fwd_shape(a.rows, row_vecs(a.width, a.x_type), [&](auto tp, auto nv) {
        using T = decltype(t);
        using PT = decltype(pt);
        constexpr int TPR = decltype(tp)::value, NV = decltype(nv)::value;
        constexpr int NT = block_threads<TPR>(), RPB = NT / TPR;
        auto go = [&](auto kern) {
          for (int64_t r = 0; r < a.rows; r += kMaxGrid * RPB) {
            const int64_t n = a.rows - r < kMaxGrid * RPB ? a.rows - r : kMaxGrid * RPB;
            kern<<<(unsigned)((n + RPB - 1) / RPB), NT, 0, stream>>>(
                (const typename T::elem*)a.x + r * a.width, n, (int)a.width,
                (const typename PT::elem*)a.w, (const typename PT::elem*)a.b, a.eps,
                (typename T::elem*)a.y + r * a.width, a.mean ? a.mean + r : nullptr, a.rstd + r);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
          }
          return hipSuccess;
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
        using T = decltype(t);
        return with_bwd_shape<T>(row_vecs(a.width, a.x_type), [&](auto nt, auto tp, auto nv) {
          using PT = decltype(pt);
          constexpr int NT = decltype(nt)::value, TPR = decltype(tp)::value,
                        NV = decltype(nv)::value;
          auto go = [&](auto kern) {
            kern<<<G, NT, 0, stream>>>((const typename T::elem*)a.dy,
                                        (const typename T::elem*)a.x, a.rows, (int)a.width,
                                        (const typename PT::elem*)a.w, a.mean, a.rstd,
                                        (typename T::elem*)a.dx, a.dw || a.db ? a.part : nullptr,
                                        (typename PT::elem*)a.dw, (typename PT::elem*)a.db);
            return hipGetLastError();
          };
          if (a.rms)
            return a.db ? go(k_norm_bwd<T, PT, NT, TPR, NV, true, true>)
                        : go(k_norm_bwd<T, PT, NT, TPR, NV, true, false>);
          return a.db ? go(k_norm_bwd<T, PT, NT, TPR, NV, false, true>)
                      : go(k_norm_bwd<T, PT, NT, TPR, NV, false, false>);
        });
      });
    });
    if (e != hipSuccess) return e;
  }
  if ((!a.dw && !a.db) || G == 1) return hipSuccess;
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
