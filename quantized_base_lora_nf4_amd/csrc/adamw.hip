// The AdamW step over many tensors at once, with states in 32 or in 8 bits.
//
//   g = c grad,  c = min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit states: blocks of 256 elements of a tensor share one fp32 scale each
// for m and for v, the block's largest |m| and v:
//   m = s c |c| / 127^2, c in -127..127      v = s (c / 255)^4, c in 0..255
// A square law on m and on sqrt(v), which is how v is used: small values next
// to a large one keep a few codes.  The nearest code in the companded domain
// is the number of thresholds (c - 1/2)^2 (v: their squares) up to |m| 127^2/s
// (v 255^4 / s); v > 0 never becomes code 0, which would divide m by eps.
// Every step from the old state and the gradient to the new codes is one
// correctly rounded fp32 operation (no fused multiply-add), so the codes are
// the same bits wherever they are computed; square roots only guess a code,
// which a comparison with the threshold then settles.
//
// One pass over the data.  32 lanes own a block, 8 elements each, so the block's
// largest values are a reduction within half a wave.  The tensors' addresses
// travel in the launch arguments, as in clip.hip.  Measured, 160 M bf16
// parameters in 448 tensors: 32-bit states (22 bytes per element) 722 us, 4.9
// TB/s, bound by HBM; 8-bit states (10 bytes) 420 us, 3.8 TB/s, where about 75 issue
// slots per element take as long as the memory.
#include "kernels.hpp"

namespace qn {
namespace {

constexpr int kNT = 256;
constexpr int kChunk = kNT / 32;  // blocks per unit of work: one per half wave
constexpr int kBlock = kAdamBlock;

template <int kCap, bool kCopy>
struct Table {
  const void* g[kCap];
  void* p[kCap];
  uint16_t* c[kCopy ? kCap : 1];
  uint32_t end[kCap];   // chunks of the tensors up to and including this one
  uint32_t first[kCap]; // its first block in the states
  uint32_t tail[kCap];  // blocks of the tensor's last chunk, less 1 (3 bits) | elements of its last
                        // block, less 1 << 3 (8 bits) | fp32 gradient << 30 | fp32 parameter << 31
  int32_t n;
};
using PlainTable = Table<136, false>;
using CopyTable = Table<104, true>;
static_assert(sizeof(PlainTable) + sizeof(AdamHyper) + 64 <= 4096 &&
                  sizeof(CopyTable) + sizeof(AdamHyper) + 64 <= 4096,
              "launch arguments");

struct State {
  void* m;
  void* v;
  float* ms;
  float* vs;
};

template <class E, int W>
struct __attribute__((packed, aligned(sizeof(E)))) Loose {
  uint32_t w[W * sizeof(E) / 4];
};

// W elements at p (aligned to their type) as they are; the first n of them
// exist, the others are zeros.
template <class E, int W>
__device__ __forceinline__ void load(Loose<E, W>& x, const E* p, int n) {
  if (n >= W) {
    x = *reinterpret_cast<const Loose<E, W>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < W * (int)sizeof(E) / 4; ++i) {
      x.w[i] = 0;
      if constexpr (sizeof(E) == 4) {
        if (i < n) x.w[i] = __builtin_bit_cast(uint32_t, p[i]);
      } else {
        if (2 * i < n) x.w[i] = p[2 * i];
        if (2 * i + 1 < n) x.w[i] |= (uint32_t)p[2 * i + 1] << 16;
      }
    }
  }
}
template <class E, int W>
__device__ __forceinline__ float element(const Loose<E, W>& x, int i) {
  if constexpr (sizeof(E) == 4) return word_to_f32(x.w[i]);
  else return i & 1 ? bf16_hi_to_f32(x.w[i >> 1]) : bf16_lo_to_f32(x.w[i >> 1]);
}

template <class E, int W>
__device__ __forceinline__ void store(E* p, const float (&x)[W], int n) {
  if (n >= W) {
    Loose<E, W> v;
#pragma unroll
    for (int i = 0; i < W * (int)sizeof(E) / 4; ++i) {
      if constexpr (sizeof(E) == 4) v.w[i] = __builtin_bit_cast(uint32_t, x[i]);
      else v.w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
    *reinterpret_cast<Loose<E, W>*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) {
        if constexpr (sizeof(E) == 4) p[i] = x[i];
        else p[i] = f32_to_bf16(x[i]);
      }
  }
}

// The largest of the 32 lanes of each half wave.
__device__ __forceinline__ uint32_t half_max(uint32_t x) {
  auto up = [&](uint32_t y) { x = x > y ? x : y; };
  up(__builtin_amdgcn_mov_dpp(x, 0xB1, 0xf, 0xf, false));   // lane ^ 1
  up(__builtin_amdgcn_mov_dpp(x, 0x4E, 0xf, 0xf, false));   // lane ^ 2
  up(__builtin_amdgcn_mov_dpp(x, 0x141, 0xf, 0xf, false));  // mirrored within 8
  up(__builtin_amdgcn_mov_dpp(x, 0x140, 0xf, 0xf, false));  // mirrored within 16
  up(__builtin_amdgcn_ds_swizzle(x, 0x401F));               // lane ^ 16
  return x;
}

// The scale of a block from the bits of its largest magnitude (as unsigned
// numbers, infinities and NaN are the largest): 0 for blocks below 2^-96,
// whose codes would need a factor beyond fp32, and NaN for a block that holds
// an infinity or NaN: it becomes NaN as a whole.
__device__ __forceinline__ float scale_of(uint32_t bits) {
  const float s = word_to_f32(bits);
  return bits >= 0x7f800000u ? __builtin_nanf("") : s < 0x1p-96f ? 0.0f : s;
}
// ... and the factor that maps it to the largest code's power.
__device__ __forceinline__ float factor_of(float s, float top) { return s > 0.0f ? top / s : 0.0f; }

// The code of a value whose power is y (at most a few roundings above the largest
// code's): the guess from a root that is within a few units in the last place,
// taken a little low, is the code or one less.
__device__ __forceinline__ float code_m(float y) {
#pragma clang fp contract(off)
  const float n = floorf(__builtin_amdgcn_sqrtf(y) + 0.4999f);
  const float h = n + 0.5f;
  return h * h <= y ? h + 0.5f : n;
}
// low: the square root of y, less 2^-20 of it, within a few units (or 0 for a
// subnormal value, whose y is below 4: code 0 or 1).  Its root is 127 2^-20 below the code's at most.
__device__ __forceinline__ float code_v(float y, float low) {
#pragma clang fp contract(off)
  const float n = rintf(__builtin_amdgcn_sqrtf(low));
  const float h = n + 0.5f, h2 = h * h;  // exact
  return h2 * h2 <= y ? h + 0.5f : n;
}
__device__ __forceinline__ float value_m(float c, float s) {
#pragma clang fp contract(off)
  return c * fabsf(c) * (1.0f / 16129.0f) * s;
}
__device__ __forceinline__ float value_v(float c, float s) {
#pragma clang fp contract(off)
  const float d = c * c;
  return d * d * (float)(1.0 / 4228250625.0) * s;
}

template <int W>
struct Codes {
  uint32_t w[W / 4];
};

// Byte i of a word as a float.
__device__ __forceinline__ float byte_f32(uint32_t w, int i) { return (float)((w >> (8 * i)) & 0xffu); }

// Scalars of a step, the same for every element.
struct Step {
  float c, b1, a1, b2, a2, keep, lr1, rb2, eps;
};

// What a launch computes from the device's scalars, once per thread.
__device__ __forceinline__ Step step_of(const AdamHyper& h) {
  Step s;
  s.b1 = (float)h.beta1;
  s.a1 = (float)(1.0 - h.beta1);
  s.b2 = (float)h.beta2;
  s.a2 = (float)(1.0 - h.beta2);
  s.eps = h.eps;
  double bc1 = h.bc1, bc2 = h.bc2, lr = h.lr;
  if (h.step_dev) {  // 1 - b^t, from the logarithms
    const double t = (double)*h.step_dev;
    bc1 = -expm1(t * h.log_beta1);
    bc2 = -expm1(t * h.log_beta2);
  }
  if (h.lr_dev) lr = (double)*h.lr_dev;
  s.keep = (float)(1.0 - lr * h.decay);
  s.lr1 = (float)(lr / bc1);
  s.rb2 = (float)(1.0 / sqrt(bc2));
  s.c = 1.0f;
  if (h.norm) {  // as in clipping: NaN passes through, an infinite norm gives 0
    const double f = h.max_norm / ((double)*h.norm + 1e-6);
    const bool free = h.max_norm == __builtin_inf() && *h.norm == __builtin_inff();
    s.c = f >= 1.0 || free ? 1.0f : (float)f;
  }
  return s;
}

// What a lane loads of a block: 8 elements, as J vectors of W.  fp32 data moves
// as 4 elements per lane and access, so that 32 lanes read whole lines; 16- and
// 8-bit data alone as 8.
template <bool k8, class PT, class GT>
struct Raw {
  static constexpr int W = k8 && sizeof(PT) == 2 && sizeof(GT) == 2 ? 8 : 4, J = 8 / W;
  Loose<GT, W> g[J];
  Loose<PT, W> p[J];
  Codes<W> cm[k8 ? J : 1], cv[k8 ? J : 1];
  f32x4 m[k8 ? 1 : J], v[k8 ? 1 : J];
  float ms, vs;

  // p, g at the block's first element, of which `count` exist; block `blk` of
  // the states
  __device__ __forceinline__ void load_block(const PT* pp, const GT* gp, const State& st, int64_t blk,
                                             int count) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = j * 32 * W + lane * W;
      load<GT, W>(g[j], gp + e, count - e);
      load<PT, W>(p[j], pp + e, count - e);
      if constexpr (k8) {
        cm[j] = *reinterpret_cast<const Codes<W>*>((const uint8_t*)st.m + blk * kBlock + e);
        cv[j] = *reinterpret_cast<const Codes<W>*>((const uint8_t*)st.v + blk * kBlock + e);
      } else {
        m[j] = *reinterpret_cast<const f32x4*>((const float*)st.m + blk * kBlock + e);
        v[j] = *reinterpret_cast<const f32x4*>((const float*)st.v + blk * kBlock + e);
      }
    }
    if constexpr (k8) {
      ms = st.ms[blk];
      vs = st.vs[blk];
    }
  }
};

// The square root of a second moment.  v_sqrt is within 1 ulp, far below the
// parameter's rounding, but takes subnormal numbers as 0: kTiny scales them.
template <bool kTiny>
__device__ __forceinline__ float root_of(float v) {
  if constexpr (!kTiny) return __builtin_amdgcn_sqrtf(v);
  const bool low = v < 0x1p-96f;
  return __builtin_amdgcn_sqrtf(low ? v * 0x1p64f : v) * (low ? 0x1p-32f : 1.0f);
}

// Whether that matters: a root of a subnormal number is below 2^-63, in the
// denominator below 2^-63 / sqrt(1 - beta2) at any step, and nothing (half a
// rounding of 2^-24) beside an eps of 2^-38 / sqrt(1 - beta2).  The usual eps of
// 1e-8 is above that up to a beta2 of 1 - 1.4e-7.  (160 M bf16 elements in one
// run, without and with it: 8-bit states 365 and 405 us, 32-bit ones 727 both.)
bool tiny_matters(const AdamHyper& h) { return !(h.eps >= 0x1p-38 / sqrt(1.0 - h.beta2)); }

// The step of one block.
template <bool k8, bool kTiny, class PT, class GT>
__device__ __forceinline__ void update_block(const Raw<k8, PT, GT>& r, PT* p, uint16_t* c,
                                             const State& st, int64_t blk, int count,
                                             const Step& s) {
  constexpr int W = Raw<k8, PT, GT>::W, J = Raw<k8, PT, GT>::J;
  const int lane = threadIdx.x & 31;
  float gv[J][W], pv[J][W], m[J][W], v[J][W], root[J][W];
  int n[J];
  Codes<W> cm[J], cv[J];
  float ms, vs;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    n[j] = count - (j * 32 * W + lane * W);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      gv[j][i] = element(r.g[j], i);
      pv[j][i] = element(r.p[j], i);
      if constexpr (k8) {
        m[j][i] = value_m(byte_f32(r.cm[j].w[i >> 2] ^ 0x80808080u, i & 3) - 128.0f, r.ms);
        v[j][i] = value_v(byte_f32(r.cv[j].w[i >> 2], i & 3), r.vs);
      } else {
        m[j][i] = r.m[j][i];
        v[j][i] = r.v[j][i];
      }
    }
  }
  uint32_t mtop = 0, vtop = 0;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      {
#pragma clang fp contract(off)
        const float x = gv[j][i] * s.c;
        m[j][i] = m[j][i] * s.b1 + x * s.a1;
        v[j][i] = v[j][i] * s.b2 + x * x * s.a2;
      }
      if constexpr (k8) {
        const uint32_t a = __builtin_bit_cast(uint32_t, m[j][i]) & 0x7fffffffu;
        const uint32_t b = __builtin_bit_cast(uint32_t, v[j][i]);  // no negative ones
        mtop = mtop > a ? mtop : a;
        vtop = vtop > b ? vtop : b;
      }
      root[j][i] = root_of<kTiny>(v[j][i]);
      const float d = root[j][i] * s.rb2 + s.eps;
      // (v_rcp is within 1 ulp too, and takes subnormal numbers as 0 too)
      if constexpr (kTiny) pv[j][i] = pv[j][i] * s.keep - s.lr1 * m[j][i] / d;
      else pv[j][i] = pv[j][i] * s.keep - s.lr1 * m[j][i] * __builtin_amdgcn_rcpf(d);
    }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = j * 32 * W + lane * W;
    store<PT, W>(p + e, pv[j], n[j]);
    if (c) store<uint16_t, W>(c + e, pv[j], n[j]);
  }
  if constexpr (!k8) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = j * 32 * W + lane * W;
      *reinterpret_cast<f32x4*>((float*)st.m + blk * kBlock + e) = f32x4{m[j][0], m[j][1], m[j][2], m[j][3]};
      *reinterpret_cast<f32x4*>((float*)st.v + blk * kBlock + e) = f32x4{v[j][0], v[j][1], v[j][2], v[j][3]};
    }
  } else {
    ms = scale_of(half_max(mtop));
    vs = scale_of(half_max(vtop));
    const float fm = factor_of(ms, 16129.0f), fv = factor_of(vs, 4228250625.0f);
    // (a block without scales, also one that holds a NaN, gets codes 0)
    const float rv = __builtin_amdgcn_sqrtf(fv) * (1.0f - 0x1p-20f);
    const uint32_t keep_m = fm > 0.0f ? ~0u : 0u, keep_v = fv > 0.0f ? ~0u : 0u;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = j * 32 * W + lane * W;
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        uint32_t wm = 0, wv = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = m[j][4 * q + i], y = v[j][4 * q + i];
          const float a = code_m(fabsf(x) * fm);
          const float c = code_v(y * fv, root[j][4 * q + i] * rv);
          const float b = y > 0.0f ? fmaxf(c, 1.0f) : c;
          wm = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_copysignf(a, x) + 128.0f, i, wm);
          wv = __builtin_amdgcn_cvt_pk_u8_f32(b, i, wv);
        }
        cm[j].w[q] = (wm ^ 0x80808080u) & keep_m;
        cv[j].w[q] = wv & keep_v;
      }
      *reinterpret_cast<Codes<W>*>((uint8_t*)st.m + blk * kBlock + e) = cm[j];
      *reinterpret_cast<Codes<W>*>((uint8_t*)st.v + blk * kBlock + e) = cv[j];
    }
    if (lane == 0) {
      st.ms[blk] = ms;
      st.vs[blk] = vs;
    }
  }
}

// The chunks k0 .. k1 - 1 of one tensor, of `blocks` blocks, the last of which
// has `tail` elements.  With 32-bit states the next chunk's loads are in flight
// under the arithmetic of this one (755 -> 722 us for 160 M bf16 elements); with
// 8-bit ones the registers cost more than that (327 us against 302 for 115 M).
template <bool k8, bool kTiny, class PT, class GT>
__device__ __forceinline__ void update_chunks(PT* p, const GT* g, uint16_t* c, const State& st,
                                              int64_t first, int64_t k0, int64_t k1, int64_t blocks,
                                              int tail, const Step& s) {
  const auto size_of = [&](int64_t b) { return b == blocks - 1 ? tail : kBlock; };
  int64_t b = k0 * kChunk + (threadIdx.x >> 5);  // this half wave's block of each chunk
  const int64_t end = k1 * kChunk < blocks ? k1 * kChunk : blocks;
  Raw<k8, PT, GT> a;
  const auto load_at = [&](Raw<k8, PT, GT>& x, int64_t i) {
    if (i < end) x.load_block(p + i * kBlock, g + i * kBlock, st, first + i, size_of(i));
  };
  if constexpr (!k8) load_at(a, b);
  for (; b < end; b += kChunk) {
    Raw<k8, PT, GT> n;
    if constexpr (k8) load_at(a, b);
    else load_at(n, b + kChunk);
    update_block<k8, kTiny>(a, p + b * kBlock, c ? c + b * kBlock : nullptr, st, first + b, size_of(b), s);
    if constexpr (!k8) a = n;
  }
}

template <bool k8, bool kTiny, bool kCopy, class Tb>
__global__ __launch_bounds__(kNT) void k_adamw(Tb tb, State st, AdamHyper hyper) {
  const Step s = step_of(hyper);
  const uint32_t total = tb.end[tb.n - 1];
  uint32_t ch = (uint32_t)((uint64_t)total * blockIdx.x / gridDim.x);
  const uint32_t che = (uint32_t)((uint64_t)total * (blockIdx.x + 1) / gridDim.x);
  if (ch >= che) return;
  int lo = 0, hi = tb.n - 1;  // the first tensor with end > ch
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (tb.end[m] > ch) hi = m;
    else lo = m + 1;
  }
  for (; ch < che; ++lo) {
    const uint32_t from = lo ? tb.end[lo - 1] : 0u, upto = tb.end[lo];
    const uint32_t tail = tb.tail[lo];
    const int64_t k0 = ch - from, k1 = (che < upto ? che : upto) - from;
    const int64_t blocks = (int64_t)(upto - from - 1) * kChunk + (tail & 7u) + 1;
    const int last = (int)((tail >> 3) & 255u) + 1;
    uint16_t* c = nullptr;
    if constexpr (kCopy) c = tb.c[lo];
    const void* g = tb.g[lo];
    void* p = tb.p[lo];
    const int64_t first = tb.first[lo];
    switch (tail >> 30) {
      case 0:
        update_chunks<k8, kTiny>((uint16_t*)p, (const uint16_t*)g, c, st, first, k0, k1, blocks, last, s);
        break;
      case 1:
        update_chunks<k8, kTiny>((uint16_t*)p, (const float*)g, c, st, first, k0, k1, blocks, last, s);
        break;
      case 2:
        update_chunks<k8, kTiny>((float*)p, (const uint16_t*)g, c, st, first, k0, k1, blocks, last, s);
        break;
      default:
        update_chunks<k8, kTiny>((float*)p, (const float*)g, c, st, first, k0, k1, blocks, last, s);
    }
    ch = from + (uint32_t)k1;
  }
}

template <class Tb, bool kCopy>
hipError_t launch(const AdamArgs& a, int cap, hipStream_t stream) {
  const State st{a.m, a.v, a.ms, a.vs};
  const bool tiny = tiny_matters(a.hyper);
  int64_t blk = 0;
  for (int64_t i = 0; i < a.n;) {
    Tb tb{};
    uint32_t end = 0;
    for (; i < a.n && tb.n < cap; ++i) {
      const int64_t blocks = (a.sizes[i] + kBlock - 1) / kBlock;
      if (blocks > 0 && a.grads[i]) {
        const int64_t chunks = (blocks + kChunk - 1) / kChunk;
        if (end + (uint64_t)chunks > 0x7fffffffu) break;  // the next launch takes it
        end += (uint32_t)chunks;
        const int k = tb.n++;
        tb.g[k] = a.grads[i];
        tb.p[k] = a.params[i];
        if constexpr (kCopy) tb.c[k] = a.copies[i];
        tb.end[k] = end;
        tb.first[k] = (uint32_t)blk;
        tb.tail[k] = (uint32_t)((blocks - 1) % kChunk) | (uint32_t)((a.sizes[i] - 1) % kBlock) << 3 |
                     (a.g_types[i] == kNormF32 ? 1u << 30 : 0u) |
                     (a.p_types[i] == kNormF32 ? 1u << 31 : 0u);
      }
      blk += blocks;
    }
    if (tb.n == 0) break;
    const dim3 grid(end < (uint32_t)kAdamGrid ? end : (uint32_t)kAdamGrid);
    auto* const k = a.bits == 8 ? (tiny ? &k_adamw<true, true, kCopy, Tb> : &k_adamw<true, false, kCopy, Tb>)
                                : (tiny ? &k_adamw<false, true, kCopy, Tb> : &k_adamw<false, false, kCopy, Tb>);
    k<<<grid, kNT, 0, stream>>>(tb, st, a.hyper);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The values that 8-bit states stand for: 4 elements of one block per thread.
__global__ __launch_bounds__(kNT) void k_adamw_values(State st, int64_t quads, float* m, float* v) {
  for (int64_t q = (int64_t)blockIdx.x * kNT + threadIdx.x; q < quads; q += (int64_t)gridDim.x * kNT) {
    const uint32_t cm = ((const uint32_t*)st.m)[q] ^ 0x80808080u, cv = ((const uint32_t*)st.v)[q];
    const float ms = st.ms[q / (kBlock / 4)], vs = st.vs[q / (kBlock / 4)];
    f32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = value_m(byte_f32(cm, i) - 128.0f, ms);
      b[i] = value_v(byte_f32(cv, i), vs);
    }
    reinterpret_cast<f32x4*>(m)[q] = a;
    reinterpret_cast<f32x4*>(v)[q] = b;
  }
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, hipStream_t stream) {
  return a.copies ? launch<CopyTable, true>(a, 104, stream) : launch<PlainTable, false>(a, 136, stream);
}

hipError_t launch_adamw_values(const void* m, const void* v, const float* ms, const float* vs,
                               int64_t blocks, float* m_out, float* v_out, hipStream_t stream) {
  const int64_t quads = blocks * (kBlock / 4);
  const int64_t groups = (quads + kNT - 1) / kNT;
  const State st{const_cast<void*>(m), const_cast<void*>(v), const_cast<float*>(ms),
                 const_cast<float*>(vs)};
  k_adamw_values<<<dim3((unsigned)(groups < 16384 ? groups : 16384)), kNT, 0, stream>>>(st, quads, m_out,
                                                                                      v_out);
  return hipGetLastError();
}

}  // namespace qn
