// Rotary positions of q and k.  Pair j of the first R elements of a head at
// position p turns by the angle a = p f_j:
//
//   (x, y) -> t (x cos a - y sin a, y cos a + x sin a)
//
// with x, y the elements j and R/2 + j (halves) or 2j and 2j + 1
// (interleaved); the other elements are copied.  The backward pass is the
// transpose: the same with -a.
//
// Bound by HBM (every element read and written once).  The angles of a token
// are the same for all its heads, so a workgroup computes cos and sin of its
// tokens once, into LDS, and streams all heads of q and k past them in one
// launch.  p f_j reaches 10^7 radians at far positions, where fp32 has no
// digits left after the whole turns: the product is taken in fp64, in turns,
// and only its fraction is rounded to fp32.
#include "kernels.hpp"

namespace qn {
namespace {

constexpr int kNT = 256;

struct __attribute__((packed, aligned(2))) Loose8 {  // 8 elements at any address
  u32x4 v;
};

struct Angle {
  float c, s;
};

// Eight elements rotated with their partners: x -> x c - y s, y -> y c + x s.
__device__ __forceinline__ void turn_halves(u32x4& x, u32x4& y, const Angle* a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Angle a0 = a[2 * i], a1 = a[2 * i + 1];
    const float x0 = bf16_lo_to_f32(x[i]), x1 = bf16_hi_to_f32(x[i]);
    const float y0 = bf16_lo_to_f32(y[i]), y1 = bf16_hi_to_f32(y[i]);
    x[i] = pack_bf16x2(x0 * a0.c - y0 * a0.s, x1 * a1.c - y1 * a1.s);
    y[i] = pack_bf16x2(y0 * a0.c + x0 * a0.s, y1 * a1.c + x1 * a1.s);
  }
}

// One pair (elements i and k of a head) of any alignment.
__device__ __forceinline__ void turn_pair(uint16_t* out, const uint16_t* in, int i, int k, Angle a) {
  const float x = bf16_to_f32(in[i]), y = bf16_to_f32(in[k]);
  out[i] = f32_to_bf16(x * a.c - y * a.s);
  out[k] = f32_to_bf16(y * a.c + x * a.s);
}

// The position of a row: given, or its place in its sequence.  False for a
// row that belongs to no sequence.
__device__ __forceinline__ bool position_of(const RopeArgs& p, int64_t b, int64_t row, double& pos) {
  if (p.pos) {
    const int64_t i = b * p.pos_sb + row * p.pos_st;
    pos = p.pos64 ? (double)static_cast<const int64_t*>(p.pos)[i]
                  : (double)static_cast<const int32_t*>(p.pos)[i];
    return true;
  }
  if (!p.cu) {
    pos = (double)row;
    return true;
  }
  int lo = 0, hi = p.nseq + 1;  // offsets up to `row`
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (p.cu[m] <= row) lo = m + 1;
    else hi = m;
  }
  if (lo == 0 || lo == p.nseq + 1) return false;
  pos = (double)(row - p.cu[lo - 1]);
  return true;
}

// LDS: per token its four row offsets (q in, k in, q out, k out) and whether
// it is rotated, then R / 2 angles.
template <bool kInterleaved>
__global__ __launch_bounds__(kNT) void k_rope(RopeArgs p, int64_t tok0, int tpw) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int64_t* off = reinterpret_cast<int64_t*>(lds);  // [tpw][4]
  Angle* ang = reinterpret_cast<Angle*>(lds + 32 * tpw);
  const int half = p.rot >> 1, tid = threadIdx.x;
  // rows padded to 8 angles, so that a chunk's angles are 16-byte reads
  const int astr = (half + 7) & ~7;
  int* turned = reinterpret_cast<int*>(ang + (int64_t)tpw * astr);  // [tpw]
  tok0 += (int64_t)blockIdx.x * tpw;
  const int nt = (int)(p.tokens - tok0 < tpw ? p.tokens - tok0 : tpw);
  for (int e = tid; e < nt * half; e += kNT) {
    const int t = e / half, j = e - t * half;
    const int64_t b = (tok0 + t) / p.rows, row = (tok0 + t) - b * p.rows;
    double pos = 0.0;
    const bool in = position_of(p, b, row, pos);
    const double turns = pos * (p.freq[j] * 0.15915494309189533577);  // 1 / (2 pi)
    const float part = (float)(turns - rint(turns));
    Angle a;
    sincospif(2.0f * part, &a.s, &a.c);
    a.c *= p.scale;
    a.s *= p.inverse ? -p.scale : p.scale;
    ang[t * astr + j] = a;
    if (j == 0) {
      off[4 * t] = b * p.q.sb + row * p.q.st;
      off[4 * t + 1] = b * p.k.sb + row * p.k.st;
      off[4 * t + 2] = b * p.qo.sb + row * p.qo.st;
      off[4 * t + 3] = b * p.ko.sb + row * p.ko.st;
      turned[t] = in;
    }
  }
  __syncthreads();

  // A thread keeps its chunk of a head and walks over (token, head).
  const int nrot = kInterleaved ? (p.rot + 7) >> 3 : (half + 7) >> 3;
  const int rest = p.D - p.rot;
  const int nch = nrot + ((rest + 7) >> 3);
  const int per = kNT / nch, heads = p.H + p.Hk;
  const int ch = tid % nch;
  if (tid / nch >= per) return;
  for (int t = 0, h = tid / nch;; h += per) {
    while (h >= heads && t < nt) h -= heads, ++t;
    if (t >= nt) break;
    const bool isq = h < p.H;
    const uint16_t* in = isq ? p.q.p + off[4 * t] + h * p.q.sh
                             : p.k.p + off[4 * t + 1] + (h - p.H) * p.k.sh;
    uint16_t* out = isq ? p.qo.p + off[4 * t + 2] + h * p.qo.sh
                        : p.ko.p + off[4 * t + 3] + (h - p.H) * p.ko.sh;
    const Angle* a = ang + t * astr;
    const bool rotate = turned[t];
    if (ch < nrot && rotate) {
      if constexpr (kInterleaved) {
        const int e0 = 8 * ch, n = p.rot - e0;  // elements left
        a += e0 >> 1;
        if (n >= 8) {
          u32x4 v = reinterpret_cast<const Loose8*>(in + e0)->v;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = bf16_lo_to_f32(v[i]), y = bf16_hi_to_f32(v[i]);
            v[i] = pack_bf16x2(x * a[i].c - y * a[i].s, y * a[i].c + x * a[i].s);
          }
          reinterpret_cast<Loose8*>(out + e0)->v = v;
        } else {
          for (int i = 0; i < n; i += 2) turn_pair(out, in, e0 + i, e0 + i + 1, a[i >> 1]);
        }
      } else {
        const int e0 = 8 * ch, n = half - e0;  // pairs left
        a += e0;
        if (n >= 8) {
          u32x4 x = reinterpret_cast<const Loose8*>(in + e0)->v;
          u32x4 y = reinterpret_cast<const Loose8*>(in + half + e0)->v;
          turn_halves(x, y, a);
          reinterpret_cast<Loose8*>(out + e0)->v = x;
          reinterpret_cast<Loose8*>(out + half + e0)->v = y;
        } else {
          for (int i = 0; i < n; ++i) turn_pair(out, in, e0 + i, half + e0 + i, a[i]);
        }
      }
    } else if (out != in) {
      // elements that are not rotated: past R, or of a row of no sequence
      int e0, n;
      if (ch < nrot) {
        e0 = (kInterleaved ? 8 : 16) * ch;
        n = p.rot - e0 < (kInterleaved ? 8 : 16) ? p.rot - e0 : (kInterleaved ? 8 : 16);
      } else {
        e0 = p.rot + 8 * (ch - nrot);
        n = p.D - e0 < 8 ? p.D - e0 : 8;
      }
      for (; n >= 8; n -= 8, e0 += 8)
        reinterpret_cast<Loose8*>(out + e0)->v = reinterpret_cast<const Loose8*>(in + e0)->v;
      for (int i = 0; i < n; ++i) out[e0 + i] = in[e0 + i];
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  const int half = a.rot / 2;
  const int astr = (half + 7) & ~7;
  // About 8 chunks per thread amortize the angles; half as many tokens while
  // that leaves compute units without a workgroup.
  const int chunks = (a.H + a.Hk) * (a.D / 8);
  int tpw = 1;
  while (tpw < 32 && tpw * chunks < 8 * kNT && 2 * tpw * astr * 8 <= 16 * 1024) tpw *= 2;
  while (tpw > 1 && a.tokens / tpw < 512) tpw /= 2;
  const size_t lds = (size_t)tpw * (32 + 8 * astr + 4);
  const int64_t most = (int64_t)1 << 22;  // a launch has fewer than 2^32 threads
  const int64_t groups = (a.tokens + tpw - 1) / tpw;
  for (int64_t g = 0; g < groups; g += most) {
    const dim3 grid((unsigned)(groups - g < most ? groups - g : most));
    if (a.interleaved) k_rope<true><<<grid, kNT, lds, stream>>>(a, g * tpw, tpw);
    else k_rope<false><<<grid, kNT, lds, stream>>>(a, g * tpw, tpw);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qn
