// How many workgroups share one tile of an attention pass, and the sums of
// their partial results.
//
// A workgroup of the forward or the dQ kernel owns 128 queries of a head and
// walks over the keys; one of the dK/dV kernel owns 128 keys and walks over
// the queries of all heads of its group.  With few such tiles (short
// sequences with few heads, a single query, few key/value heads) most of the
// chip would idle, and with a causal mask a long walk can outlast all others:
// then several workgroups share a walk, each leaves an fp32 partial result,
// and a second kernel adds them in a fixed order (8192 tokens, 8 key/value
// heads, causal: dK/dV 1318 us unshared, 998 + 25 us shared by two; the join
// reads 134 MB and writes 34, 6.7 TB/s: faster than a copy in HBM, as the partial
// results fit the Infinity Cache).
#include <math.h>

#include "attention.hpp"

namespace qn {
namespace {

using namespace attn;

// Rows of all heads on the side that a pass's columns are on.
int64_t all_rows(const AttnArgs& a, AttnPass pass) {
  const int64_t n = pass == kAttnDkv ? a.Sk * a.Hkv : a.Sq * a.H;
  return a.cu_q ? n : n * a.nseq;
}

// One partial row's 8 dimensions.
__device__ __forceinline__ void add8(float (&acc)[8], const float* p, float w) {
  const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc[e] = fmaf(w, x[e], acc[e]);
    acc[4 + e] = fmaf(w, y[e], acc[4 + e]);
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], float mul) {
  *reinterpret_cast<u32x4*>(p) =
      u32x4{pack_bf16x2(v[0] * mul, v[1] * mul), pack_bf16x2(v[2] * mul, v[3] * mul),
            pack_bf16x2(v[4] * mul, v[5] * mul), pack_bf16x2(v[6] * mul, v[7] * mul)};
}

// Row `at` of all heads ([batch][head][row] order) of a view.
__device__ __forceinline__ uint16_t* view_row(const AttnView& v, int64_t at, int64_t rows,
                                              int heads) {
  const int64_t row = at % rows, bh = at / rows;
  return v.p + bh / heads * v.sb + row * v.st + bh % heads * v.sh;
}

// O = sum over splits of exp(lse_s - lse) O_s, lse = log sum exp lse_s; 8
// dimensions per thread.
__global__ __launch_bounds__(256) void k_attn_join_fwd(AttnArgs p, int64_t rows) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = p.D / 8;
  const int64_t at = i / per;
  const int d = (int)(i % per) * 8;
  if (at >= rows) return;
  float top = -kInf;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.part_lse[s * rows + at]);
  const float base = top == -kInf ? 0.0f : top;
  float total = 0.0f, acc[8] = {};
  for (int s = 0; s < p.splits; ++s) {
    // a NaN somewhere keeps its way into the row
    const float w = __builtin_amdgcn_exp2f((p.part_lse[s * rows + at] - base) * kLog2e);
    total += w;
    add8(acc, p.part + (s * rows + at) * p.D + d, w);
  }
  store8(view_row(p.o, at, p.Sq, p.H) + d, acc, total == 0.0f ? 0.0f : 1.0f / total);
  if (d == 0) p.lse[at] = total == 0.0f ? -kInf : base + __builtin_amdgcn_logf(total) * kLn2;
}

struct JoinOut {
  AttnView v[2];
  float mul[2];
};

__global__ __launch_bounds__(256) void k_attn_join_sum(const float* part, int splits, int64_t all,
                                                       int64_t rows, int heads, int D,
                                                       JoinOut out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = D / 8;
  const int64_t at = i / per;
  const int d = (int)(i % per) * 8;
  if (at >= all) return;
  const float* src = part + (blockIdx.y * (int64_t)splits * all + at) * D + d;
  float acc[8] = {};
  for (int s = 0; s < splits; ++s) add8(acc, src + s * all * D, 1.0f);
  const int y = blockIdx.y;
  store8(view_row(y ? out.v[1] : out.v[0], at, rows, heads) + d, acc, y ? out.mul[1] : out.mul[0]);
}

}  // namespace

// The split that the following estimate finds fastest.  Times in us, from
// measurements at D = 128 (in proportion for 64 and 96): a step (64 rows of the
// walk) takes a workgroup 2.1 in the forward, 2.8 in dQ and 4.0 in dK/dV while
// two share a CU, and about 0.65 of that alone; starting and storing a tile
// about 4; a join about 6 and its partial results' bytes, written and read, at
// 4 TB/s.  Packed lengths are known to the device only: for n sequences cut at
// random the longest is taken to be 1 + log2(n) / 2 times the mean, and a
// tile's mean walk up to 1.8 times.  What the walk reads is not in it: for one
// query, 8192 keys and 32 key/value heads of 128 it expects 24 us, their bytes
// take 26 and the call 41.
int attn_splits(const AttnArgs& a, AttnPass pass) {
  const bool keys = pass == kAttnDkv;
  const int64_t cols = keys ? a.Sk : a.Sq, walk = keys ? a.Sq : a.Sk;
  const int heads = keys ? a.Hkv : a.H;
  const int64_t n = a.nseq > 0 ? a.nseq : 1;
  const int64_t tiles = a.cu_q ? (cols + kBlock - 1) / kBlock * heads
                               : (cols + kBlock - 1) / kBlock * heads * a.nseq;
  const int64_t len = a.cu_q ? (walk + n - 1) / n : walk;
  const int64_t steps = (len + kTile - 1) / kTile * (keys ? a.H / a.Hkv : 1);
  if (tiles < 1 || tiles > 65536 || steps < 2) return 1;
  const double unit = (pass == kAttnFwd ? 2.1 : pass == kAttnDq ? 2.8 : 4.0) *
                      (a.D <= 64 ? 0.5 : a.D <= 96 ? 0.75 : 1.0);
  const double uneven = a.cu_q ? 1.0 + 0.5 * log2((double)n) : 1.0;
  const double total =
      (double)tiles * steps * (uneven < 1.8 ? uneven : 1.8) * (a.causal ? 0.55 : 1.0);
  const double bytes = (double)all_rows(a, pass) * a.D * 8.0 * (keys ? 2 : 1);
  int best = 1;
  double best_t = 0.0;
  for (int s = 1; s <= 32 && s <= steps; s = s < 4 ? s + 1 : s + s / 2) {
    const double longest = (double)((steps + s - 1) / s) * uneven;
    const double slots = tiles * s < kResident ? (double)(tiles * s) : (double)kResident;
    const double step = unit * (tiles * s > kResident / 2 ? 1.0 : 0.65);
    const double rounds = total / s > 0 ? total / slots : 0.0;
    double t = (rounds > longest ? rounds : longest) * step +
               4.0 * (double)(tiles * s) / slots;
    if (s > 1) t += 6.0 + s * bytes / 4e6;
    if (s == 1 || t < 0.95 * best_t) {
      best = s;
      best_t = t;
    }
  }
  return best;
}

int64_t attn_fwd_workspace(const AttnArgs& a) {
  const int s = attn_splits(a, kAttnFwd);
  return s > 1 ? s * all_rows(a, kAttnFwd) * (a.D + 1) : 0;
}

int64_t attn_bwd_workspace(const AttnArgs& a) {
  const int sq = attn_splits(a, kAttnDq), sk = attn_splits(a, kAttnDkv);
  const int64_t q = sq > 1 ? sq * all_rows(a, kAttnDq) * a.D : 0;
  const int64_t k = sk > 1 ? 2 * sk * all_rows(a, kAttnDkv) * a.D : 0;
  const int64_t delta = (all_rows(a, kAttnDq) + 3) / 4 * 4;  // what follows is 16-byte aligned
  return delta + (q > k ? q : k);
}

hipError_t launch_attn_join_fwd(const AttnArgs& a, hipStream_t stream) {
  const int64_t rows = all_rows(a, kAttnFwd);
  const int64_t n = (rows * (a.D / 8) + 255) / 256;
  k_attn_join_fwd<<<(unsigned)n, 256, 0, stream>>>(a, rows);
  return hipGetLastError();
}

hipError_t launch_attn_join_sum(const AttnArgs& a, int n, const AttnView* out, const float* mul,
                                int64_t rows, int heads, hipStream_t stream) {
  const int64_t all = rows * heads * (a.cu_q ? 1 : a.nseq);
  JoinOut o{};
  for (int i = 0; i < n; ++i) {
    o.v[i] = out[i];
    o.mul[i] = mul[i];
  }
  const dim3 grid((unsigned)((all * (a.D / 8) + 255) / 256), n);
  k_attn_join_sum<<<grid, 256, 0, stream>>>(a.part, a.splits, all, rows, heads, a.D, o);
  return hipGetLastError();
}

}  // namespace qn
