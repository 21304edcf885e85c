// Attention forward: O = softmax(scale Q K^T) V for each head, and the
// log-sum-exp of each row's scores, which the backward pass recomputes the
// probabilities from.
//
// One pass over the keys with the running maximum and sum of the softmax:
// for each tile of 64 keys, S^T = K Q^T, P = 2^(c S - m) with c = scale
// log2(e), O^T += V^T P^T.  The reference m of a row only moves when a tile's
// maximum lies more than kSlack above it; until then the row's values are at
// most 2^kSlack, which fp32 sums and bf16 probabilities hold as well as
// values up to 1, and the output and the sum need no rescaling.
//
// P is rounded to bf16 for the product with V (the MFMA's input type; fp32
// sums); the row sum l adds the fp32 values.
//
// Four waves of 32 queries share a workgroup's K and V tiles; two workgroups
// fit on a CU (64 KB of LDS and 211 registers each at 128 dimensions), so that
// one's exponentials run beside the other's products.  The waits and fences
// in the tile keep operand reads two steps ahead of the products and no
// further: the registers that reads further ahead would take are the second
// wave's.
//
// Measured (one sequence of 8192 tokens, 32 heads over 8 key/value heads of
// 128, causal): 513 to 533 us by the card, 1030 to 1070 TFLOP/s against 1280 to
// 1390 of large bf16 library products; the MFMA pipes are busy 52 % of the
// cycles at the 1.84 GHz that the chip holds.  8 x 512 tokens, 32 heads: 40 to
// 42 us; the tile loads alone, without the arithmetic, take 30 us (135 MB).
#include "attention.hpp"

namespace qn {
namespace {

using namespace attn;

constexpr float kSlack = 8.0f;  // in powers of two

template <int DP>
struct FwdState {
  bf16x8 q[Geo<DP>::kSteps];
  f32x16 o[Geo<DP>::kDT];
  float m;   // reference, in units of c S; -inf before the first visible key
  float l;   // this half's sum
  float c;
};

// One tile of keys; this lane's query sees tile rows 0 .. last (mask: not
// all of them in some lane).
template <int DP>
__device__ __forceinline__ void fwd_tile(FwdState<DP>& st, const uint16_t* kt, const uint16_t* vt,
                                         const FragOff& f, bool mask, int last, int half) {
  constexpr int T = Geo<DP>::kDT, S = Geo<DP>::kSteps, kAhead = 2;
  const int row = opaque(f.row);
  f32x16 s[2] = {f32x16{}, f32x16{}};
  float top = -kInf;
  {
    bf16x8 x[2 * S];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = read_rows<DP>(kt, row, i, 0);
    step_fence();
#pragma unroll
    for (int i = 0; i < 2 * S; ++i) {
      if (i + kAhead < 2 * S) x[i + kAhead] = read_rows<DP>(kt, row, (i + kAhead) % S, (i + kAhead) / S);
      s[i / S] = mfma32(x[i], st.q[i % S], s[i / S]);
      step_fence();
    }
  }
  if (mask) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (32 * r + elem_row(v, half) > last) s[r][v] = -kInf;
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int v = 0; v < 16; ++v) top = fmaxf(top, s[r][v]);
  top = fmaxf(top, other_half(top)) * st.c;
  if (__any(top > st.m + kSlack)) {
    const float m = fmaxf(st.m, top);
    // a row without a visible key so far has nothing to rescale
    const float a = m == -kInf ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= a;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) st.o[t][v] *= a;
  }
  const float m = st.m == -kInf ? 0.0f : st.m;
  const int tr = opaque(f.tr);
  constexpr int N = 4 * T;
  bf16x8 x[N];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) x[j] = read_tr<DP>(vt, tr, j % T, j / T);
  float sum = 0.0f;
  u32x4 pw[4];
  // word w (elements 2 w, 2 w + 1 of the 32 of this lane) of the probabilities
  auto prob = [&](int w) {
    const int r = w / 8, v = 2 * (w % 8);
    const float a = __builtin_amdgcn_exp2f(fmaf(s[r][v], st.c, -m));
    const float b = __builtin_amdgcn_exp2f(fmaf(s[r][v + 1], st.c, -m));
    sum += a;
    sum += b;
    pw[w / 4][w % 4] = pack_bf16x2(a, b);
  };
  // The first 32 rows' probabilities, then the others' between the products
  // with the first.
#pragma unroll
  for (int w = 0; w < 8; ++w) prob(w);
  step_fence();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (j + kAhead < N) x[j + kAhead] = read_tr<DP>(vt, tr, (j + kAhead) % T, (j + kAhead) / T);
    st.o[j % T] = mfma32(x[j], as_bf16x8(pw[j / T]), st.o[j % T]);
    if (j < N / 2) {
#pragma unroll
      for (int w = 16 * j / N; w < 16 * (j + 1) / N; ++w) prob(8 + w);
    }
    step_fence();
  }
  st.l += sum;
}

template <int DP>
__global__ __launch_bounds__(kWaves * 64, 2) void k_attn_fwd(AttnArgs p, int slots) {
  // One object per buffer, so that the compiler's waits for direct-to-LDS
  // loads apply only to the buffer they fill.
  __shared__ __attribute__((aligned(16))) uint16_t k0[Geo<DP>::kElems], v0[Geo<DP>::kElems];
  __shared__ __attribute__((aligned(16))) uint16_t k1[Geo<DP>::kElems], v1[Geo<DP>::kElems];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = find_work<false>(p, slots, p.H);
  if (!w.valid) return;
  Queries t = query_tile(p, w, wave, lane);
  if (t.first - wave * kCols >= w.lq) return;
  const TileLoader ld = tile_loader<DP>(p.D, wave, lane);
  const KeyBuffers<DP> buf{k0, v0, k1, v1};
  start_keys<DP>(buf, p, w, t, ld, wave);

  FwdState<DP> st;
  load_cols<DP>(st.q, p.q.p + w.batch * p.q.sb + (w.q0 + t.rowc) * p.q.st + w.head * p.q.sh, p.D,
                lane);
#pragma unroll
  for (int i = 0; i < Geo<DP>::kDT; ++i) st.o[i] = f32x16{};
  st.m = -kInf;
  st.l = 0.0f;
  st.c = uniform(p.scale * kLog2e);
  const FragOff f = frag_off<DP>(lane);
  walk_keys<DP>(buf, p, w, t, ld, wave,
                [&](const uint16_t* kt, const uint16_t* vt, bool mask, int last) {
                  fwd_tile<DP>(st, kt, vt, f, mask, last, half);
                });
  if (t.row >= w.lq) return;
  const float l = st.l + other_half(st.l);
  // a row that sees no key: output 0, log-sum-exp -inf
  const float mul = l == 0.0f ? 0.0f : 1.0f / l;
  const float lse = l == 0.0f ? -kInf : (st.m + __builtin_amdgcn_logf(l)) * kLn2;
  const int64_t stat = (w.batch * p.H + w.head) * p.Sq + w.q0 + t.row;
  if (p.splits == 1) {
    store_cols<DP>(p.o.p + w.batch * p.o.sb + (w.q0 + t.row) * p.o.st + w.head * p.o.sh, st.o, mul,
                   p.D, lane);
    if (half == 0) p.lse[stat] = lse;
  } else {
    const int64_t at = w.split * p.all + stat;
    store_cols<DP>(p.part + at * p.D, st.o, mul, p.D, lane);
    if (half == 0) p.part_lse[at] = lse;
  }
}

}  // namespace

hipError_t launch_attn_fwd(const AttnArgs& args, float* ws, hipStream_t stream) {
  AttnArgs a = args;
  if (a.Sq == 0 || (!a.cu_q && a.nseq == 0)) return hipSuccess;
  a.splits = attn_splits(a, kAttnFwd);
  const int64_t heads = a.H * (a.cu_q ? 1 : (int64_t)a.nseq), slots = tile_slots(a, a.Sq);
  a.all = heads * a.Sq;
  a.part = ws;
  a.part_lse = ws + a.splits * heads * a.Sq * a.D;
  const hipError_t e = with_dim(a.D, [&](auto dim) {
    return launch_groups(k_attn_fwd<decltype(dim)::value>, a, slots * heads * a.splits, slots,
                         stream);
  });
  return e != hipSuccess || a.splits == 1 ? e : launch_attn_join_fwd(a, stream);
}

}  // namespace qn
