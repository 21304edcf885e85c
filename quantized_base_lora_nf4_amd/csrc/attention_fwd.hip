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

// One tile of keys.  kMask: some of its keys may be hidden: this lane's
// query sees tile rows 0 .. last.
template <int DP, bool kMask>
__device__ __forceinline__ void fwd_tile(FwdState<DP>& st, const uint16_t* kt, const uint16_t* vt,
                                         const FragOff& f, int last, int half) {
  f32x16 s[2] = {f32x16{}, f32x16{}};
#pragma unroll
  for (int i = 0; i < Geo<DP>::kSteps; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) s[r] = mfma32(read_rows<DP>(kt, f.row, i, r), st.q[i], s[r]);
  float top = -kInf;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      if (kMask && 32 * r + elem_row(v, half) > last) s[r][v] = -kInf;
      top = fmaxf(top, s[r][v]);
    }
  top = fmaxf(top, other_half(top)) * st.c;
  if (__any(top > st.m + kSlack)) {
    const float m = fmaxf(st.m, top);
    // a row without a visible key so far has nothing to rescale
    const float a = m == -kInf ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= a;
#pragma unroll
    for (int t = 0; t < Geo<DP>::kDT; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) st.o[t][v] *= a;
  }
  const float m = st.m == -kInf ? 0.0f : st.m;
  float sum = 0.0f;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      s[r][v] = __builtin_amdgcn_exp2f(fmaf(s[r][v], st.c, -m));
      sum += s[r][v];
    }
  st.l += sum;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const bf16x8 pb = pack8(s[b >> 1], b & 1);
#pragma unroll
    for (int t = 0; t < Geo<DP>::kDT; ++t) st.o[t] = mfma32(read_tr<DP>(vt, f.tr, t, b), pb, st.o[t]);
  }
}

template <int DP>
__global__ __launch_bounds__(kWaves * 64, 2) void k_attn_fwd(AttnArgs p, int64_t slots) {
  // One object per buffer, so that the compiler's waits for direct-to-LDS
  // loads apply only to the buffer they fill.
  __shared__ __attribute__((aligned(16))) uint16_t k0[Geo<DP>::kElems], v0[Geo<DP>::kElems];
  __shared__ __attribute__((aligned(16))) uint16_t k1[Geo<DP>::kElems], v1[Geo<DP>::kElems];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = find_work<false>(p, slots, p.H);
  if (!w.valid) return;
  // causal: the tiles with the most keys first
  const int tile = p.causal ? w.ntiles - 1 - w.tile : w.tile;
  const int col0 = tile * kBlock;
  if (col0 >= w.lq) return;
  const int off = w.lk - w.lq;                     // query i sees keys 0 .. i + off
  const int hk = w.head / (p.H / p.Hkv);
  const uint16_t* kb = p.k.p + w.batch * p.k.sb + w.k0 * p.k.st + hk * p.k.sh;
  const uint16_t* vb = p.v.p + w.batch * p.v.sb + w.k0 * p.v.st + hk * p.v.sh;

  const int first = col0 + wave * kCols;           // this wave's queries
  const int row = first + (lane & 31);             // this lane's
  const int rowc = row < w.lq ? row : w.lq - 1;
  FwdState<DP> st;
  load_cols<DP>(st.q, p.q.p + w.batch * p.q.sb + (w.q0 + rowc) * p.q.st + w.head * p.q.sh, p.D, lane);
#pragma unroll
  for (int t = 0; t < Geo<DP>::kDT; ++t) st.o[t] = f32x16{};
  st.m = -kInf;
  st.l = 0.0f;
  st.c = uniform(p.scale * kLog2e);
  const FragOff f = frag_off<DP>(lane);
  const TileLoader ld = tile_loader<DP>(p.D, wave, lane);

  // keys that any query of the workgroup sees
  int keys = w.lk;
  if (p.causal) {
    const int e = (col0 + kBlock < w.lq ? col0 + kBlock : w.lq) + off;
    keys = e < keys ? (e > 0 ? e : 0) : keys;
  }
  const int nt = (keys + kTile - 1) / kTile;
  // of this wave: all of the tile below `full`, none from `end` on
  const int seen_first = p.causal ? first + off : w.lk - 1;
  const int seen_last = p.causal ? (first + kCols - 1 + off < w.lk - 1 ? first + kCols - 1 + off : w.lk - 1) : w.lk - 1;
  const int mine = p.causal ? (rowc + off < w.lk - 1 ? rowc + off : w.lk - 1) : w.lk - 1;

  auto step = [&](const uint16_t* kt, const uint16_t* vt, int j) {
    const int r0 = j * kTile;
    if (first >= w.lq || r0 > seen_last) return;
    if (r0 + kTile - 1 <= seen_first && r0 + kTile <= w.lk)
      fwd_tile<DP, false>(st, kt, vt, f, 0, half);
    else
      fwd_tile<DP, true>(st, kt, vt, f, mine - r0, half);
  };
  if (nt > 0) {
    load_tile<DP>(k0, ld, kb, p.k.st, w.lk, wave);
    load_tile<DP>(v0, ld, vb, p.v.st, w.lk, wave);
  }
  for (int j = 0; j < nt; j += 2) {
    tiles_ready();
    if (j + 1 < nt) {
      load_tile<DP>(k1, ld, kb + (j + 1) * (kTile * p.k.st), p.k.st, w.lk - (j + 1) * kTile, wave);
      load_tile<DP>(v1, ld, vb + (j + 1) * (kTile * p.v.st), p.v.st, w.lk - (j + 1) * kTile, wave);
    }
    step(k0, v0, j);
    if (j + 1 >= nt) break;
    tiles_ready();
    if (j + 2 < nt) {
      load_tile<DP>(k0, ld, kb + (j + 2) * (kTile * p.k.st), p.k.st, w.lk - (j + 2) * kTile, wave);
      load_tile<DP>(v0, ld, vb + (j + 2) * (kTile * p.v.st), p.v.st, w.lk - (j + 2) * kTile, wave);
    }
    step(k1, v1, j + 1);
  }
  if (row >= w.lq) return;
  const float l = st.l + other_half(st.l);
  // a row that sees no key: output 0, log-sum-exp -inf
  store_cols<DP>(p.o.p + w.batch * p.o.sb + (w.q0 + row) * p.o.st + w.head * p.o.sh, st.o,
                 l == 0.0f ? 0.0f : 1.0f / l, p.D, lane);
  if (half == 0)
    p.lse[(w.batch * p.H + w.head) * p.Sq + w.q0 + row] =
        l == 0.0f ? -kInf : (st.m + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t stream) {
  if (a.Sq == 0 || (!a.cu_q && a.nseq == 0)) return hipSuccess;
  const int64_t slots = tile_slots(a, a.Sq);
  const int64_t grid = slots * a.H * (a.cu_q ? 1 : a.nseq);
  if (a.D <= 64) k_attn_fwd<64><<<(unsigned)grid, kWaves * 64, 0, stream>>>(a, slots);
  else k_attn_fwd<128><<<(unsigned)grid, kWaves * 64, 0, stream>>>(a, slots);
  return hipGetLastError();
}

}  // namespace qn
