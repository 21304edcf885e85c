// Attention backward, from the inputs, the output's gradient dO, the output
// O and the rows' log-sum-exp of the forward pass:
//   P  = exp(scale Q K^T - lse)          (recomputed tile by tile)
//   D  = sum over the dimension of dO O
//   dS = P (dO V^T - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
// with dK and dV summed over the query heads that share a key/value head.
//
// Two kernels, one per operand that stays: k_attn_bwd_dq keeps 32 query rows
// per wave and walks over the keys (it also computes D, for both), and
// k_attn_bwd_dkv keeps 32 keys per wave and walks over the queries of all
// heads of the group.  The scores and dO V^T are computed in both, seven
// products instead of five; in return every sum is made in registers in a
// fixed order: no atomics, no fp32 copy of dQ in memory, the same bits on
// every run.
//
// P and dS are rounded to bf16 as operands of the products that follow
// (fp32 sums), everything else is fp32.
#include <utility>

#include "attention.hpp"

namespace qn {
namespace {

using namespace attn;

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
template <int DP>
struct DqState {
  bf16x8 q[Geo<DP>::kSteps], g[Geo<DP>::kSteps];  // this lane's rows of Q and dO
  f32x16 dq[Geo<DP>::kDT];
  float c, lse, delta;  // scale log2(e); lse in powers of two, +inf if the row sees no key
};

// One tile of keys; this lane's query sees tile rows 0 .. last.
template <int DP, bool kMask>
__device__ __forceinline__ void dq_tile(DqState<DP>& st, const uint16_t* kt, const uint16_t* vt,
                                        const FragOff& f, int last, int half) {
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
    for (int i = 0; i < Geo<DP>::kSteps; ++i) {
      s = mfma32(read_rows<DP>(kt, f, i, r), st.q[i], s);
      dp = mfma32(read_rows<DP>(vt, f, i, r), st.g[i], dp);
    }
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      if (kMask && 32 * r + elem_row(v, half) > last) s[v] = -kInf;
      s[v] = __builtin_amdgcn_exp2f(fmaf(s[v], st.c, -st.lse)) * (dp[v] - st.delta);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bf16x8 ds = pack8(s, b);
#pragma unroll
      for (int t = 0; t < Geo<DP>::kDT; ++t)
        st.dq[t] = mfma32(read_tr<DP>(kt, f, t, 2 * r + b), ds, st.dq[t]);
    }
  }
}

template <int DP>
__global__ __launch_bounds__(kWaves * 64, 1) void k_attn_bwd_dq(AttnArgs p, int64_t slots) {
  __shared__ __attribute__((aligned(16))) uint16_t k0[Geo<DP>::kElems], v0[Geo<DP>::kElems];
  __shared__ __attribute__((aligned(16))) uint16_t k1[Geo<DP>::kElems], v1[Geo<DP>::kElems];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = find_work<false>(p, xcd_order(blockIdx.x, gridDim.x), slots, p.H);
  if (!w.valid) return;
  const int tile = p.causal ? w.ntiles - 1 - w.tile : w.tile;
  const int col0 = tile * kBlock;
  if (col0 >= w.lq) return;
  const int off = w.lk - w.lq;
  const int hk = w.head / (p.H / p.Hkv);
  const uint16_t* kb = p.k.p + w.batch * p.k.sb + w.k0 * p.k.st + hk * p.k.sh;
  const uint16_t* vb = p.v.p + w.batch * p.v.sb + w.k0 * p.v.st + hk * p.v.sh;

  const int first = col0 + wave * kCols;
  const int row = first + (lane & 31);
  const int rowc = row < w.lq ? row : w.lq - 1;
  const int64_t qrow = w.q0 + rowc;
  const int64_t stat = (w.batch * p.H + w.head) * p.Sq + qrow;
  DqState<DP> st;
  load_cols<DP>(st.q, p.q.p + w.batch * p.q.sb + qrow * p.q.st + w.head * p.q.sh, p.D, lane);
  load_cols<DP>(st.g, p.dout.p + w.batch * p.dout.sb + qrow * p.dout.st + w.head * p.dout.sh, p.D,
                lane);
  {
    bf16x8 o[Geo<DP>::kSteps];
    load_cols<DP>(o, p.o.p + w.batch * p.o.sb + qrow * p.o.st + w.head * p.o.sh, p.D, lane);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < Geo<DP>::kSteps; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf((float)st.g[i][e], (float)o[i][e], d);
    st.delta = d + other_half(d);
  }
  if (half == 0 && row < w.lq) p.delta[stat] = st.delta;
  const float lse = p.lse[stat];
  st.lse = lse == -kInf ? kInf : lse * kLog2e;
  st.c = p.scale * kLog2e;
#pragma unroll
  for (int t = 0; t < Geo<DP>::kDT; ++t) st.dq[t] = f32x16{};
  const FragOff f = frag_off<DP>(lane);
  TileLoader<DP> ld;
  tile_loader<DP>(ld, p.D, wave, lane);

  int keys = w.lk;
  if (p.causal) {
    const int e = (col0 + kBlock < w.lq ? col0 + kBlock : w.lq) + off;
    keys = e < keys ? (e > 0 ? e : 0) : keys;
  }
  const int nt = (keys + kTile - 1) / kTile;
  const int seen_first = p.causal ? first + off : w.lk - 1;
  int seen_last = w.lk - 1, mine = w.lk - 1;
  if (p.causal) {
    if (first + kCols - 1 + off < seen_last) seen_last = first + kCols - 1 + off;
    if (rowc + off < mine) mine = rowc + off;
  }
  auto step = [&](const uint16_t* kt, const uint16_t* vt, int j) {
    const int r0 = j * kTile;
    if (first >= w.lq || r0 > seen_last) return;
    if (r0 + kTile - 1 <= seen_first && r0 + kTile <= w.lk)
      dq_tile<DP, false>(st, kt, vt, f, 0, half);
    else
      dq_tile<DP, true>(st, kt, vt, f, mine - r0, half);
  };
  if (nt > 0) {
    load_tile<DP>(k0, ld, kb, p.k.st, 0, w.lk, wave);
    load_tile<DP>(v0, ld, vb, p.v.st, 0, w.lk, wave);
  }
  for (int j = 0; j < nt; j += 2) {
    tiles_ready();
    if (j + 1 < nt) {
      load_tile<DP>(k1, ld, kb, p.k.st, (j + 1) * kTile, w.lk, wave);
      load_tile<DP>(v1, ld, vb, p.v.st, (j + 1) * kTile, w.lk, wave);
    }
    step(k0, v0, j);
    if (j + 1 >= nt) break;
    tiles_ready();
    if (j + 2 < nt) {
      load_tile<DP>(k0, ld, kb, p.k.st, (j + 2) * kTile, w.lk, wave);
      load_tile<DP>(v0, ld, vb, p.v.st, (j + 2) * kTile, w.lk, wave);
    }
    step(k1, v1, j + 1);
  }
  if (row < w.lq)
    store_cols<DP>(p.dq.p + w.batch * p.dq.sb + qrow * p.dq.st + w.head * p.dq.sh, st.dq, p.scale,
                   p.D, lane);
}

// ---------------------------------------------------------------------------
// dK and dV
// ---------------------------------------------------------------------------
template <int DP>
struct DkvState {
  bf16x8 k[Geo<DP>::kSteps], v[Geo<DP>::kSteps];  // this lane's rows of K and V
  f32x16 dk[Geo<DP>::kDT], dv[Geo<DP>::kDT];
  float c;
};

// Row statistics of a tile, spread over the lanes: within each group of 16
// lanes, lane i holds those of the row that element i of a score accumulator
// has in this half.
struct RowStats {
  float lse[2], delta[2];  // rows 0..31 and 32..63; lse / scale, +inf for a row to leave out
};

// Lane i's value in every lane of its group of 16.
template <int I>
__device__ __forceinline__ float group_lane(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + I, 0xf, 0xf, false));
}

template <class F, int... I>
__device__ __forceinline__ void each16(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

// One tile of queries; this lane's key is seen by tile rows `from` and up.
template <int DP, bool kMask>
__device__ __forceinline__ void dkv_tile(DkvState<DP>& st, const uint16_t* qt, const uint16_t* gt,
                                         const RowStats& rs, const FragOff& f, int from,
                                         int half) {
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
    for (int i = 0; i < Geo<DP>::kSteps; ++i) {
      s = mfma32(read_rows<DP>(qt, f, i, r), st.k[i], s);
      dp = mfma32(read_rows<DP>(gt, f, i, r), st.v[i], dp);
    }
    each16(
        [&](auto vc) {
          constexpr int v = decltype(vc)::value;
          float x = (s[v] - group_lane<v>(rs.lse[r])) * st.c;
          if (kMask && 32 * r + elem_row(v, half) < from) x = -kInf;
          s[v] = __builtin_amdgcn_exp2f(x);
          dp[v] = s[v] * (dp[v] - group_lane<v>(rs.delta[r]));
        },
        std::make_integer_sequence<int, 16>{});
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bf16x8 pb = pack8(s, b), ds = pack8(dp, b);
#pragma unroll
      for (int t = 0; t < Geo<DP>::kDT; ++t) {
        st.dv[t] = mfma32(read_tr<DP>(gt, f, t, 2 * r + b), pb, st.dv[t]);
        st.dk[t] = mfma32(read_tr<DP>(qt, f, t, 2 * r + b), ds, st.dk[t]);
      }
    }
  }
}

template <int DP>
__global__ __launch_bounds__(kWaves * 64, 1) void k_attn_bwd_dkv(AttnArgs p, int64_t slots) {
  __shared__ __attribute__((aligned(16))) uint16_t q0[Geo<DP>::kElems], g0[Geo<DP>::kElems];
  __shared__ __attribute__((aligned(16))) uint16_t q1[Geo<DP>::kElems], g1[Geo<DP>::kElems];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = find_work<true>(p, xcd_order(blockIdx.x, gridDim.x), slots, p.Hkv);
  if (!w.valid) return;
  const int col0 = w.tile * kBlock;  // causal: the first keys are seen by the most queries
  if (col0 >= w.lk) return;
  const int off = w.lk - w.lq;       // query i sees keys 0 .. i + off
  const int share = p.H / p.Hkv;

  const int first = col0 + wave * kCols;
  const int row = first + (lane & 31);
  const int rowc = row < w.lk ? row : w.lk - 1;
  const int64_t krow = w.k0 + rowc;
  DkvState<DP> st;
  load_cols<DP>(st.k, p.k.p + w.batch * p.k.sb + krow * p.k.st + w.head * p.k.sh, p.D, lane);
  load_cols<DP>(st.v, p.v.p + w.batch * p.v.sb + krow * p.v.st + w.head * p.v.sh, p.D, lane);
#pragma unroll
  for (int t = 0; t < Geo<DP>::kDT; ++t) {
    st.dk[t] = f32x16{};
    st.dv[t] = f32x16{};
  }
  st.c = p.scale * kLog2e;
  const float inv_scale = 1.0f / p.scale;
  const FragOff f = frag_off<DP>(lane);
  TileLoader<DP> ld;
  tile_loader<DP>(ld, p.D, wave, lane);

  // tiles of queries that see any of the workgroup's keys
  const int ntq = (w.lq + kTile - 1) / kTile;
  int t0 = 0;
  if (p.causal && col0 - off > 0) t0 = (col0 - off) / kTile;
  const int per = ntq > t0 ? ntq - t0 : 0;
  const int nt = per * share;
  const int stat_row = elem_row(lane & 15, half);

  // Step n: query tile t0 + n % per of head n / per of the group.
  int ihead = 0, itile = t0;  // of the next step to issue
  RowStats nrs;
  auto issue = [&](uint16_t* qb, uint16_t* gb) {
    const int head = w.head * share + ihead;
    const int r0 = itile * kTile;
    load_tile<DP>(qb, ld, p.q.p + w.batch * p.q.sb + w.q0 * p.q.st + head * p.q.sh, p.q.st, r0,
                  w.lq, wave);
    load_tile<DP>(gb, ld, p.dout.p + w.batch * p.dout.sb + w.q0 * p.dout.st + head * p.dout.sh,
                  p.dout.st, r0, w.lq, wave);
    const int64_t stat = (w.batch * p.H + head) * p.Sq + w.q0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = r0 + 32 * r + stat_row;
      const int ic = i < w.lq ? i : w.lq - 1;
      const float lse = p.lse[stat + ic], delta = p.delta[stat + ic];
      // rows past the end, and rows that see no key, have no probabilities
      nrs.lse[r] = i < w.lq && lse != -kInf ? lse * inv_scale : kInf;
      nrs.delta[r] = delta;
    }
    if (++itile == ntq) {
      itile = t0;
      ++ihead;
    }
  };
  int ctile = t0;  // of the step to compute
  auto step = [&](const uint16_t* qt, const uint16_t* gt, const RowStats& rs) {
    const int r0 = ctile * kTile;
    if (++ctile == ntq) ctile = t0;
    if (first >= w.lk) return;
    if (!p.causal || r0 + off >= first + kCols - 1)
      dkv_tile<DP, false>(st, qt, gt, rs, f, 0, half);
    else if (r0 + kTile - 1 + off >= first)
      dkv_tile<DP, true>(st, qt, gt, rs, f, rowc - off - r0, half);
  };
  if (nt > 0) issue(q0, g0);
  for (int n = 0; n < nt; n += 2) {
    RowStats rs = nrs;
    tiles_ready();
    if (n + 1 < nt) issue(q1, g1);
    step(q0, g0, rs);
    if (n + 1 >= nt) break;
    rs = nrs;
    tiles_ready();
    if (n + 2 < nt) issue(q0, g0);
    step(q1, g1, rs);
  }
  if (row < w.lk) {
    store_cols<DP>(p.dk.p + w.batch * p.dk.sb + krow * p.dk.st + w.head * p.dk.sh, st.dk, p.scale,
                   p.D, lane);
    store_cols<DP>(p.dv.p + w.batch * p.dv.sb + krow * p.dv.st + w.head * p.dv.sh, st.dv, 1.0f,
                   p.D, lane);
  }
}

template <int DP>
hipError_t launch_bwd(const AttnArgs& a, hipStream_t stream) {
  const int64_t nb = a.cu_q ? 1 : a.nseq;
  if (a.Sq > 0) {
    const int64_t slots = tile_slots(a, a.Sq);
    k_attn_bwd_dq<DP><<<(unsigned)(slots * a.H * nb), kWaves * 64, 0, stream>>>(a, slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.Sk > 0) {
    const int64_t slots = tile_slots(a, a.Sk);
    k_attn_bwd_dkv<DP><<<(unsigned)(slots * a.Hkv * nb), kWaves * 64, 0, stream>>>(a, slots);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t stream) {
  if (!a.cu_q && a.nseq == 0) return hipSuccess;
  return a.D <= 64 ? launch_bwd<64>(a, stream) : launch_bwd<128>(a, stream);
}

}  // namespace qn
