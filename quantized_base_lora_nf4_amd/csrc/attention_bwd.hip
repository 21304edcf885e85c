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
//
// Both kernels run two workgroups of four waves per CU, within 256 registers
// per lane.  In the dK/dV kernel 192 of them hold K, V, dK and dV; the rest is
// enough because scores and dO V^T are computed 32 x 32 at a time, one after
// the other, the row statistics come by lane broadcast from two registers,
// and addresses are made anew in every step.  (With all reads moved ahead by
// the compiler the same kernel needed 512 registers, one wave per SIMD, or
// reloads that wait for the next tile: 1446 to 2100 us instead of 1000.)
//
// Measured (one sequence of 8192 tokens, 32 heads over 8 key/value heads of
// 128, causal): dQ 687 us, dK/dV 998 us and 25 us to join its two shares; the
// call takes 1716 to 1763 us by the card, 1090 to 1120 TFLOP/s over the seven
// products against 1280 to 1390 of large library products; MFMA pipes busy 59 to 63 % of the cycles at the 1.8 GHz
// that the chip holds, so the clock (power) bounds them.  8 x 512 tokens,
// 32 heads: 54 and 66 us; their loads and stores alone take 43 and 41 us.
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

// acc_x += rows of tile x times xb, acc_y likewise, 32 tile rows from 32 rt on;
// operands are read kAhead steps before their use.
template <int DP, int kAhead>
__device__ __forceinline__ void scores(f32x16& acc_x, f32x16& acc_y, const uint16_t* tx,
                                       const uint16_t* ty, const bf16x8 (&xb)[Geo<DP>::kSteps],
                                       const bf16x8 (&yb)[Geo<DP>::kSteps], const FragOff& f,
                                       int rt) {
  constexpr int N = Geo<DP>::kSteps;
  const int row = opaque(f.row);
  bf16x8 x[N], y[N];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    x[i] = read_rows<DP>(tx, row, i, rt);
    y[i] = read_rows<DP>(ty, row, i, rt);
  }
  step_fence();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + kAhead < N) {
      x[i + kAhead] = read_rows<DP>(tx, row, i + kAhead, rt);
      y[i + kAhead] = read_rows<DP>(ty, row, i + kAhead, rt);
    }
    acc_x = mfma32(x[i], xb[i], acc_x);
    acc_y = mfma32(y[i], yb[i], acc_y);
    step_fence();
  }
}

// One tile of keys; this lane's query sees tile rows 0 .. last (mask: not
// all of them in some lane).
template <int DP>
__device__ __forceinline__ void dq_tile(DqState<DP>& st, const uint16_t* kt, const uint16_t* vt,
                                        const FragOff& f, bool mask, int last, int half) {
  constexpr int T = Geo<DP>::kDT, kAhead = 2;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int tr = opaque(f.tr);
    f32x16 s = f32x16{}, dp = f32x16{};
    scores<DP, kAhead>(s, dp, kt, vt, st.q, st.g, f, r);
    bf16x8 x[2 * T];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) x[j] = read_tr<DP>(kt, tr, j % T, 2 * r + j / T);
    if (mask) {
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (32 * r + elem_row(v, half) > last) s[v] = -kInf;
    }
#pragma unroll
    for (int v = 0; v < 16; ++v)
      s[v] = __builtin_amdgcn_exp2f(fmaf(s[v], st.c, -st.lse)) * (dp[v] - st.delta);
    const bf16x8 ds[2] = {pack8(s, 0), pack8(s, 1)};
    step_fence();
#pragma unroll
    for (int j = 0; j < 2 * T; ++j) {
      if (j + kAhead < 2 * T)
        x[j + kAhead] = read_tr<DP>(kt, tr, (j + kAhead) % T, 2 * r + (j + kAhead) / T);
      st.dq[j % T] = mfma32(x[j], ds[j / T], st.dq[j % T]);
      step_fence();
    }
  }
}

template <int DP>
__global__ __launch_bounds__(kWaves * 64, 2) void k_attn_bwd_dq(AttnArgs p, int slots) {
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

  const int64_t qrow = w.q0 + t.rowc;
  const int64_t stat = (w.batch * p.H + w.head) * p.Sq + qrow;
  DqState<DP> st;
  const float lse = p.lse[stat];
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
  if (half == 0 && t.row < w.lq && w.split == 0) p.delta[stat] = st.delta;
  st.lse = lse == -kInf ? kInf : lse * kLog2e;
  st.c = uniform(p.scale * kLog2e);
#pragma unroll
  for (int i = 0; i < Geo<DP>::kDT; ++i) st.dq[i] = f32x16{};
  const FragOff f = frag_off<DP>(lane);
  walk_keys<DP>(buf, p, w, t, ld, wave,
                [&](const uint16_t* kt, const uint16_t* vt, bool mask, int last) {
                  dq_tile<DP>(st, kt, vt, f, mask, last, half);
                });
  if (t.row >= w.lq) return;
  if (p.splits == 1)
    store_cols<DP>(p.dq.p + w.batch * p.dq.sb + qrow * p.dq.st + w.head * p.dq.sh, st.dq, p.scale,
                   p.D, lane);
  else
    store_cols<DP>(p.part + (w.split * p.all + stat) * p.D, st.dq,
                   1.0f, p.D, lane);
}

// ---------------------------------------------------------------------------
// dK and dV
// ---------------------------------------------------------------------------
template <int DP>
struct DkvState {
  bf16x8 k[Geo<DP>::kSteps], v[Geo<DP>::kSteps];  // this lane's rows of K and V
  f32x16 dk[Geo<DP>::kDT], dv[Geo<DP>::kDT];
  float c, inv_scale;
};

// Lane i's value in every lane of its group of 16.
template <int I>
__device__ __forceinline__ float group_lane(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x150 + I, 0xf, 0xf, true));
}

template <class F, int... I>
__device__ __forceinline__ void each16(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

// One tile of queries; this lane's key is seen by tile rows `from` and up
// (mask: not by all of them in some lane).
// stats: lse and D of the tile's 64 rows.  Within each group of 16 lanes, lane
// i takes those of the row that element i of a score accumulator has in this
// half, and the elements get them by a lane broadcast within the group.
template <int DP>
__device__ __forceinline__ void dkv_tile(DkvState<DP>& st, const uint16_t* qt, const uint16_t* gt,
                                         const float* stats, int left, const FragOff& f, bool mask,
                                         int from) {
  constexpr int T = Geo<DP>::kDT;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int tr = opaque(f.tr), lane = lane_now(), half = lane >> 5;
    const int i = 32 * r + elem_row(lane & 15, half);
    float lse = stats[i];
    const float delta = stats[kTile + i];
    // rows past the end, and rows that see no key, have no probabilities
    lse = i < left && lse != -kInf ? lse * st.inv_scale : kInf;
    f32x16 s = rows_times<DP>(qt, st.k, f, r);
    if (mask) {
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (32 * r + elem_row(v, half) < from) s[v] = -kInf;
    }
    each16([&](auto vc) {
      constexpr int v = decltype(vc)::value;
      s[v] = __builtin_amdgcn_exp2f((s[v] - group_lane<v>(lse)) * st.c);
      if (v % 4 == 3) step_fence();
    }, std::make_integer_sequence<int, 16>{});
    f32x16 dp = rows_times<DP>(gt, st.v, f, r);
    bf16x8 x[2 * T], y[2 * T];
    x[0] = read_tr<DP>(gt, tr, 0, 2 * r);
    y[0] = read_tr<DP>(qt, tr, 0, 2 * r);
    u32x4 pw[2], dw[2];  // P and dS as operands
    each16([&](auto vc) {
      constexpr int v = decltype(vc)::value;
      dp[v] = s[v] * (dp[v] - group_lane<v>(delta));
      if constexpr (v % 2 == 1) {
        pw[v / 8][v / 2 % 4] = pack_bf16x2(s[v - 1], s[v]);
        dw[v / 8][v / 2 % 4] = pack_bf16x2(dp[v - 1], dp[v]);
        step_fence();
      }
    }, std::make_integer_sequence<int, 16>{});
    const bf16x8 pb[2] = {as_bf16x8(pw[0]), as_bf16x8(pw[1])};
    const bf16x8 ds[2] = {as_bf16x8(dw[0]), as_bf16x8(dw[1])};
    step_fence();
#pragma unroll
    for (int j = 0; j < 2 * T; ++j) {
      if (j + 1 < 2 * T) {
        x[j + 1] = read_tr<DP>(gt, tr, (j + 1) % T, 2 * r + (j + 1) / T);
        y[j + 1] = read_tr<DP>(qt, tr, (j + 1) % T, 2 * r + (j + 1) / T);
      }
      st.dv[j % T] = mfma32(x[j], pb[j / T], st.dv[j % T]);
      st.dk[j % T] = mfma32(y[j], ds[j / T], st.dk[j % T]);
      step_fence();
    }
  }
}

template <int DP>
__global__ __launch_bounds__(kWaves * 64, 2) void k_attn_bwd_dkv(AttnArgs p, int slots) {
  __shared__ __attribute__((aligned(16))) uint16_t q0[Geo<DP>::kElems], g0[Geo<DP>::kElems];
  __shared__ __attribute__((aligned(16))) uint16_t q1[Geo<DP>::kElems], g1[Geo<DP>::kElems];
  __shared__ float s0[2 * kTile], s1[2 * kTile];  // lse, then D, of the tile's rows
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = find_work<true>(p, slots, p.Hkv);
  if (!w.valid) return;
  // causal: the first keys are seen by the most queries, so they come first.
  // Where all workgroups start at once, two to a CU, the second half goes the
  // other way: the CU with the longest of the first half gets the shortest.
  const int mid = (w.ntiles + 1) / 2;
  const bool resident = p.groups <= kResident;
  const int tile =
      p.causal && resident && w.tile >= mid ? w.ntiles - 1 - (w.tile - mid) : w.tile;
  const int col0 = tile * kBlock;
  if (col0 >= w.lk) return;
  const int off = w.lk - w.lq;       // query i sees keys 0 .. i + off
  const int share = p.H / p.Hkv;

  const int first = col0 + wave * kCols;
  const int row = first + (lane & 31);
  const int rowc = row < w.lk ? row : w.lk - 1;
  const int64_t krow = w.k0 + rowc;
  const TileLoader ld = tile_loader<DP>(p.D, wave, lane);

  // tiles of queries that see any of the workgroup's keys
  const int ntq = (w.lq + kTile - 1) / kTile;
  int t0 = 0;
  if (p.causal && col0 - off > 0) t0 = (col0 - off) / kTile;
  const int per = ntq > t0 ? ntq - t0 : 0;
  const int n0 = (int)((int64_t)per * share * w.split / p.splits);
  const int n1 = (int)((int64_t)per * share * (w.split + 1) / p.splits);
  // Step n: query tile t0 + n % per of head n / per of the group.  The
  // pointers are those of the next step to issue.
  int itile = t0 + (per ? n0 % per : 0);
  const int head0 = w.head * share + (per ? n0 / per : 0);
  const int64_t row0 = w.q0 + (int64_t)itile * kTile;
  const uint16_t* qp = p.q.p + w.batch * p.q.sb + row0 * p.q.st + head0 * p.q.sh;
  const uint16_t* gp = p.dout.p + w.batch * p.dout.sb + row0 * p.dout.st + head0 * p.dout.sh;
  const float* sp = (wave & 1 ? p.delta : p.lse) + (w.batch * p.H + head0) * p.Sq + row0;
  const int64_t back = (int64_t)per * kTile;  // from the end of a head's rows to their start
  int ctile = itile;  // of the step to compute
  auto issue = [&](uint16_t* qb, uint16_t* gb, float* sb) {
    const int left = w.lq - itile * kTile;
    load_tile<DP>(qb, ld, qp, p.q.st, left, wave);
    load_tile<DP>(gb, ld, gp, p.dout.st, left, wave);
    if (wave < 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          bytes_rsrc(sp, 0x7fffffff),
          (__attribute__((address_space(3))) void*)(sb + wave * kTile), 4,
          4 * (lane < left ? lane : left - 1), 0, 0, 0);
    qp += kTile * p.q.st;
    gp += kTile * p.dout.st;
    sp += kTile;
    if (++itile == ntq) {
      itile = t0;
      qp += p.q.sh - back * p.q.st;
      gp += p.dout.sh - back * p.dout.st;
      sp += p.Sq - back;
    }
  };
  if (n0 < n1) issue(q0, g0, s0);
  DkvState<DP> st;
  load_cols<DP>(st.k, p.k.p + w.batch * p.k.sb + krow * p.k.st + w.head * p.k.sh, p.D, lane);
  load_cols<DP>(st.v, p.v.p + w.batch * p.v.sb + krow * p.v.st + w.head * p.v.sh, p.D, lane);
#pragma unroll
  for (int t = 0; t < Geo<DP>::kDT; ++t) {
    st.dk[t] = f32x16{};
    st.dv[t] = f32x16{};
  }
  st.c = uniform(p.scale * kLog2e);
  st.inv_scale = uniform(1.0f / p.scale);
  const FragOff f = frag_off<DP>(lane);
  auto step = [&](const uint16_t* qt, const uint16_t* gt, const float* stats) {
    const int r0 = ctile * kTile;
    if (++ctile == ntq) ctile = t0;
    if (first >= w.lk) return;
    if (p.causal && r0 + kTile - 1 + off < first) return;
    const bool mask = p.causal && r0 + off < first + kCols - 1;
    dkv_tile<DP>(st, qt, gt, stats, w.lq - r0, f, mask, rowc - off - r0);
  };
  for (int n = n0; n < n1; n += 2) {
    tiles_ready();
    if (n + 1 < n1) issue(q1, g1, s1);
    step(q0, g0, s0);
    if (n + 1 >= n1) break;
    tiles_ready();
    if (n + 2 < n1) issue(q0, g0, s0);
    step(q1, g1, s1);
  }
  if (row >= w.lk) return;
  if (p.splits > 1) {
    const int64_t at = w.split * p.all + (w.batch * p.Hkv + w.head) * p.Sk + krow;
    store_cols<DP>(p.part + at * p.D, st.dk, 1.0f, p.D, lane);
    store_cols<DP>(p.part + (p.splits * p.all + at) * p.D, st.dv, 1.0f, p.D, lane);
  } else {
    store_cols<DP>(p.dk.p + w.batch * p.dk.sb + krow * p.dk.st + w.head * p.dk.sh, st.dk, p.scale,
                   p.D, lane);
    store_cols<DP>(p.dv.p + w.batch * p.dv.sb + krow * p.dv.st + w.head * p.dv.sh, st.dv, 1.0f,
                   p.D, lane);
  }
}

template <int DP>
hipError_t launch_bwd(AttnArgs a, hipStream_t stream) {
  const int64_t nb = a.cu_q ? 1 : a.nseq;
  hipError_t e = hipSuccess;
  if (a.Sq > 0) {
    a.splits = attn_splits(a, kAttnDq);
    a.all = a.Sq * a.H * nb;
    const int64_t slots = tile_slots(a, a.Sq);
    e = launch_groups(k_attn_bwd_dq<DP>, a, slots * a.H * nb * a.splits, slots, stream);
    if (e == hipSuccess && a.splits > 1)
      e = launch_attn_join_sum(a, 1, &a.dq, &a.scale, a.Sq, a.H, stream);
  }
  if (e == hipSuccess && a.Sk > 0) {
    a.splits = attn_splits(a, kAttnDkv);
    a.all = a.Sk * a.Hkv * nb;
    const int64_t slots = tile_slots(a, a.Sk);
    e = launch_groups(k_attn_bwd_dkv<DP>, a, slots * a.Hkv * nb * a.splits, slots, stream);
    if (e == hipSuccess && a.splits > 1) {
      const AttnView out[2] = {a.dk, a.dv};
      const float mul[2] = {a.scale, 1.0f};
      e = launch_attn_join_sum(a, 2, out, mul, a.Sk, a.Hkv, stream);
    }
  }
  return e;
}

}  // namespace

hipError_t launch_attn_bwd(const AttnArgs& args, float* ws, hipStream_t stream) {
  AttnArgs a = args;
  if (!a.cu_q && a.nseq == 0) return hipSuccess;
  a.delta = ws;
  a.part = ws + (a.Sq * a.H * (a.cu_q ? 1 : a.nseq) + 3) / 4 * 4;
  return with_dim(a.D, [&](auto dim) { return launch_bwd<decltype(dim)::value>(a, stream); });
}

}  // namespace qn
