// Forward pass for rows of many adapters, from 17 rows to a few hundred: the
// decoding batch of a server.  At these sizes the tiles of qgemm.hip leave
// most of the chip idle (61 rows over 8192 x 8192: 64 workgroups of 128 steps
// each), and the cost should be that of streaming the weight.
//
// As in gemv.hip a workgroup owns 16 G weight rows and all of K, its 8 waves
// split K, codes are expanded to unscaled bf16 levels by a byte-indexed table
// in LDS, and the block constant multiplies each 64-element block's fp32 sum:
// the levels' rounding (6e-4 of a weight, level_factor) takes the place of the
// dequantized weight's (1.7e-3), and X A^T is not rounded.
// Here up to 16 T tokens share the expanded codes: T MFMA column tiles per
// code word.  Every workgroup reads all of X (from L2; G = 4 halves that
// traffic), so it comes in the order of the MFMA operands, 1 KB per load, as
// the down products write it: read in rows, whose fragments put neighbouring
// lanes 2 K bytes apart, 64 rows over 8192 x 8192 took 47 instead of 29 us.
// More tokens make more workgroups (grid dimension y), which find the weight in
// the caches.
//
// The LoRA term is added in the epilogue from U = X A^T (multi.hip), summed
// over its slices and scaled into LDS at the start; every output reads the
// adapter rows of its own token, so adapters never meet.
//
// Operand layout and double steps: see gemv.hip.
//
// Measured, 64 rows over 8192 x 8192, rank 32: 24 us (the weight alone: 7 us at
// a large copy's rate), about 8 of them before and after the loop.  128 rows
// with G = 4: 35 us, where G = 2 takes two rounds of workgroups, 46 us.  In the
// loop a compute unit's parts come close to each other: per step of 128 columns
// and 8 waves (G = 4, T = 4) 0.5 us of MFMAs, about 1 us each of vector
// instructions, of table lookups and of X through the L1; it takes 3.
#include "kernels.hpp"

namespace qn {
namespace {

constexpr int KW = 8, NT = 64 * KW;
constexpr int kLutWords = 256 * 16;
constexpr int kMaxSlices = 8;  // of multi.hip

__device__ __forceinline__ u32x4 levels8(uint32_t w, const uint32_t* lutl) {
  return u32x4{lutl[16 * (w & 0xffu)], lutl[16 * ((w >> 8) & 0xffu)],
               lutl[16 * ((w >> 16) & 0xffu)], lutl[16 * (w >> 24)]};
}

struct RowsArgs {
  const uint8_t* codes;
  const uint8_t* q8;
  const float* step;
  const uint16_t* xfrag; // X as multi.hip writes it
  int64_t M, N, K;
  const float* part;     // [slices][M][ldp]
  int slices;
  int64_t ldp;
  const uint16_t* B;     // [adapters][N][r]
  int32_t r;
  const int32_t* index;
  int adapters;
  uint16_t* Y;
  int bshift;
  UserTable ut;
};

// LDS in words: U of the workgroup's tokens, their adapters, then the byte table
// and the block constants during the main loop, the waves' sums after it.
__host__ __device__ constexpr int64_t rows_lds_words(int G, int T, int64_t ldp, int64_t kblocks) {
  const int64_t chat = 16 * G * (kblocks | 1), red = (int64_t)KW * G * T * 256;
  return 16 * T * ldp + 16 * T + (kLutWords + chat > red ? kLutWords + chat : red);
}

template <int G, int T, class CT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(2)))
void k_qrows(RowsArgs p) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  // Steps of loads in flight: a step's registers are loaded anew as soon as they
  // have been used.  A second set for the larger tiles spills outside the loop,
  // or costs time without (64 rows over 8192 x 8192: 41.3 against 37.3 us a call;
  // 17 over 28672 x 8192, G = 4: 63.5 against 61.6).
  constexpr int kAhead = G * T > 4 ? 1 : 2;
  float* ush = lds;                                            // [16 T][ldp]
  int* own = reinterpret_cast<int*>(ush + 16 * T * p.ldp);     // [16 T]
  uint32_t* lut = reinterpret_cast<uint32_t*>(own + 16 * T);
  float* chat = reinterpret_cast<float*>(lut + kLutWords);     // [16 G][kblocks | 1]
  float* red = reinterpret_cast<float*>(lut);                                           // [KW][G][T][4][64]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  const int64_t N = p.N, K = p.K, kblocks = K >> 6, kbs = kblocks | 1;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * G, m0 = (int64_t)blockIdx.y * 16 * T;
  const int mt = (int)(p.M - m0 < 16 * T ? p.M - m0 : 16 * T);  // tokens here

  // double steps of this wave (pairs of waves share a range, as in gemv.hip)
  const int64_t D = kblocks >> 1;
  const int64_t e0 = D * (wave >> 1) / (KW / 2), e1 = D * ((wave >> 1) + 1) / (KW / 2);
  const int64_t base = e0 + (wave & 1);
  const int64_t d1 = e1 > base ? (e1 - base + 1) / 2 : 0;
  const bool odd_tail = (kblocks & 1) && wave == KW - 1;

  const uint8_t* crow[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    int64_t n = n0 + 16 * g + i16;
    if (n >= N) n = N - 1;  // computed and dropped
    crow[g] = p.codes + n * kblocks * block_bytes<CT>() + (q >> 1) * block_bytes<CT>() +
              (q & 1) * half_bytes<CT>();
  }
  // token tiles past the last one are computed from it and dropped
  const uint16_t* xt[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    int64_t tile = (m0 >> 4) + t;
    if (16 * tile >= p.M) tile = (p.M - 1) >> 4;
    xt[t] = p.xfrag + tile * (K >> 5) * 512;
  }
  const float* crow_t[G];
#pragma unroll
  for (int g = 0; g < G; ++g) crow_t[g] = chat + (16 * g + i16) * kbs;

  struct Slot {
    HalfRaw<CT::kBits> c[G];
    u32x4 x[T][4];
  };
  // The parts of a step's loads: the codes, and X of its block h.
  auto issue_codes = [&](Slot& S, int64_t d, bool tail) {
    const int64_t kb = 2 * (tail ? d : base + 2 * d);
    const int64_t off = ((tail && q >= 2) ? kb - 1 : kb) * block_bytes<CT>();
#pragma unroll
    for (int g = 0; g < G; ++g) S.c[g] = load_half<CT>(crow[g] + off);
  };
  auto issue_x = [&](Slot& S, int64_t d, int h, bool tail) {
    const int64_t kb = 2 * (tail ? d : base + 2 * d) + (tail ? 0 : h);
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        S.x[t][2 * h + j] = *reinterpret_cast<const u32x4*>(xt[t] + (2 * kb + j) * 512 + lane * 8);
  };
  auto issue = [&](Slot& S, int64_t d, bool tail) {
    issue_codes(S, d, tail);
    issue_x(S, d, 0, tail);
    issue_x(S, d, 1, tail);
  };
  f32x4 acc[G][T];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[g][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // One step as 2 G chains (block h, group g): table lookups, 2 T MFMAs, scaling
  // by the block constant, in a pipeline: the lookups of chain c + 1 go out,
  // then chain c - 1 is scaled, then the MFMAs of chain c start, so that
  // neither the LDS nor the MFMA latency is waited for on its own.  The loads
  // of step d + kAhead (if `refill`) go out as soon as their registers are free.
  auto compute = [&](Slot& S, int64_t d, bool tail, bool refill) {
    const int64_t kb = 2 * (tail ? d : base + 2 * d);
    constexpr int NC = 2 * G;
    uint32_t cw[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      u32x4 c;
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = nibbles<CT>(S.c[g], j);
      // (copies: the swap overwrites both operands)
#pragma unroll
      for (int j = 0; j < 2; ++j) c[j] = __builtin_amdgcn_mov_dpp(c[j], 0xE4, 0xf, 0xf, false);
      const auto s02 = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
      const auto s13 = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
      cw[g][0] = s02[0];
      cw[g][1] = s13[0];
      cw[g][2] = s02[1];
      cw[g][3] = s13[1];
    }
    __builtin_amdgcn_sched_barrier(0);
    if (refill) issue_codes(S, d + kAhead, false);
    u32x4 wl[2][2];
    float ch[2];
    f32x4 s[T];
    auto lookup = [&](int c) {
      const int h = c / G, g = c % G;
      wl[c & 1][0] = levels8(cw[g][2 * h], lut + i16);
      wl[c & 1][1] = levels8(cw[g][2 * h + 1], lut + i16);
      ch[c & 1] = (h && tail) ? 0.0f : crow_t[g][kb + h];
    };
    lookup(0);
#pragma unroll
    for (int c = 0; c <= NC; ++c) {
      const float prev = ch[(c + 1) & 1];  // of chain c - 1, before lookup(c + 1) takes its place
      if (c + 1 < NC) lookup(c + 1);
      __builtin_amdgcn_sched_barrier(0);
      if (c > 0) {
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[(c - 1) % G][t][v] += prev * s[t][v];
      }
      if (c < NC) {
        const int h = c / G;
        const bf16x8 w0 = as_bf16x8(wl[c & 1][0]), w1 = as_bf16x8(wl[c & 1][1]);
#pragma unroll
        for (int t = 0; t < T; ++t)
          s[t] = mfma16(as_bf16x8(S.x[t][2 * h]), w0, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int t = 0; t < T; ++t) s[t] = mfma16(as_bf16x8(S.x[t][2 * h + 1]), w1, s[t]);
        __builtin_amdgcn_sched_barrier(0);
        if (refill && c % G == G - 1) issue_x(S, d + kAhead, h, false);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  Slot sl[kAhead];
  if (d1 > 0) issue(sl[0], 0, false);

  // Prologue: the tokens' adapters and U (rows without an adapter read what is
  // there, and drop it), the block constants, the byte table.  Every load goes
  // out before the first use.
  if (tid < 16 * T) {
    const int a = tid < mt ? p.index[m0 + tid] : -1;
    own[tid] = (unsigned)a < (unsigned)p.adapters ? a : -1;
  }
  const int uquads = mt * ((int)p.ldp / 4);  // U is contiguous over the tokens
  const float* up = p.part + m0 * p.ldp;
  auto sum_u = [&](int e) {
    f32x4 u[kMaxSlices];
#pragma unroll
    for (int s = 0; s < kMaxSlices; ++s)
      u[s] = *reinterpret_cast<const f32x4*>(up + (s < p.slices ? s : 0) * p.M * p.ldp + 4 * e);
    f32x4 sum = u[0];
#pragma unroll
    for (int s = 1; s < kMaxSlices; ++s)
      if (s < p.slices) sum += u[s];
    *reinterpret_cast<f32x4*>(ush + 4 * e) = sum;
  };
  const int kbl = (int)kblocks;
  if (p.bshift == 0) {
    // The constants of the workgroup's rows are contiguous: 16 per load, which
    // share a step (256 constants); bytes past the weight's read 0.
    const int64_t qtot = N * kblocks;
    const int nchunk = G * kbl, glast = (int)((qtot + 255) >> 8) - 1;
    const __amdgpu_buffer_rsrc_t qrs = bytes_rsrc(p.q8, qtot);
    for (int c0 = 0; c0 < nchunk; c0 += NT) {
      const int c = c0 + tid;
      const int o = (int)(n0 * kblocks) + 16 * c;
      const u32x4 qv = __builtin_amdgcn_raw_buffer_load_b128(qrs, c < nchunk ? o : INT32_MIN, 0, 0);
      const float st = p.step[c < nchunk && o >> 8 < glast ? o >> 8 : glast] * (1.0f / level_factor<CT>());
      if (c0 == 0 && tid < uquads) sum_u(tid);
      if (c < nchunk) {
        int row = 16 * c / kbl, kb = 16 * c - row * kbl;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          chat[row * (int)kbs + kb] = (float)((qv[i >> 2] >> (8 * (i & 3))) & 0xffu) * st;
          if (++kb == kbl) kb = 0, ++row;
        }
      }
    }
  } else {
    const int64_t cblocks = kblocks >> p.bshift;
    for (int e = tid; e < 16 * G * kbl; e += NT) {
      const int row = e / kbl, kb = e - row * kbl;
      const int64_t n = n0 + row < N ? n0 + row : N - 1;
      const int64_t ci = n * cblocks + (kb >> p.bshift);
      chat[row * kbs + kb] = (float)p.q8[ci] * (p.step[ci >> 8] * (1.0f / level_factor<CT>()));
    }
    if (tid < uquads) sum_u(tid);
  }
  for (int e = tid + NT; e < uquads; e += NT) sum_u(e);
  {
    static_assert(kLutWords == 8 * NT, "table split");
    const float lo = level_of<CT>(p.ut, (tid >> 4) & 15) * level_factor<CT>();
    const int hi0 = __builtin_amdgcn_readfirstlane(tid >> 8);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      lut[tid + NT * i] = pack_bf16x2(lo, level_of<CT>(p.ut, hi0 + 2 * i) * level_factor<CT>());
  }
  __syncthreads();

  int64_t d = 0;
  if constexpr (kAhead == 2) {
    if (d1 > 1) issue(sl[1], 1, false);
    for (; d + 4 <= d1; d += 2) {
      compute(sl[0], d, false, true);
      compute(sl[1], d + 1, false, true);
    }
    if (d + 3 <= d1) {
      compute(sl[0], d, false, true);
      compute(sl[1], d + 1, false, false);
      compute(sl[0], d + 2, false, false);
    } else {
      if (d < d1) compute(sl[0], d, false, false);
      if (d + 1 < d1) compute(sl[1], d + 1, false, false);
    }
  } else {
    for (; d + 1 < d1; ++d) compute(sl[0], d, false, true);
    if (d < d1) compute(sl[0], d, false, false);
  }
  if (odd_tail) {
    issue(sl[0], D, true);
    compute(sl[0], D, true, false);
  }
  // Outputs o = tid + NT k of [g][t][v][lane].  The first adapter columns are
  // on their way while the waves' sums go through LDS.
  constexpr int KO = G * T * 256 / NT;
  constexpr int JB = 16;
  int mk[KO];
  int64_t nk[KO];
  const uint16_t* bp[KO];
  bool store[KO], has[KO];
#pragma unroll
  for (int k = 0; k < KO; ++k) {
    const int o = tid + NT * k;
    const int l = o & 63, v = (o >> 6) & 3, t = (o >> 8) % T, g = (o >> 8) / T;
    mk[k] = 16 * t + 4 * (l >> 4) + v;
    nk[k] = n0 + 16 * g + (l & 15);
    store[k] = mk[k] < mt && nk[k] < N;
    const int a = store[k] ? own[mk[k]] : -1;
    has[k] = a >= 0;
    // (others read the first rows and drop what comes of it)
    bp[k] = p.B + (has[k] ? ((int64_t)a * N + nk[k]) * p.r : 0);
    if (!store[k]) mk[k] = 0;
  }
  u32x4 bq[KO][JB / 8];
  auto load_b = [&](int j0) {
#pragma unroll
    for (int k = 0; k < KO; ++k)
#pragma unroll
      for (int i = 0; i < JB / 8; ++i)
        bq[k][i] = load_row8(bp[k], j0 + 8 * i, p.r);
  };
  const bool bvec = p.r >= 8;
  if (bvec) load_b(0);
  __syncthreads();  // the constants become the waves' sums
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        red[(((wave * G + g) * T + t) * 4 + v) * 64 + lane] = acc[g][t][v];
  __syncthreads();
  float y[KO], lora[KO];
#pragma unroll
  for (int k = 0; k < KO; ++k) {
    y[k] = lora[k] = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) y[k] += red[w * (G * T * 256) + tid + NT * k];
  }
  if (bvec) {
    for (int j0 = 0; j0 < p.r; j0 += JB) {
      if (j0) load_b(j0);
      __builtin_amdgcn_sched_barrier(0);  // every load of the batch before the first use
#pragma unroll
      for (int i = 0; i < JB / 8; ++i) {
        if (j0 + 8 * i >= p.r) break;  // uniform
#pragma unroll
        for (int k = 0; k < KO; ++k) {
          const float* u = ush + mk[k] * p.ldp + j0 + 8 * i;
          const f32x4 u0 = *reinterpret_cast<const f32x4*>(u);
          const f32x4 u1 = *reinterpret_cast<const f32x4*>(u + 4);
          const u32x4 b = shift_row8(bq[k][i], j0 + 8 * i, p.r);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t w = b[e >> 1];
            lora[k] += (e < 4 ? u0[e] : u1[e - 4]) * ((e & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w));
          }
        }
      }
    }
  } else {
    for (int j = 0; j < p.r; ++j)
#pragma unroll
      for (int k = 0; k < KO; ++k) lora[k] += ush[mk[k] * p.ldp + j] * bf16_to_f32(bp[k][j]);
  }
#pragma unroll
  for (int k = 0; k < KO; ++k)
    if (store[k])
      p.Y[(m0 + mk[k]) * N + nk[k]] = f32_to_bf16(has[k] ? y[k] + lora[k] : y[k]);
}

template <int G, int T>
hipError_t launch(const RowsArgs& a, int code, hipStream_t stream) {
  const size_t lds = 4 * (size_t)rows_lds_words(G, T, a.ldp, a.K / 64);
  const dim3 grid((unsigned)((a.N + 16 * G - 1) / (16 * G)), (unsigned)((a.M + 16 * T - 1) / (16 * T)));
  return with_any_code(code, [&](auto ct) {
    const void* fn = reinterpret_cast<const void*>(&k_qrows<G, T, decltype(ct)>);
    const hipError_t e =
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (e != hipSuccess) return e;
    k_qrows<G, T, decltype(ct)><<<grid, dim3(NT), lds, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

namespace {

struct Shape {
  int G, T;
  double us;  // estimate; 0 if no tile fits
};

int64_t over(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile and its time, from the shapes alone: the rounds of workgroups over
// 256 compute units times a workgroup's time.  (The whole chip's, to which the
// constants are fitted: the workspace's size follows from this choice and is the
// same wherever it is asked for.)  Measured with 24 adapters of
// rank 32, us a call, G = 2 / G = 4: 64 rows over 8192 x 8192 37 / 47, 128 rows
// 58 / 48, 256 rows 100 / 79; 64 over 11008 x 4096 40 / 34; 64 over 28672 x 8192
// 106 / 83.  Up to 32 rows: 17 over 11008 x 4096 29.7 / 24.6, over 28672 x 8192
// 75.7 / 61.6, over 8192 x 8192, where G = 4 leaves half the chip idle, 28 / 35.
Shape shape_of(int64_t M, int64_t N, int64_t K, int32_t r) {
  const int T = M <= 32 ? 2 : 4;
  const auto fits = [&](int G) {
    return 4 * rows_lds_words(G, T, (r + 7) / 8 * 8, K / 64) <= 160 * 1024;
  };
  const auto rounds = [&](int G) { return (double)over(over(N, 16 * G) * over(M, 16 * T), 256); };
  if (!fits(2)) return {2, T, 0.0};
  const double two = rounds(2) * (6.0 + (T == 2 ? 0.0015 : 0.0021) * K);
  const double four = rounds(4) * (T == 2 ? 6.0 + 0.0023 * K : 5.0 + 0.0036 * K);
  return fits(4) && four < two ? Shape{4, T, four} : Shape{2, T, two};
}

}  // namespace

// Whether this kernel is the faster one, against an estimate of the tiles (128 x
// 128 while the 256 x 256 ones would leave half the chip idle): a round of
// workgroups, the weight's stream, the rows' order.  Measured as above, here /
// tiles: 256 rows over 8192 x 8192 79 / 151, 512 rows 143 / 144, 1024 rows 268 /
// 217; 384 over 11008 x 4096 121 / 125, 512 rows 144 / 126; 128 over 28672 x 8192
// 145 / 171, 256 rows 242 / 226; 512 over 4096 x 4096 60 / 88.
bool qrows_takes(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (M > kQRowsMaxM) return false;
  const Shape here = shape_of(M, N, K, r);
  const int64_t big = over(M, 256) * over(N, 256), small = over(M, 128) * over(N, 128);
  const double unit = K / 64 * 0.9 + 5.0;
  const double tiles = 2 * big <= 256 ? unit * (0.55 + 0.45 * (double)over(small, 256))
                                      : 1.9 * unit * (double)over(big, 256);
  return here.us > 0.0 && here.us < tiles + (double)N * K * 1e-7 + 8.0;
}

hipError_t launch_qrows(const Nf4View& w, const uint16_t* xfrag, int64_t M, const float* part,
                        int slices, const uint16_t* B, int32_t r, int adapters,
                        const int32_t* index, uint16_t* Y, hipStream_t stream) {
  const RowsArgs a{w.codes, w.q8, w.step, xfrag, M, w.N, w.K, part, slices, (r + 7) / 8 * 8, B, r,
                   index, adapters, Y, w.bshift, w.ut};
  const Shape s = shape_of(M, w.N, w.K, r);
  if (s.T == 4) return s.G == 4 ? launch<4, 4>(a, w.code, stream) : launch<2, 4>(a, w.code, stream);
  return s.G == 4 ? launch<4, 2>(a, w.code, stream) : launch<2, 2>(a, w.code, stream);
}

}  // namespace qn
