// What the attention kernels share: which sequence, head and tile a
// workgroup works on, K/V (or Q/dO) tiles in LDS, and the MFMA fragments.
//
// Matrix products.  Every product has one operand in registers for the whole
// kernel or fresh from the previous product (the B operand: column index =
// lane % 32), and one that comes from a tile in LDS (the A operand).  A
// wave owns 32 columns: query rows in the forward and the dQ kernel, keys
// in the dK/dV kernel.  The score tile is computed with the tile's rows as
// the MFMA's row index, so that the probabilities come out as
// "column = lane % 32, rows in registers", which is what the following
// product takes as its B operand; nothing goes through LDS in between.  An
// MFMA 32x32 result holds row 8 a + 4 h + c in element 4 a + c of half h =
// lane / 32, while the B operand of the next one wants rows 8 h + e of each
// 16-row slab in elements e = 0..7; reading tile row swap23(i) as A row i
// (bits 2 and 3 exchanged) makes the two agree.  The same exchange on the
// output columns leaves 8 consecutive output elements in a lane, so
// results are stored 16 bytes at a time.
//
// The products take the head dimension rounded up to DP = 64, 96 or 128;
// tiles in LDS are [64][64 or 128] bf16 (dimensions past D hold copies of
// valid ones, meet zeros in the register operand, and are not stored).  The
// 16-byte chunks of a row are stored in the order chunk ^ mask(row), chosen
// so that both ways of reading are free of bank conflicts: 16 rows of one
// chunk (ds_read_b128, measured 208 bytes per clock and CU) and 4 + 4 rows of
// 4 chunks (the transposing ds_read_b64_tr_b16: 188; 62 in plain order).
#pragma once

#include "kernels.hpp"

namespace qn {
namespace attn {

constexpr int kTile = 64;    // rows of a tile in LDS
constexpr int kWaves = 4;    // waves per workgroup
constexpr int kCols = 32;    // columns per wave
constexpr int kBlock = kWaves * kCols;  // columns per workgroup

constexpr unsigned kResident = 512;     // workgroups that run at once: two on each of 256 CUs

// Workgroups of a launch; a pass of more takes further launches.  HIP takes
// fewer than 2^32 threads along a dimension of the grid, 2^24 workgroups of 256
// (2^24 + 48 in one launch: most were never run, and no error came back); at
// a quarter of that a launch lasts far longer than the next one's start takes.
constexpr int64_t kMaxGrid = 1 << 22;

constexpr int kSearch = 128;            // packed sequences from which on they are found by a search

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

// ---- which tile ----

// One workgroup's work: `tile` of the columns of one sequence.
struct Work {
  int head;
  int64_t batch;           // dense: batch index (packed: 0)
  int64_t q0, k0;          // first query and key row of the sequence (packed; dense: 0)
  int lq, lk;              // lengths
  int tile, ntiles;        // tile of kBlock columns, and how many the sequence has
  int split;               // which share of the walk over the other side
  bool valid;
};

// The order of the work: workgroup id -> (head of the batch, slot).
// Workgroups go to the 8 XCDs round-robin by id, and each XCD has its own
// L2: an XCD gets a contiguous range of heads, so that those that share K
// and V share an L2.  Within its range the slots are the outer index: the
// slots that take longest come first for all heads, and the last workgroups
// to start are short ones.
struct Place {
  unsigned head, slot;
};
__device__ __forceinline__ Place place_of(unsigned id, unsigned heads) {
  Place p;
  if (heads % 8 == 0) {
    const unsigned per = heads >> 3, j = id >> 3;
    p.slot = j / per;
    p.head = (id & 7) * per + (j - p.slot * per);
  } else {
    p.slot = id / heads;
    p.head = id - p.slot * heads;
  }
  return p;
}

__device__ __forceinline__ int clamp_row(int64_t v, int64_t lo, int64_t hi) {
  return (int)(v < lo ? lo : v > hi ? hi : v);
}

// Dense: every sequence has the same tiles, ntiles = ceil(cols / kBlock).
// Packed: `slots` tiles per head, at least as many as all sequences have.
// They are taken sequence by sequence, so that tiles which share K and V run
// at the same time; up to 63 sequences, those with the most tiles first (by a
// ballot for each count), so that no long walk starts last; with more, in
// their order: up to kSearch - 1 by a prefix sum over the wave, 64 lengths at a
// time, which puts the slots without work last.  From kSearch on the slots of
// sequence s start at cu[s] / kBlock + s: one more than the whole blocks
// between two offsets is at least the tiles of the rows between them, so a
// search finds the sequence in ceil(log64(sequences)) steps, and the slots past
// a sequence's tiles have no work.  (Forward + backward, 100 sequences: 23 + 83
// us by sums, 23 + 87 by search; 128: 140 + 362 and 138 + 360; 500: 287 + 543
// and 209 + 453; 2^16 of one token: 174 and 3 ms in all.)
// After the last sequence, the rows that belong to none form one more, with
// nothing on the other side, so that outputs are zero there.  Offsets are
// clamped to the tensors' rows, so that wrong ones give wrong results but no
// access out of range.
// kKeys: the columns are keys (the dK/dV kernel), else queries.
template <bool kKeys>
__device__ __forceinline__ Work find_work(const AttnArgs& p, int slots, unsigned heads) {
  Work w;
  // heads of the whole batch, times splits, is below 2^32 (all workgroups are)
  const unsigned all = heads * (p.cu_q ? 1u : (unsigned)p.nseq) * (unsigned)p.splits;
  const Place at = place_of(p.first + blockIdx.x, all);
  const unsigned head = at.head / (unsigned)p.splits;
  w.split = (int)(at.head - head * (unsigned)p.splits);
  const unsigned batch = head / heads;
  w.head = (int)(head - batch * heads);
  const int slot = (int)at.slot;
  if (!p.cu_q) {
    w.batch = batch;
    w.q0 = w.k0 = 0;
    w.lq = (int)p.Sq;
    w.lk = (int)p.Sk;
    w.tile = slot;
    w.ntiles = slots;
    w.valid = true;
    return w;
  }
  w.batch = 0;
  w.valid = false;
  const int lane = threadIdx.x & 63;
  const int32_t* cu = kKeys ? p.cu_k : p.cu_q;
  const int64_t rows = kKeys ? p.Sk : p.Sq;
  int found = -1, tile = 0, n = 0;  // sequence, and in its lane: tiles
  auto tiles_of = [&](int s) {
    if (s > p.nseq) return 0;
    const int64_t a = clamp_row(cu[s], 0, rows);
    const int64_t b = s < p.nseq ? clamp_row(cu[s + 1], a, rows) : rows;
    return (int)((b - a + kBlock - 1) / kBlock);
  };
  if (p.nseq < 64) {
    n = tiles_of(lane);
    // the largest count below `than` (0: none)
    auto largest = [&](int than) {
      int v = n < than ? n : 0;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        const int other = __shfl_xor(v, o, 64);
        v = v > other ? v : other;
      }
      return __builtin_amdgcn_readfirstlane(v);
    };
    int left = slot;
    for (int len = largest(0x7fffffff); len > 0; --len) {
      uint64_t has = __ballot(n == len);
      if (!has) {  // a gap: on to the next count that there is
        len = largest(len);
        if (len == 0) break;
        has = __ballot(n == len);
      }
      const int count = __popcll(has) * len;
      if (left < count) {
        for (int i = left / len; i > 0; --i) has &= has - 1;
        found = __ffsll((unsigned long long)has) - 1;
        w.ntiles = len;
        tile = left % len;
        break;
      }
      left -= count;
    }
  } else if (p.nseq < kSearch) {
    int base = 0;
    for (int s0 = 0; s0 <= p.nseq; s0 += 64) {
      n = tiles_of(s0 + lane);
      int sum = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(sum, o, 64);
        if (lane >= o) sum += up;
      }
      const uint64_t past = __ballot(base + sum > slot);
      if (past) {
        const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)past) - 1);
        found = s0 + l;
        w.ntiles = __builtin_amdgcn_readlane(n, l);
        tile = slot - base - __builtin_amdgcn_readlane(sum - n, l);
        break;
      }
      base += __builtin_amdgcn_readlane(sum, 63);
    }
  } else {
    // The last sequence whose first slot is not past this one, 64 candidates at
    // a time.
    auto first_of = [&](int s) { return clamp_row(cu[s], 0, rows) / kBlock + s; };
    int s0 = 0;
    for (int left = p.nseq + 1; left > 1;) {
      const int step = (left + 63) >> 6;
      const uint64_t in = __ballot(lane * step < left && first_of(s0 + lane * step) <= slot);
      const int at = in ? (63 - __builtin_clzll(in)) * step : 0;
      s0 += at;
      left = left - at < step ? left - at : step;
    }
    n = tiles_of(s0);
    tile = slot - first_of(s0);
    if (tile >= 0 && tile < n) {
      found = s0;
      w.ntiles = n;
    }
  }
  if (found < 0) return w;
  const bool none = found == p.nseq;
  w.tile = tile;
  w.q0 = clamp_row(p.cu_q[found], 0, p.Sq);
  w.k0 = clamp_row(p.cu_k[found], 0, p.Sk);
  const int qe = none ? (kKeys ? (int)w.q0 : (int)p.Sq) : clamp_row(p.cu_q[found + 1], w.q0, p.Sq);
  const int ke = none ? (kKeys ? (int)p.Sk : (int)w.k0) : clamp_row(p.cu_k[found + 1], w.k0, p.Sk);
  w.lq = qe - (int)w.q0;
  w.lk = ke - (int)w.k0;
  w.valid = true;
  return w;
}

// Calls f(DP) for a head dimension.
template <int V>
struct Dim {
  static constexpr int value = V;
};
template <class F>
hipError_t with_dim(int D, F&& f) {
  return D <= 64 ? f(Dim<64>{}) : D <= 96 ? f(Dim<96>{}) : f(Dim<128>{});
}

// Tiles per head to launch for `cols` columns.
inline int64_t tile_slots(const AttnArgs& a, int64_t cols) {
  const int64_t n = (cols + kBlock - 1) / kBlock;
  return a.cu_q ? cols / kBlock + a.nseq + 1 : (n > 0 ? n : 1);
}

// Launches a pass of `groups` workgroups.
template <class K>
hipError_t launch_groups(K kern, AttnArgs a, int64_t groups, int64_t slots, hipStream_t stream) {
  a.groups = (uint32_t)groups;
  for (int64_t first = 0; first < groups; first += kMaxGrid) {
    a.first = (uint32_t)first;
    const int64_t n = groups - first < kMaxGrid ? groups - first : kMaxGrid;
    kern<<<(unsigned)n, kWaves * 64, 0, stream>>>(a, (int)slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- tiles in LDS ----

// v, in a form the compiler cannot compute from ahead: what is derived from
// it would otherwise be kept in registers across the loop over the tiles.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The lane, computed anew: two instructions instead of a register that lives
// through the loop.
__device__ __forceinline__ int lane_now() {
  return opaque(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)));
}

// A wave-uniform float in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}

// DP = 64, 96 or 128: the head dimension as the products see it.
template <int DP>
struct Geo {
  static constexpr int kPitch = DP <= 64 ? 64 : 128;  // elements of a row in LDS
  static constexpr int kChunks = kPitch / 8;       // 16-byte chunks per row
  static constexpr int kElems = kTile * kPitch;    // elements of a tile
  static constexpr int kSteps = DP / 16;           // 16-deep contraction steps over the dimension
  static constexpr int kDT = DP / 32;              // 32-wide tiles of the dimension
  // 16-byte loads per thread that fill a tile
  static constexpr int kLoads = kTile * kChunks / (kWaves * 64);
};

// Chunk mask of a row (see above).
template <int DP>
__device__ __forceinline__ int chunk_mask(int row) {
  if constexpr (Geo<DP>::kPitch == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
  else return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
}

// This wave's loads of a tile: load i fills 1024 consecutive bytes of LDS
// (R = 64 / kChunks rows) at row (i kWaves + wave) R, lane l's 16 bytes at 16 l,
// so the lane fetches the chunk that the mask puts there: the same one in every load,
// since the loads' rows agree in the bits that the mask looks at.  Rows past
// the last one read the last row again, chunks past D the row's first.
struct TileLoader {
  int row, col;  // row of load 0; byte offset within the row
};

template <int DP>
__device__ __forceinline__ TileLoader tile_loader(int D, int wave, int lane) {
  constexpr int C = Geo<DP>::kChunks, R = 64 / C;
  static_assert((kWaves * R) % 16 == 0, "the mask looks at four bits of the row");
  TileLoader t;
  t.row = wave * R + lane / C;
  const int c = (lane % C) ^ chunk_mask<DP>(t.row);
  t.col = c * 8 < D ? c * 16 : 0;
  return t;
}

// Issues the loads of 64 rows at `base` (row stride st elements), of which
// `left` (at least 1) exist, into the tile at `lds`.
template <int DP>
__device__ __forceinline__ void load_tile(uint16_t* lds, const TileLoader& t, const uint16_t* base,
                                          int64_t st, int left, int wave) {
  constexpr int R = kWaves * 64 / Geo<DP>::kChunks;  // rows from one load to the next
  const int st2 = (int)(st * 2);
  // 64 rows of at most 2^22 elements: below 2^31 bytes
  const __amdgpu_buffer_rsrc_t rsrc = bytes_rsrc(base, 0x7fffffff);
  if (left >= kTile) {
    const int voff = t.row * st2 + t.col;
#pragma unroll
    for (int i = 0; i < Geo<DP>::kLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(lds + (i * kWaves + wave) * 512), 16,
          voff, i * R * st2, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < Geo<DP>::kLoads; ++i) {
      int row = opaque(t.row) + i * R;
      if (row >= left) row = left - 1;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(lds + (i * kWaves + wave) * 512), 16,
          row * st2 + t.col, 0, 0, 0);
    }
  }
}

// Nothing is scheduled across this point.  The products read their LDS
// operands a fixed number of steps ahead; left to itself the compiler moves
// all reads of a tile to its front and runs out of registers.
__device__ __forceinline__ void step_fence() { __builtin_amdgcn_sched_barrier(0); }

// This wave's tile loads have landed, and every wave is here.
__device__ __forceinline__ void tiles_ready() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---- fragments ----

__device__ __forceinline__ int swap23(int r) {
  return (r & ~12) | ((r & 4) << 1) | ((r & 8) >> 1);
}

// A lane's byte offset of its fragments within a tile.  The dimension steps
// only change bits of the chunk index that nothing else adds to, so they are
// exclusive-ored into one base per kind of read.
struct FragOff {
  int row;  // rows as A rows
  int tr;   // transposed
};

// Transposed reads: A row i of the fragment is dimension swap23(i) of a
// 32-wide slab, its 16 contraction entries are tile rows.  Within each group
// g of 16 lanes, lane j reads 4 consecutive dimensions of row
// 8 (g / 2) + j / 4 (+ 4 in the second read) and receives 4 consecutive rows
// of the dimension that A row 16 (g % 2) + j stands for.
template <int DP>
__device__ __forceinline__ FragOff frag_off(int lane) {
  constexpr int P = Geo<DP>::kPitch;
  FragOff f;
  const int r = swap23(lane & 31);
  f.row = r * P * 2 + (((lane >> 5) ^ chunk_mask<DP>(r)) << 4);
  const int g = lane >> 4, j = lane & 15;
  const int x = 4 * (g & 1) + (j & 3);                       // which 4 A rows
  const int x4 = (x & 4) | ((x & 1) << 1) | ((x >> 1) & 1);  // the 4 dimensions they stand for
  const int rt = 8 * (g >> 1) + (j >> 2);
  f.tr = rt * P * 2 + (((x4 >> 1) ^ chunk_mask<DP>(rt)) << 4) + 8 * (x4 & 1);
  return f;
}

// Tile rows 32 rt + swap23(lane % 32), dimensions 16 s + 8 (lane / 32) + 0..7,
// from the offset `row`.
template <int DP>
__device__ __forceinline__ bf16x8 read_rows(const uint16_t* tile, int row, int s, int rt) {
  return *reinterpret_cast<const bf16x8*>(reinterpret_cast<const char*>(tile) + (row ^ (s << 5)) +
                                          rt * 64 * Geo<DP>::kPitch);
}

// Tile rows 16 slab + 8 (lane / 32) + 0..7 of dimension 32 d + swap23(lane % 32),
// from the offset `tr`.
template <int DP>
__device__ __forceinline__ bf16x8 read_tr(const uint16_t* tile, int tr, int d, int slab) {
  typedef short v4i16 __attribute__((ext_vector_type(4)));
  typedef short v8i16 __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
  const char* t = reinterpret_cast<const char*>(tile) + slab * 32 * Geo<DP>::kPitch;
  const int o = tr ^ (d << 6);
  // the row 4 further on has the lowest bit of its chunk mask flipped
  const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(t + o));
  const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_v4i16*)(t + (o ^ 16) + 8 * Geo<DP>::kPitch));
  const v8i16 v = v8i16{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// Tile rows 32 rt .. times xb; operands are read two steps before their use.
template <int DP>
__device__ __forceinline__ f32x16 rows_times(const uint16_t* tile,
                                             const bf16x8 (&xb)[Geo<DP>::kSteps], const FragOff& f,
                                             int rt) {
  constexpr int N = Geo<DP>::kSteps, kAhead = 2;
  const int row = opaque(f.row);
  f32x16 acc = f32x16{};
  bf16x8 x[N];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = read_rows<DP>(tile, row, i, rt);
  step_fence();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + kAhead < N) x[i + kAhead] = read_rows<DP>(tile, row, i + kAhead, rt);
    acc = mfma32(x[i], xb[i], acc);
    step_fence();
  }
  return acc;
}

// The register operand: row `r` (per lane) of a matrix, dimensions
// 16 s + 8 (lane / 32) + 0..7 in element s, zeros past D.
template <int DP>
__device__ __forceinline__ void load_cols(bf16x8 (&f)[Geo<DP>::kSteps], const uint16_t* row, int D,
                                          int lane) {
#pragma unroll
  for (int s = 0; s < Geo<DP>::kSteps; ++s) {
    const int d = 16 * s + 8 * (lane >> 5);
    const u32x4 v = *reinterpret_cast<const u32x4*>(row + (d < D ? d : 0));
    const uint32_t keep = d < D ? 0xffffffffu : 0u;
    f[s] = as_bf16x8(u32x4{v[0] & keep, v[1] & keep, v[2] & keep, v[3] & keep});
  }
}

// Stores a [dimension][column] accumulator: this lane's column is the row
// `out` of the output, times `mul`.
template <int DP>
__device__ __forceinline__ void store_cols(uint16_t* out, const f32x16 (&acc)[Geo<DP>::kDT],
                                           float mul, int D, int lane) {
#pragma unroll
  for (int t = 0; t < Geo<DP>::kDT; ++t)
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int d = 32 * t + 16 * a + 8 * (lane >> 5);
      if (d < D) {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = pack_bf16x2(acc[t][8 * a + 2 * e] * mul, acc[t][8 * a + 2 * e + 1] * mul);
        *reinterpret_cast<u32x4*>(out + d) = v;
      }
    }
}

// The same in fp32, for a partial result.
template <int DP>
__device__ __forceinline__ void store_cols(float* out, const f32x16 (&acc)[Geo<DP>::kDT],
                                           float mul, int D, int lane) {
#pragma unroll
  for (int t = 0; t < Geo<DP>::kDT; ++t)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int d = 32 * t + 16 * (a >> 1) + 8 * (lane >> 5) + 4 * (a & 1);
      if (d < D)
        *reinterpret_cast<f32x4*>(out + d) =
            f32x4{acc[t][4 * a] * mul, acc[t][4 * a + 1] * mul, acc[t][4 * a + 2] * mul,
                  acc[t][4 * a + 3] * mul};
    }
}

// Elements 8 s .. 8 s + 7 of a score accumulator as the B operand of a
// 16-deep product.
__device__ __forceinline__ bf16x8 pack8(const f32x16& x, int s) {
  u32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(x[8 * s + 2 * e], x[8 * s + 2 * e + 1]);
  return as_bf16x8(v);
}

// Tile row of element v of a score accumulator (rows 32 rt ..) in this half.
__device__ __forceinline__ int elem_row(int v, int half) {
  return 16 * (v >> 3) + 8 * half + (v & 7);
}

// The other half's value (lane ^ 32).
__device__ __forceinline__ float other_half(float x) {
  return __shfl_xor(x, 32, 64);
}

// One tile of queries in the forward and the dQ kernel.
struct Queries {
  int off;                 // causal: query i sees keys 0 .. i + off
  int first, row, rowc;    // this wave's first query, this lane's, and that or the last one
  int seen_first, seen_last, mine;  // last key seen by the wave's first, by its last, by this lane's
  int t0, t1;              // tiles of keys to walk over (of this split)
  const uint16_t* k;
  const uint16_t* v;
};

__device__ __forceinline__ Queries query_tile(const AttnArgs& p, const Work& w, int wave,
                                              int lane) {
  Queries t;
  // causal: the tiles with the most keys first
  const int tile = p.causal ? w.ntiles - 1 - w.tile : w.tile;
  const int col0 = tile * kBlock;
  t.off = w.lk - w.lq;
  t.first = col0 + wave * kCols;
  t.row = t.first + (lane & 31);
  t.rowc = t.row < w.lq ? t.row : w.lq - 1;
  int keys = w.lk;
  t.seen_first = t.seen_last = t.mine = w.lk - 1;
  if (p.causal) {
    const int e = (col0 + kBlock < w.lq ? col0 + kBlock : w.lq) + t.off;
    keys = e < keys ? (e > 0 ? e : 0) : keys;
    if (t.first + t.off < t.seen_first) t.seen_first = t.first + t.off;
    if (t.first + kCols - 1 + t.off < t.seen_last) t.seen_last = t.first + kCols - 1 + t.off;
    if (t.rowc + t.off < t.mine) t.mine = t.rowc + t.off;
  }
  const int nt = (keys + kTile - 1) / kTile;
  t.t0 = (int)((int64_t)nt * w.split / p.splits);
  t.t1 = (int)((int64_t)nt * (w.split + 1) / p.splits);
  const int hk = w.head / (p.H / p.Hkv);
  t.k = p.k.p + w.batch * p.k.sb + (w.k0 + (int64_t)t.t0 * kTile) * p.k.st + hk * p.k.sh;
  t.v = p.v.p + w.batch * p.v.sb + (w.k0 + (int64_t)t.t0 * kTile) * p.v.st + hk * p.v.sh;
  return t;
}

// Calls tile(K tile, V tile, mask, last) for the tiles of keys that any of the
// wave's queries sees (mask: not all rows of the tile in some lane; this
// lane's query sees rows 0 .. last).  Two buffers each: a tile's loads run
// during the step before it.  The first tile's loads are issued by
// start_keys, before whatever else the kernel loads.
template <int DP>
struct KeyBuffers {
  uint16_t *k0, *v0, *k1, *v1;
};

template <int DP>
__device__ __forceinline__ void start_keys(const KeyBuffers<DP>& b, const AttnArgs& p,
                                           const Work& w, const Queries& t, const TileLoader& ld,
                                           int wave) {
  if (t.t0 < t.t1) {
    load_tile<DP>(b.k0, ld, t.k, p.k.st, w.lk - t.t0 * kTile, wave);
    load_tile<DP>(b.v0, ld, t.v, p.v.st, w.lk - t.t0 * kTile, wave);
  }
}

template <int DP, class F>
__device__ __forceinline__ void walk_keys(const KeyBuffers<DP>& b, const AttnArgs& p,
                                          const Work& w, Queries& t, const TileLoader& ld,
                                          int wave, F&& tile) {
  auto issue = [&](uint16_t* kt, uint16_t* vt, int j) {
    t.k += kTile * p.k.st;
    t.v += kTile * p.v.st;
    load_tile<DP>(kt, ld, t.k, p.k.st, w.lk - j * kTile, wave);
    load_tile<DP>(vt, ld, t.v, p.v.st, w.lk - j * kTile, wave);
  };
  auto step = [&](const uint16_t* kt, const uint16_t* vt, int j) {
    const int r0 = j * kTile;
    if (t.first >= w.lq || r0 > t.seen_last) return;
    const bool mask = r0 + kTile - 1 > t.seen_first;
    tile(kt, vt, mask, t.mine - r0);
  };
  for (int j = t.t0; j < t.t1; j += 2) {
    tiles_ready();
    if (j + 1 < t.t1) issue(b.k1, b.v1, j + 1);
    step(b.k0, b.v0, j);
    if (j + 1 >= t.t1) break;
    tiles_ready();
    if (j + 2 < t.t1) issue(b.k0, b.v0, j + 2);
    step(b.k1, b.v1, j + 1);
  }
}

}  // namespace attn
}  // namespace qn
