// Internal launch interface between the C ABI (abi.hip) and the kernels.
// Every launcher enqueues on `stream` and returns hipGetLastError().
#pragma once

#include "common.hpp"

namespace qn {

// ---- nf4_quant.hip ----  (code: kId of any code type; ut: the caller's
// codebook for the CodeUser types, else unused and may be null)
// Blocks of 64 << bshift elements (bshift 0, 1, 2: block size 64, 128, 256);
// nblocks counts those blocks.
hipError_t launch_nf4_quantize(const float* W, int64_t nblocks, uint8_t* codes, uint8_t* q8,
                               float* step, int code, int bshift, const UserTable* ut,
                               hipStream_t stream);
hipError_t launch_nf4_dequantize(const uint8_t* codes, const uint8_t* q8, const float* step,
                                 int64_t nelem, uint16_t* out, int code, int bshift,
                                 const UserTable* ut, hipStream_t stream);

// ---- qgemm.hip: MFMA tile kernels with the NF4 dequantization in the prologue ----
struct Nf4View {
  const uint8_t* codes;
  const uint8_t* q8;
  const float* step;
  int64_t N, K;
  int code;     // kId of the code type
  int bshift;   // block size 64 << bshift (K is a multiple of it)
  UserTable ut; // the caller's codebook (CodeUser types only)
};

// Y[M,N] = X[M,K] W^T + bf16(s U)[M,r] B[N,r]^T.  U has row stride ldu (a
// multiple of 8, zero-padded to ceil(r/64)*64 columns).
hipError_t launch_qgemm_fwd(const Nf4View& w, const uint16_t* X, int64_t M, const uint16_t* U,
                            int64_t ldu, const uint16_t* B, int32_t r, float s, uint16_t* Y,
                            hipStream_t stream);

// dX[M,K] = dY[M,N] W + dU[M,r] A[r,K].  dU has row stride lddu (zero-padded).
hipError_t launch_qgemm_bwd(const Nf4View& w, const uint16_t* dY, int64_t M, const uint16_t* dU,
                            int64_t lddu, const uint16_t* A, int32_t r, uint16_t* dX,
                            hipStream_t stream);

// ---- gemv.hip: bandwidth-bound forward for M <= 16 ----
constexpr int kGemvMaxM = 16;
// Whether launch_qgemv takes these sizes (its per-workgroup table of block
// constants must fit in LDS: K up to about 32000 at 16 tokens and rank 256).
bool gemv_fits(int64_t M, int32_t r, int64_t K);
// Workspace of launch_qgemv: fp32 partial sums of U = X A^T.
size_t gemv_workspace_bytes(int64_t M, int32_t r, int64_t K);
// Y = X W^T + s (X A^T) B^T for M <= kGemvMaxM, and bf16 U into U_out when
// it is not null.  Two launches (U partial sums, then the weight stream);
// ev0 / ev1 (nullable) are recorded around the second one.
hipError_t launch_qgemv(const Nf4View& w, const uint16_t* X, int64_t M, const uint16_t* A,
                        const uint16_t* B, int32_t r, float s, uint16_t* Y, uint16_t* U_out,
                        float* upart, hipStream_t stream, hipEvent_t ev0, hipEvent_t ev1);

// Levels in bf16 under an fp32 constant: with every level times this factor,
// and the constants divided by it, the levels fall nearer to bf16 values (NF4:
// rms error 6.3e-4 of the levels' rms instead of 1.06e-3; found by trying
// multiples of 2^-12 from 1 to 2).
template <class CT>
constexpr float level_factor() {
  if constexpr (CT::kUser) return 1.0f;
  else return CT::kId == CodeNF4::kId   ? 1.43701171875f
              : CT::kId == CodeNF3::kId ? 1.781005859375f
              : CT::kId == CodeNF2::kId ? 1.15625f
                                        : 1.0078125f;
}

// Eight columns of an adapter's row (r >= 8 of them, at any address), from
// column j < r on: the load, of the row's last eight columns where it ends
// before, and the shift that moves them into place then, with zeros after them.
// (Column by column, 215 rows of rank 75 over 3008 x 192 took 132 us.)
struct __attribute__((packed, aligned(2))) Row8 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 load_row8(const uint16_t* row, int j, int r) {
  return reinterpret_cast<const Row8*>(row + (j < r - 8 ? j : r - 8))->v;
}
__device__ __forceinline__ u32x4 shift_row8(u32x4 v, int j, int r) {
  const int over = j + 8 > r ? j + 8 - r : 0;
  if (over & 4) v = u32x4{v[2], v[3], 0u, 0u};
  if (over & 2) v = u32x4{v[1], v[2], v[3], 0u};
  if (over & 1)
    v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return v;
}

// ---- rows of many adapters (qgemm_multi.hip, qgemv_multi.hip, qrows.hip, multi.hip) ----
// Row i has the adapter index[i] (device; none outside 0 .. adapters - 1); A
// [adapters, r, K], B [adapters, N, r], scales [adapters] fp32.
// M <= kGemvMaxM (workspace as launch_qgemv's):
hipError_t launch_qgemv_multi(const Nf4View& w, const uint16_t* X, int64_t M, const uint16_t* A,
                              const uint16_t* B, int32_t r, const float* scales, int adapters,
                              const int32_t* index, uint16_t* Y, float* upart, hipStream_t stream);
// Other M: for the tile kernels, the rows in an order that keeps adapters
// together (null: as they are; always null for qrows.hip), ...
constexpr int kMultiWindow = 4096;  // rows that are put in order together
bool multi_order_takes(int64_t K);
hipError_t launch_multi_order(const int32_t* index, int64_t M, int adapters, int32_t* order,
                              hipStream_t stream);
// ... part[s][m][j] = scale times the sum over K slice s of X A_index[j] of the
// m-th row, zeros for r <= j < ceil(r / 8) * 8, nothing for rows without an
// adapter, and, if xfrag is not null, X in the order of qrows.hip's MFMA
// operands (multi_xfrag_bytes), ...
int multi_down_slices(int64_t M, int64_t K);
size_t multi_down_bytes(int64_t M, int64_t K, int32_t r);
size_t multi_xfrag_bytes(int64_t M, int64_t K);
hipError_t launch_multi_down(const uint16_t* X, int64_t M, int64_t K, const uint16_t* A, int32_t r,
                             const float* scales, int adapters, const int32_t* index,
                             const int32_t* order, float* part, uint16_t* xfrag,
                             hipStream_t stream);
// ... which the kernel for batches of rows takes (qrows.hip) ...
constexpr int kQRowsMaxM = 4096;
bool qrows_takes(int64_t M, int64_t N, int64_t K, int32_t r);
hipError_t launch_qrows(const Nf4View& w, const uint16_t* xfrag, int64_t M, const float* part,
                        int slices, const uint16_t* B, int32_t r, int adapters,
                        const int32_t* index, uint16_t* Y, hipStream_t stream);
// ... and the tile kernels.
hipError_t launch_qgemm_multi_fwd(const Nf4View& w, const uint16_t* X, int64_t M,
                                  const float* part, int slices, const uint16_t* B, int32_t r,
                                  int adapters, const int32_t* index, const int32_t* order,
                                  uint16_t* Y, hipStream_t stream);

// ---- lora.hip: small-rank products with in-kernel reduction of contraction slices ----
// Operand element access: A-op (i, c) at a[i*a_si + c*a_sc]; B-op (c, j) at
// b[j*b_sj + c*b_sc]; one stride of each operand must be 1.
struct SkinnyOp {
  const uint16_t* a;
  int64_t a_si, a_sc;
  const uint16_t* b;
  int64_t b_sj, b_sc;
  int64_t I, J, C;
};
// One product: out[i*o_si + j] = bf16(scale * sum_c Aop(i,c) Bop(c,j)) for
// j < J, zero for J <= j < Jw, optionally also out2[i*o2_si + j] for j < J.
// part: fp32 slice partials (size from skinny_partial_bytes; unused when the
// product has one slice).
struct SkinnyJob {
  SkinnyOp op;
  float scale;
  uint16_t* out;
  int64_t o_si, Jw;
  uint16_t* out2;
  int64_t o2_si;
  float* part;
};
int skinny_tiles(int64_t I, int64_t J);
int skinny_splits(int64_t I, int64_t J, int64_t C);
size_t skinny_partial_bytes(int64_t I, int64_t J, int64_t C);
SkinnyJob make_job(const SkinnyOp& op, float scale, uint16_t* out, int64_t o_si, int64_t Jw,
                   uint16_t* out2, int64_t o2_si, float* part);
// Run one or two independent products: one launch for the partial products
// and, if any product has several contraction slices, one finish launch.
hipError_t launch_skinny(const SkinnyJob* jobs, int njobs, hipStream_t stream);

// ---- lq_init.hip: low-rank plus quantized decomposition of a weight ----
struct LqArgs {
  const float* W;      // [N, K]
  int64_t N, K;
  int code;            // code type id of the Q component
  int r, l;            // rank, subspace width (r < l <= 96, l % 16 == 0)
  const float* omega;  // [K, l] Gaussian test matrix
  int iters, power_iters;
  int start;           // 0: L step first (Q = 0), 1: Q step first (L = 0)
  float s;             // LoRA scale of the adapter outputs
  uint8_t* codes;
  uint8_t* q8;
  float* step;
  uint16_t* A;         // [r, K] bf16
  uint16_t* B;         // [N, r] bf16
  float* L1;           // [N, r]
  float* L2t;          // [K, r]
  void* ws;            // lq_workspace_bytes(N, K, l) bytes, 256-byte aligned
};
size_t lq_workspace_bytes(int64_t N, int64_t K, int32_t l);
hipError_t launch_lq_init(const LqArgs& a, hipStream_t stream);
// R = W - L1 L2t^T (fp32 [N, K]; L1 [N, r], L2t [K, r], r <= 96, K % 64 == 0)
hipError_t launch_lq_residual(const float* W, const float* L1, const float* L2t, int64_t N,
                              int64_t K, int r, float* R, hipStream_t stream);

// ---- norm.hip: layer norm and root-mean-square norm ----
constexpr int kNormBF16 = 0, kNormF32 = 1;  // element types (of clip.hip too)
struct NormArgs {
  const void* x;      // [rows, width]
  int64_t rows, width;
  int x_type;
  const void* w;      // [width]
  const void* b;      // [width] or null
  int w_type;
  float eps;
  bool rms;
  void* y;            // [rows, width], x's type
  float* mean;        // [rows] (not touched if rms)
  float* rstd;        // [rows]
};
struct NormBwdArgs {
  const void* dy;
  const void* x;
  int64_t rows, width;
  int x_type;
  const void* w;
  int w_type;
  bool rms;
  const float* mean;  // unused if rms
  const float* rstd;
  void* dx;           // or null
  void* dw;           // [width], w's type, or null
  void* db;           // or null
  float* part;        // norm_bwd_groups rows of width floats, for dw and for db
};
int64_t norm_max_width(int type);
// Workgroups of the backward pass, i.e. rows of partial parameter sums.
int norm_bwd_groups(int64_t rows, int64_t width, int type);
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream);

// ---- clip.hip: global gradient norm and clipping ----
constexpr int kClipNormTable = 240;   // tensors per launch of the sum of squares
constexpr int kClipScaleTable = 160;  // tensors per launch of the scaling
constexpr int kClipGrid = 1024;       // workgroups (and partial sums) per launch at most
struct ClipArgs {
  int64_t n;
  const void* const* grads;  // host array of device pointers
  const int64_t* sizes;      // host
  const int32_t* types;      // host: kNormBF16 / kNormF32
  void* const* out;          // host array, or null: in place
  bool scale;                // false: the norm only
  float max_norm;
  float* norm;               // device, 1 float
  double* part;              // kClipGrid slots per launch of the sum of squares
};
hipError_t launch_clip(const ClipArgs& a, hipStream_t stream);

// ---- adamw.hip: the AdamW step over many tensors ----
constexpr int kAdamBlock = 256;   // elements of a tensor per block of its 8-bit states
constexpr int kAdamGrid = 2048;   // workgroups per launch at most
struct AdamHyper {
  double lr, beta1, beta2, decay;
  double bc1, bc2;               // 1 - beta^t (host's, unless step_dev)
  double log_beta1, log_beta2;   // for step_dev
  const float* lr_dev;           // device scalars, or null
  const int64_t* step_dev;
  const float* norm;             // the gradients' norm, or null: no clipping
  double max_norm;
  float eps;
};
struct AdamArgs {
  int64_t n;
  void* const* params;           // host arrays of device pointers
  const void* const* grads;      // null: the tensor is left alone
  uint16_t* const* copies;       // bf16 copies of the parameters (entries may be null), or null
  const int64_t* sizes;
  const int32_t* p_types;        // kNormBF16 / kNormF32
  const int32_t* g_types;
  int bits;                      // of the states: 32 (fp32) or 8 (int8 m, uint8 v)
  void* m;                       // every tensor's states from a multiple of kAdamBlock on
  void* v;
  float* ms;                     // scales, one per block (8 bits)
  float* vs;
  AdamHyper hyper;
};
hipError_t launch_adamw(const AdamArgs& a, hipStream_t stream);
hipError_t launch_adamw_values(const void* m, const void* v, const float* ms, const float* vs,
                               int64_t blocks, float* m_out, float* v_out, hipStream_t stream);

// ---- attention_fwd.hip, attention_bwd.hip, attention_join.hip ----
// A [batch, token, head, dim] tensor: element strides (the last one is 1).
struct AttnView {
  uint16_t* p;
  int64_t sb, st, sh;
};
struct AttnArgs {
  AttnView q, k, v, o;         // o: output of the forward, input of the backward pass
  AttnView dout, dq, dk, dv;   // backward
  float* lse;                  // [B, H, Sq] dense, [H, Tq] packed
  float* delta;                // workspace of the backward pass, as lse
  // packed: sequence s has the query rows cu_q[s] .. cu_q[s + 1] - 1 and the
  // key rows cu_k[s] .. cu_k[s + 1] - 1 (device, int32); null if dense
  const int32_t* cu_q;
  const int32_t* cu_k;
  int nseq;                    // sequences (dense: the batch)
  int64_t Sq, Sk;              // rows: per sequence if dense, in all if packed
  int H, Hkv, D;
  float scale;
  bool causal;
  // Workgroups that share one tile's walk over the other side.  With more
  // than one, each leaves an fp32 partial result in `part` (forward: its
  // normalized output, and its log-sum-exp in part_lse), which the join adds.
  int splits;
  uint32_t groups;             // workgroups of the pass
  uint32_t first;              // the first one of this launch
  int64_t all;                 // rows of all heads
  float* part;                 // [splits][all][D]
  float* part_lse;             // [splits][all]
};
enum AttnPass { kAttnFwd, kAttnDq, kAttnDkv };
// How many workgroups share a tile in a pass (from the shapes alone).
int attn_splits(const AttnArgs& a, AttnPass pass);
// fp32 words of workspace: the forward's partial results; the backward
// pass's delta and partial results.
int64_t attn_fwd_workspace(const AttnArgs& a);
int64_t attn_bwd_workspace(const AttnArgs& a);
hipError_t launch_attn_fwd(const AttnArgs& a, float* ws, hipStream_t stream);
hipError_t launch_attn_bwd(const AttnArgs& a, float* ws, hipStream_t stream);
// Adds partial results: the forward's (weighted by their shares of the
// softmax) into o and lse; n tensors' ([n][splits][rows][D]) into out[i]
// times mul[i].
hipError_t launch_attn_join_fwd(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_join_sum(const AttnArgs& a, int n, const AttnView* out, const float* mul,
                                int64_t rows, int heads, hipStream_t stream);

// ---- rope.hip: rotary positions ----
struct RopeArgs {
  AttnView q, k, qo, ko;     // inputs and outputs (k, ko: unused if Hk == 0)
  int64_t tokens, rows;      // tokens in all; per batch entry (packed: all)
  const int32_t* cu;         // packed: sequence offsets, or null
  int nseq;
  const void* pos;           // positions, or null: a row's place in its sequence
  int64_t pos_sb, pos_st;    // element strides over the batch and the rows
  bool pos64;                // int64 positions (else int32)
  const double* freq;        // [rot / 2] radians per position
  int H, Hk, D, rot;
  bool interleaved, inverse;
  float scale;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

// ---- stream.hip: read-only HBM stream (measurement helper) ----
// Reads bytes / 16 16-byte words of src with `grid` workgroups of 256
// lanes; writes one word per workgroup to sink[0 .. grid - 1].
hipError_t launch_stream_read(const void* src, size_t bytes, uint32_t* sink, int grid,
                              hipStream_t stream);

// ---- ilp.hip: configuration errors and the budget program ----
size_t quant_error_workspace_bytes(int64_t N, int64_t K, int bits, int bshift, bool lowrank);
// *sq_err (device) = ||R - W_hat(R)||_F^2, R = W or W - L1 L2t^T (L1 non-null)
hipError_t launch_quant_error(const float* W, int64_t N, int64_t K, int code, int bshift,
                              const float* L1, const float* L2t, int r, double* sq_err, void* ws,
                              hipStream_t stream);
// host: exact minimum-error choice within the budget; false if none fits
bool ilp_plan(int M, int C, const double* err, const int64_t* bytes, int64_t budget,
              int32_t* choice, double* total_err, int64_t* total_bytes);

}  // namespace qn
