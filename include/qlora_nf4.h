/*
 * qlora_nf4.h -- C ABI of the frozen-NF4-base + LoRA linear layer for
 * AMD Instinct MI355X (gfx950).
 *
 * What the layer is (cited by page title and section):
 *  - The frozen base weight is stored in 4-bit NormalFloat (NF4): 16 levels
 *    at normal quantiles, one absmax scaling constant per block of weights,
 *    and the constants themselves quantized to 8 bits under a coarser set of
 *    constants ("QLoRA: fine-tuning a 65B model on one GPU", section
 *    "NormalFloat, double quantization, paged optimizers"; "QLoRA: efficient
 *    finetuning of quantized LLMs", Abstract, items (a) and (b)).
 *  - The base is quantized once up front and dequantized to 16 bits on the
 *    fly for every forward and backward pass; gradients reach only the
 *    low-rank adapters, which stay in 16 bits (blog section "Where the memory
 *    goes"; CoChat Abstract).
 *  - The backward pass re-materializes the low-precision weight from the
 *    quantized module instead of keeping a 16-bit copy ("ModuLoRA: Finetuning
 *    2-Bit LLMs on Consumer GPUs by Integrating with Modular Quantizers",
 *    abstract).
 *
 * Shapes (torch Linear convention, row-major, contiguous):
 *   W [N, K]  frozen weight (fp32 only as quantizer input)
 *   X [M, K]  input, bf16            Y  [M, N] output, bf16
 *   A [r, K]  LoRA down, bf16        B  [N, r] LoRA up, bf16
 *   s         LoRA scale (alpha / r), fp32
 *   Forward:  Y  = X W^T + s (X A^T) B^T
 *   Backward: dU = s dY B;  dX = dY W + dU A;  dA = dU^T X;  dB = s dY^T (X A^T)
 *   where W is the dequantized weight; there is no gradient for W.
 *
 * NF4 storage of W (the "nf4 tensor"), block size B = 64 by default (128
 * and 256 are offered too: the LQ-LoRA abstract's integer program chooses
 * the block size per matrix):
 *   codes [N*K/2] uint8  two 4-bit level indices per byte, element 2j of the
 *                        row-major flattening in the low nibble of byte j
 *   q8    [N*K/B] uint8  8-bit absmax constant of each B-element block
 *   step  [ceil(N*K/B/256)] fp32  per group of 256 consecutive blocks:
 *                        the group's largest absmax divided by 255
 *   Dequantized weight: w = bf16_rne(level[code] * (q8 * step)), both
 *   products rounded to fp32.
 *
 * Code types (the table `level[16]` behind the 4-bit codes; the capability
 * page "Qlora 4 Bit Quantization With Nf4 Fp4 Data Types And Lora Adapters"
 * names both data types, and the blog section "NormalFloat, double
 * quantization, paged optimizers" compares NF4 against a plain 4-bit float):
 *   QLORA_CODE_NF4  the 16 NF4 levels, ascending with the code, zero = code 7
 *   QLORA_CODE_FP4  4-bit float E2M1 read as: bit 3 sign, bits 2..1 exponent
 *                   (bias 1, exponent 0 subnormal), bit 0 mantissa, i.e.
 *                   magnitudes {0, 1/2, 1, 3/2, 2, 3, 4, 6}, divided by 6
 *                   so the largest is 1, rounded once to fp32; code 8 is -0
 *                   and the quantizer writes code 0 for zero.
 *   QLORA_CODE_NF3, QLORA_CODE_NF2  k-bit NormalFloat, k = 3, 2 (the
 *                   "ModuLoRA: Finetuning 2-Bit LLMs on Consumer GPUs by
 *                   Integrating with Modular Quantizers" abstract finetunes
 *                   through 2-, 3- and 4-bit weights): 2^k levels built as
 *                   NF4's are (exact zero, 2^(k-1) positive and 2^(k-1)-1
 *                   negative levels at evenly spaced normal probabilities
 *                   up to delta_k = 1 - (1/(2(2^k-1)) + 1/2^(k+1))/2, over
 *                   Phi^{-1}(delta_k)); ascending with the code.
 *   QLORA_CODE_USER4, QLORA_CODE_USER3, QLORA_CODE_USER2  a caller's
 *                   codebook of 2^k values, k = 4, 3, 2 (the ModuLoRA
 *                   abstract materializes the low-precision weight from a
 *                   black-box quantizer: the kernels only need the values
 *                   behind the codes).  The values, fp32 in code order, are
 *                   passed in nf4_tensor_t.levels (and to
 *                   qlora_quantize_user); each must be finite with
 *                   |v| <= 1, and either 0 or |v| >= 2^-20 (so that every
 *                   midpoint of two values is exact in fp64); any order,
 *                   repeats allowed.  Quantizer: the nearest value, ties to
 *                   the lower value, of equal values the lowest code; an
 *                   all-zero block takes the code of the value nearest to 0.
 *                   Accepted by the quantizer, the dequantizer and the
 *                   layer; not by qlora_lq_init and the configuration-error
 *                   calls (QLORA_ERR_UNSUPPORTED).
 *   Block scaling and double quantization are the same for all types.
 *
 * Code storage by width k (4 for NF4 and FP4): a 64-element block takes
 * 8k bytes, two halves of 4k bytes (k little-endian 32-bit words) for
 * elements 0..31 and 32..63.  k = 4: the layout above (element 2j of the
 * block in the low nibble of byte j).  k = 3, 2: within a half, element
 * 8g + 2i + p (g, i in 0..3, p in 0..1) keeps code bits 0-1 at bit 8i + 2g
 * of word p and, for k = 3, code bit 2 at bit (8i + 2 + 2g + p) mod 32 of
 * word 2.  `codes` then holds N*K*k/8 bytes.
 *
 * Conventions for every call:
 *   - bf16 tensors are passed as uint16_t bit patterns.
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library never allocates, frees or keeps them.  Scratch memory comes
 *     from a caller-provided device workspace sized by
 *     qlora_workspace_size().  Pointers must be 16-byte aligned.
 *   - Work is enqueued on `stream` (0 = the null stream) and is
 *     asynchronous; no call synchronizes.  Apart from the fixed scratch
 *     array of qlora_linear_fwd_noalloc (below), the library keeps no
 *     mutable global state: calls are reentrant and thread-safe.  Calls that
 *     share a workspace must be ordered (same stream).
 *   - Every call validates its arguments before launching anything and
 *     returns a status code (QLORA_OK or a negative error, see below).  On
 *     an argument error (QLORA_ERR_INVALID, _UNSUPPORTED, _WORKSPACE)
 *     nothing has been enqueued and no output has been touched.
 *     QLORA_ERR_LAUNCH means a launch failed after the arguments were
 *     accepted: launches of the same call made before it stay enqueued, and
 *     the outputs are undefined.
 *   - Results are deterministic: the same inputs give bit-identical outputs.
 */
#ifndef QLORA_NF4_H_
#define QLORA_NF4_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---- */
#define QLORA_OK 0
#define QLORA_ERR_INVALID (-1)     /* null pointer, bad size, misalignment   */
#define QLORA_ERR_UNSUPPORTED (-2) /* block sizes other than 64 / 256, etc.  */
#define QLORA_ERR_WORKSPACE (-3)   /* workspace smaller than required        */
#define QLORA_ERR_LAUNCH (-4)      /* a HIP launch reported an error         */
#define QLORA_ERR_INFEASIBLE (-5)  /* qlora_ilp_plan: no choice fits          */

#define QLORA_CODE_NF4 0
#define QLORA_CODE_FP4 1
#define QLORA_CODE_NF3 2
#define QLORA_CODE_NF2 3
#define QLORA_CODE_USER4 4
#define QLORA_CODE_USER3 5
#define QLORA_CODE_USER2 6
/* Smallest magnitude of a nonzero value of a caller's codebook: 2^-20. */
#define QLORA_USER_MIN_MAGNITUDE (1.0f / 1048576.0f)

#define QLORA_NF4_BLOCKSIZE 64
#define QLORA_NF4_DQ_BLOCKSIZE 256
#define QLORA_MAX_RANK 256
/* Largest N and K accepted by qlora_linear_fwd / qlora_linear_bwd (a 256-row
 * tile of X or dY must span less than 2 GiB). */
#define QLORA_LINEAR_MAX_NK (1 << 22)

/* The quantized frozen weight.  All pointers are device pointers. */
typedef struct nf4_tensor_t {
  const uint8_t* codes; /* [N*K*k/8], k = bits of code_type */
  const uint8_t* q8;    /* [N*K/blocksize] */
  const float* step;    /* [ceil(N*K/blocksize/256)] */
  int64_t N;
  int64_t K;
  int32_t blocksize;    /* 64, 128 or 256, dividing K (others give
                           QLORA_ERR_UNSUPPORTED; K not a multiple of it,
                           QLORA_ERR_INVALID) */
  int32_t dq_blocksize; /* must be 256 */
  int32_t code_type;    /* QLORA_CODE_* (the type it was quantized with);
                           others give QLORA_ERR_UNSUPPORTED */
  const float* levels;  /* QLORA_CODE_USER*: HOST pointer to the 2^k code
                           values (code order), read during each call that
                           takes the tensor and not kept; NULL or values
                           outside the contract give QLORA_ERR_INVALID.
                           Ignored for the built-in code types. */
} nf4_tensor_t;

/* Text for a status code (static storage, never NULL). */
const char* qlora_status_str(int32_t status);

/* Host-side copy of the 16 NF4 levels (ascending, fp32) and of the 15
 * decision thresholds the quantizer compares against (a value x normalized
 * by its block's absmax gets the code #{i : x > thresholds[i]}, which is the
 * nearest level with ties going to the lower one).  No device work.  Either
 * pointer may be NULL.  Levels: normal quantiles with an exact zero,
 * normalized to [-1, 1] ("QLoRA: fine-tuning a 65B model on one GPU",
 * section "NormalFloat, double quantization, paged optimizers"). */
void nf4_code_table(float* levels16, float* thresholds15);

/* Host-side copy of the value of each code of `code_type` (in code order,
 * fp32; entries past 2^k are 0) and of its decision thresholds: the fp32
 * midpoint of each pair of consecutive distinct values, rounded toward
 * -inf, ascending (NF4: 15; FP4: 14, since +0 and -0 are one value; NF3: 7;
 * NF2: 3; the rest of thresholds15 is set to 0).  Returns the number of
 * thresholds, or QLORA_ERR_UNSUPPORTED for an unknown code type.  Either
 * pointer may be NULL; no device work. */
int32_t qlora_code_table(int32_t code_type, float* levels16, float* thresholds15);

/* Host-side check of a caller's codebook for QLORA_CODE_USER* and the
 * decision thresholds the quantizer derives from it (as qlora_code_table
 * gives them for the built-in types: the fp32 midpoint of each pair of
 * consecutive distinct values, rounded toward -inf, ascending; the rest of
 * thresholds15 is set to 0).  levels: 2^k fp32 values (host).  Returns the
 * number of thresholds, QLORA_ERR_UNSUPPORTED for a code type that is not a
 * user type, or QLORA_ERR_INVALID for NULL levels or values outside the
 * contract.  thresholds15 may be NULL; no device work. */
int32_t qlora_user_table(int32_t code_type, const float* levels, float* thresholds15);

/* Bytes of the three arrays of one configuration (code type, block size 64,
 * 128 or 256) for an N x K weight: N*K*k/8 + N*K/B + 4*ceil(N*K/B/256), k
 * the code width and B the block size; 0 for invalid sizes, an unknown code
 * type or an unsupported block size. */
size_t qlora_config_bytes(int32_t code_type, int32_t blocksize, int64_t N, int64_t K);

/* Bytes of the three NF4 arrays for an N x K weight (closed form:
 * N*K/2 + N*K/64 + 4*ceil(N*K/16384)); 0 for invalid sizes. */
size_t nf4_storage_bytes(int64_t N, int64_t K);

/* The same for any code type: N*K*k/8 + N*K/64 + 4*ceil(N*K/16384) with k
 * its width in bits; 0 for invalid sizes or an unknown code type. */
size_t qlora_storage_bytes(int32_t code_type, int64_t N, int64_t K);

/* nf4_quantize -- blockwise NF4 quantization with double-quantized absmax
 * constants, once per frozen weight (blog section "NormalFloat, double
 * quantization, paged optimizers"; capability page "Qlora 4 Bit
 * Quantization With Nf4 Fp4 Data Types And Lora Adapters", NF4 entry:
 * block-wise absmax scaling and double quantization of the constants).
 *
 *   W      [N, K] fp32, device.  Must be finite.
 *   N, K   N >= 1, K >= 64, K % 64 == 0.
 *   blocksize, dq_blocksize   64, 128 or 256 (dividing K), and 256; codes
 *          are packed in 64-element units whatever the block size, q8 has
 *          N*K/blocksize bytes and step ceil(N*K/blocksize/256) floats.
 *   codes  [N*K/2] out;  q8 [N*K/64] out;  step [ceil(N*K/16384)] out.
 * Per block b of 64 consecutive elements: c_b = max|w|; each element gets
 * the level nearest to fl32(w / c_b) (ties to the lower level; an all-zero
 * block gets the zero level).  Per group g of 256 consecutive blocks (the
 * last group may be shorter): step_g = fl32(max_b c_b / 255),
 * q_b = min(255, round_half_even(fl32(c_b / step_g))), q_b = 0 if step_g = 0.
 */
int32_t nf4_quantize(const float* W, int64_t N, int64_t K, int32_t blocksize,
                     int32_t dq_blocksize, uint8_t* codes, uint8_t* q8,
                     float* step, hipStream_t stream);

/* qlora_quantize -- nf4_quantize for any code type: identical except that
 * each element gets the code of the value of `code_type` nearest to
 * fl32(w / c_b) (ties to the lower value; zero, and an all-zero block, get
 * the code of zero: 7 for NF4, 0 for FP4, 3 for NF3, 1 for NF2), stored at
 * the type's width (codes [N*K*k/8]).  An unknown code type gives
 * QLORA_ERR_UNSUPPORTED, a user code type QLORA_ERR_INVALID (it needs its
 * values: qlora_quantize_user).  nf4_quantize(...) is
 * qlora_quantize(..., QLORA_CODE_NF4, ...). */
int32_t qlora_quantize(const float* W, int64_t N, int64_t K, int32_t code_type,
                       int32_t blocksize, int32_t dq_blocksize, uint8_t* codes,
                       uint8_t* q8, float* step, hipStream_t stream);

/* qlora_quantize_user -- qlora_quantize with a caller's codebook:
 * code_type QLORA_CODE_USER4, _USER3 or _USER2 and `levels` (host, 2^k
 * fp32 values in code order, read during the call) under the contract and
 * quantizer rule above.  The division w / c_b is the IEEE-correct one for
 * every block.  A built-in code type gives QLORA_ERR_UNSUPPORTED (use
 * qlora_quantize); bad levels, QLORA_ERR_INVALID. */
int32_t qlora_quantize_user(const float* W, int64_t N, int64_t K, int32_t code_type,
                            const float* levels, int32_t blocksize, int32_t dq_blocksize,
                            uint8_t* codes, uint8_t* q8, float* step, hipStream_t stream);

/* nf4_dequantize -- materialize the bf16 weight [N, K] from its quantized
 * state, with the code table of w->code_type (for checking and interop; the
 * linear layer never does this: it dequantizes tiles on chip).  w->N, w->K
 * as in nf4_quantize.  W_bf16 [N*K] out. */
int32_t nf4_dequantize(const nf4_tensor_t* w, uint16_t* W_bf16,
                       hipStream_t stream);

/* Workspace bytes needed by qlora_linear_fwd (for_bwd = 0) or
 * qlora_linear_bwd (for_bwd = 1) at these sizes; 0 for invalid sizes. */
size_t qlora_workspace_size(int64_t M, int64_t N, int64_t K, int32_t r,
                            int32_t for_bwd);

/* qlora_linear_fwd -- Y = X W^T + s (X A^T) B^T with W dequantized on the
 * fly to bf16 (blog section "Where the memory goes").
 *
 *   w       quantized weight, N >= 1, N % 8 == 0, K % 64 == 0,
 *           N, K <= QLORA_LINEAR_MAX_NK, packed codes under 2 GiB
 *           (N K bits / 8 < 2^31)
 *   X       [M, K] bf16, M >= 1
 *   A       [r, K] bf16;  B [N, r] bf16;  1 <= r <= 256
 *   s       LoRA scale
 *   Y       [M, N] bf16 out
 *   U_out   [M, r] bf16 out, may be NULL: X A^T rounded to bf16, which
 *           qlora_linear_bwd can take back instead of recomputing it
 *   ws      device workspace of ws_bytes >= qlora_workspace_size(M,N,K,r,0)
 * Accumulation is fp32.  M <= 16 takes a bandwidth-bound path that
 * streams the packed weight once (when its per-workgroup tables fit in
 * LDS: K up to about 32000 at M = 16, r = 256); larger M, or
 * larger K, takes the MFMA tile path.  Both meet the same tolerance.
 */
int32_t qlora_linear_fwd(const nf4_tensor_t* w, const uint16_t* X, int64_t M,
                         const uint16_t* A, const uint16_t* B, int32_t r,
                         float s, uint16_t* Y, uint16_t* U_out, void* ws,
                         size_t ws_bytes, hipStream_t stream);

/* qlora_linear_bwd -- gradients of the layer for the output gradient dY,
 * re-dequantizing W on chip (ModuLoRA abstract: the backward pass
 * materializes the low-precision weight from the quantized module):
 *   dX = dY W + s (dY B) A      [M, K] bf16 out, may be NULL (skipped)
 *   dA = s (dY B)^T X           [r, K] bf16 out
 *   dB = s dY^T (X A^T)         [N, r] bf16 out
 * Outputs are overwritten, not accumulated.  U is X A^T as returned by
 * qlora_linear_fwd's U_out, or NULL to recompute it.  Other arguments as in
 * qlora_linear_fwd; ws_bytes >= qlora_workspace_size(M,N,K,r,1).
 */
int32_t qlora_linear_bwd(const nf4_tensor_t* w, const uint16_t* X,
                         const uint16_t* dY, int64_t M, const uint16_t* A,
                         const uint16_t* B, const uint16_t* U, int32_t r,
                         float s, uint16_t* dX, uint16_t* dA, uint16_t* dB,
                         void* ws, size_t ws_bytes, hipStream_t stream);

/* Measurement variants of the two layer calls: identical work, and in
 * addition `ev_begin` is recorded on `stream` right before, and `ev_end`
 * right after, the launch of the dequantizing main kernel (the MFMA tile
 * GEMM, or for M <= 16 in the forward pass the weight-streaming kernel; in
 * the backward pass the dX GEMM, so nothing is recorded when dX is NULL).
 * hipEventElapsedTime over the pair is that kernel's duration.  Either
 * event may be NULL.  The events are created and owned by the caller. */
int32_t qlora_linear_fwd_ev(const nf4_tensor_t* w, const uint16_t* X,
                            int64_t M, const uint16_t* A, const uint16_t* B,
                            int32_t r, float s, uint16_t* Y, uint16_t* U_out,
                            void* ws, size_t ws_bytes, hipStream_t stream,
                            hipEvent_t ev_begin, hipEvent_t ev_end);
int32_t qlora_linear_bwd_ev(const nf4_tensor_t* w, const uint16_t* X,
                            const uint16_t* dY, int64_t M, const uint16_t* A,
                            const uint16_t* B, const uint16_t* U, int32_t r,
                            float s, uint16_t* dX, uint16_t* dA, uint16_t* dB,
                            void* ws, size_t ws_bytes, hipStream_t stream,
                            hipEvent_t ev_begin, hipEvent_t ev_end);

/* qlora_linear_fwd_noalloc -- for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): qlora_linear_fwd with the same arguments except the
 * workspace, and the same result bit for bit.  Its scratch (U and the fp32
 * partial sums) is a fixed device array of QLORA_NOALLOC_SCRATCH_BYTES that
 * the library holds on every device it runs on until the process ends; the
 * call allocates nothing (no hipMalloc, hipFree or allocating library
 * routine).  Sizes whose workspace (qlora_workspace_size(M, N, K, r, 0))
 * exceeds the array give QLORA_ERR_WORKSPACE before any launch.  Every call
 * on one device shares that device's array and leaves its contents behind;
 * calls that overlap on one device (two host threads, or two streams not
 * ordered by events) race on it and give undefined results.  The caller
 * still owns X, A, B, Y and U_out. */
#define QLORA_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
int32_t qlora_linear_fwd_noalloc(const nf4_tensor_t* w, const uint16_t* X,
                                 int64_t M, const uint16_t* A,
                                 const uint16_t* B, int32_t r, float s,
                                 uint16_t* Y, uint16_t* U_out,
                                 hipStream_t stream);

/* qlora_linear_multi_fwd -- the layer for rows of many adapters over one
 * frozen weight (the base never changes and is shared; the adapters are small:
 * blog section "Where the memory goes"):
 *   Y_i = X_i W^T + s_a (X_i A_a^T) B_a^T,   a = index[i]
 * and Y_i = X_i W^T where index[i] lies outside 0 .. n_adapters - 1.
 *   w, X, M, Y   as in qlora_linear_fwd, M at most 2^26; Y overlaps no input (at
 *                X's address: QLORA_ERR_INVALID)
 *   A, B         [n_adapters, r, K] and [n_adapters, N, r] bf16, contiguous
 *                (adapters of smaller rank padded with zeros), n_adapters >= 1,
 *                1 <= r <= 256; any size together
 *   s            [n_adapters] fp32 (device)
 *   index        [M] int32 (device), in any order; rows of one adapter next to
 *                each other (prompts) cost least.  Read by the kernels; any
 *                value is allowed.
 *   ws           >= qlora_multi_workspace_size(M, N, K, r) bytes
 * Three kernels, chosen by M, N, K and r alone: M <= 16 streams the packed weight
 * once, as qlora_linear_fwd does, while the tables of a workgroup fit its LDS
 * (K up to about 32000 at rank 256); otherwise batches of up to a few hundred
 * rows, 4096 at most, stream it with up to 64 tokens per workgroup, where that is
 * estimated to be the faster way; the rest takes the MFMA tile path.  So a row's
 * last bits depend on how many rows come with it, though not on which ones.
 * Besides the one rounding of Y to bf16, and sums in fp32:
 *   both streams   a weight is its level rounded to bf16 (after a common factor
 *                  that brings the levels nearer to bf16 values) times an fp32
 *                  constant, where the tiles, as nf4_dequantize, round level times
 *                  constant; X A^T stays in fp32
 *   tiles          s (X A^T) is rounded to bf16 once (qlora_linear_fwd rounds
 *                  X A^T and s times that)
 * A row's result does not depend on adapters that it does not have, whatever
 * they hold; an infinity or NaN in B gives its adapter's rows an infinity or NaN
 * in that column. */
size_t qlora_multi_workspace_size(int64_t M, int64_t N, int64_t K, int32_t r);
int32_t qlora_linear_multi_fwd(const nf4_tensor_t* w, const uint16_t* X, int64_t M,
                               const uint16_t* A, const uint16_t* B, const float* s,
                               int32_t n_adapters, int32_t r, const int32_t* index, uint16_t* Y,
                               void* ws, size_t ws_bytes, hipStream_t stream);

/* Measurement helper (not part of the layer): a read-only stream over
 * `bytes` bytes of device memory at src (16-byte aligned, bytes a multiple
 * of 16), the HBM read ceiling the few-token forward's weight stream is
 * compared with.  Every 16-byte word is read once; each of the
 * QLORA_STREAM_GRID workgroups writes one uint32 to sink[0 ..
 * QLORA_STREAM_GRID - 1] (a device buffer the caller owns).  Errors as for
 * the other calls; nothing is allocated. */
#define QLORA_STREAM_GRID 1024
int32_t qlora_stream_read(const void* src, size_t bytes, uint32_t* sink,
                          hipStream_t stream);

/* ---- Low-rank plus quantized decomposition (adapter initialization) ----
 *
 * qlora_lq_init -- split a frozen weight into a quantized part Q and a
 * rank-r part L1 L2 ("LQ-LoRA: Low-rank Plus Quantized Matrix Decomposition
 * for Efficient Language Model Finetuning", abstract: an iterative
 * algorithm; the quantized part stays fixed, the low-rank part is the
 * trained adapter).  Alternating minimization of ||W - Q - L1 L2||_F:
 *   L step: L1 L2 = rank-r approximation of W - Q, by randomized subspace
 *           iteration from the caller's Gaussian test matrix `omega`
 *           (power_iters rounds, each re-orthonormalized) and
 *           Rayleigh-Ritz on its l-dimensional range;
 *   Q step: Q = qlora_quantize(W - L1 L2) with `code_type`.
 * `start` = QLORA_LQ_START_SVD begins with Q = 0 (the first L step fits W
 * itself); QLORA_LQ_START_QUANTIZE begins with L = 0 (the first Q step is
 * plain quantization).  One iteration is one L step and one Q step.
 *
 *   W       [N, K] fp32, device; K % 64 == 0
 *   r, l    rank and subspace width: 1 <= r < l <= QLORA_LQ_MAX_L,
 *           l % 16 == 0 (l - r extra directions improve the fit)
 *   omega   [K, l] fp32, i.i.d. N(0, 1) drawn by the caller
 *   iters   1..64;  power_iters 0..16
 *   s       LoRA scale of the adapter outputs (nonzero)
 *   codes, q8, step   out: Q, as qlora_quantize writes it
 *   L1      [N, r] fp32 out;  L2t [K, r] fp32 out (L2 transposed);
 *           L1 L2t^T is the low-rank part, the factors sharing each
 *           singular value evenly (both carry its square root)
 *   A       [r, K] bf16 out = bf16(L2);  B [N, r] bf16 out = bf16(L1 / s),
 *           so that s B A ~ L1 L2 as the adapter of qlora_linear_fwd
 *   ws      device workspace, 256-byte aligned, ws_bytes >=
 *           qlora_lq_workspace_size(N, K, r, l) (about 4 N K bytes)
 * The pair returned is the last Q step's Q with the L step before it
 * (start SVD) or after it (start QUANTIZE).  Sums have a fixed order:
 * results are reproducible.  Every call raises the dynamic LDS limit of the
 * two one-workgroup solver kernels (idempotent). */
#define QLORA_LQ_MAX_L 96
#define QLORA_LQ_START_SVD 0
#define QLORA_LQ_START_QUANTIZE 1
size_t qlora_lq_workspace_size(int64_t N, int64_t K, int32_t r, int32_t l);
int32_t qlora_lq_init(const float* W, int64_t N, int64_t K, int32_t code_type,
                      int32_t r, int32_t l, const float* omega, int32_t iters,
                      int32_t power_iters, int32_t start, float s,
                      uint8_t* codes, uint8_t* q8, float* step, uint16_t* A,
                      uint16_t* B, float* L1, float* L2t, void* ws,
                      size_t ws_bytes, hipStream_t stream);

/* ---- Quantization configuration per matrix under a memory budget ----
 *
 * The LQ-LoRA abstract ("LQ-LoRA: Low-rank Plus Quantized Matrix
 * Decomposition for Efficient Language Model Finetuning") chooses each
 * matrix's quantization parameters by an integer linear program so that the
 * model meets an overall memory budget.  Here a configuration is a code type
 * (QLORA_CODE_*) and a block size (64, 128 or 256, with double
 * quantization; the layer takes all of them), its memory the state bytes
 * (qlora_config_bytes) and its error on a matrix the squared Frobenius
 * error of the quantized part.
 *
 * qlora_quant_error -- *sq_err = ||R - W_hat(R)||_F^2 in fp64, where
 * R = W, or R = W - L1 L2t^T when L1 and L2t are given (the decomposition
 * error of an LQ-LoRA initialization with that configuration), and W_hat(R)
 * is R quantized with `code_type` and dequantized (as nf4_dequantize).
 *   W      [N, K] fp32, device; K % 64 == 0
 *   L1     [N, r] fp32, L2t [K, r] fp32, device, both NULL or both given;
 *          1 <= r <= QLORA_LQ_MAX_L
 *   sq_err one double, device (8-byte aligned), written on the stream
 *   ws     device workspace, 256-byte aligned, ws_bytes >=
 *          qlora_quant_error_workspace_size(N, K, code_type, L1 != NULL)
 * The sum has a fixed order: the result is reproducible. */
size_t qlora_quant_error_workspace_size(int64_t N, int64_t K, int32_t code_type,
                                        int32_t with_lowrank);
int32_t qlora_quant_error(const float* W, int64_t N, int64_t K,
                          int32_t code_type, const float* L1, const float* L2t,
                          int32_t r, double* sq_err, void* ws, size_t ws_bytes,
                          hipStream_t stream);

/* qlora_config_error -- qlora_quant_error for any configuration: code type
 * and block size (64, 128 or 256, dividing K; the abstract's "bit-width,
 * block size"); qlora_quant_error is this call at block size 64.  The
 * workspace is sized by qlora_config_error_workspace_size. */
size_t qlora_config_error_workspace_size(int64_t N, int64_t K,
                                         int32_t code_type, int32_t blocksize,
                                         int32_t with_lowrank);
int32_t qlora_config_error(const float* W, int64_t N, int64_t K,
                           int32_t code_type, int32_t blocksize,
                           const float* L1, const float* L2t, int32_t r,
                           double* sq_err, void* ws, size_t ws_bytes,
                           hipStream_t stream);

/* qlora_ilp_plan -- host only, no device work.  Given, for M matrices and
 * C configurations, the errors err[m*C + c] (finite) and the bytes
 * bytes[m*C + c] (>= 0) (host arrays), choose one configuration per matrix
 * minimizing the total error subject to total bytes <= budget.  Solved
 * exactly (dynamic programming over the Pareto front of partial choices);
 * errors are summed in matrix order, and ties go to fewer total bytes, then
 * to the lexicographically smallest choice vector.  Writes choice[M] (host),
 * *total_err and *total_bytes; returns QLORA_ERR_INFEASIBLE if no choice
 * fits.  1 <= C <= 64. */
int32_t qlora_ilp_plan(int32_t n_matrices, int32_t n_configs, const double* err,
                       const int64_t* bytes, int64_t budget, int32_t* choice,
                       double* total_err, int64_t* total_bytes);

/* ---- Around the layer: attention, rotary positions, norms, gradient clipping, AdamW ----
 *
 * The other operators of a finetuning step.  Element types of the norms and
 * of the clipping: QLORA_TYPE_BF16 or QLORA_TYPE_FP32 (others give
 * QLORA_ERR_UNSUPPORTED).  Attention is bf16 with fp32 sums. */
#define QLORA_TYPE_BF16 0
#define QLORA_TYPE_FP32 1

/* One [batch, row, head, dim] bf16 tensor: device pointer (16-byte aligned)
 * and element strides; the dim stride is 1.  Strides must be multiples of 8,
 * not negative, and the row stride at most QLORA_ATTN_MAX_STRIDE.  q, k and v
 * may be views of one projection's output; strides of 0 are allowed for
 * inputs.  An output's rows lie apart: from the smallest stride up, each
 * reaches past what the dimensions before it span (else QLORA_ERR_INVALID).
 * The batch stride is not used for packed batches. */
#define QLORA_ATTN_MAX_STRIDE ((int64_t)1 << 22)
typedef struct qlora_heads_t {
  uint16_t* data;
  int64_t batch_stride, row_stride, head_stride;
} qlora_heads_t;

/* What is attended to what.
 *   Dense: cu_seqlens_q = cu_seqlens_k = NULL; n_seq sequences of q_rows
 *   queries and k_rows keys each.
 *   Packed: q_rows and k_rows are the rows of all n_seq sequences together;
 *   cu_seqlens_q / _k (device, int32, n_seq + 1 ascending offsets from 0;
 *   both given, equal pointers for self-attention): sequence s has the query
 *   rows cu_seqlens_q[s] .. cu_seqlens_q[s + 1] - 1 and likewise the keys.
 *   Sequences may be empty on either side.  Rows past the last offset belong
 *   to no sequence: what they hold reaches no output, and outputs there are 0
 *   (lse -inf).
 *   The offsets are read by the kernels and clamped to the rows, so wrong
 *   ones give undefined outputs but no access outside the tensors.
 *   Causal: query i of a sequence of lq queries and lk keys sees the keys
 *   j <= i + lk - lq (the last query sees the last key).
 * Each key/value head serves heads / kv_heads consecutive query heads. */
typedef struct qlora_attention_t {
  int64_t n_seq;
  int64_t q_rows, k_rows;       /* >= 0, below 2^30 */
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  int32_t heads, kv_heads;      /* kv_heads divides heads */
  int32_t head_dim;             /* a multiple of 8 up to QLORA_ATTN_MAX_DIM
                                   (others: QLORA_ERR_UNSUPPORTED) */
  int32_t causal;
  float scale;                  /* QLORA_ATTN_MIN_SCALE to _MAX_SCALE */
} qlora_attention_t;
#define QLORA_ATTN_MAX_DIM 128
/* 2^-100 and 2^100: the kernels also compute with 1 / scale, and with scale
 * times log2(e), in fp32. */
#define QLORA_ATTN_MIN_SCALE 0x1p-100f
#define QLORA_ATTN_MAX_SCALE 0x1p+100f

/* qlora_attention_fwd -- per head O = softmax(scale Q K^T) V over the keys
 * that each query sees, and lse = log sum exp(scale q k) of each row (fp32,
 * natural logarithm; dense [n_seq, heads, q_rows], packed [heads, q_rows]).
 * A query that sees no key gets O = 0 and lse = -inf.  Sums and the softmax
 * are fp32; the probabilities are rounded to bf16 for the product with V.
 * Values outside a sequence never reach its outputs, whatever they are; a
 * NaN or infinity inside one may reach every row of that sequence and head.
 * o may be q itself (the same view); apart from that it overlaps no input (one
 * that starts at the same address: QLORA_ERR_INVALID).
 * ws_bytes >= qlora_attention_fwd_workspace_size(a) (16-byte aligned; 0, and
 * ws may be NULL, where the work is not split: see the backward pass). */
size_t qlora_attention_fwd_workspace_size(const qlora_attention_t* a);
int32_t qlora_attention_fwd(const qlora_attention_t* a, const qlora_heads_t* q,
                            const qlora_heads_t* k, const qlora_heads_t* v,
                            const qlora_heads_t* o, float* lse, void* ws, size_t ws_bytes,
                            hipStream_t stream);

/* qlora_attention_bwd -- the gradients of q, k and v for the output gradient
 * dout, with the probabilities recomputed from lse (o and lse as the forward
 * wrote them):
 *   P = exp(scale Q K^T - lse),  dS = P (dO V^T - rowsum(dO O)),
 *   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
 * dK and dV summed over the query heads of a key/value head.  dq, dk and dv
 * are overwritten; queries that see no key, and keys that no query sees, get
 * 0.  P and dS are rounded to bf16 for the products that follow.
 * dq may be o itself, dk k and dv v (the same view); apart from that the
 * outputs overlap neither each other nor an input (those that start at the same
 * address: QLORA_ERR_INVALID).
 * ws_bytes >= qlora_attention_bwd_workspace_size(a) (16-byte aligned; 0 for
 * invalid sizes or nothing to compute).  Both calls split long walks over
 * several workgroups where that is faster (few tiles, or few key/value heads
 * under a causal mask), by the shapes alone; the workspace then holds their
 * fp32 partial results, and a second kernel adds them in a fixed order. */
size_t qlora_attention_bwd_workspace_size(const qlora_attention_t* a);
int32_t qlora_attention_bwd(const qlora_attention_t* a, const qlora_heads_t* q,
                            const qlora_heads_t* k, const qlora_heads_t* v,
                            const qlora_heads_t* o, const float* lse,
                            const qlora_heads_t* dout, const qlora_heads_t* dq,
                            const qlora_heads_t* dk, const qlora_heads_t* dv, void* ws,
                            size_t ws_bytes, hipStream_t stream);

/* qlora_rope -- rotary positions of q and k, in one call.  The first `rot`
 * elements of every head turn in pairs: pair j of a row at position p by the
 * angle a = p inv_freq[j],
 *   (x, y) -> scale (x cos a - y sin a, y cos a + x sin a),
 * x and y being the elements j and rot / 2 + j (interleaved = 0) or 2j and
 * 2j + 1 (interleaved = 1).  The other elements are copied.  inverse = 1 turns
 * by -a, which is the backward pass: the gradients of q and k from those of the
 * outputs.  Angles are taken in fp64 (any position up to 2^40 in magnitude, also
 * negative ones), the rotation in fp32, rounded once to bf16.
 *   n_seq, rows   dense (cu_seqlens NULL): a batch of n_seq sequences of `rows`
 *                 rows; packed: `rows` rows in n_seq sequences with the offsets
 *                 cu_seqlens as in qlora_attention_t (device, int32, n_seq + 1)
 *   positions     device, int32 or int64 by position_bytes (4, 8), with element
 *                 strides over the batch (dense) and the rows (0 allowed); NULL:
 *                 a row's place in its sequence, from 0.  Given positions go
 *                 before cu_seqlens.
 *   inv_freq      device, rot / 2 doubles
 *   q, k          [batch, row, head, dim] views (head_dim a multiple of 8 up to
 *                 QLORA_ROPE_MAX_DIM; 2 <= rot <= head_dim, even); k_heads = 0: q
 *                 alone (k and k_out are not looked at)
 *   q_out, k_out  outputs whose rows lie apart; q_out may be q itself and k_out k
 *                 (the same view: in place); apart from that outputs overlap
 *                 neither inputs nor each other (those that start at the same
 *                 address: QLORA_ERR_INVALID)
 * Rows past the last offset belong to no sequence and are copied; wrong offsets
 * give wrong positions but no access outside the tensors. */
#define QLORA_ROPE_MAX_DIM 1024
typedef struct qlora_rope_t {
  int64_t n_seq, rows;
  const int32_t* cu_seqlens;
  const void* positions;
  int64_t position_batch_stride, position_row_stride;
  const double* inv_freq;
  int32_t position_bytes;
  int32_t q_heads, k_heads, head_dim, rot;
  int32_t interleaved, inverse;
  float scale;                  /* finite */
} qlora_rope_t;
int32_t qlora_rope(const qlora_rope_t* a, const qlora_heads_t* q, const qlora_heads_t* k,
                   const qlora_heads_t* q_out, const qlora_heads_t* k_out, hipStream_t stream);

/* qlora_norm_fwd -- layer norm (rms = 0) or root-mean-square norm (rms = 1) of
 * each row of x [rows, width]:
 *   mean = sum(x) / width (0 if rms),  rstd = 1 / sqrt(sum((x - mean)^2) / width + eps),
 *   y = (x - mean) rstd weight + bias.
 *   x, y          [rows, width] of x_type, 0 <= rows < 2^30, 1 <= width <=
 *                 QLORA_NORM_MAX_WIDTH_BF16 / _FP32 by x_type (more:
 *                 QLORA_ERR_UNSUPPORTED)
 *   weight, bias  [width] of w_type; bias may be NULL
 *   mean, rstd    [rows] fp32 out; mean may be NULL if rms
 * These pointers need the alignment of their elements only.  eps >= 0. */
#define QLORA_NORM_MAX_WIDTH_BF16 65536
#define QLORA_NORM_MAX_WIDTH_FP32 32768
int32_t qlora_norm_fwd(const void* x, int64_t rows, int64_t width, int32_t x_type,
                       const void* weight, const void* bias, int32_t w_type, float eps,
                       int32_t rms, void* y, float* mean, float* rstd, hipStream_t stream);

/* qlora_norm_bwd -- its gradients, from x, the row statistics and dy:
 *   z = (x - mean) rstd,  g = dy weight,
 *   dx = rstd (g - z mean(g z) - [mean(g) unless rms]),
 *   dweight = sum over rows of dy z,  dbias = sum over rows of dy.
 * dx [rows, width] of x_type; dweight, dbias [width] of w_type, summed in
 * fp32.  Each of the three may be NULL (skipped).  Outputs are overwritten.
 * ws_bytes >= qlora_norm_bwd_workspace_size(rows, width, x_type) (16-byte
 * aligned; 0 for invalid sizes; not used without dweight and dbias). */
size_t qlora_norm_bwd_workspace_size(int64_t rows, int64_t width, int32_t x_type);
int32_t qlora_norm_bwd(const void* dy, const void* x, int64_t rows, int64_t width,
                       int32_t x_type, const void* weight, int32_t w_type, int32_t rms,
                       const float* mean, const float* rstd, void* dx, void* dweight,
                       void* dbias, void* ws, size_t ws_bytes, hipStream_t stream);

/* qlora_clip_grad_norm -- the 2-norm of n gradient tensors taken together,
 * and their scaling by min(1, max_norm / (norm + 1e-6)).
 *   n          tensors, 0 <= n <= 2^20
 *   grads      HOST array of n device pointers (aligned to their elements)
 *   sizes      HOST array: elements of each (0 allowed; 2^44 in all)
 *   types      HOST array: QLORA_TYPE_* of each
 *   max_norm   >= 0 (not NaN); with +inf the factor is 1 unless the norm is NaN
 *   out        HOST array of n device pointers that take the scaled gradients
 *              (same sizes and types; each either its gradient itself or
 *              apart from all of them), or NULL: in place.  In place, nothing
 *              is written when the factor is 1.
 *   norm       one float (device) out, the norm before scaling
 * The three arrays are read during the call and not kept.  Squares are summed
 * in fp64.  A NaN norm scales by NaN, and an infinite one by 0 if max_norm is
 * finite, as min(1, max_norm / (norm + 1e-6)) says.  ws: 16-byte aligned device memory of
 * qlora_clip_workspace_size(n) bytes.
 * qlora_grad_norm is the norm alone. */
size_t qlora_clip_workspace_size(int64_t n);
int32_t qlora_clip_grad_norm(int64_t n, const void* const* grads, const int64_t* sizes,
                             const int32_t* types, float max_norm, void* const* out,
                             float* norm, void* ws, size_t ws_bytes, hipStream_t stream);
int32_t qlora_grad_norm(int64_t n, const void* const* grads, const int64_t* sizes,
                        const int32_t* types, float* norm, void* ws, size_t ws_bytes,
                        hipStream_t stream);

/* qlora_adamw_step -- one AdamW step of n parameter tensors:
 *   g = c grad,  c = min(1, max_norm / (norm + 1e-6)) as in qlora_clip_grad_norm
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32, p rounded once to its type.
 *   n            tensors, 0 <= n <= 2^20
 *   params       HOST array of n device pointers (aligned to their elements; each
 *                tensor once), updated in place
 *   grads        HOST array: the gradients; NULL leaves that tensor and its
 *                states alone
 *   copies       HOST array of bf16 tensors that take the updated parameters,
 *                rounded (for parameters held in fp32 beside a bf16 copy; NULL
 *                entries: none), or NULL
 *   sizes        HOST array: elements of each (0 allowed)
 *   param_types, grad_types   HOST arrays: QLORA_TYPE_* of each
 *   state_bits   32: m and v are fp32; 8: m is int8, v uint8, with scales below
 *   m, v         the states of all tensors one after the other, each from a
 *                multiple of QLORA_ADAMW_BLOCK elements on: QLORA_ADAMW_BLOCK
 *                state_blocks elements (16-byte aligned).  A new state is all
 *                zeros (scales too).
 *   m_scale, v_scale   8 bits: one float per block of QLORA_ADAMW_BLOCK elements
 *                (the last block of a tensor may be shorter); 32 bits: not used
 *   state_blocks >= qlora_adamw_blocks(n, sizes) (else QLORA_ERR_WORKSPACE)
 *   step         >= 1, the number of updates that the tensors have had, this one
 *                included (tensors that have had fewer: in a call of their own,
 *                with the others' gradients NULL); lr, eps, weight_decay >= 0,
 *                0 <= beta < 1
 *   lr_dev, step_dev   one float, one int64 on the device that are read by the
 *                kernels in place of lr and step (a captured step replays with
 *                their values at that time), or NULL
 *   norm         one float (device), the gradients' norm; NULL: no clipping
 *   max_norm     >= 0 (not NaN), with norm; the factor min(1, max_norm / (norm +
 *                1e-6)) is rounded once, from fp64
 * The host arrays are read during the call and not kept.
 * 8-bit states: codes with a scale s per block, the block's largest |m| and v,
 *   m = s c |c| / 127^2,  c in -127..127;   v = s (c / 255)^4,  c in 0..255.
 * c is the number of thresholds (i - 1/2)^2, i = 1..127, up to fl(|m| fl(127^2 / s))
 * with the sign of m, and of ((i - 1/2)^2)^2, i = 1..255, up to fl(v fl(255^4 / s)),
 * at least 1 where v > 0.  Blocks whose largest value is below 2^-96 get s = 0.
 * A block with an infinity or NaN gets s = NaN: it is NaN from then on.  Products
 * and sums up to the codes are rounded one by one to fp32, in the order written. */
#define QLORA_ADAMW_BLOCK 256
typedef struct qlora_adamw_t {
  int64_t n;
  void* const* params;
  const void* const* grads;
  uint16_t* const* copies;
  const int64_t* sizes;
  const int32_t* param_types;
  const int32_t* grad_types;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t state_blocks;
  int64_t step;
  double lr, beta1, beta2, weight_decay;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* norm;
  float eps;
  double max_norm;
  int32_t state_bits;
} qlora_adamw_t;
/* Blocks of states of n tensors; -1 for invalid sizes (2^31 blocks or more). */
int64_t qlora_adamw_blocks(int64_t n, const int64_t* sizes);
int32_t qlora_adamw_step(const qlora_adamw_t* a, hipStream_t stream);

/* qlora_adamw_values -- the values that 8-bit states stand for, in fp32 (for
 * inspection and conversion): m_out, v_out [blocks QLORA_ADAMW_BLOCK], 16-byte
 * aligned, from m, v, m_scale, v_scale as above. */
int32_t qlora_adamw_values(const void* m, const void* v, const float* m_scale,
                           const float* v_scale, int64_t blocks, float* m_out, float* v_out,
                           hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_NF4_H_ */
