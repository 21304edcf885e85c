// C ABI of the operators around the layer (attention, rotary positions, norms,
// gradient clipping, AdamW): argument checks and workspaces.  The declarations, with the
// meaning of every argument, are in include/qlora_nf4.h.
#include "../../include/qlora_nf4.h"

#include <math.h>

#include <algorithm>

#include "kernels.hpp"

using namespace qn;

namespace {

inline int32_t launch_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_LAUNCH; }

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool type_ok(int32_t t) { return t == QLORA_TYPE_BF16 || t == QLORA_TYPE_FP32; }
inline int64_t type_bytes(int32_t t) { return t == QLORA_TYPE_FP32 ? 4 : 2; }
static_assert(kNormBF16 == QLORA_TYPE_BF16 && kNormF32 == QLORA_TYPE_FP32, "type ids");

// ---- attention ----

constexpr int64_t kMaxRows = (int64_t)1 << 30;

int32_t attn_ok(const qlora_attention_t* a) {
  if (!a || a->n_seq < 0 || a->n_seq >= kMaxRows || a->q_rows < 0 || a->q_rows >= kMaxRows ||
      a->k_rows < 0 || a->k_rows >= kMaxRows || a->heads < 1 || a->kv_heads < 1 ||
      a->heads % a->kv_heads != 0 || !(a->scale >= QLORA_ATTN_MIN_SCALE) ||
      !(a->scale <= QLORA_ATTN_MAX_SCALE))
    return QLORA_ERR_INVALID;
  if ((a->cu_seqlens_q == nullptr) != (a->cu_seqlens_k == nullptr)) return QLORA_ERR_INVALID;
  if (!aligned(a->cu_seqlens_q, 4) || !aligned(a->cu_seqlens_k, 4)) return QLORA_ERR_INVALID;
  if (a->head_dim < 1) return QLORA_ERR_INVALID;
  if (a->head_dim > QLORA_ATTN_MAX_DIM || a->head_dim % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  // Every pass's workgroups are counted in 32 bits.  A tile has 128 rows, and
  // attn_splits gives it at most one workgroup per 64 rows of its walk, times
  // the heads of a group; beside more than 65536 tiles it gives it one.
  const int64_t rows = a->q_rows > a->k_rows ? a->q_rows : a->k_rows;
  const int64_t tiles = a->cu_seqlens_q ? rows / 32 + a->n_seq + 1
                                        : (rows / 32 + 1) * (a->n_seq > 0 ? a->n_seq : 1);
  if (tiles >= ((int64_t)1 << 31) / a->heads) return QLORA_ERR_INVALID;
  return QLORA_OK;
}

// rows == 0: the tensor is empty, its pointer is not looked at.
bool view_ok(const qlora_heads_t* t, int64_t rows) {
  if (!t) return false;
  if (rows == 0) return true;
  return t->data && aligned(t->data, 16) && t->batch_stride >= 0 && t->row_stride >= 0 &&
         t->head_stride >= 0 && t->batch_stride % 8 == 0 && t->row_stride % 8 == 0 &&
         t->head_stride % 8 == 0 && t->row_stride <= QLORA_ATTN_MAX_STRIDE;
}

// An output's rows lie apart: taken from the smallest stride up, each stride
// reaches past what the dimensions before it span.
bool rows_apart(const qlora_heads_t* t, int64_t batch, int64_t rows, int64_t heads, int64_t dim) {
  if (batch == 0 || rows == 0) return true;
  struct {
    int64_t n, stride;
  } d[3] = {{batch, t->batch_stride}, {rows, t->row_stride}, {heads, t->head_stride}};
  std::sort(d, d + 3, [](const auto& a, const auto& b) { return a.stride < b.stride; });
  __int128 span = dim;
  for (const auto& x : d) {
    if (x.n == 1) continue;
    if (x.stride < span) return false;
    span += (__int128)(x.n - 1) * x.stride;
  }
  return true;
}

// Whether output `o` starts where `t` does, unless it may be `t` itself and is.
struct Clash {
  int64_t batch, rows, heads;
  bool operator()(const qlora_heads_t* o, const qlora_heads_t* t, bool itself = false) const {
    return o->data == t->data &&
           !(itself && (batch == 1 || o->batch_stride == t->batch_stride) &&
             (rows == 1 || o->row_stride == t->row_stride) &&
             (heads == 1 || o->head_stride == t->head_stride));
  }
};

inline AttnView view(const qlora_heads_t* t) {
  return AttnView{t->data, t->batch_stride, t->row_stride, t->head_stride};
}

AttnArgs attn_args(const qlora_attention_t* a) {
  AttnArgs r{};
  r.cu_q = a->cu_seqlens_q;
  r.cu_k = a->cu_seqlens_k;
  r.nseq = (int)a->n_seq;
  r.Sq = a->q_rows;
  r.Sk = a->k_rows;
  r.H = a->heads;
  r.Hkv = a->kv_heads;
  r.D = a->head_dim;
  r.scale = a->scale;
  r.causal = a->causal != 0;
  return r;
}

// Rows of the statistics (lse, delta): one per query and head.
inline int64_t stat_rows(const qlora_attention_t* a) {
  return a->q_rows * a->heads * (a->cu_seqlens_q ? 1 : a->n_seq);
}

// ---- norms ----

int32_t norm_ok(int64_t rows, int64_t width, int32_t x_type) {
  if (!type_ok(x_type)) return QLORA_ERR_UNSUPPORTED;
  if (rows < 0 || rows >= kMaxRows || width < 1) return QLORA_ERR_INVALID;
  if (width > norm_max_width(x_type)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

// ---- clipping ----

constexpr int64_t kMaxTensors = (int64_t)1 << 20;

int32_t clip(int64_t n, const void* const* grads, const int64_t* sizes, const int32_t* types,
             bool scale, float max_norm, void* const* out, float* norm, void* ws, size_t ws_bytes,
             hipStream_t stream) {
  if (n < 0 || n > kMaxTensors || !norm || !aligned(norm, 4)) return QLORA_ERR_INVALID;
  if (n > 0 && (!grads || !sizes || !types)) return QLORA_ERR_INVALID;
  if (scale && !(max_norm >= 0.0f)) return QLORA_ERR_INVALID;
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (!type_ok(types[i])) return QLORA_ERR_UNSUPPORTED;
    if (sizes[i] < 0 || sizes[i] > ((int64_t)1 << 44)) return QLORA_ERR_INVALID;
    total += sizes[i];
    if (total > ((int64_t)1 << 44)) return QLORA_ERR_INVALID;
    if (sizes[i] == 0) continue;
    if (!grads[i] || !aligned(grads[i], type_bytes(types[i]))) return QLORA_ERR_INVALID;
    if (out && (!out[i] || !aligned(out[i], type_bytes(types[i])))) return QLORA_ERR_INVALID;
  }
  if (!ws || !aligned(ws, 16)) return QLORA_ERR_INVALID;
  if (ws_bytes < qlora_clip_workspace_size(n)) return QLORA_ERR_WORKSPACE;
  ClipArgs a{};
  a.n = n;
  a.grads = grads;
  a.sizes = sizes;
  a.types = types;
  a.out = out;
  a.scale = scale;
  a.max_norm = max_norm;
  a.norm = norm;
  a.part = static_cast<double*>(ws);
  return launch_status(launch_clip(a, stream));
}

}  // namespace

extern "C" {

int32_t qlora_attention_fwd(const qlora_attention_t* a, const qlora_heads_t* q,
                            const qlora_heads_t* k, const qlora_heads_t* v,
                            const qlora_heads_t* o, float* lse, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  const int32_t ok = attn_ok(a);
  if (ok != QLORA_OK) return ok;
  const int64_t nq = stat_rows(a), nk = a->cu_seqlens_q || a->n_seq > 0 ? a->k_rows : 0;
  if (!view_ok(q, nq) || !view_ok(o, nq) || !view_ok(k, nk) || !view_ok(v, nk))
    return QLORA_ERR_INVALID;
  if (nq == 0) return QLORA_OK;
  if (!lse || !aligned(lse, 4)) return QLORA_ERR_INVALID;
  AttnArgs r = attn_args(a);
  const size_t need = (size_t)attn_fwd_workspace(r) * 4;
  if (need > 0 && (!ws || !aligned(ws, 16))) return QLORA_ERR_INVALID;
  if (ws_bytes < need) return QLORA_ERR_WORKSPACE;
  const int64_t nb = a->cu_seqlens_q ? 1 : a->n_seq;
  if (!rows_apart(o, nb, a->q_rows, a->heads, a->head_dim)) return QLORA_ERR_INVALID;
  // a workgroup reads its queries before it, or the join, writes their outputs
  const Clash clash{nb, a->q_rows, a->heads};
  if (clash(o, q, true) || (nk > 0 && (clash(o, k) || clash(o, v))))
    return QLORA_ERR_INVALID;
  r.q = view(q);
  r.k = view(k);
  r.v = view(v);
  r.o = view(o);
  r.lse = lse;
  return launch_status(launch_attn_fwd(r, static_cast<float*>(ws), stream));
}

size_t qlora_attention_fwd_workspace_size(const qlora_attention_t* a) {
  return attn_ok(a) == QLORA_OK ? (size_t)attn_fwd_workspace(attn_args(a)) * 4 : 0;
}

size_t qlora_attention_bwd_workspace_size(const qlora_attention_t* a) {
  return attn_ok(a) == QLORA_OK ? (size_t)attn_bwd_workspace(attn_args(a)) * 4 : 0;
}

int32_t qlora_attention_bwd(const qlora_attention_t* a, const qlora_heads_t* q,
                            const qlora_heads_t* k, const qlora_heads_t* v,
                            const qlora_heads_t* o, const float* lse,
                            const qlora_heads_t* dout, const qlora_heads_t* dq,
                            const qlora_heads_t* dk, const qlora_heads_t* dv, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  const int32_t ok = attn_ok(a);
  if (ok != QLORA_OK) return ok;
  const int64_t nq = stat_rows(a), nk = a->cu_seqlens_q || a->n_seq > 0 ? a->k_rows : 0;
  if (!view_ok(q, nq) || !view_ok(o, nq) || !view_ok(dout, nq) || !view_ok(dq, nq) ||
      !view_ok(k, nk) || !view_ok(v, nk) || !view_ok(dk, nk) || !view_ok(dv, nk))
    return QLORA_ERR_INVALID;
  if (nq == 0 && nk == 0) return QLORA_OK;
  if (nq > 0 && (!lse || !aligned(lse, 4))) return QLORA_ERR_INVALID;
  AttnArgs r = attn_args(a);
  const size_t need = (size_t)attn_bwd_workspace(r) * 4;
  if (need > 0 && (!ws || !aligned(ws, 16))) return QLORA_ERR_INVALID;
  if (ws_bytes < need) return QLORA_ERR_WORKSPACE;
  const int64_t nb = a->cu_seqlens_q ? 1 : a->n_seq;
  if (!rows_apart(dq, nb, a->q_rows, a->heads, a->head_dim) ||
      !rows_apart(dk, nb, a->k_rows, a->kv_heads, a->head_dim) ||
      !rows_apart(dv, nb, a->k_rows, a->kv_heads, a->head_dim))
    return QLORA_ERR_INVALID;
  // q and dout are read again after dq is written; o is not, and a workgroup
  // reads its keys and values before it, or the join, writes their gradients
  const Clash queries{nb, a->q_rows, a->heads}, keys{nb, a->k_rows, a->kv_heads};
  if (nq > 0 && (queries(dq, q) || queries(dq, dout) || queries(dq, o, true)))
    return QLORA_ERR_INVALID;
  if (nk > 0 && (keys(dk, k, true) || keys(dk, v) || keys(dv, v, true) || keys(dv, k) ||
                 keys(dk, dv)))
    return QLORA_ERR_INVALID;
  if (nq > 0 && nk > 0) {
    if (queries(dq, k) || queries(dq, v)) return QLORA_ERR_INVALID;
    for (const qlora_heads_t* t : {dk, dv})
      if (keys(t, q) || keys(t, dout) || keys(t, o) || keys(t, dq)) return QLORA_ERR_INVALID;
  }
  r.q = view(q);
  r.k = view(k);
  r.v = view(v);
  r.o = view(o);
  r.dout = view(dout);
  r.dq = view(dq);
  r.dk = view(dk);
  r.dv = view(dv);
  r.lse = const_cast<float*>(lse);
  return launch_status(launch_attn_bwd(r, static_cast<float*>(ws), stream));
}

int32_t qlora_norm_fwd(const void* x, int64_t rows, int64_t width, int32_t x_type,
                       const void* weight, const void* bias, int32_t w_type, float eps,
                       int32_t rms, void* y, float* mean, float* rstd, hipStream_t stream) {
  const int32_t ok = norm_ok(rows, width, x_type);
  if (ok != QLORA_OK) return ok;
  if (!type_ok(w_type)) return QLORA_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || !isfinite(eps)) return QLORA_ERR_INVALID;
  if (!weight || !aligned(weight, type_bytes(w_type)) || !aligned(bias, type_bytes(w_type)))
    return QLORA_ERR_INVALID;
  if (rows == 0) return QLORA_OK;
  if (!x || !y || !rstd || (!rms && !mean) || !aligned(x, type_bytes(x_type)) ||
      !aligned(y, type_bytes(x_type)) || !aligned(rstd, 4) || !aligned(mean, 4))
    return QLORA_ERR_INVALID;
  return launch_status(launch_norm_fwd(
      NormArgs{x, rows, width, x_type, weight, bias, w_type, eps, rms != 0, y, mean, rstd},
      stream));
}

size_t qlora_norm_bwd_workspace_size(int64_t rows, int64_t width, int32_t x_type) {
  if (norm_ok(rows, width, x_type) != QLORA_OK) return 0;
  return (size_t)norm_bwd_groups(rows, width, x_type) * (size_t)width * 8;
}

int32_t qlora_norm_bwd(const void* dy, const void* x, int64_t rows, int64_t width,
                       int32_t x_type, const void* weight, int32_t w_type, int32_t rms,
                       const float* mean, const float* rstd, void* dx, void* dweight,
                       void* dbias, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int32_t ok = norm_ok(rows, width, x_type);
  if (ok != QLORA_OK) return ok;
  if (!type_ok(w_type)) return QLORA_ERR_UNSUPPORTED;
  const uintptr_t ax = type_bytes(x_type), aw = type_bytes(w_type);
  if (!weight || !aligned(weight, aw) || !aligned(dweight, aw) || !aligned(dbias, aw))
    return QLORA_ERR_INVALID;
  if (rows > 0) {
    if (!dy || !x || !rstd || (!rms && !mean) || !aligned(dy, ax) || !aligned(x, ax) ||
        !aligned(dx, ax) || !aligned(rstd, 4) || !aligned(mean, 4))
      return QLORA_ERR_INVALID;
    if (dweight || dbias) {
      if (!ws || !aligned(ws, 16)) return QLORA_ERR_INVALID;
      if (ws_bytes < qlora_norm_bwd_workspace_size(rows, width, x_type))
        return QLORA_ERR_WORKSPACE;
    }
  }
  return launch_status(launch_norm_bwd(
      NormBwdArgs{dy, x, rows, width, x_type, weight, w_type, rms != 0, mean, rstd, dx, dweight,
                  dbias, static_cast<float*>(ws)},
      stream));
}

size_t qlora_clip_workspace_size(int64_t n) {
  if (n < 0 || n > kMaxTensors) return 0;
  const int64_t launches = (n + kClipNormTable - 1) / kClipNormTable;
  return (size_t)(launches > 0 ? launches : 1) * kClipGrid * sizeof(double);
}

int32_t qlora_clip_grad_norm(int64_t n, const void* const* grads, const int64_t* sizes,
                             const int32_t* types, float max_norm, void* const* out,
                             float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  return clip(n, grads, sizes, types, true, max_norm, out, norm, ws, ws_bytes, stream);
}

int32_t qlora_grad_norm(int64_t n, const void* const* grads, const int64_t* sizes,
                        const int32_t* types, float* norm, void* ws, size_t ws_bytes,
                        hipStream_t stream) {
  return clip(n, grads, sizes, types, false, 0.0f, nullptr, norm, ws, ws_bytes, stream);
}

int32_t qlora_rope(const qlora_rope_t* a, const qlora_heads_t* q, const qlora_heads_t* k,
                   const qlora_heads_t* q_out, const qlora_heads_t* k_out, hipStream_t stream) {
  if (!a || a->n_seq < 0 || a->n_seq >= kMaxRows || a->rows < 0 || a->rows >= kMaxRows ||
      a->q_heads < 1 || a->k_heads < 0 || a->q_heads > (1 << 20) || a->k_heads > (1 << 20) ||
      a->head_dim < 1 || a->rot < 2 || a->rot % 2 != 0 || a->rot > a->head_dim ||
      !isfinite(a->scale))
    return QLORA_ERR_INVALID;
  if (a->head_dim > QLORA_ROPE_MAX_DIM || a->head_dim % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  if (!aligned(a->cu_seqlens, 4)) return QLORA_ERR_INVALID;
  if (a->positions &&
      ((a->position_bytes != 4 && a->position_bytes != 8) ||
       !aligned(a->positions, a->position_bytes) || a->position_batch_stride < 0 ||
       a->position_row_stride < 0))
    return QLORA_ERR_INVALID;
  const int64_t nb = a->cu_seqlens ? 1 : a->n_seq;
  const int64_t tokens = nb * a->rows;
  const bool keys = a->k_heads > 0;
  if (!view_ok(q, tokens) || !view_ok(q_out, tokens) ||
      (keys && (!view_ok(k, tokens) || !view_ok(k_out, tokens))))
    return QLORA_ERR_INVALID;
  if (tokens == 0) return QLORA_OK;
  if (!a->inv_freq || !aligned(a->inv_freq, 8)) return QLORA_ERR_INVALID;
  if (!rows_apart(q_out, nb, a->rows, a->q_heads, a->head_dim) ||
      (keys && !rows_apart(k_out, nb, a->rows, a->k_heads, a->head_dim)))
    return QLORA_ERR_INVALID;
  const Clash qs{nb, a->rows, a->q_heads}, ks{nb, a->rows, a->k_heads};
  if (qs(q_out, q, true)) return QLORA_ERR_INVALID;
  if (keys && (ks(k_out, k, true) || qs(q_out, k) || ks(k_out, q) || qs(q_out, k_out)))
    return QLORA_ERR_INVALID;
  RopeArgs r{};
  r.q = view(q);
  r.qo = view(q_out);
  if (keys) {
    r.k = view(k);
    r.ko = view(k_out);
  }
  r.tokens = tokens;
  r.rows = a->rows;
  r.cu = a->positions ? nullptr : a->cu_seqlens;
  r.nseq = (int)a->n_seq;
  r.pos = a->positions;
  r.pos_sb = a->position_batch_stride;
  r.pos_st = a->position_row_stride;
  r.pos64 = a->position_bytes == 8;
  r.freq = a->inv_freq;
  r.H = a->q_heads;
  r.Hk = a->k_heads;
  r.D = a->head_dim;
  r.rot = a->rot;
  r.interleaved = a->interleaved != 0;
  r.inverse = a->inverse != 0;
  r.scale = a->scale;
  return launch_status(launch_rope(r, stream));
}

static_assert(kAdamBlock == QLORA_ADAMW_BLOCK, "block of the optimizer's states");

int64_t qlora_adamw_blocks(int64_t n, const int64_t* sizes) {
  if (n < 0 || n > kMaxTensors || (n > 0 && !sizes)) return -1;
  const int64_t most = ((int64_t)1 << 31) - 1;
  int64_t blocks = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (sizes[i] < 0 || sizes[i] > most * kAdamBlock) return -1;
    blocks += (sizes[i] + kAdamBlock - 1) / kAdamBlock;
    if (blocks > most) return -1;
  }
  return blocks;
}

int32_t qlora_adamw_step(const qlora_adamw_t* a, hipStream_t stream) {
  if (!a) return QLORA_ERR_INVALID;
  if (a->state_bits != 8 && a->state_bits != 32) return QLORA_ERR_UNSUPPORTED;
  const int64_t blocks = qlora_adamw_blocks(a->n, a->sizes);
  if (blocks < 0) return QLORA_ERR_INVALID;
  const auto beta_ok = [](double b) { return b >= 0.0 && b < 1.0; };
  const auto rate_ok = [](double x) { return x >= 0.0 && isfinite(x); };
  if ((a->step < 1 && !a->step_dev) || !rate_ok(a->lr) || !beta_ok(a->beta1) ||
      !beta_ok(a->beta2) || !rate_ok(a->weight_decay) || !rate_ok(a->eps) ||
      (a->norm && !(a->max_norm >= 0.0)))
    return QLORA_ERR_INVALID;
  if (!aligned(a->lr_dev, 4) || !aligned(a->step_dev, 8) || !aligned(a->norm, 4))
    return QLORA_ERR_INVALID;
  if (a->n > 0 && (!a->params || !a->grads || !a->param_types || !a->grad_types))
    return QLORA_ERR_INVALID;
  for (int64_t i = 0; i < a->n; ++i) {
    if (!type_ok(a->param_types[i]) || !type_ok(a->grad_types[i])) return QLORA_ERR_UNSUPPORTED;
    if (a->sizes[i] == 0 || !a->grads[i]) continue;
    if (!a->params[i] || !aligned(a->params[i], type_bytes(a->param_types[i])) ||
        !aligned(a->grads[i], type_bytes(a->grad_types[i])))
      return QLORA_ERR_INVALID;
    if (a->copies && !aligned(a->copies[i], 2)) return QLORA_ERR_INVALID;
  }
  if (blocks == 0) return QLORA_OK;
  if (!a->m || !a->v || !aligned(a->m, 16) || !aligned(a->v, 16)) return QLORA_ERR_INVALID;
  if (a->state_bits == 8 &&
      (!a->m_scale || !a->v_scale || !aligned(a->m_scale, 4) || !aligned(a->v_scale, 4)))
    return QLORA_ERR_INVALID;
  if (a->state_blocks < blocks) return QLORA_ERR_WORKSPACE;
  AdamArgs r{};
  r.n = a->n;
  r.params = a->params;
  r.grads = a->grads;
  r.copies = a->copies;
  r.sizes = a->sizes;
  r.p_types = a->param_types;
  r.g_types = a->grad_types;
  r.bits = a->state_bits;
  r.m = a->m;
  r.v = a->v;
  r.ms = a->m_scale;
  r.vs = a->v_scale;
  AdamHyper& h = r.hyper;
  h.lr = a->lr;
  h.beta1 = a->beta1;
  h.beta2 = a->beta2;
  h.decay = a->weight_decay;
  if (!a->step_dev) {
    h.bc1 = 1.0 - pow(a->beta1, (double)a->step);
    h.bc2 = 1.0 - pow(a->beta2, (double)a->step);
  }
  h.log_beta1 = log(a->beta1);
  h.log_beta2 = log(a->beta2);
  h.lr_dev = a->lr_dev;
  h.step_dev = a->step_dev;
  h.norm = a->norm;
  h.max_norm = a->max_norm;
  h.eps = a->eps;
  return launch_status(launch_adamw(r, stream));
}

int32_t qlora_adamw_values(const void* m, const void* v, const float* m_scale,
                           const float* v_scale, int64_t blocks, float* m_out, float* v_out,
                           hipStream_t stream) {
  if (blocks < 0 || blocks >= (int64_t)1 << 31) return QLORA_ERR_INVALID;
  if (blocks == 0) return QLORA_OK;
  if (!m || !v || !m_scale || !v_scale || !m_out || !v_out || !aligned(m, 16) || !aligned(v, 16) ||
      !aligned(m_scale, 4) || !aligned(v_scale, 4) || !aligned(m_out, 16) || !aligned(v_out, 16))
    return QLORA_ERR_INVALID;
  return launch_status(launch_adamw_values(m, v, m_scale, v_scale, blocks, m_out, v_out, stream));
}

}  // extern "C"
