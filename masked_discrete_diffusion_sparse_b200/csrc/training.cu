// C ABI of the training form's ends: the LM head's loss, RMSNorm and the embedding, each with its
// gradient.  No handle: argument checks, workspace sizes and launches only.
#include <algorithm>

#include "ends.h"
#include "head.h"
#include "smdm.h"

using namespace smdm;

namespace {

constexpr int kMaxRows = 1 << 24, kMaxWidth = 1 << 16, kMaxVocab = 1 << 24;

bool is_dtype(int t) { return t == SMDM_F32 || t == SMDM_BF16; }
size_t size_of(int t) { return t == SMDM_F32 ? 4 : 2; }
bool on_boundary(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// fp32 or 32-bit integer tensors (a null one lies on every boundary).
template <typename... P>
bool on_words(const P*... p) { return (on_boundary(p, 4) && ...); }

// A workspace of `need` bytes: SMDM_EINVAL for none or a misaligned one, SMDM_ENOMEM for a
// small one.
smdm_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (!ws || !on_boundary(ws, 256)) return SMDM_EINVAL;
  return bytes < need ? SMDM_ENOMEM : SMDM_OK;
}

smdm_status check_head(const smdm_head_shape* s) {
  if (!s || !is_dtype(s->dtype)) return SMDM_EINVAL;
  if (s->rows < 0 || s->rows > kMaxRows || s->d_model < 1 || s->d_model > kMaxWidth ||
      s->vocab < 1 || s->vocab > kMaxVocab)
    return SMDM_ESHAPE;
  if (s->ld_hidden < s->d_model || s->ld_head < s->d_model) return SMDM_EINVAL;
  return SMDM_OK;
}

HeadArgs head_args(const smdm_head_shape* s, const void* hidden, const void* head,
                   const int32_t* target, void* ws, uint32_t* status) {
  HeadArgs a{};
  a.rows = s->rows;
  a.d = s->d_model;
  a.vocab = s->vocab;
  a.f32 = s->dtype == SMDM_F32;
  a.ld_hidden = s->ld_hidden;
  a.ld_head = s->ld_head;
  a.hidden = hidden;
  a.head = head;
  a.target = target;
  a.ws = ws;
  a.status = status;
  return a;
}

// Tensors on their element's boundary; lm_head on 16 bytes where its rows are read in place.
smdm_status check_head_ptrs(const smdm_head_shape* s, const void* hidden, const void* head,
                            const int32_t* target) {
  const size_t es = size_of(s->dtype);
  if (!head || !on_boundary(head, es)) return SMDM_EINVAL;
  if (s->rows > 0 && (!hidden || !target || !on_boundary(hidden, es) || !on_boundary(target, 4)))
    return SMDM_EINVAL;
  if (head_needs_aligned_weight(s->d_model, s->ld_head, s->dtype == SMDM_F32) &&
      !on_boundary(head, 16))
    return SMDM_EINVAL;
  return SMDM_OK;
}

smdm_status check_norm(const smdm_rmsnorm_shape* s) {
  if (!s || !is_dtype(s->x_dtype) || !is_dtype(s->dtype)) return SMDM_EINVAL;
  if (s->rows < 0 || s->rows > kMaxRows || s->d_model < 1 || s->d_model > kMaxNormWidth)
    return SMDM_ESHAPE;
  if (s->ld_x < s->d_model || s->ld_y < s->d_model || !(s->eps >= 0.f)) return SMDM_EINVAL;
  return SMDM_OK;
}

smdm_status check_embed(const smdm_embed_shape* s) {
  if (!s || !is_dtype(s->dtype) || !is_dtype(s->out_dtype)) return SMDM_EINVAL;
  if (s->rows < 0 || s->rows > kMaxRows || s->d_model < 1 || s->d_model > kMaxWidth ||
      s->n_emb < 1 || s->n_emb > kMaxVocab)
    return SMDM_ESHAPE;
  if (s->ld < s->d_model) return SMDM_EINVAL;
  return SMDM_OK;
}

smdm_status done(cudaError_t e) { return e == cudaSuccess ? SMDM_OK : SMDM_ECUDA; }

}  // namespace

extern "C" {

size_t smdm_head_loss_workspace_bytes(const smdm_head_shape* s, int grad) {
  if (check_head(s) != SMDM_OK) return 0;
  return head_workspace_bytes(std::max(1, s->rows), s->d_model, s->vocab, s->dtype == SMDM_F32,
                              grad != 0);
}

smdm_status smdm_head_loss(const smdm_head_shape* s, const void* d_hidden, const void* d_lm_head,
                           const int32_t* d_target, float* d_nll, float* d_lse, void* d_workspace,
                           size_t bytes, uint32_t* d_status, cudaStream_t st) {
  smdm_status r;
  if ((r = check_head(s)) || (r = check_head_ptrs(s, d_hidden, d_lm_head, d_target))) return r;
  if (s->rows > 0 && (!d_nll || !d_lse)) return SMDM_EINVAL;
  if (!on_words(d_nll, d_lse, d_status)) return SMDM_EINVAL;
  if ((r = check_ws(d_workspace, bytes, smdm_head_loss_workspace_bytes(s, 0)))) return r;
  if (s->rows == 0) return SMDM_OK;
  HeadArgs a = head_args(s, d_hidden, d_lm_head, d_target, d_workspace, d_status);
  a.nll = d_nll;
  a.lse_out = d_lse;
  return done(launch_head_loss(a, st));
}

smdm_status smdm_head_loss_grad(const smdm_head_shape* s, const void* d_hidden,
                                const void* d_lm_head, const int32_t* d_target,
                                const float* d_lse, const float* d_grad_nll, void* d_grad_hidden,
                                void* d_grad_lm_head, void* d_workspace, size_t bytes,
                                uint32_t* d_status, cudaStream_t st) {
  smdm_status r;
  if ((r = check_head(s)) || (r = check_head_ptrs(s, d_hidden, d_lm_head, d_target))) return r;
  const size_t es = size_of(s->dtype);
  if ((!d_grad_hidden && !d_grad_lm_head) || !on_boundary(d_grad_hidden, es) ||
      !on_boundary(d_grad_lm_head, es) || (s->rows > 0 && (!d_lse || !d_grad_nll)) ||
      !on_words(d_lse, d_grad_nll, d_status))
    return SMDM_EINVAL;
  if ((r = check_ws(d_workspace, bytes, smdm_head_loss_workspace_bytes(s, 1)))) return r;
  if (s->rows == 0)   // a sum over no rows
    return d_grad_lm_head ? done(cudaMemsetAsync(d_grad_lm_head, 0,
                                                 (size_t)s->vocab * s->d_model * es, st))
                          : SMDM_OK;
  HeadArgs a = head_args(s, d_hidden, d_lm_head, d_target, d_workspace, d_status);
  a.lse = d_lse;
  a.grad_nll = d_grad_nll;
  a.grad_hidden = d_grad_hidden;
  a.grad_head = d_grad_lm_head;
  return done(launch_head_grad(a, st));
}

smdm_status smdm_rmsnorm(const smdm_rmsnorm_shape* s, const void* d_x, const void* d_gain,
                         void* d_y, float* d_rstd, cudaStream_t st) {
  smdm_status r;
  if ((r = check_norm(s))) return r;
  const size_t xs = size_of(s->x_dtype), es = size_of(s->dtype);
  if (!d_gain || !on_boundary(d_gain, es) || !on_words(d_rstd)) return SMDM_EINVAL;
  if (s->rows == 0) return SMDM_OK;
  if (!d_x || !d_y || !on_boundary(d_x, xs) || !on_boundary(d_y, es)) return SMDM_EINVAL;
  RmsArgs a{};
  a.rows = s->rows;
  a.d = s->d_model;
  a.x_f32 = s->x_dtype == SMDM_F32;
  a.f32 = s->dtype == SMDM_F32;
  a.ld_x = s->ld_x;
  a.ld_y = s->ld_y;
  a.eps = s->eps;
  a.x = d_x;
  a.gain = d_gain;
  a.y = d_y;
  a.rstd_out = d_rstd;
  return done(launch_train_rmsnorm(a, st));
}

size_t smdm_rmsnorm_grad_workspace_bytes(const smdm_rmsnorm_shape* s) {
  if (check_norm(s) != SMDM_OK) return 0;
  return rmsnorm_grad_bytes(std::max(1, s->rows), s->d_model);
}

smdm_status smdm_rmsnorm_grad(const smdm_rmsnorm_shape* s, const void* d_x, const void* d_gain,
                              const float* d_rstd, const void* d_grad_y, const void* d_grad_add,
                              void* d_grad_x, void* d_grad_gain, void* d_workspace, size_t bytes,
                              cudaStream_t st) {
  smdm_status r;
  if ((r = check_norm(s))) return r;
  const size_t xs = size_of(s->x_dtype), es = size_of(s->dtype);
  if (!d_gain || !d_grad_gain || !on_boundary(d_gain, es) || !on_boundary(d_grad_gain, es) ||
      !on_words(d_rstd))
    return SMDM_EINVAL;
  if (s->rows > 0 && (!d_x || !d_rstd || !d_grad_y || !d_grad_x || !on_boundary(d_x, xs) ||
                      !on_boundary(d_grad_y, es) || !on_boundary(d_grad_add, xs) ||
                      !on_boundary(d_grad_x, xs)))
    return SMDM_EINVAL;
  if ((r = check_ws(d_workspace, bytes, smdm_rmsnorm_grad_workspace_bytes(s)))) return r;
  if (s->rows == 0) return done(cudaMemsetAsync(d_grad_gain, 0, (size_t)s->d_model * es, st));
  RmsArgs a{};
  a.rows = s->rows;
  a.d = s->d_model;
  a.x_f32 = s->x_dtype == SMDM_F32;
  a.f32 = s->dtype == SMDM_F32;
  a.ld_x = s->ld_x;
  a.ld_y = s->ld_y;
  a.eps = s->eps;
  a.x = d_x;
  a.gain = d_gain;
  a.rstd = d_rstd;
  a.grad_y = d_grad_y;
  a.add = d_grad_add;
  a.grad_x = d_grad_x;
  a.grad_gain = d_grad_gain;
  a.ws = static_cast<float*>(d_workspace);
  return done(launch_train_rmsnorm_grad(a, st));
}

smdm_status smdm_embed(const smdm_embed_shape* s, const int32_t* d_ids, const void* d_table,
                       void* d_out, uint32_t* d_status, cudaStream_t st) {
  smdm_status r;
  if ((r = check_embed(s))) return r;
  if (!d_table || !on_boundary(d_table, size_of(s->dtype)) || !on_words(d_ids, d_status))
    return SMDM_EINVAL;
  if (s->rows == 0) return SMDM_OK;
  if (!d_ids || !d_out || !on_boundary(d_out, size_of(s->out_dtype))) return SMDM_EINVAL;
  EmbedArgs a{};
  a.rows = s->rows;
  a.d = s->d_model;
  a.n_emb = s->n_emb;
  a.f32 = s->dtype == SMDM_F32;
  a.out_f32 = s->out_dtype == SMDM_F32;
  a.ld_table = s->ld;
  a.scale = s->scale;
  a.ids = d_ids;
  a.table = d_table;
  a.out = d_out;
  a.status = d_status;
  return done(launch_embed(a, st));
}

size_t smdm_embed_grad_workspace_bytes(const smdm_embed_shape* s) {
  if (check_embed(s) != SMDM_OK) return 0;
  return embed_grad_bytes(std::max(1, s->rows), s->d_model, s->n_emb);
}

smdm_status smdm_embed_grad(const smdm_embed_shape* s, const int32_t* d_ids,
                            const void* d_grad_out, void* d_grad_table, void* d_workspace,
                            size_t bytes, uint32_t* d_status, cudaStream_t st) {
  smdm_status r;
  if ((r = check_embed(s))) return r;
  const size_t es = size_of(s->dtype);
  if (!d_grad_table || !on_boundary(d_grad_table, es) || !on_words(d_ids, d_status))
    return SMDM_EINVAL;
  if (s->rows > 0 && (!d_ids || !d_grad_out || !on_boundary(d_grad_out, size_of(s->out_dtype))))
    return SMDM_EINVAL;
  if ((r = check_ws(d_workspace, bytes, smdm_embed_grad_workspace_bytes(s)))) return r;
  if (s->rows == 0)
    return done(cudaMemsetAsync(d_grad_table, 0, (size_t)s->n_emb * s->d_model * es, st));
  EmbedArgs a{};
  a.rows = s->rows;
  a.d = s->d_model;
  a.n_emb = s->n_emb;
  a.f32 = s->dtype == SMDM_F32;
  a.out_f32 = s->out_dtype == SMDM_F32;
  a.ld_grad = s->ld;
  a.scale = s->scale;
  a.ids = d_ids;
  a.grad_out = d_grad_out;
  a.grad_table = d_grad_table;
  a.ws = d_workspace;
  a.status = d_status;
  return done(launch_embed_grad(a, st));
}

}  // extern "C"
