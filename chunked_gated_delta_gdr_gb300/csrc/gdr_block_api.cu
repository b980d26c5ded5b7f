// gdr_block_api.cu -- the extern "C" entry points of a hybrid block's operators: validation of
// descriptors, then stream-ordered launches.
#include "gdr_block.cuh"
#include "gdr_mix_desc.cuh"

using namespace gdr;

namespace {

Heads heads(const Desc &d) { return Heads{d.p, d.stride[0], d.stride[1]}; }
Pages pages_of(const Desc &d) { return Pages{d.p, d.stride[0], d.stride[1], d.stride[2]}; }

// Written tensors whose dimensions may lie in any order: no two elements at one address.
int distinct(const Desc &d) {
  int at[4] = {0, 1, 2, 3};
  for (int i = 0; i < d.ndim; ++i)
    if (d.shape[i] == 0) return GDR_OK;
  for (int i = 1; i < d.ndim; ++i)
    for (int j = i; j > 0 && d.stride[at[j]] < d.stride[at[j - 1]]; --j) {
      const int t = at[j];
      at[j] = at[j - 1];
      at[j - 1] = t;
    }
  int64_t extent = 1;
  for (int i = 0; i < d.ndim; ++i) {
    const int64_t n = d.shape[at[i]], s = d.stride[at[i]];
    if (n <= 1) continue;
    if (s < extent) return GDR_ERR_STRIDE;
    extent += s * (n - 1);
  }
  return GDR_OK;
}

int flag(int32_t v) { return v == 0 || v == 1 ? GDR_OK : GDR_ERR_OPTION; }

// ------------------------------------------------------------------ gated linear recurrence

int read_rec(const gdr_tensor_t *x, const gdr_tensor_t *r, const gdr_tensor_t *i,
             const gdr_tensor_t *A, int32_t normalize, RecArgs *a) {
  Desc d;
  GDR_TRY(read_first(x, 2, &d, &a->f32));
  const int64_t T = d.shape[0], Dm = d.shape[1];
  if (T > kMost || Dm > kMost || Dm < 1) return GDR_ERR_SHAPE;
  a->T = (int32_t)T;
  a->D = (int32_t)Dm;
  a->x = mat(d);
  GDR_TRY(read_act(r, 2, &d, a->f32));
  GDR_TRY(shaped(d, T, Dm));
  a->r = mat(d);
  a->i = Mat{nullptr, 0};
  if (i) {
    GDR_TRY(read_act(i, 2, &d, a->f32));
    GDR_TRY(shaped(d, T, Dm));
    a->i = mat(d);
  }
  if (!A) return GDR_ERR_NULL;
  GDR_TRY(read_param(A, &a->A, Dm));
  GDR_TRY(flag(normalize));
  a->normalize = normalize;
  return GDR_OK;
}

int read_written(const gdr_tensor_t *t, const RecArgs &a, Mat *m) {
  Desc d;
  GDR_TRY(read_act(t, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.D));
  GDR_TRY(apart(d));
  *m = mat(d);
  return GDR_OK;
}

int read_rec_states(const gdr_tensor_t *t, const float **p, int64_t n, int64_t D) {
  if (t && t->ndim == 2 && t->shape[0] != n) return GDR_ERR_NSEQ;
  return read_param(t, p, n, D);
}

int64_t checkpoint_rows(int64_t T) { return (T + kRecEvery - 1) / kRecEvery; }

// ------------------------------------------------------------------ norms

int read_weight(const gdr_tensor_t *t, mix::Param *w, int64_t n) {
  *w = mix::Param{nullptr, 0};
  if (!t) return GDR_OK;
  Desc d;
  bool f32;
  GDR_TRY(read_first(t, 1, &d, &f32));
  GDR_TRY(shaped(d, n));
  *w = mix::Param{d.p, !f32};
  return GDR_OK;
}

int read_heads(const gdr_tensor_t *t, const GatedArgs &a, bool written, Heads *h) {
  Desc d;
  GDR_TRY(read_act(t, 3, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.H, a.d));
  if (written) GDR_TRY(apart(d));
  *h = heads(d);
  return GDR_OK;
}

int read_gated(const gdr_tensor_t *x, const gdr_tensor_t *z, const gdr_tensor_t *weight,
               int32_t activation, float eps, GatedArgs *a) {
  Desc d;
  GDR_TRY(read_first(x, 3, &d, &a->f32));
  if (d.shape[0] > kMost || d.shape[1] > 0xffff) return GDR_ERR_SHAPE;
  if (d.shape[2] < 1 || d.shape[2] > 1024) return GDR_ERR_DIM;
  a->T = (int32_t)d.shape[0];
  a->H = (int32_t)d.shape[1];
  a->d = (int32_t)d.shape[2];
  a->x = heads(d);
  GDR_TRY(read_heads(z, *a, false, &a->z));
  GDR_TRY(read_weight(weight, &a->w, a->d));
  if (activation != GDR_ACT_SILU && activation != GDR_ACT_SIGMOID) return GDR_ERR_OPTION;
  if (!(eps >= 0.f)) return GDR_ERR_OPTION;
  a->silu = activation == GDR_ACT_SILU;
  a->eps = eps;
  return GDR_OK;
}

int read_cols(const gdr_tensor_t *t, const ResidArgs &a, bool f32, bool written, Mat *m) {
  Desc d;
  GDR_TRY(read_act(t, 2, &d, f32));
  GDR_TRY(shaped(d, a.T, a.C));
  if (written) GDR_TRY(apart(d));
  *m = mat(d);
  return GDR_OK;
}

// `other`: the tensor that says in which type h is where there is no residual (null: x's type)
int read_resid(const gdr_tensor_t *x, const gdr_tensor_t *residual, const gdr_tensor_t *weight,
               int32_t post, const gdr_tensor_t *post_weight, const gdr_tensor_t *gate, float scale,
               float eps, const gdr_tensor_t *other, ResidArgs *a) {
  Desc d;
  GDR_TRY(read_first(x, 2, &d, &a->f32));
  if (d.shape[0] > kMost) return GDR_ERR_SHAPE;
  if (d.shape[1] < 1 || d.shape[1] > 16384) return GDR_ERR_DIM;
  a->T = (int32_t)d.shape[0];
  a->C = (int32_t)d.shape[1];
  a->x = mat(d);
  const gdr_tensor_t *type = residual ? residual : other;
  a->rf32 = a->f32;
  if (type) {
    if (type->dtype != GDR_BF16 && type->dtype != GDR_F32) return GDR_ERR_DTYPE;
    a->rf32 = type->dtype == GDR_F32;
    if (a->f32 && !a->rf32) return GDR_ERR_DTYPE;
  }
  a->res = Mat{nullptr, 0};
  if (residual) GDR_TRY(read_cols(residual, *a, a->rf32, false, &a->res));
  GDR_TRY(read_weight(weight, &a->w, a->C));
  GDR_TRY(read_weight(post_weight, &a->wp, a->C));
  GDR_TRY(read_weight(gate, &a->g, a->C));
  GDR_TRY(flag(post));
  if (post_weight && !post) return GDR_ERR_OPTION;
  if (!(eps >= 0.f)) return GDR_ERR_OPTION;
  a->post = post;
  a->scale = scale;
  a->eps = eps;
  return GDR_OK;
}

// ------------------------------------------------------------------ paged cache

int read_cache(const gdr_tensor_t *t, bool f32, bool written, Desc *d) {
  GDR_TRY(read_act(t, 4, d, f32));
  if (d->shape[0] > kMost || d->shape[1] < 1 || d->shape[1] > kMost || d->shape[2] < 1 ||
      d->shape[2] > 0xffff)
    return GDR_ERR_SHAPE;
  if (written) GDR_TRY(distinct(*d));
  return GDR_OK;
}
int alike(const Desc &a, const Desc &b) {
  for (int i = 0; i < a.ndim; ++i)
    if (a.shape[i] != b.shape[i]) return GDR_ERR_SHAPE;
  return GDR_OK;
}
int read_table(const gdr_tensor_t *t, int64_t B, int64_t page, bool written, Desc *d) {
  GDR_TRY(read_desc(t, GDR_I32, 2, d));
  if (d->shape[0] != B || d->shape[1] > kMost || d->shape[1] * page > kMost) return GDR_ERR_SHAPE;
  return written ? apart(*d) : GDR_OK;
}

}  // namespace

extern "C" {

int gdr_rec_fwd(const gdr_tensor_t *x, const gdr_tensor_t *r, const gdr_tensor_t *i,
                const gdr_tensor_t *A, int32_t normalize, const gdr_tensor_t *h0,
                const int32_t *cu_seqlens, int32_t n_seq, gdr_tensor_t *y, gdr_tensor_t *ht,
                gdr_tensor_t *checkpoints, cudaStream_t stream) {
  RecArgs a{};
  GDR_TRY(read_rec(x, r, i, A, normalize, &a));
  GDR_TRY(segments(cu_seqlens, n_seq));
  a.cu = cu_seqlens;
  a.n_seq = n_seq;
  GDR_TRY(read_rec_states(h0, &a.h0, n_seq, a.D));
  GDR_TRY(read_rec_states(ht, const_cast<const float **>(&a.ht), n_seq, a.D));
  GDR_TRY(read_written(y, a, &a.y));
  GDR_TRY(read_param(checkpoints, &a.kept, checkpoint_rows(a.T), a.D));
  GDR_TRY(device_ok());
  return done(launch_rec_fwd(a, stream));
}

int64_t gdr_rec_checkpoint_rows(int64_t T) { return T < 0 || T > kMost ? 0 : checkpoint_rows(T); }

size_t gdr_rec_bwd_workspace_bytes(int64_t T, int32_t D, int32_t n_seq, int32_t has_checkpoints) {
  if (T < 0 || T > kMost || D < 1 || n_seq < 0) return 0;
  return rec_bwd_workspace(T, D, n_seq, has_checkpoints != 0);
}

int gdr_rec_bwd(const gdr_tensor_t *x, const gdr_tensor_t *r, const gdr_tensor_t *i,
                const gdr_tensor_t *A, int32_t normalize, const gdr_tensor_t *h0,
                const int32_t *cu_seqlens, int32_t n_seq, const gdr_tensor_t *checkpoints,
                const gdr_tensor_t *dy, const gdr_tensor_t *dht, gdr_tensor_t *dx, gdr_tensor_t *dr,
                gdr_tensor_t *di, gdr_tensor_t *dA, gdr_tensor_t *dh0, void *workspace,
                size_t workspace_bytes, cudaStream_t stream) {
  RecArgs a{};
  GDR_TRY(read_rec(x, r, i, A, normalize, &a));
  GDR_TRY(segments(cu_seqlens, n_seq));
  a.cu = cu_seqlens;
  a.n_seq = n_seq;
  GDR_TRY(read_rec_states(h0, &a.h0, n_seq, a.D));
  GDR_TRY(read_rec_states(dht, &a.dht, n_seq, a.D));
  GDR_TRY(read_rec_states(dh0, const_cast<const float **>(&a.dh0), n_seq, a.D));
  GDR_TRY(read_param(checkpoints, const_cast<const float **>(&a.kept), checkpoint_rows(a.T), a.D));
  Desc d;
  GDR_TRY(read_act(dy, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.D));
  a.dy = mat(d);
  if (!i != !di) return GDR_ERR_OPTION;
  GDR_TRY(read_written(dx, a, &a.dx));
  GDR_TRY(read_written(dr, a, &a.dr));
  if (di) GDR_TRY(read_written(di, a, &a.di));
  if (!dA) return GDR_ERR_NULL;
  GDR_TRY(read_param(dA, &a.dA, a.D));
  GDR_TRY(device_ok());
  const bool kept = checkpoints != nullptr;
  GDR_TRY(scratch(workspace, workspace_bytes, rec_bwd_workspace(a.T, a.D, n_seq, kept)));
  a.work = workspace;
  return done(launch_rec_bwd(a, kept, stream));
}

int gdr_rec_step(const gdr_tensor_t *x, const gdr_tensor_t *r, const gdr_tensor_t *i,
                 const gdr_tensor_t *A, int32_t normalize, gdr_tensor_t *state,
                 const int32_t *state_indices, gdr_tensor_t *y, cudaStream_t stream) {
  RecArgs a{};
  GDR_TRY(read_rec(x, r, i, A, normalize, &a));
  Desc s;
  GDR_TRY(read_desc(state, GDR_F32, 2, &s));
  GDR_TRY(shaped(s, s.shape[0], a.D));
  GDR_TRY(packed(s));
  if (s.shape[0] > kMost) return GDR_ERR_SHAPE;
  if (!state_indices && s.shape[0] < a.T) return GDR_ERR_SHAPE;
  GDR_TRY(read_written(y, a, &a.y));
  GDR_TRY(device_ok());
  return done(launch_rec_step(a, reinterpret_cast<float *>(s.p), (int32_t)s.shape[0],
                              state_indices, stream));
}

int gdr_gated_norm_fwd(const gdr_tensor_t *x, const gdr_tensor_t *z, const gdr_tensor_t *weight,
                       int32_t activation, float eps, gdr_tensor_t *y, cudaStream_t stream) {
  GatedArgs a{};
  GDR_TRY(read_gated(x, z, weight, activation, eps, &a));
  GDR_TRY(read_heads(y, a, true, &a.y));
  GDR_TRY(device_ok());
  return done(launch_gated_fwd(a, stream));
}

size_t gdr_gated_norm_bwd_workspace_bytes(int64_t T, int32_t H, int32_t d) {
  if (T < 0 || T > kMost || H < 0 || H > 0xffff || d < 1 || d > 1024) return 0;
  return gated_bwd_workspace(T, H, d);
}

int gdr_gated_norm_bwd(const gdr_tensor_t *x, const gdr_tensor_t *z, const gdr_tensor_t *weight,
                       int32_t activation, float eps, const gdr_tensor_t *dy, gdr_tensor_t *dx,
                       gdr_tensor_t *dz, gdr_tensor_t *dweight, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  GatedArgs a{};
  GDR_TRY(read_gated(x, z, weight, activation, eps, &a));
  GDR_TRY(read_heads(dy, a, false, &a.dy));
  GDR_TRY(read_heads(dx, a, true, &a.dx));
  GDR_TRY(read_heads(dz, a, true, &a.dz));
  GDR_TRY(read_param(dweight, &a.dw, a.d));
  GDR_TRY(device_ok());
  GDR_TRY(scratch(workspace, workspace_bytes, gated_bwd_workspace(a.T, a.H, a.d)));
  a.work = workspace;
  return done(launch_gated_bwd(a, stream));
}

int gdr_residual_norm_fwd(const gdr_tensor_t *x, const gdr_tensor_t *residual,
                          const gdr_tensor_t *weight, int32_t post, const gdr_tensor_t *post_weight,
                          const gdr_tensor_t *gate, float scale, float eps, gdr_tensor_t *y,
                          gdr_tensor_t *h, cudaStream_t stream) {
  ResidArgs a{};
  GDR_TRY(read_resid(x, residual, weight, post, post_weight, gate, scale, eps, h, &a));
  GDR_TRY(read_cols(y, a, a.f32, true, &a.y));
  a.h = Mat{nullptr, 0};
  if (h) GDR_TRY(read_cols(h, a, a.rf32, true, &a.h));
  GDR_TRY(device_ok());
  return done(launch_resid_fwd(a, stream));
}

size_t gdr_residual_norm_bwd_workspace_bytes(int64_t T, int32_t C) {
  if (T < 0 || T > kMost || C < 1 || C > 16384) return 0;
  return resid_bwd_workspace(T, C);
}

int gdr_residual_norm_bwd(const gdr_tensor_t *x, const gdr_tensor_t *residual,
                          const gdr_tensor_t *weight, int32_t post, const gdr_tensor_t *post_weight,
                          const gdr_tensor_t *gate, float scale, float eps, const gdr_tensor_t *dy,
                          const gdr_tensor_t *dh, gdr_tensor_t *dx, gdr_tensor_t *dresidual,
                          gdr_tensor_t *dweight, gdr_tensor_t *dpost_weight, gdr_tensor_t *dgate,
                          void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  ResidArgs a{};
  GDR_TRY(read_resid(x, residual, weight, post, post_weight, gate, scale, eps,
                     dh ? dh : dresidual, &a));
  GDR_TRY(read_cols(dy, a, a.f32, false, &a.dy));
  a.dh = a.dres = Mat{nullptr, 0};
  if (dh) GDR_TRY(read_cols(dh, a, a.rf32, false, &a.dh));
  GDR_TRY(read_cols(dx, a, a.f32, true, &a.dx));
  if (dresidual) GDR_TRY(read_cols(dresidual, a, a.rf32, true, &a.dres));
  GDR_TRY(read_param(dweight, &a.dw, a.C));
  GDR_TRY(read_param(dpost_weight, &a.dwp, a.C));
  GDR_TRY(read_param(dgate, &a.dg, a.C));
  if (dpost_weight && !post) return GDR_ERR_OPTION;
  GDR_TRY(device_ok());
  GDR_TRY(scratch(workspace, workspace_bytes, resid_bwd_workspace(a.T, a.C)));
  a.work = workspace;
  return done(launch_resid_bwd(a, stream));
}

size_t gdr_attn_step_workspace_bytes(int32_t B, int32_t Hq, int32_t Hk, int32_t d) {
  if (B < 0 || Hq < 1 || Hk < 1 || d < 1 || d > 256) return 0;
  return attn_workspace(B, Hq, Hk, d);
}

int gdr_attn_step(const gdr_tensor_t *q, const gdr_tensor_t *k_cache, const gdr_tensor_t *v_cache,
                  const gdr_tensor_t *block_table, const int32_t *lengths, float scale,
                  int32_t window, gdr_tensor_t *o, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
  AttnArgs a{};
  Desc d, k, v, t;
  GDR_TRY(read_first(q, 3, &d, &a.f32));
  const int64_t B = d.shape[0], Hq = d.shape[1];
  if (d.shape[2] < 1 || d.shape[2] > 256) return GDR_ERR_DIM;
  a.d = (int32_t)d.shape[2];
  a.q = heads(d);
  GDR_TRY(read_cache(k_cache, a.f32, false, &k));
  GDR_TRY(read_cache(v_cache, a.f32, false, &v));
  GDR_TRY(alike(k, v));
  if (k.shape[3] != a.d) return GDR_ERR_SHAPE;
  const int64_t Hk = k.shape[2];
  if (B > kMost || Hq < 1 || Hq > 0xffff || B * Hq > 0x3fffffff) return GDR_ERR_SHAPE;
  if (Hq % Hk != 0) return GDR_ERR_HEADS;
  GDR_TRY(read_table(block_table, B, k.shape[1], false, &t));
  if (!lengths && B > 0) return GDR_ERR_NULL;
  if (window < 0) return GDR_ERR_OPTION;
  a.B = (int32_t)B;
  a.Hq = (int32_t)Hq;
  a.Hk = (int32_t)Hk;
  a.pages = (int32_t)k.shape[0];
  a.page = (int32_t)k.shape[1];
  a.width = (int32_t)t.shape[1];
  a.window = window;
  a.scale = scale;
  a.k = pages_of(k);
  a.v = pages_of(v);
  a.table = reinterpret_cast<const int32_t *>(t.p);
  a.table_st = t.stride[0];
  a.lens = lengths;
  GDR_TRY(read_act(o, 3, &d, a.f32));
  GDR_TRY(shaped(d, B, Hq, a.d));
  GDR_TRY(apart(d));
  a.o = heads(d);
  GDR_TRY(device_ok());
  GDR_TRY(scratch(workspace, workspace_bytes, attn_workspace(a.B, a.Hq, a.Hk, a.d)));
  a.work = workspace;
  return done(launch_attn_step(a, stream));
}

int gdr_cache_plan(const int32_t *lengths, const int32_t *new_tokens, int32_t B,
                   gdr_tensor_t *block_table, const gdr_tensor_t *free_pages, const int32_t *taken,
                   int32_t page_size, int32_t *slots, int32_t *positions, int32_t max_tokens,
                   int32_t *cu_seqlens, int32_t *lengths_out, int32_t *taken_out,
                   cudaStream_t stream) {
  PlanArgs a{};
  Desc t, f;
  if (B < 0 || B > kMost || max_tokens < 0 || max_tokens > kMost || page_size < 1)
    return GDR_ERR_SHAPE;
  if (B > 0 && (!lengths || !new_tokens || !lengths_out)) return GDR_ERR_NULL;
  if (!taken || !taken_out || !cu_seqlens) return GDR_ERR_NULL;
  if (max_tokens > 0 && (!slots || !positions)) return GDR_ERR_NULL;
  GDR_TRY(read_table(block_table, B, page_size, true, &t));
  GDR_TRY(read_desc(free_pages, GDR_I32, 1, &f));
  if (f.shape[0] > kMost) return GDR_ERR_SHAPE;
  GDR_TRY(device_ok());
  a.B = B;
  a.width = (int32_t)t.shape[1];
  a.page = page_size;
  a.nfree = (int32_t)f.shape[0];
  a.most = max_tokens;
  a.lens = lengths;
  a.fresh = new_tokens;
  a.table = reinterpret_cast<int32_t *>(t.p);
  a.table_st = t.stride[0];
  a.free_pages = reinterpret_cast<const int32_t *>(f.p);
  a.taken = taken;
  a.slots = slots;
  a.positions = positions;
  a.cu = cu_seqlens;
  a.lens_out = lengths_out;
  a.taken_out = taken_out;
  return done(launch_cache_plan(a, stream));
}

int gdr_cache_write(const gdr_tensor_t *k, const gdr_tensor_t *v, gdr_tensor_t *k_cache,
                    gdr_tensor_t *v_cache, const int32_t *slots, cudaStream_t stream) {
  WriteArgs a{};
  Desc d, e, kc, vc;
  GDR_TRY(read_first(k, 3, &d, &a.f32));
  GDR_TRY(read_act(v, 3, &e, a.f32));
  GDR_TRY(alike(d, e));
  GDR_TRY(read_cache(k_cache, a.f32, true, &kc));
  GDR_TRY(read_cache(v_cache, a.f32, true, &vc));
  GDR_TRY(alike(kc, vc));
  if (d.shape[2] < 1 || d.shape[2] > 0xffff) return GDR_ERR_DIM;
  if (d.shape[0] > kMost || kc.shape[2] != d.shape[1] || kc.shape[3] != d.shape[2])
    return GDR_ERR_SHAPE;
  if (d.shape[1] * d.shape[2] > kMost) return GDR_ERR_SHAPE;
  if (kc.shape[0] * kc.shape[1] > (int64_t)1 << 31) return GDR_ERR_SHAPE;  // places that no slot names
  if (!slots && d.shape[0] > 0) return GDR_ERR_NULL;
  GDR_TRY(device_ok());
  a.T = (int32_t)d.shape[0];
  a.Hk = (int32_t)d.shape[1];
  a.d = (int32_t)d.shape[2];
  a.pages = (int32_t)kc.shape[0];
  a.page = (int32_t)kc.shape[1];
  a.k = heads(d);
  a.v = heads(e);
  a.kc = pages_of(kc);
  a.vc = pages_of(vc);
  a.slots = slots;
  return done(launch_cache_write(a, stream));
}

}  // extern "C"
