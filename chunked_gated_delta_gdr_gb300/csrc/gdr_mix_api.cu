// gdr_mix_api.cu -- the extern "C" entry points of the token mixer's operators around the delta
// rule: validation of descriptors, then stream-ordered launches.
#include "gdr_mix.cuh"
#include "gdr_mix_desc.cuh"

using namespace gdr;

namespace {

// ------------------------------------------------------------------ convolution

int read_taps(const gdr_tensor_t *weight, const gdr_tensor_t *bias, int64_t C, mix::Param *w,
              mix::Param *b, int32_t *W) {
  Desc d;
  bool f32;
  GDR_TRY(read_first(weight, 2, &d, &f32));
  if (d.shape[0] != C) return GDR_ERR_SHAPE;
  if (d.shape[1] < 2 || d.shape[1] > 4) return GDR_ERR_DIM;
  GDR_TRY(packed(d));
  *w = mix::Param{d.p, !f32};
  *W = (int32_t)d.shape[1];
  *b = mix::Param{nullptr, 0};
  if (bias) {
    GDR_TRY(read_act(bias, 1, &d, f32));
    GDR_TRY(shaped(d, C));
    *b = mix::Param{d.p, !f32};
  }
  return GDR_OK;
}

int read_conv(const gdr_tensor_t *x, const gdr_tensor_t *weight, const gdr_tensor_t *bias,
              const gdr_tensor_t *h0, const int32_t *cu, int32_t n_seq, int32_t activation,
              ConvArgs *a) {
  Desc d;
  GDR_TRY(read_first(x, 2, &d, &a->f32));
  if (d.shape[0] > kMost || d.shape[1] > kMost || d.shape[1] < 1) return GDR_ERR_SHAPE;
  a->T = (int32_t)d.shape[0];
  a->C = (int32_t)d.shape[1];
  a->x = mat(d);
  GDR_TRY(read_taps(weight, bias, a->C, &a->w, &a->b, &a->W));
  if (activation != GDR_ACT_NONE && activation != GDR_ACT_SILU) return GDR_ERR_OPTION;
  a->silu = activation == GDR_ACT_SILU;
  GDR_TRY(segments(cu, n_seq));
  a->cu = cu;
  a->n_seq = n_seq;
  return read_rows(h0, &a->h0, a->f32, n_seq, a->W - 1, a->C);
}

// ------------------------------------------------------------------ state space

int read_ssm(const gdr_tensor_t *x, const gdr_tensor_t *dt, const gdr_tensor_t *A,
             const gdr_tensor_t *B, const gdr_tensor_t *C, const gdr_tensor_t *D,
             const gdr_tensor_t *z, const gdr_tensor_t *dt_bias, int32_t dt_softplus,
             SsmArgs *a) {
  Desc d;
  GDR_TRY(read_first(x, 2, &d, &a->f32));
  const int64_t T = d.shape[0], Dm = d.shape[1];
  if (T > kMost || Dm > kMost || Dm < 1) return GDR_ERR_SHAPE;
  a->T = (int32_t)T;
  a->D = (int32_t)Dm;
  a->x = mat(d);
  GDR_TRY(read_act(dt, 2, &d, a->f32));
  GDR_TRY(shaped(d, T, Dm));
  a->dt = mat(d);
  a->z = Mat{nullptr, 0};
  if (z) {
    GDR_TRY(read_act(z, 2, &d, a->f32));
    GDR_TRY(shaped(d, T, Dm));
    a->z = mat(d);
    // an empty tensor may have no address: nothing of it is read
  }
  Desc b, c;
  GDR_TRY(read_act(B, 3, &b, a->f32));
  GDR_TRY(read_act(C, 3, &c, a->f32));
  if (b.shape[0] != T) return GDR_ERR_SHAPE;
  GDR_TRY(shaped(c, b.shape[0], b.shape[1], b.shape[2]));
  if (b.shape[2] < 1 || b.shape[2] > 64) return GDR_ERR_DIM;
  if (b.shape[1] < 1 || b.shape[1] > Dm) return GDR_ERR_SHAPE;
  if (Dm % b.shape[1] != 0) return GDR_ERR_HEADS;
  a->G = (int32_t)b.shape[1];
  a->N = (int32_t)b.shape[2];
  a->B = b.p;
  a->B_st = b.stride[0];
  a->B_sg = b.stride[1];
  a->C = c.p;
  a->C_st = c.stride[0];
  a->C_sg = c.stride[1];
  if (!A) return GDR_ERR_NULL;
  GDR_TRY(read_param(A, &a->A, Dm, a->N));
  GDR_TRY(read_param(D, &a->Dskip, Dm));
  GDR_TRY(read_param(dt_bias, &a->dt_bias, Dm));
  if (dt_softplus != 0 && dt_softplus != 1) return GDR_ERR_OPTION;
  a->softplus = dt_softplus;
  return GDR_OK;
}

int read_states(const gdr_tensor_t *t, const float **p, int64_t n, int64_t D, int64_t N) {
  if (t && t->ndim == 3 && t->shape[0] != n) return GDR_ERR_NSEQ;
  return read_param(t, p, n, D, N);
}

// ------------------------------------------------------------------ q/k norm

int read_qk(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *qw,
            const gdr_tensor_t *kw, int32_t norm, float eps, const gdr_tensor_t *cos,
            const gdr_tensor_t *sin, const int32_t *positions, int32_t interleaved,
            QkArgs *a) {
  Desc d[2];
  GDR_TRY(read_first(q, 3, &d[0], &a->f32));
  GDR_TRY(read_act(k, 3, &d[1], a->f32));
  a->T = d[0].shape[0];
  if (d[1].shape[0] != a->T || d[1].shape[2] != d[0].shape[2]) return GDR_ERR_SHAPE;
  if (a->T > kMost || d[0].shape[1] > 0xffff || d[1].shape[1] > 0xffff) return GDR_ERR_SHAPE;
  if (d[0].shape[2] < 1 || d[0].shape[2] > 256) return GDR_ERR_DIM;
  a->Hq = (int32_t)d[0].shape[1];
  a->Hk = (int32_t)d[1].shape[1];
  a->d = (int32_t)d[0].shape[2];
  for (int j = 0; j < 2; ++j) {
    a->x[j] = d[j].p;
    a->x_st[j] = d[j].stride[0];
    a->x_sh[j] = d[j].stride[1];
    const gdr_tensor_t *w = j ? kw : qw;
    a->w[j] = mix::Param{nullptr, 0};
    if (w) {
      Desc e;
      bool f32;
      GDR_TRY(read_first(w, 1, &e, &f32));
      GDR_TRY(shaped(e, a->d));
      a->w[j] = mix::Param{e.p, !f32};
    }
  }
  if (norm != GDR_NORM_RMS && norm != GDR_NORM_L2) return GDR_ERR_OPTION;
  if (!(eps >= 0.f)) return GDR_ERR_OPTION;
  if (interleaved != 0 && interleaved != 1) return GDR_ERR_OPTION;
  a->rms = norm == GDR_NORM_RMS;
  a->eps = eps;
  a->interleaved = interleaved;
  a->rot = 0;
  a->places = 0;
  a->cos = a->sin = nullptr;
  a->pos = nullptr;
  if (!cos != !sin) return GDR_ERR_OPTION;
  if (cos) {
    Desc e;
    GDR_TRY(read_desc(cos, GDR_F32, 2, &e));
    if (e.shape[0] < 1 || e.shape[0] > kMost) return GDR_ERR_SHAPE;
    if (e.shape[1] > 128 || 2 * e.shape[1] > a->d) return GDR_ERR_DIM;
    GDR_TRY(packed(e));
    a->places = (int32_t)e.shape[0];
    a->rot = (int32_t)(2 * e.shape[1]);
    GDR_TRY(read_param(cos, &a->cos, a->places, a->rot / 2));
    GDR_TRY(read_param(sin, &a->sin, a->places, a->rot / 2));
    if (!positions && a->T > 0) return GDR_ERR_NULL;
    a->pos = positions;
  }
  return GDR_OK;
}

int read_pair(const gdr_tensor_t *t, const QkArgs &a, int j, bool written, void **p, int64_t *st,
              int64_t *sh) {
  Desc d;
  GDR_TRY(read_act(t, 3, &d, a.f32));
  GDR_TRY(shaped(d, a.T, j ? a.Hk : a.Hq, a.d));
  if (written) GDR_TRY(apart(d));
  *p = d.p;
  *st = d.stride[0];
  *sh = d.stride[1];
  return GDR_OK;
}

}  // namespace

extern "C" {

int gdr_conv_fwd(const gdr_tensor_t *x, const gdr_tensor_t *weight, const gdr_tensor_t *bias,
                 const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                 int32_t activation, gdr_tensor_t *y, gdr_tensor_t *ht, cudaStream_t stream) {
  ConvArgs a{};
  GDR_TRY(read_conv(x, weight, bias, h0, cu_seqlens, n_seq, activation, &a));
  Desc d;
  GDR_TRY(read_act(y, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.C));
  GDR_TRY(apart(d));
  a.y = mat(d);
  GDR_TRY(read_rows(ht, const_cast<const void **>(&a.ht), a.f32, n_seq, a.W - 1, a.C));
  GDR_TRY(device_ok());
  if (n_seq == 0) return GDR_OK;
  return done(launch_conv_fwd(a, stream));
}

size_t gdr_conv_bwd_workspace_bytes(int64_t T, int32_t C, int32_t W) {
  if (T < 0 || T > kMost || C < 1 || W < 2 || W > 4) return 0;
  return conv_bwd_workspace(T, C, W);
}

int gdr_conv_bwd(const gdr_tensor_t *x, const gdr_tensor_t *weight, const gdr_tensor_t *bias,
                 const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                 int32_t activation, const gdr_tensor_t *dy, const gdr_tensor_t *dht,
                 gdr_tensor_t *dx, gdr_tensor_t *dweight, gdr_tensor_t *dbias,
                 gdr_tensor_t *dh0, void *workspace, size_t workspace_bytes,
                 cudaStream_t stream) {
  ConvArgs a{};
  GDR_TRY(read_conv(x, weight, bias, h0, cu_seqlens, n_seq, activation, &a));
  Desc d;
  GDR_TRY(read_act(dy, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.C));
  a.dy = mat(d);
  GDR_TRY(read_act(dx, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.C));
  GDR_TRY(apart(d));
  a.dx = mat(d);
  GDR_TRY(read_rows(dht, &a.dht, a.f32, n_seq, a.W - 1, a.C));
  GDR_TRY(read_rows(dh0, const_cast<const void **>(&a.dh0), a.f32, n_seq, a.W - 1, a.C));
  if (!dweight) return GDR_ERR_NULL;
  GDR_TRY(read_param(dweight, &a.dw, a.C, a.W));
  GDR_TRY(read_param(dbias, &a.db, a.C));
  GDR_TRY(device_ok());
  GDR_TRY(scratch(workspace, workspace_bytes, conv_bwd_workspace(a.T, a.C, a.W)));
  a.work = workspace;
  return done(launch_conv_bwd(a, stream));
}

int gdr_conv_step(const gdr_tensor_t *x, const gdr_tensor_t *weight, const gdr_tensor_t *bias,
                  gdr_tensor_t *state, const int32_t *state_indices, int32_t activation,
                  gdr_tensor_t *y, cudaStream_t stream) {
  ConvStepArgs a{};
  Desc d;
  GDR_TRY(read_first(x, 2, &d, &a.f32));
  if (d.shape[0] > kMost || d.shape[1] > kMost || d.shape[1] < 1) return GDR_ERR_SHAPE;
  a.B = (int32_t)d.shape[0];
  a.C = (int32_t)d.shape[1];
  a.x = mat(d);
  GDR_TRY(read_taps(weight, bias, a.C, &a.w, &a.b, &a.W));
  if (activation != GDR_ACT_NONE && activation != GDR_ACT_SILU) return GDR_ERR_OPTION;
  a.silu = activation == GDR_ACT_SILU;
  GDR_TRY(read_act(state, 3, &d, a.f32));
  GDR_TRY(shaped(d, d.shape[0], a.W - 1, a.C));
  GDR_TRY(packed(d));
  if (d.shape[0] > kMost) return GDR_ERR_SHAPE;
  if (!state_indices && d.shape[0] < a.B) return GDR_ERR_SHAPE;
  a.slots = (int32_t)d.shape[0];
  a.state = d.p;
  a.idx = state_indices;
  GDR_TRY(read_act(y, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.B, a.C));
  GDR_TRY(apart(d));
  a.y = mat(d);
  GDR_TRY(device_ok());
  return done(launch_conv_step(a, stream));
}

size_t gdr_ssm_fwd_workspace_bytes(int64_t T, int32_t Dm, int32_t N, int32_t G) {
  if (T < 0 || T > kMost || Dm < 1 || N < 1 || N > 64 || G < 1 || Dm % G) return 0;
  return ssm_fwd_workspace(T, Dm, N, G);
}

int gdr_ssm_fwd(const gdr_tensor_t *x, const gdr_tensor_t *dt, const gdr_tensor_t *A,
                const gdr_tensor_t *B, const gdr_tensor_t *C, const gdr_tensor_t *D,
                const gdr_tensor_t *z, const gdr_tensor_t *dt_bias, int32_t dt_softplus,
                const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                gdr_tensor_t *y, gdr_tensor_t *ht, void *workspace, size_t workspace_bytes,
                cudaStream_t stream) {
  SsmArgs a{};
  GDR_TRY(read_ssm(x, dt, A, B, C, D, z, dt_bias, dt_softplus, &a));
  GDR_TRY(segments(cu_seqlens, n_seq));
  a.cu = cu_seqlens;
  a.n_seq = n_seq;
  GDR_TRY(read_states(h0, &a.h0, n_seq, a.D, a.N));
  GDR_TRY(read_states(ht, const_cast<const float **>(&a.ht), n_seq, a.D, a.N));
  Desc d;
  GDR_TRY(read_act(y, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.D));
  GDR_TRY(apart(d));
  a.y = mat(d);
  GDR_TRY(device_ok());
  if (n_seq == 0) return GDR_OK;
  GDR_TRY(scratch(workspace, workspace_bytes, ssm_fwd_workspace(a.T, a.D, a.N, a.G)));
  a.work = workspace;
  return done(launch_ssm_fwd(a, stream));
}

size_t gdr_ssm_bwd_workspace_bytes(int64_t T, int32_t Dm, int32_t N, int32_t G) {
  if (T < 0 || T > kMost || Dm < 1 || N < 1 || N > 64 || G < 1 || Dm % G) return 0;
  return ssm_bwd_workspace(T, Dm, N, G);
}

int gdr_ssm_bwd(const gdr_tensor_t *x, const gdr_tensor_t *dt, const gdr_tensor_t *A,
                const gdr_tensor_t *B, const gdr_tensor_t *C, const gdr_tensor_t *D,
                const gdr_tensor_t *z, const gdr_tensor_t *dt_bias, int32_t dt_softplus,
                const gdr_tensor_t *h0, const int32_t *cu_seqlens, int32_t n_seq,
                const gdr_tensor_t *dy, const gdr_tensor_t *dht, gdr_tensor_t *dx,
                gdr_tensor_t *ddt, gdr_tensor_t *dA, gdr_tensor_t *dB, gdr_tensor_t *dC,
                gdr_tensor_t *dD, gdr_tensor_t *dz, gdr_tensor_t *ddt_bias, gdr_tensor_t *dh0,
                void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  SsmArgs a{};
  GDR_TRY(read_ssm(x, dt, A, B, C, D, z, dt_bias, dt_softplus, &a));
  GDR_TRY(segments(cu_seqlens, n_seq));
  a.cu = cu_seqlens;
  a.n_seq = n_seq;
  GDR_TRY(read_states(h0, &a.h0, n_seq, a.D, a.N));
  GDR_TRY(read_states(dht, &a.dht, n_seq, a.D, a.N));
  GDR_TRY(read_states(dh0, const_cast<const float **>(&a.dh0), n_seq, a.D, a.N));
  if (!z != !dz) return GDR_ERR_OPTION;
  Desc d;
  GDR_TRY(read_act(dy, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.D));
  a.dout = mat(d);
  struct {
    const gdr_tensor_t *t;
    Mat *m;
  } outs[3] = {{dx, &a.dx}, {ddt, &a.ddt}, {dz, &a.dz}};
  for (auto &o : outs) {
    if (!o.t && o.m == &a.dz) continue;
    GDR_TRY(read_act(o.t, 2, &d, a.f32));
    GDR_TRY(shaped(d, a.T, a.D));
    GDR_TRY(apart(d));
    *o.m = mat(d);
  }
  if (!dA) return GDR_ERR_NULL;
  GDR_TRY(read_param(dA, &a.dA, a.D, a.N));
  GDR_TRY(read_param(dD, &a.dD, a.D));
  GDR_TRY(read_param(ddt_bias, &a.ddt_bias, a.D));
  for (int j = 0; j < 2; ++j) {
    GDR_TRY(read_act(j ? dC : dB, 3, &d, a.f32));
    GDR_TRY(shaped(d, a.T, a.G, a.N));
    GDR_TRY(packed(d));
    (j ? a.dC : a.dB) = d.p;
  }
  GDR_TRY(device_ok());
  GDR_TRY(scratch(workspace, workspace_bytes, ssm_bwd_workspace(a.T, a.D, a.N, a.G)));
  a.work = workspace;
  return done(launch_ssm_bwd(a, stream));
}

int gdr_ssm_step(const gdr_tensor_t *x, const gdr_tensor_t *dt, const gdr_tensor_t *A,
                 const gdr_tensor_t *B, const gdr_tensor_t *C, const gdr_tensor_t *D,
                 const gdr_tensor_t *z, const gdr_tensor_t *dt_bias, int32_t dt_softplus,
                 gdr_tensor_t *state, const int32_t *state_indices, gdr_tensor_t *y,
                 cudaStream_t stream) {
  SsmArgs a{};
  GDR_TRY(read_ssm(x, dt, A, B, C, D, z, dt_bias, dt_softplus, &a));
  Desc d, s;
  GDR_TRY(read_desc(state, GDR_F32, 3, &s));
  GDR_TRY(shaped(s, s.shape[0], a.D, a.N));
  GDR_TRY(packed(s));
  if (s.shape[0] > kMost) return GDR_ERR_SHAPE;
  if (!state_indices && s.shape[0] < a.T) return GDR_ERR_SHAPE;
  GDR_TRY(read_act(y, 2, &d, a.f32));
  GDR_TRY(shaped(d, a.T, a.D));
  GDR_TRY(apart(d));
  a.y = mat(d);
  GDR_TRY(device_ok());
  return done(launch_ssm_step(a, reinterpret_cast<float *>(s.p), (int32_t)s.shape[0],
                              state_indices, stream));
}

int gdr_qk_fwd(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *q_weight,
               const gdr_tensor_t *k_weight, int32_t norm, float eps, const gdr_tensor_t *cos,
               const gdr_tensor_t *sin, const int32_t *positions, int32_t interleaved,
               gdr_tensor_t *q_out, gdr_tensor_t *k_out, cudaStream_t stream) {
  QkArgs a{};
  GDR_TRY(read_qk(q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved, &a));
  for (int j = 0; j < 2; ++j)
    GDR_TRY(read_pair(j ? k_out : q_out, a, j, true, &a.y[j], &a.y_st[j], &a.y_sh[j]));
  GDR_TRY(device_ok());
  return done(launch_qk_fwd(a, stream));
}

size_t gdr_qk_bwd_workspace_bytes(int64_t T, int32_t Hq, int32_t Hk, int32_t d) {
  if (T < 0 || Hq < 0 || Hk < 0 || d < 1 || d > 256) return 0;
  return qk_bwd_workspace(T, Hq, Hk, d);
}

int gdr_qk_bwd(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *q_weight,
               const gdr_tensor_t *k_weight, int32_t norm, float eps, const gdr_tensor_t *cos,
               const gdr_tensor_t *sin, const int32_t *positions, int32_t interleaved,
               const gdr_tensor_t *dq_out, const gdr_tensor_t *dk_out, gdr_tensor_t *dq,
               gdr_tensor_t *dk, gdr_tensor_t *dq_weight, gdr_tensor_t *dk_weight,
               void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  QkArgs a{};
  GDR_TRY(read_qk(q, k, q_weight, k_weight, norm, eps, cos, sin, positions, interleaved, &a));
  for (int j = 0; j < 2; ++j) {
    GDR_TRY(read_pair(j ? dk_out : dq_out, a, j, false, &a.y[j], &a.y_st[j], &a.y_sh[j]));
    GDR_TRY(read_pair(j ? dk : dq, a, j, true, &a.dx[j], &a.dx_st[j], &a.dx_sh[j]));
    GDR_TRY(read_param(j ? dk_weight : dq_weight, &a.dw[j], a.d));
  }
  GDR_TRY(device_ok());
  GDR_TRY(scratch(workspace, workspace_bytes, qk_bwd_workspace(a.T, a.Hq, a.Hk, a.d)));
  a.work = workspace;
  return done(launch_qk_bwd(a, stream));
}

int gdr_delta_step(const gdr_tensor_t *q, const gdr_tensor_t *k, const gdr_tensor_t *v,
                   const gdr_tensor_t *g, const gdr_tensor_t *beta, float scale,
                   gdr_tensor_t *state, const int32_t *state_indices, gdr_tensor_t *o,
                   cudaStream_t stream) {
  Desc Q, K, V, Gd, Be, S, O;
  GDR_TRY(read_desc(q, GDR_BF16, 3, &Q));
  GDR_TRY(read_desc(k, GDR_BF16, 3, &K));
  GDR_TRY(read_desc(v, GDR_BF16, 3, &V));
  GDR_TRY(read_desc(g, GDR_F32, 2, &Gd));
  GDR_TRY(read_desc(beta, GDR_BF16, 2, &Be));
  GDR_TRY(read_desc(state, GDR_F32, 4, &S));
  GDR_TRY(read_desc(o, GDR_BF16, 3, &O));
  const int64_t B = Q.shape[0], Hk = Q.shape[1], D = Q.shape[2], H = V.shape[1];
  GDR_TRY(shaped(K, B, Hk, D));
  GDR_TRY(shaped(V, B, H, V.shape[2]));
  GDR_TRY(shaped(O, B, H, V.shape[2]));
  GDR_TRY(shaped(Gd, B, H));
  GDR_TRY(shaped(Be, B, H));
  if (V.shape[2] != D || (D != 64 && D != 128)) return GDR_ERR_DIM;
  if (B > kMost || Hk < 1 || H < 1 || H > 0xffff) return GDR_ERR_SHAPE;
  if (B * H * (D / 32) > 0x7fffffff) return GDR_ERR_SHAPE;
  if (H % Hk != 0) return GDR_ERR_HEADS;
  if (S.shape[1] != H || S.shape[2] != D || S.shape[3] != D || S.shape[0] > kMost)
    return GDR_ERR_SHAPE;
  if (!state_indices && S.shape[0] < B) return GDR_ERR_SHAPE;
  GDR_TRY(packed(S));
  GDR_TRY(apart(O));
  if (!aligned16(S.p)) return GDR_ERR_ALIGN;
  GDR_TRY(device_ok());
  DeltaStepArgs a{};
  a.B = (int32_t)B;
  a.Hk = (int32_t)Hk;
  a.H = (int32_t)H;
  a.D = (int32_t)D;
  a.slots = (int32_t)S.shape[0];
  a.scale = scale;
  a.q = Q.p; a.q_st = Q.stride[0]; a.q_sh = Q.stride[1];
  a.k = K.p; a.k_st = K.stride[0]; a.k_sh = K.stride[1];
  a.v = V.p; a.v_st = V.stride[0]; a.v_sh = V.stride[1];
  a.g = reinterpret_cast<const float *>(Gd.p); a.g_st = Gd.stride[0]; a.g_sh = Gd.stride[1];
  a.beta = Be.p; a.b_st = Be.stride[0]; a.b_sh = Be.stride[1];
  a.o = O.p; a.o_st = O.stride[0]; a.o_sh = O.stride[1];
  a.state = reinterpret_cast<float *>(S.p);
  a.idx = state_indices;
  return done(launch_delta_step(a, stream));
}

}  // extern "C"
