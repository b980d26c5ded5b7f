// gdr_mix_desc.cuh -- reading the descriptors of the mixer's and the block's operators, shared by their
// extern "C" entry points.
#pragma once

#include "gdr_desc.cuh"
#include "gdr_mix.cuh"

namespace gdr {

constexpr int64_t kMost = 0x7ff00000;  // tokens, rows and channels: int arithmetic stays in range

#define GDR_TRY(expr)      \
  do {                     \
    const int r_ = (expr); \
    if (r_) return r_;     \
  } while (0)

// Activations: f32 or bf16; *f32 is set by the first tensor of a call, the others must agree.
inline int read_first(const gdr_tensor_t *t, int ndim, Desc *d, bool *f32) {
  if (!t) return GDR_ERR_NULL;
  if (t->dtype != GDR_BF16 && t->dtype != GDR_F32) return GDR_ERR_DTYPE;
  *f32 = t->dtype == GDR_F32;
  return read_desc(t, t->dtype, ndim, d);
}
inline int read_act(const gdr_tensor_t *t, int ndim, Desc *d, bool f32) {
  return read_desc(t, f32 ? GDR_F32 : GDR_BF16, ndim, d);
}
inline int shaped(const Desc &d, int64_t a, int64_t b = -1, int64_t c = -1) {
  const int64_t want[3] = {a, b, c};
  for (int i = 0; i < d.ndim; ++i)
    if (d.shape[i] != want[i]) return GDR_ERR_SHAPE;
  return GDR_OK;
}
// Written tensors: no two elements at one address.
inline int apart(const Desc &d) {
  int64_t extent = 1;
  for (int i = d.ndim - 1; i >= 0; --i) {
    if (d.shape[i] > 1) {
      if (d.stride[i] < extent) return GDR_ERR_STRIDE;
      extent = d.stride[i] * (d.shape[i] - 1) + extent;
    }
    if (d.shape[i] == 0) return GDR_OK;
  }
  return GDR_OK;
}
inline int packed(const Desc &d) { return compact(d) ? GDR_OK : GDR_ERR_STRIDE; }

inline Mat mat(const Desc &d) { return Mat{d.p, d.stride[0]}; }

// An optional compact f32 tensor of these extents.
inline int read_param(const gdr_tensor_t *t, const float **p, int64_t a, int64_t b = -1,
               int64_t c = -1) {
  *p = nullptr;
  if (!t) return GDR_OK;
  Desc d;
  GDR_TRY(read_desc(t, GDR_F32, c >= 0 ? 3 : b >= 0 ? 2 : 1, &d));
  GDR_TRY(shaped(d, a, b, c));
  GDR_TRY(packed(d));
  *p = reinterpret_cast<const float *>(d.p);
  return GDR_OK;
}
inline int read_param(const gdr_tensor_t *t, float **p, int64_t a, int64_t b = -1, int64_t c = -1) {
  return read_param(t, const_cast<const float **>(p), a, b, c);
}
// Optional compact states in the activations' type.
inline int read_rows(const gdr_tensor_t *t, const void **p, bool f32, int64_t a, int64_t b, int64_t c) {
  *p = nullptr;
  if (!t) return GDR_OK;
  Desc d;
  GDR_TRY(read_act(t, 3, &d, f32));
  if (d.shape[0] != a) return GDR_ERR_NSEQ;
  GDR_TRY(shaped(d, a, b, c));
  GDR_TRY(packed(d));
  *p = d.p;
  return GDR_OK;
}

inline int segments(const int32_t *cu, int32_t n_seq) {
  if (n_seq < 0) return GDR_ERR_NSEQ;
  if (!cu && n_seq != 1) return n_seq == 0 ? GDR_OK : GDR_ERR_NULL;
  return GDR_OK;
}

inline int scratch(const void *p, size_t have, size_t need) {
  if (need == 0) return GDR_OK;
  if (!p || have < need || (reinterpret_cast<uintptr_t>(p) & 255)) return GDR_ERR_WORKSPACE;
  return GDR_OK;
}

inline int done(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace gdr
