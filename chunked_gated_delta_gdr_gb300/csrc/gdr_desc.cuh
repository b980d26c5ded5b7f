// gdr_desc.cuh -- reading gdr_tensor_t descriptors and checking the current device, shared by
// the extern "C" entry points.
#pragma once

#include "gdr_internal.cuh"

namespace gdr {

struct Desc {
  void *p;
  int ndim;
  int64_t shape[4];
  int64_t stride[4];
};

inline int read_desc(const gdr_tensor_t *t, int dtype, int ndim, Desc *d) {
  if (!t) return GDR_ERR_NULL;
  if (t->dtype != dtype) return GDR_ERR_DTYPE;
  if (t->ndim != ndim) return GDR_ERR_SHAPE;
  int64_t numel = 1;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return GDR_ERR_SHAPE;
    d->shape[i] = t->shape[i];
    numel *= t->shape[i];
  }
  if (!t->data && numel > 0) return GDR_ERR_NULL;
  d->p = t->data;
  d->ndim = ndim;
  if (t->strides) {
    for (int i = 0; i < ndim; ++i) {
      if (t->strides[i] < 0) return GDR_ERR_STRIDE;
      d->stride[i] = t->strides[i];
    }
    if (d->shape[ndim - 1] > 1 && d->stride[ndim - 1] != 1) return GDR_ERR_STRIDE;
    d->stride[ndim - 1] = 1;
  } else {
    int64_t s = 1;
    for (int i = ndim - 1; i >= 0; --i) {
      d->stride[i] = s;
      s *= d->shape[i];
    }
  }
  return GDR_OK;
}

inline bool compact(const Desc &d) {
  int64_t s = 1;
  for (int i = d.ndim - 1; i >= 0; --i) {
    if (d.shape[i] > 1 && d.stride[i] != s) return false;
    s *= d.shape[i];
  }
  return true;
}

inline int device_ok() {
  static bool fits[64] = {false};  // devices found to be sm_103: a device does not change
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDR_ERR_CUDA;
  if (dev >= 0 && dev < 64 && fits[dev]) return GDR_OK;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return GDR_ERR_CUDA;
  if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return GDR_ERR_CUDA;
  if (major != 10 || minor != 3) return GDR_ERR_DEVICE;
  if (dev >= 0 && dev < 64) fits[dev] = true;
  return GDR_OK;
}

}  // namespace gdr
