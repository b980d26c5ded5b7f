// gdr_block.cuh -- the operators of a hybrid block beside the mixer: gated linear recurrence, norms
// with gate and residual scale, attention of one new token over a paged cache, and the cache's
// bookkeeping.  Arguments of their launchers, and what their kernels share.
#pragma once

#include <atomic>

#include "gdr_mix.cuh"

namespace gdr {
namespace mix {

// A kernel's attribute, set once on each device (the first 64; others every time).
template <typename K>
cudaError_t set_once(K *kernel, cudaFuncAttribute attribute, int value, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
  if (e == cudaSuccess && !(done.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, attribute, value);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) cudaGetLastError();  // reported here, not to the next call
  return e;
}

}  // namespace mix

struct RecArgs {
  int32_t T, D, n_seq, normalize;
  bool f32;
  const int32_t *cu;
  Mat x, r, i, y;  // i.p null: no input gate
  const float *A, *h0;
  float *ht;
  float *kept;  // [ceil(T / kRecEvery), D]: the state before each token that is a multiple of it
  // backward
  Mat dy, dx, dr, di;
  const float *dht;
  float *dA, *dh0;
  void *work;
};
constexpr int kRecEvery = 8;
cudaError_t launch_rec_fwd(const RecArgs &a, cudaStream_t stream);
// the states that the backward starts from, without y
cudaError_t launch_rec_states(const RecArgs &a, cudaStream_t stream);
// the status words of the recurrence's waits (0: none ran out)
cudaError_t read_rec_bwd_status(int32_t *out);
cudaError_t clear_rec_bwd_status();
cudaError_t read_rec_status(int32_t *out);
cudaError_t clear_rec_status();
cudaError_t launch_rec_wait_selftest(uint32_t limit_us, int32_t steps, cudaStream_t stream);
size_t rec_bwd_workspace(int64_t T, int32_t D, int32_t n_seq, bool kept);
cudaError_t launch_rec_bwd(const RecArgs &a, bool kept, cudaStream_t stream);
// rows of x, r, i, y are T requests; state [slots, D] in place
cudaError_t launch_rec_step(const RecArgs &a, float *state, int32_t slots, const int32_t *idx,
                            cudaStream_t stream);

// Heads of T tokens, innermost contiguous: strides of a token and of a head.
struct Heads {
  void *p;
  int64_t st, sh;
};

struct GatedArgs {
  int32_t T, H, d, silu;
  bool f32;
  float eps;
  Heads x, z, y;
  mix::Param w;  // [d] or null
  // backward
  Heads dy, dx, dz;
  float *dw;
  void *work;
};
cudaError_t launch_gated_fwd(const GatedArgs &a, cudaStream_t stream);
size_t gated_bwd_workspace(int64_t T, int32_t H, int32_t d);
cudaError_t launch_gated_bwd(const GatedArgs &a, cudaStream_t stream);

struct ResidArgs {
  int32_t T, C;
  bool f32, rf32;  // x, y and their gradients; residual, h and theirs
  float eps, scale;
  Mat x, res, y, h;       // res.p null: zeros
  mix::Param w, wp, g;    // [C] or null; post: the norm behind the block, without or with weights
  int32_t post;
  // backward
  Mat dy, dh, dx, dres;  // dh.p null: zeros
  float *dw, *dwp, *dg;
  void *work;
};
cudaError_t launch_resid_fwd(const ResidArgs &a, cudaStream_t stream);
size_t resid_bwd_workspace(int64_t T, int32_t C);
cudaError_t launch_resid_bwd(const ResidArgs &a, cudaStream_t stream);

// Keys or values of a paged cache [pages, page, Hk, d]: strides of a page, a place in it, a head.
struct Pages {
  void *p;
  int64_t sp, st, sh;
};

struct AttnArgs {
  int32_t B, Hq, Hk, d, page, pages, width, window;
  bool f32;
  float scale;
  Heads q, o;
  Pages k, v;
  const int32_t *table;  // [B, width], rows table_st apart
  int64_t table_st;
  const int32_t *lens;   // [B]
  void *work;
};
size_t attn_workspace(int32_t B, int32_t Hq, int32_t Hk, int32_t d);
cudaError_t launch_attn_step(const AttnArgs &a, cudaStream_t stream);

struct PlanArgs {
  int32_t B, width, page, nfree, most;  // most: tokens that slots and positions hold
  const int32_t *lens, *fresh;
  int32_t *table;
  int64_t table_st;
  const int32_t *free_pages, *taken;
  int32_t *slots, *positions, *cu, *lens_out, *taken_out;
};
cudaError_t launch_cache_plan(const PlanArgs &a, cudaStream_t stream);

struct WriteArgs {
  int32_t T, Hk, d, page, pages;
  bool f32;
  Heads k, v;
  Pages kc, vc;
  const int32_t *slots;
};
cudaError_t launch_cache_write(const WriteArgs &a, cudaStream_t stream);

}  // namespace gdr
