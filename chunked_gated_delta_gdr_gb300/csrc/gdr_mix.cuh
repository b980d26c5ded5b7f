// gdr_mix.cuh -- definitions shared by the token mixer's operators around the delta rule (short
// convolution, selective state space, q/k norm with rotation, single-token steps): rows of 8
// elements in bf16 or fp32, and the device-side reading of cu_seqlens by token ranges.
#pragma once

#include "gdr_internal.cuh"

namespace gdr {
namespace mix {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ 8 elements of a row

template <typename E>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};

__device__ __forceinline__ float lo_bf(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float (&f)[8]) {
  f[0] = lo_bf(r.a.x); f[1] = hi_bf(r.a.x); f[2] = lo_bf(r.a.y); f[3] = hi_bf(r.a.y);
  f[4] = lo_bf(r.a.z); f[5] = hi_bf(r.a.z); f[6] = lo_bf(r.a.w); f[7] = hi_bf(r.a.w);
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&f)[8]) {
  f[0] = __uint_as_float(r.a.x); f[1] = __uint_as_float(r.a.y);
  f[2] = __uint_as_float(r.a.z); f[3] = __uint_as_float(r.a.w);
  f[4] = __uint_as_float(r.b.x); f[5] = __uint_as_float(r.b.y);
  f[6] = __uint_as_float(r.b.z); f[7] = __uint_as_float(r.b.w);
}

template <typename E>
__device__ __forceinline__ float ld1(const E *p);
template <>
__device__ __forceinline__ float ld1<__nv_bfloat16>(const __nv_bfloat16 *p) {
  return __bfloat162float(*p);
}
template <>
__device__ __forceinline__ float ld1<float>(const float *p) {
  return *p;
}
__device__ __forceinline__ void st1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void st1(float *p, float v) { *p = v; }

__device__ __forceinline__ Raw8<__nv_bfloat16> pack8(const float (&f)[8], __nv_bfloat16) {
  Raw8<__nv_bfloat16> r;
  r.a = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  return r;
}
__device__ __forceinline__ Raw8<float> pack8(const float (&f)[8], float) {
  Raw8<float> r;
  r.a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
  r.b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                   __float_as_uint(f[7]));
  return r;
}

template <typename E>
__device__ __forceinline__ Raw8<E> zero8() {
  Raw8<E> r;
  float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  r = pack8(z, E{});
  return r;
}

// n of 8 elements (the others 0); VEC: n is 0 or 8 and p is 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ Raw8<__nv_bfloat16> ld8(const __nv_bfloat16 *p, int n) {
  Raw8<__nv_bfloat16> r;
  r.a = make_uint4(0, 0, 0, 0);
  if (VEC) {
    if (n > 0) r.a = *reinterpret_cast<const uint4 *>(p);
  } else {
    const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? s[i] : 0;
    r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ Raw8<float> ld8(const float *p, int n) {
  Raw8<float> r;
  r.a = r.b = make_uint4(0, 0, 0, 0);
  if (VEC) {
    if (n > 0) {
      r.a = *reinterpret_cast<const uint4 *>(p);
      r.b = *reinterpret_cast<const uint4 *>(p + 4);
    }
  } else {
    const uint32_t *s = reinterpret_cast<const uint32_t *>(p);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? s[i] : 0;
    r.a = make_uint4(v[0], v[1], v[2], v[3]);
    r.b = make_uint4(v[4], v[5], v[6], v[7]);
  }
  return r;
}

template <bool VEC>
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const Raw8<__nv_bfloat16> &r, int n) {
  if (VEC) {
    if (n > 0) *reinterpret_cast<uint4 *>(p) = r.a;
  } else {
    unsigned short *s = reinterpret_cast<unsigned short *>(p);
    const uint32_t v[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) s[i] = (unsigned short)(v[i >> 1] >> ((i & 1) * 16));
  }
}
template <bool VEC>
__device__ __forceinline__ void st8(float *p, const Raw8<float> &r, int n) {
  if (VEC) {
    if (n > 0) {
      *reinterpret_cast<uint4 *>(p) = r.a;
      *reinterpret_cast<uint4 *>(p + 4) = r.b;
    }
  } else {
    uint32_t *s = reinterpret_cast<uint32_t *>(p);
    const uint32_t v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) s[i] = v[i];
  }
}

// Pairs of fp32 values: one instruction for two products.  They cost the fp32 pipes as much as two
// single ones and save an issue slot: for kernels bound by instruction issue.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(f2 v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void unpack4(const Raw8<__nv_bfloat16> &r, f2 (&f)[4]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(lo_bf(w[i]), hi_bf(w[i]));
}
__device__ __forceinline__ void unpack4(const Raw8<float> &r, f2 (&f)[4]) {
  float v[8];
  unpack8(r, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(v[2 * i], v[2 * i + 1]);
}
template <typename E>
__device__ __forceinline__ Raw8<E> pack4(const f2 (&f)[4]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(f[i], v[2 * i], v[2 * i + 1]);
  return pack8(v, E{});
}

// Launches.  A kernel is made ready while the one before it in the stream drains; its blocks wait
// here, before they touch memory, until that one has completed and its writes are visible (first
// statement of every kernel; about 1.5 us a launch).  EARLY lets the next kernel's blocks be placed
// as soon as all of this one's run: for short kernels only, for blocks that are placed while some
// SMs are still busy crowd on the others (6,619 tokens of 2,304 x 16 states: 119 us, 164 with EARLY
// everywhere; a convolution step of 37 rows 6.1 us, 3.9 with it).
template <bool EARLY = false>
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (EARLY) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream,
                   A... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = stream;
  c.attrs = &early;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // reported here, not to the next call
  return e;
}

// 16 bytes of global memory into shared memory, asynchronously (ok false: zeros instead).
__device__ __forceinline__ void copy16(uint4 *dst, const void *src, bool ok) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy16(uint4 *dst, const void *src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(void *dst, const void *src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Until at most N of this thread's groups of copies are on their way.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ functions of one value

// 2^x on the special-function unit (2 ulp; subnormal results flushed to zero)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / x on the special-function unit (1 ulp; subnormal results flushed to zero)
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-x): 2^(-x log2 e) overflows to inf for very negative x, whose reciprocal is 0
__device__ __forceinline__ float sigmoidf(float x) { return rcp(1.f + ex2(-x * kLog2e)); }
__device__ __forceinline__ f2 sigmoid2(f2 x) {
  float a, b;
  unpair(mul2(x, pair(-kLog2e, -kLog2e)), a, b);
  unpair(add2(pair(ex2(a), ex2(b)), pair(1.f, 1.f)), a, b);
  return pair(rcp(a), rcp(b));
}
// d/dx of x sigmoid(x), from s = sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float s) { return s * (1.f + x * (1.f - s)); }
__device__ __forceinline__ f2 dsilu2(f2 x, f2 s) {
  return fma2(x, fma2(mul2(s, pair(-1.f, -1.f)), s, s), s);
}
// log(1 + e^x) = max(x, 0) + log(1 + t), t = e^-|x|, and log(1 + t) = 2 atanh(s), s = t / (2 + t)
// <= 1/3, accurate relative to itself for small t too: 2 atanh(s) / s as a polynomial in s^2,
// interpolated at the Chebyshev points of [0, 1/9] (4e-9 off at most).
__device__ __forceinline__ float softplusf(float x) {
  const float t = ex2(-fabsf(x) * kLog2e), s = t * rcp(2.f + t), q = s * s;
  float p = 0.28157778f;
  p = fmaf(p, q, 0.27965158f);
  p = fmaf(p, q, 0.40024595f);
  p = fmaf(p, q, 0.66666322f);
  p = fmaf(p, q, 2.f);
  return fmaf(p, s, fmaxf(x, 0.f));
}

// A parameter vector in fp32 or bf16.
struct Param {
  const void *p;
  int bf16;
};
__device__ __forceinline__ float ldp(const Param &w, int64_t i) {
  return w.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(w.p)[i])
                : reinterpret_cast<const float *>(w.p)[i];
}

// ------------------------------------------------------------------ reading cu_seqlens
//
// Offsets are clamped to [0, T] and made non-decreasing by a running maximum b_i; segment n is
// [b_n, b_{n+1}).  A block that works on tokens [t0, t1) needs the segment alive at t0 and the
// bounds inside its range.  It finds them itself from the array, so that no launch has to come
// before it: a search by all threads for the first offset at or above t0, then one warp walks on
// tile by tile.  cu null: one segment of T tokens (n_seq = 1).

__device__ __forceinline__ int cu_at(const int32_t *cu, int i, int T) {
  return cu ? min(max(cu[i], 0), T) : (i == 0 ? 0 : T);
}

// Entries consumed so far (all with b < the next tile's first token), their running maximum (the
// start of the segment with index j - 1) and a bound below which no further entry lies.
struct SegCursor {
  int j, b, nb;
};

// All threads of the block; red: 64 ints of shared memory.
__device__ __forceinline__ SegCursor seg_find(const int32_t *cu, int n_seq, int T, int t0,
                                              int *red) {
  SegCursor c{0, 0, 0};
  if (t0 <= 0) return c;
  const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (nt + 31) >> 5;
  int m = n_seq + 1;
  for (int i = threadIdx.x; i <= n_seq; i += nt)
    if (cu_at(cu, i, T) >= t0) {
      m = i;
      break;
    }
  m = __reduce_min_sync(0xffffffffu, m);
  if (lane == 0) red[warp] = m;
  __syncthreads();
  for (int w = 0; w < nw; ++w) m = min(m, red[w]);
  int b = 0;
  for (int i = threadIdx.x; i < m; i += nt) b = max(b, cu_at(cu, i, T));
  b = __reduce_max_sync(0xffffffffu, b);
  if (lane == 0) red[32 + warp] = b;
  __syncthreads();
  for (int w = 0; w < nw; ++w) b = max(b, red[32 + w]);
  __syncthreads();
  c.j = m;
  c.b = b;
  return c;
}

// One whole warp: the bounds at tokens t0 .. t0 + n (n <= L).  mark[i] (i = 0..n) is the last
// segment index whose bound is t0 + i, or -1: the segment that starts there (n_seq: the tokens
// behind the last segment).  Returns whether there is any mark; without one, mark is not written.
// Moves the cursor to token t0 + n.
__device__ __forceinline__ bool seg_marks(const int32_t *cu, int n_seq, int T, int t0, int n,
                                          int *mark, SegCursor &c) {
  if (c.nb > t0 + n) return false;
  const int lane = threadIdx.x & 31;
  for (int i = lane; i <= n; i += 32) mark[i] = -1;
  __syncwarp();
  bool any = false;
  for (;;) {
    const int idx = c.j + lane;
    int b = idx <= n_seq ? cu_at(cu, idx, T) : 0x7fffffff;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) b = max(b, u);
    }
    b = max(b, c.b);
    const bool in = b <= t0 + n;  // a prefix of the lanes: b does not decrease
    if (in) atomicMax(&mark[b - t0], idx);  // b >= t0: what lies below was consumed
    any |= __any_sync(0xffffffffu, in);
    const int cnt = __popc(__ballot_sync(0xffffffffu, b < t0 + n));
    c.nb = __shfl_sync(0xffffffffu, b, cnt < 32 ? cnt : 31);
    if (cnt > 0) c.b = __shfl_sync(0xffffffffu, b, cnt - 1);
    c.j += cnt;
    if (cnt < 32) break;
  }
  __syncwarp();
  return any;
}

// Calls f(n) on all threads of the block for every segment n without tokens.  bits: one int of
// shared memory.
template <typename F>
__device__ __forceinline__ void for_empty_segments(const int32_t *cu, int n_seq, int T, int *bits,
                                                   F f) {
  int run = 0;  // running maximum of the entries before this round (warp 0)
  for (int base = 0; base < n_seq; base += 32) {
    if (threadIdx.x < 32) {
      const int i = base + (int)threadIdx.x;
      int b = i <= n_seq ? cu_at(cu, i, T) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, b, o);
        if ((int)threadIdx.x >= o) b = max(b, u);
      }
      b = max(b, run);
      const bool empty = i < n_seq && cu_at(cu, i + 1, T) <= b;
      run = __shfl_sync(0xffffffffu, b, 31);
      const unsigned m = __ballot_sync(0xffffffffu, empty);
      if (threadIdx.x == 0) *bits = (int)m;
    }
    __syncthreads();
    unsigned m = (unsigned)*bits;
    while (m) {
      const int k = __ffs(m) - 1;
      m &= m - 1;
      f(base + k);
    }
    __syncthreads();
  }
}

inline int sm_count() {
  static int sms[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (sms[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return 152;
    }
    sms[dev] = n;
  }
  return sms[dev];
}

}  // namespace mix

// ------------------------------------------------------------------ launchers

struct Mat {  // [rows, cols] activations, innermost contiguous; st: row stride in elements
  void *p;
  int64_t st;
};

struct ConvArgs {
  int32_t T, C, W, n_seq, silu;
  bool f32;  // activations in fp32 (else bf16)
  const int32_t *cu;
  Mat x, y;
  mix::Param w, b;  // w [C, W], b [C] or null
  const void *h0;   // [n_seq, W - 1, C] or null
  void *ht;
  // backward
  Mat dy, dx;
  const void *dht;
  void *dh0;
  float *dw, *db;
  void *work;
};
cudaError_t launch_conv_fwd(const ConvArgs &a, cudaStream_t stream);
size_t conv_bwd_workspace(int64_t T, int32_t C, int32_t W);
cudaError_t launch_conv_bwd(const ConvArgs &a, cudaStream_t stream);
// x, y [B, C]; state [slots, W - 1, C] in place; idx [B] or null (row i uses slot i)
struct ConvStepArgs {
  int32_t B, C, W, slots, silu;
  bool f32;
  Mat x, y;
  mix::Param w, b;
  void *state;  // compact
  const int32_t *idx;
};
cudaError_t launch_conv_step(const ConvStepArgs &a, cudaStream_t stream);

struct SsmArgs {
  int32_t T, D, N, G, n_seq, softplus;
  bool f32;
  bool n4;  // states in fours, 16-byte aligned (set by the launchers)
  const int32_t *cu;
  Mat x, dt, z, y;
  const void *B, *C;
  int64_t B_st, B_sg, C_st, C_sg;
  const float *A, *Dskip, *dt_bias, *h0;
  float *ht;
  void *work;
  // backward
  Mat dout, dx, ddt, dz;
  const float *dht;
  float *dA, *dD, *ddt_bias, *dh0;
  void *dB, *dC;  // compact [T, G, N]
};
size_t ssm_fwd_workspace(int64_t T, int32_t D, int32_t N, int32_t G);
cudaError_t launch_ssm_fwd(const SsmArgs &a, cudaStream_t stream);
size_t ssm_bwd_workspace(int64_t T, int32_t D, int32_t N, int32_t G);
cudaError_t launch_ssm_bwd(const SsmArgs &a, cudaStream_t stream);
// rows of x, dt, z, y, B, C are T requests; state [slots, D, N] in place
cudaError_t launch_ssm_step(const SsmArgs &a, float *state, int32_t slots, const int32_t *idx,
                            cudaStream_t stream);

struct QkArgs {
  int64_t T;
  int32_t Hq, Hk, d, rot, rms, interleaved, places;
  bool f32;
  float eps;
  // per tensor (0: q, 1: k): input, output (or the output's gradient), input's gradient
  const void *x[2];
  int64_t x_st[2], x_sh[2];
  void *y[2];
  int64_t y_st[2], y_sh[2];
  void *dx[2];
  int64_t dx_st[2], dx_sh[2];
  mix::Param w[2];
  float *dw[2];
  const float *cos, *sin;
  bool quads;  // a place's cosines and sines start on 16 bytes (set by the launcher)
  const int32_t *pos;
  void *work;
};
cudaError_t launch_qk_fwd(const QkArgs &a, cudaStream_t stream);
size_t qk_bwd_workspace(int64_t T, int32_t Hq, int32_t Hk, int32_t d);
cudaError_t launch_qk_bwd(const QkArgs &a, cudaStream_t stream);

struct DeltaStepArgs {
  int32_t B, Hk, H, D, slots;
  float scale;
  const void *q, *k, *v, *beta;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, b_st, b_sh, g_st, g_sh, o_st, o_sh;
  const float *g;
  void *o;
  float *state;
  const int32_t *idx;
};
cudaError_t launch_delta_step(const DeltaStepArgs &a, cudaStream_t stream);

}  // namespace gdr
