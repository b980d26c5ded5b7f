// gdr_norm.cu -- the norms of a hybrid block and their backward.
//
// Gated norm of the mixer's heads: y = n w f(z), n = x r, r = (mean x^2 + eps)^-1/2 over a head, f the
// gate's activation.  With e = dy w f(z):
//   dx = r (e - n mean(e n)),  dz = dy w n f'(z),  dw = sum dy f(z) n.
//
// Residual norm, between two blocks: u = x or (post) x r_x w_post, h = residual + scale gate u,
// y = h r_h w.  With n = h r_h, e = dy w:
//   dh' = dh + r_h (e - n mean(e n)) = dresidual,  dw = sum dy n,  dgate = sum scale dh' u,
//   du = scale gate dh',  dx = du, or with n_x = x r_x, e = du w_post:
//   dx = r_x (e - n_x mean(e n_x)),  dw_post = sum du n_x.
// h is computed again from x and the residual rather than read: it was rounded when it was stored.
//
// Bound by HBM: every tensor is read or written once, a row stays in registers between its sums.
#include "gdr_block.cuh"

namespace gdr {
namespace mix {
namespace {

// The sum of v over the TPR threads of a row, in all of them.  Up to 32: lanes of a warp; else the
// whole block, and `phase` names one of two places in red (which the next sum must not share).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int phase) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    constexpr int W = TPR / 32;
    if ((threadIdx.x & 31) == 0) red[phase][threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[phase][0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[phase][w];
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 (*red)[32], int phase) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (TPR > 32) {
    constexpr int W = TPR / 32;
    if ((threadIdx.x & 31) == 0) red[phase][threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[phase][0];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      v.x += red[phase][w].x;
      v.y += red[phase][w].y;
    }
  }
  return v;
}

// r (e - n mean(e n)), n = x r, for a row that one thread holds: up to 8 columns.  With few of them the
// difference cancels (with one it is r e eps r^2), so its sums are 64 bits.
__device__ __forceinline__ void row_back(const float (&x)[8], const float (&e)[8], int columns, float eps,
                                         float (&out)[8]) {
  double s = 0, p = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s += (double)x[k] * x[k];
    p += (double)e[k] * x[k];
  }
  const double q = s / columns + (double)eps, r = 1. / sqrt(q), back = p / columns / q;
#pragma unroll
  for (int k = 0; k < 8; ++k) out[k] = (float)(r * ((double)e[k] - back * x[k]));
}

// n of 8 parameters from column c on, the others 0; null: ones.
template <bool VEC>
__device__ __forceinline__ void params8(const Param &w, int64_t c, int n, float (&f)[8]) {
  if (!w.p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (w.bf16) {
    unpack8(ld8<VEC>(reinterpret_cast<const __nv_bfloat16 *>(w.p) + c, n), f);
  } else {
    unpack8(ld8<VEC>(reinterpret_cast<const float *>(w.p) + c, n), f);
  }
}

// out[c] = the sum of parts[b][c] over n blocks, in order: eight warps take every eighth.
__global__ void __launch_bounds__(256) k_sum_parts(const float *parts, int n, int64_t stride,
                                                   int count, float *out0, float *out1,
                                                   float *out2) {
  after_previous();
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float *p = parts + (int64_t)blockIdx.y * count + c;
  float v = 0.f;
  if (c < count) {
#pragma unroll 4
    for (int b = warp; b < n; b += 8) v += p[b * stride];
  }
  red[warp][lane] = v;
  __syncthreads();
  float *out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
  if (warp == 0 && c < count && out) {
#pragma unroll
    for (int w = 1; w < 8; ++w) v += red[w][lane];
    out[c] = v;
  }
}

// ------------------------------------------------------------------ gated norm of heads

constexpr int kGated = 256;  // threads of a block

// The rows (token, head) of one lane group: every G-th of them.  All lanes of a warp take the same
// number of turns.
struct Walk {
  int64_t t;
  int h, dt, dh, H, T;
  __device__ __forceinline__ Walk(int T, int H, int64_t first, int64_t step) : H(H), T(T) {
    t = first / H;
    h = (int)(first - t * H);
    dt = (int)min(step / H, (int64_t)0x7fffffff);
    dh = (int)(step - (step / H) * H);
  }
  __device__ __forceinline__ bool ok() const { return t < T; }
  __device__ __forceinline__ void next() {
    t += dt;
    h += dh;
    if (h >= H) {
      h -= H;
      ++t;
    }
  }
};
template <typename E>
__device__ __forceinline__ E *row_of(const Heads &x, const Walk &w) {
  return reinterpret_cast<E *>(x.p) + w.t * x.st + w.h * x.sh;
}

// f(z) and its derivative
__device__ __forceinline__ float gate_of(float z, int silu) {
  const float s = sigmoidf(z);
  return silu ? z * s : s;
}

template <typename E, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(kGated) k_gated_fwd(const GatedArgs a, int64_t turns) {
  after_previous();
  constexpr int RB = kGated / TPR;
  const int gl = threadIdx.x % TPR;
  Walk at(a.T, a.H, (int64_t)blockIdx.x * RB + threadIdx.x / TPR, (int64_t)gridDim.x * RB);
  float w[NV][8];
  int n[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (gl + j * TPR) * 8;
    n[j] = max(0, min(8, a.d - c));
    params8<VEC>(a.w, c, n[j], w[j]);
  }
  const float inv = 1.f / a.d;
  Raw8<E> x[NV], z[NV];
  auto load = [&] {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (gl + j * TPR) * 8, m = at.ok() ? n[j] : 0;
      x[j] = ld8<VEC>(row_of<E>(a.x, at) + c, m);
      z[j] = ld8<VEC>(row_of<E>(a.z, at) + c, m);
    }
  };
  load();
  for (int64_t i = 0; i < turns; ++i) {
    const Walk now = at;
    float xs[NV][8], zs[NV][8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack8(x[j], xs[j]);
      unpack8(z[j], zs[j]);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(xs[j][k], xs[j][k], sum);
    }
    at.next();
    load();
    sum = row_sum<TPR>(sum, nullptr, 0);
    const float r = rsqrtf(fmaf(sum, inv, a.eps));
    if (!now.ok()) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < 8; ++k) xs[j][k] *= r * w[j][k] * gate_of(zs[j][k], a.silu);
      st8<VEC>(row_of<E>(a.y, now) + (gl + j * TPR) * 8, pack8(xs[j], E{}), n[j]);
    }
  }
}

template <typename E, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(kGated) k_gated_bwd(const GatedArgs a, int64_t turns) {
  after_previous();
  constexpr int RB = kGated / TPR;
  extern __shared__ float sums[];  // [RB][TPR * NV * 8]
  const int gl = threadIdx.x % TPR, group = threadIdx.x / TPR;
  Walk at(a.T, a.H, (int64_t)blockIdx.x * RB + group, (int64_t)gridDim.x * RB);
  float w[NV][8], dw[NV][8];
  int n[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (gl + j * TPR) * 8;
    n[j] = max(0, min(8, a.d - c));
    params8<VEC>(a.w, c, n[j], w[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = 0.f;
  }
  const float inv = 1.f / a.d;
  Raw8<E> x[NV], z[NV], dy[NV];
  auto load = [&] {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (gl + j * TPR) * 8, m = at.ok() ? n[j] : 0;
      x[j] = ld8<VEC>(row_of<E>(a.x, at) + c, m);
      z[j] = ld8<VEC>(row_of<E>(a.z, at) + c, m);
      dy[j] = ld8<VEC>(row_of<E>(a.dy, at) + c, m);
    }
  };
  load();
  for (int64_t i = 0; i < turns; ++i) {
    const Walk now = at;
    float xs[NV][8], zs[NV][8], gs[NV][8];
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack8(x[j], xs[j]);
      unpack8(z[j], zs[j]);
      unpack8(dy[j], gs[j]);
    }
    at.next();
    load();
    float f[NV][8];  // f(z), then f'(z) dy w x
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float s = sigmoidf(zs[j][k]), v = a.silu ? zs[j][k] * s : s;
        const float dv = a.silu ? dsilu(zs[j][k], s) : s * (1.f - s);
        const float q = gs[j][k] * xs[j][k];  // dy x
        f[j][k] = q * w[j][k] * dv;
        zs[j][k] = q * v;              // dw's term but for r
        gs[j][k] = gs[j][k] * w[j][k] * v;  // e
        sum.x = fmaf(xs[j][k], xs[j][k], sum.x);
        sum.y = fmaf(gs[j][k], xs[j][k], sum.y);
      }
    sum = row_sum2<TPR>(sum, nullptr, 0);
    const float r = rsqrtf(fmaf(sum.x, inv, a.eps));
    if (!now.ok()) continue;
    const float back = r * r * sum.y * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dw[j][k] = fmaf(zs[j][k], r, dw[j][k]);
        f[j][k] *= r;
        if (TPR > 1) xs[j][k] = r * fmaf(-xs[j][k], back, gs[j][k]);
      }
      if (TPR == 1) row_back(xs[j], gs[j], a.d, a.eps, xs[j]);
      const int c = (gl + j * TPR) * 8;
      st8<VEC>(row_of<E>(a.dx, now) + c, pack8(xs[j], E{}), n[j]);
      st8<VEC>(row_of<E>(a.dz, now) + c, pack8(f[j], E{}), n[j]);
    }
  }
  if (!a.dw) return;
  constexpr int L = TPR * NV * 8;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[group * L + (gl + j * TPR) * 8 + k] = dw[j][k];
  __syncthreads();
  float *out = reinterpret_cast<float *>(a.work) + (int64_t)blockIdx.x * a.d;
  for (int c = threadIdx.x; c < a.d; c += kGated) {
    float v = sums[c];
#pragma unroll
    for (int g = 1; g < RB; ++g) v += sums[g * L + c];
    out[c] = v;
  }
}

bool fits16(const Heads &h, int e) {
  return reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.st * e % 16 == 0 && h.sh * e % 16 == 0;
}
bool fits16(const Mat &m, int e) {
  return !m.p || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.st * e % 16 == 0);
}
bool fits16(const Param &p) { return reinterpret_cast<uintptr_t>(p.p) % 16 == 0; }

int lanes_for(int d) {  // lanes of a row of up to 256 elements
  int l = 1;
  while (l * 8 < d) l *= 2;
  return l;
}
// Blocks: as many as run at once, or as the rows need.
int64_t gated_blocks(int64_t rows, int rows_per_block, int per_sm) {
  const int64_t most = (int64_t)sm_count() * per_sm, need = ceil_div64(rows, rows_per_block);
  return need < most ? need : most;
}
constexpr int kGatedPerSm = 8, kGatedBwdPerSm = 3;

template <typename E, int TPR, int NV, bool VEC>
cudaError_t run_gated(const GatedArgs &a, bool bwd, cudaStream_t stream) {
  constexpr int RB = kGated / TPR;
  const int64_t rows = (int64_t)a.T * a.H;
  if (!bwd) {
    const int64_t blocks = gated_blocks(rows, RB, kGatedPerSm);
    return launch(k_gated_fwd<E, TPR, NV, VEC>, (unsigned)blocks, kGated, 0, stream, a,
                  ceil_div64(rows, blocks * RB));
  }
  const int64_t blocks = gated_blocks(rows, RB, kGatedBwdPerSm);
  const int smem = a.dw ? RB * TPR * NV * 8 * 4 : 0;
  cudaError_t e = launch(k_gated_bwd<E, TPR, NV, VEC>, (unsigned)blocks, kGated, smem, stream, a,
                         ceil_div64(rows, blocks * RB));
  if (e != cudaSuccess || !a.dw) return e;
  return launch(k_sum_parts, dim3((unsigned)((a.d + 31) / 32)), 256, 0, stream,
                reinterpret_cast<const float *>(a.work), (int)blocks, (int64_t)a.d, a.d, a.dw,
                (float *)nullptr, (float *)nullptr);
}

template <typename E>
cudaError_t run_gated_for(const GatedArgs &a, bool bwd, cudaStream_t stream) {
  const int e = sizeof(E);
  bool vec = a.d % 8 == 0 && fits16(a.x, e) && fits16(a.z, e) && fits16(a.w);
  vec = vec && (bwd ? fits16(a.dy, e) && fits16(a.dx, e) && fits16(a.dz, e) : fits16(a.y, e));
  if (a.d > 512)
    return vec ? run_gated<E, 32, 4, true>(a, bwd, stream) : run_gated<E, 32, 4, false>(a, bwd, stream);
  if (a.d > 256)
    return vec ? run_gated<E, 32, 2, true>(a, bwd, stream) : run_gated<E, 32, 2, false>(a, bwd, stream);
  if (a.d <= 8)
    return vec ? run_gated<E, 1, 1, true>(a, bwd, stream) : run_gated<E, 1, 1, false>(a, bwd, stream);
  if (!vec) return a.d > 64 ? run_gated<E, 32, 1, false>(a, bwd, stream)
                            : run_gated<E, 8, 1, false>(a, bwd, stream);
  switch (lanes_for(a.d)) {
    case 32: return run_gated<E, 32, 1, true>(a, bwd, stream);
    case 16: return run_gated<E, 16, 1, true>(a, bwd, stream);
    case 8: return run_gated<E, 8, 1, true>(a, bwd, stream);
    default: return run_gated<E, 4, 1, true>(a, bwd, stream);
  }
}

// ------------------------------------------------------------------ residual norm

// A row of x and the residual to u (behind the block's norm and without the gate) and h.
template <int TPR, int NV, bool VEC>
struct Row {
  float rx;  // the first norm's factor
  __device__ __forceinline__ void make(const ResidArgs &a, float (&x)[NV][8], float (&res)[NV][8],
                                       const int (&n)[NV], int gl, float2 (*red)[32], int &phase) {
    rx = 1.f;
    if (a.post) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) s.x = fmaf(x[j][k], x[j][k], s.x);
      s = row_sum2<TPR>(s, red, phase);
      phase ^= 1;
      rx = rsqrtf(fmaf(s.x, 1.f / a.C, a.eps));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (gl + j * TPR) * 8;
      float p[8], g[8];
      params8<VEC>(a.wp, c, n[j], p);
      params8<VEC>(a.g, c, n[j], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) res[j][k] = fmaf(a.scale * g[k], x[j][k] * rx * p[k], res[j][k]);
    }
  }
};

template <typename E, typename R, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128) k_resid_fwd(const ResidArgs a) {
  after_previous<true>();
  constexpr int TH = TPR > 128 ? TPR : TPR > 32 ? TPR : 128, RB = TH / TPR;
  __shared__ float2 red[2][32];
  const int gl = threadIdx.x % TPR;
  int n[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) n[j] = max(0, min(8, a.C - (gl + j * TPR) * 8));
  int phase = 0;
  const int step = gridDim.x * RB;
  for (int64_t base = (int64_t)blockIdx.x * RB; base < a.T; base += step) {
    const int64_t t = base + threadIdx.x / TPR;
    const bool ok = t < a.T;
    float x[NV][8], h[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (gl + j * TPR) * 8, m = ok ? n[j] : 0;
      unpack8(ld8<VEC>(reinterpret_cast<const E *>(a.x.p) + t * a.x.st + c, m), x[j]);
      unpack8(a.res.p ? ld8<VEC>(reinterpret_cast<const R *>(a.res.p) + t * a.res.st + c, m)
                      : zero8<R>(),
              h[j]);
    }
    Row<TPR, NV, VEC> row;
    row.make(a, x, h, n, gl, red, phase);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) s.x = k < n[j] ? fmaf(h[j][k], h[j][k], s.x) : s.x;
    s = row_sum2<TPR>(s, red, phase);
    phase ^= 1;
    const float r = rsqrtf(fmaf(s.x, 1.f / a.C, a.eps));
    if (!ok) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (gl + j * TPR) * 8;
      if (a.h.p)
        st8<VEC>(reinterpret_cast<R *>(a.h.p) + t * a.h.st + c, pack8(h[j], R{}), n[j]);
      float w[8];
      params8<VEC>(a.w, c, n[j], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[j][k] *= r * w[k];
      st8<VEC>(reinterpret_cast<E *>(a.y.p) + t * a.y.st + c, pack8(h[j], E{}), n[j]);
    }
  }
}

// The rows of a block on their way into shared memory, `depth` of them: each thread reads only what
// it copied itself.  Without 16-byte alignment, and where a row is too long (fp32, over 8,192 columns),
// rows are loaded when they are used.
template <typename E, typename R, int TPR, int NV, bool VEC, int TH>
struct Rows4 {
  static constexpr int PE = sizeof(E) / 2, PR = sizeof(R) / 2, U = 2 * NV * (PE + PR);
  static constexpr bool kRing = VEC && U * TH * 16 <= 200 * 1024;
  uint4 *ring;
  template <typename X, int P>
  __device__ __forceinline__ void copy(int s, int unit, const Mat &m, int64_t t, int c) const {
    const X *p = reinterpret_cast<const X *>(m.p) + t * m.st + c;
#pragma unroll
    for (int i = 0; i < P; ++i) copy16(ring + (s * U + unit + i) * TH + threadIdx.x, p + i * (16 / sizeof(X)));
  }
  __device__ __forceinline__ void issue(const ResidArgs &a, int s, int64_t t, const int (&n)[NV],
                                        int gl) const {
    if (kRing) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (gl + j * TPR) * 8;
        if (t < a.T && n[j] > 0) {
          copy<E, PE>(s, j * PE, a.x, t, c);
          copy<E, PE>(s, (NV + j) * PE, a.dy, t, c);
          if (a.res.p) copy<R, PR>(s, 2 * NV * PE + j * PR, a.res, t, c);
          if (a.dh.p) copy<R, PR>(s, 2 * NV * PE + (NV + j) * PR, a.dh, t, c);
        }
      }
      copies_commit();
    }
  }
  template <typename X, int P>
  __device__ __forceinline__ Raw8<X> get(int s, int unit, const Mat &m, int64_t t, int c, int n) const {
    Raw8<X> r = zero8<X>();
    if (kRing) {
      uint4 *w = reinterpret_cast<uint4 *>(&r);
      if (m.p && n > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) w[i] = ring[(s * U + unit + i) * TH + threadIdx.x];
      }
    } else if (m.p) {
      r = ld8<VEC>(reinterpret_cast<const X *>(m.p) + t * m.st + c, n);
    }
    return r;
  }
};

template <typename E, typename R, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128) k_resid_bwd(const ResidArgs a, int depth) {
  after_previous();
  constexpr int TH = TPR > 32 ? TPR : 128, RB = TH / TPR;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 red[2][32];
  const Rows4<E, R, TPR, NV, VEC, TH> in{ring};
  using I = Rows4<E, R, TPR, NV, VEC, TH>;
  const int gl = threadIdx.x % TPR, group = threadIdx.x / TPR;
  int n[NV];
  float dw[NV][8], dp[NV][8], dg[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    n[j] = max(0, min(8, a.C - (gl + j * TPR) * 8));
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = dp[j][k] = dg[j][k] = 0.f;
  }
  const int step = gridDim.x * RB;
  const int64_t first = (int64_t)blockIdx.x * RB + group;
  for (int s = 0; s < depth - 1; ++s) in.issue(a, s, first + (int64_t)s * step, n, gl);
  int phase = 0, stage = 0;
  const float inv = 1.f / a.C;
  for (int64_t base = (int64_t)blockIdx.x * RB; base < a.T; base += step) {
    const int64_t t = base + group;
    const bool ok = t < a.T;
    // into the place of the row before; the oldest of `depth` rows is there then
    in.issue(a, stage == 0 ? depth - 1 : stage - 1, t + (int64_t)(depth - 1) * step, n, gl);
    if (I::kRing) {
      if (depth == 3) copies_wait<2>();
      else if (depth == 2) copies_wait<1>();
      else copies_wait<0>();
    }
    float x[NV][8], h[NV][8], dy[NV][8], dh[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (gl + j * TPR) * 8, m = ok ? n[j] : 0;
      unpack8(in.template get<E, I::PE>(stage, j * I::PE, a.x, t, c, m), x[j]);
      unpack8(in.template get<E, I::PE>(stage, (NV + j) * I::PE, a.dy, t, c, m), dy[j]);
      unpack8(in.template get<R, I::PR>(stage, 2 * NV * I::PE + j * I::PR, a.res, t, c, m), h[j]);
      unpack8(in.template get<R, I::PR>(stage, 2 * NV * I::PE + (NV + j) * I::PR, a.dh, t, c, m), dh[j]);
    }
    stage = stage + 1 == depth ? 0 : stage + 1;
    Row<TPR, NV, VEC> row;
    row.make(a, x, h, n, gl, red, phase);
    float2 s = make_float2(0.f, 0.f);
    float w[8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      params8<VEC>(a.w, (gl + j * TPR) * 8, n[j], w);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n[j]) {
          s.x = fmaf(h[j][k], h[j][k], s.x);
          s.y = fmaf(dy[j][k] * w[k], h[j][k], s.y);
        }
    }
    s = row_sum2<TPR>(s, red, phase);
    phase ^= 1;
    const float r = rsqrtf(fmaf(s.x, inv, a.eps)), back = r * r * s.y * inv;
    float2 q = make_float2(0.f, 0.f);
    if (ok) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (gl + j * TPR) * 8;
      float p[8], g[8];
      params8<VEC>(a.w, c, n[j], w);
      params8<VEC>(a.wp, c, n[j], p);
      params8<VEC>(a.g, c, n[j], g);
      float e[8];
      if (TPR == 1) {
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = k < n[j] ? dy[j][k] * w[k] : 0.f;
        row_back(h[j], e, a.C, a.eps, e);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dw[j][k] = fmaf(dy[j][k], h[j][k] * r, dw[j][k]);
        dh[j][k] = TPR > 1 ? fmaf(r, fmaf(-h[j][k], back, dy[j][k] * w[k]), dh[j][k]) : dh[j][k] + e[k];
        const float dv = a.scale * dh[j][k], xn = x[j][k] * row.rx, du = dv * g[k];
        dg[j][k] = fmaf(dv, xn * p[k], dg[j][k]);
        dp[j][k] = fmaf(du, xn, dp[j][k]);
        dy[j][k] = du * p[k];  // with the norm behind the block: e
        if (k < n[j]) q.x = fmaf(dy[j][k], x[j][k], q.x);
      }
      if (a.dres.p)
        st8<VEC>(reinterpret_cast<R *>(a.dres.p) + t * a.dres.st + c, pack8(dh[j], R{}), n[j]);
    }
    }
    float bx = 0.f;
    if (a.post) {
      q = row_sum2<TPR>(q, red, phase);
      phase ^= 1;
      bx = row.rx * row.rx * q.x * inv;
    }
    if (!ok) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (TPR > 1) dy[j][k] = row.rx * fmaf(-x[j][k], bx, dy[j][k]);
      if (TPR == 1 && a.post) row_back(x[j], dy[j], a.C, a.eps, dy[j]);
      st8<VEC>(reinterpret_cast<E *>(a.dx.p) + t * a.dx.st + (gl + j * TPR) * 8, pack8(dy[j], E{}),
               n[j]);
    }
  }
  if (I::kRing) copies_wait<0>();
  // the block's parts of dw, dw_post and dgate, its row groups in order
  float *out = reinterpret_cast<float *>(a.work) + (int64_t)blockIdx.x * 3 * a.C;
  if (RB == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n[j]) {
          const int c = (gl + j * TPR) * 8 + k;
          if (a.dw) out[c] = dw[j][k];
          if (a.dwp) out[a.C + c] = dp[j][k];
          if (a.dg) out[2 * a.C + c] = dg[j][k];
        }
  } else {
    __shared__ float sums[RB == 1 ? 1 : RB * TPR * NV * 8];
    constexpr int L = TPR * NV * 8;
    for (int i = 0; i < 3; ++i) {
      if (!(i == 0 ? a.dw : i == 1 ? a.dwp : a.dg)) continue;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sums[group * L + (gl + j * TPR) * 8 + k] = i == 0 ? dw[j][k] : i == 1 ? dp[j][k] : dg[j][k];
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += TH) {
        float v = sums[c];
#pragma unroll
        for (int g = 1; g < RB; ++g) v += sums[g * L + c];
        out[i * a.C + c] = v;
      }
    }
  }
}

// Blocks of the backward: as many as run at once; each leaves one row of parts.
constexpr int resid_per_sm(int threads) { return threads >= 512 ? 1 : threads >= 256 ? 2 : 4; }

template <typename E, typename R, int TPR, int NV, bool VEC>
cudaError_t run_resid(const ResidArgs &a, bool bwd, cudaStream_t stream) {
  constexpr int TH = TPR > 32 ? TPR : 128, RB = TH / TPR;
  const int64_t need = ceil_div64(a.T, RB);
  if (!bwd) {
    const int64_t most = (int64_t)sm_count() * (2048 / TH);
    return launch(k_resid_fwd<E, R, TPR, NV, VEC>, (unsigned)(need < most ? need : most), TH, 0,
                  stream, a);
  }
  using I = Rows4<E, R, TPR, NV, VEC, TH>;
  constexpr int unit = I::U * TH * 16, per_sm = resid_per_sm(TH);
  constexpr int fit = 200 * 1024 / per_sm / unit, depth = fit >= 3 ? 3 : fit == 2 ? 2 : 1;
  constexpr int smem = I::kRing ? depth * unit : 0;
  const int64_t most = (int64_t)sm_count() * per_sm;
  const int64_t blocks = need < most ? need : most;
  if (smem > 32 * 1024) {  // with the static shared memory above what needs no consent
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_once(k_resid_bwd<E, R, TPR, NV, VEC>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch(k_resid_bwd<E, R, TPR, NV, VEC>, (unsigned)blocks, TH, smem, stream, a, depth);
  if (e != cudaSuccess || !(a.dw || a.dwp || a.dg)) return e;
  return launch(k_sum_parts, dim3((unsigned)((a.C + 31) / 32), 3), 256, 0, stream,
                reinterpret_cast<const float *>(a.work), (int)blocks, (int64_t)3 * a.C, a.C, a.dw,
                a.dwp, a.dg);
}

template <typename E, typename R>
cudaError_t run_resid_for(const ResidArgs &a, bool bwd, cudaStream_t stream) {
  const int e = sizeof(E), f = sizeof(R);
  bool vec = a.C % 8 == 0 && fits16(a.x, e) && fits16(a.res, f) && fits16(a.w) && fits16(a.wp) &&
             fits16(a.g);
  vec = vec && (bwd ? fits16(a.dy, e) && fits16(a.dh, f) && fits16(a.dx, e) && fits16(a.dres, f)
                    : fits16(a.y, e) && fits16(a.h, f));
  const int C = a.C;
  if (C <= 8)
    return vec ? run_resid<E, R, 1, 1, true>(a, bwd, stream) : run_resid<E, R, 1, 1, false>(a, bwd, stream);
  if (!vec) {
    if (C <= 512) return run_resid<E, R, 32, 2, false>(a, bwd, stream);
    if (C <= 4096) return run_resid<E, R, 512, 1, false>(a, bwd, stream);
    return run_resid<E, R, 512, 4, false>(a, bwd, stream);
  }
  if (C <= 64) return run_resid<E, R, 8, 1, true>(a, bwd, stream);
  if (C <= 128) return run_resid<E, R, 16, 1, true>(a, bwd, stream);
  if (C <= 256) return run_resid<E, R, 32, 1, true>(a, bwd, stream);
  if (C <= 512) return run_resid<E, R, 64, 1, true>(a, bwd, stream);
  if (C <= 1024) return run_resid<E, R, 128, 1, true>(a, bwd, stream);
  if (C <= 2048) return run_resid<E, R, 256, 1, true>(a, bwd, stream);
  if (C <= 4096) return run_resid<E, R, 512, 1, true>(a, bwd, stream);
  if (C <= 8192) return run_resid<E, R, 512, 2, true>(a, bwd, stream);
  return run_resid<E, R, 512, 4, true>(a, bwd, stream);
}
cudaError_t run_resid_any(const ResidArgs &a, bool bwd, cudaStream_t stream) {
  if (a.f32) return run_resid_for<float, float>(a, bwd, stream);
  return a.rf32 ? run_resid_for<__nv_bfloat16, float>(a, bwd, stream)
                : run_resid_for<__nv_bfloat16, __nv_bfloat16>(a, bwd, stream);
}

__global__ void __launch_bounds__(256) k_zero(float *p, int n) {
  after_previous();
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) p[i] = 0.f;
}
// Without rows the parameters' gradients are zero.
cudaError_t zero(float *p, int n, cudaStream_t stream) {
  return p ? launch(k_zero, (n + 255) / 256, 256, 0, stream, p, n) : cudaSuccess;
}

}  // namespace
}  // namespace mix

cudaError_t launch_gated_fwd(const GatedArgs &a, cudaStream_t stream) {
  if ((int64_t)a.T * a.H == 0) return cudaSuccess;
  return a.f32 ? mix::run_gated_for<float>(a, false, stream)
               : mix::run_gated_for<__nv_bfloat16>(a, false, stream);
}
size_t gated_bwd_workspace(int64_t T, int32_t H, int32_t d) {
  return align256((size_t)mix::sm_count() * mix::kGatedBwdPerSm * d * 4);
}
cudaError_t launch_gated_bwd(const GatedArgs &a, cudaStream_t stream) {
  if ((int64_t)a.T * a.H == 0) return mix::zero(a.dw, a.d, stream);
  return a.f32 ? mix::run_gated_for<float>(a, true, stream)
               : mix::run_gated_for<__nv_bfloat16>(a, true, stream);
}
cudaError_t launch_resid_fwd(const ResidArgs &a, cudaStream_t stream) {
  return a.T == 0 ? cudaSuccess : mix::run_resid_any(a, false, stream);
}
size_t resid_bwd_workspace(int64_t T, int32_t C) {
  // one row of parts a block: no more blocks than rows, and four a multiprocessor at most
  const int64_t most = (int64_t)mix::sm_count() * 4;
  return align256((size_t)(T < most ? T : most) * 3 * C * 4);
}
cudaError_t launch_resid_bwd(const ResidArgs &a, cudaStream_t stream) {
  if (a.T == 0) {
    cudaError_t e = mix::zero(a.dw, a.C, stream);
    if (e == cudaSuccess) e = mix::zero(a.dwp, a.C, stream);
    return e == cudaSuccess ? mix::zero(a.dg, a.C, stream) : e;
  }
  return mix::run_resid_any(a, true, stream);
}

}  // namespace gdr
