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
// Bound by HBM: every tensor is read or written once, a row stays in registers between its sums.  Gated
// norm of 65,536 x 32 x 128 in bf16: 239 us, a copy's rate.  8,191 x 16 x 128, both directions: 47 us for 40
// of bytes.  Residual norm of 16,384 x 4,096 in bf16 with both norms and a gate: forward 85 us for 79 of
// bytes; backward 162 for 119: 16 warps of 124 registers an SM, of which 2.2 are ready in a cycle that issues,
// so that instructions count as much as bytes.  The blocks on a multiprocessor were chosen for bf16: in fp32
// the gated norm's forward spills some registers (32,768 x 16 x 128: 157 us for 119 of bytes, backward 311 for
// 198), and the residual norm of 16,384 x 4,096 takes 245 for 158 and 426 for 237.
#include "gdr_block.cuh"
#include "gdr_cluster.cuh"

namespace gdr {
namespace mix {
namespace {

// The sum of v over groups of TPR lanes, in all of them.
template <int TPR>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int TPR>
__device__ __forceinline__ float2 lane_sum2(float2 v) {
  v.x = lane_sum<TPR>(v.x);
  v.y = lane_sum<TPR>(v.y);
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

__device__ __forceinline__ f2 twice(float v) { return pair(v, v); }
__device__ __forceinline__ float total(f2 v) {
  float lo, hi;
  unpair(v, lo, hi);
  return lo + hi;
}

// 8 parameters from column c on in pairs; null: ones.
template <bool VEC>
__device__ __forceinline__ void params4(const Param &w, int64_t c, int n, f2 (&f)[4]) {
  float v[8];
  params8<VEC>(w, c, n, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(v[2 * i], v[2 * i + 1]);
}
// r (e - n mean(e n)) for a row of up to 8 columns in one thread (row_back), in pairs
__device__ __forceinline__ void row_back(const f2 (&x)[4], const f2 (&e)[4], int columns, float eps,
                                         f2 (&out)[4]) {
  float xs[8], es[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpair(x[i], xs[2 * i], xs[2 * i + 1]);
    unpair(e[i], es[2 * i], es[2 * i + 1]);
  }
  row_back(xs, es, columns, eps, es);
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = pair(es[2 * i], es[2 * i + 1]);
}

// out[c] = the sum of parts[b][c] over n blocks, in order: 32 warps take every 32nd.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) k_sum_parts(const float *parts, int n, int64_t stride,
                                                              int count, float *out0, float *out1,
                                                              float *out2) {
  after_previous();
  __shared__ float red[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float *out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
  if (!out) return;
  const float *p = parts + (int64_t)blockIdx.y * count + c;
  float v = 0.f;
  if (c < count) {
#pragma unroll 8
    for (int b = warp; b < n; b += kSumWarps) v += p[b * stride];
  }
  red[warp][lane] = v;
  __syncthreads();
  // a warp a column: its parts' sums by a butterfly
  v = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < count) out[col] = v;
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

// Blocks of the forward on each multiprocessor: all run at once.
constexpr int gated_per_sm(int NV) { return NV == 1 ? 5 : NV == 2 ? 3 : 1; }

template <typename E, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(kGated, gated_per_sm(NV)) k_gated_fwd(const GatedArgs a, int64_t turns) {
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
    sum = lane_sum<TPR>(sum);
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

// Rows come by cp.async into a ring in which each thread reads only what it copied itself, `depth` of
// them (0: rows are loaded when they are used); products in pairs.
template <typename E, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(kGated, NV == 4 ? 1 : 2) k_gated_bwd(const GatedArgs a, int64_t turns, int depth) {
  after_previous();
  constexpr int RB = kGated / TPR, P = sizeof(E) / 2;
  extern __shared__ __align__(16) uint4 ring[];  // then the blocks' parts of dw
  const int gl = threadIdx.x % TPR, group = threadIdx.x / TPR;
  Walk at(a.T, a.H, (int64_t)blockIdx.x * RB + group, (int64_t)gridDim.x * RB), ahead = at;
  f2 w[NV][4], dw[NV][4];
  int n[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (gl + j * TPR) * 8;
    n[j] = max(0, min(8, a.d - c));
    params4<VEC>(a.w, c, n[j], w[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = twice(0.f);
  }
  auto place = [&](int s, int unit) { return ring + (s * 3 * NV * P + unit) * kGated + threadIdx.x; };
  auto issue = [&](int s) {
    if (VEC && ahead.ok()) {
      const E *p[3] = {row_of<E>(a.x, ahead), row_of<E>(a.z, ahead), row_of<E>(a.dy, ahead)};
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (n[j] > 0) {
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i)
              copy16(place(s, (j * 3 + k) * P + i), p[k] + (gl + j * TPR) * 8 + i * (16 / sizeof(E)));
        }
    }
    copies_commit();
    ahead.next();
  };
  auto get = [&](int s, int j, int k, const Heads &m) {
    Raw8<E> r = zero8<E>();
    if (VEC) {
      uint4 *q = reinterpret_cast<uint4 *>(&r);
      if (at.ok() && n[j] > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) q[i] = *place(s, (j * 3 + k) * P + i);
      }
    } else {
      r = ld8<VEC>(row_of<E>(m, at) + (gl + j * TPR) * 8, at.ok() ? n[j] : 0);
    }
    return r;
  };
  if (VEC)
    for (int s = 0; s < depth - 1; ++s) issue(s);
  const float inv = 1.f / a.d;
  int stage = 0;
  for (int64_t t = 0; t < turns; ++t) {
    if (VEC) {
      issue(stage == 0 ? depth - 1 : stage - 1);
      if (depth >= 4) copies_wait<3>();
      else if (depth == 3) copies_wait<2>();
      else if (depth == 2) copies_wait<1>();
      else copies_wait<0>();
    }
    f2 x[NV][4], e[NV][4], f[NV][4], d[NV][4];  // x; dy w f(z); dy w f'(z) x; dy f(z) x
    f2 q = twice(0.f), p = twice(0.f);
    const f2 one = twice(1.f), minus = twice(-1.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 z[4];
      unpack4(get(stage, j, 0, a.x), x[j]);
      unpack4(get(stage, j, 1, a.z), z);
      unpack4(get(stage, j, 2, a.dy), e[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 s = sigmoid2(z[i]), g = a.silu ? mul2(z[i], s) : s;
        const f2 dg = a.silu ? dsilu2(z[i], s) : mul2(s, fma2(s, minus, one));
        const f2 yx = mul2(e[j][i], x[j][i]);
        d[j][i] = mul2(yx, g);
        f[j][i] = mul2(mul2(yx, w[j][i]), dg);
        e[j][i] = mul2(mul2(e[j][i], w[j][i]), g);
        q = fma2(x[j][i], x[j][i], q);
        p = fma2(e[j][i], x[j][i], p);
      }
    }
    stage = stage + 1 >= depth ? 0 : stage + 1;
    const float2 sum = lane_sum2<TPR>(make_float2(total(q), total(p)));
    const Walk now = at;
    at.next();
    if (!now.ok()) continue;
    const float r = rsqrtf(fmaf(sum.x, inv, a.eps)), back = r * r * sum.y * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[j][i] = fma2(d[j][i], twice(r), dw[j][i]);
        f[j][i] = mul2(f[j][i], twice(r));
        if (TPR > 1) e[j][i] = mul2(twice(r), fma2(x[j][i], twice(-back), e[j][i]));
      }
      if (TPR == 1) row_back(x[j], e[j], a.d, a.eps, e[j]);
      const int c = (gl + j * TPR) * 8;
      st8<VEC>(row_of<E>(a.dx, now) + c, pack4<E>(e[j]), n[j]);
      st8<VEC>(row_of<E>(a.dz, now) + c, pack4<E>(f[j]), n[j]);
    }
  }
  if (!a.dw) return;
  constexpr int L = TPR * NV * 8;
  float *sums = reinterpret_cast<float *>(ring);  // [RB][L]
  copies_wait<0>();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float *to = sums + group * L + (gl + j * TPR) * 8 + 2 * i;
      unpair(dw[j][i], to[0], to[1]);
    }
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
constexpr int kGatedBwdPerSm = 2;

template <typename E, int TPR, int NV, bool VEC>
cudaError_t run_gated(const GatedArgs &a, bool bwd, cudaStream_t stream) {
  constexpr int RB = kGated / TPR;
  const int64_t rows = (int64_t)a.T * a.H;
  if (!bwd) {
    const int64_t blocks = gated_blocks(rows, RB, gated_per_sm(NV));
    return launch(k_gated_fwd<E, TPR, NV, VEC>, (unsigned)blocks, kGated, 0, stream, a,
                  ceil_div64(rows, blocks * RB));
  }
  const int64_t blocks = gated_blocks(rows, RB, kGatedBwdPerSm), turns = ceil_div64(rows, blocks * RB);
  // rows ahead: up to four, what shared memory holds, and no more than a block has
  constexpr int unit = 3 * NV * (int)sizeof(E) / 2 * kGated * 16, fit = 96 * 1024 / unit;
  static_assert(fit >= 1, "a row fits");
  const int depth = !VEC ? 0 : turns < (fit < 4 ? fit : 4) ? (int)turns : fit < 4 ? fit : 4;
  constexpr int sums = RB * TPR * NV * 8 * 4;
  const int smem = depth * unit > sums ? depth * unit : sums;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = set_once(k_gated_bwd<E, TPR, NV, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024,
                 done);
  if (e != cudaSuccess) return e;
  e = launch(k_gated_bwd<E, TPR, NV, VEC>, (unsigned)blocks, kGated, smem, stream, a, turns, depth);
  if (e != cudaSuccess || !a.dw) return e;
  return launch(k_sum_parts, dim3((unsigned)((a.d + 31) / 32)), kSumWarps * 32, 0, stream,
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
  // loaded element by element, 8 neighbours a thread: 2.7 to 3.6 times the bytes' time (32,768 x 16 x 100 in bf16
  // 163 us, backward 277)
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
//
// A row is held by LANES lanes of a warp, several rows side by side, or (LANES 0) by a whole block of as
// many warps as it fills.  Products are in pairs.  Of two forms the first takes rows at any address, NV times
// 8 columns a thread, and loads them when they are used, element by element; the second takes rows at
// multiples of 16 bytes by cp.async into a ring in which each thread reads only what it copied itself.

// Sums over the threads of a row, in all of them.  With whole blocks `phase` names one of two places in
// red (which the next sum must not share).
template <int LANES>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 (*red)[32], int &phase) {
  constexpr int L = LANES ? LANES : 32;
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (LANES == 0) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[phase][threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[phase][0];
    for (int w = 1; w < warps; ++w) {
      v.x += red[phase][w].x;
      v.y += red[phase][w].y;
    }
    phase ^= 1;
  }
  return v;
}

// Columns behind the row's end (their parameters are zeros, or ones where there are none): zeros.
__device__ __forceinline__ void keep(f2 (&f)[4], int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpair(f[i], lo, hi);
    f[i] = pair(2 * i < n ? lo : 0.f, 2 * i + 1 < n ? hi : 0.f);
  }
}

// A thread's 8 columns of one row.
template <int LANES>
struct Cols {
  int first, n, group, groups;
  __device__ __forceinline__ Cols(int C) {
    const int tpr = LANES ? LANES : blockDim.x;
    first = threadIdx.x % tpr * 8;
    group = threadIdx.x / tpr;
    groups = blockDim.x / tpr;
    n = max(0, min(8, C - first));
  }
};

// Rows at any address: a thread has every S-th of 8 S columns, so that a warp's loads of one element a lane
// lie side by side (S = 32, but for rows in one thread; 4,000 x 4,098 in bf16 with neighbouring columns
// a thread: forward 114 us, backward 324; so: 50 and 270).
template <int LANES, int NV>
struct Spread {
  static constexpr int S = LANES == 1 ? 1 : 32;
  int group, groups, first, tpr;
  int n[NV];  // of the thread's columns, those that are there
  __device__ __forceinline__ Spread(int C) {
    tpr = LANES ? LANES : blockDim.x;
    const int gl = threadIdx.x % tpr;
    group = threadIdx.x / tpr;
    groups = blockDim.x / tpr;
    first = gl / S * 8 * S + gl % S;
#pragma unroll
    for (int j = 0; j < NV; ++j) n[j] = max(0, min(8, (C - at(j) + S - 1) / S));
  }
  __device__ __forceinline__ int at(int j) const { return first + j * tpr * 8; }
  __device__ __forceinline__ int at(int j, int i) const { return at(j) + i * S; }
};
template <int S>
__device__ __forceinline__ Raw8<__nv_bfloat16> gather8(const __nv_bfloat16 *p, int n) {
  const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? s[i * S] : 0;
  Raw8<__nv_bfloat16> r;
  r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  return r;
}
template <int S>
__device__ __forceinline__ Raw8<float> gather8(const float *p, int n) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i * S] : 0.f;
  return pack8(v, float{});
}
template <int S, typename X>
__device__ __forceinline__ void scatter8(X *p, const f2 (&f)[4], int n) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(f[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) st1(p + i * S, v[i]);
}
// n columns of row t from column c on, the others 0; no tensor: zeros.
template <int S, typename X>
__device__ __forceinline__ Raw8<X> row_part(const Mat &m, int64_t t, int c, int n) {
  return m.p ? gather8<S>(reinterpret_cast<const X *>(m.p) + t * m.st + c, n) : zero8<X>();
}
// Parameters; null: ones.
template <int S>
__device__ __forceinline__ void params_by(const Param &w, int c, int n, f2 (&f)[4]) {
  if (!w.p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = twice(1.f);
  } else if (w.bf16) {
    unpack4(gather8<S>(reinterpret_cast<const __nv_bfloat16 *>(w.p) + c, n), f);
  } else {
    unpack4(gather8<S>(reinterpret_cast<const float *>(w.p) + c, n), f);
  }
}

// u (behind the block's norm, without the gate) enters the residual: h.  Returns the norm's factor.
template <typename E, int LANES, int NV>
__device__ __forceinline__ float make_h(const ResidArgs &a, const Raw8<E> (&x)[NV], f2 (&h)[NV][4],
                                        const Spread<LANES, NV> &cols, float2 (*red)[32], int &phase) {
  constexpr int S = Spread<LANES, NV>::S;
  float rx = 1.f;
  if (a.post) {
    f2 q = twice(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 v[4];
      unpack4(x[j], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(v[i], v[i], q);
    }
    rx = rsqrtf(fmaf(row_sum2<LANES>(make_float2(total(q), 0.f), red, phase).x, 1.f / a.C, a.eps));
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    f2 v[4], p[4];
    unpack4(x[j], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], twice(a.scale * rx));
    if (a.wp.p) {
      params_by<S>(a.wp, cols.at(j), cols.n[j], p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], p[i]);
    }
    if (a.g.p) {
      params_by<S>(a.g, cols.at(j), cols.n[j], p);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = fma2(v[i], p[i], h[j][i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = add2(v[i], h[j][i]);
    }
    if (cols.n[j] < 8) keep(h[j], cols.n[j]);
  }
  return rx;
}

constexpr int kResidMost = 512;  // threads of a block

template <typename E, typename R, int LANES, int NV>
__global__ void __launch_bounds__(LANES ? 128 : kResidMost, LANES ? 1 : 2)
    k_resid_fwd_any(const ResidArgs a) {
  after_previous<true>();
  __shared__ float2 red[2][32];
  const Spread<LANES, NV> cols(a.C);
  constexpr int S = Spread<LANES, NV>::S;
  const int step = gridDim.x * cols.groups;
  int phase = 0;
  for (int64_t base = (int64_t)blockIdx.x * cols.groups; base < a.T; base += step) {
    const int64_t t = base + cols.group;
    const bool ok = t < a.T;
    Raw8<E> x[NV];
    f2 h[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int m = ok ? cols.n[j] : 0;
      x[j] = row_part<S, E>(a.x, t, cols.at(j), m);
      unpack4(row_part<S, R>(a.res, t, cols.at(j), m), h[j]);
    }
    make_h<E, LANES, NV>(a, x, h, cols, red, phase);
    f2 q = twice(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(h[j][i], h[j][i], q);
    const float2 s = row_sum2<LANES>(make_float2(total(q), 0.f), red, phase);
    const float r = rsqrtf(fmaf(s.x, 1.f / a.C, a.eps));
    if (!ok) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = cols.at(j);
      if (a.h.p)
        scatter8<S>(reinterpret_cast<R *>(a.h.p) + t * a.h.st + c, h[j], cols.n[j]);
      f2 w[4];
      params_by<S>(a.w, c, cols.n[j], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = mul2(mul2(h[j][i], twice(r)), w[i]);
      scatter8<S>(reinterpret_cast<E *>(a.y.p) + t * a.y.st + c, h[j], cols.n[j]);
    }
  }
}

template <typename E, typename R, int LANES, int NV>
__global__ void __launch_bounds__(LANES ? 128 : kResidMost, 1) k_resid_bwd_any(const ResidArgs a) {
  after_previous();
  __shared__ float2 red[2][32];
  const Spread<LANES, NV> cols(a.C);
  constexpr int S = Spread<LANES, NV>::S;
  f2 dw[NV][4], dp[NV][4], dg[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = dp[j][i] = dg[j][i] = twice(0.f);
  const int step = gridDim.x * cols.groups;
  int phase = 0;
  const float inv = 1.f / a.C;
  for (int64_t base = (int64_t)blockIdx.x * cols.groups; base < a.T; base += step) {
    const int64_t t = base + cols.group;
    const bool ok = t < a.T;
    Raw8<E> x[NV], dy[NV];
    f2 h[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int m = ok ? cols.n[j] : 0;
      x[j] = row_part<S, E>(a.x, t, cols.at(j), m);
      dy[j] = row_part<S, E>(a.dy, t, cols.at(j), m);
      unpack4(row_part<S, R>(a.res, t, cols.at(j), m), h[j]);
    }
    const float rx = make_h<E, LANES, NV>(a, x, h, cols, red, phase);
    f2 q = twice(0.f), p = twice(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 w[4], e[4];
      params_by<S>(a.w, cols.at(j), cols.n[j], w);
      unpack4(dy[j], e);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q = fma2(h[j][i], h[j][i], q);
        p = fma2(mul2(e[i], w[i]), h[j][i], p);
      }
    }
    const float2 s = row_sum2<LANES>(make_float2(total(q), total(p)), red, phase);
    const float r = rsqrtf(fmaf(s.x, inv, a.eps)), back = r * r * s.y * inv;
    q = twice(0.f);
    f2 du[NV][4];  // the gradient behind the gate; with the norm behind the block, times its weight
    if (ok) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = cols.at(j);
        f2 w[4], e[4], g[4], xs[4];
        params_by<S>(a.w, c, cols.n[j], w);
        unpack4(dy[j], e);
        unpack4(row_part<S, R>(a.dh, t, c, cols.n[j]), g);
        unpack4(x[j], xs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dw[j][i] = fma2(e[i], mul2(h[j][i], twice(r)), dw[j][i]);
          e[i] = mul2(e[i], w[i]);
        }
        if (LANES == 1) {
          row_back(h[j], e, a.C, a.eps, e);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = add2(g[i], e[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            g[i] = fma2(twice(r), fma2(h[j][i], twice(-back), e[i]), g[i]);
        }
        if (a.dres.p)
          scatter8<S>(reinterpret_cast<R *>(a.dres.p) + t * a.dres.st + c, g, cols.n[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = mul2(g[i], twice(a.scale));
          e[i] = mul2(xs[i], twice(rx));
        }
        if (a.wp.p) {
          params_by<S>(a.wp, c, cols.n[j], w);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = twice(1.f);
        }
        if (a.g.p) {
          f2 gate[4];
          params_by<S>(a.g, c, cols.n[j], gate);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dg[j][i] = fma2(g[i], mul2(e[i], w[i]), dg[j][i]);
            g[i] = mul2(g[i], gate[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dp[j][i] = fma2(g[i], e[i], dp[j][i]);
          du[j][i] = mul2(g[i], w[i]);
        }
        if (a.post) {
          if (cols.n[j] < 8) keep(du[j], cols.n[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) q = fma2(du[j][i], xs[i], q);
        }
      }
    }
    float bx = 0.f;
    if (a.post) bx = rx * rx * row_sum2<LANES>(make_float2(total(q), 0.f), red, phase).x * inv;
    if (!ok) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 xs[4];
      unpack4(x[j], xs);
      if (LANES == 1 && a.post) {
        row_back(xs, du[j], a.C, a.eps, du[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) du[j][i] = mul2(twice(rx), fma2(xs[i], twice(-bx), du[j][i]));
      }
      scatter8<S>(reinterpret_cast<E *>(a.dx.p) + t * a.dx.st + cols.at(j), du[j], cols.n[j]);
    }
  }
  // the block's parts of dw, dw_post and dgate, its row groups in order
  float *out = reinterpret_cast<float *>(a.work) + (int64_t)blockIdx.x * 3 * a.C;
  if (LANES == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 v[3] = {dw[j][i], dp[j][i], dg[j][i]};
#pragma unroll
        for (int b = 0; b < 3; ++b) {
          if (!(b == 0 ? a.dw : b == 1 ? a.dwp : a.dg)) continue;
          float lo, hi;
          unpair(v[b], lo, hi);
          float *to = out + (int64_t)b * a.C;
          if (2 * i < cols.n[j]) to[cols.at(j, 2 * i)] = lo;
          if (2 * i + 1 < cols.n[j]) to[cols.at(j, 2 * i + 1)] = hi;
        }
      }
  } else {
    constexpr int L = (LANES ? LANES : 1) * NV * 8;
    __shared__ float sums[LANES ? 128 / (LANES ? LANES : 1) * L : 1];
    for (int b = 0; b < 3; ++b) {
      if (!(b == 0 ? a.dw : b == 1 ? a.dwp : a.dg)) continue;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float *to = &sums[cols.group * L];
          unpair(b == 0 ? dw[j][i] : b == 1 ? dp[j][i] : dg[j][i], to[cols.at(j, 2 * i)],
                 to[cols.at(j, 2 * i + 1)]);
        }
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += 128) {
        float v = sums[c];
        for (int g = 1; g < 128 / (LANES ? LANES : 1); ++g) v += sums[g * L + c];
        out[(int64_t)b * a.C + c] = v;
      }
    }
  }
}

// ------------------------------------------------------------------ rows of 16-byte vectors
//
// One vector of 8 columns a thread, whose parameters stay in registers, and NR rows at a time, which
// share the exchanges between warps.  Rows of more columns than a block holds so (forward 8,192, backward
// 4,096, whose three gradients leave room for 512 threads) lie on a cluster of blocks (WIDE): 2 and 4
// vectors a thread in one block spilled (backward of 8,192 x 8,192 in bf16 381 us, on two blocks 235;
// 4,096 x 16,384 554, on four 256; forward of the latter 146, on two 110).

// Sums of K values over the threads of a row, in all of them: a butterfly in which half of the values
// change places while there is more than one, and for whole blocks the same once more over the
// warps' sums.
// The values from `from` to `to` count, the others come out as anything.  WIDE: over the blocks of a
// cluster, whose sums go to every one of them; a place is written again after a barrier that its readers
// came to behind their reading.
constexpr int kSums = 32 * 8;  // of a row: 64 warps' or 32 of two values, 64 of four
template <int LANES, int K, bool WIDE>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*red)[kSums], int &phase, int from = 0,
                                         int to = K) {
  static_assert(K == 1 || K == 2 || K == 4, "values");
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < from || k >= to) v[k] = 0.f;
  constexpr int L = LANES ? LANES : 32;
  const int lane = threadIdx.x & 31;
  if (LANES) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    return;
  }
  float m = v[0];  // value lane % K, summed over more and more lanes
  if (K == 4) {
    const bool up = lane & 2;
    const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 2);
    const float b = (up ? v[K - 1] : v[K > 1 ? 1 : 0]) +
                    __shfl_xor_sync(0xffffffffu, up ? v[K > 1 ? 1 : 0] : v[K - 1], 2);
    m = (lane & 1 ? b : a) + __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
  } else if (K == 2) {
    m = (lane & 1 ? v[K - 1] : v[0]) + __shfl_xor_sync(0xffffffffu, lane & 1 ? v[0] : v[K - 1], 1);
  }
#pragma unroll
  for (int o = K; o < 32; o <<= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
  int warps = blockDim.x >> 5;
  if (WIDE) {  // to all blocks of the cluster
    const int size = cluster_size(), at = (cluster_rank() * warps + (int)(threadIdx.x >> 5)) * K + lane;
    if (lane < K)
      for (int b = 0; b < size; ++b)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at_rank(&red[phase][at], b)), "f"(m) : "memory");
    cluster_arrive();
    cluster_wait();
    warps *= size;
  } else {
    if (lane < K) red[phase][(threadIdx.x >> 5) * K + lane] = m;
    __syncthreads();
  }
  m = 0.f;
  for (int i = lane; i < warps * K; i += 32) m += red[phase][i];
#pragma unroll
  for (int o = K; o < 32; o <<= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, m, k);
  phase ^= 1;
}

// A thread's parameters: weight, post_weight, and scale times gate; zeros behind the last column.
struct Params {
  f2 w[4], p[4], g[4];
  __device__ __forceinline__ Params(const ResidArgs &a, int c, int n) {
    params4<true>(a.w, c, n, w);
    params4<true>(a.wp, c, n, p);
    params4<true>(a.g, c, n, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = n > 0 ? mul2(g[i], twice(a.scale)) : twice(0.f);
  }
};

// The rows of a step: x, residual (, dy, dh) of NR rows, one vector a thread.
template <typename E, typename R, int NR, bool BWD>
struct Ahead {
  static constexpr int PE = sizeof(E) / 2, PR = sizeof(R) / 2;
  static constexpr int kX = 0, kRes = PE, kDy = PE + PR, kDh = 2 * PE + PR;
  static constexpr int kRow = (BWD ? 2 : 1) * (PE + PR), kUnits = NR * kRow;
  uint4 *ring;
  const ResidArgs &a;
  int c, n;
  __device__ __forceinline__ uint4 *place(int s, int r, int unit) const {
    return ring + (s * kUnits + r * kRow + unit) * blockDim.x + threadIdx.x;
  }
  template <typename X>
  __device__ __forceinline__ void copy(int s, int r, int unit, const Mat &m, int64_t t) const {
    const X *p = reinterpret_cast<const X *>(m.p) + t * m.st + c;
#pragma unroll
    for (int i = 0; i < (int)sizeof(X) / 2; ++i) copy16(place(s, r, unit + i), p + i * (16 / sizeof(X)));
  }
  __device__ __forceinline__ void issue(int s, int64_t t) const {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (t + r < a.T && n > 0) {
        copy<E>(s, r, kX, a.x, t + r);
        if (a.res.p) copy<R>(s, r, kRes, a.res, t + r);
        if (BWD) copy<E>(s, r, kDy, a.dy, t + r);
        if (BWD && a.dh.p) copy<R>(s, r, kDh, a.dh, t + r);
      }
    }
    copies_commit();
  }
  __device__ __forceinline__ void wait(int depth) const {  // the oldest of `depth` steps is there
    if (depth >= 4) copies_wait<3>();
    else if (depth == 3) copies_wait<2>();
    else if (depth == 2) copies_wait<1>();
    else copies_wait<0>();
  }
  template <typename X>
  __device__ __forceinline__ Raw8<X> get(int s, int r, int unit, bool there) const {
    Raw8<X> v = zero8<X>();
    uint4 *w = reinterpret_cast<uint4 *>(&v);
    if (there) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(X) / 2; ++i) w[i] = *place(s, r, unit + i);
    }
    return v;
  }
};

// The sums of x^2 over this thread's columns of a step's rows, from the ring.
template <typename E, typename In, int NR>
__device__ __forceinline__ void squares(const In &in, int s, int64_t t, float *sum) {
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    f2 v[4], q = twice(0.f);
    unpack4(in.template get<E>(s, r, In::kX, t + r < in.a.T && in.n > 0), v);
#pragma unroll
    for (int i = 0; i < 4; ++i) q = fma2(v[i], v[i], q);
    sum[r] = total(q);
  }
}

// Both kernels take the first norm's sums of the step after this one along with this one's last sums:
// one exchange less a step.

template <typename E, typename R, int LANES, int NR, bool WIDE>
__global__ void __launch_bounds__(LANES ? 128 : 1024, 1) k_resid_fwd(const ResidArgs a, int depth) {
  after_previous<true>();
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float red[2][kSums];
  const Cols<LANES> cols(a.C);
  const int size = WIDE ? cluster_size() : 1, block = blockIdx.x / size, blocks = gridDim.x / size;
  const int c = cols.first + (WIDE ? cluster_rank() * (int)blockDim.x * 8 : 0);
  const int n = WIDE ? max(0, min(8, a.C - c)) : cols.n;
  using In = Ahead<E, R, NR, false>;
  const In in{ring, a, c, n};
  const int step = blocks * cols.groups * NR;
  const int64_t first = ((int64_t)block * cols.groups + cols.group) * NR;
  for (int s = 0; s < depth - 1; ++s) in.issue(s, first + (int64_t)s * step);
  const Params par(a, c, n);
  if (WIDE) {  // every block of the cluster runs before one writes to it
    cluster_arrive();
    cluster_wait();
  }
  int phase = 0, stage = 0;
  const float inv = 1.f / a.C;
  float sum[2 * NR];  // of h^2, and of x^2 in the next step
  in.wait(depth - 1);
  if (a.post) {
    squares<E, In, NR>(in, 0, first, sum + NR);
    row_sums<LANES, 2 * NR, WIDE>(sum, red, phase, NR);
  }
  for (int64_t base = (int64_t)block * cols.groups * NR; base < a.T; base += step) {
    const int64_t t = base + cols.group * NR;
    in.issue(stage == 0 ? depth - 1 : stage - 1, t + (int64_t)(depth - 1) * step);
    f2 h[NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const bool there = t + r < a.T && n > 0;
      const float rx = a.post ? rsqrtf(fmaf(sum[NR + r], inv, a.eps)) : 1.f;
      f2 v[4], q = twice(0.f);
      unpack4(in.template get<E>(stage, r, In::kX, there), v);
      unpack4(in.template get<R>(stage, r, In::kRes, there && a.res.p), h[r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[r][i] = fma2(mul2(mul2(v[i], twice(rx)), par.p[i]), par.g[i], h[r][i]);
        q = fma2(h[r][i], h[r][i], q);
      }
      sum[r] = n > 0 ? total(q) : 0.f;
    }
    stage = stage + 1 == depth ? 0 : stage + 1;
    in.wait(depth - 1);
    if (a.post) {
      squares<E, In, NR>(in, stage, t + step, sum + NR);
      row_sums<LANES, 2 * NR, WIDE>(sum, red, phase);
    } else {
      row_sums<LANES, 2 * NR, WIDE>(sum, red, phase, 0, NR);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (t + r >= a.T || n <= 0) continue;
      if (a.h.p)
        st8<true>(reinterpret_cast<R *>(a.h.p) + (t + r) * a.h.st + c, pack4<R>(h[r]), 8);
      const float f = rsqrtf(fmaf(sum[r], inv, a.eps));
#pragma unroll
      for (int i = 0; i < 4; ++i) h[r][i] = mul2(mul2(h[r][i], twice(f)), par.w[i]);
      st8<true>(reinterpret_cast<E *>(a.y.p) + (t + r) * a.y.st + c, pack4<E>(h[r]), 8);
    }
  }
  copies_wait<0>();
}

template <typename E, typename R, int LANES, int NR, bool WIDE>
__global__ void __launch_bounds__(LANES ? 128 : 512, 1) k_resid_bwd(const ResidArgs a, int depth) {
  after_previous();
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float red[2][kSums];
  const Cols<LANES> cols(a.C);
  const int size = WIDE ? cluster_size() : 1, block = blockIdx.x / size, blocks = gridDim.x / size;
  const int c = cols.first + (WIDE ? cluster_rank() * (int)blockDim.x * 8 : 0);
  const int n = WIDE ? max(0, min(8, a.C - c)) : cols.n;
  using In = Ahead<E, R, NR, true>;
  const In in{ring, a, c, n};
  const int step = blocks * cols.groups * NR;
  const int64_t first = ((int64_t)block * cols.groups + cols.group) * NR;
  for (int s = 0; s < depth - 1; ++s) in.issue(s, first + (int64_t)s * step);
  const Params par(a, c, n);
  f2 dw[4], dp[4], dg[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = dp[i] = dg[i] = twice(0.f);
  if (WIDE) {  // every block of the cluster runs before one writes to it
    cluster_arrive();
    cluster_wait();
  }
  int phase = 0, stage = 0;
  const float inv = 1.f / a.C;
  float last[2 * NR];  // the sums of the norm behind the block, and of x^2 in the next step
  in.wait(depth - 1);
  if (a.post) {
    squares<E, In, NR>(in, 0, first, last + NR);
    row_sums<LANES, 2 * NR, WIDE>(last, red, phase, NR);
  }
  for (int64_t base = (int64_t)block * cols.groups * NR; base < a.T; base += step) {
    const int64_t t = base + cols.group * NR;
    in.issue(stage == 0 ? depth - 1 : stage - 1, t + (int64_t)(depth - 1) * step);
    f2 h[NR][4];  // then the gradient behind the gate; with the norm behind the block, times its weight
    float sum[2 * NR], rx[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const bool there = t + r < a.T && n > 0;
      rx[r] = a.post ? rsqrtf(fmaf(last[NR + r], inv, a.eps)) : 1.f;
      f2 v[4], e[4], q = twice(0.f), p = twice(0.f);
      unpack4(in.template get<E>(stage, r, In::kX, there), v);
      unpack4(in.template get<E>(stage, r, In::kDy, there), e);
      unpack4(in.template get<R>(stage, r, In::kRes, there && a.res.p), h[r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[r][i] = fma2(mul2(mul2(v[i], twice(rx[r])), par.p[i]), par.g[i], h[r][i]);
        q = fma2(h[r][i], h[r][i], q);
        p = fma2(mul2(e[i], par.w[i]), h[r][i], p);
      }
      sum[2 * r] = n > 0 ? total(q) : 0.f;
      sum[2 * r + 1] = n > 0 ? total(p) : 0.f;
    }
    row_sums<LANES, 2 * NR, WIDE>(sum, red, phase);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      last[r] = 0.f;
      if (t + r >= a.T || n <= 0) continue;
      const float f = rsqrtf(fmaf(sum[2 * r], inv, a.eps)), back = f * f * sum[2 * r + 1] * inv;
      f2 e[4], g[4], v[4], q = twice(0.f);
      unpack4(in.template get<E>(stage, r, In::kDy, true), e);
      unpack4(in.template get<R>(stage, r, In::kDh, a.dh.p), g);
      if (LANES == 1) {
        f2 ew[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ew[i] = mul2(e[i], par.w[i]);
          dw[i] = fma2(e[i], mul2(h[r][i], twice(f)), dw[i]);
        }
        row_back(h[r], ew, a.C, a.eps, ew);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = add2(g[i], ew[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dw[i] = fma2(e[i], mul2(h[r][i], twice(f)), dw[i]);
          g[i] = fma2(twice(f), fma2(h[r][i], twice(-back), mul2(e[i], par.w[i])), g[i]);
        }
      }
      if (a.dres.p)
        st8<true>(reinterpret_cast<R *>(a.dres.p) + (t + r) * a.dres.st + c, pack4<R>(g), 8);
      unpack4(in.template get<E>(stage, r, In::kX, true), v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = mul2(v[i], twice(rx[r]));  // n_x
        dg[i] = fma2(g[i], mul2(v[i], par.p[i]), dg[i]);  // but for the scale
        g[i] = mul2(g[i], par.g[i]);
        dp[i] = fma2(g[i], v[i], dp[i]);
        h[r][i] = mul2(g[i], par.p[i]);
        q = fma2(h[r][i], v[i], q);
      }
      last[r] = total(q);
    }
    const int here = stage;
    stage = stage + 1 == depth ? 0 : stage + 1;
    in.wait(depth - 1);
    if (a.post) {
      squares<E, In, NR>(in, stage, t + step, last + NR);
      row_sums<LANES, 2 * NR, WIDE>(last, red, phase);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (t + r >= a.T || n <= 0) continue;
      if (a.post) {
        f2 v[4];
        unpack4(in.template get<E>(here, r, In::kX, true), v);
        if (LANES == 1) {
          row_back(v, h[r], a.C, a.eps, h[r]);
        } else {
          const float b = -rx[r] * last[r] * inv;  // n_x mean(e n_x) = x times this
#pragma unroll
          for (int i = 0; i < 4; ++i) h[r][i] = mul2(twice(rx[r]), fma2(v[i], twice(b), h[r][i]));
        }
      }
      st8<true>(reinterpret_cast<E *>(a.dx.p) + (t + r) * a.dx.st + c, pack4<E>(h[r]), 8);
    }
  }
  copies_wait<0>();
  // the block's parts of dw, dw_post and dgate, its row groups in order
  float *out = reinterpret_cast<float *>(a.work) + (int64_t)block * 3 * a.C;
  constexpr int L = LANES ? LANES : 1;
  __shared__ float sums[LANES ? 128 * 8 : 1];
#pragma unroll
  for (int b = 0; b < 3; ++b) {
    if (!(b == 0 ? a.dw : b == 1 ? a.dwp : a.dg)) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      unpair(b == 0 ? dw[i] : b == 1 ? dp[i] : mul2(dg[i], twice(a.scale)), v[2 * i], v[2 * i + 1]);
    float *to = out + (int64_t)b * a.C;
    if (LANES == 0) {
      if (n > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) to[c + i] = v[i];
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[cols.group * L * 8 + c + i] = v[i];
      __syncthreads();
      for (int col = threadIdx.x; col < a.C; col += 128) {
        float s = sums[col];
        for (int g = 1; g < 128 / L; ++g) s += sums[g * L * 8 + col];
        to[col] = s;
      }
    }
  }
}

// Threads that share the register file and shared memory of a multiprocessor in the backward.
constexpr int kResidThreads = 512, kResidBlocks = 4;

cudaError_t sum_parts(const ResidArgs &a, int64_t blocks, cudaStream_t stream) {
  if (!(a.dw || a.dwp || a.dg)) return cudaSuccess;
  return launch(k_sum_parts, dim3((unsigned)((a.C + 31) / 32), 3), kSumWarps * 32, 0, stream,
                reinterpret_cast<const float *>(a.work), (int)blocks, (int64_t)3 * a.C, a.C, a.dw, a.dwp,
                a.dg);
}

template <typename E, typename R, int LANES, int NV>
cudaError_t run_resid_unaligned(const ResidArgs &a, bool bwd, cudaStream_t stream) {
  // a block of as many warps as a row fills, or 128 threads with a row for every LANES of them
  const int th = LANES ? 128 : (a.C + NV * 256 - 1) / (NV * 256) * 32;
  const int64_t need = ceil_div64(a.T, LANES ? 128 / LANES : 1);
  int per_sm = (bwd ? kResidThreads : 1024) / th;
  per_sm = per_sm < 1 ? 1 : bwd && per_sm > kResidBlocks ? kResidBlocks : per_sm;
  const int64_t most = (int64_t)sm_count() * per_sm, blocks = need < most ? need : most;
  if (!bwd) return launch(k_resid_fwd_any<E, R, LANES, NV>, (unsigned)blocks, th, 0, stream, a);
  const cudaError_t e = launch(k_resid_bwd_any<E, R, LANES, NV>, (unsigned)blocks, th, 0, stream, a);
  return e == cudaSuccess ? sum_parts(a, blocks, stream) : e;
}

template <typename E, typename R, int LANES, int NR>
cudaError_t run_resid(const ResidArgs &a, bool bwd, cudaStream_t stream) {
  const int th = LANES ? 128 : (a.C + 255) / 256 * 32;
  const int64_t need = ceil_div64(a.T, (LANES ? 128 / LANES : 1) * NR);
  const int unit = (bwd ? Ahead<E, R, NR, true>::kUnits : Ahead<E, R, NR, false>::kUnits) * th * 16;
  int per_sm = (bwd ? kResidThreads : 1024) / th;
  per_sm = per_sm < 1 ? 1 : bwd && per_sm > kResidBlocks ? kResidBlocks : per_sm;
  const int64_t most = (int64_t)sm_count() * per_sm, blocks = need < most ? need : most;
  // steps ahead: what shared memory holds, up to four, and no more than a block has
  const int64_t turns = ceil_div64(need, blocks);
  int depth = 200 * 1024 / per_sm / unit;
  depth = depth > 4 ? 4 : depth;
  if (turns < depth) depth = (int)turns;
  if (depth < 2) depth = 2;  // the step that is worked on, and the next one's first sums
  const int smem = depth * unit;
  static std::atomic<uint64_t> done[2];
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024)  // with the static shared memory above what needs no consent
    e = bwd ? set_once(k_resid_bwd<E, R, LANES, NR, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       200 * 1024, done[1])
            : set_once(k_resid_fwd<E, R, LANES, NR, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       200 * 1024, done[0]);
  if (e != cudaSuccess) return e;
  if (!bwd)
    return launch(k_resid_fwd<E, R, LANES, NR, false>, (unsigned)blocks, th, smem, stream, a, depth);
  e = launch(k_resid_bwd<E, R, LANES, NR, false>, (unsigned)blocks, th, smem, stream, a, depth);
  return e == cudaSuccess ? sum_parts(a, blocks, stream) : e;
}

// Rows of a cluster of blocks, as few as hold them.
template <typename E, typename R, int NR>
cudaError_t run_resid_wide(const ResidArgs &a, bool bwd, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  static std::atomic<int> known[2][64][kMostCl + 1];
  const auto kernel = bwd ? k_resid_bwd<E, R, 0, NR, true> : k_resid_fwd<E, R, 0, NR, true>;
  const int most = bwd ? 512 : 1024, cl = (a.C + most * 8 - 1) / (most * 8);
  const int th = (a.C + cl * 256 - 1) / (cl * 256) * 32;
  const int unit = (bwd ? Ahead<E, R, NR, true>::kUnits : Ahead<E, R, NR, false>::kUnits) * th * 16;
  cudaError_t e = set_once(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024, done[bwd]);
  if (e != cudaSuccess) return e;
  int clusters = clusters_at_once(kernel, cl, most, 200 * 1024, known[bwd]);
  if (clusters < 1) clusters = sm_count() / cl;
  const int64_t need = ceil_div64(a.T, NR);
  if (need < clusters) clusters = (int)need;
  const int64_t turns = ceil_div64(need, clusters);
  int depth = 200 * 1024 / unit;
  depth = depth > 4 ? 4 : depth;
  if (turns < depth) depth = (int)turns;
  if (depth < 2) depth = 2;
  e = launch_clusters(kernel, clusters * cl, cl, th, depth * unit, stream, a, depth);
  return e == cudaSuccess && bwd ? sum_parts(a, clusters, stream) : e;
}

template <typename E, typename R>
cudaError_t run_resid_for(const ResidArgs &a, bool bwd, cudaStream_t stream) {
  const int e = sizeof(E), f = sizeof(R);
  bool vec = a.C % 8 == 0 && fits16(a.x, e) && fits16(a.res, f) && fits16(a.w) && fits16(a.wp) &&
             fits16(a.g);
  vec = vec && (bwd ? fits16(a.dy, e) && fits16(a.dh, f) && fits16(a.dx, e) && fits16(a.dres, f)
                    : fits16(a.y, e) && fits16(a.h, f));
  const int C = a.C;
  if (!vec) {
    if (C <= 8) return run_resid_unaligned<E, R, 1, 1>(a, bwd, stream);
    if (C <= 256) return run_resid_unaligned<E, R, 32, 1>(a, bwd, stream);
    if (C <= 4096) return run_resid_unaligned<E, R, 0, 1>(a, bwd, stream);
    if (C <= 8192) return run_resid_unaligned<E, R, 0, 2>(a, bwd, stream);
    return run_resid_unaligned<E, R, 0, 4>(a, bwd, stream);
  }
  if (C <= 8) return run_resid<E, R, 1, 1>(a, bwd, stream);
  if (C <= 64) return run_resid<E, R, 8, 1>(a, bwd, stream);
  if (C <= 128) return run_resid<E, R, 16, 1>(a, bwd, stream);
  if (C <= 256) return run_resid<E, R, 32, 1>(a, bwd, stream);
  // two rows at a time where there are enough, and shared memory and registers hold them
  const bool wide = C > (bwd ? 4096 : 8192);
  if constexpr (sizeof(E) == 2) {
    if (a.T >= 4 * sm_count() && (bwd || wide || C <= 4096))
      return wide ? run_resid_wide<E, R, 2>(a, bwd, stream) : run_resid<E, R, 0, 2>(a, bwd, stream);
  }
  return wide ? run_resid_wide<E, R, 1>(a, bwd, stream) : run_resid<E, R, 0, 1>(a, bwd, stream);
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
  const int64_t most = (int64_t)mix::sm_count() * mix::kResidBlocks;
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
