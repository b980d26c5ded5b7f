// gdr_rec.cu -- the gated linear recurrence over packed segments, its backward and its single-token
// form.  Per channel, with sr = sigmoid(r_t), si = sigmoid(i_t) (1 without an input gate):
//
//   a_t = e^{A sr} (A <= 0),  m_t = sqrt(1 - a_t^2) (or 1),  h_t = a_t h_{t-1} + m_t si x_t,  y_t = h_t.
//
// Backward: G_t = dy_t + c_{t+1}, c_t = a_t G_t from the last token to the first (c behind a segment
// is its final state's gradient, and c of its first token the initial state's), and
//   dx = G m si,  di = G m x si (1 - si),  dL = G a_t (h_{t-1} - si x a_t / m_t)  (L = log a_t),
//   dr = dL A sr (1 - sr),  dA = sum_t dL sr.
//
// One pass over the data: a cluster of blocks walks along the tokens of 64 channels, all of them with
// the same step of CL * P * K tokens.  A thread holds two channels of K neighbouring tokens in
// registers and reduces them to one pair (A, U): h_out = A h_in + U.  The pairs of a block's warps meet
// in its shared memory, those of the cluster's blocks in everyone's (distributed shared memory), and
// each thread then runs through its tokens from its true state.  The alternative, ranges that are
// scanned from a zero state, chained and scanned again, reads and computes everything twice.
#include <initializer_list>

#include "gdr_block.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kCh = 64;      // channels of a block: two a lane
constexpr int kMostCl = 16;  // blocks of a cluster

// ------------------------------------------------------------------ two neighbouring channels

template <typename E>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
  uint32_t v;
  __device__ __forceinline__ float lo() const { return lo_bf(v); }
  __device__ __forceinline__ float hi() const { return hi_bf(v); }
};
template <>
struct Raw2<float> {
  float2 v;
  __device__ __forceinline__ float lo() const { return v.x; }
  __device__ __forceinline__ float hi() const { return v.y; }
};

// nv of two channels, the others 0; VEC: nv is 0 or 2 and p is aligned to both.
template <bool VEC>
__device__ __forceinline__ Raw2<__nv_bfloat16> ld2(const __nv_bfloat16 *p, int nv) {
  Raw2<__nv_bfloat16> r{0};
  if (VEC) {
    if (nv > 0) r.v = *reinterpret_cast<const uint32_t *>(p);
  } else {
    const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
    if (nv > 0) r.v = s[0];
    if (nv > 1) r.v |= (uint32_t)s[1] << 16;
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ Raw2<float> ld2(const float *p, int nv) {
  Raw2<float> r{make_float2(0.f, 0.f)};
  if (VEC) {
    if (nv > 0) r.v = *reinterpret_cast<const float2 *>(p);
  } else {
    if (nv > 0) r.v.x = p[0];
    if (nv > 1) r.v.y = p[1];
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ void st2(__nv_bfloat16 *p, float lo, float hi, int nv) {
  const uint32_t v = pack2(lo, hi);
  if (VEC) {
    if (nv > 0) *reinterpret_cast<uint32_t *>(p) = v;
  } else {
    unsigned short *s = reinterpret_cast<unsigned short *>(p);
    if (nv > 0) s[0] = (unsigned short)v;
    if (nv > 1) s[1] = (unsigned short)(v >> 16);
  }
}
template <bool VEC>
__device__ __forceinline__ void st2(float *p, float lo, float hi, int nv) {
  if (VEC) {
    if (nv > 0) *reinterpret_cast<float2 *>(p) = make_float2(lo, hi);
  } else {
    if (nv > 0) p[0] = lo;
    if (nv > 1) p[1] = hi;
  }
}

// ------------------------------------------------------------------ one token of one channel

// 1 - a^2 from L2 = log2 a: next to a = 1 by the series of 1 - e^y, y = 2 log a (the last term left
// out is 5e-8 of it at the border), which keeps its relative accuracy there; else as it is written.
__device__ __forceinline__ float rest_of(float L2, float a) {
  const float y = L2 * 1.3862943611198906f;
  float p = fmaf(y, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(p, y, 1.f / 24.f);
  p = fmaf(p, y, 1.f / 6.f);
  p = fmaf(p, y, 0.5f);
  p = fmaf(p, y, 1.f);
  return y > -0.25f ? -y * p : fmaf(-a, a, 1.f);
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// sqrt(s), 0 for 0 (the smallest normal number is far below what s can be); NaN for s < 0: A > 0
__device__ __forceinline__ float root_of(float s) { return s * rsqrt_approx(s + 1.1754944e-38f); }

struct Token {
  float sr, a, m;
};
__device__ __forceinline__ Token token(float r, float A2, int normalize) {
  Token t;
  t.sr = sigmoidf(r);
  const float L2 = A2 * t.sr;
  t.a = ex2(L2);
  t.m = normalize ? root_of(rest_of(L2, t.a)) : 1.f;
  return t;
}

// ------------------------------------------------------------------ pairs (A, U): h -> A h + U
//
// A = 0 says that the pair holds a segment's start: what comes before it is not looked at, be it
// infinite or NaN.  (A product of decays that underflows to 0 says the same of a state that is gone.)

struct Map {
  float A, U;
};
__device__ __forceinline__ float through(Map f, float h) { return f.A == 0.f ? f.U : fmaf(f.A, h, f.U); }
// first f, then g
__device__ __forceinline__ Map then(Map f, Map g) {
  return Map{g.A == 0.f ? 0.f : f.A * g.A, through(g, f.U)};
}

// ------------------------------------------------------------------ the cluster

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// *p of the block of this rank = v
__device__ __forceinline__ void put(float4 *p, int rank, float4 v) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), to;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int blocks, int cluster, int threads,
                            cudaStream_t stream, A... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3((unsigned)threads);
  c.stream = stream;
  c.attrs = at;
  c.numAttrs = 2;
  if (cluster > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
  }
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// ------------------------------------------------------------------ segment bounds of tiles
//
// As seg_marks, for tiles that a block meets at a distance: entries below the tile are skipped.
// alive is the segment that holds the token before the tile (-1: none), and so the tile's first
// tokens if mark[0] names no other.

__device__ __forceinline__ bool tile_marks(const int32_t *cu, int n_seq, int T, int t0, int n,
                                           int *mark, SegCursor &c, int &alive) {
  alive = c.j - 1;
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
    const bool in = b <= t0 + n && b >= t0;
    if (in) atomicMax(&mark[b - t0], idx);
    any |= __any_sync(0xffffffffu, in);
    alive += __popc(__ballot_sync(0xffffffffu, b < t0));
    const int cnt = __popc(__ballot_sync(0xffffffffu, b < t0 + n));
    c.nb = __shfl_sync(0xffffffffu, b, cnt < 32 ? cnt : 31);
    if (cnt > 0) c.b = __shfl_sync(0xffffffffu, b, cnt - 1);
    c.j += cnt;
    if (cnt < 32) break;
  }
  __syncwarp();
  return any;
}

// The same from the last tile to the first, over bounds that do not decrease.  hi: the last entry
// that is not above the tiles met so far, at bound b.
struct BackCursor {
  int hi, b;
};
__device__ __forceinline__ bool tile_marks_back(const int32_t *bounds, int t0, int n, int *mark,
                                                BackCursor &c, int &alive) {
  alive = c.hi;
  if (c.b < t0) return false;  // c.hi = -1 has c.b = -1
  const int lane = threadIdx.x & 31;
  for (int i = lane; i <= n; i += 32) mark[i] = -1;
  __syncwarp();
  bool any = false;
  int at = c.hi;
  for (;;) {
    const int idx = at - lane, b = idx >= 0 ? bounds[idx] : -1;
    const bool in = b >= t0 && b <= t0 + n;
    if (in) atomicMax(&mark[b - t0], idx);
    any |= __any_sync(0xffffffffu, in);
    const int above = __popc(__ballot_sync(0xffffffffu, b > t0 + n));
    const int low = __popc(__ballot_sync(0xffffffffu, b < t0));
    if (at == c.hi) {  // entries above this tile are above all that follow
      c.hi -= above;
      if (above < 32) c.b = __shfl_sync(0xffffffffu, b, above);
    }
    if (low > 0) {
      alive = at - (32 - low);
      break;
    }
    at -= 32;
  }
  __syncwarp();
  return any;
}

// ------------------------------------------------------------------ forward

constexpr int kFwdP = 4, kFwdK = 16;  // warps of a block, tokens of a thread
constexpr int kBwdP = 4, kBwdK = kRecEvery;

template <int P, int K>
struct Shared {
  float4 warp[P][32];          // (A, U) of both channels, for each warp of the block
  float4 block[2][kMostCl][32];  // and for each block of the cluster, by the step's parity
  int mark[2][P * K + 1];
  int any[2], alive[2];
  int red[64];
};

// The segment of a warp's first token, from the marks of its tile: the highest index up to it.
__device__ __forceinline__ int segment_at(const int *mark, int i, int alive) {
  int m = alive;
  for (int j = threadIdx.x & 31; j <= i; j += 32) m = max(m, mark[j]);
  return __reduce_max_sync(0xffffffffu, m);
}

// What the threads of a cluster exchange in a step: returns the state in front of this thread's
// tokens (of two channels) and moves `carry` past the step.  f() runs where the block's last step is
// done with, and what it writes is seen after the exchange.  BACK: warps and blocks in reverse.
template <int P, int K, bool BACK, typename F>
__device__ __forceinline__ void exchange(Shared<P, K> &s, int buf, const Map (&mine)[2],
                                         float (&carry)[2], float (&front)[2], F f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster_rank(), size = cluster_size();
  s.warp[warp][lane] = make_float4(mine[0].A, mine[0].U, mine[1].A, mine[1].U);
  __syncthreads();
  f();
  Map all[2] = {{1.f, 0.f}, {1.f, 0.f}}, pre[2] = {{1.f, 0.f}, {1.f, 0.f}};
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int w = BACK ? P - 1 - j : j;
    if (w == warp) {
      pre[0] = all[0];
      pre[1] = all[1];
    }
    const float4 v = s.warp[w][lane];
    all[0] = then(all[0], Map{v.x, v.y});
    all[1] = then(all[1], Map{v.z, v.w});
  }
  const float4 out = make_float4(all[0].A, all[0].U, all[1].A, all[1].U);
  for (int to = warp; to < size; to += P) put(&s.block[buf][rank][lane], to, out);
  cluster_arrive();
  cluster_wait();
  float h[2] = {carry[0], carry[1]};
  for (int j = 0; j < size; ++j) {
    const int b = BACK ? size - 1 - j : j;
    if (b == rank) {
      front[0] = h[0];
      front[1] = h[1];
    }
    const float4 v = s.block[buf][b][lane];
    h[0] = through(Map{v.x, v.y}, h[0]);
    h[1] = through(Map{v.z, v.w}, h[1]);
  }
  carry[0] = h[0];
  carry[1] = h[1];
  front[0] = through(pre[0], front[0]);
  front[1] = through(pre[1], front[1]);
}

// OUT: y is written (without it only the kept states: the backward's first pass).
template <typename E, bool VEC, bool OUT>
__global__ void __launch_bounds__(kFwdP * 32, 4) k_rec_fwd(const RecArgs a) {
  after_previous();
  constexpr int P = kFwdP, K = kFwdK, N = P * K;
  __shared__ Shared<P, K> s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster_rank(), size = cluster_size();
  const int c0 = (int)(blockIdx.x / size) * kCh + lane * 2, nv = max(0, min(2, a.D - c0));
  const float A2[2] = {nv > 0 ? a.A[c0] * kLog2e : 0.f, nv > 1 ? a.A[c0 + 1] * kLog2e : 0.f};
  const E *x = reinterpret_cast<const E *>(a.x.p) + c0, *r = reinterpret_cast<const E *>(a.r.p) + c0;
  const E *ig = a.i.p ? reinterpret_cast<const E *>(a.i.p) + c0 : nullptr;
  E *y = reinterpret_cast<E *>(a.y.p) + c0;
  SegCursor cursor{0, 0, 0};
  auto look = [&](int buf, int t0) {  // warp 0: the bounds of a tile
    int alive = -1;
    const bool any = t0 < a.T && tile_marks(a.cu, a.n_seq, a.T, t0, min(N, a.T - t0), s.mark[buf],
                                            cursor, alive);
    if (lane == 0) {
      s.any[buf] = any;
      s.alive[buf] = alive;
    }
  };
  if (warp == 0) look(0, rank * N);
  cluster_arrive();  // every block of the cluster runs before one writes to it
  cluster_wait();
  float carry[2] = {0.f, 0.f};
  int buf = 0;
  for (int base = 0; base < a.T; base += size * N, buf ^= 1) {
    const int t0 = base + rank * N, tw = t0 + warp * K, left = a.T - tw;
    float at[K][2], u[K][2];
    {
      Raw2<E> xr[K], rr[K], ir[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int64_t t = tw + k;
        const int n = k < left ? nv : 0;
        xr[k] = ld2<VEC>(x + t * a.x.st, n);
        rr[k] = ld2<VEC>(r + t * a.r.st, n);
        if (ig) ir[k] = ld2<VEC>(ig + t * a.i.st, n);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float xs[2] = {xr[k].lo(), xr[k].hi()}, rs[2] = {rr[k].lo(), rr[k].hi()};
        float is[2] = {1.f, 1.f};
        if (ig) {
          is[0] = sigmoidf(ir[k].lo());
          is[1] = sigmoidf(ir[k].hi());
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const Token v = token(rs[c], A2[c], a.normalize);
          at[k][c] = k < left ? v.a : 1.f;
          u[k][c] = k < left ? v.m * is[c] * xs[c] : 0.f;
        }
      }
    }
    // segments that start among this warp's tokens: their state goes into the first token
    const bool any = s.any[buf];
    int seg = s.alive[buf];
    uint32_t starts = 0;
    if (any) {
      const int *mark = s.mark[buf];
      seg = left > 0 ? segment_at(mark, warp * K, seg) : seg;
#pragma unroll 1
      for (int k = 0; k < K; ++k)
        if (k < left && mark[warp * K + k] >= 0) starts |= 1u << k;
      if (starts && a.h0) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (starts >> k & 1) {
            const int n = mark[warp * K + k];
            if (n < a.n_seq) {
              const float *q = a.h0 + (int64_t)n * a.D + c0;
              if (nv > 0) u[k][0] = fmaf(at[k][0], q[0], u[k][0]);
              if (nv > 1) u[k][1] = fmaf(at[k][1], q[1], u[k][1]);
            }
          }
      }
    }
    Map mine[2] = {{1.f, 0.f}, {1.f, 0.f}};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool first = starts >> k & 1;
        mine[c].U = first ? u[k][c] : fmaf(at[k][c], mine[c].U, u[k][c]);
        mine[c].A = first ? 0.f : mine[c].A * at[k][c];
      }
    float h[2];
    exchange<P, K, false>(s, buf, mine, carry, h, [&] {
      if (warp == 0) look(buf ^ 1, t0 + size * N);
    });
    if (left <= 0) continue;
    if (!any && left >= K) {
      const bool in = seg >= 0 && seg < a.n_seq;
      const int n = in ? nv : 0;
      E *to = y + (int64_t)tw * a.y.st;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (a.kept && k % kRecEvery == 0) {
          float *q = a.kept + (int64_t)((tw + k) / kRecEvery) * a.D + c0;
          st2<VEC>(q, h[0], h[1], nv);
        }
        h[0] = fmaf(at[k][0], h[0], u[k][0]);
        h[1] = fmaf(at[k][1], h[1], u[k][1]);
        if (OUT) st2<VEC>(to, h[0], h[1], n);
        to += a.y.st;
      }
    } else {
      const int *mark = s.mark[buf] + warp * K;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k >= left) break;
        if (a.kept && k % kRecEvery == 0) {
          float *q = a.kept + (int64_t)((tw + k) / kRecEvery) * a.D + c0;
          st2<VEC>(q, h[0], h[1], nv);
        }
        const bool first = starts >> k & 1;
        if (first) seg = mark[k];
        h[0] = first ? u[k][0] : fmaf(at[k][0], h[0], u[k][0]);
        h[1] = first ? u[k][1] : fmaf(at[k][1], h[1], u[k][1]);
        if (seg >= 0 && seg < a.n_seq) {
          if (OUT) st2<VEC>(y + (int64_t)(tw + k) * a.y.st, h[0], h[1], nv);
          if (a.ht && any && mark[k + 1] >= 0) {
            float *q = a.ht + (int64_t)seg * a.D + c0;
            if (nv > 0) q[0] = h[0];
            if (nv > 1) q[1] = h[1];
          }
        }
      }
    }
  }
  // segments without tokens end as they start
  if (a.ht && rank == 0)
    for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
      if (warp == 0)
        for (int c = 0; c < nv; ++c)
          a.ht[(int64_t)n * a.D + c0 + c] = a.h0 ? a.h0[(int64_t)n * a.D + c0 + c] : 0.f;
    });
}

// ------------------------------------------------------------------ backward

// cu_seqlens as the kernels read it, non-decreasing in [0, T], for one that walks backwards.
__global__ void __launch_bounds__(1024) k_rec_bounds(const int32_t *cu, int n, int T, int32_t *out) {
  after_previous();
  __shared__ int top[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int run = 0;
  for (int base = 0; base < n; base += 1024) {
    const int i = base + (int)threadIdx.x;
    int b = i < n ? cu_at(cu, i, T) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) b = max(b, u);
    }
    if (lane == 31) top[warp] = b;
    __syncthreads();
    for (int w = 0; w < warp; ++w) b = max(b, top[w]);
    int next = run;
    for (int w = 0; w < 32; ++w) next = max(next, top[w]);
    if (i < n) out[i] = max(b, run);
    run = next;
    __syncthreads();
  }
}

template <typename E, bool VEC>
__global__ void __launch_bounds__(kBwdP * 32, 3) k_rec_bwd(const RecArgs a, const int32_t *bounds) {
  after_previous();
  constexpr int P = kBwdP, K = kBwdK, N = P * K;
  __shared__ Shared<P, K> s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster_rank(), size = cluster_size();
  const int c0 = (int)(blockIdx.x / size) * kCh + lane * 2, nv = max(0, min(2, a.D - c0));
  const float A[2] = {nv > 0 ? a.A[c0] : 0.f, nv > 1 ? a.A[c0 + 1] : 0.f};
  const E *x = reinterpret_cast<const E *>(a.x.p) + c0, *r = reinterpret_cast<const E *>(a.r.p) + c0;
  const E *dy = reinterpret_cast<const E *>(a.dy.p) + c0;
  const E *ig = a.i.p ? reinterpret_cast<const E *>(a.i.p) + c0 : nullptr;
  E *dx = reinterpret_cast<E *>(a.dx.p) + c0, *dr = reinterpret_cast<E *>(a.dr.p) + c0;
  E *di = reinterpret_cast<E *>(a.di.p) + c0;
  const int steps = (a.T + size * N - 1) / (size * N);
  BackCursor cursor{a.n_seq, bounds[a.n_seq]};
  auto look = [&](int buf, int t0) {  // warp 0: the bounds of a tile
    int alive = -1;
    const bool any = t0 >= 0 && t0 < a.T &&
                     tile_marks_back(bounds, t0, min(N, a.T - t0), s.mark[buf], cursor, alive);
    if (lane == 0) {
      s.any[buf] = any;
      s.alive[buf] = alive;
    }
  };
  if (warp == 0) look(0, ((steps - 1) * size + rank) * N);
  cluster_arrive();
  cluster_wait();
  float carry[2] = {0.f, 0.f}, dA[2] = {0.f, 0.f};
  int buf = 0;
  for (int step = steps - 1; step >= 0; --step, buf ^= 1) {
    const int t0 = (step * size + rank) * N, tw = t0 + warp * K, left = a.T - tw;
    Raw2<E> xr[K], ir[K];
    float g[K][2], sr[K][2], at[K][2], m[K][2], hb[K][2];
    float h[2] = {0.f, 0.f};
    if (left > 0) {
      const Raw2<float> q = ld2<VEC>(a.kept + (int64_t)(tw / kRecEvery) * a.D + c0, nv);
      h[0] = q.lo();
      h[1] = q.hi();
    }
    {
      Raw2<E> rr[K], gr[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int64_t t = tw + k;
        const int n = k < left ? nv : 0;
        rr[k] = ld2<VEC>(r + t * a.r.st, n);
        gr[k] = ld2<VEC>(dy + t * a.dy.st, n);
        xr[k] = ld2<VEC>(x + t * a.x.st, n);
        if (ig) ir[k] = ld2<VEC>(ig + t * a.i.st, n);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float rs[2] = {rr[k].lo(), rr[k].hi()};
        g[k][0] = gr[k].lo();
        g[k][1] = gr[k].hi();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const Token v = token(rs[c], A[c] * kLog2e, a.normalize);
          sr[k][c] = v.sr;
          at[k][c] = k < left ? v.a : 1.f;
          m[k][c] = v.m;
        }
      }
    }
    const bool any = s.any[buf];
    const int *mark = s.mark[buf] + warp * K;
    const int seg0 = any && left > 0 ? segment_at(s.mark[buf], warp * K, s.alive[buf]) : s.alive[buf];
    // bit k: a segment starts with token k (of K + 1)
    uint32_t starts = 0;
    if (any) {
#pragma unroll 1
      for (int k = 0; k <= K; ++k)
        if (k <= left && mark[k] >= 0) starts |= 1u << k;
    }
    // the states before the tokens, and the final states' gradients
    int seg = seg0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float is[2] = {1.f, 1.f};
      if (ig) {
        is[0] = sigmoidf(ir[k].lo());
        is[1] = sigmoidf(ir[k].hi());
      }
      if (starts >> k & 1) {
        seg = mark[k];
        const float *q = a.h0 && seg < a.n_seq ? a.h0 + (int64_t)seg * a.D + c0 : nullptr;
        h[0] = q && nv > 0 ? q[0] : 0.f;
        h[1] = q && nv > 1 ? q[1] : 0.f;
      }
      const bool in = seg >= 0 && seg < a.n_seq;
      if (starts >> (k + 1) & 1 && in && a.dht) {
        const float *q = a.dht + (int64_t)seg * a.D + c0;
        if (nv > 0) g[k][0] += q[0];
        if (nv > 1) g[k][1] += q[1];
      }
      hb[k][0] = h[0];
      hb[k][1] = h[1];
      h[0] = fmaf(at[k][0], h[0], m[k][0] * is[0] * xr[k].lo());
      h[1] = fmaf(at[k][1], h[1], m[k][1] * is[1] * xr[k].hi());
    }
    Map mine[2] = {{1.f, 0.f}, {1.f, 0.f}};
#pragma unroll
    for (int k = K - 1; k >= 0; --k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool last = starts >> (k + 1) & 1;
        const float in = last ? g[k][c] : g[k][c] + mine[c].U;
        mine[c].A = last ? 0.f : mine[c].A * at[k][c];
        mine[c].U = at[k][c] * in;
      }
    float c1[2];
    exchange<P, K, true>(s, buf, mine, carry, c1, [&] {
      if (warp == 0) look(buf ^ 1, t0 - size * N);
    });
    if (left <= 0) continue;
    seg = any ? -2 : seg0;
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      if (k >= left) continue;
      int own = seg;
      if (any) own = segment_at(mark, k, seg0);
      const bool in = own >= 0 && own < a.n_seq;
      const bool last = starts >> (k + 1) & 1;
      float ox[2], orr[2], oi[2];
      const float xs[2] = {xr[k].lo(), xr[k].hi()};
      float is[2] = {1.f, 1.f};
      if (ig) {
        is[0] = sigmoidf(ir[k].lo());
        is[1] = sigmoidf(ir[k].hi());
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float G = last ? g[k][c] : g[k][c] + c1[c];
        const float dv = G * m[k][c], v = is[c] * xs[c];
        // the normaliser's part of d/dL; none where a is 1 and it has no derivative
        const float ratio = a.normalize && m[k][c] != 0.f ? at[k][c] * rcp(m[k][c]) : 0.f;
        const float dL = G * at[k][c] * (hb[k][c] - v * ratio);
        ox[c] = in ? dv * is[c] : 0.f;
        oi[c] = in ? dv * v * (1.f - is[c]) : 0.f;
        orr[c] = in ? dL * A[c] * sr[k][c] * (1.f - sr[k][c]) : 0.f;
        dA[c] += in ? dL * sr[k][c] : 0.f;
        c1[c] = at[k][c] * G;
      }
      const int64_t t = tw + k;
      st2<VEC>(dx + t * a.dx.st, ox[0], ox[1], nv);
      st2<VEC>(dr + t * a.dr.st, orr[0], orr[1], nv);
      if (ig) st2<VEC>(di + t * a.di.st, oi[0], oi[1], nv);
      if (a.dh0 && in && starts >> k & 1) {
        float *q = a.dh0 + (int64_t)own * a.D + c0;
        if (nv > 0) q[0] = c1[0];
        if (nv > 1) q[1] = c1[1];
      }
    }
  }
  // dA: the warps' sums in order, then the blocks' of the cluster
  __syncthreads();
  s.warp[warp][lane] = make_float4(dA[0], dA[1], 0.f, 0.f);
  __syncthreads();
  if (warp == 0) {
    float4 v = s.warp[0][lane];
#pragma unroll
    for (int w = 1; w < P; ++w) {
      v.x += s.warp[w][lane].x;
      v.y += s.warp[w][lane].y;
    }
    put(&s.block[buf][rank][lane], 0, v);
  }
  cluster_arrive();
  cluster_wait();
  if (rank == 0) {
    if (warp == 0) {
      float4 v = s.block[buf][0][lane];
      for (int b = 1; b < size; ++b) {
        v.x += s.block[buf][b][lane].x;
        v.y += s.block[buf][b][lane].y;
      }
      if (nv > 0) a.dA[c0] = v.x;
      if (nv > 1) a.dA[c0 + 1] = v.y;
    }
    if (a.dh0)
      for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
        if (warp == 0)
          for (int c = 0; c < nv; ++c)
            a.dh0[(int64_t)n * a.D + c0 + c] = a.dht ? a.dht[(int64_t)n * a.D + c0 + c] : 0.f;
      });
  }
}

// ------------------------------------------------------------------ single tokens

// Two channels of one request a thread.
template <typename E, bool VEC>
__global__ void __launch_bounds__(128) k_rec_step(const RecArgs a, float *state, int slots,
                                                  const int32_t *idx) {
  after_previous<true>();
  const int c0 = ((int)blockIdx.x * 128 + (int)threadIdx.x) * 2, row = blockIdx.y;
  const int nv = max(0, min(2, a.D - c0));
  if (nv == 0) return;
  const int slot = idx ? idx[row] : row;
  E *y = reinterpret_cast<E *>(a.y.p) + (int64_t)row * a.y.st + c0;
  if (slot < 0 || slot >= slots) {
    st2<VEC>(y, 0.f, 0.f, nv);
    return;
  }
  float *q = state + (int64_t)slot * a.D + c0;
  const Raw2<float> h = ld2<VEC>(q, nv), A = ld2<VEC>(a.A + c0, nv);
  const Raw2<E> x = ld2<VEC>(reinterpret_cast<const E *>(a.x.p) + (int64_t)row * a.x.st + c0, nv);
  const Raw2<E> r = ld2<VEC>(reinterpret_cast<const E *>(a.r.p) + (int64_t)row * a.r.st + c0, nv);
  float is[2] = {1.f, 1.f};
  if (a.i.p) {
    const Raw2<E> i =
        ld2<VEC>(reinterpret_cast<const E *>(a.i.p) + (int64_t)row * a.i.st + c0, nv);
    is[0] = sigmoidf(i.lo());
    is[1] = sigmoidf(i.hi());
  }
  const Token u = token(r.lo(), A.lo() * kLog2e, a.normalize);
  const Token v = token(r.hi(), A.hi() * kLog2e, a.normalize);
  const float lo = fmaf(u.a, h.lo(), u.m * is[0] * x.lo());
  const float hi = fmaf(v.a, h.hi(), v.m * is[1] * x.hi());
  st2<VEC>(q, lo, hi, nv);
  st2<VEC>(y, lo, hi, nv);
}

// ------------------------------------------------------------------ launches

// Pairs of channels at addresses that are multiples of a pair.
template <typename E>
bool pairs(const RecArgs &a, std::initializer_list<Mat> mats, std::initializer_list<const void *> f) {
  bool ok = a.D % 2 == 0;
  for (const Mat &m : mats)
    ok = ok && reinterpret_cast<uintptr_t>(m.p) % (2 * sizeof(E)) == 0 && m.st % 2 == 0;
  for (const void *p : f) ok = ok && reinterpret_cast<uintptr_t>(p) % 8 == 0;
  return ok;
}

// Blocks of a cluster: as many as the tokens fill, while all blocks run at once.
int cluster_for(int T, int D, int tile, int per_sm) {
  const int64_t groups = (D + kCh - 1) / kCh, slots = (int64_t)sm_count() * per_sm;
  int cl = 1;
  while (cl < 8 && (int64_t)cl * tile < T && groups * cl * 2 <= slots) cl *= 2;
  return cl;
}

template <typename E, bool OUT>
cudaError_t run_fwd(const RecArgs &a, cudaStream_t stream) {
  const int cl = cluster_for(a.T, a.D, kFwdP * kFwdK, 4), groups = (a.D + kCh - 1) / kCh;
  const bool vec = OUT ? pairs<E>(a, {a.x, a.r, a.i, a.y}, {a.kept})
                       : pairs<E>(a, {a.x, a.r, a.i}, {a.kept});
  return vec ? launch_clusters(k_rec_fwd<E, true, OUT>, groups * cl, cl, kFwdP * 32, stream, a)
             : launch_clusters(k_rec_fwd<E, false, OUT>, groups * cl, cl, kFwdP * 32, stream, a);
}

size_t kept_bytes(int64_t T, int32_t D) {
  return align256((size_t)((T + kRecEvery - 1) / kRecEvery) * D * 4);
}

template <typename E>
cudaError_t run_bwd(RecArgs a, bool kept, cudaStream_t stream) {
  char *w = reinterpret_cast<char *>(a.work);
  int32_t *bounds = reinterpret_cast<int32_t *>(w);
  cudaError_t e = launch(k_rec_bounds, 1, 1024, 0, stream, a.cu, a.n_seq + 1, a.T, bounds);
  if (e != cudaSuccess) return e;
  if (!kept) {
    a.kept = reinterpret_cast<float *>(w + align256(((size_t)a.n_seq + 1) * 4));
    a.ht = nullptr;
    e = run_fwd<E, false>(a, stream);
    if (e != cudaSuccess) return e;
  }
  const int cl = cluster_for(a.T, a.D, kBwdP * kBwdK, 3), groups = (a.D + kCh - 1) / kCh;
  return pairs<E>(a, {a.x, a.r, a.i, a.dy, a.dx, a.dr, a.di}, {a.kept})
             ? launch_clusters(k_rec_bwd<E, true>, groups * cl, cl, kBwdP * 32, stream, a, bounds)
             : launch_clusters(k_rec_bwd<E, false>, groups * cl, cl, kBwdP * 32, stream, a, bounds);
}

template <typename E>
cudaError_t run_step(const RecArgs &a, float *state, int32_t slots, const int32_t *idx,
                     cudaStream_t stream) {
  const bool vec = pairs<E>(a, {a.x, a.r, a.i, a.y}, {state, a.A});
  // rows beyond a grid's second dimension in further launches
  RecArgs p = a;
  for (int32_t row = 0; row < a.T; row += 65535) {
    const int32_t rows = a.T - row < 65535 ? a.T - row : 65535;
    auto at = [&](const Mat &m) {
      return Mat{m.p ? reinterpret_cast<E *>(m.p) + (int64_t)row * m.st : nullptr, m.st};
    };
    p.x = at(a.x);
    p.r = at(a.r);
    p.i = at(a.i);
    p.y = at(a.y);
    const dim3 grid((unsigned)((a.D + 255) / 256), (unsigned)rows);
    float *s = idx ? state : state + (int64_t)row * a.D;
    const int32_t n = idx ? slots : slots - row;
    const cudaError_t e =
        vec ? launch(k_rec_step<E, true>, grid, 128, 0, stream, p, s, n, idx ? idx + row : idx)
            : launch(k_rec_step<E, false>, grid, 128, 0, stream, p, s, n, idx ? idx + row : idx);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace mix

cudaError_t launch_rec_fwd(const RecArgs &a, cudaStream_t stream) {
  return a.f32 ? mix::run_fwd<float, true>(a, stream)
               : mix::run_fwd<__nv_bfloat16, true>(a, stream);
}
size_t rec_bwd_workspace(int64_t T, int32_t D, int32_t n_seq, bool kept) {
  return align256(((size_t)n_seq + 1) * 4) + (kept ? 0 : mix::kept_bytes(T, D));
}
cudaError_t launch_rec_bwd(const RecArgs &a, bool kept, cudaStream_t stream) {
  return a.f32 ? mix::run_bwd<float>(a, kept, stream)
               : mix::run_bwd<__nv_bfloat16>(a, kept, stream);
}
cudaError_t launch_rec_step(const RecArgs &a, float *state, int32_t slots, const int32_t *idx,
                            cudaStream_t stream) {
  return a.f32 ? mix::run_step<float>(a, state, slots, idx, stream)
               : mix::run_step<__nv_bfloat16>(a, state, slots, idx, stream);
}

}  // namespace gdr
