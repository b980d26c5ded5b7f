// gdr_conv.cu -- the short causal convolution over packed segments, its backward and its
// single-token form.
//
//   u_t = b + sum_{k < W} w_k x_{t-W+1+k},   y_t = u_t or u_t sigmoid(u_t)          (per channel)
//
// with the W - 1 inputs before a segment taken from its initial state (oldest first) or zero.
// Backward, with du_t = dy_t y'(u_t) and sums inside the segment:
//   dx_t = sum_k w_k du_{t+W-1-k} (+ the final state's gradient at the last W - 1 places),
//   dw_k = sum_t du_t x_{t-W+1+k},  db = sum_t du_t.
//
// Bound by HBM: every x is read and every y written once.  A thread owns 8 neighbouring channels
// (16 bytes of bf16) and marches over a range of tokens with the last W - 1 inputs in registers,
// so that the taps cost no second load; ranges are long enough for the W - 1 tokens read again at
// each range's start not to matter.
#include "gdr_mix.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 16;  // tokens between two looks at the segment bounds
constexpr int kAhead = 4;    // groups of 4 tokens in a forward thread's ring (bf16; fp32 half)
constexpr int kFwdCtas = 3;  // blocks on each SM of the forward: all of them run at once

// Marks of one tile, written by warp 0 one tile ahead.
struct Marks {
  int mark[2][kTile + 1];
  int any[2];
  int red[64];
  int seg, start;
};

template <typename E, int W, bool VEC>
struct Rows {  // 8 channels of x and of the states
  const E *x;
  int64_t st;
  const E *h0;
  int C, c0, nv;
  __device__ __forceinline__ Raw8<E> load(int t) const {
    return ld8<VEC>(x + (int64_t)t * st + c0, nv);
  }
  // the W - 1 inputs before place p of segment seg (token t); win[W - 2] is the newest
  __device__ __forceinline__ void fill(float (&win)[W - 1][8], int seg, int t, int p) const {
#pragma unroll
    for (int b = 1; b < W; ++b) {
      Raw8<E> r = zero8<E>();
      if (p >= b)
        r = load(t - b);
      else if (h0)
        r = ld8<VEC>(h0 + ((int64_t)seg * (W - 1) + (W - 1 + p - b)) * C + c0, nv);
      unpack8(r, win[W - 1 - b]);
    }
  }
};

template <int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c0, int nv, float (&w)[W][8],
                                          float (&bias)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = i < nv ? ldp(a.w, (int64_t)(c0 + i) * W + k) : 0.f;
    bias[i] = (i < nv && a.b.p) ? ldp(a.b, c0 + i) : 0.f;
  }
}

template <int W>
__device__ __forceinline__ void taps(const float (&w)[W][8], const float (&bias)[8],
                                     const float (&win)[W - 1][8], const float (&x)[8],
                                     float (&u)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s = bias[i];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) s = fmaf(w[k][i], win[k][i], s);
    u[i] = fmaf(w[W - 1][i], x[i], s);
  }
}

template <int W>
__device__ __forceinline__ void shift(float (&win)[W - 1][8], const float (&x)[8]) {
#pragma unroll
  for (int k = 0; k + 1 < W - 1; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) win[k][i] = win[k + 1][i];
#pragma unroll
  for (int i = 0; i < 8; ++i) win[W - 2][i] = x[i];
}

// Copies the state rows of segments without tokens (src null: zeros).
template <typename E, bool VEC>
__device__ void empty_rows(const ConvArgs &a, int rows, const void *src, void *dst, int c0, int nv,
                           int *bits) {
  for_empty_segments(a.cu, a.n_seq, a.T, bits, [&](int n) {
    for (int k = 0; k < rows; ++k) {
      const int64_t at = ((int64_t)n * rows + k) * a.C + c0;
      const Raw8<E> r = src ? ld8<VEC>(reinterpret_cast<const E *>(src) + at, nv) : zero8<E>();
      st8<VEC>(reinterpret_cast<E *>(dst) + at, r, nv);
    }
  });
}

template <typename E>
__device__ __forceinline__ Raw8<E> activated(float (&v)[8], int silu) {
  if (silu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= sigmoidf(v[e]);
  }
  return pack8(v, E{});
}

// A thread's next rows of x on their way into shared memory: groups of G tokens, S of them in a
// ring in which each thread reads only what it copied itself.  Without 16-byte alignment rows are
// loaded when they are used.
template <typename E, bool VEC>
struct Ahead {
  static constexpr int G = 4;
  static constexpr int P = (int)sizeof(E) / 2;  // 16-byte parts of a row's 8 elements
  static constexpr int S = kAhead / P;
  static constexpr int kBytes = VEC ? S * G * P * kThreads * 16 : 0;
  uint4 *ring;
  const E *x;
  int64_t st;
  int nv, end;

  __device__ __forceinline__ uint4 *at(int s, int g) const {
    return ring + ((s * G + g) * P) * kThreads + threadIdx.x;
  }
  __device__ __forceinline__ void issue(int s, int t) const {
    if (VEC) {
      const E *p = x + (int64_t)t * st;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (t + g < end && nv > 0) {
#pragma unroll
          for (int i = 0; i < P; ++i) copy16(at(s, g) + i * kThreads, p + i * 4);
        }
        p += st;
      }
      copies_commit();
    }
  }
  __device__ __forceinline__ void wait() const {
    if (VEC) copies_wait<S - 1>();
  }
  __device__ __forceinline__ Raw8<E> get(int s, int g, int t) const {
    Raw8<E> r;
    if (VEC) {
      uint4 *w = reinterpret_cast<uint4 *>(&r);
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = at(s, g)[i * kThreads];
    } else {
      r = ld8<VEC>(x + (int64_t)t * st, nv);
    }
    return r;
  }
};

template <typename E, int W, bool VEC>
__global__ void __launch_bounds__(kThreads, kFwdCtas)
    k_conv_fwd(const ConvArgs a, int range, int cblocks, int nranges) {
  using R = Ahead<E, VEC>;
  constexpr int G = R::G, S = R::S;
  __shared__ Marks m;
  extern __shared__ __align__(16) uint4 ring[];
  const int cb = blockIdx.x % cblocks, r = blockIdx.x / cblocks;
  const int c0 = (cb * kThreads + threadIdx.x) * 8, nv = max(0, min(8, a.C - c0));
  if (r == nranges) {
    empty_rows<E, VEC>(a, W - 1, a.h0, a.ht, c0, nv, m.red);
    return;
  }
  const int t0 = r * range, t1 = min(a.T, t0 + range);
  const Rows<E, W, VEC> rows{reinterpret_cast<const E *>(a.x.p), a.x.st,
                             reinterpret_cast<const E *>(a.h0), a.C, c0, nv};
  const R in{ring, rows.x + c0, a.x.st, nv, t1};
#pragma unroll
  for (int s = 0; s < S - 1; ++s) in.issue(s, t0 + s * G);
  E *y = reinterpret_cast<E *>(a.y.p) + c0;
  E *ht = reinterpret_cast<E *>(a.ht);
  float w[W][8], bias[8], win[W - 1][8];
  load_taps<W>(a, c0, nv, w, bias);
  SegCursor cursor = seg_find(a.cu, a.n_seq, a.T, t0, m.red);
  int seg = cursor.j - 1;
  if (threadIdx.x < 32) {
    const int start = cursor.b;
    const bool any = seg_marks(a.cu, a.n_seq, a.T, t0, min(kTile, t1 - t0), m.mark[0], cursor);
    if (threadIdx.x == 0) {
      m.any[0] = any;
      m.start = start;
    }
  }
  __syncthreads();
  if (seg >= 0 && seg < a.n_seq) {
    rows.fill(win, seg, t0, t0 - m.start);
  } else {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) win[k][i] = 0.f;
  }
  int buf = 0, stage = 0;
  for (int tb = t0; tb < t1; tb += kTile, buf ^= 1) {
    if (threadIdx.x < 32 && tb + kTile < t1) {
      const bool any = seg_marks(a.cu, a.n_seq, a.T, tb + kTile, min(kTile, t1 - tb - kTile),
                                 m.mark[buf ^ 1], cursor);
      if (threadIdx.x == 0) m.any[buf ^ 1] = any;
    }
    const bool any = m.any[buf];
    const int *mark = m.mark[buf];
#pragma unroll 1
    for (int tu = tb; tu < min(tb + kTile, t1); tu += G) {
      in.issue(stage == 0 ? S - 1 : stage - 1, tu + (S - 1) * G);
      in.wait();
      E *to = y + (int64_t)tu * a.y.st;
      if (!any && tu + G <= t1 && seg >= 0 && seg < a.n_seq) {
        // inside one segment: no bounds to look at, the window moves by renaming
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float x[8], v[8];
          unpack8(in.get(stage, g, tu + g), x);
          taps<W>(w, bias, win, x, v);
          st8<VEC>(to, activated<E>(v, a.silu), nv);
          to += a.y.st;
          shift<W>(win, x);
        }
      } else {
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
          const int t = tu + g, i = t - tb;
          if (t >= t1) break;
          float x[8], v[8];
          unpack8(in.get(stage, g, t), x);
          if (any && mark[i] >= 0) {
            seg = mark[i];
            if (seg < a.n_seq) rows.fill(win, seg, t, 0);
          }
          if (seg >= 0 && seg < a.n_seq) {
            taps<W>(w, bias, win, x, v);
            st8<VEC>(to, activated<E>(v, a.silu), nv);
            shift<W>(win, x);
            if (any && ht && mark[i + 1] >= 0) {
#pragma unroll
              for (int k = 0; k < W - 1; ++k)
                st8<VEC>(ht + ((int64_t)seg * (W - 1) + k) * a.C + c0, pack8(win[k], E{}), nv);
            }
          }
          to += a.y.st;
        }
      }
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    __syncthreads();
  }
}

// The backward over the same ranges.  acc[j] gathers the gradient of the input j + 1 tokens back
// until its last tap is in.  A range owns the gradients of its own tokens and of the initial
// states of the segments that start in it; it runs on W - 1 tokens into the next range for them.
template <typename E, int W, bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_conv_bwd(const ConvArgs a, int range, int cblocks, int nranges) {
  __shared__ Marks m;
  constexpr int U = 4;
  const int cb = blockIdx.x % cblocks, r = blockIdx.x / cblocks;
  const int c0 = (cb * kThreads + threadIdx.x) * 8, nv = max(0, min(8, a.C - c0));
  if (r == nranges) {
    empty_rows<E, VEC>(a, W - 1, a.dht, a.dh0, c0, nv, m.red);
    return;
  }
  const int t0 = r * range, t1 = min(a.T, t0 + range), t2 = min(a.T, t1 + W - 1);
  const Rows<E, W, VEC> rows{reinterpret_cast<const E *>(a.x.p), a.x.st,
                             reinterpret_cast<const E *>(a.h0), a.C, c0, nv};
  const E *dy = reinterpret_cast<const E *>(a.dy.p) + c0;
  E *dx = reinterpret_cast<E *>(a.dx.p) + c0;
  E *dh0 = reinterpret_cast<E *>(a.dh0);
  const E *dht = reinterpret_cast<const E *>(a.dht);
  float w[W][8], bias[8], win[W - 1][8], acc[W - 1][8], dw[W][8], db[8];
  load_taps<W>(a, c0, nv, w, bias);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][i] = 0.f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) acc[k][i] = win[k][i] = 0.f;
  }
  SegCursor cursor = seg_find(a.cu, a.n_seq, a.T, t0, m.red);
  int seg = cursor.j - 1;
  if (threadIdx.x < 32) {
    const int start = cursor.b;
    const bool any = seg_marks(a.cu, a.n_seq, a.T, t0, min(kTile, t2 - t0), m.mark[0], cursor);
    if (threadIdx.x == 0) {
      m.any[0] = any;
      m.start = start;
    }
  }
  __syncthreads();
  int start = m.start;
  if (seg >= 0 && seg < a.n_seq) rows.fill(win, seg, t0, t0 - start);

  auto emit = [&](int t, const float (&v)[8]) {  // the finished gradient of the input of token t
    if (t >= start) {
      if (t >= t0 && t < t1) st8<VEC>(dx + (int64_t)t * a.dx.st, pack8(v, E{}), nv);
    } else if (dh0 && start >= t0) {
      st8<VEC>(dh0 + ((int64_t)seg * (W - 1) + (W - 1 + t - start)) * a.C + c0, pack8(v, E{}), nv);
    }
  };

  int buf = 0;
  bool stop = false;
  for (int tb = t0; tb < t2; tb += kTile, buf ^= 1) {
    if (threadIdx.x < 32 && tb + kTile < t2) {
      const bool any = seg_marks(a.cu, a.n_seq, a.T, tb + kTile, min(kTile, t2 - tb - kTile),
                                 m.mark[buf ^ 1], cursor);
      if (threadIdx.x == 0) m.any[buf ^ 1] = any;
    }
    const bool any = m.any[buf];
    const int *mark = m.mark[buf];
#pragma unroll 1
    for (int u0 = 0; u0 < kTile && !stop; u0 += U) {
      Raw8<E> rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u0 + u;
        rx[u] = t < t2 ? rows.load(t) : zero8<E>();
        rd[u] = t < t2 ? ld8<VEC>(dy + (int64_t)t * a.dy.st, nv) : zero8<E>();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = u0 + u, t = tb + i;
        if (t < t2 && !stop) {
          if (any && mark[i] >= 0) {
            if (t >= t1) {
              stop = true;
            } else {
              seg = mark[i];
              start = t;
              if (seg < a.n_seq) rows.fill(win, seg, t, 0);
#pragma unroll
              for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
            }
          }
          if (!stop) {
            if (seg >= 0 && seg < a.n_seq) {
              float x[8], g[8];
              unpack8(rx[u], x);
              unpack8(rd[u], g);
              if (a.silu) {
                float v[8];
                taps<W>(w, bias, win, x, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] *= dsilu(v[e], sigmoidf(v[e]));
              }
              if (t < t1) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  db[e] += g[e];
#pragma unroll
                  for (int k = 0; k < W - 1; ++k) dw[k][e] = fmaf(g[e], win[k][e], dw[k][e]);
                  dw[W - 1][e] = fmaf(g[e], x[e], dw[W - 1][e]);
                }
              }
              float done[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                done[e] = fmaf(w[0][e], g[e], acc[W - 2][e]);
#pragma unroll
                for (int j = W - 2; j > 0; --j)
                  acc[j][e] = fmaf(w[W - 1 - j][e], g[e], acc[j - 1][e]);
                acc[0][e] = w[W - 1][e] * g[e];
              }
              emit(t - (W - 1), done);
              shift<W>(win, x);
              if (any && mark[i + 1] >= 0) {  // the segment's last token
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                  if (dht) {
                    float f[8];
                    unpack8(ld8<VEC>(dht + ((int64_t)seg * (W - 1) + (W - 2 - j)) * a.C + c0, nv),
                            f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[j][e] += f[e];
                  }
                  emit(t - j, acc[j]);
                }
              }
            } else if (t < t1) {  // no segment: no gradient
              st8<VEC>(dx + (int64_t)t * a.dx.st, zero8<E>(), nv);
            }
          }
        }
      }
    }
    __syncthreads();
  }
  float *work = reinterpret_cast<float *>(a.work) + (int64_t)r * (W + 1) * a.C;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < nv) {
#pragma unroll
      for (int k = 0; k < W; ++k) work[(int64_t)k * a.C + c0 + i] = dw[k][i];
      work[(int64_t)W * a.C + c0 + i] = db[i];
    }
}

// Sums the ranges' parts of dw and db in range order.
__global__ void k_conv_sum(const float *work, int nranges, int C, int W, float *dw, float *db) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x, k = blockIdx.y;
  if (c >= C || (k == W && !db)) return;
  const float *p = work + (int64_t)k * C + c;
  const int64_t st = (int64_t)(W + 1) * C;
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  int r = 0;
  for (; r + 8 <= nranges; r += 8)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += p[(r + i) * st];
  for (; r < nranges; ++r) s[0] += p[r * st];
  const float v = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  if (k < W)
    dw[(int64_t)c * W + k] = v;
  else
    db[c] = v;
}

template <typename E, int W, bool VEC>
__global__ void __launch_bounds__(kThreads) k_conv_step(const ConvStepArgs a, int cblocks) {
  const int c0 = (blockIdx.x % cblocks * kThreads + threadIdx.x) * 8, row = blockIdx.x / cblocks;
  const int nv = max(0, min(8, a.C - c0));
  if (nv == 0) return;
  E *y = reinterpret_cast<E *>(a.y.p) + (int64_t)row * a.y.st + c0;
  const int slot = a.idx ? a.idx[row] : row;
  if (slot < 0 || slot >= a.slots) {
    st8<VEC>(y, zero8<E>(), nv);
    return;
  }
  const Raw8<E> rx = ld8<VEC>(reinterpret_cast<const E *>(a.x.p) + (int64_t)row * a.x.st + c0, nv);
  E *s = reinterpret_cast<E *>(a.state) + (int64_t)slot * (W - 1) * a.C + c0;
  Raw8<E> old[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) old[k] = ld8<VEC>(s + (int64_t)k * a.C, nv);
  float win[W - 1][8], w[W][8], bias[8], x[8], v[8];
  ConvArgs ca{};
  ca.w = a.w;
  ca.b = a.b;
  load_taps<W>(ca, c0, nv, w, bias);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) unpack8(old[k], win[k]);
  unpack8(rx, x);
  taps<W>(w, bias, win, x, v);
  st8<VEC>(y, activated<E>(v, a.silu), nv);
#pragma unroll
  for (int k = 0; k + 1 < W - 1; ++k) st8<VEC>(s + (int64_t)k * a.C, old[k + 1], nv);
  st8<VEC>(s + (int64_t)(W - 2) * a.C, rx, nv);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// whether every 8-channel group of these rows starts on a 16-byte boundary
bool rows_ok(const Mat &m, bool f32) {
  return !m.p || (aligned16(m.p) && m.st % (f32 ? 4 : 8) == 0);
}

int conv_ranges(int64_t T, int32_t C, int ctas_per_sm) {
  const int64_t cblocks = ceil_div64(C, kThreads * 8);
  int64_t n = (int64_t)sm_count() * ctas_per_sm / cblocks;
  const int64_t most = ceil_div64(T, 4 * kTile);
  if (n > most) n = most;
  return (int)(n < 1 ? 1 : n);
}
int range_of(int64_t T, int n) {
  const int64_t r = ceil_div64(ceil_div64(T, n), kTile) * kTile;
  return (int)(r < kTile ? kTile : r);
}

template <typename E, int W, bool VEC>
cudaError_t run_fwd(const ConvArgs &a, cudaStream_t stream) {
  const int cblocks = (int)ceil_div64(a.C, kThreads * 8);
  const int range = range_of(a.T, conv_ranges(a.T, a.C, kFwdCtas));
  const int nranges = (int)ceil_div64(a.T, range);
  const int64_t blocks = (int64_t)cblocks * (nranges + (a.ht ? 1 : 0));
  if (blocks == 0) return cudaSuccess;
  constexpr int smem = Ahead<E, VEC>::kBytes;
  static_assert(smem <= 46 * 1024, "more shared memory than a launch has without asking");
  k_conv_fwd<E, W, VEC><<<(unsigned)blocks, kThreads, smem, stream>>>(a, range, cblocks, nranges);
  return cudaGetLastError();
}

template <typename E, int W, bool VEC>
cudaError_t run_bwd(const ConvArgs &a, cudaStream_t stream) {
  const int cblocks = (int)ceil_div64(a.C, kThreads * 8);
  const int range = range_of(a.T, conv_ranges(a.T, a.C, 4));
  const int nranges = (int)ceil_div64(a.T, range);
  const int64_t blocks = (int64_t)cblocks * (nranges + (a.dh0 ? 1 : 0));
  if (blocks > 0)
    k_conv_bwd<E, W, VEC><<<(unsigned)blocks, kThreads, 0, stream>>>(a, range, cblocks, nranges);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_conv_sum<<<dim3((unsigned)ceil_div64(a.C, 256), W + 1), 256, 0, stream>>>(
      reinterpret_cast<const float *>(a.work), nranges, a.C, W, a.dw, a.db);
  return cudaGetLastError();
}

template <typename E, int W, bool VEC>
cudaError_t run_step(const ConvStepArgs &a, cudaStream_t stream) {
  const int cblocks = (int)ceil_div64(a.C, kThreads * 8);
  k_conv_step<E, W, VEC><<<(unsigned)((int64_t)cblocks * a.B), kThreads, 0, stream>>>(a, cblocks);
  return cudaGetLastError();
}

#define GDR_CONV_DISPATCH(run, f32, W, vec)                                              \
  do {                                                                                   \
    if (f32) {                                                                           \
      if (W == 2) return vec ? run<float, 2, true>(a, stream) : run<float, 2, false>(a, stream); \
      if (W == 3) return vec ? run<float, 3, true>(a, stream) : run<float, 3, false>(a, stream); \
      return vec ? run<float, 4, true>(a, stream) : run<float, 4, false>(a, stream);     \
    }                                                                                    \
    if (W == 2)                                                                          \
      return vec ? run<__nv_bfloat16, 2, true>(a, stream)                                \
                 : run<__nv_bfloat16, 2, false>(a, stream);                              \
    if (W == 3)                                                                          \
      return vec ? run<__nv_bfloat16, 3, true>(a, stream)                                \
                 : run<__nv_bfloat16, 3, false>(a, stream);                              \
    return vec ? run<__nv_bfloat16, 4, true>(a, stream)                                  \
               : run<__nv_bfloat16, 4, false>(a, stream);                                \
  } while (0)

}  // namespace
}  // namespace mix

cudaError_t launch_conv_fwd(const ConvArgs &a, cudaStream_t stream) {
  using namespace mix;
  const bool vec = a.C % 8 == 0 && rows_ok(a.x, a.f32) && rows_ok(a.y, a.f32) &&
                   aligned16(a.h0) && aligned16(a.ht);
  GDR_CONV_DISPATCH(run_fwd, a.f32, a.W, vec);
}

size_t conv_bwd_workspace(int64_t T, int32_t C, int32_t W) {
  const int range = mix::range_of(T, mix::conv_ranges(T, C, 4));
  return align256((size_t)ceil_div64(T, range) * (W + 1) * C * sizeof(float));
}

cudaError_t launch_conv_bwd(const ConvArgs &a, cudaStream_t stream) {
  using namespace mix;
  const bool vec = a.C % 8 == 0 && rows_ok(a.x, a.f32) && rows_ok(a.dy, a.f32) &&
                   rows_ok(a.dx, a.f32) && aligned16(a.h0) && aligned16(a.dht) &&
                   aligned16(a.dh0);
  GDR_CONV_DISPATCH(run_bwd, a.f32, a.W, vec);
}

cudaError_t launch_conv_step(const ConvStepArgs &a, cudaStream_t stream) {
  using namespace mix;
  if (a.B == 0 || a.C == 0) return cudaSuccess;
  const bool vec = a.C % 8 == 0 && rows_ok(a.x, a.f32) && rows_ok(a.y, a.f32) &&
                   aligned16(a.state);
  GDR_CONV_DISPATCH(run_step, a.f32, a.W, vec);
}

}  // namespace gdr
