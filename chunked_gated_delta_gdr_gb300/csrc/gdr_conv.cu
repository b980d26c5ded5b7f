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
// each range's start not to matter.  65,536 x 12,288 in bf16: 509 us, 6.3 TB/s of 6.8.  The backward
// recomputes the taps for the activation's derivative and is bound by latency: 236 registers leave
// it 2 warps a scheduler, which issue in 43 % of the cycles and reach 5.0 TB/s.  16,384 x 6,144: forward 72
// us for 59 of bytes, backward 118 (with its sums over the ranges, 6) for 89; the two in turn 190, with
// four segments' states 204.
#include "gdr_mix.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kThreads = 128;  // of a step's block; the others' TH: 128, or 32 for few channels
constexpr int kTile = 16;  // tokens between two looks at the segment bounds
constexpr int kFwdCtas = 3;  // blocks on each SM: all of them run at once
constexpr int kBwdCtas = 2;

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
  __device__ __forceinline__ void fill(f2 (&win)[W - 1][4], int seg, int t, int p) const {
#pragma unroll
    for (int b = 1; b < W; ++b) {
      Raw8<E> r = zero8<E>();
      if (p >= b)
        r = load(t - b);
      else if (h0)
        r = ld8<VEC>(h0 + ((int64_t)seg * (W - 1) + (W - 1 + p - b)) * C + c0, nv);
      unpack4(r, win[W - 1 - b]);
    }
  }
};

template <int N>
__device__ __forceinline__ void clear(f2 (&v)[N][4]) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[k][i] = pair(0.f, 0.f);
}

// n contiguous parameters, a multiple of 8 of them 16-byte aligned
template <int N>
__device__ __forceinline__ void load_params(const Param &p, int64_t at, float (&v)[N]) {
  if (p.bf16) {
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(p.p) + at);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      float f[8];
      unpack8(Raw8<__nv_bfloat16>{q[i]}, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * i + j] = f[j];
    }
  } else {
    const float4 *q = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p.p) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 f = q[i];
      v[4 * i] = f.x;
      v[4 * i + 1] = f.y;
      v[4 * i + 2] = f.z;
      v[4 * i + 3] = f.w;
    }
  }
}

// The taps and bias of 8 channels (those from nv on are zero).
template <int W>
__device__ __forceinline__ void load_taps(const Param &weight, const Param &b, int c0, int nv,
                                          f2 (&w)[W][4], f2 (&bias)[4]) {
  float v[8 * W], u[8];
  const uintptr_t at = reinterpret_cast<uintptr_t>(weight.p) | reinterpret_cast<uintptr_t>(b.p);
  if (nv == 8 && (at & 15) == 0) {
    load_params<8 * W>(weight, (int64_t)c0 * W, v);
    if (b.p) load_params<8>(b, c0, u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k)
        v[i * W + k] = i < nv ? ldp(weight, (int64_t)(c0 + i) * W + k) : 0.f;
      u[i] = i < nv && b.p ? ldp(b, c0 + i) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = pair(v[2 * i * W + k], v[(2 * i + 1) * W + k]);
    bias[i] = b.p ? pair(u[2 * i], u[2 * i + 1]) : pair(0.f, 0.f);
  }
}

template <int W>
__device__ __forceinline__ void taps(const f2 (&w)[W][4], const f2 (&bias)[4],
                                     const f2 (&win)[W - 1][4], const f2 (&x)[4], f2 (&u)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[i] = bias[i];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) u[i] = fma2(w[k][i], win[k][i], u[i]);
    u[i] = fma2(w[W - 1][i], x[i], u[i]);
  }
}

template <int W>
__device__ __forceinline__ void shift(f2 (&win)[W - 1][4], const f2 (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
    win[W - 2][i] = x[i];
  }
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

// The forward's output: single products, which it has the issue slots for; pairs measured 7 %
// slower here (554 against 519 us for 65,536 x 12,288), their latency longer.
template <typename E, int W>
__device__ __forceinline__ Raw8<E> output(const f2 (&w)[W][4], const f2 (&bias)[4],
                                          const f2 (&win)[W - 1][4], const f2 (&x)[4], int silu) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b, c, d, e, f;
    unpair(bias[i], a, b);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      unpair(w[k][i], c, d);
      unpair(k < W - 1 ? win[k < W - 1 ? k : 0][i] : x[i], e, f);
      a = fmaf(c, e, a);
      b = fmaf(d, f, b);
    }
    v[2 * i] = silu ? a * sigmoidf(a) : a;
    v[2 * i + 1] = silu ? b * sigmoidf(b) : b;
  }
  return pack8(v, E{});
}

// A thread's next rows on their way into shared memory: groups of G tokens, S of them in a ring in
// which each thread reads only what it copied itself.  Without 16-byte alignment rows are loaded
// when they are used.
template <typename E, bool VEC, int G_, int S_, int TH>
struct Ahead {
  static constexpr int G = G_, S = S_;
  static constexpr int P = (int)sizeof(E) / 2;  // 16-byte parts of a row's 8 elements
  static constexpr int kSlots = VEC ? S * G * P * TH : 0;
  uint4 *ring;
  const E *x;
  int64_t st;
  int nv, end;

  __device__ __forceinline__ uint4 *at(int s, int g) const {
    return ring + ((s * G + g) * P) * TH + threadIdx.x;
  }
  __device__ __forceinline__ void issue(int s, int t) const {
    if (VEC) {
      const E *p = x + (int64_t)t * st;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (t + g < end && nv > 0) {
#pragma unroll
          for (int i = 0; i < P; ++i) copy16(at(s, g) + i * TH, p + i * 4);
        }
        p += st;
      }
    }
  }
  static __device__ __forceinline__ void commit() {
    if (VEC) copies_commit();
  }
  static __device__ __forceinline__ void wait() {
    if (VEC) copies_wait<S - 1>();
  }
  __device__ __forceinline__ Raw8<E> get(int s, int g, int t) const {
    Raw8<E> r;
    if (VEC) {
      uint4 *w = reinterpret_cast<uint4 *>(&r);
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = at(s, g)[i * TH];
    } else {
      r = ld8<VEC>(x + (int64_t)t * st, nv);
    }
    return r;
  }
};
// the forward's and the backward's (x and dy), less deep in fp32: a row is twice the bytes
template <typename E, bool VEC, int TH>
using FwdAhead = Ahead<E, VEC, 4, sizeof(E) == 2 ? 4 : 2, TH>;
template <typename E, bool VEC, int TH>
using BwdAhead = Ahead<E, VEC, sizeof(E) == 2 ? 4 : 2, 2, TH>;

template <typename E, int W, bool VEC, int TH>
__global__ void __launch_bounds__(TH, kFwdCtas * kThreads / TH)
    k_conv_fwd(const ConvArgs a, int range, int cblocks, int nranges) {
  after_previous();
  using R = FwdAhead<E, VEC, TH>;
  constexpr int G = R::G, S = R::S;
  __shared__ Marks m;
  extern __shared__ __align__(16) uint4 ring[];
  const int cb = blockIdx.x % cblocks, r = blockIdx.x / cblocks;
  const int c0 = (cb * TH + threadIdx.x) * 8, nv = max(0, min(8, a.C - c0));
  if (r == nranges) {
    empty_rows<E, VEC>(a, W - 1, a.h0, a.ht, c0, nv, m.red);
    return;
  }
  const int t0 = r * range, t1 = min(a.T, t0 + range);
  const Rows<E, W, VEC> rows{reinterpret_cast<const E *>(a.x.p), a.x.st,
                             reinterpret_cast<const E *>(a.h0), a.C, c0, nv};
  const R in{ring, rows.x + c0, a.x.st, nv, t1};
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    in.issue(s, t0 + s * G);
    in.commit();
  }
  E *y = reinterpret_cast<E *>(a.y.p) + c0;
  E *ht = reinterpret_cast<E *>(a.ht);
  f2 w[W][4], bias[4], win[W - 1][4];
  load_taps<W>(a.w, a.b, c0, nv, w, bias);
  clear<W - 1>(win);
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
  if (seg >= 0 && seg < a.n_seq) rows.fill(win, seg, t0, t0 - m.start);
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
      in.commit();
      in.wait();
      E *to = y + (int64_t)tu * a.y.st;
      if (!any && tu + G <= t1 && seg >= 0 && seg < a.n_seq) {
        // inside one segment: no bounds to look at, the window moves by renaming
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f2 x[4];
          unpack4(in.get(stage, g, tu + g), x);
          st8<VEC>(to, output<E, W>(w, bias, win, x, a.silu), nv);
          to += a.y.st;
          shift<W>(win, x);
        }
      } else {
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
          const int t = tu + g, i = t - tb;
          if (t >= t1) break;
          f2 x[4];
          unpack4(in.get(stage, g, t), x);
          if (any && mark[i] >= 0) {
            seg = mark[i];
            if (seg < a.n_seq) rows.fill(win, seg, t, 0);
          }
          if (seg >= 0 && seg < a.n_seq) {
            st8<VEC>(to, output<E, W>(w, bias, win, x, a.silu), nv);
            shift<W>(win, x);
            if (any && ht && mark[i + 1] >= 0) {
#pragma unroll
              for (int k = 0; k < W - 1; ++k)
                st8<VEC>(ht + ((int64_t)seg * (W - 1) + k) * a.C + c0, pack4<E>(win[k]), nv);
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
template <typename E, int W, bool VEC, int TH>
__global__ void __launch_bounds__(TH, kBwdCtas * kThreads / TH)
    k_conv_bwd(const ConvArgs a, int range, int cblocks, int nranges) {
  after_previous();
  using R = BwdAhead<E, VEC, TH>;
  constexpr int G = R::G, S = R::S;
  __shared__ Marks m;
  extern __shared__ __align__(16) uint4 ring[];
  const int cb = blockIdx.x % cblocks, r = blockIdx.x / cblocks;
  const int c0 = (cb * TH + threadIdx.x) * 8, nv = max(0, min(8, a.C - c0));
  if (r == nranges) {
    empty_rows<E, VEC>(a, W - 1, a.dht, a.dh0, c0, nv, m.red);
    return;
  }
  const int t0 = r * range, t1 = min(a.T, t0 + range), t2 = min(a.T, t1 + W - 1);
  const Rows<E, W, VEC> rows{reinterpret_cast<const E *>(a.x.p), a.x.st,
                             reinterpret_cast<const E *>(a.h0), a.C, c0, nv};
  const R inx{ring, rows.x + c0, a.x.st, nv, t2};
  const R ing{ring + R::kSlots, reinterpret_cast<const E *>(a.dy.p) + c0, a.dy.st, nv, t2};
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    inx.issue(s, t0 + s * G);
    ing.issue(s, t0 + s * G);
    R::commit();
  }
  E *dx = reinterpret_cast<E *>(a.dx.p) + c0;
  E *dh0 = reinterpret_cast<E *>(a.dh0);
  const E *dht = reinterpret_cast<const E *>(a.dht);
  f2 w[W][4], bias[4], win[W - 1][4], acc[W - 1][4], dw[W][4], db[1][4];
  load_taps<W>(a.w, a.b, c0, nv, w, bias);
  clear<W - 1>(win);
  clear<W - 1>(acc);
  clear<W>(dw);
  clear<1>(db);
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

  // one token: its x and dy; `done` is the finished gradient of the input W - 1 tokens back
  auto token = [&](const Raw8<E> &rx, const Raw8<E> &rg, bool own, f2 (&done)[4]) {
    f2 x[4], g[4];
    unpack4(rx, x);
    unpack4(rg, g);
    if (a.silu) {
      f2 u[4];
      taps<W>(w, bias, win, x, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], dsilu2(u[i], sigmoid2(u[i])));
    }
    if (own) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        db[0][i] = add2(db[0][i], g[i]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) dw[k][i] = fma2(g[i], win[k][i], dw[k][i]);
        dw[W - 1][i] = fma2(g[i], x[i], dw[W - 1][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      done[i] = fma2(w[0][i], g[i], acc[W - 2][i]);
#pragma unroll
      for (int j = W - 2; j > 0; --j) acc[j][i] = fma2(w[W - 1 - j][i], g[i], acc[j - 1][i]);
      acc[0][i] = mul2(w[W - 1][i], g[i]);
    }
    shift<W>(win, x);
  };
  auto emit = [&](int t, const f2 (&v)[4]) {  // the finished gradient of the input of token t
    if (t >= start) {
      if (t >= t0 && t < t1) st8<VEC>(dx + (int64_t)t * a.dx.st, pack4<E>(v), nv);
    } else if (dh0 && start >= t0) {
      st8<VEC>(dh0 + ((int64_t)seg * (W - 1) + (W - 1 + t - start)) * a.C + c0, pack4<E>(v), nv);
    }
  };

  int buf = 0, stage = 0;
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
    for (int tu = tb; tu < min(tb + kTile, t2) && !stop; tu += G) {
      const int ahead = stage == 0 ? S - 1 : stage - 1;
      inx.issue(ahead, tu + (S - 1) * G);
      ing.issue(ahead, tu + (S - 1) * G);
      R::commit();
      R::wait();
      if (!any && tu + G <= t1 && seg >= 0 && seg < a.n_seq && tu - (W - 1) >= max(t0, start)) {
        // inside one segment, all finished gradients this range's own
        E *to = dx + (int64_t)(tu - (W - 1)) * a.dx.st;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f2 done[4];
          token(inx.get(stage, g, tu + g), ing.get(stage, g, tu + g), true, done);
          st8<VEC>(to, pack4<E>(done), nv);
          to += a.dx.st;
        }
      } else {
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
          const int t = tu + g, i = t - tb;
          if (t >= t2) break;
          if (any && mark[i] >= 0) {
            if (t >= t1) {  // the next range's segment
              stop = true;
              break;
            }
            seg = mark[i];
            start = t;
            if (seg < a.n_seq) rows.fill(win, seg, t, 0);
            clear<W - 1>(acc);
          }
          if (seg >= 0 && seg < a.n_seq) {
            f2 done[4];
            token(inx.get(stage, g, t), ing.get(stage, g, t), t < t1, done);
            emit(t - (W - 1), done);
            if (any && mark[i + 1] >= 0) {  // the segment's last token
#pragma unroll
              for (int j = 0; j < W - 1; ++j) {
                if (dht) {
                  f2 f[4];
                  unpack4(ld8<VEC>(dht + ((int64_t)seg * (W - 1) + (W - 2 - j)) * a.C + c0, nv), f);
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[j][e] = add2(acc[j][e], f[e]);
                }
                emit(t - j, acc[j]);
              }
            }
          } else if (t < t1) {  // no segment: no gradient
            st8<VEC>(dx + (int64_t)t * a.dx.st, zero8<E>(), nv);
          }
        }
      }
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    __syncthreads();
  }
  if (VEC) copies_wait<0>();  // a range that stopped early has copies on their way
  float *work = reinterpret_cast<float *>(a.work) + (int64_t)r * (W + 1) * a.C + c0;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(k < W ? dw[k < W ? k : 0][i] : db[0][i], v[2 * i], v[2 * i + 1]);
    if (VEC) {
      if (nv > 0) {
        float4 *q = reinterpret_cast<float4 *>(work + (int64_t)k * a.C);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < nv) work[(int64_t)k * a.C + i] = v[i];
    }
  }
}

// Sums the ranges' parts of dw and db: 32 channels a block, its 8 warps taking every 8th range.
__global__ void __launch_bounds__(256)
    k_conv_sum(const float *work, int nranges, int C, int W, float *dw, float *db) {
  after_previous<true>();
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
  if (k == W && !db) return;
  const int64_t st = (int64_t)(W + 1) * C;
  float s[4] = {0, 0, 0, 0};
  if (c < C) {
    const float *p = work + (int64_t)k * C + c;
    int r = q;
    for (; r + 24 < nranges; r += 32)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += p[(r + 8 * i) * st];
    for (; r < nranges; r += 8) s[0] += p[r * st];
  }
  part[q][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (q != 0 || c >= C) return;
  float v = part[0][lane];
#pragma unroll
  for (int i = 1; i < 8; ++i) v += part[i][lane];
  if (k < W)
    dw[(int64_t)c * W + k] = v;
  else
    db[c] = v;
}

template <typename E, int W, bool VEC>
__global__ void __launch_bounds__(kThreads) k_conv_step(const ConvStepArgs a, int cblocks) {
  after_previous<true>();
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
  f2 win[W - 1][4], w[W][4], bias[4], x[4];
  load_taps<W>(a.w, a.b, c0, nv, w, bias);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) unpack4(old[k], win[k]);
  unpack4(rx, x);
  st8<VEC>(y, output<E, W>(w, bias, win, x, a.silu), nv);
#pragma unroll
  for (int k = 0; k + 1 < W - 1; ++k) st8<VEC>(s + (int64_t)k * a.C, old[k + 1], nv);
  st8<VEC>(s + (int64_t)(W - 2) * a.C, rx, nv);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// whether every 8-channel group of these rows starts on a 16-byte boundary
bool rows_ok(const Mat &m, bool f32) {
  return !m.p || (aligned16(m.p) && m.st % (f32 ? 4 : 8) == 0);
}

// How the channels and tokens are cut: blocks of 32 threads (256 channels) where blocks of 128
// would leave a quarter of their threads without channels, and as many ranges as run at once, of
// at least one tile of tokens.
struct Plan {
  int threads, cblocks, range, nranges;
};
Plan plan_for(int64_t T, int32_t C, int ctas) {
  Plan p;
  p.threads = ceil_div64(C, kThreads * 8) * kThreads * 8 * 3 > (int64_t)C * 4 ? 32 : kThreads;
  p.cblocks = (int)ceil_div64(C, p.threads * 8);
  int64_t n = (int64_t)sm_count() * ctas * (kThreads / p.threads) / p.cblocks;
  const int64_t most = ceil_div64(T, kTile);
  if (n > most) n = most;
  if (n < 1) n = 1;
  const int64_t r = ceil_div64(ceil_div64(T, n), kTile) * kTile;
  p.range = (int)(r < kTile ? kTile : r);
  p.nranges = (int)ceil_div64(T, p.range);
  return p;
}

template <typename E, int W, bool VEC, int TH>
cudaError_t fwd_threads(const ConvArgs &a, const Plan &p, cudaStream_t stream) {
  const int64_t blocks = (int64_t)p.cblocks * (p.nranges + (a.ht ? 1 : 0));
  if (blocks == 0) return cudaSuccess;
  constexpr int smem = FwdAhead<E, VEC, TH>::kSlots * 16;
  static_assert(smem <= 46 * 1024, "more shared memory than a launch has without asking");
  return launch(k_conv_fwd<E, W, VEC, TH>, (unsigned)blocks, TH, smem, stream, a, p.range,
                p.cblocks, p.nranges);
}
template <typename E, int W, bool VEC>
cudaError_t run_fwd(const ConvArgs &a, cudaStream_t stream) {
  const Plan p = plan_for(a.T, a.C, kFwdCtas);
  return p.threads == 32 ? fwd_threads<E, W, VEC, 32>(a, p, stream)
                         : fwd_threads<E, W, VEC, kThreads>(a, p, stream);
}

template <typename E, int W, bool VEC, int TH>
cudaError_t bwd_threads(const ConvArgs &a, const Plan &p, cudaStream_t stream) {
  const int64_t blocks = (int64_t)p.cblocks * (p.nranges + (a.dh0 ? 1 : 0));
  constexpr int smem = 2 * BwdAhead<E, VEC, TH>::kSlots * 16;
  static_assert(smem <= 46 * 1024, "more shared memory than a launch has without asking");
  cudaError_t e;
  if (blocks > 0 &&
      (e = launch(k_conv_bwd<E, W, VEC, TH>, (unsigned)blocks, TH, smem, stream, a, p.range,
                  p.cblocks, p.nranges)) != cudaSuccess)
    return e;
  return launch(k_conv_sum, dim3((unsigned)ceil_div64(a.C, 32), W + 1), 256, 0, stream,
                reinterpret_cast<const float *>(a.work), p.nranges, a.C, W, a.dw, a.db);
}
template <typename E, int W, bool VEC>
cudaError_t run_bwd(const ConvArgs &a, cudaStream_t stream) {
  const Plan p = plan_for(a.T, a.C, kBwdCtas);
  return p.threads == 32 ? bwd_threads<E, W, VEC, 32>(a, p, stream)
                         : bwd_threads<E, W, VEC, kThreads>(a, p, stream);
}

template <typename E, int W, bool VEC>
cudaError_t run_step(const ConvStepArgs &a, cudaStream_t stream) {
  const int cblocks = (int)ceil_div64(a.C, kThreads * 8);
  return launch(k_conv_step<E, W, VEC>, (unsigned)((int64_t)cblocks * a.B), kThreads, 0, stream, a,
                cblocks);
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
  return align256((size_t)mix::plan_for(T, C, mix::kBwdCtas).nranges * (W + 1) * C *
                  sizeof(float));
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
