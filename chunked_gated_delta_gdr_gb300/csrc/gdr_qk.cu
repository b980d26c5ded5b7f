// gdr_qk.cu -- the norm of queries and keys for each head with the position rotation in the same
// pass, forward and backward.  For a row x of d elements (one token and head):
//
//   r = (sum x^2 / d + eps)^-1/2  (RMS)   or   (sum x^2 + eps)^-1/2  (L2),      u = x r w,
//   y = R(p) u: pairs (a, b) -> (a cos - b sin, b cos + a sin), elements from `rot` on unchanged.
//
// Backward, with e = R(p)^T dy and m = w e:
//   dx = r m - x r^3 (sum x m) / d  (L2: without / d),   dw = sum over rows of e x r.
//
// Bound by HBM: each row is read once and written once.  8 elements a lane, 16 bytes of bf16; a
// group of lanes keeps one token's cosines and sines in registers while it runs over the token's
// heads, q's and then k's.  65,536 tokens of 48 heads of 128 in bf16: 277 us, 5.8 TB/s of 6.8; the
// backward 424 us, 5.7 TB/s.  L2 without a rotation 271 and 414.
#include <type_traits>

#include "gdr_mix.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kThreads = 128;
constexpr int kCtas = 4;    // blocks on each SM; each runs over many tokens
constexpr int kAnyCtas = 10;  // for any strides, where only warps hide the loads' latency
constexpr int kStages = 4;  // batches of rows on their way or in use (bf16)

__device__ __forceinline__ int place_of(const QkArgs &a, int64_t t) {
  return min(max(a.pos[t], 0), a.places - 1);
}

// Sums K (2 or 4) values of each lane over the LR lanes of a group: every lane gets all of them.
// A transposing butterfly: log2 K exchanges leave a lane with one of the sums, the rest of the
// butterfly completes it.  f is applied to the sums, once a lane.
template <int LR, int K, typename F>
__device__ __forceinline__ void group_sums(float (&v)[K], int gl, F f) {
  float b;
  int k = 0;
  const bool hi = gl & (LR / 2);
  if (K == 4) {
    const bool lo = gl & (LR / 4);
    const float a0 = (hi ? v[K - 2] : v[0]) +
                     __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[K - 2], LR / 2);
    const float a1 = (hi ? v[K - 1] : v[1]) +
                     __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[K - 1], LR / 2);
    b = (lo ? a1 : a0) + __shfl_xor_sync(0xffffffffu, lo ? a0 : a1, LR / 4);
    k = (hi ? 2 : 0) + (lo ? 1 : 0);
  } else {
    b = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], LR / 2);
    k = hi;
  }
#pragma unroll
  for (int o = LR / (2 * K); o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
  b = f(b, k);
#pragma unroll
  for (int i = 0; i < K; ++i)
    v[i] = __shfl_sync(0xffffffffu, b,
                       K == 4 ? (i >> 1) * (LR / 2) + (i & 1) * (LR / 4) : i * (LR / 2), LR);
}

// How a row of d elements lies over the lanes, 8 to each, d / 8 of a group's LR, so that the two
// elements of a rotated pair share a lane:
//   kNear    8 neighbours: four interleaved pairs, or no rotation
//   kHalves  4 neighbours and the 4 half the rotated part away (pairs i, i + rot / 2; rot a multiple
//            of 8), behind the rotated part 8 neighbours.  Partners by shuffles between lanes of 8
//            neighbours are slower for all their wider copies: 307 against 281 us at 65,536 tokens
//            of 48 heads of 128 in bf16, 713 against 516 in fp32.
enum Layout { kNear, kHalves };

// Cosines and sines of a lane's 8 elements, the sine with its sign for the forward rotation
// (u_e cos + u_partner sin).
struct Angles {
  f2 c[4], s[4];
};
__device__ __forceinline__ void load_angles(const QkArgs &a, int64_t t, int e0, float4 &c,
                                            float4 &s) {
  const int half = a.rot >> 1, at = e0 >> 1;
  const float *cos = a.cos + (int64_t)place_of(a, t) * half + at;
  const float *sin = a.sin + (int64_t)place_of(a, t) * half + at;
  if (a.quads) {
    c = *reinterpret_cast<const float4 *>(cos);
    s = *reinterpret_cast<const float4 *>(sin);
  } else {  // the rotated part may end inside the lane's elements: no rotation behind it
    float *cf = reinterpret_cast<float *>(&c), *sf = reinterpret_cast<float *>(&s);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i < half) {
        cf[i] = cos[i];
        sf[i] = sin[i];
      }
  }
}
template <int LAY>
__device__ __forceinline__ Angles signed_angles(const float4 &c, const float4 &s) {
  Angles r;
  if (LAY == kNear) {
    r.c[0] = pair(c.x, c.x);
    r.c[1] = pair(c.y, c.y);
    r.c[2] = pair(c.z, c.z);
    r.c[3] = pair(c.w, c.w);
    r.s[0] = pair(-s.x, s.x);
    r.s[1] = pair(-s.y, s.y);
    r.s[2] = pair(-s.z, s.z);
    r.s[3] = pair(-s.w, s.w);
  } else {
    r.c[0] = r.c[2] = pair(c.x, c.y);
    r.c[1] = r.c[3] = pair(c.z, c.w);
    r.s[0] = pair(-s.x, -s.y);
    r.s[1] = pair(-s.z, -s.w);
    r.s[2] = pair(s.x, s.y);
    r.s[3] = pair(s.z, s.w);
  }
  return r;
}

// The partners of a lane's 8 elements.
template <int LAY>
__device__ __forceinline__ void partners(const f2 (&u)[4], f2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpair(u[i], lo, hi);
    v[i] = LAY == kNear ? pair(hi, lo) : u[i ^ 2];
  }
}

// A lane's 8 elements to the row, the second four `gap` elements behind the first.
template <int LAY>
__device__ __forceinline__ void put_row(__nv_bfloat16 *p, int gap, const Raw8<__nv_bfloat16> &r) {
  if (LAY == kHalves) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(r.a.x, r.a.y);
    *reinterpret_cast<uint2 *>(p + gap) = make_uint2(r.a.z, r.a.w);
  } else {
    *reinterpret_cast<uint4 *>(p) = r.a;
  }
}
template <int LAY>
__device__ __forceinline__ void put_row(float *p, int gap, const Raw8<float> &r) {
  *reinterpret_cast<uint4 *>(p) = r.a;
  *reinterpret_cast<uint4 *>(p + (LAY == kHalves ? gap : 4)) = r.b;
}

struct Groups {
  int hp;  // lane groups of a block that share a token (its heads in turn)
  int tp;  // tokens of a block
};

template <typename E, bool BWD>
struct Ring {
  static constexpr int U = 2;                           // rows of a lane group in a batch
  static constexpr int P = (int)sizeof(E) / 2;          // 16-byte parts of a lane's 8 elements
  static constexpr int S = sizeof(E) == 2 ? kStages : 2;  // batches in the ring
  static constexpr int kSlot = U * (BWD ? 2 : 1) * P;
  static constexpr int kBytes = S * kSlot * kThreads * 16;
};

// A block runs over tokens tb, tb + gridDim.x and so on, and for each over batches of the heads of
// q, then of k, U rows a lane group.  The next S - 1 batches are on their way into a ring in shared
// memory in which each thread reads only what it copied itself.  The weights' products with the
// angles are formed once a token:
//   y_e = r (x_e (w_e cos_e) + x_partner (w_partner sin_e)).
template <typename E, int LR, int LAY, bool BWD>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_qk(const QkArgs a, const Groups gr, int token_blocks) {
  after_previous();
  using R = Ring<E, BWD>;
  constexpr int RP = kThreads / LR, U = R::U, S = R::S;
  __shared__ __align__(16) float ws[2][LR * 8];
  extern __shared__ __align__(16) uint4 ring[];
  const int grp = threadIdx.x / LR, gl = threadIdx.x % LR, e0 = gl * 8;
  const int hp = gr.hp, first = grp % hp, mine = grp / hp, rows = hp * U;
  const bool rotated = a.rot > 0, turned = e0 < a.rot;
  const bool has = e0 < a.d;  // the lane has elements
  // the lane's first element, and from it to its second four
  const int at0 = LAY == kHalves && turned ? gl * 4 : e0;
  const int gap = LAY == kHalves && turned ? a.rot >> 1 : 4;
  const float inv = a.rms ? 1.f / (float)a.d : 1.f;
  const int stride = gridDim.x, j0 = a.Hq > 0 ? 0 : 1;
  // whether a batch of q (k) has a row in every place, for a block of tokens inside T
  const bool even[2] = {hp * gr.tp == RP && a.Hq % rows == 0, hp * gr.tp == RP && a.Hk % rows == 0};
  auto inside = [&](int tb) { return (int64_t)(tb + 1) * gr.tp <= a.T; };
  auto alive = [&](int tb) { return mine < gr.tp && (int64_t)tb * gr.tp + mine < a.T; };
  auto slot = [&](int s, int u, int q) {
    return ring + ((s * R::kSlot + (u * (BWD ? 2 : 1) + q) * R::P) * kThreads + threadIdx.x);
  };
  // this lane group's first row of a tensor at its first token, and the step to its next token
  const int64_t t0 = (int64_t)blockIdx.x * gr.tp + mine, tstep = (int64_t)stride * gr.tp;
  auto start = [&](const void *base, int64_t st, int64_t sh) {
    return reinterpret_cast<const E *>(base) + t0 * st + first * sh + at0;
  };
  auto copy = [&](uint4 *to, const E *p) {  // a lane's 8 elements into its slot
    if (LAY == kHalves && sizeof(E) == 2) {
      copy8(to, p);
      copy8(reinterpret_cast<char *>(to) + 8, p + gap);
    } else {
#pragma unroll
      for (int i = 0; i < R::P; ++i) copy16(to + i * kThreads, p + (i ? gap : 0));
    }
  };

  // the copies' place: block of tokens, tensor, head, stage; the first rows at that token
  int at_tb = blockIdx.x, at_j = j0, at_h = 0, at_s = 0;
  const E *xb[2], *gb[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    xb[j] = start(a.x[j], a.x_st[j], a.x_sh[j]);
    gb[j] = start(a.y[j], a.y_st[j], a.y_sh[j]);
  }
  auto issue = [&]() {
    if (at_tb < token_blocks) {
      const bool k = at_j;
      const int heads = k ? a.Hk : a.Hq;
      const int64_t xs = hp * (k ? a.x_sh[1] : a.x_sh[0]), gs = hp * (k ? a.y_sh[1] : a.y_sh[0]);
      const E *x = k ? xb[1] : xb[0], *g = k ? gb[1] : gb[0];
      if (at_h > 0) {
        x += at_h * (k ? a.x_sh[1] : a.x_sh[0]);
        if (BWD) g += at_h * (k ? a.y_sh[1] : a.y_sh[0]);
      }
      const bool full = (k ? even[1] : even[0]) && inside(at_tb);
      const bool live = has && (full || alive(at_tb));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (live && (full || at_h + u * hp + first < heads)) {
          copy(slot(at_s, u, 0), x);
          if (BWD) copy(slot(at_s, u, 1), g);
        }
        x += xs;
        if (BWD) g += gs;
      }
      at_s = at_s + 1 == S ? 0 : at_s + 1;
      at_h += rows;
      if (at_h >= heads) {
        at_h = 0;
        at_j = !k && a.Hk > 0 ? 1 : j0;
        if (k || a.Hk == 0) {
          at_tb += stride;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            xb[j] += tstep * a.x_st[j];
            if (BWD) gb[j] += tstep * a.y_st[j];
          }
        }
      }
    }
    copies_commit();
  };
  auto row = [&](int s, int u, int q) {
    Raw8<E> r;
    uint4 *w = reinterpret_cast<uint4 *>(&r);
#pragma unroll
    for (int i = 0; i < R::P; ++i) w[i] = slot(s, u, q)[i * kThreads];
    return r;
  };
  // slots that a lane never fills read as zero; one that it leaves out holds an older row, whose
  // results go nowhere
  for (int i = threadIdx.x; i < R::kBytes / 16; i += kThreads) ring[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue();
  float4 ca = make_float4(1.f, 1.f, 1.f, 1.f), sa = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turned && alive(blockIdx.x)) load_angles(a, t0, e0, ca, sa);
  for (int i = threadIdx.x; i < 2 * LR * 8; i += kThreads) {
    const Param &w = i < LR * 8 ? a.w[0] : a.w[1];
    const int e = i % (LR * 8);
    ws[i / (LR * 8)][e] = e >= a.d ? 0.f : w.p ? ldp(w, e) : 1.f;
  }
  f2 dw[2][4];
  E *ob[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    ob[j] = const_cast<E *>(BWD ? start(a.dx[j], a.dx_st[j], a.dx_sh[j])
                                : start(a.y[j], a.y_st[j], a.y_sh[j]));
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = pair(0.f, 0.f);
  }
  __syncthreads();

  int stage = 0;
  for (int tb = blockIdx.x; tb < token_blocks; tb += stride) {
    const bool live = alive(tb), in = inside(tb);
    const Angles ang = signed_angles<LAY>(ca, sa);
    if (turned && tb + stride < token_blocks && alive(tb + stride))
      load_angles(a, (int64_t)(tb + stride) * gr.tp + mine, e0, ca, sa);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int heads = j ? a.Hk : a.Hq;
      const bool full = in && even[j];
      const int64_t os = hp * (BWD ? a.dx_sh[j] : a.y_sh[j]);
      E *p = ob[j];
      ob[j] += tstep * (BWD ? a.dx_st[j] : a.y_st[j]);
      f2 cw[4], sw[4];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float4 u = *reinterpret_cast<const float4 *>(&ws[j][i ? at0 + gap : at0]);
        cw[i] = pair(u.x, u.y);
        cw[i + 1] = pair(u.z, u.w);
        if (!BWD) {
          // the partners' weights
          float4 v = make_float4(u.y, u.x, u.w, u.z);
          if (LAY == kHalves) v = *reinterpret_cast<const float4 *>(&ws[j][i ? at0 : at0 + gap]);
          cw[i] = mul2(cw[i], ang.c[i]);
          cw[i + 1] = mul2(cw[i + 1], ang.c[i + 1]);
          sw[i] = mul2(pair(v.x, v.y), ang.s[i]);
          sw[i + 1] = mul2(pair(v.z, v.w), ang.s[i + 1]);
        }
      }
#pragma unroll 1
      for (int h = 0; h < heads; h += rows) {
        issue();
        copies_wait<S - 1>();
        Raw8<E> cx[U], cd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          cx[u] = row(stage, u, 0);
          if (BWD) cd[u] = row(stage, u, 1);
        }
        stage = stage + 1 == S ? 0 : stage + 1;
        if (!BWD) {
          float v[U];
          f2 x[U][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            unpack4(cx[u], x[u]);
            f2 q = mul2(x[u][0], x[u][0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) q = fma2(x[u][i], x[u][i], q);
            float q0, q1;
            unpair(q, q0, q1);
            v[u] = q0 + q1;
          }
          group_sums<LR>(v, gl, [&](float q, int) { return rsqrtf(fmaf(q, inv, a.eps)); });
#pragma unroll
          for (int u = 0; u < U; ++u) {
            f2 o[4];
            const f2 r = pair(v[u], v[u]);
            if (rotated) {
              partners<LAY>(x[u], o);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = mul2(fma2(x[u][i], cw[i], mul2(o[i], sw[i])), r);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = mul2(mul2(x[u][i], cw[i]), r);
            }
            if (has && (full || (live && h + u * hp + first < heads)))
              put_row<LAY>(p, gap, pack4<E>(o));
            p += os;
          }
        } else {
          f2 e[U][4], x[U][4];  // e: the rotation undone
          float v[2 * U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            unpack4(cx[u], x[u]);
            unpack4(cd[u], e[u]);
            if (rotated) {
              f2 o[4];
              partners<LAY>(e[u], o);
              const f2 minus = pair(-1.f, -1.f);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                e[u][i] = fma2(e[u][i], ang.c[i], mul2(mul2(o[i], minus), ang.s[i]));
            }
            f2 q = mul2(x[u][0], x[u][0]), d = mul2(mul2(e[u][0], cw[0]), x[u][0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              q = fma2(x[u][i], x[u][i], q);
              d = fma2(mul2(e[u][i], cw[i]), x[u][i], d);
            }
            float q0, q1;
            unpair(q, q0, q1);
            v[u] = q0 + q1;
            unpair(d, q0, q1);
            v[U + u] = q0 + q1;
          }
          group_sums<LR>(v, gl, [&](float q, int k) {
            return k < U ? rsqrtf(fmaf(q, inv, a.eps)) : q * inv;
          });
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const bool ok = has && (full || (live && h + u * hp + first < heads));
            const float rr = v[u], dd = -v[U + u] * rr * rr * rr;
            const f2 r = pair(rr, rr), d = pair(dd, dd);
            f2 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (ok) dw[j][i] = fma2(mul2(e[u][i], x[u][i]), r, dw[j][i]);
              o[i] = fma2(mul2(e[u][i], cw[i]), r, mul2(x[u][i], d));
            }
            if (ok) put_row<LAY>(p, gap, pack4<E>(o));
            p += os;
          }
        }
      }
    }
  }
  if (BWD) {  // this block's part of dw, its lane groups added in order
    __shared__ float part[RP][LR * 8];
    float *work = reinterpret_cast<float *>(a.work) + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (!a.dw[j]) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (has) {
          float *q = &part[grp][(i < 2 ? at0 : at0 + gap) + 2 * (i & 1)];
          unpair(dw[j][i], q[0], q[1]);
        }
      __syncthreads();
      for (int e = threadIdx.x; e < a.d; e += kThreads) {
        float v = 0.f;
        for (int k = 0; k < RP; ++k) v += part[k][e];
        work[j * a.d + e] = v;
      }
      __syncthreads();
    }
  }
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Any head size up to 256, any strides: one warp for each row, the row read again for the
// partners of the rotation (36,939 tokens of 15 heads of 232, half of each rotated by halves: 465 us
// where interleaved pairs take the fast path's 98; backward 1,419 and 149).  WIDE: the backward's row sums and its last
// difference are in 64 bits, for heads of a few elements: there r m and x r^3 (sum x m) / d nearly
// cancel (at d = 1 only eps is left).
template <typename E, bool BWD, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_qk_any(const QkArgs a, int64_t rows) {
  after_previous();
  constexpr int M = 8;  // elements of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = kThreads / 32;
  const int heads = a.Hq + a.Hk, half = a.rot >> 1;
  float dw[2][M];
#pragma unroll
  for (int i = 0; i < M; ++i) dw[0][i] = dw[1][i] = 0.f;
  for (int64_t row = blockIdx.x * (int64_t)nw + warp; row < rows; row += (int64_t)gridDim.x * nw) {
    const int64_t t = row / heads;
    const int h = (int)(row % heads), j = h < a.Hq ? 0 : 1, hj = j ? h - a.Hq : h;
    const E *x = reinterpret_cast<const E *>(a.x[j]) + t * a.x_st[j] + hj * a.x_sh[j];
    const E *y = reinterpret_cast<const E *>(a.y[j]) + t * a.y_st[j] + hj * a.y_sh[j];
    const int64_t base = a.rot > 0 ? (int64_t)place_of(a, t) * half : 0;
    using S = typename std::conditional<WIDE, double, float>::type;
    S q = 0;
    for (int e = lane; e < a.d; e += 32) q += (S)ld1(x + e) * (S)ld1(x + e);
    q = warp_sum(q) / (S)(a.rms ? a.d : 1) + (S)a.eps;
    const float r = rsqrtf((float)q);
    // element e of R v (back: R^T v), v read through f
    auto turned = [&](int e, bool back, auto f) {
      if (e >= a.rot) return f(e);
      const int at = a.interleaved ? e >> 1 : (e < half ? e : e - half);
      const bool low = a.interleaved ? (e & 1) == 0 : e < half;
      const int other = a.interleaved ? e ^ 1 : (low ? e + half : e - half);
      const float n = low != back ? -a.sin[base + at] : a.sin[base + at];
      return fmaf(f(other), n, f(e) * a.cos[base + at]);
    };
    if (!BWD) {
      E *out = reinterpret_cast<E *>(a.y[j]) + t * a.y_st[j] + hj * a.y_sh[j];
      for (int e = lane; e < a.d; e += 32)
        st1(out + e, turned(e, false, [&](int i) {
              return ld1(x + i) * r * (a.w[j].p ? ldp(a.w[j], i) : 1.f);
            }));
    } else {
      float m[M];
      S dot = 0;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const int e = lane + i * 32;
        m[i] = 0.f;
        if (e < a.d) {
          const float g = turned(e, true, [&](int k) { return ld1(y + k); });
          const float xv = ld1(x + e), gx = g * xv * r;
          if (j)
            dw[1][i] += gx;
          else
            dw[0][i] += gx;
          m[i] = g * (a.w[j].p ? ldp(a.w[j], e) : 1.f);
          dot += (S)m[i] * (S)xv;
        }
      }
      // dx = r (m - x dot / (d q)), q = mean x^2 + eps (L2: d = 1)
      dot = warp_sum(dot) / ((S)(a.rms ? a.d : 1) * q);
      E *out = reinterpret_cast<E *>(a.dx[j]) + t * a.dx_st[j] + hj * a.dx_sh[j];
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const int e = lane + i * 32;
        if (e < a.d) st1(out + e, r * (float)((S)m[i] - (S)ld1(x + e) * dot));
      }
    }
  }
  if (BWD) {
    __shared__ float part[kThreads / 32][32 * M];
    float *work = reinterpret_cast<float *>(a.work) + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (!a.dw[j]) continue;
#pragma unroll
      for (int i = 0; i < M; ++i) part[warp][lane + i * 32] = dw[j][i];
      __syncthreads();
      for (int e = threadIdx.x; e < a.d; e += kThreads) {
        float v = 0.f;
        for (int k = 0; k < nw; ++k) v += part[k][e];
        work[j * a.d + e] = v;
      }
      __syncthreads();
    }
  }
}

// dw: the blocks' parts, added by one block for each (tensor, 32 elements) in a fixed order.
__global__ void __launch_bounds__(1024)
    k_qk_sum(const float *work, int blocks, int d, float *dwq, float *dwk) {
  after_previous<true>();
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, j = blockIdx.y;
  const int e = blockIdx.x * 32 + lane;
  float *out = j ? dwk : dwq;
  if (!out) return;
  float v = 0.f;
  if (e < d) {
#pragma unroll 8
    for (int b = k; b < blocks; b += 32) v += work[((int64_t)b * 2 + j) * d + e];
  }
  part[k][lane] = v;
  __syncthreads();
  v = warp_sum(part[lane][k]);  // element k of the 32, over the rows
  if (lane == 0 && blockIdx.x * 32 + k < d) out[blockIdx.x * 32 + k] = v;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether every row starts on a boundary of `g` elements.
bool rows_on(const QkArgs &a, bool bwd, int g) {
  const uintptr_t bytes = (uintptr_t)g * (a.f32 ? 4 : 2) - 1;
  auto on = [&](const void *p, int64_t st, int64_t sh) {
    return (reinterpret_cast<uintptr_t>(p) & bytes) == 0 && ((st | sh) & (g - 1)) == 0;
  };
  for (int j = 0; j < 2; ++j) {
    if (!on(a.x[j], a.x_st[j], a.x_sh[j]) || !on(a.y[j], a.y_st[j], a.y_sh[j])) return false;
    if (bwd && !on(a.dx[j], a.dx_st[j], a.dx_sh[j])) return false;
  }
  return true;
}
// The layout that the head size, the rotation and the alignment allow, or -1.
int layout_of(const QkArgs &a, bool bwd) {
  if (a.d % 8 != 0) return -1;
  const bool whole = rows_on(a, bwd, a.f32 ? 4 : 8);
  if (a.interleaved || a.rot == 0) return whole ? kNear : -1;
  return a.rot % 8 == 0 && rows_on(a, bwd, 4) ? kHalves : -1;
}

int lanes_of(int d) {  // of a row's group: a power of two
  int n = 8;
  while (n * 8 < d) n *= 2;
  return n;
}

// hp: where the fewest places of a token's batches stay empty, and then the most heads (9 heads of
// 64 on as many lane groups as the block has: 35 us for 12,170 tokens, on 4 of them: 10 us).
template <int U>
Groups groups_for(const QkArgs &a) {
  const int rp = kThreads / lanes_of(a.d);
  int64_t least = 0;
  int hp = 1;
  for (int h = 1; h <= rp; h *= 2) {
    const int64_t places = h * (ceil_div64(a.Hq, h * U) + ceil_div64(a.Hk, h * U));
    if (h == 1 || places <= least) {
      least = places;
      hp = h;
    }
  }
  return Groups{hp, rp / hp};
}

int64_t most_blocks() { return (int64_t)sm_count() * kCtas; }

template <typename E, int LR, bool BWD>
cudaError_t run_fast(const QkArgs &a, int layout, cudaStream_t stream, int *blocks_out) {
  const Groups gr = groups_for<Ring<E, BWD>::U>(a);
  const int64_t tb = ceil_div64(a.T, gr.tp);
  int64_t blocks = tb;
  if (blocks > most_blocks()) blocks = most_blocks();
  *blocks_out = (int)blocks;
  constexpr int smem = Ring<E, BWD>::kBytes;
  static_assert(smem + 2 * LR * 8 * 4 + kThreads * 8 * 4 <= 48 * 1024,
                "more shared memory than a launch has without asking");
  if (layout == kNear)
    return launch(k_qk<E, LR, kNear, BWD>, (unsigned)blocks, kThreads, smem, stream, a, gr,
                  (int)tb);
  return launch(k_qk<E, LR, kHalves, BWD>, (unsigned)blocks, kThreads, smem, stream, a, gr,
                (int)tb);
}

template <typename E, bool BWD>
cudaError_t run(const QkArgs &args, cudaStream_t stream, int *blocks) {
  QkArgs a = args;
  a.quads = a.rot % 8 == 0 && aligned16(a.cos) && aligned16(a.sin);
  *blocks = 0;
  const int64_t rows = a.T * (a.Hq + a.Hk);
  if (rows == 0) return cudaSuccess;
  const int layout = layout_of(a, BWD);
  if (layout >= 0) {
    if (a.d <= 64) return run_fast<E, 8, BWD>(a, layout, stream, blocks);
    if (a.d <= 128) return run_fast<E, 16, BWD>(a, layout, stream, blocks);
    return run_fast<E, 32, BWD>(a, layout, stream, blocks);
  }
  int64_t n = ceil_div64(rows, kThreads / 32);
  const int64_t most = (int64_t)sm_count() * kAnyCtas;
  if (n > most) n = most;
  *blocks = (int)n;
  if (BWD && a.d <= 8)
    return launch(k_qk_any<E, BWD, BWD>, (unsigned)n, kThreads, 0, stream, a, rows);
  return launch(k_qk_any<E, BWD, false>, (unsigned)n, kThreads, 0, stream, a, rows);
}

}  // namespace
}  // namespace mix

cudaError_t launch_qk_fwd(const QkArgs &a, cudaStream_t stream) {
  int blocks;
  return a.f32 ? mix::run<float, false>(a, stream, &blocks)
               : mix::run<__nv_bfloat16, false>(a, stream, &blocks);
}

size_t qk_bwd_workspace(int64_t, int32_t, int32_t, int32_t d) {
  return align256((size_t)mix::sm_count() * mix::kAnyCtas * 2 * d * sizeof(float));
}

cudaError_t launch_qk_bwd(const QkArgs &a, cudaStream_t stream) {
  int blocks;
  cudaError_t e = a.f32 ? mix::run<float, true>(a, stream, &blocks)
                        : mix::run<__nv_bfloat16, true>(a, stream, &blocks);
  if (e != cudaSuccess || (!a.dw[0] && !a.dw[1])) return e;
  return mix::launch(mix::k_qk_sum, dim3((unsigned)ceil_div64(a.d, 32), 2), 1024, 0, stream,
                     reinterpret_cast<const float *>(a.work), blocks, a.d, a.dw[0], a.dw[1]);
}

}  // namespace gdr
