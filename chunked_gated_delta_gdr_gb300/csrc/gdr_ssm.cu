// gdr_ssm.cu -- the selective state space scan over packed segments (forward) and its
// single-token form.  Per channel d and state n, with dt = softplus(raw + bias):
//
//   h_t = e^{dt_t A_dn} h_{t-1} + dt_t x_t B_tn,   y_t = sum_n C_tn h_t + D_d x_t,
//   out_t = y_t z_t sigmoid(z_t).
//
// Everything is computed in fp32.  One token of one channel moves 8 bytes (bf16) and costs N
// exponentials and 4 N products: at N = 16 the special-function unit (8 lanes a cycle and
// sub-partition: 4 cycles for a warp) and the fp32 pipes are the bound before HBM is.
//
// The token axis is cut into ranges of equal length, whatever the segments are, so that a long
// prompt fills the GPU and ragged ones stay balanced.  Pass 1 runs each range from a zero state
// and keeps the state at its end and the sum of dt (a range's decay is e^{A sum dt}); pass 2
// chains the ends before its range, runs it from its true state and writes y.  When one range is
// enough, only pass 2 runs.  1,537 tokens of 1,002 x 12 states in fp32: 33 us, the latency of the
// passes; 2,048 of 4,096 x 16: 92 us.
#include "gdr_ssm.cuh"

namespace gdr {
namespace ssm {
namespace {

using namespace mix;

// Blocks of pass 2 on each SM, by which the ranges are cut: all of them run at once for up to 16
// states in bf16 and 8 in fp32.  A tile's tokens grow with the lanes of a channel, and the partial
// sums of y with both: 74 KB a block for 17 to 32 states, 138 KB above (fp32 93 and 157, 67 for 9 to 16
// states) leave 3 and 1 blocks (2 and 1, 3), so that the grid runs in up to four waves: 8,192 x
// 2,048 x 16, 32 and 64 in bf16 160, 358 and 1,016 us.
constexpr int kFwdCtas = 4;
constexpr int kEndCtas = 5;
constexpr int kAhead = 3;    // tiles in the rings
constexpr int kLeast = 4;    // tiles of a range at least where there are over kFew ranges
constexpr int kFew = 64;

template <int LN>
struct __align__(16) Tile1 {
  using Y = Lay<LN>;
  float2 pair[Y::L * Y::PT];
  float b[Y::L * Y::NP];
  float bias[Y::CH];
  int red[64];
};

// Pass 1: the state at the end of a range.  Only the segment alive there counts, from its start or
// the range's on.
template <typename E, int LN, bool VEC>
__global__ void __launch_bounds__(kThreads, kEndCtas)
    k_ssm_ends(const SsmArgs a, const Ranges rg, int tiles_per_group) {
  after_previous();
  using Y = Lay<LN>;
  using R = TileRing<E, VEC, kAhead>;
  constexpr int L = Y::L, NP = Y::NP, CH = Y::CH, Q = R::S;
  extern __shared__ __align__(16) char smem_raw[];
  Tile1<LN> &s = *reinterpret_cast<Tile1<LN> *>(smem_raw);
  uint4 *ring = reinterpret_cast<uint4 *>(&s + 1);
  const Place<LN> P(a, tiles_per_group);
  const int r0 = P.r * rg.range, t1 = min(a.T, r0 + rg.range);
  const int lt = P.tid / Y::CG, lc = P.tid % Y::CG * 8, nv = max(0, min(8, P.nch - lc));
  R xr(ring, a.x.p, P.c0 + lc, a.x.st, nv);
  R dr(ring + R::kSlots, a.dt.p, P.c0 + lc, a.dt.st, nv);
  const E *Bp = reinterpret_cast<const E *>(a.B) + P.grp * a.B_sg;
  for (int i = P.tid; i < CH; i += kThreads)
    s.bias[i] = step_bias(a.dt_bias, P.c0, P.nch, i);
  float A2[2][4], h[2][4], S[2] = {0.f, 0.f};
  const float most = P.decays(a, A2);
  const SegCursor c = seg_find(a.cu, a.n_seq, a.T, t1, s.red);
  const int seg = c.j - 1;
  const bool covered = seg >= 0 && seg < a.n_seq, reset = seg >= 0 && c.b >= r0;
  const int t0 = reset ? c.b : r0;
  P.read(a, covered && reset ? a.h0 : nullptr, seg, h);
  if (covered) {
    BcTile<E, NP, L, VEC> rb;
    auto issue = [&](int q, int tb) {
      const int n = tb + lt < t1 ? nv : 0;
      xr.issue(q, tb + lt, n);
      dr.issue(q, tb + lt, n);
      copies_commit();
    };
#pragma unroll
    for (int q = 0; q < Q - 1; ++q) issue(q, t0 + q * L);
    rb.fetch(Bp, a.B_st, t0, t1, a.N);
    __syncthreads();
    int stage = 0;
    for (int tb = t0; tb < t1; tb += L) {
      issue(stage == 0 ? Q - 1 : stage - 1, tb + (Q - 1) * L);
      copies_wait<Q - 1>();
      put_pairs<E, LN>(s.pair, s.bias, a.softplus, lt, lc, xr.get(stage),
                       dr.get(stage));
      stage = stage + 1 == Q ? 0 : stage + 1;
      rb.put(s.b);
      if (tb + L < t1) rb.fetch(Bp, a.B_st, tb + L, t1, a.N);
      __syncthreads();
      tile_tokens<L>(0, min(L, t1 - tb), [&](int i) {
        const float4 d = *reinterpret_cast<const float4 *>(
            &s.pair[i * Y::PT + P.pair]);
        const float4 B = *reinterpret_cast<const float4 *>(&s.b[i * NP + P.nl * 4]);
        const float dt[2] = {d.x, d.z}, dx[2] = {d.y, d.w}, Bv[4] = {B.x, B.y, B.z, B.w};
        const float more = raised(dt, most);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          S[k] += dt[k];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[k][j] = fmaf(decay(dt[k], A2[k][j], more), h[k][j], dx[k] * Bv[j]);
        }
      });
      __syncthreads();
    }
  }
  P.write(a, rg.state, P.r, h);
  if (P.nl == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (P.ch[k] < P.nch) rg.sum[(int64_t)P.r * a.D + P.c0 + P.ch[k]] = S[k];
  }
  if (P.ct == 0 && P.tid == 0) rg.reset[P.r] = reset;
}

// h = the state that enters range r: over the ranges before it, next = e^{A sum} state + end, or the
// end alone where a segment starts in the range.  Where the ranges are few, each block of pass 2
// does this itself: a launch less.
template <int LN>
__device__ __forceinline__ void entering_state(const SsmArgs &a, const Ranges &rg,
                                               const Place<LN> &P, int r,
                                               const float (&A2)[2][4], float (&h)[2][4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) h[k][j] = 0.f;
#pragma unroll 4
  for (int q = 0; q < r; ++q) {
    float end[2][4];
    P.read(a, rg.state, q, end);
    const bool reset = rg.reset[q] != 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float sum = P.ch[k] < P.nch ? rg.sum[(int64_t)q * a.D + P.c0 + P.ch[k]] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[k][j] = reset ? end[k][j] : fmaf(ex2(A2[k][j] * sum), h[k][j], end[k][j]);
    }
  }
}

// The states that enter the ranges, in the places of their ends: by a kernel of its own where the
// ranges are many (chained).
__global__ void k_ssm_chain(const float *A, const Ranges rg, int D, int N) {
  after_previous<true>();
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, size = (int64_t)D * N;
  if (i >= size) return;
  chain_ranges(rg.state, rg.sum, rg.reset, rg.n, D, size, i, (int)(i / N), A[i] * kLog2e, false);
}

template <int LN>
struct __align__(16) Tile2 {  // shared memory of one tile of pass 2
  using Y = Lay<LN>;
  float2 pair[Y::L * Y::PT];  // (dt, dt x)
  float b[Y::L * Y::NP], c[Y::L * Y::NP];
  float part[Y::L * Y::ST];
  float bias[Y::CH], skip[Y::CH];
  int mark[Y::L + 1], seg[Y::L], any, same;
  int red[64];
};

// Pass 2: a range from its true state.
template <typename E, int LN, bool VEC>
__global__ void __launch_bounds__(kThreads, kFwdCtas)
    k_ssm_fwd(const SsmArgs a, const Ranges rg, int tiles_per_group) {
  after_previous();
  using Y = Lay<LN>;
  using R = TileRing<E, VEC, kAhead>;
  constexpr int L = Y::L, NP = Y::NP, CH = Y::CH, Q = R::S;
  extern __shared__ __align__(16) char smem_raw[];
  Tile2<LN> &s = *reinterpret_cast<Tile2<LN> *>(smem_raw);
  uint4 *ring = reinterpret_cast<uint4 *>(&s + 1);
  const Place<LN> P(a, tiles_per_group);
  if (P.r == rg.n) {  // final states of the segments without tokens
    for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
      const int64_t at = ((int64_t)n * a.D + P.c0) * a.N;
      for (int i = P.tid; i < P.nch * a.N; i += kThreads)
        a.ht[at + i] = a.h0 ? a.h0[at + i] : 0.f;
    });
    return;
  }
  const int t0 = P.r * rg.range, t1 = min(a.T, t0 + rg.range);
  const int lt = P.tid / Y::CG, lc = P.tid % Y::CG * 8, nv = max(0, min(8, P.nch - lc));
  R xr(ring, a.x.p, P.c0 + lc, a.x.st, nv);
  R dr(ring + R::kSlots, a.dt.p, P.c0 + lc, a.dt.st, nv);
  R zr(ring + 2 * R::kSlots, a.z.p, P.c0 + lc, a.z.st, nv);
  const bool gated = a.z.p != nullptr;
  E *yp = reinterpret_cast<E *>(a.y.p) + P.c0 + lc;
  const E *Bp = reinterpret_cast<const E *>(a.B) + P.grp * a.B_sg;
  const E *Cp = reinterpret_cast<const E *>(a.C) + P.grp * a.C_sg;
  for (int i = P.tid; i < CH; i += kThreads) {
    s.bias[i] = step_bias(a.dt_bias, P.c0, P.nch, i);
    s.skip[i] = a.Dskip && i < P.nch ? a.Dskip[P.c0 + i] : 0.f;
  }
  BcTile<E, NP, L, VEC> rb, rc;
  auto issue = [&](int q, int tb) {
    const int n = tb + lt < t1 ? nv : 0;
    xr.issue(q, tb + lt, n);
    dr.issue(q, tb + lt, n);
    if (gated) zr.issue(q, tb + lt, n);
    copies_commit();
  };
#pragma unroll
  for (int q = 0; q < Q - 1; ++q) issue(q, t0 + q * L);
  rb.fetch(Bp, a.B_st, t0, t1, a.N);
  rc.fetch(Cp, a.C_st, t0, t1, a.N);
  float A2[2][4], h[2][4];
  const float most = P.decays(a, A2);
  SegCursor cursor = seg_find(a.cu, a.n_seq, a.T, t0, s.red);
  int seg = cursor.j - 1;
  const bool enters = P.r > 0 && seg >= 0 && seg < a.n_seq;
  if (rg.n > kChainRanges)
    P.read(a, enters ? rg.state : nullptr, P.r, h);
  else
    entering_state<LN>(a, rg, P, enters ? P.r : 0, A2, h);
  __syncthreads();

  // where this thread's partial sums of its two channels go in a token's row
  int po[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) po[k] = Y::part_at(0, P.ch[k]) + P.nl;
  auto scan = [&](int i0, int i1) {
    tile_tokens<L>(i0, i1, [&](int i) {
      const float4 d = *reinterpret_cast<const float4 *>(
          &s.pair[i * Y::PT + P.pair]);
      const float4 B = *reinterpret_cast<const float4 *>(&s.b[i * NP + P.nl * 4]);
      const float4 C = *reinterpret_cast<const float4 *>(&s.c[i * NP + P.nl * 4]);
      const float dt[2] = {d.x, d.z}, dx[2] = {d.y, d.w}, Bv[4] = {B.x, B.y, B.z, B.w};
      const float more = raised(dt, most);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[k][j] = fmaf(decay(dt[k], A2[k][j], more), h[k][j], dx[k] * Bv[j]);
        s.part[po[k] + i * Y::ST] =
            fmaf(h[k][0], C.x, fmaf(h[k][1], C.y, fmaf(h[k][2], C.z, h[k][3] * C.w)));
      }
    });
  };

  int stage = 0;
  for (int tb = t0; tb < t1; tb += L) {
    const int n = min(L, t1 - tb);
    issue(stage == 0 ? Q - 1 : stage - 1, tb + (Q - 1) * L);
    copies_wait<Q - 1>();
    put_pairs<E, LN>(s.pair, s.bias, a.softplus, lt, lc, xr.get(stage),
                     dr.get(stage));
    rb.put(s.b);
    rc.put(s.c);
    if (P.warp == 0) {
      const int carry = cursor.j - 1;
      const bool any = seg_marks(a.cu, a.n_seq, a.T, tb, n, s.mark, cursor);
      if (any) {
        int base = carry;
        for (int i0 = 0; i0 < L; i0 += 32) {
          int v = i0 + P.lane < n ? s.mark[i0 + P.lane] : -1;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (P.lane >= o) v = max(v, u);
          }
          v = max(v, base);
          if (i0 + P.lane < L) s.seg[i0 + P.lane] = v;
          base = __shfl_sync(0xffffffffu, v, 31);
        }
      }
      if (P.lane == 0) {
        s.any = any;
        s.same = carry;
      }
    }
    if (tb + L < t1) {
      rb.fetch(Bp, a.B_st, tb + L, t1, a.N);
      rc.fetch(Cp, a.C_st, tb + L, t1, a.N);
    }
    __syncthreads();
    const bool any = s.any;
    if (!any) {
      if (seg >= 0 && seg < a.n_seq) scan(0, n);
    } else {
      for (int i = 0; i < n;) {
        if (s.mark[i] >= 0) {
          seg = s.mark[i];
          P.read(a, seg < a.n_seq ? a.h0 : nullptr, seg, h);
        }
        int e = i + 1;
        while (e < n && s.mark[e] < 0) ++e;
        if (seg >= 0 && seg < a.n_seq) {
          scan(i, e);
          if (a.ht && s.mark[e] >= 0) P.write(a, a.ht, seg, h);
        }
        i = e;
      }
    }
    __syncthreads();
    const int own = any ? s.seg[lt] : s.same;
    if (lt < n && own >= 0 && own < a.n_seq) {
      float x[8], v[8];
      unpack8(xr.get(stage), x);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 w = *reinterpret_cast<const float4 *>(&s.skip[lc + i]);
        const float *part = &s.part[Y::part_at(lt, lc) + i * LN];
        v[i] = fmaf(w.x, x[i], sum_parts<LN>(part));
        v[i + 1] = fmaf(w.y, x[i + 1], sum_parts<LN>(part + LN));
        v[i + 2] = fmaf(w.z, x[i + 2], sum_parts<LN>(part + 2 * LN));
        v[i + 3] = fmaf(w.w, x[i + 3], sum_parts<LN>(part + 3 * LN));
      }
      if (gated) {
        unpack8(zr.get(stage), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= x[i] * sigmoidf(x[i]);
      }
      st8<VEC>(yp + (int64_t)(tb + lt) * a.y.st, pack8(v, E{}), nv);
    }
    stage = stage + 1 == Q ? 0 : stage + 1;
    __syncthreads();
  }
}

// Four neighbouring elements as fp32, in one read (VEC) or the first n of them.
template <bool VEC>
__device__ __forceinline__ void four(const __nv_bfloat16 *p, int n, float (&f)[4]) {
  if (VEC) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    f[0] = lo_bf(v.x);
    f[1] = hi_bf(v.x);
    f[2] = lo_bf(v.y);
    f[3] = hi_bf(v.y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? ld1(p + i) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void four(const float *p, int n, float (&f)[4]) {
  if (VEC) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? p[i] : 0.f;
  }
}

// One token for each row: state slot idx[row] in place.  Bound by HBM: the states are read and
// written once.  A warp takes CW neighbouring channels of a row: LN lanes hold a channel's states,
// 4 each, and K times PER channels follow one another, so that each of its K loads of states is one
// run of 512 bytes.  What belongs to a channel alone (step size, skip, gate, output) is one lane's
// each, and the sums over states come back to it.  128 rows of 4,096 x 16 states: 14.5 us with
// the states in HBM (4.8 TB/s; one fill and one drain of the GPU are a third of it), 9.3 us from L2.
template <typename E, int LN>
__global__ void __launch_bounds__(kThreads)
    k_ssm_step(const SsmArgs a, float *state, int slots, const int32_t *idx, int cblocks) {
  after_previous<true>();
  constexpr int PER = 32 / LN, K = LN < 8 ? LN : 8, CW = PER * K;
  const int row = blockIdx.x / cblocks, lane = threadIdx.x & 31;
  const int d0 = (blockIdx.x % cblocks * (kThreads / 32) + (threadIdx.x >> 5)) * CW;
  if (d0 >= a.D) return;
  const int slot = idx ? idx[row] : row, d = d0 + lane;
  const bool own = lane < CW && d < a.D;  // lane's own channel
  E *y = reinterpret_cast<E *>(a.y.p) + (int64_t)row * a.y.st + d;
  if (slot < 0 || slot >= slots) {
    if (own) st1(y, 0.f);
    return;
  }
  const int g = lane / LN, nl = lane % LN, n0 = nl * 4;
  const bool in = n0 < a.N;
  const int64_t at = (int64_t)(d0 + g) * a.N + n0;
  float *s = state + (int64_t)slot * a.D * a.N + at;
  float4 h[K], A[K];
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const bool ok = in && d0 + g + c * PER < a.D;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    h[c] = ok ? *reinterpret_cast<const float4 *>(s + c * PER * a.N) : zero;
    A[c] = ok ? *reinterpret_cast<const float4 *>(a.A + at + c * PER * a.N) : zero;
  }
  float B[4] = {0, 0, 0, 0}, C[4] = {0, 0, 0, 0}, x = 0.f, v = 0.f, z = 0.f, skip = 0.f;
  if (in) {
    const int grp = a.G == 1 ? 0 : d0 / (a.D / a.G);
    four<true>(reinterpret_cast<const E *>(a.B) + (int64_t)row * a.B_st + grp * a.B_sg + n0, 4, B);
    four<true>(reinterpret_cast<const E *>(a.C) + (int64_t)row * a.C_st + grp * a.C_sg + n0, 4, C);
  }
  if (own) {
    x = ld1(reinterpret_cast<const E *>(a.x.p) + (int64_t)row * a.x.st + d);
    v = ld1(reinterpret_cast<const E *>(a.dt.p) + (int64_t)row * a.dt.st + d);
    if (a.z.p) z = ld1(reinterpret_cast<const E *>(a.z.p) + (int64_t)row * a.z.st + d);
    if (a.dt_bias) v += a.dt_bias[d];
    if (a.Dskip) skip = a.Dskip[d];
    if (a.softplus) v = softplusf(v);
  }
  const float v2 = v * kLog2e, dx = v * x;
  float part[K];
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const float w = __shfl_sync(0xffffffffu, v2, c * PER + g);
    const float u = __shfl_sync(0xffffffffu, dx, c * PER + g);
    const bool lasts = A[c].x == 0.f || A[c].y == 0.f || A[c].z == 0.f || A[c].w == 0.f;
    const float more = raised(w, lasts ? 0.f : kShort);
    h[c].x = fmaf(decay(w, A[c].x, more), h[c].x, u * B[0]);
    h[c].y = fmaf(decay(w, A[c].y, more), h[c].y, u * B[1]);
    h[c].z = fmaf(decay(w, A[c].z, more), h[c].z, u * B[2]);
    h[c].w = fmaf(decay(w, A[c].w, more), h[c].w, u * B[3]);
    if (in && d0 + g + c * PER < a.D) *reinterpret_cast<float4 *>(s + c * PER * a.N) = h[c];
    part[c] = in ? fmaf(h[c].x, C[0], fmaf(h[c].y, C[1], fmaf(h[c].z, C[2], h[c].w * C[3]))) : 0.f;
  }
  // sums over a channel's lanes, each exchange halving what a lane sums
#pragma unroll
  for (int o = LN / 2, k = K; o > 0; o >>= 1) {
    const bool hi = nl & o;
    if (k > 1) {
      k /= 2;
#pragma unroll
      for (int c = 0; c < k; ++c) {
        const float send = hi ? part[c] : part[c + k];
        part[c] = (hi ? part[c + k] : part[c]) + __shfl_xor_sync(0xffffffffu, send, o);
      }
    } else {
      part[0] += __shfl_xor_sync(0xffffffffu, part[0], o);
    }
  }
  const int q = lane % CW;  // channel q's sum: lane q / PER (K of LN hold one) of group q % PER
  float sum = __shfl_sync(0xffffffffu, part[0], q % PER * LN + q / PER * (LN / K));
  sum = fmaf(skip, x, sum);
  if (a.z.p) sum *= z * sigmoidf(z);
  if (own) st1(y, sum);
}

// The same for any alignment and any groups: a thread holds 4 states of 4 neighbouring channels.
template <typename E, int LN>
__global__ void __launch_bounds__(kThreads)
    k_ssm_step_any(const SsmArgs a, float *state, int slots, const int32_t *idx, int cblocks) {
  after_previous<true>();
  constexpr int CB = kThreads / LN * 4;  // channels of a block
  const int row = blockIdx.x / cblocks;
  const int d0 = blockIdx.x % cblocks * CB + threadIdx.x / LN * 4, n0 = threadIdx.x % LN * 4;
  const int nd = max(0, min(4, a.D - d0)), nn = max(0, min(4, a.N - n0));
  const int slot = idx ? idx[row] : row;
  E *y = reinterpret_cast<E *>(a.y.p) + (int64_t)row * a.y.st + d0;
  if (slot < 0 || slot >= slots) {
    if (n0 == 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < nd) st1(y + c, 0.f);
    }
    return;
  }
  const bool on = nd > 0 && nn > 0;
  const int64_t at = (int64_t)d0 * a.N + n0;
  float *s = state + (int64_t)slot * a.D * a.N + at;
  float h[4][4], A[4][4], x[4], dt[4], z[4], bias[4], skip[4], B[4], C[4], part[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    x[c] = dt[c] = z[c] = bias[c] = skip[c] = B[c] = C[c] = part[c] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[c][j] = A[c][j] = 0.f;
  }
  const int Dg = a.D / a.G;
  const E *Bp = reinterpret_cast<const E *>(a.B) + (int64_t)row * a.B_st + n0;
  const E *Cp = reinterpret_cast<const E *>(a.C) + (int64_t)row * a.C_st + n0;
  if (on) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < nd) {
        four<false>(s + c * a.N, nn, h[c]);
        four<false>(a.A + at + c * a.N, nn, A[c]);
      }
  }
  if (nd > 0) {
    four<false>(reinterpret_cast<const E *>(a.x.p) + (int64_t)row * a.x.st + d0, nd, x);
    four<false>(reinterpret_cast<const E *>(a.dt.p) + (int64_t)row * a.dt.st + d0, nd, dt);
    if (a.z.p) four<false>(reinterpret_cast<const E *>(a.z.p) + (int64_t)row * a.z.st + d0, nd, z);
    if (a.dt_bias) four<false>(a.dt_bias + d0, nd, bias);
    if (a.Dskip) four<false>(a.Dskip + d0, nd, skip);
  }
  if (on) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c >= nd) break;
      four<false>(Bp + (d0 + c) / Dg * a.B_sg, nn, B);
      four<false>(Cp + (d0 + c) / Dg * a.C_sg, nn, C);
      float v = dt[c] + bias[c];
      if (a.softplus) v = softplusf(v);
      const float dx = v * x[c];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float more = raised(v, A[c][j] == 0.f ? 0.f : kShort);
        h[c][j] = fmaf(decay(v, A[c][j] * kLog2e, more), h[c][j], dx * B[j]);
        part[c] = fmaf(h[c][j], C[j], part[c]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < nn) s[c * a.N + j] = h[c][j];
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) part[c] += __shfl_xor_sync(0xffffffffu, part[c], o);
    part[c] = fmaf(skip[c], x[c], part[c]);
    if (a.z.p) part[c] *= z[c] * sigmoidf(z[c]);
  }
  if (n0 == 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < nd) st1(y + c, part[c]);
  }
}

// Tokens of a range: as many ranges as run at once, but no more than make a long chain.  Short
// ranges shorten the two passes of little work: 339 tokens of 448 channels of 32 states in fp32 27 us
// in ranges of four tiles, 15 us in ranges of one, 1,537 of 1,002 of 12 36 and 32; 7,922 of 128 of 16
// 29.7 us and, with the chain over two and a half times the ranges, 31.7.
int range_for(int64_t T, int32_t D, int32_t N, int32_t G) {
  const int LN = lanes_for(N), tile = 4 * LN;
  const int64_t ctiles = channel_tiles(D, G, LN);
  int64_t n = (int64_t)sm_count() * kFwdCtas / ctiles;
  int64_t most = ceil_div64(T, kLeast * tile);
  if (most < kFew) most = min((int64_t)kFew, ceil_div64(T, tile));
  if (n > most) n = most;
  if (n < 1) n = 1;
  const int64_t r = ceil_div64(ceil_div64(T, n), tile) * tile;
  return (int)(r < tile ? tile : r);
}

template <typename E, int LN, bool VEC>
cudaError_t run_fwd(const SsmArgs &a, cudaStream_t stream) {
  const int tpg = (int)ceil_div64(a.D / a.G, Lay<LN>::CH), ctiles = tpg * a.G;
  const Carve c = carve_ranges(a.work, a.T, a.D, a.N, range_for(a.T, a.D, a.N, a.G));
  constexpr int slots = TileRing<E, VEC, kAhead>::kSlots * 16;
  constexpr int smem1 = (int)sizeof(Tile1<LN>) + 2 * slots,
                smem2 = (int)sizeof(Tile2<LN>) + 3 * slots;
  cudaError_t e;
  if (c.rg.n > 1) {
    if (smem1 > 48 * 1024 && (e = allow_smem(k_ssm_ends<E, LN, VEC>, smem1)) != cudaSuccess)
      return e;
    if ((e = launch(k_ssm_ends<E, LN, VEC>, (unsigned)((int64_t)ctiles * (c.rg.n - 1)), kThreads,
                    smem1, stream, a, c.rg, tpg)) != cudaSuccess)
      return e;
    if (c.rg.n > kChainRanges) {
      if ((e = launch(k_ssm_chain, (unsigned)ceil_div64((int64_t)a.D * a.N, 128), 128, 0, stream,
                      a.A, c.rg, a.D, a.N)) != cudaSuccess)
        return e;
    }
  }
  const int64_t blocks = (int64_t)ctiles * (c.rg.n + (a.ht ? 1 : 0));
  if (blocks == 0) return cudaSuccess;
  if (smem2 > 48 * 1024 && (e = allow_smem(k_ssm_fwd<E, LN, VEC>, smem2)) != cudaSuccess) return e;
  return launch(k_ssm_fwd<E, LN, VEC>, (unsigned)blocks, kThreads, smem2, stream, a, c.rg, tpg);
}

template <typename E>
cudaError_t fwd_by_lanes(const SsmArgs &a, bool vec, cudaStream_t stream) {
  switch (lanes_for(a.N)) {
    case 2: return vec ? run_fwd<E, 2, true>(a, stream) : run_fwd<E, 2, false>(a, stream);
    case 4: return vec ? run_fwd<E, 4, true>(a, stream) : run_fwd<E, 4, false>(a, stream);
    case 8: return vec ? run_fwd<E, 8, true>(a, stream) : run_fwd<E, 8, false>(a, stream);
    default: return vec ? run_fwd<E, 16, true>(a, stream) : run_fwd<E, 16, false>(a, stream);
  }
}

template <typename E, int LN>
cudaError_t run_step(const SsmArgs &a, float *state, int32_t slots, const int32_t *idx,
                     cudaStream_t stream) {
  constexpr int CW = 32 / LN * (LN < 8 ? LN : 8);  // channels of a warp
  const uintptr_t four = a.f32 ? 15 : 7;           // four elements of B and C
  auto fit = [&](const void *p, int64_t st, int64_t sg) {
    return (reinterpret_cast<uintptr_t>(p) & four) == 0 && ((st | sg) & 3) == 0;
  };
  if (a.N % 4 == 0 && aligned16(state) && aligned16(a.A) && (a.G == 1 || a.D / a.G % CW == 0) &&
      fit(a.B, a.B_st, a.B_sg) && fit(a.C, a.C_st, a.C_sg)) {
    const int64_t cblocks = ceil_div64(a.D, kThreads / 32 * CW);
    return launch(k_ssm_step<E, LN>, (unsigned)(cblocks * a.T), kThreads, 0, stream, a, state,
                  slots, idx, (int)cblocks);
  }
  const int64_t cblocks = ceil_div64(a.D, kThreads / LN * 4);
  return launch(k_ssm_step_any<E, LN>, (unsigned)(cblocks * a.T), kThreads, 0, stream, a, state,
                slots, idx, (int)cblocks);
}
template <typename E>
cudaError_t step_by_lanes(const SsmArgs &a, float *state, int32_t slots, const int32_t *idx,
                          cudaStream_t stream) {
  switch (lanes_for(a.N)) {
    case 2: return run_step<E, 2>(a, state, slots, idx, stream);
    case 4: return run_step<E, 4>(a, state, slots, idx, stream);
    case 8: return run_step<E, 8>(a, state, slots, idx, stream);
    default: return run_step<E, 16>(a, state, slots, idx, stream);
  }
}

}  // namespace
}  // namespace ssm

size_t ssm_fwd_workspace(int64_t T, int32_t D, int32_t N, int32_t G) {
  // the layout also goes by the tensors' type and alignment: room for either (fp32 takes the wide one
  // wherever bf16 does)
  const size_t lanes = ssm::carve_ranges(nullptr, T, D, N, ssm::range_for(T, D, N, G)).bytes;
  const int wide = ssm::wide_range(T, D, N, G, true);
  const size_t bytes = wide ? ssm::carve_ranges(nullptr, T, D, N, wide).bytes : 0;
  return bytes > lanes ? bytes : lanes;
}

cudaError_t launch_ssm_fwd(const SsmArgs &args, cudaStream_t stream) {
  using namespace ssm;
  SsmArgs a = args;
  a.n4 = states_ok(a);
  const bool vec = (a.D / a.G) % 8 == 0 && rows_ok(a.x, a.f32) && rows_ok(a.dt, a.f32) &&
                   rows_ok(a.z, a.f32) && rows_ok(a.y, a.f32) && bc_ok(a);
  const int wide = vec ? wide_range(a.T, a.D, a.N, a.G, a.f32) : 0;
  if (wide) return launch_wide(a, wide, stream);
  return a.f32 ? fwd_by_lanes<float>(a, vec, stream)
               : fwd_by_lanes<__nv_bfloat16>(a, vec, stream);
}

cudaError_t launch_ssm_step(const SsmArgs &a, float *state, int32_t slots, const int32_t *idx,
                            cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return a.f32 ? ssm::step_by_lanes<float>(a, state, slots, idx, stream)
               : ssm::step_by_lanes<__nv_bfloat16>(a, state, slots, idx, stream);
}

}  // namespace gdr
