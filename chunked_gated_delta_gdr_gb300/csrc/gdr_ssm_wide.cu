// gdr_ssm_wide.cu -- the selective state space scan (forward) for much work: one thread a channel,
// all its states in registers (up to 16), where gdr_ssm.cu spreads a channel over lanes.
//
// A token's B and C are the same for every lane, one broadcast read of shared memory for four
// states, and y needs no sum over lanes: 8.2 instructions a token, channel and state against 8.8,
// and under half the shared-memory traffic, which bounds the other layout beside issue.  It takes
// four times the tokens and channels to fill the GPU, and a lone token takes longer: the launcher
// takes this layout where the work is enough for it.
//
// What bounds it: an exponential takes about two of the issue slots of the products beside it (8
// of them with 32 products: 49 cycles a warp and sub-partition), so that a token's 16 states cost
// at least 98 cycles, with the step size, gate and traffic about 150; measured 195.
//
// Ranges, pass 1 and pass 2 are those of gdr_ssm.cu; the decays are the approximate exponential's as
// they are, without what gdr_ssm.cuh's decay adds.  20,468 tokens of 4,096 x 16 states in bf16: 680 us
// (258 and 427 under the profiler), 76 and 72 % of the issue slots.
#include "gdr_ssm.cuh"

namespace gdr {
namespace ssm {
namespace {

using namespace mix;

constexpr int kL = 16;        // tokens of a tile
constexpr int kCtas = 4;      // blocks on each SM: the ranges are cut to run all at once
constexpr int kMost = 32;     // ranges at most

template <typename E>
struct Stages {
  static constexpr int S = sizeof(E) == 2 ? 3 : 2;  // tiles of x, dt and z in shared memory
};

template <typename E, int NS, int TENSORS>
struct __align__(16) Shared {
  E in[Stages<E>::S][TENSORS][kL][kThreads];
  float b[2][kL][NS], c[2][kL][NS];
  int mark[2][kL + 1], any[2];
  int red[64];
};

// A block's range and channels; this thread's channel.
struct Wide {
  int tid, r, grp, c0, nch;
  int64_t d;
  bool on;
  __device__ __forceinline__ Wide(const SsmArgs &a, int tiles_per_group) {
    tid = threadIdx.x;
    const int ctiles = tiles_per_group * a.G, Dg = a.D / a.G, ct = blockIdx.x % ctiles;
    r = blockIdx.x / ctiles;
    grp = ct / tiles_per_group;
    c0 = grp * Dg + ct % tiles_per_group * kThreads;
    nch = min(kThreads, (grp + 1) * Dg - c0);
    on = tid < nch;
    d = c0 + tid;
  }
  template <int NS>
  __device__ __forceinline__ void read(const SsmArgs &a, const float *p, int64_t row,
                                       float (&h)[NS]) const {
    const float *q = p + (row * a.D + d) * a.N;
    const bool in = p && on;
#pragma unroll
    for (int j = 0; j < NS; j += 4) {
      if (a.n4) {
        const float4 v = in && j < a.N ? *reinterpret_cast<const float4 *>(q + j)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
        h[j] = v.x;
        h[j + 1] = v.y;
        h[j + 2] = v.z;
        h[j + 3] = v.w;
      } else {
#pragma unroll
        for (int i = j; i < j + 4; ++i) h[i] = in && i < a.N ? q[i] : 0.f;
      }
    }
  }
  template <int NS>
  __device__ __forceinline__ void write(const SsmArgs &a, float *p, int64_t row,
                                        const float (&h)[NS]) const {
    float *q = p + (row * a.D + d) * a.N;
    if (!on) return;
#pragma unroll
    for (int j = 0; j < NS; j += 4) {
      if (a.n4) {
        if (j < a.N)
          *reinterpret_cast<float4 *>(q + j) = make_float4(h[j], h[j + 1], h[j + 2], h[j + 3]);
      } else {
#pragma unroll
        for (int i = j; i < j + 4; ++i)
          if (i < a.N) q[i] = h[i];
      }
    }
  }
};

// Copies a tile of one tensor's rows into shared memory, 16 bytes at a time.
template <typename E>
__device__ __forceinline__ void copy_tile(E (&to)[kL][kThreads], const void *base, int64_t st,
                                          const Wide &W, int tb, int t1) {
  constexpr int V = 16 / (int)sizeof(E), C = kThreads / V;  // elements a copy, copies a row
#pragma unroll
  for (int q = 0; q < kL * C / kThreads; ++q) {
    const int e = W.tid + q * kThreads, i = e / C, col = e % C * V;
    if (tb + i < t1 && col < W.nch)
      copy16(reinterpret_cast<uint4 *>(&to[i][col]),
             reinterpret_cast<const E *>(base) + (int64_t)(tb + i) * st + W.c0 + col);
  }
}

// The state's step: h <- e^{v A} h + dx B of one token.  The products are made in pairs, which
// saves issue slots; the sums are not: a paired multiply-add reads six registers and takes longer
// than two single ones.
template <int NS>
__device__ __forceinline__ void step(float (&h)[NS], const f2 (&A2)[NS / 2], const float *b,
                                     float v, float dx) {
  const f2 vv = pair(v, v), dd = pair(dx, dx);
#pragma unroll
  for (int j = 0; j < NS; j += 4) {
    const float4 B = *reinterpret_cast<const float4 *>(b + j);
    float e[4], u[4];
    unpair(mul2(vv, A2[j / 2]), e[0], e[1]);
    unpair(mul2(vv, A2[j / 2 + 1]), e[2], e[3]);
    unpair(mul2(dd, pair(B.x, B.y)), u[0], u[1]);
    unpair(mul2(dd, pair(B.z, B.w)), u[2], u[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[j + i] = fmaf(ex2(e[i]), h[j + i], u[i]);
  }
}

// A's rows times log2 e, in pairs.
template <int NS>
__device__ __forceinline__ void decay_pairs(const SsmArgs &a, const Wide &W, f2 (&A2)[NS / 2]) {
  float v[NS];
  W.read(a, a.A, 0, v);
#pragma unroll
  for (int j = 0; j < NS / 2; ++j) A2[j] = pair(v[2 * j] * kLog2e, v[2 * j + 1] * kLog2e);
}

template <typename E, int NS>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_ssm_wide_ends(const SsmArgs a, const Ranges rg, int tiles_per_group) {
  after_previous();
  constexpr int S = Stages<E>::S;
  extern __shared__ __align__(16) char smem_raw[];
  auto &s = *reinterpret_cast<Shared<E, NS, 2> *>(smem_raw);
  const Wide W(a, tiles_per_group);
  const int r0 = W.r * rg.range, t1 = min(a.T, r0 + rg.range);
  const E *Bp = reinterpret_cast<const E *>(a.B) + W.grp * a.B_sg;
  const float bias = a.dt_bias && W.on ? a.dt_bias[W.d] : 0.f;
  f2 A2[NS / 2];
  float h[NS], sum = 0.f;
  decay_pairs<NS>(a, W, A2);
  const SegCursor c = seg_find(a.cu, a.n_seq, a.T, t1, s.red);
  const int seg = c.j - 1;
  const bool covered = seg >= 0 && seg < a.n_seq, reset = seg >= 0 && c.b >= r0;
  const int t0 = reset ? c.b : r0;
  W.read(a, covered && reset ? a.h0 : nullptr, seg, h);
  if (covered) {
    BcTile<E, NS, kL, true> rb;
    auto issue = [&](int q, int tb) {
      copy_tile(s.in[q][0], a.x.p, a.x.st, W, tb, t1);
      copy_tile(s.in[q][1], a.dt.p, a.dt.st, W, tb, t1);
      copies_commit();
    };
#pragma unroll
    for (int q = 0; q < S - 1; ++q) issue(q, t0 + q * kL);
    rb.fetch(Bp, a.B_st, t0, t1, a.N);
    int stage = 0, buf = 0;
    for (int tb = t0; tb < t1; tb += kL, buf ^= 1) {
      rb.put(s.b[buf][0]);
      copies_wait<S - 2>();
      __syncthreads();  // the tile is there, and the one before it has been read
      issue(stage == 0 ? S - 1 : stage - 1, tb + (S - 1) * kL);
      if (tb + kL < t1) rb.fetch(Bp, a.B_st, tb + kL, t1, a.N);
      tile_tokens<kL>(0, min(kL, t1 - tb), [&](int i) {
        const float x = ld1(&s.in[stage][0][i][W.tid]);
        float v = ld1(&s.in[stage][1][i][W.tid]) + bias;
        if (a.softplus) v = softplusf(v);
        sum += v;
        step<NS>(h, A2, s.b[buf][i], v, v * x);
      });
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    copies_wait<0>();
  }
  W.write(a, rg.state, W.r, h);
  if (W.on) rg.sum[(int64_t)W.r * a.D + W.d] = sum;
  if (blockIdx.x % (tiles_per_group * a.G) == 0 && W.tid == 0) rg.reset[W.r] = reset;
}

template <typename E, int NS>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_ssm_wide(const SsmArgs a, const Ranges rg, int tiles_per_group) {
  after_previous();
  constexpr int S = Stages<E>::S;
  extern __shared__ __align__(16) char smem_raw[];
  auto &s = *reinterpret_cast<Shared<E, NS, 3> *>(smem_raw);
  const Wide W(a, tiles_per_group);
  if (W.r == rg.n) {  // final states of the segments without tokens
    for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
      const int64_t at = ((int64_t)n * a.D + W.c0) * a.N;
      for (int i = W.tid; i < W.nch * a.N; i += kThreads) a.ht[at + i] = a.h0 ? a.h0[at + i] : 0.f;
    });
    return;
  }
  const int t0 = W.r * rg.range, t1 = min(a.T, t0 + rg.range);
  const E *Bp = reinterpret_cast<const E *>(a.B) + W.grp * a.B_sg;
  const E *Cp = reinterpret_cast<const E *>(a.C) + W.grp * a.C_sg;
  const bool gated = a.z.p != nullptr;
  BcTile<E, NS, kL, true> rb, rc;
  auto issue = [&](int q, int tb) {
    copy_tile(s.in[q][0], a.x.p, a.x.st, W, tb, t1);
    copy_tile(s.in[q][1], a.dt.p, a.dt.st, W, tb, t1);
    if (gated) copy_tile(s.in[q][2], a.z.p, a.z.st, W, tb, t1);
    copies_commit();
  };
#pragma unroll
  for (int q = 0; q < S - 1; ++q) issue(q, t0 + q * kL);
  rb.fetch(Bp, a.B_st, t0, t1, a.N);
  rc.fetch(Cp, a.C_st, t0, t1, a.N);
  const float bias = a.dt_bias && W.on ? a.dt_bias[W.d] : 0.f;
  const float skip = a.Dskip && W.on ? a.Dskip[W.d] : 0.f;
  f2 A2[NS / 2];
  float h[NS];
  decay_pairs<NS>(a, W, A2);
#pragma unroll
  for (int j = 0; j < NS; ++j) h[j] = 0.f;
  SegCursor cursor = seg_find(a.cu, a.n_seq, a.T, t0, s.red);
  int seg = cursor.j - 1;
  if (seg >= 0 && seg < a.n_seq) {
#pragma unroll 2
    for (int q = 0; q < W.r; ++q) {  // the state that enters this range
      float end[NS];
      W.read(a, rg.state, q, end);
      const float sum = W.on ? rg.sum[(int64_t)q * a.D + W.d] : 0.f;
      const bool reset = rg.reset[q] != 0;
#pragma unroll
      for (int j = 0; j < NS; j += 2) {
        float u, v;
        unpair(A2[j / 2], u, v);
        h[j] = reset ? end[j] : fmaf(ex2(u * sum), h[j], end[j]);
        h[j + 1] = reset ? end[j + 1] : fmaf(ex2(v * sum), h[j + 1], end[j + 1]);
      }
    }
  }
  if (W.tid < 32) {
    const bool any = seg_marks(a.cu, a.n_seq, a.T, t0, min(kL, t1 - t0), s.mark[0], cursor);
    if (W.tid == 0) s.any[0] = any;
  }
  E *y = reinterpret_cast<E *>(a.y.p) + W.d;
  int stage = 0, buf = 0;
  for (int tb = t0; tb < t1; tb += kL, buf ^= 1) {
    const int n = min(kL, t1 - tb);
    rb.put(s.b[buf][0]);
    rc.put(s.c[buf][0]);
    copies_wait<S - 2>();
    __syncthreads();  // the tile and its marks are there, and the one before it has been read
    issue(stage == 0 ? S - 1 : stage - 1, tb + (S - 1) * kL);
    if (tb + kL < t1) {
      rb.fetch(Bp, a.B_st, tb + kL, t1, a.N);
      rc.fetch(Cp, a.C_st, tb + kL, t1, a.N);
      if (W.tid < 32) {
        const bool any = seg_marks(a.cu, a.n_seq, a.T, tb + kL, min(kL, t1 - tb - kL),
                                   s.mark[buf ^ 1], cursor);
        if (W.tid == 0) s.any[buf ^ 1] = any;
      }
    }
    auto scan = [&](int i0, int i1) {
      tile_tokens<kL>(i0, i1, [&](int i) {
        const float x = ld1(&s.in[stage][0][i][W.tid]);
        float v = ld1(&s.in[stage][1][i][W.tid]) + bias;
        if (a.softplus) v = softplusf(v);
        step<NS>(h, A2, s.b[buf][i], v, v * x);
        float p[4];
#pragma unroll
        for (int j = 0; j < NS; j += 4) {
          const float4 C = *reinterpret_cast<const float4 *>(&s.c[buf][i][j]);
          p[0] = j ? fmaf(h[j], C.x, p[0]) : h[j] * C.x;
          p[1] = j ? fmaf(h[j + 1], C.y, p[1]) : h[j + 1] * C.y;
          p[2] = j ? fmaf(h[j + 2], C.z, p[2]) : h[j + 2] * C.z;
          p[3] = j ? fmaf(h[j + 3], C.w, p[3]) : h[j + 3] * C.w;
        }
        float o = fmaf(skip, x, (p[0] + p[1]) + (p[2] + p[3]));
        if (gated) {
          const float z = ld1(&s.in[stage][2][i][W.tid]);
          o *= z * sigmoidf(z);
        }
        if (W.on) st1(y + (int64_t)(tb + i) * a.y.st, o);
      });
    };
    if (!s.any[buf]) {
      if (seg >= 0 && seg < a.n_seq) scan(0, n);
    } else {
      const int *mark = s.mark[buf];
#pragma unroll 1
      for (int i = 0; i < n;) {
        if (mark[i] >= 0) {
          seg = mark[i];
          W.read(a, seg < a.n_seq ? a.h0 : nullptr, seg, h);
        }
        int e = i + 1;
        while (e < n && mark[e] < 0) ++e;
        if (seg >= 0 && seg < a.n_seq) {
          scan(i, e);
          if (a.ht && mark[e] >= 0) W.write(a, a.ht, seg, h);
        }
        i = e;
      }
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }
}

template <typename E, int NS>
cudaError_t run_wide(const SsmArgs &a, int range, cudaStream_t stream) {
  const int tpg = (int)ceil_div64(a.D / a.G, kThreads), ctiles = tpg * a.G;
  const Ranges rg = carve_ranges(a.work, a.T, a.D, a.N, range).rg;
  constexpr int smem1 = (int)sizeof(Shared<E, NS, 2>), smem2 = (int)sizeof(Shared<E, NS, 3>);
  cudaError_t e;
  if (smem1 > 48 * 1024 && (e = allow_smem(k_ssm_wide_ends<E, NS>, smem1)) != cudaSuccess) return e;
  if (smem2 > 48 * 1024 && (e = allow_smem(k_ssm_wide<E, NS>, smem2)) != cudaSuccess) return e;
  if (rg.n > 1) {
    if ((e = launch(k_ssm_wide_ends<E, NS>, (unsigned)((int64_t)ctiles * (rg.n - 1)), kThreads,
                    smem1, stream, a, rg, tpg)) != cudaSuccess)
      return e;
  }
  return launch(k_ssm_wide<E, NS>, (unsigned)((int64_t)ctiles * (rg.n + (a.ht ? 1 : 0))), kThreads,
                smem2, stream, a, rg, tpg);
}

}  // namespace

int wide_range(int64_t T, int32_t D, int32_t N, int32_t G, bool f32) {
  if (N > 16) return 0;
  const int64_t ctiles = G * ceil_div64(D / G, kThreads), room = (int64_t)sm_count() * kCtas;
  // enough work, 16 tiles of tokens for each block that could run, and the channels of a group fill
  // at least 3 in 4 lanes.  Lanes / this layout in us, 16 states in bf16: 2,437 x 4,096 (8 tiles)
  // 103 / 102, 4,869 (16) 196 / 181, 20,373 (67) 788 / 679; 8 states 133 / 125 with 16 tiles
  if (T * ctiles < room * 16 * kL || (int64_t)D * 4 < ctiles * kThreads * 3) return 0;
  int64_t n = room / ctiles;
  if (n > kMost) {
    n = kMost;
    // few channels: kMost ranges of them do not fill the GPU, however long the prompt.  bf16 with
    // 67 tiles: 2,304 channels (95 % of the blocks) 792 / 714, 2,048 (84 %) 754 / 800, 1,024 (42 %)
    // 756 / 1,022, 512 (21 %) 761 / 1,672.  fp32, whose rings leave the lanes fewer blocks an SM:
    // 2,048 1,251 / 806, 1,024 1,250 / 1,030, 512 1,196 / 1,710
    if (n * ctiles * 10 < room * (f32 ? 4 : 9)) return 0;
  }
  if (n < 1) n = 1;
  return (int)(ceil_div64(ceil_div64(T, n), kL) * kL);
}

cudaError_t launch_wide(const SsmArgs &a, int range, cudaStream_t stream) {
  if (a.f32)
    return a.N <= 8 ? run_wide<float, 8>(a, range, stream) : run_wide<float, 16>(a, range, stream);
  return a.N <= 8 ? run_wide<__nv_bfloat16, 8>(a, range, stream)
                  : run_wide<__nv_bfloat16, 16>(a, range, stream);
}

}  // namespace ssm
}  // namespace gdr
