// gdr_ssm.cuh -- the thread layout that the selective state space kernels share.
//
// A block of 128 threads owns CH = 256 / LN channels of one group.  LN neighbouring lanes share a
// channel and hold 4 states each (LN = 4 for up to 16 states); a thread holds two channels, so
// that a token's B and C, read from shared memory, serve 8 states.
#pragma once

#include <string.h>

#include <type_traits>

#include "gdr_mix.cuh"

namespace gdr {
namespace ssm {

constexpr int kThreads = 128;

// e^{dt A}, A2 = A log2 e (or dt's product with it, and A).  The approximate exponential falls
// short: by 2e-8 of its value on average for exponents between -0.5 and -0.004, by 6e-9 for smaller
// ones (measured).  Over a state's tokens that adds up, most of all in dA, whose terms weigh by the
// time that states last (at 4,067 tokens of 512 x 16 states 9.7e-7 of dA's norm; 4.8e-7 with the
// middle of the two added to the exponent).  A state that must last is kept exactly: with dt = 0
// (the tokens behind a short tile's last, too) or A = 0 the exponent is 0, for which the instruction
// promises 1.  So what is added is no more than |dt| (of either of a thread's two channels: one
// minimum of three instead of two of two; 8,192 x 2,048 x 16, forward and backward: 806 us without,
// 820 and 827), and nothing by a thread that holds a state with A = 0.
constexpr float kShort = 1.9e-8f;  // 1.3e-8 / ln 2
__device__ __forceinline__ float raised(float dt, float most) { return fminf(fabsf(dt), most); }
__device__ __forceinline__ float raised(const float (&dt)[2], float most) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(dt[0])), "f"(fabsf(dt[1])), "f"(most));
  return r;
}
__device__ __forceinline__ float decay(float dt, float A2, float more) {
  return mix::ex2(fmaf(dt, A2, more));
}

template <int LN>
struct Lay {
  static constexpr int NP = 4 * LN;      // states, padded
  static constexpr int CW = 32 / LN;     // channels of a warp, for each of a thread's two
  static constexpr int CH = 256 / LN;    // channels of a block
  static constexpr int L = 4 * LN;       // tokens of a tile: 8 elements of x for each thread
  static constexpr int CG = CH / 8;      // groups of 8 channels

  // channel k (0, 1) of a thread, in the block
  static __device__ __forceinline__ int channel(int warp, int lane, int k) {
    return warp * 2 * CW + k * CW + lane / LN;
  }
  // A token's pairs (two floats for each channel) in shared memory, in float2: a thread's two
  // channels are neighbours, one 16-byte load.  Two more pairs behind each warp's channels spread
  // the stores of a thread's 8 neighbouring channels, and the next token's, over the banks.
  static constexpr int PW = 2 * CW + 2, PT = 4 * PW;
  static __device__ __forceinline__ int pair_at(int t, int ch) {
    return t * PT + ch / (2 * CW) * PW + ch % CW * 2 + (ch / CW & 1);
  }
  // A token's LN partial sums of each channel, in floats: one more place behind every 8 channels
  // spreads the reads of a thread's 8 channels.
  static constexpr int ST = (CH + CG) * LN;
  static __device__ __forceinline__ int part_at(int t, int ch) {
    return t * ST + (ch + (ch >> 3)) * LN;
  }
};

// A block's range and channels, a thread's channels and states (4 nl .. 4 nl + 3 of both).
template <int LN>
struct Place {
  using Y = Lay<LN>;
  int tid, warp, lane, nl, cl, ct, r, grp, c0, nch;
  int ch[2];
  int pair;  // where this thread's pairs are in a token's row
  __device__ __forceinline__ Place(const SsmArgs &a, int tiles_per_group) {
    tid = threadIdx.x;
    warp = tid >> 5;
    lane = tid & 31;
    nl = lane % LN;
    cl = lane / LN;
    const int ctiles = tiles_per_group * a.G, Dg = a.D / a.G;
    ct = blockIdx.x % ctiles;
    r = blockIdx.x / ctiles;
    grp = ct / tiles_per_group;
    c0 = grp * Dg + ct % tiles_per_group * Y::CH;
    nch = min(Y::CH, (grp + 1) * Dg - c0);
    ch[0] = Y::channel(warp, lane, 0);
    ch[1] = Y::channel(warp, lane, 1);
    pair = Y::pair_at(0, ch[0]);
  }
  // h = the states of this row of p [rows, D, N], zeros where p is null; and back
  __device__ __forceinline__ void read(const SsmArgs &a, const float *p, int64_t row,
                                       float (&h)[2][4]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float *q = p + ((row * a.D + c0 + ch[k]) * a.N + nl * 4);
      const bool in = p && ch[k] < nch;
      if (a.n4) {
        const float4 v = in && nl * 4 < a.N ? *reinterpret_cast<const float4 *>(q)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
        h[k][0] = v.x;
        h[k][1] = v.y;
        h[k][2] = v.z;
        h[k][3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] = in && nl * 4 + j < a.N ? q[j] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void write(const SsmArgs &a, float *p, int64_t row,
                                        const float (&h)[2][4]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float *q = p + ((row * a.D + c0 + ch[k]) * a.N + nl * 4);
      if (ch[k] >= nch) continue;
      if (a.n4) {
        if (nl * 4 < a.N)
          *reinterpret_cast<float4 *>(q) = make_float4(h[k][0], h[k][1], h[k][2], h[k][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (nl * 4 + j < a.N) q[j] = h[k][j];
      }
    }
  }
  // A2 = A log2 e; returns what decay's exponents may be raised by
  __device__ __forceinline__ float decays(const SsmArgs &a, float (&A2)[2][4]) const {
    read(a, a.A, 0, A2);
    float most = kShort;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A2[k][j] *= mix::kLog2e;
        if (A2[k][j] == 0.f && ch[k] < nch && nl * 4 + j < a.N) most = 0.f;
      }
    return most;
  }
};

template <int LN>
__device__ __forceinline__ float sum_parts(const float *p) {
  if constexpr (LN == 2) {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    return v.x + v.y;
  } else {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < LN; i += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(p + i);
      s += (v.x + v.y) + (v.z + v.w);
    }
    return s;
  }
}

// A tile of B (or C) in shared memory as fp32, padded to NP states; read from global memory one
// tile ahead, two elements at a time (VEC: N and the strides are even, addresses aligned).
template <typename E, int NP, int L, bool VEC>
struct BcTile {
  static constexpr int M = (L * NP / 2 + kThreads - 1) / kThreads;
  using Two = typename std::conditional<sizeof(E) == 2, uint32_t, uint2>::type;
  Two v[M];
  __device__ __forceinline__ void fetch(const E *p, int64_t st, int tb, int t1, int N) {
#pragma unroll
    for (int q = 0; q < M; ++q) {
      const int e = (threadIdx.x + q * kThreads) * 2, t = tb + e / NP, n = e % NP;
      const bool row = e < L * NP && t < t1;
      v[q] = Two{};
      if (VEC) {
        if (row && n < N) v[q] = *reinterpret_cast<const Two *>(p + t * st + n);
      } else {
        E w[2] = {E(0.f), E(0.f)};
        if (row && n < N) w[0] = p[t * st + n];
        if (row && n + 1 < N) w[1] = p[t * st + n + 1];
        memcpy(&v[q], w, sizeof(Two));
      }
    }
  }
  __device__ __forceinline__ void put(float *s) const {
#pragma unroll
    for (int q = 0; q < M; ++q) {
      const int e = (threadIdx.x + q * kThreads) * 2;
      if (e < L * NP) *reinterpret_cast<float2 *>(s + e) = both(v[q]);
    }
  }
  static __device__ __forceinline__ float2 both(uint32_t u) {
    return make_float2(mix::lo_bf(u), mix::hi_bf(u));
  }
  static __device__ __forceinline__ float2 both(uint2 u) {
    return make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
};

// A thread's 8 elements of each tile of x (dt, z, dout) on their way into shared memory, S tiles
// in a ring in which each thread reads only what it copied itself: they take no registers while
// they wait.  Elements that were not copied read as anything (no token) or as 0 (no channel).
// Without 16-byte alignment they wait in registers, one tile ahead.  issue is called for each tile
// in turn, S - 1 tiles before its get.
template <typename E, bool VEC, int S_>
struct TileRing {
  static constexpr int S = VEC ? S_ : 2, P = (int)sizeof(E) / 2;
  static constexpr int kSlots = VEC ? S * P * kThreads : 0;
  uint4 *ring;
  const E *p;
  int64_t st;
  mix::Raw8<E> now, next;

  __device__ __forceinline__ TileRing(uint4 *ring_, const void *base, int64_t at, int64_t st_,
                                      int nv)
      : ring(ring_), p(reinterpret_cast<const E *>(base) + at), st(st_) {
    if (!VEC) {
      now = next = mix::zero8<E>();
    } else if (nv == 0) {
      for (int i = 0; i < S * P; ++i) ring[i * kThreads + threadIdx.x] = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void issue(int s, int t, int n) {
    if (VEC) {
      if (n > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i)
          mix::copy16(ring + (s * P + i) * kThreads + threadIdx.x, p + t * st + i * 4);
      }
    } else {
      now = next;
      next = mix::ld8<false>(p + t * st, n);
    }
  }
  __device__ __forceinline__ mix::Raw8<E> get(int s) const {
    if (!VEC) return now;
    mix::Raw8<E> r;
    uint4 *w = reinterpret_cast<uint4 *>(&r);
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = ring[(s * P + i) * kThreads + threadIdx.x];
    return r;
  }
};

// What a step's raw size is raised by; 1 where the block has no channel, whose step must not be 0
// for the sake of the channel that shares its threads (raised).
__device__ __forceinline__ float step_bias(const float *dt_bias, int c0, int nch, int i) {
  return i >= nch ? 1.f : dt_bias ? dt_bias[c0 + i] : 0.f;
}

// (dt, dt x) of a thread's 8 elements of a tile.
template <typename E, int LN>
__device__ __forceinline__ void put_pairs(float2 *pair, const float *bias, int softplus, int lt,
                                          int lc, const mix::Raw8<E> &rx, const mix::Raw8<E> &rd) {
  float x[8], d[8];
  mix::unpack8(rx, x);
  mix::unpack8(rd, d);
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 b = *reinterpret_cast<const float4 *>(bias + lc + i);
    d[i] += b.x;
    d[i + 1] += b.y;
    d[i + 2] += b.z;
    d[i + 3] += b.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = softplus ? mix::softplusf(d[i]) : d[i];
    pair[Lay<LN>::pair_at(lt, lc) + Lay<LN>::pair_at(0, i)] = make_float2(v, v * x[i]);
  }
}

// Calls f(i) for tokens [i0, i1) of a tile; a whole tile is unrolled, so that its addresses are
// constants.
template <int L, typename F>
__device__ __forceinline__ void tile_tokens(int i0, int i1, F f) {
  constexpr int U = L < 16 ? L : 16;
  if (i1 - i0 == L) {
#pragma unroll 1
    for (int i = 0; i < L; i += U)
#pragma unroll
      for (int u = 0; u < U; ++u) f(i + u);
  } else {
#pragma unroll 2
    for (int i = i0; i < i1; ++i) f(i);
  }
}

// Rows that may be read 16 bytes at a time, and B and C two elements at a time.
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool rows_ok(const Mat &m, bool f32) {
  return !m.p || (aligned16(m.p) && m.st % (f32 ? 4 : 8) == 0);
}

inline bool bc_ok(const SsmArgs &a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C);
  return a.N % 2 == 0 && a.B_st % 2 == 0 && a.B_sg % 2 == 0 && a.C_st % 2 == 0 &&
         a.C_sg % 2 == 0 && (at & (a.f32 ? 7 : 3)) == 0;
}

inline bool states_ok(const SsmArgs &a) {
  return a.N % 4 == 0 && aligned16(a.A) && aligned16(a.h0) && aligned16(a.ht) &&
         aligned16(a.dht) && aligned16(a.dh0);
}

inline int lanes_for(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

// Replaces val[r] of state i, the end of range r from a zero state, by the state that enters the
// range; with `back` the same for gradients, from the last range to the first.  A warp is alone on
// its scheduler here and its instructions follow one another slowly: pointers that step from
// range to range keep them few.
__device__ __forceinline__ void chain_ranges(float *val, const float *sum, const int *reset, int n,
                                             int D, int64_t size, int64_t i, int d, float A2,
                                             bool back) {
  const int64_t first = back ? n - 1 : 0;
  val += first * size + i;
  sum += first * D + d;
  reset += first;
  if (back) size = -size;
  const int64_t dstep = back ? -(int64_t)D : D;
  const int step = back ? -1 : 1;
  float cur = 0.f;
  auto batch = [&](auto U) {
    float own[U.value], s[U.value];
    int rs[U.value];
    float *v = val;
#pragma unroll
    for (int u = 0; u < U.value; ++u) {
      own[u] = *v;
      s[u] = *sum;
      rs[u] = *reset;
      v += size;
      sum += dstep;
      reset += step;
    }
#pragma unroll
    for (int u = 0; u < U.value; ++u) {
      *val = cur;
      cur = rs[u] ? own[u] : fmaf(mix::ex2(A2 * s[u]), cur, own[u]);
      val += size;
    }
  };
  int k = 0;
  for (; k + 16 < n; k += 16) batch(std::integral_constant<int, 16>());
  for (; k + 4 < n; k += 4) batch(std::integral_constant<int, 4>());
  for (; k + 1 < n; ++k) batch(std::integral_constant<int, 1>());
  *val = cur;  // the last range's end goes nowhere
}

constexpr int kChainRanges = 16;  // more ranges than this are chained by a kernel of its own

// The ranges of the forward's scan, and what pass 1 leaves of each.
struct Ranges {
  int range, n;      // tokens of a range, ranges
  float *state;      // [n][D][N]: the state at the end, from a zero state at the start
  float *sum;        // [n][D]: sum of dt from the last segment start in the range (or its start)
  int *reset;        // [n]: a segment starts in the range
};

struct Carve {
  Ranges rg;
  size_t bytes;
};
inline Carve carve_ranges(void *work, int64_t T, int32_t D, int32_t N, int range) {
  Carve c{};
  c.rg.range = range;
  c.rg.n = (int)ceil_div64(T, range);
  if (c.rg.n <= 1) return c;
  char *p = reinterpret_cast<char *>(work);
  c.rg.state = reinterpret_cast<float *>(p);
  size_t off = align256((size_t)c.rg.n * D * N * sizeof(float));
  c.rg.sum = reinterpret_cast<float *>(p + off);
  off += align256((size_t)c.rg.n * D * sizeof(float));
  c.rg.reset = reinterpret_cast<int *>(p + off);
  off += align256((size_t)c.rg.n * sizeof(int));
  c.bytes = off;
  return c;
}

template <typename K>
cudaError_t allow_smem(K k, int bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// The layout of one thread a channel (gdr_ssm_wide.cu): its tokens of a range where it is worth
// while (aligned rows), else 0.
int wide_range(int64_t T, int32_t D, int32_t N, int32_t G, bool f32);
cudaError_t launch_wide(const SsmArgs &a, int range, cudaStream_t stream);

inline int64_t channel_tiles(int D, int G, int LN) {
  return (int64_t)G * ceil_div64(D / G, 256 / LN);
}

}  // namespace ssm
}  // namespace gdr
