// gdr_rec.cuh -- what the gated linear recurrence's forward and backward share: products of a token, pairs
// (A, U), the layout of lanes, rows on their way, and the chain of a cluster's blocks.
//
// A lane holds two channels of kK neighbouring tokens.  A warp's lanes lie in SUB groups over one row of
// 64 / SUB channels, each with the kK tokens behind the group's before: few channels then still fill the
// GPU's blocks, which share the channels among clusters and the tokens inside one.
#pragma once

#include <initializer_list>

#include "gdr_block.cuh"
#include "gdr_cluster.cuh"

namespace gdr {
namespace mix {
namespace {

// Nonzero once a wait for another block of a cluster ran out; read by gdr_device_status.
__device__ int32_t g_rec_status = 0;
constexpr uint64_t kRecWaitNs = 2000000000ull;  // 2 s, once a block

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

__device__ __forceinline__ f2 both(float v) { return pair(v, v); }
// sqrt(x) on the special-function unit (2^-23; NaN below 0)
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename E>
__device__ __forceinline__ f2 wide(const Raw2<E> &r) {
  return pair(r.lo(), r.hi());
}

// a = 2^L2 and 1 - a^2.  Next to a = 1, above it too, both come from the series of d = 1 - a (the first term
// left out is 1e-9 of it at the border, |ln a| = 1/16): the special-function unit's 2^x falls short by 2e-8 on
// average, which a state that lasts for hundreds of tokens adds up, and 1 - a^2 would lose its
// relative accuracy (8,192 x 2,560: error of dA 6.2e-6 of its norm without the series for a).  Nothing
// is added to a state with A = 0, and nothing taken from it: d = 0.
__device__ __forceinline__ f2 short_of_one(f2 L2) {
  f2 p = fma2(L2, both(-0.0013333558f), both(-0.0096181291f));
  p = fma2(p, L2, both(-0.055504109f));
  p = fma2(p, L2, both(-0.24022651f));
  p = fma2(p, L2, both(-0.69314718f));
  return mul2(p, L2);
}
constexpr float kNear = 0.09016844f;  // |L2| below: the series
__device__ __forceinline__ f2 decay_of(f2 L2) {
  const f2 near = fma2(short_of_one(L2), both(-1.f), both(1.f));
  float l0, l1, n0, n1;
  unpair(L2, l0, l1);
  unpair(near, n0, n1);
  return pair(fabsf(l0) < kNear ? n0 : ex2(l0), fabsf(l1) < kNear ? n1 : ex2(l1));
}

struct Token {
  f2 sr, a, m;
};
// A2: A log2 e; sr: sigmoid(r).  m is NaN for a > 1 (A > 0).
template <bool NORM>
__device__ __forceinline__ Token token(f2 sr, f2 A2) {
  Token t;
  t.sr = sr;
  const f2 L2 = mul2(A2, sr), d = short_of_one(L2), near = fma2(d, both(-1.f), both(1.f));
  float l0, l1, n0, n1, a0, a1;
  unpair(L2, l0, l1);
  unpair(near, n0, n1);
  a0 = fabsf(l0) < kNear ? n0 : ex2(l0);
  a1 = fabsf(l1) < kNear ? n1 : ex2(l1);
  t.a = pair(a0, a1);
  t.m = both(1.f);
  if (NORM) {
    float s0, s1;
    unpair(mul2(d, add2(near, both(1.f))), s0, s1);
    t.m = pair(sqrt_approx(fabsf(l0) < kNear ? s0 : fmaf(-a0, a0, 1.f)),
               sqrt_approx(fabsf(l1) < kNear ? s1 : fmaf(-a1, a1, 1.f)));
  }
  return t;
}
// Two sigmoids for one reciprocal, which is twice an exponential's time: 1 / (1 + e) (1 + f) times the other
// factor.  q: the reciprocals; 0 where the product overflowed (both far below 0), and the two have to be
// computed on their own.
__device__ __forceinline__ void sigmoids(f2 r, f2 i, f2 &sr, f2 &si, float &q) {
  float a, b, c, d;
  unpair(mul2(r, both(-kLog2e)), a, b);
  unpair(mul2(i, both(-kLog2e)), c, d);
  const f2 e = add2(pair(ex2(a), ex2(b)), both(1.f)), f = add2(pair(ex2(c), ex2(d)), both(1.f));
  unpair(mul2(e, f), a, b);
  a = rcp(a);
  b = rcp(b);
  q = fminf(a, b);
  sr = mul2(pair(a, b), f);
  si = mul2(pair(a, b), e);
}
// The same for every value, to the bit where the reciprocals are not 0: a token's results do not depend on
// which of the two its warp takes, nor so on the tokens of other sequences beside it or on what is left in
// places that no token was copied to.
__device__ __forceinline__ void sigmoids_apart(f2 r, f2 i, f2 &sr, f2 &si) {
  float q;
  sigmoids(r, i, sr, si, q);
  if (q == 0.f) {
    sr = sigmoid2(r);
    si = sigmoid2(i);
  }
}

// ------------------------------------------------------------------ pairs (A, U): h -> A h + U
//
// A = -0 says that the pair holds a segment's start: what comes before it is not looked at, be it
// infinite or NaN.  Decays are never negative, so that no product of them is -0 but one with such a
// pair in it.  A product that underflowed to +0 is a product like any other: an infinity or NaN in
// front of it is still one behind it (0 times it is NaN).

struct Map {
  f2 A, U;
};
__device__ __forceinline__ f2 pick(bool lo, bool hi, f2 yes, f2 no) {
  float a, b, c, d;
  unpair(yes, a, b);
  unpair(no, c, d);
  return pair(lo ? a : c, hi ? b : d);
}
__device__ __forceinline__ f2 start_mark() { return both(-0.f); }
__device__ __forceinline__ bool is_start(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ f2 through(Map f, f2 h) {
  float lo, hi;
  unpair(f.A, lo, hi);
  return pick(is_start(lo), is_start(hi), f.U, fma2(f.A, h, f.U));
}
// first f, then g
__device__ __forceinline__ Map then(Map f, Map g) {
  float f0, f1, g0, g1;
  unpair(f.A, f0, f1);
  unpair(g.A, g0, g1);
  return Map{pick(is_start(f0) || is_start(g0), is_start(f1) || is_start(g1), start_mark(), mul2(f.A, g.A)),
             through(g, f.U)};
}
// the same where neither holds a segment's start
__device__ __forceinline__ Map then_inside(Map f, Map g) {
  return Map{mul2(f.A, g.A), fma2(g.A, f.U, g.U)};
}
__device__ __forceinline__ float4 packed(Map f) {
  float4 v;
  unpair(f.A, v.x, v.y);
  unpair(f.U, v.z, v.w);
  return v;
}
__device__ __forceinline__ Map unpacked(float4 v) { return Map{pair(v.x, v.y), pair(v.z, v.w)}; }

// ------------------------------------------------------------------ to the cluster's blocks

// *p of the block of this rank = v, before the next barrier of the cluster
__device__ __forceinline__ void put(float4 *p, int rank, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at_rank(p, rank)), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
// the same, counted as 16 bytes by that block's *bar
__device__ __forceinline__ void send(float4 *p, uint64_t *bar, int rank, float4 v) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          at_rank(p, rank)),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(at_rank(bar, rank))
      : "memory");
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

// ------------------------------------------------------------------ a warp's tokens

constexpr int kP = 8, kK = 8;  // warps of a block, tokens of a thread
constexpr int kHold = kP - 1;             // warps with tokens
constexpr int kMostSub = 4;
constexpr int channels_of(int sub) { return 64 / sub; }     // of a block
constexpr int tile_of(int sub) { return kHold * kK * sub; }  // tokens of a block
static_assert(kRecEvery == kK, "a kept state for each thread's tokens");

// Of a block's eight warps seven hold tokens and one chains their maps.  The holders compute the maps of
// step s + 1 while the chain of step s is on its way through the cluster, and then run through step
// s: nobody waits for a map that was sent just now.  Places are written again when a later meeting
// has shown that they were read: maps and states two steps on, bounds (looked up two steps ahead) four.
template <int SUB>
struct Shared {
  float4 warp[2][kHold][32 / SUB];     // (A, U) of both channels, for each warp with tokens
  float4 block[2][kMostCl][32 / SUB];  // and for each block of the cluster
  f2 front[2][kHold][32 / SUB];        // the state in front of each warp's tokens
  uint64_t bar[2];                     // every block's map is here
  int mark[4][tile_of(SUB) + 1];
  int any[4], alive[4];
  int red[64];
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      tc::mbar_init(&bar[0], 1);
      tc::mbar_init(&bar[1], 1);
      tc::fence_mbar_init();
    }
  }
};

// Meetings of holders and chain, two of each kind in turn.
__device__ __forceinline__ void arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(kP * 32) : "memory");
}
__device__ __forceinline__ void meet(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(kP * 32) : "memory");
}
constexpr int kMaps = 1, kFronts = 3;

// A lane's group and its place in it (what a warp of one group knows when it is compiled).
template <int SUB>
__device__ __forceinline__ int group_of(int lane) {
  return SUB == 1 ? 0 : lane / (32 / SUB);
}
template <int SUB>
__device__ __forceinline__ int place_of(int lane) {
  return SUB == 1 ? lane : lane % (32 / SUB);
}

// The N tensors of a step on their way into shared memory, into one of S places of a warp's own, a step
// ahead.  MODE 2: rows come 16 bytes at a time; 1: each lane's two channels, for rows that fit no better;
// 0 (rows at any address): they are loaded when they are used.
template <typename E, int MODE, int N, int S, int SUB>
struct Tokens {
  static constexpr int kLanes = 32 / SUB;                      // of a row
  static constexpr int kRow = channels_of(SUB) * (int)sizeof(E);  // bytes
  static constexpr int kRows = kK * SUB;                       // of a warp's step
  static constexpr int kGap = SUB > 1 ? kK + 1 : kK;           // rows of a group: one spare spreads the banks
  static constexpr int kPlace = N * SUB * kGap * kRow;
  static constexpr int kBytes = MODE ? S * kHold * kPlace : 0;  // of a block
  static constexpr int kL = kRow / 16, kR = 32 / kL;           // lanes of a row and rows, 16 bytes a lane
  const E *p[N];  // at this block's first channel; null: not there
  int64_t st[N];
  unsigned char *mine;  // this warp's places
  int lane, cols, nv, T;
  const E *from[N];  // what this lane copies first of the next step

  // rows from token t on are the first to come, then those `step` tokens on each time
  __device__ __forceinline__ void start(int t) {
    if (MODE == 0) return;
#pragma unroll
    for (int n = 0; n < N; ++n)
      from[n] = MODE == 2 ? p[n] + (int64_t)(t + lane / kL) * st[n] + lane % kL * (16 / (int)sizeof(E))
                          : p[n] + (int64_t)(t + group_of<SUB>(lane) * kK) * st[n] + place_of<SUB>(lane) * 2;
  }
  __device__ __forceinline__ unsigned char *at(int place, int n, int k) const {
    return mine + place * kPlace + (n * SUB * kGap + group_of<SUB>(lane) * kGap + k) * kRow +
           place_of<SUB>(lane) * 2 * (int)sizeof(E);
  }
  __device__ __forceinline__ void issue(int place, int t, int step) {
    if (MODE == 0) return;
    __syncwarp();  // the place was read by all lanes
    if (MODE == 2) {
      const int r0 = lane / kL;
      const int left = lane % kL * (16 / (int)sizeof(E)) < cols ? T - t - r0 : 0;
      unsigned char *to = mine + place * kPlace + (r0 + (SUB > 1 ? r0 / kK : 0)) * kRow + lane % kL * 16;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n == 2 && !p[n]) continue;
        const E *q = from[n];
#pragma unroll
        for (int r = 0; r < kRows; r += kR) {
          constexpr int kSpare = SUB > 1 ? kK : 1 << 20;
          if (r < left)
            copy16(reinterpret_cast<uint4 *>(to + (n * SUB * kGap + r + r / kSpare) * kRow), q);
          q += kR * st[n];
        }
        from[n] += step * st[n];
      }
    } else {
      const int left = nv > 0 ? T - t - group_of<SUB>(lane) * kK : 0;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n == 2 && !p[n]) continue;
        const E *q = from[n];
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          if (k < left) {
            if (sizeof(E) == 2) copy4(at(place, n, k), q);
            else copy8(at(place, n, k), q);
          }
          q += st[n];
        }
        from[n] += step * st[n];
      }
    }
    copies_commit();
  }
  __device__ __forceinline__ void wait() const {
    if (MODE) {
      copies_wait<1>();
      __syncwarp();
    }
  }
  // the lane's two channels of its k-th token, which is t
  __device__ __forceinline__ f2 get(int place, int n, int k, int t) const {
    if (MODE) return wide(*reinterpret_cast<const Raw2<E> *>(at(place, n, k)));
    return wide(ld2<false>(p[n] + (int64_t)t * st[n] + place_of<SUB>(lane) * 2, t < T ? nv : 0));
  }
};

// Bit k: a segment starts with the lane's token k (of n), of which `left` are there.
template <int SUB>
__device__ __forceinline__ uint32_t starts_of(const int *mark, int left, int n) {
  if (SUB == 1) {
    const int k = threadIdx.x & 31;
    return __ballot_sync(0xffffffffu, k < n && k <= left && left > 0 && mark[min(k, max(left, 0))] >= 0);
  }
  uint32_t bits = 0;
#pragma unroll 1
  for (int k = 0; k < n; ++k)
    if (left > 0 && k <= left && mark[k] >= 0) bits |= 1u << k;
  return bits;
}
// The segment of the lane's token k, from what starts among its tokens and that of the first.
__device__ __forceinline__ int own_segment(uint32_t starts, const int *mark, int k, int first) {
  const uint32_t upto = starts & ((2u << k) - 1);
  return upto ? mark[31 - __clz(upto)] : first;
}

__device__ __forceinline__ int uniform_warp() {
  return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
}

// The segment of a warp's first token, from the marks of its tile: the highest index up to it.
__device__ __forceinline__ int segment_at(const int *mark, int i, int alive) {
  int m = alive;
  for (int j = threadIdx.x & 31; j <= i; j += 32) m = max(m, mark[j]);
  return __reduce_max_sync(0xffffffffu, m);
}

// The same for each group of lanes: its first token is the tile's i-th, then those kK on.
template <int SUB>
__device__ __forceinline__ int segments_at(const int *mark, int i, int alive) {
  int seg = 0;
#pragma unroll
  for (int j = 0; j < SUB; ++j) {
    const int v = segment_at(mark, i + j * kK, alive);
    if (SUB == 1 || (int)(threadIdx.x & 31) / (32 / SUB) == j) seg = v;
  }
  return seg;
}

// nv of two fp32 values at any address
__device__ __forceinline__ f2 load_state(const float *p, int nv) {
  return pair(nv > 0 ? p[0] : 0.f, nv > 1 ? p[1] : 0.f);
}
__device__ __forceinline__ void store_state(float *p, f2 v, int nv) {
  float lo, hi;
  unpair(v, lo, hi);
  if (nv > 0) p[0] = lo;
  if (nv > 1) p[1] = hi;
}
template <bool VEC, typename E>
__device__ __forceinline__ void store(E *p, f2 v, int nv) {
  float lo, hi;
  unpair(v, lo, hi);
  st2<VEC>(p, lo, hi, nv);
}

// ------------------------------------------------------------------ forward

// The chain warp's work in step s, once the holders' maps are there: the block's map to all blocks, and
// from theirs the state in front of each warp.  The block's map goes out as counted stores, so that
// nobody waits for this block's other writes as at a cluster's barrier.  A place is written again two
// steps later: by a block that has seen all maps of the step between, whose senders had read this one's.
// BACK: warps and blocks in reverse.  Only the lanes of one group have maps of their own.
// lost: a wait of this block ran out.  The results are void then, and it neither sends nor waits any more,
// but goes on to the end, where the cluster's blocks meet: the others, which miss its maps, do the same within
// one wait of their own.
template <bool BACK, int SUB>
__device__ __forceinline__ void chain(Shared<SUB> &s, int step, bool any, f2 &carry, bool &lost,
                                      uint64_t limit_ns = kRecWaitNs) {
  constexpr int L = 32 / SUB;
  const int lane = place_of<SUB>(threadIdx.x & 31), buf = step & 1, rank = cluster_rank(), size = cluster_size();
  const bool speaks = SUB == 1 || (threadIdx.x & 31) < L;
  auto map = [&](int j) { return unpacked(s.warp[buf][BACK ? kHold - 1 - j : j][lane]); };
  Map all = map(0);
  if (any) {
#pragma unroll 1
    for (int j = 1; j < kHold; ++j) all = then(all, map(j));
  } else {
#pragma unroll
    for (int j = 1; j < kHold; ++j) all = then_inside(all, map(j));
  }
  const float4 out = packed(all);
  if (!lost) {
#pragma unroll 2
    for (int to = 0; to < size; ++to)
      if (speaks) send(&s.block[buf][rank][lane], &s.bar[buf], to, out);
    if ((threadIdx.x & 31) == 0) tc::mbar_expect_tx(&s.bar[buf], size * L * 16);
    __syncwarp();
    lost = __any_sync(0xffffffffu, !tc::mbar_wait(&s.bar[buf], step >> 1 & 1, nullptr, limit_ns));
    if (lost) atomicCAS(&g_rec_status, 0, BACK ? 0x602 : 0x601);
  }
  f2 h = carry, front = carry;
#pragma unroll 4
  for (int j = 0; j < size; ++j) {
    const int b = BACK ? size - 1 - j : j;
    const Map v = unpacked(s.block[buf][b][lane]);
    if (b == rank) front = h;
    h = through(v, h);
  }
  carry = h;
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    if (speaks) s.front[buf][BACK ? kHold - 1 - j : j][lane] = front;
    if (j < kHold - 1) front = through(map(j), front);
  }
}

// A warp's groups in order: its map for the chain, and returned the map in front of the lane's tokens.
template <bool BACK, int SUB>
__device__ __forceinline__ Map post(Shared<SUB> &s, int step, int warp, bool any, Map mine) {
  constexpr int L = 32 / SUB;
  const int lane = threadIdx.x & 31, group = BACK ? SUB - 1 - lane / L : lane / L;
  Map all = mine, front = {both(1.f), both(0.f)};
  if constexpr (SUB > 1) {
    auto from = [&](Map m, int groups) {  // that of the lane so many groups before
      float4 v = packed(m);
      const int at = BACK ? lane + groups * L : lane - groups * L;
      v.x = __shfl_sync(0xffffffffu, v.x, at & 31);
      v.y = __shfl_sync(0xffffffffu, v.y, at & 31);
      v.z = __shfl_sync(0xffffffffu, v.z, at & 31);
      v.w = __shfl_sync(0xffffffffu, v.w, at & 31);
      return unpacked(v);
    };
#pragma unroll
    for (int d = 1; d < SUB; d *= 2) {
      const Map before = from(all, d);
      if (group >= d) all = any ? then(before, all) : then_inside(before, all);
    }
    const Map before = from(all, 1);
    if (group > 0) front = before;
  }
  if (SUB == 1 || group == SUB - 1) s.warp[step & 1][warp][place_of<SUB>(lane)] = packed(all);
  __syncwarp();
  arrive(kMaps + (step & 1));
  return front;
}

// Rows at multiples of n bytes, floats of pairs at multiples of 8.
template <typename E>
bool rows_fit(const RecArgs &a, int n, std::initializer_list<Mat> mats,
              std::initializer_list<const void *> f) {
  bool ok = a.D * (int64_t)sizeof(E) % n == 0;
  for (const Mat &m : mats)
    ok = ok && reinterpret_cast<uintptr_t>(m.p) % n == 0 && m.st * (int64_t)sizeof(E) % n == 0;
  for (const void *p : f) ok = ok && reinterpret_cast<uintptr_t>(p) % 8 == 0;
  return ok;
}

// Blocks of a cluster: as many as the tokens fill, while all clusters run at once (a cluster's blocks lie
// in one part of the GPU, so that fewer fit than their number of blocks says).
template <typename K>
int cluster_for(K *kernel, int T, int D, int sub, int smem,
                std::atomic<int> (&known)[64][kMostCl + 1]) {
  const int64_t groups = ceil_div64(D, channels_of(sub)), tiles = ceil_div64(T, tile_of(sub));
  int cl = tiles < 1 ? 1 : tiles > kMostCl ? kMostCl : (int)tiles;
  while (cl > 1 && clusters_at_once(kernel, cl, kP * 32, smem, known) < groups) --cl;
  return cl;
}

template <auto kernel, typename... A>
cudaError_t run_clusters(const RecArgs &a, int sub, int smem, cudaStream_t stream, A... more) {
  static std::atomic<uint64_t> bytes{0}, size{0};
  static std::atomic<int> known[64][kMostCl + 1];
  cudaError_t e = set_once(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, bytes);
  if (e == cudaSuccess) e = set_once(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, size);
  if (e != cudaSuccess) return e;
  const int cl = cluster_for(kernel, a.T, a.D, sub, smem, known);
  return launch_clusters(kernel, (int)ceil_div64(a.D, channels_of(sub)) * cl, cl, kP * 32, smem, stream, a, more...);
}

// Groups of lanes: as few as fill the blocks that run at once, or those that give the most blocks; no more for
// tokens that are four steps or fewer of the largest clusters.  Blocks that run at once are counted as two
// a multiprocessor, as they are in bf16, for which the rule was made; the fp32 backward's rows ahead
// (172,032 bytes) leave room for one.  The rule takes two groups where one is the better by a little
// (4,096 x 1,024).  Forward and backward with 1, 2 and 4 groups in us, bf16: 65,536 x 128 102 + 172, 64 + 101, 56 + 94; 30,000 x 512
// 73 + 135, 58 + 96, 55 + 88; 30,000 x 1,024 96 + 188, 83 + 156, 91 + 157; 8,192 x 2,560 56 + 104, 62 + 111,
// 97 + 169; 32,768 x 4,096 277 + 544, 297 + 555, 339 + 608; 4,096 x 1,024 20 + 31, 21 + 35, 21 + 38;
// 1,500 x 680 11 + 17, 11 + 19, 14 + 24; 10 x 64 6 + 9, with 4 groups 8 + 12.
inline int groups_of_lanes(int T, int D) {
  int64_t best = 0;
  int sub = 1;
  for (int s = 1; s <= kMostSub; s *= 2) {
    const int64_t tiles = ceil_div64(T, tile_of(s)), cl = tiles < kMostCl ? tiles : kMostCl;
    const int64_t blocks = ceil_div64(D, channels_of(s)) * (cl < 1 ? 1 : cl);
    if (blocks > best) {
      best = blocks;
      sub = s;
    }
    if (blocks >= 2 * (int64_t)sm_count() || tiles <= 4 * kMostCl) break;
  }
  return sub;
}

}  // namespace
}  // namespace mix
}  // namespace gdr
