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
#include "gdr_tc.cuh"

namespace gdr {
namespace mix {
namespace {

// Nonzero once a wait for another block of a cluster ran out; read by gdr_device_status.
__device__ int32_t g_rec_status = 0;
constexpr uint64_t kRecWaitNs = 2000000000ull;  // 2 s a wait

constexpr int kCh = 64;      // channels of a block: two a lane
constexpr int kMostCl = 16;  // blocks of a cluster (over 8 with the device's consent)

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

// a = 2^L2 and 1 - a^2.  Next to a = 1 both come from the series of d = 1 - a (the first term left out is
// 1e-9 of it at the border, ln a = -1/16): the special-function unit's 2^x falls short by 2e-8 on
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
constexpr float kNear = -0.09016844f;  // L2 above: the series
__device__ __forceinline__ f2 decay_of(f2 L2) {
  const f2 near = fma2(short_of_one(L2), both(-1.f), both(1.f));
  float l0, l1, n0, n1;
  unpair(L2, l0, l1);
  unpair(near, n0, n1);
  return pair(l0 > kNear ? n0 : ex2(l0), l1 > kNear ? n1 : ex2(l1));
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
  a0 = l0 > kNear ? n0 : ex2(l0);
  a1 = l1 > kNear ? n1 : ex2(l1);
  t.a = pair(a0, a1);
  t.m = both(1.f);
  if (NORM) {
    float s0, s1;
    unpair(mul2(d, add2(near, both(1.f))), s0, s1);
    t.m = pair(sqrt_approx(l0 > kNear ? s0 : fmaf(-a0, a0, 1.f)),
               sqrt_approx(l1 > kNear ? s1 : fmaf(-a1, a1, 1.f)));
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

// ------------------------------------------------------------------ pairs (A, U): h -> A h + U
//
// A = 0 says that the pair holds a segment's start: what comes before it is not looked at, be it
// infinite or NaN.  (A product of decays that underflows to 0 says the same of a state that is gone.)

struct Map {
  f2 A, U;
};
__device__ __forceinline__ f2 pick(bool lo, bool hi, f2 yes, f2 no) {
  float a, b, c, d;
  unpair(yes, a, b);
  unpair(no, c, d);
  return pair(lo ? a : c, hi ? b : d);
}
__device__ __forceinline__ f2 through(Map f, f2 h) {
  float lo, hi;
  unpair(f.A, lo, hi);
  return pick(lo == 0.f, hi == 0.f, f.U, fma2(f.A, h, f.U));
}
// first f, then g
__device__ __forceinline__ Map then(Map f, Map g) {
  float lo, hi;
  unpair(g.A, lo, hi);
  return Map{pick(lo == 0.f, hi == 0.f, both(0.f), mul2(f.A, g.A)), through(g, f.U)};
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
// No block ends while another may write to it.
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  cluster_wait();
}
__device__ __forceinline__ uint32_t at_rank(const void *p, int rank) {
  uint32_t to;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(p)), "r"(rank));
  return to;
}
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

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int blocks, int cluster, int threads,
                            int smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = stream;
  c.attrs = at;
  c.numAttrs = 2;
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

// ------------------------------------------------------------------ a warp's tokens

constexpr int kP = 8, kK = 8;  // warps of a block, tokens of a thread
constexpr int kHold = kP - 1, kTile = kHold * kK;  // warps with tokens, tokens of a block
static_assert(kRecEvery == kK, "a kept state for each thread's tokens");

// Of a block's eight warps seven hold tokens and one chains their maps.  The holders compute the maps of
// step s + 1 while the chain of step s is on its way through the cluster, and then run through step
// s: nobody waits for a map that was sent just now.  Places are written again when a later meeting
// has shown that they were read: maps and states two steps on, bounds (looked up two steps ahead) four.
struct Shared {
  float4 warp[2][kHold][32];     // (A, U) of both channels, for each warp with tokens
  float4 block[2][kMostCl][32];  // and for each block of the cluster
  f2 front[2][kHold][32];        // the state in front of each warp's tokens
  uint64_t bar[2];               // every block's map is here
  int mark[4][kTile + 1];
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

// The N tensors of a step on their way into shared memory: a warp's rows of 64 channels come 16 bytes
// at a time into one of S places of its own, a step ahead, and are read two channels a lane.
// Without 16-byte alignment (RING false) they are loaded when they are used.
template <typename E, bool RING, int N, int S>
struct Tokens {
  static constexpr int kRow = kCh * (int)sizeof(E);          // bytes
  static constexpr int kPlace = N * kK * kRow;               // of a warp's step
  static constexpr int kBytes = RING ? S * kHold * kPlace : 0;  // of a block
  const E *p[N];  // at this block's first channel; null: not there
  int64_t st[N];
  unsigned char *mine;  // this warp's places
  int lane, cols, nv, T;
  const E *from[N];  // the lane's part of the next step's first rows

  // rows from token t on are the first to come, then those `step` tokens on each time
  __device__ __forceinline__ void start(int t) {
    if (RING) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        from[n] = p[n] + (int64_t)(t + lane / kL) * st[n] + lane % kL * (16 / (int)sizeof(E));
    }
  }
  static constexpr int kL = kRow / 16, kR = 32 / kL;  // lanes of a row, rows of an instruction
  __device__ __forceinline__ void issue(int place, int t, int step) {
    if (RING) {
      __syncwarp();  // the place was read by all lanes
      const int left = lane % kL * (16 / (int)sizeof(E)) < cols ? T - t - lane / kL : 0;
      unsigned char *to = mine + place * kPlace + lane * 16;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n == 2 && !p[n]) continue;
        const E *q = from[n];
#pragma unroll
        for (int k = 0; k < kK; k += kR) {
          if (k < left) copy16(reinterpret_cast<uint4 *>(to + (n * kK + k) * kRow), q);
          q += kR * st[n];
        }
        from[n] += step * st[n];
      }
      copies_commit();
    }
  }
  __device__ __forceinline__ void wait() const {
    if (RING) {
      copies_wait<1>();
      __syncwarp();
    }
  }
  // the lane's two channels of token t = t0 + k
  __device__ __forceinline__ f2 get(int place, int n, int k, int t) const {
    if (RING)
      return wide(*reinterpret_cast<const Raw2<E> *>(mine + place * kPlace + (n * kK + k) * kRow +
                                                     lane * 2 * (int)sizeof(E)));
    return wide(ld2<false>(p[n] + (int64_t)t * st[n] + lane * 2, t < T ? nv : 0));
  }
};

// Bit k: a segment starts with token k of n, of which `left` are there.
__device__ __forceinline__ uint32_t starts_of(const int *mark, int left, int n) {
  const int k = threadIdx.x & 31;
  return __ballot_sync(0xffffffffu, k < n && k <= left && left > 0 && mark[min(k, max(left, 0))] >= 0);
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
// BACK: warps and blocks in reverse.
template <bool BACK>
__device__ __forceinline__ void chain(Shared &s, int step, bool any, f2 &carry) {
  const int lane = threadIdx.x & 31, buf = step & 1, rank = cluster_rank(), size = cluster_size();
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
#pragma unroll 2
  for (int to = 0; to < size; ++to) send(&s.block[buf][rank][lane], &s.bar[buf], to, out);
  if (lane == 0) tc::mbar_expect_tx(&s.bar[buf], size * 512);
  __syncwarp();
  if (!tc::mbar_wait(&s.bar[buf], step >> 1 & 1, nullptr, kRecWaitNs))
    atomicCAS(&g_rec_status, 0, BACK ? 0x602 : 0x601);  // the results are void; go on to the end
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
    s.front[buf][BACK ? kHold - 1 - j : j][lane] = front;
    if (j < kHold - 1) front = through(map(j), front);
  }
}

// A warp's tokens of a step: decays and inputs, and what starts among them.
struct Step {
  f2 at[kK], u[kK];
  uint32_t starts;  // bit k: a segment starts with token k
};

// OUT: y is written (without it only the kept states: the backward's first pass).
template <typename E, bool VEC, bool OUT, bool NORM>
__global__ void __launch_bounds__(kP * 32, 2) k_rec_fwd(const RecArgs a) {
  after_previous();
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ Shared s;
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int rank = cluster_rank(), size = cluster_size();
  const int cb = (int)(blockIdx.x / size) * kCh, c0 = cb + lane * 2, nv = max(0, min(2, a.D - c0));
  const int stride = size * kTile, steps = (a.T + stride - 1) / stride;
  s.init();
  if (warp == kHold) {
    SegCursor cursor{0, 0, 0};
    auto look = [&](int step) {  // the bounds of a tile
      const int buf = step & 3;
      const int64_t t0 = (int64_t)step * stride + rank * kTile;
      int alive = -1;
      const bool any = t0 < a.T && tile_marks(a.cu, a.n_seq, a.T, (int)t0, min(kTile, a.T - (int)t0),
                                              s.mark[buf], cursor, alive);
      if (lane == 0) {
        s.any[buf] = any;
        s.alive[buf] = alive;
      }
      return any;
    };
    bool any0 = look(0), any1 = look(1);
    cluster_arrive();  // every block of the cluster runs before one writes to it
    cluster_wait();
    f2 carry = both(0.f);
    for (int step = 0; step < steps; ++step) {
      meet(kMaps + (step & 1));
      const bool any2 = look(step + 2);
      chain<false>(s, step, any0, carry);
      any0 = any1;
      any1 = any2;
      __syncwarp();
      arrive(kFronts + (step & 1));
    }
  } else {
    const f2 A2 = mul2(load_state(a.A + c0, nv), both(kLog2e));
    using In = Tokens<E, VEC, 3, 2>;
    In in{{reinterpret_cast<const E *>(a.x.p) + cb, reinterpret_cast<const E *>(a.r.p) + cb,
           a.i.p ? reinterpret_cast<const E *>(a.i.p) + cb : nullptr},
          {a.x.st, a.r.st, a.i.st},
          raw + warp * 2 * In::kPlace, lane, a.D - cb, nv, a.T};
    const bool gate = a.i.p;
    E *y = reinterpret_cast<E *>(a.y.p) + c0;
    const int first = rank * kTile + warp * kK;
    in.start(first);
    in.issue(0, first, stride);
    in.issue(1, first + stride, stride);
    cluster_arrive();
    cluster_wait();

    auto hold = [&](int step, Step &v) {  // the step's tokens, and their map for the chain
      const int place = step & 1, tw = first + step * stride, left = a.T - tw;
      in.wait();
      auto make = [&](int k, f2 sr, f2 x) {
        const Token t = token<NORM>(sr, A2);
        v.at[k] = t.a;
        v.u[k] = NORM ? mul2(t.m, x) : x;
      };
      bool alone = !gate;
      if (gate) {
        float q = 1.f;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          f2 sr, si;
          float p;
          sigmoids(in.get(place, 1, k, tw + k), in.get(place, 2, k, tw + k), sr, si, p);
          q = fminf(q, p);
          make(k, sr, mul2(si, in.get(place, 0, k, tw + k)));
        }
        alone = __any_sync(0xffffffffu, q == 0.f);
      }
      if (alone) {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          f2 x = in.get(place, 0, k, tw + k);
          if (gate) x = mul2(x, sigmoid2(in.get(place, 2, k, tw + k)));
          make(k, sigmoid2(in.get(place, 1, k, tw + k)), x);
        }
      }
      // segments that start among the tokens: their state goes into the first one
      const bool any = s.any[step & 3];
      v.starts = 0;
      if (any || left < kK) {
        const int *mark = s.mark[step & 3] + warp * kK;
        if (any && left > 0) {
#pragma unroll 1
          for (int k = 0; k < kK; ++k)
            if (k < left && mark[k] >= 0) v.starts |= 1u << k;
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          if (k >= left) {
            v.at[k] = both(1.f);
            v.u[k] = both(0.f);
          } else if (v.starts >> k & 1 && a.h0 && mark[k] < a.n_seq) {
            v.u[k] = fma2(v.at[k], load_state(a.h0 + (int64_t)mark[k] * a.D + c0, nv), v.u[k]);
          }
        }
      }
      Map mine = {v.at[0], v.u[0]};
      if (v.starts == 0) {
#pragma unroll
        for (int k = 1; k < kK; ++k) mine = Map{mul2(mine.A, v.at[k]), fma2(v.at[k], mine.U, v.u[k])};
      } else {
        if (v.starts & 1) mine.A = both(0.f);
#pragma unroll
        for (int k = 1; k < kK; ++k)
          mine = v.starts >> k & 1 ? Map{both(0.f), v.u[k]}
                                   : Map{mul2(mine.A, v.at[k]), fma2(v.at[k], mine.U, v.u[k])};
      }
      s.warp[step & 1][warp][lane] = packed(mine);
      __syncwarp();
      arrive(kMaps + (step & 1));
    };
    auto run = [&](int step, const Step &v) {  // through the tokens from their true state
      const int tw = first + step * stride, left = a.T - tw;
      meet(kFronts + (step & 1));
      f2 h = s.front[step & 1][warp][lane];
      if (left <= 0) return;
      const bool any = s.any[step & 3];
      int seg = s.alive[step & 3];
      if (a.kept) store<VEC>(a.kept + (int64_t)(tw / kK) * a.D + c0, h, nv);
      E *to = y + (int64_t)tw * a.y.st;
      if (!any && left >= kK) {
        const int n = seg >= 0 && seg < a.n_seq ? nv : 0;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          h = fma2(v.at[k], h, v.u[k]);
          if (OUT) store<VEC>(to, h, n);
          to += a.y.st;
        }
      } else {
        if (any) seg = segment_at(s.mark[step & 3], warp * kK, seg);
        const int *mark = s.mark[step & 3] + warp * kK;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          if (k >= left) break;
          const bool starts = v.starts >> k & 1;
          if (starts) seg = mark[k];
          h = starts ? v.u[k] : fma2(v.at[k], h, v.u[k]);
          if (seg >= 0 && seg < a.n_seq) {
            if (OUT) store<VEC>(to, h, nv);
            if (a.ht && any && mark[k + 1] >= 0) store_state(a.ht + (int64_t)seg * a.D + c0, h, nv);
          }
          to += a.y.st;
        }
      }
    };
    Step even, odd;
    if (steps > 0) hold(0, even);
    for (int step = 0; step < steps; step += 2) {
      in.issue(0, first + (step + 2) * stride, stride);
      if (step + 1 < steps) hold(step + 1, odd);
      run(step, even);
      if (step + 1 < steps) {
        in.issue(1, first + (step + 3) * stride, stride);
        if (step + 2 < steps) hold(step + 2, even);
        run(step + 1, odd);
      }
    }
    if (VEC) copies_wait<0>();
  }
  __syncthreads();
  cluster_leave();
  // segments without tokens end as they start
  if (a.ht && rank == 0)
    for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
      if (warp == 0) {
        const int64_t at = (int64_t)n * a.D + c0;
        store_state(a.ht + at, a.h0 ? load_state(a.h0 + at, nv) : both(0.f), nv);
      }
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

template <typename E, bool VEC, bool NORM>
__global__ void __launch_bounds__(kP * 32, 2) k_rec_bwd(const RecArgs a, const int32_t *bounds) {
  after_previous();
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ Shared s;
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int rank = cluster_rank(), size = cluster_size();
  const int cb = (int)(blockIdx.x / size) * kCh, c0 = cb + lane * 2, nv = max(0, min(2, a.D - c0));
  const int stride = size * kTile, steps = (a.T + stride - 1) / stride;
  const f2 one = both(1.f), minus = both(-1.f);
  f2 dA = both(0.f);
  s.init();
  if (warp == kHold) {
    BackCursor cursor{a.n_seq, bounds[a.n_seq]};
    auto look = [&](int step) {  // the bounds of a tile
      const int buf = step & 3, t0 = (steps - 1 - step) * stride + rank * kTile;
      int alive = -1;
      const bool any = step < steps && t0 < a.T &&
                       tile_marks_back(bounds, t0, min(kTile, a.T - t0), s.mark[buf], cursor, alive);
      if (lane == 0) {
        s.any[buf] = any;
        s.alive[buf] = alive;
      }
      return any;
    };
    bool any0 = look(0), any1 = look(1);
    cluster_arrive();  // every block of the cluster runs before one writes to it
    cluster_wait();
    f2 carry = both(0.f);
    for (int step = 0; step < steps; ++step) {
      meet(kMaps + (step & 1));
      const bool any2 = look(step + 2);
      chain<true>(s, step, any0, carry);
      any0 = any1;
      any1 = any2;
      __syncwarp();
      arrive(kFronts + (step & 1));
    }
  } else {
    const f2 A = load_state(a.A + c0, nv), A2 = mul2(A, both(kLog2e));
    using In = Tokens<E, VEC, 4, 3>;
    In in{{reinterpret_cast<const E *>(a.x.p) + cb, reinterpret_cast<const E *>(a.r.p) + cb,
           a.i.p ? reinterpret_cast<const E *>(a.i.p) + cb : nullptr,
           reinterpret_cast<const E *>(a.dy.p) + cb},
          {a.x.st, a.r.st, a.i.st, a.dy.st},
          raw + warp * 3 * In::kPlace, lane, a.D - cb, nv, a.T};
    const bool gate = a.i.p;
    E *dx = reinterpret_cast<E *>(a.dx.p) + c0, *dr = reinterpret_cast<E *>(a.dr.p) + c0;
    E *di = reinterpret_cast<E *>(a.di.p) + c0;
    const int first = (steps - 1) * stride + rank * kTile + warp * kK;
    in.start(first);
    in.issue(0, steps > 0 ? first : a.T, -stride);
    in.issue(1, steps > 1 ? first - stride : a.T, -stride);
    cluster_arrive();
    cluster_wait();

    // the state that a segment starts from, the gradient of the one it ends with
    auto origin = [&](int n) {
      return a.h0 && n < a.n_seq ? load_state(a.h0 + (int64_t)n * a.D + c0, nv) : both(0.f);
    };
    auto ending = [&](int n) {
      return a.dht && n >= 0 && n < a.n_seq ? load_state(a.dht + (int64_t)n * a.D + c0, nv) : both(0.f);
    };
    // what a step's tokens have among them; one that ends with the last does not count
    auto starts_in = [&](int step, int left) {
      return s.any[step & 3] ? starts_of(s.mark[step & 3] + warp * kK, left, kK + 1) : 0u;
    };
    auto hold = [&](int place, int step) {  // the map of the step's tokens, for the chain
      const int tw = first - step * stride, left = a.T - tw;
      in.wait();
      const uint32_t starts = starts_in(step, left);
      Map mine = {one, both(0.f)};
      if (starts == 0 && left >= kK) {
        f2 at[kK];
#pragma unroll
        for (int k = 0; k < kK; ++k) at[k] = decay_of(mul2(A2, sigmoid2(in.get(place, 1, k, tw + k))));
        mine = Map{at[kK - 1], mul2(at[kK - 1], in.get(place, 3, kK - 1, tw + kK - 1))};
#pragma unroll
        for (int k = kK - 2; k >= 0; --k)
          mine = Map{mul2(mine.A, at[k]), mul2(at[k], add2(in.get(place, 3, k, tw + k), mine.U))};
      } else if (left > 0) {
        const int *mark = s.mark[step & 3];
#pragma unroll 1
        for (int k = min(kK, left) - 1; k >= 0; --k) {
          const f2 at = decay_of(mul2(A2, sigmoid2(in.get(place, 1, k, tw + k))));
          f2 g = in.get(place, 3, k, tw + k);
          if (starts >> (k + 1) & 1) {
            g = add2(g, ending(segment_at(mark, warp * kK + k, s.alive[step & 3])));
            mine = Map{both(0.f), mul2(at, g)};
          } else {
            mine = Map{mul2(mine.A, at), mul2(at, add2(g, mine.U))};
          }
        }
      }
      s.warp[step & 1][warp][lane] = packed(mine);
      __syncwarp();
      arrive(kMaps + (step & 1));
    };
    // The gradients of one token from its parts; G: dL/dh.  Moves dA on.
    auto grads = [&](f2 G, f2 at, f2 m, f2 sr, f2 si, f2 x, f2 before, f2 &ox, f2 &orr, f2 &oi) {
      const f2 w = mul2(si, x), dv = mul2(G, m);
      f2 past = before;
      if (NORM) {
        // the normaliser's part of d/dL; none where a is 1 and it has no derivative
        float lo, hi;
        unpair(m, lo, hi);
        const f2 ratio = mul2(at, pair(lo != 0.f ? rcp(lo) : 0.f, hi != 0.f ? rcp(hi) : 0.f));
        past = fma2(mul2(w, minus), ratio, past);
      }
      const f2 q = mul2(mul2(mul2(G, at), past), sr);  // dL sr
      ox = mul2(dv, si);
      oi = mul2(mul2(dv, w), fma2(si, minus, one));
      orr = mul2(mul2(A, q), fma2(sr, minus, one));
      return q;
    };
    auto run = [&](int place, int step) {  // the gradients of the step's tokens
      const int tw = first - step * stride, left = a.T - tw;
      f2 h = both(0.f);
      if (left > 0) h = wide(ld2<VEC>(a.kept + (int64_t)(tw / kK) * a.D + c0, nv));
      const uint32_t starts = starts_in(step, left);
      int seg = s.alive[step & 3];
      if (s.any[step & 3] && left > 0) seg = segment_at(s.mark[step & 3], warp * kK, seg);
      if (starts == 0 && left >= kK && seg >= 0 && seg < a.n_seq) {
        f2 sr[kK], si[kK], at[kK], m[kK], hb[kK];
        bool alone = !gate;
        if (gate) {
          float q = 1.f;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            float p;
            sigmoids(in.get(place, 1, k, tw + k), in.get(place, 2, k, tw + k), sr[k], si[k], p);
            q = fminf(q, p);
          }
          alone = __any_sync(0xffffffffu, q == 0.f);
        }
        if (alone) {
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            sr[k] = sigmoid2(in.get(place, 1, k, tw + k));
            si[k] = gate ? sigmoid2(in.get(place, 2, k, tw + k)) : one;
          }
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const Token v = token<NORM>(sr[k], A2);
          at[k] = v.a;
          m[k] = v.m;
          hb[k] = h;
          h = fma2(at[k], h, mul2(m[k], mul2(si[k], in.get(place, 0, k, tw + k))));
        }
        meet(kFronts + (step & 1));
        f2 c = s.front[step & 1][warp][lane];
        const int64_t t = tw + kK - 1;
        E *px = dx + t * a.dx.st, *pr = dr + t * a.dr.st, *pi = di + t * a.di.st;
#pragma unroll
        for (int k = kK - 1; k >= 0; --k) {
          f2 ox, orr, oi;
          const f2 G = add2(in.get(place, 3, k, tw + k), c);
          dA = add2(dA, grads(G, at[k], m[k], sr[k], si[k], in.get(place, 0, k, tw + k), hb[k], ox, orr,
                              oi));
          c = mul2(at[k], G);
          store<VEC>(px, ox, nv);
          store<VEC>(pr, orr, nv);
          if (gate) store<VEC>(pi, oi, nv);
          px -= a.dx.st;
          pr -= a.dr.st;
          pi -= a.di.st;
        }
        return;
      }
      // one by one: where a segment starts, before and behind all of them, behind the last token
      const int *mark = s.mark[step & 3] + warp * kK;
      f2 hb[kK];  // not in registers
      auto part = [&](int k, f2 &sr, f2 &si, f2 &at, f2 &m) {
        sr = sigmoid2(in.get(place, 1, k, tw + k));
        si = gate ? sigmoid2(in.get(place, 2, k, tw + k)) : one;
        const Token v = token<NORM>(sr, A2);
        at = v.a;
        m = v.m;
      };
      f2 sr, si, at, m;
#pragma unroll 1
      for (int k = 0; k < min(kK, left); ++k) {
        if (starts >> k & 1) h = origin(mark[k]);
        hb[k] = h;
        part(k, sr, si, at, m);
        h = fma2(at, h, mul2(m, mul2(si, in.get(place, 0, k, tw + k))));
      }
      meet(kFronts + (step & 1));
      f2 c = s.front[step & 1][warp][lane];
#pragma unroll 1
      for (int k = min(kK, left) - 1; k >= 0; --k) {
        const int own = s.any[step & 3] ? segment_at(mark, k, seg) : seg;
        part(k, sr, si, at, m);
        f2 G = in.get(place, 3, k, tw + k), ox, orr, oi;
        G = starts >> (k + 1) & 1 ? add2(G, ending(own)) : add2(G, c);
        const f2 q = grads(G, at, m, sr, si, in.get(place, 0, k, tw + k), hb[k], ox, orr, oi);
        c = mul2(at, G);
        if (own >= 0 && own < a.n_seq) {
          dA = add2(dA, q);
          if (a.dh0 && starts >> k & 1) store_state(a.dh0 + (int64_t)own * a.D + c0, c, nv);
        } else {
          ox = oi = orr = both(0.f);
        }
        const int64_t t = tw + k;
        store<VEC>(dx + t * a.dx.st, ox, nv);
        store<VEC>(dr + t * a.dr.st, orr, nv);
        if (gate) store<VEC>(di + t * a.di.st, oi, nv);
      }
    };
    if (steps > 0) hold(0, 0);
    int place = 0;  // of the step that is run
    auto after = [](int p) { return p == 2 ? 0 : p + 1; };
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      const int next = after(place);
      // the step after next into the place of the one before this
      in.issue(after(next), step + 2 < steps ? first - (step + 2) * stride : a.T, -stride);
      if (step + 1 < steps) hold(next, step + 1);
      run(place, step);
      place = next;
    }
    if (VEC) copies_wait<0>();
  }
  // dA: the warps' sums in order, then the blocks' of the cluster
  __syncthreads();
  if (warp < kHold) s.warp[0][warp][lane] = packed(Map{dA, both(0.f)});
  __syncthreads();
  if (warp == 0) {
    f2 v = unpacked(s.warp[0][0][lane]).A;
#pragma unroll
    for (int w = 1; w < kHold; ++w) v = add2(v, unpacked(s.warp[0][w][lane]).A);
    put(&s.block[steps & 1][rank][lane], 0, packed(Map{v, both(0.f)}));
  }
  cluster_arrive();
  cluster_wait();
  if (rank == 0) {
    if (warp == 0) {
      f2 v = unpacked(s.block[steps & 1][0][lane]).A;
      for (int b = 1; b < size; ++b) v = add2(v, unpacked(s.block[steps & 1][b][lane]).A);
      store_state(a.dA + c0, v, nv);
    }
    if (a.dh0)
      for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
        if (warp == 0) {
          const int64_t at = (int64_t)n * a.D + c0;
          store_state(a.dh0 + at, a.dht ? load_state(a.dht + at, nv) : both(0.f), nv);
        }
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
  f2 u = wide(x);
  if (a.i.p)
    u = mul2(u, sigmoid2(wide(
                    ld2<VEC>(reinterpret_cast<const E *>(a.i.p) + (int64_t)row * a.i.st + c0, nv))));
  const f2 A2 = mul2(wide(A), both(kLog2e));
  const Token v = a.normalize ? token<true>(sigmoid2(wide(r)), A2) : token<false>(sigmoid2(wide(r)), A2);
  const f2 out = fma2(v.a, wide(h), mul2(v.m, u));
  store<VEC>(q, out, nv);
  store<VEC>(y, out, nv);
}

// ------------------------------------------------------------------ launches

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

// Clusters of `cl` blocks that run at once (asked for once for each device and size; -1: unknown).
template <typename K>
int clusters_at_once(K *kernel, int cl, int smem, std::atomic<int> (&known)[64][kMostCl + 1]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev >= 0 && dev < 64) {
    const int n = known[dev][cl].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)cl;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)cl);
  c.blockDim = dim3(kP * 32);
  c.dynamicSmemBytes = (size_t)smem;
  c.attrs = &at;
  c.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &c) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  if (n > 0 && dev >= 0 && dev < 64) known[dev][cl].store(n, std::memory_order_relaxed);
  return n;
}

// Blocks of a cluster: as many as the tokens fill, while all clusters run at once (a cluster's blocks lie
// in one part of the GPU, so that fewer fit than their number of blocks says).
template <typename K>
int cluster_for(K *kernel, int T, int D, int tile, int smem,
                std::atomic<int> (&known)[64][kMostCl + 1]) {
  const int64_t groups = (D + kCh - 1) / kCh, tiles = ceil_div64(T, tile);
  int cl = tiles < 1 ? 1 : tiles > kMostCl ? kMostCl : (int)tiles;
  while (cl > 1 && clusters_at_once(kernel, cl, smem, known) < groups) --cl;
  return cl;
}

template <auto kernel, typename... A>
cudaError_t run_clusters(const RecArgs &a, int tile, int smem, cudaStream_t stream, A... more) {
  static std::atomic<uint64_t> bytes{0}, size{0};
  static std::atomic<int> known[64][kMostCl + 1];
  cudaError_t e = set_once(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, bytes);
  if (e == cudaSuccess) e = set_once(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, size);
  if (e != cudaSuccess) return e;
  const int cl = cluster_for(kernel, a.T, a.D, tile, smem, known);
  return launch_clusters(kernel, (a.D + kCh - 1) / kCh * cl, cl, kP * 32, smem, stream, a, more...);
}

template <typename E, bool VEC, bool OUT, bool NORM>
cudaError_t run_fwd_as(const RecArgs &a, cudaStream_t stream) {
  return run_clusters<k_rec_fwd<E, VEC, OUT, NORM>>(a, kTile, Tokens<E, VEC, 3, 2>::kBytes, stream);
}
template <typename E, bool OUT>
cudaError_t run_fwd(const RecArgs &a, cudaStream_t stream) {
  const bool vec = OUT ? rows_fit<E>(a, 16, {a.x, a.r, a.i, a.y}, {a.kept})
                       : rows_fit<E>(a, 16, {a.x, a.r, a.i}, {a.kept});
  if (a.normalize)
    return vec ? run_fwd_as<E, true, OUT, true>(a, stream)
               : run_fwd_as<E, false, OUT, true>(a, stream);
  return vec ? run_fwd_as<E, true, OUT, false>(a, stream)
             : run_fwd_as<E, false, OUT, false>(a, stream);
}

size_t kept_bytes(int64_t T, int32_t D) {
  return align256((size_t)((T + kRecEvery - 1) / kRecEvery) * D * 4);
}

template <typename E, bool VEC, bool NORM>
cudaError_t run_bwd_as(const RecArgs &a, const int32_t *bounds, cudaStream_t stream) {
  return run_clusters<k_rec_bwd<E, VEC, NORM>>(a, kTile, Tokens<E, VEC, 4, 3>::kBytes, stream, bounds);
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
  const bool vec = rows_fit<E>(a, 16, {a.x, a.r, a.i, a.dy, a.dx, a.dr, a.di}, {a.kept});
  if (a.normalize)
    return vec ? run_bwd_as<E, true, true>(a, bounds, stream)
               : run_bwd_as<E, false, true>(a, bounds, stream);
  return vec ? run_bwd_as<E, true, false>(a, bounds, stream)
             : run_bwd_as<E, false, false>(a, bounds, stream);
}

template <typename E>
cudaError_t run_step(const RecArgs &a, float *state, int32_t slots, const int32_t *idx,
                     cudaStream_t stream) {
  const bool vec = a.D % 2 == 0 && rows_fit<E>(a, 2 * sizeof(E), {a.x, a.r, a.i, a.y}, {state, a.A});
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

cudaError_t read_rec_status(int32_t *out) {
  return cudaMemcpyFromSymbol(out, mix::g_rec_status, sizeof(int32_t));
}
cudaError_t clear_rec_status() {
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(mix::g_rec_status, &zero, sizeof(int32_t));
}

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
