// gdr_ssm_bwd.cu -- backward of the selective state space scan.  With y's gradient after the gate
// dy = dout z sigmoid(z), a_t = e^{dt_t A} and the states' gradient
//
//   g_t = C_t dy_t + a_{t+1} g_{t+1}      (+ the final state's gradient at the segment's end)
//
//   dC_t = sum_d dy h_t,   dB_t = sum_d dt x g_t,   p_t = sum_n B g_t,   c_t = a_t h_{t-1} g_t,
//   dx = dt p + D dy,   ddt = (x p + sum_n A c_t) sigmoid(raw),   dA = sum_t dt c_t,
//   dD = sum_t dy x,   dz = dout y (z sigmoid(z))',   dh0 = a g at the segment's first token.
//
// The token axis is cut into ranges of 64 tokens.  Pass 1 runs each range once, forwards, from a
// zero state: it keeps the state at its end and, with the running product of the a, the gradient
// that its own tokens send to the state before it.  A short kernel chains both over the ranges.
// Pass 2 then has a range's true state at its start and true gradient at its end.  It takes the
// range in tiles of up to 8 tokens of one segment: a sweep forwards keeps the state before every
// tile that continues a segment, then the tiles go last to first, each recomputing its states and
// walking back through them.  Both the kept states and a tile's states (8 fp32 a thread each) live
// in Tensor Memory, 128 columns a block, each thread reading back its own lane: in registers and
// shared memory they would leave room for 3 blocks on an SM instead of 4.
//
// Sums over states (p, c A, y) are left as partial sums of LN lanes in shared memory; sums over
// channels (dB, dC) go over the warp's lanes by a transposing butterfly, over its warps in shared
// memory and over the blocks in a last kernel, always in the same order.
//
// 16 products and 3 exponentials for each token, channel and state in pass 2, of about 41 instructions (the
// others move and sum: shared and Tensor Memory, the sums over channels), and 6 and 1 in pass 1: bound
// by instruction issue and, with 16 warps an SM, its latencies: 60 % of the slots.  8,192 tokens of
// 2,048 x 16 states in bf16: 650 us (under the profiler pass 1 131, chain 27, pass 2 475, sums 25); of 32
// and 64 states 1,153 and 2,478 us.
#include "gdr_ssm.cuh"
#include "gdr_tc.cuh"

namespace gdr {
namespace ssm {
namespace {

using namespace mix;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBwdCtas = 4;   // blocks on each SM
constexpr int kBT = 8;        // tokens of a tile of pass 2
constexpr int kRange = 64;    // tokens of a range at most
// Ranges get shorter where the GPU has room for more blocks at once, and the chain over them stays
// short.
constexpr int kLeast = 16, kMostShort = 256;
constexpr int kKept = kRange / kBT;  // states kept at most: tiles that continue a segment
constexpr uint32_t kCols = 8 * (kKept + kBT);  // Tensor Memory columns: kept, then a tile's

struct BwdWork {
  int range, n;     // tokens of a range, ranges
  float *state;     // [n][D][N]: states at the ranges' ends, then at their starts, then dA's parts
  float *grad;      // [n][D][N]: gradients at the ranges' starts, then at their ends
  float *sum;       // [n][D]: sum of dt
  float *pd, *pb;   // [n][D]: parts of dD and ddt_bias
  int *reset;       // [n]
  float *bc;        // [channel tiles][T][2][NP]: parts of dB and dC, T x D x LN^2 / 8 bytes
  size_t bytes;
};

template <typename E, int M>
struct Elems {
  E v[M];
};
template <bool VEC, typename E, int M>
__device__ __forceinline__ Elems<E, M> ldm(const E *p, int n) {
  Elems<E, M> r;
  constexpr int bytes = M * (int)sizeof(E);
  if constexpr (VEC && bytes >= 4) {
    constexpr int w = bytes >= 16 ? 16 : bytes;
    if constexpr (w == 16) {
      uint4 q[bytes / 16];
#pragma unroll
      for (int i = 0; i < bytes / 16; ++i)
        q[i] = n > 0 ? reinterpret_cast<const uint4 *>(p)[i] : make_uint4(0, 0, 0, 0);
      memcpy(&r, q, bytes);
    } else if constexpr (w == 8) {
      const uint2 q = n > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0, 0);
      memcpy(&r, &q, 8);
    } else {
      const uint32_t q = n > 0 ? *reinterpret_cast<const uint32_t *>(p) : 0u;
      memcpy(&r, &q, 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) r.v[i] = i < n ? p[i] : E(0.f);
  }
  return r;
}
template <bool VEC, typename E, int M>
__device__ __forceinline__ void stm(E *p, const float (&f)[M], int n) {
  Elems<E, M> r;
#pragma unroll
  for (int i = 0; i < M; ++i) st1(&r.v[i], f[i]);
  constexpr int bytes = M * (int)sizeof(E);
  if constexpr (VEC && bytes >= 4) {
    if (n <= 0) return;
    if constexpr (bytes >= 16) {
      uint4 q[bytes / 16];
      memcpy(q, &r, bytes);
#pragma unroll
      for (int i = 0; i < bytes / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = q[i];
    } else if constexpr (bytes == 8) {
      uint2 q;
      memcpy(&q, &r, 8);
      *reinterpret_cast<uint2 *>(p) = q;
    } else {
      uint32_t q;
      memcpy(&q, &r, 4);
      *reinterpret_cast<uint32_t *>(p) = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i)
      if (i < n) p[i] = r.v[i];
  }
}

// The whole range's segment bounds: marks, and each token's segment.
struct RangeSegs {
  int mark[kRange + 1], seg[kRange];
  int red[64];
};
__device__ __forceinline__ int warp_max_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = max(v, u);
  }
  return v;
}
// All threads; only the first warp has filled s on return.
__device__ __forceinline__ void range_segments(const SsmArgs &a, int t0, int n, RangeSegs &s) {
  SegCursor c = seg_find(a.cu, a.n_seq, a.T, t0, s.red);
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int base = c.j - 1;
    if (!seg_marks(a.cu, a.n_seq, a.T, t0, n, s.mark, c))
      for (int i = lane; i <= n; i += 32) s.mark[i] = -1;
    __syncwarp();
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int v = max(warp_max_scan(i0 + lane < n ? s.mark[i0 + lane] : -1, lane), base);
      if (i0 + lane < n) s.seg[i0 + lane] = v;
      base = __shfl_sync(0xffffffffu, v, 31);
    }
    __syncwarp();
  }
}
// The first warp: cuts the range into tiles of up to kBT tokens that cross no bound; tile q is
// tokens at[q] .. at[q + 1] - 1.  Returns their number.
__device__ __forceinline__ int range_tiles(int n, const RangeSegs &s, int *at) {
  const int lane = threadIdx.x;
  int base = 0, count = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int run = max(warp_max_scan(i < n && s.mark[i] >= 0 ? i : 0, lane), base);
    base = __shfl_sync(0xffffffffu, run, 31);
    const bool first = i < n && (i - run) % kBT == 0;
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if (first) at[count + __popc(m & ((1u << lane) - 1))] = i;
    count += __popc(m);
  }
  if (lane == 0) at[count] = n;
  return count;
}

template <int LN>
struct __align__(16) Tile1 {
  using Y = Lay<LN>;
  float2 pair[Y::L * Y::PT];
  float dy[Y::L * Y::PT];
  float b[Y::L * Y::NP], c[Y::L * Y::NP];
  float bias[Y::CH];
  RangeSegs s;
};

// Pass 1.
template <typename E, int LN, bool VEC>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
    k_ssm_bwd_ends(const SsmArgs a, const BwdWork w, int tiles_per_group) {
  after_previous();
  using Y = Lay<LN>;
  using R = TileRing<E, VEC, 2>;
  constexpr int L = Y::L, NP = Y::NP, Q = R::S;
  extern __shared__ __align__(16) char smem_raw[];
  Tile1<LN> &s = *reinterpret_cast<Tile1<LN> *>(smem_raw);
  uint4 *ring = reinterpret_cast<uint4 *>(&s + 1);
  const Place<LN> P(a, tiles_per_group);
  const int t0 = P.r * w.range, n = min(w.range, a.T - t0);
  const int lt = P.tid / Y::CG, lc = P.tid % Y::CG * 8, nv = max(0, min(8, P.nch - lc));
  const int64_t c = P.c0 + lc;
  R xr(ring, a.x.p, c, a.x.st, nv);
  R dr(ring + R::kSlots, a.dt.p, c, a.dt.st, nv);
  R gr(ring + 2 * R::kSlots, a.dout.p, c, a.dout.st, nv);
  R zr(ring + 3 * R::kSlots, a.z.p, c, a.z.st, nv);
  const bool gated = a.z.p != nullptr;
  const E *Bp = reinterpret_cast<const E *>(a.B) + P.grp * a.B_sg;
  const E *Cp = reinterpret_cast<const E *>(a.C) + P.grp * a.C_sg;
  BcTile<E, NP, L, VEC> rb, rc;
  auto issue = [&](int q, int i0) {
    const int m = i0 + lt < n ? nv : 0, t = t0 + i0 + lt;
    xr.issue(q, t, m);
    dr.issue(q, t, m);
    gr.issue(q, t, m);
    if (gated) zr.issue(q, t, m);
    copies_commit();
  };
#pragma unroll
  for (int q = 0; q < Q - 1; ++q) issue(q, q * L);
  rb.fetch(Bp, a.B_st, t0, t0 + n, a.N);
  rc.fetch(Cp, a.C_st, t0, t0 + n, a.N);
  for (int i = P.tid; i < Y::CH; i += kThreads)
    s.bias[i] = step_bias(a.dt_bias, P.c0, P.nch, i);
  float A2[2][4], h[2][4], pr[2][4], gs[2][4], S[2] = {0.f, 0.f};
  const float most = P.decays(a, A2);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[k][j] = gs[k][j] = 0.f;
      pr[k][j] = 1.f;
    }
  range_segments(a, t0, n, s.s);
  __syncthreads();
  bool reset = false;  // a segment has started: nothing from here on reaches the state before
  int stage = 0;
  for (int i0 = 0; i0 < n; i0 += L) {
    const int m = min(L, n - i0);
    issue(stage == 0 ? Q - 1 : stage - 1, i0 + (Q - 1) * L);
    copies_wait<Q - 1>();
    put_pairs<E, LN>(s.pair, s.bias, a.softplus, lt, lc, xr.get(stage),
                     dr.get(stage));
    {
      float g[8], z[8];
      unpack8(gr.get(stage), g);
      if (gated) {
        unpack8(zr.get(stage), z);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= z[i] * sigmoidf(z[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s.dy[Y::pair_at(lt, lc) + Y::pair_at(0, i)] = g[i];
    }
    stage = stage + 1 == Q ? 0 : stage + 1;
    rb.put(s.b);
    rc.put(s.c);
    if (i0 + L < n) {
      rb.fetch(Bp, a.B_st, t0 + i0 + L, t0 + n, a.N);
      rc.fetch(Cp, a.C_st, t0 + i0 + L, t0 + n, a.N);
    }
    __syncthreads();
    // ENTERS: of the segment that enters the range, whose tokens' gradients reach the state before
    // it; a later segment's do not, whatever they are (an infinity times 0 would be NaN)
    auto scan = [&](auto ENTERS, int from, int to) {
      tile_tokens<L>(from, to, [&](int i) {
        const int at = i * Y::PT + P.pair;
        const float4 q = *reinterpret_cast<const float4 *>(&s.pair[at]);
        const float4 B = *reinterpret_cast<const float4 *>(&s.b[i * NP + P.nl * 4]);
        const float dt[2] = {q.x, q.z}, dx[2] = {q.y, q.w}, Bv[4] = {B.x, B.y, B.z, B.w};
        float dy[2], Cv[4];
        if (ENTERS) {
          const float2 d = *reinterpret_cast<const float2 *>(&s.dy[at]);
          const float4 C = *reinterpret_cast<const float4 *>(&s.c[i * NP + P.nl * 4]);
          dy[0] = d.x;
          dy[1] = d.y;
          Cv[0] = C.x;
          Cv[1] = C.y;
          Cv[2] = C.z;
          Cv[3] = C.w;
        }
        const float more = raised(dt, most);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          S[k] += dt[k];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = decay(dt[k], A2[k][j], more);
            h[k][j] = fmaf(e, h[k][j], dx[k] * Bv[j]);
            if (ENTERS) {
              pr[k][j] *= e;
              gs[k][j] = fmaf(pr[k][j], Cv[j] * dy[k], gs[k][j]);
            }
          }
        }
      });
    };
    for (int i = 0; i < m;) {
      if (s.s.mark[i0 + i] >= 0) {
        const int next = s.s.mark[i0 + i];
        P.read(a, next < a.n_seq ? a.h0 : nullptr, next, h);
        S[0] = S[1] = 0.f;
        reset = true;
      }
      int e = i + 1;
      while (e < m && s.s.mark[i0 + e] < 0) ++e;
      const int seg = s.s.seg[i0 + i];
      if (seg >= 0 && seg < a.n_seq) {
        if (reset) {
          scan(std::false_type(), i, e);
        } else {
          scan(std::true_type(), i, e);
          if (s.s.mark[i0 + e] >= 0 && a.dht) {
            float f[2][4];
            P.read(a, a.dht, seg, f);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) gs[k][j] = fmaf(pr[k][j], f[k][j], gs[k][j]);
          }
        }
      }
      i = e;
    }
    __syncthreads();
  }
  P.write(a, w.state, P.r, h);
  P.write(a, w.grad, P.r, gs);
  if (P.nl == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (P.ch[k] < P.nch) w.sum[(int64_t)P.r * a.D + P.c0 + P.ch[k]] = S[k];
  }
  if (P.ct == 0 && P.tid == 0) w.reset[P.r] = reset;
}

// States forwards to the ranges' starts, gradients backwards to the ranges' ends.
__global__ void k_ssm_bwd_chain(const float *A, const BwdWork w, int D, int N) {
  after_previous<true>();
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, size = (int64_t)D * N;
  if (i >= size) return;
  const bool back = blockIdx.y != 0;
  chain_ranges(back ? w.grad : w.state, w.sum, w.reset, w.n, D, size, i, (int)(i / N),
               A[i] * kLog2e, back);
}

template <int LN>
struct Tile2 {
  using Y = Lay<LN>;
  float2 pair[kBT * Y::PT];                // (dt, dt x)
  float dy[kBT * Y::PT];
  float b[kBT * Y::NP], c[kBT * Y::NP];
  float pp[kBT * Y::ST], pc[kBT * Y::ST], py[kBT * Y::ST];
  float red[kThreads / 32][kBT][2 * Y::NP];
  float bias[Y::CH], skip[Y::CH];
  RangeSegs s;
  int at[kRange + 1], tiles;
  uint32_t tmem;
};

// 8 of a thread's own fp32 values in its lane of Tensor Memory.  Whole warps.
__device__ __forceinline__ void keep8(uint32_t addr, const float (&h)[2][4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
               "f"(h[0][0]), "f"(h[0][1]), "f"(h[0][2]), "f"(h[0][3]), "f"(h[1][0]), "f"(h[1][1]),
               "f"(h[1][2]), "f"(h[1][3])
               : "memory");
}
// The read is complete after got8 of the same values.
__device__ __forceinline__ void get8(uint32_t addr, float (&h)[2][4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(h[0][0]), "=f"(h[0][1]), "=f"(h[0][2]), "=f"(h[0][3]), "=f"(h[1][0]),
                 "=f"(h[1][1]), "=f"(h[1][2]), "=f"(h[1][3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void got8(float (&h)[2][4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(h[0][0]), "+f"(h[0][1]), "+f"(h[0][2]), "+f"(h[0][3]), "+f"(h[1][0]),
                 "+f"(h[1][1]), "+f"(h[1][2]), "+f"(h[1][3])::"memory");
}

// M floats of shared memory.
template <int M>
__device__ __forceinline__ void lds(const float *p, float (&v)[M]) {
  if constexpr (M % 4 == 0) {
#pragma unroll
    for (int i = 0; i < M; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + i);
      v[i] = q.x;
      v[i + 1] = q.y;
      v[i + 2] = q.z;
      v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = p[i];
  }
}

// Sums v[0..3] (dB) and v[4..7] (dC) over the lanes that hold the same states; each lane is left
// with 8 / CW of the sums, the first being number `first`.
template <int LN>
__device__ __forceinline__ int channel_sums(float (&v)[8], int lane) {
  int first = 0;
  auto half = [&](int off, int cnt) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt) {
        const float send = up ? v[i] : v[i + cnt], keep = up ? v[i + cnt] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
    if (up) first += cnt;
  };
  half(16, 4);
  if (LN <= 8) half(8, 2);
  if (LN <= 4) half(4, 1);
  if (LN <= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return first;
}

// Pass 2.
template <typename E, int LN, bool VEC>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
    k_ssm_bwd(const SsmArgs a, const BwdWork w, int tiles_per_group) {
  after_previous();
  using Y = Lay<LN>;
  constexpr int NP = Y::NP, CH = Y::CH;
  // tokens of a tile unrolled: all of them outgrow the instruction cache (8,192 tokens of 2,048
  // channels of 16 states with the forward: 848 us, by fours 824), but for two lanes a channel,
  // where indexes in registers cost more (4,124 x 832 x 8: 176 and 198 us) than the spills of the whole
  // tile's addresses (160 to 360 bytes a thread)
  constexpr int kUnroll = LN > 2 ? 4 : kBT;
  constexpr int M = kBT * CH / kThreads;  // elements of x a thread has of a tile
  constexpr int LEFT = LN <= 4 ? 1 : LN / 4;  // channel sums left to a lane
  extern __shared__ __align__(16) char smem_raw[];
  Tile2<LN> &s = *reinterpret_cast<Tile2<LN> *>(smem_raw);
  const Place<LN> P(a, tiles_per_group);
  if (P.r == w.n) {  // initial states' gradients of the segments without tokens
    for_empty_segments(a.cu, a.n_seq, a.T, s.s.red, [&](int q) {
      const int64_t at = ((int64_t)q * a.D + P.c0) * a.N;
      for (int i = P.tid; i < P.nch * a.N; i += kThreads)
        a.dh0[at + i] = a.dht ? a.dht[at + i] : 0.f;
    });
    return;
  }
  if (P.warp == 0) {
    tc::tmem_alloc(&s.tmem, kCols);
    tc::tmem_relinquish();
  }
  const int t0 = P.r * w.range, n = min(w.range, a.T - t0);
  const int lt = P.tid / (CH / M), lc = P.tid % (CH / M) * M, nv = max(0, min(M, P.nch - lc));
  const int64_t c = P.c0 + lc;
  const E *xp = reinterpret_cast<const E *>(a.x.p) + c, *dp = reinterpret_cast<const E *>(a.dt.p) + c;
  const E *gp = reinterpret_cast<const E *>(a.dout.p) + c;
  const E *zp = a.z.p ? reinterpret_cast<const E *>(a.z.p) + c : nullptr;
  const E *Bp = reinterpret_cast<const E *>(a.B) + P.grp * a.B_sg;
  const E *Cp = reinterpret_cast<const E *>(a.C) + P.grp * a.C_sg;
  for (int i = P.tid; i < CH; i += kThreads) {
    s.bias[i] = step_bias(a.dt_bias, P.c0, P.nch, i);
    s.skip[i] = a.Dskip && i < P.nch ? a.Dskip[P.c0 + i] : 0.f;
  }
  float A2[2][4], h[2][4];
  const float most = P.decays(a, A2);
  range_segments(a, t0, n, s.s);
  if (P.warp == 0) {
    const int tiles = range_tiles(n, s.s, s.at);
    if (P.lane == 0) s.tiles = tiles;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t kept = s.tmem + ((uint32_t)(P.warp * 32) << 16);
  const uint32_t hist = kept + 8 * kKept;
  const int tiles = s.tiles;
  auto covered = [&](int i) { return s.s.seg[i] >= 0 && s.s.seg[i] < a.n_seq; };
  auto starts = [&](int q) { return s.s.mark[s.at[q]] >= 0; };

  Elems<E, M> rx, rd, rg, rz;
  BcTile<E, NP, kBT, VEC> rb, rc;
  // a tile's elements; a token without a segment, and one past the tile, is neutral: zeros
  auto fetch = [&](int q, bool all) {
    const int i0 = s.at[q], m = s.at[q + 1] - i0, live = covered(i0) ? m : 0;
    const int64_t t = t0 + i0 + lt;
    const int k = lt < live ? nv : 0;
    rx = ldm<VEC, E, M>(xp + t * a.x.st, k);
    rd = ldm<VEC, E, M>(dp + t * a.dt.st, k);
    rb.fetch(Bp, a.B_st, t0 + i0, t0 + i0 + live, a.N);
    if (all) {
      rg = ldm<VEC, E, M>(gp + t * a.dout.st, k);
      if (zp) rz = ldm<VEC, E, M>(zp + t * a.z.st, k);
      rc.fetch(Cp, a.C_st, t0 + i0, t0 + i0 + live, a.N);
    }
  };
  auto put = [&](bool in) {
    if (in) {
      float b[M];
      lds<M>(&s.bias[lc], b);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float v = ld1(&rd.v[i]) + b[i];
        if (a.softplus) v = softplusf(v);
        s.pair[Y::pair_at(lt, lc + i)] = make_float2(v, v * ld1(&rx.v[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < M; ++i) s.pair[Y::pair_at(lt, lc + i)] = make_float2(0.f, 0.f);
    }
    rb.put(s.b);
  };
  auto advance = [&](int i, float (&v)[2][4]) {  // the state after token i of the tile
    const float4 q = *reinterpret_cast<const float4 *>(&s.pair[i * Y::PT + P.pair]);
    const float4 B = *reinterpret_cast<const float4 *>(&s.b[i * NP + P.nl * 4]);
    const float dt[2] = {q.x, q.z}, dx[2] = {q.y, q.w}, Bv[4] = {B.x, B.y, B.z, B.w};
    const float more = raised(dt, most);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[k][j] = fmaf(decay(dt[k], A2[k][j], more), v[k][j], dx[k] * Bv[j]);
    }
  };

  // the sweep: the state before each tile that continues a segment
  P.read(a, P.r > 0 && covered(0) ? w.state : nullptr, P.r, h);
  fetch(0, false);
  for (int q = 0; q < tiles; ++q) {
    const int i0 = s.at[q];
    if (starts(q))
      P.read(a, covered(i0) ? a.h0 : nullptr, s.s.seg[i0], h);
    else
      keep8(kept + (i0 / kBT) * 8, h);
    if (q + 1 == tiles) break;
    const bool on = !starts(q + 1);  // the next tile goes on from here
    if (on) {
      put(covered(i0) && lt < s.at[q + 1] - i0);
    }
    fetch(q + 1, false);
    if (on) {
      __syncthreads();
#pragma unroll kUnroll
      for (int i = 0; i < kBT; ++i) advance(i, h);
      __syncthreads();
    }
  }
  tc::tmem_st_wait();

  float g[2][4], dA[2][4], sd[M], sb[M];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) dA[k][j] = 0.f;
#pragma unroll
  for (int i = 0; i < M; ++i) sd[i] = sb[i] = 0.f;
  // the gradient that arrives at the range's end
  P.read(a, w.n > 1 ? w.grad : nullptr, P.r, g);
  fetch(tiles - 1, true);
  for (int q = tiles - 1; q >= 0; --q) {
    const int i0 = s.at[q], m = s.at[q + 1] - i0;
    const bool live = covered(i0), in = live && lt < m, first = starts(q);
    const int64_t t = t0 + i0 + lt;
    if (s.s.mark[i0 + m] >= 0) P.read(a, live ? a.dht : nullptr, s.s.seg[i0], g);
    put(in);
    if (in) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float dy = ld1(&rg.v[i]);
        if (zp) {
          const float z = ld1(&rz.v[i]);
          dy *= z * sigmoidf(z);
        }
        s.dy[Y::pair_at(lt, lc + i)] = dy;
      }
    } else {
#pragma unroll
      for (int i = 0; i < M; ++i) s.dy[Y::pair_at(lt, lc + i)] = 0.f;
    }
    rc.put(s.c);
    const Elems<E, M> cx = rx, cd = rd, cg = rg, cz = rz;
    if (q > 0) fetch(q - 1, true);
    __syncthreads();
    float now[2][4], before[2][4], next[2][4];  // states after token i, before it, before that
    if (first) {
      P.read(a, live ? a.h0 : nullptr, s.s.seg[i0], before);
    } else {
      get8(kept + (i0 / kBT) * 8, before);
      got8(before);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) now[k][j] = before[k][j];
    keep8(hist, now);
#pragma unroll kUnroll
    for (int i = 0; i < kBT; ++i) {
      advance(i, now);
      if (i + 1 < kBT) keep8(hist + (i + 1) * 8, now);
      if (zp) {
        const float4 C = *reinterpret_cast<const float4 *>(&s.c[i * NP + P.nl * 4]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          s.py[Y::part_at(i, P.ch[k]) + P.nl] =
              fmaf(now[k][0], C.x, fmaf(now[k][1], C.y, fmaf(now[k][2], C.z, now[k][3] * C.w)));
      }
    }
    tc::tmem_st_wait();
    get8(hist + (kBT - 1) * 8, before);
    got8(before);
#pragma unroll kUnroll
    for (int i = kBT - 1; i >= 0; --i) {
      if (i > 0) get8(hist + (i - 1) * 8, next);
      const int at = i * Y::PT + P.pair;
      const float4 v = *reinterpret_cast<const float4 *>(&s.pair[at]);
      const float2 dyv = *reinterpret_cast<const float2 *>(&s.dy[at]);
      const float4 B = *reinterpret_cast<const float4 *>(&s.b[i * NP + P.nl * 4]);
      const float4 C = *reinterpret_cast<const float4 *>(&s.c[i * NP + P.nl * 4]);
      const float dt[2] = {v.x, v.z}, dx[2] = {v.y, v.w}, dy[2] = {dyv.x, dyv.y};
      const float Bv[4] = {B.x, B.y, B.z, B.w}, Cv[4] = {C.x, C.y, C.z, C.w};
      const float more = raised(dt, most);
      float bc[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float p = 0.f, cs = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[k][j] = fmaf(Cv[j], dy[k], g[k][j]);
          bc[j] = k ? fmaf(dx[k], g[k][j], bc[j]) : dx[k] * g[k][j];
          bc[4 + j] = k ? fmaf(dy[k], now[k][j], bc[4 + j]) : dy[k] * now[k][j];
          p = j ? fmaf(g[k][j], Bv[j], p) : g[k][j] * Bv[j];
          g[k][j] *= decay(dt[k], A2[k][j], more);
          const float cr = g[k][j] * before[k][j];
          dA[k][j] = fmaf(dt[k], cr, dA[k][j]);
          cs = j ? fmaf(cr, A2[k][j], cs) : cr * A2[k][j];
        }
        const int o = Y::part_at(i, P.ch[k]) + P.nl;
        s.pp[o] = p;
        s.pc[o] = cs;
      }
      const int f = channel_sums<LN>(bc, P.lane);
      if (LN > 2 || !(P.lane & 2)) {
#pragma unroll
        for (int u = 0; u < LEFT; ++u)
          s.red[P.warp][i][((f + u) >> 2) * NP + P.nl * 4 + ((f + u) & 3)] = bc[u];
      }
      if (i > 0) {
        got8(next);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            now[k][j] = before[k][j];
            before[k][j] = next[k][j];
          }
      }
    }
    if (first && live && a.dh0) P.write(a, a.dh0, s.s.seg[i0], g);
    __syncthreads();
    if (lt < m) {
      float ox[M], od[M], oz[M];
      if (in) {
        float skip[M], b[M];
        lds<M>(&s.skip[lc], skip);
        lds<M>(&s.bias[lc], b);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const int o = Y::part_at(lt, lc + i), at = Y::pair_at(lt, lc + i);
          const float p = sum_parts<LN>(&s.pp[o]), cs = sum_parts<LN>(&s.pc[o]) * kLn2;
          const float x = ld1(&cx.v[i]), dt = s.pair[at].x, dy = s.dy[at];
          if (zp) {
            const float z = ld1(&cz.v[i]), sg = sigmoidf(z);
            oz[i] = ld1(&cg.v[i]) * fmaf(skip[i], x, sum_parts<LN>(&s.py[o])) * dsilu(z, sg);
          }
          ox[i] = fmaf(dt, p, skip[i] * dy);
          od[i] = fmaf(x, p, cs);
          if (a.softplus) od[i] *= sigmoidf(ld1(&cd.v[i]) + b[i]);
          sd[i] = fmaf(dy, x, sd[i]);
          sb[i] += od[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < M; ++i) ox[i] = od[i] = oz[i] = 0.f;
      }
      stm<VEC, E, M>(reinterpret_cast<E *>(a.dx.p) + t * a.dx.st + c, ox, nv);
      stm<VEC, E, M>(reinterpret_cast<E *>(a.ddt.p) + t * a.ddt.st + c, od, nv);
      if (zp) stm<VEC, E, M>(reinterpret_cast<E *>(a.dz.p) + t * a.dz.st + c, oz, nv);
    }
    float *bc = w.bc + ((int64_t)P.ct * a.T + t0 + i0) * (2 * NP);
    for (int e = P.tid; e < m * 2 * NP; e += kThreads) {
      const int i = e / (2 * NP), o = e % (2 * NP);
      bc[e] = (s.red[0][i][o] + s.red[1][i][o]) + (s.red[2][i][o] + s.red[3][i][o]);
    }
    __syncthreads();
  }
  P.write(a, w.state, P.r, dA);
  // dD and ddt_bias: over the threads that hold the same channels
  float *part = s.pp;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    part[lt * CH + lc + i] = sd[i];
    part[(kBT + lt) * CH + lc + i] = sb[i];
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (P.warp == 0) tc::tmem_dealloc(s.tmem, kCols);
  for (int e = P.tid; e < P.nch; e += kThreads) {
    float u = 0.f, v = 0.f;
#pragma unroll
    for (int i = 0; i < kBT; ++i) {
      u += part[i * CH + e];
      v += part[(kBT + i) * CH + e];
    }
    w.pd[(int64_t)P.r * a.D + P.c0 + e] = u;
    w.pb[(int64_t)P.r * a.D + P.c0 + e] = v;
  }
}

// out[i] = sum over n parts of in[r * size + i], for up to three arrays (blockIdx.y): 32 columns a
// block, its 8 warps taking every 8th part.
struct PartSums {
  const float *in[3];
  float *out[3];
  int64_t size[3];
  int n;
};
__global__ void __launch_bounds__(256) k_ssm_part_sums(const PartSums p) {
  after_previous<true>();
  __shared__ float part[8][32];
  const int y = blockIdx.y, lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t i = blockIdx.x * (int64_t)32 + lane;
  const int64_t size = y == 0 ? p.size[0] : y == 1 ? p.size[1] : p.size[2];
  const float *in = y == 0 ? p.in[0] : y == 1 ? p.in[1] : p.in[2];
  float *out = y == 0 ? p.out[0] : y == 1 ? p.out[1] : p.out[2];
  if (!out || blockIdx.x * (int64_t)32 >= size) return;
  float s[4] = {0, 0, 0, 0};
  if (i < size) {
    int r = k;
    for (; r + 24 < p.n; r += 32)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += in[(r + 8 * u) * size + i];
    for (; r < p.n; r += 8) s[0] += in[r * size + i];
  }
  part[k][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (k == 0 && i < size) {
    float v = part[0][lane];
#pragma unroll
    for (int u = 1; u < 8; ++u) v += part[u][lane];
    out[i] = v;
  }
}

// dB and dC: over the channel tiles of a group.
template <typename E>
__global__ void k_ssm_bc_sums(const float *bc, int64_t T, int G, int N, int NP, int tpg, E *dB,
                              E *dC) {
  after_previous();
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int64_t row = (int64_t)G * 2 * N, t = i / row;  // of a token: past 32 bits for many groups
  if (t >= T) return;
  const int64_t part = (i - t * row) / N;
  const int m = (int)(i - t * row - part * N);
  const int grp = (int)(part >> 1), kind = (int)(part & 1);  // 0: dB, 1: dC
  const float *q = bc + ((int64_t)grp * tpg * T + t) * (2 * NP) + kind * NP + m;
  const int64_t st = T * (2 * NP);
  float s[4] = {0, 0, 0, 0};
  int r = 0;
  for (; r + 4 <= tpg; r += 4)
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += q[(r + u) * st];
  for (; r < tpg; ++r) s[0] += q[r * st];
  st1((kind ? dC : dB) + (t * G + grp) * N + m, (s[0] + s[1]) + (s[2] + s[3]));
}

BwdWork carve_bwd(void *work, int64_t T, int32_t D, int32_t N, int32_t G) {
  BwdWork w{};
  const int LN = lanes_for(N);
  const int64_t ctiles = channel_tiles(D, G, LN);
  w.range = kRange;
  while (w.range > kLeast && ceil_div64(T, w.range / 2) * ctiles <= sm_count() * kBwdCtas &&
         ceil_div64(T, w.range / 2) <= kMostShort)
    w.range /= 2;
  w.n = (int)ceil_div64(T, w.range);
  const int64_t R = w.n < 1 ? 1 : w.n;
  char *p = reinterpret_cast<char *>(work);
  size_t off = 0;
  auto take = [&](int64_t floats) {
    float *q = reinterpret_cast<float *>(p + off);
    off += align256((size_t)floats * 4);
    return q;
  };
  w.state = take(R * D * N);
  w.grad = take(R * D * N);
  w.sum = take(R * D);
  w.pd = take(R * D);
  w.pb = take(R * D);
  w.reset = reinterpret_cast<int *>(take(R));
  w.bc = take(ctiles * T * 2 * 4 * LN);
  w.bytes = off;
  return w;
}

template <typename E, int LN, bool VEC>
cudaError_t run_bwd(const SsmArgs &a, cudaStream_t stream) {
  const int tpg = (int)ceil_div64(a.D / a.G, Lay<LN>::CH), ctiles = tpg * a.G;
  const BwdWork w = carve_bwd(a.work, a.T, a.D, a.N, a.G);
  constexpr int smem1 = (int)sizeof(Tile1<LN>) + 4 * 16 * TileRing<E, VEC, 2>::kSlots;
  constexpr int smem2 = (int)sizeof(Tile2<LN>);
  cudaError_t e = cudaFuncSetAttribute(k_ssm_bwd<E, LN, VEC>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem2);
  if (e != cudaSuccess) return e;
  if (smem1 > 48 * 1024 &&
      (e = cudaFuncSetAttribute(k_ssm_bwd_ends<E, LN, VEC>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, smem1)) != cudaSuccess)
    return e;
  const int64_t size = (int64_t)a.D * a.N;
  if (w.n > 1) {
    if ((e = launch(k_ssm_bwd_ends<E, LN, VEC>, (unsigned)((int64_t)ctiles * w.n), kThreads, smem1,
                    stream, a, w, tpg)) != cudaSuccess)
      return e;
    if ((e = launch(k_ssm_bwd_chain, dim3((unsigned)ceil_div64(size, 128), 2), 128, 0, stream, a.A,
                    w, a.D, a.N)) != cudaSuccess)
      return e;
  }
  const int64_t blocks = (int64_t)ctiles * (w.n + (a.dh0 ? 1 : 0));
  if (blocks > 0) {
    if ((e = launch(k_ssm_bwd<E, LN, VEC>, (unsigned)blocks, kThreads, smem2, stream, a, w,
                    tpg)) != cudaSuccess)
      return e;
  }
  const PartSums ps{{w.state, w.pd, w.pb}, {a.dA, a.dD, a.ddt_bias}, {size, a.D, a.D}, w.n};
  if ((e = launch(k_ssm_part_sums, dim3((unsigned)ceil_div64(size, 32), 3), 256, 0, stream, ps)) !=
          cudaSuccess ||
      a.T == 0)
    return e;
  return launch(k_ssm_bc_sums<E>, (unsigned)ceil_div64((int64_t)a.T * a.G * 2 * a.N, 256), 256, 0,
                stream, w.bc, a.T, a.G, a.N, Lay<LN>::NP, tpg, reinterpret_cast<E *>(a.dB),
                reinterpret_cast<E *>(a.dC));
}

template <typename E>
cudaError_t by_lanes(const SsmArgs &a, bool vec, cudaStream_t stream) {
  switch (lanes_for(a.N)) {
    case 2: return vec ? run_bwd<E, 2, true>(a, stream) : run_bwd<E, 2, false>(a, stream);
    case 4: return vec ? run_bwd<E, 4, true>(a, stream) : run_bwd<E, 4, false>(a, stream);
    case 8: return vec ? run_bwd<E, 8, true>(a, stream) : run_bwd<E, 8, false>(a, stream);
    default: return vec ? run_bwd<E, 16, true>(a, stream) : run_bwd<E, 16, false>(a, stream);
  }
}

}  // namespace
}  // namespace ssm

size_t ssm_bwd_workspace(int64_t T, int32_t D, int32_t N, int32_t G) {
  return ssm::carve_bwd(nullptr, T, D, N, G).bytes;
}

cudaError_t launch_ssm_bwd(const SsmArgs &args, cudaStream_t stream) {
  using namespace ssm;
  SsmArgs a = args;
  a.n4 = states_ok(a);
  const bool vec = (a.D / a.G) % 8 == 0 && rows_ok(a.x, a.f32) && rows_ok(a.dt, a.f32) &&
                   rows_ok(a.z, a.f32) && rows_ok(a.dout, a.f32) && rows_ok(a.dx, a.f32) &&
                   rows_ok(a.ddt, a.f32) && rows_ok(a.dz, a.f32) && bc_ok(a);
  return a.f32 ? by_lanes<float>(a, vec, stream) : by_lanes<__nv_bfloat16>(a, vec, stream);
}

}  // namespace gdr
