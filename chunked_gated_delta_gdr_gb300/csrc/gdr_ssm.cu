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
// and keeps the state at its end and the sum of dt (a range's decay is e^{A sum dt}); a short
// kernel chains these ends over the ranges; pass 2 runs each range from its true state and writes
// y.  When one range is enough, only pass 2 runs.
#include "gdr_ssm.cuh"

namespace gdr {
namespace ssm {
namespace {

using namespace mix;

struct Ranges {
  int range, n;      // tokens of a range, ranges
  float *state;      // [n][D][N]: pass 1 the state at the end, after the chain the one at the start
  float *sum;        // [n][D]: sum of dt from the last segment start in the range (or its start)
  int *reset;        // [n]: a segment starts in the range
};

template <int LN>
struct Tile {  // shared memory of one tile
  using Y = Lay<LN>;
  float2 pair[Y::L * Y::CH];  // (dt, dt x)
  float b[Y::L * Y::NP], c[Y::L * Y::NP];
  float part[Y::L * Y::CH * LN];
  int mark[Y::L + 1], seg[Y::L], any, same;
  int red[64];
};

// One range.  ENDS: pass 1 (no y).  VEC: every group of 8 channels is whole and 16-byte aligned.
template <typename E, int LN, bool ENDS, bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_ssm_fwd(const SsmArgs a, const Ranges rg, int tiles_per_group) {
  using Y = Lay<LN>;
  constexpr int L = Y::L, NP = Y::NP, CH = Y::CH;
  constexpr int NB = (L * NP + kThreads - 1) / kThreads;  // elements of B a thread loads for a tile
  extern __shared__ __align__(16) char smem_raw[];
  Tile<LN> &s = *reinterpret_cast<Tile<LN> *>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctiles = tiles_per_group * a.G;
  const int ct = blockIdx.x % ctiles, r = blockIdx.x / ctiles;
  const int grp = ct / tiles_per_group, Dg = a.D / a.G;
  const int c0 = grp * Dg + ct % tiles_per_group * CH;
  const int nch = min(CH, (grp + 1) * Dg - c0);
  const int N = a.N;

  if (!ENDS && r == rg.n) {  // final states of the segments without tokens
    for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
      const int64_t at = ((int64_t)n * a.D + c0) * N;
      for (int i = tid; i < nch * N; i += kThreads) a.ht[at + i] = a.h0 ? a.h0[at + i] : 0.f;
    });
    return;
  }
  const int t0 = r * rg.range, t1 = min(a.T, t0 + rg.range);

  // this thread's states: channels ch[k], states 4 nl .. 4 nl + 3
  const int nl = lane % LN, cl = lane / LN;
  float A2[2][4], h[2][4], S[2] = {0.f, 0.f};
  int ch[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    ch[k] = Y::channel(warp, lane, k);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = nl * 4 + j;
      A2[k][j] = (ch[k] < nch && n < N) ? a.A[(int64_t)(c0 + ch[k]) * N + n] * kLog2e : 0.f;
      h[k][j] = 0.f;
    }
  }
  auto read_state = [&](const float *p, int64_t row) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nl * 4 + j;
        h[k][j] = (p && ch[k] < nch && n < N) ? p[(row * a.D + c0 + ch[k]) * N + n] : 0.f;
      }
  };
  auto write_state = [&](float *p, int64_t row) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nl * 4 + j;
        if (ch[k] < nch && n < N) p[(row * a.D + c0 + ch[k]) * N + n] = h[k][j];
      }
  };

  // this thread's 8 elements of a tile of x, dt, z and y
  const int lt = tid / Y::CG, lc = tid % Y::CG * 8, nv = max(0, min(8, nch - lc));
  const E *xp = reinterpret_cast<const E *>(a.x.p) + c0 + lc;
  const E *dp = reinterpret_cast<const E *>(a.dt.p) + c0 + lc;
  const E *zp = a.z.p ? reinterpret_cast<const E *>(a.z.p) + c0 + lc : nullptr;
  E *yp = reinterpret_cast<E *>(a.y.p) + c0 + lc;
  const E *Bp = reinterpret_cast<const E *>(a.B) + grp * a.B_sg;
  const E *Cp = reinterpret_cast<const E *>(a.C) + grp * a.C_sg;
  float bias[8], skip[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bias[i] = (a.dt_bias && i < nv) ? a.dt_bias[c0 + lc + i] : 0.f;
    skip[i] = (!ENDS && a.Dskip && i < nv) ? a.Dskip[c0 + lc + i] : 0.f;
  }

  Raw8<E> rx, rd, rz = zero8<E>();
  E rb[NB], rc[NB];
  auto fetch = [&](int tb) {
    const int t = tb + lt, n = t < t1 ? nv : 0;
    rx = ld8<VEC>(xp + (int64_t)t * a.x.st, n);
    rd = ld8<VEC>(dp + (int64_t)t * a.dt.st, n);
    if (!ENDS && zp) rz = ld8<VEC>(zp + (int64_t)t * a.z.st, n);
  };
  auto fetch_bc = [&](int tb) {
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int e = tid + q * kThreads, t = tb + e / NP, n = e % NP;
      const bool ok = e < L * NP && t < t1 && n < N;
      rb[q] = ok ? Bp[t * a.B_st + n] : E(0.f);
      if (!ENDS) rc[q] = ok ? Cp[t * a.C_st + n] : E(0.f);
    }
  };

  SegCursor cursor = seg_find(a.cu, a.n_seq, a.T, t0, s.red);
  int seg = cursor.j - 1;
  bool reset = false;
  if (!ENDS && r > 0 && seg >= 0 && seg < a.n_seq) read_state(rg.state, r);
  fetch(t0);
  fetch_bc(t0);

  // the scan of tokens [i0, i1) of the tile
  auto scan = [&](int i0, int i1) {
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const float4 d = *reinterpret_cast<const float4 *>(
          &s.pair[i * CH + Y::pair_slot(i, warp, cl) * 2]);
      const float4 B = *reinterpret_cast<const float4 *>(&s.b[i * NP + nl * 4]);
      const float dt[2] = {d.x, d.z}, dx[2] = {d.y, d.w}, Bv[4] = {B.x, B.y, B.z, B.w};
      float4 C;
      if (!ENDS) C = *reinterpret_cast<const float4 *>(&s.c[i * NP + nl * 4]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[k][j] = fmaf(ex2(dt[k] * A2[k][j]), h[k][j], dx[k] * Bv[j]);
        if (ENDS)
          S[k] += dt[k];
        else
          s.part[Y::part_at(i, ch[k]) + nl] =
              fmaf(h[k][0], C.x, h[k][1] * C.y) + fmaf(h[k][2], C.z, h[k][3] * C.w);
      }
    }
  };

  for (int tb = t0; tb < t1; tb += L) {
    const int n = min(L, t1 - tb);
    // this tile's elements into shared memory, the next tile's from global memory
    float x[8], d[8], z[8];
    unpack8(rx, x);
    unpack8(rd, d);
    unpack8(rz, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = d[i] + bias[i];
      if (a.softplus) v = softplusf(v);
      s.pair[Y::pair_at(lt, lc + i)] = make_float2(v, v * x[i]);
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int e = tid + q * kThreads;
      if (e < L * NP) {
        s.b[e] = ld1(&rb[q]);
        if (!ENDS) s.c[e] = ld1(&rc[q]);
      }
    }
    if (warp == 0) {
      const int carry = cursor.j - 1;
      const bool any = seg_marks(a.cu, a.n_seq, a.T, tb, n, s.mark, cursor);
      if (any) {
        int base = carry;
        for (int i0 = 0; i0 < L; i0 += 32) {
          int v = i0 + lane < n ? s.mark[i0 + lane] : -1;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = max(v, u);
          }
          v = max(v, base);
          if (i0 + lane < L) s.seg[i0 + lane] = v;
          base = __shfl_sync(0xffffffffu, v, 31);
        }
      }
      if (lane == 0) {
        s.any = any;
        s.same = carry;
      }
    }
    if (tb + L < t1) {
      fetch(tb + L);
      fetch_bc(tb + L);
    }
    __syncthreads();
    const bool any = s.any;
    if (!any) {
      if (seg >= 0 && seg < a.n_seq) scan(0, n);
    } else {
      for (int i = 0; i < n;) {
        if (s.mark[i] >= 0) {
          seg = s.mark[i];
          if (seg < a.n_seq) read_state(a.h0, seg);
          S[0] = S[1] = 0.f;
          reset = true;
        }
        int e = i + 1;
        while (e < n && s.mark[e] < 0) ++e;
        if (seg >= 0 && seg < a.n_seq) {
          scan(i, e);
          if (!ENDS && a.ht && s.mark[e] >= 0) write_state(a.ht, seg);
        }
        i = e;
      }
    }
    __syncthreads();
    if (!ENDS) {
      const int own = any ? s.seg[lt] : s.same;
      if (lt < n && own >= 0 && own < a.n_seq) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = fmaf(skip[i], x[i], sum_parts<LN>(&s.part[Y::part_at(lt, lc + i)]));
          if (zp) v[i] *= z[i] * sigmoidf(z[i]);
        }
        st8<VEC>(yp + (int64_t)(tb + lt) * a.y.st, pack8(v, E{}), nv);
      }
      __syncthreads();
    }
  }
  if (ENDS) {
    write_state(rg.state, r);
    if (nl == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (ch[k] < nch) rg.sum[(int64_t)r * a.D + c0 + ch[k]] = S[k];
    }
    if (ct == 0 && tid == 0) rg.reset[r] = reset;
  }
}

// The state at the start of each range from the ends of pass 1: next = e^{A sum} state + end, or
// the end alone where a segment starts in the range.
__global__ void k_ssm_chain(const float *A, const Ranges rg, int D, int N) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, size = (int64_t)D * N;
  if (i >= size) return;
  const float A2 = A[i] * kLog2e;
  const int d = (int)(i / N);
  float cur = 0.f;
  constexpr int U = 8;
  for (int r0 = 0; r0 < rg.n; r0 += U) {
    float end[U], sum[U];
    int rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool ok = r0 + u < rg.n - 1;  // the last range's end goes nowhere
      end[u] = ok ? rg.state[(r0 + u) * size + i] : 0.f;
      sum[u] = ok ? rg.sum[(int64_t)(r0 + u) * D + d] : 0.f;
      rs[u] = ok ? rg.reset[r0 + u] : 1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u < rg.n) {
        rg.state[(r0 + u) * size + i] = cur;
        cur = rs[u] ? end[u] : fmaf(ex2(A2 * sum[u]), cur, end[u]);
      }
  }
}

// One token for each row: state slot idx[row] in place.  A thread holds 4 states of one channel.
template <typename E, int LN>
__global__ void __launch_bounds__(kThreads)
    k_ssm_step(const SsmArgs a, float *state, int slots, const int32_t *idx, int cblocks) {
  constexpr int CB = kThreads / LN;  // channels of a block
  const int row = blockIdx.x / cblocks, d = blockIdx.x % cblocks * CB + threadIdx.x / LN;
  const int nl = threadIdx.x % LN, N = a.N;
  const bool in = d < a.D;
  const int slot = idx ? idx[row] : row;
  E *y = reinterpret_cast<E *>(a.y.p) + (int64_t)row * a.y.st + d;
  if (slot < 0 || slot >= slots) {
    if (in && nl == 0) st1(y, 0.f);
    return;
  }
  float part = 0.f, x = 0.f;
  if (in) {
    const int grp = d / (a.D / a.G);
    const E *B = reinterpret_cast<const E *>(a.B) + row * a.B_st + grp * a.B_sg;
    const E *C = reinterpret_cast<const E *>(a.C) + row * a.C_st + grp * a.C_sg;
    float *s = state + ((int64_t)slot * a.D + d) * N;
    const float *A = a.A + (int64_t)d * N;
    x = ld1(reinterpret_cast<const E *>(a.x.p) + (int64_t)row * a.x.st + d);
    float dt = ld1(reinterpret_cast<const E *>(a.dt.p) + (int64_t)row * a.dt.st + d);
    if (a.dt_bias) dt += a.dt_bias[d];
    if (a.softplus) dt = softplusf(dt);
    const float dx = dt * x;
    const int n0 = nl * 4;
    if (N % 4 == 0) {
      if (n0 < N) {
        const float4 h = *reinterpret_cast<const float4 *>(s + n0);
        const float4 Av = *reinterpret_cast<const float4 *>(A + n0);
        float4 o;
        o.x = fmaf(ex2(dt * (Av.x * kLog2e)), h.x, dx * ld1(B + n0));
        o.y = fmaf(ex2(dt * (Av.y * kLog2e)), h.y, dx * ld1(B + n0 + 1));
        o.z = fmaf(ex2(dt * (Av.z * kLog2e)), h.z, dx * ld1(B + n0 + 2));
        o.w = fmaf(ex2(dt * (Av.w * kLog2e)), h.w, dx * ld1(B + n0 + 3));
        *reinterpret_cast<float4 *>(s + n0) = o;
        part = fmaf(o.x, ld1(C + n0), o.y * ld1(C + n0 + 1)) +
               fmaf(o.z, ld1(C + n0 + 2), o.w * ld1(C + n0 + 3));
      }
    } else {
      for (int n = n0; n < min(N, n0 + 4); ++n) {
        const float o = fmaf(ex2(dt * (A[n] * kLog2e)), s[n], dx * ld1(B + n));
        s[n] = o;
        part = fmaf(o, ld1(C + n), part);
      }
    }
  }
#pragma unroll
  for (int o = LN / 2; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (in && nl == 0) {
    if (a.Dskip) part = fmaf(a.Dskip[d], x, part);
    if (a.z.p) {
      const float z = ld1(reinterpret_cast<const E *>(a.z.p) + (int64_t)row * a.z.st + d);
      part *= z * sigmoidf(z);
    }
    st1(y, part);
  }
}

template <int LN>
int fwd_range(int64_t T, int D, int G) {
  return range_tokens(T, channel_tiles(D, G, LN), Lay<LN>::L, 8, 128);
}

struct Carve {
  Ranges rg;
  size_t bytes;
};
Carve carve(void *work, int64_t T, int32_t D, int32_t N, int range) {
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

int range_for(int64_t T, int32_t D, int32_t N, int32_t G) {
  switch (lanes_for(N)) {
    case 2: return fwd_range<2>(T, D, G);
    case 4: return fwd_range<4>(T, D, G);
    case 8: return fwd_range<8>(T, D, G);
    default: return fwd_range<16>(T, D, G);
  }
}

template <typename K>
cudaError_t allow_smem(K k, int bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename E, int LN, bool VEC>
cudaError_t run_fwd(const SsmArgs &a, cudaStream_t stream) {
  const int tpg = (int)ceil_div64(a.D / a.G, Lay<LN>::CH), ctiles = tpg * a.G;
  const Carve c = carve(a.work, a.T, a.D, a.N, fwd_range<LN>(a.T, a.D, a.G));
  constexpr int smem = (int)sizeof(Tile<LN>);
  cudaError_t e;
  if (smem > 48 * 1024) {
    if ((e = allow_smem(k_ssm_fwd<E, LN, true, VEC>, smem)) != cudaSuccess) return e;
    if ((e = allow_smem(k_ssm_fwd<E, LN, false, VEC>, smem)) != cudaSuccess) return e;
  }
  if (c.rg.n > 1) {
    k_ssm_fwd<E, LN, true, VEC>
        <<<(unsigned)((int64_t)ctiles * (c.rg.n - 1)), kThreads, smem, stream>>>(a, c.rg, tpg);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k_ssm_chain<<<(unsigned)ceil_div64((int64_t)a.D * a.N, 128), 128, 0, stream>>>(a.A, c.rg, a.D,
                                                                                   a.N);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int64_t blocks = (int64_t)ctiles * (c.rg.n + (a.ht ? 1 : 0));
  if (blocks == 0) return cudaSuccess;
  k_ssm_fwd<E, LN, false, VEC><<<(unsigned)blocks, kThreads, smem, stream>>>(a, c.rg, tpg);
  return cudaGetLastError();
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool rows_ok(const Mat &m, bool f32) {
  return !m.p || (aligned16(m.p) && m.st % (f32 ? 4 : 8) == 0);
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
  const int cblocks = (int)ceil_div64(a.D, kThreads / LN);
  k_ssm_step<E, LN><<<(unsigned)((int64_t)cblocks * a.T), kThreads, 0, stream>>>(a, state, slots,
                                                                                 idx, cblocks);
  return cudaGetLastError();
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
  return ssm::carve(nullptr, T, D, N, ssm::range_for(T, D, N, G)).bytes;
}

cudaError_t launch_ssm_fwd(const SsmArgs &a, cudaStream_t stream) {
  using namespace ssm;
  const bool vec = (a.D / a.G) % 8 == 0 && rows_ok(a.x, a.f32) && rows_ok(a.dt, a.f32) &&
                   rows_ok(a.z, a.f32) && rows_ok(a.y, a.f32);
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
