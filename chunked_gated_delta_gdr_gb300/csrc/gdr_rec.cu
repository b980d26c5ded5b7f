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
// One pass over the data: a cluster of blocks walks along the tokens of 64, 32 or 16 channels, all of them
// with the same step.  A lane holds two channels of eight neighbouring tokens in registers and reduces
// them to one pair (A, U): h_out = A h_in + U.  The pairs of a block's warps meet in its shared memory,
// those of the cluster's blocks in everyone's (distributed shared memory), and each lane then runs
// through its tokens from its true state.  The alternative, ranges that are scanned from a zero state,
// chained and scanned again, reads and computes everything twice.
//
// What bounds it: latency, before HBM.  32,768 x 4,096 in bf16 with an input gate: 260 us for 158 of bytes
// (60 % of a copy's rate); 16 warps an SM, as many as 128 registers a thread leave, issue in about half of
// the cycles: most of what they wait for is an instruction's own latency (decay, normaliser and two
// gates are 3 exponentials, a reciprocal and a square root a token) and the chain's meetings.  The chain
// behind the next step's products instead of between a step's two halves, rows by asynchronous copies,
// packed products and counted stores together: 460 -> 250 us (the series of decays next to 1 then added 14).
#include "gdr_rec.cuh"

namespace gdr {
namespace mix {
namespace {

// ------------------------------------------------------------------ forward

// A warp's tokens of a step: decays and inputs, and what starts among them.
struct Step {
  f2 at[kK], u[kK];
  uint32_t starts;  // bit k: a segment starts with token k
  Map front;        // of the groups before the lane's
};

// OUT: y is written (without it only the kept states: the backward's first pass).
template <typename E, int MODE, int SUB, bool OUT, bool NORM>
__global__ void __launch_bounds__(kP * 32, 2) k_rec_fwd(const RecArgs a) {
  after_previous();
  constexpr int kTile = tile_of(SUB), L = 32 / SUB;
  constexpr bool VEC = MODE > 0;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ Shared<SUB> s;
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int rank = cluster_rank(), size = cluster_size();
  const int cb = (int)(blockIdx.x / size) * channels_of(SUB), c0 = cb + place_of<SUB>(lane) * 2;
  const int nv = max(0, min(2, a.D - c0));
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
    bool lost = false;
    for (int step = 0; step < steps; ++step) {
      meet(kMaps + (step & 1));
      const bool any2 = look(step + 2);
      chain<false, SUB>(s, step, any0, carry, lost);
      any0 = any1;
      any1 = any2;
      __syncwarp();
      arrive(kFronts + (step & 1));
    }
  } else {
    const f2 A2 = mul2(load_state(a.A + c0, nv), both(kLog2e));
    using In = Tokens<E, MODE, 3, 2, SUB>;
    In in{{reinterpret_cast<const E *>(a.x.p) + cb, reinterpret_cast<const E *>(a.r.p) + cb,
           a.i.p ? reinterpret_cast<const E *>(a.i.p) + cb : nullptr},
          {a.x.st, a.r.st, a.i.st},
          raw + warp * 2 * In::kPlace, lane, a.D - cb, nv, a.T};
    const bool gate = a.i.p;
    E *y = reinterpret_cast<E *>(a.y.p) + c0;
    const int first = rank * kTile + warp * kK * SUB, mine0 = warp * kK * SUB + group_of<SUB>(lane) * kK;
    in.start(first);
    in.issue(0, first, stride);
    in.issue(1, first + stride, stride);
    cluster_arrive();
    cluster_wait();

    auto hold = [&](int step, Step &v) {  // the step's tokens, and their map for the chain
      const int place = step & 1, tw = first + step * stride + group_of<SUB>(lane) * kK, left = a.T - tw;
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
          const f2 x = in.get(place, 0, k, tw + k), r = in.get(place, 1, k, tw + k);
          if (gate) {
            f2 sr, si;
            sigmoids_apart(r, in.get(place, 2, k, tw + k), sr, si);
            make(k, sr, mul2(si, x));
          } else {
            make(k, sigmoid2(r), x);
          }
        }
      }
      // segments that start among the tokens: their state goes into the first one
      const bool any = s.any[step & 3];
      v.starts = 0;
      if (any || left < kK) {
        const int *mark = s.mark[step & 3] + mine0;
        if (any) v.starts = starts_of<SUB>(mark, left, kK);
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          if (k >= left) {
            v.starts &= ~(1u << k);
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
        if (v.starts & 1) mine.A = start_mark();
#pragma unroll
        for (int k = 1; k < kK; ++k)
          mine = v.starts >> k & 1 ? Map{start_mark(), v.u[k]}
                                   : Map{mul2(mine.A, v.at[k]), fma2(v.at[k], mine.U, v.u[k])};
      }
      if (SUB > 1) __syncwarp();
      v.front = post<false, SUB>(s, step, warp, any, mine);
    };
    auto run = [&](int step, const Step &v) {  // through the tokens from their true state
      const int tw = first + step * stride + group_of<SUB>(lane) * kK, left = a.T - tw;
      meet(kFronts + (step & 1));
      f2 h = s.front[step & 1][warp][place_of<SUB>(lane)];
      if (SUB > 1) h = through(v.front, h);
      const bool any = s.any[step & 3];
      int seg = s.alive[step & 3];
      if (SUB > 1 && any && a.T - first - step * stride > 0)
        seg = segments_at<SUB>(s.mark[step & 3], warp * kK * SUB, seg);
      if (left <= 0) return;
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
        if (SUB == 1 && any) seg = segment_at(s.mark[step & 3], warp * kK, seg);
        const int *mark = s.mark[step & 3] + mine0;
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
      if (warp == 0 && lane < L) {
        const int64_t at = (int64_t)n * a.D + c0;
        store_state(a.ht + at, a.h0 ? load_state(a.h0 + at, nv) : both(0.f), nv);
      }
    });
}

// ------------------------------------------------------------------ waits that run out

// The chain of the first of a cluster's two blocks, of which the second sends nothing: its first wait runs
// out, the others are not begun.
__global__ void __launch_bounds__(32) k_rec_wait_selftest(int steps, uint64_t limit_ns) {
  __shared__ Shared<1> s;
  s.init();
  for (int i = threadIdx.x; i < 2 * kHold * 32; i += 32) (&s.warp[0][0][0])[i] = packed(Map{both(1.f), both(0.f)});
  cluster_arrive();
  cluster_wait();
  if (cluster_rank() == 0) {
    f2 carry = both(0.f);
    bool lost = false;
    for (int step = 0; step < steps; ++step) chain<false, 1>(s, step, false, carry, lost, limit_ns);
  }
  __syncwarp();
  cluster_leave();
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

template <typename E, int MODE, int SUB, bool OUT, bool NORM>
cudaError_t run_fwd_as(const RecArgs &a, cudaStream_t stream) {
  return run_clusters<k_rec_fwd<E, MODE, SUB, OUT, NORM>>(a, SUB, Tokens<E, MODE, 3, 2, SUB>::kBytes, stream);
}
// The lanes' groups go by the sizes alone, so that the states are the same with and without y.  Without the
// normaliser there is one group, for fewer instances to compile: few channels then cost what the
// table at groups_of_lanes has for one (65,536 x 128: 1.8 times the time).
template <typename E, int MODE, bool OUT, bool NORM>
cudaError_t run_fwd_by(const RecArgs &a, cudaStream_t stream) {
  if (NORM) {
    const int sub = groups_of_lanes(a.T, a.D);
    if (sub == 4) return run_fwd_as<E, MODE, NORM ? 4 : 1, OUT, NORM>(a, stream);
    if (sub == 2) return run_fwd_as<E, MODE, NORM ? 2 : 1, OUT, NORM>(a, stream);
  }
  return run_fwd_as<E, MODE, 1, OUT, NORM>(a, stream);
}
template <typename E, bool OUT, bool NORM>
cudaError_t run_fwd(const RecArgs &a, cudaStream_t stream) {
  const std::initializer_list<Mat> mats = {a.x, a.r, a.i, OUT ? a.y : a.x};
  if (rows_fit<E>(a, 16, mats, {a.kept})) return run_fwd_by<E, 2, OUT, NORM>(a, stream);
  if (rows_fit<E>(a, 2 * sizeof(E), mats, {a.kept})) return run_fwd_by<E, 1, OUT, NORM>(a, stream);
  return run_fwd_by<E, 0, OUT, NORM>(a, stream);
}
template <typename E, bool OUT>
cudaError_t run_fwd(const RecArgs &a, cudaStream_t stream) {
  return a.normalize ? run_fwd<E, OUT, true>(a, stream) : run_fwd<E, OUT, false>(a, stream);
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
  const cudaError_t e = cudaMemcpyFromSymbol(out, mix::g_rec_status, sizeof(int32_t));
  return e == cudaSuccess && *out == 0 ? read_rec_bwd_status(out) : e;
}
cudaError_t clear_rec_status() {
  const int32_t zero = 0;
  const cudaError_t e = cudaMemcpyToSymbol(mix::g_rec_status, &zero, sizeof(int32_t));
  return e == cudaSuccess ? clear_rec_bwd_status() : e;
}

cudaError_t launch_rec_wait_selftest(uint32_t limit_us, int32_t steps, cudaStream_t stream) {
  return mix::launch_clusters(mix::k_rec_wait_selftest, 2, 2, 32, 0, stream, steps, (uint64_t)limit_us * 1000);
}

cudaError_t launch_rec_states(const RecArgs &a, cudaStream_t stream) {
  return a.f32 ? mix::run_fwd<float, false>(a, stream)
               : mix::run_fwd<__nv_bfloat16, false>(a, stream);
}
cudaError_t launch_rec_fwd(const RecArgs &a, cudaStream_t stream) {
  return a.f32 ? mix::run_fwd<float, true>(a, stream)
               : mix::run_fwd<__nv_bfloat16, true>(a, stream);
}
cudaError_t launch_rec_step(const RecArgs &a, float *state, int32_t slots, const int32_t *idx,
                            cudaStream_t stream) {
  return a.f32 ? mix::run_step<float>(a, state, slots, idx, stream)
               : mix::run_step<__nv_bfloat16>(a, state, slots, idx, stream);
}

}  // namespace gdr
