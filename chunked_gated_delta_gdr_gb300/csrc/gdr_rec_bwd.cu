// gdr_rec_bwd.cu -- the backward of the gated linear recurrence (formulas in gdr_rec.cu): the same walk
// from the last token to the first, over the states that the forward kept before every kK-th token.  A
// step's maps need the decays and dy alone; its gradients are computed while the next step's maps are on
// their way.  8,192 x 2,560: 100 us in bf16 for 43 of bytes (x, r, i, dy, dx, dr, di), 134 in fp32 for 86, bound as
// the forward is: 16 warps an SM (8 in fp32), which recompute each state from the last one kept, where that
// costs no bytes (keeping all of them in fp32 would be 84 MB more written and read, 25 us of a copy).
#include "gdr_rec.cuh"

namespace gdr {
namespace mix {
namespace {

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

template <typename E, int MODE, int SUB, bool NORM>
__global__ void __launch_bounds__(kP * 32, 2) k_rec_bwd(const RecArgs a, const int32_t *bounds) {
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
    bool lost = false;
    for (int step = 0; step < steps; ++step) {
      meet(kMaps + (step & 1));
      const bool any2 = look(step + 2);
      chain<true, SUB>(s, step, any0, carry, lost);
      any0 = any1;
      any1 = any2;
      __syncwarp();
      arrive(kFronts + (step & 1));
    }
  } else {
    const f2 A = load_state(a.A + c0, nv), A2 = mul2(A, both(kLog2e));
    using In = Tokens<E, MODE, 4, 3, SUB>;
    In in{{reinterpret_cast<const E *>(a.x.p) + cb, reinterpret_cast<const E *>(a.r.p) + cb,
           a.i.p ? reinterpret_cast<const E *>(a.i.p) + cb : nullptr,
           reinterpret_cast<const E *>(a.dy.p) + cb},
          {a.x.st, a.r.st, a.i.st, a.dy.st},
          raw + warp * 3 * In::kPlace, lane, a.D - cb, nv, a.T};
    const bool gate = a.i.p;
    E *dx = reinterpret_cast<E *>(a.dx.p) + c0, *dr = reinterpret_cast<E *>(a.dr.p) + c0;
    E *di = reinterpret_cast<E *>(a.di.p) + c0;
    const int first = (steps - 1) * stride + rank * kTile + warp * kK * SUB;
    const int mine0 = warp * kK * SUB + group_of<SUB>(lane) * kK;  // the lane's first token in the tile
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
    auto starts_in = [&](int step, int left) {
      return s.any[step & 3] ? starts_of<SUB>(s.mark[step & 3] + mine0, left, kK + 1) : 0u;
    };
    auto segments_in = [&](int step) {  // of the lanes' first tokens
      int seg = s.alive[step & 3];
      if (s.any[step & 3] && a.T - (first - step * stride) > 0)
        seg = segments_at<SUB>(s.mark[step & 3], warp * kK * SUB, seg);
      return seg;
    };
    // all of a warp's tokens are there, and none of them starts or ends a segment but the last
    auto plain = [&](int step, uint32_t starts) {
      const bool whole = a.T - (first - step * stride) >= kK * SUB;
      return SUB == 1 ? whole && starts == 0 : whole && !__any_sync(0xffffffffu, starts != 0);
    };
    auto hold = [&](int place, int step) {  // the map of the step's tokens, for the chain
      const int tw = first - step * stride + group_of<SUB>(lane) * kK, left = a.T - tw;
      in.wait();
      const uint32_t starts = starts_in(step, left);
      Map mine = {one, both(0.f)};
      if (plain(step, starts)) {
        f2 at[kK];
#pragma unroll
        for (int k = 0; k < kK; ++k) at[k] = decay_of(mul2(A2, sigmoid2(in.get(place, 1, k, tw + k))));
        mine = Map{at[kK - 1], mul2(at[kK - 1], in.get(place, 3, kK - 1, tw + kK - 1))};
#pragma unroll
        for (int k = kK - 2; k >= 0; --k)
          mine = Map{mul2(mine.A, at[k]), mul2(at[k], add2(in.get(place, 3, k, tw + k), mine.U))};
      } else {
        const int seg = segments_in(step);
        const int *mark = s.mark[step & 3] + mine0;
#pragma unroll 1
        for (int k = min(kK, left) - 1; k >= 0; --k) {
          const f2 at = decay_of(mul2(A2, sigmoid2(in.get(place, 1, k, tw + k))));
          f2 g = in.get(place, 3, k, tw + k);
          if (starts >> (k + 1) & 1) {
            g = add2(g, ending(own_segment(starts, mark, k, seg)));
            mine = Map{start_mark(), mul2(at, g)};
          } else {
            mine = Map{mul2(mine.A, at), mul2(at, add2(g, mine.U))};
          }
        }
        __syncwarp();
      }
      return post<true, SUB>(s, step, warp, s.any[step & 3], mine);
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
    auto run = [&](int place, int step, const Map &before) {  // the gradients of the step's tokens
      const int tw = first - step * stride + group_of<SUB>(lane) * kK, left = a.T - tw;
      f2 h = both(0.f);
      if (left > 0) h = wide(ld2<VEC>(a.kept + (int64_t)(tw / kK) * a.D + c0, nv));
      const uint32_t starts = starts_in(step, left);
      const int seg = segments_in(step);
      const bool inside = seg >= 0 && seg < a.n_seq;
      if (plain(step, starts) && (SUB == 1 ? inside : __all_sync(0xffffffffu, inside))) {
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
            const f2 r = in.get(place, 1, k, tw + k);
            si[k] = one;
            if (gate) sigmoids_apart(r, in.get(place, 2, k, tw + k), sr[k], si[k]);
            else sr[k] = sigmoid2(r);
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
        f2 c = s.front[step & 1][warp][place_of<SUB>(lane)];
        if (SUB > 1) c = through(before, c);
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
      const int *mark = s.mark[step & 3] + mine0;
      f2 hb[kK];  // not in registers
      auto part = [&](int k, f2 &sr, f2 &si, f2 &at, f2 &m) {
        const f2 r = in.get(place, 1, k, tw + k);
        si = one;
        if (gate) sigmoids_apart(r, in.get(place, 2, k, tw + k), sr, si);
        else sr = sigmoid2(r);
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
      __syncwarp();
      meet(kFronts + (step & 1));
      f2 c = s.front[step & 1][warp][place_of<SUB>(lane)];
      if (SUB > 1) c = through(before, c);
#pragma unroll 1
      for (int k = min(kK, left) - 1; k >= 0; --k) {
        const int own = own_segment(starts, mark, k, seg);
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
    Map before = {one, both(0.f)};  // of the groups behind the lane's
    if (steps > 0) before = hold(0, 0);
    int place = 0;  // of the step that is run
    auto after = [](int p) { return p == 2 ? 0 : p + 1; };
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      const int next = after(place);
      // the step after next into the place of the one before this
      in.issue(after(next), step + 2 < steps ? first - (step + 2) * stride : a.T, -stride);
      Map then_before = before;
      if (step + 1 < steps) then_before = hold(next, step + 1);
      run(place, step, before);
      __syncwarp();
      before = then_before;
      place = next;
    }
    if (VEC) copies_wait<0>();
  }
  // dA: the warps' sums in order, then the blocks' of the cluster
  float d0, d1;
  unpair(dA, d0, d1);
#pragma unroll
  for (int o = L; o < 32; o *= 2) {
    d0 += __shfl_xor_sync(0xffffffffu, d0, o);
    d1 += __shfl_xor_sync(0xffffffffu, d1, o);
  }
  dA = pair(d0, d1);
  __syncthreads();
  if (warp < kHold && lane < L) s.warp[0][warp][lane] = packed(Map{dA, both(0.f)});
  __syncthreads();
  if (warp == 0 && lane < L) {
    f2 v = unpacked(s.warp[0][0][lane]).A;
#pragma unroll
    for (int w = 1; w < kHold; ++w) v = add2(v, unpacked(s.warp[0][w][lane]).A);
    put(&s.block[steps & 1][rank][lane], 0, packed(Map{v, both(0.f)}));
  }
  cluster_arrive();
  cluster_wait();
  if (rank == 0) {
    if (warp == 0 && lane < L) {
      f2 v = unpacked(s.block[steps & 1][0][lane]).A;
      for (int b = 1; b < size; ++b) v = add2(v, unpacked(s.block[steps & 1][b][lane]).A);
      store_state(a.dA + c0, v, nv);
    }
    if (a.dh0)
      for_empty_segments(a.cu, a.n_seq, a.T, s.red, [&](int n) {
        if (warp == 0 && lane < L) {
          const int64_t at = (int64_t)n * a.D + c0;
          store_state(a.dh0 + at, a.dht ? load_state(a.dht + at, nv) : both(0.f), nv);
        }
      });
  }
}

// ------------------------------------------------------------------ launches

size_t kept_bytes(int64_t T, int32_t D) {
  return align256((size_t)((T + kRecEvery - 1) / kRecEvery) * D * 4);
}

template <typename E, int MODE, int SUB, bool NORM>
cudaError_t run_bwd_as(const RecArgs &a, const int32_t *bounds, cudaStream_t stream) {
  return run_clusters<k_rec_bwd<E, MODE, SUB, NORM>>(a, SUB, Tokens<E, MODE, 4, 3, SUB>::kBytes, stream,
                                                     bounds);
}
template <typename E, int MODE, bool NORM>
cudaError_t run_bwd_by(const RecArgs &a, const int32_t *bounds, cudaStream_t stream) {
  if (NORM) {
    const int sub = groups_of_lanes(a.T, a.D);
    if (sub == 4) return run_bwd_as<E, MODE, NORM ? 4 : 1, NORM>(a, bounds, stream);
    if (sub == 2) return run_bwd_as<E, MODE, NORM ? 2 : 1, NORM>(a, bounds, stream);
  }
  return run_bwd_as<E, MODE, 1, NORM>(a, bounds, stream);
}
template <typename E, bool NORM>
cudaError_t run_bwd_for(const RecArgs &a, const int32_t *bounds, cudaStream_t stream) {
  const std::initializer_list<Mat> mats = {a.x, a.r, a.i, a.dy, a.dx, a.dr, a.di};
  if (rows_fit<E>(a, 16, mats, {a.kept})) return run_bwd_by<E, 2, NORM>(a, bounds, stream);
  if (rows_fit<E>(a, 2 * sizeof(E), mats, {a.kept})) return run_bwd_by<E, 1, NORM>(a, bounds, stream);
  return run_bwd_by<E, 0, NORM>(a, bounds, stream);
}

cudaError_t run_bwd(RecArgs a, bool kept, cudaStream_t stream) {
  char *w = reinterpret_cast<char *>(a.work);
  int32_t *bounds = reinterpret_cast<int32_t *>(w);
  cudaError_t e = launch(k_rec_bounds, 1, 1024, 0, stream, a.cu, a.n_seq + 1, a.T, bounds);
  if (e != cudaSuccess) return e;
  if (!kept) {
    a.kept = reinterpret_cast<float *>(w + align256(((size_t)a.n_seq + 1) * 4));
    a.ht = nullptr;
    e = launch_rec_states(a, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.f32)
    return a.normalize ? run_bwd_for<float, true>(a, bounds, stream)
                       : run_bwd_for<float, false>(a, bounds, stream);
  return a.normalize ? run_bwd_for<__nv_bfloat16, true>(a, bounds, stream)
                     : run_bwd_for<__nv_bfloat16, false>(a, bounds, stream);
}

}  // namespace
}  // namespace mix

cudaError_t read_rec_bwd_status(int32_t *out) {
  return cudaMemcpyFromSymbol(out, mix::g_rec_status, sizeof(int32_t));
}
cudaError_t clear_rec_bwd_status() {
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(mix::g_rec_status, &zero, sizeof(int32_t));
}

size_t rec_bwd_workspace(int64_t T, int32_t D, int32_t n_seq, bool kept) {
  return align256(((size_t)n_seq + 1) * 4) + (kept ? 0 : mix::kept_bytes(T, D));
}
cudaError_t launch_rec_bwd(const RecArgs &a, bool kept, cudaStream_t stream) {
  return mix::run_bwd(a, kept, stream);
}

}  // namespace gdr
