// gdr_qk.cu -- the norm of queries and keys for each head with the position rotation in the same
// pass, forward and backward.  For a row x of d elements (one token and head):
//
//   r = (sum x^2 / d + eps)^-1/2  (RMS)   or   (sum x^2 + eps)^-1/2  (L2),      u = x r w,
//   y = R(p) u: pairs (a, b) -> (a cos - b sin, b cos + a sin), elements from `rot` on unchanged.
//
// Backward, with e = R(p)^T dy and m = w e:
//   dx = r m - x r^3 (sum x m) / d  (L2: without / d),   dw = sum over rows of e x r.
//
// Bound by HBM: each row is read once and written once.  d / 8 lanes hold a row, 16 bytes of bf16
// each; a group of lanes keeps one token's cosines and sines in registers while it runs over the
// token's heads, q's and then k's.
#include <type_traits>

#include "gdr_mix.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kThreads = 128;
constexpr int kCtas = 4;  // blocks on each SM; each runs over many tokens

__device__ __forceinline__ int place_of(const QkArgs &a, int64_t t) {
  return min(max(a.pos[t], 0), a.places - 1);
}

// Sums four values of each lane over the LR lanes of a group: every lane gets all four.  A
// transposing butterfly: two exchanges leave a lane with one of the four sums, the rest of the
// butterfly completes it.  f is applied to the four sums, once a lane.
template <int LR, typename F>
__device__ __forceinline__ void four_sums(float (&v)[4], int gl, F f) {
  const bool hi = gl & (LR / 2), lo = gl & (LR / 4);
  const float a0 = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], LR / 2);
  const float a1 = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], LR / 2);
  float b = (lo ? a1 : a0) + __shfl_xor_sync(0xffffffffu, lo ? a0 : a1, LR / 4);
#pragma unroll
  for (int o = LR / 8; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
  b = f(b, (hi ? 2 : 0) + (lo ? 1 : 0));
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v[k] = __shfl_sync(0xffffffffu, b, (k >> 1) * (LR / 2) + (k & 1) * (LR / 4), LR);
}

// Cosines and sines of a lane's 8 elements, the sine with its sign for the forward rotation
// (u_e cos + u_partner sin); all 8 elements are in the rotated part or none.
struct Angles {
  float c[8], s[8];
};
template <bool INTER>
__device__ __forceinline__ void load_angles(const QkArgs &a, int64_t t, int e0, float4 (&c)[2],
                                            float4 (&s)[2]) {
  const int half = a.rot >> 1, at = INTER ? e0 >> 1 : (e0 < half ? e0 : e0 - half);
  const int64_t base = (int64_t)place_of(a, t) * half + at;
#pragma unroll
  for (int i = 0; i < (INTER ? 1 : 2); ++i) {
    c[i] = reinterpret_cast<const float4 *>(a.cos + base)[i];
    s[i] = reinterpret_cast<const float4 *>(a.sin + base)[i];
  }
}
template <bool INTER>
__device__ __forceinline__ Angles signed_angles(const float4 (&c)[2], const float4 (&s)[2],
                                                bool lower) {
  Angles r;
  const float cc[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
  const float ss[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.c[i] = cc[INTER ? i >> 1 : i];
    const float v = ss[INTER ? i >> 1 : i];
    r.s[i] = (INTER ? (i & 1) == 0 : lower) ? -v : v;
  }
  return r;
}

// The partners of a lane's 8 elements.
template <typename E, int LR, bool INTER>
__device__ __forceinline__ void partners(const Raw8<E> &own, int other, float (&v)[8]) {
  if (INTER) {
    float u[8];
    unpack8(own, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i ^ 1];
  } else {
    Raw8<E> r = own;
    uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r) / 4); ++i)
      w[i] = __shfl_sync(0xffffffffu, w[i], other, LR);
    unpack8(r, v);
  }
}

struct Groups {
  int hp;  // lane groups of a block that share a token (its heads in turn)
  int tp;  // tokens of a block
};

// A block runs over tokens tb, tb + gridDim.x, ...; for each, over batches of the heads of q, then
// of k: U rows a lane group, the next batch's rows (and the next token's angles) on their way.
// The weights' products with the angles are formed once a token:
//   y_e = r (x_e (w_e cos_e) + x_partner (w_partner sin_e)).
template <typename E, int LR, bool INTER, bool BWD>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_qk(const QkArgs a, const Groups gr, int64_t token_blocks) {
  constexpr int RP = kThreads / LR;
  constexpr int U = BWD ? 2 : 4;
  __shared__ __align__(16) float ws[2][LR * 8];
  const int grp = threadIdx.x / LR, gl = threadIdx.x % LR, e0 = gl * 8;
  const int first = grp % gr.hp;
  const bool rotated = a.rot > 0, turned = e0 < a.rot, lower = e0 < (a.rot >> 1);
  const int ro = a.rot >> 4;  // lanes of half the rotated part
  const int other = INTER || !turned ? gl : (lower ? gl + ro : gl - ro);
  const float inv = a.rms ? 1.f / (float)a.d : 1.f;
  for (int i = threadIdx.x; i < 2 * LR * 8; i += kThreads) {
    const mix::Param &w = i < LR * 8 ? a.w[0] : a.w[1];
    ws[i / (LR * 8)][i % (LR * 8)] = w.p ? ldp(w, i % (LR * 8)) : 1.f;
  }
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  __syncthreads();

  auto token = [&](int64_t tb) { return tb * gr.tp + grp / gr.hp; };
  auto alive = [&](int64_t tb) {
    return tb < token_blocks && grp < gr.hp * gr.tp && token(tb) < a.T;
  };
  Raw8<E> rx[U], rd[U];
  auto fetch = [&](int64_t tb, int j, int h0) {
    const int heads = j ? a.Hk : a.Hq;
    const int64_t t = token(tb);
    const int n = alive(tb) ? 8 : 0;
    const E *p = reinterpret_cast<const E *>(a.x[j]) + t * a.x_st[j] + (h0 + first) * a.x_sh[j] + e0;
    const int64_t step = gr.hp * a.x_sh[j];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rx[u] = ld8<true>(p, h0 + u * gr.hp + first < heads ? n : 0);
      p += step;
    }
    if (BWD) {
      p = reinterpret_cast<const E *>(a.y[j]) + t * a.y_st[j] + (h0 + first) * a.y_sh[j] + e0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        rd[u] = ld8<true>(p, h0 + u * gr.hp + first < heads ? n : 0);
        p += gr.hp * a.y_sh[j];
      }
    }
  };
  float4 ca[2], sa[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ca[i] = make_float4(1.f, 1.f, 1.f, 1.f);
    sa[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (turned && alive(blockIdx.x)) load_angles<INTER>(a, token(blockIdx.x), e0, ca, sa);
  int j = a.Hq > 0 ? 0 : 1, h0 = 0;
  fetch(blockIdx.x, j, 0);
  for (int64_t tb = blockIdx.x; tb < token_blocks; tb += gridDim.x) {
    const int64_t t = token(tb);
    const bool live = alive(tb);
    const Angles ang = signed_angles<INTER>(ca, sa, lower);
    if (turned && alive(tb + gridDim.x)) load_angles<INTER>(a, token(tb + gridDim.x), e0, ca, sa);
    float cw[8], sw[8];
    int formed = -1;  // the tensor that cw, sw are of
    for (bool last = false; !last;) {
      const int jj = j, hh = h0, heads = jj ? a.Hk : a.Hq;
      Raw8<E> cx[U], cd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        cx[u] = rx[u];
        if (BWD) cd[u] = rd[u];
      }
      h0 += gr.hp * U;
      if (h0 >= heads) {
        h0 = 0;
        if (jj == 0 && a.Hk > 0) {
          j = 1;
        } else {
          j = a.Hq > 0 ? 0 : 1;
          last = true;
        }
      }
      fetch(last ? tb + gridDim.x : tb, j, h0);
      if (formed != jj) {
        formed = jj;
        float w[8], wp[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(&ws[jj][e0 + i]);
          const float4 v = *reinterpret_cast<const float4 *>(&ws[jj][other * 8 + i]);
          w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
          wp[i] = v.x; wp[i + 1] = v.y; wp[i + 2] = v.z; wp[i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cw[i] = BWD ? w[i] : w[i] * ang.c[i];
          sw[i] = (INTER ? w[i ^ 1] : wp[i]) * ang.s[i];
        }
      }
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (!BWD) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[8];
          unpack8(cx[u], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u] = fmaf(x[i], x[i], v[u]);
        }
        four_sums<LR>(v, gl, [&](float q, int) { return rsqrtf(fmaf(q, inv, a.eps)); });
        E *p = reinterpret_cast<E *>(a.y[jj]) + t * a.y_st[jj] + (hh + first) * a.y_sh[jj] + e0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (hh + u * gr.hp >= heads) break;  // no lane group has a row left
          float x[8], o[8];
          unpack8(cx[u], x);
          if (rotated) {
            partners<E, LR, INTER>(cx[u], other, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(x[i], cw[i], o[i] * sw[i]) * v[u];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = x[i] * cw[i] * v[u];
          }
          st8<true>(p, pack8(o, E{}), live && hh + u * gr.hp + first < heads ? 8 : 0);
          p += gr.hp * a.y_sh[jj];
        }
      } else {
        float e[U][8];  // the rotation undone
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[8];
          unpack8(cx[u], x);
          unpack8(cd[u], e[u]);
          if (rotated) {
            float o[8];
            partners<E, LR, INTER>(cd[u], other, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[u][i] = fmaf(e[u][i], ang.c[i], -o[i] * ang.s[i]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[u] = fmaf(x[i], x[i], v[u]);
            v[2 + u] = fmaf(e[u][i] * cw[i], x[i], v[2 + u]);
          }
        }
        four_sums<LR>(v, gl, [&](float q, int k) {
          return k < 2 ? rsqrtf(fmaf(q, inv, a.eps)) : q * inv;
        });
        E *p = reinterpret_cast<E *>(a.dx[jj]) + t * a.dx_st[jj] + (hh + first) * a.dx_sh[jj] + e0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (hh + u * gr.hp >= heads) break;
          const bool ok = live && hh + u * gr.hp + first < heads;
          const float r = ok ? v[u] : 0.f, d = v[2 + u] * r * r * r;  // eps may be 0
          float x[8], o[8];
          unpack8(cx[u], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float g = e[u][i] * x[i];  // rows past the end are zero
            if (jj)
              dw[1][i] = fmaf(g, r, dw[1][i]);
            else
              dw[0][i] = fmaf(g, r, dw[0][i]);
            o[i] = fmaf(e[u][i] * cw[i], r, -x[i] * d);
          }
          st8<true>(p, pack8(o, E{}), ok ? 8 : 0);
          p += gr.hp * a.dx_sh[jj];
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
      for (int i = 0; i < 8; ++i) part[grp][e0 + i] = dw[j][i];
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
// partners of the rotation.  The backward's row sums and its last difference are in 64 bits: in a
// head of a few elements r m and x r^3 (sum x m) / d nearly cancel (at d = 1 only eps is left),
// and this path is not the fast one.
template <typename E, bool BWD>
__global__ void __launch_bounds__(kThreads) k_qk_any(const QkArgs a, int64_t rows) {
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
    using S = typename std::conditional<BWD, double, float>::type;
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
__global__ void __launch_bounds__(256)
    k_qk_sum(const float *work, int blocks, int d, float *dwq, float *dwk) {
  __shared__ float part[8][32];
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5, j = blockIdx.y;
  float *out = j ? dwk : dwq;
  if (!out) return;
  float v = 0.f;
  if (e < d)
    for (int b = k; b < blocks; b += 8) v += work[((int64_t)b * 2 + j) * d + e];
  part[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k == 0 && e < d) {
    for (int i = 1; i < 8; ++i) v += part[i][threadIdx.x];
    out[e] = v;
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool fast_rows(const QkArgs &a, bool bwd) {
  const int g = a.f32 ? 4 : 8;
  const bool pow2 = a.d == 64 || a.d == 128 || a.d == 256;
  if (!pow2 || a.rot % (a.interleaved ? 8 : 16) != 0) return false;
  if (!aligned16(a.cos) || !aligned16(a.sin)) return false;
  for (int j = 0; j < 2; ++j) {
    if (!aligned16(a.x[j]) || a.x_st[j] % g || a.x_sh[j] % g) return false;
    if (!aligned16(a.y[j]) || a.y_st[j] % g || a.y_sh[j] % g) return false;
    if (bwd && (!aligned16(a.dx[j]) || a.dx_st[j] % g || a.dx_sh[j] % g)) return false;
  }
  return true;
}

Groups groups_for(const QkArgs &a) {
  const int rp = kThreads / (a.d / 8);
  int hp = 1;
  while (hp < rp && hp < a.Hq + a.Hk) hp *= 2;
  return Groups{hp, rp / hp};
}

int64_t most_blocks() { return (int64_t)sm_count() * kCtas; }

template <typename E, int LR, bool BWD>
cudaError_t run_fast(const QkArgs &a, cudaStream_t stream, int *blocks_out) {
  const Groups gr = groups_for(a);
  const int64_t tb = ceil_div64(a.T, gr.tp);
  int64_t blocks = tb;
  if (blocks > most_blocks()) blocks = most_blocks();
  *blocks_out = (int)blocks;
  if (a.interleaved)
    k_qk<E, LR, true, BWD><<<(unsigned)blocks, kThreads, 0, stream>>>(a, gr, tb);
  else
    k_qk<E, LR, false, BWD><<<(unsigned)blocks, kThreads, 0, stream>>>(a, gr, tb);
  return cudaGetLastError();
}

template <typename E, bool BWD>
cudaError_t run(const QkArgs &a, cudaStream_t stream, int *blocks) {
  *blocks = 0;
  const int64_t rows = a.T * (a.Hq + a.Hk);
  if (rows == 0) return cudaSuccess;
  if (fast_rows(a, BWD)) {
    if (a.d == 64) return run_fast<E, 8, BWD>(a, stream, blocks);
    if (a.d == 128) return run_fast<E, 16, BWD>(a, stream, blocks);
    return run_fast<E, 32, BWD>(a, stream, blocks);
  }
  int64_t n = ceil_div64(rows, kThreads / 32);
  if (n > most_blocks()) n = most_blocks();
  *blocks = (int)n;
  k_qk_any<E, BWD><<<(unsigned)n, kThreads, 0, stream>>>(a, rows);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mix

cudaError_t launch_qk_fwd(const QkArgs &a, cudaStream_t stream) {
  int blocks;
  return a.f32 ? mix::run<float, false>(a, stream, &blocks)
               : mix::run<__nv_bfloat16, false>(a, stream, &blocks);
}

size_t qk_bwd_workspace(int64_t, int32_t, int32_t, int32_t d) {
  return align256((size_t)mix::most_blocks() * 2 * d * sizeof(float));
}

cudaError_t launch_qk_bwd(const QkArgs &a, cudaStream_t stream) {
  int blocks;
  cudaError_t e = a.f32 ? mix::run<float, true>(a, stream, &blocks)
                        : mix::run<__nv_bfloat16, true>(a, stream, &blocks);
  if (e != cudaSuccess || (!a.dw[0] && !a.dw[1])) return e;
  mix::k_qk_sum<<<dim3((unsigned)ceil_div64(a.d, 32), 2), 256, 0, stream>>>(
      reinterpret_cast<const float *>(a.work), blocks, a.d, a.dw[0], a.dw[1]);
  return cudaGetLastError();
}

}  // namespace gdr
