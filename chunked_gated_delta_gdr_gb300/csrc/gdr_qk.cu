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

__device__ __forceinline__ int place_of(const QkArgs &a, int64_t t) {
  return min(max(a.pos[t], 0), a.places - 1);
}

template <int LR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Cosines and sines of a lane's 8 elements (interleaved pairs: the first 4).
template <bool INTER>
__device__ __forceinline__ void angles(const QkArgs &a, int64_t t, int e0, float (&c)[8],
                                       float (&s)[8]) {
  const int half = a.rot >> 1;
  const int64_t base = (int64_t)place_of(a, t) * half;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = INTER ? (e0 >> 1) + i : (e0 + i < half ? e0 + i : e0 + i - half);
    const bool ok = INTER ? (i < 4 && e0 + 2 * i < a.rot) : e0 + i < a.rot;
    c[i] = ok ? a.cos[base + at] : 1.f;
    s[i] = ok ? a.sin[base + at] : 0.f;
  }
}

// The rotation (back: its transpose) of a row spread over the lanes.
template <int LR, bool INTER>
__device__ __forceinline__ void rotate(float (&u)[8], const float (&c)[8], const float (&s)[8],
                                       int gl, int rot, bool back) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = u[2 * i], q = u[2 * i + 1], n = back ? -s[i] : s[i];
      u[2 * i] = p * c[i] - q * n;
      u[2 * i + 1] = q * c[i] + p * n;
    }
  } else {
    const int ro = rot >> 4;  // lanes of half the rotated part
    const bool lower = gl < ro;
    const int other = gl < 2 * ro ? (lower ? gl + ro : gl - ro) : gl;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = __shfl_sync(0xffffffffu, u[i], other, LR);
      const float n = lower != back ? -s[i] : s[i];
      u[i] = fmaf(v, n, u[i] * c[i]);
    }
  }
}

struct Groups {
  int hp;  // lane groups of a block that share a token (its heads in turn)
  int tp;  // tokens of a block
};

template <typename E, int LR, bool INTER, bool BWD>
__global__ void __launch_bounds__(kThreads)
    k_qk(const QkArgs a, const Groups gr, int64_t token_blocks) {
  constexpr int RP = kThreads / LR;
  constexpr int U = BWD ? 2 : 4;  // rows in flight
  const int grp = threadIdx.x / LR, gl = threadIdx.x % LR, e0 = gl * 8;
  const int heads = a.Hq + a.Hk;
  const float inv = a.rms ? 1.f / (float)a.d : 1.f;
  float w[2][8], dw[2][8];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[j][i] = a.w[j].p ? ldp(a.w[j], e0 + i) : 1.f;
      dw[j][i] = 0.f;
    }
  for (int64_t tb = blockIdx.x; tb < token_blocks; tb += gridDim.x) {
    const int64_t t = tb * gr.tp + grp / gr.hp;
    const bool live = grp < gr.hp * gr.tp && t < a.T;
    float c[8], s[8];
    if (a.rot > 0 && live) {
      angles<INTER>(a, t, e0, c, s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
      }
    }
    // the loop runs the same number of times in every lane: shuffles inside
    const int first = grp % gr.hp;
    for (int h0 = 0; h0 < heads; h0 += gr.hp * U) {
      Raw8<E> rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * gr.hp + first;
        const bool ok = live && h < heads;
        const int j = h < a.Hq ? 0 : 1, hj = j ? h - a.Hq : h;
        rx[u] = ld8<true>(reinterpret_cast<const E *>(a.x[j]) + t * a.x_st[j] + hj * a.x_sh[j] + e0,
                          ok ? 8 : 0);
        if (BWD)
          rd[u] = ld8<true>(
              reinterpret_cast<const E *>(a.y[j]) + t * a.y_st[j] + hj * a.y_sh[j] + e0, ok ? 8 : 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h0 + u * gr.hp >= heads) break;  // no lane group has a row left
        const int h = h0 + u * gr.hp + first;
        const bool ok = live && h < heads;
        const int j = h < a.Hq ? 0 : 1, hj = j ? h - a.Hq : h;
        float x[8], v[8], q = 0.f;
        unpack8(rx[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(x[i], x[i], q);
        q = row_sum<LR>(q);
        const float r = ok ? rsqrtf(fmaf(q, inv, a.eps)) : 0.f;  // eps may be 0
        if (!BWD) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = x[i] * r * (j ? w[1][i] : w[0][i]);
          if (a.rot > 0) rotate<LR, INTER>(v, c, s, gl, a.rot, false);
          st8<true>(reinterpret_cast<E *>(a.y[j]) + t * a.y_st[j] + hj * a.y_sh[j] + e0,
                    pack8(v, E{}), ok ? 8 : 0);
        } else {
          unpack8(rd[u], v);
          if (a.rot > 0) rotate<LR, INTER>(v, c, s, gl, a.rot, true);
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float g = v[i] * x[i] * r;  // rows past the end are zero
            if (j)
              dw[1][i] += g;
            else
              dw[0][i] += g;
            v[i] *= j ? w[1][i] : w[0][i];
            dot = fmaf(v[i], x[i], dot);
          }
          dot = row_sum<LR>(dot) * inv * r * r * r;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], r, -x[i] * dot);
          st8<true>(reinterpret_cast<E *>(a.dx[j]) + t * a.dx_st[j] + hj * a.dx_sh[j] + e0,
                    pack8(v, E{}), ok ? 8 : 0);
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
  if (!pow2 || (!a.interleaved && a.rot % 16 != 0)) return false;
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

constexpr int kBwdCtas = 6;  // blocks on each SM of the backward, which keeps dw in registers

int64_t bwd_blocks() { return (int64_t)sm_count() * kBwdCtas; }

template <typename E, int LR, bool BWD>
cudaError_t run_fast(const QkArgs &a, cudaStream_t stream, int *blocks_out) {
  const Groups gr = groups_for(a);
  const int64_t tb = ceil_div64(a.T, gr.tp);
  int64_t blocks = tb;
  if (BWD && blocks > bwd_blocks()) blocks = bwd_blocks();
  if (blocks > 0x7fffffff) blocks = 0x7fffffff;
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
  if (n > bwd_blocks()) n = bwd_blocks();
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
  return align256((size_t)mix::bwd_blocks() * 2 * d * sizeof(float));
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
