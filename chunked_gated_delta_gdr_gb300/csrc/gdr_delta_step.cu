// gdr_delta_step.cu -- the gated delta rule for single tokens (decoding), states in a pool of
// slots, updated in place.  With K = e^g S (S [dk, dv] of one request and value head):
//
//   s = k^T K,   S' = K + beta k (v - s)^T,   o = scale S'^T q = scale (q^T K + beta (q.k) (v - s)),
//
// so that both products over the rows, k^T K and q^T K, come from one look at the state, and o
// needs no second.  Bound by HBM: the state is read once and written once, in fp32.  Columns are
// independent: a block owns a tile of CT columns of one head, all rows of it in registers.
// 256 requests of 32 heads of 128: 155 us, all of the measured copy bandwidth.
#include "gdr_mix.cuh"

namespace gdr {
namespace mix {
namespace {

// D rows x CT columns; 4 columns a thread, D * CT / 4 / THREADS rows a thread.
template <int D, int CT, int THREADS>
__global__ void __launch_bounds__(THREADS) k_delta_step(const DeltaStepArgs a) {
  after_previous<true>();
  constexpr int CL = CT / 4, RG = THREADS / CL, R = D / RG;  // column lanes, row groups, rows each
  __shared__ float ks[D], qs[D];
  __shared__ float4 red[2][RG][CL];
  const int tiles = D / CT;
  const int tile = blockIdx.x % tiles;
  const int h = (int)(blockIdx.x / tiles % a.H), row = (int)(blockIdx.x / tiles / a.H);
  const int cl = threadIdx.x % CL, rg = threadIdx.x / CL, col = tile * CT + cl * 4;
  const int slot = a.idx ? a.idx[row] : row;
  __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(a.o) + row * a.o_st + h * a.o_sh + col;
  if (slot < 0 || slot >= a.slots) {
    if (rg == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __float2bfloat16_rn(0.f);
    }
    return;
  }
  float4 *S = reinterpret_cast<float4 *>(a.state + (((int64_t)slot * a.H + h) * D + rg * R) * D + col);
  float4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) s[i] = S[i * (D / 4)];
  const int hk = h / (a.H / a.Hk);
  for (int i = threadIdx.x; i < D; i += THREADS) {
    ks[i] = ldbf(a.k, row * a.k_st + hk * a.k_sh + i);
    qs[i] = ldbf(a.q, row * a.q_st + hk * a.q_sh + i);
  }
  const float eg = expf(a.g[row * a.g_st + h * a.g_sh]);
  const float beta = ldbf(a.beta, row * a.b_st + h * a.b_sh);
  const int64_t vat = row * a.v_st + h * a.v_sh + col;
  const float4 v = make_float4(ldbf(a.v, vat), ldbf(a.v, vat + 1), ldbf(a.v, vat + 2),
                               ldbf(a.v, vat + 3));
  __syncthreads();
  float4 sk = make_float4(0, 0, 0, 0), sq = make_float4(0, 0, 0, 0);
  float qk = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float k = ks[rg * R + i], q = qs[rg * R + i];
    s[i].x *= eg; s[i].y *= eg; s[i].z *= eg; s[i].w *= eg;
    sk.x = fmaf(k, s[i].x, sk.x); sk.y = fmaf(k, s[i].y, sk.y);
    sk.z = fmaf(k, s[i].z, sk.z); sk.w = fmaf(k, s[i].w, sk.w);
    sq.x = fmaf(q, s[i].x, sq.x); sq.y = fmaf(q, s[i].y, sq.y);
    sq.z = fmaf(q, s[i].z, sq.z); sq.w = fmaf(q, s[i].w, sq.w);
  }
  red[0][rg][cl] = sk;
  red[1][rg][cl] = sq;
  __syncthreads();
  sk = red[0][0][cl];
#pragma unroll
  for (int i = 1; i < RG; ++i) {
    const float4 p = red[0][i][cl];
    sk.x += p.x; sk.y += p.y; sk.z += p.z; sk.w += p.w;
  }
  const float4 d = make_float4(beta * (v.x - sk.x), beta * (v.y - sk.y), beta * (v.z - sk.z),
                               beta * (v.w - sk.w));
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float k = ks[rg * R + i];
    s[i].x = fmaf(k, d.x, s[i].x); s[i].y = fmaf(k, d.y, s[i].y);
    s[i].z = fmaf(k, d.z, s[i].z); s[i].w = fmaf(k, d.w, s[i].w);
    S[i * (D / 4)] = s[i];
  }
  if (rg == 0) {
    sq = red[1][0][cl];
#pragma unroll
    for (int i = 1; i < RG; ++i) {
      const float4 p = red[1][i][cl];
      sq.x += p.x; sq.y += p.y; sq.z += p.z; sq.w += p.w;
    }
#pragma unroll 8
    for (int i = 0; i < D; ++i) qk = fmaf(qs[i], ks[i], qk);
    o[0] = __float2bfloat16_rn(a.scale * fmaf(qk, d.x, sq.x));
    o[1] = __float2bfloat16_rn(a.scale * fmaf(qk, d.y, sq.y));
    o[2] = __float2bfloat16_rn(a.scale * fmaf(qk, d.z, sq.z));
    o[3] = __float2bfloat16_rn(a.scale * fmaf(qk, d.w, sq.w));
  }
}

template <int D, int CT, int THREADS>
cudaError_t run(const DeltaStepArgs &a, cudaStream_t stream) {
  const int64_t blocks = (int64_t)a.B * a.H * (D / CT);
  return launch(k_delta_step<D, CT, THREADS>, (unsigned)blocks, THREADS, 0, stream, a);
}

}  // namespace
}  // namespace mix

cudaError_t launch_delta_step(const DeltaStepArgs &a, cudaStream_t stream) {
  if (a.B == 0) return cudaSuccess;
  if (a.D == 64) return mix::run<64, 32, 64>(a, stream);
  return mix::run<128, 32, 128>(a, stream);
}

}  // namespace gdr
