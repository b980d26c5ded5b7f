// gdr_ssm.cuh -- the thread layout that the selective state space kernels share.
//
// A block of 128 threads owns CH = 256 / LN channels of one group.  LN neighbouring lanes share a
// channel and hold 4 states each (LN = 4 for up to 16 states); a thread holds two channels, so
// that a token's B and C, read from shared memory, serve 8 states.
#pragma once

#include "gdr_mix.cuh"

namespace gdr {
namespace ssm {

constexpr int kThreads = 128;

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
  __device__ __forceinline__ void read(const SsmArgs &a, const float *p, int64_t row,
                                       float (&h)[2][4]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nl * 4 + j;
        h[k][j] = (p && ch[k] < nch && n < a.N) ? p[(row * a.D + c0 + ch[k]) * a.N + n] : 0.f;
      }
  }
  __device__ __forceinline__ void write(const SsmArgs &a, float *p, int64_t row,
                                        const float (&h)[2][4]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nl * 4 + j;
        if (ch[k] < nch && n < a.N) p[(row * a.D + c0 + ch[k]) * a.N + n] = h[k][j];
      }
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

inline int lanes_for(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

inline int64_t channel_tiles(int D, int G, int LN) {
  return (int64_t)G * ceil_div64(D / G, 256 / LN);
}

}  // namespace ssm
}  // namespace gdr
