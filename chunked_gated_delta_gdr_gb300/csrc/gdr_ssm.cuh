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
  // A token's pairs (two floats for each channel) in shared memory: a thread's two channels are
  // neighbours, one 16-byte load.  The XOR spreads the stores of 8 neighbouring channels, which
  // stand 16 bytes apart, over the banks.
  static __device__ __forceinline__ int pair_slot(int t, int warp, int cl) {
    const int f = CW >= 8 ? (warp + ((t & 1) << 2)) & 7 : 0;
    return warp * CW + (cl ^ f);
  }
  // index (in float2) of channel ch's pair of token t
  static __device__ __forceinline__ int pair_at(int t, int ch) {
    const int warp = ch / (2 * CW), k = (ch / CW) & 1, cl = ch % CW;
    return t * CH + pair_slot(t, warp, cl) * 2 + k;
  }
  // index of channel ch's LN partial sums of token t; the XOR spreads the reads of a thread's 8
  // channels
  static __device__ __forceinline__ int part_at(int t, int ch) {
    const int g = ch >> 3;
    return (t * CH + g * 8 + ((ch & 7) ^ (g & 7))) * LN;
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

// Tokens of a range of the scan (a multiple of the tile) for `want` blocks on each SM.
inline int range_tokens(int64_t T, int64_t ctiles, int tile, int want, int least) {
  int64_t n = (int64_t)mix::sm_count() * want / (ctiles < 1 ? 1 : ctiles);
  const int64_t most = ceil_div64(T, least);
  if (n > most) n = most;
  if (n < 1) n = 1;
  const int64_t r = ceil_div64(ceil_div64(T, n), tile) * tile;
  return (int)(r < tile ? tile : r);
}

inline int lanes_for(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

inline int64_t channel_tiles(int D, int G, int LN) {
  return (int64_t)G * ceil_div64(D / G, 256 / LN);
}

}  // namespace ssm
}  // namespace gdr
