// gdr_attn.cu -- attention of one new token for each request over a paged key-value cache:
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = e^{scale q.k_j - max},  j over the request's last keys.
//
// Bound by HBM: keys and values are read once for up to 16 query heads that share them, once more for
// every further 16 (64 requests of 4,096 keys, 2 key heads of 128: 128 us with 64 query heads, 232 with 128).
// The work is cut over the keys, whatever the requests' lengths are: all (request, head) pairs' keys
// in a row, in units of 64, are dealt to the blocks in equal ranges, which every block finds from
// the lengths on the device.  A block keeps a running maximum, sum and output for each pair in its
// range; a pair that lies in one range is finished there, parts of others are joined by a second
// kernel, in order.
//
// A warp takes 16 keys of a unit: its rows come by cp.async into a ring of its own, so that no barrier
// is needed before a range's end, and go through mma.sync with the 16 keys (or 16 columns of the values) as
// its rows and one or two tiles of 8 query heads as its columns, of which a group of fewer heads leaves
// some empty: its rate is far above what HBM feeds, and one instruction needs no accumulator in Tensor
// Memory that the softmax would have to fetch.  Scores, maxima, sums and outputs are fp32; the probabilities
// go to the second product as three bf16 parts each, which hold all of their 24 bits (with two parts, 17
// bits, the case below takes 192 us as well).
//
// 64 requests of up to 16,384 keys, 32 / 4 heads of 128: 192 us, 86 % of a copy's rate.  One request of 32,768
// keys, 32 / 8 heads: 33 us for 20 of bytes; start, drain and the second kernel are the rest.  8 heads a tile and
// three blocks an SM where they fit; heads over 128 leave room for one block of four warps (146 requests of
// 3,314 keys x 256: 60 us for 41 of bytes).
#include "gdr_block.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kRows = 16;           // query heads of a pair at most
constexpr int kWarps = 4, kUnit = 16 * kWarps;  // keys of a unit
constexpr int kMostCtas = 1024;     // blocks with parts in the workspace

__device__ __forceinline__ float low() { return __uint_as_float(0xff800000u); }  // -inf

// ------------------------------------------------------------------ dealing out the work

// The keys of a request that its token sees, first .. end - 1, in units from base on: a warp's 16 keys
// start at a multiple of 16, and lie on one page where pages hold a multiple of that.
struct Span {
  int base, first, end;
  __device__ __forceinline__ Span(const AttnArgs &a, int b) {
    const int64_t room = (int64_t)a.width * a.page;
    const int64_t n = max((int64_t)0, min((int64_t)a.lens[b], room));
    end = (int)n;
    first = a.window > 0 && n > a.window ? (int)(n - a.window) : 0;
    base = first & ~15;
  }
  __device__ __forceinline__ int units() const { return (int)(((int64_t)end - base + kUnit - 1) / kUnit); }
};

// All threads: the sum of v over the block.  red: 32 values.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < (int)blockDim.x >> 5; ++w) v += red[w];
  return v;
}

// Units of all requests, and of those before request b.
__device__ __forceinline__ void count_units(const AttnArgs &a, int b, int64_t *red, int64_t &all,
                                            int64_t &before) {
  int64_t s = 0, p = 0;
  for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
    const int u = Span(a, i).units();
    s += u;
    if (i < b) p += u;
  }
  all = block_sum(s, red);
  before = b > 0 ? block_sum(p, red) : 0;
}

// Units of a block's range: equal for all blocks.
__device__ __forceinline__ int64_t share_of(int64_t units, int ctas) {
  return max((int64_t)1, (units + ctas - 1) / ctas);
}

// The request whose units hold unit x of the whole (x < all pairs' units), and where they start.
__device__ __forceinline__ int find_request(const AttnArgs &a, int pairs, int64_t x, int64_t *red,
                                            int64_t *found, int64_t &start) {
  int64_t run = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int base = 0; base < a.B; base += blockDim.x) {
    const int i = base + threadIdx.x;
    const int64_t u = i < a.B ? (int64_t)Span(a, i).units() * pairs : 0;
    int64_t v = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) v += red[w];
      total += red[w];
    }
    if (run + v - u <= x && x < run + v) {
      found[0] = i;
      found[1] = run + v - u;
    }
    run += total;
    if (run > x) break;
  }
  __syncthreads();
  start = found[1];
  return (int)found[0];
}

// ------------------------------------------------------------------ tensor instructions

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// c += a b: 16 x 8 x 16 in bf16
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of a warp's pairs, transposed
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Two weights as three bf16 parts each, the leading 8 bits of what is left each time: all 24 bits of them.
// No part of a weight is 0 but the weight itself: 0 times an infinite value would be NaN, and so would
// parts of either sign be.  (2^-126 in the place of a 0 is less of the largest weight, 1, than fp32 holds.)
__device__ __forceinline__ void split3(float x, float y, uint32_t (&part)[3]) {
  const float least = __uint_as_float(0x00800000u);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    part[i] = __byte_perm(a, b, 0x7632);  // the upper halves, cut off
    x = fmaxf(x - __uint_as_float(a & 0xffff0000u), least);
    y = fmaxf(y - __uint_as_float(b & 0xffff0000u), least);
  }
}

// ------------------------------------------------------------------ the split kernel

// A part of a (request, key head, group of query heads): O [16][D], m and l [16].
template <int D>
constexpr int kPart = kRows * D + 2 * kRows;

// H: query heads of a pair, 8 or 16
template <int D, int H, int S>
struct AttnSmem {
  uint4 ring[kWarps][S][2][16 * D / 8];  // each warp's keys and values, rows of 16-byte parts
  float out[2][H * D];
  float m[kWarps][H], l[kWarps][H];
  int64_t red[32], found[2];
  // element (head, column) of a warp's output: a lane's heads 2 t, 2 t + 1 beside 8 columns
  static __device__ __forceinline__ int at(int h, int c) { return h * D + (c ^ ((h >> 1 & 3) << 3)); }
};

// Where a block is in the sequence of units: a warp's walk over requests, pairs and units.
struct Cursor {
  int b, pair, unit, units, base, first, end;
  __device__ __forceinline__ void request(const AttnArgs &a) {
    // past the requests without keys
    for (; b < a.B; ++b) {
      const Span s(a, b);
      base = s.base;
      first = s.first;
      end = s.end;
      units = s.units();
      if (units > 0) return;
    }
    units = 0;
  }
  __device__ __forceinline__ void next(const AttnArgs &a, int pairs) {
    if (++unit < units) return;
    unit = 0;
    if (++pair < pairs) return;
    pair = 0;
    ++b;
    request(a);
  }
};

// blocks on each multiprocessor: what shared memory and registers hold
constexpr int attn_per_sm(int D, int H) { return D == 256 ? 1 : H == 8 ? 3 : 2; }

template <int D, int H, int S>
__global__ void __launch_bounds__(kWarps * 32, attn_per_sm(D, H))
    k_attn_split(const AttnArgs a, int groups) {
  after_previous<true>();
  extern __shared__ __align__(128) unsigned char raw[];
  using Smem = AttnSmem<D, H, S>;
  Smem &s = *reinterpret_cast<Smem *>(raw);
  constexpr int NT = H / 8;  // tiles of 8 query heads
  constexpr int C = D / 8;  // 16-byte parts of a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int pairs = a.Hk * groups, G = a.Hq / a.Hk, parts = a.d / 8;
  int64_t all, before;
  count_units(a, 0, s.red, all, before);
  all *= pairs;
  const int64_t share = share_of(all, gridDim.x), w0 = (int64_t)blockIdx.x * share;
  if (w0 >= all) return;
  const int64_t w1 = min(all, w0 + share);
  Cursor at;
  int64_t start;
  at.b = find_request(a, pairs, w0, s.red, s.found, start);
  at.request(a);
  at.pair = (int)((w0 - start) / at.units);
  at.unit = (int)((w0 - start) % at.units);
  Cursor ahead = at;

  // parts of a row that the head does not have are zeros for the products
  if (parts < C)
    for (int i = lane; i < S * 2 * 16 * C; i += 32)
      (&s.ring[warp][0][0][0])[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();

  // The copies of one unit.  A unit's pages are looked up while the one before it is copied.
  const __nv_bfloat16 *kp = reinterpret_cast<const __nv_bfloat16 *>(a.k.p);
  const __nv_bfloat16 *vp = reinterpret_cast<const __nv_bfloat16 *>(a.v.p);
  const bool one_page = a.page % 16 == 0;
  int page = -1;  // of key `lane` of 16 (one page: of all of them)
  auto look = [&] {
    const int key = ahead.base + ahead.unit * kUnit + warp * 16 + (one_page ? 0 : lane & 15);
    page = -1;
    if (ahead.units > 0 && key < ahead.end) page = a.table[ahead.b * a.table_st + key / a.page];
  };
  auto issue = [&](int place, bool in) -> uint32_t {  // which of the 16 keys are there
    uint32_t good = 0;
    if (in) {
      const int key0 = ahead.base + ahead.unit * kUnit + warp * 16, key = key0 + (lane & 15);
      const bool fine = key >= ahead.first && key < ahead.end && page >= 0 && page < a.pages;
      good = __ballot_sync(0xffffffffu, fine) & 0xffffu;
      const int head = ahead.pair / groups;
      uint4 *ks = s.ring[warp][place][0], *vs = s.ring[warp][place][1];
      if (one_page) {
        const int r0 = lane / C, c = lane % C;  // C <= 32
        const int at0 = key0 % a.page + r0;
        const __nv_bfloat16 *k = kp, *v = vp;
        if (good) {
          k += page * a.k.sp + at0 * a.k.st + head * a.k.sh + c * 8;
          v += page * a.v.sp + at0 * a.v.st + head * a.v.sh + c * 8;
        }
        if (c < parts) {
#pragma unroll
          for (int i = 0; i < 16 * C / 32; ++i) {
            const int r = r0 + i * (32 / C);
            const bool there = good >> r & 1;
            copy16(ks + r * C + (c ^ (r & 7)), there ? k : kp, there);
            copy16(vs + r * C + (c ^ (r & 7)), there ? v : vp, there);
            k += (32 / C) * a.k.st;
            v += (32 / C) * a.v.st;
          }
        }
      } else {
        const int at0 = key % a.page;
        const int64_t ka = fine ? page * a.k.sp + at0 * a.k.st + head * a.k.sh : 0;
        const int64_t va = fine ? page * a.v.sp + at0 * a.v.st + head * a.v.sh : 0;
#pragma unroll 2
        for (int i = 0; i < 16 * C / 32; ++i) {
          const int r = (i * 32 + lane) / C, c = (i * 32 + lane) % C;
          const int64_t kr = __shfl_sync(0xffffffffu, ka, r), vr = __shfl_sync(0xffffffffu, va, r);
          const bool there = good >> r & 1;
          if (c < parts) {
            copy16(ks + r * C + (c ^ (r & 7)), kp + kr + c * 8, there);
            copy16(vs + r * C + (c ^ (r & 7)), vp + vr + c * 8, there);
          }
        }
      }
      ahead.next(a, pairs);
      look();
    }
    copies_commit();
    return good;
  };
  look();
  uint64_t ok = 0;  // of the units on their way, 16 keys each
#pragma unroll
  for (int i = 0; i < S - 1; ++i) ok |= (uint64_t)issue(i, w0 + i < w1) << (16 * i);

  // Products with keys and values as the first factor, so that a tile of 8 heads is enough: scores
  // [16 keys, 8 heads], outputs [16 columns, 8 heads].  A lane has heads 2 t4 and 2 t4 + 1 of both.
  uint32_t q[D / 16][NT][2];
  float o[D / 16][NT][4], m[NT][2], l[NT][2];
  const float scale = a.scale * kLog2e;
  bool fresh = true;
  bool whole_start = at.unit == 0;  // the pair's first unit is in this range
  int stage = 0;
#pragma unroll 1
  for (int64_t u = w0; u < w1;) {
    const uint32_t good = (uint32_t)ok & 0xffffu;
    ok = ok >> 16 | (uint64_t)issue(stage == 0 ? S - 1 : stage - 1, u + S - 1 < w1) << (16 * (S - 2));
    copies_wait<S - 1>();
    __syncwarp();
    const int head = at.pair / groups, row0 = at.pair % groups * H;
    if (fresh) {  // a pair's queries, and nothing seen yet
      fresh = false;
      const __nv_bfloat16 *qp = reinterpret_cast<const __nv_bfloat16 *>(a.q.p) + at.b * a.q.st;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = row0 + n * 8 + g;
        const uint32_t *qh = reinterpret_cast<const uint32_t *>(qp + (int64_t)(head * G + h) * a.q.sh);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          q[k][n][0] = 16 * k < a.d && h < G ? qh[8 * k + t4] : 0;
          q[k][n][1] = 16 * k + 8 < a.d && h < G ? qh[8 * k + 4 + t4] : 0;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;
        m[n][0] = m[n][1] = low();
        l[n][0] = l[n][1] = 0.f;
      }
    }
    const uint32_t kbase = static_cast<uint32_t>(__cvta_generic_to_shared(s.ring[warp][stage][0]));
    const uint32_t vbase = static_cast<uint32_t>(__cvta_generic_to_shared(s.ring[warp][stage][1]));
    float c[NT][4];
    {
      float e[2][NT][4];  // even and odd steps: two shorter chains
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[0][n][i] = e[1][n][i] = 0.f;
      const int r = lane & 15, half = lane >> 4;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t x[4];
        ldm4(x, kbase + (r * C + ((2 * k + half) ^ (r & 7))) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(e[k & 1][n], x, q[k][n][0], q[k][n][1]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = (e[0][n][i] + e[1][n][i]) * scale;
    }
    // scores in powers of two; keys that are not there count for nothing
    if (good != 0xffffu) {
      const bool lo = good >> g & 1, hi = good >> (g + 8) & 1;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        c[n][0] = lo ? c[n][0] : low();
        c[n][1] = lo ? c[n][1] : low();
        c[n][2] = hi ? c[n][2] : low();
        c[n][3] = hi ? c[n][3] : low();
      }
    }
    bool moved = false;
    float to[NT][2], shift[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) to[n][i] = fmaxf(c[n][i], c[n][2 + i]);
#pragma unroll
    for (int w = 4; w < 32; w <<= 1)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) to[n][i] = fmaxf(to[n][i], __shfl_xor_sync(0xffffffffu, to[n][i], w));
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        to[n][i] = fmaxf(m[n][i], to[n][i]);
        moved |= to[n][i] != m[n][i];
        shift[n][i] = to[n][i] == low() ? 0.f : to[n][i];  // nothing seen: all weights 2^-inf
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = ex2(m[n][i] - shift[n][i]);
          l[n][i] *= f;
          m[n][i] = to[n][i];
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[j][n][i] *= f;
            o[j][n][2 + i] *= f;
          }
        }
    }
    uint32_t p[NT][2][3];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[n][i] = ex2(c[n][i] - shift[n][i & 1]);
        l[n][i & 1] += c[n][i];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        split3(c[n][2 * i], c[n][2 * i + 1], p[n][i]);
#pragma unroll
        for (int k = 0; k < 3; ++k) p[n][i][k] = turned(p[n][i][k]);
      }
    }
    {
      const int r = (lane & 7) + (lane >> 4) * 8, half = lane >> 3 & 1;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t x[4];
        ldm4t(x, vbase + (r * C + ((2 * j + half) ^ (r & 7))) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 3; ++k) mma(o[j][n], x, p[n][0][k], p[n][1][k]);
      }
    }
    __syncwarp();  // the ring's place is free for the copies of the next turn
    stage = stage + 1 == S ? 0 : stage + 1;
    ++u;
    const bool pair_ends = at.unit + 1 == at.units;
    if (pair_ends || u == w1) {
      // the warps' parts become one: their maxima and sums, then their outputs two by two
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          for (int w = 4; w < 32; w <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], w);
          if (g == 0) {
            s.m[warp][n * 8 + 2 * t4 + i] = m[n][i];
            s.l[warp][n * 8 + 2 * t4 + i] = l[n][i];
          }
        }
      __syncthreads();
      auto most = [&](int h) {
        float v = s.m[0][h];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = fmaxf(v, s.m[w][h]);
        return v;
      };
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float M = most(n * 8 + 2 * t4 + i), f = ex2(m[n][i] - (M == low() ? 0.f : M));
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[j][n][i] *= f;
            o[j][n][2 + i] *= f;
          }
        }
      float *mine = s.out[warp & 1];
#pragma unroll
      for (int turn = 0; turn < 2; ++turn) {
        if (warp >> 1 == 1 - turn) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float &to_ = mine[Smem::at(n * 8 + 2 * t4 + (i & 1), 16 * j + (i >> 1) * 8 + g)];
                to_ = turn == 0 ? o[j][n][i] : to_ + o[j][n][i];
              }
        }
        __syncthreads();
      }
      const int rows = min(H, G - row0);
      const bool done = pair_ends && whole_start;
      // part 0: the pair that the range starts in; part 1: the one that it ends in
      float *part = reinterpret_cast<float *>(a.work) +
                    ((int64_t)blockIdx.x * 2 + (u - (at.unit + 1) <= w0 ? 0 : 1)) * kPart<D>;
      for (int i = threadIdx.x; i < rows * (D / 2); i += kWarps * 32) {
        const int h = i / (D / 2), col = i % (D / 2) * 2, from = Smem::at(h, col);
        const float x = s.out[0][from] + s.out[1][from], y = s.out[0][from + 1] + s.out[1][from + 1];
        const float M = most(h), by = M == low() ? 0.f : M;
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) L += s.l[w][h] * ex2(s.m[w][h] - by);
        if (done) {
          const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;
          if (col < a.d) {
            __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.o.p) + at.b * a.o.st;
            *reinterpret_cast<uint32_t *>(op + (int64_t)(head * G + row0 + h) * a.o.sh + col) =
                pack2(x * inv, y * inv);
          }
        } else {
          *reinterpret_cast<float2 *>(part + h * D + col) = make_float2(x, y);
          if (col == 0) {
            part[kRows * D + h] = M;
            part[kRows * D + kRows + h] = L;
          }
        }
      }
      fresh = true;
      whole_start = true;
      __syncthreads();  // what the warps left for one another has been read
    }
    at.next(a, pairs);
  }
  copies_wait<0>();
}

// Joins the parts of the pairs that lie in several ranges, one block a query head of a pair; rows
// without keys get zeros.  The warps take every eighth part, a lane D / 32 columns.  A block looks for
// its pair by its number; where there are more pairs than ranges (BY_RANGE), by the range that the pair
// starts in, as at most one goes on behind a range's end, and most pairs have nothing to join.
constexpr int kJoin = 8;  // warps

template <int D, bool BY_RANGE>
__global__ void __launch_bounds__(kJoin * 32) k_attn_join(const AttnArgs a, int groups, int per_group, int ctas, int rows) {
  after_previous<true>();
  constexpr int N = D / 32;
  __shared__ int64_t red[32], found[2];
  __shared__ float ms[kJoin], ls[kJoin], os[kJoin][D];
  const int pairs = a.Hk * groups, G = a.Hq / a.Hk;
  const int r = blockIdx.x % rows;
  int b, pair;
  int64_t all, before;
  if (BY_RANGE) {
    const int c = blockIdx.x / rows;
    for (int i = c; i < a.B; i += ctas) {
      if (Span(a, i).units() > 0) continue;
      __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.o.p) + i * a.o.st;
      for (int p = 0; p < pairs; ++p) {
        const int h = p % groups * per_group + r;
        if (h >= G) continue;
        for (int d = threadIdx.x; d < a.d; d += kJoin * 32)
          op[(int64_t)(p / groups * G + h) * a.o.sh + d] = __float2bfloat16_rn(0.f);
      }
    }
    count_units(a, 0, red, all, before);
    const int64_t share = share_of(all * pairs, ctas), end = (c + 1) * share;
    if (end >= all * pairs) return;  // the last range
    int64_t start;
    b = find_request(a, pairs, end - 1, red, found, start);
    const int units = Span(a, b).units();
    pair = (int)((end - 1 - start) / units);
    before = start / pairs;
    if (start + (int64_t)pair * units < c * share) return;  // an earlier range's
  } else {
    b = blockIdx.x / rows / pairs, pair = blockIdx.x / rows % pairs;
    if (pair % groups * per_group + r >= G) return;
    count_units(a, b, red, all, before);
  }
  const int head = pair / groups, h = pair % groups * per_group + r;
  if (h >= G) return;
  const int units = Span(a, b).units();
  const int64_t share = share_of(all * pairs, ctas);
  const int64_t u0 = before * pairs + (int64_t)pair * units, u1 = u0 + units;
  const int64_t c0 = u0 / share, c1 = units > 0 ? (u1 - 1) / share : c0;
  if (units > 0 && c0 == c1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = low(), l = 0.f, acc[N] = {};
  if (units > 0) {
    // a range's part 0 is the pair that it starts in, part 1 the one that it ends in
    const float *w = reinterpret_cast<const float *>(a.work) + (u0 > c0 * share ? kPart<D> : 0);
    for (int64_t c = c0 + warp; c <= c1; c += 4 * kJoin) {
      float pm[4], pl[4], po[4][N];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = c + kJoin * i;
        const float *p = (at == c0 ? w : reinterpret_cast<const float *>(a.work)) + at * 2 * kPart<D>;
        const bool in = at <= c1;
        pm[i] = in ? p[kRows * D + r] : low();
        pl[i] = in ? p[kRows * D + kRows + r] : 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) po[i][j] = in ? p[r * D + j * 32 + lane] : 0.f;
      }
      float to = m;
#pragma unroll
      for (int i = 0; i < 4; ++i) to = fmaxf(to, pm[i]);
      const float by = to == low() ? 0.f : to, f = ex2(m - by);
      m = to;
      l *= f;
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g = ex2(pm[i] - by);
        l = fmaf(pl[i], g, l);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = fmaf(po[i][j], g, acc[j]);
      }
    }
  }
  if (lane == 0) {
    ms[warp] = m;
    ls[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) os[warp][j * 32 + lane] = acc[j];
  __syncthreads();
  m = ms[0];
#pragma unroll
  for (int w = 1; w < kJoin; ++w) m = fmaxf(m, ms[w]);
  const float by = m == low() ? 0.f : m;
  float f[kJoin];
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoin; ++w) {
    f[w] = ex2(ms[w] - by);
    l = fmaf(ls[w], f[w], l);
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.o.p) + b * a.o.st + (int64_t)(head * G + h) * a.o.sh;
  for (int c = threadIdx.x; c < a.d; c += kJoin * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kJoin; ++w) v = fmaf(os[w][c], f[w], v);
    op[c] = __float2bfloat16_rn(v * inv);
  }
}

// ------------------------------------------------------------------ any type, size and alignment
//
// One block for a request's query head: its warps take every 16th key, a lane 8 of the head's
// elements.  Every query head reads its keys again, and one request fills as many blocks as it has heads:
// far from the bytes (64 requests of 4,096 keys, 32 / 4 heads of 128: 2,131 us in fp32 for 158, 2,002 in bf16 off
// 16 bytes for 79; one of 32,768 keys, 32 / 8 heads, in fp32: 2,363 for 40).

constexpr int kPlainWarps = 16;

template <typename E>
__global__ void __launch_bounds__(kPlainWarps * 32) k_attn_plain(const AttnArgs a) {
  after_previous();
  __shared__ float out[kPlainWarps][257], ms[kPlainWarps], ls[kPlainWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.Hk);
  const Span span(a, b);
  const E *q = reinterpret_cast<const E *>(a.q.p) + b * a.q.st + h * a.q.sh;
  float qs[8], o[8], m = low(), l = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    qs[i] = lane + 32 * i < a.d ? ld1(q + lane + 32 * i) * (a.scale * kLog2e) : 0.f;
    o[i] = 0.f;
  }
  for (int64_t key = (int64_t)span.first + warp; key < span.end; key += kPlainWarps) {
    const int page = a.table[b * a.table_st + key / a.page];
    if (page < 0 || page >= a.pages) continue;
    const int64_t place = key % a.page;
    const E *k = reinterpret_cast<const E *>(a.k.p) + page * a.k.sp + place * a.k.st + hk * a.k.sh;
    const E *v = reinterpret_cast<const E *>(a.v.p) + page * a.v.sp + place * a.v.st + hk * a.v.sh;
    float x[8], c = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = lane + 32 * i < a.d;
      c = in ? fmaf(qs[i], ld1(k + lane + 32 * i), c) : c;
      x[i] = in ? ld1(v + lane + 32 * i) : 0.f;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) c += __shfl_xor_sync(0xffffffffu, c, s);
    const float to = fmaxf(m, c), by = to == low() ? 0.f : to;
    const float f = ex2(m - by), p = ex2(c - by);
    m = to;
    l = fmaf(l, f, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(o[i], f, p * x[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) out[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    ms[warp] = m;
    ls[warp] = l;
  }
  __syncthreads();
  float M = low(), L = 0.f;
#pragma unroll
  for (int w = 0; w < kPlainWarps; ++w) M = fmaxf(M, ms[w]);
  const float by = M == low() ? 0.f : M;
#pragma unroll
  for (int w = 0; w < kPlainWarps; ++w) L += ls[w] * ex2(ms[w] - by);
  const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;
  for (int c = threadIdx.x; c < a.d; c += kPlainWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kPlainWarps; ++w) v = fmaf(out[w][c], ex2(ms[w] - by), v);
    st1(reinterpret_cast<E *>(a.o.p) + b * a.o.st + h * a.o.sh + c, v * inv);
  }
}

// ------------------------------------------------------------------ launches

int wide_for(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
int ctas_for(int D, int H) { return min(kMostCtas, sm_count() * attn_per_sm(D, H)); }

template <int D, int H, int S>
cudaError_t run_split(const AttnArgs &a, cudaStream_t stream) {
  const int G = a.Hq / a.Hk, groups = (G + H - 1) / H, ctas = ctas_for(D, H);
  constexpr int smem = sizeof(AttnSmem<D, H, S>);
  static_assert((smem + 1024) * attn_per_sm(D, H) <= 228 * 1024, "shared memory of the blocks");
  static std::atomic<uint64_t> done{0};
  cudaError_t e =
      set_once(k_attn_split<D, H, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
  if (e != cudaSuccess) return e;
  e = launch(k_attn_split<D, H, S>, (unsigned)ctas, kWarps * 32, smem, stream, a, groups);
  if (e != cudaSuccess) return e;
  const int rows = G < H ? G : H;
  const int64_t all = (int64_t)a.B * a.Hk * groups;
  if (all <= ctas)
    return launch(k_attn_join<D, false>, (unsigned)(all * rows), kJoin * 32, 0, stream, a, groups, H,
                  ctas, rows);
  return launch(k_attn_join<D, true>, (unsigned)(ctas * rows), kJoin * 32, 0, stream, a, groups, H,
                ctas, rows);
}

bool fits16(const Pages &h) {
  return reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.sp % 8 == 0 && h.st % 8 == 0 && h.sh % 8 == 0;
}
bool fits4(const Heads &h) {
  return reinterpret_cast<uintptr_t>(h.p) % 4 == 0 && h.st % 2 == 0 && h.sh % 2 == 0;
}

}  // namespace
}  // namespace mix

size_t attn_workspace(int32_t B, int32_t Hq, int32_t Hk, int32_t d) {
  const int D = mix::wide_for(d);
  return align256((size_t)mix::ctas_for(D, 8) * 2 * (mix::kRows * D + 2 * mix::kRows) * 4);
}

cudaError_t launch_attn_step(const AttnArgs &a, cudaStream_t stream) {
  if (a.B == 0) return cudaSuccess;
  // (a cache without pages has no address that a copy, even of nothing, may name)
  if (!a.f32 && a.pages > 0 && a.d % 8 == 0 && mix::fits16(a.k) && mix::fits16(a.v) && mix::fits4(a.q) &&
      mix::fits4(a.o)) {
    if (a.Hq / a.Hk <= 8) {
      if (a.d <= 64) return mix::run_split<64, 8, 4>(a, stream);
      if (a.d <= 128) return mix::run_split<128, 8, 2>(a, stream);
      return mix::run_split<256, 8, 3>(a, stream);
    }
    if (a.d <= 64) return mix::run_split<64, 16, 5>(a, stream);
    if (a.d <= 128) return mix::run_split<128, 16, 3>(a, stream);
    return mix::run_split<256, 16, 2>(a, stream);
  }
  const unsigned blocks = (unsigned)((int64_t)a.B * a.Hq);
  return a.f32 ? mix::launch(mix::k_attn_plain<float>, blocks, mix::kPlainWarps * 32, 0, stream, a)
               : mix::launch(mix::k_attn_plain<__nv_bfloat16>, blocks, mix::kPlainWarps * 32, 0,
                             stream, a);
}

}  // namespace gdr
