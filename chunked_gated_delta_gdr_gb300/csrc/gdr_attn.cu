// gdr_attn.cu -- attention of one new token for each request over a paged key-value cache:
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = e^{scale q.k_j - max},  j over the request's last keys.
//
// Bound by HBM: keys and values are read once, for all of the query heads that share them.
// The work is cut over the keys, whatever the requests' lengths are: all (request, head) pairs' keys
// in a row, in units of 64, are dealt to the blocks in equal ranges, which every block finds from
// the lengths on the device.  A block keeps a running maximum, sum and output for each pair in its
// range; a pair that lies in one range is finished there, parts of others are joined by a second
// kernel, in order.
//
// A warp takes 16 keys of a unit: its rows come by cp.async into a ring of its own, so that no barrier
// is needed before a range's end, and go through mma.sync (16 query rows, of which a group of fewer
// heads leaves some empty): its rate is far above what HBM feeds, and one instruction needs no
// accumulator in Tensor Memory that the softmax would have to fetch.  Scores, maxima, sums and
// outputs are fp32; the probabilities go to the second product as two bf16 parts each, whose error is
// 2^-17 instead of 2^-9.
#include "gdr_block.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kRows = 16;           // query heads of a pair
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
// two values as bf16, and what that leaves of them
__device__ __forceinline__ uint32_t split2(float x, float y, uint32_t &rest) {
  const uint32_t hi = pack2(x, y);
  rest = pack2(x - lo_bf(hi), y - hi_bf(hi));
  return hi;
}

// ------------------------------------------------------------------ the split kernel

// One (request, key head, 16 of its query heads); parts in the workspace are O [16][D], m and l [16].
template <int D>
constexpr int kPart = kRows * D + 2 * kRows;

template <int D, int S>
struct AttnSmem {
  uint4 ring[kWarps][S][2][16 * D / 8];  // each warp's keys and values, rows of 16-byte parts
  float out[2][kRows * D];
  float m[kWarps][kRows], l[kWarps][kRows];
  int64_t red[32], found[2];
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

template <int D, int S>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 1 : 2)
    k_attn_split(const AttnArgs a, int groups, int rows) {
  after_previous<true>();
  extern __shared__ __align__(128) unsigned char raw[];
  AttnSmem<D, S> &s = *reinterpret_cast<AttnSmem<D, S> *>(raw);
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

  uint32_t q[D / 16][4];
  float o[D / 8][4], m[2], l[2];
  const float scale = a.scale * kLog2e;
  bool fresh = true;
  bool whole_start = at.unit == 0;  // the pair's first unit is in this range
  int stage = 0;
#pragma unroll 1
  for (int64_t u = w0; u < w1;) {
    {
      const uint32_t good = (uint32_t)ok & 0xffffu;
      ok = ok >> 16 | (uint64_t)issue(stage == 0 ? S - 1 : stage - 1, u + S - 1 < w1) << (16 * (S - 2));
      copies_wait<S - 1>();
      __syncwarp();
      const int head = at.pair / groups, row0 = at.pair % groups * kRows;
      if (fresh) {  // a pair's queries, and nothing seen yet
        fresh = false;
        const __nv_bfloat16 *qp = reinterpret_cast<const __nv_bfloat16 *>(a.q.p) + at.b * a.q.st;
        const int h0 = row0 + g, h1 = row0 + g + 8;
        const uint32_t *q0 = reinterpret_cast<const uint32_t *>(qp + (int64_t)(head * G + h0) * a.q.sh);
        const uint32_t *q1 = reinterpret_cast<const uint32_t *>(qp + (int64_t)(head * G + h1) * a.q.sh);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const bool lo = 16 * k < a.d, hi = 16 * k + 8 < a.d;
          q[k][0] = lo && h0 < G ? q0[8 * k + t4] : 0;
          q[k][1] = lo && h1 < G ? q1[8 * k + t4] : 0;
          q[k][2] = hi && h0 < G ? q0[8 * k + 4 + t4] : 0;
          q[k][3] = hi && h1 < G ? q1[8 * k + 4 + t4] : 0;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        m[0] = m[1] = low();
        l[0] = l[1] = 0.f;
      }
      const uint4 *ks = s.ring[warp][stage][0], *vs = s.ring[warp][stage][1];
      const uint32_t kbase = static_cast<uint32_t>(__cvta_generic_to_shared(ks));
      const uint32_t vbase = static_cast<uint32_t>(__cvta_generic_to_shared(vs));
      float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int r = (lane & 7) + (lane >> 4) * 8, half = lane >> 3 & 1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          ldm4(b, kbase + (r * C + ((2 * k + half) ^ (r & 7))) * 16);
          mma(c[0], q[k], b[0], b[1]);
          mma(c[1], q[k], b[2], b[3]);
        }
      }
      // scores in powers of two; keys that are not there count for nothing
      float top[2] = {low(), low()};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[n][e] *= scale;
          if (good != 0xffffu && !(good >> (8 * n + 2 * t4 + (e & 1)) & 1)) c[n][e] = low();
          top[e >> 1] = fmaxf(top[e >> 1], c[n][e]);
        }
      bool moved = false;
      float to[2], shift[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        to[i] = fmaxf(m[i], top[i]);
        moved |= to[i] != m[i];
        shift[i] = to[i] == low() ? 0.f : to[i];  // nothing seen: all weights 2^-inf
      }
      if (__any_sync(0xffffffffu, moved)) {
        const float f0 = ex2(m[0] - shift[0]), f1 = ex2(m[1] - shift[1]);
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
        m[0] = to[0];
        m[1] = to[1];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[n][e] = ex2(c[n][e] - shift[e >> 1]);
          l[e >> 1] += c[n][e];
        }
      uint32_t p[4], rest[4];
      p[0] = split2(c[0][0], c[0][1], rest[0]);
      p[1] = split2(c[0][2], c[0][3], rest[1]);
      p[2] = split2(c[1][0], c[1][1], rest[2]);
      p[3] = split2(c[1][2], c[1][3], rest[3]);
      {
        const int r = lane & 15, half = lane >> 4;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t b[4];
          ldm4t(b, vbase + (r * C + ((2 * j + half) ^ (r & 7))) * 16);
          mma(o[2 * j], p, b[0], b[1]);
          mma(o[2 * j + 1], p, b[2], b[3]);
          mma(o[2 * j], rest, b[0], b[1]);
          mma(o[2 * j + 1], rest, b[2], b[3]);
        }
      }
      __syncwarp();  // the ring's place is free for the copies of the next turn
      stage = stage + 1 == S ? 0 : stage + 1;
      ++u;
      const bool pair_ends = at.unit + 1 == at.units;
      if (pair_ends || u == w1) {
        // the warps' parts become one: their maxima and sums, then their outputs two by two
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        if (t4 == 0) {
          s.m[warp][g] = m[0];
          s.m[warp][g + 8] = m[1];
          s.l[warp][g] = l[0];
          s.l[warp][g + 8] = l[1];
        }
        __syncthreads();
        float M[2], L[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = g + 8 * i;
          M[i] = s.m[0][r];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) M[i] = fmaxf(M[i], s.m[w][r]);
          const float by = M[i] == low() ? 0.f : M[i];
          L[i] = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) L[i] += s.l[w][r] * ex2(s.m[w][r] - by);
          const float f = ex2(m[i] - by);
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][2 * i] *= f;
            o[j][2 * i + 1] *= f;
          }
        }
        auto place = [&](int slot, int r, int j) {
          return reinterpret_cast<float2 *>(&s.out[slot][r * D + ((j * 8 + 2 * t4) ^ ((r & 3) << 3))]);
        };
        auto give = [&](int slot) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            *place(slot, g, j) = make_float2(o[j][0], o[j][1]);
            if (rows > 8) *place(slot, g + 8, j) = make_float2(o[j][2], o[j][3]);
          }
        };
        auto take = [&](int slot) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            const float2 x = *place(slot, g, j);
            o[j][0] += x.x;
            o[j][1] += x.y;
            if (rows > 8) {
              const float2 y = *place(slot, g + 8, j);
              o[j][2] += y.x;
              o[j][3] += y.y;
            }
          }
        };
        if (warp >= 2) give(warp - 2);
        __syncthreads();
        if (warp < 2) take(warp);
        if (warp == 1) give(1);
        __syncthreads();
        if (warp == 0) {
          take(1);
          if (pair_ends && whole_start) {
            __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.o.p) + at.b * a.o.st;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int h = row0 + g + 8 * i;
              if (h >= G) continue;
              const float inv = L[i] > 0.f ? 1.f / L[i] : L[i] == 0.f ? 0.f : L[i];
              uint32_t *to_ = reinterpret_cast<uint32_t *>(op + (int64_t)(head * G + h) * a.o.sh);
#pragma unroll
              for (int j = 0; j < D / 8; ++j)
                if (8 * j < a.d)
                  to_[4 * j + t4] = pack2(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
            }
          } else {
            // part 0: the pair that the range starts in; part 1: the one that it ends in
            const bool first = u - (at.unit + 1) <= w0;
            float *w = reinterpret_cast<float *>(a.work) +
                       ((int64_t)blockIdx.x * 2 + (first ? 0 : 1)) * kPart<D>;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = g + 8 * i;
#pragma unroll
              for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<float2 *>(w + r * D + j * 8 + 2 * t4) =
                    make_float2(o[j][2 * i], o[j][2 * i + 1]);
              if (t4 == 0) {
                w[kRows * D + r] = M[i];
                w[kRows * D + kRows + r] = L[i];
              }
            }
          }
        }
        fresh = true;
        whole_start = true;
      }
      at.next(a, pairs);
    }
  }
  copies_wait<0>();
}

// Joins the parts of the pairs that lie in several ranges, one block a pair and query head; rows
// without keys get zeros.  The warps take every fourth part, a lane D / 32 columns.
template <int D>
__global__ void __launch_bounds__(128) k_attn_join(const AttnArgs a, int groups, int ctas, int rows) {
  after_previous<true>();
  constexpr int N = D / 32;
  __shared__ int64_t red[32];
  __shared__ float ms[4], ls[4], os[4][D];
  const int pairs = a.Hk * groups, G = a.Hq / a.Hk;
  const int r = blockIdx.x % rows, b = blockIdx.x / rows / pairs, pair = blockIdx.x / rows % pairs;
  const int head = pair / groups, h = pair % groups * kRows + r;
  if (h >= G) return;
  int64_t all, before;
  count_units(a, b, red, all, before);
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
    for (int64_t c = c0 + warp; c <= c1; c += 16) {
      float pm[4], pl[4], po[4][N];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = c + 4 * i;
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
  m = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]));
  const float by = m == low() ? 0.f : m;
  float f[4];
  l = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = ex2(ms[w] - by);
    l = fmaf(ls[w], f[w], l);
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.o.p) + b * a.o.st + (int64_t)(head * G + h) * a.o.sh;
  for (int c = threadIdx.x; c < a.d; c += 128) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v = fmaf(os[w][c], f[w], v);
    op[c] = __float2bfloat16_rn(v * inv);
  }
}

// ------------------------------------------------------------------ any type, size and alignment
//
// One block for a request's query head: its warps take every 16th key, a lane 8 of the head's
// elements.

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
int ctas_for(int D) { return min(kMostCtas, sm_count() * (D == 256 ? 1 : 2)); }

template <int D, int S>
cudaError_t run_split(const AttnArgs &a, cudaStream_t stream) {
  const int G = a.Hq / a.Hk, groups = (G + kRows - 1) / kRows, ctas = ctas_for(D);
  constexpr int smem = sizeof(AttnSmem<D, S>);
  static_assert(smem <= (D == 256 ? 227 : 113) * 1024, "shared memory of a block");
  static std::atomic<uint64_t> done{0};
  cudaError_t e =
      set_once(k_attn_split<D, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
  if (e != cudaSuccess) return e;
  e = launch(k_attn_split<D, S>, (unsigned)ctas, kWarps * 32, smem, stream, a, groups,
             G < kRows ? G : kRows);
  if (e != cudaSuccess) return e;
  const int rows = G < kRows ? G : kRows;
  return launch(k_attn_join<D>, (unsigned)((int64_t)a.B * a.Hk * groups * rows), 128, 0, stream, a, groups,
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
  return align256((size_t)mix::ctas_for(D) * 2 * (mix::kRows * D + 2 * mix::kRows) * 4);
}

cudaError_t launch_attn_step(const AttnArgs &a, cudaStream_t stream) {
  if (a.B == 0) return cudaSuccess;
  if (!a.f32 && a.d % 8 == 0 && mix::fits16(a.k) && mix::fits16(a.v) && mix::fits4(a.q) &&
      mix::fits4(a.o)) {
    if (a.d <= 64) return mix::run_split<64, 5>(a, stream);
    if (a.d <= 128) return mix::run_split<128, 3>(a, stream);
    return mix::run_split<256, 3>(a, stream);
  }
  const unsigned blocks = (unsigned)((int64_t)a.B * a.Hq);
  return a.f32 ? mix::launch(mix::k_attn_plain<float>, blocks, mix::kPlainWarps * 32, 0, stream, a)
               : mix::launch(mix::k_attn_plain<__nv_bfloat16>, blocks, mix::kPlainWarps * 32, 0,
                             stream, a);
}

}  // namespace gdr
