// gdr_cache.cu -- the bookkeeping of a paged key-value cache on the GPU: pages and slots of new tokens,
// and their keys and values written into the pages.  Both are bound by launch latency for single
// tokens; writing a prompt's rows is bound by HBM.  256 requests of one token, plan and write: 8.9 us, the
// host side of two calls.  12 prompts of up to 2,500 tokens x 8 x 128 in bf16: 24 us for 15 of bytes, three
// kernels in turn.
#include "gdr_block.cuh"

namespace gdr {
namespace mix {
namespace {

constexpr int kPlan = 1024;  // requests of a round, one a thread

// Inclusive sums over the block's threads, and the block's total.  red: 32 values.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *red, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // red is free
  if (lane == 31) red[warp] = v;
  __syncthreads();
  int64_t w = lane < warps ? red[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return warp > 0 ? v + before : v;
}

// The first of n rows that ends behind x (ends do not decrease).
__device__ __forceinline__ int row_of_place(const int *ends, int n, int64_t x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] <= x) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t slot_of(const PlanArgs &a, int row, int pos) {
  const int page = a.table[row * a.table_st + pos / a.page];
  const int64_t slot = (int64_t)page * a.page + pos % a.page;
  return page >= 0 && slot <= 0x7fffffff ? (int32_t)slot : -1;
}

// One block.  Requests in rounds of one a thread; what a request may take depends on those before it
// through three running sums: tokens asked for, pages needed, tokens granted.
__global__ void __launch_bounds__(kPlan) k_cache_plan(const PlanArgs a, int tokens_too) {
  after_previous<true>();
  __shared__ int64_t red[32];
  __shared__ int page_end[kPlan], tok_end[kPlan], had[kPlan], len0[kPlan];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int64_t room = (int64_t)a.width * a.page;
  const int used = min(max(*a.taken, 0), a.nfree);
  const int64_t left = a.nfree - used;
  int64_t asked = 0, needed = 0, granted = 0;  // of the rounds before
  for (int base = 0; base < a.B; base += nt) {
    const int i = base + tid, rows = min(nt, a.B - base);
    int64_t len = 0, n = 0, total;
    if (i < a.B) {
      len = max(a.lens[i], 0);
      n = max((int64_t)0, min((int64_t)a.fresh[i], room - len));
    }
    int64_t end = asked + block_scan(n, red, total);
    n = min(end, (int64_t)a.most) - min(end - n, (int64_t)a.most);
    asked += total;
    const int64_t have = (len + a.page - 1) / a.page;
    const int64_t need = n > 0 ? (len + n + a.page - 1) / a.page - have : 0;
    end = needed + block_scan(need, red, total);
    const int64_t start = min(end - need, left), got = min(end, left) - start;
    const int p0 = (int)min(needed, left);  // pages of the rounds before, and with this one
    needed += total;
    const int p1 = (int)min(needed, left);
    n = max((int64_t)0, min(n, (have + got) * a.page - len));
    end = granted + block_scan(n, red, total);
    page_end[tid] = (int)(start + got);
    tok_end[tid] = (int)end;
    had[tid] = (int)min(have, (int64_t)0x7fffffff);
    len0[tid] = (int)len;
    if (i < a.B) {
      a.cu[i + 1] = (int)end;
      a.lens_out[i] = (int)(len + n);
      if (i == 0) a.cu[0] = 0;
    }
    const int64_t tok0 = granted;
    granted += total;
    __syncthreads();
    // new pages of these requests, in their order
    for (int p = p0 + tid; p < p1; p += nt) {
      const int r = row_of_place(page_end, rows, p);
      const int before = r > 0 ? page_end[r - 1] : p0;
      a.table[(int64_t)(base + r) * a.table_st + had[r] + (p - before)] = a.free_pages[used + p];
    }
    __syncthreads();
    if (tokens_too) {
      for (int64_t t = tok0 + tid; t < granted; t += nt) {
        const int r = row_of_place(tok_end, rows, t);
        const int pos = len0[r] + (int)(t - (r > 0 ? tok_end[r - 1] : tok0));
        a.positions[t] = pos;
        a.slots[t] = slot_of(a, base + r, pos);
      }
      __syncthreads();
    }
  }
  if (tid == 0) {
    *a.taken_out = used + (int)min(needed, left);
    if (a.B == 0) a.cu[0] = 0;
  }
  if (tokens_too)
    for (int64_t t = granted + tid; t < a.most; t += nt) {
      a.positions[t] = 0;
      a.slots[t] = -1;
    }
}

// Slots and positions of many tokens, one a thread.
__global__ void __launch_bounds__(256) k_cache_slots(const PlanArgs a) {
  after_previous();
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.most) return;
  int pos = 0, slot = -1;
  if (a.B > 0 && t < a.cu[a.B]) {
    const int r = row_of_place(a.cu + 1, a.B, t);
    pos = a.lens_out[r] - (a.cu[r + 1] - (int)t);
    slot = slot_of(a, r, pos);
  }
  a.positions[t] = pos;
  a.slots[t] = slot;
}

// U: a unit of copying.  A warp a token: four units a lane of keys and of values are on their way
// before the slot is looked at.
template <typename U>
__global__ void __launch_bounds__(256) k_cache_write(const WriteArgs a, int per_head) {
  after_previous<true>();
  const int lane = threadIdx.x & 31, units = a.Hk * per_head;
  constexpr int E = sizeof(U);
  const int e = a.f32 ? 4 : 2;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t < a.T) {
    const int slot = a.slots[t];
    const char *k = reinterpret_cast<const char *>(a.k.p) + t * a.k.st * e;
    const char *v = reinterpret_cast<const char *>(a.v.p) + t * a.v.st * e;
    for (int base = 0; base < units; base += 128) {
      U x[4], y[4];
      int h[4];
      int64_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = base + j * 32 + lane;
        if (i >= units) continue;
        h[j] = i / per_head;
        c[j] = (int64_t)(i - h[j] * per_head) * E;
        x[j] = *reinterpret_cast<const U *>(k + h[j] * a.k.sh * e + c[j]);
        y[j] = *reinterpret_cast<const U *>(v + h[j] * a.v.sh * e + c[j]);
      }
      const int page = slot / a.page, place = slot % a.page;
      if (slot < 0 || page >= a.pages) break;
      char *kc = reinterpret_cast<char *>(a.kc.p) + (page * a.kc.sp + place * a.kc.st) * e;
      char *vc = reinterpret_cast<char *>(a.vc.p) + (page * a.vc.sp + place * a.vc.st) * e;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (base + j * 32 + lane >= units) continue;
        *reinterpret_cast<U *>(kc + h[j] * a.kc.sh * e + c[j]) = x[j];
        *reinterpret_cast<U *>(vc + h[j] * a.vc.sh * e + c[j]) = y[j];
      }
    }
  }
}

bool fits16(const Heads &h, int e) {
  return reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.st * e % 16 == 0 && h.sh * e % 16 == 0;
}
bool fits16(const Pages &h, int e) {
  return reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.sp * e % 16 == 0 && h.st * e % 16 == 0 &&
         h.sh * e % 16 == 0;
}

}  // namespace
}  // namespace mix

cudaError_t launch_cache_plan(const PlanArgs &a, cudaStream_t stream) {
  // few tokens: all in one launch (a block writes some 2,000 in the time of a second launch)
  const int both = a.most <= 4096;
  // a small block starts sooner and has shorter sums (256 requests of a token: 3.3 us, 4.5 with 1,024
  // threads), and writes many tokens more slowly (1,024 of them: 5.2 and 4.8)
  const int threads = a.B <= 256 && a.most <= 1024 ? 256 : mix::kPlan;
  const cudaError_t e = mix::launch(mix::k_cache_plan, 1, threads, 0, stream, a, both);
  if (e != cudaSuccess || both) return e;
  return mix::launch(mix::k_cache_slots, (unsigned)ceil_div64(a.most, 256), 256, 0, stream, a);
}

cudaError_t launch_cache_write(const WriteArgs &a, cudaStream_t stream) {
  if (a.T == 0 || a.pages == 0) return cudaSuccess;
  const int e = a.f32 ? 4 : 2;
  const unsigned grid = (unsigned)ceil_div64(a.T, 8);
  if (a.d * e % 16 == 0 && mix::fits16(a.k, e) && mix::fits16(a.v, e) && mix::fits16(a.kc, e) &&
      mix::fits16(a.vc, e))
    return mix::launch(mix::k_cache_write<uint4>, grid, 256, 0, stream, a, a.d * e / 16);
  return a.f32 ? mix::launch(mix::k_cache_write<uint32_t>, grid, 256, 0, stream, a, a.d)
               : mix::launch(mix::k_cache_write<uint16_t>, grid, 256, 0, stream, a, a.d);
}

}  // namespace gdr
