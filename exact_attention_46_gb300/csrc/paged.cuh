// paged.cuh -- what the kernels of attention over a paged cache share: the list of key tiles and how
// it is cut over the CTAs, and the asynchronous copies outside TMA.
//
// A unit is (sequence, key/value head); its keys are cut into 128-key tiles.  The tiles of all units, in
// the order sequence, key/value head, key, form one list, every unit led by p.lead empty entries that
// stand for the time a CTA takes to change units; of the W entries group i of N takes [i W / N,
// (i + 1) W / N).  A group is one CTA, or one per tile of packed query rows where there are several:
// its CTAs go through the same keys at the same time, so all but the first find them in L2.
// Everything is computed from the lengths on the device.
#pragma once

#include <cstdint>

#include "cache.h"
#include "ptx.cuh"

namespace ea46 {

constexpr float LN2_P = 0.69314718055994530942f;
enum : int { WHERE_PAGED_LOAD = 51, WHERE_PAGED_USE = 52, WHERE_PAGED_LENS = 53, WHERE_PAGED_PAGE = 54,
             WHERE_PAGED_MMA = 55 };

// Loads of what another kernel of the same stream wrote: ordered after the wait for it, past L1.  (The
// kernels here may start before that kernel has ended, so they use no read-only-cache loads, which the
// compiler may move above the wait.)
__device__ __forceinline__ float ld_l2(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ float2 ld_l2(const float2* p) {
  float2 v;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_l2(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ int4 ld_l2(const int4* p) {
  int4 v;
  asm volatile("ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// 16-byte asynchronous copy global -> shared, and an arrival on `bar` when this thread's copies so
// far have landed (counted in the barrier's initial count).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void wait_drain_paged(uint32_t bar, uint32_t parity, long long limit) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit) return;
}

// List entries of sequence b, per key/value head; ok becomes false if its lengths are out of range.
__device__ __forceinline__ int tiles_of(const PagedParams& p, int b, bool& ok) {
  const int ctx = *(p.ctx_lens + b), ql = p.q_lens != nullptr ? *(p.q_lens + b) : p.T;
  const bool fine = ctx >= 0 && ql >= 0 && ql <= p.T &&
                    static_cast<long long>(ctx) + ql <= static_cast<long long>(p.max_pages) * p.page_size;
  ok = ok && fine;
  return fine && ql > 0 ? ((ctx + ql + 127) >> 7) + p.lead : 0;
}

// Prefix sums of the sequences' list entries into pre[0 .. B]; returns 0 if any length is out of
// range.  Called by all `n` threads of the block (a multiple of 32, at most 1024).
__device__ __forceinline__ bool tile_prefix(const PagedParams& p, int* pre, int* scratch, int n) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool ok = true;
  if (p.B <= 32) {                             // every warp sums for itself
    int incl = lane < p.B ? tiles_of(p, lane, ok) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (warp == 0 && lane < p.B) pre[lane + 1] = incl;
    if (tid == 0) pre[0] = 0;
    ok = __all_sync(0xffffffffu, ok);
    __syncthreads();
    return ok;
  }
  const int per = (p.B + n - 1) / n, b0 = tid * per, b1 = min(p.B, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int tiles = tiles_of(p, b, ok);
    pre[b + 1] = tiles;                       // own entries only, until the scan below
    sum += tiles;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scratch[warp] = incl;
  ok = __syncthreads_and(ok);
  int off = incl - sum;
  for (int w = 0; w < warp; ++w) off += scratch[w];
  for (int b = b0; b < b1; ++b) {
    off += pre[b + 1];
    pre[b + 1] = off;
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  return ok;
}

// The piece of the list that starts at x and ends at x1 or with its unit.
struct Segment {
  int b, hkv;           // sequence, key/value head
  int t0, t1, n;        // tiles [t0, t1) of the unit's n (none where the piece holds lead entries only)
  int len;              // list entries
};

// x / y for y > 0, in 32 bits where both fit (the 64-bit division is a few hundred cycles).
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// Token of packed row r: r / G by multiplication (r, G < 2^16).
__device__ __forceinline__ int token_of(const PagedParams& p, int r) {
  return p.g_magic == 0 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), p.g_magic));
}

__device__ __forceinline__ Segment find_segment(const PagedParams& p, const int* pre, long long x, long long x1) {
  const long long hr = p.Hkv;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * hr <= x) lo = mid; else hi = mid;
  }
  // x lies in sequence lo: empty ones before it have pre[lo + 1] == pre[lo]
  Segment s;
  s.b = lo;
  const int all = pre[lo + 1] - pre[lo];
  const long long y = x - pre[lo] * hr;
  s.hkv = static_cast<int>(quotient(y, all));
  const int at = static_cast<int>(y - static_cast<long long>(s.hkv) * all);
  const long long left = x1 - x;
  s.len = left < all - at ? static_cast<int>(left) : all - at;
  s.n = all - p.lead;
  s.t0 = max(0, at - p.lead);
  s.t1 = max(0, at + s.len - p.lead);
  return s;
}

// The next piece with tiles in it, from x on; x becomes its end.  False: none before x1.
__device__ __forceinline__ bool next_segment(const PagedParams& p, const int* pre, long long& x, long long x1, Segment& s) {
  while (x < x1) {
    s = find_segment(p, pre, x, x1);
    x += s.len;
    if (s.t1 > s.t0) return true;
  }
  return false;
}

__device__ __forceinline__ long long cta_start(long long i, long long W, long long N) { return quotient(i * W, N); }

// What the merge has to do about the start of group i's tiles (i > 0): where that is the first cut inside a
// unit, the unit and the number of its parts (groups i - 1 ..); otherwise no parts.  One thread.
__device__ __forceinline__ void write_cut(const PagedParams& p, const int* pre, int i, long long W, long long N) {
  if (p.cuts == nullptr || i == 0) return;
  int4 c = make_int4(0, 0, 0, 0);
  if (i < N) {
    const long long x = cta_start(i, W, N);
    const Segment s = find_segment(p, pre, x, W);
    // the group that holds list position y is the last c with c W / N <= y; x - t0 is tile 0's
    const long long c0 = quotient((x - s.t0 + 1) * N - 1, W), c1 = quotient((x - s.t0 + s.n) * N - 1, W);
    if (s.t0 > 0 && c0 == i - 1)
      c = make_int4(static_cast<int>(c1 - c0) + 1, s.b, s.hkv, p.q_lens != nullptr ? *(p.q_lens + s.b) : p.T);
  }
  p.cuts[i] = c;
}

}  // namespace ea46
