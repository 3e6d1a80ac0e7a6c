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
#include <cuda_bf16.h>

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

// Units of more parts than this are merged by the blocks of all their cuts, others by those of the first.
constexpr int MANY_PARTS = 8;

// What the merge has to do about the start of group i's tiles (i > 0), one thread: the unit cut there, if it is the
// unit's first cut or one of many, as its parts (of groups i - 1 - k ..) + (k << 16), sequence, key/value head and
// q_len; k counts the unit's cuts before this one.  Otherwise no parts.
__device__ __forceinline__ void write_cut(const PagedParams& p, const int* pre, int i, long long W, long long N) {
  if (p.cuts == nullptr || i == 0) return;
  int4 c = make_int4(0, 0, 0, 0);
  if (i < N) {
    const long long x = cta_start(i, W, N);
    const Segment s = find_segment(p, pre, x, W);
    if (s.t0 > 0) {
      // the group that holds list position y is the last c with c W / N <= y; x - t0 is tile 0's
      const int c0 = static_cast<int>(quotient((x - s.t0 + 1) * N - 1, W));
      const int parts = static_cast<int>(quotient((x - s.t0 + s.n) * N - 1, W)) - c0 + 1;
      if (c0 == i - 1 || parts > MANY_PARTS)
        c = make_int4(parts + ((i - 1 - c0) << 16), s.b, s.hkv, p.q_lens != nullptr ? *(p.q_lens + s.b) : p.T);
    }
  }
  p.cuts[i] = c;
}

// ---- E4M3 terms ----

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// x (two fp16) as two E4M3 terms: hi = E4M3(x), lo = E4M3(x - hi); the pairs in the low 16 bits.
__device__ __forceinline__ void e4m3_terms(uint32_t x, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 b, d;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 b, h;\n\t"
      "sub.rn.f16x2 d, %2, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, d;\n\t"
      "cvt.u32.u16 %0, h;\n\tcvt.u32.u16 %1, l;\n\t}"
      : "=r"(hi), "=r"(lo) : "r"(x));
}

__device__ __forceinline__ void e4m3_terms4(float a, float b, float c, float d, uint32_t& hi, uint32_t& lo) {
  uint32_t h0, l0, h1, l1;
  e4m3_terms(f16x2(a, b), h0, l0);
  e4m3_terms(f16x2(c, d), h1, l1);
  hi = __byte_perm(h0, h1, 0x5410);
  lo = __byte_perm(l0, l1, 0x5410);
}

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) < INFINITY; }

// Numerators over an E4M3 cache in the kernels on tcgen05: lazily rescaled when they pass 2^TAU (log2), scaled by
// 2^(15 - TAU), so that the sum of their terms spans E5M2's [2^-17, 2^15]: of a sequence of 2^17 keys that lie
// 2^-20 under one other, none is lost.  (E4M3 terms span 2^19 and lose them.)
constexpr float TAU_E4M3 = 4.0f, TOP_E4M3 = 2048.0f;

// Four numerators in [0, 2^15] as three E5M2 terms (packed bytes): fp16 first (2^-11), whose upper byte is
// the first term, the remainder's upper byte the second, and what is left then rounded: each takes three bits
// at least, so the sum is off by 2^-9 of the number, or 2^-17, half of E5M2's smallest step.
__device__ __forceinline__ void e5m2_terms4(float a, float b, float c, float d, uint32_t (&t)[3]) {
  asm("{\n\t.reg .b32 x, y, p, q, r, s;\n\t.reg .b16 u, v;\n\t"
      "cvt.rn.f16x2.f32 x, %4, %3;\n\tcvt.rn.f16x2.f32 y, %6, %5;\n\t"
      "prmt.b32 %0, x, y, 0x7531;\n\t"
      "and.b32 p, x, 0xff00ff00;\n\tand.b32 q, y, 0xff00ff00;\n\t"
      "sub.rn.f16x2 x, x, p;\n\tsub.rn.f16x2 y, y, q;\n\t"
      "prmt.b32 %1, x, y, 0x7531;\n\t"
      "and.b32 r, x, 0xff00ff00;\n\tand.b32 s, y, 0xff00ff00;\n\t"
      "sub.rn.f16x2 x, x, r;\n\tsub.rn.f16x2 y, y, s;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 u, x;\n\tcvt.rn.satfinite.e5m2x2.f16x2 v, y;\n\t"
      "mov.b32 %2, {u, v};\n\t}"
      : "=r"(t[0]), "=r"(t[1]), "=r"(t[2]) : "f"(a), "f"(b), "f"(c), "f"(d));
}

// ---- issue and loads of the kernels on tcgen05 ----

// Whether the phase with this parity has completed.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}

// One lane of a converged warp.  The branch on it tells the compiler that one thread issues: 16 MMAs in
// a branch on lane == 0 take 738 cycles to issue, in a branch on this 424.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// D (+)= A B with shared-memory descriptors whose upper halves are constants of the kernel.
template <bool FP8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (FP8)
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                 "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n\t}\n"
                 ::"r"(d), "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate) : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                 "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}\n"
                 ::"r"(d), "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate) : "memory");
}

// Shared memory and barriers of the rings of K tiles, V tiles and (E4M3) 128 key and 128 value scales.
struct TileRings {
  uint32_t k, v, sc;
  uint32_t full_k, empty_k, full_v, empty_v, full_s, empty_s;
};

// One warp loads the K tiles (what = 0), the V tiles (1) or the scales (2) of list entries [x0, x1).  C: the
// kernel's configuration.  Box i of a segment's list of boxes is br rows of one page; lane i % 32 looks its page
// up, one batch of 32 boxes ahead, and issues its copies.
template <class C>
__device__ __forceinline__ void load_tiles(const PagedParams& p, const int* pre, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                           const TileRings& g, int what, int rt0, long long x0, long long x1,
                                           const WaitCtl& ctl) {
  const int lane = static_cast<int>(lane_id());
  const bool is_k = what == 0, is_s = what == 2;
  const CUtensorMap* tm = is_k ? &tmK : &tmV;
  const uint32_t data = is_k ? g.k : g.v;
  const uint32_t fulls = is_s ? g.full_s : (is_k ? g.full_k : g.full_v), empties = is_s ? g.empty_s : (is_k ? g.empty_k : g.empty_v);
  const int ps_log = 31 - __clz(p.page_size), br_log = ps_log < 7 ? ps_log : 7;
  const int pt_log = 7 - br_log, per_tile = 1 << pt_log, batch = 32 >> pt_log;
  const int stages = is_s ? C::NSC : (is_k ? C::NK : C::NV);
  const uint64_t pol = p.row_tiles > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
  int it = 0, slot = 0;
  uint32_t par = 1;
  bool dead = false;                           // a wait gave up (the same in every lane)
  Segment s;
  for (int rt = rt0; rt < p.row_tiles && !dead; rt += p.group_ctas)
    for (long long x = x0; !dead && next_segment(p, pre, x, x1, s);) {
      const int L = *(p.ctx_lens + s.b) + (p.q_lens != nullptr ? *(p.q_lens + s.b) : p.T);
      const int* table = p.page_table + static_cast<long long>(s.b) * p.max_pages;
      auto look_up = [&](int j) {
        const int at = (128 * j + (lane << br_log)) >> ps_log;
        return j < s.t1 && at < p.max_pages ? *(table + at) : -1;
      };
      int next = look_up(s.t0);
      for (int j0 = s.t0; j0 < s.t1 && !dead; j0 += batch) {
        const int page = next;
        next = look_up(j0 + batch);
        const int key = 128 * j0 + (lane << br_log);
        const bool wanted = key < L && j0 + (lane >> pt_log) < s.t1;
        const bool good = wanted && page >= 0 && page < p.n_pages;
        if (is_k && wanted && !good && atomicCAS(p.err_word, 0, 1) == 0) atomicExch(p.err_info, WHERE_PAGED_PAGE);
        const unsigned boxes = __ballot_sync(0xffffffffu, good);
        const int row = key & (p.page_size - 1);
        for (int i = 0; i < batch && j0 + i < s.t1; ++i, ++it) {
          dead = !warp_wait(empties + 8u * slot, par, ctl, WHERE_PAGED_LOAD);
          if (dead) break;
          const uint32_t full = fulls + 8u * slot;
          if (!is_s) {
            const uint32_t dst = data + slot * C::TILE_BYTES;
            const unsigned mine = (boxes >> (i << pt_log)) & ((1u << per_tile) - 1);
            if (lane == 0) mbar_arrive_expect_tx(full, (__popc(mine) << br_log) * C::ROW_BYTES);
            __syncwarp();
            const int box = lane & (per_tile - 1);
            if ((lane >> pt_log) == i && ((mine >> box) & 1)) {
#pragma unroll
              for (int pn = 0; pn < C::NPANEL; ++pn)
                tma_load_4d(dst + pn * C::PANEL_BYTES + (box << br_log) * C::PANEL_ROW, tm, full,
                            pn * (C::PANEL_ROW / C::ESZ), row, s.hkv, page, pol);
            }
          } else {
            // lane: the scales of four keys of the tile
            const uint32_t dst = g.sc + 1024 * slot + 16 * lane;
            const int src = (i << pt_log) + (lane >> (br_log - 2));
            const int pg = __shfl_sync(0xffffffffu, page, src);
            const int r0 = __shfl_sync(0xffffffffu, row, src) + ((4 * lane) & ((1 << br_log) - 1));
            if ((boxes >> src) & 1) {
              const long long e = (static_cast<long long>(pg) * p.Hkv + s.hkv) * p.page_size + r0;
              cp_async16(dst, p.k_scale + e);
              cp_async16(dst + 512, p.v_scale + e);
            }
            cp_async_arrive(full);
          }
          if (++slot == stages) {
            slot = 0;
            par ^= 1;
          }
        }
      }
    }
  if (dead) {
    cp_async_wait_all();
    if (lane == 0 && !is_s) {
      // this warp's copies in flight: the slots issued last
      const int n = it < stages ? it : stages;
      for (int i = 0; i < n; ++i)
        wait_drain_paged(fulls + 8u * ((it - 1 - i) % stages), ((it - 1 - i) / stages) & 1, p.spin_limit);
    }
  }
}

}  // namespace ea46
