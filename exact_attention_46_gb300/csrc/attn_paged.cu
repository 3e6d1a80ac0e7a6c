// attn_paged.cu -- attention of one or a few (drafted) query tokens per sequence over a paged
// key/value cache, for sm_103a.  The hada.io FA3 summary ("Weitere Optimierungen und künftige
// Integration") names LLM inference as future work and defines nothing; the readings are below.
//
// Sequence b has ctx_lens[b] cached keys and after them the q_lens[b] drafted tokens' own keys,
// L = ctx + q_len in all; key j lies in page page_table[b, j / page_size].  Drafted token t sees
// the keys j < ctx and, of the drafted keys, i = j - ctx where bit i of tree_mask[b, t] is set
// (no mask: i <= t).  Per query row (t, query head) of key/value head h / G:
//     x_j = scale q . k_j,  lse = log sum_j exp x_j,  o = sum_j exp(x_j - lse) v_j,
// rows that see no key: o = 0, lse = -inf; rows t >= q_len are not written.
//
// The work is one pass over K and V: 2 L D bytes (E4M3) or 4 L D (bf16) per key/value head, for
// G * T <= 32 query rows far below the tensor pipe's rate, so HBM bounds it and the kernel is built
// to keep loads in flight whatever the lengths are:
//   * the unit is (sequence, key/value head, tile of RB packed rows r = t * G + g); its keys are cut
//     into 128-key tiles and the tiles of all units form one list.  CTA i of N (one per SM) takes
//     tiles [i W / N, (i + 1) W / N) of the W, so every SM streams the same number of bytes for
//     any mix of lengths, and the lengths stay on the device.  A unit that several CTAs share
//     leaves one partial (o, lse) per CTA in the workspace; a second, dependent kernel merges them
//     in a fixed order;
//   * a producer warp looks the pages up and fills a ring of (K tile, V tile) stages by TMA, one
//     box per page and swizzle panel; a page number outside the cache is not loaded and reported;
//   * a consumer warp takes 32 keys of a tile, from S = Q K^T to its own running (max, sum, O): no
//     barrier between warps inside a unit.  With at most 32 rows an MMA tile of 128 rows would
//     stand mostly empty and its hand-offs (S, P, O through Tensor Memory) would set the pace, so
//     the products run on mma.sync m16n8k16 from registers.  Two groups of four warps: with up to
//     16 rows they take every other tile, with up to 32 each takes 16 of the rows;
//   * E4M3 rows become fp16 in registers (exact), with queries in fp16 after an exact
//     power-of-two scaling of each row; the key's scale multiplies its logit, the value's scale
//     its numerator, over a power-of-two reference that keeps fp16 in range.  Numerators are rounded to bf16 (fp16 with E4M3)
//     because the tensor core takes no wider operand; sums and statistics are fp32.
// Hidden keys never reach a sum: their logit is replaced by -inf, their numerator by 0, and in tiles
// that hold drafted keys or the end of the sequence a value row that is past the end or not finite
// is masked out of the product and, where it is seen, enters by itself (bf16: element by element;
// E4M3: by its scale, which is not finite where a code is NaN).
// Every mbarrier wait is bounded.
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "cache.h"
#include "ptx.cuh"

namespace ea46 {

namespace {

constexpr float LN2_P = 0.69314718055994530942f;
constexpr int NWARP = 8;                        // consumer warps
constexpr int NTHREADS = 32 * (NWARP + 1);
enum : int { WHERE_PAGED_LOAD = 51, WHERE_PAGED_USE = 52, WHERE_PAGED_LENS = 53, WHERE_PAGED_PAGE = 54 };

// WIDE: 32 rows per unit, one warp group per 16; otherwise 16 rows, the groups take turns by tile.
template <int D, bool FP8, bool WIDE>
struct PagedCfg {
  static constexpr int RB = WIDE ? 32 : 16;
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int ROW_BYTES = D * ESZ;
  static constexpr int PANEL_ROW = ROW_BYTES >= 128 ? 128 : ROW_BYTES;
  static constexpr int NPANEL = ROW_BYTES / PANEL_ROW;
  static constexpr int PANEL_BYTES = 128 * PANEL_ROW;
  static constexpr int TILE_BYTES = 128 * ROW_BYTES;
  static constexpr int SCALE_BYTES = FP8 ? 2 * 128 * 4 : 0;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES + SCALE_BYTES;
  static constexpr int KS = D / 16;                          // k-steps of Q K^T
  static constexpr int NB = D / 8;                           // n-blocks of O
  static constexpr int PARTS = WIDE ? 4 : 8;                 // warps that hold a part of a row
  static constexpr int MCOLS = 32;                           // columns merged at a time
  static constexpr int MSTRIDE = MCOLS + 8;
  static constexpr int Q_BYTES = RB / 16 * KS * 32 * 16;
  static constexpr int REST = 1024 + Q_BYTES + NWARP * 16 * MSTRIDE * 4 + NWARP * 16 * 8 + RB * 12 +
                              (PAGED_MAX_BATCH + 2) * 4 + 16 * 16 + 64;
  static constexpr int FIT = (227 * 1024 - REST) / STAGE_BYTES, WANT = 196608 / (2 * TILE_BYTES);
  static constexpr int NSTAGE = FIT < WANT ? FIT : WANT;     // up to 192 KB of K/V in flight
  static constexpr int Q_OFF = NSTAGE * STAGE_BYTES;
  static constexpr int M_OFF = Q_OFF + Q_BYTES;              // merge buffer [NWARP][16][MSTRIDE]
  static constexpr int M_BYTES = NWARP * 16 * MSTRIDE * 4;
  static constexpr int ML_OFF = M_OFF + M_BYTES;             // [NWARP][16] (max, sum)
  static constexpr int BITS_OFF = ML_OFF + NWARP * 16 * 8;   // [RB] visible drafts
  static constexpr int RQ_OFF = BITS_OFF + RB * 8;           // [RB] power of two of a query row
  static constexpr int PRE_OFF = RQ_OFF + RB * 4;            // [PAGED_MAX_BATCH + 1] tile prefix
  static constexpr int BAR_OFF = PRE_OFF + (PAGED_MAX_BATCH + 2) * 4;
  static constexpr int SMEM_BYTES = 1024 + BAR_OFF + 2 * NSTAGE * 8 + 64;
  static_assert(BAR_OFF % 8 == 0, "barrier alignment");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four E4M3 bytes -> fp16 pairs (bytes 0, 1) and (bytes 2, 3); exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ void wait_drain_paged(uint32_t bar, uint32_t parity, long long limit) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit) return;
}

// Prefix sums of the sequences' key tiles into pre[0 .. B]; returns 0 if any length is out of
// range.  Called by all `n` threads (n >= 32 a multiple of 32, n <= 1024).
__device__ __forceinline__ bool tile_prefix(const PagedParams& p, int* pre, int* scratch, int n) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + n - 1) / n, b0 = tid * per, b1 = min(p.B, b0 + per);
  bool ok = true;
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int ctx = __ldg(p.ctx_lens + b), ql = p.q_lens != nullptr ? __ldg(p.q_lens + b) : p.T;
    const bool fine = ctx >= 0 && ql >= 0 && ql <= p.T &&
                      static_cast<long long>(ctx) + ql <= static_cast<long long>(p.max_pages) * p.page_size;
    ok = ok && fine;
    const int tiles = fine && ql > 0 ? (ctx + ql + 127) >> 7 : 0;
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

// The piece of the tile list that starts at x and ends at x1 or with its unit.
struct Segment {
  int b, hkv, rt;       // sequence, key/value head, row tile
  int t0, t1, n;        // tiles [t0, t1) of the unit's n
};

__device__ __forceinline__ Segment find_segment(const PagedParams& p, const int* pre, long long x, long long x1) {
  const long long hr = static_cast<long long>(p.Hkv) * p.row_tiles;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * hr <= x) lo = mid; else hi = mid;
  }
  // x lies in sequence lo: empty ones before it have pre[lo + 1] == pre[lo]
  Segment s;
  s.b = lo;
  s.n = pre[lo + 1] - pre[lo];
  const long long y = x - pre[lo] * hr;
  const int u = static_cast<int>(y / s.n);
  s.hkv = u / p.row_tiles;
  s.rt = u % p.row_tiles;
  s.t0 = static_cast<int>(y - static_cast<long long>(u) * s.n);
  const long long left = x1 - x;
  s.t1 = left < s.n - s.t0 ? s.t0 + static_cast<int>(left) : s.n;
  return s;
}

__device__ __forceinline__ long long cta_start(long long i, long long W, long long N) { return i * W / N; }

template <int D, bool FP8, bool WIDE>
__global__ void __launch_bounds__(NTHREADS, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedParams p) {
  using C = PagedCfg<D, FP8, WIDE>;
  constexpr int RB = C::RB, NSTAGE = C::NSTAGE;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  int* pre = reinterpret_cast<int*>(base + C::PRE_OFF);
  const uint32_t bar0 = base_u32 + C::BAR_OFF;
  auto BAR_FULL = [&](int s) { return bar0 + 8u * s; };
  auto BAR_EMPTY = [&](int s) { return bar0 + 8u * (NSTAGE + s); };
  int* flags = reinterpret_cast<int*>(base + C::BAR_OFF + 2 * NSTAGE * 8);
  volatile int* abort_flag = flags;
  int* scratch = flags + 1;                      // [NWARP + 1]

  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  if (threadIdx.x == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(BAR_FULL(s), 1);
      mbar_init(BAR_EMPTY(s), NWARP);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  grid_launch_dependents();
  if (!tile_prefix(p, pre, scratch, NTHREADS)) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && atomicCAS(p.err_word, 0, 1) == 0) atomicExch(p.err_info, WHERE_PAGED_LENS);
    return;
  }
  const long long W = static_cast<long long>(pre[p.B]) * p.Hkv * p.row_tiles;
  const long long N = W < p.n_cta ? W : p.n_cta;
  if (static_cast<long long>(blockIdx.x) >= N) return;
  const long long x0 = cta_start(blockIdx.x, W, N), x1 = cta_start(blockIdx.x + 1ll, W, N);
  const WaitCtl ctl{p.spin_limit, abort_flag, p.err_word, p.err_info};

  if (warp == NWARP) {
    // ---- producer: page look-up and TMA ----
    // Box i of the list of boxes of a segment is br rows of one page; lane i % 32 looks its page up,
    // one batch of 32 boxes ahead of their use, and issues its copies.
    const int ps_log = 31 - __clz(p.page_size);
    const int br_log = ps_log < 7 ? ps_log : 7, br = 1 << br_log;
    const int pt_log = 7 - br_log, per_tile = 1 << pt_log;       // boxes of a tile (1 .. 8)
    const uint64_t pol = l2_policy_evict_first();
    int it = 0;
    for (long long x = x0; x < x1;) {
      const Segment s = find_segment(p, pre, x, x1);
      const int L = __ldg(p.ctx_lens + s.b) + (p.q_lens != nullptr ? __ldg(p.q_lens + s.b) : p.T);
      const int* table = p.page_table + static_cast<long long>(s.b) * p.max_pages;
      // first key of this lane's box in the batch that starts at tile j, and its page (-1: past the end)
      auto look_up = [&](int j) {
        const int key = 128 * j + (lane << br_log);
        return j < s.t1 && key < L ? __ldg(table + (key >> ps_log)) : -1;
      };
      const int batch = 32 >> pt_log;              // tiles of a batch
      int next = look_up(s.t0);
      for (int j0 = s.t0; j0 < s.t1; j0 += batch) {
        const int page = next;
        next = look_up(j0 + batch);
        const int key = 128 * j0 + (lane << br_log);
        const bool wanted = key < L && j0 + (lane >> pt_log) < s.t1;
        const bool good = wanted && page >= 0 && page < p.n_pages;
        if (wanted && !good && atomicCAS(p.err_word, 0, 1) == 0) atomicExch(p.err_info, WHERE_PAGED_PAGE);
        const unsigned boxes = __ballot_sync(0xffffffffu, good);
        const int row = key & (p.page_size - 1);
        const long long e = (static_cast<long long>(page) * p.Hkv + s.hkv) * p.page_size + row;
        for (int i = 0; i < batch && j0 + i < s.t1; ++i, ++it) {
          const int slot = it % NSTAGE;
          if (!warp_wait(BAR_EMPTY(slot), ((it / NSTAGE) & 1) ^ 1u, ctl, WHERE_PAGED_LOAD)) break;
          const unsigned mine = (boxes >> (i << pt_log)) & ((1u << per_tile) - 1);
          if (lane == 0)
            mbar_arrive_expect_tx(BAR_FULL(slot), (__popc(mine) << br_log) * (2u * C::ROW_BYTES + (FP8 ? 8u : 0u)));
          __syncwarp();
          if (good && (lane >> pt_log) == i) {
            const int box = lane & (per_tile - 1);
            const uint32_t sK = base_u32 + slot * C::STAGE_BYTES + (box << br_log) * C::PANEL_ROW;
#pragma unroll
            for (int pn = 0; pn < C::NPANEL; ++pn) {
              tma_load_4d(sK + pn * C::PANEL_BYTES, &tmK, BAR_FULL(slot), pn * (C::PANEL_ROW / C::ESZ), row, s.hkv, page, pol);
              tma_load_4d(sK + C::TILE_BYTES + pn * C::PANEL_BYTES, &tmV, BAR_FULL(slot), pn * (C::PANEL_ROW / C::ESZ),
                          row, s.hkv, page, pol);
            }
            if (FP8) {
              const uint32_t sS = base_u32 + slot * C::STAGE_BYTES + 2 * C::TILE_BYTES + (4 * box << br_log);
              bulk_load(sS, p.k_scale + e, 4 * br, BAR_FULL(slot), pol);
              bulk_load(sS + 512, p.v_scale + e, 4 * br, BAR_FULL(slot), pol);
            }
          }
        }
        if (*abort_flag) break;
      }
      if (*abort_flag) break;
      x += s.t1 - s.t0;
    }
    if (*abort_flag && lane == 0)
      for (int i = it > NSTAGE ? it - NSTAGE : 0; i < it; ++i)
        wait_drain_paged(BAR_FULL(i % NSTAGE), (i / NSTAGE) & 1, p.spin_limit);
    return;
  }

  // ---- consumers: warp w takes keys 32 (w & 3) .. of a tile; the two groups of four warps take
  // the unit's row halves (WIDE) or every other tile ----
  const int g = lane >> 2, t4 = lane & 3;
  const int kw = 32 * (warp & 3), group = warp >> 2;
  const int rlo = WIDE ? 16 * group : 0;         // first row of this warp
  uint4* qfrag = reinterpret_cast<uint4*>(base + C::Q_OFF);
  float* mbuf = reinterpret_cast<float*>(base + C::M_OFF);
  float2* ml = reinterpret_cast<float2*>(base + C::ML_OFF);
  unsigned long long* bits = reinterpret_cast<unsigned long long*>(base + C::BITS_OFF);
  float* rq = reinterpret_cast<float*>(base + C::RQ_OFF);
  // key (within the warp's 32) of column e of n-block nb of this thread's S
  auto key_of = [&](int nb, int e) { return FP8 ? 8 * nb + t4 + 4 * e : 8 * nb + 2 * t4 + e; };
  int it = 0;
  for (long long x = x0; x < x1;) {
    const Segment sg = find_segment(p, pre, x, x1);
    const int ctx = __ldg(p.ctx_lens + sg.b), ql = p.q_lens != nullptr ? __ldg(p.q_lens + sg.b) : p.T;
    const int L = ctx + ql;
    const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(p.q) +
                              (static_cast<long long>(sg.b) * p.T * p.Hq + static_cast<long long>(sg.hkv) * p.G) * D;
    auto row_ptr = [&](int r) -> const __nv_bfloat16* {          // packed row of the tile, or null
      const int pr = sg.rt * RB + r, t = pr / p.G;
      return t < ql ? qb + (static_cast<long long>(t) * p.Hq + pr % p.G) * D : nullptr;
    };
    // the last segment's readers of the shared arrays below are past them (barrier at its end).
    // Query fragments: entry (16-row block, k-step, lane) holds the A registers of that lane
    if (FP8) {
      // per-row power of two that brings the largest element into [1, 2): exact, and the logit
      // multiplier takes it back
      for (int r = warp; r < RB; r += NWARP) {
        const __nv_bfloat16* src = row_ptr(r);
        float m = 0.f;
        if (src != nullptr)
          for (int d = 2 * lane; d < D; d += 64) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(src + d));
            m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        int ex = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        ex = ex < -110 ? -110 : (ex > 110 ? 110 : ex);
        if (lane == 0) rq[r] = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
      }
      named_bar_sync(1, 32 * NWARP);
    }
    for (int i = threadIdx.x; i < RB / 16 * C::KS * 32; i += 32 * NWARP) {
      const int l = i & 31, ks = (i >> 5) % C::KS, mt = (i >> 5) / C::KS;
      const int lg = l >> 2, lt = l & 3;
      uint32_t a[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * mt + lg + 8 * h;
        const __nv_bfloat16* src = row_ptr(r);
        uint32_t lo = 0, hi = 0;
        if (src != nullptr) {
          // bf16: k = 2t, 2t + 1 and 2t + 8, 2t + 9 of the step; E4M3: four elements in a row, the
          // order in which a thread reads the key's bytes
          const int d = FP8 ? 16 * (lt + 4 * (ks >> 2)) + 4 * (ks & 3) : 16 * ks + 2 * lt;
          lo = *reinterpret_cast<const uint32_t*>(src + d);
          hi = *reinterpret_cast<const uint32_t*>(src + d + (FP8 ? 2 : 8));
          if (FP8) {
            const float inv = 1.f / rq[r];
            lo = pack_f16x2(__uint_as_float(lo << 16) * inv, __uint_as_float(lo & 0xffff0000u) * inv);
            hi = pack_f16x2(__uint_as_float(hi << 16) * inv, __uint_as_float(hi & 0xffff0000u) * inv);
          }
        }
        a[h] = lo;
        a[2 + h] = hi;
      }
      qfrag[i] = make_uint4(a[0], a[1], a[2], a[3]);
    }
    if (threadIdx.x < RB) {
      const int t = (sg.rt * RB + static_cast<int>(threadIdx.x)) / p.G;
      unsigned long long m = 0;
      if (t < ql)
        m = p.tree_mask != nullptr ? __ldg(p.tree_mask + static_cast<long long>(sg.b) * p.T + t)
                                   : (t >= 63 ? ~0ull : (2ull << t) - 1);
      bits[threadIdx.x] = m;
    }
    named_bar_sync(1, 32 * NWARP);
    float cr[2];                                   // logit multiplier of rows g, g + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) cr[h] = FP8 ? p.c_log2 * rq[rlo + g + 8 * h] : p.c_log2;
    const uint4* qf = qfrag + (WIDE ? group : 0) * C::KS * 32 + lane;

    float o[C::NB][4];
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float vref = 0.f, vup = 0.f;                   // E4M3: power of two above the value scales seen, 2^10 / vref
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[nb][i] = 0.f;

    for (int j = sg.t0; j < sg.t1; ++j, ++it) {
      const int slot = it % NSTAGE;
      // every warp waits for and frees every tile, its own or not: a parity wait can only follow a
      // barrier whose phases it sees one by one
      const bool ok = warp_wait(BAR_FULL(slot), (it / NSTAGE) & 1, ctl, WHERE_PAGED_USE);
      const int k0 = 128 * j + kw;                 // first key of this warp
      // TAIL: the warp's keys hold drafted ones, or the end of the sequence
      auto visit = [&](auto tail_c) {
        constexpr bool TAIL = decltype(tail_c)::value;
        const uint32_t sK = base_u32 + slot * C::STAGE_BYTES, sV = sK + C::TILE_BYTES;
        float s[4][4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nb][i] = 0.f;
        // ---- S = Q K^T ----
        if constexpr (!FP8) {
          const int r = kw + (lane & 7) + 8 * (lane >> 4), half = (lane >> 3) & 1;
#pragma unroll
          for (int ks = 0; ks < C::KS; ++ks) {
            uint32_t kf[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y)
              ldsm4(sK + (ks >> 2) * C::PANEL_BYTES + (r + 16 * y) * 128 + (((2 * (ks & 3) + half) ^ (r & 7)) << 4), kf[y]);
            const uint4 a = qf[ks * 32];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              mma16816<false>(s[2 * y], a, kf[y][0], kf[y][1]);
              mma16816<false>(s[2 * y + 1], a, kf[y][2], kf[y][3]);
            }
          }
        } else {
          // S's column n of an n-block is key (n >> 1) + 4 (n & 1): with the swizzle, the two rows
          // that eight lanes read at once then lie in different banks
          const int rg = (g >> 1) + 4 * (g & 1);
#pragma unroll
          for (int i = 0; i < C::KS / 4; ++i) {
            uint4 w[4];
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
              const int r = kw + 8 * nb + rg;
              const int ch = C::PANEL_ROW == 128 ? ((t4 + 4 * i) ^ rg) : (t4 ^ ((r >> 1) & 3));
              w[nb] = lds128(sK + r * C::PANEL_ROW + 16 * ch);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 a = qf[(4 * i + c) * 32];
#pragma unroll
              for (int nb = 0; nb < 4; ++nb) {
                uint32_t b0, b1;
                e4m3x4_to_f16(c == 0 ? w[nb].x : (c == 1 ? w[nb].y : (c == 2 ? w[nb].z : w[nb].w)), b0, b1);
                mma16816<true>(s[nb], a, b0, b1);
              }
            }
          }
        }
        // ---- scales of this thread's eight keys (pairs: columns 0, 1 of an n-block) ----
        uint64_t ksc[4], vsc[4];
        uint32_t vbad = 0;                         // E4M3, tail: value rows past the end or without a finite scale
        if constexpr (FP8) {
          const float* sc = reinterpret_cast<const float*>(base + slot * C::STAGE_BYTES + 2 * C::TILE_BYTES) + kw;
          float top = 0.f, vs[4][2];
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            ksc[nb] = f2_pack(sc[key_of(nb, 0)], sc[key_of(nb, 1)]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              vs[nb][e] = sc[128 + key_of(nb, e)];
              if (TAIL) {
                if (k0 + key_of(nb, e) >= L) vs[nb][e] = 0.f;
                if (!(vs[nb][e] < INFINITY) || k0 + key_of(nb, e) >= L) vbad |= 1u << (2 * nb + e);
                top = fmaxf(top, vs[nb][e] < INFINITY ? vs[nb][e] : 0.f);
              }
            }
            if (!TAIL) top = max3(top, vs[nb][0], vs[nb][1]);
          }
          if (__any_sync(0xffffffffu, top > vref)) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // next power of two above
            const float nref = __uint_as_float((__float_as_uint(top) & 0x7f800000u) + (top < 0x1p126f ? 0x00800000u : 0u));
            const float f = vref / nref;
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[nb][i] *= f;
            vref = nref;
            vup = 1024.f / nref;
          }
          const uint64_t up = f2_pack(vup, vup);
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) vsc[nb] = f2_mul(f2_pack(vs[nb][0], vs[nb][1]), up);
        }
        // ---- logits (before the row's multiplier cr, which is positive), mask, running maximum ----
        uint64_t xs[2][4];
        float mt_max[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            xs[h][nb] = f2_pack(s[nb][2 * h], s[nb][2 * h + 1]);
            if (FP8) xs[h][nb] = f2_mul(xs[h][nb], ksc[nb]);
            if (TAIL) {
              float v[2];
              f2_unpack(xs[h][nb], v[0], v[1]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = k0 + key_of(nb, e);
                const bool sees = key < ctx || (key < L && ((bits[rlo + g + 8 * h] >> (key - ctx)) & 1));
                v[e] = sees ? v[e] : -INFINITY;
              }
              xs[h][nb] = f2_pack(v[0], v[1]);
            }
          }
          float mx = -INFINITY;
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            float v0, v1;
            f2_unpack(xs[h][nb], v0, v1);
            mx = max3(mx, v0, v1);
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mt_max[h] = mx * cr[h];
        }
        if (__any_sync(0xffffffffu, mt_max[0] > m_run[0] + 4.f || mt_max[1] > m_run[1] + 4.f)) {
          // lazily: O and the sum are only rescaled when some maximum moved by a factor of 2^4
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m_run[h], mt_max[h]);
            const float f = m_run[h] == -INFINITY ? 0.f : ex2(m_run[h] - mn);
            m_run[h] = mn;
            l_run[h] *= f;
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) {
              o[nb][2 * h] *= f;
              o[nb][2 * h + 1] *= f;
            }
          }
        }
        // ---- numerators ----
        uint4 pa[2];
        {
          uint32_t w[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float off = m_run[h] == -INFINITY ? 0.f : -m_run[h];
            const uint64_t off2 = f2_pack(off, off), cr2 = f2_pack(cr[h], cr[h]);
            uint64_t sum = f2_pack(l_run[h], 0.f);
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
              float q0, q1;
              f2_unpack(f2_fma(xs[h][nb], cr2, off2), q0, q1);
              q0 = ex2(q0);
              q1 = ex2(q1);
              const uint64_t q = f2_pack(q0, q1);
              sum = f2_add(sum, q);
              if constexpr (FP8) {
                float y0, y1;
                f2_unpack(f2_mul(q, vsc[nb]), y0, y1);
                if (TAIL) {                        // a hidden key's scale may be anything: its numerator is 0
                  y0 = q0 == 0.f ? 0.f : y0;
                  y1 = q1 == 0.f ? 0.f : y1;
                }
                w[h][nb] = pack_f16x2(y0, y1);
              } else {
                s[nb][2 * h] = q0;
                s[nb][2 * h + 1] = q1;
                w[h][nb] = pack_bf16x2(q0, q1);
              }
            }
            float l0, l1;
            f2_unpack(sum, l0, l1);
            l_run[h] = l0 + l1;
          }
          pa[0] = make_uint4(w[0][0], w[1][0], w[0][1], w[1][1]);
          pa[1] = make_uint4(w[0][2], w[1][2], w[0][3], w[1][3]);
        }
        // ---- O += P V ----
        if constexpr (!FP8) {
          uint32_t odd = 0;                        // value rows past the end, or not finite: out of the product
          if (TAIL) {
            for (int r = 0; r < 32; ++r) {
              bool strange = k0 + r >= L;
              if (!strange && k0 + r >= ctx) {
                bool inf = false;
                for (int c = lane; c < D / 2; c += 32) {
                  const uint32_t w = *reinterpret_cast<const uint32_t*>(base + (sV - base_u32) + (c >> 5) * C::PANEL_BYTES +
                                                                        (kw + r) * 128 + (c & 31) * 4);
                  inf = inf || (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
                }
                strange = __any_sync(0xffffffffu, inf);
              }
              if (strange) odd |= 1u << r;
            }
            // those that some row may see are added element by element
            const uint32_t seen = k0 + 32 <= L ? odd : odd & ((1u << (L - k0)) - 1);
            if (seen != 0) {
#pragma unroll
              for (int rb = 0; rb < 4; ++rb)
                for (int r8 = 0; r8 < 8; ++r8) {
                  const int r = 8 * rb + r8;
                  if (!((seen >> r) & 1)) continue;
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    // the lane of each quad that holds key r's numerators
                    float pv = (r8 & 1) ? s[rb][2 * h + 1] : s[rb][2 * h];
                    pv = __shfl_sync(0xffffffffu, pv, (lane & ~3) | (r8 >> 1));
                    if (pv != 0.f) {
#pragma unroll
                      for (int nb = 0; nb < C::NB; ++nb) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(
                            base + (sV - base_u32) + (nb >> 3) * C::PANEL_BYTES + (kw + r) * 128 +
                            (((nb & 7) ^ ((kw + r) & 7)) << 4) + 4 * t4);
                        o[nb][2 * h] += pv * __uint_as_float(w << 16);
                        o[nb][2 * h + 1] += pv * __uint_as_float(w & 0xffff0000u);
                      }
                    }
                  }
                }
            }
          }
          // value fragment register b of 16 keys: keys 2 t + 8 b and the next
          uint32_t keep[2][2];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t two = odd >> (16 * kk + 8 * y + 2 * t4);
              keep[kk][y] = ((two & 1u) ? 0u : 0xffffu) | ((two & 2u) ? 0u : 0xffff0000u);
            }
          const int r = kw + (lane & 15), hi = lane >> 4;
          auto add = [&](bool masked) {
#pragma unroll
            for (int nb = 0; nb < C::NB; nb += 2)
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                uint32_t vf[4];
                ldsm4t(sV + (nb >> 3) * C::PANEL_BYTES + (r + 16 * kk) * 128 + ((((nb & 7) + hi) ^ (r & 7)) << 4), vf);
                if (masked) {
#pragma unroll
                  for (int y = 0; y < 4; ++y) vf[y] &= keep[kk][y & 1];
                }
                mma16816<false>(o[nb], pa[kk], vf[0], vf[1]);
                mma16816<false>(o[nb + 1], pa[kk], vf[2], vf[3]);
              }
          };
          if (TAIL && odd != 0) add(true);
          else add(false);
        } else {
          // lane g reads D / 8 bytes of rows t, t + 4, t + 8, t + 12 of each 16 -- the keys of S's
          // columns; a row that must not show is read as zeros (its codes may be NaN), and shows in
          // the rows that see it through its scale
          constexpr int NW = D / 32;
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            uint32_t w[4][NW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = kw + 16 * kk + t4 + 4 * i;
              if constexpr (D == 128) {
                const uint4 u = lds128(sV + r * 128 + ((((g >> 1) | ((g & 1) << 2)) ^ (r & 7)) << 4));
                w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
              } else {
                const int ch = ((g >> 2) & 1) | (((g >> 1) & 1) << 1);
                const uint2 u = lds64(sV + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4) + 8 * (g & 1));
                w[i][0] = u.x; w[i][1] = u.y;
              }
              if (TAIL && ((vbad >> (4 * kk + i)) & 1)) {
#pragma unroll
                for (int c = 0; c < NW; ++c) w[i][c] = 0u;
              }
            }
#pragma unroll
            for (int c = 0; c < NW; ++c)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                // bytes e, e + 1 of two rows: (row, row + 4) of element e, then of e + 1
                const uint32_t sel = e == 0 ? 0x5140u : 0x7362u;
                uint32_t b0, b1, d0, d1;
                e4m3x4_to_f16(__byte_perm(w[0][c], w[1][c], sel), b0, d0);
                e4m3x4_to_f16(__byte_perm(w[2][c], w[3][c], sel), b1, d1);
                mma16816<true>(o[4 * c + e], pa[kk], b0, b1);
                mma16816<true>(o[4 * c + e + 1], pa[kk], d0, d1);
              }
          }
        }
      };
      if (ok && k0 < L && (WIDE || (it & 1) == group)) {
        if (k0 + 32 > ctx) visit(std::true_type{});
        else visit(std::false_type{});
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR_EMPTY(slot));
    }

    // ---- the warps' partial results meet ----
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_run[h];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (t4 == 0) ml[warp * 16 + g + 8 * h] = make_float2(m_run[h], l);
    }
    named_bar_sync(1, 32 * NWARP);
    // (max, sum) over the warps that hold a part of row r of the unit
    auto whole_row = [&](int r, float& M, float& l) {
      const float2* e = ml + (WIDE ? (r >> 4) * 4 * 16 : 0) + (r & 15);
      M = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int w = 0; w < C::PARTS; ++w) M = fmaxf(M, e[16 * w].x);
#pragma unroll
      for (int w = 0; w < C::PARTS; ++w) l += e[16 * w].x == -INFINITY ? e[16 * w].y : e[16 * w].y * ex2(e[16 * w].x - M);
    };
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float M, l;
      whole_row(rlo + g + 8 * h, M, l);
      f[h] = m_run[h] == -INFINITY ? 0.f : ex2(m_run[h] - M) / l;
      if (FP8) f[h] *= vref * 0x1p-10f;            // the 2^10 of the numerators
    }
    const bool whole = sg.t0 == 0 && sg.t1 == sg.n;
    const long long ws_slot = 2ll * blockIdx.x + (sg.t0 > 0 ? 0 : 1);
    if (threadIdx.x < RB) {
      const int r = threadIdx.x;
      float M, l;
      whole_row(r, M, l);
      const float lse2 = l == 0.f ? -INFINITY : M + __log2f(l);
      const int pr = sg.rt * RB + r, t = pr / p.G;
      if (!whole) p.ws_l[ws_slot * RB + r] = lse2;
      else if (t < ql && p.lse != nullptr)
        p.lse[(static_cast<long long>(sg.b) * p.Hq + sg.hkv * p.G + pr % p.G) * p.T + t] = lse2 * LN2_P;
    }
    constexpr int KB = C::MCOLS / 8;               // n-blocks per pass
#pragma unroll
    for (int pass = 0; pass < C::NB / KB; ++pass) {
      if (pass > 0) named_bar_sync(1, 32 * NWARP);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nb = 0; nb < KB; ++nb)
          *reinterpret_cast<float2*>(mbuf + (warp * 16 + g + 8 * h) * C::MSTRIDE + 8 * nb + 2 * t4) =
              make_float2(o[pass * KB + nb][2 * h] * f[h], o[pass * KB + nb][2 * h + 1] * f[h]);
      named_bar_sync(1, 32 * NWARP);
#pragma unroll
      for (int r0 = 0; r0 < RB; r0 += 16) {
        // thread: two output columns of one row
        const int r = r0 + static_cast<int>(threadIdx.x) / 16, c2 = threadIdx.x % 16;
        int i0, i1, d;
        if (FP8) {                                 // n-blocks 2y, 2y + 1 of column n: neighbours in d
          const int n = c2 & 7, y = c2 >> 3;
          i0 = 16 * y + n;
          i1 = i0 + 8;
          const int lt = n >> 1;
          const int first = D == 128 ? 16 * (lt + 4 * (n & 1)) : 16 * (((lt & 1) << 1) | (lt >> 1)) + 8 * (n & 1);
          d = first + pass * KB + 2 * y;
        } else {
          i0 = 2 * c2;
          i1 = i0 + 1;
          d = pass * C::MCOLS + 2 * c2;
        }
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int w = 0; w < C::PARTS; ++w) {
          const float* src = mbuf + ((WIDE ? (r0 >> 4) * 4 : 0) + w) * 16 * C::MSTRIDE + (r & 15) * C::MSTRIDE;
          a += src[i0];
          b += src[i1];
        }
        const int pr = sg.rt * RB + r, t = pr / p.G;
        if (t < ql) {
          if (whole)
            *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) +
                                         ((static_cast<long long>(sg.b) * p.T + t) * p.Hq + sg.hkv * p.G + pr % p.G) * D + d) =
                pack_bf16x2(a, b);
          else
            *reinterpret_cast<float2*>(p.ws_o + (ws_slot * RB + r) * D + d) = make_float2(a, b);
        }
      }
    }
    named_bar_sync(1, 32 * NWARP);                 // the next unit rewrites the shared arrays
    x += sg.t1 - sg.t0;
  }
}

// Merge of the units that several CTAs share: one block per unit, one warp per row.
template <int D, int RB>
__global__ void __launch_bounds__(128) paged_combine_kernel(const PagedParams p) {
  __shared__ int pre[PAGED_MAX_BATCH + 1];
  __shared__ int scratch[4];
  const bool ok = tile_prefix(p, pre, scratch, 128);
  grid_dependency_wait();       // in every block: this grid's end stands for the key kernel's too
  if (!ok) return;
  const long long hr = static_cast<long long>(p.Hkv) * p.row_tiles;
  const int b = static_cast<int>(blockIdx.x / hr), u = static_cast<int>(blockIdx.x % hr);
  const int hkv = u / p.row_tiles, rt = u % p.row_tiles;
  const int n = pre[b + 1] - pre[b];
  if (n == 0) return;
  const long long W = pre[p.B] * hr, N = W < p.n_cta ? W : p.n_cta;
  const long long a = pre[b] * hr + static_cast<long long>(u) * n;
  // the CTA that holds list position x is the last i with i W / N <= x
  const long long c0 = ((a + 1) * N - 1) / W, c1 = ((a + n) * N - 1) / W;
  if (c0 == c1) return;
  const int ql = p.q_lens != nullptr ? __ldg(p.q_lens + b) : p.T;
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < RB; r += 4) {
    const int pr = rt * RB + r, t = pr / p.G;
    if (t >= ql) break;
    float mx = -INFINITY;
    for (long long c = c0 + lane; c <= c1; c += 32) mx = fmaxf(mx, p.ws_l[(2 * c + (c == c0 ? 1 : 0)) * RB + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float acc[D / 32], sum = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
    for (long long c = c0; c <= c1; ++c) {
      const long long slot = 2 * c + (c == c0 ? 1 : 0);
      const float l = p.ws_l[slot * RB + r];
      const float w = l == -INFINITY ? 0.f : ex2(l - mx);
      sum += w;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(w, p.ws_o[(slot * RB + r) * D + lane * (D / 32) + e], acc[e]);
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const long long h = static_cast<long long>(hkv) * p.G + pr % p.G;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + ((static_cast<long long>(b) * p.T + t) * p.Hq + h) * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
      p.lse[(static_cast<long long>(b) * p.Hq + h) * p.T + t] = mx == -INFINITY ? -INFINITY : (mx + __log2f(sum)) * LN2_P;
  }
}

template <int D, bool FP8, bool WIDE>
cudaError_t launch_paged_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, bool combine, cudaStream_t st) {
  using C = PagedCfg<D, FP8, WIDE>;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((configured.load() & bit) == 0) {
    e = cudaFuncSetAttribute(attn_paged_kernel<D, FP8, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  attn_paged_kernel<D, FP8, WIDE><<<p.n_cta, NTHREADS, C::SMEM_BYTES, st>>>(tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess || !combine) return e;
  // the merge starts while the last CTAs finish and waits for them on the device
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * p.row_tiles);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D, C::RB>, p);
}

template <int D, bool FP8>
cudaError_t launch_paged_m(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, bool combine, cudaStream_t st) {
  return paged_rows(p.G * p.T) == 16 ? launch_paged_d<D, FP8, false>(tk, tv, p, combine, st)
                                     : launch_paged_d<D, FP8, true>(tk, tv, p, combine, st);
}

}  // namespace

cudaError_t launch_attn_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int D, bool fp8,
                              bool combine, cudaStream_t st) {
  if (D == 64) return fp8 ? launch_paged_m<64, true>(tk, tv, p, combine, st) : launch_paged_m<64, false>(tk, tv, p, combine, st);
  return fp8 ? launch_paged_m<128, true>(tk, tv, p, combine, st) : launch_paged_m<128, false>(tk, tv, p, combine, st);
}

}  // namespace ea46
