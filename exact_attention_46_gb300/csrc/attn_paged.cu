// attn_paged.cu -- attention of one or a few (drafted) query tokens per sequence over a paged
// key/value cache, for up to 32 query rows (heads of a group x tokens) per key/value head, 8 of E4M3,
// for sm_103a; attn_lanes.cu takes up to 64 rows and attn_tree.cu more.  The hada.io FA3 summary ("Weitere Optimierungen und künftige
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
//   * the unit is (sequence, key/value head) with its RB packed rows r = t * G + g; its keys are cut into
//     128-key tiles and the tiles of all units form one list.  CTA i of N (one per SM) takes
//     tiles [i W / N, (i + 1) W / N) of the W, so every SM streams the same number of bytes for
//     any mix of lengths, and the lengths stay on the device.  A unit that several CTAs share
//     leaves one partial (o, lse) per CTA in the workspace; a second, dependent kernel merges them
//     in a fixed order;
//   * producer warps look the pages up and fill a ring of (K tile, V tile) stages by TMA, one box per
//     page and swizzle panel; a page number outside the cache is not loaded and reported;
//   * a consumer warp takes 32 keys of a tile, from S = Q K^T to its own running (max, sum, O): no
//     barrier between warps inside a unit.  The products run on mma.sync m16n8k16 from registers, with the
//     keys as its 16 rows: with so few query rows the hand-offs of tcgen05 (S, P, O through Tensor Memory)
//     cost more than they save (figures at launch_attn_paged).  Two groups of four warps: with up to
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
//
// Measured: 16 sequences of up to 8192 keys, 32 query and 8 key/value heads, D = 128, T = 1: E4M3 42 us for
// 240 MB (5.7 TB/s; 35.4 us at the copy rate), bf16 71.4 us for 465 MB (6.5 TB/s; 68.6 us).  HBM bounds the middle;
// the first logits come 4 us after the launch may start (lengths, page numbers and the first tile are three
// dependent reads), and the merge ends 3 us after the last tile.  One sequence of 1000 keys takes 7 us, all of it such steps.
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "cache.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ea46 {

namespace {

constexpr int NWARP = 8;                        // consumer warps
constexpr int NPROD = 4;                        // producer warps: (key, value) x (even, odd copies)
constexpr int NTHREADS = 32 * (NWARP + NPROD);

// NRB: 8-row blocks of a warp (1, 2).  WIDE: a warp group per 16 of 32 rows; otherwise the two
// groups take the same rows and turns by tile.
template <int D, bool FP8, int NRB, bool WIDE>
struct PagedCfg {
  static constexpr int RW = 8 * NRB, RB = WIDE ? 2 * RW : RW;
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int ROW_BYTES = D * ESZ;
  static constexpr int PANEL_ROW = ROW_BYTES >= 128 ? 128 : ROW_BYTES;
  static constexpr int NPANEL = ROW_BYTES / PANEL_ROW;
  static constexpr int PANEL_BYTES = 128 * PANEL_ROW;
  static constexpr int TILE_BYTES = 128 * ROW_BYTES;
  static constexpr int SCALE_BYTES = FP8 ? 2 * 128 * 4 : 0;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES + SCALE_BYTES;
  static constexpr int KS = D / 16;                          // k-steps of K Q^T
  static constexpr int MB = D / 16;                          // 16-row blocks of O^T
  static constexpr int PARTS = WIDE ? 4 : 8;                 // warps that hold a part of a row
  static constexpr int MCOLS = 32, MSTRIDE = MCOLS + 4;      // columns merged at a time
  static constexpr int Q_BYTES = RB / 8 * KS * 32 * 8;
  static constexpr int M_BYTES = NWARP * RW * MSTRIDE * 4;
  static constexpr int REST = 1024 + Q_BYTES + M_BYTES + NWARP * RW * 8 + RB * 12 + (PAGED_MAX_BATCH + 2) * 4 + 16 * 16 + 64;
  static constexpr int FIT = (227 * 1024 - REST) / STAGE_BYTES, WANT = 196608 / (2 * TILE_BYTES);
  static constexpr int NSTAGE = FIT < WANT ? FIT : WANT;     // up to 192 KB of K/V in flight
  static constexpr int Q_OFF = NSTAGE * STAGE_BYTES;         // query fragments [RB / 8][KS][32] x 8 bytes
  static constexpr int M_OFF = Q_OFF + Q_BYTES;              // merge buffer [NWARP][RW][MSTRIDE]
  static constexpr int ML_OFF = M_OFF + M_BYTES;             // [NWARP][RW] (max, sum)
  static constexpr int BITS_OFF = ML_OFF + NWARP * RW * 8;   // [RB] visible drafts
  static constexpr int RQ_OFF = BITS_OFF + RB * 8;           // [RB] largest magnitude of a query row (bits)
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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

template <int D, bool FP8, int NRB, bool WIDE>
__global__ void __launch_bounds__(NTHREADS, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedParams p) {
  using C = PagedCfg<D, FP8, NRB, WIDE>;
  constexpr int RB = C::RB, RW = C::RW, NSTAGE = C::NSTAGE;
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
  int* scratch = flags + 1;                      // [NWARP + NPROD]

  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  if (threadIdx.x == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(BAR_FULL(s), NPROD + (FP8 ? 64 : 0));
      mbar_init(BAR_EMPTY(s), NWARP);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  grid_launch_dependents();
  grid_dependency_wait();       // everything below reads what earlier kernels may have written
  if (!tile_prefix(p, pre, scratch, NTHREADS)) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && atomicCAS(p.err_word, 0, 1) == 0) atomicExch(p.err_info, WHERE_PAGED_LENS);
    if (threadIdx.x == 0) write_cut(p, pre, blockIdx.x, 0, 0);
    return;
  }
  const long long W = static_cast<long long>(pre[p.B]) * p.Hkv;
  const long long N = W < p.n_cta ? W : p.n_cta;
  if (static_cast<long long>(blockIdx.x) >= N) {
    if (threadIdx.x == 0) write_cut(p, pre, blockIdx.x, W, N);
    return;
  }
  const long long x0 = cta_start(blockIdx.x, W, N), x1 = cta_start(blockIdx.x + 1ll, W, N);
  const WaitCtl ctl{p.spin_limit, abort_flag, p.err_word, p.err_info};

  if (warp >= NWARP) {
    // ---- producers: page look-up and copies.  Warp pw takes the keys (pw even) or the values, and
    // every other copy of a tile; with E4M3 the first two also bring the scales ----
    // Box i of the list of boxes of a segment is br rows of one page; lane i % 32 looks its page up,
    // one batch of 32 boxes ahead of their use, and issues its copies.
    const int pw = warp - NWARP, kv = pw & 1, odd = pw >> 1;
    const CUtensorMap* tm = kv == 0 ? &tmK : &tmV;
    const float* scales = kv == 0 ? p.k_scale : p.v_scale;
    const int ps_log = 31 - __clz(p.page_size);
    const int br_log = ps_log < 7 ? ps_log : 7;
    const int pt_log = 7 - br_log, per_tile = 1 << pt_log;       // boxes of a tile (1 .. 8)
    // two panels: this warp's panel of every box; one panel: every other box
    const unsigned my_boxes = C::NPANEL == 2 ? 0xffu : (odd ? 0xaau : 0x55u);
    const int panel = C::NPANEL == 2 ? odd : 0;
    const uint64_t pol = l2_policy_evict_first();
    int it = 0;
    bool dead = false;                             // a wait gave up (the same in every lane)
    Segment s;
    for (long long x = x0; !dead && next_segment(p, pre, x, x1, s);) {
      const int L = *(p.ctx_lens + s.b) + (p.q_lens != nullptr ? *(p.q_lens + s.b) : p.T);
      const int* table = p.page_table + static_cast<long long>(s.b) * p.max_pages;
      // page of this lane's box in the batch that starts at tile j (-1: past the end).  The entry is
      // read before the length is known -- it lies in the table -- so the two loads overlap
      auto look_up = [&](int j) {
        const int at = (128 * j + (lane << br_log)) >> ps_log;
        return j < s.t1 && at < p.max_pages ? *(table + at) : -1;
      };
      const int batch = 32 >> pt_log;              // tiles of a batch
      int next = look_up(s.t0);
      for (int j0 = s.t0; j0 < s.t1 && !dead; j0 += batch) {
        const int page = next;
        next = look_up(j0 + batch);
        const int key = 128 * j0 + (lane << br_log);
        const bool wanted = key < L && j0 + (lane >> pt_log) < s.t1;
        const bool good = wanted && page >= 0 && page < p.n_pages;
        if (pw == 0 && wanted && !good && atomicCAS(p.err_word, 0, 1) == 0) atomicExch(p.err_info, WHERE_PAGED_PAGE);
        const unsigned boxes = __ballot_sync(0xffffffffu, good);
        const int row = key & (p.page_size - 1);
        for (int i = 0; i < batch && j0 + i < s.t1; ++i, ++it) {
          const int slot = it % NSTAGE;
          dead = !warp_wait(BAR_EMPTY(slot), ((it / NSTAGE) & 1) ^ 1u, ctl, WHERE_PAGED_LOAD);
          if (dead) break;
          const unsigned mine = (boxes >> (i << pt_log)) & ((1u << per_tile) - 1) & my_boxes;
          if (lane == 0) mbar_arrive_expect_tx(BAR_FULL(slot), (__popc(mine) << br_log) * C::PANEL_ROW);
          __syncwarp();
          const uint32_t st = base_u32 + slot * C::STAGE_BYTES;
          const int box = lane & (per_tile - 1);
          if ((lane >> pt_log) == i && ((mine >> box) & 1))
            tma_load_4d(st + kv * C::TILE_BYTES + panel * C::PANEL_BYTES + (box << br_log) * C::PANEL_ROW, tm, BAR_FULL(slot),
                        panel * (C::PANEL_ROW / C::ESZ), row, s.hkv, page, pol);
          if (FP8 && odd == 0) {
            // lane: the scales of four keys of the tile
            const int src = (i << pt_log) + (lane >> (br_log - 2));
            const int pg = __shfl_sync(0xffffffffu, page, src);
            const int r0 = __shfl_sync(0xffffffffu, row, src) + ((4 * lane) & ((1 << br_log) - 1));
            if ((boxes >> src) & 1)
              cp_async16(st + 2 * C::TILE_BYTES + 512 * kv + 16 * lane,
                         scales + (static_cast<long long>(pg) * p.Hkv + s.hkv) * p.page_size + r0);
            cp_async_arrive(BAR_FULL(slot));
          }
        }
      }
    }
    if (pw == 0 && lane == 0) write_cut(p, pre, blockIdx.x, W, N);   // the loads are all on their way
    if (dead) {
      cp_async_wait_all();
      if (lane == 0)
        for (int i = it > NSTAGE ? it - NSTAGE : 0; i < it; ++i)
          wait_drain_paged(BAR_FULL(i % NSTAGE), (i / NSTAGE) & 1, p.spin_limit);
    }
    return;
  }

  // ---- consumers: warp w takes keys 32 (w & 3) .. of a tile; the two groups of four warps take
  // the unit's row halves (WIDE) or every other tile ----
  const int g = lane >> 2, t4 = lane & 3;
  const int kw = 32 * (warp & 3), group = warp >> 2;
  const int rlo = WIDE ? RW * group : 0;         // first row of this warp
  uint2* qfrag = reinterpret_cast<uint2*>(base + C::Q_OFF);
  float* mbuf = reinterpret_cast<float*>(base + C::M_OFF);
  float2* ml = reinterpret_cast<float2*>(base + C::ML_OFF);
  unsigned long long* bits = reinterpret_cast<unsigned long long*>(base + C::BITS_OFF);
  int* qmax = reinterpret_cast<int*>(base + C::RQ_OFF);
  // key (within 8) that row g of an S^T block stands for.  E4M3: with the swizzle, the two rows that
  // eight lanes read at once then lie in different banks
  const int kg = FP8 ? (g >> 1) + 4 * (g & 1) : g;
  auto key_of = [&](int kb, int y) { return 16 * kb + 8 * y + kg; };

  // What a segment needs from memory before its first tile, fetched while the last one ends: its
  // lengths, query elements (item i of a thread: B registers of lane i % 32, k-step, 8-row block)
  // and visible drafts.
  constexpr int QI = RB / 8 * C::KS * 32 / (32 * NWARP);
  static_assert(QI >= 1 || RB / 8 * C::KS * 32 == 128, "query items");
  constexpr int QN = QI > 0 ? QI : 1;
  Segment sg;
  int ctx, ql;
  uint2 qraw[QN];
  unsigned long long my_bits;
  auto fetch = [&](long long& x) -> bool {
    if (!next_segment(p, pre, x, x1, sg)) return false;
    ctx = *(p.ctx_lens + sg.b);
    ql = p.q_lens != nullptr ? *(p.q_lens + sg.b) : p.T;
    const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(p.q) +
                              (static_cast<long long>(sg.b) * p.T * p.Hq + static_cast<long long>(sg.hkv) * p.G) * D;
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int e = static_cast<int>(threadIdx.x) + i * 32 * NWARP;
      const int l = e & 31, ks = (e >> 5) % C::KS, rb = (e >> 5) / C::KS;
      const int pr = 8 * rb + (l >> 2), t = token_of(p, pr);
      qraw[i] = make_uint2(0u, 0u);
      if (rb < RB / 8 && t < p.T) {                // rows past q_len are computed and not written
        const __nv_bfloat16* src = qb + (static_cast<long long>(t) * p.Hq + pr - t * p.G) * D;
        // bf16: k = 2t, 2t + 1 and 2t + 8, 2t + 9 of the step; E4M3: four elements in a row, the order in
        // which a thread reads the key's bytes
        if (FP8) {
          qraw[i] = *reinterpret_cast<const uint2*>(src + 16 * ((l & 3) + 4 * (ks >> 2)) + 4 * (ks & 3));
        } else {
          qraw[i].x = *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * (l & 3));
          qraw[i].y = *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * (l & 3) + 8);
        }
      }
    }
    my_bits = 0;
    if (threadIdx.x < RB) {
      const int t = token_of(p, static_cast<int>(threadIdx.x));
      if (t < p.T)
        my_bits = p.tree_mask != nullptr ? *(p.tree_mask + static_cast<long long>(sg.b) * p.T + t)
                                         : (t >= 63 ? ~0ull : (2ull << t) - 1);
    }
    return true;
  };
  if (threadIdx.x < RB) qmax[threadIdx.x] = 0;
  long long x = x0;
  bool more = fetch(x);
  named_bar_sync(1, 32 * NWARP);
  int it = 0;
  while (more) {
    const int L = ctx + ql;
    if (FP8) {
#pragma unroll
      for (int i = 0; i < QN; ++i) {
        const int e = static_cast<int>(threadIdx.x) + i * 32 * NWARP;
        const int rb = (e >> 5) / C::KS;
        float m = fmaxf(fmaxf(fabsf(__uint_as_float(qraw[i].x << 16)), fabsf(__uint_as_float(qraw[i].x & 0xffff0000u))),
                        fmaxf(fabsf(__uint_as_float(qraw[i].y << 16)), fabsf(__uint_as_float(qraw[i].y & 0xffff0000u))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (t4 == 0 && rb < RB / 8) atomicMax(qmax + 8 * rb + g, __float_as_int(m));   // m >= 0: ordered as integers
      }
      named_bar_sync(1, 32 * NWARP);
    }
    // per-row power of two that brings the largest query element into [1, 2): exact, and the logit
    // multiplier takes it back
    auto row_pow2 = [&](int r) {
      int ex = (qmax[r] >> 23) - 127;
      ex = ex < -110 ? -110 : (ex > 110 ? 110 : ex);
      return __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
    };
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int e = static_cast<int>(threadIdx.x) + i * 32 * NWARP;
      uint2 v = qraw[i];
      if ((e >> 5) / C::KS >= RB / 8) break;
      if (FP8) {
        const float inv = 1.f / row_pow2(8 * ((e >> 5) / C::KS) + g);
        v.x = pack_f16x2(__uint_as_float(v.x << 16) * inv, __uint_as_float(v.x & 0xffff0000u) * inv);
        v.y = pack_f16x2(__uint_as_float(v.y << 16) * inv, __uint_as_float(v.y & 0xffff0000u) * inv);
      }
      qfrag[e] = v;
    }
    if (threadIdx.x < RB) bits[threadIdx.x] = my_bits;
    named_bar_sync(1, 32 * NWARP);
    // rows of this thread: rlo + 8 rb + 2 t4 + e; everything per row is a pair (e = 0, 1)
    uint64_t cr[NRB];                              // logit multipliers
#pragma unroll
    for (int rb = 0; rb < NRB; ++rb) {
      const int r = rlo + 8 * rb + 2 * t4;
      cr[rb] = FP8 ? f2_pack(p.c_log2 * row_pow2(r), p.c_log2 * row_pow2(r + 1)) : f2_pack(p.c_log2, p.c_log2);
    }
    const uint2* qf = qfrag + (WIDE ? group * NRB : 0) * C::KS * 32 + lane;

    float o[NRB][C::MB][4];                        // O^T: (d, row 2t), (d, 2t + 1), (d', 2t), (d', 2t + 1)
    float m_run[NRB][2];
    uint64_t l_run[NRB];
    float vref = 0.f, vup = 0.f;                   // E4M3: power of two above the value scales seen, 2^10 / vref
#pragma unroll
    for (int rb = 0; rb < NRB; ++rb) {
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[rb][mb][i] = 0.f;
      m_run[rb][0] = m_run[rb][1] = -INFINITY;
      l_run[rb] = f2_pack(0.f, 0.f);
    }

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
        float s[2][NRB][4];                        // S^T of 16 keys: (key g, rows 2t, 2t + 1), (key g + 8, ..)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[kb][rb][i] = 0.f;
        // ---- S^T = K Q^T ----
        if constexpr (!FP8) {
          const int r = kw + (lane & 15), half = lane >> 4;
#pragma unroll
          for (int ks = 0; ks < C::KS; ++ks) {
            uint2 q[NRB];
#pragma unroll
            for (int rb = 0; rb < NRB; ++rb) q[rb] = qf[(rb * C::KS + ks) * 32];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              uint32_t a[4];
              ldsm4(sK + (ks >> 2) * C::PANEL_BYTES + (r + 16 * kb) * 128 + (((2 * (ks & 3) + half) ^ (r & 7)) << 4), a);
#pragma unroll
              for (int rb = 0; rb < NRB; ++rb)
                mma16816<false>(s[kb][rb], make_uint4(a[0], a[1], a[2], a[3]), q[rb].x, q[rb].y);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < C::KS / 4; ++i) {
            uint4 w[2][2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int r = kw + key_of(kb, y);
                const int ch = C::PANEL_ROW == 128 ? ((t4 + 4 * i) ^ kg) : (t4 ^ ((r >> 1) & 3));
                w[kb][y] = lds128(sK + r * C::PANEL_ROW + 16 * ch);
              }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint2 q[NRB];
#pragma unroll
              for (int rb = 0; rb < NRB; ++rb) q[rb] = qf[(rb * C::KS + 4 * i + c) * 32];
#pragma unroll
              for (int kb = 0; kb < 2; ++kb) {
                uint4 a;
                e4m3x4_to_f16(c == 0 ? w[kb][0].x : (c == 1 ? w[kb][0].y : (c == 2 ? w[kb][0].z : w[kb][0].w)), a.x, a.z);
                e4m3x4_to_f16(c == 0 ? w[kb][1].x : (c == 1 ? w[kb][1].y : (c == 2 ? w[kb][1].z : w[kb][1].w)), a.y, a.w);
#pragma unroll
                for (int rb = 0; rb < NRB; ++rb) mma16816<true>(s[kb][rb], a, q[rb].x, q[rb].y);
              }
            }
          }
        }
        // ---- scales of this thread's four keys ----
        [[maybe_unused]] float ksc[2][2], vsc[2][2];
        if constexpr (FP8) {
          const float* sc = reinterpret_cast<const float*>(base + slot * C::STAGE_BYTES + 2 * C::TILE_BYTES) + kw;
          float top = 0.f;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              ksc[kb][y] = sc[key_of(kb, y)];
              vsc[kb][y] = sc[128 + key_of(kb, y)];
              // an infinite or NaN scale goes to the rows that see it only
              if (TAIL && k0 + key_of(kb, y) >= L) vsc[kb][y] = 0.f;
              top = fmaxf(top, !TAIL || vsc[kb][y] < INFINITY ? vsc[kb][y] : 0.f);
            }
          if (__any_sync(0xffffffffu, top > vref)) {
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
            // next power of two above
            const float nref = __uint_as_float((__float_as_uint(top) & 0x7f800000u) + (top < 0x1p126f ? 0x00800000u : 0u));
            const float f = vref / nref;
#pragma unroll
            for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
              for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[rb][mb][i] *= f;
            vref = nref;
            vup = 1024.f / nref;
          }
        }
        // ---- logits (before the row's multiplier, which is positive), mask, running maximum ----
        uint64_t xs[NRB][2][2];
        float top2[NRB][2];
        bool grow = false;
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb) {
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint64_t v = f2_pack(s[kb][rb][2 * y], s[kb][rb][2 * y + 1]);
              if (FP8) v = f2_mul(v, f2_pack(ksc[kb][y], ksc[kb][y]));
              float v0, v1;
              f2_unpack(v, v0, v1);
              if (TAIL) {
                const int key = k0 + key_of(kb, y);
                const int r = rlo + 8 * rb + 2 * t4;
                const bool in = key < L;
                v0 = key < ctx || (in && ((bits[r] >> (key - ctx)) & 1)) ? v0 : -INFINITY;
                v1 = key < ctx || (in && ((bits[r + 1] >> (key - ctx)) & 1)) ? v1 : -INFINITY;
              }
              xs[rb][kb][y] = f2_pack(v0, v1);
              m0 = fmaxf(m0, v0);
              m1 = fmaxf(m1, v1);
            }
          f2_unpack(f2_mul(f2_pack(m0, m1), cr[rb]), top2[rb][0], top2[rb][1]);
          grow = grow || top2[rb][0] > m_run[rb][0] + 4.f || top2[rb][1] > m_run[rb][1] + 4.f;
        }
        if (__any_sync(0xffffffffu, grow)) {
          // lazily: the maxima are only looked up over the lanes, and O and the sum rescaled, when some
          // logit lies a factor of 2^4 above its row's reference
#pragma unroll
          for (int rb = 0; rb < NRB; ++rb) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = top2[rb][e];
#pragma unroll
              for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
              const float mn = fmaxf(m_run[rb][e], mx);
              f[e] = m_run[rb][e] == -INFINITY ? 0.f : ex2(m_run[rb][e] - mn);
              m_run[rb][e] = mn;
            }
            l_run[rb] = f2_mul(l_run[rb], f2_pack(f[0], f[1]));
#pragma unroll
            for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[rb][mb][i] *= f[i & 1];
          }
        }
        // ---- numerators, and their blocks turned into B operands (keys along k) ----
        uint32_t pb[NRB][2][2];
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb) {
          const uint64_t off = f2_pack(m_run[rb][0] == -INFINITY ? 0.f : -m_run[rb][0],
                                       m_run[rb][1] == -INFINITY ? 0.f : -m_run[rb][1]);
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float q0, q1;
              f2_unpack(f2_fma(xs[rb][kb][y], cr[rb], off), q0, q1);
              q0 = ex2(q0);
              q1 = ex2(q1);
              const uint64_t q = f2_pack(q0, q1);
              l_run[rb] = f2_add(l_run[rb], q);
              if constexpr (FP8) {
                const float vs = vsc[kb][y] * vup;
                float y0, y1;
                f2_unpack(f2_mul(q, f2_pack(vs, vs)), y0, y1);
                if (TAIL) {                        // a hidden key's scale may be anything: its numerator is 0
                  y0 = q0 == 0.f ? 0.f : y0;
                  y1 = q1 == 0.f ? 0.f : y1;
                }
                pb[rb][kb][y] = transpose8x8(pack_f16x2(y0, y1));
              } else {
                s[kb][rb][2 * y] = q0;
                s[kb][rb][2 * y + 1] = q1;
                pb[rb][kb][y] = transpose8x8(pack_bf16x2(q0, q1));
              }
            }
        }
        // ---- O^T += V^T P^T ----
        if constexpr (!FP8) {
          uint32_t odd = 0;                        // value rows past the end, or not finite: out of the product
          if (TAIL) {
            if (k0 + 32 > L) odd = ~0u << (L - k0);
            for (int r = ctx > k0 ? ctx - k0 : 0; r < 32 && k0 + r < L; ++r) {
              bool inf = false;
              for (int c = lane; c < D / 2; c += 32) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(base + (sV - base_u32) + (c >> 5) * C::PANEL_BYTES +
                                                                      (kw + r) * 128 + (c & 31) * 4);
                inf = inf || (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
              }
              if (__any_sync(0xffffffffu, inf)) odd |= 1u << r;
            }
            // those that some row may see are added element by element
            const uint32_t seen = k0 + 32 <= L ? odd : odd & ((1u << (L - k0)) - 1);
            if (seen != 0) {
#pragma unroll
              for (int ky = 0; ky < 4; ++ky)
                for (int r8 = 0; r8 < 8; ++r8) {
                  const int r = 8 * ky + r8;
                  if (!((seen >> r) & 1)) continue;
#pragma unroll
                  for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      // lane (r8, t) holds key r's numerators of rows 2t, 2t + 1
                      const float pv = __shfl_sync(0xffffffffu, s[ky >> 1][rb][2 * (ky & 1) + e], 4 * r8 + t4);
                      if (pv != 0.f) {
#pragma unroll
                        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
                          for (int y = 0; y < 2; ++y) {
                            const int ch = 2 * mb + y;
                            const __nv_bfloat16 v = *reinterpret_cast<const __nv_bfloat16*>(
                                base + (sV - base_u32) + (ch >> 3) * C::PANEL_BYTES + (kw + r) * 128 +
                                (((ch & 7) ^ ((kw + r) & 7)) << 4) + 2 * g);
                            o[rb][mb][2 * y + e] += pv * __bfloat162float(v);
                          }
                      }
                    }
                }
            }
          }
          // value fragment registers 0, 1 (2, 3) of 16 keys hold keys 2t, 2t + 1 (+ 8)
          uint32_t keep[2][2];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t two = odd >> (16 * kk + 8 * y + 2 * t4);
              keep[kk][y] = ((two & 1u) ? 0u : 0xffffu) | ((two & 2u) ? 0u : 0xffff0000u);
            }
          const int r = kw + (lane & 7) + 8 * (lane >> 4), half = (lane >> 3) & 1;
          auto add = [&](bool masked) {
#pragma unroll
            for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                uint32_t a[4];
                ldsm4t(sV + (mb >> 2) * C::PANEL_BYTES + (r + 16 * kk) * 128 + (((2 * (mb & 3) + half) ^ (r & 7)) << 4), a);
                if (masked) {
#pragma unroll
                  for (int y = 0; y < 4; ++y) a[y] &= keep[kk][y >> 1];
                }
#pragma unroll
                for (int rb = 0; rb < NRB; ++rb)
                  mma16816<false>(o[rb][mb], make_uint4(a[0], a[1], a[2], a[3]), pb[rb][kk][0], pb[rb][kk][1]);
              }
          };
          if (TAIL && odd != 0) add(true);
          else add(false);
        } else {
          // lane g reads D / 8 bytes of rows t, t + 4, t + 8, t + 12 of each 16 -- the keys of S^T's rows
          // 2t, 2t + 1 (+ 8).  A row that must not show is read as zeros (its codes may be NaN), and
          // shows in the rows that see it through its scale
          constexpr int NW = D / 32;
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            uint32_t w[4][NW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kr = 16 * kk + t4 + 4 * i, r = kw + kr;
              if constexpr (D == 128) {
                const uint4 u = lds128(sV + r * 128 + ((((g >> 1) | ((g & 1) << 2)) ^ (r & 7)) << 4));
                w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
              } else {
                const int ch = ((g >> 2) & 1) | (((g >> 1) & 1) << 1);
                const uint2 u = lds64(sV + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4) + 8 * (g & 1));
                w[i][0] = u.x; w[i][1] = u.y;
              }
              if (TAIL) {
                const float vs = reinterpret_cast<const float*>(base + slot * C::STAGE_BYTES + 2 * C::TILE_BYTES)[128 + r];
                if (k0 + kr >= L || !(vs < INFINITY)) {
#pragma unroll
                  for (int c = 0; c < NW; ++c) w[i][c] = 0u;
                }
              }
            }
#pragma unroll
            for (int mb = 0; mb < C::MB; ++mb) {
              // bytes 2 mb, 2 mb + 1 of the lane's piece, of rows (t, t + 4) and (t + 8, t + 12)
              const int c = mb >> 1;
              const uint32_t sel = (mb & 1) == 0 ? 0x5140u : 0x7362u;
              uint4 a;
              e4m3x4_to_f16(__byte_perm(w[0][c], w[1][c], sel), a.x, a.y);
              e4m3x4_to_f16(__byte_perm(w[2][c], w[3][c], sel), a.z, a.w);
#pragma unroll
              for (int rb = 0; rb < NRB; ++rb) mma16816<true>(o[rb][mb], a, pb[rb][kk][0], pb[rb][kk][1]);
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

    // ---- the warps' partial results meet; the next segment's inputs are on their way meanwhile ----
    const Segment dn = sg;
    const int ql_dn = ql;
    more = fetch(x);
#pragma unroll
    for (int rb = 0; rb < NRB; ++rb) {
      float l[2];
      f2_unpack(l_run[rb], l[0], l[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], sh);
        if (g == 0) ml[warp * RW + 8 * rb + 2 * t4 + e] = make_float2(m_run[rb][e], l[e]);
      }
    }
    named_bar_sync(1, 32 * NWARP);
    // (max, sum) over the warps that hold a part of row r of the unit
    auto whole_row = [&](int r, float& M, float& l) {
      const float2* e = ml + (WIDE ? (r / RW) * 4 * RW : 0) + r % RW;
      M = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int w = 0; w < C::PARTS; ++w) M = fmaxf(M, e[RW * w].x);
#pragma unroll
      for (int w = 0; w < C::PARTS; ++w) l += e[RW * w].x == -INFINITY ? e[RW * w].y : e[RW * w].y * ex2(e[RW * w].x - M);
    };
    float f[NRB][2];
#pragma unroll
    for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M, l;
        whole_row(rlo + 8 * rb + 2 * t4 + e, M, l);
        f[rb][e] = m_run[rb][e] == -INFINITY ? 0.f : ex2(m_run[rb][e] - M) / l;
        if (FP8) f[rb][e] *= vref * 0x1p-10f;      // the 2^10 of the numerators
      }
    const bool whole = dn.t0 == 0 && dn.t1 == dn.n;
    const long long ws_slot = 2ll * blockIdx.x + (dn.t0 > 0 ? 0 : 1);
    if (threadIdx.x < RB) {
      const int r = threadIdx.x;
      qmax[r] = 0;
      float M, l;
      whole_row(r, M, l);
      const float lse2 = l == 0.f ? -INFINITY : M + __log2f(l);
      const int t = token_of(p, r);
      if (!whole) p.ws_l[ws_slot * RB + r] = lse2;
      else if (t < ql_dn && p.lse != nullptr)
        p.lse[(static_cast<long long>(dn.b) * p.Hq + dn.hkv * p.G + r - t * p.G) * p.T + t] = lse2 * LN2_P;
    }
    // 32 columns at a time: column 16 m + 8 y + g of the buffer is row g + 8 y of O^T's block m
#pragma unroll
    for (int pass = 0; pass < D / 32; ++pass) {
      if (pass > 0) named_bar_sync(1, 32 * NWARP);
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mbuf[(warp * RW + 8 * rb + 2 * t4 + (i & 1)) * C::MSTRIDE + 16 * m + 8 * (i >> 1) + g] =
                o[rb][2 * pass + m][i] * f[rb][i & 1];
      named_bar_sync(1, 32 * NWARP);
#pragma unroll
      for (int r0 = 0; r0 < RB; r0 += 16) {
        // thread: two output columns of one row
        const int r = r0 + static_cast<int>(threadIdx.x) / 16, c2 = threadIdx.x % 16;
        if (r >= RB) continue;
        int i0, i1, d;
        if (FP8) {                                 // d of block m, row g + 8 y: piece(g) + 2 m + y
          const int n = c2 & 7, m = c2 >> 3;
          i0 = 16 * m + n;
          i1 = i0 + 8;
          const int first = D == 128 ? 16 * ((n >> 1) | ((n & 1) << 2))
                                     : 16 * (((n >> 2) & 1) | (((n >> 1) & 1) << 1)) + 8 * (n & 1);
          d = first + 2 * (2 * pass + m);
        } else {
          i0 = 2 * c2;
          i1 = i0 + 1;
          d = 32 * pass + 2 * c2;
        }
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int w = 0; w < C::PARTS; ++w) {
          const float* src = mbuf + ((WIDE ? (r / RW) * 4 : 0) + w) * RW * C::MSTRIDE + (r % RW) * C::MSTRIDE;
          a += src[i0];
          b += src[i1];
        }
        const int t = token_of(p, r);
        if (t < ql_dn) {
          if (whole)
            *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) +
                                         ((static_cast<long long>(dn.b) * p.T + t) * p.Hq + dn.hkv * p.G + r - t * p.G) * D + d) =
                pack_bf16x2(a, b);
          else
            *reinterpret_cast<float2*>(p.ws_o + (ws_slot * RB + r) * D + d) = make_float2(a, b);
        }
      }
    }
    named_bar_sync(1, 32 * NWARP);                 // the next unit rewrites the shared arrays
  }
}

// Rows of a merge block of eight warps where a unit has many parts: one a warp where a unit has 64 rows or more; few
// rows a unit: the parts of a row are read by several warps at once.  (Four rows a warp, one after the other:
// 3 us more on 128 rows.)
template <int RB>
constexpr int COMBINE_ROWS = RB >= 64 ? 8 : RB / 8;

// Merge of the units that several groups share.  A block takes rows of one row tile of the unit that group
// i + 1's start cuts, as write_cut says.
template <int D, int RB>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p) {
  constexpr int NW = 8, E = D / 32, SHARE = NW / COMBINE_ROWS<RB>;
  constexpr int BATCH = SHARE == 1 ? 4 : 8;                     // parts of a row in flight
  __shared__ float part[NW][D + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int at = static_cast<int>(blockIdx.x / p.row_tiles), rt = static_cast<int>(blockIdx.x % p.row_tiles);
  grid_launch_dependents();
  grid_dependency_wait();       // in every block: this grid's end stands for the key kernel's too
  const int4 cut = ld_l2(p.cuts + at + 1);
  const int n = cut.x & 0xffff, k_cut = cut.x >> 16, c0 = at - k_cut;        // parts: groups c0 .. c0 + n - 1
  // warps of a row.  16 and 32 rows of few parts take half the blocks, which then are on the device at once:
  // 1.2 and 1.9 us less over 128 units; 8 rows want all the warps.
  // Many parts: a row a block, over the blocks of all the unit's cuts (one unit of 152 parts and 32 rows: 22 us in
  // the blocks of one cut).
  const int share = n > MANY_PARTS ? NW : (SHARE > 1 && SHARE < 8 && n <= 4 ? SHARE / 2 : SHARE);
  const int first = (NW / share) * (blockIdx.y + k_cut * gridDim.y), rows = min(RB, cut.w * p.G - rt * RB) - first;
  if (n == 0 || rows <= 0) return;
  // c0's part is its last unit's (slot 1), the others' their first's (slot 0)
  auto slot = [&](int c) { return 2ll * ((c0 + c) * static_cast<long long>(p.row_tiles) + rt) + (c == 0 ? 1 : 0); };
  const int r = first + warp / share, sub = warp % share;
  const bool live = r - first < rows;
  float mx = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  // add a part of (lse l, weight s, output v); one that saw no key has l = -inf and weight 0, and zeros (or
  // NaN, which stays)
  auto add = [&](float l, float s, const float* v) {
    const float m = fmaxf(mx, l);
    const float f = mx == -INFINITY ? 1.f : ex2(mx - m), w = l == -INFINITY ? 1.f : ex2(l - m);
    mx = m;
    sum = fmaf(sum, f, s * w);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, w * v[e]);
  };
  if (live) {
    // lane: columns E lane ..
    for (int cb = sub; cb < n; cb += BATCH * share) {
      float l[BATCH], v[BATCH][E];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        // past the last part: that part again, not added (no branch between the loads)
        const int c = cb + k * share < n ? cb + k * share : n - 1;
        l[k] = ld_l2(p.ws_l + slot(c) * RB + r);
        const float* src = p.ws_o + (slot(c) * RB + r) * D + lane * E;
        if constexpr (E == 4) {
          const float4 u = ld_l2(reinterpret_cast<const float4*>(src));
          v[k][0] = u.x; v[k][1] = u.y; v[k][2] = u.z; v[k][3] = u.w;
        } else {
          const float2 u = ld_l2(reinterpret_cast<const float2*>(src));
          v[k][0] = u.x; v[k][1] = u.y;
        }
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (cb + k * share >= n) break;
        add(l[k], l[k] == -INFINITY ? 0.f : 1.f, v[k]);
      }
    }
  }
  if (share > 1) {
    if (live) {
#pragma unroll
      for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
      if (lane == 0) {
        part[warp][D] = mx;
        part[warp][D + 1] = sum;
      }
    }
    __syncthreads();
    if (live && sub == 0)
      for (int w = 1; w < share; ++w) add(part[warp + w][D], part[warp + w][D + 1], &part[warp + w][lane * E]);
  }
  if (live && sub == 0) {
    const int pr = rt * RB + r, t = token_of(p, pr);
    const float inv = sum == 0.f ? 1.f : 1.f / sum;          // no key at all: the parts' zeros
    const long long h = static_cast<long long>(cut.z) * p.G + pr - t * p.G;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + ((static_cast<long long>(cut.y) * p.T + t) * p.Hq + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
      p.lse[(static_cast<long long>(cut.y) * p.Hq + h) * p.T + t] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * LN2_P;
  }
}

// The merge starts while the key kernel's last CTAs finish and waits for them on the device.
template <int D, int RB>
cudaError_t launch_paged_combine(const PagedParams& p, cudaStream_t st) {
  if (p.n_cta < 2) return cudaSuccess;
  const int rows = p.G * p.T < RB ? p.G * p.T : RB;
  return launch_overlapped(paged_combine_kernel<D, RB>,
                           dim3(static_cast<unsigned>(p.n_cta - 1) * p.row_tiles, (rows + COMBINE_ROWS<RB> - 1) / COMBINE_ROWS<RB>),
                           256, 0, st, p);
}

template <int D, bool FP8, int NRB, bool WIDE>
cudaError_t launch_paged_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, cudaStream_t st) {
  using C = PagedCfg<D, FP8, NRB, WIDE>;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((configured.load() & bit) == 0) {
    e = cudaFuncSetAttribute(attn_paged_kernel<D, FP8, NRB, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return launch_overlapped(attn_paged_kernel<D, FP8, NRB, WIDE>, dim3(p.n_cta), NTHREADS, C::SMEM_BYTES, st, tk, tv, p);
}

template <int D>
cudaError_t launch_combine_rows(const PagedParams& p, int rb, cudaStream_t st) {
  return rb == 8    ? launch_paged_combine<D, 8>(p, st)
         : rb == 16  ? launch_paged_combine<D, 16>(p, st)
         : rb == 32 ? launch_paged_combine<D, 32>(p, st)
         : rb == 64 ? launch_paged_combine<D, 64>(p, st)
                    : launch_paged_combine<D, PAGED_TREE_ROWS>(p, st);
}

}  // namespace

cudaError_t launch_attn_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int D, bool fp8,
                              bool combine, cudaStream_t st) {
  const int rb = paged_rows(p.G * p.T);
  cudaError_t e;
  if (rb == PAGED_TREE_ROWS) {
    e = launch_attn_tree(tk, tv, p, D, fp8, st);
  } else if (rb == 64 || (fp8 && rb > 8)) {
    // 16 sequences of up to 8192 keys, and of 700, there and in this file's kernel: 4 rows of E4M3 43.8 and 42.2 us
    // (14.9, 12.2), 16 45.5 and 46.5 (15.6, 16.6), 32 50.1 and 72.5; of bf16 16 rows 77.8 and 74.8 (18.9, 16.9), 32 79.3
    // and 76.1 (22.0, 18.6).
    e = launch_attn_lanes(tk, tv, p, D, fp8, st);
  } else if (fp8) {
    e = D == 64 ? launch_paged_d<64, true, 1, false>(tk, tv, p, st) : launch_paged_d<128, true, 1, false>(tk, tv, p, st);
  } else if (rb == 8) {
    e = D == 64 ? launch_paged_d<64, false, 1, false>(tk, tv, p, st) : launch_paged_d<128, false, 1, false>(tk, tv, p, st);
  } else if (rb == 16) {
    e = D == 64 ? launch_paged_d<64, false, 2, false>(tk, tv, p, st) : launch_paged_d<128, false, 2, false>(tk, tv, p, st);
  } else {
    e = D == 64 ? launch_paged_d<64, false, 2, true>(tk, tv, p, st) : launch_paged_d<128, false, 2, true>(tk, tv, p, st);
  }
  if (e != cudaSuccess || !combine) return e;
  return D == 64 ? launch_combine_rows<64>(p, rb, st) : launch_combine_rows<128>(p, rb, st);
}

}  // namespace ea46
