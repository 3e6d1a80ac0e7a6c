// attn_tree.cu -- attention of a drafted tree (or many heads) over a paged key/value cache: more than 32
// query rows (heads of a group x drafted tokens) per key/value head, for sm_103a.  What it
// computes, the readings and the list of key tiles are attn_paged.cu's and paged.cuh's.
//
// With 33 or more rows the 128-row tile of tcgen05 is used well: S = Q K^T and O += P V run on it with
// S, P and O in Tensor Memory.  128 rows take about 1100 cycles of the
// tensor pipe and about as many of the exp2 units per 128-key tile of D = 128 in bf16, against the 2800
// the tile takes from HBM at an SM's share of it, so one row tile is bound by HBM and several by
// compute; the CTAs of a group take one row tile each and the same keys, which all but the first find
// in L2.
//   * warps 0..7 softmax (thread = row and half of the tile's keys; the two warps of a quarter of Tensor
//     Memory exchange their maxima, and hide each other's latencies), 8 issues the MMAs, 9 and 10
//     load K and V tiles by TMA (one box per page and swizzle panel) through a ring each, 11 the
//     E4M3 scales;
//   * S and P are double-buffered: S(i + 1) is issued before PV(i).  The running maximum is lazy (O is
//     rescaled in Tensor Memory only when a maximum moves by more than 2^TAU);
//   * the next unit's queries are written to shared memory before the last unit's epilogue, so its
//     first S is computed meanwhile;
//   * E4M3: the products run on the codes themselves.  A query row, scaled by a power of two into
//     E4M3's range, is the exact sum of two E4M3 terms (bf16 has eight significant bits, each term
//     four; below 2^-10 of the row's largest element the second loses bits, 2^-18 of the largest at
//     most), and a numerator times its value's scale is rounded to the sum of three E5M2 terms: 2^-9 of it, as bf16
//     would be.  (One E4M3 term would be off by 2^-4, two lose what lies 2^-17 under the largest.)
//     Each term is one more MMA over the same tile;
//   * hidden keys: logits replaced by -inf before the maximum.  In tiles with drafted keys or the end of
//     the sequence the value rows past the end are zeroed in shared memory, and so is what is not
//     finite in a drafted row; the rows that see it get it in the epilogue (E4M3: a scale that is
//     not finite makes their numerators NaN).
// Every mbarrier wait is bounded.
//
// Measured: 8 sequences of up to 8192 keys, trees of 32 of 32 query over 8 key/value heads (128 rows), bf16, 218 MB,
// 32.2 us at the copy rate: 46.4 us; the key kernel ends 36 us after it may start, the merge takes 6.  256 rows: bf16
// 119 us (two row tiles, the second's keys from L2), E4M3 232 us, bound by the softmax and by the
// terms' conversion.
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <type_traits>

#include "cache.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ea46 {

namespace {

template <int D, bool FP8>
struct TreeCfg {
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int ROW_BYTES = D * ESZ;
  static constexpr int PANEL_ROW = ROW_BYTES >= 128 ? 128 : ROW_BYTES;
  static constexpr int NPANEL = ROW_BYTES / PANEL_ROW;
  static constexpr int PANEL_BYTES = 128 * PANEL_ROW;
  static constexpr int TILE_BYTES = 128 * ROW_BYTES;
  static constexpr int NQ = FP8 ? 2 : 1;                      // query tiles: terms of the queries
  static constexpr int NP = FP8 ? 3 : 1;                      // terms of the numerators
  // K and V tiles in flight
  static constexpr int NK = TILE_BYTES == 32768 ? 3 : (TILE_BYTES == 16384 ? 5 : 8);
  static constexpr int NV = TILE_BYTES == 32768 ? 2 : (TILE_BYTES == 16384 ? 5 : 8);
  static constexpr int NSC = FP8 ? 4 : 0;                     // stages of 128 key and 128 value scales
  static constexpr uint32_t SBO = 8 * PANEL_ROW;
  static constexpr uint32_t LAYOUT = PANEL_ROW == 128 ? 2u : 4u;
  static constexpr int KSTEPS_QK = ROW_BYTES / 32;
  static constexpr int STEPS_PER_PANEL = PANEL_ROW / 32;
  static constexpr int UMMA_K = FP8 ? 32 : 16;
  static constexpr int KSTEPS_PV = 128 / UMMA_K;
  static constexpr uint32_t FMT = FP8 ? 0u : 1u;
  static constexpr uint32_t IDESC_QK = instr_desc(FMT, 0, 128, 128);
  static constexpr uint32_t IDESC_PV = instr_desc(FMT, 1, 128, D) | (FP8 ? 1u << 7 : 0u);     // A: E5M2 (bf16: FMT)
  // Tensor Memory: S buffers at columns 0 and 128, O at 256, after it two P buffers of 64 columns (E4M3: one, 32
  // columns for each term)
  static constexpr uint32_t O_COL = 256, P_COL = 256 + D;
  static constexpr int K_OFF = NQ * TILE_BYTES, V_OFF = K_OFF + NK * TILE_BYTES;
  static constexpr int SC_OFF = V_OFF + NV * TILE_BYTES;
  static constexpr int PRE_OFF = SC_OFF + NSC * 1024;
  static constexpr int RED_OFF = PRE_OFF + (PAGED_MAX_BATCH + 4) * 4;       // [3][2][128] floats: maxima (twice), sums
  static constexpr int FLAG_OFF = RED_OFF + 3 * 2 * 128 * 4;                // vodd [2] x 8, tmem, abort, scratch
  static constexpr int STAGE_ROW = 20;                                      // floats: 16 columns and padding
  static constexpr int STAGE_OFF = FLAG_OFF + 96;                           // [8 warps][32][STAGE_ROW]
  static constexpr int BAR_OFF = STAGE_OFF + 8 * 32 * STAGE_ROW * 4;
  static constexpr int NBAR = 8 + 2 * (NK + NV + NSC);
  static constexpr int SMEM_BYTES = 1024 + BAR_OFF + NBAR * 8;
  static_assert(FLAG_OFF % 8 == 0 && STAGE_OFF % 16 == 0 && BAR_OFF % 8 == 0, "alignment");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(P_COL + 128 <= 512, "Tensor Memory budget");
};

constexpr int TREE_THREADS = 384;
constexpr int MMA_WARP = 8, K_WARP = 9, S_WARP = 11;
constexpr float TAU_BF16 = 8.0f;        // lazy rescale threshold (log2): numerators reach 2^TAU

// Registers of a warpgroup, out of the block's: 384 threads x 168 = 2 x 128 x 200 + 128 x 104.  The E4M3
// softmax spills 588 bytes in 168; bf16 fits.
__device__ __forceinline__ void softmax_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 200;"); }
__device__ __forceinline__ void other_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }

template <int D, bool FP8>
__global__ void __launch_bounds__(TREE_THREADS, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PagedParams p) {
  using C = TreeCfg<D, FP8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  const uint32_t sQ = base_u32, sK = base_u32 + C::K_OFF, sV = base_u32 + C::V_OFF;
  int* pre = reinterpret_cast<int*>(base + C::PRE_OFF);
  unsigned long long* vodd_sh = reinterpret_cast<unsigned long long*>(base + C::FLAG_OFF);   // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::FLAG_OFF + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::FLAG_OFF + 20);
  int* scratch = reinterpret_cast<int*>(base + C::FLAG_OFF + 24);                            // [12]
  float* red = reinterpret_cast<float*>(base + C::RED_OFF);                                  // [3][2][128]
  const uint32_t bar0 = base_u32 + C::BAR_OFF;
  const uint32_t BAR_Q = bar0, BAR_O = bar0 + 8, BAR_DONE = bar0 + 16, BAR_PV = bar0 + 24;
  auto BAR_S = [&](int b) { return bar0 + 32 + 8u * b; };
  auto BAR_P = [&](int b) { return bar0 + 48 + 8u * b; };
  auto FULLK = [&](int s) { return bar0 + 64 + 8u * s; };
  auto EMPTYK = [&](int s) { return bar0 + 64 + 8u * (C::NK + s); };
  auto FULLV = [&](int s) { return bar0 + 64 + 8u * (2 * C::NK + s); };
  auto EMPTYV = [&](int s) { return bar0 + 64 + 8u * (2 * C::NK + C::NV + s); };
  auto FULLS = [&](int s) { return bar0 + 64 + 8u * (2 * (C::NK + C::NV) + s); };
  auto EMPTYS = [&](int s) { return bar0 + 64 + 8u * (2 * (C::NK + C::NV) + C::NSC + s); };

  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  if (threadIdx.x == 0) {
    mbar_init(BAR_Q, 8);
    mbar_init(BAR_O, 1);
    mbar_init(BAR_DONE, 1);
    mbar_init(BAR_PV, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(BAR_S(b), 1);
      mbar_init(BAR_P(b), 8);
    }
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(FULLK(s), 1);
      mbar_init(EMPTYK(s), 1);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(FULLV(s), 1);
      mbar_init(EMPTYV(s), 1);
    }
    for (int s = 0; s < C::NSC; ++s) {
      mbar_init(FULLS(s), 32);
      mbar_init(EMPTYS(s), 8);
    }
    *abort_flag = 0;
    vodd_sh[0] = vodd_sh[1] = 0;
    fence_barrier_init();
  }
  grid_launch_dependents();
  grid_dependency_wait();       // everything below reads what earlier kernels may have written
  const bool fine = tile_prefix(p, pre, scratch, TREE_THREADS);
  if (!fine) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && atomicCAS(p.err_word, 0, 1) == 0) atomicExch(p.err_info, WHERE_PAGED_LENS);
    if (threadIdx.x == 0 && blockIdx.x % p.group_ctas == 0) write_cut(p, pre, blockIdx.x / p.group_ctas, 0, 0);
    return;
  }
  const long long W = static_cast<long long>(pre[p.B]) * p.Hkv;
  const long long N = W < p.n_cta ? W : p.n_cta;
  const int group = blockIdx.x / p.group_ctas, rt0 = blockIdx.x % p.group_ctas;
  if (group >= N) {
    if (threadIdx.x == 0 && rt0 == 0) write_cut(p, pre, group, W, N);
    return;
  }
  const long long x0 = cta_start(group, W, N), x1 = cta_start(group + 1ll, W, N);
  if (warp == MMA_WARP) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{p.spin_limit, abort_flag, p.err_word, p.err_info};
  const TileRings rings{sK, sV, base_u32 + C::SC_OFF, FULLK(0), EMPTYK(0), FULLV(0), EMPTYV(0), FULLS(0), EMPTYS(0)};

  if constexpr (FP8) {
    if (warp >= MMA_WARP) other_registers();
    else softmax_registers();
  }

  if (warp >= K_WARP) {
    if (FP8 || warp < S_WARP) load_tiles<C>(p, pre, tmK, tmV, rings, warp - K_WARP, rt0, x0, x1, ctl);
    if (warp == K_WARP && rt0 == 0 && lane == 0) write_cut(p, pre, group, W, N);
  } else if (warp == MMA_WARP) {
    // ---- MMA issue ----
    if (elect_one()) {
      const uint64_t dq = smem_desc(sQ, 16, C::SBO, C::LAYOUT);
      const uint64_t dk0 = smem_desc(sK, 16, C::SBO, C::LAYOUT);
      const uint64_t dv0 = smem_desc(sV, C::PANEL_BYTES, C::SBO, C::LAYOUT);
      bool ok = true;
      Segment s;
      int it = 0, seg = 0;
      auto qk = [&](int i) -> bool {
        const int ks = i % C::NK;
        if (!wait_bounded(FULLK(ks), (i / C::NK) & 1, ctl, WHERE_PAGED_MMA)) return false;
        tc_fence_after();
        const uint64_t bk = dk0 + ((ks * C::TILE_BYTES) >> 4);
#pragma unroll
        for (int term = 0; term < C::NQ; ++term)
#pragma unroll
          for (int kk = 0; kk < C::KSTEPS_QK; ++kk) {
            const uint32_t off = ((kk / C::STEPS_PER_PANEL) * C::PANEL_BYTES + (kk % C::STEPS_PER_PANEL) * 32) >> 4;
            const uint64_t aq = dq + off + ((term * C::TILE_BYTES) >> 4);
            if (FP8) mma_f8_ss(tmem + 128u * (i & 1), aq, bk + off, C::IDESC_QK, (kk > 0 || term > 0) ? 1u : 0u);
            else     mma_f16_ss(tmem + 128u * (i & 1), aq, bk + off, C::IDESC_QK, kk > 0 ? 1u : 0u);
          }
        mma_commit(BAR_S(i & 1));
        mma_commit(EMPTYK(ks));
        return true;
      };
      for (int rt = rt0; ok && rt < p.row_tiles; rt += p.group_ctas)
        for (long long x = x0; ok && next_segment(p, pre, x, x1, s); ++seg) {
          const int n = s.t1 - s.t0;
          if (!(ok = wait_bounded(BAR_Q, seg & 1, ctl, WHERE_PAGED_MMA))) break;
          if (!(ok = qk(it))) break;
          for (int j = 0; j < n; ++j, ++it) {
            // S(it + 1) overwrites S(it - 1), which the softmax read before it handed over P(it - 1)
            if (j + 1 < n && !(ok = qk(it + 1))) break;
            if (!(ok = wait_bounded(BAR_P(it & 1), (it >> 1) & 1, ctl, WHERE_PAGED_MMA))) break;
            const int vs = it % C::NV;
            if (!(ok = wait_bounded(FULLV(vs), (it / C::NV) & 1, ctl, WHERE_PAGED_MMA))) break;
            tc_fence_after();
            const uint64_t bv = dv0 + ((vs * C::TILE_BYTES) >> 4);
            const uint32_t pa = tmem + C::P_COL + (FP8 ? 0u : 64u * (it & 1));
#pragma unroll
            for (int term = 0; term < C::NP; ++term)
#pragma unroll
              for (int kk = 0; kk < C::KSTEPS_PV; ++kk) {
                const uint32_t off = (kk * C::UMMA_K * C::PANEL_ROW) >> 4;
                const uint32_t acc = (j > 0 || kk > 0 || term > 0) ? 1u : 0u;
                if (FP8) mma_f8_ts(tmem + C::O_COL, pa + 32u * term + 8u * kk, bv + off, C::IDESC_PV, acc);
                else     mma_f16_ts(tmem + C::O_COL, pa + 8u * kk, bv + off, C::IDESC_PV, acc);
              }
            mma_commit(BAR_PV);
            mma_commit(EMPTYV(vs));
          }
          if (ok) mma_commit(BAR_O);
        }
      mma_commit(BAR_DONE);
      wait_drain_paged(BAR_DONE, 0, p.spin_limit);
    }
  } else {
    // ---- softmax: warps w and w + 4 share the rows of Tensor Memory's quarter w & 3 (its own SM
    // sub-partition); thread = row r, half hf of the tile's keys, of the head and of the output ----
    const int r = 32 * (warp & 3) + lane, hf = warp >> 2;
    const uint32_t tl = tmem + (static_cast<uint32_t>(warp & 3) << 21);      // this warp's 32 lanes
    const uint32_t pair_bar = 2u + (warp & 3);
    Segment sg;
    int ctx = 0, ql = 0;
    unsigned long long bits = 0;
    float cmul = p.c_log2;
    bool bad = false;                              // a wait of this warp gave up; it still meets the barriers
    // Lengths, mask and query row of the segment that starts at x; the row goes to shared memory.  Runs when
    // the last segment's S = Q K^T are complete.
    auto fetch = [&](int rt, long long& x) -> bool {
      if (!next_segment(p, pre, x, x1, sg)) return false;
      const int pr = rt * PAGED_TREE_ROWS + r, t = token_of(p, pr);
      const bool there = t < p.T;
      // this half of the row, all of it on its way before anything is waited for: behind the first K and V tiles in
      // the memory's queues it takes 3 us longer
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(p.q) +
          ((static_cast<long long>(sg.b) * p.T + t) * p.Hq + sg.hkv * p.G + pr - t * p.G) * D);
      uint4 u[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) u[i] = there ? src[hf * (D / 16) + i] : make_uint4(0u, 0u, 0u, 0u);
      ctx = *(p.ctx_lens + sg.b);
      ql = p.q_lens != nullptr ? *(p.q_lens + sg.b) : p.T;
      bits = 0;
      if (there)
        bits = p.tree_mask != nullptr ? *(p.tree_mask + static_cast<long long>(sg.b) * p.T + t)
                                      : (t >= 63 ? ~0ull : (2ull << t) - 1);
      if (ql < 64) bits &= (1ull << ql) - 1;
      if constexpr (!FP8) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int c = hf * (D / 16) + i;
          st_shared_v4(sQ + (c >> 3) * C::PANEL_BYTES + r * 128 + (((c & 7) ^ (r & 7)) << 4), u[i].x, u[i].y, u[i].z, u[i].w);
        }
      } else {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
        }
        // the row's largest element over its two threads (the sums' array is free here), and the power of
        // two that brings it into [128, 256): exact
        named_bar_sync(pair_bar, 64u);
        red[512 + 128 * hf + r] = m;
        named_bar_sync(pair_bar, 64u);
        m = fmaxf(m, red[512 + 128 * (hf ^ 1) + r]);
        int ex = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        ex = ex < -100 ? -100 : (ex > 100 ? 100 : ex);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - ex) << 23);
        // (an infinite element, which E4M3 cannot hold, makes the row's logits NaN)
        cmul = m == INFINITY ? __int_as_float(0x7fffffff) : p.c_log2 * __uint_as_float(static_cast<uint32_t>(127 - 7 + ex) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int c = hf * (D / 32) + i;
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint4 w = u[2 * i + y];
            e4m3_terms4(__uint_as_float(w.x << 16) * up, __uint_as_float(w.x & 0xffff0000u) * up,
                        __uint_as_float(w.y << 16) * up, __uint_as_float(w.y & 0xffff0000u) * up, hi[2 * y], lo[2 * y]);
            e4m3_terms4(__uint_as_float(w.z << 16) * up, __uint_as_float(w.z & 0xffff0000u) * up,
                        __uint_as_float(w.w << 16) * up, __uint_as_float(w.w & 0xffff0000u) * up, hi[2 * y + 1],
                        lo[2 * y + 1]);
          }
          const uint32_t at = sQ + r * C::PANEL_ROW +
                              ((C::PANEL_ROW == 128 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3))) << 4);
          st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(at + C::TILE_BYTES, lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR_Q);
      return true;
    };
    int it = 0, seg = 0, sslot = 0;
    uint32_t spar = 0;
    long long x = x0;
    bool more = fetch(rt0, x);
    for (int rt = rt0; more; ++seg) {
      const Segment dn = sg;
      const int dn_rt = rt;
      const int my_ctx = ctx, my_ql = ql, L = ctx + ql;
      const unsigned long long my_bits = bits;
      const float my_cmul = cmul;
      float m_run = -INFINITY, l_run = 0.f;      // the maximum of the row, the sum of this half
      float vref = 0.f;                          // E4M3: power of two above the value scales
      for (int j = dn.t0; j < dn.t1; ++j, ++it) {
        const int kb = 128 * j, c0 = 64 * hf;    // this thread's keys: kb + c0 ..
        const bool tail = kb + 128 > my_ctx;     // drafted keys, or the end of the sequence
        if (!bad && !warp_wait(BAR_S(it & 1), (it >> 1) & 1, ctl, WHERE_PAGED_USE)) bad = true;
        if (FP8 && !bad && !warp_wait(FULLS(sslot), spar, ctl, WHERE_PAGED_USE)) bad = true;
        const float* sc = reinterpret_cast<const float*>(base + C::SC_OFF + 1024 * sslot);
        if (!bad) tc_fence_after();
        float alpha = 1.f;
        bool vscale_odd = false, rescale = false;
        if constexpr (FP8) {
          // largest finite value scale of the tile's keys
          const float4 v4 = reinterpret_cast<const float4*>(sc + 128)[lane];
          const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = kb + 4 * lane + i < L;
            top = fmaxf(top, in && finite_f(vv[i]) ? vv[i] : 0.f);
            vscale_odd = vscale_odd || (in && !finite_f(vv[i]));
          }
          vscale_odd = __any_sync(0xffffffffu, vscale_odd);
          if (__any_sync(0xffffffffu, top > vref)) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float nref = __uint_as_float((__float_as_uint(top) & 0x7f800000u) + (top < 0x1p126f ? 0x00800000u : 0u));
            alpha = vref / nref;
            rescale = true;
            vref = nref;
          }
        }
        // 32 columns of S from column c, times the keys' scales, hidden ones -inf
        auto load_s = [&](int c, uint32_t (&s)[32]) {
          if (!bad) {
            tmem_ld32(tl + 128u * (it & 1) + c, s);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) reg_fence(s[i]);
          if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 k4 = reinterpret_cast<const float4*>(sc + c)[i];
              float y[4];
              f2_unpack(f2_mul(f2_pack(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), f2_pack(k4.x, k4.y)), y[0],
                        y[1]);
              f2_unpack(f2_mul(f2_pack(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), f2_pack(k4.z, k4.w)),
                        y[2], y[3]);
#pragma unroll
              for (int h = 0; h < 4; ++h) s[4 * i + h] = __float_as_uint(y[h]);
            }
          }
          if (tail) {
            // the columns' visibility: the context, then this row's drafts (bits past q_len are clear)
            const int rel = kb + c - my_ctx;
            const uint32_t vis = rel >= 0    ? (rel < 64 ? static_cast<uint32_t>(my_bits >> rel) : 0u)
                                 : rel > -32 ? (static_cast<uint32_t>(my_bits << -rel) | ((1u << -rel) - 1))
                                             : ~0u;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((vis >> i) & 1)) s[i] = __float_as_uint(-INFINITY);
          }
        };
        auto max_of = [&](const uint32_t (&s)[32], float m) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) m = max3(m, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          return m;
        };
        float mt = -INFINITY;
        [[maybe_unused]] uint32_t sr[2][32];
        if constexpr (FP8) {
          // the logits are read from Tensor Memory again below: a tile whose 64 columns are unrolled is
          // 1.2x slower, it misses the instruction cache
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t s[32];
            load_s(c0 + 32 * q, s);
            mt = max_of(s, mt);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q) load_s(c0 + 32 * q, sr[q]);
          mt = max_of(sr[1], max_of(sr[0], mt));
        }
        // the halves' maxima meet; both threads of a row then decide alike
        float* rm = red + 256 * (it & 1);
        rm[128 * hf + r] = mt;
        named_bar_sync(pair_bar, 64u);
        mt = fmaxf(mt, rm[128 * (hf ^ 1) + r]) * my_cmul;
        if (mt > m_run + (FP8 ? TAU_E4M3 : TAU_BF16) || (m_run == -INFINITY && mt != -INFINITY)) {
          const float f = m_run == -INFINITY ? 0.f : ex2(m_run - mt);
          alpha *= f;
          l_run *= f;
          m_run = mt;
          rescale = true;
        }
        const float off = m_run == -INFINITY ? 0.f : m_run;
        const uint32_t pb = tl + C::P_COL + (FP8 ? 0u : 64u * (it & 1));
        // E4M3: numerators times 2^11 / vref, a power of two that goes into the exponent (no scale seen: 1);
        // what would leave fp32's range there (scales below 2^-49 or above 2^71) is multiplied on
        const int want = FP8 && vref > 0.f ? 138 - static_cast<int>(__float_as_uint(vref) >> 23) : 0;
        const int shift = want > 60 ? 60 : (want < -60 ? -60 : want);
        const float extra = __uint_as_float(static_cast<uint32_t>(127 + want - shift) << 23);
        const float off_v = off - (FP8 ? static_cast<float>(shift) : 0.f);
        const uint64_t cm2 = f2_pack(my_cmul, my_cmul), of2 = f2_pack(-off_v, -off_v);
        uint64_t sum = f2_pack(0.f, 0.f);
        if constexpr (!FP8) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float a, b;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[q][2 * i]), __uint_as_float(sr[q][2 * i + 1])), cm2, of2), a, b);
              a = ex2(a);
              b = ex2(b);
              sum = f2_add(sum, f2_pack(a, b));
              pk[i] = pack_bf16x2(a, b);
            }
            if (!bad) tmem_st16(pb + c0 / 2 + 16u * q, pk);
          }
        } else {
          // one P buffer: PV of the tile before must be through with it
          if (!bad && j > dn.t0) {
            if (!warp_wait(BAR_PV, (it - 1) & 1, ctl, WHERE_PAGED_USE)) bad = true;
            else tc_fence_after();
          }
          // FIX: tiles where some numerator may meet a scale that is not finite, or needs `extra`
          auto numerators = [&](auto fix_c) {
            constexpr bool FIX = decltype(fix_c)::value;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
              uint32_t s[32], tt[3][8];
              load_s(c0 + 32 * q, s);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 v4 = reinterpret_cast<const float4*>(sc + 128 + c0 + 32 * q)[i];
                float e[4], y[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  f2_unpack(f2_fma(f2_pack(__uint_as_float(s[4 * i + 2 * h]), __uint_as_float(s[4 * i + 2 * h + 1])), cm2,
                                   of2), e[2 * h], e[2 * h + 1]);
                  e[2 * h] = ex2(e[2 * h]);
                  e[2 * h + 1] = ex2(e[2 * h + 1]);
                  const uint64_t e2 = f2_pack(e[2 * h], e[2 * h + 1]);
                  sum = f2_add(sum, e2);
                  f2_unpack(f2_mul(e2, h == 0 ? f2_pack(v4.x, v4.y) : f2_pack(v4.z, v4.w)), y[2 * h], y[2 * h + 1]);
                }
                if (FIX) {                       // hidden: 0 whatever the scale; seen and not finite: NaN
                  const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                  for (int h = 0; h < 4; ++h)
                    y[h] = e[h] == 0.f ? 0.f : (finite_f(v[h]) ? y[h] * extra : __int_as_float(0x7fffffff));
                }
                uint32_t w[3];
                e5m2_terms4(y[0], y[1], y[2], y[3], w);
#pragma unroll
                for (int h = 0; h < 3; ++h) tt[h][i] = w[h];
              }
              if (!bad) {
#pragma unroll
                for (int h = 0; h < 3; ++h) tmem_st8(pb + 32u * h + c0 / 4 + 8u * q, tt[h]);
              }
            }
          };
          if (tail || vscale_odd || extra != 1.f) numerators(std::true_type{});
          else numerators(std::false_type{});
        }
        {
          float s0, s1;
          f2_unpack(sum, s0, s1);
          l_run += FP8 ? (s0 + s1) * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23) : s0 + s1;
        }
        if (!bad && j > dn.t0 && __any_sync(0xffffffffu, rescale)) {
          // O must hold PV(it - 1) complete; PV(it) waits for both warps' arrivals below.  Each half of the
          // columns is one warp's
          if (!warp_wait(BAR_PV, (it - 1) & 1, ctl, WHERE_PAGED_USE)) {
            bad = true;
          } else {
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < D / 64; ++q) {
              const uint32_t at = tl + C::O_COL + hf * (D / 2) + 32u * q;
              uint32_t o[32];
              tmem_ld32(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                reg_fence(o[i]);
                o[i] = __float_as_uint(__uint_as_float(o[i]) * (rescale ? alpha : 1.f));
              }
              tmem_st32(at, o);
            }
          }
        }
        if (tail) {
          // thread = half of key row r of the value tile: what must not meet a zero numerator is taken out
          if (!bad && !warp_wait(FULLV(it % C::NV), (it / C::NV) & 1, ctl, WHERE_PAGED_USE)) bad = true;
          const int key = kb + r;
          if (!bad && key >= my_ctx) {
            uint8_t* row = base + C::V_OFF + (it % C::NV) * C::TILE_BYTES + r * C::PANEL_ROW;
            bool clear = key >= L;
            if (FP8 && !clear) clear = !finite_f(sc[128 + r]);
            bool odd = false;
            constexpr int NC = C::ROW_BYTES / 32;
#pragma unroll 1
            for (int i = 0; i < NC; ++i) {
              const int c = hf * NC + i;
              uint4* at = reinterpret_cast<uint4*>(row + (c >> 3) * C::PANEL_BYTES + (((c & 7) ^ (r & (NC - 1) & 3)) << 4));
              if (clear) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else if (!FP8) {
                uint4 u = *at;
                uint32_t* w = reinterpret_cast<uint32_t*>(&u);
                bool hit = false;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  if ((w[y] & 0x7f80u) == 0x7f80u) { w[y] &= 0xffff0000u; hit = true; }
                  if ((w[y] & 0x7f800000u) == 0x7f800000u) { w[y] &= 0xffffu; hit = true; }
                }
                if (hit) *at = u;
                odd = odd || hit;
              }
            }
            if (odd) atomicOr(vodd_sh + (seg & 1), 1ull << (key - my_ctx));
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(BAR_P(it & 1));
          if (FP8) mbar_arrive(EMPTYS(sslot));
        }
        if (FP8 && ++sslot == C::NSC) {
          sslot = 0;
          spar ^= 1;
        }
      }
      // ---- end of the segment: the halves' sums, what the value rows held that was not finite, the next
      // segment's queries, then the output ----
      red[512 + 128 * hf + r] = l_run;
      named_bar_sync(1, 256);
      l_run = red[512 + r] + red[512 + 128 + r];
      const unsigned long long vodd = vodd_sh[seg & 1] & my_bits;
      if (threadIdx.x == 0) vodd_sh[(seg & 1) ^ 1] = 0;    // read by all before this barrier; next written after BAR_Q
      more = fetch(rt, x);
      if (!more && rt + p.group_ctas < p.row_tiles) {      // the same keys for the CTA's next row tile
        rt += p.group_ctas;
        x = x0;
        more = fetch(rt, x);
      }
      if (!bad && !warp_wait(BAR_O, seg & 1, ctl, WHERE_PAGED_USE)) bad = true;
      if (!bad) {
        tc_fence_after();
        const int pr = dn_rt * PAGED_TREE_ROWS + r, t = token_of(p, pr);
        const bool valid = t < my_ql;
        const bool whole = dn.t0 == 0 && dn.t1 == dn.n;
        const long long ws_slot = 2ll * (group * static_cast<long long>(p.row_tiles) + dn_rt) + (dn.t0 > 0 ? 0 : 1);
        float inv = l_run == 0.f ? 0.f : 1.f / l_run;
        if (FP8) inv *= vref * (1.f / TOP_E4M3);
        const float lse2 = l_run == 0.f ? -INFINITY : m_run + __log2f(l_run);
        const long long head = static_cast<long long>(dn.hkv) * p.G + pr - t * p.G;
        // a thread holds a row, whose columns lie side by side in memory: 16 columns of the warp's 32 rows at
        // a time go through shared memory, so that a store covers rows in pieces of 32 or 64 bytes
        float* stage = reinterpret_cast<float*>(base + C::STAGE_OFF) + warp * 32 * C::STAGE_ROW;
#pragma unroll 1
        for (int q = hf * (D / 64); q < (hf + 1) * (D / 64); ++q) {
          uint32_t o[32];
          tmem_ld32(tl + C::O_COL + 32u * q, o);
          tmem_wait_ld();
          float f[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            reg_fence(o[i]);
            f[i] = __uint_as_float(o[i]) * inv;
          }
          if (valid && !FP8 && vodd != 0) {
            // infinities and NaN of drafted value rows that this row sees
            for (unsigned long long left = vodd; left != 0; left &= left - 1) {
              const int key = my_ctx + __ffsll(left) - 1;
              if (key < 128 * dn.t0 || key >= 128 * dn.t1) continue;
              const int page = p.page_table[static_cast<long long>(dn.b) * p.max_pages + key / p.page_size];
              if (page < 0 || page >= p.n_pages) continue;
              const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v_cache) + page * p.page_stride +
                                       dn.hkv * p.head_stride + (key % p.page_size) * p.tok_stride + 32 * q;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float e = __bfloat162float(v[i]);
                if (!finite_f(e)) f[i] += e;
              }
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(stage + lane * C::STAGE_ROW + 4 * i) =
                  make_float4(f[16 * y + 4 * i], f[16 * y + 4 * i + 1], f[16 * y + 4 * i + 2], f[16 * y + 4 * i + 3]);
            __syncwarp();
            const int per = whole ? 2 : 4;       // lanes of a row
            for (int k = 0; k < per; ++k) {
              const int row = k * (32 / per) + lane / per, col = (lane % per) * (16 / per);
              const int row_pr = dn_rt * PAGED_TREE_ROWS + 32 * (warp & 3) + row, row_t = token_of(p, row_pr);
              if (row_t >= my_ql) continue;
              const float* src = stage + row * C::STAGE_ROW + col;
              const float4 a = *reinterpret_cast<const float4*>(src);
              if (whole) {
                const float4 e = *reinterpret_cast<const float4*>(src + 4);
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) +
                                     ((static_cast<long long>(dn.b) * p.T + row_t) * p.Hq + dn.hkv * p.G + row_pr - row_t * p.G) * D +
                                     32 * q + 16 * y + col;
                *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w),
                                                            pack_bf16x2(e.x, e.y), pack_bf16x2(e.z, e.w));
              } else {
                *reinterpret_cast<float4*>(p.ws_o + (ws_slot * PAGED_TREE_ROWS + 32 * (warp & 3) + row) * D + 32 * q +
                                           16 * y + col) = a;
              }
            }
          }
          __syncwarp();
        }
        if (hf == 0) {
          if (!whole) p.ws_l[ws_slot * PAGED_TREE_ROWS + r] = lse2;
          else if (valid && p.lse != nullptr) p.lse[(static_cast<long long>(dn.b) * p.Hq + head) * p.T + t] = lse2 * LN2_P;
        }
        tc_fence_before();                       // these reads of O before the next P's arrival
      }
      }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool FP8>
cudaError_t launch_tree_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, cudaStream_t st) {
  using C = TreeCfg<D, FP8>;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((configured.load() & bit) == 0) {
    e = cudaFuncSetAttribute(attn_tree_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return launch_overlapped(attn_tree_kernel<D, FP8>, dim3(p.n_cta * p.group_ctas), TREE_THREADS, C::SMEM_BYTES, st, tk, tv, p);
}

}  // namespace

cudaError_t launch_attn_tree(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int D, bool fp8,
                             cudaStream_t st) {
  if (D == 64) return fp8 ? launch_tree_d<64, true>(tk, tv, p, st) : launch_tree_d<64, false>(tk, tv, p, st);
  return fp8 ? launch_tree_d<128, true>(tk, tv, p, st) : launch_tree_d<128, false>(tk, tv, p, st);
}

}  // namespace ea46
