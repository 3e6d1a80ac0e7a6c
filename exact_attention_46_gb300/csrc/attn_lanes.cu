// attn_lanes.cu -- attention of a few drafted tokens over a paged key/value cache: 9 to 64 query rows
// (heads of a group x drafted tokens) per key/value head over E4M3, 33 to 64 over bf16, for sm_103a.  What it computes, the
// readings and the list of key tiles are attn_paged.cu's and paged.cuh's.
//
// The keys of a tile take the 128 rows of tcgen05's tile and the NR = 16, 32 or 64 query rows its columns:
//     S^T = K Q^T      [128 keys x NR]      K as it lies in the cache, Q row-major
//     O^T += V^T P^T   [D x NR]             V and the numerators with the long side contiguous
// so no product is spent on rows that are not there, a softmax thread holds one key (its scales, its place
// in the tree are one scalar each) and the cache's E4M3 codes go to the tensor core unconverted.
//   * warps 0..7 softmax, in two teams.  A tile's way through the softmax is mostly waiting (for S, the vote, the
//     copies into shared memory to be seen), so with 16 and 32 rows the teams take every other tile, each with maxima,
//     sums and O of its own that the unit's end adds up; with 64 rows, whose arithmetic takes longer than the loads,
//     each has half of the rows.  Thread = key: its numerators go to shared memory as one row of P (three tiles of
//     terms for E4M3), its sums stay in registers.  The maxima of the rows run over threads, and moving them is rare:
//     a team votes once per tile whether any logit passed its row's maximum by 2^TAU, and only then reduces
//     them over the lanes;
//   * warp 8 issues the MMAs, S up to three tiles ahead of PV and across units; 9 to 11 load K, V and scales
//     (load_tiles); 12..15 bring the next unit's queries, a buffer ahead;
//   * O^T's lanes are the columns of an output row, so the epilogue's stores cover rows as they are.
// E4M3: queries are two E4M3 terms (attn_tree.cu has the arithmetic), numerators three E5M2 terms; a thread
// multiplies its numerators by its value's scale over vref, a power of two at or above the scales so far.
// Hidden keys, value rows past the end and drafted values that are not finite: as in attn_tree.cu.
// Every mbarrier wait is bounded.
//
// Measured on 16 sequences of up to 8192 keys, 8 key/value heads, D = 128 (240 MB of E4M3, 35.5 us at the copy rate):
// 16 rows 45.5 us, 32 50.1, 64 79; 64 rows of bf16 (465 MB, 69.3 us) 81.2.  Three sequences of up to 65536 keys, 32
// rows of E4M3 (345 MB, 50.8 us): 62.4.  Up to 32 rows a tile takes 1400 to 1600 cycles, HBM's share of an SM; with 64
// the way of a tile through the softmax, 2600 cycles of which about half are waits, is longer.  The first logits
// come 4 us after the launch may start and a unit's first tile takes 1 to 2 us more, its code being cold.
#include <atomic>
#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>

#include "cache.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ea46 {

namespace {

template <int D, bool FP8, int NR>
struct LanesCfg {
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int ROW_BYTES = D * ESZ;
  static constexpr int PANEL_ROW = ROW_BYTES >= 128 ? 128 : ROW_BYTES;
  static constexpr int NPANEL = ROW_BYTES / PANEL_ROW;
  static constexpr int PANEL_BYTES = 128 * PANEL_ROW;
  static constexpr int TILE_BYTES = 128 * ROW_BYTES;
  static constexpr int NQ = FP8 ? 2 : 1;                       // terms of queries
  static constexpr int NP = FP8 ? 3 : 1;                       // terms of numerators
  // 16 and 32 rows: two teams of four warps take every other tile; 64: each the half of the rows of every tile
  static constexpr int TURNS = NR == 64 ? 1 : 2;
  static constexpr int COLS = NR == 16 ? 16 : 32;              // rows of a softmax thread
  static constexpr int Q_TERM = NR * ROW_BYTES;
  static constexpr int P_ROW = NR * ESZ > 64 ? 128 : 64;       // bytes of a key's row of P, swizzled as wide
  static constexpr int P_TERM = 128 * P_ROW;
  static constexpr int NSC = FP8 ? 6 : 0;                      // stages of 128 key and 128 value scales
  static constexpr uint32_t SBO = 8 * PANEL_ROW, LAYOUT = PANEL_ROW == 128 ? 2u : 4u;
  static constexpr uint32_t P_SBO = 8 * P_ROW, P_LAYOUT = P_ROW == 128 ? 2u : 4u;
  static constexpr int KSTEPS_QK = ROW_BYTES / 32, STEPS_PER_PANEL = PANEL_ROW / 32;
  static constexpr int UMMA_K = FP8 ? 32 : 16, KSTEPS_PV = 128 / UMMA_K;
  static constexpr uint32_t FMT = FP8 ? 0u : 1u;
  static constexpr uint32_t IDESC_QK = instr_desc(FMT, 0, 128, NR);
  // A = V^T with its rows (the columns of V) contiguous: bit 15.  The tile has 128 rows for D = 64 too: the upper
  // half multiplies whatever lies behind the panel in shared memory, and its lanes are never read.
  static constexpr uint32_t IDESC_PV = instr_desc(FMT, 1, 128, NR) | (1u << 15) | (FP8 ? 1u << 10 : 0u);
  static_assert(!FP8 || FMT == 0, "bits 7 and 10: formats of A (E4M3) and B (E5M2)");
  // Tensor Memory: four S buffers, O of either team or of both
  static constexpr uint32_t O_COL = 4 * NR, TMEM_COLS = NR == 64 ? 512 : (NR == 32 ? 256 : 128);
  // shared memory from the end of what the K and V rings leave
  static constexpr int SMALL = 1024 * NSC + (PAGED_MAX_BATCH + 4) * 4 + 8 * COLS * 16 + 8 * NR * 8 + 2 * NR * 12 + 1024;
  static constexpr int ROOM = (227 * 1024 - 1024 - SMALL - 2 * (NP * P_TERM + NQ * Q_TERM)) / TILE_BYTES;
  static constexpr int NK = ROOM >= 16 ? 8 : (ROOM + 1) / 2, NV = ROOM >= 16 ? 8 : ROOM / 2;
  static constexpr int V_OFF = NK * TILE_BYTES;
  static constexpr int P_OFF = V_OFF + NV * TILE_BYTES;         // [2][NP]
  static constexpr int Q_OFF = P_OFF + 2 * NP * P_TERM;         // [2][NQ]
  static constexpr int SC_OFF = Q_OFF + 2 * NQ * Q_TERM;
  static constexpr int VIS_OFF = SC_OFF + NSC * 1024;           // [2][NR] u64: drafted keys a row sees
  static constexpr int ROWAT_OFF = VIS_OFF + 2 * NR * 8;        // [8 warps][NR / 2] i64: where an output row begins
  static constexpr int QMUL_OFF = ROWAT_OFF + 8 * NR * 4;       // [2][NR] floats: softmax scale of a row's codes
  static constexpr int NMAX_OFF = QMUL_OFF + 2 * NR * 4;        // [8 warps][COLS] minus the running maxima
  static constexpr int STEP_OFF = NMAX_OFF + 8 * COLS * 4;      // [8 warps][COLS] what they move by
  static constexpr int FAC_OFF = STEP_OFF + 8 * COLS * 4;       // [8 warps][NR]
  static constexpr int RED_OFF = FAC_OFF + 8 * NR * 4;          // [2][8 warps][COLS]: maxima, sums
  static constexpr int PRE_OFF = RED_OFF + 2 * 8 * COLS * 4;
  static constexpr int FLAG_OFF = PRE_OFF + (PAGED_MAX_BATCH + 4) * 4;   // vodd [4] x 8, vtop [8], vmul [2], tmem, abort, scratch [16]
  static constexpr int BAR_OFF = FLAG_OFF + 32 + 32 + 8 + 8 + 64;
  static constexpr int NBAR = 14 + 2 * (NK + NV + NSC);
  static constexpr int SMEM_BYTES = 1024 + BAR_OFF + NBAR * 8;
  static_assert(VIS_OFF % 16 == 0 && QMUL_OFF % 16 == 0 && NMAX_OFF % 16 == 0 && FLAG_OFF % 8 == 0 && BAR_OFF % 8 == 0, "alignment");
  static_assert(Q_OFF % 1024 == 0 && Q_TERM % 1024 == 0, "swizzle atoms");
  static_assert(2 * NP * P_TERM >= PANEL_BYTES, "the panel behind the last V tile");
  static_assert(NV >= 2 && SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

constexpr int LANES_THREADS = 512;
constexpr int MMA_WARP = 8, K_WARP = 9, S_WARP = 11, Q_WARP = 12;
constexpr float TAU_BF16 = 8.0f;        // lazy rescale threshold (log2): numerators reach 2^TAU

// Registers of a warpgroup for 32 and 64 rows, out of the block's: 512 threads x 128 = 256 x 176 + 256 x 80 =
// 256 x 184 + 256 x 72, what neither side spills in.
template <int NR>
__device__ __forceinline__ void softmax_registers() {
  if constexpr (NR == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
  if constexpr (NR == 32) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
}
template <int NR>
__device__ __forceinline__ void other_registers() {
  if constexpr (NR == 64) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  if constexpr (NR == 32) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
}

// N columns of this warp's 32 lanes of Tensor Memory.
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(at));
}
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(at));
}
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[32]) { tmem_ld32(at, r); }

// Whether any thread of named barrier `id`'s n threads brings `mine`; a barrier among them.
__device__ __forceinline__ bool named_bar_any(uint32_t id, uint32_t n, bool mine) {
  uint32_t any;
  asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %3, 0;\n\tbarrier.cta.red.or.pred b, %1, %2, a;\n\t"
               "selp.u32 %0, 1, 0, b;\n\t}" : "=r"(any) : "r"(id), "r"(n), "r"(mine ? 1u : 0u) : "memory");
  return any != 0;
}

// Over the warp's lanes, of column lane % N: N - 1 exchanges for the first log2 N steps of all columns at once
// (32 warp-wide reductions instead of the maxima of 32 columns took 3.5 us on a unit's first tile).
template <bool MAX, int N>
__device__ __forceinline__ float column_reduce(float (&v)[N]) {
  const uint32_t lane = lane_id();
  auto both = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = (lane & o) != 0;
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + o], o);
      v[i] = both(up ? v[i + o] : v[i], other);
    }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] = both(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

template <int D, bool FP8, int NR>
__global__ void __launch_bounds__(LANES_THREADS, 1)
    attn_lanes_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedParams p) {
  using C = LanesCfg<D, FP8, NR>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  const uint32_t sK = base_u32, sV = base_u32 + C::V_OFF, sP = base_u32 + C::P_OFF, sQ = base_u32 + C::Q_OFF;
  unsigned long long* vis_sh = reinterpret_cast<unsigned long long*>(base + C::VIS_OFF);
  float* qmul_sh = reinterpret_cast<float*>(base + C::QMUL_OFF);
  float* red = reinterpret_cast<float*>(base + C::RED_OFF);
  int* pre = reinterpret_cast<int*>(base + C::PRE_OFF);
  unsigned long long* vodd_sh = reinterpret_cast<unsigned long long*>(base + C::FLAG_OFF);   // [4]
  uint32_t* vtop_sh = reinterpret_cast<uint32_t*>(base + C::FLAG_OFF + 32);                  // [8 warps]
  float* vmul_sh = reinterpret_cast<float*>(base + C::FLAG_OFF + 64);                        // [2 groups]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::FLAG_OFF + 72);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::FLAG_OFF + 76);
  int* scratch = reinterpret_cast<int*>(base + C::FLAG_OFF + 80);                            // [16]
  const uint32_t bar0 = base_u32 + C::BAR_OFF;
  const uint32_t BAR_O = bar0, BAR_DONE = bar0 + 8;
  auto BAR_PV = [&](int g) { return bar0 + 16 + 8u * g; };
  auto BAR_P = [&](int g) { return bar0 + 32 + 8u * g; };
  auto FULLQ = [&](int b) { return bar0 + 48 + 8u * b; };
  auto EMPTYQ = [&](int b) { return bar0 + 64 + 8u * b; };
  auto BAR_S = [&](int b) { return bar0 + 80 + 8u * b; };                                    // [4]
  auto FULLK = [&](int s) { return bar0 + 112 + 8u * s; };
  auto EMPTYK = [&](int s) { return bar0 + 112 + 8u * (C::NK + s); };
  auto FULLV = [&](int s) { return bar0 + 112 + 8u * (2 * C::NK + s); };
  auto EMPTYV = [&](int s) { return bar0 + 112 + 8u * (2 * C::NK + C::NV + s); };
  auto FULLS = [&](int s) { return bar0 + 112 + 8u * (2 * (C::NK + C::NV) + s); };
  auto EMPTYS = [&](int s) { return bar0 + 112 + 8u * (2 * (C::NK + C::NV) + C::NSC + s); };

  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  if (threadIdx.x == 0) {
    mbar_init(BAR_O, 1);
    mbar_init(BAR_DONE, 1);
    for (int b = 0; b < 4; ++b) mbar_init(BAR_S(b), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(BAR_PV(b), 1);
      mbar_init(BAR_P(b), C::TURNS == 2 ? 4 : 8);
      mbar_init(FULLQ(b), 4);
      mbar_init(EMPTYQ(b), 1 + 8);
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
      mbar_init(EMPTYS(s), C::TURNS == 2 ? 4 : 8);
    }
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) vodd_sh[i] = 0;
    fence_barrier_init();
  }
  grid_launch_dependents();
  grid_dependency_wait();       // everything below reads what earlier kernels may have written
  const bool fine = tile_prefix(p, pre, scratch, LANES_THREADS);
  if (!fine) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && atomicCAS(p.err_word, 0, 1) == 0) atomicExch(p.err_info, WHERE_PAGED_LENS);
    if (threadIdx.x == 0) write_cut(p, pre, blockIdx.x, 0, 0);
    return;
  }
  const long long W = static_cast<long long>(pre[p.B]) * p.Hkv;
  const long long N = W < p.n_cta ? W : p.n_cta;
  const int group = blockIdx.x;
  if (group >= N) {
    if (threadIdx.x == 0) write_cut(p, pre, group, W, N);
    return;
  }
  const long long x0 = cta_start(group, W, N), x1 = cta_start(group + 1ll, W, N);
  if (warp == MMA_WARP) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{p.spin_limit, abort_flag, p.err_word, p.err_info};
  const TileRings rings{sK, sV, base_u32 + C::SC_OFF, FULLK(0), EMPTYK(0), FULLV(0), EMPTYV(0), FULLS(0), EMPTYS(0)};

  if (warp >= MMA_WARP) other_registers<NR>();
  else softmax_registers<NR>();

  if (warp >= Q_WARP) {
    // ---- queries: a warp every fourth row, lane = D / 32 elements ----
    constexpr int E = D / 32, ROWS = NR / 4, BATCH = ROWS < 8 ? ROWS : 8;
    const int w = warp - Q_WARP;
    Segment s;
    long long x = x0;
    for (int seg = 0; next_segment(p, pre, x, x1, s); ++seg) {
      const int buf = seg & 1;
      if (!warp_wait(EMPTYQ(buf), ((seg >> 1) & 1) ^ 1, ctl, WHERE_PAGED_LOAD)) break;
      const int ql = p.q_lens != nullptr ? *(p.q_lens + s.b) : p.T;
      // the drafted keys that row mr sees (the load is under way with the queries')
      const int mr = 32 * w + lane;
      const bool masks = mr < NR;
      unsigned long long bits = 0;
      if (masks) {
        const int t = token_of(p, mr);
        if (t < p.T)
          bits = p.tree_mask != nullptr ? *(p.tree_mask + static_cast<long long>(s.b) * p.T + t)
                                        : (t >= 63 ? ~0ull : (2ull << t) - 1);
      }
#pragma unroll 1
      for (int i0 = 0; i0 < ROWS; i0 += BATCH) {
        uint32_t u[BATCH][E / 2];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int r = 4 * (i0 + i) + w, t = token_of(p, r);
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
              ((static_cast<long long>(s.b) * p.T + t) * p.Hq + s.hkv * p.G + r - t * p.G) * D + E * lane;
#pragma unroll
          for (int k = 0; k < E / 2; ++k) u[i][k] = 0;
          if (t < p.T) {
            if constexpr (E == 4) {
              const uint2 y = *reinterpret_cast<const uint2*>(src);
              u[i][0] = y.x;
              u[i][E / 2 - 1] = y.y;
            } else {
              u[i][0] = *reinterpret_cast<const uint32_t*>(src);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int r = 4 * (i0 + i) + w;
          const int at = E * C::ESZ * lane, pb = at % C::PANEL_ROW;      // this lane's bytes of the row
          const int swz = C::PANEL_ROW == 128 ? (r & 7) : ((r >> 1) & 3);
          const uint32_t dst = sQ + buf * C::NQ * C::Q_TERM + (at / C::PANEL_ROW) * (NR * C::PANEL_ROW) + r * C::PANEL_ROW +
                               (((pb >> 4) ^ swz) << 4) + (pb & 15);
          if constexpr (!FP8) {
            if constexpr (E == 4)
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(u[i][0]), "r"(u[i][E / 2 - 1]) : "memory");
            else
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(u[i][0]) : "memory");
          } else {
            // the row's largest element and the power of two that brings it into [128, 256): exact
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < E / 2; ++k) m = max(m, max(u[i][k] & 0x7fffu, (u[i][k] >> 16) & 0x7fffu));
            m = __reduce_max_sync(0xffffffffu, m);
            int ex = static_cast<int>(m >> 7) - 127;
            ex = ex < -100 ? -100 : (ex > 100 ? 100 : ex);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - ex) << 23);
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              f[k] = k < E ? __uint_as_float((k & 1) ? u[i][(k / 2) % (E / 2)] & 0xffff0000u : u[i][(k / 2) % (E / 2)] << 16) * up : 0.f;
            uint32_t hi, lo;
            e4m3_terms4(f[0], f[1], f[2], f[3], hi, lo);
            if constexpr (E == 4) {
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(hi) : "memory");
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + C::Q_TERM), "r"(lo) : "memory");
            } else {
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(static_cast<uint16_t>(hi)) : "memory");
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + C::Q_TERM), "h"(static_cast<uint16_t>(lo)) : "memory");
            }
            // an infinite query element, which E4M3 cannot hold, makes its row's logits NaN
            if (lane == 0)
              qmul_sh[buf * NR + r] = m >= 0x7f80u ? __int_as_float(0x7fffffff)
                                                   : p.c_log2 * __uint_as_float(static_cast<uint32_t>(127 - 7 + ex) << 23);
          }
        }
      }
      if (masks) {
        if (ql < 64) bits &= (1ull << ql) - 1;
        vis_sh[buf * NR + mr] = bits;
        if (!FP8) qmul_sh[buf * NR + mr] = p.c_log2;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(FULLQ(buf));
    }
  } else if (warp >= K_WARP) {
    if (FP8 || warp < S_WARP) load_tiles<C>(p, pre, tmK, tmV, rings, warp - K_WARP, 0, x0, x1, ctl);
    if (warp == K_WARP && lane == 0) write_cut(p, pre, group, W, N);
  } else if (warp == MMA_WARP) {
    // ---- MMA issue ----
    if (elect_one()) {
      const uint64_t dk0 = smem_desc(sK, 16, C::SBO, C::LAYOUT);
      const uint64_t dv0 = smem_desc(sV, C::PANEL_BYTES, C::SBO, C::LAYOUT);
      const uint64_t dq0 = smem_desc(sQ, 16, C::SBO, C::LAYOUT);
      const uint64_t dp0 = smem_desc(sP, C::P_TERM, C::P_SBO, C::P_LAYOUT);
      const uint32_t hk = static_cast<uint32_t>(dk0 >> 32), hq = static_cast<uint32_t>(dq0 >> 32);
      const uint32_t hv = static_cast<uint32_t>(dv0 >> 32), hp = static_cast<uint32_t>(dp0 >> 32);
      // S of up to three tiles ahead of PV, whichever can go: S(i) overwrites S(i - 4), which the softmax read
      // before it handed over P(i - 4)
      Segment s;
      long long x = x0;
      bool more = next_segment(p, pre, x, x1, s);
      int tile = 0, seg = 0;                     // next tile of S: its place in segment `seg`
      int qi = 0, pi = 0;                        // tiles of S and PV issued
      int ks = 0, vs = 0;                        // ring positions
      uint32_t kpar = 0, vpar = 0, fresh = 0, last = 0;        // bit i & 3: first tile of its O, last of its segment
      long long t0 = clock64();
      while (more || pi < qi) {
        bool moved = false;
        if (pi < qi && mbar_test(BAR_P(pi & 1), (pi >> 1) & 1) && mbar_test(FULLV(vs), vpar)) {
          tc_fence_after();
          const uint32_t av = static_cast<uint32_t>(dv0) + ((vs * C::TILE_BYTES) >> 4);
          const uint32_t bp = static_cast<uint32_t>(dp0) + (((pi & 1) * C::NP * C::P_TERM) >> 4);
          const uint32_t d = tmem + C::O_COL + (C::TURNS == 2 ? NR * (pi & 1) : 0);
          const uint32_t acc0 = ((fresh >> (pi & 3)) & 1) ^ 1;
#pragma unroll
          for (int term = 0; term < C::NP; ++term)
#pragma unroll
            for (int kk = 0; kk < C::KSTEPS_PV; ++kk)
              mma_ss<FP8>(d, av + ((kk * C::UMMA_K * C::PANEL_ROW) >> 4), hv,
                          bp + ((term * C::P_TERM + kk * C::UMMA_K * C::P_ROW) >> 4), hp, C::IDESC_PV,
                          kk > 0 || term > 0 ? 1u : acc0);
          mma_commit(BAR_PV(pi & 1));
          mma_commit(EMPTYV(vs));
          if ((last >> (pi & 3)) & 1) mma_commit(BAR_O);
          if (++vs == C::NV) {
            vs = 0;
            vpar ^= 1;
          }
          ++pi;
          moved = true;
        }
        if (more && qi - pi < 4 && (tile > 0 || mbar_test(FULLQ(seg & 1), (seg >> 1) & 1)) && mbar_test(FULLK(ks), kpar)) {
          tc_fence_after();
          const uint32_t ak = static_cast<uint32_t>(dk0) + ((ks * C::TILE_BYTES) >> 4);
          const uint32_t bq = static_cast<uint32_t>(dq0) + (((seg & 1) * C::NQ * C::Q_TERM) >> 4);
          const uint32_t d = tmem + NR * (qi & 3);
#pragma unroll
          for (int term = 0; term < C::NQ; ++term)
#pragma unroll
            for (int kk = 0; kk < C::KSTEPS_QK; ++kk) {
              const uint32_t in = (kk % C::STEPS_PER_PANEL) * 32, pn = kk / C::STEPS_PER_PANEL;
              mma_ss<FP8>(d, ak + ((pn * C::PANEL_BYTES + in) >> 4), hk,
                          bq + ((term * C::Q_TERM + pn * (NR * C::PANEL_ROW) + in) >> 4), hq, C::IDESC_QK,
                          (kk > 0 || term > 0) ? 1u : 0u);
            }
          mma_commit(BAR_S(qi & 3));
          mma_commit(EMPTYK(ks));
          const uint32_t bit = 1u << (qi & 3);
          fresh = tile < C::TURNS ? fresh | bit : fresh & ~bit;
          last &= ~bit;
          if (++tile == s.t1 - s.t0) {
            last |= bit;
            mma_commit(EMPTYQ(seg & 1));
            more = next_segment(p, pre, x, x1, s);
            tile = 0;
            ++seg;
          }
          if (++ks == C::NK) {
            ks = 0;
            kpar ^= 1;
          }
          ++qi;
          moved = true;
        }
        if (moved) {
          t0 = clock64();
        } else {
          if (*abort_flag) break;
          if (clock64() - t0 > p.spin_limit) {
            *abort_flag = 1;
            if (atomicCAS(p.err_word, 0, 4 /* ATTN_ERR_TIMEOUT */) == 0) atomicExch(p.err_info, WHERE_PAGED_MMA);
            break;
          }
        }
      }
      mma_commit(BAR_DONE);
      wait_drain_paged(BAR_DONE, 0, p.spin_limit);
    }
  } else {
    // ---- softmax: a team of four warps has maxima and sums of its own; thread = key r, COLS rows from cb ----
    constexpr int COLS = C::COLS, TURNS = C::TURNS;
    constexpr float TAU = FP8 ? TAU_E4M3 : TAU_BF16;
    const int quarter = warp & 3, team = warp >> 2, r = 32 * quarter + lane, cb = TURNS == 1 ? COLS * team : 0;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter) << 21);       // this warp's 32 lanes
    const uint32_t o_at = tl + C::O_COL + (TURNS == 2 ? NR * team : cb), team_bar = 2u + team;
    const bool holds_o = 32 * quarter < D;                                    // lanes of O^T (D = 64: the lower half)
    float* nmax0 = reinterpret_cast<float*>(base + C::NMAX_OFF);
    float* nmax = nmax0 + warp * COLS;                                        // minus the rows' maxima
    float* step = reinterpret_cast<float*>(base + C::STEP_OFF) + warp * COLS;
    float* fac = reinterpret_cast<float*>(base + C::FAC_OFF) + warp * NR;
    long long* row_at = reinterpret_cast<long long*>(base + C::ROWAT_OFF) + warp * (NR / 2);
    float* red_max = red + 4 * team * COLS;
    float* red_sum = red + 8 * COLS;
    const int swz = C::P_ROW == 128 ? (r & 7) : ((r >> 1) & 3);
    bool bad = false;                              // a wait of this warp gave up; it still meets the barriers
    Segment s;
    long long x = x0;
    int it = 0;                                    // tiles before the segment
    int sslot = TURNS == 2 ? team : 0;
    uint32_t spar = 0;
    for (int seg = 0; next_segment(p, pre, x, x1, s); ++seg) {
      const int buf = seg & 1;
      const int ctx = *(p.ctx_lens + s.b), ql = p.q_lens != nullptr ? *(p.q_lens + s.b) : p.T, L = ctx + ql;
      const float* qmul = qmul_sh + buf * NR + cb;
      const unsigned long long* vis = vis_sh + buf * NR;
      if (lane < COLS) nmax[lane] = 0.f;
      __syncwarp();
      if (!bad && !warp_wait(FULLQ(buf), (seg >> 1) & 1, ctl, WHERE_PAGED_USE)) bad = true;
      uint64_t l[COLS / 2];                        // this thread's keys' part of the rows' sums, in pairs
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) l[i] = 0;
      float vref = 0.f, rv = 0.f;                  // E4M3: power of two at or above the value scales, its reciprocal
      const int first = s.t0 + (TURNS == 2 ? (team ^ it) & 1 : 0);
      for (int j = first; j < s.t1; j += TURNS) {
        const int at = it + j - s.t0;              // place among the CTA's tiles
        const int key = 128 * j + r;
        const bool tail = 128 * j + 128 > ctx;     // drafted keys, or the end of the sequence
        float ks = 1.f, vsc = 0.f;
        bool odd = false;                          // this key's value scale is not finite
        const bool ready = mbar_test(BAR_S(at & 3), (at >> 2) & 1) && (!FP8 || mbar_test(FULLS(sslot), spar));
        if (!__all_sync(0xffffffffu, ready) && !bad) {
          if (!warp_wait(BAR_S(at & 3), (at >> 2) & 1, ctl, WHERE_PAGED_USE)) bad = true;
          if (FP8 && !bad && !warp_wait(FULLS(sslot), spar, ctl, WHERE_PAGED_USE)) bad = true;
        }
        if constexpr (FP8) {
          const float* sc = reinterpret_cast<const float*>(base + C::SC_OFF + 1024 * sslot);
          ks = sc[r];
          vsc = key < L ? sc[128 + r] : 0.f;
          odd = !finite_f(vsc);
        }
        // logits in log2 units less the maxima so far; hidden ones -inf
        float y[COLS];
        float top = -INFINITY;
        {
          uint32_t u[COLS];
          if (!bad) {
            tc_fence_after();
            tmem_ld(tl + NR * (at & 3) + cb, u);
            tmem_wait_ld();
          }
#pragma unroll
          for (int k = 0; k < COLS; ++k) reg_fence(u[k]);
          const uint64_t ks2 = f2_pack(ks, ks);
#pragma unroll
          for (int k = 0; k < COLS; k += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(qmul + k);
            const float4 a4 = *reinterpret_cast<const float4*>(nmax + k);
            uint64_t lo = f2_pack(__uint_as_float(u[k]), __uint_as_float(u[k + 1]));
            uint64_t hi = f2_pack(__uint_as_float(u[k + 2]), __uint_as_float(u[k + 3]));
            if constexpr (FP8) {
              lo = f2_mul(lo, ks2);
              hi = f2_mul(hi, ks2);
            }
            f2_unpack(f2_fma(lo, f2_pack(c4.x, c4.y), f2_pack(a4.x, a4.y)), y[k], y[k + 1]);
            f2_unpack(f2_fma(hi, f2_pack(c4.z, c4.w), f2_pack(a4.z, a4.w)), y[k + 2], y[k + 3]);
          }
          if (tail) {
            const int rel = key - ctx;
#pragma unroll
            for (int k = 0; k < COLS; ++k)
              if (rel >= 0 && (rel >= 64 || !((vis[cb + k] >> rel) & 1))) y[k] = -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < COLS; k += 2) top = max3(top, y[k], y[k + 1]);
        }
        // a unit's first tile sets the maxima
        const bool any = named_bar_any(team_bar, 128, j == first || top > TAU || (FP8 && !odd && vsc > vref));
        // P's buffer (and, in turns, O) are free with PV of the tile two before
        if (at >= 2 && !bad) {
          if (!__all_sync(0xffffffffu, mbar_test(BAR_PV(at & 1), ((at >> 1) - 1) & 1)) &&
              !warp_wait(BAR_PV(at & 1), ((at >> 1) - 1) & 1, ctl, WHERE_PAGED_USE)) bad = true;
          else tc_fence_after();
        }
        if (any) {
          // some row's maximum moves (or the scales' bound): the rows' maxima over the tile's keys
#pragma unroll
          for (int i = 0; i < COLS; i += 16) {
            float z[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] = y[i + k];
            const float m = column_reduce<true>(z);            // (a NaN counts for nothing)
            if (lane < 16) red_max[quarter * COLS + i + lane] = m;
          }
          if constexpr (FP8) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, odd ? 0u : __float_as_uint(vsc));
            if (lane == 0) vtop_sh[warp] = m;
          }
          named_bar_sync(team_bar, 128);
          float vfac = 1.f;
          if constexpr (FP8) {
            float vt = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) vt = fmaxf(vt, __uint_as_float(vtop_sh[4 * team + w]));
            if (vt > vref) {
              const float nref = __uint_as_float((__float_as_uint(vt) & 0x7f800000u) + (vt < 0x1p126f ? 0x00800000u : 0u));
              vfac = vref / nref;
              vref = nref;
              rv = 1.f / nref;
            }
          }
          if (lane < COLS) {
            float m = red_max[lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) m = fmaxf(m, red_max[w * COLS + lane]);
            // The first tile's maxima replace the zeros that stand for none; later ones only rise.  A row that
            // sees nothing of its team's first tile keeps 0: such a tile begins with drafted keys, of which there are
            // at most 64, so the row has no other tile.
            const float up = m == -INFINITY ? 0.f : (j == first ? m : fmaxf(m, 0.f));
            nmax[lane] -= up;
            step[lane] = -up;
            fac[lane] = ex2(-up);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < COLS; i += 4) {
            const float4 d4 = *reinterpret_cast<const float4*>(step + i);
            f2_unpack(f2_add(f2_pack(y[i], y[i + 1]), f2_pack(d4.x, d4.y)), y[i], y[i + 1]);
            f2_unpack(f2_add(f2_pack(y[i + 2], y[i + 3]), f2_pack(d4.z, d4.w)), y[i + 2], y[i + 3]);
          }
          if (j > first) {
#pragma unroll
            for (int i = 0; i < COLS; i += 4) {
              const float4 f4 = *reinterpret_cast<const float4*>(fac + i);
              l[i / 2] = f2_mul(l[i / 2], f2_pack(f4.x, f4.y));
              l[i / 2 + 1] = f2_mul(l[i / 2 + 1], f2_pack(f4.z, f4.w));
            }
            // O must hold PV of this O's last tile; PV of this one waits for the team's arrival below.  (In the state
            // of its barrier nothing older can stand for that: PV two tiles before is complete.)
            if (TURNS == 1 && !bad) {
              if (!warp_wait(BAR_PV((at - 1) & 1), ((at - 1) >> 1) & 1, ctl, WHERE_PAGED_USE)) bad = true;
              else tc_fence_after();
            }
            if (!bad && holds_o) {
#pragma unroll 1
              for (int i = 0; i < COLS; i += 8) {
                uint32_t o[8];
                tmem_ld(o_at + i, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  reg_fence(o[k]);
                  o[k] = __float_as_uint(__uint_as_float(o[k]) * fac[i + k] * vfac);
                }
                tmem_st8(o_at + i, o);
              }
              tmem_wait_st();
            }
          }
        }
        // numerators
        const uint32_t prow = sP + (at & 1) * C::NP * C::P_TERM + r * C::P_ROW;
        if constexpr (!FP8) {
#pragma unroll
          for (int i = 0; i < COLS; i += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              const float a = ex2(y[i + k]), b = ex2(y[i + k + 1]);
              l[(i + k) / 2] = f2_add(l[(i + k) / 2], f2_pack(a, b));
              pk[k / 2] = pack_bf16x2(a, b);
            }
            st_shared_v4(prow + ((((cb + i) >> 3) ^ swz) << 4), pk[0], pk[1], pk[2], pk[3]);
          }
        } else {
          const float w = odd ? __int_as_float(0x7fffffff) : vsc * rv * TOP_E4M3;
          const bool fix = __any_sync(0xffffffffu, odd);       // hidden: 0 whatever the scale; seen and not finite: NaN
#pragma unroll
          for (int i = 0; i < COLS; i += 16) {
            uint32_t tt[4][3];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              float e[4], f[4];
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                e[k] = ex2(y[i + 4 * h + k]);
                e[k + 1] = ex2(y[i + 4 * h + k + 1]);
                const uint64_t e2 = f2_pack(e[k], e[k + 1]);
                uint64_t& lc = l[(i + 4 * h + k) / 2];
                lc = f2_add(lc, e2);
                f2_unpack(f2_mul(e2, f2_pack(w, w)), f[k], f[k + 1]);
              }
              if (fix) {
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = e[k] == 0.f ? 0.f : f[k];
              }
              e5m2_terms4(f[0], f[1], f[2], f[3], tt[h]);
            }
            const uint32_t dst = prow + ((((cb + i) >> 4) ^ swz) << 4);
#pragma unroll
            for (int k = 0; k < 3; ++k) st_shared_v4(dst + k * C::P_TERM, tt[0][k], tt[1][k], tt[2][k], tt[3][k]);
          }
        }
        if (tail) {
          // thread = key row r of the value tile (in turns; else a team half the row): what must not meet a zero
          // numerator is taken out.  (PV two tiles before is complete, so the slot's phase before this one is too.)
          if (!bad && !warp_wait(FULLV(at % C::NV), (at / C::NV) & 1, ctl, WHERE_PAGED_USE)) bad = true;
          if (!bad && key >= ctx) {
            uint8_t* row = base + C::V_OFF + (at % C::NV) * C::TILE_BYTES + r * C::PANEL_ROW;
            const bool clear = key >= L || odd;
            bool hits = false;
            constexpr int PC = C::PANEL_ROW / 16, NC = C::ROW_BYTES / 16;
            const int vswz = C::PANEL_ROW == 128 ? (r & 7) : ((r >> 1) & 3);
#pragma unroll 1
            for (int i = TURNS == 1 ? team * (NC / 2) : 0; i < (TURNS == 1 ? (team + 1) * (NC / 2) : NC); ++i) {
              uint4* v = reinterpret_cast<uint4*>(row + (i / PC) * C::PANEL_BYTES + (((i % PC) ^ vswz) << 4));
              if (clear) {
                *v = make_uint4(0u, 0u, 0u, 0u);
              } else if (!FP8) {
                uint4 u = *v;
                uint32_t* q = reinterpret_cast<uint32_t*>(&u);
                bool hit = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((q[k] & 0x7f80u) == 0x7f80u) { q[k] &= 0xffff0000u; hit = true; }
                  if ((q[k] & 0x7f800000u) == 0x7f800000u) { q[k] &= 0xffffu; hit = true; }
                }
                if (hit) *v = u;
                hits = hits || hit;
              }
            }
            if (hits) atomicOr(vodd_sh + (seg & 3), 1ull << (key - ctx));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(BAR_P(at & 1));
          if (FP8) mbar_arrive(EMPTYS(sslot));
        }
        if constexpr (FP8) {
          sslot += TURNS;
          if (sslot >= C::NSC) {
            sslot -= C::NSC;
            spar ^= 1;
          }
        }
      }
      // ---- end of the segment: the sums over the lanes and the teams, then the output; a team's warps take
      // columns c0 .. c0 + NR / 2 of O, or of both teams' O ----
#pragma unroll
      for (int c = 0; c < COLS; c += 16) {
        float part[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) f2_unpack(l[(c + i) / 2], part[i], part[i + 1]);
        const float sum = column_reduce<false>(part);
        if (lane < 16) red_sum[warp * COLS + c + lane] = sum;
      }
      if (FP8 && lane == 0 && quarter == 0) vmul_sh[team] = vref * (1.f / TOP_E4M3);
      const int n = s.t1 - s.t0;
      // teams with tiles in the segment; one without left nothing of it in its O
      const bool has0 = TURNS == 1 || n > 1 || (it & 1) == 0, has1 = TURNS == 2 && (n > 1 || (it & 1) == 1);
      it += n;
      named_bar_sync(1, 256);
      const unsigned long long vodd = vodd_sh[seg & 3];
      // last read two segments ago, next written after the next segment's barrier
      if (threadIdx.x == 0) vodd_sh[(seg + 2) & 3] = 0;
      const bool whole = s.t0 == 0 && s.t1 == s.n;
      const long long ws_row = (2ll * group + (s.t0 > 0 ? 0 : 1)) * NR;
      constexpr int HALF = NR / 2;
      const int c0 = HALF * team;
      if (lane < HALF) {
        const int pr = c0 + lane, t = token_of(p, pr);
        float sums[2] = {0.f, 0.f}, m, f[2] = {1.f, 1.f};
        if constexpr (TURNS == 2) {
#pragma unroll
          for (int k = 0; k < 8; ++k) sums[k >> 2] += red_sum[k * COLS + pr];
          const float m0 = sums[0] == 0.f ? -FLT_MAX : -nmax0[pr], m1 = sums[1] == 0.f ? -FLT_MAX : -nmax0[4 * COLS + pr];
          m = fmaxf(m0, m1);
          f[0] = ex2(m0 - m);
          f[1] = ex2(m1 - m);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) sums[0] += red_sum[(4 * team + k) * COLS + lane];
          m = -nmax[lane];
        }
        const float sum = sums[0] * f[0] + sums[1] * f[1], inv = sum == 0.f ? 0.f : 1.f / sum;
        fac[lane] = f[0] * inv;
        fac[HALF + lane] = f[1] * inv;
        const long long head = static_cast<long long>(s.hkv) * p.G + pr - t * p.G;
        row_at[lane] = t >= ql ? -1 : (whole ? ((static_cast<long long>(s.b) * p.T + t) * p.Hq + head) * D : (ws_row + pr) * D);
        if (quarter == 0) {
          const float lse2 = sum == 0.f ? -INFINITY : __log2f(sum) + m;
          if (!whole) p.ws_l[ws_row + pr] = lse2;
          else if (t < ql && p.lse != nullptr) p.lse[(static_cast<long long>(s.b) * p.Hq + head) * p.T + t] = lse2 * LN2_P;
        }
      }
      __syncwarp();
      if (!bad && !warp_wait(BAR_O, seg & 1, ctl, WHERE_PAGED_USE)) bad = true;
      if (!bad && holds_o) {
        tc_fence_after();
        const float v0 = FP8 ? vmul_sh[TURNS == 2 ? 0 : team] : 1.f, v1 = FP8 ? vmul_sh[1] : 1.f;
#pragma unroll 1
        for (int i = 0; i < HALF; i += 8) {
          uint32_t a[8], b[8];
          tmem_ld(tl + C::O_COL + c0 + i, a);
          if (TURNS == 2) tmem_ld(tl + C::O_COL + NR + c0 + i, b);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            reg_fence(a[k]);
            if (TURNS == 2) reg_fence(b[k]);
            float f = has0 ? __uint_as_float(a[k]) * fac[i + k] * v0 : 0.f;
            if (TURNS == 2 && has1) f += __uint_as_float(b[k]) * fac[HALF + i + k] * v1;
            const long long to = row_at[i + k];
            if (to < 0) continue;
            if (!FP8 && vodd != 0) {
              // infinities and NaN of drafted value rows that this row sees
              for (unsigned long long left = vodd & vis[c0 + i + k]; left != 0; left &= left - 1) {
                const int at_key = ctx + __ffsll(left) - 1;
                if (at_key < 128 * s.t0 || at_key >= 128 * s.t1) continue;
                const int page = p.page_table[static_cast<long long>(s.b) * p.max_pages + at_key / p.page_size];
                if (page < 0 || page >= p.n_pages) continue;
                const float e = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[page * p.page_stride +
                    s.hkv * p.head_stride + (at_key % p.page_size) * p.tok_stride + r]);
                if (!finite_f(e)) f += e;
              }
            }
            if (whole) static_cast<__nv_bfloat16*>(p.o)[to + r] = __float2bfloat16(f);
            else p.ws_o[to + r] = f;
          }
        }
      }
      tc_fence_before();                         // all reads of O before the next P's arrival
      named_bar_sync(1, 256);
      if (lane == 0) mbar_arrive(EMPTYQ(buf));
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool FP8, int NR>
cudaError_t launch_lanes_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, cudaStream_t st) {
  using C = LanesCfg<D, FP8, NR>;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if ((configured.load() & bit) == 0) {
    e = cudaFuncSetAttribute(attn_lanes_kernel<D, FP8, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return launch_overlapped(attn_lanes_kernel<D, FP8, NR>, dim3(p.n_cta), LANES_THREADS, C::SMEM_BYTES, st, tk, tv, p);
}

template <int D>
cudaError_t launch_lanes_n(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, bool fp8, cudaStream_t st) {
  const int rb = paged_rows(p.G * p.T);
  if (!fp8) return launch_lanes_d<D, false, 64>(tk, tv, p, st);
  return rb == 16   ? launch_lanes_d<D, true, 16>(tk, tv, p, st)
         : rb == 32 ? launch_lanes_d<D, true, 32>(tk, tv, p, st)
                    : launch_lanes_d<D, true, 64>(tk, tv, p, st);
}

}  // namespace

cudaError_t launch_attn_lanes(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int D, bool fp8, cudaStream_t st) {
  return D == 64 ? launch_lanes_n<64>(tk, tv, p, fp8, st) : launch_lanes_n<128>(tk, tv, p, fp8, st);
}

}  // namespace ea46
