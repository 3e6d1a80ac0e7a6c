// kv_cache.cu -- rotary positions on their own, and the writes and read-back of a paged key/value
// cache, for sm_103a.  The pages name rotary embedding as the bandwidth-bound op beside the
// quantiser (hada.io FA3 summary, "Niedrige FP8-Präzision und incoherent processing") and LLM
// inference as future work; the formulas are RoFormer's (Su et al. 2021, section 3.2).
//
// Rotation of a row x at position p, first `rot` elements, c_i = cos(p theta_i), s_i = sin(p theta_i)
// from a table evaluated in fp64:
//     y_a = x_a c_i - x_b s_i,  y_b = x_a s_i + x_b c_i,
// (a, b) = (2i, 2i + 1) interleaved or (i, i + rot / 2) half; the gradient is the transposed turn
// (s -> -s).  Cache write, E4M3: scale = max|y| / 448 of the row, code = E4M3(y / scale).
//
// All three kernels move each byte once and are bound by HBM.  A row of D elements is D / 16 lanes, each
// with two 16-byte chunks (bf16); in the half layout they hold the two elements of each pair, so a
// turn never leaves its lane.  A lane group takes HEADS heads of one token: the
// token's cos/sin are read once for them and every lane keeps 2 HEADS loads in flight.  Consecutive
// groups take consecutive heads, then tokens, so a block reads and writes one contiguous piece.
// Measured, back to back: rotation of 16384 x 16 x 128 19.7 us (134 MB, 6.8 TB/s); rotation and E4M3 write of 16384
// tokens, 32 query and 8 key/value heads of 128, 58.7 us (370 MB, 6.3 TB/s); read-back of 263 MB 42.1 us (6.2 TB/s).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache.h"
#include "ptx.cuh"

namespace ea46 {

namespace {

// Rows (heads of one token) a lane group works on at once, threads of a block and blocks an SM is compiled for (64
// registers).  Measured, us: 2 rows instead of 4 takes the rotation of 16384 x 16 x 128 from 20.3 to 22.7 and the
// E4M3 write of 16384 tokens (32 + 2 x 8 heads of 128) from 63.7 to 69.2; three quarters of the threads give 21.7
// and 65.8; blocks of 256 threads 20.1 and 63.4 against 19.8 and 62.2 of 128 (and of 64).
constexpr int HEADS = 4, THREADS = 128, BLOCKS_PER_SM = 8;
enum : int { WHERE_ROPE_POS = 41, WHERE_APPEND_SLOT = 42, WHERE_GATHER = 43 };

__device__ __forceinline__ void note_bad(int* err_word, int* err_info, int where) {
  if (atomicCAS(err_word, 0, 1 /* ATTN_ERR_INVALID_ARG */) == 0) atomicExch(err_info, where);
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// First elements of the two chunks of lane l of a row: l and l + D / 16, so that the lanes of one load lie
// side by side; in the half layout the lanes of the turned part take the chunks whose elements pair
// up, and the others split the rest the same way.
template <int D, bool HALF>
__device__ __forceinline__ void chunks_of(int l, int rot, int& c0, int& c1) {
  const int hl = HALF ? rot / 16 : 0;
  if (HALF && l < hl) {
    c0 = 8 * l;
    c1 = c0 + rot / 2;
  } else {
    c0 = 8 * (l + hl);
    c1 = c0 + 8 * (D / 16 - hl);
  }
}

// The cos and sin of a lane's eight pairs: four of each chunk (interleaved), or elementwise (half).
template <bool HALF>
struct Turn {
  float4 e[4];          // (c, s, c, s)
  bool on[2];           // the chunk's elements turn

  __device__ __forceinline__ void load(const RopeParams& r, int p, int c0, int c1) {
    const bool any = r.cs != nullptr && p >= 0;
    on[0] = any && c0 < r.rot;
    on[1] = any && c1 < r.rot;
    const float* row = r.cs + static_cast<long long>(p) * r.rot;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (on[k]) {
        // entries (c, s) of pairs from c0 on (half), or from chunk k's first pair
        const float4* t = reinterpret_cast<const float4*>(row + (HALF ? 2 * c0 + 8 * k : (k ? c1 : c0)));
        e[2 * k] = *(t);
        e[2 * k + 1] = *(t + 1);
      }
  }

  __device__ __forceinline__ bool any() const { return on[0] || on[1]; }

  // f: the two chunks' elements.
  __device__ __forceinline__ void apply(float (&f)[16], float sign) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!on[i >> 2]) continue;
      const float c = (i & 1) ? e[i >> 1].z : e[i >> 1].x, s = ((i & 1) ? e[i >> 1].w : e[i >> 1].y) * sign;
      float& a = f[HALF ? i : 2 * i];
      float& b = f[HALF ? i + 8 : 2 * i + 1];
      const float x = a, y = b;
      a = fmaf(x, c, -(y * s));
      b = fmaf(y, c, x * s);
    }
  }
};

// Position of token t, or -1 (reported) when the table has no row for it.
__device__ __forceinline__ int position(const RopeParams& r, uint32_t t, int* err_word, int* err_info) {
  const int p = r.pos != nullptr ? *(r.pos + t) : static_cast<int>(t % static_cast<uint32_t>(r.pos_wrap));
  if (p >= 0 && p < r.n_pos) return p;
  note_bad(err_word, err_info, WHERE_ROPE_POS);
  return -1;
}

// Item of this thread's lane group in block `block`, as (token, chunk of heads) of n chunks a token; 32
// bits by the host.
__device__ __forceinline__ void item_of(uint32_t block, int lanes, int n, uint32_t& t, int& sub) {
  const uint32_t item = block * (THREADS / lanes) + threadIdx.x / lanes;
  t = item / static_cast<uint32_t>(n);
  sub = static_cast<int>(item - t * static_cast<uint32_t>(n));
}

template <int D, bool HALF>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM) rope_apply_kernel(const RopeApplyParams p) {
  grid_launch_dependents();
  grid_dependency_wait();       // everything below reads what earlier kernels may have written
  constexpr int LPR = D / 16;
  const int l = threadIdx.x % LPR;
  uint32_t t;
  int sub;
  item_of(blockIdx.x, LPR, (p.H + HEADS - 1) / HEADS, t, sub);
  if (t >= static_cast<uint32_t>(p.n_tokens)) return;
  const int h0 = sub * HEADS;
  const int pos = position(p.rope, t, p.err_word, p.err_info);
  int c0, c1;
  chunks_of<D, HALF>(l, p.rope.rot, c0, c1);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.x) + t * p.x_stride + static_cast<long long>(h0) * D;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + t * p.out_stride + static_cast<long long>(h0) * D;
  uint4 u[HEADS][2];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h0 + h < p.H) {
      u[h][0] = *reinterpret_cast<const uint4*>(src + h * D + c0);
      u[h][1] = *reinterpret_cast<const uint4*>(src + h * D + c1);
    }
  if (pos < 0) return;
  Turn<HALF> turn;
  turn.load(p.rope, pos, c0, c1);
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h0 + h < p.H) {
      if (turn.any()) {
        float f[16];
        unpack8(u[h][0], f);
        unpack8(u[h][1], f + 8);
        turn.apply(f, p.rope.sin_sign);
        u[h][0] = pack8(f);
        u[h][1] = pack8(f + 8);
      }
      *reinterpret_cast<uint4*>(dst + h * D + c0) = u[h][0];
      *reinterpret_cast<uint4*>(dst + h * D + c1) = u[h][1];
    }
}

// A row's scale: largest magnitude / 448.  A row below 2^-117 throughout is written as zeros with
// scale 1 (a smaller scale would be subnormal); NaN anywhere makes the scale NaN, an infinity
// makes it infinite, and either way the row reads back as NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <int D, bool HALF, bool FP8>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM) cache_append_kernel(const AppendParams p) {
  grid_launch_dependents();
  grid_dependency_wait();       // everything below reads what earlier kernels may have written
  constexpr int LPR = D / 16;
  const int l = threadIdx.x % LPR;
  // A block's groups do like work, queries or keys and values, and the two kinds of blocks take turns: the
  // quantiser's instructions run beside the queries' loads, and a token's kinds read its cos and sin
  // soon after each other (62.2 us to 59.1; queries first, then the others).
  const uint32_t kv_before = static_cast<uint32_t>((blockIdx.x * p.kv_step) >> 32);
  const bool queries = kv_before == static_cast<uint32_t>(((blockIdx.x + 1ull) * p.kv_step) >> 32);
  const int nkv = (p.cache.Hkv + HEADS - 1) / HEADS;
  uint32_t t;
  int sub;
  if (queries) item_of(blockIdx.x - kv_before, LPR, (p.Hq + HEADS - 1) / HEADS, t, sub);
  else item_of(kv_before, LPR, 2 * nkv, t, sub);
  if (t >= static_cast<uint32_t>(p.n_tokens)) return;
  const int which = queries ? 0 : (sub < nkv ? 1 : 2);                // q, k, v
  const int h0 = (which == 2 ? sub - nkv : sub) * HEADS;
  const int H = which == 0 ? p.Hq : p.cache.Hkv;
  const bool turns = p.rope.cs != nullptr && which != 2;
  const int pos = turns ? position(p.rope, t, p.err_word, p.err_info) : 0;
  // where the rows go: a slot below 0 is a padded token, one past the cache is reported
  const int ps_log = 31 - __clz(p.cache.page_size);
  long long slot = 0;
  bool store = pos >= 0;
  if (which != 0) {
    slot = *(p.slots + t);
    const bool in = slot < static_cast<long long>(p.cache.n_pages) << ps_log;
    if (!in) note_bad(p.err_word, p.err_info, WHERE_APPEND_SLOT);
    store = store && slot >= 0 && in;
  }
  int c0, c1;
  chunks_of<D, HALF>(l, turns ? p.rope.rot : 0, c0, c1);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which == 0 ? p.q : (which == 1 ? p.k : p.v)) +
                             t * (which == 0 ? p.q_stride : (which == 1 ? p.k_stride : p.v_stride)) +
                             static_cast<long long>(h0) * D;
  uint4 u[HEADS][2];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h0 + h < H) {
      u[h][0] = *reinterpret_cast<const uint4*>(src + h * D + c0);
      u[h][1] = *reinterpret_cast<const uint4*>(src + h * D + c1);
    }
  if (!store) return;                                   // a whole lane group, as in every branch here
  Turn<HALF> turn;
  turn.load(p.rope, turns ? pos : -1, c0, c1);
  const long long page = slot >> ps_log;
  const int off = static_cast<int>(slot) & (p.cache.page_size - 1);
  const unsigned group = (LPR == 32 ? ~0u : (1u << (LPR & 31)) - 1) << (threadIdx.x & 31 & ~(LPR - 1));
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h0 + h >= H) break;
    if (which == 0 || !FP8) {
      if (turn.any()) {
        float f[16];
        unpack8(u[h][0], f);
        unpack8(u[h][1], f + 8);
        turn.apply(f, 1.f);
        u[h][0] = pack8(f);
        u[h][1] = pack8(f + 8);
      }
      __nv_bfloat16* dst =
          which == 0 ? static_cast<__nv_bfloat16*>(p.q_out) + (static_cast<long long>(t) * p.Hq + h0 + h) * D
                     : static_cast<__nv_bfloat16*>(which == 1 ? p.cache.k : p.cache.v) + page * p.cache.page_stride +
                           (h0 + h) * p.cache.head_stride + off * p.cache.tok_stride;
      *reinterpret_cast<uint4*>(dst + c0) = u[h][0];
      *reinterpret_cast<uint4*>(dst + c1) = u[h][1];
    } else {
      float f[16];
      unpack8(u[h][0], f);
      unpack8(u[h][1], f + 8);
      turn.apply(f, 1.f);
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max_nan(m, fabsf(f[i]));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(group, m, o));
      const float scale = m < 0x1p-117f ? 1.f : m / 448.f;
      // x / scale for the row's elements from one reciprocal: r = fl(1 / scale), q = fl(x r), one correction
      // by the exact remainder x - q scale (Markstein 1990: the correctly rounded quotient)
      const float r = 1.f / scale;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float q = f[i] * r;
        f[i] = fmaf(fmaf(-q, scale, f[i]), r, q);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = pack_e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      uint8_t* dst = static_cast<uint8_t*>(which == 1 ? p.cache.k : p.cache.v) + page * p.cache.page_stride +
                     (h0 + h) * p.cache.head_stride + off * p.cache.tok_stride;
      *reinterpret_cast<uint2*>(dst + c0) = make_uint2(c[0], c[1]);
      *reinterpret_cast<uint2*>(dst + c1) = make_uint2(c[2], c[3]);
      if (l == 0)
        (which == 1 ? p.cache.k_scale : p.cache.v_scale)[((page * p.cache.Hkv + h0 + h) << ps_log) + off] = scale;
    }
  }
}

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[0]), "=f"(f[1]) : "r"(lo));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[2]), "=f"(f[3]) : "r"(hi));
}

// One lane group per token and HEADS heads of k and of v, two chunks of eight elements
// a lane (as above).
template <int D, bool FP8>
__global__ void __launch_bounds__(THREADS) cache_gather_kernel(const GatherParams p) {
  grid_launch_dependents();
  grid_dependency_wait();       // everything below reads what earlier kernels may have written
  constexpr int LPR = D / 16;
  const int l = threadIdx.x % LPR;
  const int ps_log = 31 - __clz(p.cache.page_size);
  uint32_t t;
  int sub;
  item_of(blockIdx.x, LPR, (p.cache.Hkv + HEADS - 1) / HEADS, t, sub);
  const int tok = static_cast<int>(t), h0 = sub * HEADS;
  if (t >= static_cast<uint32_t>(p.total)) return;
  // the sequence of the token: the last s with cu[s] <= tok.  The search stays inside the array
  // whatever it holds; a token that lies in no sequence is reported and not written.
  int lo = 0, hi = p.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (*(p.cu_seqlens + mid) <= tok) lo = mid; else hi = mid;
  }
  const long long off = static_cast<long long>(tok) - *(p.cu_seqlens + lo);
  const bool in = off >= 0 && tok < *(p.cu_seqlens + lo + 1) && (off >> ps_log) < p.max_pages;
  long long page = -1;
  if (in) page = *(p.page_table + static_cast<long long>(lo) * p.max_pages + (off >> ps_log));
  if (page < 0 || page >= p.cache.n_pages) {
    note_bad(p.err_word, p.err_info, WHERE_GATHER);
    return;
  }
  const int at = static_cast<int>(off) & (p.cache.page_size - 1);
  const long long e0 = page * p.cache.page_stride + h0 * p.cache.head_stride + at * p.cache.tok_stride + 8 * l;
  uint4 u[2][HEADS][2];                // E4M3: eight codes in .x, .y
  float scale[2][HEADS];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
      if (h0 + h < p.cache.Hkv) {
        const long long e = e0 + h * p.cache.head_stride;
        if constexpr (FP8) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv ? p.cache.v : p.cache.k) + e + c * (D / 2));
            u[kv][h][c].x = w.x;
            u[kv][h][c].y = w.y;
          }
          scale[kv][h] = *((kv ? p.cache.v_scale : p.cache.k_scale) + ((page * p.cache.Hkv + h0 + h) << ps_log) + at);
        } else {
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(kv ? p.cache.v : p.cache.k) + e;
          u[kv][h][0] = *reinterpret_cast<const uint4*>(src);
          u[kv][h][1] = *reinterpret_cast<const uint4*>(src + D / 2);
        }
      }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
      if (h0 + h < p.cache.Hkv) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(kv ? p.v_out : p.k_out) +
                             (static_cast<long long>(tok) * p.cache.Hkv + h0 + h) * D + 8 * l;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (FP8) {
            float f[8];
            e4m3x4_to_f32(u[kv][h][c].x, f);
            e4m3x4_to_f32(u[kv][h][c].y, f + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= scale[kv][h];
            u[kv][h][c] = pack8(f);
          }
          *reinterpret_cast<uint4*>(dst + c * (D / 2)) = u[kv][h][c];
        }
      }
}

unsigned blocks_for(int subs, int tokens, int D) {
  const long long groups = THREADS / (D / 16);
  return static_cast<unsigned>((static_cast<long long>(subs) * tokens + groups - 1) / groups);
}

template <int D>
cudaError_t rope_d(const RopeApplyParams& p, bool half, cudaStream_t st) {
  const unsigned grid = blocks_for((p.H + HEADS - 1) / HEADS, p.n_tokens, D);
  return launch_overlapped(half ? rope_apply_kernel<D, true> : rope_apply_kernel<D, false>, dim3(grid), THREADS, 0, st, p);
}

template <int D>
cudaError_t append_d(AppendParams p, bool half, cudaStream_t st) {
  const unsigned q_blocks = p.q != nullptr ? blocks_for((p.Hq + HEADS - 1) / HEADS, p.n_tokens, D) : 0;
  const unsigned kv_blocks = blocks_for(2 * ((p.cache.Hkv + HEADS - 1) / HEADS), p.n_tokens, D), grid = q_blocks + kv_blocks;
  // rounded up: floor(grid * kv_step / 2^32) is kv_blocks
  p.kv_step = ((static_cast<unsigned long long>(kv_blocks) << 32) + grid - 1) / grid;
  const bool fp8 = p.cache.k_scale != nullptr;
  void (*kernel)(AppendParams) = half ? (fp8 ? cache_append_kernel<D, true, true> : cache_append_kernel<D, true, false>)
                                      : (fp8 ? cache_append_kernel<D, false, true> : cache_append_kernel<D, false, false>);
  return launch_overlapped(kernel, dim3(grid), THREADS, 0, st, p);
}

template <int D>
cudaError_t gather_d(const GatherParams& p, cudaStream_t st) {
  const unsigned grid = blocks_for((p.cache.Hkv + HEADS - 1) / HEADS, p.total, D);
  return launch_overlapped(p.cache.k_scale != nullptr ? cache_gather_kernel<D, true> : cache_gather_kernel<D, false>,
                           dim3(grid), THREADS, 0, st, p);
}

}  // namespace

cudaError_t launch_rope_apply(const RopeApplyParams& p, int D, bool half, cudaStream_t st) {
  return D == 64 ? rope_d<64>(p, half, st) : (D == 128 ? rope_d<128>(p, half, st) : rope_d<256>(p, half, st));
}

cudaError_t launch_cache_append(const AppendParams& p, int D, bool half, cudaStream_t st) {
  return D == 64 ? append_d<64>(p, half, st) : (D == 128 ? append_d<128>(p, half, st) : append_d<256>(p, half, st));
}

cudaError_t launch_cache_gather(const GatherParams& p, int D, cudaStream_t st) {
  return D == 64 ? gather_d<64>(p, st) : (D == 128 ? gather_d<128>(p, st) : gather_d<256>(p, st));
}

}  // namespace ea46
