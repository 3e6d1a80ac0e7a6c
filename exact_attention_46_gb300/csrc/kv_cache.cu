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
// All three kernels move each byte once and are bound by HBM.  A row of D bf16 elements is D / 8
// lanes x 16 bytes; a lane group takes one token and HEADS heads of it, so the token's cos/sin are
// read once for HEADS rows and every lane keeps HEADS 16-byte loads in flight.  Pairs of the
// interleaved layout lie within a lane; those of the half layout are rot / 16 lanes apart and
// meet by shuffle.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache.h"
#include "ptx.cuh"

namespace ea46 {

namespace {

constexpr int HEADS = 4;          // rows (heads of one token) a lane group works on at once
constexpr int THREADS = 256;
enum : int { WHERE_ROPE_POS = 41, WHERE_APPEND_SLOT = 42, WHERE_GATHER = 43 };

__device__ __forceinline__ void note_bad(int* err_word, int* err_info, int where) {
  if (atomicCAS(err_word, 0, 1 /* ATTN_ERR_INVALID_ARG */) == 0) atomicExch(err_info, where);
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// The cos and sin of one lane's eight elements (interleaved: four pairs, both entries of a pair
// alike; half: eight).  Lanes past `rot` get the identity.
template <bool HALF>
struct Turn {
  float c[HALF ? 8 : 4], s[HALF ? 8 : 4];
  bool on;              // this lane's elements turn
  int partner;          // half: the lane with the other elements of the pairs
  bool second;          // half: this lane holds the pairs' second elements

  __device__ __forceinline__ void load(const RopeParams& r, int p, int lane_in_row, int lane_base) {
    on = r.cs != nullptr && 8 * lane_in_row < r.rot;
    second = false;
    partner = lane_base + lane_in_row;
    int first = 4 * lane_in_row;                      // table index of the lane's first entry
    if (HALF) {
      const int hl = r.rot / 16;
      second = on && lane_in_row >= hl;
      if (on) partner = lane_base + (second ? lane_in_row - hl : lane_in_row + hl);
      first = 8 * (second ? lane_in_row - hl : lane_in_row);
    }
#pragma unroll
    for (int i = 0; i < (HALF ? 8 : 4); ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    if (on) {
      const float4* t = reinterpret_cast<const float4*>(r.cs + (static_cast<long long>(p) * (r.rot / 2) + first) * 2);
#pragma unroll
      for (int i = 0; i < (HALF ? 4 : 2); ++i) {
        const float4 e = __ldg(t + i);
        c[2 * i] = e.x;
        s[2 * i] = e.y * r.sin_sign;
        c[2 * i + 1] = e.z;
        s[2 * i + 1] = e.w * r.sin_sign;
      }
    }
  }

  // Every lane of the warp calls this (shuffle).
  __device__ __forceinline__ void apply(float (&f)[8]) const {
    if constexpr (HALF) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, f[i], partner);
        // first element: x_a c - x_b s;  second: x_b c + x_a s
        if (on) f[i] = second ? fmaf(f[i], c[i], o * s[i]) : fmaf(f[i], c[i], -(o * s[i]));
      }
    } else {
      if (on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = f[2 * i], b = f[2 * i + 1];
          f[2 * i] = fmaf(a, c[i], -(b * s[i]));
          f[2 * i + 1] = fmaf(b, c[i], a * s[i]);
        }
      }
    }
  }
};

// Position of token t, or -1 (reported) when the table has no row for it.
__device__ __forceinline__ int position(const RopeParams& r, long long t, int* err_word, int* err_info) {
  const int p = r.pos != nullptr ? __ldg(r.pos + t) : static_cast<int>(t % r.pos_wrap);
  if (p >= 0 && p < r.n_pos) return p;
  note_bad(err_word, err_info, WHERE_ROPE_POS);
  return -1;
}

template <int D, bool HALF>
__global__ void __launch_bounds__(THREADS) rope_apply_kernel(const RopeApplyParams p) {
  constexpr int LPR = D / 8;
  const int lr = threadIdx.x % LPR, base = (threadIdx.x & 31) - lr;
  const int chunks = (p.H + HEADS - 1) / HEADS;
  const long long item = (static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x) / LPR;
  const long long t = item / chunks;
  const int h0 = static_cast<int>(item % chunks) * HEADS;
  const bool live = t < p.n_tokens;
  uint4 u[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (live && h0 + h < p.H)
      u[h] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + t * p.x_stride +
                                             static_cast<long long>(h0 + h) * D + 8 * lr);
  const int pos = live ? position(p.rope, t, p.err_word, p.err_info) : -1;
  Turn<HALF> turn;
  RopeParams r = p.rope;
  if (pos < 0) r.cs = nullptr;
  turn.load(r, pos, lr, base);
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float f[8] = {};
    const bool there = live && h0 + h < p.H;
    if (there) unpack8(u[h], f);
    turn.apply(f);
    if (there && pos >= 0)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + t * p.out_stride +
                                static_cast<long long>(h0 + h) * D + 8 * lr) = pack8(f);
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
__global__ void __launch_bounds__(THREADS) cache_append_kernel(const AppendParams p) {
  constexpr int LPR = D / 8;
  const int lr = threadIdx.x % LPR, base = (threadIdx.x & 31) - lr;
  // items of one token: its q chunks, then k chunks, then v chunks of HEADS heads
  const int nq = p.q != nullptr ? (p.Hq + HEADS - 1) / HEADS : 0;
  const int nkv = (p.cache.Hkv + HEADS - 1) / HEADS;
  const int per_token = nq + 2 * nkv;
  const long long item = (static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x) / LPR;
  const long long t = item / per_token;
  const int sub = static_cast<int>(item % per_token);
  const bool live = t < p.n_tokens;
  const int which = sub < nq ? 0 : (sub < nq + nkv ? 1 : 2);          // q, k, v
  const int h0 = (which == 0 ? sub : (which == 1 ? sub - nq : sub - nq - nkv)) * HEADS;
  const int H = which == 0 ? p.Hq : p.cache.Hkv;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which == 0 ? p.q : (which == 1 ? p.k : p.v)) +
                             t * (which == 0 ? p.q_stride : (which == 1 ? p.k_stride : p.v_stride)) + 8 * lr;
  uint4 u[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (live && h0 + h < H) u[h] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(h0 + h) * D);

  // where the row goes: a slot below 0 is a padded token, one past the cache is reported
  bool store = live;
  long long page = 0;
  int off = 0;
  if (live && which != 0) {
    const long long slot = __ldg(p.slots + t);
    store = slot >= 0 && slot < static_cast<long long>(p.cache.n_pages) * p.cache.page_size;
    if (slot >= 0 && !store) note_bad(p.err_word, p.err_info, WHERE_APPEND_SLOT);
    if (store) {
      page = slot / p.cache.page_size;
      off = static_cast<int>(slot - page * p.cache.page_size);
    }
  }
  RopeParams r = p.rope;
  if (which == 2 || !store) r.cs = nullptr;
  int pos = 0;
  if (r.cs != nullptr) {
    pos = position(r, t, p.err_word, p.err_info);
    if (pos < 0) {
      r.cs = nullptr;
      store = false;
    }
  }
  Turn<HALF> turn;
  turn.load(r, pos, lr, base);
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float f[8] = {};
    const bool there = live && h0 + h < H;
    if (there) unpack8(u[h], f);
    turn.apply(f);
    const bool put = there && store;
    if (FP8) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (which != 0) {
        const float scale = m < 0x1p-117f ? 1.f : m / 448.f;
        if (put) {
          uint2 c;
          c.x = pack_e4m3x4(f[0] / scale, f[1] / scale, f[2] / scale, f[3] / scale);
          c.y = pack_e4m3x4(f[4] / scale, f[5] / scale, f[6] / scale, f[7] / scale);
          uint8_t* dst = static_cast<uint8_t*>(which == 1 ? p.cache.k : p.cache.v) + page * p.cache.page_stride +
                         (h0 + h) * p.cache.head_stride + off * p.cache.tok_stride + 8 * lr;
          *reinterpret_cast<uint2*>(dst) = c;
          if (lr == 0)
            (which == 1 ? p.cache.k_scale : p.cache.v_scale)[(page * p.cache.Hkv + h0 + h) * p.cache.page_size + off] =
                scale;
        }
      } else if (put) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) +
                                  (t * p.Hq + h0 + h) * static_cast<long long>(D) + 8 * lr) = pack8(f);
      }
    } else if (put) {
      __nv_bfloat16* dst =
          which == 0 ? static_cast<__nv_bfloat16*>(p.q_out) + (t * p.Hq + h0 + h) * static_cast<long long>(D)
                     : static_cast<__nv_bfloat16*>(which == 1 ? p.cache.k : p.cache.v) + page * p.cache.page_stride +
                           (h0 + h) * p.cache.head_stride + off * p.cache.tok_stride;
      *reinterpret_cast<uint4*>(dst + 8 * lr) = pack8(f);
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

// One lane group per token and HEADS heads of k and of v.
template <int D, bool FP8>
__global__ void __launch_bounds__(THREADS) cache_gather_kernel(const GatherParams p) {
  constexpr int LPR = D / 8;
  const int lr = threadIdx.x % LPR;
  const int chunks = (p.cache.Hkv + HEADS - 1) / HEADS;
  const long long item = (static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x) / LPR;
  const long long t = item / chunks;
  const int h0 = static_cast<int>(item % chunks) * HEADS;
  if (t >= p.total) return;
  // the sequence of token t: the last s with cu[s] <= t.  The search stays inside the array
  // whatever it holds; a token that lies in no sequence is reported and not written.
  int lo = 0, hi = p.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
  }
  const long long off = t - __ldg(p.cu_seqlens + lo);
  const bool in = off >= 0 && t < __ldg(p.cu_seqlens + lo + 1) && off / p.cache.page_size < p.max_pages;
  long long page = -1;
  if (in) page = __ldg(p.page_table + static_cast<long long>(lo) * p.max_pages + off / p.cache.page_size);
  if (page < 0 || page >= p.cache.n_pages) {
    note_bad(p.err_word, p.err_info, WHERE_GATHER);
    return;
  }
  const int at = static_cast<int>(off % p.cache.page_size);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const void* cache = kv == 0 ? p.cache.k : p.cache.v;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(kv == 0 ? p.k_out : p.v_out);
    const float* sc = kv == 0 ? p.cache.k_scale : p.cache.v_scale;
    uint4 u[HEADS];
    float scale[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      if (h0 + h >= p.cache.Hkv) continue;
      const long long e = page * p.cache.page_stride + (h0 + h) * p.cache.head_stride + at * p.cache.tok_stride + 8 * lr;
      if (FP8) {
        const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + e);
        u[h].x = c.x;
        u[h].y = c.y;
        scale[h] = __ldg(sc + (page * p.cache.Hkv + h0 + h) * p.cache.page_size + at);
      } else {
        u[h] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + e);
      }
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      if (h0 + h >= p.cache.Hkv) continue;
      uint4 w = u[h];
      if (FP8) {
        float f[8];
        e4m3x4_to_f32(u[h].x, f);
        e4m3x4_to_f32(u[h].y, f + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= scale[h];
        w = pack8(f);
      }
      *reinterpret_cast<uint4*>(out + (t * p.cache.Hkv + h0 + h) * static_cast<long long>(D) + 8 * lr) = w;
    }
  }
}

unsigned blocks_for(long long items, int D) { return static_cast<unsigned>((items * (D / 8) + THREADS - 1) / THREADS); }

template <int D>
cudaError_t rope_d(const RopeApplyParams& p, bool half, cudaStream_t st) {
  const unsigned grid = blocks_for(static_cast<long long>(p.n_tokens) * ((p.H + HEADS - 1) / HEADS), D);
  if (half) rope_apply_kernel<D, true><<<grid, THREADS, 0, st>>>(p);
  else rope_apply_kernel<D, false><<<grid, THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t append_d(const AppendParams& p, bool half, cudaStream_t st) {
  const int nq = p.q != nullptr ? (p.Hq + HEADS - 1) / HEADS : 0, nkv = (p.cache.Hkv + HEADS - 1) / HEADS;
  const unsigned grid = blocks_for(static_cast<long long>(p.n_tokens) * (nq + 2 * nkv), D);
  const bool fp8 = p.cache.k_scale != nullptr;
  if (half) {
    if (fp8) cache_append_kernel<D, true, true><<<grid, THREADS, 0, st>>>(p);
    else cache_append_kernel<D, true, false><<<grid, THREADS, 0, st>>>(p);
  } else {
    if (fp8) cache_append_kernel<D, false, true><<<grid, THREADS, 0, st>>>(p);
    else cache_append_kernel<D, false, false><<<grid, THREADS, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t gather_d(const GatherParams& p, cudaStream_t st) {
  const unsigned grid = blocks_for(static_cast<long long>(p.total) * ((p.cache.Hkv + HEADS - 1) / HEADS), D);
  if (p.cache.k_scale != nullptr) cache_gather_kernel<D, true><<<grid, THREADS, 0, st>>>(p);
  else cache_gather_kernel<D, false><<<grid, THREADS, 0, st>>>(p);
  return cudaGetLastError();
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
