// api_cache.cu -- the C ABI of rotary positions and the paged key/value cache (include/attn46.h):
// argument checks and launches.  No computation happens here.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn46.h"
#include "cache.h"

namespace {

using namespace ea46;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_head_dim(int D, bool d256) {
  if (D == 64 || D == 128 || (D == 256 && d256)) return ATTN_OK;
  return api_fail(D > 0 ? ATTN_ERR_UNSUPPORTED : ATTN_ERR_INVALID_ARG, "head dimension D = %d not supported (64, 128%s)",
                  D, d256 ? ", 256" : "");
}

// Rows of `heads` heads of D elements, one token every `stride` elements: extent in elements.
long long extent(long long tokens, long long stride, int heads, int D) {
  return (tokens - 1) * stride + static_cast<long long>(heads) * D;
}

// The row kernels number lane groups (a token's heads in fours, at worst one) in 31 bits.
bool rows_fit(long long tokens, long long heads) { return tokens * (heads + 3) < 0x7fffff00ll; }

int check_rows(const char* name, const void* ptr, long long stride, int n_tokens, int heads, int D) {
  if (ptr == nullptr || !api_aligned16(ptr))
    return api_fail(ATTN_ERR_INVALID_ARG, "%s must be a non-null, 16-byte aligned device pointer", name);
  if (stride < static_cast<long long>(heads) * D || stride % 8 != 0 || stride > (1ll << 40))
    return api_fail(ATTN_ERR_INVALID_ARG, "%s: the token stride %lld must be a multiple of 8 elements and at least "
                    "heads * D = %lld", name, stride, static_cast<long long>(heads) * D);
  if (extent(n_tokens, stride, heads, D) > (1ll << 40))
    return api_fail(ATTN_ERR_INVALID_ARG, "%s is too large", name);
  return ATTN_OK;
}

int check_rope(const float* cs, int n_pos, int rot, int D, int layout) {
  if (cs == nullptr || !api_aligned16(cs))
    return api_fail(ATTN_ERR_INVALID_ARG, "rope_cs must be a non-null, 16-byte aligned device pointer");
  if (n_pos < 1) return api_fail(ATTN_ERR_INVALID_ARG, "n_pos must be >= 1 (got %d)", n_pos);
  if (layout != ATTN_ROPE_INTERLEAVED && layout != ATTN_ROPE_HALF)
    return api_fail(ATTN_ERR_INVALID_ARG, "rope_layout must be ATTN_ROPE_INTERLEAVED (0) or ATTN_ROPE_HALF (1)");
  if (rot < 16 || rot > D || rot % 16 != 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [16, D] (got %d)", rot);
  return ATTN_OK;
}

// The cache arguments of every entry point; fills the view.
int check_cache(CacheView* c, const void* k, const void* v, const float* ks, const float* vs, int n_pages, int page_size,
                int Hkv, int D, int layout, int dtype) {
  if (dtype != ATTN_BF16 && dtype != ATTN_FP8_E4M3)
    return api_fail(ATTN_ERR_INVALID_ARG, "dtype must be ATTN_BF16 (0) or ATTN_FP8_E4M3 (1)");
  if (layout != ATTN_CACHE_HEAD_MAJOR && layout != ATTN_CACHE_TOKEN_MAJOR)
    return api_fail(ATTN_ERR_INVALID_ARG, "cache_layout must be ATTN_CACHE_HEAD_MAJOR (0) or ATTN_CACHE_TOKEN_MAJOR (1)");
  if (k == nullptr || v == nullptr || !api_aligned16(k) || !api_aligned16(v))
    return api_fail(ATTN_ERR_INVALID_ARG, "k_cache and v_cache must be non-null, 16-byte aligned device pointers");
  if (n_pages < 1 || Hkv < 1 || Hkv > 65535)
    return api_fail(ATTN_ERR_INVALID_ARG, "need n_pages >= 1 and 1 <= Hkv <= 65535 (got %d, %d)", n_pages, Hkv);
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return api_fail(page_size > 0 ? ATTN_ERR_UNSUPPORTED : ATTN_ERR_INVALID_ARG,
                    "page_size must be a power of two in [16, 1024] (got %d)", page_size);
  const unsigned __int128 n = static_cast<unsigned __int128>(n_pages) * page_size * Hkv * D;
  if (n > (1ull << 40)) return api_fail(ATTN_ERR_INVALID_ARG, "the cache is too large");
  const bool fp8 = dtype == ATTN_FP8_E4M3;
  if (fp8 != (ks != nullptr) || fp8 != (vs != nullptr))
    return api_fail(ATTN_ERR_INVALID_ARG, "k_scale and v_scale go with an E4M3 cache, both, and only with one");
  if (!api_aligned16(ks) || !api_aligned16(vs)) return api_fail(ATTN_ERR_INVALID_ARG, "cache scales must be 16-byte aligned");
  c->k = const_cast<void*>(k);
  c->v = const_cast<void*>(v);
  c->k_scale = const_cast<float*>(ks);
  c->v_scale = const_cast<float*>(vs);
  c->n_pages = n_pages;
  c->page_size = page_size;
  c->Hkv = Hkv;
  c->page_stride = static_cast<long long>(page_size) * Hkv * D;
  c->head_stride = layout == ATTN_CACHE_HEAD_MAJOR ? static_cast<long long>(page_size) * D : D;
  c->tok_stride = layout == ATTN_CACHE_HEAD_MAJOR ? D : static_cast<long long>(Hkv) * D;
  return ATTN_OK;
}

struct Range {
  const void* p;
  size_t n;
};

// No output may overlap another output or an input (null ranges are skipped).
int check_disjoint(const Range* outs, int n_outs, const Range* ins, int n_ins) {
  for (int i = 0; i < n_outs; ++i) {
    if (outs[i].p == nullptr || outs[i].n == 0) continue;
    for (int j = 0; j < n_ins; ++j)
      if (ins[j].p != nullptr && api_overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
        return api_fail(ATTN_ERR_INVALID_ARG, "an output overlaps an input");
    for (int j = i + 1; j < n_outs; ++j)
      if (outs[j].p != nullptr && api_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return api_fail(ATTN_ERR_INVALID_ARG, "outputs overlap each other");
  }
  return ATTN_OK;
}

size_t cache_bytes(const CacheView& c, int D) {
  return static_cast<size_t>(c.n_pages) * c.page_size * c.Hkv * D * (c.k_scale != nullptr ? 1 : 2);
}

size_t scale_bytes(const CacheView& c) { return 4ull * c.n_pages * c.page_size * c.Hkv; }

int append(const void* q, const void* k, const void* v, void* q_out, const float* cs, const int* positions, void* kc,
           void* vc, float* ks, float* vs, const long long* slots, int n_tokens, int Hq, int Hkv, int D,
           long long q_stride, long long k_stride, long long v_stride, int n_pages, int page_size, int cache_layout,
           int dtype, int n_pos, int rot, int rope_layout, void* stream) {
  const bool rope = q != nullptr;
  if (n_tokens < 1) return api_fail(ATTN_ERR_INVALID_ARG, "n_tokens must be >= 1 (got %d)", n_tokens);
  AppendParams p{};
  int rc = check_head_dim(D, true);
  if (rc == ATTN_OK) rc = check_cache(&p.cache, kc, vc, ks, vs, n_pages, page_size, Hkv, D, cache_layout, dtype);
  if (rc == ATTN_OK) rc = check_rows("k", k, k_stride, n_tokens, Hkv, D);
  if (rc == ATTN_OK) rc = check_rows("v", v, v_stride, n_tokens, Hkv, D);
  if (rc != ATTN_OK) return rc;
  if (slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return api_fail(ATTN_ERR_INVALID_ARG, "slots must be a non-null, 8-byte aligned device pointer");
  if (rope) {
    if (Hq < 1 || Hq > 65535) return api_fail(ATTN_ERR_INVALID_ARG, "need 1 <= Hq <= 65535 (got %d)", Hq);
    if ((rc = check_rows("q", q, q_stride, n_tokens, Hq, D)) != ATTN_OK) return rc;
    if (q_out == nullptr || !api_aligned16(q_out))
      return api_fail(ATTN_ERR_INVALID_ARG, "q_out must be a non-null, 16-byte aligned device pointer");
    if (positions == nullptr || !aligned4(positions))
      return api_fail(ATTN_ERR_INVALID_ARG, "positions must be a non-null, 4-byte aligned device pointer");
    if ((rc = check_rope(cs, n_pos, rot, D, rope_layout)) != ATTN_OK) return rc;
  }
  if (!rows_fit(n_tokens, (rope ? Hq : 0) + 2ll * Hkv)) return api_fail(ATTN_ERR_INVALID_ARG, "too many rows");
  const size_t cb = cache_bytes(p.cache, D), sb = scale_bytes(p.cache);
  const Range outs[5] = {{kc, cb}, {vc, cb}, {ks, sb}, {vs, sb}, {q_out, 2ull * n_tokens * (rope ? Hq : 0) * D}};
  const Range ins[6] = {{q, rope ? 2ull * extent(n_tokens, q_stride, Hq, D) : 0},
                        {k, 2ull * extent(n_tokens, k_stride, Hkv, D)},
                        {v, 2ull * extent(n_tokens, v_stride, Hkv, D)},
                        {slots, 8ull * n_tokens},
                        {positions, 4ull * n_tokens},
                        {cs, 4ull * n_pos * (rope ? rot : 0)}};
  if ((rc = check_disjoint(outs, 5, ins, 6)) != ATTN_OK) return rc;
  if ((rc = api_err_words(&p.err_word)) != ATTN_OK) return rc;
  p.err_info = p.err_word + 1;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.n_tokens = n_tokens;
  p.Hq = Hq;
  p.rope = RopeParams{rope ? cs : nullptr, positions, 1, n_pos, rot, 1.f};
  const cudaError_t e = launch_cache_append(p, D, rope && rope_layout == ATTN_ROPE_HALF, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_fail(ATTN_ERR_CUDA, "cache write launch failed: %s", cudaGetErrorString(e));
  return api_ok();
}

// CTAs of attn_decode_paged's key kernel on the current device: one per SM, in groups of one per row tile.
int paged_ctas() {
  static std::atomic<int> known[64];               // SM count by device: a constant of the hardware
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// A unit can be shared by CTAs only if some sequence can have more than one 128-key tile.
bool paged_combines(int page_size, int max_pages) { return static_cast<long long>(page_size) * max_pages > 128; }

// Two partial units a CTA (the one it starts in and the one it ends in): RB rows of D + 1 floats; and a
// CTA's cut (16 bytes).  Where
// there are more row tiles than CTAs there is one group and nothing is cut.
size_t paged_workspace(int n_cta, int RB, int D) { return 8ull * n_cta * RB * (static_cast<size_t>(D) + 1) + 16ull * n_cta; }

}  // namespace

extern "C" {

int rope_scaled_table(float* cs, int n_pos, int rot_dim, double base, int scaling, double factor, double original_length,
                      void* stream) {
  if (cs == nullptr || (reinterpret_cast<uintptr_t>(cs) & 7u))
    return api_fail(ATTN_ERR_INVALID_ARG, "cs must be a non-null, 8-byte aligned device pointer");
  if (n_pos < 1 || n_pos > (1 << 26)) return api_fail(ATTN_ERR_INVALID_ARG, "n_pos must be in [1, 2^26] (got %d)", n_pos);
  if (rot_dim < 4 || rot_dim % 2 != 0 || rot_dim > 4096)
    return api_fail(ATTN_ERR_INVALID_ARG, "rot_dim must be even and in [4, 4096] (got %d)", rot_dim);
  if (!(base > 0.0) || !std::isfinite(base)) return api_fail(ATTN_ERR_INVALID_ARG, "base must be finite and > 0");
  if (scaling < ATTN_ROPE_UNSCALED || scaling > ATTN_ROPE_YARN)
    return api_fail(ATTN_ERR_INVALID_ARG, "scaling must be one of ATTN_ROPE_UNSCALED .. ATTN_ROPE_YARN (got %d)", scaling);
  if (!(factor >= 1.0) || !std::isfinite(factor)) return api_fail(ATTN_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (scaling == ATTN_ROPE_YARN && (!(original_length >= 1.0) || !std::isfinite(original_length)))
    return api_fail(ATTN_ERR_INVALID_ARG, "original_length must be finite and >= 1 for this scaling");
  const cudaError_t e =
      launch_rope_scaled_table(cs, n_pos, rot_dim, base, scaling, factor, original_length, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_fail(ATTN_ERR_CUDA, "rotary table launch failed: %s", cudaGetErrorString(e));
  return api_ok();
}

int rope_apply(const void* x, void* out, const float* rope_cs, const int* positions, int n_tokens, int seq_len, int H,
               int D, long long x_stride, long long out_stride, int n_pos, int rot_dim, int rope_layout, int transpose,
               void* stream) {
  if (n_tokens < 1 || H < 1 || H > 65535)
    return api_fail(ATTN_ERR_INVALID_ARG, "need n_tokens >= 1 and 1 <= H <= 65535 (got %d, %d)", n_tokens, H);
  int rc = check_head_dim(D, true);
  if (rc == ATTN_OK) rc = check_rows("x", x, x_stride, n_tokens, H, D);
  if (rc == ATTN_OK) rc = check_rows("out", out, out_stride, n_tokens, H, D);
  if (rc == ATTN_OK) rc = check_rope(rope_cs, n_pos, rot_dim, D, rope_layout);
  if (rc != ATTN_OK) return rc;
  if (!aligned4(positions)) return api_fail(ATTN_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  if (positions == nullptr && (seq_len < 1 || seq_len > n_pos))
    return api_fail(ATTN_ERR_INVALID_ARG, "without positions, seq_len must be in [1, n_pos] (got %d, n_pos = %d)", seq_len, n_pos);
  if (transpose != 0 && transpose != 1) return api_fail(ATTN_ERR_INVALID_ARG, "transpose must be 0 or 1");
  if (!rows_fit(n_tokens, H)) return api_fail(ATTN_ERR_INVALID_ARG, "too many rows");
  const size_t xb = 2ull * extent(n_tokens, x_stride, H, D), ob = 2ull * extent(n_tokens, out_stride, H, D);
  const bool in_place = x == out && x_stride == out_stride;
  const Range outs[1] = {{out, ob}};
  const Range ins[3] = {{in_place ? nullptr : x, xb}, {rope_cs, 4ull * n_pos * rot_dim}, {positions, 4ull * n_tokens}};
  if ((rc = check_disjoint(outs, 1, ins, 3)) != ATTN_OK) return rc;
  RopeApplyParams p{};
  if ((rc = api_err_words(&p.err_word)) != ATTN_OK) return rc;
  p.err_info = p.err_word + 1;
  p.x = x;
  p.out = out;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  p.n_tokens = n_tokens;
  p.H = H;
  p.rope = RopeParams{rope_cs, positions, positions != nullptr ? 1 : seq_len, n_pos, rot_dim, transpose ? -1.f : 1.f};
  const cudaError_t e = launch_rope_apply(p, D, rope_layout == ATTN_ROPE_HALF, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_fail(ATTN_ERR_CUDA, "rotary launch failed: %s", cudaGetErrorString(e));
  return api_ok();
}

int kv_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                    const long long* slots, int n_tokens, int Hkv, int D, long long k_stride, long long v_stride,
                    int n_pages, int page_size, int cache_layout, int dtype, void* stream) {
  return append(nullptr, k, v, nullptr, nullptr, nullptr, k_cache, v_cache, k_scale, v_scale, slots, n_tokens, 0, Hkv, D,
                0, k_stride, v_stride, n_pages, page_size, cache_layout, dtype, 0, 0, 0, stream);
}

int rope_kv_cache_append(const void* q, const void* k, const void* v, void* q_out, const float* rope_cs,
                         const int* positions, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         const long long* slots, int n_tokens, int Hq, int Hkv, int D, long long q_stride,
                         long long k_stride, long long v_stride, int n_pages, int page_size, int cache_layout, int dtype,
                         int n_pos, int rot_dim, int rope_layout, void* stream) {
  if (q == nullptr) return api_fail(ATTN_ERR_INVALID_ARG, "q must be a non-null device pointer");
  return append(q, k, v, q_out, rope_cs, positions, k_cache, v_cache, k_scale, v_scale, slots, n_tokens, Hq, Hkv, D,
                q_stride, k_stride, v_stride, n_pages, page_size, cache_layout, dtype, n_pos, rot_dim, rope_layout, stream);
}

int kv_cache_gather(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                    const int* page_table, const int* cu_seqlens, void* k_out, void* v_out, int n_seq, int total, int Hkv,
                    int D, int n_pages, int page_size, int max_pages, int cache_layout, int dtype, void* stream) {
  GatherParams p{};
  int rc = check_head_dim(D, true);
  if (rc == ATTN_OK) rc = check_cache(&p.cache, k_cache, v_cache, k_scale, v_scale, n_pages, page_size, Hkv, D, cache_layout, dtype);
  if (rc != ATTN_OK) return rc;
  if (n_seq < 1 || total < 1 || max_pages < 1)
    return api_fail(ATTN_ERR_INVALID_ARG, "need n_seq, total, max_pages >= 1 (got %d, %d, %d)", n_seq, total, max_pages);
  if (page_table == nullptr || cu_seqlens == nullptr || !aligned4(page_table) || !aligned4(cu_seqlens))
    return api_fail(ATTN_ERR_INVALID_ARG, "page_table and cu_seqlens must be non-null, 4-byte aligned device pointers");
  if (k_out == nullptr || v_out == nullptr || !api_aligned16(k_out) || !api_aligned16(v_out))
    return api_fail(ATTN_ERR_INVALID_ARG, "k_out and v_out must be non-null, 16-byte aligned device pointers");
  if (!rows_fit(total, Hkv)) return api_fail(ATTN_ERR_INVALID_ARG, "too many rows");
  const size_t cb = cache_bytes(p.cache, D), sb = scale_bytes(p.cache), ob = 2ull * total * Hkv * D;
  const Range outs[2] = {{k_out, ob}, {v_out, ob}};
  const Range ins[6] = {{k_cache, cb}, {v_cache, cb}, {k_scale, sb}, {v_scale, sb},
                        {page_table, 4ull * n_seq * max_pages}, {cu_seqlens, 4ull * n_seq + 4}};
  if ((rc = check_disjoint(outs, 2, ins, 6)) != ATTN_OK) return rc;
  if ((rc = api_err_words(&p.err_word)) != ATTN_OK) return rc;
  p.err_info = p.err_word + 1;
  p.page_table = page_table;
  p.cu_seqlens = cu_seqlens;
  p.k_out = k_out;
  p.v_out = v_out;
  p.n_seq = n_seq;
  p.total = total;
  p.max_pages = max_pages;
  const cudaError_t e = launch_cache_gather(p, D, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_fail(ATTN_ERR_CUDA, "cache read-back launch failed: %s", cudaGetErrorString(e));
  return api_ok();
}

size_t attn_decode_paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int page_size, int max_pages) {
  if (B < 1 || T < 1 || T > PAGED_MAX_DRAFT || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128) ||
      page_size < 1 || max_pages < 1)
    return 0;
  if (!paged_combines(page_size, max_pages)) return 0;
  return paged_workspace(paged_ctas(), paged_rows(Hq / Hkv * T), D);
}

int attn_decode_paged(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                      void* o, float* lse, const int* page_table, const int* ctx_lens, const int* q_lens,
                      const unsigned long long* tree_mask, void* workspace, size_t workspace_bytes, int B, int T, int Hq,
                      int Hkv, int D, int n_pages, int page_size, int max_pages, int cache_layout, int dtype, float scale,
                      void* stream) {
  CacheView c{};
  int rc = check_head_dim(D, false);
  if (rc == ATTN_OK) rc = check_cache(&c, k_cache, v_cache, k_scale, v_scale, n_pages, page_size, Hkv, D, cache_layout, dtype);
  if (rc != ATTN_OK) return rc;
  if (B < 1 || B > PAGED_MAX_BATCH)
    return api_fail(B < 1 ? ATTN_ERR_INVALID_ARG : ATTN_ERR_UNSUPPORTED, "B must be in [1, %d] (got %d)", PAGED_MAX_BATCH, B);
  if (T < 1 || T > PAGED_MAX_DRAFT)
    return api_fail(T < 1 ? ATTN_ERR_INVALID_ARG : ATTN_ERR_UNSUPPORTED, "T must be in [1, %d] (got %d)", PAGED_MAX_DRAFT, T);
  if (Hq < 1 || Hq > 65535 || Hq % Hkv != 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "Hq (%d) must be a positive multiple of Hkv (%d)", Hq, Hkv);
  if (!std::isfinite(scale) || scale < 0.f)
    return api_fail(ATTN_ERR_INVALID_ARG, "scale must be finite and >= 0 (0 selects 1/sqrt(D))");
  if (q == nullptr || o == nullptr || !api_aligned16(q) || !api_aligned16(o))
    return api_fail(ATTN_ERR_INVALID_ARG, "q and o must be non-null, 16-byte aligned device pointers");
  if (page_table == nullptr || ctx_lens == nullptr || !aligned4(page_table) || !aligned4(ctx_lens) || !aligned4(q_lens) ||
      !aligned4(lse) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return api_fail(ATTN_ERR_INVALID_ARG, "page_table and ctx_lens must be non-null; page_table, ctx_lens, q_lens and lse "
                    "4-byte, tree_mask 8-byte aligned");
  if (max_pages < 1 || static_cast<long long>(max_pages) * page_size > 0x7fff0000ll)
    return api_fail(ATTN_ERR_INVALID_ARG, "need max_pages >= 1 and max_pages * page_size < 2^31 (got %d)", max_pages);
  const long long tiles = (static_cast<long long>(max_pages) * page_size + 127) / 128;
  if ((tiles + 16) * B > 0x7fffffffll) return api_fail(ATTN_ERR_INVALID_ARG, "the page table spans too many keys");
  const int G = Hq / Hkv;
  if (G * static_cast<long long>(T) > 65535)
    return api_fail(ATTN_ERR_UNSUPPORTED, "(Hq / Hkv) * T = %lld query rows per key/value head, at most 65535",
                    G * static_cast<long long>(T));
  const int RB = paged_rows(G * T), row_tiles = (G * T + RB - 1) / RB;
  const int sms = paged_ctas(), group = row_tiles < sms ? row_tiles : sms, n_cta = sms / group;
  const size_t need = paged_combines(page_size, max_pages) ? paged_workspace(sms, RB, D) : 0;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need || !api_aligned16(workspace))
      return api_fail(ATTN_ERR_INVALID_ARG, "a 16-byte aligned workspace of %zu bytes is needed "
                      "(attn_decode_paged_workspace_bytes)", need);
  }
  const size_t cb = cache_bytes(c, D), sb = scale_bytes(c), qb = 2ull * B * T * Hq * D;
  const Range outs[3] = {{o, qb}, {lse, 4ull * B * Hq * T}, {need > 0 ? workspace : nullptr, need}};
  const Range ins[9] = {{q, qb}, {k_cache, cb}, {v_cache, cb}, {k_scale, sb}, {v_scale, sb},
                        {page_table, 4ull * B * max_pages}, {ctx_lens, 4ull * B}, {q_lens, 4ull * B},
                        {tree_mask, 8ull * B * T}};
  if ((rc = check_disjoint(outs, 3, ins, 9)) != ATTN_OK) return rc;
  PagedParams p{};
  if ((rc = api_err_words(&p.err_word)) != ATTN_OK) return rc;
  p.err_info = p.err_word + 1;
  CUtensorMap tk, tv;
  const bool fp8 = dtype == ATTN_FP8_E4M3;
  if ((rc = api_make_cache_map(&tk, c, k_cache, D, fp8)) != ATTN_OK) return rc;
  if ((rc = api_make_cache_map(&tv, c, v_cache, D, fp8)) != ATTN_OK) return rc;
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.page_table = page_table;
  p.ctx_lens = ctx_lens;
  p.q_lens = q_lens;
  p.tree_mask = tree_mask;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.v_cache = v_cache;
  p.page_stride = c.page_stride;
  p.head_stride = c.head_stride;
  p.tok_stride = c.tok_stride;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.g_magic = G == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + G - 1) / G);
  p.n_pages = n_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.row_tiles = row_tiles;
  p.lead = PAGED_LEAD;
  p.n_cta = n_cta;
  p.group_ctas = group;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_l = need > 0 ? p.ws_o + 2ll * sms * RB * D : nullptr;
  p.cuts = need > 0 ? reinterpret_cast<int4*>(p.ws_l + 2ll * sms * RB) : nullptr;
  const float sc = scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(D));
  p.c_log2 = sc * 1.4426950408889634f;
  p.spin_limit = api_spin_limit();
  const cudaError_t e = launch_attn_paged(tk, tv, p, D, fp8, need > 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_fail(ATTN_ERR_CUDA, "paged attention launch failed: %s", cudaGetErrorString(e));
  return api_ok();
}

}  // extern "C"
