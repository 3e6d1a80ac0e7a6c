// cache.h -- declarations shared by the C-ABI layer of the paged key/value cache (api_cache.cu)
// and its kernels: rotary positions, cache write and read-back, attention over the cache.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace ea46 {

// A paged cache of keys and values.  Row (page, head, offset) of D elements starts at element
// page * page_stride + head * head_stride + offset * tok_stride; the scales of an E4M3 cache are
// [n_pages, Hkv, page_size] fp32.
struct CacheView {
  void* k;
  void* v;
  float* k_scale;       // nullptr: bf16 rows
  float* v_scale;
  long long page_stride, head_stride, tok_stride;   // elements
  int n_pages, page_size, Hkv;
};

// Rotation of the first `rot` elements of rows of D; cs [n_pos, rot / 2, 2] (cos, sin).
struct RopeParams {
  const float* cs;      // nullptr: no rotation
  const int* pos;       // [n_tokens], or nullptr: token index modulo pos_wrap
  int pos_wrap;
  int n_pos, rot;
  float sin_sign;       // -1: the transposed rotation (gradient)
};

struct RopeApplyParams {
  const void* x;        // bf16 rows: token t, head h at t * x_stride + h * D
  void* out;
  long long x_stride, out_stride;                   // elements
  int n_tokens, H;
  RopeParams rope;
  int* err_word;
  int* err_info;
};

struct AppendParams {
  const void* q;        // nullptr: keys and values only
  const void* k;
  const void* v;
  void* q_out;          // [n_tokens, Hq, D] bf16
  long long q_stride, k_stride, v_stride;           // elements between tokens
  const long long* slots;                           // [n_tokens] page * page_size + offset, < 0: none
  int n_tokens, Hq;
  unsigned long long kv_step;                       // blocks for keys and values, of 2^32 (set by the launch)
  CacheView cache;
  RopeParams rope;
  int* err_word;
  int* err_info;
};

struct GatherParams {
  CacheView cache;
  const int* page_table;                            // [n_seq, max_pages]
  const int* cu_seqlens;                            // [n_seq + 1]
  void* k_out;          // [total, Hkv, D] bf16
  void* v_out;
  int n_seq, total, max_pages;
  int* err_word;
  int* err_info;
};

cudaError_t launch_rope_apply(const RopeApplyParams& p, int D, bool half, cudaStream_t st);
cudaError_t launch_cache_append(const AppendParams& p, int D, bool half, cudaStream_t st);
cudaError_t launch_cache_gather(const GatherParams& p, int D, cudaStream_t st);

enum RopeScaling { ROPE_NONE = 0, ROPE_LINEAR = 1, ROPE_NTK = 2, ROPE_YARN = 3 };
cudaError_t launch_rope_scaled_table(float* cs, int n_pos, int rot, double base, int scaling, double factor,
                                     double original_length, cudaStream_t st);

// Attention of T query tokens per sequence over the cache.
struct PagedParams {
  const void* q;        // [B, T, Hq, D] bf16
  void* o;              // [B, T, Hq, D] bf16
  float* lse;           // [B, Hq, T] fp32 or nullptr
  const int* page_table;                            // [B, max_pages]
  const int* ctx_lens;  // [B]
  const int* q_lens;    // [B] or nullptr: T
  const unsigned long long* tree_mask;              // [B, T] or nullptr: chain
  const float* k_scale; // E4M3: [n_pages, Hkv, page_size]
  const float* v_scale;
  const void* v_cache;  // bf16: read element by element for drafted rows that are not finite
  long long page_stride, head_stride, tok_stride;   // elements
  float* ws_o;          // [slots][RB][D] partial outputs
  float* ws_l;          // [slots][RB] partial lse, log2 units
  int4* cuts;           // [n_cta] (parts, sequence, key/value head, q_len) of the units to merge; nullptr: none
  int B, T, Hq, Hkv, G;
  uint32_t g_magic;     // ceil(2^32 / G), 0 for G = 1
  int n_pages, page_size, max_pages;
  int row_tiles;        // ceil(G * T / RB)
  int lead;             // list entries a change of units costs (paged.cuh)
  int n_cta;            // groups of CTAs that share the key tiles out; a group has one CTA per row tile,
  int group_ctas;       // at most group_ctas
  float c_log2;         // softmax scale * log2(e)
  long long spin_limit;
  int* err_word;
  int* err_info;
};

constexpr int PAGED_MAX_BATCH = 1024;
constexpr int PAGED_MAX_DRAFT = 64;

// Query rows per work unit for R = G * T packed rows.
constexpr int PAGED_TREE_ROWS = 128;
constexpr int paged_rows(int R) {
  return R <= 8 ? 8 : (R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : PAGED_TREE_ROWS)));
}

// List entries (128-key tiles) that a change of units is taken to cost.  Measured with 0, 2, 3, 4 and 6: trees
// of 8 over long e4m3 contexts 92.2, 90.3, 89.4, 88.3, 87.8 us, trees of 32 bf16 50.0, 49.1, 48.3, 47.8, 47.5,
// 30 e4m3 sequences of up to 2000 keys 25.8, 25.5, 25.2, 24.9, 25.1, bf16 units of 64 tiles 72.2, 72.2, 72.8, 73.4,
// 73.6.
constexpr int PAGED_LEAD = 4;

// tk, tv: the cache as (D, page_size, Hkv, n_pages) with a box of one swizzle panel x
// min(page_size, 128) rows.
cudaError_t launch_attn_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int D, bool fp8,
                              bool combine, cudaStream_t st);

cudaError_t launch_attn_tree(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int D, bool fp8,
                             cudaStream_t st);
cudaError_t launch_attn_lanes(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, int D, bool fp8,
                              cudaStream_t st);

// Launch a kernel that may become resident while the one before it on the stream ends; it waits for that
// one's completion (griddepcontrol.wait) before it reads or writes anything.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                              const A&... a) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a...);
}

// Shared pieces of the C-ABI layer (api.cu).
int api_fail(int code, const char* fmt, ...);
int api_ok();
int api_err_words(int** out);
long long api_spin_limit();
bool api_aligned16(const void* p);
bool api_overlap(const void* a, size_t na, const void* b, size_t nb);
int api_make_cache_map(CUtensorMap* m, const CacheView& c, const void* ptr, int D, bool fp8);

}  // namespace ea46
