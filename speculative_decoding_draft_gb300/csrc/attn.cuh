// Arguments and shared device code of the operators around a ragged verification step: norm and
// rotation of heads, the paged cache in 4 bits, attention over it and the logits' penalties.
//
// The cache.  An element is kept as e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) with one e4m3 scale
// for 16 dimensions and a power of two for the whole cache.  element * scale has 2 + 4 significant
// bits and is a multiple of 2^-10 below 2^12, so it is exact in fp16: what the attention multiplies
// is what the cache holds, with no rounding in between.  The unit of the layout is a tile of 16
// tokens of one head, 18 D contiguous bytes (keys, values, key scales, value scales), so that one
// bulk copy brings a tile and every tile of a page is alike whatever the page size.  Keys lie token
// by token; values lie in 8 chunks of D/8 dimensions with the 8 tokens of a half-tile side by side
// in each: a thread of the product P V finds its tokens' pieces of one chunk next to each other.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "dspark_internal.cuh"

namespace dspark {

constexpr int kTileTokens = 16;

__host__ __device__ constexpr int tile_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int tile_k(int D, int t) { return t * (D / 2); }
__host__ __device__ constexpr int tile_v(int D, int t, int chunk) {
  return 8 * D + (D / 16) * (64 * (t >> 3) + 8 * chunk + (t & 7));
}
__host__ __device__ constexpr int tile_ks(int D, int t, int c) { return 16 * D + t * (D / 16) + c; }
__host__ __device__ constexpr int tile_vs(int D, int t, int c) {
  return 17 * D + (t >> 3) * (D / 2) + 8 * c + (t & 7);
}

struct HeadsArgs {
  const void *q, *k, *v;              // [rows, heads, D] with strides in elements
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;
  void *q_out, *k_out;                // contiguous [rows, heads, D]
  const void *q_weight, *k_weight;    // [D] or null
  const int32_t *positions;           // [rows] or null (append: the rows' places in the cache)
  const unsigned long long *turns;    // [rot / 2] or null: no rotation
  int64_t rows;
  int Hq, Hkv, D, rot, interleaved, dtype;
  float gain, eps;
  // append
  uint8_t *cache;
  int64_t pages, max_pages, B;
  int page_size;
  float k_inv, v_inv, k_unit, v_unit;   // the cache's scales and their reciprocals, powers of two
  const int32_t *row_off, *kv_len, *table;
  int32_t *dev_status;
};

struct CacheReadArgs {
  const uint8_t *cache;
  int64_t pages, max_pages, B, rows;
  int Hkv, D, page_size;
  const int32_t *row_off, *kv_len, *table;
  uint8_t *k, *ks, *v, *vs;
  int32_t *dev_status;
};

struct AttendArgs {
  const void *q;                      // [rows, Hq, D] with strides in elements
  int64_t q_row, q_head;
  void *out;                          // contiguous [rows, Hq, D]
  float *lse;                         // [rows, Hq] or null
  const uint8_t *cache;
  int64_t pages, max_pages, B, rows;
  int Hq, Hkv, D, page_size, group, causal, window, max_rows, dtype;
  float scale_log2, out_scale;        // on q.k in units of log2, on the output
  float *partial;                     // workspace of the split form
  const int32_t *row_off, *kv_len, *table;
  int32_t *dev_status;
};

struct PenalizeArgs {
  const void *logits;
  void *out;                          // may be `logits`
  int64_t rows, B, V, hist_cap, draft_cap, bias_cap, mask_words;
  int dtype;
  const int32_t *row_off, *hist, *hist_len, *prompt_len, *draft_tok, *bias_tok;
  const uint32_t *mask;
  const float *repetition, *presence, *frequency, *bias_val;
  int32_t *dev_status;
};

cudaError_t launch_norm_rope(const HeadsArgs &a, cudaStream_t s);
cudaError_t launch_cache_append(const HeadsArgs &a, cudaStream_t s);
cudaError_t launch_cache_read(const CacheReadArgs &a, cudaStream_t s);
cudaError_t launch_attend(const AttendArgs &a, cudaStream_t s, int sms);
// Bytes of AttendArgs::partial that a call needs; len: tokens that its page table can name.
int64_t attend_workspace_bytes(int64_t B, int Hkv, int group, int D, int64_t len, int64_t max_rows, int64_t rows, int sms);
cudaError_t launch_penalize(const PenalizeArgs &a, cudaStream_t s, int sms);

// The status word as a kernel finds it, through the SM's first-level cache: a warp a row means thousands of
// warps that ask for the same word, and from the second level these answers come one after the other (the
// read-back of 8190 rows 7.1 us, 8.2 so).
__device__ __forceinline__ int status_on_entry(const int32_t *status) {
  int s;
  asm volatile("ld.global.ca.s32 %0, [%1];" : "=r"(s) : "l"(status) : "memory");
  return s;
}

// A launch in clusters as a programmatic dependent of what precedes it in the stream, so that its CTAs
// stand ready when that ends: such a kernel waits (grid_dep_wait) before its first access to global
// memory and lets the next one in (grid_dep_launch) at once.  For the attention, which needs this form
// of launch for its clusters and its joining kernel: a single token's call takes 7.9 us (10.2 without).
// The other operators' plain launches cost the host 1 us less, which is what bounds their small calls.
template <class... P>
cudaError_t launch_next(void (*kernel)(P...), int64_t grid, int threads, int smem, int cluster, cudaStream_t s, P... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The request of a row: the last r with row_off[r] <= row, by one warp, 64 probes a step (two steps for
// 2048 requests, where halving would take eleven dependent loads).
__device__ __forceinline__ int64_t request_of_row(const int32_t *row_off, int64_t B, int64_t row, int lane) {
  int lo = 0, len = (int)B;
  while (len > 1) {
    const int step = (len + 63) >> 6, at = lane * step, at2 = at + 32 * step;
    const int32_t x = at < len ? row_off[lo + at] : INT32_MAX, y = at2 < len ? row_off[lo + at2] : INT32_MAX;
    const uint32_t m = __ballot_sync(0xffffffffu, at < len && x <= row);
    const uint32_t m2 = __ballot_sync(0xffffffffu, at2 < len && y <= row);
    const int last = m2 ? 63 - __clz(m2) : (m ? 31 - __clz(m) : 0);
    const int end = lo + len;
    lo += last * step;
    len = min(end - lo, step);
  }
  return lo;
}

// A row's place in the cache, in two steps so that what needs the position alone need not wait for the
// page: find_row looks the position up and starts the load of the page's id, place_row checks that.
// Both return false for rows past row_off[B] and for inconsistent arguments, which they record in the
// status word.  Loads that do not depend on one another are issued together.
struct RowPlace {
  int64_t pos, tile;   // token position; index of its tile of head 0 in units of tiles
  int32_t page;
  int in_page, t;      // its tile in the page, token in the tile
};
__device__ __forceinline__ bool find_row(const int32_t *row_off, const int32_t *kv_len, const int32_t *table, int64_t B,
                                         int64_t max_pages, int page_size, int64_t row, int lane, int32_t *status,
                                         RowPlace *p) {
  const int64_t r = request_of_row(row_off, B, row, lane);
  const int64_t a = row_off[r], b = row_off[r + 1], all = row_off[B], len = kv_len[r];
  if (row < a || row >= b) {
    if (row < all) set_status(status, DSPARK_ERR_OFFSETS);
    return false;
  }
  const int64_t pos = len - b + row;
  if (pos < 0 || pos >= max_pages * page_size) {
    set_status(status, DSPARK_ERR_LENGTHS);
    return false;
  }
  // positions are below 2^31: a 32-bit division, the only one
  const uint32_t tile = (uint32_t)pos / kTileTokens, per = (uint32_t)page_size / kTileTokens, at = tile / per;
  p->page = table[r * max_pages + at];
  p->pos = pos;
  p->in_page = (int)(tile - at * per);
  p->t = (int)((uint32_t)pos % kTileTokens);
  return true;
}
__device__ __forceinline__ bool place_row(int64_t pages, int page_size, int Hkv, int32_t *status, RowPlace *p) {
  if (p->page < 0 || p->page >= pages) {
    set_status(status, DSPARK_ERR_PAGES);
    return false;
  }
  p->tile = p->page * ((int64_t)Hkv * (page_size / kTileTokens)) + p->in_page;
  return true;
}

// 8 elements of a row as floats, and back.
template <int DT>
struct Elem;
template <>
struct Elem<DSPARK_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float to(T x) { return __bfloat162float(x); }
  static __device__ __forceinline__ T from(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<DSPARK_F16> {
  using T = __half;
  static __device__ __forceinline__ float to(T x) { return __half2float(x); }
  static __device__ __forceinline__ T from(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<DSPARK_F32> {
  using T = float;
  static __device__ __forceinline__ float to(T x) { return x; }
  static __device__ __forceinline__ T from(float x) { return x; }
};

template <int DT>
struct alignas(16) Eight {
  typename Elem<DT>::T e[8];
};

}  // namespace dspark
