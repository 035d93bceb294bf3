// history.h -- parameters and launchers of the history-cache kernels: per-head norm and rotation, the paged 4-bit
// cache's append and read, and the attention over it.
#pragma once

#include "sm100.cuh"

namespace rocs {

// ---------------------------------------------------------------- per-head norm + rotation
struct NormRopeSide {
  const void* x;
  void* out;
  const int32_t* pos;  // [n], or null without rotation
  const float* gamma;  // [dh] or null
  const float* beta;   // [dh] or null
  int64_t ld_x, ld_out;
  int n, heads;
};
struct NormRopeParams {
  NormRopeSide side[2];  // queries, keys
  int64_t warps0, warps;  // warps of side 0, of both
  const float* rope;      // [max_pos, rot] or null
  int max_pos, rot, interleaved, norm;
  float eps;
  WsHeader* ws;
};
cudaError_t launch_norm_rope(const NormRopeParams& p, int dh, bool f32, int unroll, cudaStream_t st);
// rows that a warp of the kernels below holds at a time; with few of them (less than the device's warps) a warp takes one
// such set, so that as many SMs as possible work on a small call, otherwise several, so that more loads are in flight
inline int rows_per_warp(int64_t dh) { return (int)(512 / dh); }
inline int unroll_for(int64_t rows, int64_t dh, int sms, int most) { return rows >= (int64_t)sms * 32 * rows_per_warp(dh) ? most : 1; }
constexpr int kNormSets = 2, kAppendSets = 2, kReadSets = 4;
cudaError_t launch_rope_table(float* table, int64_t max_pos, int rot, double base, cudaStream_t st);

// ---------------------------------------------------------------- the paged 4-bit cache
// codes [pages, heads, page, dh/2] bytes, scale [pages, heads, page, 2] bf16 (step, minimum)
struct CacheQ4 {
  uint8_t* codes[2];          // K, V
  __nv_bfloat162* scale[2];
  int pages, page_log2, heads;
};
struct CacheMoveParams {  // append and read
  CacheQ4 c;
  void* x[2];              // append: k, v in;  read: k, v out
  int64_t ld[2];           // token stride in elements
  const int32_t* tok_off;  // [R+1]
  const int32_t* base;     // [R]
  const int32_t* table;    // [R, max_pages]
  const int32_t* pos;      // [T] or null
  const float* rope;
  int R, max_pages, max_pos, rot, interleaved;
  int64_t rows, warps;     // T * heads; warps for one of keys and values
  WsHeader* ws;
};
cudaError_t launch_cache_append(const CacheMoveParams& p, int dh, bool f32, int unroll, cudaStream_t st);
cudaError_t launch_cache_read(const CacheMoveParams& p, int dh, int unroll, cudaStream_t st);

// ---------------------------------------------------------------- attention over the cache
struct CacheAttnParams {
  CacheQ4 c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                // or null
  const int32_t* cand_off;   // [R+1]
  const int32_t* seq_len;    // [R]
  const int32_t* table;      // [R, max_pages]
  const int32_t* key_limit;  // [C] or null
  int64_t q_ld;              // elements from one query token to the next
  int R, C, q_tokens, H, G;  // G: query heads to a key head
  int max_pages, capacity;   // capacity: slots that a row of the page table reaches
  int rows_lo, rows_hi;      // requests with rows_lo < rows (of one key head) <= rows_hi are this launch's
  float scale_log2;          // softmax scale * log2(e)
  float* part;               // partial results, two per CTA
  int* cnt;                  // [CTAs], zeroed before the launch
  WsHeader* ws;
};
constexpr int kFewRows = 16;   // rows of a unit of the kernel for few rows, at most
size_t cache_few_part_bytes(int dh);
int cache_few_grid(int sms);
struct CacheManyParams {
  CUtensorMap tm_q;          // Q viewed as [tokens][H][dh], box {64, G, 128 / G}
  CacheAttnParams a;
  int min_share;             // blocks of keys in a CTA's run, at least
  long long wait_limit_ns;
};
size_t cache_many_part_bytes(int dh);  // partial results of one unit
cudaError_t launch_cache_many(const CacheManyParams& p, int dh, int grid, cudaStream_t st);
// rows: the most that a key head of a request of this launch has
cudaError_t launch_cache_few(const CacheAttnParams& p, int dh, int rows, int grid, cudaStream_t st);

}  // namespace rocs
