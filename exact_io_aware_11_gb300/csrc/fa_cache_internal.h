// Launch descriptions of the rotary and cache entry points (fa_cache_api.cu)
// and the kernels behind them (fa_rotary.cu, fa_cache.cu, fa_cache_attn.cu, fa_cache_rows.cuh,
// fa_cache_tile.cuh, fa_cache_shared.cu, fa_cache_pages.cu).
#pragma once

#include "fa.h"
#include "fa_internal.h"

namespace fa {

// Element strides {batch, head, row} of one 16-bit [B, H, N, d] tensor.
struct RowStrides {
  long long b, h, n;
};

struct RotaryTensor {
  const uint16_t* x;
  uint16_t* y;
  RowStrides sx, sy;
};

struct RotaryLaunch {
  RotaryTensor t[2];  // queries, keys
  int B, Hq, Hk, N, d, r;
  int interleaved, fp16, inner;  // inner: a row's heads lie closer together than a head's rows
  float fcos, fsin;  // factor, and factor with the direction's sign
  const unsigned long long* turns;
  const int32_t* pos;
  long long pos_b, pos_n;
  int offset;
};
cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t stream);

// The page pool and a page table over it.
struct CacheView {
  uint8_t* code[2];  // K, V
  float* scale[2];
  int num_pages, H, page, d, log2_page;
  int int8;
  const int32_t* table;
  long long table_stride;
  int table_width;
};

struct CacheRows {
  CacheView c;
  uint16_t* x[2];  // k, v of the call
  RowStrides st;
  int B, N, fp16;
  const int32_t* start;
  const int32_t* count;
  int* status;
};
cudaError_t launch_cache_write(const CacheRows& a, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheRows& a, cudaStream_t stream);

struct CacheAttnLaunch {
  CUtensorMap tm[2];  // K's and V's codes as rows of d bytes, boxes of a page
  CacheView c;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  RowStrides sq, so;
  int B, Hq, N, G;  // G: query heads per cache head
  int fp16, causal;
  float scale_log2;
  const int32_t* kv_len;
  const int32_t* q_len;
  int* status;
  long long wait_limit;
  uint8_t* ws;
  size_t ws_bytes;
};
cudaError_t launch_cache_attention(const CacheAttnLaunch& a, cudaStream_t stream);
size_t cache_attention_workspace(int B, int HK, int G, int N, int d, int page, int table_width);
constexpr int kSharedGroups = 2048;  // groups of a call with shared prefixes
cudaError_t launch_shared_attention(const CacheAttnLaunch& a, const int32_t* prefix_of, const int32_t* prefix_len, int groups,
                                    cudaStream_t stream);
size_t shared_attention_workspace(int B, int HK, int G, int N, int d, int page, int table_width, int groups);

constexpr int kPageTableRows = 16384;  // at most
// A page table with the counts of its pages' users (fa_page_table).
struct PageTable {
  int* entry;
  long long stride;
  int rows, width;
  int* refs;
  int num_pages, page;
};

constexpr int kCopyLayers = 64;  // layers of a launch
struct PageCopyLaunch {
  const int* src;
  const int* dst;
  const int* count;  // moves (device), nullptr: n
  int n, num_pages, H, layers, piece;
  long long page_bytes;  // codes of a page, K or V
  int* status;
  long long wait_limit;
  struct Layer {
    uint8_t* code[2];
    float* scale[2];
  } layer[kCopyLayers];
};
// a: src, dst, count, n, status, wait_limit; the rest comes from the caches.
cudaError_t launch_page_copy(PageCopyLaunch a, const fa_cache* caches, int layers, cudaStream_t stream);

struct PageForkLaunch {
  PageTable t;
  const int* parent;
  const int* keep;
  int* status;
  int log2_cols;  // of a CTA
};
cudaError_t launch_page_fork(PageForkLaunch a, cudaStream_t stream);

struct PageReserveLaunch {
  PageTable t;
  const int* start;
  const int* count;
  int tokens;  // of every row, where count is nullptr
  int* ok;
  int* status;
  // workspace
  int* moves;  // pages to be copied
  int* src;    // [rows]
  int* dst;
  int* list;   // free pages
};
size_t reserve_workspace(int rows, int width, int num_pages);
cudaError_t launch_page_reserve(PageReserveLaunch a, const fa_cache* caches, int layers, uint8_t* ws, cudaStream_t stream);

struct PageCompactLaunch {
  PageTable t;
  int* where;
  int* live;
  int* status;
  // workspace
  int* moves;
  int* src;
  int* dst;
};
size_t compact_workspace(int num_pages);
cudaError_t launch_page_compact(PageCompactLaunch a, const fa_cache* caches, int layers, uint8_t* ws, cudaStream_t stream);

bool encode_code_rows(CUtensorMap* map, const void* base, long long rows, int d, int box_rows);

// Records a page table entry out of range (fa_device_status).
static __device__ __noinline__ void report_bad_page(int* status) {
  atomicCAS(status, FA_OK, FA_ERR_BAD_PAGE);
}

}  // namespace fa
