// Launch descriptions of the rotary and cache entry points (fa_cache_api.cu)
// and the kernels behind them (fa_rotary.cu, fa_cache.cu, fa_cache_attn.cu, fa_cache_tile.cuh).
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

bool encode_code_rows(CUtensorMap* map, const void* base, long long rows, int d, int box_rows);

// Records a page table entry out of range (fa_device_status).
static __device__ __noinline__ void report_bad_page(int* status) {
  atomicCAS(status, FA_OK, FA_ERR_BAD_PAGE);
}

}  // namespace fa
