// C-ABI of the rotary and cache entry points (declared in include/fa.h):
// argument validation and dispatch. Nothing is launched and nothing written
// when an argument is refused.
#include <climits>
#include <cmath>
#include <cstring>

#include "fa.h"
#include "fa_cache_internal.h"

namespace fa {
namespace {

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool ranges_meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

// A [B, H, N, d] tensor of 16-bit elements as a call gives it.
struct Tensor {
  const void* p;
  int B, H, N, d;
  Strides st;
  size_t bytes() const { return span_bytes(B, H, N, d, st, 2); }
  RowStrides rows() const { return RowStrides{st.b, st.h, st.n}; }
};

int make_tensor(const void* p, int B, int H, int N, int d, const int64_t* s, Tensor* t) {
  if (p == nullptr || !aligned(p, 16)) return FA_ERR_INVALID_ARG;
  *t = Tensor{p, B, H, N, d, Strides{}};
  const bool dense = s[0] == 0 && s[1] == 0 && s[2] == 0;
  if (!(dense ? dense_strides(B, H, N, d, &t->st) : make_strides(B, H, N, d, s[0], s[1], s[2], &t->st)))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Whether two tensors of a call, which differ in their heads at most, may share an element: exactly
// where their strides are the same (of axes that both step), by their address ranges otherwise.
bool tensors_meet(const Tensor& a, const Tensor& b) {
  Strides st = a.st;
  if (a.H == 1) st.h = b.st.h;
  if ((a.B == 1 || st.b == b.st.b) && (b.H == 1 || st.h == b.st.h) && (a.N == 1 || st.n == b.st.n))
    return strided_overlap(a.p, b.p, a.B, a.H, b.H, a.N, a.d, st);
  return ranges_meet(a.p, a.bytes(), b.p, b.bytes());
}
bool same_place(const Tensor& a, const Tensor& b) {
  return a.p == b.p && a.st.b == b.st.b && a.st.h == b.st.h && a.st.n == b.st.n;
}

int check_sizes(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || B > 65535 || H > 65535) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int rotary(const void* q, void* q_out, const void* k, void* k_out, int B, int Hq, int Hk, int N, int d,
           const fa_rotary_options* opt, cudaStream_t stream, bool back) {
  if (opt == nullptr || Hk < 0 || Hk > 65535) return FA_ERR_INVALID_ARG;
  int st = check_sizes(B, Hq, N, d);
  if (st != FA_OK) return st;
  if ((k == nullptr) != (Hk == 0) || (k_out == nullptr) != (Hk == 0)) return FA_ERR_INVALID_ARG;
  if (opt->rotary_dim < 2 || opt->rotary_dim > d || (opt->rotary_dim & 1)) return FA_ERR_INVALID_ARG;
  if ((opt->interleaved != 0 && opt->interleaved != 1) || !std::isfinite(opt->factor)) return FA_ERR_INVALID_ARG;
  if (opt->dtype != FA_BF16 && opt->dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (opt->turns == nullptr || !aligned(opt->turns, 8)) return FA_ERR_INVALID_ARG;
  if (!aligned(opt->positions, 4) || opt->pos_stride_b < 0 || opt->pos_stride_n < 0) return FA_ERR_INVALID_ARG;
  const size_t turns_bytes = static_cast<size_t>(opt->rotary_dim) / 2 * 8;
  const long long lim = 1LL << 31;  // their products with B and N fit 64 bits
  if (opt->pos_stride_b > lim || opt->pos_stride_n > lim) return FA_ERR_INVALID_ARG;
  if (opt->positions == nullptr && opt->offset > INT_MAX - (N - 1)) return FA_ERR_INVALID_ARG;
  const size_t pos_bytes = static_cast<size_t>((B - 1) * opt->pos_stride_b + (N - 1) * opt->pos_stride_n + 1) * 4;
  Tensor in[2], out[2];
  const int tensors = Hk > 0 ? 2 : 1;
  const int64_t* sin[2] = {opt->q_stride, opt->k_stride};
  const int64_t* sout[2] = {opt->q_out_stride, opt->k_out_stride};
  for (int i = 0; i < tensors; ++i) {
    if ((st = make_tensor(i ? k : q, B, i ? Hk : Hq, N, d, sin[i], &in[i])) != FA_OK) return st;
    if ((st = make_tensor(i ? k_out : q_out, B, i ? Hk : Hq, N, d, sout[i], &out[i])) != FA_OK) return st;
  }
  for (int i = 0; i < tensors; ++i) {
    for (int j = 0; j < tensors; ++j)
      if (!(i == j && same_place(out[i], in[j])) && tensors_meet(out[i], in[j])) return FA_ERR_INVALID_ARG;
    if (ranges_meet(out[i].p, out[i].bytes(), opt->turns, turns_bytes) ||
        ranges_meet(out[i].p, out[i].bytes(), opt->positions, pos_bytes))
      return FA_ERR_INVALID_ARG;
  }
  if (tensors == 2 && tensors_meet(out[0], out[1])) return FA_ERR_INVALID_ARG;
  int* status = nullptr;
  if ((st = device_status_word(&status)) != FA_OK) return st;
  RotaryLaunch a;
  std::memset(&a, 0, sizeof(a));
  for (int i = 0; i < tensors; ++i)
    a.t[i] = RotaryTensor{static_cast<const uint16_t*>(in[i].p),
                          const_cast<uint16_t*>(static_cast<const uint16_t*>(out[i].p)), in[i].rows(), out[i].rows()};
  a.B = B;
  a.Hq = Hq;
  a.Hk = Hk;
  a.N = N;
  a.d = d;
  a.r = opt->rotary_dim;
  a.interleaved = opt->interleaved;
  a.fp16 = opt->dtype == FA_FP16;
  a.inner = Hq > 1 && N > 1 && in[0].st.h < in[0].st.n;
  a.fcos = opt->factor;
  a.fsin = back ? -opt->factor : opt->factor;
  a.turns = reinterpret_cast<const unsigned long long*>(opt->turns);
  a.pos = opt->positions;
  a.pos_b = opt->pos_stride_b;
  a.pos_n = opt->pos_stride_n;
  a.offset = opt->offset;
  return launch_rotary(a, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The pool's codes of one tensor in bytes, and the checks of a cache.
size_t pool_bytes(const fa_cache* c) {
  return static_cast<size_t>(c->num_pages) * c->H * c->page_size * c->d;
}
size_t scale_bytes(const fa_cache* c) { return static_cast<size_t>(c->num_pages) * c->H * 4; }

int check_cache_sizes(const fa_cache* c) {
  if (c == nullptr || c->num_pages < 1 || c->H < 1 || c->H > 65535) return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return FA_ERR_UNSUPPORTED;
  if (c->format != FA_CACHE_E4M3 && c->format != FA_CACHE_INT8) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int check_cache(const fa_cache* c, const int32_t* table, int64_t table_stride, int width, CacheView* v) {
  const int st = check_cache_sizes(c);
  if (st != FA_OK) return st;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !table) return FA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(table, 4))
    return FA_ERR_INVALID_ARG;
  if (width < 1 || table_stride < 0 || table_stride > (1LL << 40) ||
      static_cast<long long>(width) * c->page_size > INT_MAX - 1024)
    return FA_ERR_INVALID_ARG;
  v->code[0] = static_cast<uint8_t*>(c->k);
  v->code[1] = static_cast<uint8_t*>(c->v);
  v->scale[0] = c->k_scale;
  v->scale[1] = c->v_scale;
  v->num_pages = c->num_pages;
  v->H = c->H;
  v->page = c->page_size;
  v->d = c->d;
  v->log2_page = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  v->int8 = c->format == FA_CACHE_INT8;
  v->table = table;
  v->table_stride = table_stride;
  v->table_width = width;
  return FA_OK;
}

// Whether [p, p + n) meets a part of the cache.
bool meets_cache(const fa_cache* c, const void* p, size_t n) {
  return ranges_meet(p, n, c->k, pool_bytes(c)) || ranges_meet(p, n, c->v, pool_bytes(c)) ||
         ranges_meet(p, n, c->k_scale, scale_bytes(c)) || ranges_meet(p, n, c->v_scale, scale_bytes(c));
}
// Whether the cache's own parts share memory.
bool cache_meets_itself(const fa_cache* c) {
  return ranges_meet(c->k, pool_bytes(c), c->v, pool_bytes(c)) ||
         ranges_meet(c->k, pool_bytes(c), c->k_scale, scale_bytes(c)) ||
         ranges_meet(c->k, pool_bytes(c), c->v_scale, scale_bytes(c)) ||
         ranges_meet(c->v, pool_bytes(c), c->k_scale, scale_bytes(c)) ||
         ranges_meet(c->v, pool_bytes(c), c->v_scale, scale_bytes(c)) ||
         ranges_meet(c->k_scale, scale_bytes(c), c->v_scale, scale_bytes(c));
}
size_t table_bytes(int B, int64_t stride, int width) {
  return static_cast<size_t>((B - 1) * stride + width) * 4;
}

int cache_rows(const fa_cache* cache, const void* k, const void* v, int B, int N, const fa_cache_range* range,
               cudaStream_t stream, bool write) {
  if (range == nullptr) return FA_ERR_INVALID_ARG;
  CacheRows a;
  std::memset(&a, 0, sizeof(a));
  int st = check_cache(cache, range->page_table, range->table_stride, range->table_width, &a.c);
  if (st != FA_OK) return st;
  if ((st = check_sizes(B, cache->H, N, cache->d)) != FA_OK) return st;
  if (range->dtype != FA_BF16 && range->dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (!aligned(range->start, 4) || !aligned(range->count, 4)) return FA_ERR_INVALID_ARG;
  Tensor t[2];
  if ((st = make_tensor(k, B, cache->H, N, cache->d, range->stride, &t[0])) != FA_OK) return st;
  if ((st = make_tensor(v, B, cache->H, N, cache->d, range->stride, &t[1])) != FA_OK) return st;
  const size_t len = static_cast<size_t>(B) * 4, tab = table_bytes(B, range->table_stride, range->table_width);
  for (const Tensor& x : t) {
    if (meets_cache(cache, x.p, x.bytes())) return FA_ERR_INVALID_ARG;
    if (!write && (ranges_meet(x.p, x.bytes(), range->page_table, tab) ||
                   ranges_meet(x.p, x.bytes(), range->start, len) || ranges_meet(x.p, x.bytes(), range->count, len)))
      return FA_ERR_INVALID_ARG;
  }
  if (write) {
    if (cache_meets_itself(cache) || meets_cache(cache, range->page_table, tab) ||
        meets_cache(cache, range->start, len) || meets_cache(cache, range->count, len))
      return FA_ERR_INVALID_ARG;
  } else if (tensors_meet(t[0], t[1])) {
    return FA_ERR_INVALID_ARG;
  }
  if ((st = device_status_word(&a.status)) != FA_OK) return st;
  a.x[0] = const_cast<uint16_t*>(static_cast<const uint16_t*>(k));
  a.x[1] = const_cast<uint16_t*>(static_cast<const uint16_t*>(v));
  a.st = t[0].rows();
  a.B = B;
  a.N = N;
  a.fp16 = range->dtype == FA_FP16;
  a.start = range->start;
  a.count = range->count;
  return (write ? launch_cache_write(a, stream) : launch_cache_read(a, stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Sizes of a call of the attention that the kernels count in 32 bits.
int check_attention_sizes(const fa_cache* cache, int B, int Hq, int N, int table_width) {
  const int st = check_cache_sizes(cache);
  if (st != FA_OK) return st;
  if (B < 1 || B > 65535 || Hq < 1 || Hq > 65535 || N < 1 || table_width < 1 || Hq % cache->H != 0)
    return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(table_width) * cache->page_size > INT_MAX - 1024) return FA_ERR_INVALID_ARG;
  // rows of the pool are coordinates of its tensor map
  if (static_cast<long long>(cache->num_pages) * cache->H > INT_MAX / cache->page_size) return FA_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(N) * (Hq / cache->H);
  if (rows > INT_MAX - 1024 || static_cast<long long>(B) * (rows / 8 + 1) > INT_MAX - 1024) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_rotary_fwd(const void* q, void* q_out, const void* k, void* k_out, int B, int Hq, int Hk, int N, int d,
                  const fa_rotary_options* opt, struct CUstream_st* stream) {
  return rotary(q, q_out, k, k_out, B, Hq, Hk, N, d, opt, stream, false);
}

int fa_rotary_bwd(const void* dq_out, void* dq, const void* dk_out, void* dk, int B, int Hq, int Hk, int N, int d,
                  const fa_rotary_options* opt, struct CUstream_st* stream) {
  return rotary(dq_out, dq, dk_out, dk, B, Hq, Hk, N, d, opt, stream, true);
}

int fa_cache_write(const fa_cache* cache, const void* k, const void* v, int B, int N, const fa_cache_range* range,
                   struct CUstream_st* stream) {
  return cache_rows(cache, k, v, B, N, range, stream, true);
}

int fa_cache_read(const fa_cache* cache, void* k, void* v, int B, int N, const fa_cache_range* range,
                  struct CUstream_st* stream) {
  return cache_rows(cache, k, v, B, N, range, stream, false);
}

size_t fa_cache_attention_workspace_bytes(const fa_cache* cache, int B, int Hq, int N, int table_width) {
  if (check_attention_sizes(cache, B, Hq, N, table_width) != FA_OK) return 0;
  return cache_attention_workspace(B, cache->H, Hq / cache->H, N, cache->d, cache->page_size, table_width);
}

int fa_cache_attention(const void* q, void* o, float* lse, const fa_cache* cache, int B, int Hq, int N,
                       const fa_cache_attention_options* opt, void* workspace, size_t workspace_bytes,
                       struct CUstream_st* stream) {
  if (opt == nullptr) return FA_ERR_INVALID_ARG;
  CacheAttnLaunch a;
  std::memset(&a, 0, sizeof(a));
  int st = check_cache(cache, opt->page_table, opt->table_stride, opt->table_width, &a.c);
  if (st != FA_OK) return st;
  if ((st = check_attention_sizes(cache, B, Hq, N, opt->table_width)) != FA_OK) return st;
  if (opt->dtype != FA_BF16 && opt->dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (opt->causal != 0 && opt->causal != 1) return FA_ERR_INVALID_ARG;
  const float scale_log2 = opt->scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2) || !(opt->scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (opt->kv_len == nullptr || !aligned(opt->kv_len, 4) || !aligned(opt->q_len, 4)) return FA_ERR_INVALID_ARG;
  if (lse == nullptr || !aligned(lse, 16)) return FA_ERR_INVALID_ARG;
  if ((workspace == nullptr && workspace_bytes != 0) || !aligned(workspace, 16)) return FA_ERR_INVALID_ARG;
  Tensor tq, to;
  if ((st = make_tensor(q, B, Hq, N, cache->d, opt->q_stride, &tq)) != FA_OK) return st;
  if ((st = make_tensor(o, B, Hq, N, cache->d, opt->o_stride, &to)) != FA_OK) return st;
  const size_t lse_bytes = static_cast<size_t>(B) * Hq * N * 4, len = static_cast<size_t>(B) * 4;
  const size_t tab = table_bytes(B, opt->table_stride, opt->table_width);
  if (tensors_meet(to, tq) || ranges_meet(lse, lse_bytes, q, tq.bytes()) || ranges_meet(lse, lse_bytes, o, to.bytes()))
    return FA_ERR_INVALID_ARG;
  const struct {
    const void* p;
    size_t n;
  } outs[] = {{o, to.bytes()}, {lse, lse_bytes}, {workspace, workspace_bytes}};
  for (const auto& x : outs)
    if (meets_cache(cache, x.p, x.n) || ranges_meet(x.p, x.n, opt->page_table, tab) ||
        ranges_meet(x.p, x.n, opt->kv_len, len) || ranges_meet(x.p, x.n, opt->q_len, len))
      return FA_ERR_INVALID_ARG;
  if (ranges_meet(workspace, workspace_bytes, q, tq.bytes()) || ranges_meet(workspace, workspace_bytes, o, to.bytes()) ||
      ranges_meet(workspace, workspace_bytes, lse, lse_bytes))
    return FA_ERR_INVALID_ARG;
  if ((st = device_status_word(&a.status)) != FA_OK) return st;
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.sq = tq.rows();
  a.so = to.rows();
  a.B = B;
  a.Hq = Hq;
  a.N = N;
  a.G = Hq / cache->H;
  a.fp16 = opt->dtype == FA_FP16;
  a.causal = opt->causal;
  a.scale_log2 = scale_log2;
  a.kv_len = opt->kv_len;
  a.q_len = opt->q_len;
  a.wait_limit = kWaitLimitCycles;
  const long long pool_rows = static_cast<long long>(cache->num_pages) * cache->H * cache->page_size;
  if (!encode_code_rows(&a.tm[0], cache->k, pool_rows, cache->d, cache->page_size) ||
      !encode_code_rows(&a.tm[1], cache->v, pool_rows, cache->d, cache->page_size))
    return FA_ERR_CUDA;
  a.ws = static_cast<uint8_t*>(workspace);
  a.ws_bytes = workspace_bytes;
  return launch_cache_attention(a, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
