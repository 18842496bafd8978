// Writing K and V into the paged 8-bit cache and reading them back
// (fa_cache_write, fa_cache_read).
//
// Mathematics: the rows of one (page, head) of K or V share a scale s, a power
// of two: s = 2^e with e the smallest integer such that amax <= s * QMAX (448
// for e4m3, 127 for int8). e comes from amax's exponent and one compare of its
// mantissa, and x * 2^-e is exact, so a code depends on x and s alone and every
// path forms the same one. A page that is partly filled keeps its rows when
// the scale grows: their codes times 2^(e_old - e_new), rounded once more. In
// e4m3 that is exact but for values that become subnormal; in int8 the errors of
// repeated moves form a geometric series, at most one step in all.
//
// What bounds it: memory (2 bytes read and 1 written per element) for prompts,
// latency for single tokens. Measured (GPU time): prompts of 1021 to 4099 tokens, 5 sequences, 8
// heads, d = 128, int8: 19.7 us, 4000 GB/s (bursts of four to five rounds of blocks); 4 of 8192,
// e4m3: 37 us, 5450 GB/s; one token of 64 sequences 5.4 us; reading 16384 tokens of 16 heads back:
// 36.9 us, 5450 GB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (FP16) return __half22float2(*reinterpret_cast<__half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (FP16) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  return pack_bf16(lo, hi);
}

// |x| where x is finite, else 0: an infinity or NaN does not set a scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// The magnitudes of two packed 16-bit values, and their maxima, NaN on top.
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & 0x7fff7fffu; }
template <bool FP16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t m;
  if constexpr (FP16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
template <bool FP16>
__device__ __forceinline__ void values8(const uint4& x, float (&v)[2][4]) {
  const float2 f0 = unpack2<FP16>(x.x), f1 = unpack2<FP16>(x.y), f2 = unpack2<FP16>(x.z), f3 = unpack2<FP16>(x.w);
  v[0][0] = f0.x;
  v[0][1] = f0.y;
  v[0][2] = f1.x;
  v[0][3] = f1.y;
  v[1][0] = f2.x;
  v[1][1] = f2.y;
  v[1][2] = f3.x;
  v[1][3] = f3.y;
}
template <bool FP16>
__device__ __forceinline__ bool has_nonfinite(uint32_t mag) {
  return mag >= (FP16 ? 0x7c00u : 0x7f80u);
}

// The smallest power of two s >= 2^-126 with amax <= s * QMAX, exactly; 0 for
// amax = 0. QMAX is 1.75 * 2^8 (e4m3) or 1.984375 * 2^6 (int8).
template <bool INT8>
__device__ __forceinline__ float scale_for(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  constexpr uint32_t kMant = INT8 ? 0x7e0000u : 0x600000u;  // mantissa of QMAX
  constexpr int kExp = INT8 ? 6 : 8;
  int e = static_cast<int>(u >> 23) - kExp + ((u & 0x7fffffu) > kMant ? 1 : 0);  // biased
  e = max(e, 1);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}
// The smallest power of two that is not below s. A page of another scale (a pool filled elsewhere) takes
// one with its next tokens: x / s is then exact, and every path forms the same codes.
__device__ __forceinline__ float ceil_power(float s) {
  return __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0xff800000u);
}
// What values are multiplied by to become codes. Of a page of scale 0 the finite ones are zeros,
// and infinities and NaN have to stay what they are.
__device__ __forceinline__ float inverse(float s) { return s > 0.f ? __frcp_rn(s) : 1.f; }

// Two values to codes (ties to even, saturating), `lo` in the low byte.
template <bool INT8>
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  if constexpr (INT8) {
    const int a = min(max(__float2int_rn(lo), -127), 127), b = min(max(__float2int_rn(hi), -127), 127);
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8);
  } else {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
}
// The two codes in the low 16 bits of w.
template <bool INT8>
__device__ __forceinline__ float2 decode2(uint32_t w) {
  if constexpr (INT8) {
    return make_float2(static_cast<float>(static_cast<int8_t>(w & 0xff)),
                       static_cast<float>(static_cast<int8_t>((w >> 8) & 0xff)));
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w & 0xffffu)));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
  }
}
// Four finite values times f to codes, |x f| <= QMAX. int8: adding 1.5 * 2^23 leaves the
// nearest integer (ties to even) in the low bits, in one fma with the product.
template <bool INT8>
__device__ __forceinline__ uint32_t encode4_finite(const float (&x)[4], float f) {
  if constexpr (INT8) {
    const float k = 12582912.f;
    const uint32_t a = __float_as_uint(fmaf(x[0], f, k)), b = __float_as_uint(fmaf(x[1], f, k));
    const uint32_t c = __float_as_uint(fmaf(x[2], f, k)), d = __float_as_uint(fmaf(x[3], f, k));
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  }
  return encode2<INT8>(x[0] * f, x[1] * f) | (encode2<INT8>(x[2] * f, x[3] * f) << 16);
}
template <bool INT8>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float f) {
  return encode2<INT8>(x[0] * f, x[1] * f) | (encode2<INT8>(x[2] * f, x[3] * f) << 16);
}
// Four codes times f, as codes again.
template <bool INT8>
__device__ __forceinline__ uint32_t move4(uint32_t w, float f) {
  const float2 a = decode2<INT8>(w), b = decode2<INT8>(w >> 16);
  const float x[4] = {a.x, a.y, b.x, b.y};
  return encode4<INT8>(x, f);
}

// The tokens of sequence b that a call writes or reads: [first, end).
struct Span {
  long long first, end;
};
__device__ __forceinline__ Span span_of(const CacheRows& a, int b) {
  const long long room = static_cast<long long>(a.c.table_width) << a.c.log2_page;
  Span s;
  s.first = a.start != nullptr ? max(0, a.start[b]) : 0;
  const int cnt = a.count != nullptr ? min(a.N, max(0, a.count[b])) : a.N;
  s.end = min(s.first + cnt, room);
  return s;
}
// The page that entry i of sequence b's table row names, or -1 (reported).
__device__ __forceinline__ int page_of(const CacheRows& a, int b, long long i) {
  const int p = a.c.table[b * a.c.table_stride + i];
  if (p >= 0 && p < a.c.num_pages) return p;
  report_bad_page(a.status);
  return -1;
}

// Unit number to (sequence, page, head).
struct UnitAt {
  int h, rel, b;
  __device__ __forceinline__ UnitAt(unsigned unit, int H, int pages_per_seq) {
    const unsigned q = unit / static_cast<unsigned>(H);
    h = static_cast<int>(unit - q * static_cast<unsigned>(H));
    b = static_cast<int>(q / static_cast<unsigned>(pages_per_seq));
    rel = static_cast<int>(q - static_cast<unsigned>(b) * static_cast<unsigned>(pages_per_seq));
  }
};

// Pages (more than kFew tokens). A unit is one (sequence, page, head), K and V together; its R d / 32
// threads hold its R new rows in registers (R: a page, or the power of two that holds N), 32
// elements of each, so they are read once: the loads, the maxima over the unit, then the codes.
// 16 bytes in and 8 bytes out per thread and piece, coalesced over the unit's rows. Beside the
// memory the instructions around few elements bind it, so K and V share a thread's place, places
// within the page are 32-bit, and a thread's four pieces lie a constant stride apart. 38 tokens of
// 224 sequences, 12 heads, pages of 128 take 29 us with R = 64 and 60 with R = 128.
template <bool FP16, bool INT8>
__global__ void __launch_bounds__(512) cache_write_pages_kernel(const CacheRows a, int log2_t, int pages_per_seq,
                                                                unsigned units) {
  __shared__ uint32_t warp_max[2][16];
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x & ((1 << log2_t) - 1);
  const unsigned unit = blockIdx.x * (blockDim.x >> log2_t) + (threadIdx.x >> log2_t);
  const int log2_chunks = a.c.d == 128 ? 4 : 3;
  int h = 0, b = 0, page = -1;
  int lo = 0, hi = 0;    // rows of the page that are written
  long long before = 0;  // the page's first row counted from the call's first token
  if (unit < units) {
    const UnitAt u(unit, a.c.H, pages_per_seq);
    h = u.h;
    b = u.b;
    const Span sp = span_of(a, b);
    const long long pi = (sp.first >> a.c.log2_page) + u.rel, page0 = pi << a.c.log2_page;
    before = page0 - sp.first;
    lo = static_cast<int>(max(0LL, -before));
    hi = static_cast<int>(min(static_cast<long long>(a.c.page), sp.end - page0));
    if (lo < hi) page = page_of(a, b, pi);  // needed after the loads below, which do not wait for it
  }
  const int row0 = lo + (t >> log2_chunks), row_step = 1 << (log2_t - log2_chunks);
  const long long at0 = b * a.st.b + h * a.st.h + (before + row0) * a.st.n + (t & ((1 << log2_chunks) - 1)) * 8;
  const long long src_step = row_step * a.st.n;
  uint4 x[2][4];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint16_t* const src = a.x[kv] + at0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = row0 + k * row_step;
      x[kv][k] = row < hi ? *reinterpret_cast<const uint4*>(src + k * src_step) : make_uint4(0, 0, 0, 0);
    }
  }
  const long long ph = static_cast<long long>(page) * a.c.H + h;
  const bool held = page >= 0 && lo > 0;  // earlier tokens of this sequence lie in the page
  float s_old[2], amax[2];
  uint32_t big[2];  // maxima of magnitudes, as patterns; NaN and infinities on top
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    // by every thread, before the barriers below; written after them
    s_old[kv] = held ? fmaxf(a.c.scale[kv][ph], 0.f) : 0.f;
    uint32_t m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = max2<FP16>(max2<FP16>(magnitudes(x[kv][k].x), magnitudes(x[kv][k].y)),
                        max2<FP16>(magnitudes(x[kv][k].z), magnitudes(x[kv][k].w)));
    const uint32_t v = max2<FP16>(max2<FP16>(m[0], m[1]), max2<FP16>(m[2], m[3]));
    big[kv] = __reduce_max_sync(0xffffffffu, max(v & 0xffffu, v >> 16));
  }
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, unit_warps = 1 << max(0, log2_t - 5);
  const int peer = (w & ~(unit_warps - 1)) + (lane & (unit_warps - 1));  // a warp of this unit, by lane
  if (log2_t > 5) {  // units of several warps
    if (lane < 2) warp_max[lane][w] = lane == 0 ? big[0] : big[1];
    __syncthreads();
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) big[kv] = __reduce_max_sync(0xffffffffu, warp_max[kv][peer]);
  }
  const bool finite = !has_nonfinite<FP16>(max(big[0], big[1]));
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) amax[kv] = unpack2<FP16>(big[kv]).x;
  // Infinities and NaN are rare: only then second maxima, over the finite values (a
  // block's units of several warps share barriers, so all of them take them).
  if (log2_t > 5 ? __syncthreads_or(!finite) : !finite) {
    for (int kv = 0; kv < 2; ++kv) {
      float f = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 q = kv ? x[1][k] : x[0][k];
        const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 e = unpack2<FP16>(v[i]);
          f = fmaxf(f, fmaxf(finite_abs(e.x), finite_abs(e.y)));
        }
      }
      uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(f));
      if (log2_t > 5) {
        __syncthreads();
        if (lane == 0) warp_max[0][w] = bits;
        __syncthreads();
        bits = __reduce_max_sync(0xffffffffu, warp_max[0][peer]);
      }
      if (kv)
        amax[1] = __uint_as_float(bits);
      else
        amax[0] = __uint_as_float(bits);
    }
  }
  if (page < 0) return;
  if (log2_t == 5) __syncwarp();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float s = fmaxf(ceil_power(s_old[kv]), scale_for<INT8>(amax[kv]));
    const float inv = inverse(s);
    uint8_t* const dst = a.c.code[kv] + ((ph << a.c.log2_page) + lo) * a.c.d + t * 8;
    if (finite) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[2][4];
        values8<FP16>(x[kv][k], v);
        if (row0 + k * row_step < hi)
          *reinterpret_cast<uint2*>(dst + (k * 8 << log2_t)) =
              make_uint2(encode4_finite<INT8>(v[0], inv), encode4_finite<INT8>(v[1], inv));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[2][4];
        values8<FP16>(x[kv][k], v);
        if (row0 + k * row_step < hi)
          *reinterpret_cast<uint2*>(dst + (k * 8 << log2_t)) = make_uint2(encode4<INT8>(v[0], inv), encode4<INT8>(v[1], inv));
      }
    }
    if (lo > 0 && s > s_old[kv]) {  // the page's older rows move to the new scale
      uint8_t* const old = a.c.code[kv] + (ph << a.c.log2_page) * a.c.d + t * 8;
#pragma unroll 1
      for (int row = t >> log2_chunks, k = 0; row < lo; row += row_step, ++k) {
        uint2* const at = reinterpret_cast<uint2*>(old + (k * 8 << log2_t));
        const uint2 c = *at;
        *at = make_uint2(move4<INT8>(c.x, s_old[kv] * inv), move4<INT8>(c.y, s_old[kv] * inv));
      }
    }
    if (t == 0) a.c.scale[kv][ph] = s;
  }
}

// A few tokens (N <= kFew; us here and by the kernel above: 1 token of 64 sequences 5.5, 6.2; 8 tokens
// of 4 5.1, 6.2, of 64 6.2, 6.2, of 256 8.4, 10.3 in e4m3 and 10.2, 10.1 in int8): one warp per
// (sequence, page, head) of K or V, a
// row per lane group: lane l holds channels [4 l', 4 l' + 4) of a row, l' = l
// modulo d / 4. The page's older rows are touched only when the scale grows.
constexpr int kFew = 8;
template <bool FP16, bool INT8>
__global__ void __launch_bounds__(128) cache_write_few_kernel(const CacheRows a, int pages_per_seq, unsigned units) {
  grid_dep_wait();
  grid_dep_launch();
  const unsigned unit = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int lane = threadIdx.x & 31;
  const int per_row = a.c.d >> 2, rows = 32 / per_row;  // lanes of a row, rows a warp takes at once: 1 or 2
  const int sub = lane / per_row, ch = (lane - sub * per_row) * 4;
  const UnitAt u(unit >> 1, a.c.H, pages_per_seq);
  const int kv = static_cast<int>(unit & 1u), h = u.h, b = u.b;
  const Span sp = span_of(a, b);
  const long long pi = (sp.first >> a.c.log2_page) + u.rel, page0 = pi << a.c.log2_page;
  if (sp.first >= sp.end || page0 >= sp.end) return;
  const int page = page_of(a, b, pi);
  if (page < 0) return;
  const long long t0 = max(sp.first, page0), t1 = min(sp.end, page0 + (1LL << a.c.log2_page));
  float* const scale = a.c.scale[kv] + static_cast<long long>(page) * a.c.H + h;
  const bool held = sp.first > page0;
  const float s_old = held ? fmaxf(*scale, 0.f) : 0.f;
  const uint16_t* src = a.x[kv] + b * a.st.b + h * a.st.h + ch;
  uint2 x[kFew];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kFew; ++k) {
    const long long tok = t0 + k * rows + sub;
    x[k] = make_uint2(0, 0);
    if (tok < t1) x[k] = *reinterpret_cast<const uint2*>(src + (tok - sp.first) * a.st.n);
  }
#pragma unroll
  for (int k = 0; k < kFew; ++k) {
    const float2 f = unpack2<FP16>(x[k].x), g = unpack2<FP16>(x[k].y);
    amax = fmaxf(fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y))), fmaxf(finite_abs(g.x), finite_abs(g.y)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = fmaxf(ceil_power(s_old), scale_for<INT8>(amax));
  const float inv = inverse(s);
  uint8_t* const dst = a.c.code[kv] + ((static_cast<long long>(page) * a.c.H + h) << a.c.log2_page) * a.c.d + ch;
  if (s > s_old && held) {
    const float f = s_old * inv;
    const int n = static_cast<int>(sp.first - page0);
#pragma unroll 4
    for (int row = sub; row < n; row += rows) {
      uint32_t* const at = reinterpret_cast<uint32_t*>(dst + row * a.c.d);
      *at = move4<INT8>(*at, f);
    }
  }
#pragma unroll
  for (int k = 0; k < kFew; ++k) {
    const long long tok = t0 + k * rows + sub;
    if (tok < t1) {
      const float2 f = unpack2<FP16>(x[k].x), g = unpack2<FP16>(x[k].y);
      const float v[4] = {f.x, f.y, g.x, g.y};
      *reinterpret_cast<uint32_t*>(dst + (tok - page0) * a.c.d) = encode4<INT8>(v, inv);
    }
  }
  __syncwarp();  // the old scale has been read by every lane
  if (lane == 0) *scale = s;
}

// Reading back: a thread takes 16 codes (one 16-byte load, two 16-byte
// stores) of kRead rows a block's width apart, so that several loads are in
// flight (16384 tokens of 16 heads: 1 row 37.0 us, 2 36.9, 4 42.1).
constexpr int kRead = 2;
template <bool FP16, bool INT8>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheRows a, int tiles) {
  grid_dep_wait();
  grid_dep_launch();
  const int log2_chunks = a.c.d == 128 ? 3 : 2;
  const unsigned bh = blockIdx.x / static_cast<unsigned>(tiles);
  const int tile = static_cast<int>(blockIdx.x - bh * static_cast<unsigned>(tiles));
  const int b = static_cast<int>(bh / static_cast<unsigned>(a.c.H)), h = static_cast<int>(bh) - b * a.c.H, kv = blockIdx.y;
  const Span sp = span_of(a, b);
  const int rows = 256 >> log2_chunks, ch = (threadIdx.x & ((1 << log2_chunks) - 1)) * 16;
  const int n0 = tile * rows * kRead + (threadIdx.x >> log2_chunks);
  uint16_t* const dst = a.x[kv] + b * a.st.b + h * a.st.h + ch;
  uint4 w[kRead];
  float s[kRead];
#pragma unroll
  for (int k = 0; k < kRead; ++k) {
    const int n = n0 + k * rows;
    const long long tok = sp.first + n;
    w[k] = make_uint4(0, 0, 0, 0);
    s[k] = 0.f;
    if (n < a.N && tok < sp.end) {
      const int page = page_of(a, b, tok >> a.c.log2_page);
      if (page >= 0) {
        const long long ph = static_cast<long long>(page) * a.c.H + h;
        const long long row = (ph << a.c.log2_page) + (tok & ((1 << a.c.log2_page) - 1));
        w[k] = *reinterpret_cast<const uint4*>(a.c.code[kv] + row * a.c.d + ch);
        s[k] = a.c.scale[kv][ph];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kRead; ++k) {
    const int n = n0 + k * rows;
    if (n >= a.N) return;
    const uint32_t in[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 lo = decode2<INT8>(in[i]), hi = decode2<INT8>(in[i] >> 16);
      out[2 * i] = pack2<FP16>(lo.x * s[k], lo.y * s[k]);
      out[2 * i + 1] = pack2<FP16>(hi.x * s[k], hi.y * s[k]);
    }
    uint4* const at = reinterpret_cast<uint4*>(dst + n * a.st.n);
    at[0] = make_uint4(out[0], out[1], out[2], out[3]);
    at[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

template <bool FP16, bool INT8>
cudaError_t write_variant(const CacheRows& a, cudaStream_t stream) {
  // a run of N tokens touches at most this many pages, wherever it starts
  const long long span_pages = ((static_cast<long long>(a.N) + a.c.page - 2) >> a.c.log2_page) + 1;
  const int pages = static_cast<int>(span_pages < a.c.table_width ? span_pages : a.c.table_width);
  const long long units = static_cast<long long>(a.B) * pages * a.c.H;
  if (units > 0x3fffffffLL) return cudaErrorInvalidValue;
  const unsigned n = static_cast<unsigned>(units);
  if (a.N <= kFew) {
    return launch_pdl(cache_write_few_kernel<FP16, INT8>, dim3((2 * n + 3) / 4), dim3(128), 0, stream, a, pages, 2 * n);
  }
  int log2_rows = 4;
  while (log2_rows < a.c.log2_page && (1 << log2_rows) < a.N) ++log2_rows;
  const int log2_t = log2_rows + (a.c.d == 128 ? 7 : 6) - 5;
  // a unit a block, of 128 threads at least: smaller blocks end and begin more evenly (19.7 us
  // where blocks of 256 took 20.7)
  const int threads = log2_t > 8 ? 512 : log2_t > 7 ? 256 : 128;
  const unsigned per = static_cast<unsigned>(threads >> log2_t);
  return launch_pdl(cache_write_pages_kernel<FP16, INT8>, dim3((n + per - 1) / per), dim3(threads), 0, stream, a,
                    log2_t, pages, n);
}

template <bool FP16, bool INT8>
cudaError_t read_variant(const CacheRows& a, cudaStream_t stream) {
  const int rows = (a.c.d == 128 ? 32 : 64) * kRead, tiles = (a.N + rows - 1) / rows;
  const long long blocks = static_cast<long long>(a.B) * a.c.H * tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(cache_read_kernel<FP16, INT8>, dim3(static_cast<unsigned>(blocks), 2), dim3(256), 0, stream, a,
                    tiles);
}

}  // namespace

cudaError_t launch_cache_write(const CacheRows& a, cudaStream_t stream) {
  if (a.fp16) return a.c.int8 ? write_variant<true, true>(a, stream) : write_variant<true, false>(a, stream);
  return a.c.int8 ? write_variant<false, true>(a, stream) : write_variant<false, false>(a, stream);
}

cudaError_t launch_cache_read(const CacheRows& a, cudaStream_t stream) {
  if (a.fp16) return a.c.int8 ? read_variant<true, true>(a, stream) : read_variant<true, false>(a, stream);
  return a.c.int8 ? read_variant<false, true>(a, stream) : read_variant<false, false>(a, stream);
}

}  // namespace fa
