// What the kernels of the attention over the cache share: the conversions of
// 16-bit types and of the 8-bit codes, the weights' reference, NaN in V.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache_internal.h"
#include "fa_ptx.cuh"

namespace fa {

constexpr float kLn2Cache = 0.69314718055994530942f;
// Log2 units a weight may stand above the reference before that moves (a chunk with 4 210.8 us, 6
// 203.0, 8 201.3, 10 201.1: heavy-tailed scores move it often, and moving O costs a tile more than a
// step's weights). Weights within 2^21 below the reference keep fp16's 11 bits.
constexpr float kSlack = 8.f;
constexpr float kBias = 15.f - kSlack;       // weights are at most 2^15
constexpr float kMinScale = 0x1p-100f;       // a page whose V scale is not above it counts as zeros
// V scale that stands in for a page of zeros, whose weights count in the sum alone. A weight whose
// exponent lies 2^-133 below the reference is lost to the sum as well, so the stand-in is
// near the scales that occur: pages of zeros keep 2^-43 of the sum beside scales up to 2^30.
constexpr float kZeroScale = 0x1p-60f;

__device__ __forceinline__ float2 unpack16(uint32_t w, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<__half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  return fp16 ? pack_half(lo, hi) : pack_bf16(lo, hi);
}

// 16 bytes to shared memory, `bytes` of them (0 or 16) from p and zeros behind; and the wait
// for all of the thread's copies.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* p, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(p)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// The codes in bytes 0, 1 (lo) and 2, 3 (hi) of a word, as fp16 pairs. For
// int8 the byte plus 128 becomes the mantissa of 1024 + b and 1152 comes off.
template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (INT8) {
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const uint32_t k = 0x64806480u;
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&k));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&k));
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// Channels [c0, c0 + 4 W) of V, c0 a multiple of 4, that are NaN at one of the keys [first, end) of a
// sequence and cache head, from entry `tab` of the page table on: a bit each. For rows that see a NaN which was taken out of a tile because other
// rows of the unit do not see all of its keys: at most a tile's keys and a unit's rows of them.
template <int W>
__device__ __forceinline__ unsigned long long seen_nan(const CacheView& c, long long tab, int h, int first, int end, int c0) {
  unsigned long long bits = 0ull;
#pragma unroll 1
  for (int key = first; key < end; ++key) {
    const int p = __ldcg(c.table + tab + (key >> c.log2_page));
    if (p < 0 || p >= c.num_pages) continue;  // not read
    const long long row = ((static_cast<long long>(p) * c.H + h) << c.log2_page) + (key & (c.page - 1));
    const uint32_t* const at = reinterpret_cast<const uint32_t*>(c.code[1] + row * c.d + c0);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t nan = __vcmpeq4(__ldcg(at + w) & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0x08040201u;  // a bit of each byte
      bits |= static_cast<unsigned long long>(nan * 0x01010101u >> 24) << (4 * w);
    }
  }
  return bits;
}

}  // namespace fa
