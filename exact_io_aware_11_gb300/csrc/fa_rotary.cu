// Rotary positions of queries and keys, forward and backward (fa_rotary_fwd,
// fa_rotary_bwd).
//
// Mathematics: pair i of the row at position p is turned by theta = p w_i.
// The caller gives w_i / 2 pi as a 64-bit binary fraction T_i; the integer
// product p T_i mod 2^64 is then the exact fraction of a turn, whatever the
// position, where an fp32 p w_i would be off by p 2^-24 radians. Its top 32
// bits, as a signed number of 2^-31 half turns, go to sincospi: the angle that
// reaches it is off by at most 2^-25 half turns, as from an exact fp32 angle.
// The gradient of a rotation is the rotation back: only the sine's sign differs.
//
// What bounds it: memory, 4 bytes moved per element. A sine and cosine cost
// about as many instructions as moving ten pairs, so a thread keeps those of
// its pairs of one (batch, row) for several heads when there are enough
// threads to fill the GPU (heads_per_thread), and with one token per sequence
// takes one head, where only latency counts. Queries and keys share the
// launch: their heads are one list.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (FP16) return __half22float2(*reinterpret_cast<__half2*>(&w));
  // bf16 is the upper half of fp32
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
template <bool FP16>
__device__ __forceinline__ float unpack1(uint16_t w) {
  return unpack2<FP16>(w).x;
}
template <bool FP16>
__device__ __forceinline__ uint16_t pack1(float x) {
  return static_cast<uint16_t>(pack2<FP16>(x, 0.f));
}

__device__ __forceinline__ void turn_of(unsigned long long turns, int p, float fcos, float fsin,
                                        float& c, float& s) {
  // p is negative before the first token of a shifted window: the product wraps the same way
  const unsigned long long t = turns * static_cast<unsigned long long>(static_cast<long long>(p));
  const float half_turns = static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f;
  sincospif(half_turns, &s, &c);
  c *= fcos;
  s *= fsin;
}

__device__ __forceinline__ int position(const RotaryLaunch& a, int b, int n) {
  return a.pos != nullptr ? __ldg(a.pos + b * a.pos_b + n * a.pos_n)
                          : static_cast<int>(static_cast<unsigned>(a.offset) + static_cast<unsigned>(n));
}

// Offsets of row (b, h, n) in the input and output of the tensor that head h
// of the joint list belongs to.
struct RowAt {
  const uint16_t* x;
  uint16_t* y;
};
__device__ __forceinline__ RowAt row_at(const RotaryLaunch& a, int b, int h, int n) {
  const bool key = h >= a.Hq;
  const RotaryTensor& t = a.t[key];
  const int hh = key ? h - a.Hq : h;
  return RowAt{t.x + b * t.sx.b + hh * t.sx.h + n * t.sx.n, t.y + b * t.sy.b + hh * t.sy.h + n * t.sy.n};
}

// One thread: 8 pairs (half layout: two 16-byte chunks r/2 apart) or 4 pairs
// (interleaved: one chunk) of `hpt` heads of one row, or one chunk of channels
// behind the rotated ones, which are copied.
template <bool FP16, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryLaunch a, int jobs, int hpt, int hgroups,
                                                     long long total) {
  grid_dep_wait();
  grid_dep_launch();
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= total) return;
  const int job = static_cast<int>(idx % jobs);
  const long long rest = idx / jobs;
  const int n = static_cast<int>(rest % a.N);
  const long long bg = rest / a.N;
  const int hg = static_cast<int>(bg % hgroups), b = static_cast<int>(bg / hgroups);
  const int h0 = hg * hpt, h1 = min(h0 + hpt, a.Hq + a.Hk);
  const int rot_jobs = INTERLEAVED ? (a.r + 7) / 8 : a.r / 16;
  if (job >= rot_jobs) {  // copied channels
    const int c = INTERLEAVED ? job * 8 : a.r + (job - rot_jobs) * 8;
    for (int h = h0; h < h1; ++h) {
      const RowAt p = row_at(a, b, h, n);
      if (p.x != p.y) *reinterpret_cast<uint4*>(p.y + c) = *reinterpret_cast<const uint4*>(p.x + c);
    }
    return;
  }
  const int pos = position(a, b, n);
  if constexpr (INTERLEAVED) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (job * 8 + 2 * i < a.r) turn_of(__ldg(a.turns + job * 4 + i), pos, a.fcos, a.fsin, c[i], s[i]);
    }
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      const RowAt p = row_at(a, b, h, n);
      uint4 v = *reinterpret_cast<const uint4*>(p.x + job * 8);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (job * 8 + 2 * i < a.r) {
          const float2 x = unpack2<FP16>(w[i]);
          w[i] = pack2<FP16>(x.x * c[i] - x.y * s[i], x.x * s[i] + x.y * c[i]);
        }
      }
      *reinterpret_cast<uint4*>(p.y + job * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_of(__ldg(a.turns + job * 8 + i), pos, a.fcos, a.fsin, c[i], s[i]);
    const int hi = a.r / 2;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      const RowAt p = row_at(a, b, h, n);
      const uint4 va = *reinterpret_cast<const uint4*>(p.x + job * 8);
      const uint4 vb = *reinterpret_cast<const uint4*>(p.x + hi + job * 8);
      uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 xa = unpack2<FP16>(wa[i]), xb = unpack2<FP16>(wb[i]);
        wa[i] = pack2<FP16>(xa.x * c[2 * i] - xb.x * s[2 * i], xa.y * c[2 * i + 1] - xb.y * s[2 * i + 1]);
        wb[i] = pack2<FP16>(xa.x * s[2 * i] + xb.x * c[2 * i], xa.y * s[2 * i + 1] + xb.y * c[2 * i + 1]);
      }
      *reinterpret_cast<uint4*>(p.y + job * 8) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
      *reinterpret_cast<uint4*>(p.y + hi + job * 8) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
    }
  }
}

// Half layout whose second channels do not start on a chunk (r / 2 not a
// multiple of 8): a thread takes one pair, or one copied channel, at a time.
template <bool FP16>
__global__ void __launch_bounds__(256) rotary_pairs_kernel(const RotaryLaunch a, int jobs, int hpt, int hgroups,
                                                           long long total) {
  grid_dep_wait();
  grid_dep_launch();
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= total) return;
  const int job = static_cast<int>(idx % jobs);
  const long long rest = idx / jobs;
  const int n = static_cast<int>(rest % a.N);
  const long long bg = rest / a.N;
  const int hg = static_cast<int>(bg % hgroups), b = static_cast<int>(bg / hgroups);
  const int h0 = hg * hpt, h1 = min(h0 + hpt, a.Hq + a.Hk);
  const int half = a.r / 2;
  if (job >= half) {
    const int ch = a.r + (job - half);
    for (int h = h0; h < h1; ++h) {
      const RowAt p = row_at(a, b, h, n);
      if (p.x != p.y) p.y[ch] = p.x[ch];
    }
    return;
  }
  float c, s;
  turn_of(__ldg(a.turns + job), position(a, b, n), a.fcos, a.fsin, c, s);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const RowAt p = row_at(a, b, h, n);
    const float xa = unpack1<FP16>(p.x[job]), xb = unpack1<FP16>(p.x[half + job]);
    p.y[job] = pack1<FP16>(xa * c - xb * s);
    p.y[half + job] = pack1<FP16>(xa * s + xb * c);
  }
}

// Heads a thread takes: as many as leave the GPU 4096 threads per SM twice
// over, at most 8 (more brings nothing: the sines are then a tenth of the work).
int heads_per_thread(long long threads_at_one, int heads) {
  const long long enough = static_cast<long long>(sm_count()) * 4096;
  int hpt = 1;
  while (hpt < 8 && hpt < heads && threads_at_one / (hpt * 2) >= enough) hpt *= 2;
  return hpt;
}

}  // namespace

cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t stream) {
  const int heads = a.Hq + a.Hk;
  const bool chunks = a.interleaved || a.r % 16 == 0;
  const int jobs = a.interleaved ? a.d / 8 : chunks ? a.r / 16 + (a.d - a.r) / 8 : a.r / 2 + (a.d - a.r);
  const long long rows = static_cast<long long>(a.B) * a.N;
  const int hpt = heads_per_thread(rows * jobs * heads, heads);
  const int hgroups = (heads + hpt - 1) / hpt;
  const long long total = rows * jobs * hgroups, blocks = (total + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(256);
  if (!chunks)
    return a.fp16 ? launch_pdl(rotary_pairs_kernel<true>, grid, block, 0, stream, a, jobs, hpt, hgroups, total)
                  : launch_pdl(rotary_pairs_kernel<false>, grid, block, 0, stream, a, jobs, hpt, hgroups, total);
  if (a.interleaved)
    return a.fp16 ? launch_pdl(rotary_kernel<true, true>, grid, block, 0, stream, a, jobs, hpt, hgroups, total)
                  : launch_pdl(rotary_kernel<false, true>, grid, block, 0, stream, a, jobs, hpt, hgroups, total);
  return a.fp16 ? launch_pdl(rotary_kernel<true, false>, grid, block, 0, stream, a, jobs, hpt, hgroups, total)
                : launch_pdl(rotary_kernel<false, false>, grid, block, 0, stream, a, jobs, hpt, hgroups, total);
}

}  // namespace fa
