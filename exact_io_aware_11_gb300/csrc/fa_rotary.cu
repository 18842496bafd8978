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
// launch: their heads are one list. Measured figures stand at kBatch; one token of 32 sequences,
// 16 + 4 heads: 5.8 us with its launch.
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
  return a.pos != nullptr ? a.pos[b * a.pos_b + n * a.pos_n]
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

// A thread's row and heads from its index. Of the G = hgroups threads of a row, thread g takes
// heads g, g + G, g + 2G ... The job runs fastest, then what lies closer in memory: the row
// or, where the heads of a row lie together (a.inner), the thread of the row; batches last.
// I: 32 bits where the indices fit (a 64-bit division costs as much as two pairs' sines).
template <typename I>
struct Item {
  int job, n, b, h0, heads;
  __device__ __forceinline__ Item(const RotaryLaunch& a, I idx, int jobs, int hgroups) {
    const I first = static_cast<I>(a.inner ? hgroups : a.N), second = static_cast<I>(a.inner ? a.N : hgroups);
    const I rest = idx / static_cast<I>(jobs);
    job = static_cast<int>(idx - rest * static_cast<I>(jobs));
    const I up = rest / first;
    const int lo = static_cast<int>(rest - up * first);
    b = static_cast<int>(up / second);
    const int hi = static_cast<int>(up - static_cast<I>(b) * second);
    n = a.inner ? hi : lo;
    h0 = a.inner ? lo : hi;
    heads = a.Hq + a.Hk;
  }
};

// Heads' loads in flight, threads of a block, and heads of a thread at most. GPU time of
// 8 x 24 x 1024 x 64 and of 1 x 32 x 16384 x 128, one direction: (2, 128, 4) 11.5, 43.2 us (4390,
// 6210 GB/s); 8 heads 11.5, 44.8; blocks of 256 12.0, 45.5; batches of 4 and 8 heads 12.7, 51.5;
// batches of 8 (120 registers) 11.8, 43.1.
constexpr int kBatch = 2, kThreads = 128, kMaxHeads = 4;
// One thread: 32 bytes of some heads of one row. Half layout: 8 pairs, two chunks r/2
// apart, or two chunks of the channels behind the rotated ones; interleaved: 8 pairs, two
// adjacent chunks. Channels that are not rotated go the same way and keep their bits, so
// that the lanes of a warp stay together.
template <bool FP16, bool INTERLEAVED, typename I>
__global__ void __launch_bounds__(kThreads, 8) rotary_kernel(const RotaryLaunch a, int jobs, int hgroups, I total) {
  grid_dep_wait();
  grid_dep_launch();
  const I idx = static_cast<I>(blockIdx.x) * kThreads + threadIdx.x;
  if (idx >= total) return;
  const Item<I> it(a, idx, jobs, hgroups);
  const int rot_jobs = INTERLEAVED ? (a.r + 15) / 16 : a.r / 16;
  const bool rot = it.job < rot_jobs;
  const int ca = INTERLEAVED ? it.job * 16 : rot ? it.job * 8 : a.r + (it.job - rot_jobs) * 8;
  const int cb = INTERLEAVED ? ca + 8 : rot ? a.r / 2 + it.job * 8 : ca + (a.d - a.r) / 2;
  const int pairs = rot ? min(8, a.r / 2 - it.job * 8) : 0;  // fewer: interleaved, the last rotated chunks
  // A batch of heads' loads in flight: written out, because the compiler may not move a load
  // ahead of another head's store (the call may be in place). The first one's cross the sines.
  uint4 v[kBatch][2];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (h0 + k * hgroups < it.heads) {
        const uint16_t* const x = row_at(a, it.b, h0 + k * hgroups, it.n).x;
        v[k][0] = *reinterpret_cast<const uint4*>(x + ca);
        v[k][1] = *reinterpret_cast<const uint4*>(x + cb);
      }
    }
  };
  load(it.h0);
  float c[8], s[8];
  if (rot) {
    const int pos = position(a, it.b, it.n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (i < pairs) turn_of(a.turns[it.job * 8 + i], pos, a.fcos, a.fsin, c[i], s[i]);
    }
  }
  for (int h0 = it.h0; h0 < it.heads; h0 += kBatch * hgroups) {
    if (h0 > it.h0) load(h0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (h0 + k * hgroups >= it.heads) break;
      uint32_t wa[4] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w};
      uint32_t wb[4] = {v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
      if (rot) {
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<FP16>(wa[i]), y = unpack2<FP16>(wb[i]);
            if (i < pairs) wa[i] = pack2<FP16>(x.x * c[i] - x.y * s[i], x.x * s[i] + x.y * c[i]);
            if (4 + i < pairs) wb[i] = pack2<FP16>(y.x * c[4 + i] - y.y * s[4 + i], y.x * s[4 + i] + y.y * c[4 + i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<FP16>(wa[i]), y = unpack2<FP16>(wb[i]);
            wa[i] = pack2<FP16>(x.x * c[2 * i] - y.x * s[2 * i], x.y * c[2 * i + 1] - y.y * s[2 * i + 1]);
            wb[i] = pack2<FP16>(x.x * s[2 * i] + y.x * c[2 * i], x.y * s[2 * i + 1] + y.y * c[2 * i + 1]);
          }
        }
      }
      uint16_t* const y = row_at(a, it.b, h0 + k * hgroups, it.n).y;
      *reinterpret_cast<uint4*>(y + ca) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
      *reinterpret_cast<uint4*>(y + cb) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
    }
  }
}

// Half layout whose second channels do not start on a chunk (r / 2 not a multiple of 8): a
// warp takes 1 KB of one (batch, row) at a time, several heads, through shared memory, in as
// 16-byte chunks, turned two channels a lane and word, and out as chunks; its sines serve all
// its heads, every hgroups-th KB of the row. GPU time of 16 + 16 heads x 8192, 100 of 128
// channels: 32.7 us, with 1 KB a warp 44.8; one pair a thread, straight from memory, took 112 (96 channels by chunks 28.6).
template <int D, bool FP16, typename I>
__global__ void __launch_bounds__(kThreads) rotary_rows_kernel(const RotaryLaunch a, int hgroups, I units) {
  constexpr int kHeads = 512 / D, kLoads = 2, kWords = D / 64;  // heads of a warp, chunks and words of a lane
  __shared__ uint4 in[kThreads / 32][kLoads * 32], out[kThreads / 32][kLoads * 32];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const I unit = static_cast<I>(blockIdx.x) * (kThreads / 32) + warp;
  if (unit >= units) return;
  const I bn = unit / static_cast<I>(hgroups);
  int h0 = static_cast<int>(unit - bn * static_cast<I>(hgroups)) * kHeads;
  const int b = static_cast<int>(bn / static_cast<I>(a.N)), n = static_cast<int>(bn - static_cast<I>(b) * static_cast<I>(a.N));
  const int heads = a.Hq + a.Hk, half = a.r / 2;
  uint4 v[kLoads] = {};
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = i * 32 + lane, h = h0 + q / (D / 8);
      if (h < heads) v[i] = *reinterpret_cast<const uint4*>(row_at(a, b, h, n).x + (q % (D / 8)) * 8);
    }
  };
  load();
  const int pos = position(a, b, n);
  float c[kWords][2], s[kWords][2];  // s with the sign that the channel's partner gets
  int other[kWords][2];              // the partner; -1: not rotated
#pragma unroll
  for (int j = 0; j < kWords; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int ch = 2 * (lane + 32 * j) + e;
      other[j][e] = ch < half ? ch + half : ch < a.r ? ch - half : -1;
      c[j][e] = 1.f;
      s[j][e] = 0.f;
      if (ch < a.r) turn_of(a.turns[min(ch, other[j][e])], pos, a.fcos, ch < half ? -a.fsin : a.fsin, c[j][e], s[j][e]);
    }
  while (true) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) in[warp][i * 32 + lane] = v[i];
    __syncwarp();  // also: the chunks that went out have been read
    const int now = h0;
    h0 += hgroups * kHeads;
    const bool more = h0 < heads;
    if (more) load();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (now + h >= heads) break;
      const uint16_t* const x = reinterpret_cast<const uint16_t*>(in[warp]) + h * D;
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        const uint32_t own = reinterpret_cast<const uint32_t*>(x)[lane + 32 * j];
        const float2 f = unpack2<FP16>(own);
        const float y0 = other[j][0] < 0 ? 0.f : unpack1<FP16>(x[other[j][0]]);
        const float y1 = other[j][1] < 0 ? 0.f : unpack1<FP16>(x[other[j][1]]);
        uint32_t w = pack2<FP16>(f.x * c[j][0] + y0 * s[j][0], f.y * c[j][1] + y1 * s[j][1]);
        if (other[j][0] < 0) w = own;  // r is even: both or neither
        reinterpret_cast<uint32_t*>(out[warp])[h * (D / 2) + lane + 32 * j] = w;
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = i * 32 + lane, h = now + q / (D / 8);
      if (h < heads) *reinterpret_cast<uint4*>(row_at(a, b, h, n).y + (q % (D / 8)) * 8) = out[warp][q];
    }
    if (!more) break;
  }
}

// Heads a thread takes: as many as leave every SM 1024 threads, at most kMaxHeads (the
// sines are then a third of a thread's instructions).
int heads_per_thread(long long threads_at_one, int heads) {
  const long long enough = static_cast<long long>(sm_count()) * 1024;
  int hpt = 1;
  while (hpt < kMaxHeads && hpt < heads && threads_at_one / (hpt * 2) >= enough) hpt *= 2;
  return hpt;
}

template <bool FP16, typename I>
cudaError_t launch_chunks(const RotaryLaunch& a, unsigned blocks, int jobs, int hgroups, long long total,
                          cudaStream_t stream) {
  const dim3 grid(blocks), block(kThreads);
  const I n = static_cast<I>(total);
  if (a.interleaved) return launch_pdl(rotary_kernel<FP16, true, I>, grid, block, 0, stream, a, jobs, hgroups, n);
  return launch_pdl(rotary_kernel<FP16, false, I>, grid, block, 0, stream, a, jobs, hgroups, n);
}
template <bool FP16, typename I>
cudaError_t launch_rows(const RotaryLaunch& a, unsigned blocks, int hgroups, long long units, cudaStream_t stream) {
  const dim3 grid(blocks), block(kThreads);
  const I n = static_cast<I>(units);
  if (a.d == 128) return launch_pdl(rotary_rows_kernel<128, FP16, I>, grid, block, 0, stream, a, hgroups, n);
  return launch_pdl(rotary_rows_kernel<64, FP16, I>, grid, block, 0, stream, a, hgroups, n);
}

}  // namespace

cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t stream) {
  const int heads = a.Hq + a.Hk;
  const long long rows = static_cast<long long>(a.B) * a.N;
  if (!a.interleaved && a.r % 16 != 0) {
    // KBs of a row that a warp takes: as many as leave every SM 32 warps, at most 4
    const int kbs = (heads * a.d + 511) / 512;
    int each = 1;
    while (each < 4 && each < kbs && rows * kbs / (each * 2) >= static_cast<long long>(sm_count()) * 32) each *= 2;
    const int hgroups = (kbs + each - 1) / each;
    const long long units = rows * hgroups, blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned nb = static_cast<unsigned>(blocks);
    if (units + kThreads <= 0xffffffffLL)
      return a.fp16 ? launch_rows<true, unsigned>(a, nb, hgroups, units, stream)
                    : launch_rows<false, unsigned>(a, nb, hgroups, units, stream);
    return a.fp16 ? launch_rows<true, unsigned long long>(a, nb, hgroups, units, stream)
                  : launch_rows<false, unsigned long long>(a, nb, hgroups, units, stream);
  }
  const int jobs = a.d / 16;
  const int hpt = heads_per_thread(rows * jobs * heads, heads);
  const int hgroups = (heads + hpt - 1) / hpt;
  const long long total = rows * jobs * hgroups, blocks = (total + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned nb = static_cast<unsigned>(blocks);
  if (total + kThreads <= 0xffffffffLL)
    return a.fp16 ? launch_chunks<true, unsigned>(a, nb, jobs, hgroups, total, stream)
                  : launch_chunks<false, unsigned>(a, nb, jobs, hgroups, total, stream);
  return a.fp16 ? launch_chunks<true, unsigned long long>(a, nb, jobs, hgroups, total, stream)
                : launch_chunks<false, unsigned long long>(a, nb, jobs, hgroups, total, stream);
}

}  // namespace fa
