// Attention over the paged 8-bit cache, few query rows per cache head
// (single tokens and drafted ones), and the merge of units that were cut.
//
// Mathematics: with codes kc, vc and scales ks, vs of each page,
//   x_j = scale log2e ks (q . kc_j),  y_j = x_j + log2 vs_j,  M = max_j y_j,
//   w_j = 2^(y_j - M + 15),  O = sum_j w_j vc_j / sum_j w_j / vs_j,
//   LSE = (M - 15 + log2 sum_j w_j / vs_j) ln 2.
// Taking V's scale into the exponent keeps it out of the products, and the
// running maximum then sits on the weight that V is really given: the weights are
// rounded to fp16 (11 bits, against bf16's 8) and 2^15 below the largest one
// they still have all of them. The sum is formed from the unrounded weights. Codes of
// either format are exact in fp16. A row of q is scaled by a power of two so that
// its largest value lies in [2^14, 2^15): exact for every value within 2^-28 of it.
//
// What bounds it: reading the cache, d bytes per token, head and tensor. Each
// warp streams its own key tiles (32 keys, K and V: 8 KB at d = 128) through a
// ring of kStages cp.async stages of its own, with no barrier between warps
// until a unit ends; 8 warps per SM keep 128 KB and more in flight, three times
// what the latency asks for. Products run on the warp matrix instruction with
// keys (K) and channels (V) on its 16 rows and the query rows on its 8 columns,
// so that a group of 8 query rows costs one pass over the converted codes:
// the tcgen05 form needs 128 rows and would convert through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache_internal.h"
#include "fa_cache_sched.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kWarps = 4, kThreads = kWarps * 32, kStages = 3;
constexpr int kTile = 32;                    // keys of a warp's tile
constexpr float kBias = 15.f;                // weights are at most 2^15
constexpr float kMinScale = 0x1p-100f;       // a page whose V scale is below it counts as zeros

template <int D>
struct Layout {
  static constexpr int kMat = kTile * D;               // K or V of a tile
  static constexpr int kStage = 2 * kMat;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kScales = kWarps * kStages * 16;  // ks, vs of two 16-key groups
  static constexpr int kMerge = kWarps * 8 * D * 4;
  static constexpr int kSmem = kRing + kScales + kMerge;  // two CTAs per SM
  static_assert(2 * (kSmem + 1024 + 512) <= 228 * 1024, "two CTAs per SM");
};

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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Byte offset of 16-byte chunk c of row r in a tile: chunks are permuted
// within 128-byte lines so that the reads of 8 lanes meet all banks.
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// One row of queries in fp16, scaled by a power of two (its inverse comes
// back): lane t of the row's four holds channels [D/4 t, D/4 (t + 1)).
template <int D>
__device__ __forceinline__ float load_query(const uint16_t* row, bool real, bool fp16, int t, uint32_t (&q)[D / 8]) {
  float x[D / 4];
  float mx = 0.f;
#pragma unroll
  for (int v = 0; v < D / 32; ++v) {
    const uint4 w = real ? __ldg(reinterpret_cast<const uint4*>(row + t * (D / 4)) + v) : make_uint4(0, 0, 0, 0);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16(ww[i], fp16);
      x[v * 8 + 2 * i] = f.x;
      x[v * 8 + 2 * i + 1] = f.y;
      mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const int e = max(15, static_cast<int>(__float_as_uint(mx) >> 23));
  const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) q[i] = pack_half(x[2 * i] * f, x[2 * i + 1] * f);
  return __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
}

// A weight of zero does not mask a NaN. Where the rows of a unit see different
// parts of a tile, V's NaN codes (e4m3 0x7f, 0xff) are taken out of it, and the
// rows that see one of them get a NaN sum. Lane: keys key, + 1, + 8, + 9.
template <int NT, int W>
__device__ __forceinline__ void poison_unseen(uint32_t (&v)[4][W], int key, const int (&lim)[NT][2], float (&l)[NT][2]) {
  int first = 0x7fffffff;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t nan = __vcmpeq4(v[k][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);
      if (nan != 0u) {
        v[k][w] &= ~nan;
        first = min(first, key + (k & 1) + 8 * (k >> 1));
      }
    }
  first = __reduce_min_sync(0xffffffffu, first);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (first < lim[n][k]) l[n][k] = __int_as_float(0x7fffffff);
}

// NT groups of 8 query rows per unit.
template <int D, int NT, bool INT8>
__global__ void __launch_bounds__(kThreads, 2) cache_attn_kernel(const CacheAttnLaunch a, const AttnGrid g) {
  using L = Layout<D>;
  constexpr int kM = D / 16;  // 16-channel tiles of O
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ AttnShare share;
  __shared__ long long part[kWarps];
  __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t = lane & 3;
  grid_dep_wait();
  grid_dep_launch();

  AttnCursor cur = attn_share<kThreads>(g, &share, part);
  if (g.split && threadIdx.x == 0) g.record[blockIdx.x] = make_int4(-1, 0, 0, 0);

  const uint32_t ring = smem_u32(smem) + warp * kStages * L::kStage;
  const uint32_t scales = smem_u32(smem) + L::kRing + warp * kStages * 16;
  float* const merge = reinterpret_cast<float*>(smem + L::kRing + L::kScales);

  // ---- the load side: this warp's tile of the load cursor's step
  AttnCursor ld = cur;
  const CacheView& c = a.c;
  int pid[2];
  // page ids of the load cursor's tile (-1 where no key is needed or bad);
  // a page holds one or both of the tile's 16-key groups
  auto look_up = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = (ld.step << g.log2_keys) + warp * kTile + u * 16;
      pid[u] = -1;
      if (!ld.done(g) && key < ld.x.seen) {
        pid[u] = __ldg(c.table + ld.x.b * c.table_stride + (key >> c.log2_page));
      }
    }
  };
  auto issue = [&](int stage) {
    if (!ld.done(g)) {
      const int key0 = (ld.step << g.log2_keys) + warp * kTile;
      const uint32_t dst = ring + stage * L::kStage;
      const uint8_t* base[2][2];
      int left[2];  // rows of each group that are read
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key = key0 + u * 16;
        const bool want = key < ld.x.seen, good = want && pid[u] >= 0 && pid[u] < c.num_pages;
        if (want && !good && lane == 0) report_bad_page(a.status);
        left[u] = good ? min(16, ld.x.seen - key) : 0;
        const long long ph = good ? static_cast<long long>(pid[u]) * c.H + ld.h : 0;
        const long long row = good ? (ph << c.log2_page) + (key & (c.page - 1)) : 0;
        base[u][0] = c.code[0] + row * D;
        base[u][1] = c.code[1] + row * D;
        if (lane < 2) {  // lane: K's or V's scale
          const uint32_t at = scales + stage * 16 + u * 8 + lane * 4;
          if (good)
            cp_async4(at, c.scale[lane] + ph);
          else
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(-1.f) : "memory");
        }
      }
      constexpr int kChunks = D / 16, kPer = 32 / kChunks;  // rows a warp copies at once
      const int ch = lane % kChunks, r0 = lane / kChunks;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int i = 0; i < kTile / kPer; ++i) {
          const int r = r0 + i * kPer, u = (i * kPer) >> 4;
          const int ru = r - u * 16;
          cp_async16(dst + kv * L::kMat + tile_offset<D>(r, ch), base[u][kv] + ru * D + ch * 16, ru < left[u]);
        }
      ld.next(g);
    }
    cp_async_commit();
    look_up();
  };
  look_up();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  int stage = 0;

  while (!cur.done(g)) {
    // ---- a unit (or the CTA's part of one)
    const AttnEntry x = cur.x;
    const int h = cur.h, step0 = cur.step;
    const long long unit_first = cur.pos - cur.step;
    uint32_t q[NT][D / 8];
    float rf[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = x.row0 + n * 8 + gq, i = r / g.G;
      const bool real = i < x.ql;
      const uint16_t* row = a.q + x.b * a.sq.b + static_cast<long long>(h * g.G + (r - i * g.G)) * a.sq.h + i * a.sq.n;
      const float inv = load_query<D>(row, real, a.fp16, t, q[n]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        rf[n][k] = __shfl_sync(0xffffffffu, inv, (2 * t + k) * 4) * a.scale_log2;
        lim[n][k] = attn_limit(g, x, n * 8 + 2 * t + k);
      }
    }
    int low = lim[0][0];
#pragma unroll
    for (int n = 0; n < NT; ++n) low = min(low, min(lim[n][0], lim[n][1]));
    low = __reduce_min_sync(0xffffffffu, low);  // keys below it are seen by every row

    float o[kM][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][n][k] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    int step = step0;
    bool more = true;
    while (more) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      // the stage read in the last iteration is free: refill it
      issue(stage == 0 ? kStages - 1 : stage - 1);
      const int key0 = (step << g.log2_keys) + warp * kTile;
      const uint32_t kt = ring + stage * L::kStage, vt = kt + L::kMat;
      if (key0 < x.seen) {
        const uint4 sc = lds128(scales + stage * 16);
        const float ks[2] = {__uint_as_float(sc.x), __uint_as_float(sc.z)};
        const float vs[2] = {fmaxf(__uint_as_float(sc.y), kMinScale), fmaxf(__uint_as_float(sc.w), kMinScale)};
        // S^T = K Q^T: keys gq, gq + 8 of each group, queries 2t, 2t + 1
        float s[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[u][n][k] = 0.f;
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const int ch = (D / 64) * t + j;
            const uint4 ka = lds128(kt + tile_offset<D>(u * 16 + gq, ch));
            const uint4 kb = lds128(kt + tile_offset<D>(u * 16 + gq + 8, ch));
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t a0, a1, a2, a3;
              decode4<INT8>(wa[w], a0, a2);
              decode4<INT8>(wb[w], a1, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816(s[u][n], a0, a1, a2, a3, q[n][(j * 4 + w) * 2], q[n][(j * 4 + w) * 2 + 1]);
            }
          }
        }
        // y, the running maximum, the weights
        const float lv[2] = {__log2f(vs[0]), __log2f(vs[1])};
        const float iv[2] = {__fdividef(1.f, vs[0]), __fdividef(1.f, vs[1])};
        const bool mixed = min(key0 + kTile, x.seen) > low;  // rows see different parts of the tile
        const bool edge = key0 + kTile > low || ks[0] < 0.f || ks[1] < 0.f;
        bool moved = false;
        float al[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float f = rf[n][k] * ks[u];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float y = fmaf(s[u][n][2 * e + k], f, lv[u]);
                if (edge && (key0 + u * 16 + gq + 8 * e >= lim[n][k] || ks[u] < 0.f)) y = -INFINITY;
                s[u][n][2 * e + k] = y;
                mx = fmaxf(mx, y);
              }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[n][k], mx);
            const float base = mn == -INFINITY ? 0.f : mn;
            al[n][k] = ex2(m[n][k] - base);
            moved |= mn > m[n][k];
            m[n][k] = mn;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float su = 0.f;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float p = ex2(s[u][n][2 * e + k] - base + kBias);
                s[u][n][2 * e + k] = p;
                su += p;
              }
              sum = fmaf(su, iv[u], sum);
            }
            l[n][k] = fmaf(l[n][k], al[n][k], sum);
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < kM; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[i][n][k] *= al[n][k & 1];
        }
        // O^T += V^T P^T: channels (D/8) gq + 2i, + 1 on the rows of tile i
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t p0[NT], p1[NT];
          const bool zero = !(vs[u] > kMinScale);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            p0[n] = transpose8x8(zero ? 0u : pack_half(s[u][n][0], s[u][n][1]));
            p1[n] = transpose8x8(zero ? 0u : pack_half(s[u][n][2], s[u][n][3]));
          }
          uint32_t v[4][D / 32];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = u * 16 + 2 * t + (k & 1) + 8 * (k >> 1);
            if constexpr (D == 128) {
              const uint4 w = lds128(vt + tile_offset<D>(r, gq));
              v[k][0] = w.x;
              v[k][1] = w.y;
              v[k][2] = w.z;
              v[k][3] = w.w;
            } else {
              const uint2 w = lds64(vt + tile_offset<D>(r, gq >> 1) + (gq & 1) * 8);
              v[k][0] = w.x;
              v[k][1] = w.y;
            }
          }
          if (!INT8 && mixed) poison_unseen(v, key0 + u * 16 + 2 * t, lim, l);
#pragma unroll
          for (int i = 0; i < kM; ++i) {
            const uint32_t sel = (i & 1) ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            decode4<INT8>(__byte_perm(v[0][i >> 1], v[1][i >> 1], sel), a0, a1);
            decode4<INT8>(__byte_perm(v[2][i >> 1], v[3][i >> 1], sel), a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[i][n], a0, a1, a2, a3, p0[n], p1[n]);
          }
        }
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
      ++step;
      const bool same = cur.next(g);
      more = same && !cur.done(g);
    }

    // ---- join the warps' keys
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], w);
        if (gq == 0) {
          sm_m[warp][n * 8 + 2 * t + k] = m[n][k];
          sm_l[warp][n * 8 + 2 * t + k] = l[n][k];
        }
      }
    __syncthreads();
    const bool whole = step0 == 0 && step == x.steps;
    const int slot = 2 * blockIdx.x + (step0 == 0 ? 1 : 0);
    if (g.split && !whole && step == x.steps && threadIdx.x == 0)
      g.record[blockIdx.x] =
          make_int4(x.b * g.row_tiles + x.row0 / g.rows, h, attn_cta_of(unit_first, share.total, share.ctas), 0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = n * 8 + 2 * t + k;
        float M = sm_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm_m[w][r]);
        const float f = ex2(m[n][k] - (M == -INFINITY ? 0.f : M));
        float* const at = merge + (warp * 8 + 2 * t + k) * D + gq * (D / 8);
#pragma unroll
        for (int i = 0; i < kM; ++i)
          *reinterpret_cast<float2*>(at + 2 * i) = make_float2(o[i][n][k] * f, o[i][n][2 + k] * f);
      }
      __syncthreads();
      {
        constexpr int kPer = 8 * D / kThreads;  // channels of a row per thread
        const int r8 = threadIdx.x / 16, d0 = (threadIdx.x & 15) * kPer, r = n * 8 + r8;
        float M = sm_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm_m[w][r]);
        float sum = 0.f, acc[kPer];
#pragma unroll
        for (int d = 0; d < kPer; ++d) acc[d] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          sum = fmaf(sm_l[w][r], ex2(sm_m[w][r] - (M == -INFINITY ? 0.f : M)), sum);
#pragma unroll
          for (int d = 0; d < kPer; ++d) acc[d] += merge[(w * 8 + r8) * D + d0 + d];
        }
        const int row = x.row0 + r, i = row / g.G;
        if (!whole) {
          const long long pr = static_cast<long long>(slot) * g.rows + r;
#pragma unroll
          for (int d = 0; d < kPer; d += 4)
            *reinterpret_cast<float4*>(g.o_part + pr * D + d0 + d) =
                make_float4(acc[d], acc[d + 1], acc[d + 2], acc[d + 3]);
          if (d0 == 0) {
            g.m_part[pr] = M;
            g.l_part[pr] = sum;
          }
        } else if (i < g.N) {
          const bool none = sum == 0.f;  // a row that sees no key; NaN stays NaN
          const float inv = none ? 0.f : 1.f / sum;
          const int head = h * g.G + (row - i * g.G);
          uint16_t* const dst = a.o + x.b * a.so.b + head * a.so.h + i * a.so.n + d0;
          uint32_t w[kPer / 2];
#pragma unroll
          for (int d = 0; d < kPer / 2; ++d)
            w[d] = none ? 0u : pack16(acc[2 * d] * inv, acc[2 * d + 1] * inv, a.fp16);
          if constexpr (kPer == 8)
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
          if (d0 == 0)
            a.lse[(static_cast<long long>(x.b) * a.Hq + head) * g.N + i] =
                none ? -INFINITY : (M - kBias + log2f(sum)) * kLn2;
        }
      }
      __syncthreads();
    }
  }
  cp_async_wait<0>();
}

// Merges the units that were cut. Block (c, y) looks at CTA c's record (the
// unit whose last part c ran); each warp takes rows of it: with m_q, l_q, O_q
// of part q and M = max_q m_q, O = sum 2^(m_q - M) O_q / sum 2^(m_q - M) l_q.
// Lane: four consecutive channels (two at d = 64) of every part, 16-byte loads.
template <int D>
__global__ void __launch_bounds__(256) cache_attn_merge_kernel(const CacheAttnLaunch a, const AttnGrid g) {
  grid_dep_wait();
  grid_dep_launch();
  const int4 rec = g.record[blockIdx.x];
  if (rec.x < 0) return;
  const AttnEntry x = attn_entry(g, rec.x);
  const int c0 = rec.z, c1 = blockIdx.x, lane = threadIdx.x & 31;
  constexpr int kV = D / 32;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < g.rows; r += gridDim.y * 8) {
    const int row = x.row0 + r, i = row / g.G;
    if (i >= g.N) continue;
    float M = -INFINITY;
    for (int q = c0 + lane; q <= c1; q += 32) {
      const int slot = 2 * q + (q == c0 ? 1 : 0);
      M = fmaxf(M, g.m_part[static_cast<long long>(slot) * g.rows + r]);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    const float base = M == -INFINITY ? 0.f : M;
    float acc[kV], sum = 0.f;
#pragma unroll
    for (int d = 0; d < kV; ++d) acc[d] = 0.f;
#pragma unroll 4
    for (int q = c0; q <= c1; ++q) {
      const long long pr = static_cast<long long>(2 * q + (q == c0 ? 1 : 0)) * g.rows + r;
      const float f = ex2(g.m_part[pr] - base);
      sum = fmaf(g.l_part[pr], f, sum);
      float v[kV];
      if constexpr (kV == 4) {
        const float4 w = *reinterpret_cast<const float4*>(g.o_part + pr * D + lane * 4);
        v[0] = w.x;
        v[1] = w.y;
        v[2] = w.z;
        v[3] = w.w;
      } else {
        const float2 w = *reinterpret_cast<const float2*>(g.o_part + pr * D + lane * 2);
        v[0] = w.x;
        v[1] = w.y;
      }
#pragma unroll
      for (int d = 0; d < kV; ++d) acc[d] = fmaf(v[d], f, acc[d]);
    }
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const int head = rec.y * g.G + (row - i * g.G);
    uint16_t* const dst = a.o + x.b * a.so.b + head * a.so.h + i * a.so.n + lane * kV;
    uint32_t w[kV / 2];
#pragma unroll
    for (int d = 0; d < kV / 2; ++d) w[d] = none ? 0u : pack16(acc[2 * d] * inv, acc[2 * d + 1] * inv, a.fp16);
    if constexpr (kV == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (lane == 0)
      a.lse[(static_cast<long long>(x.b) * a.Hq + head) * g.N + i] =
          none ? -INFINITY : (M - kBias + log2f(sum)) * kLn2;
  }
}

template <int D, int NT, bool INT8>
cudaError_t launch_rows(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  auto kern = cache_attn_kernel<D, NT, INT8>;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = set_smem_once(smem_set, reinterpret_cast<const void*>(kern), Layout<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), Layout<D>::kSmem, stream, a, g);
}

template <int D, bool INT8>
cudaError_t launch_variant(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  cudaError_t e = g.rows == 8 ? launch_rows<D, 1, INT8>(a, g, ctas, stream) : launch_rows<D, 2, INT8>(a, g, ctas, stream);
  if (e != cudaSuccess || !g.split) return e;
  return launch_pdl(cache_attn_merge_kernel<D>, dim3(ctas, (g.rows + 7) / 8), dim3(256), 0, stream, a, g);
}

struct AttnWorkspace {
  size_t m_off, l_off, o_off, total;
};
AttnWorkspace attn_workspace(int ctas, int rows, int d) {
  AttnWorkspace w{};
  const size_t parts = 2 * static_cast<size_t>(ctas) * rows;
  w.m_off = align256(static_cast<size_t>(ctas) * 16);
  w.l_off = w.m_off + align256(parts * 4);
  w.o_off = w.l_off + align256(parts * 4);
  w.total = w.o_off + align256(parts * d * 4);
  return w;
}

}  // namespace

AttnPlan attn_plan(int B, int HK, long long rows, long long cap) {
  AttnPlan p{};
  p.rows = rows <= 8 ? 8 : 16;
  p.log2_keys = 7;
  p.units = static_cast<long long>(B) * HK * ((rows + p.rows - 1) / p.rows);
  p.cap_steps = (cap + 127) >> 7;
  if (p.cap_steps < 1) p.cap_steps = 1;
  const long long most = 2LL * sm_count();
  p.ctas = static_cast<int>(p.units >= most || p.units * p.cap_steps >= most ? most : p.units * p.cap_steps);
  return p;
}

size_t cache_attention_workspace(int B, int HK, int G, int N, int d, int page, int table_width) {
  const AttnPlan p = attn_plan(B, HK, static_cast<long long>(N) * G, static_cast<long long>(table_width) * page);
  return p.cap_steps > 1 ? attn_workspace(p.ctas, p.rows, d).total : 0;
}

cudaError_t launch_cache_attention(const CacheAttnLaunch& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.N) * a.G, cap = static_cast<long long>(a.c.table_width) * a.c.page;
  const AttnPlan p = attn_plan(a.B, a.c.H, rows, cap);
  AttnGrid g{};
  g.B = a.B;
  g.HK = a.c.H;
  g.N = a.N;
  g.G = a.G;
  g.D = a.c.d;
  g.rows = p.rows;
  g.row_tiles = static_cast<int>((rows + p.rows - 1) / p.rows);
  g.log2_keys = p.log2_keys;
  g.cap = static_cast<int>(cap);
  g.causal = a.causal;
  g.kv_len = a.kv_len;
  g.q_len = a.q_len;
  const AttnWorkspace w = attn_workspace(p.ctas, p.rows, a.c.d);
  g.split = p.cap_steps > 1 && a.ws != nullptr && a.ws_bytes >= w.total;
  if (g.split) {
    g.record = reinterpret_cast<int4*>(a.ws);
    g.m_part = reinterpret_cast<float*>(a.ws + w.m_off);
    g.l_part = reinterpret_cast<float*>(a.ws + w.l_off);
    g.o_part = reinterpret_cast<float*>(a.ws + w.o_off);
  }
  if (a.c.d == 128)
    return a.c.int8 ? launch_variant<128, true>(a, g, p.ctas, stream) : launch_variant<128, false>(a, g, p.ctas, stream);
  return a.c.int8 ? launch_variant<64, true>(a, g, p.ctas, stream) : launch_variant<64, false>(a, g, p.ctas, stream);
}

}  // namespace fa
