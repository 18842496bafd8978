// Attention over the paged 8-bit cache: which kernel a call takes (fa_cache_rows.cuh, fa_cache_tile.cuh),
// whether its units are cut, and the merge of those that were.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache_internal.h"
#include "fa_cache_math.cuh"
#include "fa_cache_rows.cuh"
#include "fa_cache_sched.cuh"

namespace fa {
namespace {

// Merges the units that were cut. Blocks (c, y) look at CTA c's record (the unit
// whose last part c ran) and share its rows out: with m_q, l_q, O_q of part q and
// M = max_q m_q, O = sum 2^(m_q - M) O_q / sum 2^(m_q - M) l_q. A lane holds D / 32
// consecutive channels and loads five parts at a time, statistics and all. A unit
// of few parts gives each of the block's 8 warps a row; one of more parts gives a row
// four or all of them, which take every fourth or eighth part and then join theirs (a
// row of 76 parts with one warp, four at a time: 36 us by itself, with four warps 8 us). g is read where it
// lies: copied to registers, single tokens of 64 sequences of 2458 to 4096, 32 heads on 8, d = 64, 56.5 -> 57 to 63 us.
template <int D>
__global__ void __launch_bounds__(256) cache_attn_merge_kernel(const __grid_constant__ CacheAttnLaunch a, const __grid_constant__ AttnGrid g) {
  constexpr int kV = D / 32, kBatch = 5, kRowWarps = 8;
  __shared__ float sm_m[kRowWarps], sm_l[kRowWarps], sm_o[kRowWarps][D];
  grid_dep_wait();
  grid_dep_launch();
  const int4 rec = g.record[blockIdx.x];
  if (rec.x < 0) return;
  const int c0 = rec.z, c1 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = c1 - c0 < kBatch ? 1 : c1 - c0 < 4 * kBatch ? 4 : kRowWarps, sub = warp & (W - 1);  // warps of a row
  const int b = rec.x / g.row_tiles, row0 = (rec.x - b * g.row_tiles) * g.rows;
  const int live = static_cast<int>(min(static_cast<long long>(g.rows), static_cast<long long>(g.N) * g.G - row0));
  for (int r0 = blockIdx.y * (kRowWarps / W); r0 < live; r0 += gridDim.y * (kRowWarps / W)) {  // uniform over the block
    const int r = r0 + warp / W;
    float acc[kV], sum = 0.f, M = -INFINITY;
#pragma unroll
    for (int d = 0; d < kV; ++d) acc[d] = 0.f;
    for (int q0 = c0 + sub; q0 <= c1 && r < live; q0 += W * kBatch) {
      float mq[kBatch], lq[kBatch], v[kBatch][kV];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int q = q0 + W * k;
        mq[k] = -INFINITY;
        lq[k] = 0.f;
#pragma unroll
        for (int d = 0; d < kV; ++d) v[k][d] = 0.f;
        if (q <= c1) {
          const long long pr = static_cast<long long>(2 * q + (q == c0 ? 1 : 0)) * g.rows + r;
          mq[k] = g.m_part[pr];
          lq[k] = g.l_part[pr];
          if constexpr (kV == 4) {
            const float4 w = *reinterpret_cast<const float4*>(g.o_part + pr * D + lane * 4);
            v[k][0] = w.x;
            v[k][1] = w.y;
            v[k][2] = w.z;
            v[k][3] = w.w;
          } else {
            const float2 w = *reinterpret_cast<const float2*>(g.o_part + pr * D + lane * 2);
            v[k][0] = w.x;
            v[k][1] = w.y;
          }
        }
      }
      float Mn = M;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) Mn = fmaxf(Mn, mq[k]);
      const float base = Mn == -INFINITY ? 0.f : Mn, e = ex2(M - base);
      M = Mn;
      sum *= e;
#pragma unroll
      for (int d = 0; d < kV; ++d) acc[d] *= e;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float f = ex2(mq[k] - base);
        sum = fmaf(lq[k], f, sum);
#pragma unroll
        for (int d = 0; d < kV; ++d) acc[d] = fmaf(v[k][d], f, acc[d]);
      }
    }
    if (W > 1) {
#pragma unroll
      for (int d = 0; d < kV; ++d) sm_o[warp][lane * kV + d] = acc[d];
      if (lane == 0) {
        sm_m[warp] = M;
        sm_l[warp] = sum;
      }
      __syncthreads();
      if (sub == 0) {
        for (int w = 1; w < W; ++w) M = fmaxf(M, sm_m[warp + w]);
        const float base = M == -INFINITY ? 0.f : M;
        sum = 0.f;
#pragma unroll
        for (int d = 0; d < kV; ++d) acc[d] = 0.f;
        for (int w = 0; w < W; ++w) {
          const float f = ex2(sm_m[warp + w] - base);
          sum = fmaf(sm_l[warp + w], f, sum);
#pragma unroll
          for (int d = 0; d < kV; ++d) acc[d] = fmaf(sm_o[warp + w][lane * kV + d], f, acc[d]);
        }
      }
      __syncthreads();
    }
    if (sub != 0 || r >= live) continue;
    const int row = row0 + r, i = row / g.G, head = rec.y * g.G + (row - i * g.G);
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    uint16_t* const dst = a.o + b * a.so.b + head * a.so.h + i * a.so.n + lane * kV;
    uint32_t w[kV / 2];
#pragma unroll
    for (int d = 0; d < kV / 2; ++d) w[d] = none ? 0u : pack16(acc[2 * d] * inv, acc[2 * d + 1] * inv, a.fp16);
    if constexpr (kV == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (lane == 0)
      a.lse[(static_cast<long long>(b) * a.Hq + head) * g.N + i] = none ? -INFINITY : (M - kBias + log2f(sum)) * kLn2Cache;
  }
}

// The same for the tile kernel's parts, which lie in its registers' order: lane i holds row
// i of 32, warp w of block (c, y) channels [16 w, 16 w + 16) of the y-th 32 rows. Loads are 512
// bytes a warp, stores a sector of 32 bytes a lane.
template <int D>
__global__ void __launch_bounds__(D * 2)
    cache_attn_merge_tiles_kernel(const __grid_constant__ CacheAttnLaunch a, const AttnGrid g) {
  constexpr int kBatch = 4;  // parts in flight
  grid_dep_wait();
  grid_dep_launch();
  const int4 rec = g.record[blockIdx.x];
  if (rec.x < 0) return;
  const int c0 = rec.z, c1 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = rec.x / g.row_tiles, row0 = (rec.x - b * g.row_tiles) * g.rows;
  const int r = blockIdx.y * 32 + lane, row = row0 + r, i = row / g.G;
  if (i >= g.N) return;
  float acc[16], sum = 0.f, M = -INFINITY;
#pragma unroll
  for (int d = 0; d < 16; ++d) acc[d] = 0.f;
  for (int q0 = c0; q0 <= c1; q0 += kBatch) {
    float mq[kBatch], lq[kBatch];
    float4 v[kBatch][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int q = q0 + k;
      mq[k] = -INFINITY;
      lq[k] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q <= c1) {
        const long long block = static_cast<long long>(2 * q + (q == c0 ? 1 : 0)) * (g.rows / 32) + blockIdx.y;
        mq[k] = g.m_part[block * 32 + lane];
        lq[k] = g.l_part[block * 32 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[k][j] = reinterpret_cast<const float4*>(g.o_part)[(block * (D / 4) + warp * 4 + j) * 32 + lane];
      }
    }
    float Mn = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) Mn = fmaxf(Mn, mq[k]);
    const float base = Mn == -INFINITY ? 0.f : Mn, e = ex2(M - base);
    M = Mn;
    sum *= e;
#pragma unroll
    for (int d = 0; d < 16; ++d) acc[d] *= e;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float f = ex2(mq[k] - base);
      sum = fmaf(lq[k], f, sum);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[4 * j] = fmaf(v[k][j].x, f, acc[4 * j]);
        acc[4 * j + 1] = fmaf(v[k][j].y, f, acc[4 * j + 1]);
        acc[4 * j + 2] = fmaf(v[k][j].z, f, acc[4 * j + 2]);
        acc[4 * j + 3] = fmaf(v[k][j].w, f, acc[4 * j + 3]);
      }
    }
  }
  const int head = rec.y * g.G + (row - i * g.G);
  const bool none = sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
  uint32_t w[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) w[d] = none ? 0u : pack16(acc[2 * d] * inv, acc[2 * d + 1] * inv, a.fp16);
  uint4* const dst = reinterpret_cast<uint4*>(a.o + b * a.so.b + head * a.so.h + i * a.so.n + warp * 16);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (warp == 0)
    a.lse[(static_cast<long long>(b) * a.Hq + head) * g.N + i] = none ? -INFINITY : (M - kBias + log2f(sum)) * kLn2Cache;
}

template <int D, bool INT8>
cudaError_t launch_variant(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  cudaError_t e = g.rows > 16  ? (INT8 ? launch_cache_attention_tiles_int8(a, g, ctas, stream)
                                       : launch_cache_attention_tiles_e4m3(a, g, ctas, stream))
                  : g.rows > 8 ? launch_rows<D, 2, INT8>(a, g, ctas, stream)
                               : launch_rows<D, 1, INT8>(a, g, ctas, stream);
  if (e != cudaSuccess || !g.split) return e;
  const long long live = min(static_cast<long long>(g.rows), static_cast<long long>(g.N) * g.G);
  if (g.rows > 16)
    return launch_pdl(cache_attn_merge_tiles_kernel<D>, dim3(ctas, static_cast<unsigned>((live + 31) / 32)), dim3(D * 2), 0,
                      stream, a, g);
  // blocks of a unit: a row each (most CTAs have no record)
  return launch_pdl(cache_attn_merge_kernel<D>, dim3(ctas, static_cast<unsigned>(live)), dim3(256), 0, stream, a, g);
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

// Rows of a unit, from the rows of a (sequence, cache head); GPU time in us at d = 128, pages of 64:
//   up to 8, 16: one or two groups of the few-row kernel (8 rows of 64 sequences 103.2 as one
//     group, 106.0 as two, 156 as a tile; 16 rows 110 and 158);
//   up to 64: a tile with its rows twice (40 rows of 16 sequences 33.1, in a tile of 128 34.8) where
//     the CTAs have 3 steps each; otherwise groups of 16, which start and end sooner though each
//     reads the cache (2 steps a CTA, 32 rows: 18.8 in groups, 24.2 as tiles; 64 rows 22.7 and 26.4;
//     7 steps 28.1 and 25.7; 54 steps 94.3 and 73.8; 1024 units of 4 steps 75.3 and 74.0);
//   up to 128: one tile (128 rows 29.0, in a unit of two tiles 31.3);
//   above: a unit of two tiles, whose step costs some 1.4 times one tile's, where the CTAs have about
//     6 steps each to make good its longer start and larger merge (107 steps a CTA 197, with
//     single tiles 267; 13 steps 45.6 and 51.3; 7 steps 37.1 and 36.9; 3 steps 36.3 and 31.6; 384
//     rows, which leave half a tile empty, at 54 steps 112.9 and 118.7).
// lead: beginning one more unit costs a CTA 1 us (rows of up to 16, steps of 0.7 us) and 5 us (tiles,
// steps of 1 to 2 us); counting it shares ragged batches out more evenly: drafts 39.9 us with
// none, 37.0 with 4, 36.9 with 8; a chunk 243.3, 242.5, 247.0; single tokens of 64 sequences
// 102.7 with none, 101.5 with 1, 101.5 with 4.
AttnPlan attn_plan(int B, int HK, long long rows, long long cap, int d) {
  AttnPlan p{};
  p.log2_keys = 7;
  p.cap_steps = (cap + 127) >> 7;
  if (p.cap_steps < 1) p.cap_steps = 1;
  const long long heads = static_cast<long long>(B) * HK, two = (rows + 255) / 256, enough = 6LL * sm_count();
  const bool wide = rows > 128 && (heads * two >= enough || heads * two * p.cap_steps >= enough);
  const bool brief = heads * p.cap_steps < 3LL * sm_count();  // as tiles of up to 64 rows
  p.rows = rows <= 8 ? 8 : rows <= 16 || (rows <= 64 && brief) ? 16 : rows <= 64 ? 64 : wide ? 256 : 128;
  p.lead = p.rows <= 16 ? 1 : 4;
  p.units = heads * ((rows + p.rows - 1) / p.rows);
  const long long most = (p.rows > 16 ? 1LL : few_row_ctas(d, p.rows)) * sm_count();
  p.ctas = static_cast<int>(p.units >= most || p.units * p.cap_steps >= most ? most : p.units * p.cap_steps);
  return p;
}

// Whether units are cut, from the sizes that the host knows (capacities, not lengths).
// Cutting shares the steps out evenly but adds the merge and, with many rows, units that
// begin within a CTA's run: worth about 6 steps (GPU time in us, cut and whole: single tokens,
// 12 units of 4 steps 10.3, 10.2, of 8 steps 10.3, 12.3; 64 of 8 steps 12.5, 14.4; 192 of 16 steps,
// which saves 5.9, 29.2, 26.0; 320 of 8 steps 26.7, 28.6; 32 tiles of 4 steps 22.6, 20.6, of 8
// steps 24.7, 27.4; 256 tiles of 16 steps 82.7, 79.4). Beyond 16 steps unequal lengths may cost
// more than that, so those are always cut.
static bool attn_cut(const AttnPlan& p) {
  if (p.cap_steps <= 4) return false;
  if (p.cap_steps > 16) return true;
  const long long rounds = (p.units + p.ctas - 1) / p.ctas;
  return static_cast<double>(rounds * p.cap_steps) - static_cast<double>(p.units * p.cap_steps) / p.ctas > 6.1;
}

size_t cache_attention_workspace(int B, int HK, int G, int N, int d, int page, int table_width) {
  const AttnPlan p = attn_plan(B, HK, static_cast<long long>(N) * G, static_cast<long long>(table_width) * page, d);
  return attn_cut(p) ? attn_workspace(p.ctas, p.rows, d).total : 0;
}

cudaError_t launch_cache_attention(const CacheAttnLaunch& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.N) * a.G, cap = static_cast<long long>(a.c.table_width) * a.c.page;
  const AttnPlan p = attn_plan(a.B, a.c.H, rows, cap, a.c.d);
  AttnGrid g{};
  g.B = a.B;
  g.HK = a.c.H;
  g.N = a.N;
  g.G = a.G;
  g.rows = p.rows;
  g.row_tiles = static_cast<int>((rows + p.rows - 1) / p.rows);
  g.log2_keys = p.log2_keys;
  g.lead = p.lead;
  g.cap = static_cast<int>(cap);
  g.causal = a.causal;
  g.kv_len = a.kv_len;
  g.q_len = a.q_len;
  const AttnWorkspace w = attn_workspace(p.ctas, p.rows, a.c.d);
  g.split = attn_cut(p) && a.ws != nullptr && a.ws_bytes >= w.total;
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
