// Attention over the paged 8-bit cache, many query rows per cache head (drafted
// tokens of large groups, chunks of a prompt): tiles of 128 query rows on
// tcgen05. Which calls come here: attn_plan.
//
// Mathematics, units, shares and parts: as in fa_cache_attn.cu. A unit has NQ tiles of
// 128 query rows, whose S = Q K^T and O += P V run as 128 x
// 128 x d products with fp16 operands and fp32 accumulators in TMEM. A task is one
// tile's step; task k uses S buffer k mod 2, and the issue order
//   S(0) S(1) | PV(0) S(2) PV(1) S(3) ...
// lets one task's softmax run under the other's products: the two tiles of a
// unit at NQ = 2, a tile's consecutive steps at NQ = 1.
//
// Warps: 4 NQ softmax warps (a thread owns a query row, the TMEM lane of its
// warp's quarter), 4 / NQ converter warps (codes to fp16 tiles in the swizzled form
// the products read), the MMA issuer, 2 / NQ loaders (TMA copies of whole pages). The codes are
// converted unscaled: K's scale multiplies the scores and V's joins the exponent, both
// constant over 16 columns, so that the converters do nothing but convert.
//
// What bounds it, and what it measured (GPU time, d = 128):
//   Chunks (NQ = 2; 2048 tokens of 16 heads on 4 over 16384, e4m3, pages of 64): 196 us, 1317
//   TFLOP/s with the merge. A step is 2048 cycles of products and takes some 3200: softmax,
//   P V and the next S follow one another within a tile, and the two tiles cover each other only in
//   part. Tensor pipe 58 %, issue slots 45 %, no other pipe above 37 %. Tried and slower: one
//   pass over the scores with the reference moved afterwards (304 us where two passes took 230:
//   spills) or chunk by chunk (326). int8 codes take three instructions on the busiest pipe where
//   e4m3 takes two conversions: 127 us where e4m3 takes 113 (2 sequences of 1024 on 8192), 218 us for the
//   chunk above. At d = 64 that chunk takes 187 us in either format: the exponentials of a step stay.
//   Drafts (REP = 2; 5 tokens of 16 heads on 2, 16 sequences of 2000 to 16384, pages of 16): 35 us,
//   of which 15 steps of 1 us (5 TB/s of codes), 5 us of start, 3 us of end and the merge's 4; 6 to 8
//   are not accounted for.
#pragma once

#include "fa_cache_internal.h"
#include "fa_cache_math.cuh"
#include "fa_cache_sched.cuh"

namespace fa {
namespace {

constexpr int kKeys = 128;
constexpr int kChunkBytes = 128 * 128;  // 128 rows x 64 fp16 columns, 128-byte swizzle
constexpr int kScaleSlots = 8;          // steps whose scales are kept

template <int D, int NQ>
struct TileLayout {
  // NQ = 2: 12 warps, so that a softmax thread can hold a step's 128 scores (168 registers)
  static constexpr int kConvWarps = NQ == 2 ? 2 : 4;
  static constexpr int kConv = 4 * NQ, kMma = kConv + kConvWarps, kLoad = kMma + 1;  // warps
  static constexpr int kLoaders = NQ == 1 ? 2 : 1;  // NQ = 1: a warp each for K and V
  static constexpr int kThreads = (kLoad + kLoaders) * 32;
  static constexpr int kTile = (D / 64) * kChunkBytes;  // one fp16 tile
  static constexpr int kRaw = kKeys * D;                // K or V codes of a step
  static constexpr int kStg = D == 128 ? (NQ == 2 ? 2 : 4) : 8;  // raw tiles in flight
  static constexpr int oQ = 0, oK = NQ * kTile, oV = oK + 2 * kTile, oRaw = oV + 2 * kTile;
  static constexpr int oScales = oRaw + kStg * kRaw;    // [slots][8 groups] ks, log2 vs, 1 / vs, 1 (0: V of zeros, -1: not read)
  static constexpr int oNan = oScales + kScaleSlots * 128;  // [8] first NaN key of V per unit
  // Slots for the descriptions of units (TileUnit). Units have a step at least. The producer
  // describes a unit three steps before it issues K(n), for which K(n - kStg / 2) is
  // converted, so the scores of the step two before that are formed, so the weights of
  // the step NQ = 1: two, NQ = 2: one before that are done; that step's unit may still be read.
  static constexpr int kUnits = kStg <= 2 ? 8 : 16;
  static_assert(3 + kStg / 2 + 2 + (NQ == 1 ? 2 : 1) < kUnits, "a unit's description outlives its use");
  static constexpr int oUnits = oNan + 32;
  static constexpr int oBars = oUnits + kUnits * 32;
  static constexpr int kBars = 2 * kStg + 17 + kUnits + 7;
  static constexpr int kSmem = oBars + kBars * 8 + 16 + 1024;
  static_assert(kSmem + sizeof(AttnShare) + 16 <= 227 * 1024, "shared memory of one CTA");
  static constexpr uint32_t cO = 256;                   // TMEM column of O
};

// A unit (or the CTA's part of one), as the producer writes it down for the other warps,
// which then carry little more than counters through their loops. steps 0: no more.
struct __align__(16) TileUnit {
  int b, row0, h, first;  // sequence, first row, cache head, first step
  int steps, kv, ql, seen_last;  // seen: tokens the last row sees; top bit: the unit ends here
};
__device__ __forceinline__ int unit_limit(const AttnGrid& g, const TileUnit& x, int r) {
  const int i = (x.row0 + r) / g.G;
  if (i >= x.ql) return 0;
  return g.causal ? max(0, x.kv - x.ql + i + 1) : x.kv;
}

// f32 += f16 x f16
constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return idesc_bf16(M, N, false, b_mn_major) & ~((1u << 7) | (1u << 10));
}

struct TileBars {
  uint64_t *raw_full, *raw_empty, *kfull, *kempty, *vfull, *vempty, *qfull, *sfull, *pfull, *odone, *fin, *ufull, *rep_out, *rep_in, *rep_done, *phalf;
};

// Producer: the raw tiles K(n), V(n) of every step, as pages. Lane i < 8 looks
// after the step's i-th group of 16 keys (page id three steps ahead, scales two: one step is
// less than their way from memory).
// With NQ = 1 K and V have a warp each: a step of 16-token pages is 16 copies, which take one
// warp some 75 cycles each to issue. K's also describes the units to the other warps (TileLayout::kUnits), and
// writes the record of a cut unit that the CTA ends, well before that end.
template <int D, int NQ>
__device__ __forceinline__ void tile_produce(const CacheAttnLaunch& a, const AttnGrid& g, AttnCursor ld,
                                             const AttnShare& share, uint8_t* smem, const TileBars& b,
                                             const Watchdog& wd, int loader, int lane) {
  using L = TileLayout<D, NQ>;
  const CacheView& c = a.c;
  const int rows = min(c.page, kKeys), per_page = rows >> 4;
  const bool group = lane < kKeys / 16, leader = group && lane % per_page == 0;
  struct Step {
    bool live, want;
    int pid, h, row;
    float ks, vs;
  };
  int units = 0;
  bool first = true;
  auto describe = [&](const TileUnit& u) {
    if (lane == 0) {
      *reinterpret_cast<TileUnit*>(smem + L::oUnits + units % L::kUnits * 32) = u;
      mbar_arrive(b.ufull + units % L::kUnits);
    }
    ++units;
  };
  auto look = [&]() {
    Step s{!ld.done(g), false, -1, 0, 0, 1.f, 1.f};
    if (s.live) {
      if (loader == 0 && (first || ld.step == 0)) {
        const int steps = ld.run(g);
        const bool ends = ld.step + steps == ld.x.steps;
        describe(TileUnit{ld.x.b, ld.x.row0, ld.h, ld.step, steps, ld.x.kv, ld.x.ql,
                          static_cast<int>(static_cast<unsigned>(ld.x.seen) | (ends ? 0x80000000u : 0u))});
        if (ld.step > 0 && ends && g.split && lane == 0)
          g.record[blockIdx.x] = make_int4(ld.e, ld.h, attn_cta_of(ld.pos - ld.step, share), 0);
        first = false;
      }
      const int key = (ld.step << g.log2_keys) + lane * 16;
      s.want = group && key < ld.x.seen;
      s.h = ld.h;
      s.row = key & (c.page - 1);
      if (s.want) s.pid = c.table[ld.x.b * c.table_stride + (key >> c.log2_page)];
      ld.next(g);
    }
    return s;
  };
  auto scales = [&](Step& s) {
    const bool good = s.want && s.pid >= 0 && s.pid < c.num_pages;
    if (s.want && !good) report_bad_page(a.status);
    s.want = good;
    if (good) {
      const int ph = s.pid * c.H + s.h;
      s.row += ph << c.log2_page;
      s.ks = c.scale[0][ph];
      s.vs = c.scale[1][ph];
    }
  };
  Step now = look(), next = look();
  scales(now);
  scales(next);
  Step third = look();
  int tile = 0, issued = 0;  // raw tiles: K(n) is 2 n, V(n) 2 n + 1
  bool ok = true;
  for (int n = 0; now.live && ok; ++n) {
    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, leader && now.want)) * rows * D;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      if (L::kLoaders == 2 && kv != loader) continue;
      tile = 2 * n + kv;
      const int st = tile % L::kStg;
      if (tile >= L::kStg && !mbar_wait_warp(b.raw_empty + st, ((tile / L::kStg) - 1) & 1, wd)) {
        ok = false;
        break;
      }
      if (leader && now.want)
        tma_load_2d(smem + L::oRaw + st * L::kRaw + lane * 16 * D, &a.tm[kv], b.raw_full + st, now.row);
      if (kv == 0 && group) {
        const bool counts = now.vs > kMinScale;
        const float v = counts ? now.vs : kZeroScale;
        *reinterpret_cast<float4*>(smem + L::oScales + (n % kScaleSlots) * 128 + lane * 16) =
            make_float4(now.ks, __log2f(v), 1.f / v, !now.want ? -1.f : counts ? 1.f : 0.f);
      }
      __syncwarp();
      if (lane == 0) {
        if (bytes > 0)
          mbar_expect_tx(b.raw_full + st, bytes);
        else
          mbar_arrive(b.raw_full + st);
      }
      issued = tile + 1;
    }
    now = next;
    next = third;
    scales(next);  // before the next load of a page id: waiting for one waits for all of its kind
    third = look();
  }
  if (loader == 0) describe(TileUnit{0, 0, 0, 0, 0, 0, 0, 0});
  for (int i = max(0, issued - L::kStg); i < issued; ++i)  // copies in flight land before the CTA exits
    if (L::kLoaders == 1 || (i & 1) == loader) mbar_wait_drain(b.raw_full + i % L::kStg, (i / L::kStg) & 1, a.wait_limit);
}

// V's rows [row0, row0 + rows) of a step that holds keys which a row of queries may not see (from
// `low` on), pages of zeros or groups of keys that were not read: such groups become zeros, and so do pages of
// zeros but for their NaN codes. NaN codes at keys >= low are taken out, and the first such key < seen
// is kept for the unit: the rows that see it look for the channels (seen_nan). A call, because few
// steps come here: within the converters' loop it cost every step (a chunk in int8 131 us, so 127).
template <int D, bool INT8>
__device__ __noinline__ void convert_checked(uint32_t src, uint32_t dst, const float4* scales, int row0, int rows, int key0,
                                             int low, int seen, int* nan_key, int lane) {
#pragma unroll 2
  for (int i = lane; i < rows * (D / 16); i += 32) {  // pieces in tile_convert's order
    const int ch = D == 128 ? (i & 3) | ((i >> 1) & 4) : i & 3;
    const int p = D == 128 ? ((i >> 4) & 3) + 8 * (i >> 6) : i >> 2, r = row0 + (D == 128 && (i & 4) ? p ^ 5 : p), key = key0 + r;
    const uint4 v = lds128(src + (D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)));
    const float counts = scales[r >> 4].w;
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, any = 0u;
    if (counts != 1.f) {
      const bool keep = !INT8 && counts == 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] &= keep ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) : 0u;
    }
    if (!INT8 && key >= low) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t nan = __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        w[k] &= ~nan;
        any |= nan;
      }
      if (any != 0u && key < seen) atomicMin(nan_key, key);
    }
    const uint32_t at = dst + (D == 128 ? (ch >> 2) * kChunkBytes : 0) + r * 128 + (((ch & 3) * 2 ^ (r & 7)) << 4);
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) decode4<INT8>(w[k], h[2 * k], h[2 * k + 1]);
    st_shared_v4(at, h[0], h[1], h[2], h[3]);
    st_shared_v4(at ^ 16u, h[4], h[5], h[6], h[7]);
  }
}

// Converters: each warp takes its 32 (64) rows of every raw tile, 16 codes a lane at a
// time. At d = 128 the 8 lanes of a shared-memory phase take four chunks of rows r
// and r ^ 5: the rows differ in bit 2 (so their raw chunks, at c ^ (r & 7), fall
// apart) and in bit 0 (so do the results, at 2 c ^ (r & 7)), and every bank is met
// once in both directions.
template <int D, int NQ, bool INT8>
__device__ __forceinline__ void tile_convert(const CacheAttnLaunch& a, const AttnGrid& g, uint8_t* smem,
                                             const TileBars& b, const Watchdog& wd, int cw, int lane) {
  using L = TileLayout<D, NQ>;
  // The lane's pieces: chunk ch of its row of 8 + 8 g, e < kPer, g < kGroups, at constant
  // distances of a piece with g = 0 (both swizzles repeat every 8 rows).
  constexpr int kRows = kKeys / L::kConvWarps, kPer = D / 64, kGroups = kRows / 8;
  const int ch = D == 128 ? (lane & 3) | ((lane >> 1) & 4) : lane & 3;
  uint32_t raw_at[kPer], half_at[kPer];  // in the raw and the fp16 tile; the second half's place is the first's ^ 16
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int p = D == 128 ? (lane >> 4) + 2 * e : lane >> 2, r = cw * kRows + (D == 128 && (lane & 4) ? p ^ 5 : p);
    raw_at[e] = D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
    half_at[e] = (D == 128 ? (ch >> 2) * kChunkBytes : 0) + r * 128 + (((ch & 3) * 2 ^ (r & 7)) << 4);
  }
  int* const nan_key = reinterpret_cast<int*>(smem + L::oNan);
  int n = 0;  // steps converted
  for (int unit = 0;; ++unit) {
    if (!mbar_wait_warp(b.ufull + unit % L::kUnits, (unit / L::kUnits) & 1, wd)) return;
    const TileUnit x = *reinterpret_cast<const TileUnit*>(smem + L::oUnits + unit % L::kUnits * 32);
    if (x.steps == 0) return;
    // slot of the unit three on; the one five back, which used it, has ended (a unit
    // has a step at least, and K(n) waits for the scores of step n - 2)
    if (cw == 0 && lane == 0) nan_key[(unit + 3) & 7] = 0x7fffffff;
    const int seen = x.seen_last & 0x7fffffff, low = unit_limit(g, x, 0);
    int key0 = x.first << g.log2_keys;
    for (const int end = n + x.steps; n < end; ++n, key0 += kKeys) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int tile = 2 * n + kv, st = tile % L::kStg, slot = n & 1;
        if (!mbar_wait_warp(b.raw_full + st, (tile / L::kStg) & 1, wd)) return;
        if (n >= 2 && !mbar_wait_warp((kv ? b.vempty : b.kempty) + slot, ((n >> 1) - 1) & 1, wd)) return;
        const uint32_t src = smem_u32(smem) + L::oRaw + st * L::kRaw;
        const uint32_t dst = smem_u32(smem) + (kv ? L::oV : L::oK) + slot * L::kTile;
        bool check = false;
        if (kv == 1) {
          const float counts = *reinterpret_cast<const float*>(smem + L::oScales + (n % kScaleSlots) * 128 + (lane & 7) * 16 + 12);
          check = (!INT8 && key0 + kKeys > low) || __any_sync(0xffffffffu, counts != 1.f);
        }
        auto put = [&](const uint4& v, int e, int g) {
          uint32_t w[8];
          decode4<INT8>(v.x, w[0], w[1]);
          decode4<INT8>(v.y, w[2], w[3]);
          decode4<INT8>(v.z, w[4], w[5]);
          decode4<INT8>(v.w, w[6], w[7]);
          st_shared_v4(dst + half_at[e] + g * 1024, w[0], w[1], w[2], w[3]);
          st_shared_v4(dst + (half_at[e] ^ 16u) + g * 1024, w[4], w[5], w[6], w[7]);
        };
        if (!check) {
          constexpr int kBatch = D / 16;  // loads in flight
#pragma unroll 1
          for (int g0 = 0; g0 < kGroups; g0 += kBatch / kPer) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = lds128(src + raw_at[i % kPer] + (g0 + i / kPer) * (8 * D));
#pragma unroll
            for (int i = 0; i < kBatch; ++i) put(v[i], i % kPer, g0 + i / kPer);
          }
        } else {
          convert_checked<D, INT8>(src, dst, reinterpret_cast<const float4*>(smem + L::oScales + (n % kScaleSlots) * 128), cw * kRows,
                                   kRows, key0, low, seen, nan_key + (unit & 7), lane);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive((kv ? b.vfull : b.kfull) + slot);
          mbar_arrive(b.raw_empty + st);
        }
      }
    }
  }
}

// Copies a warp's 32 rows of queries (lane r knows row r's offset, -1: zeros) into the
// swizzled tile at `dst`, D / 8 lanes to a row. fp16 rows already are what the products take;
// bf16 rows become fp16 there, scaled by a power of two that puts their largest value into
// [2^14, 2^15): a lane takes its own row, and its inverse factor comes back. Short loops: this
// runs once a unit, and code met for the first time costs more than its instructions (unrolled,
// with the rows in registers, 4.5 us for a CTA's first unit and 2.6 us for its next).
template <int D>
__device__ __forceinline__ float tile_queries(const uint16_t* q, long long q_at, bool fp16, uint32_t dst, int lane) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows at once
  const int c = lane % kLanes, sub = lane / kLanes;
  auto place = [&](int r, int chunk) { return dst + (chunk >> 3) * kChunkBytes + r * 128 + (((chunk & 7) ^ (r & 7)) << 4); };
#pragma unroll 2
  for (int r = sub; r < 32; r += kAtOnce) {
    const long long at = __shfl_sync(0xffffffffu, q_at, r);
    cp_async_16(place(r, c), q + (at >= 0 ? at + c * 8 : 0), at >= 0 ? 16u : 0u);
  }
  cp_async_wait();
  __syncwarp();
  if (fp16) return 1.f;
  uint32_t mx = 0u;  // the largest magnitude as an integer: bf16 patterns order like their values
#pragma unroll 4
  for (int i = 0; i < kLanes; ++i) {
    const uint4 w = lds128(place(lane, i));
    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
  }
  const int e = max(15, static_cast<int>(max(mx & 0xffffu, mx >> 16) >> 7));
  const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
  auto half2_of = [&](uint32_t w) { return pack_half(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f); };
#pragma unroll 4
  for (int i = 0; i < kLanes; ++i) {
    const uint4 w = lds128(place(lane, i));
    st_shared_v4(place(lane, i), half2_of(w.x), half2_of(w.y), half2_of(w.z), half2_of(w.w));
  }
  return __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
}

static __device__ __noinline__ unsigned long long seen_nan64(const CacheView& c, int b, int h, int first, int end, int c0) {
  return seen_nan<16>(c, b, h, first, end, c0);
}

// Writes 32 rows x 128 bytes, a lane's row as 8 pieces, to the rows' own places: through `box`
// (4 KB of shared memory, pieces permuted within a row), so that 8 lanes write a row's bytes
// together. at: of row `lane`, nullptr: not written.
__device__ __forceinline__ void store_rows(uint32_t box, const uint4 (&w)[8], uint8_t* at, int lane) {
  __syncwarp();  // the box's last pieces have been read
#pragma unroll
  for (int i = 0; i < 8; ++i) st_shared_v4(box + lane * 128 + ((i ^ (lane & 7)) << 4), w[i].x, w[i].y, w[i].z, w[i].w);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = k * 4 + lane / 8;
    const uint4 v = lds128(box + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
    uint8_t* const p = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(at), r));
    if (p != nullptr) *reinterpret_cast<uint4*>(p + (lane & 7) * 16) = v;
  }
}

// The largest of N scores from column c0 of a chunk.
template <int N>
__device__ __forceinline__ float largest_of(const uint32_t (&v)[32], int c0) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = __uint_as_float(v[c0 + i]);
#pragma unroll
  for (int q = 4; q + 8 <= N; q += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m[i] = max3(m[i], __uint_as_float(v[c0 + q + i]), __uint_as_float(v[c0 + q + 4 + i]));
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], __uint_as_float(v[c0 + N - 4 + i]));
  return max3(max3(m[0], m[1], m[2]), m[3], m[3]);
}

// Weights 2^(v mul + add) of 16 scores, packed to fp16 pairs; their sum comes back,
// unrounded. Pairs of columns share the packed fp32 instructions.
__device__ __forceinline__ float weigh16(const uint32_t (&v)[32], int c0, float mul, float add, uint32_t (&p)[8]) {
  const uint64_t mul2 = f2_pack(mul, mul), add2 = f2_pack(add, add);
  uint64_t sum = 0ull;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c0 + 2 * q]), __uint_as_float(v[c0 + 2 * q + 1])), mul2, add2), x0, x1);
    const float w0 = ex2(x0), w1 = ex2(x1);
    p[q] = pack_half(w0, w1);
    sum = f2_add(sum, f2_pack(w0, w1));
  }
  float s0, s1;
  f2_unpack(sum, s0, s1);
  return s0 + s1;
}

// P16: pages of 16 tokens, whose scales change every 16 columns (32 and more
// otherwise). REP = 2 (units of up to 64 rows): the rows stand in the tile twice, and each
// copy's warps take half of a step's keys, with weights of zero for the others; a unit ends
// with the copies joined. All four softmax warps then work, each on half the columns.
template <int D, int NQ, int REP, bool INT8, bool P16>
__global__ void __launch_bounds__(TileLayout<D, NQ>::kThreads, 1)
    cache_attn_tile_kernel(const __grid_constant__ CacheAttnLaunch a, const AttnGrid g) {
  using L = TileLayout<D, NQ>;
  // The weights are handed over in halves of 64 keys, so that P V begins under the second
  // half's exponentials: a chunk in e4m3 207.0 us as a whole, 197.3 in halves; in int8, where
  // the converters are behind, 219.4 and 221.3; in units of one tile (384 rows, e4m3) 118.7 and 130.2.
  constexpr bool kHalves = NQ == 2 && !INT8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnShare share;
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  TileBars b;
  {
    uint64_t* p = reinterpret_cast<uint64_t*>(smem + L::oBars);
    b.raw_full = p;
    b.raw_empty = p + L::kStg;
    p += 2 * L::kStg;
    b.kfull = p;
    b.kempty = p + 2;
    b.vfull = p + 4;
    b.vempty = p + 6;
    b.qfull = p + 8;
    b.sfull = p + 10;
    b.pfull = p + 12;
    b.odone = p + 14;
    b.fin = p + 16;
    b.ufull = p + 17;
    b.rep_out = p + 17 + L::kUnits;  // [2] pairs of warps
    b.rep_in = b.rep_out + 2;        // [2]
    b.rep_done = b.rep_out + 4;
    b.phalf = b.rep_out + 5;         // [2]
  }
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::oBars + L::kBars * 8);
  int* const abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  check_init(a.status);
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStg; ++i) {
      mbar_init(b.raw_full + i, 1);
      mbar_init(b.raw_empty + i, L::kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b.kfull + i, L::kConvWarps);
      mbar_init(b.kempty + i, 1);
      mbar_init(b.vfull + i, L::kConvWarps);
      mbar_init(b.vempty + i, 1);
      mbar_init(b.qfull + i, 4);
      mbar_init(b.sfull + i, 1);
      mbar_init(b.pfull + i, 4);
      mbar_init(b.phalf + i, 4);
      mbar_init(b.odone + i, 1);
    }
    mbar_init(b.fin, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b.rep_out + i, 1);
      mbar_init(b.rep_in + i, 1);
    }
    mbar_init(b.rep_done, 2);
    for (int i = 0; i < L::kUnits; ++i) mbar_init(b.ufull + i, 1);
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) reinterpret_cast<int*>(smem + L::oNan)[i] = 0x7fffffff;
    fence_mbar_init();
    tma_prefetch_desc(&a.tm[0]);
    tma_prefetch_desc(&a.tm[1]);
  }
  if (warp == L::kMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  grid_dep_wait();
  grid_dep_launch();
  // its barriers publish the above; the slots of the scales are not in use yet
  AttnCursor cur = attn_share<L::kThreads>(g, &share, reinterpret_cast<long long*>(smem + L::oScales));
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{a.wait_limit, a.status, abort_flag};
  if (warp >= L::kLoad) {
    if (g.split && warp == L::kLoad && lane == 0) g.record[blockIdx.x] = make_int4(-1, 0, 0, 0);
    tile_produce<D, NQ>(a, g, cur, share, smem, b, wd, warp - L::kLoad, lane);
  } else if (warp == L::kMma) {
    // ------------------------------------------------------------ MMA issuer (whole warp)
    constexpr uint32_t kIdS = idesc_f16(128, 128, false), kIdO = idesc_f16(128, D, true);
    const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::oQ), 16, 1024);
    const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::oK), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::oV), kChunkBytes, 1024);  // MN-major
    int task0 = 0, step0 = 0;  // of the unit, over the CTA's run
    bool ok = true;
    for (int unit = 0; ok; ++unit) {
      if (!mbar_wait_spin_w(b.ufull + unit % L::kUnits, (unit / L::kUnits) & 1, wd)) break;
      const int steps = reinterpret_cast<const TileUnit*>(smem + L::oUnits + unit % L::kUnits * 32)->steps, tasks = steps * NQ;
      if (steps == 0) break;
      for (int t = 0; ok && t < NQ; ++t) ok = mbar_wait_spin_w(b.qfull + t, unit & 1, wd);
      if (!ok) break;
      auto issue_s = [&](int i) -> bool {
        const int t = NQ == 2 ? i & 1 : 0, n = step0 + (NQ == 2 ? i >> 1 : i), buf = (task0 + i) & 1;
        if (!mbar_wait_spin_w(b.kfull + (n & 1), (n >> 1) & 1, wd)) return false;
        tc_fence_after();  // the softmax has read the buffer's last scores (pfull was awaited)
        const uint64_t qd = desc_adv(q_desc, t * L::kTile), kd = desc_adv(k_desc, (n & 1) * L::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
          mma_ss_w(tmem + buf * 128, desc_adv(qd, off), desc_adv(kd, off), kIdS, kk > 0 ? 1u : 0u);
        }
        mma_commit_w(b.sfull + buf);
        if (t == NQ - 1) mma_commit_w(b.kempty + (n & 1));
        return true;
      };
      auto issue_pv = [&](int i) -> bool {
        const int t = NQ == 2 ? i & 1 : 0, n = step0 + (NQ == 2 ? i >> 1 : i), buf = (task0 + i) & 1;
        const uint32_t ph = ((task0 + i) >> 1) & 1;
        if (!mbar_wait_spin_w((kHalves ? b.phalf : b.pfull) + buf, ph, wd)) return false;
        if (!mbar_wait_spin_w(b.vfull + (n & 1), (n >> 1) & 1, wd)) return false;
        tc_fence_after();
        const uint64_t vd = desc_adv(v_desc, (n & 1) * L::kTile);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) {
          if (kHalves && kk == kKeys / 32) {  // the second half of the weights
            if (!mbar_wait_spin_w(b.pfull + buf, ph, wd)) return false;
            tc_fence_after();
          }
          mma_ts_w(tmem + L::cO + t * D, tmem + buf * 128 + kk * 8, desc_adv(vd, kk * 2048), kIdO,
                   (kk > 0 || i >= NQ) ? 1u : 0u);
        }
        mma_commit_w(b.odone + buf);
        if (t == NQ - 1) mma_commit_w(b.vempty + (n & 1));
        return true;
      };
      ok = issue_s(0);
      if (ok && tasks > 1) ok = issue_s(1);
      for (int i = 0; ok && i < tasks; ++i) {
        ok = issue_pv(i);
        if (ok && i + 2 < tasks) ok = issue_s(i + 2);
      }
      task0 += tasks;
      step0 += steps;
    }
    mma_commit_w(b.fin);
    mbar_wait_drain(b.fin, 0, a.wait_limit);
    __syncwarp();
  } else if (warp >= L::kConv && warp < L::kMma) {
    tile_convert<D, NQ, INT8>(a, g, smem, b, wd, warp - L::kConv, lane);
  } else if (warp < L::kConv) {
    // ------------------------------------------------------------ softmax
    static_assert(REP == 1 || NQ == 1, "copies of rows stand in one tile");
    constexpr int kCols = kKeys / REP, kChunks = kCols / 32;  // this warp's columns
    const int t = NQ == 2 ? warp >> 2 : 0;
    const int rep = REP == 2 ? (warp >> 1) & 1 : 0, pair = warp & 1;
    const int rl = (REP == 2 ? pair : warp & 3) * 32 + lane;  // row of the unit's tile
    const int col0 = rep * kCols;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // this warp's rows of the tile of queries: also its box for whole rows on their way out
    const uint32_t q_at = smem_u32(smem) + L::oQ + t * L::kTile + (warp & 3) * 4096;
    int task = t, step_n = 0;  // of this tile; steps so far (for the slots of the scales)
    for (int unit = 0;; ++unit) {
      if (!mbar_wait_warp<true>(b.ufull + unit % L::kUnits, (unit / L::kUnits) & 1, wd)) break;
      const TileUnit* const ux = reinterpret_cast<const TileUnit*>(smem + L::oUnits + unit % L::kUnits * 32);
      const int steps = ux->steps;
      if (steps == 0) break;
      int lim, low;
      float rf;
      bool live;
      {
        const TileUnit x = *ux;
        if (REP == 2 && unit > 0 && !mbar_wait_warp<true>(b.rep_done, (unit - 1) & 1, wd)) break;
        const int row = x.row0 + t * 128 + rl, qi = row / g.G;
        lim = unit_limit(g, x, t * 128 + rl);
        // The warp's 32 rows of queries to fp16, scaled by a power of two each, into the
        // swizzled tile (the last unit's scores are done: its last P V was awaited).
        const long long at = qi < x.ql ? x.b * a.sq.b + static_cast<long long>(x.h * g.G + (row - qi * g.G)) * a.sq.h + qi * a.sq.n : -1;
        rf = a.scale_log2 * tile_queries<D>(a.q, at, a.fp16, q_at, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b.qfull + t);
        live = __any_sync(0xffffffffu, lim > 0);  // rows of this warp see keys
        // rows that stand for no query (their q is zero) do not make a step an edge
        low = __reduce_min_sync(0xffffffffu, qi < x.ql ? lim : 0x7fffffff) - (x.first << g.log2_keys) - col0;
        lim -= (x.first << g.log2_keys) + col0;  // both from here on relative to the step's first key of these columns
      }
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < steps; ++j, task += NQ, ++step_n, lim -= kKeys, low -= kKeys) {
        const uint32_t s_tm = lane_base + (task & 1) * 128;
        if (!mbar_wait_warp<true>(b.sfull + (task & 1), (task >> 1) & 1, wd)) {
          ok = false;
          break;
        }
        tc_fence_after();
        auto half_done = [&]() {  // the first half of the weights stands
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b.phalf + (task & 1));
        };
        if (kHalves && !live) half_done();
        if (live) {
          // constants of the step's groups of 16 columns (plain loads, free to move ahead of
          // the stores to TMEM below)
          const float4* const scp = reinterpret_cast<const float4*>(smem + L::oScales + (step_n % kScaleSlots) * 128) + col0 / 16;
          auto sc = [&](int i) { return scp[i]; };
          // The whole row at once, held: a round trip to TMEM takes about 300 cycles while
          // products run, whatever it brings.
          uint32_t v[kChunks][32];
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tmem_ld32(s_tm + col0 + c * 32, v[c]);
          // whether every row sees every key, and every page was read and counts
          const bool plain = kCols <= low && !__any_sync(0xffffffffu, sc(lane & (kCols / 16 - 1)).w != 1.f);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kChunks; ++c) reg_fence(v[c]);
          if (!plain) {
#pragma unroll
            for (int u = 0; u < kCols / 16; ++u) {
              const int lim16 = sc(u).w < 0.f ? 0 : lim - u * 16;
#pragma unroll
              for (int q = 0; q < 16; ++q)
                v[u >> 1][(u & 1) * 16 + q] = q < lim16 ? v[u >> 1][(u & 1) * 16 + q] : 0xff800000u;
            }
          }
          // the largest y of the row; the factor stays above zero, so that masked scores stay at -inf
          constexpr int kG = P16 ? 16 : 32;  // columns that share their scales
          float tmax = -INFINITY;
#pragma unroll
          for (int u = 0; u < kCols / kG; ++u) {
            const float4 f = sc(u * (kG / 16));
            tmax = fmaxf(tmax, fmaf(largest_of<kG>(v[u * kG / 32], (u * kG) & 31), fmaxf(rf * f.x, 1e-37f), f.y));
          }
          const bool grow = tmax > m + kSlack;
          const bool moved = __any_sync(0xffffffffu, grow);
          const float alpha = grow ? ex2(m - tmax) : 1.f;
          if (grow) m = tmax;
          l *= alpha;
          const float base = (m == -INFINITY ? 0.f : m) - kBias;
          // the weights, over the first half of the score columns
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t p[2][8];
            float part[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float4 f = sc(c * 2 + (P16 ? u : 0));
              part[u] = f.z * weigh16(v[c], u * 16, fmaxf(rf * f.x, 1e-37f), f.y - base, p[u]);
            }
            l += part[0] + part[1];
            tmem_st8x2(s_tm + col0 / 2 + c * 16, p);
            // Between the halves also a line that the compiler does not schedule across: without
            // one the chunk spilled registers (221 us where 212).
            if (kChunks == 4 && c == 1) {
              if (kHalves && !moved)
                half_done();
              else
                __syncwarp();
            }
          }
          if constexpr (REP == 2) {  // the other copy's keys
            const uint32_t none[2][8] = {};
#pragma unroll
            for (int c = 0; c < kChunks; ++c) tmem_st8x2(s_tm + (kCols - col0) / 2 + c * 16, none);
          }
          if (moved && j > 0) {  // the tile's last P V is done before O is rescaled
            const int kp = task - NQ;
            if (!mbar_wait_warp<true>(b.odone + (kp & 1), (kp >> 1) & 1, wd)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              const uint32_t at = lane_base + L::cO + t * D + c * 32;
              uint32_t o[32];
              tmem_ld32(at, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
              tmem_st32(at, o);
            }
          }
          if (kHalves && moved) half_done();
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b.pfull + (task & 1));
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (!mbar_wait_warp<true>(b.odone + ((task - NQ) & 1), ((task - NQ) >> 1) & 1, wd)) break;
      tc_fence_after();
      const uint32_t o_tm = lane_base + L::cO + t * D;
      // rows leave through boxes of 4 KB in the tile of queries, which is done with: this warp's
      // own part of it; REP = 2: the places where the other copy left them
      const uint32_t box = REP == 2 ? smem_u32(smem) + L::oQ + pair * (L::kTile / 2) : q_at;
      float f0 = 1.f, f1 = 0.f;  // REP = 2: what both copies' O are multiplied by
      if constexpr (REP == 2) {
        if (rep == 1) {
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(box + lane * 8), "f"(m), "f"(l) : "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(b.rep_out + pair);
          if (!mbar_wait_warp<true>(b.rep_in + pair, unit & 1, wd)) break;
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[2][32];
#pragma unroll
            for (int e = 0; e < 2; ++e) tmem_ld32(o_tm + (c * 2 + e) * 32, o[e]);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              reg_fence(o[e]);
#pragma unroll
              for (int v = 0; v < 8; ++v)
                st_shared_v4(box + (c * 2 + e) * 4096 + v * 512 + lane * 16, o[e][4 * v], o[e][4 * v + 1], o[e][4 * v + 2], o[e][4 * v + 3]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(b.rep_out + pair);
          tc_fence_before();
          continue;
        }
        if (!mbar_wait_warp<true>(b.rep_out + pair, 0, wd)) break;
        const uint2 other = lds64(box + lane * 8);
        __syncwarp();
        if (lane == 0) mbar_arrive(b.rep_in + pair);
        const float M = fmaxf(m, __uint_as_float(other.x)), base = M == -INFINITY ? 0.f : M;
        f0 = ex2(m - base);
        f1 = ex2(__uint_as_float(other.x) - base);
        l = l * f0 + __uint_as_float(other.y) * f1;
        m = M;
        if (!mbar_wait_warp<true>(b.rep_out + pair, 1, wd)) break;
      }
      const TileUnit x = *ux;
      const int r = t * 128 + rl, row = x.row0 + r, qi = row / g.G, head = x.h * g.G + (row - qi * g.G);
      int nan_key = 0x7fffffff, end = 0;  // keys of V with a NaN that was taken out, and seen by this row
      if (!INT8) {
        nan_key = *reinterpret_cast<volatile int*>(smem + L::oNan + (unit & 7) * 4);
        end = unit_limit(g, x, r);
      }
      // 64 channels of the row's O, from column 64 c
      auto read_o = [&](int c, uint32_t (&o)[2][32]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) tmem_ld32(o_tm + (c * 2 + e) * 32, o[e]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          reg_fence(o[e]);
          if constexpr (REP == 2) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const uint4 w = lds128(box + (c * 2 + e) * 4096 + v * 512 + lane * 16);
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                o[e][4 * v + q] = __float_as_uint(__uint_as_float(o[e][4 * v + q]) * f0 + __uint_as_float(ww[q]) * f1);
            }
          }
        }
        if (!INT8 && nan_key < end) {
          const unsigned long long nan = seen_nan64(a.c, x.b, x.h, nan_key, end, c * 64);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (nan >> (e * 32 + q) & 1ull) o[e][q] = 0x7fffffffu;
        }
      };
      if (qi >= x.ql) {
        l = 0.f;
        m = -INFINITY;
      }
      const bool none = l == 0.f, row_ok = qi < g.N;
      if (x.first == 0 && x.seen_last < 0) {  // the whole unit
        const float inv = none ? 0.f : 1.f / l;
        uint16_t* const dst = a.o + x.b * a.so.b + static_cast<long long>(head) * a.so.h + qi * a.so.n;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[2][32];
          read_o(c, o);
          uint4 w[8];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            uint32_t hw[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int k = (v & 3) * 8 + 2 * q;
              hw[q] = none ? 0u : pack16(__uint_as_float(o[v >> 2][k]) * inv, __uint_as_float(o[v >> 2][k + 1]) * inv, a.fp16);
            }
            w[v] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          }
          store_rows(box + (REP == 2 ? c * 8192 : 0), w, row_ok ? reinterpret_cast<uint8_t*>(dst + c * 64) : nullptr, lane);
        }
        if (row_ok)
          a.lse[(static_cast<long long>(x.b) * a.Hq + head) * g.N + qi] = none ? -INFINITY : (m - kBias + log2f(l)) * kLn2Cache;
      } else {
        // a part, in the order of the registers: 512 bytes a warp and store
        const long long pr = static_cast<long long>(2 * blockIdx.x + (x.first == 0 ? 1 : 0)) * g.rows + r;
        if (row_ok) {
          g.m_part[pr] = m;
          g.l_part[pr] = l;
        }
        uint4* const dst = reinterpret_cast<uint4*>(g.o_part) + (pr >> 5) * (D / 4 * 32) + lane;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[2][32];
          read_o(c, o);
          if (row_ok) {  // rows that see nothing leave zeros: their accumulators hold whatever P was
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const uint32_t* const w = o[v >> 3] + (v & 7) * 4;
              dst[(c * 16 + v) * 32] = none ? make_uint4(0, 0, 0, 0) : make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      __syncwarp();       // the boxes have been read
      tc_fence_before();  // O is read before the next unit's P V
      if (REP == 2 && lane == 0) mbar_arrive(b.rep_done);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int NQ, int REP, bool INT8, bool P16>
cudaError_t launch_tile_variant(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  using L = TileLayout<D, NQ>;
  auto kern = cache_attn_tile_kernel<D, NQ, REP, INT8, P16>;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = set_smem_once(smem_set, reinterpret_cast<const void*>(kern), L::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(L::kThreads), L::kSmem, stream, a, g);
}

template <int D, bool INT8, bool P16>
cudaError_t launch_tile_rows(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  if (g.rows == 64) return launch_tile_variant<D, 1, 2, INT8, P16>(a, g, ctas, stream);
  return g.rows == 128 ? launch_tile_variant<D, 1, 1, INT8, P16>(a, g, ctas, stream)
                       : launch_tile_variant<D, 2, 1, INT8, P16>(a, g, ctas, stream);
}

template <int D, bool INT8>
cudaError_t launch_tiles(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  return a.c.page == 16 ? launch_tile_rows<D, INT8, true>(a, g, ctas, stream)
                        : launch_tile_rows<D, INT8, false>(a, g, ctas, stream);
}

}  // namespace
}  // namespace fa
