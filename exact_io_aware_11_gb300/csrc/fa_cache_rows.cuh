// Attention over the paged 8-bit cache in units of 8 or 16 query rows per cache head
// (single tokens, drafted ones, up to 64 rows over short caches: attn_plan).
//
// Mathematics: with codes kc, vc and scales ks, vs of each page,
//   x_j = scale log2e ks (q . kc_j),  y_j = x_j + log2 vs_j,  M = max_j y_j,
//   w_j = 2^(y_j - M + 7),  O = sum_j w_j vc_j / sum_j w_j / vs_j,
//   LSE = (M - 7 + log2 sum_j w_j / vs_j) ln 2.
// Taking V's scale into the exponent keeps it out of the products, and the
// running maximum then sits on the weight that V is really given: the weights are
// rounded to fp16 (11 bits, against bf16's 8) and 2^21 below the reference
// they still have all of them. The sum is formed from the unrounded weights. Codes of
// either format are exact in fp16. A row of q is scaled by a power of two so that
// its largest value lies in [2^14, 2^15): exact for every value within 2^-28 of it.
//
// What bounds it: reading the cache, d bytes per token, head and tensor. A CTA
// is one producer warp, which walks the page table and fills a ring of stages
// (128 keys, K and V: 32 KB at d = 128) with TMA copies of whole pages, and four
// consumer warps, each with 32 keys of every stage and a softmax of its own, which
// meet only when a unit ends. The reference maximum moves only when a weight
// would pass 2^15, so that most tiles need no reduction across lanes. Products run
// on the warp matrix instruction with keys (K) and channels (V) on its 16 rows and
// the query rows on its 8 columns, so that a group of 8 query rows costs one pass
// over the converted codes: the tcgen05 form needs 128 rows and would convert
// through shared memory.
//
// Measured (GPU time): one token of 64 sequences of 1000 to 8192, 32 heads on 8, d = 128, e4m3: 101
// to 102.6 us, 5900 GB/s; 16 heads on 16 (16 sequences of 8192) 92 us, 5840 GB/s; 64
// sequences of 4096, 12 heads, d = 64: 75 us, 5370 GB/s, where scores and weights weigh twice as
// much beside a row's bytes; one sequence of 131071, 16 heads on 4, int8: 33.5 us, 4000 GB/s, of which
// 17 us stream at the memory's rate, 2 us share the steps out, 3 us bring the first tile and 4 us
// merge; one of 1024, 12 heads, d = 64: 10.3 us, launches and latencies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache_internal.h"
#include "fa_cache_math.cuh"
#include "fa_cache_sched.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;                    // consumer warps; the producer follows them
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kTile = 32;                    // keys of a warp's tile
constexpr int kKeys = kWarps * kTile;        // keys of a step

// CTAs of the few-row kernel that an SM holds: at d = 64 with one group of rows its registers
// leave room for a third, which hides more of the steps' latencies (64 sequences of 4096, 12
// heads: 75 us, with two 90).
constexpr int few_row_ctas(int d, int rows) { return d == 64 && rows <= 8 ? 3 : 2; }

template <int D, int NT>
struct Layout {
  static constexpr int kCtas = few_row_ctas(D, 8 * NT);  // on an SM
  static constexpr int kStages = D == 128 ? 3 : kCtas == 3 ? 4 : 6;
  static constexpr int kMat = kKeys * D;               // K or V of a step
  static constexpr int kStage = 2 * kMat;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kScales = kRing;                // [stages][8 groups of 16 keys] ks, vs
  static constexpr int kQuery = kScales + kStages * 64;  // NT = 2: fragments of q, rows' factors
  static_assert(kWarps * 8 * NT * D * 4 <= kStage, "the warps' O of a unit fits a stage");
  static constexpr int kBars = kQuery + (NT > 1 ? NT * (D / 16) * 256 + NT * 32 : 0);
  static constexpr int kSmem = kBars + 2 * kStages * 8 + 1024;  // slack: 1024-byte alignment
  static_assert(kCtas * (kSmem + 1024 + 1024) <= 228 * 1024, "kCtas CTAs on an SM");
};

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

// Byte offset of 16-byte chunk c of row r in a tile, as the TMA copy's swizzle
// leaves it: the reads of 8 lanes meet all banks (d = 64: of V, half of them).
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// One row of queries as it lies in memory, zeros where it is none: lane t of the row's four has channels
// [D/4 t, D/4 (t + 1)).
template <int D, bool SH>
__device__ __forceinline__ void load_query(const uint16_t* row, bool real, int t, uint4 (&w)[D / 32]) {
#pragma unroll
  for (int v = 0; v < D / 32; ++v)
    w[v] = real ? attn_load<SH>(reinterpret_cast<const uint4*>(row + t * (D / 4)) + v) : make_uint4(0, 0, 0, 0);
}
// The same in fp16, scaled by a power of two (its inverse comes back).
template <int D>
__device__ __forceinline__ float scale_query(const uint4 (&raw)[D / 32], bool fp16, uint32_t (&q)[D / 8]) {
  float x[D / 4];
  float mx = 0.f;
#pragma unroll
  for (int v = 0; v < D / 32; ++v) {
    const uint32_t ww[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
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

// A weight of zero does not mask a NaN. Where not every row of a unit sees all
// of a tile (its keys may be leftovers behind the sequence's end), V's NaN codes
// (e4m3 0x7f, 0xff) are taken out of it; the first key that had one comes back, 0x7fffffff if there
// was none. `gone`: no row sees any (a page that was not read). Lane: keys key, + 1, + 8, + 9.
template <int W>
__device__ __forceinline__ int take_out_nan(uint32_t (&v)[4][W], bool gone, int key) {
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
  return gone ? 0x7fffffff : __reduce_min_sync(0xffffffffu, first);
}
// The rows of a unit that see such keys, of which `first` is the least, get NaN in the channels
// that have it: in O, or in the part that the unit leaves, where this thread has just written them.
// A call after the rows, because it is rare: code among theirs cost launches without any NaN 0.6 of 10 us.
template <int D, int NT>
__device__ __noinline__ void put_nan(const CacheAttnLaunch& a, int b, int row0, int kv, int ql, int h, int first,
                                     float* o_part, int warp, int lane) {
  constexpr int kPer = D / 32;
  const int d0 = lane * kPer;
  for (int r = warp; r < 8 * NT; r += kWarps) {
    const int row = row0 + r, i = row / a.G, end = i >= ql ? 0 : a.causal ? kv - ql + i + 1 : kv;  // attn_limit
    const unsigned nan = static_cast<unsigned>(seen_nan<1>(a.c, b * a.c.table_stride, h, first, end, d0 & ~3)) >> (d0 & 3);
    uint16_t* const o = a.o + b * a.so.b + (h * a.G + (row - i * a.G)) * a.so.h + i * a.so.n + d0;
#pragma unroll
    for (int d = 0; d < kPer; ++d) {
      if (!(nan >> d & 1u)) continue;
      if (o_part != nullptr)
        o_part[r * D + d0 + d] = __int_as_float(0x7fffffff);
      else
        o[d] = 0x7fffu;  // NaN in bf16 and in fp16
    }
  }
}

// The same for an entry of a list (SharedGrid::entry).
template <int D, int NT>
__device__ __noinline__ void put_nan_shared(const CacheAttnLaunch& a, const int* member, SharedEntry x, int h, int first,
                                            float* o_part, int warp, int lane) {
  constexpr int kPer = D / 32;
  const int d0 = lane * kPer;
  SharedGrid g{};
  g.N = a.N;
  g.G = a.G;
  g.causal = a.causal;
  g.q_len = a.q_len;
  g.member = member;
  for (int r = warp; r < 8 * NT; r += kWarps) {
    const AttnRow y = shared_row(g, x, r);
    const unsigned nan = static_cast<unsigned>(seen_nan<1>(a.c, x.b * a.c.table_stride + x.col, h, first, y.limit, d0 & ~3)) >> (d0 & 3);
    uint16_t* const o = a.o + y.b * a.so.b + (h * a.G + y.head) * a.so.h + y.i * a.so.n + d0;
#pragma unroll
    for (int d = 0; d < kPer; ++d) {
      if (!(nan >> d & 1u)) continue;
      if (o_part != nullptr)
        o_part[r * D + d0 + d] = __int_as_float(0x7fffffff);
      else
        o[d] = 0x7fffu;  // NaN in bf16 and in fp16
    }
  }
}

// The producer warp: every step of the CTA's run, a stage each. Lane i < 8 looks
// after the step's i-th group of 16 keys: its page id is loaded three steps ahead,
// the page's scales two steps ahead (one step is less than their way from memory),
// and the first lane of each page copies its rows (the pages' K and V lie in rows of d bytes of one tensor map each).
template <int D, int NT, bool SH>
__device__ __forceinline__ void produce(const CacheAttnLaunch& a, const AttnGridOf<SH>& g, AttnCursor<SH> ld, uint8_t* smem,
                                        uint64_t* full, uint64_t* empty, const Watchdog& wd, int lane) {
  using L = Layout<D, NT>;
  constexpr int kStages = L::kStages;
  const CacheView& c = a.c;
  const int per_page = min(c.page, kKeys) >> 4;  // groups of a page
  const bool group = lane < kKeys / 16, leader = group && lane % per_page == 0;
  // what is known of a coming step, per lane
  struct Step {
    bool live, want;  // within the run; the group holds keys that are seen
    int pid, h, row;  // row: of the page, where the step's rows start
    float ks, vs;
  };
  auto look = [&]() {  // the cursor's step, then on
    Step s{!ld.done(g), false, -1, 0, 0, -1.f, -1.f};
    if (s.live) {
      const int key = (ld.step << g.log2_keys) + lane * 16;
      s.want = group && key < ld.x.seen;
      s.h = ld.h;
      s.row = key & (c.page - 1);
      if (s.want) s.pid = attn_load<SH>(c.table + ld.x.b * c.table_stride + first_column(ld.x) + (key >> c.log2_page));
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
      s.ks = attn_load<SH>(c.scale[0] + ph);
      s.vs = attn_load<SH>(c.scale[1] + ph);
    }
  };
  Step now = look(), next = look();
  scales(now);
  scales(next);
  Step third = look();
  int n = 0;  // steps issued
  for (; now.live; ++n) {
    const int st = n % kStages;
    if (n >= kStages && !mbar_wait_warp(empty + st, ((n / kStages) - 1) & 1, wd)) break;
    // The copies go out before their bytes are announced (the phase cannot end
    // before lane 0 arrives) and before the scales, which may still be on their way.
    if (leader && now.want) {
      uint8_t* const dst = smem + st * L::kStage + lane * 16 * D;
      tma_load_2d(dst, &a.tm[0], full + st, now.row);
      tma_load_2d(dst + L::kMat, &a.tm[1], full + st, now.row);
    }
    const int copies = __popc(__ballot_sync(0xffffffffu, leader && now.want));
    if (group)
      *reinterpret_cast<float2*>(smem + L::kScales + st * 64 + lane * 8) = make_float2(now.ks, now.vs);
    __syncwarp();
    if (lane == 0) {
      if (copies > 0)
        mbar_expect_tx(full + st, copies * 2 * min(c.page, kKeys) * D);
      else
        mbar_arrive(full + st);
    }
    now = next;
    next = third;
    scales(next);  // before the next load of a page id: waiting for one waits for all of its kind
    third = look();
  }
  // let every copy in flight land before the CTA can exit
  for (int i = max(0, n - kStages); i < n; ++i)
    mbar_wait_drain(full + i % kStages, (i / kStages) & 1, a.wait_limit);
}

// NT groups of 8 query rows per unit. SH: the units are a list's, and their rows' parts are joined
// afterwards, but where a sequence shares nothing (SharedGrid::entry).
template <int D, int NT, bool INT8, bool SH>
__global__ void __launch_bounds__(kThreads, Layout<D, NT>::kCtas)
    cache_attn_kernel(const __grid_constant__ CacheAttnLaunch a, const AttnGridOf<SH> g) {
  using L = Layout<D, NT>;
  constexpr int kStages = L::kStages;
  constexpr int kM = D / 16;  // 16-channel tiles of O
  constexpr int kRows = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnShareOf<SH> share;
  __shared__ long long part[kThreads / 32];
  __shared__ float sm_m[2][kWarps][kRows], sm_l[2][kWarps][kRows];  // of a unit, in turn
  __shared__ int sm_nan[2][kWarps];  // likewise: the warps' nan_key
  __shared__ int abort_flag;
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t = lane & 3;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* const empty = full + kStages;
  check_init(a.status);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&a.tm[0]);
    tma_prefetch_desc(&a.tm[1]);
  }
  attn_wait<SH>(g, false);
  grid_dep_launch();
  const Watchdog wd{a.wait_limit, a.status, &abort_flag};
  AttnCursor<SH> cur = attn_share<kThreads, SH>(g, &share, part);  // its barriers publish the above
  if (warp == kWarps) {
    produce<D, NT, SH>(a, g, cur, smem, full, empty, wd, lane);
    attn_wait<SH>(g, true);
    return;
  }
  if (!SH && g.split && threadIdx.x == 0) g.record[blockIdx.x] = make_int4(-1, 0, 0, 0);
  bool alive = true;  // no wait has given up
  int stage = 0, turn = 0;
  uint32_t phase = 0;

  // The queries of the cursor's unit, this lane's part of group n of 8 rows
  auto query = [&](int n, uint4 (&w)[D / 32]) {
    const int r = n * 8 + gq;
    if constexpr (SH) {
      const AttnRow y = shared_row(g, cur.x, r);
      load_query<D, SH>(a.q + y.b * a.sq.b + static_cast<long long>(cur.h * g.G + y.head) * a.sq.h + y.i * a.sq.n, y.real, t, w);
    } else {
      const int row = cur.x.row0 + r, i = row / g.G;
      load_query<D, SH>(a.q + cur.x.b * a.sq.b + static_cast<long long>(cur.h * g.G + (row - i * g.G)) * a.sq.h + i * a.sq.n,
                        i < cur.x.ql, t, w);
    }
  };
  // A list's units are short (a sequence's own tokens): their queries are loaded a unit ahead (64 sequences of 50 to 2000
  // tokens 38.1 -> 36.4 us; 64 of 1000 to 8192, which is not a list, 100.2 -> 101.1: registers). Two groups of
  // rows leave no registers for it (200 bytes of spills at d = 128).
  constexpr bool kAhead = SH && NT == 1;
  uint4 ahead[kAhead ? D / 32 : 1];
  if constexpr (kAhead)
    if (!cur.done(g)) query(0, ahead);

  while (!cur.done(g)) {
    // ---- a unit (or the CTA's part of one)
    const typename AttnEntryOf<SH>::type x = cur.x;
    const int h = cur.h, step0 = cur.step, steps = cur.run(g), unit = cur.e * g.HK + h;
    const long long unit_first = cur.pos - cur.step;
    // Queries: lane (gq, t) holds what the products take of row gq, channels
    // [D/4 t, D/4 (t + 1)). Two groups of rows would take too many registers: each is
    // then loaded by one warp and shared, in the order of the products.
    uint32_t q[NT == 1 ? D / 8 : 1];
    uint2* const qs = reinterpret_cast<uint2*>(smem + L::kQuery);
    float* const rfs = reinterpret_cast<float*>(smem + L::kQuery + NT * (D / 16) * 256);
    float rf[NT][2];
    int lim[NT][2];
    if constexpr (NT == 1) {
      uint4 raw[D / 32];
      if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[i] = ahead[kAhead ? i : 0];
      } else {
        query(0, raw);
      }
      const float f = scale_query<D>(raw, a.fp16, q) * a.scale_log2;
      rf[0][0] = __shfl_sync(0xffffffffu, f, 2 * t * 4);
      rf[0][1] = __shfl_sync(0xffffffffu, f, (2 * t + 1) * 4);
    } else {
      if (warp < NT) {
        uint4 raw[D / 32];
        query(warp, raw);
        uint32_t w[D / 8];
        const float f = scale_query<D>(raw, a.fp16, w) * a.scale_log2;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) qs[(warp * (D / 16) + i) * 32 + lane] = make_uint2(w[2 * i], w[2 * i + 1]);
        if (t == 0) rfs[warp * 8 + gq] = f;
      }
      named_bar_sync(1, kWarps * 32);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        rf[n][0] = rfs[n * 8 + 2 * t];
        rf[n][1] = rfs[n * 8 + 2 * t + 1];
      }
    }
    int low = 0x7fffffff;  // keys below it are seen by every row
    bool real[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = n * 8 + 2 * t + k;
        // columns that stand for no query (their q is zero) do not make a tile an edge
        if constexpr (SH) {
          const AttnRow y = shared_row(g, x, r);
          lim[n][k] = y.limit;
          real[n][k] = y.real;
        } else {
          lim[n][k] = attn_limit(g, x, r);
          real[n][k] = (x.row0 + r) / g.G < x.ql;
        }
        if (real[n][k]) low = min(low, lim[n][k]);
      }
    low = __reduce_min_sync(0xffffffffu, low);

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

    int nan_key = 0x7fffffff;  // first key of V with a NaN that was taken out
    int key0 = (step0 << g.log2_keys) + warp * kTile;
    for (int step = 0; step < steps; ++step, key0 += kKeys) {
      alive = alive && mbar_wait_warp(full + stage, phase, wd);
      if (alive && key0 < x.seen) {
        const uint32_t kt = smem_u32(smem) + stage * L::kStage, vt = kt + L::kMat;
        const uint4 sc = lds128(smem_u32(smem) + L::kScales + stage * 64 + warp * 16);
        const float ks[2] = {__uint_as_float(sc.x), __uint_as_float(sc.z)};
        const bool zero[2] = {!(__uint_as_float(sc.y) > kMinScale), !(__uint_as_float(sc.w) > kMinScale)};
        const float vs[2] = {zero[0] ? kZeroScale : __uint_as_float(sc.y), zero[1] ? kZeroScale : __uint_as_float(sc.w)};
        // S^T = K Q^T: keys gq, gq + 8 of each group, queries 2t, 2t + 1
        float s[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[u][n][k] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t kw[2][2][4];  // group, half of its keys, word
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 v = lds128(kt + tile_offset<D>(warp * kTile + u * 16 + e * 8 + gq, (D / 64) * t + j));
              kw[u][e][0] = v.x;
              kw[u][e][1] = v.y;
              kw[u][e][2] = v.z;
              kw[u][e][3] = v.w;
            }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint2 qf[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
              qf[n] = NT == 1 ? make_uint2(q[NT == 1 ? (j * 4 + w) * 2 : 0], q[NT == 1 ? (j * 4 + w) * 2 + 1 : 0])
                              : qs[(n * (D / 16) + j * 4 + w) * 32 + lane];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t a0, a1, a2, a3;
              decode4<INT8>(kw[u][0][w], a0, a2);
              decode4<INT8>(kw[u][1][w], a1, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(s[u][n], a0, a1, a2, a3, qf[n].x, qf[n].y);
            }
          }
        }
        // y, the reference maximum, the weights
        const float lv[2] = {__log2f(vs[0]), __log2f(vs[1])};
        const float iv[2] = {__fdividef(1.f, vs[0]), __fdividef(1.f, vs[1])};
        const bool edge = key0 + kTile > low || ks[0] < 0.f || ks[1] < 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[u][n][k] = fmaf(s[u][n][k], rf[n][k & 1] * ks[u], lv[u]);
        if (edge) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (key0 + u * 16 + gq + 8 * (k >> 1) >= lim[n][k & 1] || ks[u] < 0.f) s[u][n][k] = -INFINITY;
        }
        float mx[NT][2];
        bool above = false;  // a weight would pass 2^15
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mx[n][k] = fmaxf(fmaxf(s[0][n][k], s[0][n][2 + k]), fmaxf(s[1][n][k], s[1][n][2 + k]));
            above |= mx[n][k] > m[n][k] + kSlack;
          }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float al[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              mx[n][k] = fmaxf(mx[n][k], __shfl_xor_sync(0xffffffffu, mx[n][k], 4));
              mx[n][k] = fmaxf(mx[n][k], __shfl_xor_sync(0xffffffffu, mx[n][k], 8));
              mx[n][k] = fmaxf(mx[n][k], __shfl_xor_sync(0xffffffffu, mx[n][k], 16));
              const float mn = fmaxf(m[n][k], mx[n][k]);
              al[k] = ex2(m[n][k] - (mn == -INFINITY ? 0.f : mn));
              m[n][k] = mn;
              l[n][k] *= al[k];
            }
#pragma unroll
            for (int i = 0; i < kM; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[i][n][k] *= al[k & 1];
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float base = (m[n][k] == -INFINITY ? 0.f : m[n][k]) - kBias;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float p0 = ex2(s[u][n][k] - base), p1 = ex2(s[u][n][2 + k] - base);
              s[u][n][k] = p0;
              s[u][n][2 + k] = p1;
              l[n][k] = fmaf(p0 + p1, iv[u], l[n][k]);
            }
          }
        // O^T += V^T P^T: channels (D/8) gq + 2i, + 1 on the rows of tile i
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t p0[NT], p1[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            p0[n] = transpose8x8(zero[u] ? 0u : pack_half(s[u][n][0], s[u][n][1]));
            p1[n] = transpose8x8(zero[u] ? 0u : pack_half(s[u][n][2], s[u][n][3]));
          }
          uint32_t v[4][D / 32];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = warp * kTile + u * 16 + 2 * t + (k & 1) + 8 * (k >> 1);
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
          if (!INT8 && (key0 + kTile > low || ks[u] < 0.f))
            nan_key = min(nan_key, take_out_nan(v, ks[u] < 0.f, key0 + u * 16 + 2 * t));
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
      __syncwarp();  // every lane has read the stage
      if (step + 1 == steps) break;  // the unit's last stage is kept: the warps join in it
      if (lane == 0) mbar_arrive(empty + stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    cur.skip(g, steps);
    if constexpr (kAhead)
      if (!cur.done(g)) query(0, ahead);  // the next unit's, on their way while this one ends

    // ---- join the warps' keys, through the last step's stage
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], w);
        if (!real[n][k]) {
          l[n][k] = 0.f;
          m[n][k] = -INFINITY;
        }
        if (gq == 0) {
          sm_m[turn][warp][n * 8 + 2 * t + k] = m[n][k];
          sm_l[turn][warp][n * 8 + 2 * t + k] = l[n][k];
        }
      }
    if (!INT8 && lane == 0) sm_nan[turn][warp] = nan_key;
    named_bar_sync(1, kWarps * 32);  // also: every warp has read its part of the stage
    const bool last = step0 + steps == x.steps, whole = step0 == 0 && last;
    const int slot = SH && whole ? 2 * gridDim.x + unit : 2 * blockIdx.x + (step0 == 0 ? 1 : 0);
    bool direct = whole;  // straight to O and LSE
    if constexpr (SH) {
      direct = whole && x.list < 0 && x.count == 1;
      if (last && threadIdx.x == 0)
        g.unit_parts[unit] = whole ? make_int2(-1, 0) : make_int2(attn_cta_of(unit_first, share), blockIdx.x);
    } else if (g.split && !whole && last && threadIdx.x == 0) {
      g.record[blockIdx.x] =
          make_int4(x.b * g.row_tiles + x.row0 / g.rows, h, attn_cta_of(unit_first, share), 0);
    }
    // O of warp w, row r: D words at (w kRows + r) D; pair i of group gq at 2 (8 i + gq), and half the
    // banks on for every other pair of rows, so that a warp's 64 words meet every bank twice
    float* const merge = reinterpret_cast<float*>(smem + stage * L::kStage);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = n * 8 + 2 * t + k;
        float M = sm_m[turn][0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm_m[turn][w][r]);
        const float f = ex2(m[n][k] - (M == -INFINITY ? 0.f : M));
        float* const at = merge + (warp * kRows + r) * D;
#pragma unroll
        for (int i = 0; i < kM; ++i)
          *reinterpret_cast<float2*>(at + ((16 * i + 2 * gq) ^ ((t & 1) << 4))) = make_float2(o[i][n][k] * f, o[i][n][2 + k] * f);
      }
    named_bar_sync(1, kWarps * 32);
    constexpr int kPer = D / 32;  // channels of a row per lane
    const int d0 = lane * kPer;
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {  // a warp joins every fourth row
      const int r = warp + kWarps * j;
      float M = sm_m[turn][0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm_m[turn][w][r]);
      float sum = 0.f, acc[kPer];
#pragma unroll
      for (int d = 0; d < kPer; ++d) acc[d] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sum = fmaf(sm_l[turn][w][r], ex2(sm_m[turn][w][r] - (M == -INFINITY ? 0.f : M)), sum);
#pragma unroll
        for (int d = 0; d < kPer; d += 2) {
          const int pair = (d0 + d) % (D / 8) / 2;
          const float2 v = *reinterpret_cast<const float2*>(merge + (w * kRows + r) * D +
                                                            ((16 * pair + 2 * (d0 / (D / 8))) ^ ((r >> 1 & 1) << 4)));
          acc[d] += v.x;
          acc[d + 1] += v.y;
        }
      }
      const int row = x.row0 + r, i = row / g.G;
      if (!direct) {
        const long long pr = static_cast<long long>(slot) * g.rows + r;
#pragma unroll
        for (int d = 0; d < kPer; d += 2)
          *reinterpret_cast<float2*>(g.o_part + pr * D + d0 + d) = make_float2(acc[d], acc[d + 1]);
        if (lane == 0) {
          g.m_part[pr] = M;
          g.l_part[pr] = sum;
        }
      } else if (i < g.N) {
        const bool none = sum == 0.f;  // a row that sees no key; NaN stays NaN
        const float inv = none ? 0.f : 1.f / sum;
        const int head = h * g.G + (row - i * g.G);
        uint16_t* const dst = a.o + x.b * a.so.b + head * a.so.h + i * a.so.n + d0;
#pragma unroll
        for (int d = 0; d < kPer; d += 2)
          *reinterpret_cast<uint32_t*>(dst + d) = none ? 0u : pack16(acc[d] * inv, acc[d + 1] * inv, a.fp16);
        if (lane == 0)
          a.lse[(static_cast<long long>(x.b) * a.Hq + head) * g.N + i] =
              none ? -INFINITY : (M - kBias + log2f(sum)) * kLn2Cache;
      }
    }
    if constexpr (!INT8) {
      int first = sm_nan[turn][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) first = min(first, sm_nan[turn][w]);
      if (first != 0x7fffffff) {
        float* const at = direct ? nullptr : g.o_part + static_cast<long long>(slot) * g.rows * D;
        if constexpr (SH)
          put_nan_shared<D, NT>(a, g.member, x, h, first, at, warp, lane);
        else
          put_nan<D, NT>(a, x.b, x.row0, x.kv, x.ql, h, first, at, warp, lane);
      }
    }
    // the stage goes back, and the statistics' other half is next: a warp that is a unit ahead
    // has passed that unit's barriers, and with it all that read these
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + stage);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
    turn ^= 1;
  }
}

template <int D, int NT, bool INT8, bool SH = false>
cudaError_t launch_rows(const CacheAttnLaunch& a, const AttnGridOf<SH>& g, int ctas, cudaStream_t stream) {
  auto kern = cache_attn_kernel<D, NT, INT8, SH>;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = set_smem_once(smem_set, reinterpret_cast<const void*>(kern), Layout<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), Layout<D, NT>::kSmem, stream, a, g);
}

}  // namespace
}  // namespace fa
