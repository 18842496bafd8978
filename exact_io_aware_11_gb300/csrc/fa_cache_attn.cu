// Attention over the paged 8-bit cache in units of 8 or 16 query rows per cache head
// (single tokens, drafted ones, up to 64 rows over short caches: attn_plan), and the merge of
// units that were cut.
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

// One row of queries in fp16, scaled by a power of two (its inverse comes
// back): lane t of the row's four holds channels [D/4 t, D/4 (t + 1)).
template <int D>
__device__ __forceinline__ float load_query(const uint16_t* row, bool real, bool fp16, int t, uint32_t (&q)[D / 8]) {
  float x[D / 4];
  float mx = 0.f;
#pragma unroll
  for (int v = 0; v < D / 32; ++v) {
    const uint4 w = real ? reinterpret_cast<const uint4*>(row + t * (D / 4))[v] : make_uint4(0, 0, 0, 0);
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
    const unsigned nan = static_cast<unsigned>(seen_nan<1>(a.c, b, h, first, end, d0 & ~3)) >> (d0 & 3);
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

// The producer warp: every step of the CTA's run, a stage each. Lane i < 8 looks
// after the step's i-th group of 16 keys: its page id is loaded three steps ahead,
// the page's scales two steps ahead (one step is less than their way from memory),
// and the first lane of each page copies its rows (the pages' K and V lie in rows of d bytes of one tensor map each).
template <int D, int NT>
__device__ __forceinline__ void produce(const CacheAttnLaunch& a, const AttnGrid& g, AttnCursor ld, uint8_t* smem,
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

// NT groups of 8 query rows per unit.
template <int D, int NT, bool INT8>
__global__ void __launch_bounds__(kThreads, Layout<D, NT>::kCtas)
    cache_attn_kernel(const __grid_constant__ CacheAttnLaunch a, const AttnGrid g) {
  using L = Layout<D, NT>;
  constexpr int kStages = L::kStages;
  constexpr int kM = D / 16;  // 16-channel tiles of O
  constexpr int kRows = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnShare share;
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
  grid_dep_wait();
  grid_dep_launch();
  const Watchdog wd{a.wait_limit, a.status, &abort_flag};
  AttnCursor cur = attn_share<kThreads>(g, &share, part);  // its barriers publish the above
  if (warp == kWarps) {
    produce<D, NT>(a, g, cur, smem, full, empty, wd, lane);
    return;
  }
  if (g.split && threadIdx.x == 0) g.record[blockIdx.x] = make_int4(-1, 0, 0, 0);
  bool alive = true;  // no wait has given up
  int stage = 0, turn = 0;
  uint32_t phase = 0;

  while (!cur.done(g)) {
    // ---- a unit (or the CTA's part of one)
    const AttnEntry x = cur.x;
    const int h = cur.h, step0 = cur.step, steps = cur.run(g);
    const long long unit_first = cur.pos - cur.step;
    // Queries: lane (gq, t) holds what the products take of row gq, channels
    // [D/4 t, D/4 (t + 1)). Two groups of rows would take too many registers: each is
    // then loaded by one warp and shared, in the order of the products.
    uint32_t q[NT == 1 ? D / 8 : 1];
    uint2* const qs = reinterpret_cast<uint2*>(smem + L::kQuery);
    float* const rfs = reinterpret_cast<float*>(smem + L::kQuery + NT * (D / 16) * 256);
    float rf[NT][2];
    int lim[NT][2];
    auto query = [&](int n, uint32_t (&w)[D / 8]) {
      const int r = x.row0 + n * 8 + gq, i = r / g.G;
      const uint16_t* row = a.q + x.b * a.sq.b + static_cast<long long>(h * g.G + (r - i * g.G)) * a.sq.h + i * a.sq.n;
      return load_query<D>(row, i < x.ql, a.fp16, t, w) * a.scale_log2;
    };
    if constexpr (NT == 1) {
      const float f = query(0, q);
      rf[0][0] = __shfl_sync(0xffffffffu, f, 2 * t * 4);
      rf[0][1] = __shfl_sync(0xffffffffu, f, (2 * t + 1) * 4);
    } else {
      if (warp < NT) {
        uint32_t w[D / 8];
        const float f = query(warp, w);
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
        lim[n][k] = attn_limit(g, x, r);
        // columns that stand for no query (their q is zero) do not make a tile an edge
        real[n][k] = (x.row0 + r) / g.G < x.ql;
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
    const int slot = 2 * blockIdx.x + (step0 == 0 ? 1 : 0);
    if (g.split && !whole && last && threadIdx.x == 0)
      g.record[blockIdx.x] =
          make_int4(x.b * g.row_tiles + x.row0 / g.rows, h, attn_cta_of(unit_first, share), 0);
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
      if (!whole) {
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
      if (first != 0x7fffffff)
        put_nan<D, NT>(a, x.b, x.row0, x.kv, x.ql, h, first, whole ? nullptr : g.o_part + static_cast<long long>(slot) * g.rows * D, warp, lane);
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

// Merges the units that were cut. Blocks (c, y) look at CTA c's record (the unit
// whose last part c ran) and share its rows out: with m_q, l_q, O_q of part q and
// M = max_q m_q, O = sum 2^(m_q - M) O_q / sum 2^(m_q - M) l_q. A lane holds D / 32
// consecutive channels and loads five parts at a time, statistics and all. A unit
// of few parts gives each of the block's 8 warps a row; one of more parts gives a row
// four or all of them, which take every fourth or eighth part and then join theirs (a
// row of 76 parts with one warp, four at a time: 36 us by itself, with four warps 8 us).
template <int D>
__global__ void __launch_bounds__(256) cache_attn_merge_kernel(const __grid_constant__ CacheAttnLaunch a, const AttnGrid g) {
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

template <int D, int NT, bool INT8>
cudaError_t launch_rows(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  auto kern = cache_attn_kernel<D, NT, INT8>;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = set_smem_once(smem_set, reinterpret_cast<const void*>(kern), Layout<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), Layout<D, NT>::kSmem, stream, a, g);
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
