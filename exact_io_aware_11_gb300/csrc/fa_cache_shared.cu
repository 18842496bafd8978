// Attention over the paged 8-bit cache for a batch whose sequences share prefixes
// (fa_cache_attention_shared). It is the attention of fa_cache_attention, row by row; only who reads
// the keys changes.
//
// Mathematics: the softmax of a row over [prefix | own tokens] is joined from parts over any runs of its
// keys: with m_q, l_q, O_q of part q and M = max m_q, O = sum 2^(m_q - M) O_q / sum 2^(m_q - M) l_q.
// So the rows of all of a group's sequences stand together in tiles over the prefix, whose keys
// are then read once for all of them, and each sequence's rows go over its own tokens.
//
// Four launches: the plan (one CTA: who belongs to which group, the lists of entries), the tile
// kernel (fa_cache_tile.cuh) over list A, prefixes of groups with more than 16 rows to a cache
// head; the kernel for the sequences' own tokens over list B, with few rows (fa_cache_rows.cuh) also
// the prefixes of small groups; and the join. Parts are in 32 bits.
//
// The two lists run beside each other, because one is bound by products and latencies and the other by
// memory: the plan gives each as many SMs as its share of the estimated cost, the
// other CTAs of list A's kernel leave at once, and list B's kernel, let go by them, begins there without
// waiting (its own wait, for list A's kernel, comes at its end, so that the join's covers both).
// It may: list A's CTAs let it go after their wait for the plan, whose writes, and all
// before them, it has by the plan's mark (attn_wait). It cannot keep a CTA of list A from running,
// as they have all begun.
//
// What bounds it, and what it measured (GPU time; fa_cache_attention on the same sequences in brackets): 64 sequences behind
// 8192 tokens with 50 to 2000 of their own, 32 heads on 8, d = 128, e4m3: 50 us (118), of which plan, first scores, last
// results, join and launches are some 27; 256 behind 32768 with 256 to 2048: 207 to 213 us (1548), bound by the SMs: 1.72 us
// a step of 256 rows and 128 keys (1480 TFLOP/s on all SMs), 0.42 us of an SM a step of own tokens (32 KB: 78 GB/s). Short
// prefixes are sooner served without sharing: 64 sequences with 500 to 2000 tokens behind 128 52 us (37).
#include <chrono>

#include "fa_cache_rows.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024, kMaxGroups = kSharedGroups;

struct PlanLaunch {
  int B, groups, N, G, page, cap, causal;
  int rows_a, rows_b, tiles_b, few;  // few: list B's kernel takes few rows
  int HK, sms, ctas_a, per_sm_b;        // CTAs of list A's kernel, of list B's that an SM holds
  int step_a, start_a, step_b, start_b;  // what an SM takes for a step and for beginning a unit, in ns
  const int32_t* of;
  const int32_t* len;
  const int32_t* kv_len;
  const int32_t* q_len;
  // workspace
  int* entries;      // of list A, its CTAs; of list B, its CTAs
  SharedEntry* entry_a;
  SharedEntry* entry_b;
  int* member;       // [B]
  int4* seq;         // [B] where the sequence's part over the prefix is: list (0 none, 1 A, 2 B), its
                     // first row in the group, the group's first entry
  PlanMark mark;
};

__device__ __forceinline__ SharedEntry make_entry(int b, int row0, int kv, int ql, int seen, int list, int count, int col) {
  SharedEntry x;
  x.b = b;
  x.row0 = row0;
  x.kv = kv;
  x.ql = ql;
  x.seen = seen;
  x.steps = max(1, (seen + 127) >> 7);
  x.list = list;
  x.count = count;
  x.col = col;
  x.pad[0] = x.pad[1] = x.pad[2] = 0;
  return x;
}

struct Sequence {
  int kv, ql, group, prefix;  // group -1: on its own
};
// A sequence counts as one of its group where every one of its rows sees the whole prefix.
__device__ __forceinline__ Sequence sequence(const PlanLaunch& a, const int* tokens, int group, int kv_len, int q_len) {
  Sequence s;
  s.kv = min(a.cap, max(0, kv_len));
  s.ql = min(a.N, max(0, q_len));
  s.group = group;
  s.prefix = 0;
  if (s.group >= 0 && s.group < a.groups && s.ql > 0) s.prefix = tokens[s.group];
  if (s.prefix == 0 || (a.causal ? s.kv - s.ql + 1 : s.kv) < s.prefix) {
    s.group = -1;
    s.prefix = 0;
  }
  return s;
}
__device__ __forceinline__ Sequence sequence(const PlanLaunch& a, const int* tokens, int b) {
  return sequence(a, tokens, a.of[b], a.kv_len[b], a.q_len != nullptr ? a.q_len[b] : a.N);
}

// A block of as many threads as there are sequences or groups, 1024 at most; what is said of a
// sequence stays in its thread's registers where each has one.
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const __grid_constant__ PlanLaunch a) {
  __shared__ int count[kMaxGroups], start[kMaxGroups], base[kMaxGroups], first[kMaxGroups];
  __shared__ int tokens[kMaxGroups];  // of the prefixes, in whole pages
  __shared__ int rank[kPlanThreads];
  __shared__ int sums[3][kPlanThreads / 32];
  __shared__ unsigned long long cost[2];  // of the lists, in ns of an SM
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, NG = a.N * a.G;
  const bool one = a.B <= threads;
  __shared__ int shortest, longest;       // list A's prefixes, in steps
  if (tid < 2) cost[tid] = 0ull;
  if (tid == 0) {
    shortest = 0x7fffffff;
    longest = 0;
  }
  unsigned long long cost_a = 0ull, cost_b = 0ull;
  grid_dep_wait();
  grid_dep_launch();
  // (a sequence's group and lengths are on their way at the same time)
  Sequence own{};
  int group = tid < a.B ? a.of[tid] : -1, kv_len = tid < a.B ? a.kv_len[tid] : 0, q_len = a.q_len != nullptr && tid < a.B ? a.q_len[tid] : a.N;
  for (int g = tid; g < a.groups; g += threads) {
    count[g] = 0;
    tokens[g] = min(max(0, a.len[g]), a.cap) / a.page * a.page;
  }
  __syncthreads();
  // ---- each sequence's place in its group, in the order of the batch
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + tid;
    own.group = -1;
    if (b < a.B) own = b0 == 0 ? sequence(a, tokens, group, kv_len, q_len) : sequence(a, tokens, b);
    rank[tid] = own.group;
    __syncthreads();
    if (warp == 0)
      for (int c = 0; c < threads && b0 + c < a.B; c += 32) {
        const int g = rank[c + lane];
        const unsigned same = __match_any_sync(0xffffffffu, g);
        const int before = g >= 0 ? count[g] : 0, r = before + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (g >= 0) {
          if (lane == __ffs(same) - 1) count[g] = before + __popc(same);
          if (r == 0) first[g] = b0 + c + lane;
          rank[c + lane] = r;
        }
        __syncwarp();
      }
    __syncthreads();
    if (!one) {
      if (b < a.B) a.seq[b] = make_int4(0, rank[tid], 0, 0);
      __syncthreads();
    }
  }
  // ---- groups: their sequences' places in the list, their entries
  int at_member = 0, at_a = 0, at_b = a.B * a.tiles_b;  // list B begins with the sequences' own tokens
  for (int g0 = 0; g0 < a.groups; g0 += threads) {
    const int g = g0 + tid;
    int n = g < a.groups ? count[g] : 0;
    if (n < 2) n = 0;  // alone, it shares nothing
    const long long rows = static_cast<long long>(n) * NG;
    const bool small = a.few && rows <= 16;
    const int per = small ? a.rows_b : a.rows_a, tiles = static_cast<int>((rows + per - 1) / per);
    const int v[3] = {n, small ? 0 : tiles, small ? tiles : 0};
    int incl[3], total[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      incl[k] = v[k];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl[k], o);
        if (lane >= o) incl[k] += u;
      }
      if (lane == 31) sums[k][warp] = incl[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      int before = 0, sum = 0;
      for (int w = 0; w < threads >> 5; ++w) {
        if (w < warp) before += sums[k][w];
        sum += sums[k][w];
      }
      incl[k] += before - v[k];  // exclusive
      total[k] = sum;
    }
    if (g < a.groups) {
      count[g] = n;
      start[g] = at_member + incl[0];
      base[g] = small ? at_b + incl[2] : at_a + incl[1];
      if (n > 0) {
        const int seen = tokens[g];
        SharedEntry* const to = small ? a.entry_b : a.entry_a;
        const unsigned long long steps = static_cast<unsigned long long>(tiles) * ((seen + 127) >> 7);
        if (small) {
          cost_b += steps * a.step_b + static_cast<unsigned long long>(tiles) * a.start_b;
        } else {
          cost_a += steps * a.step_a + static_cast<unsigned long long>(tiles) * a.start_a;
          atomicMin(&shortest, (seen + 127) >> 7);
          atomicMax(&longest, (seen + 127) >> 7);
        }
        for (int t = 0; t < tiles; ++t) to[base[g] + t] = make_entry(first[g], t * per, seen, 0, seen, start[g], n, 0);
      }
    }
    at_member += total[0];
    at_a += total[1];
    at_b += total[2];
    __syncthreads();
  }
  // ---- sequences: their own tokens
  for (int b = tid; b < a.B; b += threads) {
    const Sequence s = one ? own : sequence(a, tokens, b);
    int4 to = make_int4(0, 0, 0, 0);
    int prefix = 0;
    if (s.group >= 0 && count[s.group] > 0) {
      const int r = one ? rank[tid] : a.seq[b].y;
      prefix = s.prefix;
      a.member[start[s.group] + r] = b;
      to = make_int4(a.few && static_cast<long long>(count[s.group]) * NG <= 16 ? 2 : 1, r * NG, base[s.group], 0);
    }
    a.seq[b] = to;
    const int kv = s.kv - prefix;
    for (int t = 0; t < a.tiles_b; ++t) {
      const int row0 = t * a.rows_b, rows = min(a.rows_b, s.ql * a.G - row0);
      const int seen = rows <= 0 ? 0 : a.causal ? max(0, kv - s.ql + (row0 + rows - 1) / a.G + 1) : kv;
      a.entry_b[b * a.tiles_b + t] = make_entry(b, row0, kv, s.ql, seen, -1, to.x == 0 ? 1 : 0, prefix / a.page);
      cost_b += static_cast<unsigned long long>(max(1, (seen + 127) >> 7)) * a.step_b + a.start_b;
    }
  }
  // ---- how many SMs each list has
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    cost_a += __shfl_xor_sync(0xffffffffu, cost_a, o);
    cost_b += __shfl_xor_sync(0xffffffffu, cost_b, o);
  }
  if (lane == 0) {
    atomicAdd(&cost[0], cost_a);
    atomicAdd(&cost[1], cost_b);
  }
  __syncthreads();
  if (tid == 0) {
    // list A's CTAs take some 3 us more for their beginning and end; both end together where cost_a / n + 3 us
    // = cost_b / (sms - n)
    const float fa = static_cast<float>(cost[0]) * a.HK, fb = static_cast<float>(cost[1]) * a.HK;
    float x = a.sms * fa / (fa + fb);
#pragma unroll 1
    for (int k = 0; k < 4; ++k) x = fa / fmaxf((fa + fb + 3000.f * x) / a.sms - 3000.f, fa / a.sms);
    int n = at_a == 0 ? 0 : max(1, min(min(a.ctas_a, a.sms - 1), static_cast<int>(x + 0.5f)));
    // a whole number of CTAs to a unit, if these are equal: one that ends a unit and begins another takes some 6 us longer, so where the
    // other share costs less than that (batch of 64 behind 8192 tokens 53.7 -> 50.2 us)
    const int units = at_a * a.HK, whole = units > 0 ? (n + units / 2) / units * units : 0;
    if (shortest == longest && whole > 0 && whole <= min(a.ctas_a, a.sms - 1) && abs(whole - n) * (fa / n) <= 6000.f * min(n, a.sms - n)) n = whole;
    a.entries[0] = at_a;
    a.entries[1] = n;
    a.entries[2] = at_b;
    a.entries[3] = (a.sms - n) * a.per_sm_b;
    // after a barrier of the CTA, so for all of its writes
    asm volatile("st.release.gpu.u64 [%0], %1;" ::"l"(__cvta_generic_to_global(a.mark.word)), "l"(a.mark.call) : "memory");
  }
}

// Rows from which on a warp of the join takes four: 256 sequences of 32 heads behind four prefixes 84.7 us, with one row a
// warp 87.7; 64 sequences (2048 rows) 50.9 and 50.5.
constexpr long long kJoinMany = 4096;

// One list's parts, as the kernels leave them.
struct JoinList {
  const int2* unit_parts;
  const float* m;
  const float* l;
  const float* o;
  int rows, ctas;
};
struct JoinLaunch {
  JoinList list[2];  // A, B
  const int4* seq;
  int rows_b, tiles_b, HK;
  PlanMark mark;
};

// The parts of every row of O whose units have not written it: R rows a warp, 32 / R lanes a row. A row's lanes look up
// a part and its weight each, then sum D R / 32 channels each, up to eight parts in flight. Bound: latency and the L2
// cache (a part is 4 D + 8 bytes a row). One row a warp for few rows, four for many (kJoinMany); the former would spill
// with the registers of three blocks an SM.
template <int D, int R>
__global__ void __launch_bounds__(256, R == 1 ? 2 : 3) shared_join_kernel(const __grid_constant__ CacheAttnLaunch a, const __grid_constant__ JoinLaunch j) {
  constexpr int kLanes = 32 / R, kQuads = D / 4 < kLanes ? 1 : D / 4 / kLanes;  // of a row; 4 channels each, of a lane
  constexpr int kBatch = 8 / kQuads;
  plan_wait(j.mark);  // rows are looked up while the lists' kernels end
  const int lane = threadIdx.x & (kLanes - 1);
  const bool active = lane < D / 4;
  const long long row = blockIdx.x * (8LL * R) + threadIdx.x / kLanes;
  const int bh = static_cast<int>(row / a.N), i = static_cast<int>(row - static_cast<long long>(bh) * a.N);
  const int b = bh / a.Hq, head = bh - b * a.Hq, hk = head / a.G, r = i * a.G + head - hk * a.G;
  const int tile = r / j.rows_b, own = (b * j.tiles_b + tile) * j.HK + hk;
  const bool row_ok = row < static_cast<long long>(a.B) * a.Hq * a.N;
  const int4 s = row_ok ? __ldcg(j.seq + b) : make_int4(0, 0, 0, 0);
  const JoinList& pl = j.list[s.x == 2 ? 1 : 0];  // where the prefix's parts are
  int unit = 0, at = 0;
  if (s.x != 0) {
    const int x = s.y + r, t = x / pl.rows;
    unit = (s.z + t) * j.HK + hk;
    at = x - t * pl.rows;
  }
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *j.mark.word = 0ull;  // a graph may run this call again
  if (R == 1 && !row_ok) return;
  const int2 none2 = make_int2(0, -1);
  const int2 parts = row_ok ? j.list[1].unit_parts[own] : none2, p = s.x != 0 ? pl.unit_parts[unit] : none2;
  const bool write = row_ok && !(s.x == 0 && parts.x < 0);  // otherwise straight from its unit
  if (R == 1 && !write) return;
  // the prefix's parts, then the row's own; each list's first CTA, and how many
  const bool whole = p.x < 0;
  const int first = whole ? 0 : p.x, n = whole ? 1 : p.y - p.x + 1;
  const int all = !write ? 0 : n + (parts.x < 0 ? 1 : parts.y - parts.x + 1);
  int most = all;  // of the warp's rows
  if constexpr (R > 1) {
    most = __reduce_max_sync(0xffffffffu, all);
    if (most == 0) return;
  }
  float4 acc[kQuads];
#pragma unroll
  for (int c = 0; c < kQuads; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f, M = -INFINITY;
  for (int q0 = 0; q0 < most; q0 += kLanes) {
    // this lane's part
    const int q = q0 + lane;
    const float* o = nullptr;
    float m = -INFINITY, l = 0.f;
    if (q < all) {
      const JoinList& x = q < n ? pl : j.list[1];
      long long pr;
      if (q < n)
        pr = static_cast<long long>(whole ? 2 * x.ctas + unit : 2 * (first + q) + (q == 0 ? 1 : 0)) * x.rows + at;
      else
        pr = static_cast<long long>(parts.x < 0 ? 2 * x.ctas + own : 2 * (parts.x + q - n) + (q == n ? 1 : 0)) * x.rows + (r - tile * j.rows_b);
      m = x.m[pr];
      l = x.l[pr];
      o = x.o + pr * D;
    }
    const int count = min(kLanes, most - q0);
    // the first parts' values are on their way while their weights are formed
    float4 v[kBatch][kQuads];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float4* const from = reinterpret_cast<const float4*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), (k0 + k) & (kLanes - 1), kLanes));
#pragma unroll
        for (int c = 0; c < kQuads; ++c)
          v[k][c] = k0 + k < count && active && (R == 1 || from != nullptr) ? from[c * kLanes + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    load(0);
    float Mn = fmaxf(M, m);
#pragma unroll
    for (int w = kLanes / 2; w > 0; w >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, w));
    const float zero = Mn == -INFINITY ? 0.f : Mn, e = ex2(M - zero), f = ex2(m - zero);
    M = Mn;
    float part = l * f;
#pragma unroll
    for (int w = kLanes / 2; w > 0; w >>= 1) part += __shfl_xor_sync(0xffffffffu, part, w);
    sum = sum * e + part;
#pragma unroll
    for (int c = 0; c < kQuads; ++c) {
      acc[c].x *= e;
      acc[c].y *= e;
      acc[c].z *= e;
      acc[c].w *= e;
    }
    for (int k0 = 0; k0 < count; k0 += kBatch) {
      if (k0 > 0) load(k0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, (k0 + k) & (kLanes - 1), kLanes);
#pragma unroll
        for (int c = 0; c < kQuads; ++c) {
          acc[c].x = fmaf(v[k][c].x, w, acc[c].x);
          acc[c].y = fmaf(v[k][c].y, w, acc[c].y);
          acc[c].z = fmaf(v[k][c].z, w, acc[c].z);
          acc[c].w = fmaf(v[k][c].w, w, acc[c].w);
        }
      }
    }
  }
  if (!write) return;
  const bool none = sum == 0.f;  // a row that sees no key; NaN stays NaN
  const float inv = none ? 0.f : 1.f / sum;
  if (active) {
#pragma unroll
    for (int c = 0; c < kQuads; ++c) {
      uint2 w = make_uint2(0u, 0u);
      if (!none) w = make_uint2(pack16(acc[c].x * inv, acc[c].y * inv, a.fp16), pack16(acc[c].z * inv, acc[c].w * inv, a.fp16));
      *reinterpret_cast<uint2*>(a.o + b * a.so.b + head * a.so.h + i * a.so.n + (c * kLanes + lane) * 4) = w;
    }
  }
  if (lane == 0) a.lse[row] = none ? -INFINITY : (M - kBias + log2f(sum)) * kLn2Cache;
}

// What a step and the beginning of a unit take of an SM, in ns, both lists at work (least squares over the CTAs of 64
// to 256 sequences with 50 to 2000 tokens of their own behind prefixes of 8192 to 32768; two or three CTAs of
// few rows share an SM).
struct ListCost {
  int step, start;
};
ListCost tile_cost(int d, int rows) {
  if (rows == 256) return ListCost{d == 128 ? 1800 : 1500, 9000};
  return ListCost{rows == 128 ? (d == 128 ? 1570 : 1250) : d == 128 ? 1080 : 930, 4000};
}
ListCost few_cost(int d, int rows) {
  if (d == 128) return rows <= 8 ? ListCost{430, 1100} : ListCost{530, 2000};
  return rows <= 8 ? ListCost{300, 400} : ListCost{410, 1100};
}

// Rows of a unit and CTAs of both lists, and the workspace.
struct SharedPlan {
  bool plain;   // as fa_cache_attention
  bool only_b;  // list A is empty: no group has more than 16 rows
  int rows_a, rows_b, tiles_b, ctas_a, ctas_b, lead_a, lead_b;
  long long max_a, max_b;  // entries
  size_t entry_a, entry_b, member, seq, unit_a, unit_b, m_a, l_a, o_a, m_b, l_b, o_b, total;
};
SharedPlan shared_plan(int B, int HK, int G, int N, int d, int page, int table_width, int groups) {
  SharedPlan p{};
  const long long NG = static_cast<long long>(N) * G, cap = static_cast<long long>(table_width) * page;
  const AttnPlan own = attn_plan(B, HK, NG, cap, d);
  const long long sms = sm_count(), slots = own.rows <= 16 ? few_row_ctas(d, own.rows) * sms : sms;
  // Sharing takes some 20 us whatever there is to do (the plan, a tile kernel's beginning and end, the join): not
  // where the table has room for few steps a CTA without it. GPU time in us, shared and plain, one group
  // with 128 tokens of its own a sequence: 8 rows at d = 128, 15 steps 24.7, 22.6, 28 steps 28.1, 33.0; at d = 64 7 steps 21.1,
  // 16.5, 14 steps 24.4, 25.5; 16 rows, 8 steps 28.4, 24.0, 14 steps 29.6, 30.8; 40 rows, 14 steps 35.8, 27.8, 27 steps 44.1, 42.3; 80 rows,
  // 28 steps 43.0, 32.3, 55 steps 51.1, 49.6.
  const long long enough = NG <= 8 ? (d == 64 ? 11 : 18) : NG <= 16 ? 13 : NG <= 64 ? 29 : 58;
  p.plain = NG > 128 || B < 2 || own.units * own.cap_steps <= enough * slots;
  // units are numbered in 32 bits
  p.plain = p.plain || (static_cast<long long>(B) * (NG / 8 + 2) + groups) * HK > (1LL << 30);
  if (p.plain) {
    p.total = cache_attention_workspace(B, HK, G, N, d, page, table_width);
    return p;
  }
  // Own tokens are short: up to 32 rows go as groups of 16, which begin in a quarter of a tile's time
  // (20 rows of 64 sequences with 50 to 1000 tokens, 109.1 us in tiles, 93.9; 32 rows 149.2, 123.7; 32 rows of 32 sequences with 3000 to 6000 139.9, 134.3).
  const bool few = NG <= 32;
  p.rows_b = NG <= 8 ? 8 : few ? 16 : NG <= 64 ? 64 : 128;
  p.lead_b = !few ? (p.rows_b == 64 ? 6 : 4) : d == 64 && p.rows_b <= 8 ? 2 : 3;
  // One gap for tiles of every size, although pairs of them take some 5 steps to begin: with 3, 6 and 8 of them 128 sequences behind two
  // prefixes of 2000 and 16000 tokens 65.4, 65.5, 68.2 us (GPU time), 192 behind three of 1000 to 9000 (int8) 66.6, 68.7, 69.9, 512 behind
  // eight of 1000 to 6000 128.6, 131.7, 134.2; 64 behind one of 8192 49.4, 50.2, 50.1, 256 behind 32768 209.0, 208.7, 208.7.
  p.lead_a = 3;
  p.only_b = few && B * NG <= 16;
  p.tiles_b = static_cast<int>((NG + p.rows_b - 1) / p.rows_b);
  // (with the other SMs at work on list B, few steps a CTA are no reason for smaller tiles)
  const long long rows_of_group = (B + groups - 1) / groups * NG;
  p.rows_a = rows_of_group <= 64 ? 64 : rows_of_group <= 128 ? 128 : 256;
  const long long pairs = groups < B / 2 ? groups : B / 2;  // groups of two and more
  p.max_a = B * NG / p.rows_a + pairs;
  p.max_b = static_cast<long long>(B) * p.tiles_b + (few ? B * NG / p.rows_b + pairs : 0);
  const long long steps = (cap + 127) / 128, most_b = few ? few_row_ctas(d, p.rows_b) * sms : sms;
  p.ctas_a = static_cast<int>(p.max_a * HK >= sms || p.max_a * HK * steps >= sms ? sms : p.max_a * HK * steps);
  p.ctas_b = static_cast<int>(p.max_b * HK >= most_b || p.max_b * HK * steps >= most_b ? most_b : p.max_b * HK * steps);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  p.entry_a = take(p.max_a * sizeof(SharedEntry));
  p.entry_b = take(p.max_b * sizeof(SharedEntry));
  p.member = take(static_cast<size_t>(B) * 4);
  p.seq = take(static_cast<size_t>(B) * 16);
  p.unit_a = take(p.max_a * HK * 8);
  p.unit_b = take(p.max_b * HK * 8);
  const size_t parts_a = (2LL * p.ctas_a + p.max_a * HK) * p.rows_a, parts_b = (2LL * p.ctas_b + p.max_b * HK) * p.rows_b;
  p.m_a = take(parts_a * 4);
  p.l_a = take(parts_a * 4);
  p.o_a = take(parts_a * d * 4);
  p.m_b = take(parts_b * 4);
  p.l_b = take(parts_b * 4);
  p.o_b = take(parts_b * d * 4);
  p.total = at;
  return p;
}

template <int D, bool INT8>
cudaError_t launch_shared(const CacheAttnLaunch& a, const SharedGrid& ga, const SharedGrid& gb, const SharedPlan& p, const JoinLaunch& j,
                          cudaStream_t stream) {
  auto tiles = [&](const SharedGrid& g, int ctas) {
    return INT8 ? launch_shared_tiles_int8(a, g, ctas, stream) : launch_shared_tiles_e4m3(a, g, ctas, stream);
  };
  cudaError_t e = p.only_b ? cudaSuccess : tiles(ga, p.ctas_a);
  if (e != cudaSuccess) return e;
  e = p.rows_b > 16  ? tiles(gb, p.ctas_b)
      : p.rows_b > 8 ? launch_rows<D, 2, INT8, true>(a, gb, p.ctas_b, stream)
                     : launch_rows<D, 1, INT8, true>(a, gb, p.ctas_b, stream);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(a.B) * a.Hq * a.N;
  if (rows < kJoinMany) return launch_pdl(shared_join_kernel<D, 1>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, stream, a, j);
  return launch_pdl(shared_join_kernel<D, 4>, dim3(static_cast<unsigned>((rows + 31) / 32)), dim3(256), 0, stream, a, j);
}

}  // namespace

size_t shared_attention_workspace(int B, int HK, int G, int N, int d, int page, int table_width, int groups) {
  return shared_plan(B, HK, G, N, d, page, table_width, groups).total;
}

cudaError_t launch_shared_attention(const CacheAttnLaunch& a, const int32_t* prefix_of, const int32_t* prefix_len, int groups,
                                    cudaStream_t stream) {
  const SharedPlan p = shared_plan(a.B, a.c.H, a.G, a.N, a.c.d, a.c.page, a.c.table_width, groups);
  if (p.plain) return launch_cache_attention(a, stream);
  const int cap = a.c.table_width * a.c.page;
  PlanLaunch pl{};
  pl.B = a.B;
  pl.groups = groups;
  pl.N = a.N;
  pl.G = a.G;
  pl.page = a.c.page;
  pl.cap = cap;
  pl.causal = a.causal;
  pl.rows_a = p.rows_a;
  pl.rows_b = p.rows_b;
  pl.tiles_b = p.tiles_b;
  pl.few = p.rows_b <= 16;
  pl.HK = a.c.H;
  pl.sms = sm_count();
  pl.ctas_a = p.ctas_a;
  pl.per_sm_b = pl.few ? few_row_ctas(a.c.d, p.rows_b) : 1;
  ListCost ca = tile_cost(a.c.d, p.rows_a), cb = pl.few ? few_cost(a.c.d, p.rows_b) : tile_cost(a.c.d, p.rows_b);
  if (!pl.few) cb.start = 7500;  // units of few steps, one after another (64 sequences, 64 rows to a head, 16 to 64 own tokens: 216 us with 4000, 166)
  pl.step_a = ca.step;
  pl.start_a = ca.start;
  pl.step_b = cb.step;
  pl.start_b = cb.start;
  pl.of = prefix_of;
  pl.len = prefix_len;
  pl.kv_len = a.kv_len;
  pl.q_len = a.q_len;
  pl.entries = reinterpret_cast<int*>(a.ws);
  pl.entry_a = reinterpret_cast<SharedEntry*>(a.ws + p.entry_a);
  pl.entry_b = reinterpret_cast<SharedEntry*>(a.ws + p.entry_b);
  pl.member = reinterpret_cast<int*>(a.ws + p.member);
  pl.seq = reinterpret_cast<int4*>(a.ws + p.seq);
  static std::atomic<unsigned long long> calls{static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count()) << 16 | 1};
  pl.mark = PlanMark{reinterpret_cast<unsigned long long*>(a.ws + 128), calls.fetch_add(2, std::memory_order_relaxed)};  // never 0
  const int most = a.B > groups ? a.B : groups, threads = most >= kPlanThreads ? kPlanThreads : (most + 31) / 32 * 32;
  cudaError_t e = launch_pdl(shared_plan_kernel, dim3(1), dim3(threads), 0, stream, pl);
  if (e != cudaSuccess) return e;
  SharedGrid g{};
  g.B = a.B;
  g.HK = a.c.H;
  g.N = a.N;
  g.G = a.G;
  g.log2_keys = 7;
  g.cap = cap;
  g.causal = a.causal;
  g.split = 1;
  g.kv_len = a.kv_len;
  g.q_len = a.q_len;
  g.member = pl.member;
  SharedGrid ga = g, gb = g;
  ga.rows = p.rows_a;
  ga.lead = p.lead_a;
  ga.entry = pl.entry_a;
  ga.entries = pl.entries;
  ga.unit_parts = reinterpret_cast<int2*>(a.ws + p.unit_a);
  ga.m_part = reinterpret_cast<float*>(a.ws + p.m_a);
  ga.l_part = reinterpret_cast<float*>(a.ws + p.l_a);
  ga.o_part = reinterpret_cast<float*>(a.ws + p.o_a);
  gb.rows = p.rows_b;
  gb.lead = p.lead_b;
  gb.entry = pl.entry_b;
  gb.entries = pl.entries + 2;
  if (!p.only_b) gb.mark = pl.mark;
  gb.unit_parts = reinterpret_cast<int2*>(a.ws + p.unit_b);
  gb.m_part = reinterpret_cast<float*>(a.ws + p.m_b);
  gb.l_part = reinterpret_cast<float*>(a.ws + p.l_b);
  gb.o_part = reinterpret_cast<float*>(a.ws + p.o_b);
  JoinLaunch j{};
  j.list[0] = JoinList{ga.unit_parts, ga.m_part, ga.l_part, ga.o_part, p.rows_a, p.ctas_a};
  j.list[1] = JoinList{gb.unit_parts, gb.m_part, gb.l_part, gb.o_part, p.rows_b, p.ctas_b};
  j.seq = pl.seq;
  j.rows_b = p.rows_b;
  j.tiles_b = p.tiles_b;
  j.HK = a.c.H;
  j.mark = pl.mark;
  if (a.c.d == 128)
    return a.c.int8 ? launch_shared<128, true>(a, ga, gb, p, j, stream) : launch_shared<128, false>(a, ga, gb, p, j, stream);
  return a.c.int8 ? launch_shared<64, true>(a, ga, gb, p, j, stream) : launch_shared<64, false>(a, ga, gb, p, j, stream);
}

}  // namespace fa
