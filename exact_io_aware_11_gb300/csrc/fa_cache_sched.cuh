// How the attention over the cache shares its work out, computed on the
// device because the sequences' lengths live there.
//
// A unit is one (sequence, tile of query rows, cache head): row r of a tile is
// query row r / G of head r % G of the cache head's group of G. A unit's steps
// are the key tiles its rows see (at least one, so that units without keys
// still write their rows). All units' steps lie end to end, ordered by
// (sequence, row tile), then head, and before each unit's first a gap of `lead` steps: about
// what it costs a CTA to begin one more unit (AttnPlan). CTA c of C takes T / C of the T
// places, and one more if c < T mod C, an equal share whatever the lengths. A unit cut by a
// boundary leaves parts in the workspace: slot 2 c for the part CTA c starts in the middle of, slot
// 2 c + 1 for one it starts and does not finish. The CTA with a unit's last part
// writes the unit's merge record.
#pragma once

#include <type_traits>

#include "fa_cache_internal.h"
#include "fa_ptx.cuh"

namespace fa {

struct SharedEntry;

struct AttnGrid {
  int B, HK, N, G;
  int rows;       // query rows of a tile
  int row_tiles;  // tiles of N * G rows (one sequence's)
  int log2_keys;  // keys of a step
  int cap;        // tokens a page table row has room for
  int causal, split;
  int lead;       // places without a step before each unit
  const int32_t* kv_len;
  const int32_t* q_len;
  // workspace (split only)
  int4* record;   // [C]: entry, head, first CTA of a cut unit that c ends; entry -1: none
  float* m_part;  // [2 C][rows]
  float* l_part;
  float* o_part;  // [2 C][rows][D]; tiles (but not a list's): [2 C][rows / 32][D / 4][32 rows][4]
};
// What tells a kernel that the call's plan is made: the plan writes `call`, a number that no other call has, when all
// else is written; the join takes it away. See plan_wait.
struct PlanMark {
  unsigned long long* word;
  unsigned long long call;
};
// Shared prefixes (fa_cache_shared.cu): the entries, made on the device before, the sequences of
// the groups, and per unit the CTAs that its parts come from: {-1, 0} where a slot 2 C + unit has it whole.
// A struct of its own: with these in AttnGrid as well, that is past the size up to which a kernel's argument is
// held in registers, which cost the tile kernels without lists 1 to 3 % (128 rows of 16 sequences, 32 heads on 8,
// e4m3, pages of 16: 84.6 -> 86.0 us; d = 64 75.4 -> 77.5).
struct SharedGrid : AttnGrid {
  const SharedEntry* entry;
  const int* entries;  // how many, and the CTAs that work on them
  const int* member;
  int2* unit_parts;
  PlanMark mark;  // word set: the kernel runs beside the one before it, and waits for it at its end (attn_wait)
};

template <bool SH>
using AttnGridOf = std::conditional_t<SH, SharedGrid, AttnGrid>;

// One (sequence, row tile).
struct AttnEntry {
  int b, row0, kv, ql;  // first row of the tile; tokens and query rows of the sequence
  int seen;             // tokens the tile's last row sees
  int steps;
};
// An entry of a list: its keys begin at column `col` of b's row of the page table, and kv and seen
// count from there. list >= 0: the rows are those of all `count` sequences member[list],
// member[list + 1], ..., one sequence after another, over the same keys, of which all
// see every one. list < 0: count 1 where no part of b's rows comes from elsewhere.
struct __align__(16) SharedEntry : AttnEntry {
  int list, count, col, pad[3];
};
__device__ __forceinline__ int first_column(const AttnEntry&) { return 0; }
__device__ __forceinline__ int first_column(const SharedEntry& x) { return x.col; }
template <bool SH>
struct AttnEntryOf {
  using type = AttnEntry;
};
template <>
struct AttnEntryOf<true> {
  using type = SharedEntry;
};
template <bool SH>
__device__ __forceinline__ typename AttnEntryOf<SH>::type attn_entry(const AttnGridOf<SH>& g, int e) {
  typename AttnEntryOf<SH>::type x;
  if constexpr (SH) {
    const int4* const p = reinterpret_cast<const int4*>(g.entry + e);
    const int4 u = __ldcg(p), v = __ldcg(p + 1);
    x.b = u.x;
    x.row0 = u.y;
    x.kv = u.z;
    x.ql = u.w;
    x.seen = v.x;
    x.steps = v.y;
    x.list = v.z;
    x.count = v.w;
    x.col = __ldcg(reinterpret_cast<const int*>(p + 2));
  } else {
    x.b = e / g.row_tiles;
    x.row0 = (e - x.b * g.row_tiles) * g.rows;
    x.kv = min(g.cap, max(0, g.kv_len[x.b]));
    x.ql = g.q_len != nullptr ? min(g.N, max(0, g.q_len[x.b])) : g.N;
    const int rows = min(g.rows, x.ql * g.G - x.row0);
    x.seen = 0;
    if (rows > 0) x.seen = g.causal ? max(0, x.kv - x.ql + (x.row0 + rows - 1) / g.G + 1) : x.kv;
    x.steps = max(1, (x.seen + (1 << g.log2_keys) - 1) >> g.log2_keys);
  }
  return x;
}
// Tokens that row r of the tile sees.
__device__ __forceinline__ int attn_limit(const AttnGrid& g, const AttnEntry& x, int r) {
  const int i = (x.row0 + r) / g.G;
  if (i >= x.ql) return 0;
  return g.causal ? max(0, x.kv - x.ql + i + 1) : x.kv;
}

// Row r of an entry's tile. exists: it has a place in O and LSE; real: it stands for a query;
// limit: the keys that it sees, from the entry's first on.
struct AttnRow {
  int b, i, head, limit;  // sequence, query row, head of the cache head's group
  bool exists, real;
};
template <typename X>
__device__ __forceinline__ AttnRow shared_row(const SharedGrid& g, const X& x, int r) {
  AttnRow y;
  int row = x.row0 + r, ql = x.ql;
  y.b = x.b;
  y.exists = true;
  if (x.list >= 0) {
    const int rows = g.N * g.G, m = row / rows;
    y.exists = m < x.count;
    row -= m * rows;
    if (y.exists) {
      y.b = __ldcg(g.member + x.list + m);
      ql = g.q_len != nullptr ? min(g.N, max(0, __ldcg(g.q_len + y.b))) : g.N;
    }
  }
  y.i = row / g.G;
  y.head = row - y.i * g.G;
  y.exists = y.exists && y.i < g.N;
  y.real = y.exists && y.i < ql;
  y.limit = !y.real ? 0 : x.list >= 0 || !g.causal ? x.kv : max(0, x.kv - ql + y.i + 1);
  return y;
}

template <bool SH>
__device__ __forceinline__ int attn_entries(const AttnGridOf<SH>& g) {
  if constexpr (SH) return __ldcg(g.entries);
  return g.B * g.row_tiles;
}

// A CTA's place in the list: unit (e, h) at `step`, which is `pos` places from the
// list's start; the CTA's run lasts until `end`.
template <bool SH>
struct AttnCursor {
  typename AttnEntryOf<SH>::type x;
  int e, h, step;
  long long pos, end;
  __device__ __forceinline__ bool done(const AttnGridOf<SH>& g) const {
    // without a workspace a CTA finishes the units that start in its run
    return pos >= end && (g.split || step == 0);
  }
  __device__ __forceinline__ void next(const AttnGridOf<SH>& g) {
    ++pos;
    if (++step == x.steps) next_unit(g);
  }
  // Steps of this unit that are the CTA's.
  __device__ __forceinline__ int run(const AttnGridOf<SH>& g) const {
    const int left = x.steps - step;
    return g.split && end - pos < left ? static_cast<int>(end - pos) : left;
  }
  __device__ __forceinline__ void skip(const AttnGridOf<SH>& g, int n) {
    pos += n;
    step += n;
    if (step == x.steps) next_unit(g);
  }
  __device__ __forceinline__ void next_unit(const AttnGridOf<SH>& g) {
    step = 0;
    pos += g.lead;
    if (++h == g.HK) {
      h = 0;
      if (++e < attn_entries<SH>(g)) x = attn_entry<SH>(g, e);
    }
  }
};

// The places' division: CTA c starts at c * each + min(c, extra).
struct AttnShare {
  long long first;  // the first place of `entry`
  long long each;
  int extra, ctas, entry;
};
template <bool SH>
struct AttnShareOf : AttnShare {
  typename AttnEntryOf<SH>::type x;  // of `entry`
};
// A list's division is even to the place: CTA c starts at floor(c * total / ctas), so that the
// boundaries of equal units are boundaries of CTAs where there is a whole number of these to a unit.
template <>
struct AttnShareOf<true> : AttnShare {
  SharedEntry x;
  long long total;
};

// n / d for n that mostly fits 32 bits (a 64-bit division takes some 400 cycles).
__device__ __forceinline__ long long attn_div(long long n, long long d) {
  if (((n | d) >> 32) == 0) return static_cast<unsigned>(n) / static_cast<unsigned>(d);
  return n / d;
}
__device__ __forceinline__ long long attn_start(const AttnShareOf<false>& s, int c) {
  return c * s.each + min(c, s.extra);
}
__device__ __forceinline__ long long attn_start(const AttnShareOf<true>& s, int c) { return attn_div(c * s.total, s.ctas); }

// This CTA's cursor. Called by the whole CTA of kThreads threads; `sh` and
// `part` (kThreads / 32 words) are shared memory.
template <int kThreads, bool SH>
__device__ __forceinline__ AttnCursor<SH> attn_share(const AttnGridOf<SH>& g, AttnShareOf<SH>* sh, long long* part) {
  const int E = attn_entries<SH>(g), per = (E + kThreads - 1) / kThreads;
  const int e0 = min(E, static_cast<int>(threadIdx.x) * per), e1 = min(E, e0 + per);
  typename AttnEntryOf<SH>::type own{};  // the thread's only entry, where it has just one
  long long mine = 0;
  for (int e = e0; e < e1; ++e) {
    own = attn_entry<SH>(g, e);
    mine += own.steps + g.lead;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if ((threadIdx.x & 31) >= o) incl += v;
  }
  if ((threadIdx.x & 31) == 31) part[threadIdx.x >> 5] = incl;
  if (threadIdx.x == 0) sh->entry = E;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long v = part[w];
    if (w < static_cast<int>(threadIdx.x >> 5)) before += v;
    total += v;
  }
  before += incl - mine;
  total *= g.HK;
  AttnShareOf<SH> d{};
  int ctas = gridDim.x;
  if constexpr (SH) ctas = min(ctas, __ldcg(g.entries + 1));
  d.ctas = static_cast<int>(min(static_cast<long long>(ctas), total));
  if constexpr (SH) {
    d.total = total;
  } else {
    d.each = attn_div(total, d.ctas);
    d.extra = static_cast<int>(total - d.each * d.ctas);
  }
  const int c = blockIdx.x;
  const long long s0 = c < d.ctas ? attn_start(d, c) : total;
  long long p = before * g.HK;
  if (s0 >= p && s0 < p + mine * g.HK) {
    for (int e = e0; e < e1; ++e) {
      const typename AttnEntryOf<SH>::type x = per == 1 ? own : attn_entry<SH>(g, e);
      const long long n = static_cast<long long>(x.steps + g.lead) * g.HK;
      if (s0 < p + n) {
        sh->entry = e;
        sh->first = p;
        sh->x = x;
        break;
      }
      p += n;
    }
  }
  if (threadIdx.x == 0) {
    if constexpr (SH) {
      sh->total = d.total;
    } else {
      sh->each = d.each;
      sh->extra = d.extra;
    }
    sh->ctas = d.ctas;
  }
  __syncthreads();
  AttnCursor<SH> cur;
  cur.e = sh->entry;
  cur.h = 0;
  cur.step = 0;
  cur.pos = s0;
  cur.end = c < d.ctas ? attn_start(d, c + 1) : total;
  if (cur.e < E) {
    cur.x = sh->x;
    const long long rem = s0 - sh->first;
    const int places = cur.x.steps + g.lead;
    cur.h = static_cast<int>(attn_div(rem, places));
    const int at = static_cast<int>(rem - static_cast<long long>(cur.h) * places) - g.lead;
    cur.step = max(0, at);
    cur.pos += cur.step - at;
    if (!g.split && cur.step > 0) {  // the unit belongs to the CTA that it starts in
      cur.pos += cur.x.steps - cur.step;
      cur.next_unit(g);
    }
  } else {
    cur.pos = cur.end = total;
  }
  return cur;
}

// The CTA whose run holds place s.
__device__ __forceinline__ int attn_cta_of(long long s, const AttnShareOf<true>& d) {
  return static_cast<int>(attn_div((s + 1) * d.ctas - 1, d.total));
}
__device__ __forceinline__ int attn_cta_of(long long s, const AttnShareOf<false>& d) {
  const long long longer = d.extra * (d.each + 1);  // steps of the CTAs that have one more
  return static_cast<int>(s < longer ? attn_div(s, d.each + 1) : d.extra + attn_div(s - longer, d.each));
}

// Loads of what earlier kernels wrote: a list's, which may have been written while the kernel was being set up, past the L1 cache.
template <bool SH, typename T>
__device__ __forceinline__ T attn_load(const T* p) {
  if constexpr (SH) return __ldcg(p);
  return *p;
}
// Called by a whole CTA that has not waited for the kernels before it: what the plan wrote, and all kernels before the
// plan, is visible to the CTA from here on. A release after those writes and an acquire that reads its value order
// them; that the kernel which let this one go had waited is no promise to this one. Where the mark is not there, the CTA
// waits after all (it always is: the plan has ended before list A's kernel lets the next one go). One thread looks, of a
// warp that prepares nothing: 64 sequences behind 8192 tokens 49.4 -> 50.4 us, d = 64 55.8 -> 56.6, others within 1 %.
__device__ __forceinline__ void plan_wait(const PlanMark& m) {
  if (threadIdx.x == 64) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.u64 %0, [%1];" : "=l"(v) : "l"(__cvta_generic_to_global(m.word)) : "memory");
    if (v != m.call) grid_dep_wait();
  }
  __syncthreads();
}
// At the start (end false) and at the end of a kernel: the wait for the kernels before it. A list's kernel that runs beside
// the one before it waits for the plan at its start, for that kernel at its end.
template <bool SH>
__device__ __forceinline__ void attn_wait(const AttnGridOf<SH>& g, bool end) {
  if constexpr (SH) {
    if (g.mark.word == nullptr) {
      if (end) return;
    } else if (!end) {
      plan_wait(g.mark);
      return;
    }
  } else if (end) {
    return;
  }
  grid_dep_wait();
}

// Keys of a step and rows of a tile of the kernel that a call of `rows` = N * G
// query rows per (sequence, cache head) takes, and its CTAs.
struct AttnPlan {
  int rows, log2_keys, ctas, lead;
  long long units, cap_steps;
};
AttnPlan attn_plan(int B, int HK, long long rows, long long cap, int d);

// Tiles of 64, 128 (g.rows) or 2 x 128 query rows on tcgen05 (fa_cache_tile.cuh), one
// translation unit for each format.
cudaError_t launch_cache_attention_tiles_e4m3(const CacheAttnLaunch& a, const AttnGrid& g, int ctas,
                                              cudaStream_t stream);
cudaError_t launch_cache_attention_tiles_int8(const CacheAttnLaunch& a, const AttnGrid& g, int ctas,
                                              cudaStream_t stream);
// The same over a list of entries (SharedGrid::entry).
cudaError_t launch_shared_tiles_e4m3(const CacheAttnLaunch& a, const SharedGrid& g, int ctas, cudaStream_t stream);
cudaError_t launch_shared_tiles_int8(const CacheAttnLaunch& a, const SharedGrid& g, int ctas, cudaStream_t stream);

}  // namespace fa
