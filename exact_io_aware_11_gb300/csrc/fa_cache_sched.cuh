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

#include "fa_cache_internal.h"

namespace fa {

struct AttnGrid {
  int B, HK, N, G;
  int rows;       // query rows of a tile
  int row_tiles;  // tiles of N * G rows
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
  float* o_part;  // [2 C][rows][D]; tiles: [2 C][rows / 32][D / 4][32 rows][4]
};

// One (sequence, row tile).
struct AttnEntry {
  int b, row0, kv, ql;  // first row of the tile; tokens and query rows of the sequence
  int seen;             // tokens the tile's last row sees
  int steps;
};
__device__ __forceinline__ AttnEntry attn_entry(const AttnGrid& g, int e) {
  AttnEntry x;
  x.b = e / g.row_tiles;
  x.row0 = (e - x.b * g.row_tiles) * g.rows;
  x.kv = min(g.cap, max(0, g.kv_len[x.b]));
  x.ql = g.q_len != nullptr ? min(g.N, max(0, g.q_len[x.b])) : g.N;
  const int rows = min(g.rows, x.ql * g.G - x.row0);
  x.seen = 0;
  if (rows > 0) x.seen = g.causal ? max(0, x.kv - x.ql + (x.row0 + rows - 1) / g.G + 1) : x.kv;
  x.steps = max(1, (x.seen + (1 << g.log2_keys) - 1) >> g.log2_keys);
  return x;
}
// Tokens that row r of the tile sees.
__device__ __forceinline__ int attn_limit(const AttnGrid& g, const AttnEntry& x, int r) {
  const int i = (x.row0 + r) / g.G;
  if (i >= x.ql) return 0;
  return g.causal ? max(0, x.kv - x.ql + i + 1) : x.kv;
}

// A CTA's place in the list: unit (e, h) at `step`, which is `pos` places from the
// list's start; the CTA's run lasts until `end`.
struct AttnCursor {
  AttnEntry x;
  int e, h, step;
  long long pos, end;
  __device__ __forceinline__ bool done(const AttnGrid& g) const {
    // without a workspace a CTA finishes the units that start in its run
    return pos >= end && (g.split || step == 0);
  }
  __device__ __forceinline__ void next(const AttnGrid& g) {
    ++pos;
    if (++step == x.steps) next_unit(g);
  }
  // Steps of this unit that are the CTA's.
  __device__ __forceinline__ int run(const AttnGrid& g) const {
    const int left = x.steps - step;
    return g.split && end - pos < left ? static_cast<int>(end - pos) : left;
  }
  __device__ __forceinline__ void skip(const AttnGrid& g, int n) {
    pos += n;
    step += n;
    if (step == x.steps) next_unit(g);
  }
  __device__ __forceinline__ void next_unit(const AttnGrid& g) {
    step = 0;
    pos += g.lead;
    if (++h == g.HK) {
      h = 0;
      if (++e < g.B * g.row_tiles) x = attn_entry(g, e);
    }
  }
};

// The places' division: CTA c starts at c * each + min(c, extra).
struct AttnShare {
  long long first;  // the first place of `entry`
  long long each;
  int extra, ctas, entry;
  AttnEntry x;      // of `entry`
};

// n / d for n that mostly fits 32 bits (a 64-bit division takes some 400 cycles).
__device__ __forceinline__ long long attn_div(long long n, long long d) {
  if (((n | d) >> 32) == 0) return static_cast<unsigned>(n) / static_cast<unsigned>(d);
  return n / d;
}
__device__ __forceinline__ long long attn_start(const AttnShare& s, int c) {
  return c * s.each + min(c, s.extra);
}

// This CTA's cursor. Called by the whole CTA of kThreads threads; `sh` and
// `part` (kThreads / 32 words) are shared memory.
template <int kThreads>
__device__ __forceinline__ AttnCursor attn_share(const AttnGrid& g, AttnShare* sh, long long* part) {
  const int E = g.B * g.row_tiles, per = (E + kThreads - 1) / kThreads;
  const int e0 = min(E, static_cast<int>(threadIdx.x) * per), e1 = min(E, e0 + per);
  AttnEntry own{};  // the thread's only entry, where it has just one
  long long mine = 0;
  for (int e = e0; e < e1; ++e) {
    own = attn_entry(g, e);
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
  AttnShare d{};
  d.ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  d.each = attn_div(total, d.ctas);
  d.extra = static_cast<int>(total - d.each * d.ctas);
  const int c = blockIdx.x;
  const long long s0 = c < d.ctas ? attn_start(d, c) : total;
  long long p = before * g.HK;
  if (s0 >= p && s0 < p + mine * g.HK) {
    for (int e = e0; e < e1; ++e) {
      const AttnEntry x = per == 1 ? own : attn_entry(g, e);
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
    sh->each = d.each;
    sh->extra = d.extra;
    sh->ctas = d.ctas;
  }
  __syncthreads();
  AttnCursor cur;
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
__device__ __forceinline__ int attn_cta_of(long long s, const AttnShare& d) {
  const long long longer = d.extra * (d.each + 1);  // steps of the CTAs that have one more
  return static_cast<int>(s < longer ? attn_div(s, d.each + 1) : d.extra + attn_div(s - longer, d.each));
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

}  // namespace fa
