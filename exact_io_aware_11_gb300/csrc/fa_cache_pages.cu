// The pages of the 8-bit cache: copying them in every layer, sequences that share them
// (fa_cache_fork), pages for tokens to come (fa_cache_reserve), and moving the pages in use
// together (fa_cache_compact). What these do is counting and copying; the definitions are in fa.h.
//
// refs[p] counts the table entries that name page p; a page is free where it is 0. The counts
// change by integer adds, whose order does not matter, so that every call has one result.
#include "fa_cache_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

__device__ __forceinline__ bool is_page(int p, int num_pages) { return p >= 0 && p < num_pages; }

// ------------------------------------------------------------------ copying
// Every (move, layer, K or V) is a run of contiguous codes, cut into pieces. A CTA's first warp sends
// its pieces through a ring in shared memory with bulk copies (no registers, no cache lines held); the
// other warps copy the scales. Bound: memory, two bytes moved per code: 500 pages of 64 KB, K and V, in 8 layers 167 us,
// 6280 GB/s; 3 pages of 12 KB 2.6 us.
constexpr int kCopyWarps = 4, kCopyStages = 6, kCopyAhead = 4;  // pieces that are loaded ahead
constexpr int kCopyPiece = 32768;  // at most
constexpr int kCopySmem(int piece) { return kCopyStages * piece + 128; }

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(__cvta_generic_to_global(dst)),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Move m's pages; false where there is none.
__device__ __forceinline__ bool move_of(const PageCopyLaunch& a, int m, int* src, int* dst) {
  *src = a.src[m];
  *dst = a.dst[m];
  if (*src == -1 || *dst == -1 || *src == *dst) return false;
  if (is_page(*src, a.num_pages) && is_page(*dst, a.num_pages)) return true;
  report_bad_page(a.status);
  return false;
}

__global__ void __launch_bounds__(kCopyWarps * 32) page_copy_kernel(const __grid_constant__ PageCopyLaunch a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kCopyStages];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  check_init(a.status);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kCopyStages; ++i) mbar_init(full + i, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const int n = a.count != nullptr ? min(a.n, *a.count) : a.n;
  const int per_layer = 2, tensors = a.layers * per_layer;
  if (warp > 0) {  // scales
    const long long items = static_cast<long long>(n) * tensors;
    for (long long i = blockIdx.x * (kCopyWarps - 1LL) + warp - 1; i < items; i += gridDim.x * (kCopyWarps - 1LL)) {
      const int m = static_cast<int>(i / tensors), t = static_cast<int>(i - static_cast<long long>(m) * tensors);
      int src, dst;
      if (!move_of(a, m, &src, &dst)) continue;
      float* const s = a.layer[t >> 1].scale[t & 1];
      for (int h = lane; h < a.H; h += 32) s[static_cast<long long>(dst) * a.H + h] = s[static_cast<long long>(src) * a.H + h];
    }
    return;
  }
  const int pieces = static_cast<int>(a.page_bytes / a.piece);
  const long long items = static_cast<long long>(n) * tensors * pieces;
  const Watchdog wd{a.wait_limit, a.status, &abort_flag};
  // Lane l looks up the warp's pieces l, l + 32, ...; lane 0 issues them.
  const uint8_t* from = nullptr;
  uint8_t* to = nullptr;
  auto look = [&](long long k) {
    const long long i = blockIdx.x + k * gridDim.x;
    from = nullptr;
    if (i >= items) return;
    const long long mt = i / pieces;
    const int part = static_cast<int>(i - mt * pieces), m = static_cast<int>(mt / tensors), t = static_cast<int>(mt - static_cast<long long>(m) * tensors);
    int src, dst;
    if (!move_of(a, m, &src, &dst)) return;
    uint8_t* const c = a.layer[t >> 1].code[t & 1] + static_cast<long long>(part) * a.piece;
    from = c + src * a.page_bytes;
    to = c + dst * a.page_bytes;
  };
  const long long mine = items > blockIdx.x ? (items - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  long long loaded = 0, stored = 0;    // pieces
  unsigned long long go[kCopyAhead];   // where the pieces that are loaded go to, in turn
  // Lane 0 keeps the destinations; every lane walks the same loop.
  bool ok = true;
  for (long long k0 = 0; k0 < mine && ok; k0 += 32) {
    look(k0 + lane);
    const int batch = static_cast<int>(min(32LL, mine - k0));
    for (int j = 0; j < batch && ok; ++j) {
      const unsigned long long f = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), j);
      const unsigned long long d = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), j);
      if (f == 0ull) continue;  // no move
      const int st = static_cast<int>(loaded % kCopyStages);
      if (lane == 0) {
        // the store that used the stage before has read it: at most the latest few have not
        if (loaded >= kCopyStages) bulk_wait_read<kCopyStages - kCopyAhead - 1>();
        mbar_expect_tx(full + st, a.piece);
        bulk_load(smem + st * a.piece, reinterpret_cast<const void*>(f), a.piece, full + st);
      }
      __syncwarp();
      // the destinations move up; [0] is the oldest piece that is not stored once the ring is full
      const bool drain = loaded - stored == kCopyAhead;
      if (drain) {
        const int os = static_cast<int>(stored % kCopyStages);
        ok = mbar_wait_warp(full + os, static_cast<uint32_t>(stored / kCopyStages) & 1u, wd);
        if (ok) {
          if (lane == 0) {
            bulk_store(reinterpret_cast<void*>(go[0]), smem + os * a.piece, a.piece);
            bulk_commit();
          }
          ++stored;
#pragma unroll
          for (int i = 0; i + 1 < kCopyAhead; ++i) go[i] = go[i + 1];
        }
      }
      const int at = static_cast<int>(loaded - stored);
#pragma unroll
      for (int i = 0; i < kCopyAhead; ++i)
        if (i == at) go[i] = d;
      ++loaded;
    }
  }
  for (; stored < loaded; ++stored) {
    const int os = static_cast<int>(stored % kCopyStages);
    const bool landed = mbar_wait_drain(full + os, static_cast<uint32_t>(stored / kCopyStages) & 1u, a.wait_limit);
    if (!landed) {
      ok = false;
      if (lane == 0) watchdog_fire(a.status, &abort_flag);
    }
    if (ok && lane == 0) {
      bulk_store(reinterpret_cast<void*>(go[0]), smem + os * a.piece, a.piece);
      bulk_commit();
    }
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
#pragma unroll
    for (int i = 0; i + 1 < kCopyAhead; ++i) go[i] = go[i + 1];
  }
  if (lane == 0) bulk_wait0();
}

// ------------------------------------------------------------------ forking
// A CTA takes some columns of every row, so that rows can be exchanged in place: all that the new
// entries are made from is read into shared memory before any is written. Bound: latency (the parent, its entry, the
// store), for large tables memory.
constexpr int kForkThreads = 512, kForkWords = 16384;

__global__ void __launch_bounds__(kForkThreads) page_fork_kernel(const __grid_constant__ PageForkLaunch a) {
  extern __shared__ int2 stage[];  // [rows][cols]: an entry as it was, as it will be
  grid_dep_wait();
  grid_dep_launch();
  const PageTable& t = a.t;
  const int c0 = blockIdx.x << a.log2_cols, cols = 1 << a.log2_cols;
  const int n = t.rows << a.log2_cols;
#pragma unroll 2
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int b = i >> a.log2_cols, c = c0 + (i & (cols - 1));
    if (c >= t.width) continue;
    int p = a.parent != nullptr ? a.parent[b] : b;
    const int keep = a.keep != nullptr ? a.keep[b] : 0, old = t.entry[b * t.stride + c];
    if (p < -1 || p >= t.rows) {  // such a row stays as it is, but for `keep`
      if (c0 == 0) report_bad_page(a.status);
      p = b;
    }
    const bool kept = p >= 0 && (a.keep == nullptr || static_cast<long long>(c) * t.page < keep);
    int now = -1;
    if (kept) now = p == b ? old : t.entry[p * t.stride + c];
    if (p != b && now != -1 && !is_page(now, t.num_pages)) {
      report_bad_page(a.status);
      now = -1;
    }
    stage[i] = make_int2(old, now);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int b = i >> a.log2_cols, c = c0 + (i & (cols - 1));
    if (c >= t.width) continue;
    const int2 e = stage[i];
    if (e.x == e.y) continue;
    t.entry[b * t.stride + c] = e.y;
    if (e.y >= 0) atomicAdd(t.refs + e.y, 1);
    if (is_page(e.x, t.num_pages))
      atomicAdd(t.refs + e.x, -1);
    else if (e.x != -1)
      report_bad_page(a.status);
  }
}

// ------------------------------------------------------------------ CTAs that count
// One CTA for pools of up to 8192 pages, a cluster of eight for others.
constexpr int kCluster = 8, kSmallPool = 8192;
constexpr int count_threads(int ctas) { return ctas == 1 ? 1024 : 512; }

template <int C>
__device__ __forceinline__ void cluster_sync() {
  if constexpr (C == 1)
    __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int load_l2(const int* p) {
  int v;
  asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)) : "memory");
  return v;
}

// Exclusive prefix of v over the CTA's threads, and the sum. `part`: a word a warp.
template <int C>
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // part's last values have been read
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  int p = lane < count_threads(C) / 32 ? part[lane] : 0, sum = p;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  *total = __shfl_sync(0xffffffffu, sum, 31);
  return __shfl_sync(0xffffffffu, sum - p, warp) + incl - v;
}
// Each CTA's v written to `slot` (a word a CTA of shared memory, used once) of all; a barrier of the cluster.
template <int C>
__device__ __forceinline__ void write_slot(int v, int* slot, int rank) {
  if constexpr (C > 1) {
    if (threadIdx.x < C) {
      uint32_t to;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(slot + rank)), "r"(threadIdx.x));
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
    }
  } else if (threadIdx.x == 0) {
    slot[0] = v;
  }
}
template <int C>
__device__ __forceinline__ void exchange(int v, int* slot, int rank) {
  write_slot<C>(v, slot, rank);
  cluster_sync<C>();
}
// What the CTAs before this one have in `slot`, and all.
template <int C>
__device__ __forceinline__ int sum_slots(const int* slot, int rank, int* total) {
  int before = 0, sum = 0;
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const int x = slot[r];
    if (r < rank) before += x;
    sum += x;
  }
  *total = sum;
  return before;
}
template <int C>
__device__ __forceinline__ int cluster_scan(int v, int* slot, int rank, int* total) {
  exchange<C>(v, slot, rank);
  return sum_slots<C>(slot, rank, total);
}
// The CTA's share of the pages.
struct PageSlice {
  int first, end;
};
template <int C>
__device__ __forceinline__ PageSlice page_slice(int num_pages, int rank) {
  const int per = ((num_pages + C - 1) / C + 3) & ~3;
  const long long f = static_cast<long long>(per) * rank;
  return PageSlice{static_cast<int>(min(f, static_cast<long long>(num_pages))),
                   static_cast<int>(min(f + per, static_cast<long long>(num_pages)))};
}
// Pages p of the slice with want(p, refs[p]), counted.
template <int C, typename Want>
__device__ __forceinline__ int count_pages(const PageSlice& s, const int* refs, int* part, Want want) {
  int mine = 0, total;
#pragma unroll 4
  for (int p = s.first + threadIdx.x; p < s.end; p += count_threads(C)) mine += want(p, load_l2(refs + p)) ? 1 : 0;
  block_scan<C>(mine, part, &total);
  return total;
}
// The same pages, in order: the k-th, from `rank0` on, goes to list[k] where k < most.
template <int C, typename Want>
__device__ __forceinline__ void list_pages(const PageSlice& s, const int* refs, int* part, int rank0, int most, int* list, Want want) {
  for (int p0 = s.first; p0 < s.end && rank0 < most; p0 += 4 * count_threads(C)) {
    const int p = p0 + 4 * threadIdx.x;
    int w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p + i < s.end && want(p + i, load_l2(refs + p + i))) w |= 1 << i;
    int total;
    int k = rank0 + block_scan<C>(__popc(w), part, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (w >> i & 1) {
        if (k < most) list[k] = p + i;
        ++k;
      }
    rank0 += total;
  }
}

// ------------------------------------------------------------------ reserving
// The items are the columns of the rows' ranges, in the order of rows; each CTA has an equal run of them. An
// item without a page takes one, an item whose page has no other user keeps it. Who copies a page that several
// items write to: all but the last one, which keeps it if nobody outside the call has it. That is
// found in refs itself: every such item takes itself off its page's count; where nothing is left the last
// item, by an atomic minimum of -(2^30 + its number), keeps the page.
// Bound: latency, four to eight round trips to memory between barriers of the cluster: 10 rows of which 8 share pages 8 us,
// 160 rows with 9200 new pages 12 us.
constexpr int kItemCache = 4096;  // items of a CTA that are kept in shared memory
enum : int { kTakes = 0, kOwn = 1, kShared = 2, kKeeps = 3 };  // kShared: takes one, once the keepers are known
constexpr int reserve_smem(int rows) { return kItemCache * 8 + (2 * rows + 1) * 4; }

template <int C>
__global__ void __launch_bounds__(count_threads(C), 1)
    page_reserve_kernel(const __grid_constant__ PageReserveLaunch a) {
  extern __shared__ int2 cache[];  // row and state, entry
  constexpr int kThreads = count_threads(C);
  __shared__ int part[kThreads / 32];
  __shared__ int slots[4][C];  // items that take a page (and whether any is shared), these after the election, free pages, the first row that fails
  __shared__ int fail_row, any_shared;
  const PageTable& t = a.t;
  const int rank = C == 1 ? 0 : blockIdx.x;  // the grid is one cluster
  int* const first_item = reinterpret_cast<int*>(cache + kItemCache);  // [rows + 1]
  int* const first_col = first_item + t.rows + 1;                      // [rows]
  cluster_sync<C>();  // every CTA has begun: its shared memory may be written to
  grid_dep_wait();
  if (threadIdx.x == 0) {
    fail_row = t.rows;
    any_shared = 0;
    if (rank == 0) *a.moves = 0;
  }
  // ---- the rows' ranges: every CTA has all of them
  int all_items = 0;
  for (int r0 = 0; r0 < t.rows; r0 += kThreads) {
    const int b = r0 + threadIdx.x;
    int n = 0;
    if (b < t.rows) {
      const long long s = a.start != nullptr ? a.start[b] : 0;
      const long long c = max(0, a.count != nullptr ? a.count[b] : a.tokens);
      const bool fits = c == 0 || (s >= 0 && s + c <= static_cast<long long>(t.width) * t.page);
      const int col = fits && c > 0 ? static_cast<int>(s / t.page) : 0;
      if (fits && c > 0) n = static_cast<int>((s + c + t.page - 1) / t.page) - col;
      first_col[b] = col;
      if (rank == 0) a.ok[b] = fits ? 1 : 0;
    }
    int total;
    const int k = block_scan<C>(n, part, &total);
    if (b < t.rows) first_item[b] = all_items + k;
    all_items += total;
  }
  if (threadIdx.x == 0) first_item[t.rows] = all_items;
  __syncthreads();
  const int item0 = static_cast<int>(static_cast<long long>(all_items) * rank / C);
  const int items = static_cast<int>(static_cast<long long>(all_items) * (rank + 1) / C) - item0;
  struct Item {
    int row, col, entry, state;
  };
  auto row_of = [&](int i) {  // the last row with first_item <= i
    int lo = 0, hi = t.rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      (first_item[mid] <= i ? lo : hi) = mid;
    }
    return lo;
  };
  auto column = [&](int row, int i) { return first_col[row] + item0 + i - first_item[row]; };
  auto item = [&](int i) {
    Item x;
    if (i < kItemCache) {
      const int2 v = cache[i];
      x.row = v.x >> 2;
      x.state = v.x & 3;
      x.entry = v.y;
      x.col = column(x.row, i);
    } else {
      x.row = row_of(item0 + i);
      x.col = column(x.row, i);
      x.entry = t.entry[x.row * t.stride + x.col];
      x.state = is_page(x.entry, t.num_pages) ? kShared : kTakes;
    }
    return x;
  };
  auto code = [&](int i) { return -(1 << 30) - (item0 + i); };
  // ---- what each item has
  constexpr int kAtOnce = 4;
  int mine = 0;
  for (int i0 = 0; i0 < items; i0 += kAtOnce * kThreads) {
    int row[kAtOnce], entry[kAtOnce], refs[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads + threadIdx.x;
      row[k] = 0;
      entry[k] = -1;
      if (i < items) {
        row[k] = row_of(item0 + i);
        entry[k] = t.entry[row[k] * t.stride + column(row[k], i)];
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) refs[k] = is_page(entry[k], t.num_pages) ? load_l2(t.refs + entry[k]) : 0;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kThreads + threadIdx.x;
      if (i >= items) continue;
      int state = kTakes;
      if (is_page(entry[k], t.num_pages))
        state = i < kItemCache && refs[k] == 1 ? kOwn : kShared;
      else if (entry[k] != -1)
        report_bad_page(a.status);
      if (state == kTakes) ++mine;
      if (state == kShared) any_shared = 1;
      if (i < kItemCache) cache[i] = make_int2(row[k] << 2 | state, entry[k]);
    }
  }
  int need, wanted, all_free;
  auto is_free = [](int, int refs) { return refs == 0; };
  const PageSlice s = page_slice<C>(t.num_pages, rank);
  const int have = count_pages<C>(s, t.refs, part, is_free);
  block_scan<C>(mine, part, &need);
  // (need is at most the pages of the table's rows, 2^30: a bit is left for any_shared)
  write_slot<C>(have, slots[2], rank);
  exchange<C>(need | (any_shared != 0 ? 1 << 31 : 0), slots[0], rank);
  const int free_before = sum_slots<C>(slots[2], rank, &all_free);
  int before = 0;
  bool shared = false;
  wanted = 0;
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const int v = slots[0][r];
    shared |= v < 0;
    if (r < rank) before += v & 0x7fffffff;
    wanted += v & 0x7fffffff;
  }
  // whether item i takes a page; final once `shared` has been dealt with
  auto takes = [&](const Item& x, int i) {
    return x.state == kTakes || (x.state == kShared && (i < kItemCache || load_l2(t.refs + x.entry) != code(i)));
  };
  if (shared) {
    // ---- such items off their pages' counts; pages that nobody else has: the last item keeps them
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const Item x = item(i);
      if (x.state == kShared) atomicAdd(t.refs + x.entry, -1);
    }
    cluster_sync<C>();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const Item x = item(i);
      if (x.state == kShared && load_l2(t.refs + x.entry) <= 0) atomicMin(t.refs + x.entry, code(i));
    }
    cluster_sync<C>();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const Item x = item(i);
      if (x.state != kShared) continue;
      if (load_l2(t.refs + x.entry) != code(i))
        ++mine;
      else if (i < kItemCache)
        cache[i].x = x.row << 2 | kKeeps;
    }
    block_scan<C>(mine, part, &need);
    before = cluster_scan<C>(need, slots[1], rank, &wanted);
  }
  int f = t.rows;  // the first row that fails
  if (wanted > 0) {  // the same in every CTA
    if (wanted > all_free) {
      int k0 = before;
      for (int i0 = 0; i0 < items; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        Item x{};
        const bool take = i < items && (x = item(i), takes(x, i));
        int total;
        const int k = k0 + block_scan<C>(take ? 1 : 0, part, &total);
        if (take && k >= all_free) atomicMin(&fail_row, x.row);
        k0 += total;
      }
      __syncthreads();
      exchange<C>(fail_row, slots[3], rank);
#pragma unroll
      for (int r = 0; r < C; ++r) f = min(f, slots[3][r]);
    }
    list_pages<C>(s, t.refs, part, free_before, min(wanted, all_free), a.list, is_free);
    cluster_sync<C>();
  }
  // ---- pages dealt out
  if (shared || wanted > 0) {
    int k0 = before;
    for (int i0 = 0; i0 < items; i0 += kAtOnce * kThreads) {
      Item x[kAtOnce];
      int take = 0;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = i0 + kAtOnce * threadIdx.x + k;
        x[k].state = kOwn;
        if (i >= items) continue;
        x[k] = item(i);
        if (takes(x[k], i)) take |= 1 << k;
      }
      int total, at = k0 + block_scan<C>(__popc(take), part, &total), page[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (take >> k & 1) page[k] = x[k].row < f ? load_l2(a.list + at++) : -1;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int b = x[k].row, p = page[k];
        if (!(take >> k & 1)) {
          // (below, the rows that fail come back to their pages' counts)
          if (x[k].state == kKeeps || x[k].state == kShared) t.refs[x[k].entry] = b < f ? 1 : 0;
        } else if (b < f && is_page(p, t.num_pages)) {  // (it is one, if refs counts the entries)
          t.entry[b * t.stride + x[k].col] = p;
          t.refs[p] = 1;
          // earlier tokens of the sequence in the page
          if (x[k].state == kShared && x[k].col == first_col[b] && (a.start != nullptr ? a.start[b] : 0) % t.page != 0) {
            const int m = atomicAdd(a.moves, 1);
            a.src[m] = x[k].entry;
            a.dst[m] = p;
          }
        }
      }
      k0 += total;
    }
  }
  if (f < t.rows) {
    cluster_sync<C>();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const Item x = item(i);
      if ((x.state == kShared || x.state == kKeeps) && x.row >= f) atomicAdd(t.refs + x.entry, 1);
    }
    cluster_sync<C>();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const Item x = item(i);
      if (x.row >= f && x.state != kOwn && (x.state == kTakes || load_l2(t.refs + x.entry) != 1)) a.ok[x.row] = 0;
    }
  }
  grid_dep_launch();
}

// ------------------------------------------------------------------ compacting
// L pages are in use. The k-th of them with a number >= L goes to the k-th free number below L, so
// that no page is read and written, and no more pages move than have to. Bound: latency (2048 pages 5 us) beside the copies.
template <int C>
__global__ void __launch_bounds__(count_threads(C), 1)
    page_compact_kernel(const __grid_constant__ PageCompactLaunch a) {
  constexpr int kThreads = count_threads(C);
  __shared__ int part[kThreads / 32];
  __shared__ int slots[3][C];
  const int rank = C == 1 ? 0 : blockIdx.x, P = a.t.num_pages;
  int* const refs = a.t.refs;
  cluster_sync<C>();  // every CTA has begun: its shared memory may be written to
  grid_dep_wait();
  const PageSlice s = page_slice<C>(P, rank);
  int live, moves, holes;
  cluster_scan<C>(count_pages<C>(s, refs, part, [](int, int r) { return r != 0; }), slots[0], rank, &live);
  auto mover = [live](int p, int r) { return p >= live && r != 0; };
  auto hole = [live](int p, int r) { return p < live && r == 0; };
  const int m0 = cluster_scan<C>(count_pages<C>(s, refs, part, mover), slots[1], rank, &moves);
  const int h0 = cluster_scan<C>(count_pages<C>(s, refs, part, hole), slots[2], rank, &holes);
  list_pages<C>(s, refs, part, m0, moves, a.src, mover);
  list_pages<C>(s, refs, part, h0, moves, a.dst, hole);
  for (int p = s.first + threadIdx.x; p < s.end; p += kThreads) a.where[p] = load_l2(refs + p) != 0 ? p : -1;
  if (rank == 0 && threadIdx.x == 0) {
    *a.live = live;
    *a.moves = moves;
  }
  cluster_sync<C>();
  for (int k = rank * kThreads + threadIdx.x; k < moves; k += C * kThreads) {
    const int from = load_l2(a.src + k), to = load_l2(a.dst + k);
    a.where[from] = to;
    refs[to] = load_l2(refs + from);
    refs[from] = 0;
  }
  grid_dep_launch();
}

__global__ void __launch_bounds__(256) page_rename_kernel(const __grid_constant__ PageCompactLaunch a) {
  grid_dep_wait();
  grid_dep_launch();
  const PageTable& t = a.t;
  const long long n = static_cast<long long>(t.rows) * t.width;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const long long b = i / t.width;
    int* const at = t.entry + b * t.stride + (i - b * t.width);
    const int e = *at;
    if (is_page(e, t.num_pages))
      *at = a.where[e];
    else if (e != -1)
      report_bad_page(a.status);
  }
}

// Launches a kernel of one CTA or of one cluster.
template <typename... KArgs, typename... Args>
cudaError_t launch_counting(void (*kern)(KArgs...), int ctas, size_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(count_threads(ctas));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

size_t words(long long n) { return align256(static_cast<size_t>(n) * 4); }

}  // namespace

cudaError_t launch_page_copy(PageCopyLaunch a, const fa_cache* caches, int layers, cudaStream_t stream) {
  const fa_cache& c = caches[0];
  a.page_bytes = static_cast<long long>(c.H) * c.page_size * c.d;
  a.H = c.H;
  a.num_pages = c.num_pages;
  for (int l0 = 0; l0 < layers; l0 += kCopyLayers) {
    a.layers = layers - l0 < kCopyLayers ? layers - l0 : kCopyLayers;
    for (int l = 0; l < a.layers; ++l) {
      const fa_cache& x = caches[l0 + l];
      a.layer[l] = PageCopyLaunch::Layer{{static_cast<uint8_t*>(x.k), static_cast<uint8_t*>(x.v)}, {x.k_scale, x.v_scale}};
    }
    // pieces of 32 KB (500 pages of 64 KB in 8 layers 166.8 us, of 16 KB 169.0), smaller ones where there would be few
    const long long runs = static_cast<long long>(a.n) * a.layers * 2;
    long long piece = a.page_bytes;
    while (piece > kCopyPiece || (piece > 2048 && runs * (a.page_bytes / piece) < 4LL * sm_count())) {
      if (piece % 2 == 0 && (piece / 2) % 128 == 0) {
        piece /= 2;
        continue;
      }
      // an odd number of heads: a multiple of 1024 bytes that divides the page
      long long best = 1024;
      for (long long p = 2048; p < piece && p <= kCopyPiece; p += 1024)
        if (a.page_bytes % p == 0) best = p;
      piece = best;
      break;
    }
    a.piece = static_cast<int>(piece);
    const long long items = runs * (a.page_bytes / piece);
    const int grid = static_cast<int>(items < sm_count() ? items : sm_count());
    static std::atomic<unsigned long long> smem_set{0};
    cudaError_t e = set_smem_once(smem_set, reinterpret_cast<const void*>(page_copy_kernel), kCopySmem(kCopyPiece));
    if (e != cudaSuccess) return e;
    e = launch_pdl(page_copy_kernel, dim3(grid), dim3(kCopyWarps * 32), kCopySmem(a.piece), stream, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_page_fork(PageForkLaunch a, cudaStream_t stream) {
  // 32 columns a CTA, fewer where the staged entries would not fit or most SMs would be idle (256 rows of 66: 7.6 us with 8
  // columns, 2.4 with one)
  a.log2_cols = 5;
  while (a.log2_cols > 0 && ((a.t.rows << a.log2_cols) > kForkWords || (a.t.width >> a.log2_cols) < sm_count())) --a.log2_cols;
  const int smem = (a.t.rows << a.log2_cols) * 8;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = set_smem_once(smem_set, reinterpret_cast<const void*>(page_fork_kernel), kForkWords * 8);
  if (e != cudaSuccess) return e;
  const int grid = (a.t.width + (1 << a.log2_cols) - 1) >> a.log2_cols;
  return launch_pdl(page_fork_kernel, dim3(grid), dim3(kForkThreads), smem, stream, a);
}

size_t reserve_workspace(int rows, int width, int num_pages) {
  const long long most = static_cast<long long>(rows) * width;  // pages that a call can take
  return 256 + 2 * words(rows) + words(most < num_pages ? most : num_pages);
}
cudaError_t launch_page_reserve(PageReserveLaunch a, const fa_cache* caches, int layers, uint8_t* ws, cudaStream_t stream) {
  a.moves = reinterpret_cast<int*>(ws);
  a.src = reinterpret_cast<int*>(ws + 256);
  a.dst = reinterpret_cast<int*>(ws + 256 + words(a.t.rows));
  a.list = reinterpret_cast<int*>(ws + 256 + 2 * words(a.t.rows));
  const bool small = a.t.num_pages <= kSmallPool;
  auto kern = small ? page_reserve_kernel<1> : page_reserve_kernel<kCluster>;
  static std::atomic<unsigned long long> smem_set[2];
  cudaError_t e = set_smem_once(smem_set[small], reinterpret_cast<const void*>(kern), reserve_smem(kPageTableRows));
  if (e != cudaSuccess) return e;
  e = launch_counting(kern, small ? 1 : kCluster, reserve_smem(a.t.rows), stream, a);
  if (e != cudaSuccess) return e;
  PageCopyLaunch c{};
  c.src = a.src;
  c.dst = a.dst;
  c.n = a.t.rows;
  c.count = a.moves;
  c.status = a.status;
  c.wait_limit = kWaitLimitCycles;
  return launch_page_copy(c, caches, layers, stream);
}

size_t compact_workspace(int num_pages) { return 256 + 2 * words(num_pages / 2 + 1); }
cudaError_t launch_page_compact(PageCompactLaunch a, const fa_cache* caches, int layers, uint8_t* ws, cudaStream_t stream) {
  a.moves = reinterpret_cast<int*>(ws);
  a.src = reinterpret_cast<int*>(ws + 256);
  a.dst = reinterpret_cast<int*>(ws + 256 + words(a.t.num_pages / 2 + 1));
  const bool small = a.t.num_pages <= kSmallPool;
  cudaError_t e = launch_counting(small ? page_compact_kernel<1> : page_compact_kernel<kCluster>, small ? 1 : kCluster, 0, stream, a);
  if (e != cudaSuccess) return e;
  const long long n = static_cast<long long>(a.t.rows) * a.t.width, blocks = (n + 255) / 256, most = 4LL * sm_count();
  e = launch_pdl(page_rename_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  PageCopyLaunch c{};
  c.src = a.src;
  c.dst = a.dst;
  c.n = a.t.num_pages / 2 > 0 ? a.t.num_pages / 2 : 1;
  c.count = a.moves;
  c.status = a.status;
  c.wait_limit = kWaitLimitCycles;
  return launch_page_copy(c, caches, layers, stream);
}

}  // namespace fa
