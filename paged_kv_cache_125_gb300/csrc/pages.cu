// kv_pages_fork / kv_pages_extend / kv_pages_compact: the pages of a cache
// handled on the device.
//
// The pool is described by three int32 arrays: block_tables [rows,
// max_blocks], context_lens [rows] (a row's first ceil(len / block_size)
// entries are its pages) and ref_counts [num_blocks] (holders of each page; 0
// = free).  Each operator is two launches: a plan kernel that computes the new
// arrays and the list of page copies, and a copy kernel (its programmatic
// dependent) that moves the pages in every plane of the cache.
//
// The plan kernel is one thread-block cluster: its phases depend on one
// another through a few integers per page (counts, the ranks of free pages),
// so they are separated by cluster barriers inside one launch, and the CTAs
// exchange partial counts through the workspace.  Every choice is made by
// rank (lowest page first, rows in order) and integer atomics only add or
// take minima, so results do not depend on the order of execution.
//
// The plans are chains of dependent look-ups, bound by latency: a beam step of
// 256 rows 13 us, a token for each of 512 rows over 150,000 pages 25 us, the
// plan of a compaction 7 us.  The copies are bound by HBM (see below).
#include "kvp_device.cuh"
#include "pages.h"

namespace kvp {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kIntMax = 0x7fffffff;
constexpr int kMaxTeam = 8;  // CTAs of a plan cluster (the portable limit)

// The CTAs of the plan kernel's cluster.
struct Team {
  int rank, size;
  __device__ Team() {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  }
  // Barrier over every thread of the team; orders their global memory accesses.
  __device__ void sync() const {
    __threadfence();
    asm volatile(
        "barrier.cluster.arrive.release;\n\t"
        "barrier.cluster.wait.acquire;" ::
            : "memory");
  }
  __device__ int64_t thread() const { return (int64_t)rank * kPlanThreads + threadIdx.x; }
  __device__ int64_t threads() const { return (int64_t)size * kPlanThreads; }
};

__device__ __forceinline__ int ld_cg(const int* p) { return __ldcg(p); }

// How the team's threads walk table rows: 1 .. 32 lanes of a warp per row, as
// many as the row has entries for.
struct RowWalk {
  int lanes, lane, first, step;
  __device__ RowWalk(int max_blocks, int rank, int size) {
    lanes = 32;
    while (lanes > 1 && lanes / 2 >= max_blocks) lanes /= 2;
    lane = threadIdx.x & (lanes - 1);
    const int per_cta = kPlanThreads / lanes;
    first = rank + (int)threadIdx.x / lanes * size;
    step = per_cta * size;
  }
};

// Exclusive prefix sum of v over the block's threads; *total = the sum.
// `warp_sums` holds kPlanThreads / 32 sums.
template <typename T>
__device__ T block_scan(T v, long long* warp_sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = (long long)incl;
  __syncthreads();
  const T s = (T)warp_sums[lane];  // kPlanThreads / 32 == 32 sums
  T ws = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) ws += y;
  }
  *total = __shfl_sync(0xffffffffu, ws, 31);
  const T before = __shfl_sync(0xffffffffu, ws - s, warp);
  return before + incl - v;
}
static_assert(kPlanThreads == 1024, "block_scan needs 32 warps");

__device__ __forceinline__ int row_pages(int len, int block_size) {
  return (int)(((unsigned)len + (unsigned)block_size - 1u) / (unsigned)block_size);
}

// context_lens[r] if it fits its table row, else 0 (recorded): such a row has
// no pages that could be trusted.
__device__ __forceinline__ int row_len(const PagesArgs& a, int r) {
  const int c = a.context_lens[r];
  if (c < 0 || c > (int64_t)a.max_blocks * a.block_size) {
    record_error(a.status, KVP_ERR_DEVICE_DATA);
    return 0;
  }
  return c;
}

// This CTA's segment of the pages.  A thread looks at four consecutive pages
// at a time (segments start at multiples of four).
struct Segment {
  int64_t begin, end;
  int64_t base, total;  // counted pages before the segment / in the pool
};
constexpr int kPagesPerThread = 4;
constexpr int kPagesPerRound = kPlanThreads * kPagesPerThread;

__device__ __forceinline__ Segment segment_of(const PagesArgs& a, const Team& t) {
  Segment s;
  const int64_t per = ((a.num_blocks + t.size - 1) / t.size + 3) / 4 * 4;
  s.begin = min(per * t.rank, a.num_blocks);
  s.end = min(s.begin + per, a.num_blocks);
  s.base = s.total = 0;
  return s;
}

// Entries p .. p + 3 of an array of the pages (those past the end read as
// `past`); one load where the array allows it.
__device__ __forceinline__ int4 load_pages(const int* v, int64_t p, int64_t end, int past) {
  if (p + 4 <= end && (reinterpret_cast<uintptr_t>(v) & 15u) == 0)
    return __ldcg(reinterpret_cast<const int4*>(v + p));
  int4 r;
  r.x = p < end ? __ldcg(v + p) : past;
  r.y = p + 1 < end ? __ldcg(v + p + 1) : past;
  r.z = p + 2 < end ? __ldcg(v + p + 2) : past;
  r.w = p + 3 < end ? __ldcg(v + p + 3) : past;
  return r;
}
__device__ __forceinline__ void store_pages(int* v, int64_t p, int64_t end, const int4& x) {
  if (p + 4 <= end && (reinterpret_cast<uintptr_t>(v) & 15u) == 0) {
    *reinterpret_cast<int4*>(v + p) = x;
    return;
  }
  if (p < end) v[p] = x.x;
  if (p + 1 < end) v[p + 1] = x.y;
  if (p + 2 < end) v[p + 2] = x.z;
  if (p + 3 < end) v[p + 3] = x.w;
}

// Publishes this CTA's count and sums those of the CTAs before it (a team
// barrier).
__device__ void rank_segment(const PagesArgs& a, const Team& t, long long* warp_sums, int mine,
                             Segment* s) {
  int total;
  block_scan(mine, warp_sums, &total);
  if (threadIdx.x == 0) a.ws.team_counts[t.rank] = total;
  t.sync();
  s->base = s->total = 0;
  for (int i = 0; i < t.size; ++i) {
    const int c = ld_cg(&a.ws.team_counts[i]);
    if (i < t.rank) s->base += c;
    s->total += c;
  }
}

__device__ __forceinline__ int zeros(const int4& x) {
  return (x.x == 0) + (x.y == 0) + (x.z == 0) + (x.w == 0);
}

// Calls use(page, rank) for the free pages (counts[p] == 0) of the segment in
// order, with their ranks among the pool's; stops after rank limit - 1.
template <typename Use>
__device__ void for_free_pages(const int* counts, const Segment& s, int64_t limit,
                               long long* warp_sums, Use use) {
  int64_t base = s.base;
  for (int64_t p0 = s.begin; p0 < s.end && base < limit; p0 += kPagesPerRound) {
    const int64_t p = p0 + threadIdx.x * kPagesPerThread;
    const int4 c = p < s.end ? load_pages(counts, p, s.end, 1) : make_int4(1, 1, 1, 1);
    int total;
    int64_t k = base + block_scan(zeros(c), warp_sums, &total);
    const int v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v[i] == 0) {
        if (k < limit) use(p + i, k);
        ++k;
      }
    base += total;
  }
}

// ------------------------------------------------------------------ fork

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[32];
  const Team t;
  const int bs = a.block_size;
  const int64_t mb = a.max_blocks;
  const RowWalk rows(a.max_blocks, t.rank, t.size);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Segment s = segment_of(a, t);
  for (int64_t p = s.begin + threadIdx.x * kPagesPerThread; p < s.end; p += kPagesPerRound) {
    store_pages(a.out_counts, p, s.end, load_pages(a.ref_counts, p, s.end, 0));
    // ws.page: the lowest new row whose unfilled last page this is
    store_pages(a.ws.page, p, s.end, make_int4(kIntMax, kIntMax, kIntMax, kIntMax));
  }
  t.sync();

  // Every old row lets go of its pages; every new row takes its parent's,
  // except an unfilled last page, which goes to one new row (below).
  for (int r = rows.first; r < a.num_rows; r += rows.step) {
    const int n = row_pages(row_len(a, r), bs);
    for (int j = rows.lane; j < n; j += rows.lanes) {
      const int e = a.block_tables[r * mb + j];
      if (e < 0 || e >= a.num_blocks)
        record_error(a.status, KVP_ERR_DEVICE_DATA);
      else
        atomicAdd(&a.out_counts[e], -1);
    }
  }
  for (int r = rows.first; r < a.num_out; r += rows.step) {
    int p = a.parents[r];
    if (p < -1 || p >= a.num_rows) {
      record_error(a.status, KVP_ERR_DEVICE_DATA);
      p = -1;
    }
    const int len = p >= 0 ? row_len(a, p) : 0;
    const int n = row_pages(len, bs);
    if (rows.lane == 0) a.out_lens[r] = len;
    for (int j = rows.lane; j < a.max_blocks; j += rows.lanes) {
      int e = j < n ? a.block_tables[p * mb + j] : -1;
      if (e >= a.num_blocks || e < 0) e = -1;  // recorded above, with the parent's row
      a.out_tables[r * mb + j] = e;
      if (e < 0) continue;
      if (j == n - 1 && len % bs)
        atomicMin(&a.ws.page[e], r);
      else
        atomicAdd(&a.out_counts[e], 1);
    }
  }
  t.sync();

  // The lowest new row on an unfilled page keeps it; the others, in row
  // order, get copies.
  if (t.rank == 0) {
    int copies = 0;
    for (int r0 = 0; r0 < a.num_out; r0 += kPlanThreads) {
      const int r = r0 + (int)threadIdx.x;
      bool copy = false;
      if (r < a.num_out) {
        const int len = ld_cg(&a.out_lens[r]);
        if (len % bs) {
          const int e = ld_cg(&a.out_tables[r * mb + row_pages(len, bs) - 1]);
          if (e >= 0) {
            copy = ld_cg(&a.ws.page[e]) != r;
            if (!copy) atomicAdd(&a.out_counts[e], 1);
          }
        }
      }
      int total;
      const int k = copies + block_scan(copy ? 1 : 0, warp_sums, &total);
      if (copy) a.ws.row[k] = r;
      copies += total;
    }
    if (threadIdx.x == 0) a.ws.head->copies = copies;
  }
  t.sync();
  const int copies = ld_cg(&a.ws.head->copies);
  int mine = 0;
  for (int64_t p = s.begin + threadIdx.x * kPagesPerThread; p < s.end; p += kPagesPerRound)
    mine += zeros(load_pages(a.out_counts, p, s.end, 1));
  rank_segment(a, t, warp_sums, mine, &s);
  for_free_pages(a.out_counts, s, copies, warp_sums, [&](int64_t p, int64_t k) {
    const int r = ld_cg(&a.ws.row[k]);
    const int len = ld_cg(&a.out_lens[r]);
    int* entry = &a.out_tables[r * mb + row_pages(len, bs) - 1];
    a.ws.pairs[k] = PagePair{ld_cg(entry), (int)p, len % bs, 0};
    *entry = (int)p;
    a.out_counts[p] = 1;
  });
  if (s.total >= copies) return;
  // The pool ran out: rows past the last free page are dropped.
  t.sync();
  if (t.rank) return;
  record_error(a.status, KVP_ERR_DEVICE_DATA);
  if (threadIdx.x == 0) a.ws.head->copies = (int)s.total;
  for (int64_t k = s.total; k < copies; ++k) {
    const int r = ld_cg(&a.ws.row[k]);
    const int n = row_pages(ld_cg(&a.out_lens[r]), bs);
    for (int j = threadIdx.x; j < n; j += kPlanThreads) {
      const int e = ld_cg(&a.out_tables[r * mb + j]);
      if (j < n - 1 && e >= 0) atomicAdd(&a.out_counts[e], -1);
      a.out_tables[r * mb + j] = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.out_lens[r] = 0;
    __syncthreads();
  }
}

// ---------------------------------------------------------------- extend

// Last index i with v[i] <= x of the non-decreasing v[0 .. n), v[0] <= x.
__device__ __forceinline__ int last_at_most(const int* v, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)v[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

constexpr int kRowsInSmem = 2048;

__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[32];
  __shared__ int s_page0[kRowsInSmem], s_token0[kRowsInSmem];
  const Team t;
  const int bs = a.block_size;
  const int64_t mb = a.max_blocks;

  // The rows, by CTA 0: pages needed and new tokens, and their prefix sums.
  if (t.rank == 0) {
    long long pages = 0, tokens = 0;
    for (int r0 = 0; r0 < a.num_rows; r0 += kPlanThreads) {
      const int r = r0 + (int)threadIdx.x;
      long long need = 0, asked = 0;
      int add = 0, len = 0;
      bool bad = false;
      if (r < a.num_rows) {
        add = a.new_tokens[r];
        len = row_len(a, r);
        bad = len != a.context_lens[r];
        if (add < 0 || (int64_t)len + add > mb * bs) {  // does not fit the row: takes no slots
          bad = true;
          add = 0;
        }
        asked = add;
        if (!bad && add > 0 && len % bs) {  // the new tokens start in the last page: no one else's
          const int e = a.block_tables[r * mb + row_pages(len, bs) - 1];
          bad = e < 0 || e >= a.num_blocks || a.ref_counts[e] > 1;
        }
        if (bad) {
          record_error(a.status, KVP_ERR_DEVICE_DATA);
          add = 0;
        }
        need = row_pages(len + add, bs) - row_pages(len, bs);
      }
      long long total;
      const long long page0 = pages + block_scan(need, warp_sums, &total);
      pages += total;
      const long long token0 = tokens + block_scan(asked, warp_sums, &total);
      tokens += total;
      if (r < a.num_rows)
        a.ws.grow[r] = RowGrowth{(int)min(page0, (long long)kIntMax),
                                 (int)min(token0, (long long)kIntMax), len, add};
    }
    if (threadIdx.x == 0) {
      a.ws.head->copies = (int)min(pages, (long long)kIntMax);
      a.ws.head->tokens = (int)min(tokens, (long long)kIntMax);
      if (tokens > a.num_slots) record_error(a.status, KVP_ERR_DEVICE_DATA);
    }
  }
  // Meanwhile the others: the tables as they were (new pages follow below).
  const int copiers = t.size > 1 ? t.size - 1 : 1, me = t.size > 1 ? t.rank - 1 : 0;
  if (me >= 0) {
    const RowWalk rows(a.max_blocks, me, copiers);
    const bool in_place = a.out_tables == a.block_tables;
    for (int r = rows.first; r < a.num_rows; r += rows.step) {
      const int had = row_pages(row_len(a, r), bs);
      const int32_t* from = a.block_tables + r * mb;
      int32_t* to = a.out_tables + r * mb;
      int j = rows.lane;
      if (in_place) j += had / rows.lanes * rows.lanes;
#pragma unroll 4
      for (; j < a.max_blocks; j += rows.lanes)
        if (j >= had)
          to[j] = -1;
        else if (!in_place)
          to[j] = from[j];
    }
  }
  // The counts as they were, and the free pages among them.
  Segment s = segment_of(a, t);
  int mine = 0;
  for (int64_t p = s.begin + threadIdx.x * kPagesPerThread; p < s.end; p += kPagesPerRound) {
    const int4 c = load_pages(a.ref_counts, p, s.end, 1);
    mine += zeros(c);
    if (a.out_counts != a.ref_counts) store_pages(a.out_counts, p, s.end, c);
  }
  rank_segment(a, t, warp_sums, mine, &s);  // (a team barrier)

  // The rows' prefix sums, to search in: in shared memory, or (too many rows)
  // packed in the workspace, by every CTA for itself, all writing the same.
  const bool small = a.num_rows <= kRowsInSmem;
  int* page0 = small ? s_page0 : a.ws.row;
  int* token0 = small ? s_token0 : a.ws.row2;
  for (int r = threadIdx.x; r < a.num_rows; r += kPlanThreads) {
    const int2 g = __ldcg(reinterpret_cast<const int2*>(&a.ws.grow[r]));
    page0[r] = g.x;
    token0[r] = g.y;
  }
  __syncthreads();
  // Free page of rank k goes to the last row whose pages start at or before k.
  const int pages = ld_cg(&a.ws.head->copies);
  if (pages > 0) {
    for_free_pages(a.ref_counts, s, pages, warp_sums, [&](int64_t p, int64_t k) {
      const int r = last_at_most(page0, a.num_rows, k);
      const int4 g = __ldcg(reinterpret_cast<const int4*>(&a.ws.grow[r]));  // page0, token0, len, add
      const int had = row_pages(g.z, bs), need = row_pages(g.z + g.w, bs) - had;
      if (g.x + need > s.total) return;  // not enough pages left for the whole row
      a.out_tables[r * mb + had + (k - g.x)] = (int)p;
      a.out_counts[p] = 1;
    });
    t.sync();
  }

  // Whether the pool had the pages that a row needs.
  auto served = [&](const int4& g) {
    const int need = row_pages(g.z + g.w, bs) - row_pages(g.z, bs);
    return need == 0 || (int64_t)g.x + need <= s.total;
  };
  for (int64_t r = t.thread(); r < a.num_rows; r += t.threads()) {
    const int4 g = __ldcg(reinterpret_cast<const int4*>(&a.ws.grow[r]));
    if (!served(g)) record_error(a.status, KVP_ERR_DEVICE_DATA);
    a.out_lens[r] = served(g) ? g.z + g.w : g.z;
  }
  const int tokens = ld_cg(&a.ws.head->tokens);
  for (int64_t i = t.thread(); i < a.num_slots; i += t.threads()) {
    int slot = -1;
    if (i < tokens) {
      const int r = last_at_most(token0, a.num_rows, i);
      const int4 g = __ldcg(reinterpret_cast<const int4*>(&a.ws.grow[r]));
      const int pos = g.z + (int)(i - g.y);
      if (served(g) && pos < g.z + g.w)
        slot = ld_cg(&a.out_tables[r * mb + pos / bs]) * bs + pos % bs;
    }
    a.slot_mapping[i] = slot;
  }
}

// --------------------------------------------------------------- compact

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[32];
  const Team t;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Segment s = segment_of(a, t);
  auto live4 = [](const int4& c) { return (c.x > 0) + (c.y > 0) + (c.z > 0) + (c.w > 0); };
  int mine = 0;
  for (int64_t p = s.begin + threadIdx.x * kPagesPerThread; p < s.end; p += kPagesPerRound)
    mine += live4(load_pages(a.ref_counts, p, s.end, 0));
  rank_segment(a, t, warp_sums, mine, &s);
  const int64_t live = s.total;  // pages [0, live) hold everything afterwards

  // Live pages before each page; free page p < live is hole p - before(p).
  int64_t base = s.base;
  for (int64_t p0 = s.begin; p0 < s.end; p0 += kPagesPerRound) {
    const int64_t p = p0 + threadIdx.x * kPagesPerThread;
    const int4 c = p < s.end ? load_pages(a.ref_counts, p, s.end, 0) : make_int4(0, 0, 0, 0);
    int total;
    int before = (int)base + block_scan(live4(c), warp_sums, &total);
    base += total;
    const int v[4] = {c.x, c.y, c.z, c.w};
    int o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = before;
      if (v[i] > 0)
        ++before;
      else if (p + i < s.end && p + i < live)
        a.ws.page2[p + i - before] = (int)(p + i);
    }
    if (p < s.end) store_pages(a.ws.page, p, s.end, make_int4(o[0], o[1], o[2], o[3]));
  }
  t.sync();
  const int64_t staying = live < a.num_blocks ? ld_cg(&a.ws.page[live]) : live;
  if (t.thread() == 0) a.ws.head->copies = (int)(live - staying);
  for (int64_t p = t.thread(); p < a.num_blocks; p += t.threads()) {
    const int c = a.ref_counts[p];
    int place = -1;
    if (c > 0 && p >= live) {  // the k-th live page above moves into the k-th hole below
      const int64_t k = ld_cg(&a.ws.page[p]) - staying;
      place = ld_cg(&a.ws.page2[k]);
      a.ws.pairs[k] = PagePair{(int)p, place, a.block_size, 0};
      a.out_counts[place] = c;
    } else if (c > 0) {
      place = (int)p;
      a.out_counts[p] = c;
    }
    if (p >= live) a.out_counts[p] = 0;
    a.places[p] = place;
  }
  t.sync();
  const RowWalk rows(a.max_blocks, t.rank, t.size);
  for (int r = rows.first; r < a.num_rows; r += rows.step) {
    const int n = row_pages(row_len(a, r), a.block_size);
    for (int j = rows.lane; j < a.max_blocks; j += rows.lanes) {
      int e = -1;
      if (j < n) {
        const int old = a.block_tables[(int64_t)r * a.max_blocks + j];
        if (old >= 0 && old < a.num_blocks) e = ld_cg(&a.places[old]);
        if (e < 0) record_error(a.status, KVP_ERR_DEVICE_DATA);  // a row's page is outside or free
      }
      a.out_tables[(int64_t)r * a.max_blocks + j] = e;
    }
  }
}

// ------------------------------------------------------------------ copy
//
// Copies the first `tokens` rows of each listed page in every plane; the
// number of pairs is the plan kernel's.  Sources and destinations of one plan
// are disjoint, so the order of the copies does not matter.

// 16-byte path: one warp per SM streams 16 KiB chunks through a ring in shared
// memory (bulk copies in, bulk copies out), so that loads and stores are always
// under way together.  HBM-bound.  Half of the pages of 16 planes moved (4.3 GB
// read and written): 664 us with 64 KiB of loads in flight per SM, 6.47 TB/s;
// more of them cost (690 us with 128 KiB: reads and writes get in each other's
// way), fewer starve (880 us with 32 KiB).  Eight blocks of 256 threads with
// eight 16-byte loads each took 715 us.
constexpr uint32_t kChunkBytes = 16384;
constexpr int kRing = 8;            // chunks in shared memory
constexpr int kStoresInFlight = 4;  // of them being written out
constexpr uint32_t kRingBytes = kRing * kChunkBytes + kRing * 8;

// x / y; nearly always both fit 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

__global__ void __launch_bounds__(32) stream_pages_kernel(uint8_t* __restrict__ cache, int64_t num_planes,
                                                          int64_t plane_bytes, int64_t block_bytes,
                                                          int64_t row_bytes, int64_t chunks_per_block,
                                                          const PagesHead* head, const PagePair* pairs,
                                                          int* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing * kChunkBytes);
  const int lane = threadIdx.x;
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("fence.proxy.async.global;" ::: "memory");
  const int64_t per_pair = num_planes * chunks_per_block;
  const int64_t items = ld_cg(&head->copies) * per_pair;
  // An item is a chunk of one page of one plane.  The lanes look up 32 items
  // of this CTA at a time (those past a page's filled rows drop out).
  int64_t next = blockIdx.x;
  unsigned ready = 0;
  uint8_t *src = nullptr, *dst = nullptr;
  uint32_t bytes = 0;
  auto look_up = [&]() {
    while (!ready && next < items) {
      const int64_t w = next + (int64_t)lane * gridDim.x;
      next += 32 * (int64_t)gridDim.x;
      bytes = 0;
      if (w < items) {
        const int64_t pair = quotient(w, per_pair), rest = w - pair * per_pair;
        const int64_t plane = quotient(rest, chunks_per_block), chunk = rest - plane * chunks_per_block;
        const int4 pr = __ldcg(reinterpret_cast<const int4*>(pairs + pair));
        const int64_t at = chunk * kChunkBytes, size = pr.z * row_bytes;
        uint8_t* base = cache + plane * plane_bytes + at;
        src = base + pr.x * block_bytes;
        dst = base + pr.y * block_bytes;
        bytes = at >= size ? 0u : (uint32_t)min(size - at, (int64_t)kChunkBytes);
      }
      ready = __ballot_sync(0xffffffffu, bytes > 0);
    }
    return ready != 0;
  };
  uint8_t* out[kRing];  // of the chunk in each slot
  uint32_t out_bytes[kRing];
  uint32_t loads = 0, stores = 0;
  auto load = [&]() {
    if (!look_up()) return false;
    const int i = __ffs(ready) - 1;
    ready &= ready - 1;
    const uint32_t slot = loads++ % kRing;
    const uint32_t n = __shfl_sync(0xffffffffu, bytes, i);
    const uint8_t* from = reinterpret_cast<const uint8_t*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), i));
    out[slot] = reinterpret_cast<uint8_t*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), i));
    out_bytes[slot] = n;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[slot], n);
      bulk_g2s(smem + slot * kChunkBytes, from, n, &full[slot]);
    }
    return true;
  };
  bool more = true, ok = true;
  while (more && loads < kRing - kStoresInFlight) more = load();
  for (; stores < loads; ++stores) {
    const uint32_t slot = stores % kRing;
    ok = mbar_wait(&full[slot], (stores / kRing) & 1, status);
    if (!ok) break;
    if (lane == 0) {
      bulk_s2g(out[slot], smem + slot * kChunkBytes, out_bytes[slot]);
      bulk_commit();
      bulk_wait_read<kStoresInFlight - 1>();  // of these, the oldest leaves its slot to the next load
    }
    __syncwarp();
    if (more) more = load();
  }
  // After an expired wait: no copy of this CTA is in flight when it exits.
  for (; !ok && stores < loads; ++stores) mbar_wait(&full[stores % kRing], (stores / kRing) & 1, status);
  if (lane == 0) bulk_wait_all();
}

// Any alignment: element by element.
constexpr int kCopyThreads = 256;
constexpr int64_t kChunkElems = 16384;

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(
    uint16_t* __restrict__ cache, int64_t num_planes, int64_t plane_stride, int64_t block_elems,
    int64_t row_elems, int64_t chunks_per_block, const PagesHead* head, const PagePair* pairs) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t items = (int64_t)ld_cg(&head->copies) * num_planes * chunks_per_block;
  for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
    const int64_t chunk = w % chunks_per_block;
    const int64_t pp = w / chunks_per_block;
    const int4 pr = __ldcg(reinterpret_cast<const int4*>(pairs + pp / num_planes));
    uint16_t* base = cache + pp % num_planes * plane_stride;
    const uint16_t* src = base + (int64_t)pr.x * block_elems;
    uint16_t* dst = base + (int64_t)pr.y * block_elems;
    const int64_t e0 = chunk * kChunkElems, e1 = min(e0 + kChunkElems, pr.z * row_elems);
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kCopyThreads) dst[e] = src[e];
  }
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, int threads, size_t smem, int cluster, bool pdl,
                   cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs of the plan: enough to see its largest array in one round.
int team_size(const PagesArgs& a) {
  const int64_t rows = a.num_rows > a.num_out ? a.num_rows : a.num_out;
  int64_t n = rows * a.max_blocks;
  if (a.num_blocks > n) n = a.num_blocks;
  if (a.num_slots > n) n = a.num_slots;
  int size = 1;
  while (size < kMaxTeam && (int64_t)size * kPlanThreads < n) size *= 2;
  return size;
}

cudaError_t launch_copies(const PagesArgs& a, const PagesCache& c, int num_sms, cudaStream_t stream) {
  const int64_t block_elems = (int64_t)a.block_size * c.row_elems;
  const bool vec = (reinterpret_cast<uintptr_t>(c.cache) & 15u) == 0 && c.plane_stride % 8 == 0 &&
                   c.row_elems % 8 == 0;
  const PagesHead* head = a.ws.head;
  const PagePair* pairs = a.ws.pairs;
  if (!vec)
    return launch(copy_pages_kernel, num_sms * 8, kCopyThreads, 0, 0, true, stream, c.cache, c.num_planes,
                  c.plane_stride, block_elems, c.row_elems, (block_elems + kChunkElems - 1) / kChunkElems,
                  head, pairs);
  cudaError_t e = cudaFuncSetAttribute(stream_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kRingBytes);
  if (e != cudaSuccess) return e;
  return launch(stream_pages_kernel, num_sms, 32, kRingBytes, 0, true, stream,
                reinterpret_cast<uint8_t*>(c.cache), c.num_planes, c.plane_stride * 2, block_elems * 2,
                c.row_elems * 2, (block_elems * 2 + kChunkBytes - 1) / kChunkBytes, head, pairs, a.status);
}

}  // namespace

size_t pages_workspace_bytes(int64_t num_blocks, int64_t rows) {
  const int64_t pairs = num_blocks > rows ? num_blocks : rows;
  const int64_t pages = (num_blocks + 3) / 4 * 4;
  return 256 + (size_t)pairs * sizeof(PagePair) + (size_t)rows * (sizeof(RowGrowth) + 2 * sizeof(int)) +
         (size_t)(2 * pages) * sizeof(int);
}

PagesWorkspace pages_workspace(void* base, int64_t num_blocks, int64_t rows) {
  PagesWorkspace w;
  uint8_t* p = static_cast<uint8_t*>(base);
  const int64_t pairs = num_blocks > rows ? num_blocks : rows;
  const int64_t pages = (num_blocks + 3) / 4 * 4;
  w.head = reinterpret_cast<PagesHead*>(p);
  w.team_counts = reinterpret_cast<int*>(p + 64);
  w.pairs = reinterpret_cast<PagePair*>(p + 256);
  w.grow = reinterpret_cast<RowGrowth*>(w.pairs + pairs);
  w.page = reinterpret_cast<int*>(w.grow + rows);
  w.page2 = w.page + pages;
  w.row = w.page2 + pages;
  w.row2 = w.row + rows;
  return w;
}

cudaError_t launch_pages_fork(const PagesArgs& a, const PagesCache& c, int num_sms,
                              cudaStream_t stream) {
  const int size = team_size(a);
  cudaError_t e = launch(fork_plan_kernel, size, kPlanThreads, 0, size, false, stream, a);
  return e != cudaSuccess ? e : launch_copies(a, c, num_sms, stream);
}

cudaError_t launch_pages_extend(const PagesArgs& a, cudaStream_t stream) {
  const int size = team_size(a);
  return launch(extend_plan_kernel, size, kPlanThreads, 0, size, false, stream, a);
}

cudaError_t launch_pages_compact(const PagesArgs& a, const PagesCache& c, int num_sms,
                                 cudaStream_t stream) {
  const int size = team_size(a);
  cudaError_t e = launch(compact_plan_kernel, size, kPlanThreads, 0, size, false, stream, a);
  return e != cudaSuccess ? e : launch_copies(a, c, num_sms, stream);
}

}  // namespace kvp
