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
// 256 rows 12 us, a token for each of 512 rows over 150,000 pages 12 us (25 with
// a barrier pair and a load per round of 4096 pages, and the team keeping the
// table rows), the plan of a compaction of 1024 pages 9 us, of a few rows or
// pages 6 to 9.  The copies are bound by HBM (see below).
#include "kvp_device.cuh"
#include "pages.h"

namespace kvp {
namespace {

constexpr int kPlanThreads = 1024;  // of a plan CTA, at most
constexpr int kFewThreads = 256;    // where there is little to do (kRounds warps at least)
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
    asm volatile(
        "barrier.cluster.arrive.release;\n\t"
        "barrier.cluster.wait.acquire;" ::
            : "memory");
  }
  __device__ int64_t thread() const { return (int64_t)rank * blockDim.x + threadIdx.x; }
  __device__ int64_t threads() const { return (int64_t)size * blockDim.x; }
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
    const int per_cta = (int)blockDim.x / lanes;
    first = rank + (int)threadIdx.x / lanes * size;
    step = per_cta * size;
  }
};

// Exclusive prefix sums of N values at once over the block's threads; total[i] =
// the sum of v[i].  `sums` holds the warps' sums.
template <typename T, int N>
__device__ __forceinline__ void block_scan(T (&v)[N], T (&total)[N], long long (*sums)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    incl[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, incl[i], o);
      if (lane >= o) incl[i] += y;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 31) sums[i][warp] = (long long)incl[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const T s = lane < (int)blockDim.x / 32 ? (T)sums[i][lane] : T(0);
    T ws = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, ws, o);
      if (lane >= o) ws += y;
    }
    total[i] = __shfl_sync(0xffffffffu, ws, 31);
    v[i] = __shfl_sync(0xffffffffu, ws - s, warp) + incl[i] - v[i];
  }
}
static_assert(kPlanThreads <= 1024, "block_scan takes 32 warps");

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

// The pages of a kind (free, in use) are numbered from the lowest on.  Each CTA
// of the team has a segment of the pool, which it takes in spans of 8 rounds; in
// a round a thread looks at four consecutive pages (segments start at multiples
// of four).  The marks of a whole span are kept in registers, four bits a round,
// and ranked by one scan over packed byte counts, so that a pool of 260,000 pages
// is read once and ranked with three barriers in each CTA.
struct Segment {
  int64_t begin, end;
  int64_t base, total;  // marked pages before the segment / in the pool
};
constexpr int kRounds = 8;
static_assert(kFewThreads / 32 >= kRounds, "a warp ranks the marks of a round");
__device__ __forceinline__ int pages_per_round() { return (int)blockDim.x * 4; }
__device__ __forceinline__ int pages_per_span() { return (int)blockDim.x * 4 * kRounds; }

__device__ __forceinline__ Segment segment_of(const PagesArgs& a, const Team& t) {
  Segment s;
  const int64_t per = ((a.num_blocks + t.size - 1) / t.size + 3) / 4 * 4;
  s.begin = min(per * t.rank, a.num_blocks);
  s.end = min(s.begin + per, a.num_blocks);
  s.base = s.total = 0;
  return s;
}

__device__ __forceinline__ bool quads(const void* v) { return (reinterpret_cast<uintptr_t>(v) & 15u) == 0; }

// Entries p .. p + 3 of an array of the pages (those past the end read as
// `past`); one load where the array allows it.
__device__ __forceinline__ int4 load_pages(const int* v, int64_t p, int64_t end, int past) {
  if (p + 4 <= end && quads(v)) return __ldcg(reinterpret_cast<const int4*>(v + p));
  int4 r;
  r.x = p < end ? __ldcg(v + p) : past;
  r.y = p + 1 < end ? __ldcg(v + p + 1) : past;
  r.z = p + 2 < end ? __ldcg(v + p + 2) : past;
  r.w = p + 3 < end ? __ldcg(v + p + 3) : past;
  return r;
}
__device__ __forceinline__ void store_pages(int* v, int64_t p, int64_t end, const int4& x) {
  if (p + 4 <= end && quads(v)) {
    *reinterpret_cast<int4*>(v + p) = x;
    return;
  }
  if (p < end) v[p] = x.x;
  if (p + 1 < end) v[p + 1] = x.y;
  if (p + 2 < end) v[p + 2] = x.z;
  if (p + 3 < end) v[p + 3] = x.w;
}

// The page of entry 0 that a thread looks at in round i of a span.
__device__ __forceinline__ int64_t page_of(int64_t p0, int i) {
  return p0 + i * pages_per_round() + (int)threadIdx.x * 4;
}

// Rounds of the span at p0.
__device__ __forceinline__ int rounds_of(int64_t p0, int64_t end) {
  return (int)(((int)min(end - p0, (int64_t)pages_per_span()) + pages_per_round() - 1) / (unsigned)pages_per_round());
}

struct RankScratch {
  uint2 warp[32];           // marks of each warp: a byte per even / odd round
  int before[kRounds][32];  // marks of a round in the warps before
  int round[kRounds];       // marks of a round
};

struct Marks {
  unsigned bits;       // four a round
  unsigned even, odd;  // marks of the lanes before, a byte per even / odd round
};

__device__ __forceinline__ int span_total(const RankScratch& s) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) n += s.round[i];
  return n;
}

// Marks the pages p of the span at p0 with flag(v[p]) (false for `past`) and
// ranks them; copies v to `copy` (null: does not).
template <typename Flag>
__device__ __forceinline__ Marks mark_span(const int* v, int64_t p0, int64_t end, int past, RankScratch& s,
                                           Flag flag, int* copy = nullptr) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rounds = rounds_of(p0, end);
  Marks m{0, 0, 0};
  auto take = [&](const int4& c, int i) {
    const unsigned b = (unsigned)flag(c.x) | (unsigned)flag(c.y) << 1 | (unsigned)flag(c.z) << 2 |
                       (unsigned)flag(c.w) << 3;
    m.bits |= b << (4 * i);
    if (copy && page_of(p0, i) < end) store_pages(copy, page_of(p0, i), end, c);
  };
  if (quads(v) && end % 4 == 0) {
#pragma unroll 1
    for (int i0 = 0; i0 < rounds; i0 += 4) {
      int4 c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t p = page_of(p0, i0 + i);
        c[i] = p < end ? __ldcg(reinterpret_cast<const int4*>(v + p)) : make_int4(past, past, past, past);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) take(c[i], i0 + i);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) take(load_pages(v, page_of(p0, i), end, past), i);
  }
  unsigned n = m.bits - (m.bits >> 1 & 0x55555555u);
  n = (n & 0x33333333u) + (n >> 2 & 0x33333333u);  // marks of each round, 4 bits
  const unsigned even = n & 0x0f0f0f0fu, odd = n >> 4 & 0x0f0f0f0fu;
  m.even = even, m.odd = odd;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {  // (a warp has at most 128 marks a round)
    const unsigned e = __shfl_up_sync(0xffffffffu, m.even, o), d = __shfl_up_sync(0xffffffffu, m.odd, o);
    if (lane >= o) m.even += e, m.odd += d;
  }
  __syncthreads();  // the span before has been used
  if (lane == 31) s.warp[warp] = make_uint2(m.even, m.odd);
  m.even -= even, m.odd -= odd;
  __syncthreads();
  if (warp < kRounds) {
    const uint2 w = lane < (int)blockDim.x / 32 ? s.warp[lane] : make_uint2(0, 0);
    const int mine = ((warp & 1 ? w.y : w.x) >> (warp / 2 * 8)) & 255;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    s.before[warp][lane] = incl - mine;
    if (lane == 31) s.round[warp] = incl;
  }
  __syncthreads();
  return m;
}

// Marked pages of round i before this thread's four.
__device__ __forceinline__ int rank_in_round(const Marks& m, const RankScratch& s, int i) {
  return s.before[i][threadIdx.x >> 5] + (((i & 1 ? m.odd : m.even) >> (i / 2 * 8)) & 255);
}

// Marks the team's pages: their number in the pool and before each segment, and
// the marks of this CTA's span (of the last one, if there are several).  (A
// team barrier.)
template <typename Flag>
__device__ __forceinline__ Marks mark_segment(const PagesArgs& a, const Team& t, const int* v, int past,
                                              RankScratch& scratch, Segment* s, Flag flag,
                                              int* copy = nullptr) {
  Marks m{0, 0, 0};
  int mine = 0;
  for (int64_t p0 = s->begin; p0 < s->end; p0 += pages_per_span()) {
    m = mark_span(v, p0, s->end, past, scratch, flag, copy);
    mine += span_total(scratch);
  }
  if (threadIdx.x == 0) a.ws.team_counts[t.rank] = mine;
  t.sync();
  s->base = s->total = 0;
  for (int i = 0; i < t.size; ++i) {
    const int c = ld_cg(&a.ws.team_counts[i]);
    if (i < t.rank) s->base += c;
    s->total += c;
  }
  return m;
}

template <typename Flag>
__device__ __noinline__ Marks mark_again(const int* v, int64_t p0, int64_t end, int past, RankScratch& s,
                                         Flag flag) {
  return mark_span(v, p0, end, past, s, flag);
}

// Calls use(p0, m, rank) for each span of the segment, with its first page, its
// marks and the marked pages of the pool before it.  m: of mark_segment.
template <typename Flag, typename Use>
__device__ __forceinline__ void for_spans(const int* v, int past, RankScratch& scratch, const Segment& s,
                                          Marks m, int64_t limit, Flag flag, Use use) {
  int64_t rank = s.base;
  for (int64_t p0 = s.begin; p0 < s.end && rank < limit; p0 += pages_per_span()) {
    if (s.end - s.begin > pages_per_span()) m = mark_again(v, p0, s.end, past, scratch, flag);
    use(p0, m, rank);
    rank += span_total(scratch);
  }
}

__device__ __forceinline__ bool is_free(int count) { return count == 0; }

// Calls use(page, four, rank) for the free pages of the segment with ranks <
// limit, four at a time: free page number rank is page + i of the lowest bit i of
// `four`, and so on.
template <typename Use>
__device__ __forceinline__ void for_free_pages(const int* counts, RankScratch& scratch, const Segment& s,
                                               const Marks& marks, int64_t limit, Use use) {
  for_spans(counts, 1, scratch, s, marks, limit, is_free, [&](int64_t p0, const Marks& m, int64_t rank) {
#pragma unroll 1
    for (int i = 0; i < rounds_of(p0, s.end) && rank < limit; ++i) {
      const int64_t k = rank + rank_in_round(m, scratch, i);
      unsigned four = m.bits >> (4 * i) & 15u;
      while (four && k + __popc(four) > limit) four &= 0x7fffffffu >> __clz(four);  // without its highest
      if (four) use(page_of(p0, i), four, k);
      rank += scratch.round[i];
    }
  });
}

// A plan is launched in the shadow of the kernel before it on the stream, and
// lets the copies, which wait for it, get ready.
__device__ __forceinline__ void plan_begins() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ fork

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[1][32];
  __shared__ RankScratch scratch;
  const Team t;
  const int bs = a.block_size;
  const int64_t mb = a.max_blocks;
  const RowWalk rows(a.max_blocks, t.rank, t.size);
  plan_begins();

  Segment s = segment_of(a, t);
#pragma unroll 4
  for (int64_t p = s.begin + threadIdx.x * 4; p < s.end; p += pages_per_round()) {
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
      // (one of the rows on an unfilled page is its holder, whichever it is)
      if (j != n - 1 || len % bs == 0 || atomicMin(&a.ws.page[e], r) == kIntMax)
        atomicAdd(&a.out_counts[e], 1);
    }
  }
  t.sync();

  // The lowest new row on an unfilled page keeps it; the others, in row order,
  // get copies.  Copy k is noted as {page, its place in the row, tokens, row}.
  if (t.rank == 0) {
    int copies = 0;
    for (int r0 = 0; r0 < a.num_out; r0 += blockDim.x) {
      const int r = r0 + (int)threadIdx.x;
      int len = 0, e = -1;
      if (r < a.num_out) {
        len = ld_cg(&a.out_lens[r]);
        if (len % bs) e = ld_cg(&a.out_tables[r * mb + row_pages(len, bs) - 1]);
      }
      const bool copy = e >= 0 && ld_cg(&a.ws.page[e]) != r;
      int k[1] = {copy ? 1 : 0}, total[1];
      block_scan(k, total, warp_sums);
      if (copy) a.ws.pairs[copies + k[0]] = PagePair{e, row_pages(len, bs) - 1, len % bs, r};
      copies += total[0];
    }
    if (threadIdx.x == 0) a.ws.head->copies = copies;
  }
  const Marks marks = mark_segment(a, t, a.out_counts, 1, scratch, &s, is_free);
  const int copies = ld_cg(&a.ws.head->copies);
  auto noted = [&](int64_t k) { return __ldcg(reinterpret_cast<const int4*>(&a.ws.pairs[k])); };
  for_free_pages(a.out_counts, scratch, s, marks, copies, [&](int64_t p0, unsigned four, int64_t k) {
    const int n = __popc(four);
    int4 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) c[i] = noted(k + i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) {
        const int p = (int)p0 + __ffs(four) - 1;
        four &= four - 1;
        a.out_tables[c[i].w * mb + c[i].y] = p;
        a.out_counts[p] = 1;
        a.ws.pairs[k + i] = PagePair{c[i].x, p, c[i].z, 0};
      }
  });
  if (s.total >= copies) return;
  // The pool ran out: rows past the last free page are dropped.
  t.sync();
  if (t.rank) return;
  record_error(a.status, KVP_ERR_DEVICE_DATA);
  if (threadIdx.x == 0) a.ws.head->copies = (int)s.total;
  for (int64_t k = s.total; k < copies; ++k) {
    const int4 c = noted(k);
    for (int j = threadIdx.x; j <= c.y; j += blockDim.x) {
      const int e = ld_cg(&a.out_tables[c.w * mb + j]);
      if (j < c.y && e >= 0) atomicAdd(&a.out_counts[e], -1);
      a.out_tables[c.w * mb + j] = -1;
    }
    if (threadIdx.x == 0) a.out_lens[c.w] = 0;
  }
}

// ---------------------------------------------------------------- extend

// Last row i with rows[i].*first <= x, of n >= 1 rows in which it never falls
// and starts at 0.
__device__ __forceinline__ int last_at_most(const RowGrowth* rows, int n, int RowGrowth::*first, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)(rows[mid].*first) <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

constexpr int kRowsInSmem = 2048;

// Pages that a row of length len asks for (0: its new length does not fit).
__device__ __forceinline__ int asked_pages(const PagesArgs& a, int r, int len) {
  const int add = a.new_tokens[r];
  if (add < 0 || (int64_t)len + add > (int64_t)a.max_blocks * a.block_size) return 0;
  return row_pages(len + add, a.block_size) - row_pages(len, a.block_size);
}

// The table rows as they were, by CTA `me` of `n`: all entries but those of the
// pages that a row asks for, which the team writes.
__device__ void keep_rows(const PagesArgs& a, int me, int n) {
  const int64_t mb = a.max_blocks;
  if (a.out_tables == a.block_tables) {
    const RowWalk rows(a.max_blocks, me, n);
    for (int r = rows.first; r < a.num_rows; r += rows.step) {
      const int len = row_len(a, r), from = row_pages(len, a.block_size) + asked_pages(a, r, len);
      for (int j = from + rows.lane; j < a.max_blocks; j += rows.lanes) a.out_tables[r * mb + j] = -1;
    }
    return;
  }
  const int64_t entries = a.num_rows * mb, step = (int64_t)n * blockDim.x;
#pragma unroll 4
  for (int64_t i = (int64_t)me * blockDim.x + threadIdx.x; i < entries; i += step) {
    const int r = (int)(entries <= kIntMax ? (unsigned)i / (unsigned)a.max_blocks : i / mb);
    const int j = (int)(i - r * mb);
    const int len = row_len(a, r), had = row_pages(len, a.block_size);
    if (j < had)
      a.out_tables[i] = a.block_tables[i];
    else if (j >= had + asked_pages(a, r, len))
      a.out_tables[i] = -1;
  }
}

// The first cluster is the team; CTAs behind it, if there are any, keep the
// table rows.  Nothing orders the two, so the team reads no entry that they write.
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[2][32];
  __shared__ RowGrowth s_grow[kRowsInSmem];
  __shared__ RankScratch scratch;
  const Team t;
  const int bs = a.block_size;
  const int64_t mb = a.max_blocks;
  plan_begins();
  const int keepers = (int)gridDim.x - t.size;
  if ((int)blockIdx.x >= t.size) {
    keep_rows(a, (int)blockIdx.x - t.size, keepers);
    return;
  }

  // The rows, by CTA 0: pages needed and new tokens, and their prefix sums.
  if (t.rank == 0) {
    long long pages = 0, tokens = 0;
    for (int r0 = 0; r0 < a.num_rows; r0 += blockDim.x) {
      const int r = r0 + (int)threadIdx.x;
      long long v[2] = {0, 0}, total[2];  // pages needed, tokens asked for
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
        v[1] = add;
        if (!bad && add > 0 && len % bs) {  // the new tokens start in the last page: no one else's
          const int e = a.block_tables[r * mb + row_pages(len, bs) - 1];
          bad = e < 0 || e >= a.num_blocks || a.ref_counts[e] > 1;
        }
        if (bad) {
          record_error(a.status, KVP_ERR_DEVICE_DATA);
          add = 0;
        }
        v[0] = row_pages(len + add, bs) - row_pages(len, bs);
      }
      block_scan(v, total, warp_sums);
      if (r < a.num_rows)
        a.ws.grow[r] = RowGrowth{(int)min(pages + v[0], (long long)kIntMax),
                                 (int)min(tokens + v[1], (long long)kIntMax), len, add};
      pages += total[0];
      tokens += total[1];
    }
    if (threadIdx.x == 0) {
      a.ws.head->copies = (int)min(pages, (long long)kIntMax);
      a.ws.head->tokens = (int)min(tokens, (long long)kIntMax);
      if (tokens > a.num_slots) record_error(a.status, KVP_ERR_DEVICE_DATA);
    }
  }
  // Meanwhile the others: the tables as they were.
  if (keepers == 0 && (t.rank > 0 || t.size == 1))
    keep_rows(a, t.size > 1 ? t.rank - 1 : 0, t.size > 1 ? t.size - 1 : 1);
  // The counts as they were, and the free pages among them.
  Segment s = segment_of(a, t);
  const Marks marks = mark_segment(a, t, a.ref_counts, 1, scratch, &s, is_free,
                                   a.out_counts != a.ref_counts ? a.out_counts : nullptr);

  // The rows, to search in: in shared memory unless there are too many.
  if (a.num_rows <= kRowsInSmem)
    for (int r = threadIdx.x; r < a.num_rows; r += blockDim.x)
      *reinterpret_cast<int4*>(&s_grow[r]) = __ldcg(reinterpret_cast<const int4*>(&a.ws.grow[r]));
  const RowGrowth* grow = a.num_rows <= kRowsInSmem ? s_grow : a.ws.grow;
  __syncthreads();
  // Whether the pool had the pages that a row needs.
  auto served = [&](const RowGrowth& g) {
    const int need = row_pages(g.len + g.add, bs) - row_pages(g.len, bs);
    return need == 0 || (int64_t)g.page0 + need <= s.total;
  };
  // Free page of rank k goes to the last row whose pages start at or before k.
  const int pages = ld_cg(&a.ws.head->copies), tokens = ld_cg(&a.ws.head->tokens);
  if (pages > 0) {
    for_free_pages(a.ref_counts, scratch, s, marks, pages, [&](int64_t p0, unsigned four, int64_t k) {
      for (; four; four &= four - 1, ++k) {
        const int r = last_at_most(grow, a.num_rows, &RowGrowth::page0, k);
        const RowGrowth g = grow[r];
        if (!served(g)) return;  // not enough pages left for the whole row
        const int64_t p = p0 + __ffs(four) - 1;
        a.out_tables[r * mb + row_pages(g.len, bs) + (k - g.page0)] = (int)p;
        a.out_counts[p] = 1;
      }
    });
    t.sync();
  }

  for (int64_t r = t.thread(); r < a.num_rows; r += t.threads()) {
    const RowGrowth g = grow[r];
    const bool ok = served(g);
    if (!ok) record_error(a.status, KVP_ERR_DEVICE_DATA);
    a.out_lens[r] = ok ? g.len + g.add : g.len;
    if (!ok || g.add == 0) {  // entries that no page came for
      const int had = row_pages(g.len, bs), asked = asked_pages(a, (int)r, g.len);
      for (int j = had; j < had + asked; ++j) a.out_tables[r * mb + j] = -1;
    }
  }
  for (int64_t i = t.thread(); i < a.num_slots; i += t.threads()) {
    int slot = -1;
    if (i < tokens) {
      const int r = last_at_most(grow, a.num_rows, &RowGrowth::token0, i);
      const RowGrowth g = grow[r];
      const int pos = g.len + (int)(i - g.token0);
      // A page that the row had comes from the input: keep_rows may be CTAs of
      // other clusters, which no barrier of the team orders.  (In place too: the
      // entries that a row had are never written.)
      if (served(g) && pos < g.len + g.add)
        slot = (pos / bs < row_pages(g.len, bs) ? a.block_tables[r * mb + pos / bs]
                                                : ld_cg(&a.out_tables[r * mb + pos / bs])) * bs + pos % bs;
    }
    a.slot_mapping[i] = slot;
  }
}

// --------------------------------------------------------------- compact

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PagesArgs a) {
  __shared__ RankScratch scratch;
  const Team t;
  plan_begins();
  Segment s = segment_of(a, t);
  auto in_use = [](int count) { return count > 0; };
  const Marks marks = mark_segment(a, t, a.ref_counts, 0, scratch, &s, in_use);
  const int64_t live = s.total;  // pages [0, live) hold everything afterwards

  // Free page p < live is hole p - (pages in use before it); and how many of
  // the pages in use stay.
  if (t.rank == 0 && threadIdx.x == 0 && live == a.num_blocks) a.ws.head->copies = 0;
  for_spans(a.ref_counts, 0, scratch, s, marks, kIntMax, in_use, [&](int64_t p0, const Marks& m, int64_t rank) {
#pragma unroll 1
    for (int i = 0; i < rounds_of(p0, s.end) && p0 + i * pages_per_round() <= live; ++i) {
      int64_t k = rank + rank_in_round(m, scratch, i);
      const unsigned four = m.bits >> (4 * i) & 15u;
      for (int j = 0; j < 4; ++j) {
        const int64_t p = page_of(p0, i) + j;
        if (p >= s.end) break;
        if (p == live) a.ws.head->copies = (int)(live - k);
        if (four >> j & 1)
          ++k;
        else if (p < live)
          a.ws.page[p - k] = (int)p;
      }
      rank += scratch.round[i];
    }
  });
  t.sync();
  const int64_t staying = live - ld_cg(&a.ws.head->copies);
  for_spans(a.ref_counts, 0, scratch, s, marks, kIntMax, in_use, [&](int64_t p0, const Marks& m, int64_t rank) {
#pragma unroll 1
    for (int i = 0; i < rounds_of(p0, s.end); ++i) {
      const int64_t p = page_of(p0, i);
      if (p < s.end) {
        int64_t k = rank + rank_in_round(m, scratch, i);
        const int4 c4 = load_pages(a.ref_counts, p, s.end, 0);
        const int c[4] = {c4.x, c4.y, c4.z, c4.w};
        int place[4];
        int64_t at[4];  // the k-th page in use above moves into the k-th hole below
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          at[j] = c[j] > 0 && p + j >= live ? k - staying : -1;
          place[j] = at[j] >= 0 ? ld_cg(&a.ws.page[at[j]]) : c[j] > 0 ? (int)(p + j) : -1;
          k += c[j] > 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (at[j] >= 0) a.ws.pairs[at[j]] = PagePair{(int)(p + j), place[j], a.block_size, 0};
          if (c[j] > 0) a.out_counts[place[j]] = c[j];
          if (p + j >= live && p + j < s.end) a.out_counts[p + j] = 0;
        }
        store_pages(a.places, p, s.end, make_int4(place[0], place[1], place[2], place[3]));
      }
      rank += scratch.round[i];
    }
  });
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

// The plan's launch: enough threads to see its largest array in one round, the
// pages four at a time.
struct TeamShape {
  int size, threads;
};
TeamShape team_shape(const PagesArgs& a) {
  const int64_t rows = a.num_rows > a.num_out ? a.num_rows : a.num_out;
  int64_t n = rows * a.max_blocks;
  if (a.num_blocks / 4 > n) n = a.num_blocks / 4;
  if (a.num_slots > n) n = a.num_slots;
  // (256 threads up to 512 of them: 8.0 against 9.7 us for a token for each of 8
  // rows, 11.1 against 11.5 for a compaction of 400 pages; up to 1024 the latter
  // of 1000 pages takes 15.9 against 13.7.)
  if (n <= 2 * kFewThreads) return {1, kFewThreads};
  int size = 1;
  while (size < kMaxTeam && (int64_t)size * kPlanThreads < n) size *= 2;
  return {size, kPlanThreads};
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
  return 256 + (size_t)pairs * sizeof(PagePair) + (size_t)rows * sizeof(RowGrowth) +
         (size_t)pages * sizeof(int);
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
  return w;
}

cudaError_t launch_pages_fork(const PagesArgs& a, const PagesCache& c, int num_sms,
                              cudaStream_t stream) {
  const TeamShape t = team_shape(a);
  cudaError_t e = launch(fork_plan_kernel, t.size, t.threads, 0, t.size, true, stream, a);
  return e != cudaSuccess ? e : launch_copies(a, c, num_sms, stream);
}

cudaError_t launch_pages_extend(const PagesArgs& a, int num_sms, cudaStream_t stream) {
  const TeamShape t = team_shape(a);
  // CTAs that keep the table rows, two entries a thread.  In place there is
  // little to keep, and the lengths must be read before the team writes them.
  const int64_t entries = (int64_t)a.num_rows * a.max_blocks;
  int keepers = 0;
  if (t.size == kMaxTeam && a.out_tables != a.block_tables && a.out_lens != a.context_lens) {
    const int64_t cluster = 2ll * t.threads * t.size;
    const int64_t want = (entries + cluster - 1) / cluster, room = num_sms / t.size - 1;
    keepers = t.size * (int)(want < room ? want : room);
  }
  return launch(extend_plan_kernel, t.size + keepers, t.threads, 0, t.size, true, stream, a);
}

cudaError_t launch_pages_compact(const PagesArgs& a, const PagesCache& c, int num_sms,
                                 cudaStream_t stream) {
  const TeamShape t = team_shape(a);
  cudaError_t e = launch(compact_plan_kernel, t.size, t.threads, 0, t.size, true, stream, a);
  return e != cudaSuccess ? e : launch_copies(a, c, num_sms, stream);
}

}  // namespace kvp
