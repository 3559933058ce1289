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
  return (int)(((int64_t)len + block_size - 1) / block_size);
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

// This CTA's segment of the pages, and the rank of its first counted page:
// counts the pages of the segment that `pick` accepts, publishes the count in
// the workspace, and sums those of the CTAs before it.
struct Segment {
  int64_t begin, end;
  int64_t base, total;  // counted pages before the segment / in the pool
};

template <typename Pick>
__device__ Segment count_pages(const PagesArgs& a, const Team& t, long long* warp_sums, Pick pick) {
  Segment s;
  const int64_t per = (a.num_blocks + t.size - 1) / t.size;
  s.begin = min(per * t.rank, a.num_blocks);
  s.end = min(s.begin + per, a.num_blocks);
  int mine = 0;
  for (int64_t p = s.begin + threadIdx.x; p < s.end; p += kPlanThreads) mine += pick(p) ? 1 : 0;
  int total;
  block_scan(mine, warp_sums, &total);
  if (threadIdx.x == 0) a.ws.team_counts[t.rank] = total;
  t.sync();
  s.base = s.total = 0;
  for (int i = 0; i < t.size; ++i) {
    const int c = ld_cg(&a.ws.team_counts[i]);
    if (i < t.rank) s.base += c;
    s.total += c;
  }
  return s;
}

// Calls use(page, rank) for every page of the segment that `pick` accepts, in
// order, with its rank among the pool's; stops after rank limit - 1.
template <typename Pick, typename Use>
__device__ void for_pages(const Segment& s, int64_t limit, long long* warp_sums, Pick pick, Use use) {
  int64_t base = s.base;
  for (int64_t p0 = s.begin; p0 < s.end && base < limit; p0 += kPlanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const bool ok = p < s.end && pick(p);
    int total;
    const int64_t k = base + block_scan(ok ? 1 : 0, warp_sums, &total);
    if (ok && k < limit) use(p, k);
    base += total;
  }
}

// ------------------------------------------------------------------ fork

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[32];
  const Team t;
  const int bs = a.block_size;
  const int64_t mb = a.max_blocks;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int64_t p = t.thread(); p < a.num_blocks; p += t.threads()) {
    a.out_counts[p] = a.ref_counts[p];
    a.ws.page[p] = kIntMax;  // lowest new row whose unfilled last page this is
  }
  t.sync();

  // Every old row lets go of its pages; every new row takes its parent's,
  // except an unfilled last page, which goes to one new row (below).
  for (int64_t i = t.thread(); i < (int64_t)a.num_rows * mb; i += t.threads()) {
    const int r = (int)(i / mb), j = (int)(i % mb);
    if (j >= row_pages(row_len(a, r), bs)) continue;
    const int e = a.block_tables[i];
    if (e < 0 || e >= a.num_blocks)
      record_error(a.status, KVP_ERR_DEVICE_DATA);
    else
      atomicAdd(&a.out_counts[e], -1);
  }
  for (int64_t i = t.thread(); i < (int64_t)a.num_out * mb; i += t.threads()) {
    const int r = (int)(i / mb), j = (int)(i % mb);
    int p = a.parents[r];
    if (p < -1 || p >= a.num_rows) {
      record_error(a.status, KVP_ERR_DEVICE_DATA);
      p = -1;
    }
    const int len = p >= 0 ? row_len(a, p) : 0;
    const int n = row_pages(len, bs);
    if (j == 0) a.out_lens[r] = len;
    int e = j < n ? a.block_tables[(int64_t)p * mb + j] : -1;
    if (e >= a.num_blocks || e < 0) e = -1;  // recorded above, with the parent's row
    a.out_tables[i] = e;
    if (e < 0) continue;
    if (j == n - 1 && len % bs)
      atomicMin(&a.ws.page[e], r);
    else
      atomicAdd(&a.out_counts[e], 1);
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
  auto is_free = [&](int64_t p) { return ld_cg(&a.out_counts[p]) == 0; };
  const Segment s = count_pages(a, t, warp_sums, is_free);
  for_pages(s, copies, warp_sums, is_free, [&](int64_t p, int64_t k) {
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

// The number of entries of the non-decreasing v[0 .. n) that are <= x.
__device__ __forceinline__ int upper_bound(const int* v, int n, int64_t x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)ld_cg(&v[mid]) <= x)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[32];
  const Team t;
  const int bs = a.block_size;
  const int64_t mb = a.max_blocks;

  // Rows: pages needed and new tokens, with their prefix sums over the rows.
  if (t.rank == 0) {
    long long pages = 0, tokens = 0;
    for (int r0 = 0; r0 < a.num_rows; r0 += kPlanThreads) {
      const int r = r0 + (int)threadIdx.x;
      long long need = 0, asked = 0;
      int add = 0, len = 0;
      bool bad = false;
      if (r < a.num_rows) {
        len = row_len(a, r);
        bad = len != a.context_lens[r];
        add = a.new_tokens[r];
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
      if (r < a.num_rows) {
        a.ws.row[r] = (int)min(page0, (long long)kIntMax);  // past every page and slot
        a.ws.row2[r] = (int)min(token0, (long long)kIntMax);
        a.ws.row3[r] = len;
        a.ws.row4[r] = add;
      }
    }
    if (threadIdx.x == 0) {
      a.ws.head->copies = (int)min(pages, (long long)kIntMax);
      a.ws.head->tokens = (int)min(tokens, (long long)kIntMax);
      if (tokens > a.num_slots) record_error(a.status, KVP_ERR_DEVICE_DATA);
    }
  }
  auto is_free = [&](int64_t p) { return ld_cg(&a.ref_counts[p]) == 0; };
  const Segment s = count_pages(a, t, warp_sums, is_free);  // (a team barrier)
  const int pages = ld_cg(&a.ws.head->copies);

  // The tables as they were; the new entries follow below.
  for (int64_t i = t.thread(); i < a.num_rows * mb; i += t.threads()) {
    const int r = (int)(i / mb), j = (int)(i % mb);
    const int len = ld_cg(&a.ws.row3[r]);
    const int had = row_pages(len, bs), add = ld_cg(&a.ws.row4[r]);
    const int has = row_pages(len + add, bs);
    const bool fits = (int64_t)ld_cg(&a.ws.row[r]) + (has - had) <= s.total;
    if (j < had)
      a.out_tables[i] = a.block_tables[i];
    else if (j >= has || !fits)
      a.out_tables[i] = -1;
    if (j == 0) {
      if (!fits && has > had) record_error(a.status, KVP_ERR_DEVICE_DATA);
      a.out_lens[r] = !fits && has > had ? len : len + add;
    }
  }
  // Free page of rank k goes to the row whose pages start at or before k.
  if (a.out_counts != a.ref_counts)
    for (int64_t p = s.begin + threadIdx.x; p < s.end; p += kPlanThreads)
      a.out_counts[p] = a.ref_counts[p];
  __syncthreads();
  for_pages(s, pages, warp_sums, is_free, [&](int64_t p, int64_t k) {
    const int r = upper_bound(a.ws.row, a.num_rows, k) - 1;
    const int len = ld_cg(&a.ws.row3[r]), add = ld_cg(&a.ws.row4[r]), page0 = ld_cg(&a.ws.row[r]);
    const int had = row_pages(len, bs), need = row_pages(len + add, bs) - had;
    if (page0 + need > s.total) return;  // not enough pages left for the whole row
    a.out_tables[r * mb + had + (k - page0)] = (int)p;
    a.out_counts[p] = 1;
  });
  t.sync();

  const int tokens = ld_cg(&a.ws.head->tokens);
  for (int64_t i = t.thread(); i < a.num_slots; i += t.threads()) {
    int slot = -1;
    if (i < tokens) {
      const int r = upper_bound(a.ws.row2, a.num_rows, i) - 1;
      const int len = ld_cg(&a.ws.row3[r]);
      const int64_t pos = len + (i - ld_cg(&a.ws.row2[r]));
      if (pos < ld_cg(&a.out_lens[r]))
        slot = ld_cg(&a.out_tables[r * mb + pos / bs]) * bs + (int)(pos % bs);
    }
    a.slot_mapping[i] = slot;
  }
}

// --------------------------------------------------------------- compact

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PagesArgs a) {
  __shared__ long long warp_sums[32];
  const Team t;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto is_live = [&](int64_t p) { return a.ref_counts[p] > 0; };
  const Segment s = count_pages(a, t, warp_sums, is_live);
  const int64_t live = s.total;  // pages [0, live) hold everything afterwards

  // Live pages before each page; free page p < live is hole p - before(p).
  int64_t base = s.base;
  for (int64_t p0 = s.begin; p0 < s.end; p0 += kPlanThreads) {
    const int64_t p = p0 + threadIdx.x;
    const bool ok = p < s.end && is_live(p);
    int total;
    const int64_t before = base + block_scan(ok ? 1 : 0, warp_sums, &total);
    if (p < s.end) {
      a.ws.page[p] = (int)before;
      if (!ok && p < live) a.ws.page2[p - before] = (int)p;
    }
    base += total;
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
  for (int64_t i = t.thread(); i < (int64_t)a.num_rows * a.max_blocks; i += t.threads()) {
    const int r = (int)(i / a.max_blocks), j = (int)(i % a.max_blocks);
    int e = -1;
    if (j < row_pages(row_len(a, r), a.block_size)) {
      const int old = a.block_tables[i];
      if (old >= 0 && old < a.num_blocks) e = ld_cg(&a.places[old]);
      if (e < 0) record_error(a.status, KVP_ERR_DEVICE_DATA);  // a row's page is outside or free
    }
    a.out_tables[i] = e;
  }
}

// ------------------------------------------------------------------ copy

constexpr int kCopyThreads = 256;
constexpr int kVecPerThread = 8;
constexpr int64_t kChunkVecs = (int64_t)kCopyThreads * kVecPerThread;  // 32 KiB

__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ void st_once(uint4* p, const uint4& v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Copies the first `tokens` rows of each listed page in every plane.  The
// number of pairs is the plan kernel's.  Sources and destinations of one plan
// are disjoint, so the order of the copies does not matter.
template <bool kVec>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(
    uint16_t* __restrict__ cache, int64_t num_planes, int64_t plane_stride, int64_t block_elems,
    int64_t row_elems, int64_t chunks_per_block, const PagesHead* head, const PagePair* pairs) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t items = (int64_t)ld_cg(&head->copies) * num_planes * chunks_per_block;
  for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
    const int64_t chunk = w % chunks_per_block;
    const int64_t pp = w / chunks_per_block;
    const int64_t plane = pp % num_planes;
    const int4 pr = __ldcg(reinterpret_cast<const int4*>(pairs + pp / num_planes));
    uint16_t* base = cache + plane * plane_stride;
    const uint16_t* src = base + (int64_t)pr.x * block_elems;
    uint16_t* dst = base + (int64_t)pr.y * block_elems;
    const int64_t elems = (int64_t)pr.z * row_elems;
    if constexpr (kVec) {
      const uint4* s4 = reinterpret_cast<const uint4*>(src);
      uint4* d4 = reinterpret_cast<uint4*>(dst);
      const int64_t v0 = chunk * kChunkVecs, v1 = min(v0 + kChunkVecs, elems >> 3);
      if (v1 - v0 == kChunkVecs) {
        uint4 r[kVecPerThread];
#pragma unroll
        for (int i = 0; i < kVecPerThread; ++i) r[i] = ld_once(s4 + v0 + i * kCopyThreads + threadIdx.x);
#pragma unroll
        for (int i = 0; i < kVecPerThread; ++i) st_once(d4 + v0 + i * kCopyThreads + threadIdx.x, r[i]);
      } else {
        for (int64_t v = v0 + threadIdx.x; v < v1; v += kCopyThreads) st_once(d4 + v, ld_once(s4 + v));
      }
    } else {
      const int64_t e0 = chunk * kChunkVecs, e1 = min(e0 + kChunkVecs, elems);
      for (int64_t e = e0 + threadIdx.x; e < e1; e += kCopyThreads) dst[e] = src[e];
    }
  }
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, int threads, int cluster, bool pdl,
                   cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
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

// CTAs of the plan: one per 4096 elements of its largest array.
int team_size(const PagesArgs& a) {
  const int64_t rows = a.num_rows > a.num_out ? a.num_rows : a.num_out;
  int64_t n = rows * a.max_blocks;
  if (a.num_blocks > n) n = a.num_blocks;
  if (a.num_slots > n) n = a.num_slots;
  int size = 1;
  while (size < kMaxTeam && size * 4096 < n) size *= 2;
  return size;
}

cudaError_t launch_copies(const PagesArgs& a, const PagesCache& c, int num_sms, cudaStream_t stream) {
  const int64_t block_elems = (int64_t)a.block_size * c.row_elems;
  const bool vec = (reinterpret_cast<uintptr_t>(c.cache) & 15u) == 0 && c.plane_stride % 8 == 0 &&
                   c.row_elems % 8 == 0;
  const int64_t units = vec ? block_elems / 8 : block_elems;
  const int64_t chunks = (units + kChunkVecs - 1) / kChunkVecs;
  return launch(vec ? copy_pages_kernel<true> : copy_pages_kernel<false>, num_sms * 8, kCopyThreads, 0,
                true, stream, c.cache, c.num_planes, c.plane_stride, block_elems, c.row_elems, chunks,
                (const PagesHead*)a.ws.head, (const PagePair*)a.ws.pairs);
}

}  // namespace

size_t pages_workspace_bytes(int64_t num_blocks, int64_t rows) {
  const int64_t pairs = num_blocks > rows ? num_blocks : rows;
  return 256 + (size_t)pairs * sizeof(PagePair) + (size_t)(2 * num_blocks + 4 * rows) * sizeof(int);
}

PagesWorkspace pages_workspace(void* base, int64_t num_blocks, int64_t rows) {
  PagesWorkspace w;
  uint8_t* p = static_cast<uint8_t*>(base);
  const int64_t pairs = num_blocks > rows ? num_blocks : rows;
  w.head = reinterpret_cast<PagesHead*>(p);
  w.team_counts = reinterpret_cast<int*>(p + 64);
  w.pairs = reinterpret_cast<PagePair*>(p + 256);
  w.page = reinterpret_cast<int*>(w.pairs + pairs);
  w.page2 = w.page + num_blocks;
  w.row = w.page2 + num_blocks;
  w.row2 = w.row + rows;
  w.row3 = w.row2 + rows;
  w.row4 = w.row3 + rows;
  return w;
}

cudaError_t launch_pages_fork(const PagesArgs& a, const PagesCache& c, int num_sms,
                              cudaStream_t stream) {
  const int size = team_size(a);
  cudaError_t e = launch(fork_plan_kernel, size, kPlanThreads, size, false, stream, a);
  return e != cudaSuccess ? e : launch_copies(a, c, num_sms, stream);
}

cudaError_t launch_pages_extend(const PagesArgs& a, cudaStream_t stream) {
  const int size = team_size(a);
  return launch(extend_plan_kernel, size, kPlanThreads, size, false, stream, a);
}

cudaError_t launch_pages_compact(const PagesArgs& a, const PagesCache& c, int num_sms,
                                 cudaStream_t stream) {
  const int size = team_size(a);
  cudaError_t e = launch(compact_plan_kernel, size, kPlanThreads, size, false, stream, a);
  return e != cudaSuccess ? e : launch_copies(a, c, num_sms, stream);
}

}  // namespace kvp
