// attn_shared_plan / attn_decode_shared(_append): paged decode of a batch whose
// sequences share leading pages.
//
// Sources: "【nano-vllm 学习】04 - 自顶向下的引擎调度层源码学习2", section
// "场景优化1：Parallel Memory Shared" (sequences of one prompt map their prompt
// blocks to the same physical blocks), and the prefix cache of "nano-vLLM-1",
// BlockManager "3. 核心方法一：分配 (allocate)"; the attention is that of
// attn_decode_paged.
//
// With the keys of sequence b cut into a part that its group shares and a part
// of its own, softmax(q K^T) V is put together from partial results (m = the
// largest scaled score, l = sum 2^(s - m), acc = sum 2^(s - m) v, all fp32):
//     M = max_p m_p,  out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p.
// So a group's shared keys can be read once, as a matrix product with all the
// queries of the group, which turns the part that is read B times by
// attn_decode_paged from HBM-bound into tensor-core work.
//
// Four kernels: the plan (once per step: groups, tiles, where each CTA starts),
// and per layer the own parts (HBM-bound), the prefixes (tcgen05) and the
// merge.  The two in the middle are sized to share every SM (shared memory
// 131 + 99 of 228 KB, registers, 256 tensor-memory columns), one CTA each: the
// tensor core works on the prefixes under the stream of the own parts, whatever
// their proportion, with nothing to choose on the host.  The grids depend on
// the SM count alone, so a captured call serves any batch of its size.
//
// Measured on one GB300 (device time of plan + call, its bytes read once):
//   512 sequences, 32/8/128, 8192 keys shared, 64 .. 1000 own    216 us
//     (own parts alone 162 us = 6.7 TB/s, prefixes alone 64 us = 1080 TFLOP/s;
//      together 192: the prefixes are through after 113, and the own parts run
//      at 70% until then, which is not one resource's doing: neither without the
//      MMAs of either, nor with the bytes of either from L2 or halved, does it
//      come near 162; 20 merge and plan)
//   64 sequences, 16/8/128, 2048 shared, 100 .. 1500 own           46.5 us
//   16 sequences, 64/8/128, 32768 shared, up to 64 own             44 us
//   against attn_decode_paged on such tables, 16/8/128: 64 sequences with 2048
//   shared and 100 .. 600 own 33 against 100 us, with 8192 35 against 323; on tables
//   that share nothing: 64 sequences of 100 .. 1500 46 against 45, 128 of 500 .. 4000
//   178 against 182, 512 of 64 .. 1000 (32/8/128) 177 against 195.
// Break-even of the default min_shared_len (128 tokens; groups joined / not, 16/8/128,
// 64 sequences of 100 .. 600 own tokens, +-1 us): 4 groups of 16 28.8 / 30.6 us, one of
// 64 28.7 / 30.8.  Groups of four gain from 256 tokens on (32 groups: 46.6 / 53.4; 128
// tokens 46.2 / 47.1), of two from 512 to 1024 (32 groups: 512 tokens 41.7 / 42.2, 1024
// 54.7 / 57.9, 8192 188 / 311); below, pairs lose up to 2 us, with few tokens of their
// own 4 (100 pairs with up to 64: 128 tokens 41.4 / 32.8, 512 61.5 / 72.5).
#include "decode_shared.h"

#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "kvp_warp.cuh"

namespace kvp {
namespace {

constexpr int kPlanMagic = 0x53504c31;
constexpr int kTileRows = 128;  // query rows of a prefix tile
constexpr int kTileKeys = 64;   // keys of a prefix step

// Both split kernels cut their work, laid end to end, into one equal chunk
// per CTA; a chunk's pieces are its segments.  Segment (item i, CTA c) has its
// own rows of partial results: items and CTAs only ever advance together, so
// (rows of the items before i) + c * (rows of an item) is never taken twice.
__host__ __device__ constexpr int prefix_ctas(int sms) { return 2 * sms; }
__host__ __device__ constexpr int own_ctas(int sms) { return sms; }
// Prefix steps of a CTA: each CTA that touches an item adds a part to its rows'
// merge, but a chain of steps is latency (8 sequences behind 1024 tokens, four
// layers: 51.7 / 50.1 / 53.1 / 66.7 us with at least 1 / 2 / 4 / 8).
constexpr int kLeastSteps = 2;
// An SM holds one prefix CTA beside its own-part CTA; the second one begins when
// either has ended.  So the first gets as many steps more as it can do beside the
// own part: kLeadSteps for the latency of that kernel, and one per kLeadOwn tokens
// x kv heads of its share.  Equal chunks / these (us): 16 sequences behind 4096
// tokens 23.1 / 19.8, 128 behind 8192 49.7 / 46.8, 64 behind 32768 with 500 ..
// 2500 own 101.8 / 97.8.  (kLeadSteps 0, 4, 6: 128 behind 8192 49.7, 48.1, 49.1;
// kLeadOwn 64 as 128, 256 loses 9 us of the last.)
constexpr int kLeadSteps = 2;
constexpr int kLeadOwn = 128;
// A sequence in a CTA costs about as much as two or three stages of its stream
// (query, page and plan look-ups, partials): in the own-part kernel's split it
// counts three stages of tokens more than it has (16 prompts x 8 samples 63.1 us
// with two, 62.3 with three, 62.5 with four).  A CTA takes as much at least (one
// document for 16 sequences: 44.5 us, 45.3 with twice that).
__host__ __device__ constexpr int own_gap(int num_kv_heads) { return 3 * 64 / num_kv_heads; }
__device__ __forceinline__ long long chunk_of(long long total, int ctas, int least) {
  const long long c = (total + ctas - 1) / ctas;
  return c < least ? least : c;
}

// x / y for the plan's work positions, which nearly always fit 32 bits.
__device__ __forceinline__ long long quotient(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// Where the prefix CTAs' chunks begin: an SM takes one of the first wave beside
// its own-part CTA and one of the second when either has ended.
struct PrefixSplit {
  int wave;  // CTAs of the first wave
  long long first, second;
  __device__ explicit PrefixSplit(const SharedPlanHead& h)
      : wave(h.sms), first(h.prefix_chunk), second(h.prefix_chunk2) {}
  __device__ PrefixSplit(int sms, long long a, long long b) : wave(sms), first(a), second(b) {}
  __device__ long long begin(int cta) const {
    return cta < wave ? cta * first : wave * first + (cta - wave) * second;
  }
  __device__ long long end(int cta) const { return begin(cta) + (cta < wave ? first : second); }
  // The CTA of step x.
  __device__ long long cta(long long x) const {
    const long long y = x - wave * first;
    return y < 0 ? quotient(x, first) : wave + quotient(y, second);
  }
};

__device__ __forceinline__ PrefixSplit split_prefixes(long long total, long long own, int sms) {
  const long long per_sm = (total + sms - 1) / sms, lead = kLeadSteps + own / kLeadOwn;
  long long first = (per_sm + lead + 1) / 2;
  if (first > per_sm) first = per_sm;
  if (first < kLeastSteps) first = kLeastSteps;
  const long long rest = total - first * sms;
  return PrefixSplit(sms, first, chunk_of(rest > 0 ? rest : 0, sms, kLeastSteps));
}

// The weights are rounded to bf16 for the matrix products with V.  With one or two
// query heads per kv head, where attn_decode_paged has them in fp32, they go in as two
// bf16 numbers, the second being what the first leaves out (split_bf16x2: within 2^-15).
// Against 64 bits, 2-norm, 16/8/128, 16 sequences of 1000 to 1200 keys, shared or not:
// 0.00166, as a result rounded once and as attn_decode_paged (32/8/128 0.0023, both).
// In the own parts that takes no more products (see own_consumer); the prefixes have
// twice those with V: 512 sequences of 16/8/128 behind 8192 tokens 67.7 against 59.5 us
// with one number, with own parts of 64 .. 1000 tokens 201 against 190, 64 behind 2048
// with 100 .. 1500 48.7 against 47.9.  (A barrier of its own for the second number, so
// that its arithmetic runs under the first product: 104 us, registers spill.)
// With four or eight heads one number, as in attn_decode_paged.
__host__ __device__ constexpr bool fine_weights(int group) { return group <= 2; }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ plan

struct PlanArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  int max_blocks;
  int num_seqs;
  int64_t num_blocks;
  int block_size;
  int group;         // query heads per kv head
  int num_kv_heads;
  int gap;           // own_gap
  int min_shared;    // tokens
  int sms;
  SharedPlan plan;
  int* status;
};

// Exclusive prefix sums of N values at once over the block's threads; total[i]
// = the sum of v[i].  `sums` holds the warps' sums.
template <int T, int N>
__device__ void block_scan(long long (&v)[N], long long (&total)[N], long long (*sums)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    incl[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl[i], o);
      if (lane >= o) incl[i] += y;
    }
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i][warp] = incl[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long s = lane < T / 32 ? sums[i][lane] : 0;
    long long ws = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, ws, o);
      if (lane >= o) ws += y;
    }
    total[i] = __shfl_sync(0xffffffffu, ws, 31);
    v[i] = __shfl_sync(0xffffffffu, ws - s, warp) + incl[i] - v[i];
  }
}
__device__ __forceinline__ int plan_ctx(const PlanArgs& a, int b) {
  const int c = a.context_lens[b];
  const int64_t cap = (int64_t)a.max_blocks * a.block_size;
  if (c < 0 || c > cap) {
    record_error(a.status, KVP_ERR_DEVICE_DATA);
    return c < 0 ? 0 : (int)cap;
  }
  return c;
}

// Leading pages that rows b - 1 and b of the table share, by one warp.  Only
// pages before each sequence's last token count, so that every sequence keeps
// at least one token of its own.  *ctx = sequence b's context length.
__device__ int shared_pages(const PlanArgs& a, int b, int* ctx) {
  const int lane = threadIdx.x & 31;
  const int32_t* y = a.block_tables + (int64_t)b * a.max_blocks;
  const int32_t* x = b > 0 ? y - a.max_blocks : y;
  constexpr int U = 4;  // rounds of 32 entries with their loads in flight together
  int ex[U], ey[U];
  auto load = [&](int j0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + 32 * u + lane;
      ex[u] = j < a.max_blocks ? x[j] : -1;
      ey[u] = j < a.max_blocks ? y[j] : -2;
    }
  };
  load(0);  // beside the lengths that say how many of them count
  const int prev = b > 0 ? plan_ctx(a, b - 1) : 0;
  *ctx = plan_ctx(a, b);
  const int n = prev > 0 && *ctx > 0 ? (min(prev, *ctx) - 1) / a.block_size : 0;
  for (int j0 = 0; j0 < n; j0 += 32 * U) {
    if (j0) load(j0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool same = j0 + 32 * u + lane < n && ex[u] == ey[u] && ex[u] >= 0 && ex[u] < a.num_blocks;
      const unsigned diff = ~__ballot_sync(0xffffffffu, same);
      if (diff) return j0 + 32 * u + __ffs(diff) - 1;
    }
  }
  return n;
}

// Stores v in CTA 0's copy of a shared variable of the cluster.
__device__ __forceinline__ void store_cta0(int* p, int v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// Sequence b reads its first pages together with sequence b - 1: it shares
// enough of them, and not less than half of what either neighbour shares
// (a page or two that all requests have in common, e.g. a short system
// prompt, must not join groups that share much more among themselves).
__device__ __forceinline__ bool plan_joined(const PlanArgs& a, int b, int prev, int same, int next) {
  if (b == 0 || same == 0 || (int64_t)same * a.block_size < a.min_shared) return false;
  return 2 * (int64_t)same >= max(prev, next);
}

// One cluster.  The warps of all its CTAs compare the table rows; after a
// cluster barrier CTA 0 forms the groups and tiles by prefix sums over the
// sequences, T at a time.  Up to T sequences' shared-page counts and groups
// stay in shared memory (of more, they go through the plan buffer): the
// kernel is a chain of small dependent steps, and each round trip to L2 that
// it does without is 0.7 us of a step's latency.
template <int T>
__global__ void __launch_bounds__(T) shared_plan_kernel(const PlanArgs a) {
  __shared__ long long sums[3][32];
  __shared__ int s_same[T + 2], s_min[T + 1], s_seq[T + 1],
      s_ctx[T];
  __shared__ long long s_tokens[T + 1], s_steps[T + 1];
  const SharedPlan& p = a.plan;
  const int B = a.num_seqs, bs = a.block_size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool small = B <= T;
  // (Launched in the shadow of the kernel before.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Every CTA of the cluster runs before one writes to another's shared memory.
  asm volatile(
      "barrier.cluster.arrive.relaxed;\n\t"
      "barrier.cluster.wait;" ::
          : "memory");
  for (int b = blockIdx.x + warp * gridDim.x; b < B; b += gridDim.x * (T / 32)) {
    int ctx;
    const int same = shared_pages(a, b, &ctx);
    if (lane == 0) {
      p.ctx[b] = ctx;
      if (small) {
        store_cta0(&s_same[b + 1], same);
        store_cta0(&s_ctx[b], ctx);
      } else {
        p.same[b] = same;
      }
    }
  }
  if (!small) __threadfence();
  asm volatile(
      "barrier.cluster.arrive.release;\n\t"
      "barrier.cluster.wait.acquire;" ::
          : "memory");
  if (blockIdx.x) return;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Groups: maximal runs of joined sequences; all of a group read the pages
  // that every one of them shares.
  int* group_min = small ? s_min : p.group_min;
  int* group_seq = small ? s_seq : p.group_seq;
  for (int b = threadIdx.x; b < B; b += T) group_min[b] = 0x7fffffff;
  int my_ctx = 0, my_group = 0;  // of sequence threadIdx.x
  long long groups = 0;
  for (int b0 = 0; b0 < B; b0 += T) {
    const int b = b0 + (int)threadIdx.x;
    // s_same[i]: sequence b0 - 1 + i
    if (!small) {
      s_same[threadIdx.x + 1] = b < B ? __ldcg(&p.same[b]) : 0;
      if (threadIdx.x == 0) s_same[0] = b > 0 ? __ldcg(&p.same[b - 1]) : 0;
      if (threadIdx.x == 1)
        s_same[T + 1] = b0 + T < B ? __ldcg(&p.same[b0 + T]) : 0;
    } else if (b < B) {
      my_ctx = s_ctx[b];
    }
    __syncthreads();
    const int same = s_same[threadIdx.x + 1];
    const bool joined = b < B && plan_joined(a, b, b > 0 ? s_same[threadIdx.x] : 0, same,
                                             b + 1 < B ? s_same[threadIdx.x + 2] : 0);
    long long v[1] = {b < B && !joined ? 1 : 0}, total[1];
    block_scan<T>(v, total, sums);
    if (b < B) {
      const int g = (int)(groups + v[0]) - (joined ? 1 : 0);
      if (b0 == 0) my_group = g;
      if (!small) p.tile_of[b] = g;
      if (joined)
        atomicMin(&group_min[g], same);
      else
        group_seq[g] = b;
    }
    groups += total[0];
    __syncthreads();
  }

  // Tiles of 128 query rows within a group, and the prefix sums the kernels
  // find their work by: (tiles, sequences in tiles), steps, own positions.
  const int tile_seqs = kTileRows / a.group;
  long long base[3] = {0, 0, 0};
  for (int b0 = 0; b0 < B; b0 += T) {
    const int b = b0 + (int)threadIdx.x;
    int ctx = 0, prefix = 0;
    bool start = false;
    if (b < B) {
      const int g = small ? my_group : p.tile_of[b], m = *(volatile int*)&group_min[g];
      ctx = small ? my_ctx : __ldcg(&p.ctx[b]);
      prefix = m == 0x7fffffff ? 0 : m * bs;
      start = prefix > 0 && (b - *(volatile int*)&group_seq[g]) % tile_seqs == 0;
    }
    const int steps = start ? a.num_kv_heads * ((prefix + kTileKeys - 1) / kTileKeys) : 0;
    const int len = ctx > 0 ? a.gap + ctx - prefix : 0;
    long long v[3] = {((long long)(start ? 1 : 0) << 32) | (prefix > 0 ? 1 : 0), steps, len};
    long long total[3];
    block_scan<T>(v, total, sums);
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] += base[i], base[i] += total[i];
    if (b < B) {
      const int t = (int)(v[0] >> 32) - (start ? 0 : 1);
      const int r = (int)(v[0] & 0xffffffffll);
      p.prefix[b] = prefix;
      p.tile_of[b] = prefix > 0 ? t : -1;
      p.cum_tokens[b] = v[2];
      if (start) {
        p.tile_seq[t] = b;
        p.cum_rows[t] = r;
        p.cum_steps[t] = v[1];
      }
      if (small) {  // for the starts below, in arrays that the groups are done with
        s_same[b] = prefix;
        s_tokens[b] = v[2];
        if (start) {
          s_seq[t] = b;
          s_min[t] = r;
          s_steps[t] = v[1];
        }
      }
    }
  }
  const int tiles = (int)(base[0] >> 32);
  const long long ochunk = chunk_of(base[2], own_ctas(a.sms), a.gap);
  const PrefixSplit split = split_prefixes(base[1], ochunk * a.num_kv_heads, a.sms);
  if (threadIdx.x == 0) {
    p.cum_tokens[B] = base[2];
    p.cum_rows[tiles] = (int)(base[0] & 0xffffffffll);
    p.cum_steps[tiles] = base[1];
    SharedPlanHead h;
    h.magic = kPlanMagic;
    h.num_seqs = B;
    h.group = a.group;
    h.num_kv_heads = a.num_kv_heads;
    h.block_size = bs;
    h.max_blocks = a.max_blocks;
    h.num_tiles = tiles;
    h.sms = a.sms;
    h.gap = a.gap;
    h.pad = 0;
    h.prefix_chunk = split.first;
    h.prefix_chunk2 = split.second;
    h.prefix_total = base[1];
    h.own_chunk = ochunk;
    h.own_total = base[2];
    *p.head = h;
  }
  if (threadIdx.x == 0 && small) {
    s_tokens[B] = base[2];
    s_min[tiles] = (int)(base[0] & 0xffffffffll);
    s_steps[tiles] = base[1];
  }
  __syncthreads();
  // Where each CTA starts: the last sequence (tile) whose positions (steps)
  // begin at or before its first one.
  const long long *tokens = small ? s_tokens : p.cum_tokens, *tsteps = small ? s_steps : p.cum_steps;
  const int *prefixes = small ? s_same : p.prefix, *ctxs = small ? s_ctx : p.ctx;
  const int *tile_seq = small ? s_seq : p.tile_seq, *tile_rows = small ? s_min : p.cum_rows;
  for (int i = threadIdx.x; i < own_ctas(a.sms) + prefix_ctas(a.sms); i += T) {
    const bool own = i < own_ctas(a.sms);
    const int c = own ? i : i - own_ctas(a.sms);
    const long long x = own ? c * ochunk : split.begin(c);
    if (x >= (own ? base[2] : base[1])) continue;
    const long long* v = own ? tokens : tsteps;
    int lo = 0, hi = own ? B : tiles;  // the answer is in [lo, hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (v[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    if (own) {
      p.own_start[c] = SharedOwnStart{lo, ctxs[lo], ctxs[lo] - prefixes[lo], 0, v[lo + 1], 0};
    } else {
      const int seq0 = tile_seq[lo];
      p.prefix_start[c] = SharedPrefixStart{
          lo, seq0, tile_rows[lo + 1] - tile_rows[lo], prefixes[seq0], v[lo], v[lo + 1]};
    }
  }
}

// ------------------------------------------------------------- attention

// Row of partial results in the workspace: accumulator[D], m, l and two pad
// floats, so that every row starts on a 16-byte boundary.
template <int D>
__host__ __device__ constexpr int part_stride() {
  return D + 4;
}

struct SharedArgs {
  const uint16_t* q;
  int64_t q_stride;
  int64_t num_blocks;
  int block_size;
  const int32_t* block_tables;
  int max_blocks;
  int num_seqs, num_heads, num_kv_heads;
  float scale_log2;
  float prefix_scale_log2;  // its magnitude, for the prefix kernel: never 0
  uint32_t prefix_negate;   // and its sign, as the negate-A bit of an MMA
  SharedPlan plan;
  float* prefix_part;  // rows of the prefix kernel's segments
  float* own_part;     // rows of the own-part kernel's segments
  int sms;
  uint16_t* out;
  int64_t out_stride;
  int* status;
};

// Fused store of the step's new rows (null k_new: none).
struct SharedAppend {
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t k_stride, v_stride;
  const int32_t* slot_mapping;
  uint16_t* k_cache;
  uint16_t* v_cache;
};

// True if the plan was made for this call's batch and shape.
__device__ __forceinline__ bool plan_fits(const SharedArgs& a) {
  // The head's first eight fields: magic, num_seqs, group, num_kv_heads;
  // block_size, max_blocks, num_tiles, sms.
  const int4* h = reinterpret_cast<const int4*>(a.plan.head);
  const int4 x = h[0], y = h[1];
  return (x.x == kPlanMagic) & (x.y == a.num_seqs) & (x.z == a.num_heads / a.num_kv_heads) &
         (x.w == a.num_kv_heads) & (y.x == a.block_size) & (y.y == a.max_blocks) & (y.w == a.sms);
}

// ------------------------------------------------- the shared prefixes
//
// Item: a tile t of up to 128 query rows (128 / G sequences of a group x the G
// query heads of kv head h) against all keys of the group's prefix, taken 64
// at a time ("step").  The items' steps, laid end to end, are split over the
// CTAs; a CTA's pieces ("segments") leave un-normalised partials.
// Per step: S = Q K^T (tcgen05, M128, K = D) -> row maxima and weights in
// registers -> P in tensor memory -> O += P V.  Rows of a group share the
// same keys, so nothing but the last step's ragged end is masked.
//
// 192 threads: warps 0-3 softmax (thread = row), warp 4 TMA producer, warp 5
// tensor memory and MMA issue.  S of two steps is one product (N 128), so that Q
// is read from shared memory half as often: alone the kernel takes the same, but
// the own parts beside it gain (231 to 216 us for 512 sequences).  The softmax of
// the second step runs on while the first one's PV is issued.
// 512 x 32 rows over 8192 keys: 64 us, 1080 TFLOP/s (128 with one S of 64 keys and
// the MMAs issued by a lane alone).  What bounds it is the chain of a step, 1960
// cycles: softmax 690 (552 of them arithmetic), PV and S of the next steps 1000,
// half of it issue; the tensor pipe is active 51% of the time with two CTAs on an
// SM, issue slots 38%.  K and V are read once per tile from L2 (552 MB for those
// rows; 39 MB from HBM).

constexpr int kPrefixThreads = 192;
// Two warps of this kernel and three of the own-part kernel must fit one SM
// sub-partition's 16384 registers: 32 * (2 * 112 + 3 * 96).
constexpr int kPrefixRegs = 112;

enum : int {
  P_KFULL = 0,   // [2]
  P_KEMPTY = 2,  // [2]
  P_VFULL = 4,   // [2]
  P_VEMPTY = 6,  // [2]
  P_SFULL = 8,   // [2]
  P_PFULL = 10,  // [2]
  P_QFULL = 12,
  P_QEMPTY,
  P_PVDONE,  // a step's PV
  P_ODONE,   // a segment's last PV
  P_OFREE,
  P_DRAIN,
  P_BARS
};

template <int D>
struct PrefixLayout {
  static constexpr uint32_t kPanels = D / 64;
  static constexpr uint32_t kQPanel = kTileRows * 128;  // 128 rows x 64 columns, 128-byte swizzle
  static constexpr uint32_t kPanel = kTileKeys * 128;   // 64 keys x 64 columns
  static constexpr uint32_t kQBytes = kTileRows * D * 2;
  static constexpr uint32_t kSlot = kTileKeys * D * 2;  // a step's K or V
  static constexpr uint32_t kQ = 0, kK = kQBytes, kV = kK + 2 * kSlot;  // two slots of K and V
  static constexpr uint32_t kBar = kV + 2 * kSlot;
  static constexpr uint32_t kAlloc = kBar + P_BARS * 8 + 16;
};
constexpr int kMaxSub = kTileKeys / 16;    // pages of a step (the smallest page has 16 tokens)
// Tensor memory: S of even steps | S of odd steps (P over each one's first half, what
// bf16 leaves of it over the second) | O.
constexpr uint32_t kColO = 2 * kTileKeys, kPrefixTmem = 256;

// Steps of the next unit, of `left` in the segment: an even step and the one
// after it have their S in one matrix product of 128 keys, which reads Q once.
__device__ __forceinline__ int unit_of(uint32_t n, int left) { return !(n & 1) && left > 1 ? 2 : 1; }

// The segments of this CTA, one after the other.
struct PrefixSegment {
  long long pos, end;  // flat steps left
  // the current tile
  int t;
  int seq0, nseq;      // its sequences
  int prefix;          // its keys
  long long c0, c1;    // its steps of the flat order
  // the segment
  int h, s0, s1;       // kv head, steps [s0, s1) of the item
  long long row0;      // first row of partials, after those of the tiles before

  __device__ void begin(const SharedPrefixStart& s) {
    t = s.tile;
    seq0 = s.seq0;
    nseq = s.nseq;
    prefix = s.prefix;
    c0 = s.step0;
    c1 = s.step1;
  }

  __device__ bool next(const SharedArgs& a) {
    if (pos >= end) return false;
    const int Hkv = a.num_kv_heads, G = a.num_heads / Hkv;
    if (pos == c1) {
      ++t;
      seq0 = a.plan.tile_seq[t];
      nseq = a.plan.cum_rows[t + 1] - a.plan.cum_rows[t];
      prefix = a.plan.prefix[seq0];
      c0 = c1;
      c1 = a.plan.cum_steps[t + 1];
    }
    const int st = (int)(c1 - c0) / Hkv, rel = (int)(pos - c0);  // (at most 8 x 2^24 steps)
    h = rel / st;
    s0 = rel - h * st;
    const long long left = end - pos;
    s1 = st - s0 < left ? st : s0 + (int)left;
    row0 = (long long)h * nseq * G + (long long)blockIdx.x * kTileRows;
    pos += s1 - s0;
    return true;
  }
};

template <int D>
__device__ void prefix_producer(const SharedArgs& a, PrefixSegment sg, const CUtensorMap* tmQ,
                                const CUtensorMap* tmK, const CUtensorMap* tmV, uint8_t* smem,
                                uint64_t* bars) {
  using Lay = PrefixLayout<D>;
  const int lane = threadIdx.x & 31;
  const int box = a.block_size < kTileKeys ? a.block_size : kTileKeys;
  const int nsub = kTileKeys / box;
  const int shift = __ffs(a.block_size) - 1;  // block_size is a power of two
  const int past = (int)(a.num_blocks * a.block_size);  // a row past the pool: loads zeros
  if (lane == 0) {
    prefetch_tensormap(tmQ);
    prefetch_tensormap(tmK);
    prefetch_tensormap(tmV);
  }
  // Other tiles read the same keys: hold on to them in L2.
  const uint64_t keep = policy_evict_last();
  const int G = a.num_heads / a.num_kv_heads;
  uint32_t n = 0, segs = 0;    // steps and segments begun; step n uses slot n & 1
  uint32_t issued[2] = {0, 0};  // loads of K, of V
  bool ok = true;
  while (ok && sg.next(a)) {
    if (!mbar_wait(&bars[P_QEMPTY], (segs & 1) ^ 1u, a.status)) {
      ok = false;
      break;
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[P_QFULL], Lay::kQBytes);
      for (int p = 0; p < (int)Lay::kPanels; ++p)
        tma_load_3d(smem + Lay::kQ + p * Lay::kQPanel, tmQ, p * 64, sg.h * G, sg.seq0,
                    &bars[P_QFULL]);
    }
    ++segs;
    const int32_t* table = a.block_tables + (int64_t)sg.seq0 * a.max_blocks;
    // Lane i has the row of sub-box i & 3 of the (i / 4)-th of 8 steps from w on.
    int rows = past, w = sg.s0 - 8;
    for (int s = sg.s0; ok && s < sg.s1;) {
      const int unit = unit_of(n, sg.s1 - s);
      if (s + unit > w + 8) {
        w = s;
        const int key = (w + (lane >> 2)) * kTileKeys + (lane & 3) * box;
        rows = past;
        if ((lane & 3) < nsub && key < sg.prefix && w + (lane >> 2) < sg.s1) {
          int phys = table[key >> shift];
          if (phys < 0 || phys >= a.num_blocks) {
            record_error(a.status, KVP_ERR_DEVICE_DATA);
            phys = 0;  // never address a block outside the pool
          }
          rows = (phys << shift) + (key & (a.block_size - 1));
        }
      }
#pragma unroll 1
      for (int i = 0; ok && i < 2 * unit; ++i) {  // K of the unit's steps, then V
        const int kv = i >= unit, u = i - kv * unit;
        const uint32_t slot = (n + u) & 1, par = ((n + u) >> 1 & 1) ^ 1u;
        const int full = (kv == 0 ? P_KFULL : P_VFULL) + slot;
        const int empty = (kv == 0 ? P_KEMPTY : P_VEMPTY) + slot;
        int row[kMaxSub];
#pragma unroll
        for (int k = 0; k < kMaxSub; ++k) row[k] = __shfl_sync(0xffffffffu, rows, (s + u - w) * 4 + k);
        if (!mbar_wait(&bars[empty], par, a.status)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[full], Lay::kSlot);
          uint8_t* dst = smem + (kv == 0 ? Lay::kK + slot * Lay::kPanel : Lay::kV + slot * Lay::kSlot);
          const uint32_t panel = kv == 0 ? 2 * Lay::kPanel : Lay::kPanel;
          const CUtensorMap* map = kv == 0 ? tmK : tmV;
#pragma unroll
          for (int k = 0; k < kMaxSub; ++k)
            if (k < nsub)
              for (int p = 0; p < (int)Lay::kPanels; ++p)
                tma_load_3d_hint(dst + p * panel + k * box * 128, map, p * 64, sg.h, row[k], &bars[full],
                                 keep);
        }
        ++issued[kv];
      }
      s += unit;
      n += unit;
    }
  }
  if (ok) return;  // the MMA thread has waited for every copy
  // After an expired wait: no copy of this CTA is in flight when it exits.
  if (segs) mbar_wait(&bars[P_QFULL], (segs - 1) & 1, a.status);
  for (int kv = 0; kv < 2; ++kv)
    for (uint32_t i = issued[kv] > 2 ? issued[kv] - 2 : 0; i < issued[kv]; ++i)
      mbar_wait(&bars[(kv == 0 ? P_KFULL : P_VFULL) + (i & 1)], (i >> 1) & 1, a.status);
}

// MMAs and commits of a converged warp, by one of its lanes (the same each time).
// A lane that runs alone has its operands in vector registers and moves each to
// the uniform ones that these instructions take: 70 cycles an MMA.
__device__ __forceinline__ void warp_umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t"
      ".reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void warp_umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t"
      ".reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A bounded wait with one outcome for the warp, which stays converged.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}
__device__ __forceinline__ void warp_umma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t"
      ".reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
      "}" ::"r"(smem_u32(bar))
      : "memory");
}

template <int D, bool kFine>
__device__ void prefix_mma(const SharedArgs& a, PrefixSegment sg, uint8_t* smem, uint64_t* bars,
                           uint32_t tbase) {
  using Lay = PrefixLayout<D>;
  const uint32_t idesc_s1 = idesc_bf16_f32(kTileRows, kTileKeys, 0, 0) | a.prefix_negate;
  const uint32_t idesc_s2 = idesc_bf16_f32(kTileRows, 2 * kTileKeys, 0, 0) | a.prefix_negate;
  constexpr uint32_t idesc_o = idesc_bf16_f32(kTileRows, D, 0, 1);
  const uint64_t dq = smem_desc(smem_u32(smem + Lay::kQ), 16, 1024, 2);
  const uint64_t dk0 = smem_desc(smem_u32(smem + Lay::kK), 16, 1024, 2);
  const uint64_t dv0 = smem_desc(smem_u32(smem + Lay::kV), Lay::kPanel, 1024, 2);
  uint32_t n = 0, segs = 0;
  while (sg.next(a)) {
    const int steps = sg.s1 - sg.s0;
    if (!warp_wait(&bars[P_QFULL], segs & 1, a.status)) goto drain;
    for (int j = 0; j < steps;) {
      // S = Q K^T of the unit.  The P that it overwrites have been read: their
      // PV were issued before.
      const int unit = unit_of(n, steps - j);
      for (int u = 0; u < unit; ++u)
        if (!warp_wait(&bars[P_KFULL + ((n + u) & 1)], ((n + u) >> 1) & 1, a.status)) goto drain;
      tc_fence_after();
      const uint64_t dk = dk0 + (((n & 1) * Lay::kPanel) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t in = (kk & 3) * 32;
        warp_umma_ss(tbase + (n & 1) * kTileKeys, dq + (((kk >> 2) * Lay::kQPanel + in) >> 4),
                    dk + (((kk >> 2) * 2 * Lay::kPanel + in) >> 4), unit == 2 ? idesc_s2 : idesc_s1, kk > 0);
      }
      for (int u = 0; u < unit; ++u) {
        warp_umma_commit(&bars[P_SFULL + ((n + u) & 1)]);
        warp_umma_commit(&bars[P_KEMPTY + ((n + u) & 1)]);
      }
      if (j + unit == steps) warp_umma_commit(&bars[P_QEMPTY]);
      for (int u = 0; u < unit; ++u, ++j, ++n) {
        const uint32_t slot = n & 1, par = (n >> 1) & 1;
        if (!warp_wait(&bars[P_VFULL + slot], par, a.status)) goto drain;
        if (j == 0 && segs > 0 && !warp_wait(&bars[P_OFREE], (segs - 1) & 1, a.status)) goto drain;
        if (!warp_wait(&bars[P_PFULL + slot], par, a.status)) goto drain;
        tc_fence_after();
        const uint64_t dv = dv0 + ((slot * Lay::kSlot) >> 4);
#pragma unroll
        for (int kk = 0; kk < (kFine ? 2 : 1) * kTileKeys / 16; ++kk)  // P, then its rest
          warp_umma_ts(tbase + kColO, tbase + slot * kTileKeys + kk * 8,
                       dv + ((kk % (kTileKeys / 16) * 16 * 128) >> 4), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
        warp_umma_commit(&bars[P_VEMPTY + slot]);
        warp_umma_commit(&bars[P_PVDONE]);
        if (j + 1 == steps) warp_umma_commit(&bars[P_ODONE]);
      }
    }
    ++segs;
  }
drain:
  // Every MMA this thread issued has completed before the CTA tears down.
  warp_umma_commit(&bars[P_DRAIN]);
  warp_wait(&bars[P_DRAIN], 0, a.status);
}

template <int D, bool kFine>
__device__ void prefix_softmax(const SharedArgs& a, PrefixSegment sg, uint64_t* bars,
                               uint32_t tbase) {
  constexpr int S = part_stride<D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = threadIdx.x;  // row == TMEM lane
  const int G = a.num_heads / a.num_kv_heads;
  const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
  const uint32_t t_row = tbase + lane_base, o_col = t_row + kColO;
  const float2 scale2 = make_float2(a.prefix_scale_log2, a.prefix_scale_log2);
  uint32_t n = 0, segs = 0;
  while (sg.next(a)) {
    const bool valid = r < sg.nseq * G;
    const long long row0 = (long long)a.num_heads * a.plan.cum_rows[sg.t] + sg.row0;
    float m = -INFINITY, l = 0.f;
    for (int s = sg.s0; s < sg.s1; ++s, ++n) {
      if (!mbar_wait(&bars[P_SFULL + (n & 1)], (n >> 1) & 1, a.status)) return;
      tc_fence_after();
      const uint32_t s_col = t_row + (n & 1) * kTileKeys;
      const int lim = sg.prefix - s * kTileKeys;  // columns < lim exist
      uint32_t v[2][32];
      tmem_ld32(s_col, v[0]);
      tmem_ld32(s_col + 32, v[1]);
      tmem_ld_wait();
      if (lim < kTileKeys) {
#pragma unroll
        for (int i = 0; i < kTileKeys; ++i)
          if (i >= lim) v[i >> 5][i & 31] = 0xff800000u;  // -inf
      }
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kTileKeys; ++i)
        mx4[i & 3] = fmaxf(mx4[i & 3], __uint_as_float(v[i >> 5][i & 31]));
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.prefix_scale_log2;
      // The reference max m moves only when the step's max exceeds it by more
      // than 2^8; O and l keep the same stale reference, so this is exact, and
      // P <= 2^8 is well inside bf16's range.
      float alpha = 1.f;
      bool rescale = false;
      if (mx > m + 8.0f) {
        rescale = s > sg.s0;
        alpha = fast_exp2(m - mx);  // 0 while m is -inf
        m = mx;
      }
      const float mu = m == -INFINITY ? 0.f : m;
      const float2 negm = make_float2(-mu, -mu);
      float2 sum2 = make_float2(0.f, 0.f);
      // P over the S columns, which this thread has read: in bf16, and (kFine)
      // what that leaves of each weight in the slot's other half.
      constexpr int kHalf = kTileKeys / 2, W = kFine ? kHalf / 4 : kHalf;  // columns of a store
#pragma unroll
      for (int c = 0; c < kHalf; c += W) {
        uint32_t w[W], rest[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const int i = c + j;
          const float2 x = make_float2(__uint_as_float(v[i >> 4][(2 * i) & 31]),
                                       __uint_as_float(v[i >> 4][(2 * i + 1) & 31]));
          const float2 y = __ffma2_rn(x, scale2, negm);
          const float2 p = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          sum2 = __fadd2_rn(sum2, p);
          if constexpr (kFine)
            split_bf16x2(p.x, p.y, w[j], rest[j]);
          else
            w[j] = pack_bf16x2(p.x, p.y);
        }
        if constexpr (kFine) {
          tmem_st8(s_col + c, w);
          tmem_st8(s_col + kHalf + c, rest);
        } else {
          tmem_st32(s_col + c, w);
        }
      }
      if (__any_sync(0xffffffffu, rescale)) {
        // The step before is in O.  (One phase back at most: S(n) was issued
        // after PV(n - 2) and is complete.)
        if (!mbar_wait(&bars[P_PVDONE], (n - 1) & 1, a.status)) return;
        tc_fence_after();
        l *= alpha;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_col + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(o_col + c * 32, o);
        }
      }
      l += sum2.x + sum2.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[P_PFULL + (n & 1)]);
    }
    // The segment's partials: O, m, l of the tile's rows.
    if (!mbar_wait(&bars[P_ODONE], segs & 1, a.status)) return;
    ++segs;
    tc_fence_after();
    float* row = valid ? a.prefix_part + (row0 + r) * S : nullptr;
    if (valid) *reinterpret_cast<float2*>(row + D) = make_float2(m, l);
    const int qb = lane & ~3, jq = lane & 3;
    float* qrow[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      qrow[k] = reinterpret_cast<float*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), qb + k));
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      // A quad of lanes exchanges 16-byte chunks so that each of its stores
      // covers 64 contiguous bytes of one row.
      uint32_t v[16], w[4][4];
      tmem_ld16(o_col + c * 16, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i >> 2][i & 3] = v[i];
      quad_transpose16(w, lane);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (qrow[k] != nullptr)
          *reinterpret_cast<uint4*>(qrow[k] + c * 16 + jq * 4) =
              make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[P_OFREE]);
  }
}

template <int D, bool kFine>
__global__ void __maxnreg__(kPrefixRegs)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const SharedArgs a) {
  using Lay = PrefixLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  PrefixSegment sg;
  sg.pos = 0;
  sg.end = 0;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + P_BARS);
  // (A plan of another shape is reported by the own-part kernel.)
  const SharedPrefixStart start = a.plan.prefix_start[blockIdx.x];
  if (threadIdx.x == 4 * 32) {
    for (int i = 0; i < P_BARS; ++i) mbar_init(&bars[i], i == P_PFULL || i == P_PFULL + 1 || i == P_OFREE ? 4 : 1);
    fence_mbar_init();
  }
  if (plan_fits(a)) {
    const PrefixSplit split(*a.plan.head);
    sg.pos = split.begin(blockIdx.x);
    sg.end = min(split.end(blockIdx.x), a.plan.head->prefix_total);
    sg.begin(start);
  }
  if (sg.pos < sg.end && !(smem_u32(smem) & 1023u)) {
    uint32_t tbase = 0;
    if (warp == 4) {
      // The producer has set the barriers up itself and needs no tensor memory:
      // its first loads are under way before the others have theirs.
      __syncwarp();
      asm volatile("bar.arrive 1, %0;" ::"n"(kPrefixThreads) : "memory");
      prefix_producer<D>(a, sg, &tmQ, &tmK, &tmV, smem, bars);
    } else {
      if (warp == 5) {
        tmem_alloc(tmem_slot, kPrefixTmem);
        tmem_relinquish();
      }
      tc_fence_before();
      named_barrier_sync(1, kPrefixThreads);
      tc_fence_after();
      tbase = *tmem_slot;
      if (warp < 4)
        prefix_softmax<D, kFine>(a, sg, bars, tbase);
      else
        prefix_mma<D, kFine>(a, sg, smem, bars, tbase);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tbase, kPrefixTmem);
  } else if (sg.pos < sg.end && threadIdx.x == 0) {
    record_error(a.status, KVP_ERR_DEVICE_DATA);  // the 128-byte swizzle needs a 1 KiB aligned base
  }
  // The grid, launched beside the own-part kernel, must not complete before it.
  // One CTA waits for it, the others leave at once: their SMs take the CTAs
  // that did not fit beside the own-part kernel at first.
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// --------------------------------------------- each sequence's own part
//
// Tokens [prefix, ctx) of every sequence, laid end to end and split evenly
// over one persistent CTA per SM.  A producer warp streams stages of 64 /
// Hkv tokens of one page (K and V, all heads, one tensor copy each) into a
// shared-memory ring; eight consumer warps, each with one kv head and 8
// tokens of a stage, run S = q K^T and O^T += V^T P^T as warp MMAs (M = the G
// query heads of the kv head).  Every segment leaves partials, one row per
// query head and consumer warp of its kv head.  With the fused store, the
// stage that ends at a sequence's last token takes that token's K / V row
// from the new rows, and the producer warp writes them to the cache.
//
// HBM-bound: alone it reads 1.09 GB in 162 us and 2.06 GB in 290 us (6.7 and
// 7.1 TB/s), every byte once where a page has 64 / Hkv tokens or more; of smaller
// pages (16 or 32 tokens with one kv head, 16 with two) a copy brings what lies behind
// the page too, masked: two or four times the bytes.  Four 32 KiB stages beside a prefix CTA's 99 KB
// (three: 2% slower).  The loads are marked evict-first: they are read once and
// would push the prefixes out of L2 (own parts of 512 sequences 171 us without).

constexpr int kOwnWarps = 8;  // consumer warps
constexpr int kOwnThreads = (kOwnWarps + 1) * 32;
constexpr int kOwnRegs = 96;
static_assert(32 * (2 * kPrefixRegs + 3 * kOwnRegs) <= 16384, "registers of a sub-partition");
constexpr int kStageRows = 64;  // tokens x kv heads of a stage

enum : int { F_NEW = 1, F_LAST = 2, F_DONE = 4, F_TAIL = 8 };

struct StageMeta {
  int b, n, flags, pad;
};

template <int D>
struct OwnLayout {
  static constexpr uint32_t kHalf = kStageRows * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kMeta = 2 * kStages * kHalf;
  static constexpr uint32_t kBar = kMeta + kStages * (uint32_t)sizeof(StageMeta);
  static constexpr uint32_t kAlloc = kBar + 2 * kStages * 8;
};
// One CTA of each kernel, or two of the prefix kernel, fit an SM (228 KiB,
// 1 KiB of it per CTA reserved).
static_assert(OwnLayout<128>::kAlloc + PrefixLayout<128>::kAlloc + 2048 <= 228 * 1024, "smem");

template <int D>
__device__ void own_producer(const SharedArgs& a, const SharedAppend& app, const SharedOwnStart& start,
                             long long pos, const long long end, const CUtensorMap* tmK,
                             const CUtensorMap* tmV, uint8_t* smem, StageMeta* meta, uint64_t* full,
                             uint64_t* empty) {
  using Lay = OwnLayout<D>;
  constexpr int RS = Lay::kStages;
  const int lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads, T = kStageRows / Hkv, bs = a.block_size;
  const int shift = __ffs(bs) - 1;  // block_size is a power of two
  uint8_t *ringK = smem, *ringV = smem + RS * Lay::kHalf;
  int s = 0;
  uint32_t ph = 0, issued = 0, issued_ph = 0;
  bool ok = true;
  // Read once: these keys must not push the shared prefixes out of L2.
  const uint64_t once = policy_evict_first();
  if (pos < end) {
    // Lane i knows sequence base + i; the pages of the current window of the
    // current sequence are one per lane, and the next sequence's first window
    // is loaded ahead.
    int base = start.seq, b = base;
    long long seq_end;
    int ctx, own;  // context length; tokens of its own
    auto load_seqs = [&]() {
      const int i = base + lane;
      const bool in = i < a.num_seqs;
      seq_end = in ? a.plan.cum_tokens[i + 1] : 0;
      ctx = in ? a.plan.ctx[i] : 0;
      own = in ? ctx - a.plan.prefix[i] : 0;
    };
    auto load_pages = [&](int seq, int page, int last) {
      return page + lane <= last ? a.block_tables[(int64_t)seq * a.max_blocks + page + lane] : -1;
    };
    // The first sequence comes with the start record; its first pages are under
    // way before the look-ups of the others.
    int ahead, ahead_seq = b;
    {
      const long long c0 = start.seq_end - start.own, p0 = pos > c0 ? pos : c0;
      const long long p1 = end < start.seq_end ? end : start.seq_end;
      ahead = p0 < p1 ? load_pages(b, (start.ctx - (int)(start.seq_end - p0)) >> shift,
                                   (start.ctx - (int)(start.seq_end - p1) - 1) >> shift)
                      : -1;
    }
    load_seqs();
    while (ok && pos < end) {
      if (b - base == 32) {
        base = b;
        load_seqs();
      }
      const long long c1 = __shfl_sync(0xffffffffu, seq_end, b - base);
      const int L = __shfl_sync(0xffffffffu, ctx, b - base);
      const long long c0 = c1 - __shfl_sync(0xffffffffu, own, b - base);  // its first token
      if (pos < c0) pos = c0;
      if (pos >= end) break;
      if (c1 <= pos) {  // no tokens of its own (a padding row)
        ++b;
        continue;
      }
      int t = L - (int)(c1 - pos);
      pos = end < c1 ? end : c1;
      const int t1 = L - (int)(c1 - pos);
      const int last_page = (t1 - 1) >> shift;
      int page0 = t >> shift;
      int pages = ahead_seq == b ? ahead : load_pages(b, page0, last_page);
      ahead_seq = -1;
      if (b + 1 - base < 32 && b + 1 < a.num_seqs) {
        const int L1 = __shfl_sync(0xffffffffu, ctx, b + 1 - base);
        const int o1 = __shfl_sync(0xffffffffu, own, b + 1 - base);
        const long long c2 = __shfl_sync(0xffffffffu, seq_end, b + 1 - base);
        if (o1 > 0 && c2 - o1 < end) {
          const int n1 = L1 - (int)(c2 - (end < c2 ? end : c2));
          ahead = load_pages(b + 1, (L1 - o1) >> shift, (n1 - 1) >> shift);
          ahead_seq = b + 1;
        }
      }
      bool first = true;
      while (t < t1) {
        const int page = t >> shift, off = t & (bs - 1);
        if (page - page0 == 32) {
          page0 = page;
          pages = load_pages(b, page0, last_page);
        }
        int n = bs - off;
        if (n > T) n = T;
        if (n > t1 - t) n = t1 - t;
        int phys = __shfl_sync(0xffffffffu, pages, page - page0);
        if (phys < 0 || phys >= a.num_blocks) {
          if (lane == 0) record_error(a.status, KVP_ERR_DEVICE_DATA);
          phys = 0;  // never address a block outside the pool
        }
        if (!mbar_wait(&empty[s], ph ^ 1u, a.status)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const bool tail = app.k_new != nullptr && t + n == L;
          meta[s] = StageMeta{
              b, n, (first ? F_NEW : 0) | (t + n == t1 ? F_LAST : 0) | (tail ? F_TAIL : 0), 0};
          uint8_t *dk = ringK + s * Lay::kHalf, *dv = ringV + s * Lay::kHalf;
          mbar_arrive_expect_tx(&full[s], 2 * Lay::kHalf);
          const int row = (phys << shift) + off;
          // Rows past n (of the next page, or past the pool) are masked by the consumers.
          tma_load_4d_hint(dk, tmK, 0, row, 0, 0, &full[s], once);
          tma_load_4d_hint(dv, tmV, 0, row, 0, 0, &full[s], once);
        }
        issued |= 1u << s;
        issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
        first = false;
        t += n;
        if (++s == RS) {
          s = 0;
          ph ^= 1u;
        }
      }
      ++b;
    }
  }
  if (ok && mbar_wait(&empty[s], ph ^ 1u, a.status)) {
    if (lane == 0) {
      meta[s].flags = F_DONE;
      mbar_arrive(&full[s]);
    }
  } else {
    // A wait expired: let every copy this CTA issued land before the CTA exits.
    for (int i = 0; i < RS; ++i)
      if (issued >> i & 1u) mbar_wait(&full[i], issued_ph >> i & 1u, a.status);
  }
  __syncwarp();
  if (app.k_new == nullptr) return;
  // The store of the step's new rows: this CTA writes those of sequences
  // blockIdx.x, blockIdx.x + gridDim.x, ...
  const int row_elems = Hkv * D;
  const int64_t slots = a.num_blocks * bs;
  for (int i = blockIdx.x; i < a.num_seqs; i += gridDim.x) {
    const int slot = app.slot_mapping[i];
    if (slot < 0) continue;
    if (slot >= slots) {
      if (lane == 0) record_error(a.status, KVP_ERR_DEVICE_DATA);
      continue;
    }
    const int L = a.plan.ctx[i];
    if (L > 0 && lane == 0) {
      const int lb = (L - 1) / bs;
      const int phys = a.block_tables[(int64_t)i * a.max_blocks + lb];
      if ((int64_t)phys * bs + (L - 1 - lb * bs) != slot) record_error(a.status, KVP_ERR_DEVICE_DATA);
    }
    const uint4* ks = reinterpret_cast<const uint4*>(app.k_new + (int64_t)i * app.k_stride);
    const uint4* vs = reinterpret_cast<const uint4*>(app.v_new + (int64_t)i * app.v_stride);
    uint4* kd = reinterpret_cast<uint4*>(app.k_cache + (int64_t)slot * row_elems);
    uint4* vd = reinterpret_cast<uint4*>(app.v_cache + (int64_t)slot * row_elems);
    for (int j = lane; j < row_elems / 8; j += 32) {
      kd[j] = ks[j];
      vd[j] = vs[j];
    }
  }
}

// Byte offset of 16-byte chunk q of token row `row` in a stage half
// ([head][panel][token][128 bytes], 128-byte swizzle).
__device__ __forceinline__ uint32_t stage_off(uint32_t region, int T, int row, int q) {
  return region + (uint32_t)(((q >> 3) * T + row) * 128 + (((q & 7) ^ (row & 7)) << 4));
}

template <int D, int G>
__device__ void own_consumer(const SharedArgs& a, const SharedAppend& app, uint8_t* smem,
                             const StageMeta* meta, uint64_t* full, uint64_t* empty, int first_seq) {
  using Lay = OwnLayout<D>;
  constexpr int RS = Lay::kStages;
  constexpr int P = D / 64, NQ = D / 8, KS = D / 16, S = part_stride<D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads, NS = kOwnWarps / Hkv, T = kStageRows / Hkv;
  const int g = warp % Hkv, sub = warp / Hkv;
  const int head0 = g * G;
  const int r = lane >> 2, c = lane & 3;
  // S row r is that of head r.  With fine weights rows 4 .. 7 are the heads of rows
  // 0 .. 3 again (there is room: at most two), and the product with V takes the weights
  // in the former and what bf16 leaves of them in the latter, as columns of one MMA.
  constexpr bool kTwice = fine_weights(G);
  const int head = kTwice ? r & 3 : r;
  const bool srow = head < G;  // this thread's S row is a real head
  const uint32_t region = (uint32_t)(g * P * T * 128);
  const int mrow = sub * 8 + (lane & 7), msel = lane >> 3;
  const uint32_t kbase = smem_u32(smem), vbase = kbase + RS * Lay::kHalf;

  uint32_t qa[KS][2];
  float ot[KS][4];
  float m = -INFINITY, l = 0.f;
  int s = 0;
  uint32_t ph = 0;
  int qseq = -1;  // the sequence whose query qa holds
  auto load_q = [&](int b) {
    qseq = b;
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(a.q + (int64_t)b * a.q_stride +
                                                             (int64_t)(head0 + head) * D);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qa[ks][0] = srow ? qrow[ks * 8 + c] : 0u;
      qa[ks][1] = srow ? qrow[ks * 8 + 4 + c] : 0u;
    }
  };
  if (first_seq >= 0) load_q(first_seq);  // while the first keys are on their way
  while (true) {
    if (!mbar_wait(&full[s], ph, a.status)) return;
    const StageMeta md = meta[s];
    if (md.flags & F_DONE) break;
    if (md.flags & F_NEW) {
      if (md.b != qseq) load_q(md.b);
#pragma unroll
      for (int i = 0; i < KS; ++i) ot[i][0] = ot[i][1] = ot[i][2] = ot[i][3] = 0.f;
      m = -INFINITY;
      l = 0.f;
    }
    const uint32_t kst = kbase + s * Lay::kHalf, vst = vbase + s * Lay::kHalf;
    const int nt = md.n - sub * 8;  // this warp's tokens in the stage (<= 0: none)
    bool patched = false;
    if (nt > 0) {
      if ((md.flags & F_TAIL) && (md.n - 1) >> 3 == sub) {
        // The sequence's last token: its row comes from the new rows (the
        // cache slot is written in this launch).  Lanes 0..15 patch K, 16..31 V.
        const int row = md.n - 1, q = lane & 15;
        if (q < NQ) {
          const uint16_t* src = (lane < 16 ? app.k_new + (int64_t)md.b * app.k_stride
                                           : app.v_new + (int64_t)md.b * app.v_stride) +
                                (int64_t)g * D + q * 8;
          const uint4 u = *reinterpret_cast<const uint4*>(src);
          const uint32_t dst = (lane < 16 ? kst : vst) + stage_off(region, T, row, q);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(u.x), "r"(u.y),
                       "r"(u.z), "r"(u.w)
                       : "memory");
        }
        __syncwarp();
        patched = true;
      }
      // S = q K^T for the warp's 8 tokens; two accumulators halve the chain.
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NQ / 4; ++j) {
        uint32_t k0, k1, k2, k3;
        ldsm_x4(kst + stage_off(region, T, mrow, 4 * j + msel), k0, k1, k2, k3);
        mma_k16(sa, qa[2 * j][0], qa[2 * j][1], k0, k1);
        mma_k16(sb, qa[2 * j + 1][0], qa[2 * j + 1][1], k2, k3);
      }
      float x0 = (sa[0] + sb[0]) * a.scale_log2, x1 = (sa[1] + sb[1]) * a.scale_log2;
      if (2 * c >= nt) x0 = -INFINITY;
      if (2 * c + 1 >= nt) x1 = -INFINITY;
      float mx = fmaxf(x0, x1);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const bool grow = mx > m + 8.0f;  // as in the prefix kernel
      if (__any_sync(0xffffffffu, grow)) {
        const float alpha = grow ? fast_exp2(m - mx) : 1.f;
        if (grow) {
          m = mx;
          l *= alpha;
        }
        const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * c);
        const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * c + 4);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          ot[i][0] *= a0;
          ot[i][1] *= a1;
          ot[i][2] *= a0;
          ot[i][3] *= a1;
        }
      }
      const float mu = m == -INFINITY ? 0.f : m;
      const float p0 = fast_exp2(x0 - mu), p1 = fast_exp2(x1 - mu);
      l += p0 + p1;
      uint32_t pb;
      if constexpr (kTwice) {
        uint32_t rest;
        split_bf16x2(p0, p1, pb, rest);
        if (r >= 4) pb = rest;
      } else {
        pb = pack_bf16x2(p0, p1);
      }
      // V rows past the warp's tokens may hold anything: zero them.
      const uint32_t keep = 2 * c >= nt ? 0u : (2 * c + 1 >= nt ? 0x0000ffffu : 0xffffffffu);
#pragma unroll
      for (int j = 0; j < NQ / 4; ++j) {
        uint32_t v0, v1, v2, v3;
        ldsm_x4_t(vst + stage_off(region, T, mrow, 4 * j + msel), v0, v1, v2, v3);
        mma_k8(ot[2 * j], v0 & keep, v1 & keep, pb);
        mma_k8(ot[2 * j + 1], v2 & keep, v3 & keep, pb);
      }
    }
    if (patched) fence_proxy_async_smem();  // generic writes before the next tensor copy
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (++s == RS) {
      s = 0;
      ph ^= 1u;
    }
    if (!(md.flags & F_LAST)) continue;
    // The segment's partials: heads 2c, 2c + 1 of each thread.
    if constexpr (kTwice) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) ot[i][x] += __shfl_xor_sync(0xffffffffu, ot[i][x], 2);
    }
    float lt = l;
    lt += __shfl_xor_sync(0xffffffffu, lt, 1);
    lt += __shfl_xor_sync(0xffffffffu, lt, 2);
    const long long row0 =
        (((long long)md.b + blockIdx.x) * NS + sub) * a.num_heads + head0 + 2 * c;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float mh = __shfl_sync(0xffffffffu, m, 8 * c + 4 * x);
      const float lh = __shfl_sync(0xffffffffu, lt, 8 * c + 4 * x);
      if (2 * c + x >= G) continue;
      float* dst = a.own_part + (row0 + x) * S;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        dst[16 * i + r] = ot[i][x];
        dst[16 * i + r + 8] = ot[i][2 + x];
      }
      if (r == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(mh, lh);
    }
  }
}

template <int D, int G>
__global__ void __maxnreg__(kOwnRegs)
    shared_own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const SharedArgs a, const SharedAppend app) {
  using Lay = OwnLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  StageMeta* meta = reinterpret_cast<StageMeta*>(smem + Lay::kMeta);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* empty = full + Lay::kStages;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    for (int i = 0; i < Lay::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kOwnWarps);
    }
    fence_mbar_init();
  }
  // The call's first kernel: everything before it on the stream is complete
  // from here on.  Only then may the prefix kernel start beside it, so that
  // kernel can rely on the same.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (One round trip for all of these, and for the head that plan_fits looks at.)
  const SharedOwnStart start = a.plan.own_start[blockIdx.x];
  const long long chunk = a.plan.head->own_chunk, total = a.plan.head->own_total;
  if (!plan_fits(a) || (smem_u32(smem) & 1023u)) {
    if (threadIdx.x == 0) record_error(a.status, KVP_ERR_DEVICE_DATA);
    return;
  }
  __syncthreads();
  const long long pos = chunk * blockIdx.x, end = min(pos + chunk, total);
  if ((threadIdx.x >> 5) == kOwnWarps)
    own_producer<D>(a, app, start, pos, end, &tmK, &tmV, smem, meta, full, empty);
  else
    own_consumer<D, G>(a, app, smem, meta, full, empty, pos < end ? start.seq : -1);
}

// ----------------------------------------------------------------- merge
//
// out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p over a row's partials:
// W warps per (sequence, query head), a lane per D / 32 elements.  Launched as
// a programmatic dependent of the prefix kernel: its plan look-ups overlap the
// kernels before it.  Bound by latency: a few parts of 528 bytes a row, from
// L2; 10 us for 16384 rows, 4 us for 1024.

constexpr int kMergeWarps = 8;

// One row (sequence b, query head h) by W warps; `hand` passes the sums of the
// row's warps to the first of them.
template <int D, int W>
__device__ __forceinline__ void merge_row(const SharedArgs& a, int b, int h, int lane, int warp, int wi,
                                          int ns, long long orow, int hg, int st, long long first,
                                          const PrefixSplit& split, long long prow, float4 (*hand)[33]) {
  constexpr int E = D / 32, S = part_stride<D>();
  constexpr int U = 4;  // parts whose loads are in flight together
  float acc[E], M = -INFINITY, den = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  // Prefix parts: one per CTA that steps [first, first + st) reach; each CTA's
  // rows start 128 rows after the one before's.
  int np = 0;
  if (st > 0) {
    const long long p0 = split.cta(first);
    np = (int)(split.cta(first + st - 1) - p0) + 1;
    prow += p0 * kTileRows + hg;
  }
  const int parts = np + ns;
  const float* pp = a.prefix_part + prow * S;
  const float* op = a.own_part + orow * S;
  const long long ostep = (long long)a.num_heads * S;
  // Warp wi of the row takes parts wi, wi + W, ...; every lane has their m and l.
  for (int k0 = wi; k0 < parts; k0 += U * W) {
    float v[U][E], mk[U], lk[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = k0 + i * W;
      mk[i] = -INFINITY;
      lk[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = 0.f;
      if (k < parts) {
        const float* p = k < np ? pp + (long long)k * kTileRows * S : op + (k - np) * ostep;
        const float2 ml = *reinterpret_cast<const float2*>(p + D);
        mk[i] = ml.x;
        lk[i] = ml.y;
        if constexpr (E == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p + lane * E);
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(p + lane * E);
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
    }
    float Mn = M;
#pragma unroll
    for (int i = 0; i < U; ++i) Mn = fmaxf(Mn, mk[i]);
    const float mu = Mn == -INFINITY ? 0.f : Mn;
    const float alpha = fast_exp2(M - mu);
    M = Mn;
    den *= alpha;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float w = fast_exp2(mk[i] - mu);
      den += w * lk[i];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w * v[i][e];
    }
  }
  if constexpr (W > 1) {
    // The row's warps hand their sums to the first of them.
    float4 mine = make_float4(0.f, 0.f, 0.f, 0.f);
    mine.x = acc[0];
    mine.y = acc[1];
    if constexpr (E == 4) {
      mine.z = acc[2];
      mine.w = acc[3];
    }
    hand[warp][lane] = mine;
    if (lane == 0) hand[warp][32] = make_float4(M, den, 0.f, 0.f);
    named_barrier_sync(1 + warp / W, W * 32);
    if (wi == 0) {
#pragma unroll
      for (int j = 1; j < W; ++j) M = fmaxf(M, hand[warp + j][32].x);
      const float mu = M == -INFINITY ? 0.f : M;
      den = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float4 ml = hand[warp + j][32], v = hand[warp + j][lane];
        const float w = fast_exp2(ml.x - mu);
        den += w * ml.y;
        acc[0] += w * v.x;
        acc[1] += w * v.y;
        if constexpr (E == 4) {
          acc[2] += w * v.z;
          acc[3] += w * v.w;
        }
      }
    }
    named_barrier_sync(1 + warp / W, W * 32);  // the buffer is free for the next row
    if (wi != 0) return;
  }
  const float inv = parts > 0 ? 1.f / den : 0.f;
  __nv_bfloat16* out =
      reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)b * a.out_stride + (int64_t)h * D + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

template <int D, int W>
__global__ void __launch_bounds__(kMergeWarps * 32, 4) shared_merge_kernel(const SharedArgs a,
                                                                        int heads) {
  __shared__ float4 hand[W > 1 ? kMergeWarps : 1][33];  // acc of each lane; {M, den, 0, 0}
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wi = warp % W;
  const int Hkv = a.num_kv_heads, G = a.num_heads / Hkv, NS = kOwnWarps / Hkv;
  const int blocks = a.num_heads / heads;  // of a sequence
  const int b = (int)(blockIdx.x / (unsigned)blocks);
  const int h0 = (int)(blockIdx.x % (unsigned)blocks) * heads;
  const bool fits = plan_fits(a);
  int ns = 0;
  long long orow = 0, prow = 0, first = 0;
  PrefixSplit split(1, 1, 1);
  int st = 0, rows_of_item = 0;
  if (fits) {
    const long long k1 = a.plan.cum_tokens[b + 1];
    const int own = a.plan.ctx[b] - a.plan.prefix[b];
    const int t = a.plan.tile_of[b];
    if (own > 0) {  // every sequence with a context has tokens of its own
      const long long chunk = a.plan.head->own_chunk;
      const long long c0 = quotient(k1 - own, chunk), c1 = quotient(k1 - 1, chunk);
      ns = (int)(c1 - c0 + 1) * NS;
      orow = (b + c0) * NS * a.num_heads;
    }
    if (t >= 0) {
      split = PrefixSplit(*a.plan.head);
      first = a.plan.cum_steps[t];
      st = (int)((a.plan.cum_steps[t + 1] - first) / Hkv);
      const int r0 = a.plan.cum_rows[t];
      rows_of_item = (a.plan.cum_rows[t + 1] - r0) * G;
      prow = (long long)Hkv * G * r0 + (long long)(b - a.plan.tile_seq[t]) * G;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (The next call's first kernel may get ready now; it waits for this grid.)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!fits) return;
  for (int h = h0 + warp / W; h < h0 + heads; h += kMergeWarps / W)
    merge_row<D, W>(a, b, h, lane, warp, wi, ns, orow + h, h % G, st, first + (long long)(h / G) * st,
                    split, prow + (long long)(h / G) * rows_of_item, hand);
}

// Sets a split kernel up for its dynamic shared memory, once per device.  The
// split kernels share SMs: without the carve-out an SM is set up with as much
// shared memory as the first of them needs, and the other does not fit.
template <typename... Params>
cudaError_t allow_smem(void (*kernel)(Params...), size_t smem, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);  // (device_info takes devices 0 .. 63)
  if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches a kernel, as a programmatic dependent of the stream's previous one
// when pdl is set.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), unsigned grid, int threads, size_t smem, bool pdl,
                   cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int G>
cudaError_t launch_shared_t(const CUtensorMap& mq, const CUtensorMap& mpk, const CUtensorMap& mpv,
                            const CUtensorMap& mok, const CUtensorMap& mov, const SharedArgs& a,
                            const SharedAppend& app, cudaStream_t stream) {
  static std::atomic<uint64_t> own_set, prefix_set;
  const auto prefix_kernel = shared_prefix_kernel<D, fine_weights(G)>;
  cudaError_t e = allow_smem(shared_own_kernel<D, G>, OwnLayout<D>::kAlloc, &own_set);
  if (e == cudaSuccess) e = allow_smem(prefix_kernel, PrefixLayout<D>::kAlloc, &prefix_set);
  if (e != cudaSuccess) return e;
  e = launch(shared_own_kernel<D, G>, own_ctas(a.sms), kOwnThreads, OwnLayout<D>::kAlloc, true,
                         stream, mok, mov, a, app);
  if (e != cudaSuccess) return e;
  e = launch(prefix_kernel, prefix_ctas(a.sms), kPrefixThreads, PrefixLayout<D>::kAlloc, true,
             stream, mq, mpk, mpv, a);
  if (e != cudaSuccess) return e;
  // Few rows: several warps share a row's parts.  A block takes as many heads
  // of a sequence as leave up to four blocks per SM, all resident at once.
  const long long rows = (long long)a.num_seqs * a.num_heads, warps = 4ll * a.sms * kMergeWarps;
  const int W = rows * 4 <= warps ? 4 : rows * 2 <= warps ? 2 : 1;
  int heads = kMergeWarps / W < a.num_heads ? kMergeWarps / W : a.num_heads;
  while (heads < a.num_heads && rows / heads > 4 * a.sms) heads *= 2;
  const unsigned grid = (unsigned)(rows / heads);
  auto merge = W == 4 ? shared_merge_kernel<D, 4> : W == 2 ? shared_merge_kernel<D, 2> : shared_merge_kernel<D, 1>;
  return launch(merge, grid, kMergeWarps * 32, 0, true, stream, a, heads);
}

}  // namespace

// ------------------------------------------------------------- host side

size_t shared_plan_bytes(int num_seqs, int num_sms) {
  const size_t B = (size_t)num_seqs;
  return (sizeof(SharedPlanHead) + own_ctas(num_sms) * sizeof(SharedOwnStart) +
          prefix_ctas(num_sms) * sizeof(SharedPrefixStart) + 16 * (B + 1) + 4 * (8 * B + 2) + 255) /
         256 * 256;
}

SharedPlan shared_plan_view(void* base, int num_seqs, int num_sms) {
  const size_t B = (size_t)num_seqs;
  SharedPlan p;
  p.head = static_cast<SharedPlanHead*>(base);
  p.own_start = reinterpret_cast<SharedOwnStart*>(p.head + 1);
  p.prefix_start = reinterpret_cast<SharedPrefixStart*>(p.own_start + own_ctas(num_sms));
  p.cum_tokens = reinterpret_cast<long long*>(p.prefix_start + prefix_ctas(num_sms));
  p.cum_steps = p.cum_tokens + B + 1;
  p.ctx = reinterpret_cast<int*>(p.cum_steps + B + 1);
  p.prefix = p.ctx + B;
  p.tile_of = p.prefix + B;
  p.tile_seq = p.tile_of + B;
  p.cum_rows = p.tile_seq + B + 1;
  p.same = p.cum_rows + B + 1;
  p.group_min = p.same + B;
  p.group_seq = p.group_min + B;
  return p;
}

cudaError_t launch_shared_plan(const int32_t* block_tables, int max_blocks, const int32_t* ctx,
                               int num_seqs, int64_t num_blocks, int block_size, int group,
                               int num_kv_heads, int min_shared_len, const SharedPlan& plan,
                               int num_sms, int* status, cudaStream_t stream) {
  const PlanArgs a{block_tables, ctx,   max_blocks,   num_seqs,       num_blocks,
                   block_size,   group, num_kv_heads, own_gap(num_kv_heads), min_shared_len, num_sms,
                   plan,         status};
  // A warp compares one pair of rows at a time: up to 8 CTAs (a portable
  // cluster).  Few sequences: smaller CTAs, whose barriers cost less (64
  // sequences 5.1 us with 256 threads, 6.9 with 1024), as long as there are
  // warps enough (138: 8.1 us with 256 threads, 6.9 with 512, 7.4 with 1024;
  // 512: 9.5 us with 512, 8.9 with 1024).
  const int threads = num_seqs <= 128 ? 256 : num_seqs <= 256 ? 512 : 1024;
  int ctas = 1;
  while (ctas < 8 && ctas * (threads / 32) < num_seqs) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg,
                            threads == 256   ? shared_plan_kernel<256>
                            : threads == 512 ? shared_plan_kernel<512>
                                             : shared_plan_kernel<1024>,
                            a);
}

// Rows of partial results: see chunk_of.
static size_t prefix_rows(int num_seqs, int num_heads, int ctas) {
  return (size_t)num_seqs * num_heads + (size_t)ctas * kTileRows;
}
static size_t own_rows(int num_seqs, int num_heads, int num_kv_heads, int ctas) {
  return ((size_t)num_seqs + ctas) * (kOwnWarps / num_kv_heads) * num_heads;
}

size_t shared_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                              int num_sms) {
  const size_t rows = prefix_rows(num_seqs, num_heads, prefix_ctas(num_sms)) +
                      own_rows(num_seqs, num_heads, num_kv_heads, own_ctas(num_sms));
  return rows * (head_dim + 4) * sizeof(float);
}

cudaError_t launch_decode_shared(const SharedCall& c, const SharedPlan& plan,
                                 const DecodeAppend* app, int num_sms, int* status,
                                 cudaStream_t stream) {
  const int D = c.head_dim, Hkv = c.num_kv_heads, G = c.num_heads / Hkv;
  SharedArgs a;
  a.q = c.q;
  a.q_stride = c.q_stride;
  a.num_blocks = c.num_blocks;
  a.block_size = c.block_size;
  a.block_tables = c.block_tables;
  a.max_blocks = c.max_blocks;
  a.num_seqs = c.num_seqs;
  a.num_heads = c.num_heads;
  a.num_kv_heads = Hkv;
  a.scale_log2 = c.softmax_scale * 1.4426950408889634f;
  // The prefix kernel takes the maximum of a row before it scales it and masks
  // with -inf, so its scale is positive: the sign goes to the matrix product
  // (bit 13 of an instruction descriptor negates A), and 0 becomes a magnitude
  // at which all scores below 10^32 are 0 to 2^-19.
  a.prefix_scale_log2 = std::fmax(std::fabs(a.scale_log2), FLT_MIN);
  a.prefix_negate = a.scale_log2 < 0.f ? 1u << 13 : 0u;
  a.plan = plan;
  a.sms = num_sms;
  a.prefix_part = static_cast<float*>(c.workspace);
  a.own_part = a.prefix_part + prefix_rows(c.num_seqs, c.num_heads, prefix_ctas(num_sms)) * (D + 4);
  a.out = c.out;
  a.out_stride = c.out_stride;
  a.status = status;
  SharedAppend ap{};
  if (app) ap = {app->k, app->v, app->k_stride, app->v_stride, app->slot_mapping, app->k_cache, app->v_cache};
  const int64_t rows = c.num_blocks * c.block_size;
  const int box = c.block_size < kTileKeys ? c.block_size : kTileKeys;
  CUtensorMap mq, mpk, mpv, mok, mov;
  if (!rows_tensor_map(&mq, c.q, c.num_seqs, c.num_heads, D, c.q_stride, G, kTileRows / G) ||
      !rows_tensor_map(&mpk, c.k_cache, rows, Hkv, D, (int64_t)Hkv * D, 1, box) ||
      !rows_tensor_map(&mpv, c.v_cache, rows, Hkv, D, (int64_t)Hkv * D, 1, box) ||
      !stage_tensor_map(&mok, c.k_cache, rows, Hkv, D, kStageRows / Hkv) ||
      !stage_tensor_map(&mov, c.v_cache, rows, Hkv, D, kStageRows / Hkv))
    return cudaErrorInvalidValue;
  auto run = [&](auto d, auto g) {
    return launch_shared_t<decltype(d)::value, decltype(g)::value>(mq, mpk, mpv, mok, mov, a, ap, stream);
  };
  auto with_group = [&](auto d) {
    switch (G) {
      case 1: return run(d, std::integral_constant<int, 1>{});
      case 2: return run(d, std::integral_constant<int, 2>{});
      case 4: return run(d, std::integral_constant<int, 4>{});
      case 8: return run(d, std::integral_constant<int, 8>{});
    }
    return cudaErrorInvalidValue;
  };
  if (D == 128) return with_group(std::integral_constant<int, 128>{});
  if (D == 64) return with_group(std::integral_constant<int, 64>{});
  return cudaErrorInvalidValue;
}

}  // namespace kvp
