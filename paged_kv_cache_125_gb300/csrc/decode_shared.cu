// attn_shared_plan / attn_decode_shared: paged decode of a batch whose
// sequences share leading pages.
#include "decode_shared.h"

#include <type_traits>

#include "kvp_device.cuh"

namespace kvp {
namespace {

constexpr int kPlanMagic = 0x53504c31;
constexpr int kTileRows = 128;  // query rows of a prefix tile
constexpr int kTileKeys = 128;  // keys of a prefix step

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  int max_blocks;
  int num_seqs;
  int64_t num_blocks;
  int block_size;
  int group;         // query heads per kv head
  int num_kv_heads;
  int min_shared;    // tokens
  SharedPlan plan;
  int* status;
};

// Exclusive prefix sum over the block's threads; *total = the sum.
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
  const T s = (T)warp_sums[lane];
  T ws = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) ws += y;
  }
  *total = __shfl_sync(0xffffffffu, ws, 31);
  return __shfl_sync(0xffffffffu, ws - s, warp) + incl - v;
}
static_assert(kPlanThreads == 1024, "block_scan needs 32 warps");

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
// at least one token of its own.
__device__ int shared_pages(const PlanArgs& a, int b, int prev_ctx, int ctx) {
  const int lane = threadIdx.x & 31;
  const int n = prev_ctx > 0 && ctx > 0 ? (min(prev_ctx, ctx) - 1) / a.block_size : 0;
  const int32_t* x = a.block_tables + (int64_t)(b - 1) * a.max_blocks;
  const int32_t* y = x + a.max_blocks;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    bool same = false;
    if (j < n) {
      const int e = x[j];
      same = e == y[j] && e >= 0 && e < a.num_blocks;
    }
    const unsigned diff = ~__ballot_sync(0xffffffffu, same);
    if (diff) return j0 + __ffs(diff) - 1;
  }
  return n;
}

// Sequence b reads its first pages together with sequence b - 1: it shares
// enough of them, and not less than half of what either neighbour shares
// (a page or two that all requests have in common, e.g. a short system
// prompt, must not join groups that share much more among themselves).
__device__ __forceinline__ bool plan_joined(const PlanArgs& a, int b, int same) {
  if (b == 0 || same == 0 || (int64_t)same * a.block_size < a.min_shared) return false;
  const int prev = a.plan.same[b - 1];
  const int next = b + 1 < a.num_seqs ? a.plan.same[b + 1] : 0;
  return 2 * (int64_t)same >= max(prev, next);
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const PlanArgs a) {
  __shared__ long long warp_sums[32];
  const SharedPlan& p = a.plan;
  const int B = a.num_seqs, bs = a.block_size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = warp; b < B; b += kPlanThreads / 32) {
    const int ctx = plan_ctx(a, b);
    const int same = b > 0 ? shared_pages(a, b, plan_ctx(a, b - 1), ctx) : 0;
    if (lane == 0) {
      p.ctx[b] = ctx;
      p.same[b] = same;
      p.group_min[b] = 0x7fffffff;
    }
  }
  __syncthreads();
  // Groups: maximal runs of joined sequences; all of a group read the pages
  // that every one of them shares.
  int groups = 0;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + (int)threadIdx.x;
    const int same = b < B ? p.same[b] : 0;
    const bool joined = b < B && plan_joined(a, b, same);
    int total;
    const int before = block_scan(b < B && !joined ? 1 : 0, warp_sums, &total);
    if (b < B) {
      const int g = groups + before - (joined ? 1 : 0);
      p.tile_of[b] = g;
      if (joined)
        atomicMin(&p.group_min[g], same);
      else
        p.group_seq[g] = b;
    }
    groups += total;
  }
  __syncthreads();
  // Tiles of 128 query rows within a group, and the prefix sums the kernels
  // find their work by.
  const int tile_seqs = kTileRows / a.group;
  int tiles = 0, rows = 0;
  long long steps = 0, tokens = 0;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + (int)threadIdx.x;
    int ctx = 0, prefix = 0;
    bool start = false;
    if (b < B) {
      const int g = p.tile_of[b], m = *(volatile int*)&p.group_min[g];
      ctx = p.ctx[b];
      prefix = m == 0x7fffffff ? 0 : m * bs;
      start = prefix > 0 && (b - p.group_seq[g]) % tile_seqs == 0;
    }
    int total;
    const int t = tiles + block_scan(start ? 1 : 0, warp_sums, &total) + (start ? 1 : 0) - 1;
    tiles += total;
    const int r = rows + block_scan(prefix > 0 ? 1 : 0, warp_sums, &total);
    rows += total;
    const int n = start ? (prefix + kTileKeys - 1) / kTileKeys : 0;
    long long ltotal;
    const long long st = steps + block_scan((long long)n, warp_sums, &ltotal);
    steps += ltotal;
    const long long tok = tokens + block_scan((long long)(ctx - prefix), warp_sums, &ltotal);
    tokens += ltotal;
    if (b < B) {
      p.prefix[b] = prefix;
      p.tile_of[b] = prefix > 0 ? t : -1;
      p.cum_tokens[b] = tok;
      if (start) {
        p.tile_seq[t] = b;
        p.cum_rows[t] = r;
        p.cum_steps[t] = st;
      }
    }
  }
  if (threadIdx.x == 0) {
    p.cum_tokens[B] = tokens;
    p.cum_rows[tiles] = rows;
    p.cum_steps[tiles] = steps;
    SharedPlanHead h;
    h.magic = kPlanMagic;
    h.num_seqs = B;
    h.group = a.group;
    h.num_kv_heads = a.num_kv_heads;
    h.block_size = bs;
    h.max_blocks = a.max_blocks;
    h.num_tiles = tiles;
    h.pad = 0;
    h.steps = steps;
    h.tokens = tokens;
    *p.head = h;
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
  SharedPlan plan;
  float* prefix_part;  // rows of the prefix kernel's segments
  float* own_part;     // rows of the own-part kernel's segments
  int prefix_ctas, own_ctas;
  int tma_per_head;
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
  const SharedPlanHead& h = *a.plan.head;
  return h.magic == kPlanMagic && h.num_seqs == a.num_seqs &&
         h.group == a.num_heads / a.num_kv_heads && h.num_kv_heads == a.num_kv_heads &&
         h.block_size == a.block_size && h.max_blocks == a.max_blocks;
}

// Both split kernels cut their work, laid end to end, into one equal chunk
// per CTA; a chunk's pieces are its segments.  Segment (item i, CTA c) has its
// own rows of partial results: items and CTAs only ever advance together, so
// (rows of the items before i) + c * (rows of an item) is never taken twice.
__device__ __forceinline__ long long chunk_of(long long total, int ctas, int least) {
  const long long c = (total + ctas - 1) / ctas;
  return c < least ? least : c;
}
constexpr int kLeastSteps = 1;    // prefix steps of 128 keys per CTA
constexpr int kLeastTokens = 32;  // own tokens per CTA

// ------------------------------------------------- the shared prefixes
//
// Item: a tile t of up to 128 query rows (128 / G sequences of a group x the G
// query heads of kv head h) against all keys of the group's prefix, taken 128
// at a time ("step").  The items' steps, laid end to end, are split evenly
// over the CTAs; a CTA's pieces ("segments") leave un-normalised partials.
// Per step: S = Q K^T (tcgen05, M128 N128 K = D) -> row maxima and weights in
// registers -> P in tensor memory -> O += P V.  Rows of a group share the
// same keys, so nothing but the last step's ragged end is masked.
//
// 192 threads: warps 0-3 softmax (thread = row), warp 4 TMA producer, warp 5
// tensor memory and MMA issue.  One K and one V slot each: K(j + 1) loads
// while the softmax of step j runs, V(j + 1) while S(j + 1) and its softmax
// do.  Shared and tensor memory and registers are small enough for two CTAs
// per SM (which alternate on the tensor core) or for one beside a CTA of the
// own-part kernel, whose HBM stream it overlaps.

constexpr int kPrefixThreads = 192;

enum : int { P_QFULL, P_QEMPTY, P_KFULL, P_KEMPTY, P_VFULL, P_VEMPTY, P_SFULL, P_PFULL, P_PVDONE,
             P_OFREE, P_DRAIN, P_BARS };

template <int D>
struct PrefixLayout {
  static constexpr uint32_t kPanels = D / 64;
  static constexpr uint32_t kPanelBytes = 128 * 128;
  static constexpr uint32_t kTileBytes = 128 * D * 2;
  static constexpr uint32_t kQ = 0, kK = kTileBytes, kV = 2 * kTileBytes;
  static constexpr uint32_t kBar = 3 * kTileBytes;
  static constexpr uint32_t kAlloc = kBar + P_BARS * 8 + 16;
};
constexpr uint32_t kPrefixTmem = 256;  // S (P over its first half) | O

// The segments of this CTA, one after the other.
struct PrefixSegment {
  long long pos, end;  // flat steps left
  int t;               // current tile
  // the segment
  int h, s0, s1;       // kv head, steps [s0, s1) of the item
  int seq0, nseq;      // the tile's sequences
  int prefix;          // its keys
  long long row0;      // first row of partials

  __device__ bool next(const SharedArgs& a) {
    if (pos >= end) return false;
    const int Hkv = a.num_kv_heads, G = a.num_heads / Hkv;
    const long long c0 = a.plan.cum_steps[t], c1 = a.plan.cum_steps[t + 1];
    const long long st = c1 - c0, rel = pos - Hkv * c0;
    h = (int)(rel / st);
    s0 = (int)(rel - h * st);
    const long long left = end - pos;
    s1 = st - s0 < left ? (int)st : s0 + (int)left;
    const int r0 = a.plan.cum_rows[t];
    nseq = a.plan.cum_rows[t + 1] - r0;
    seq0 = a.plan.tile_seq[t];
    prefix = a.plan.prefix[seq0];
    row0 = (long long)Hkv * G * r0 + (long long)h * nseq * G + (long long)blockIdx.x * kTileRows;
    pos += s1 - s0;
    if (pos == Hkv * c1) ++t;
    return true;
  }
};

template <int D>
__device__ void prefix_producer(const SharedArgs& a, PrefixSegment sg, const CUtensorMap* tmQ,
                                const CUtensorMap* tmK, const CUtensorMap* tmV, uint8_t* smem,
                                uint64_t* bars) {
  using Lay = PrefixLayout<D>;
  const int lane = threadIdx.x & 31;
  const int G = a.num_heads / a.num_kv_heads;
  const int box = a.block_size < kTileKeys ? a.block_size : kTileKeys;
  const int nsub = kTileKeys / box;
  const int past = (int)(a.num_blocks * a.block_size);  // a row past the pool: loads zeros
  if (lane == 0) {
    prefetch_tensormap(tmQ);
    prefetch_tensormap(tmK);
    prefetch_tensormap(tmV);
  }
  uint32_t nq = 0, nk = 0, nv = 0;
  bool ok = true;
  while (ok && sg.next(a)) {
    if (nq > 0 && !mbar_wait(&bars[P_QEMPTY], (nq - 1) & 1, a.status)) break;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[P_QFULL], Lay::kTileBytes);
      for (int p = 0; p < (int)Lay::kPanels; ++p)
        tma_load_3d(smem + Lay::kQ + p * Lay::kPanelBytes, tmQ, p * 64, sg.h * G, sg.seq0,
                    &bars[P_QFULL]);
    }
    ++nq;
    const int32_t* table = a.block_tables + (int64_t)sg.seq0 * a.max_blocks;
    for (int s = sg.s0; s < sg.s1; ++s) {
      // Lane i looks up sub-box i of the step (at most 8).
      int row = past;
      const int key = s * kTileKeys + lane * box;
      if (lane < nsub && key < sg.prefix) {
        int phys = table[key / a.block_size];
        if (phys < 0 || phys >= a.num_blocks) {
          record_error(a.status, KVP_ERR_DEVICE_DATA);
          phys = 0;  // never address a block outside the pool
        }
        row = phys * a.block_size + key % a.block_size;
      }
      int rows[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) rows[i] = __shfl_sync(0xffffffffu, row, i);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint32_t& n = kv == 0 ? nk : nv;
        const int full = kv == 0 ? P_KFULL : P_VFULL, empty = kv == 0 ? P_KEMPTY : P_VEMPTY;
        if (n > 0 && !mbar_wait(&bars[empty], (n - 1) & 1, a.status)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[full], Lay::kTileBytes);
          uint8_t* dst = smem + (kv == 0 ? Lay::kK : Lay::kV);
          const CUtensorMap* map = kv == 0 ? tmK : tmV;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < nsub)
              for (int p = 0; p < (int)Lay::kPanels; ++p)
                tma_load_3d(dst + p * Lay::kPanelBytes + i * box * 128, map, p * 64, sg.h, rows[i],
                            &bars[full]);
        }
        ++n;
      }
      if (!ok) break;
    }
  }
  // No copy of this CTA is in flight when it exits (after an expired wait
  // nobody else may have waited for them).
  if (nq) mbar_wait(&bars[P_QFULL], (nq - 1) & 1, a.status);
  if (nk) mbar_wait(&bars[P_KFULL], (nk - 1) & 1, a.status);
  if (nv) mbar_wait(&bars[P_VFULL], (nv - 1) & 1, a.status);
}

template <int D>
__device__ void prefix_mma(const SharedArgs& a, PrefixSegment sg, uint8_t* smem, uint64_t* bars,
                           uint32_t tbase) {
  using Lay = PrefixLayout<D>;
  constexpr uint32_t idesc_s = idesc_bf16_f32(kTileRows, kTileKeys, 0, 0);
  constexpr uint32_t idesc_o = idesc_bf16_f32(kTileRows, D, 0, 1);
  const uint64_t dq = smem_desc(smem_u32(smem + Lay::kQ), 16, 1024, 2);
  const uint64_t dk = smem_desc(smem_u32(smem + Lay::kK), 16, 1024, 2);
  const uint64_t dv = smem_desc(smem_u32(smem + Lay::kV), Lay::kPanelBytes, 1024, 2);
  const uint32_t ts = tbase, to = tbase + kTileKeys;
  uint32_t n = 0, segs = 0;
  while (sg.next(a)) {
    if (!mbar_wait(&bars[P_QFULL], segs & 1, a.status)) goto drain;
    for (int s = sg.s0; s < sg.s1; ++s, ++n) {
      if (!mbar_wait(&bars[P_KFULL], n & 1, a.status)) goto drain;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * Lay::kPanelBytes + (kk & 3) * 32) >> 4;
        umma_f16_ss(ts, dq + off, dk + off, idesc_s, kk > 0);
      }
      umma_commit(&bars[P_SFULL]);
      umma_commit(&bars[P_KEMPTY]);
      if (s + 1 == sg.s1) umma_commit(&bars[P_QEMPTY]);
      if (!mbar_wait(&bars[P_VFULL], n & 1, a.status)) goto drain;
      if (s == sg.s0 && segs > 0 && !mbar_wait(&bars[P_OFREE], (segs - 1) & 1, a.status)) goto drain;
      if (!mbar_wait(&bars[P_PFULL], n & 1, a.status)) goto drain;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kTileKeys / 16; ++kk)
        umma_f16_ts(to, ts + kk * 8, dv + ((kk * 16 * 128) >> 4), idesc_o,
                    (s > sg.s0 || kk > 0) ? 1u : 0u);
      umma_commit(&bars[P_VEMPTY]);
      if (s + 1 == sg.s1) umma_commit(&bars[P_PVDONE]);
    }
    ++segs;
  }
drain:
  // Every MMA this thread issued has completed before the CTA tears down.
  umma_commit(&bars[P_DRAIN]);
  mbar_wait(&bars[P_DRAIN], 0, a.status);
}

template <int D>
__device__ void prefix_softmax(const SharedArgs& a, PrefixSegment sg, uint64_t* bars,
                               uint32_t tbase) {
  constexpr int S = part_stride<D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = threadIdx.x;  // row == TMEM lane
  const int G = a.num_heads / a.num_kv_heads;
  const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
  const uint32_t s_col = tbase + lane_base, o_col = s_col + kTileKeys;
  const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
  uint32_t n = 0, segs = 0;
  while (sg.next(a)) {
    float m = -INFINITY, l = 0.f;
    for (int s = sg.s0; s < sg.s1; ++s, ++n) {
      if (!mbar_wait(&bars[P_SFULL], n & 1, a.status)) return;
      tc_fence_after();
      const int lim = sg.prefix - s * kTileKeys;  // columns < lim exist
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < kTileKeys / 64; ++c) {
        uint32_t v0[32], v1[32];
        tmem_ld32(s_col + c * 64, v0);
        tmem_ld32(s_col + c * 64 + 32, v1);
        tmem_ld_wait();
        if (lim >= kTileKeys) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            mx = fmaxf(mx, fmaxf(__uint_as_float(v0[i]), __uint_as_float(v1[i])));
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (c * 64 + i < lim) mx = fmaxf(mx, __uint_as_float(v0[i]));
            if (c * 64 + 32 + i < lim) mx = fmaxf(mx, __uint_as_float(v1[i]));
          }
        }
      }
      mx *= a.scale_log2;
      // The reference max m moves only when the step's max exceeds it by more
      // than 2^8; O and l keep the same stale reference, so this is exact, and
      // P <= 2^8 is well inside bf16's range.  S(j) complete implies that PV(j
      // - 1) is (it was issued earlier): O may be rescaled here.
      float alpha = 1.f;
      bool rescale = false;
      if (mx > m + 8.0f) {
        rescale = s > sg.s0;
        alpha = fast_exp2(m - mx);  // 0 while m is -inf
        m = mx;
      }
      if (__any_sync(0xffffffffu, rescale)) {
        l *= alpha;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(o_col + c * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tmem_st32(o_col + c * 32, v);
        }
      }
      const float mu = m == -INFINITY ? 0.f : m;
      const float2 negm = make_float2(-mu, -mu);
      float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kTileKeys / 64; ++c) {
        uint32_t v[2][32], w[32];
        tmem_ld32(s_col + c * 64, v[0]);
        tmem_ld32(s_col + c * 64 + 32, v[1]);
        tmem_ld_wait();
        if (lim < kTileKeys) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (c * 64 + i >= lim) v[i >> 5][i & 31] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 x = make_float2(__uint_as_float(v[i >> 4][(2 * i) & 31]),
                                       __uint_as_float(v[i >> 4][(2 * i + 1) & 31]));
          const float2 y = __ffma2_rn(x, scale2, negm);
          const float2 p = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          sum2 = __fadd2_rn(sum2, p);
          w[i] = pack_bf16x2(p.x, p.y);
        }
        // P over S columns that this thread has read already.
        tmem_st32(s_col + c * 32, w);
      }
      l += sum2.x + sum2.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[P_PFULL]);
    }
    // The segment's partials: O, m, l of the tile's rows.
    if (!mbar_wait(&bars[P_PVDONE], segs & 1, a.status)) return;
    ++segs;
    tc_fence_after();
    const bool valid = r < sg.nseq * G;
    float* row = valid ? a.prefix_part + (sg.row0 + r) * S : nullptr;
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

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 2)
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
  sg.t = 0;
  // (A plan of another shape is reported by the own-part kernel.)
  if (plan_fits(a)) {
    const long long total = a.num_kv_heads * a.plan.head->steps;
    const long long chunk = chunk_of(total, gridDim.x, kLeastSteps);
    sg.pos = chunk * blockIdx.x;
    sg.end = sg.pos + chunk < total ? sg.pos + chunk : total;
  }
  if (sg.pos < sg.end && !(smem_u32(smem) & 1023u)) {
    // The tile that holds the first step: the last one that starts at or before it.
    const int tiles = a.plan.head->num_tiles;
    for (int t0 = 0; t0 < tiles; t0 += kPrefixThreads) {
      const int t = t0 + (int)threadIdx.x;
      sg.t += __syncthreads_count(t < tiles && a.num_kv_heads * a.plan.cum_steps[t] <= sg.pos);
    }
    --sg.t;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + P_BARS);
    if (threadIdx.x == 0) {
      for (int i = 0; i < P_BARS; ++i) mbar_init(&bars[i], i == P_PFULL || i == P_OFREE ? 4 : 1);
      fence_mbar_init();
    }
    if (warp == 5) {
      tmem_alloc(tmem_slot, kPrefixTmem);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    if (warp == 4)
      prefix_producer<D>(a, sg, &tmQ, &tmK, &tmV, smem, bars);
    else if (warp < 4)
      prefix_softmax<D>(a, sg, bars, tbase);
    else if ((threadIdx.x & 31) == 0)
      prefix_mma<D>(a, sg, smem, bars, tbase);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tbase, kPrefixTmem);
  } else if (sg.pos < sg.end && threadIdx.x == 0) {
    record_error(a.status, KVP_ERR_DEVICE_DATA);  // the 128-byte swizzle needs a 1 KiB aligned base
  }
  // Launched beside the own-part kernel: do not complete before it.
  if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
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

constexpr int kOwnWarps = 8;  // consumer warps
constexpr int kOwnThreads = (kOwnWarps + 1) * 32;
constexpr int kStageRows = 64;  // tokens x kv heads of a stage

enum : int { F_NEW = 1, F_LAST = 2, F_DONE = 4, F_TAIL = 8 };

struct StageMeta {
  int b, n, flags, pad;
};

template <int D>
struct OwnLayout {
  static constexpr uint32_t kHalf = kStageRows * D * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kMeta = 2 * kStages * kHalf;
  static constexpr uint32_t kBar = kMeta + kStages * (uint32_t)sizeof(StageMeta);
  static constexpr uint32_t kAlloc = kBar + 2 * kStages * 8;
};
// One CTA of each kernel, or two of the prefix kernel, fit an SM (228 KiB,
// 1 KiB of it per CTA reserved).
static_assert(OwnLayout<128>::kAlloc + PrefixLayout<128>::kAlloc + 2048 <= 228 * 1024, "smem");
static_assert(2 * PrefixLayout<128>::kAlloc + 2048 <= 228 * 1024, "smem");

// Last index i of the non-decreasing v[0 .. n) with v[i] <= x (v[0] <= x), by
// one warp: 32 probes a round.
__device__ int last_at_most(const long long* v, int n, long long x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < hi && v[i] <= x);
    const int k = 31 - __clz(le);  // v is sorted: lanes 0 .. k
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

template <int D>
__device__ void own_producer(const SharedArgs& a, const SharedAppend& app, const CUtensorMap* tmK,
                             const CUtensorMap* tmV, uint8_t* smem, StageMeta* meta,
                             uint64_t* full, uint64_t* empty) {
  using Lay = OwnLayout<D>;
  constexpr int RS = Lay::kStages;
  const int lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads, T = kStageRows / Hkv, bs = a.block_size;
  const long long total = a.plan.head->tokens;
  const long long chunk = chunk_of(total, gridDim.x, kLeastTokens);
  long long pos = chunk * blockIdx.x;
  const long long end = pos + chunk < total ? pos + chunk : total;
  int b = pos < end ? last_at_most(a.plan.cum_tokens, a.num_seqs, pos) : 0;
  uint8_t *ringK = smem, *ringV = smem + RS * Lay::kHalf;
  if (lane == 0) {
    prefetch_tensormap(tmK);
    prefetch_tensormap(tmV);
    int s = 0;
    uint32_t ph = 0, issued = 0, issued_ph = 0;
    bool ok = true;
    for (; ok && pos < end; ++b) {
      const long long c0 = a.plan.cum_tokens[b], c1 = a.plan.cum_tokens[b + 1];
      if (c1 <= pos) continue;
      const int start = a.plan.prefix[b], ctx = a.plan.ctx[b];
      int t = start + (int)(pos - c0);
      const int t1 = start + (int)((end < c1 ? end : c1) - c0);
      pos = end < c1 ? end : c1;
      bool first = true;
      int page = -1, phys = 0;
      while (t < t1) {
        const int bi = t / bs, off = t - bi * bs;
        int n = bs - off;
        if (n > T) n = T;
        if (n > t1 - t) n = t1 - t;
        if (bi != page) {
          page = bi;
          phys = a.block_tables[(int64_t)b * a.max_blocks + bi];
          if (phys < 0 || phys >= a.num_blocks) {
            record_error(a.status, KVP_ERR_DEVICE_DATA);
            phys = 0;  // never address a block outside the pool
          }
        }
        if (!mbar_wait(&empty[s], ph ^ 1u, a.status)) {
          ok = false;
          break;
        }
        const bool tail = app.k_new != nullptr && t + n == ctx;
        meta[s] = StageMeta{b, n, (first ? F_NEW : 0) | (t + n == t1 ? F_LAST : 0) | (tail ? F_TAIL : 0), 0};
        uint8_t *dk = ringK + s * Lay::kHalf, *dv = ringV + s * Lay::kHalf;
        mbar_arrive_expect_tx(&full[s], 2 * Lay::kHalf);
        const int row = phys * bs + off;
        // Rows past n (of the next page, or past the pool) are masked by the consumers.
        if (!a.tma_per_head) {
          tma_load_4d(dk, tmK, 0, row, 0, 0, &full[s]);
          tma_load_4d(dv, tmV, 0, row, 0, 0, &full[s]);
        } else {
          for (int h = 0; h < Hkv; ++h)
            for (int p = 0; p < D / 64; ++p) {
              const uint32_t at = (uint32_t)((h * (D / 64) + p) * T * 128);
              tma_load_3d(dk + at, tmK, p * 64, h, row, &full[s]);
              tma_load_3d(dv + at, tmV, p * 64, h, row, &full[s]);
            }
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
    }
    if (ok && mbar_wait(&empty[s], ph ^ 1u, a.status)) {
      meta[s].flags = F_DONE;
      mbar_arrive(&full[s]);
    } else {
      // A wait expired: let every copy this CTA issued land before the CTA exits.
      for (int i = 0; i < RS; ++i)
        if (issued >> i & 1u) mbar_wait(&full[i], issued_ph >> i & 1u, a.status);
    }
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
                             const StageMeta* meta, uint64_t* full, uint64_t* empty) {
  using Lay = OwnLayout<D>;
  constexpr int RS = Lay::kStages;
  constexpr int P = D / 64, NQ = D / 8, KS = D / 16, S = part_stride<D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads, NS = kOwnWarps / Hkv, T = kStageRows / Hkv;
  const int g = warp % Hkv, sub = warp / Hkv;
  const int head0 = g * G;
  const int r = lane >> 2, c = lane & 3;
  const bool srow = r < G;  // this thread's S row is a real head
  const uint32_t region = (uint32_t)(g * P * T * 128);
  const int mrow = sub * 8 + (lane & 7), msel = lane >> 3;
  const uint32_t kbase = smem_u32(smem), vbase = kbase + RS * Lay::kHalf;

  uint32_t qa[KS][2];
  float ot[KS][4];
  float m = -INFINITY, l = 0.f;
  int s = 0;
  uint32_t ph = 0;
  while (true) {
    if (!mbar_wait(&full[s], ph, a.status)) return;
    const StageMeta md = meta[s];
    if (md.flags & F_DONE) break;
    if (md.flags & F_NEW) {
      const uint32_t* qrow = reinterpret_cast<const uint32_t*>(a.q + (int64_t)md.b * a.q_stride +
                                                               (int64_t)(head0 + r) * D);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qa[ks][0] = srow ? qrow[ks * 8 + c] : 0u;
        qa[ks][1] = srow ? qrow[ks * 8 + 4 + c] : 0u;
      }
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
      const uint32_t pb = pack_bf16x2(p0, p1);
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
__global__ void __launch_bounds__(kOwnThreads, 2)
    shared_own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const SharedArgs a, const SharedAppend app) {
  using Lay = OwnLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  StageMeta* meta = reinterpret_cast<StageMeta*>(smem + Lay::kMeta);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* empty = full + Lay::kStages;
  // The prefix kernel may start beside this one.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!plan_fits(a) || (smem_u32(smem) & 1023u)) {
    if (threadIdx.x == 0) record_error(a.status, KVP_ERR_DEVICE_DATA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kOwnWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if ((threadIdx.x >> 5) == kOwnWarps)
    own_producer<D>(a, app, &tmK, &tmV, smem, meta, full, empty);
  else
    own_consumer<D, G>(a, app, smem, meta, full, empty);
}

// ----------------------------------------------------------------- merge
//
// out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p over a row's partials:
// one warp per (sequence, query head), a lane per D / 32 elements.  Launched
// as a programmatic dependent of the prefix kernel: its plan look-ups overlap
// the kernels before it.

constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(const SharedArgs a) {
  constexpr int E = D / 32, S = part_stride<D>();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const bool real = row < (long long)a.num_seqs * a.num_heads && plan_fits(a);
  int b = 0, h = 0, np = 0, ns = 0;
  long long prow = 0, orow = 0;  // first part's row; parts of a kind are a fixed distance apart
  const int Hkv = a.num_kv_heads, G = a.num_heads / Hkv, NS = kOwnWarps / Hkv;
  bool some = false;
  if (real) {
    b = (int)(row / a.num_heads);
    h = (int)(row - (long long)b * a.num_heads);
    const int g = h / G;
    some = a.plan.ctx[b] > 0;
    if (some) {
      const long long chunk = chunk_of(a.plan.head->tokens, a.own_ctas, kLeastTokens);
      const long long c0 = a.plan.cum_tokens[b] / chunk, c1 = (a.plan.cum_tokens[b + 1] - 1) / chunk;
      ns = (int)(c1 - c0 + 1) * NS;
      orow = (b + c0) * NS * a.num_heads + h;
      const int t = a.plan.tile_of[b];
      if (t >= 0) {
        const long long pchunk = chunk_of(Hkv * a.plan.head->steps, a.prefix_ctas, kLeastSteps);
        const long long s0 = a.plan.cum_steps[t], st = a.plan.cum_steps[t + 1] - s0;
        const long long first = Hkv * s0 + g * st;
        const long long p0 = first / pchunk, p1 = (first + st - 1) / pchunk;
        const int r0 = a.plan.cum_rows[t], n = a.plan.cum_rows[t + 1] - r0;
        np = (int)(p1 - p0 + 1);
        prow = (long long)Hkv * G * r0 + (long long)g * n * G + p0 * kTileRows +
               (long long)(b - a.plan.tile_seq[t]) * G + h % G;
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!real) return;
  __nv_bfloat16* out =
      reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)b * a.out_stride + (int64_t)h * D + lane * E;
  float acc[E], M = -INFINITY, den = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (some) {
    const int parts = np + ns;
    for (int k0 = 0; k0 < parts; k0 += 32) {
      // Lane k has part k0 + k: its address, m and l.
      const int k = k0 + lane;
      const float* mine = nullptr;
      float mk = -INFINITY, lk = 0.f;
      if (k < parts) {
        mine = k < np ? a.prefix_part + (prow + (long long)k * kTileRows) * S
                      : a.own_part + (orow + (long long)(k - np) * a.num_heads) * S;
        const float2 ml = *reinterpret_cast<const float2*>(mine + D);
        mk = ml.x;
        lk = ml.y;
      }
      float mx = mk;
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float Mn = fmaxf(M, mx);
      const float mu = Mn == -INFINITY ? 0.f : Mn;
      const float alpha = fast_exp2(M - mu), w = fast_exp2(mk - mu);
      M = Mn;
      float lw = w * lk;
#pragma unroll
      for (int o = 16; o; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
      den = den * alpha + lw;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= alpha;
      const int n = min(32, parts - k0);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float* p = reinterpret_cast<const float*>(
                             __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), i)) +
                         lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(p);
          acc[0] += wi * v.x;
          acc[1] += wi * v.y;
          acc[2] += wi * v.z;
          acc[3] += wi * v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(p);
          acc[0] += wi * v.x;
          acc[1] += wi * v.y;
        }
      }
    }
    const float inv = 1.f / den;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= inv;
  }
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
  else
    *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(acc[0], acc[1]);
}

// Launches a kernel, as a programmatic dependent of the stream's previous one
// when pdl is set.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), unsigned grid, int threads, size_t smem, bool pdl,
                   cudaStream_t stream, Args... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
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
  cudaError_t e = launch(shared_own_kernel<D, G>, a.own_ctas, kOwnThreads, OwnLayout<D>::kAlloc, false,
                         stream, mok, mov, a, app);
  if (e != cudaSuccess) return e;
  e = launch(shared_prefix_kernel<D>, a.prefix_ctas, kPrefixThreads, PrefixLayout<D>::kAlloc, true,
             stream, mq, mpk, mpv, a);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.num_seqs * a.num_heads;
  return launch(shared_merge_kernel<D>, (unsigned)((rows + kMergeWarps - 1) / kMergeWarps),
                kMergeWarps * 32, 0, true, stream, a);
}

}  // namespace

// ------------------------------------------------------------- host side

size_t shared_plan_bytes(int num_seqs) {
  const size_t B = (size_t)num_seqs;
  return (sizeof(SharedPlanHead) + 16 * (B + 1) + 4 * (8 * B + 2) + 255) / 256 * 256;
}

SharedPlan shared_plan_view(void* base, int num_seqs) {
  const size_t B = (size_t)num_seqs;
  SharedPlan p;
  p.head = static_cast<SharedPlanHead*>(base);
  p.cum_tokens = reinterpret_cast<long long*>(p.head + 1);
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
                               int* status, cudaStream_t stream) {
  const PlanArgs a{block_tables, ctx,   max_blocks,   num_seqs,       num_blocks,
                   block_size,   group, num_kv_heads, min_shared_len, plan,
                   status};
  shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
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
  const size_t rows = prefix_rows(num_seqs, num_heads, 2 * num_sms) +
                      own_rows(num_seqs, num_heads, num_kv_heads, num_sms);
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
  a.plan = plan;
  a.prefix_ctas = 2 * num_sms;
  a.own_ctas = num_sms;
  a.prefix_part = static_cast<float*>(c.workspace);
  a.own_part = a.prefix_part + prefix_rows(c.num_seqs, c.num_heads, a.prefix_ctas) * (D + 4);
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
      !stage_tensor_maps(c.k_cache, c.v_cache, rows, Hkv, D, kStageRows / Hkv, &mok, &mov,
                         &a.tma_per_head))
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
