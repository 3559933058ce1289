// attn_shared_plan / attn_decode_shared: paged decode of a batch whose
// sequences share leading pages.
#include "decode_shared.h"
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

struct SharedArgs {
  SharedCall c;
  SharedPlan plan;
  const int32_t* slot_mapping;  // fused store: checked against the plan
  float scale_log2;
  int* status;
};

// True if the plan was made for this call's batch and shape.
__device__ __forceinline__ bool plan_fits(const SharedArgs& a) {
  const SharedPlanHead& h = *a.plan.head;
  return h.magic == kPlanMagic && h.num_seqs == a.c.num_seqs &&
         h.group == a.c.num_heads / a.c.num_kv_heads && h.num_kv_heads == a.c.num_kv_heads &&
         h.block_size == a.c.block_size && h.max_blocks == a.c.max_blocks;
}

// One warp per (sequence, query head).
template <int D>
__global__ void __launch_bounds__(128) shared_decode_kernel(const SharedArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)a.c.num_seqs * a.c.num_heads) return;
  const int b = (int)(row / a.c.num_heads), h = (int)(row % a.c.num_heads);
  if (!plan_fits(a)) {
    if (lane == 0) record_error(a.status, KVP_ERR_DEVICE_DATA);
    return;
  }
  const int L = a.plan.ctx[b], bs = a.c.block_size;
  const int64_t row_elems = (int64_t)a.c.num_kv_heads * D;
  const int g = h / (a.c.num_heads / a.c.num_kv_heads);
  if (a.slot_mapping && h == 0 && lane == 0 && L > 0 && a.slot_mapping[b] >= 0) {
    const int lb = (L - 1) / bs;
    const int phys = a.c.block_tables[(int64_t)b * a.c.max_blocks + lb];
    if ((int64_t)phys * bs + (L - 1 - lb * bs) != a.slot_mapping[b])
      record_error(a.status, KVP_ERR_DEVICE_DATA);
  }
  const __nv_bfloat16* q =
      reinterpret_cast<const __nv_bfloat16*>(a.c.q) + (int64_t)b * a.c.q_stride + (int64_t)h * D;
  float qf[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qf[i] = __bfloat162float(q[i * 32 + lane]) * a.scale_log2;
    acc[i] = 0.f;
  }
  int phys = 0, cur = -1;
  for (int t = 0; t < L; ++t) {
    const int lb = t / bs;
    if (lb != cur) {
      cur = lb;
      phys = a.c.block_tables[(int64_t)b * a.c.max_blocks + lb];
      if (phys < 0 || phys >= a.c.num_blocks) {
        if (lane == 0) record_error(a.status, KVP_ERR_DEVICE_DATA);
        phys = 0;
      }
    }
    const int64_t at = ((int64_t)phys * bs + (t - lb * bs)) * row_elems + (int64_t)g * D;
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(a.c.k_cache) + at;
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.c.v_cache) + at;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) x += qf[i] * __bfloat162float(k[i * 32 + lane]);
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    const float mn = fmaxf(m, x);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float alpha = fast_exp2(m - mu), p = fast_exp2(x - mu);
    l = l * alpha + p;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * alpha + p * __bfloat162float(v[i * 32 + lane]);
    m = mn;
  }
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.c.out) + (int64_t)b * a.c.out_stride +
                     (int64_t)h * D;
  const float inv = L > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) o[i * 32 + lane] = __float2bfloat16_rn(acc[i] * inv);
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

size_t shared_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                              int num_sms) {
  (void)num_seqs, (void)num_heads, (void)num_kv_heads, (void)head_dim, (void)num_sms;
  return 256;
}

cudaError_t launch_decode_shared(const SharedCall& c, const SharedPlan& plan,
                                 const DecodeAppend* app, int num_sms, int* status,
                                 cudaStream_t stream) {
  if (app) {
    cudaError_t e = launch_kv_store(app->k, app->v, app->k_stride, app->v_stride, app->slot_mapping,
                                    c.num_seqs, app->k_cache, app->v_cache,
                                    c.num_blocks * c.block_size, c.num_kv_heads * c.head_dim, true,
                                    num_sms, status, stream);
    if (e != cudaSuccess) return e;
  }
  const SharedArgs a{c, plan, app ? app->slot_mapping : nullptr,
                     c.softmax_scale * 1.4426950408889634f, status};
  const unsigned grid = (unsigned)(((int64_t)c.num_seqs * c.num_heads + 3) / 4);
  if (c.head_dim == 128)
    shared_decode_kernel<128><<<grid, 128, 0, stream>>>(a);
  else
    shared_decode_kernel<64><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvp
