// C ABI of the shared-prefix decode and the page operators: argument
// validation and dispatch.  The contract of every entry point is in kvpaged.h.
#include "decode_shared.h"
#include "kvp_internal.h"
#include "pages.h"

namespace {

using kvp::set_last_error;

// Prefix shared without a min_shared_len of the caller's.
constexpr int kDefaultMinShared = 128;
constexpr int kMaxRows = 1 << 20;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

int cuda_error(cudaError_t e, const char* fn) {
  return set_last_error(KVP_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
}

// The checks of an attention call over a planned batch (and, with app, of
// its new rows).
int check_shared(const char* fn, const kvp::SharedCall& c, const void* plan, size_t plan_bytes,
                 size_t workspace_bytes, const kvp::DecodeAppend* app) {
  if (c.num_seqs < 0 || c.num_seqs >= kMaxRows || c.num_blocks <= 0 || c.max_blocks < 0)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (!kvp::decode_supported(c.num_heads, c.num_kv_heads, c.head_dim) ||
      !kvp::prefill_supported(c.num_heads, c.num_kv_heads, c.head_dim, c.block_size))
    return set_last_error(KVP_ERR_UNSUPPORTED,
                          "%s: unsupported heads %d/%d, head_dim %d or block_size %d", fn,
                          c.num_heads, c.num_kv_heads, c.head_dim, c.block_size);
  const int64_t q_row = (int64_t)c.num_heads * c.head_dim, kv_row = (int64_t)c.num_kv_heads * c.head_dim;
  if (c.q_stride < q_row || c.out_stride < q_row ||
      (app && (app->k_stride < kv_row || app->v_stride < kv_row)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: row stride too small", fn);
  if ((int64_t)c.max_blocks * c.block_size > (int64_t)1 << 30)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: context capacity too large", fn);
  if (c.num_blocks >= ((int64_t)1 << 31) / c.block_size)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: pool has 2^31 or more slots", fn);
  if (c.num_seqs == 0) return KVP_OK;
  if (!c.q || !c.k_cache || !c.v_cache || !c.block_tables || !plan || !c.out ||
      (app && (!app->k || !app->v || !app->slot_mapping)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(c.q) || !aligned16(c.k_cache) || !aligned16(c.v_cache) || !aligned16(c.out) ||
      !aligned16(plan) || c.q_stride % 8 || c.out_stride % 8 ||
      (app && (!aligned16(app->k) || !aligned16(app->v) || app->k_stride % 8 || app->v_stride % 8)))
    return set_last_error(KVP_ERR_INVALID_ARG,
                          "%s: q, k, v, caches, plan and out need 16-byte alignment and row strides "
                          "that are multiples of 8 elements",
                          fn);
  int sms;
  int rc = kvp::device_sm_count(&sms);
  if (rc) return rc;
  if (plan_bytes < kvp::shared_plan_bytes(c.num_seqs, sms))
    return set_last_error(KVP_ERR_WORKSPACE, "%s: plan needs %zu bytes (got %zu)", fn,
                          kvp::shared_plan_bytes(c.num_seqs, sms), plan_bytes);
  const size_t need =
      kvp::shared_workspace_bytes(c.num_seqs, c.num_heads, c.num_kv_heads, c.head_dim, sms);
  if (!c.workspace || workspace_bytes < need || !aligned16(c.workspace))
    return set_last_error(KVP_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu)", fn, need,
                          workspace_bytes);
  return KVP_OK;
}

int run_shared(const char* fn, const kvp::SharedCall& c, const void* plan, size_t plan_bytes,
               size_t workspace_bytes, const kvp::DecodeAppend* app, kvp_stream_t stream) {
  int rc = check_shared(fn, c, plan, plan_bytes, workspace_bytes, app);
  if (rc || c.num_seqs == 0) return rc;
  int *status, sms;
  rc = kvp::device_handles(&status, &sms);
  if (rc) return rc;
  const cudaError_t e =
      kvp::launch_decode_shared(c, kvp::shared_plan_view(const_cast<void*>(plan), c.num_seqs, sms), app,
                                sms, status, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

// The checks the page operators share.  rows: the larger of num_rows and
// num_out.
int check_pages(const char* fn, const kvp::PagesArgs& a, const kvp::PagesCache* c, void* workspace,
                size_t workspace_bytes) {
  if (a.num_rows < 0 || a.num_rows >= kMaxRows || a.num_out < 0 || a.num_out >= kMaxRows ||
      a.max_blocks < 0 || a.num_blocks <= 0 || a.block_size <= 0 || a.num_slots < 0)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (a.num_blocks >= (((int64_t)1 << 31) + a.block_size - 1) / a.block_size ||
      a.num_slots >= (int64_t)1 << 31)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: 2^31 or more slots", fn);
  if ((int64_t)a.max_blocks * a.block_size > (int64_t)1 << 30)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: context capacity too large", fn);
  const int rows = a.num_rows > a.num_out ? a.num_rows : a.num_out;
  if (c) {
    if (c->num_planes <= 0 || c->row_elems <= 0)
      return set_last_error(KVP_ERR_INVALID_ARG, "%s: non-positive cache shape", fn);
    if (c->row_elems > (int64_t)1 << 20)
      return set_last_error(KVP_ERR_UNSUPPORTED, "%s: row too long", fn);
    if (c->plane_stride < a.num_blocks * a.block_size * c->row_elems)
      return set_last_error(KVP_ERR_INVALID_ARG, "%s: plane_stride smaller than the pool", fn);
    if (!c->cache) return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  }
  if (!a.ref_counts || !a.out_counts ||
      (a.num_rows > 0 && (!a.context_lens || (a.max_blocks > 0 && !a.block_tables))))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  const size_t need = kvp::pages_workspace_bytes(a.num_blocks, rows);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return set_last_error(KVP_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu)", fn, need,
                          workspace_bytes);
  return KVP_OK;
}

struct Range {
  const void* p;
  size_t bytes;
};

// Outputs must not overlap inputs or one another; same(i, j) allows output i
// to be input j itself.
template <int NI, int NO, typename Same>
int check_overlap(const char* fn, const Range (&in)[NI], const Range (&out)[NO], Same same) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes) &&
          !(same(i, j) && out[i].p == in[j].p))
        return set_last_error(KVP_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return set_last_error(KVP_ERR_INVALID_ARG, "%s: outputs overlap", fn);
  }
  return KVP_OK;
}

size_t ints(int64_t n) { return (size_t)n * sizeof(int32_t); }

}  // namespace

extern "C" {

size_t attn_shared_plan_size(int num_seqs, int num_heads, int num_kv_heads) {
  if (num_seqs < 0 || num_seqs >= kMaxRows || !kvp::decode_supported(num_heads, num_kv_heads, 128)) {
    set_last_error(KVP_ERR_INVALID_ARG, "attn_shared_plan_size: bad shape");
    return 0;
  }
  int sms;
  if (kvp::device_sm_count(&sms)) return 0;
  return kvp::shared_plan_bytes(num_seqs, sms);
}

int attn_shared_plan(const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, int num_seqs, int64_t num_blocks, int block_size,
                     int num_heads, int num_kv_heads, int min_shared_len, void* plan,
                     size_t plan_bytes, kvp_stream_t stream) {
  const char* fn = "attn_shared_plan";
  if (num_seqs < 0 || num_seqs >= kMaxRows || num_blocks <= 0 || max_blocks_per_seq < 0 ||
      min_shared_len < 0)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (!kvp::decode_supported(num_heads, num_kv_heads, 128) ||
      !kvp::prefill_supported(num_heads, num_kv_heads, 128, block_size))
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: unsupported heads %d/%d or block_size %d", fn,
                          num_heads, num_kv_heads, block_size);
  if ((int64_t)max_blocks_per_seq * block_size > (int64_t)1 << 30)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: context capacity too large", fn);
  if (num_seqs == 0) return KVP_OK;
  if (!block_tables || !context_lens || !plan)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(plan))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: plan needs 16-byte alignment", fn);
  int *status, sms;
  int rc = kvp::device_handles(&status, &sms);
  if (rc) return rc;
  if (plan_bytes < kvp::shared_plan_bytes(num_seqs, sms))
    return set_last_error(KVP_ERR_WORKSPACE, "%s: plan needs %zu bytes (got %zu)", fn,
                          kvp::shared_plan_bytes(num_seqs, sms), plan_bytes);
  const cudaError_t e = kvp::launch_shared_plan(
      block_tables, max_blocks_per_seq, context_lens, num_seqs, num_blocks, block_size,
      num_heads / num_kv_heads, num_kv_heads, min_shared_len ? min_shared_len : kDefaultMinShared,
      kvp::shared_plan_view(plan, num_seqs, sms), sms, status, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

size_t attn_decode_shared_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                         int head_dim) {
  if (num_seqs < 0 || num_seqs >= kMaxRows ||
      !kvp::decode_supported(num_heads, num_kv_heads, head_dim)) {
    set_last_error(KVP_ERR_INVALID_ARG, "attn_decode_shared_workspace_size: bad shape");
    return 0;
  }
  int sms;
  if (kvp::device_sm_count(&sms)) return 0;
  return kvp::shared_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, sms);
}

int attn_decode_shared(const kvp_bf16* q, int64_t q_stride_tok, const kvp_bf16* k_cache,
                       const kvp_bf16* v_cache, int64_t num_blocks, int block_size,
                       const int32_t* block_tables, int max_blocks_per_seq, const void* plan,
                       size_t plan_bytes, int num_seqs, int num_heads, int num_kv_heads,
                       int head_dim, float softmax_scale, void* workspace, size_t workspace_bytes,
                       kvp_bf16* out, int64_t out_stride_tok, kvp_stream_t stream) {
  const kvp::SharedCall c{q,          q_stride_tok, k_cache,      v_cache,            num_blocks,
                          block_size, block_tables, max_blocks_per_seq, num_seqs,     num_heads,
                          num_kv_heads, head_dim,   softmax_scale, workspace,         out,
                          out_stride_tok};
  return run_shared("attn_decode_shared", c, plan, plan_bytes, workspace_bytes, nullptr, stream);
}

int attn_decode_shared_append(const kvp_bf16* q, int64_t q_stride_tok, const kvp_bf16* k,
                              const kvp_bf16* v, int64_t k_stride_tok, int64_t v_stride_tok,
                              const int32_t* slot_mapping, kvp_bf16* k_cache, kvp_bf16* v_cache,
                              int64_t num_blocks, int block_size, const int32_t* block_tables,
                              int max_blocks_per_seq, const void* plan, size_t plan_bytes,
                              int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                              float softmax_scale, void* workspace, size_t workspace_bytes,
                              kvp_bf16* out, int64_t out_stride_tok, kvp_stream_t stream) {
  const kvp::SharedCall c{q,          q_stride_tok, k_cache,      v_cache,            num_blocks,
                          block_size, block_tables, max_blocks_per_seq, num_seqs,     num_heads,
                          num_kv_heads, head_dim,   softmax_scale, workspace,         out,
                          out_stride_tok};
  const kvp::DecodeAppend app{k, v, k_stride_tok, v_stride_tok, slot_mapping, k_cache, v_cache};
  return run_shared("attn_decode_shared_append", c, plan, plan_bytes, workspace_bytes, &app, stream);
}

size_t kv_pages_workspace_size(int64_t num_blocks, int num_rows) {
  if (num_blocks <= 0 || num_blocks >= (int64_t)1 << 31 || num_rows < 0 || num_rows >= kMaxRows) {
    set_last_error(KVP_ERR_INVALID_ARG, "kv_pages_workspace_size: bad shape");
    return 0;
  }
  return kvp::pages_workspace_bytes(num_blocks, num_rows);
}

int kv_pages_fork(kvp_bf16* cache, int64_t num_planes, int64_t plane_stride, int64_t num_blocks,
                  int block_size, int64_t row_elems, const int32_t* block_tables,
                  int max_blocks_per_seq, const int32_t* context_lens, int num_rows,
                  const int32_t* ref_counts, const int32_t* parents, int num_out,
                  int32_t* out_tables, int32_t* out_context_lens, int32_t* out_ref_counts,
                  void* workspace, size_t workspace_bytes, kvp_stream_t stream) {
  const char* fn = "kv_pages_fork";
  kvp::PagesArgs a{};
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.ref_counts = ref_counts;
  a.num_rows = num_rows;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.parents = parents;
  a.num_out = num_out;
  a.out_tables = out_tables;
  a.out_lens = out_context_lens;
  a.out_counts = out_ref_counts;
  const kvp::PagesCache c{cache, num_planes, plane_stride, row_elems};
  int rc = check_pages(fn, a, &c, workspace, workspace_bytes);
  if (rc) return rc;
  if (num_out > 0 && (!parents || !out_context_lens || (max_blocks_per_seq > 0 && !out_tables)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  const Range in[] = {{block_tables, ints((int64_t)num_rows * max_blocks_per_seq)},
                      {context_lens, ints(num_rows)},
                      {ref_counts, ints(num_blocks)},
                      {parents, ints(num_out)}};
  const Range out[] = {{out_tables, ints((int64_t)num_out * max_blocks_per_seq)},
                       {out_context_lens, ints(num_out)},
                       {out_ref_counts, ints(num_blocks)},
                       {workspace, workspace_bytes}};
  rc = check_overlap(fn, in, out, [](int, int) { return false; });
  if (rc) return rc;
  a.ws = kvp::pages_workspace(workspace, num_blocks, num_rows > num_out ? num_rows : num_out);
  int sms;
  rc = kvp::device_handles(&a.status, &sms);
  if (rc) return rc;
  const cudaError_t e = kvp::launch_pages_fork(a, c, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

int kv_pages_extend(const int32_t* block_tables, int max_blocks_per_seq,
                    const int32_t* context_lens, int num_rows, const int32_t* ref_counts,
                    int64_t num_blocks, int block_size, const int32_t* new_tokens,
                    int64_t num_slots, int32_t* out_tables, int32_t* out_context_lens,
                    int32_t* out_ref_counts, int32_t* slot_mapping, void* workspace,
                    size_t workspace_bytes, kvp_stream_t stream) {
  const char* fn = "kv_pages_extend";
  kvp::PagesArgs a{};
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.ref_counts = ref_counts;
  a.num_rows = num_rows;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.new_tokens = new_tokens;
  a.num_slots = num_slots;
  a.slot_mapping = slot_mapping;
  a.out_tables = out_tables;
  a.out_lens = out_context_lens;
  a.out_counts = out_ref_counts;
  int rc = check_pages(fn, a, nullptr, workspace, workspace_bytes);
  if (rc) return rc;
  if ((num_rows > 0 && (!new_tokens || !out_context_lens || (max_blocks_per_seq > 0 && !out_tables))) ||
      (num_slots > 0 && !slot_mapping))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  const size_t tables = ints((int64_t)num_rows * max_blocks_per_seq);
  const Range in[] = {{block_tables, tables},
                      {context_lens, ints(num_rows)},
                      {ref_counts, ints(num_blocks)},
                      {new_tokens, ints(num_rows)}};
  const Range out[] = {{out_tables, tables},
                       {out_context_lens, ints(num_rows)},
                       {out_ref_counts, ints(num_blocks)},
                       {slot_mapping, ints(num_slots)},
                       {workspace, workspace_bytes}};
  rc = check_overlap(fn, in, out, [](int i, int j) { return i == j && i < 3; });
  if (rc) return rc;
  a.ws = kvp::pages_workspace(workspace, num_blocks, num_rows);
  int sms;
  rc = kvp::device_handles(&a.status, &sms);
  if (rc) return rc;
  const cudaError_t e = kvp::launch_pages_extend(a, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

int kv_pages_compact(kvp_bf16* cache, int64_t num_planes, int64_t plane_stride, int64_t num_blocks,
                     int block_size, int64_t row_elems, const int32_t* block_tables,
                     int max_blocks_per_seq, const int32_t* context_lens, int num_rows,
                     const int32_t* ref_counts, int32_t* out_tables, int32_t* out_ref_counts,
                     int32_t* places, void* workspace, size_t workspace_bytes,
                     kvp_stream_t stream) {
  const char* fn = "kv_pages_compact";
  kvp::PagesArgs a{};
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.ref_counts = ref_counts;
  a.num_rows = num_rows;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.places = places;
  a.out_tables = out_tables;
  a.out_counts = out_ref_counts;
  const kvp::PagesCache c{cache, num_planes, plane_stride, row_elems};
  int rc = check_pages(fn, a, &c, workspace, workspace_bytes);
  if (rc) return rc;
  if (!places || (num_rows > 0 && max_blocks_per_seq > 0 && !out_tables))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  const size_t tables = ints((int64_t)num_rows * max_blocks_per_seq);
  const Range in[] = {{block_tables, tables},
                      {context_lens, ints(num_rows)},
                      {ref_counts, ints(num_blocks)}};
  const Range out[] = {{out_tables, tables},
                       {out_ref_counts, ints(num_blocks)},
                       {places, ints(num_blocks)},
                       {workspace, workspace_bytes}};
  rc = check_overlap(fn, in, out, [](int, int) { return false; });
  if (rc) return rc;
  a.ws = kvp::pages_workspace(workspace, num_blocks, num_rows);
  int sms;
  rc = kvp::device_handles(&a.status, &sms);
  if (rc) return rc;
  const cudaError_t e = kvp::launch_pages_compact(a, c, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

}  // extern "C"
