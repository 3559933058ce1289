// C ABI of rotary positions and the 8-bit cache: argument validation and
// dispatch.  The contract of every entry point is in kvpaged.h.
#include <cmath>

#include "kvp_internal.h"
#include "quant.h"

namespace {

using kvp::set_last_error;

constexpr int kMaxScaleTokens = 256;
constexpr int kMaxHeads = 1 << 16;
constexpr double kTwoPi = 6.283185307179586476925;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool power_of_two(int x) { return x > 0 && (x & (x - 1)) == 0; }

int cuda_error(cudaError_t e, const char* fn) {
  return set_last_error(KVP_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
}

int log2_of(int x) {
  int s = 0;
  while (1 << s < x) ++s;
  return s;
}

// Shape of an 8-bit cache.
int check_cache_shape(const char* fn, int format, int64_t num_blocks, int block_size, int scale_tokens,
                      int num_kv_heads, int head_dim) {
  if (num_blocks <= 0 || block_size <= 0 || scale_tokens <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: non-positive cache shape", fn);
  if (format != KVP_E4M3 && format != KVP_INT8)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: unknown format %d", fn, format);
  if (head_dim != 64 && head_dim != 128)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: unsupported head_dim %d", fn, head_dim);
  if (!power_of_two(scale_tokens) || scale_tokens > kMaxScaleTokens || block_size % scale_tokens)
    return set_last_error(KVP_ERR_UNSUPPORTED,
                          "%s: scale_tokens %d is no power of two up to %d that divides block_size %d", fn,
                          scale_tokens, kMaxScaleTokens, block_size);
  if (num_kv_heads > kMaxHeads / 128)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: too many kv heads", fn);
  if (num_blocks >= ((int64_t)1 << 31) / block_size)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: pool has 2^31 or more slots", fn);
  return KVP_OK;
}

int check_cache_pointers(const char* fn, const kvp::QuantCache& c) {
  if (!c.k || !c.v || !c.k_scales || !c.v_scales)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(c.k) || !aligned16(c.v) || !aligned16(c.k_scales) || !aligned16(c.v_scales))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: caches and scales need 16-byte alignment", fn);
  return KVP_OK;
}

kvp::QuantCache cache_of(const void* k, const void* v, const float* ks, const float* vs, int format,
                         int64_t num_blocks, int block_size, int scale_tokens, int num_kv_heads, int head_dim) {
  return {static_cast<uint8_t*>(const_cast<void*>(k)),
          static_cast<uint8_t*>(const_cast<void*>(v)),
          const_cast<float*>(ks),
          const_cast<float*>(vs),
          format,
          num_blocks,
          block_size,
          log2_of(scale_tokens),
          num_kv_heads,
          head_dim};
}

// Rotary arguments and the rows they apply to, without the pointers.
int check_rope_shape(const char* fn, int64_t num_tokens, int rotary_dim, int num_heads, int num_kv_heads,
                     int head_dim, int64_t q_stride, int64_t q_out_stride, int64_t k_stride,
                     int64_t k_out_stride) {
  if (num_tokens < 0 || num_heads < 0 || num_kv_heads < 0 || num_heads + num_kv_heads == 0 || head_dim <= 0)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (num_heads > kMaxHeads || num_kv_heads > kMaxHeads || head_dim > 1024 || num_tokens >= (int64_t)1 << 31)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: row too long or too many tokens", fn);
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: rotary_dim %d is not even or not in 2 .. head_dim", fn,
                          rotary_dim);
  const int64_t q_row = (int64_t)num_heads * head_dim, k_row = (int64_t)num_kv_heads * head_dim;
  if (q_stride < q_row || q_out_stride < q_row || k_stride < k_row || k_out_stride < k_row)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: row stride too small", fn);
  return KVP_OK;
}

int check_store_rows(const char* fn, const kvp::QuantStoreRows& r, int num_kv_heads, int head_dim) {
  if (r.num_tokens < 0) return set_last_error(KVP_ERR_INVALID_ARG, "%s: num_tokens < 0", fn);
  if (r.num_tokens >= (int64_t)1 << 31)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: too many tokens", fn);
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (r.k_stride < row || r.v_stride < row)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: row stride too small", fn);
  if (r.num_tokens == 0) return KVP_OK;
  if (!r.k || !r.v || !r.slots) return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(r.k) || !aligned16(r.v) || r.k_stride % 8 || r.v_stride % 8)
    return set_last_error(KVP_ERR_INVALID_ARG,
                          "%s: k and v need 16-byte alignment and row strides that are multiples of 8 elements",
                          fn);
  return KVP_OK;
}

}  // namespace

extern "C" {

int attn_rope_freqs(int rotary_dim, double base, int scaling, double factor, double original_len, double low,
                    double high, uint64_t* freqs, float* magnitude) {
  const char* fn = "attn_rope_freqs";
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 1024)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: rotary_dim %d is not even or not in 2 .. 1024", fn, rotary_dim);
  if (!(base > 1) || !std::isfinite(base))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: base must be above 1", fn);
  if (scaling < KVP_ROPE_NONE || scaling > KVP_ROPE_WAVELENGTH)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: unknown scaling %d", fn, scaling);
  if (scaling != KVP_ROPE_NONE && (!(factor >= 1) || !std::isfinite(factor)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: factor must be 1 or more", fn);
  const bool by_turns = scaling == KVP_ROPE_YARN || scaling == KVP_ROPE_WAVELENGTH;
  if (by_turns && (!(original_len >= 1) || !std::isfinite(original_len) || !(low > 0) || !(high > low) ||
                   !std::isfinite(high)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: original_len must be 1 or more, and 0 < low < high", fn);
  if (!freqs || !magnitude) return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  const int pairs = rotary_dim / 2;
  if (scaling == KVP_ROPE_NTK && rotary_dim > 2)
    base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
  // The pair that turns `turns` times over the original length.
  auto pair_of = [&](double turns) {
    return rotary_dim * std::log(original_len / (turns * kTwoPi)) / (2 * std::log(base));
  };
  double from = 0, to = 1;
  if (scaling == KVP_ROPE_YARN) {
    from = std::fmax(0, std::floor(pair_of(high)));
    to = std::fmin(rotary_dim - 1, std::ceil(pair_of(low)));
  }
  for (int i = 0; i < pairs; ++i) {
    double w = std::pow(base, -2.0 * i / rotary_dim);
    double stretched = 0;  // share of the pair's angle that is divided by the factor
    if (scaling == KVP_ROPE_LINEAR) stretched = 1;
    if (scaling == KVP_ROPE_YARN) stretched = (i - from) / std::fmax(to - from, 0.001);
    if (scaling == KVP_ROPE_WAVELENGTH) stretched = 1 - (original_len * w / kTwoPi - low) / (high - low);
    stretched = std::fmin(1, std::fmax(0, stretched));
    if (stretched > 0) w = w * (1 - stretched) + w / factor * stretched;
    freqs[i] = (uint64_t)std::ldexp(w / kTwoPi, 64);  // w <= 1: below 2^62
  }
  *magnitude = scaling == KVP_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1) : 1.f;
  return KVP_OK;
}

int attn_rope(const kvp_bf16* q, int64_t q_stride_tok, const kvp_bf16* k, int64_t k_stride_tok,
              const int64_t* positions, int64_t num_tokens, const uint64_t* freqs, int rotary_dim, int interleaved,
              float magnitude, int num_heads, int num_kv_heads, int head_dim, kvp_bf16* q_out,
              int64_t q_out_stride_tok, kvp_bf16* k_out, int64_t k_out_stride_tok, kvp_stream_t stream) {
  const char* fn = "attn_rope";
  int rc = check_rope_shape(fn, num_tokens, rotary_dim, num_heads, num_kv_heads, head_dim, q_stride_tok,
                            q_out_stride_tok, k_stride_tok, k_out_stride_tok);
  if (rc || num_tokens == 0) return rc;
  if (!positions || !freqs || (num_heads && (!q || !q_out)) || (num_kv_heads && (!k || !k_out)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  if ((q == q_out && num_heads && q_stride_tok != q_out_stride_tok) ||
      (k == k_out && num_kv_heads && k_stride_tok != k_out_stride_tok))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: rows rotated in place need one row stride", fn);
  int *status, sms;
  rc = kvp::device_handles(&status, &sms);
  if (rc) return rc;
  const cudaError_t e = kvp::launch_rope({positions, freqs, rotary_dim, interleaved != 0, magnitude},
                                         {q, q_stride_tok, q_out, q_out_stride_tok, num_heads},
                                         {k, k_stride_tok, k_out, k_out_stride_tok, num_kv_heads}, num_tokens,
                                         head_dim, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

int kv_quant_store(const kvp_bf16* k, const kvp_bf16* v, int64_t k_stride_tok, int64_t v_stride_tok,
                   const int32_t* slot_mapping, int64_t num_tokens, void* k_cache, void* v_cache, float* k_scales,
                   float* v_scales, int format, int64_t num_blocks, int block_size, int scale_tokens,
                   int num_kv_heads, int head_dim, kvp_stream_t stream) {
  const char* fn = "kv_quant_store";
  int rc = check_cache_shape(fn, format, num_blocks, block_size, scale_tokens, num_kv_heads, head_dim);
  if (rc) return rc;
  const kvp::QuantStoreRows rows{k, v, k_stride_tok, v_stride_tok, slot_mapping, num_tokens};
  rc = check_store_rows(fn, rows, num_kv_heads, head_dim);
  if (rc || num_tokens == 0) return rc;
  const kvp::QuantCache c = cache_of(k_cache, v_cache, k_scales, v_scales, format, num_blocks, block_size,
                                     scale_tokens, num_kv_heads, head_dim);
  rc = check_cache_pointers(fn, c);
  if (rc) return rc;
  int *status, sms;
  rc = kvp::device_handles(&status, &sms);
  if (rc) return rc;
  const cudaError_t e = kvp::launch_quant_store(rows, c, nullptr, nullptr, sms, status, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

int kv_quant_store_rope(const kvp_bf16* q, int64_t q_stride_tok, const kvp_bf16* k, const kvp_bf16* v,
                        int64_t k_stride_tok, int64_t v_stride_tok, const int64_t* positions,
                        const int32_t* slot_mapping, int64_t num_tokens, const uint64_t* freqs, int rotary_dim,
                        int interleaved, float magnitude, int num_heads, kvp_bf16* q_out,
                        int64_t q_out_stride_tok, void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                        int format, int64_t num_blocks, int block_size, int scale_tokens, int num_kv_heads,
                        int head_dim, kvp_stream_t stream) {
  const char* fn = "kv_quant_store_rope";
  int rc = check_cache_shape(fn, format, num_blocks, block_size, scale_tokens, num_kv_heads, head_dim);
  if (rc) return rc;
  rc = check_rope_shape(fn, num_tokens, rotary_dim, num_heads, num_kv_heads, head_dim, q_stride_tok,
                        q_out_stride_tok, k_stride_tok, k_stride_tok);
  if (rc) return rc;
  const kvp::QuantStoreRows rows{k, v, k_stride_tok, v_stride_tok, slot_mapping, num_tokens};
  rc = check_store_rows(fn, rows, num_kv_heads, head_dim);
  if (rc || num_tokens == 0) return rc;
  const kvp::QuantCache c = cache_of(k_cache, v_cache, k_scales, v_scales, format, num_blocks, block_size,
                                     scale_tokens, num_kv_heads, head_dim);
  rc = check_cache_pointers(fn, c);
  if (rc) return rc;
  if (!positions || !freqs || (num_heads && (!q || !q_out)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (q == q_out && num_heads && q_stride_tok != q_out_stride_tok)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: rows rotated in place need one row stride", fn);
  int *status, sms;
  rc = kvp::device_handles(&status, &sms);
  if (rc) return rc;
  const kvp::RopeArgs rope{positions, freqs, rotary_dim, interleaved != 0, magnitude};
  const kvp::RopeRows q_rows{q, q_stride_tok, q_out, q_out_stride_tok, num_heads};
  const cudaError_t e = kvp::launch_quant_store(rows, c, &rope, &q_rows, sms, status, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

int kv_quant_load(const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
                  int format, int64_t num_blocks, int block_size, int scale_tokens, const int32_t* block_tables,
                  int max_blocks_per_seq, const int32_t* context_lens, const int32_t* starts, int num_seqs,
                  int max_context_len, int num_kv_heads, int head_dim, int64_t num_rows, kvp_bf16* k,
                  int64_t k_stride_tok, kvp_bf16* v, int64_t v_stride_tok, kvp_stream_t stream) {
  const char* fn = "kv_quant_load";
  int rc = check_cache_shape(fn, format, num_blocks, block_size, scale_tokens, num_kv_heads, head_dim);
  if (rc) return rc;
  if (num_seqs < 0 || max_blocks_per_seq < 0 || max_context_len < 0 || num_rows < 0)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if ((int64_t)max_blocks_per_seq * block_size > (int64_t)1 << 30)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: context capacity too large", fn);
  if (num_seqs > 65535) return set_last_error(KVP_ERR_UNSUPPORTED, "%s: more than 65535 sequences", fn);
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (k_stride_tok < row || v_stride_tok < row)
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: row stride too small", fn);
  if (num_seqs == 0 || max_blocks_per_seq == 0) return KVP_OK;
  const kvp::QuantCache c = cache_of(k_cache, v_cache, k_scales, v_scales, format, num_blocks, block_size,
                                     scale_tokens, num_kv_heads, head_dim);
  rc = check_cache_pointers(fn, c);
  if (rc) return rc;
  if (!block_tables || !context_lens || !starts || (num_rows > 0 && (!k || !v)))
    return set_last_error(KVP_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(k) || !aligned16(v) || k_stride_tok % 8 || v_stride_tok % 8)
    return set_last_error(KVP_ERR_INVALID_ARG,
                          "%s: k and v need 16-byte alignment and row strides that are multiples of 8 elements",
                          fn);
  int *status, sms;
  rc = kvp::device_handles(&status, &sms);
  if (rc) return rc;
  const kvp::QuantLoadArgs a{block_tables, max_blocks_per_seq, context_lens, starts, num_seqs, max_context_len,
                             num_rows,     k,                  v,            k_stride_tok, v_stride_tok};
  const cudaError_t e = kvp::launch_quant_load(a, c, sms, status, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

size_t attn_decode_quant_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                        int max_context_len) {
  if (num_seqs < 0 || max_context_len < 0 || !kvp::decode_supported(num_heads, num_kv_heads, head_dim)) {
    set_last_error(KVP_ERR_INVALID_ARG, "attn_decode_quant_workspace_size: bad shape");
    return 0;
  }
  int sms;
  if (kvp::device_sm_count(&sms)) return 0;
  return kvp::quant_decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len, sms);
}

int attn_decode_quant(const kvp_bf16* q, int64_t q_stride_tok, const void* k_cache, const void* v_cache,
                      const float* k_scales, const float* v_scales, int format, int64_t num_blocks, int block_size,
                      int scale_tokens, const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* context_lens, int num_seqs, int max_context_len, int num_heads,
                      int num_kv_heads, int head_dim, float softmax_scale, void* workspace, size_t workspace_bytes,
                      kvp_bf16* out, int64_t out_stride_tok, kvp_stream_t stream) {
  const char* fn = "attn_decode_quant";
  int rc = check_cache_shape(fn, format, num_blocks, block_size, scale_tokens, num_kv_heads, head_dim);
  if (rc) return rc;
  rc = kvp::check_decode_args(fn, q, q_stride_tok, static_cast<const kvp_bf16*>(k_cache),
                              static_cast<const kvp_bf16*>(v_cache), num_blocks, block_size, block_tables,
                              max_blocks_per_seq, context_lens, num_seqs, max_context_len, num_heads, num_kv_heads,
                              head_dim, out, out_stride_tok);
  if (rc || num_seqs == 0) return rc;
  // The kernel counts work in units of up to 16 tokens of a page.
  if ((int64_t)num_seqs * max_blocks_per_seq * ((block_size + 15) / 16) >= (int64_t)1 << 31)
    return set_last_error(KVP_ERR_UNSUPPORTED, "%s: tables of 2^31 or more units of 16 tokens", fn);
  const kvp::QuantCache c = cache_of(k_cache, v_cache, k_scales, v_scales, format, num_blocks, block_size,
                                     scale_tokens, num_kv_heads, head_dim);
  rc = check_cache_pointers(fn, c);
  if (rc) return rc;
  int *status, sms;
  rc = kvp::device_handles(&status, &sms);
  if (rc) return rc;
  const size_t need =
      kvp::quant_decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len, sms);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return set_last_error(KVP_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu)", fn, need, workspace_bytes);
  const kvp::QuantDecodeArgs a{q,        q_stride_tok, block_tables,  max_blocks_per_seq, context_lens, num_seqs,
                               max_context_len, num_heads, softmax_scale, workspace, out, out_stride_tok};
  const cudaError_t e = kvp::launch_quant_decode(a, c, sms, status, (cudaStream_t)stream);
  return e == cudaSuccess ? KVP_OK : cuda_error(e, fn);
}

}  // extern "C"
