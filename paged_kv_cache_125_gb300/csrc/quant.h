// Internal interface between api_quant.cu and the kernels of rotary positions
// and the 8-bit cache.  Not installed; not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kvp {

// Quotients of n < 2^31 by a number that the host knows: with 2^s >= d and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (n + floor(m n / 2^32)) >> s.
struct Divisor {
  uint32_t m, s;
};
inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1u << s) < d) ++s;
  return {(uint32_t)((((uint64_t)1 << 32) * ((1u << s) - d)) / d + 1), s};
}

// Launches a kernel in the shadow of the stream's previous one: it may become
// resident while that one drains, and waits (griddepcontrol.wait) before it
// touches memory.
template <typename... Params, typename... As>
inline cudaError_t launch_shadow(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                          As... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Rotary positions (rope.cu): freqs[i] is pair i's angle per position in turns,
// as a fraction of 2^64.
struct RopeArgs {
  const int64_t* positions;
  const uint64_t* freqs;
  int rotary_dim;
  bool interleaved;
  float magnitude;
};

// Rows [num_tokens, heads, head_dim] in and out (heads 0: none).
struct RopeRows {
  const uint16_t* in;
  int64_t in_stride;
  uint16_t* out;
  int64_t out_stride;
  int heads;
};
cudaError_t launch_rope(const RopeArgs& r, const RopeRows& q, const RopeRows& k, int64_t num_tokens,
                        int head_dim, int num_sms, cudaStream_t stream);

// One layer's 8-bit cache: codes [num_blocks, block_size, num_kv_heads,
// head_dim], scales [num_blocks, block_size / scale_tokens, num_kv_heads].
struct QuantCache {
  uint8_t* k;
  uint8_t* v;
  float* k_scales;
  float* v_scales;
  int format;
  int64_t num_blocks;
  int block_size;
  int scale_shift;  // log2 of scale_tokens
  int num_kv_heads;
  int head_dim;
};

struct QuantStoreRows {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  int64_t num_tokens;
};
// rope: rotates k on the way (null: none); q: rows rotated in the same launch.
cudaError_t launch_quant_store(const QuantStoreRows& rows, const QuantCache& c, const RopeArgs* rope,
                               const RopeRows* q, int num_sms, int* status, cudaStream_t stream);

struct QuantLoadArgs {
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* context_lens;
  const int32_t* starts;
  int num_seqs;
  int max_context_len;
  int64_t num_rows;
  uint16_t* k;
  uint16_t* v;
  int64_t k_stride, v_stride;
};
cudaError_t launch_quant_load(const QuantLoadArgs& a, const QuantCache& c, int num_sms, int* status,
                              cudaStream_t stream);

struct QuantDecodeArgs {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* context_lens;
  int num_seqs;
  int max_context_len;
  int num_heads;
  float softmax_scale;
  void* workspace;
  uint16_t* out;
  int64_t out_stride;
};
size_t quant_decode_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                    int max_context_len, int num_sms);
cudaError_t launch_quant_decode(const QuantDecodeArgs& a, const QuantCache& c, int num_sms, int* status,
                                cudaStream_t stream);

}  // namespace kvp
