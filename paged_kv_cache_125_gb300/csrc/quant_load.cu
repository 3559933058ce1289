// kv_quant_load: sequences of the 8-bit cache read back as bf16 rows.
//
// Row starts[b] + p of the output is token p of sequence b: code * scale,
// rounded once to bf16.  Memory bound: a code is read once, a number written
// once.  A thread turns 16 codes (one 16-byte load) into 16 numbers (two
// 16-byte stores); the codes of a token's heads are contiguous, so a warp's
// loads and stores are too.
#include "quant_device.cuh"

namespace kvp {
namespace {

constexpr int kLoadThreads = 256;
constexpr int kLoadTokens = 32;  // tokens of one CTA's step

template <int kFormat>
__global__ void __launch_bounds__(kLoadThreads) quant_load_kernel(const QuantLoadArgs a, const QuantCache c,
                                                                  int* status) {
  const int b = blockIdx.y;
  const int cap = a.max_blocks * c.block_size;
  int len = a.context_lens[b];
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_error(status, KVP_ERR_DEVICE_DATA);
    len = len < 0 ? 0 : cap;
  }
  const int64_t start = a.starts[b];
  const int vecs = c.num_kv_heads * c.head_dim / 16;  // chunks of 16 codes in a token's row
  const int per_block = c.block_size >> c.scale_shift;
  for (int t0 = blockIdx.x * kLoadTokens; t0 < len; t0 += gridDim.x * kLoadTokens) {
    const int n = len - t0 < kLoadTokens ? len - t0 : kLoadTokens;
    for (int i = threadIdx.x; i < n * vecs; i += kLoadThreads) {
      const int j = i / vecs, x = i - j * vecs, t = t0 + j;
      const int page = t / c.block_size, off = t - page * c.block_size;
      const int block = a.block_tables[(int64_t)b * a.max_blocks + page];
      const int64_t row = start + t;
      if (block < 0 || block >= c.num_blocks || row < 0 || row >= a.num_rows) {
        record_error(status, KVP_ERR_DEVICE_DATA);
        continue;
      }
      const int64_t at = ((int64_t)block * c.block_size + off) * vecs + x;
      const int64_t sc = ((int64_t)block * per_block + (off >> c.scale_shift)) * c.num_kv_heads +
                         x * 16 / c.head_dim;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint4 u = reinterpret_cast<const uint4*>(kv ? c.v : c.k)[at];
        const float scale = (kv ? c.v_scales : c.k_scales)[sc];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = decode2<kFormat>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
          o[e] = pack_bf16x2(f.x * scale, f.y * scale);
        }
        uint4* dst = reinterpret_cast<uint4*>((kv ? a.v + row * a.v_stride : a.k + row * a.k_stride) + x * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_quant_load(const QuantLoadArgs& a, const QuantCache& c, int num_sms, int* status,
                              cudaStream_t stream) {
  const int tiles = (a.max_context_len + kLoadTokens - 1) / kLoadTokens;
  const dim3 grid(tiles < 1 ? 1 : tiles, a.num_seqs);
  if (c.format == KVP_E4M3)
    quant_load_kernel<KVP_E4M3><<<grid, kLoadThreads, 0, stream>>>(a, c, status);
  else
    quant_load_kernel<KVP_INT8><<<grid, kLoadThreads, 0, stream>>>(a, c, status);
  return cudaGetLastError();
}

}  // namespace kvp
