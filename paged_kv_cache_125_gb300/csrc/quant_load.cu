// kv_quant_load: sequences of the 8-bit cache read back as bf16 rows.
//
// Row starts[b] + p of the output is token p of sequence b: code * scale,
// rounded once to bf16.  Memory bound: a code is read once, a number written
// once.  A thread turns 16 codes (one 16-byte load) into 16 numbers (two 16-byte
// stores that pass L2 by); the codes of a token's heads are contiguous, so a
// warp's loads and stores are too.  A CTA has 8 or 16 tokens of K or of V: with both
// in one CTA, or with several tokens' loads of a thread in flight together, a
// sequence of 131072 tokens took 143 to 162 us; so it takes 131 (93% of the
// copy's rate).  Eight prefixes of 100 .. 2048 tokens, 53 MB: 11.8 us (4.5 TB/s),
// three dependent trips (length, page, codes) and a start in it.
#include "quant_device.cuh"

namespace kvp {
namespace {

constexpr int kLoadThreads = 256;

struct LoadShape {
  int columns;    // threads of a row: of its chunks of 16 codes, as many as fit a CTA
  int rows;       // of a CTA's pass
  int tile;       // tokens of a CTA's step
  Divisor by_columns, by_block;
};

template <int kFormat>
__global__ void __launch_bounds__(kLoadThreads) quant_load_kernel(const QuantLoadArgs a, const QuantCache c,
                                                                  const LoadShape s, int* status) {
  out_of_shadow();
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z;
  const int cap = a.max_blocks * c.block_size;
  int len = a.context_lens[b];
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_error(status, KVP_ERR_DEVICE_DATA);
    len = len < 0 ? 0 : cap;
  }
  const int y = quotient(threadIdx.x, s.by_columns), x0 = threadIdx.x - y * s.columns;
  if (y >= s.rows) return;
  const int64_t start = a.starts[b];
  const int vecs = c.num_kv_heads * c.head_dim / 16;
  const uint8_t* codes = is_v ? c.v : c.k;
  const float* scales = is_v ? c.v_scales : c.k_scales;
  uint16_t* to = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  for (int t0 = blockIdx.x * s.tile; t0 < len; t0 += gridDim.x * s.tile) {
#pragma unroll 1
    for (int i = y; i < s.tile; i += s.rows) {
      const int t = t0 + i;
      if (t >= len) break;
      const int page = quotient(t, s.by_block);
      const int block = a.block_tables[(int64_t)b * a.max_blocks + page];
      if (block < 0 || block >= c.num_blocks || start + t < 0 || start + t >= a.num_rows) {
        record_error(status, KVP_ERR_DEVICE_DATA);
        continue;
      }
      const int slot = block * c.block_size + t - page * c.block_size;
      for (int x = x0; x < vecs; x += s.columns) {
        const uint4 u = load_once(codes + ((int64_t)slot * vecs + x) * 16);
        const float scale = scales[(int64_t)(slot >> c.scale_shift) * c.num_kv_heads + x * 16 / c.head_dim];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = decode2<kFormat>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
          o[e] = pack_bf16x2(f.x * scale, f.y * scale);
        }
        uint4* dst = reinterpret_cast<uint4*>(to + (start + t) * stride + x * 16);
        __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
}

}  // namespace

cudaError_t launch_quant_load(const QuantLoadArgs& a, const QuantCache& c, int num_sms, int* status,
                              cudaStream_t stream) {
  const int vecs = c.num_kv_heads * c.head_dim / 16;
  // (no sequence is longer than its row of the table: up to 2^30 tokens)
  const int cap = a.max_blocks * c.block_size, longest = a.max_context_len < cap ? a.max_context_len : cap;
  LoadShape s;
  s.columns = vecs < kLoadThreads ? vecs : kLoadThreads;
  s.rows = kLoadThreads / s.columns;
  s.by_columns = divisor(s.columns);
  s.by_block = divisor(c.block_size);
  // 16 tokens for a CTA; 8 where that leaves each SM fewer than 16 CTAs (five
  // sequences of up to 1400 tokens: 18.1 us for 19.7 with the store before; one of
  // 131072: 131.9 for 135.9 the other way).
  s.tile = (int64_t)a.num_seqs * longest < (int64_t)num_sms * 128 ? 8 : 16;
  const int tiles = (longest + s.tile - 1) / s.tile;
  const dim3 grid(tiles < 1 ? 1 : tiles, a.num_seqs, 2);
  return launch_shadow(c.format == KVP_E4M3 ? quant_load_kernel<KVP_E4M3> : quant_load_kernel<KVP_INT8>, grid,
                       kLoadThreads, 0, stream, a, c, s, status);
}

}  // namespace kvp
