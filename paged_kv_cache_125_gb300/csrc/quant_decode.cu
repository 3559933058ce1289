// attn_decode_quant: one query token per sequence over the 8-bit cache.
//
//   out[b, h] = sum_p softmax_p(q[b, h] . kc_p * ks_p * scale) * vs_p * vc_p
//
// with codes kc, vc and the scales ks, vs of their block of tokens and kv head.
// One CTA per (sequence, kv head): a warp takes every eighth token, a lane
// head_dim / 32 numbers of it; the warps' softmax states are joined in shared
// memory.
#include "quant_device.cuh"

namespace kvp {
namespace {

constexpr int kWarps = 8;

template <int kFormat, int D, int G>
__global__ void __launch_bounds__(kWarps * 32) quant_decode_kernel(const QuantDecodeArgs a, const QuantCache c,
                                                                   int* status) {
  constexpr int E = D / 32;
  const int b = blockIdx.x, g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cap = a.max_blocks * c.block_size;
  int len = a.context_lens[b];
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0) record_error(status, KVP_ERR_DEVICE_DATA);
    len = len < 0 ? 0 : cap;
  }
  const int per_block = c.block_size >> c.scale_shift;
  const float scale = a.softmax_scale * 1.4426950408889634f;
  float q[G][E], acc[G][E], m[G], l[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[h][e] = bf16lo(a.q[b * a.q_stride + (int64_t)(g * G + h) * D + lane * E + e]) * scale;
      acc[h][e] = 0.f;
    }
  }
  for (int t = warp; t < len; t += kWarps) {
    const int page = t / c.block_size, off = t - page * c.block_size;
    const int block = a.block_tables[(int64_t)b * a.max_blocks + page];
    if (block < 0 || block >= c.num_blocks) {
      if (lane == 0) record_error(status, KVP_ERR_DEVICE_DATA);
      continue;
    }
    const int64_t row = (((int64_t)block * c.block_size + off) * c.num_kv_heads + g) * D + lane * E;
    const int64_t sc = ((int64_t)block * per_block + (off >> c.scale_shift)) * c.num_kv_heads + g;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = decode2<kFormat>(*reinterpret_cast<const uint16_t*>(c.k + row + e));
      const float2 y = decode2<kFormat>(*reinterpret_cast<const uint16_t*>(c.v + row + e));
      k[e] = x.x, k[e + 1] = x.y, v[e] = y.x, v[e + 1] = y.y;
    }
    const float ks = c.k_scales[sc], vs = c.v_scales[sc];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += q[h][e] * k[e];
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= ks;
      const float top = fmaxf(m[h], s), old = m[h] == top ? 1.f : exp2f(m[h] - top), p = exp2f(s - top);
      m[h] = top;
      l[h] = l[h] * old + p;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[h][e] = acc[h][e] * old + p * vs * v[e];
    }
  }
  __shared__ float all[kWarps][G][D + 2];
#pragma unroll
  for (int h = 0; h < G; ++h) {
#pragma unroll
    for (int e = 0; e < E; ++e) all[warp][h][lane * E + e] = acc[h][e];
    if (lane == 0) all[warp][h][D] = m[h], all[warp][h][D + 1] = l[h];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += kWarps * 32) {
    const int h = i / D, e = i - h * D;
    float top = -INFINITY, num = 0.f, den = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, all[w][h][D]);
    for (int w = 0; w < kWarps; ++w) {
      const float x = all[w][h][D] == -INFINITY ? 0.f : exp2f(all[w][h][D] - top);
      num += x * all[w][h][e];
      den += x * all[w][h][D + 1];
    }
    const uint32_t r = pack_bf16x2(len == 0 ? 0.f : num / den, 0.f);
    a.out[b * a.out_stride + (int64_t)(g * G + h) * D + e] = (uint16_t)r;
  }
}

template <int kFormat, int D>
cudaError_t launch(const QuantDecodeArgs& a, const QuantCache& c, int* status, cudaStream_t stream) {
  const dim3 grid(a.num_seqs, c.num_kv_heads);
  switch (a.num_heads / c.num_kv_heads) {
    case 1: quant_decode_kernel<kFormat, D, 1><<<grid, kWarps * 32, 0, stream>>>(a, c, status); break;
    case 2: quant_decode_kernel<kFormat, D, 2><<<grid, kWarps * 32, 0, stream>>>(a, c, status); break;
    case 4: quant_decode_kernel<kFormat, D, 4><<<grid, kWarps * 32, 0, stream>>>(a, c, status); break;
    default: quant_decode_kernel<kFormat, D, 8><<<grid, kWarps * 32, 0, stream>>>(a, c, status); break;
  }
  return cudaGetLastError();
}

}  // namespace

size_t quant_decode_workspace_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_quant_decode(const QuantDecodeArgs& a, const QuantCache& c, int num_sms, int* status,
                                cudaStream_t stream) {
  if (c.format == KVP_E4M3)
    return c.head_dim == 128 ? launch<KVP_E4M3, 128>(a, c, status, stream) : launch<KVP_E4M3, 64>(a, c, status, stream);
  return c.head_dim == 128 ? launch<KVP_INT8, 128>(a, c, status, stream) : launch<KVP_INT8, 64>(a, c, status, stream);
}

}  // namespace kvp
