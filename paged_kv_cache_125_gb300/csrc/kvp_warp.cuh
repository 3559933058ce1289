// Warp-level building blocks of the shared-prefix decode: ldmatrix, the two
// warp MMAs of its own-part consumers, a 4 x 4 chunk transpose, and the tensor
// maps of a layer's caches.
#pragma once

#include <cudaTypedefs.h>

#include "kvp_device.cuh"

namespace kvp {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                        uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                          uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// d += a b: m16n8k16, bf16 inputs, fp32 accumulate (rows 8..15 of a are zero).
__device__ __forceinline__ void mma_k16(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1));
}

// d += a b: m16n8k8, bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// x and y >= 0 as two bf16 numbers each: `hi` is x (1 - 2^-8) rounded, so always
// below x, and `rest` what it leaves out, between 2^-16 x and 2^-7 x (exact before
// it is rounded, by 2^-15 x at most).  Both have x's sign: a product with an
// infinity keeps it, where a rest of 0 or below would make a NaN.
__device__ __forceinline__ void split_bf16x2(float x, float y, uint32_t& hi, uint32_t& rest) {
  const float2 v = make_float2(x, y);
  const float2 low = __fmul2_rn(v, make_float2(0.99609375f, 0.99609375f));
  hi = pack_bf16x2(low.x, low.y);
  const float2 h = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
  const float2 r = __ffma2_rn(h, make_float2(-1.f, -1.f), v);
  rest = pack_bf16x2(r.x, r.y);
}

// Transpose of a 4 x 4 matrix of 16-byte chunks held by the 4 lanes of a
// quad: on entry lane j holds chunks 0..3 of its row in w[0..3]; on exit lane
// j holds chunk j of rows 0..3 of the quad.  Two butterfly stages; in each, a
// chunk moves to the partner lane when one bit of its chunk index differs
// from the same bit of the lane index.
__device__ __forceinline__ void quad_transpose16(uint32_t (&w)[4][4], int lane) {
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    const bool hi = (lane & m) != 0;
#pragma unroll
    for (int k0 = 0; k0 < 4; ++k0) {
      if (k0 & m) continue;
      const int k1 = k0 | m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t send = hi ? w[k0][i] : w[k1][i];
        const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, m);
        if (hi)
          w[k0][i] = recv;
        else
          w[k1][i] = recv;
      }
    }
  }
}

// 3-D map over [rows, heads, D] bf16 (row stride in elements), 128-byte
// swizzle, box {64, box_heads, box_rows}.
inline bool rows_tensor_map(CUtensorMap* m, const void* base, int64_t rows, int heads, int D,
                            int64_t row_stride, int box_heads, int box_rows) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)row_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D map (column, token row, panel, head) of a [rows, heads, D] cache that
// lands T token rows as [head][64-column panel][token][64] in one box.
inline bool stage_tensor_map(CUtensorMap* m, const void* cache, int64_t rows, int heads, int D, int T) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(D / 64), (cuuint64_t)heads};
  cuuint64_t strides[3] = {(cuuint64_t)heads * D * 2, 128, (cuuint64_t)D * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)T, (cuuint32_t)(D / 64), (cuuint32_t)heads};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(cache), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kvp
