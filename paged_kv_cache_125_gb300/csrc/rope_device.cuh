// Rotation of query and key rows, shared by attn_rope and the rotating store.
#pragma once

#include "quant_device.cuh"

namespace kvp {

struct RopeShape {
  int64_t num_tokens;
  int head_dim;
  bool vec;        // 16-byte chunks; else number by number
  int units;       // threads per token and slice of heads
  int turns;       // of which rotate; the others pass numbers on
  int slices;      // slices of the heads
  int per_slice;   // heads in each
};

// The shape of a launch for these rows (rope.cu).  A thread has fewer heads where
// that makes up to `fill` threads.
RopeShape rope_shape(const RopeArgs& r, const RopeRows& q, const RopeRows& k, int64_t num_tokens, int head_dim,
                     int64_t fill);

// Head h of the call: q's heads first, then k's.
struct Head {
  const uint16_t* in;
  uint16_t* out;
};
__device__ __forceinline__ Head head_of(const RopeRows& q, const RopeRows& k, int64_t t, int h, int d) {
  if (h < q.heads) return {q.in + t * q.in_stride + (int64_t)h * d, q.out + t * q.out_stride + (int64_t)h * d};
  h -= q.heads;
  return {k.in + t * k.in_stride + (int64_t)h * d, k.out + t * k.out_stride + (int64_t)h * d};
}

// Thread i of rows in 16-byte chunks.
template <bool kInterleaved>
__device__ __forceinline__ void rope_vec(const RopeArgs& r, const RopeRows& q, const RopeRows& k,
                                         const RopeShape& s, int64_t i) {
  const int64_t t = i / (s.units * s.slices);
  if (t >= s.num_tokens) return;
  const int rest = (int)(i - t * (s.units * s.slices));
  const int slice = rest / s.units, unit = rest - slice * s.units;
  const int h0 = slice * s.per_slice, heads = q.heads + k.heads;
  const int h1 = h0 + s.per_slice < heads ? h0 + s.per_slice : heads;
  const int d = s.head_dim;
  if (unit >= s.turns) {  // a chunk behind the rotated part
    const int e = r.rotary_dim + (unit - s.turns) * 8;
    for (int h = h0; h < h1; ++h) {
      const Head x = head_of(q, k, t, h, d);
      *reinterpret_cast<uint4*>(x.out + e) = *reinterpret_cast<const uint4*>(x.in + e);
    }
    return;
  }
  // Four heads at a time; the first batch's loads are on their way while the angles
  // are made.
  constexpr int kPairs = kInterleaved ? 4 : 8, kBatch = 4;
  const int e = unit * 8, e2 = e + r.rotary_dim / 2;
  uint4 a4[kBatch], b4[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (h + j >= h1) break;
      const Head x = head_of(q, k, t, h + j, d);
      a4[j] = load_once(x.in + e);
      if (!kInterleaved) b4[j] = load_once(x.in + e2);
    }
  };
  load(h0);
  float2 cs[kPairs];
  const int64_t pos = r.positions[t];
#pragma unroll
  for (int p = 0; p < kPairs; ++p) cs[p] = rope_turn<true>(pos, r.freqs[unit * kPairs + p], r.magnitude);
  for (int h = h0;;) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (h + j >= h1) break;
      const Head x = head_of(q, k, t, h + j, d);
      float a[8], b[8], c[8];
      bf16_floats(a4[j], a);
      if constexpr (kInterleaved) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          c[2 * p] = a[2 * p] * cs[p].x - a[2 * p + 1] * cs[p].y;
          c[2 * p + 1] = a[2 * p + 1] * cs[p].x + a[2 * p] * cs[p].y;
        }
      } else {
        bf16_floats(b4[j], b);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          c[p] = a[p] * cs[p].x - b[p] * cs[p].y;
          b[p] = b[p] * cs[p].x + a[p] * cs[p].y;
        }
        *reinterpret_cast<uint4*>(x.out + e2) = floats_bf16(b);
      }
      *reinterpret_cast<uint4*>(x.out + e) = floats_bf16(c);
    }
    h += kBatch;
    if (h >= h1) return;
    load(h);
  }
}

// Thread i with any rotary_dim, alignment and stride: one pair of each head, or
// one number behind the rotated part.
__device__ __forceinline__ void rope_any(const RopeArgs& r, const RopeRows& q, const RopeRows& k,
                                         const RopeShape& s, int64_t i) {
  const int64_t t = i / (s.units * s.slices);
  if (t >= s.num_tokens) return;
  const int rest = (int)(i - t * (s.units * s.slices));
  const int slice = rest / s.units, unit = rest - slice * s.units;
  const int h0 = slice * s.per_slice, heads = q.heads + k.heads;
  const int h1 = h0 + s.per_slice < heads ? h0 + s.per_slice : heads;
  const int half = r.rotary_dim / 2;
  const bool turns = unit < half;
  const int e = !turns ? half + unit : r.interleaved ? 2 * unit : unit;
  const int e2 = r.interleaved ? e + 1 : e + half;
  const float2 cs = turns ? rope_turn<true>(r.positions[t], r.freqs[unit], r.magnitude) : make_float2(0.f, 0.f);
  for (int h = h0; h < h1; ++h) {
    const Head x = head_of(q, k, t, h, s.head_dim);
    if (!turns) {
      x.out[e] = x.in[e];
      continue;
    }
    const float a = bf16lo(x.in[e]), b = bf16lo(x.in[e2]);
    const uint32_t w = pack_bf16x2(a * cs.x - b * cs.y, b * cs.x + a * cs.y);
    x.out[e] = (uint16_t)w;
    x.out[e2] = (uint16_t)(w >> 16);
  }
}

__device__ __forceinline__ void rope_thread(const RopeArgs& r, const RopeRows& q, const RopeRows& k,
                                            const RopeShape& s, int64_t i) {
  if (!s.vec)
    rope_any(r, q, k, s, i);
  else if (r.interleaved)
    rope_vec<true>(r, q, k, s, i);
  else
    rope_vec<false>(r, q, k, s, i);
}

}  // namespace kvp
