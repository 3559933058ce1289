// Device code shared by the kernels of the 8-bit cache: codes, scales, and
// rotary angles.
#pragma once

#include "kvp_device.cuh"
#include "quant.h"

namespace kvp {

__device__ __forceinline__ int quotient(int n, Divisor d) {
  return (int)(((uint32_t)n + __umulhi(d.m, (uint32_t)n)) >> d.s);
}

// The start of a kernel launched in the shadow of the one before: nothing of
// memory is touched before that one is done, and the next may come up.
__device__ __forceinline__ void out_of_shadow() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 16 bytes that pass through once.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

constexpr float kLeastScale = 5.421010862427522e-20f;  // 2^-64

// The largest code is 448 = 1.75 * 2^8 (e4m3) or 127 = 1.984375 * 2^6 (int8).
template <int kFormat>
__device__ __forceinline__ float largest_code() {
  return kFormat == KVP_E4M3 ? 448.f : 127.f;
}

// The least power of two p with top <= p * (the largest code), and at least
// 2^-64: exponent arithmetic, so exact.  Powers of two cost e4m3 nothing (its
// precision is relative) and int8 at most one bit; in exchange a code is the
// number's own rounding with no division's before it, and a block whose scale
// grows keeps what its codes hold, up to one rounding of the new, larger step.
template <int kFormat>
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t bits = __float_as_uint(top);
  const uint32_t part = bits & 0x7fffffu;
  int e = (int)(bits >> 23) - 127;
  e += kFormat == KVP_E4M3 ? (part > 0x600000u) - 8 : (part > 0x7e0000u) - 6;
  return e <= -64 ? kLeastScale : __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two numbers, already divided by their scale, as two codes (ties to even,
// infinities to the largest code, NaN to NaN in e4m3 and to 0 in int8).
template <int kFormat>
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  if constexpr (kFormat == KVP_E4M3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    int a, b;
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(a) : "f"(lo));
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(b) : "f"(hi));
    a = a < -127 ? -127 : a;  // -infinity saturates to -128
    b = b < -127 ? -127 : b;
    return (uint32_t)(a & 0xff) | (uint32_t)(b & 0xff) << 8;
  }
}

// The same for four finite numbers times inv, none above the largest code: int8 by
// adding 1.5 * 2^23, whose last place is 1 (the conversion instruction runs at a
// quarter of that rate).
__device__ __forceinline__ uint32_t encode4_int8(float a, float b, float c, float d, float inv) {
  const uint32_t w[4] = {__float_as_uint(fmaf(a, inv, 12582912.f)), __float_as_uint(fmaf(b, inv, 12582912.f)),
                         __float_as_uint(fmaf(c, inv, 12582912.f)), __float_as_uint(fmaf(d, inv, 12582912.f))};
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

template <int kFormat>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv, bool finite = false) {
  uint2 r;
  if (kFormat == KVP_INT8 && finite) {
    r.x = encode4_int8(x[0], x[1], x[2], x[3], inv);
    r.y = encode4_int8(x[4], x[5], x[6], x[7], inv);
    return r;
  }
  r.x = encode2<kFormat>(x[0] * inv, x[1] * inv) | encode2<kFormat>(x[2] * inv, x[3] * inv) << 16;
  r.y = encode2<kFormat>(x[4] * inv, x[5] * inv) | encode2<kFormat>(x[6] * inv, x[7] * inv) << 16;
  return r;
}

// The two codes in the low half of w as two fp16 numbers (exact: e4m3 is a
// subset of fp16, and so are -127 .. 127).
template <int kFormat>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (kFormat == KVP_E4M3) {
    asm("{\n\t.reg .b16 x;\n\tmov.b32 {x, _}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(w));
  } else {
    // 1024 + (code + 128) has the biased code in its low bits
    uint32_t biased;
    asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(biased) : "r"(w ^ 0x8080u), "r"(0x64646464u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(biased), "r"(0x64806480u));  // 1152
  }
  return r;
}

// All four codes of w: lo has the first two.
template <int kFormat>
__device__ __forceinline__ void codes_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kFormat == KVP_E4M3) {
    lo = codes_f16x2<KVP_E4M3>(w);
    hi = codes_f16x2<KVP_E4M3>(w >> 16);
  } else {
    const uint32_t biased = w ^ 0x80808080u;
    uint32_t a = __byte_perm(biased, 0x64646464u, 0x4140), b = __byte_perm(biased, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  }
}

__device__ __forceinline__ float2 f16x2_floats(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .f16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

template <int kFormat>
__device__ __forceinline__ float2 decode2(uint32_t w) {
  return f16x2_floats(codes_f16x2<kFormat>(w));
}

// Cosine and sine of position * freq.  The angle is held in turns as a 64-bit
// fixed-point fraction, in which the product with a 64-bit position wraps as
// the angle does: far positions lose nothing.  Its upper 32 bits, signed, are
// the angle in units of pi * 2^-31.  The fast functions are off by at most 2^-21,
// 2^-12 of the step that bf16 rows are rounded to (16384 tokens of 40 heads: 54.4
// us, with the full ones 56.6); keys that become codes get the full ones, as the
// fast ones' error rounds a few in a million the other way.
template <bool kFast>
__device__ __forceinline__ float2 rope_turn(int64_t position, uint64_t freq, float magnitude) {
  const float half_turns = (float)(int32_t)(uint32_t)(((uint64_t)position * freq) >> 32);
  float s, c;
  if constexpr (kFast)
    __sincosf(half_turns * 1.4629180792671596e-9f, &s, &c);  // pi * 2^-31
  else
    sincospif(half_turns * 4.656612873077393e-10f, &s, &c);  // 2^-31
  return make_float2(c * magnitude, s * magnitude);
}

__device__ __forceinline__ void bf16_floats(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}

__device__ __forceinline__ uint4 floats_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

}  // namespace kvp
