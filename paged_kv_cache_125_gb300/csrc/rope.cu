// attn_rope: rotary positions of a step's query and key rows.
//
// Pair i of a head is turned by the angle position * w_i:
//   x' = x cos - y sin,  y' = y cos + x sin
// with (x, y) the numbers (i, i + R/2) of the head in the half layout and
// (2i, 2i + 1) in the interleaved one, R = rotary_dim; the rest of the head is
// passed on.
//
// Memory bound: every row is read and written once, the angles are made from
// the position and 8 bytes per pair (no table of cosines).  A thread holds the
// cosines and sines of one 16-byte chunk's pairs (of two chunks' in the half
// layout, where x and y stand in different ones) in registers and applies them
// to several heads, so that a head costs two or four 16-byte accesses and the
// rotation itself.  Neighbouring threads have neighbouring chunks.  16384 tokens
// of 32/8/128: 51.6 us, 6.5 TB/s (a copy: 6.7).
#include "rope_device.cuh"

namespace kvp {
namespace {

constexpr int kRopeThreads = 128;

__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs r, const RopeRows q, const RopeRows k,
                                                            const RopeShape s) {
  out_of_shadow();
  rope_thread(r, q, k, s, (int64_t)blockIdx.x * kRopeThreads + threadIdx.x);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool chunks(const RopeRows& x) {
  return x.heads == 0 || (aligned16(x.in) && aligned16(x.out) && x.in_stride % 8 == 0 && x.out_stride % 8 == 0);
}

bool in_place(const RopeRows& x) { return x.heads == 0 || x.in == x.out; }

}  // namespace

RopeShape rope_shape(const RopeArgs& r, const RopeRows& q, const RopeRows& k, int64_t num_tokens, int head_dim,
                     int64_t fill) {
  RopeShape s;
  s.num_tokens = num_tokens;
  s.head_dim = head_dim;
  s.vec = head_dim % 8 == 0 && r.rotary_dim % (r.interleaved ? 8 : 16) == 0 && chunks(q) && chunks(k);
  s.turns = s.vec ? r.rotary_dim / (r.interleaved ? 8 : 16) : r.rotary_dim / 2;
  s.units = s.turns;
  if (!in_place(q) || !in_place(k)) s.units += (head_dim - r.rotary_dim) / (s.vec ? 8 : 1);
  // Heads per thread: eight, or as few as make `fill` threads.
  const int heads = q.heads + k.heads;
  s.per_slice = 8;
  while (s.per_slice > 1 && num_tokens * s.units * ((heads + s.per_slice - 1) / s.per_slice) < fill)
    s.per_slice /= 2;
  s.slices = (heads + s.per_slice - 1) / s.per_slice;
  return s;
}

cudaError_t launch_rope(const RopeArgs& r, const RopeRows& q, const RopeRows& k, int64_t num_tokens,
                        int head_dim, int num_sms, cudaStream_t stream) {
  const RopeShape s = rope_shape(r, q, k, num_tokens, head_dim, (int64_t)num_sms * 4 * kRopeThreads);
  const int64_t ctas = (num_tokens * s.units * s.slices + kRopeThreads - 1) / kRopeThreads;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_shadow(rope_kernel, dim3((unsigned)ctas), kRopeThreads, 0, stream, r, q, k, s);
}

}  // namespace kvp
