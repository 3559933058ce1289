// attn_decode_quant: one query token per sequence over the 8-bit cache.
//
//   out[b, h] = sum_p softmax_p(q[b, h] . kc_p * ks_p * scale) * vs_p * vc_p
//
// with codes kc, vc and the scales ks, vs of their block of tokens and kv head.
// Memory bound: every code of a context is read once.  512 sequences of 1000 ..
// 8000 tokens (32/8/128, e4m3, 4.7 GB): 659 us, 7.2 TB/s, more than a copy's 6.7
// (reads alone are faster).  64 of 512 .. 4096 (16/8/128, 294 MB): 50 us, 5.8 TB/s,
// of which the split kernel's stream is 42 us, its start 3 and the merge 4.  One of
// 131071 (64/8/128, int8): 51.5 us, of which the merge of 152 parts is 6.
//
// * Work is counted in units of one page: 16 tokens of eight kv heads, up to 128 of
//   fewer where pages are long enough.  The units of all sequences, end to end, are
//   cut into equal contiguous shares, one per CTA, one CTA per SM.  A sequence that a
//   cut falls into leaves partial results, which the merge kernel joins.
// * A producer warp streams units through a ring of stages in shared memory:
//   one tensor copy each for K and V lands a unit as [kv head][token][head_dim]
//   bytes, swizzled so that the consumers' 16-byte loads fall in different banks;
//   the tokens' scales come by 4-byte asynchronous copies that arrive on the same
//   barrier.  A lane looks up the page of one unit, 32 units ahead at a time.
//   Codes are marked as read once: L2 drops them first.
// * Eight consumer warps: warp w has one piece of 16 tokens of a stage (two of
//   head_dim 64) of kv head w % Hkv.
//   S = q K^T, N = 8 tokens, the query heads of the kv head in M.  The numbers of
//   head_dim may come in any order, the same in q and K, so a thread's operand is
//   32 (16) contiguous bytes of a token.  e4m3: m16n8k32 on the codes as they lie;
//   q, scaled per head by a power of two to at most 2^8, is the sum of two e4m3
//   numbers (rows r and r + 8, the second times 2^4): all of bf16's 8 bits, to
//   2^-21 of the head's largest number.  int8: m16n8k16 on codes made fp16.
//   O^T += V^T W: m16n8k16 in fp16, M = 16 columns of head_dim, N = 8 heads, K = the
//   piece's 16 tokens; the transposing 8-bit load gives a thread four tokens of a
//   column, which two conversions make its operand.  The weights W are the
//   thread's own S.
//   Both kinds of instruction sum in fp32.
// * Softmax: m is a running reference for p * vs, l = sum p and O = sum (p vs) vc
//   are both relative to it.  W = p * vs is rounded to fp16: V's scales, which may
//   differ by any factor between blocks, thus stay out of fp16's range.  m moves, and O
//   and l with it, only when a weight would exceed 2^15, and then to where that one
//   is 2^11 .. 2^12.  So fp16's range lies below the largest weight: one down to 2^-25
//   of it is off by 2^-11 of itself, a smaller one by 2^-36 of the largest, and what
//   lies behind a key that takes nearly all of the weight keeps its bits.  (A step
//   whose weights are below 1/2 could be raised apart: 5 to 10% of the time for all
//   calls, and 25% for those.)
// * Where scale_tokens is 16 or more (kUniform), a unit has one scale of K and
//   one of V per kv head.
#include <cudaTypedefs.h>

#include "kvp_internal.h"
#include "quant_device.cuh"

namespace kvp {
namespace {

constexpr int kConsumers = 8;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kPiece = 16;  // tokens of a warp's step
// Stages of the ring: as many as fit beside the join's buffer.  (Four and six of
// head_dim 128 measured 1 to 2% slower at decode B512, two CTAs of three 12%.)
template <int D>
__host__ __device__ constexpr int stages() {
  return 5;
}
constexpr int kTold = 16;  // segments that the producer may be ahead by, at most
static_assert(stages<64>() + 2 <= kTold, "a segment is told over one that all warps have finished");

// Pieces that a warp takes from a stage: two of head_dim 64, whose 1 KB would not pay
// for the stage's waits (64 sequences of 16384 tokens, 16/8/64 e4m3: 172 us; with one
// 208).
template <int D>
__host__ __device__ constexpr int warp_pieces() {
  return D == 128 ? 1 : 2;
}
// Pieces of a stage, each of one kv head, of K and of V.
template <int D>
__host__ __device__ constexpr int stage_pieces() {
  return kConsumers * warp_pieces<D>();
}
template <int D>
__host__ __device__ constexpr int half_bytes() {
  return stage_pieces<D>() * kPiece * D;
}

enum : int { F_LAST = 1, F_WHOLE = 2, F_ENTERED = 4 };

struct StageMeta {
  uint8_t n[16];  // tokens of each unit
  int flags;
};

// A sequence that is cut: its first and last CTA (last < first: not cut).
struct alignas(16) Chain {
  int b;
  int first;
  int last;
  int pad;
};

struct Args {
  QuantDecodeArgs a;
  int64_t num_blocks;
  int block_size;
  int unit;        // tokens of a unit: 16 << piece_shift
  int piece_shift;
  int least;       // units of the smallest share
  int page_units;  // units of a full page
  Divisor by_block, by_page_units;
  int scale_shift;
  int num_kv_heads;
  int head_shift;  // log2 of num_kv_heads
  const float* k_scales;
  const float* v_scales;
  float scale_log2;
  float* part;    // [ctas][2][Hq][D + 4]: O[D], m, l
  Chain* chains;  // per sequence, or per CTA that one begins in where those are fewer
  bool by_seq;
  bool whole;     // CTA i has sequences i, i + CTAs, ...: none is cut
  int* status;
};

// Units start .. end - 1 of the batch: CTA i has `each` of them, and one more where
// i < more.  The first are units skip, skip + 1, ... of sequence seq.
struct Share {
  int start, end, each, more;
  int seq, skip, len;
};

template <int D, int G>
struct Smem {
  alignas(1024) uint8_t k[stages<D>()][half_bytes<D>()];
  alignas(1024) uint8_t v[stages<D>()][half_bytes<D>()];
  alignas(16) float scales[stages<D>()][2][stage_pieces<D>() * kPiece];  // [piece][token], or (K, V) of each
  alignas(16) StageMeta meta[stages<D>()];
  alignas(8) float join[kConsumers - 1][G][D + 2];  // O, m, l
  alignas(8) uint64_t full[stages<D>()], empty[stages<D>()], told[kTold];
  uint64_t joined[kConsumers], taken[kConsumers];
  int2 warp_sums[kConsumers + 1];  // units and sequences that have any, of each warp's run
  Share share;
  int seg_seq[kTold];  // the sequence of segment i at i % kTold
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// d += a b: m16n8k16, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}

// d += a b: m16n8k32, e4m3 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two 16 x 16 byte matrices, transposed: lane l gives the address of row l % 16 of
// matrix l / 16; thread (r, c) gets rows 4c .. 4c + 3 of columns r and r + 8.
__device__ __forceinline__ void ldsm_bytes_t(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr));
}

__device__ __forceinline__ void copy4_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// An arrival on bar once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ int clamp_len(int c, int cap) { return c < 0 ? 0 : c > cap ? cap : c; }

// Units of a sequence of n tokens.
__device__ __forceinline__ int units_of(const Args& x, int n) {
  if (x.page_units * x.unit == x.block_size) return (n + x.unit - 1) >> (4 + x.piece_shift);
  const int pages = quotient(n, x.by_block), rest = n - pages * x.block_size;
  return pages * x.page_units + ((rest + x.unit - 1) >> (4 + x.piece_shift));
}

// ---------------------------------------------------------------- shares

// This CTA's share of the batch's units, found by all of its threads at once (one
// trip to the context lengths): each has a run of neighbouring sequences.
template <int D, int G>
__device__ void find_share(const Args& x, Smem<D, G>& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = blockIdx.x;
  const int cap = x.a.max_blocks * x.block_size;
  const int per = x.a.num_seqs <= kThreads ? 1 : (x.a.num_seqs + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * per, b1 = b0 + per < x.a.num_seqs ? b0 + per : x.a.num_seqs;
  int mine = 0, live = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = x.a.context_lens[b];
    if (c < 0 || c > cap) record_error(x.status, KVP_ERR_DEVICE_DATA);
    const int u = units_of(x, clamp_len(c, cap));
    mine += u;
    live += u > 0;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  live = __reduce_add_sync(0xffffffffu, live);
  if (lane == 31) sm.warp_sums[warp] = make_int2(incl, live);
  __syncthreads();
  int before = incl - mine, total = 0;
  live = 0;
#pragma unroll
  for (int w = 0; w <= kConsumers; ++w) {
    const int2 y = sm.warp_sums[w];
    if (w < warp) before += y.x;
    total += y.x;
    live += y.y;
  }
  // CTAs that get a share: one for 64 tokens (a unit, where those are longer) or one
  // for a sequence, whichever are more.
  int ctas = (int)((unsigned)(total + x.least - 1) / (unsigned)x.least);
  if (ctas < live) ctas = live;
  if (ctas > (int)gridDim.x) ctas = gridDim.x;
  if (ctas < 1) ctas = 1;
  const int q = (unsigned)total / (unsigned)ctas, rest = total - q * ctas;
  const int start = me < ctas ? me * q + (me < rest ? me : rest) : total;
  const int end = me < ctas ? start + q + (me < rest) : total;
  if (threadIdx.x == 0) sm.share = {start, end, q, rest, 0, 0, 0};
  __syncthreads();
  if (start < end && before <= start && start < before + mine) {  // one thread
    for (int b = b0; b < b1; ++b) {
      const int len = clamp_len(x.a.context_lens[b], cap), u = units_of(x, len);
      if (start < before + u) {
        sm.share.seq = b;
        sm.share.skip = start - before;
        sm.share.len = len;
        break;
      }
      before += u;
    }
  }
  __syncthreads();
}

// Rows without a context are zero, and not cut.
template <int D>
__device__ void empty_rows(const Args& x) {
  const int cap = x.a.max_blocks * x.block_size;
  for (int b = blockIdx.x + gridDim.x * (threadIdx.x >> 5); b < x.a.num_seqs; b += gridDim.x * (kThreads / 32)) {
    if (clamp_len(x.a.context_lens[b], cap) != 0) continue;
    uint4* o = reinterpret_cast<uint4*>(x.a.out + (int64_t)b * x.a.out_stride);
    for (int j = threadIdx.x & 31; j < x.a.num_heads * D / 8; j += 32) o[j] = make_uint4(0, 0, 0, 0);
    if (x.by_seq && !x.whole && (threadIdx.x & 31) == 0) x.chains[b] = {b, 0, -1, 0};
  }
}

// ---------------------------------------------------------------- producer

template <int D, int G, bool kUniform>
struct Producer {
  const Args& x;
  Smem<D, G>& sm;
  const CUtensorMap *mapK, *mapV;
  int left;     // units of the share behind the present segment
  int b, skip;  // the next segment: its sequence and first unit
  int seq = 0, u = 0, u1 = 0, at = 0, len = 0, seg_flags = 0;
  int row = 0, n = 0, row_next = 0, n_next = 0;  // this lane's unit of the present 32, and of the next
  int s = 0;
  uint32_t ph = 0, segs = 0, issued = 0, issued_ph = 0;
  const uint64_t once = policy_evict_first();
  bool more = true;

  __device__ __forceinline__ Producer(const Args& x_, Smem<D, G>& sm_, const CUtensorMap* k, const CUtensorMap* v)
      : x(x_), sm(sm_), mapK(k), mapV(v) {
    left = x.whole ? 1 << 30 : sm.share.end - sm.share.start;
    b = x.whole ? (int)blockIdx.x : sm.share.seq;
    skip = x.whole ? 0 : sm.share.skip;
    len = sm.share.len;
  }

  __device__ __forceinline__ void look_up(int unit, int& r, int& m) {
    r = m = 0;
    if (unit >= u1) return;
    const int page = quotient(unit, x.by_page_units), off = (unit - page * x.page_units) * x.unit;
    int block = x.a.block_tables[(int64_t)seq * x.a.max_blocks + page];
    if (block < 0 || block >= x.num_blocks) {
      record_error(x.status, KVP_ERR_DEVICE_DATA);
      block = 0;  // never read a page outside the pool
    }
    r = block * x.block_size + off;
    m = x.block_size - off < x.unit ? x.block_size - off : x.unit;
    const int rest = len - page * x.block_size - off;
    if (m > rest) m = rest;
  }

  // Tells the consumers the next segment's sequence (-1: no more), whose query they
  // fetch while its first unit is on its way.  Nothing reads slot segs % kTold any more:
  // of the segments that came after the one in it, all stages but the last
  // stages() were given back, and kTold - 1 segments have as many stages or more.
  __device__ __forceinline__ void tell(int sequence) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
      sm.seg_seq[segs & (kTold - 1)] = sequence;
      mbar_arrive(&sm.told[segs & (kTold - 1)]);
    }
    ++segs;
  }

  __device__ __forceinline__ void next_segment() {
    const int lane = threadIdx.x & 31, cap = x.a.max_blocks * x.block_size;
    int units = 0;
    if (segs == 0 && left > 0 && !x.whole) {
      units = units_of(x, len);
    } else {
      for (; left > 0 && b < x.a.num_seqs; b += x.whole ? gridDim.x : 1) {
        const int c = x.a.context_lens[b];
        if (x.whole && (c < 0 || c > cap)) record_error(x.status, KVP_ERR_DEVICE_DATA);
        len = clamp_len(c, cap);
        units = units_of(x, len);
        if (units) break;
      }
    }
    if (!units) {
      more = false;
      tell(-1);
      return;
    }
    tell(b);
    const int begins = sm.share.end - left - skip;  // the sequence's first unit among all
    const int take = left < units - skip ? left : units - skip;
    seq = b;
    b += x.whole ? gridDim.x : 1;
    u = skip;
    u1 = u + take;
    if (!x.whole) left -= take;
    skip = 0;
    at = 0;
    look_up(u + lane, row_next, n_next);
    const bool cut = u > 0 || u1 < units;
    if (u == 0 && lane == 0 && !x.whole) {  // it begins here: the CTA of its last unit
      const int end = begins + units - 1, each = sm.share.each, longer = sm.share.more * (each + 1);
      const int last = !cut ? (int)blockIdx.x - 1
                            : end < longer ? end / (each + 1) : sm.share.more + (end - longer) / each;
      if (x.by_seq)
        x.chains[seq] = {seq, (int)blockIdx.x, last, 0};
      else if (cut)
        x.chains[blockIdx.x] = {seq, (int)blockIdx.x, last, 0};
    }
    seg_flags = (cut ? 0 : F_WHOLE) | (u > 0 ? F_ENTERED : 0);
  }

  // Copies of one stage, once its slot is given back.  False: a wait expired.
  __device__ __forceinline__ bool step() {
    if (!more) return true;
    if (u >= u1) {
      next_segment();
      if (!more) return true;
    }
    const int lane = threadIdx.x & 31;
    const int Hkv = x.num_kv_heads, per_stage = stage_pieces<D>() >> x.head_shift >> x.piece_shift;
    const uint32_t unit_bytes = (uint32_t)(x.unit * Hkv * D);
    const int pieces = (1 << x.piece_shift) - 1;  // of a unit, less one
    if (at == 0) {
      row = row_next;
      n = n_next;
      look_up(u + 32 + lane, row_next, n_next);
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.empty[s], ph ^ 1u, x.status))) return false;
    const int unit = lane - at;  // of the stage
    const bool mine = unit >= 0 && unit < per_stage;
    if (mine) sm.meta[s].n[unit] = (uint8_t)n;
    if (lane == 0) sm.meta[s].flags = seg_flags | (u + per_stage >= u1 ? F_LAST : 0);
    const int count = __popc(__ballot_sync(0xffffffffu, mine && n > 0));
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], 2u * count * unit_bytes);
    __syncwarp();
    if (mine && n > 0) {
      tma_load_3d_hint(sm.k[s] + unit * unit_bytes, mapK, 0, row, 0, &sm.full[s], once);
      tma_load_3d_hint(sm.v[s] + unit * unit_bytes, mapV, 0, row, 0, &sm.full[s], once);
    }
    if constexpr (kUniform) {
      constexpr int kPieces = stage_pieces<D>();  // 8 or 16: K's and V's scales are a warp's at most
      const int i = lane & (kPieces - 1), sub = i >> x.head_shift, off = (sub & pieces) * kPiece;
      const int r = __shfl_sync(0xffffffffu, row, at + (sub >> x.piece_shift)) + off;
      const int m = __shfl_sync(0xffffffffu, n, at + (sub >> x.piece_shift)) - off;
      if (lane < 2 * kPieces && m > 0)
        copy4_async(&sm.scales[s][0][2 * i + lane / kPieces],
                    (lane < kPieces ? x.k_scales : x.v_scales) + ((int64_t)(r >> x.scale_shift) << x.head_shift) +
                        (i & (Hkv - 1)));
    } else {
#pragma unroll
      for (int j = 0; j < stage_pieces<D>() * kPiece / 32; ++j) {
        const int i = j * 32 + lane, sub = i / kPiece >> x.head_shift, head = i / kPiece & (Hkv - 1);
        const int t = (sub & pieces) * kPiece + lane % kPiece;
        const int r = __shfl_sync(0xffffffffu, row, at + (sub >> x.piece_shift));
        const int m = __shfl_sync(0xffffffffu, n, at + (sub >> x.piece_shift));
        if (t < m) {
          const int64_t src = ((int64_t)((r + t) >> x.scale_shift) << x.head_shift) + head;
          copy4_async(&sm.scales[s][0][i], x.k_scales + src);
          copy4_async(&sm.scales[s][1][i], x.v_scales + src);
        }
      }
    }
    arrive_after_copies(&sm.full[s]);
    issued |= 1u << s;
    issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
    if (++s == stages<D>()) {
      s = 0;
      ph ^= 1u;
    }
    u += per_stage;
    at = (at + per_stage) & 31;
    return true;
  }

  // After an expired wait: let every copy that was issued land before the CTA exits.
  __device__ void drain() {
    for (int i = 0; i < stages<D>(); ++i)
      if (issued >> i & 1u) mbar_wait(&sm.full[i], issued_ph >> i & 1u, x.status);
  }
};

// ---------------------------------------------------------------- consumers

// S of 8 tokens for the query heads; thread (r, c): head r, the tokens that the
// lanes' rows 2c and 2c + 1 are.
template <int kFormat, int D>
struct Scores;

template <int D>
struct Scores<KVP_E4M3, D> {
  uint32_t a[D / 32][4];

  // raw: D / 8 words of bf16 of head r, largest below 2^e (e a biased exponent)
  __device__ __forceinline__ float load(const uint32_t (&raw)[D / 8], uint32_t e) {
    e = e < 8 ? 8 : e;
    const float up = __uint_as_float((261 - e) << 23);  // to below 2^8
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float q0 = bf16lo(raw[2 * i + y]) * up, q1 = bf16hi(raw[2 * i + y]) * up;
        const uint32_t h = encode2<KVP_E4M3>(q0, q1);
        const float2 f = decode2<KVP_E4M3>(h);
        hi |= h << 16 * y;
        lo |= encode2<KVP_E4M3>((q0 - f.x) * 16.f, (q1 - f.y) * 16.f) << 16 * y;
      }
      a[i >> 1][2 * (i & 1)] = hi;
      a[i >> 1][2 * (i & 1) + 1] = lo;
    }
    return __uint_as_float((e - 7) << 23);
  }
  // chunk(i): the i-th 16 bytes of this thread's part of its token
  template <typename F>
  __device__ __forceinline__ void of(F chunk, float& x0, float& x1) const {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 u = lds128(chunk(i));
      mma_e4m3(s, a[2 * i], u.x, u.y);
      mma_e4m3(s, a[2 * i + 1], u.z, u.w);
    }
    x0 = fmaf(s[2], 0.0625f, s[0]);
    x1 = fmaf(s[3], 0.0625f, s[1]);
  }
};

template <int D>
struct Scores<KVP_INT8, D> {
  uint32_t a[D / 16][2];

  __device__ __forceinline__ float load(const uint32_t (&raw)[D / 8], uint32_t e) {
    e = e < 1 ? 1 : e > 253 ? 253 : e;
    const float down = __uint_as_float((254 - e) << 23);  // to below 2
#pragma unroll
    for (int i = 0; i < D / 8; ++i) a[i >> 1][i & 1] = pack_f16x2(bf16lo(raw[i]) * down, bf16hi(raw[i]) * down);
    return __uint_as_float(e << 23);
  }
  template <typename F>
  __device__ __forceinline__ void of(F chunk, float& x0, float& x1) const {
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};  // two sums halve the chain
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 u = lds128(chunk(i));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t lo, hi;
        codes_f16x4<KVP_INT8>(w[y], lo, hi);
        mma_f16(y & 1 ? s1 : s0, a[4 * i + y][0], 0, a[4 * i + y][1], 0, lo, hi);
      }
    }
    x0 = s0[0] + s1[0];
    x1 = s0[1] + s1[1];
  }
};

// O += V^T W over a unit's tokens (n of them, where kCut).
template <int kFormat, int D, bool kCut>
__device__ __forceinline__ void add_values(uint32_t addr, int n, int c, const uint32_t (&wt)[2],
                                           float (&o)[D / 16][4]) {
  const int left = n - 4 * c;  // what lies behind the context may be anything
  const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << 8 * left) - 1;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t w[4];
    ldsm_bytes_t(addr ^ (uint32_t)(i << 5), w);
    if constexpr (kCut) {
#pragma unroll
      for (int y = 0; y < 4; ++y) w[y] &= keep;
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t a[4];
      codes_f16x4<kFormat>(w[2 * y], a[0], a[2]);
      codes_f16x4<kFormat>(w[2 * y + 1], a[1], a[3]);
      mma_f16(o[2 * i + y], a[0], a[1], a[2], a[3], wt[0], wt[1]);
    }
  }
}

// log2 of the largest weight that there may be, and of the one that m moves for.
constexpr float kMostWeight = 15.f, kFirstWeight = 12.f;

// V's scales are taken times 2^-16, and outputs times 2^16: the largest p is then
// 2^(27 - e) .. 2^(30 - e) for scales of 2^e, between 2^95 and 2^-100 whatever they are
// (sums over a context stay finite, and a p counts down to 2^-26 of it at least).
constexpr float kValueUnit = 1.52587890625e-05f;

// log2 of a scale times 2^-16, rounded up; a scale below 2^-64 counts as that.
__device__ __forceinline__ float log2_above(float scale) {
  const int e = (int)(__float_as_uint(scale) >> 23) - 126;
  return (float)(e < -80 ? -80 : e);
}

// Thread (r, c) of a warp (r = lane / 4, c = lane % 4) has head r's scores of
// tokens 4c .. 4c + 3 of a unit and the sums of heads 2c, 2c + 1 in columns
// 16 i + r + 8 z: o[i][y + 2 z] is head 2c + y.
template <int kFormat, int D, int G, bool kUniform>
__device__ __forceinline__ void consume(const Args& x, Smem<D, G>& sm) {
  constexpr int KS = D / 16;  // tiles of O
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = x.num_kv_heads;
  const int g = warp & (Hkv - 1), sub = warp >> x.head_shift, subs = kConsumers >> x.head_shift;
  const int head0 = g * G;
  const int r = lane >> 2, c = lane & 3;
  const bool oc[2] = {2 * c < G, 2 * c + 1 < G};
  // This warp's pieces: sub * PW, sub * PW + 1, ... of kv head g.
  constexpr int PW = warp_pieces<D>();
  auto place = [&](int p) {  // of one in a stage half
    const int piece = sub * PW + p, unit = piece >> x.piece_shift;
    return (uint32_t)(((unit * Hkv + g) * x.unit + (piece - (unit << x.piece_shift)) * kPiece) * D);
  };
  // A thread's 16 bytes: chunk q of row t is at chunk q ^ (t & 7) (D 64: t >> 1 & 3),
  // the copies' swizzle.  K: rows krow (tokens of scores 0, 1) and krow + 2, chunks
  // D / 64 * c + i.  V: row lane % 16, chunks 2i + lane / 16.
  const int krow = (r >> 1) * 4 + (r & 1);
  const uint32_t koff = (uint32_t)(krow * D + ((c * (D / 64) ^ (D == 128 ? krow & 7 : krow >> 1 & 3)) << 4));
  const uint32_t voff =
      (uint32_t)((lane & 15) * D + (((D == 128 ? lane & 7 : lane >> 1 & 3) ^ (lane >> 4)) << 4));
  constexpr uint32_t kRowFlip = D == 128 ? 32 : 16;  // of the swizzle from krow to krow + 2

  Scores<kFormat, D> q;
  float o[KS][4];
  int s = 0;
  uint32_t ph = 0;

  for (uint32_t seg = 0;; ++seg) {
    float m = -INFINITY, l = 0.f, cq;
    {
      // The segment's query: D / 4 contiguous numbers of head r.
      if (!mbar_wait(&sm.told[seg & (kTold - 1)], seg / kTold & 1, x.status)) return;
      const int b = sm.seg_seq[seg & (kTold - 1)];
      if (b < 0) return;
      uint32_t raw[D / 8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (r < G)
          u = *reinterpret_cast<const uint4*>(x.a.q + (int64_t)b * x.a.q_stride + (int64_t)(head0 + r) * D +
                                              c * (D / 4) + i * 8);
        raw[4 * i] = u.x, raw[4 * i + 1] = u.y, raw[4 * i + 2] = u.z, raw[4 * i + 3] = u.w;
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = fmaxf(top, fmaxf(fabsf(bf16lo(raw[i])), fabsf(bf16hi(raw[i]))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t e = __float_as_uint(top) >> 23;
      cq = q.load(raw, e) * x.scale_log2;
      // An infinity in q: every score is infinite or NaN, and the softmax NaN.  (A NaN's
      // own code is one.)
      if (e == 255) cq = __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    int flags;
    do {
      if (!mbar_wait(&sm.full[s], ph, x.status)) return;
      flags = sm.meta[s].flags;
      int n[PW];
#pragma unroll
      for (int p = 0; p < PW; ++p) {
        const int piece = sub * PW + p, unit = piece >> x.piece_shift;
        n[p] = (int)sm.meta[s].n[unit] - (piece - (unit << x.piece_shift)) * kPiece;
      }
      if (n[0] > 0) {
        const uint32_t half = (uint32_t)(s * half_bytes<D>());
        float sc[PW][4], vs[PW][4];  // tokens 4c + i
        float top = -INFINITY;
#pragma unroll
        for (int p = 0; p < PW; ++p) {
          const uint32_t at = (smem_u32(sm.k[0]) + half + place(p)) + koff;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            q.of([&](int i) { return (at ^ (j * kRowFlip ^ i << 4)) + 2 * j * D; }, sc[p][2 * j], sc[p][2 * j + 1]);
        }
#pragma unroll
        for (int p = 0; p < PW; ++p) {
          const int at = ((sub * PW + p) << x.head_shift) + g;
          float lv[4];
          if constexpr (kUniform) {
            const float2 scale = *reinterpret_cast<const float2*>(&sm.scales[s][0][2 * at]);
            const float kq = scale.x * cq, v = PW == 1 || n[p] > 0 ? scale.y * kValueUnit : 0.f;
            const float lu = log2_above(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[p][i] *= kq, vs[p][i] = v, lv[i] = lu;
          } else {
            const float4 ks = *reinterpret_cast<const float4*>(&sm.scales[s][0][at * kPiece + 4 * c]);
            const float4 v4 = *reinterpret_cast<const float4*>(&sm.scales[s][1][at * kPiece + 4 * c]);
            sc[p][0] *= cq * ks.x, sc[p][1] *= cq * ks.y, sc[p][2] *= cq * ks.z, sc[p][3] *= cq * ks.w;
            vs[p][0] = v4.x, vs[p][1] = v4.y, vs[p][2] = v4.z, vs[p][3] = v4.w;
#pragma unroll
            for (int i = 0; i < 4; ++i) vs[p][i] *= kValueUnit, lv[i] = log2_above(vs[p][i]);
          }
          if (n[p] < kPiece) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool valid = 4 * c + i < n[p];
              sc[p][i] = valid ? sc[p][i] : -INFINITY;
              if (!kUniform && !valid) vs[p][i] = lv[i] = 0.f;
            }
          }
          top = fmaxf(top, fmaxf(fmaxf(sc[p][0] + lv[0], sc[p][1] + lv[1]), fmaxf(sc[p][2] + lv[2], sc[p][3] + lv[3])));
        }
        if (__any_sync(0xffffffffu, top > m + kMostWeight)) {  // also a sequence's first unit
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const bool grow = top > m + kMostWeight;
          const float to = top - kFirstWeight, alpha = grow ? fast_exp2(m - to) : 1.f;
          if (grow) {
            m = to;
            l *= alpha;
          }
          const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * c), a1 = __shfl_sync(0xffffffffu, alpha, 8 * c + 4);
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[i][0] *= a0;
            o[i][1] *= a1;
            o[i][2] *= a0;
            o[i][3] *= a1;
          }
        }
#pragma unroll
        for (int p = 0; p < PW; ++p) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[p][i] = fast_exp2(sc[p][i] - m);
          l += (sc[p][0] + sc[p][1]) + (sc[p][2] + sc[p][3]);
          const uint32_t wt[2] = {pack_f16x2(sc[p][0] * vs[p][0], sc[p][1] * vs[p][1]),
                                  pack_f16x2(sc[p][2] * vs[p][2], sc[p][3] * vs[p][3])};
          const uint32_t at = (smem_u32(sm.v[0]) + half + place(p)) + voff;
          if (n[p] >= kPiece)
            add_values<kFormat, D, false>(at, n[p], c, wt, o);
          else
            add_values<kFormat, D, true>(at, n[p], c, wt, o);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[s]);
      if (++s == stages<D>()) {
        s = 0;
        ph ^= 1u;
      }
    } while (!(flags & F_LAST));

    // ---- the end of the CTA's part of sequence b: heads 2c, 2c + 1
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    float mh[2] = {__shfl_sync(0xffffffffu, m, 8 * c), __shfl_sync(0xffffffffu, m, 8 * c + 4)};
    float lh[2] = {__shfl_sync(0xffffffffu, l, 8 * c), __shfl_sync(0xffffffffu, l, 8 * c + 4)};
    if (subs > 1) {
      // Warps of the same kv head: sub 0 takes the others' parts (bounded waits
      // both ways).
      if (sub > 0) {
        if (seg > 0 && !mbar_wait(&sm.taken[g], (seg - 1) & 1, x.status)) return;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (!oc[y]) continue;
          float* to = sm.join[warp - Hkv][2 * c + y];
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            to[16 * i + r] = o[i][y];
            to[16 * i + r + 8] = o[i][y + 2];
          }
          if (r == 0) *reinterpret_cast<float2*>(to + D) = make_float2(mh[y], lh[y]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.joined[g]);
        continue;
      }
      if (!mbar_wait(&sm.joined[g], seg & 1, x.status)) return;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (!oc[y]) continue;
        float top = mh[y];
        for (int k = 1; k < subs; ++k) top = fmaxf(top, sm.join[(k - 1) * Hkv + g][2 * c + y][D]);
        float w = mh[y] == -INFINITY ? 0.f : fast_exp2(mh[y] - top);
        lh[y] *= w;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          o[i][y] *= w;
          o[i][y + 2] *= w;
        }
        for (int k = 1; k < subs; ++k) {
          const float* from = sm.join[(k - 1) * Hkv + g][2 * c + y];
          const float2 ml = *reinterpret_cast<const float2*>(from + D);
          w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - top);
          lh[y] += w * ml.y;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[i][y] += w * from[16 * i + r];
            o[i][y + 2] += w * from[16 * i + r + 8];
          }
        }
        mh[y] = top;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.taken[g]);
    }
    const int b = sm.seg_seq[seg & (kTold - 1)];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (!oc[y]) continue;
      const int h = head0 + 2 * c + y;
      if (flags & F_WHOLE) {
        const float inv = 1.f / kValueUnit / lh[y];
        __nv_bfloat16* to =
            reinterpret_cast<__nv_bfloat16*>(x.a.out + (int64_t)b * x.a.out_stride + (int64_t)h * D) + r;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          to[16 * i] = __float2bfloat16_rn(o[i][y] * inv);
          to[16 * i + 8] = __float2bfloat16_rn(o[i][y + 2] * inv);
        }
      } else {
        float* to = x.part + (((size_t)blockIdx.x * 2 + (flags & F_ENTERED ? 0 : 1)) * x.a.num_heads + h) * (D + 4);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          to[16 * i + r] = o[i][y];
          to[16 * i + r + 8] = o[i][y + 2];
        }
        if (r == 0) *reinterpret_cast<float2*>(to + D) = make_float2(mh[y], lh[y]);
      }
    }
  }
}

template <int kFormat, int D, int G, bool kUniform>
__global__ void __launch_bounds__(kThreads, 1)
    quant_split_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                       const Args x) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<D, G>& sm = *reinterpret_cast<Smem<D, G>*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages<D>(); ++i) {
      mbar_init(&sm.full[i], 33);  // the copies' bytes, and the producer's 32 lanes' own copies
      mbar_init(&sm.empty[i], kConsumers);
    }
    for (int i = 0; i < kTold; ++i) mbar_init(&sm.told[i], 1);
    const int subs = kConsumers / x.num_kv_heads;
    for (int i = 0; i < kConsumers; ++i) {
      mbar_init(&sm.joined[i], subs > 1 ? subs - 1 : 1);
      mbar_init(&sm.taken[i], 1);
    }
    fence_mbar_init();
    prefetch_tensormap(&mapK);
    prefetch_tensormap(&mapV);
  }
  out_of_shadow();
  __syncthreads();
  if (!x.whole) find_share<D, G>(x, sm);
  if (!x.by_seq && !x.whole && threadIdx.x == kThreads - 32) x.chains[blockIdx.x] = {0, 0, -1, 0};  // before the producer's
  if (threadIdx.x >> 5 == kConsumers) {
    // The tensor copies read what kernels before this one stored.
    asm volatile("fence.proxy.async.global;" ::: "memory");
    Producer<D, G, kUniform> feed(x, sm, &mapK, &mapV);
    bool ok = true;
    while (ok && feed.more) ok = feed.step();
    if (!ok) feed.drain();
  } else {
    consume<kFormat, D, G, kUniform>(x, sm);
  }
  empty_rows<D>(x);
}

// Joins the parts of the sequences that are cut.  A warp has one head of one chain,
// or a slice of its parts (then the block's warps join theirs in shared memory).
// Small blocks of few registers: one comes up on every SM beside the split
// kernel's CTA and waits there for that grid's end; then two dependent trips to L2
// (the chain, its parts) remain.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32, 4)
    quant_merge_kernel(const Args x, int chains, int head_shift, int slice_shift) {
  constexpr int E = D / 32, kBatch = 8;  // parts in flight
  __shared__ float all[kMergeWarps][D + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = (blockIdx.x * kMergeWarps + warp) >> slice_shift, slice = warp & ((1 << slice_shift) - 1);
  const int chain = item >> head_shift, h = item & ((1 << head_shift) - 1);
  out_of_shadow();
  Chain ch{0, 0, -1, 0};
  if (chain < chains) {
    const int4 c = *reinterpret_cast<const int4*>(&x.chains[chain]);
    ch = {c.x, c.y, c.z, c.w};
  }
  float m = -INFINITY, l = 0.f, o[E] = {};
  for (int i = ch.first + slice; i <= ch.last; i += kBatch << slice_shift) {
    float a[kBatch][E];
    float2 s = make_float2(-INFINITY, 0.f);  // lane k: part k's m and l
    auto of = [&](int part) {  // (at most 5.2 million numbers)
      return x.part + ((part * 2 + (part == ch.first ? 1 : 0)) * x.a.num_heads + h) * (D + 4);
    };
    if (lane < kBatch && i + (lane << slice_shift) <= ch.last)
      s = *reinterpret_cast<const float2*>(of(i + (lane << slice_shift)) + D);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int part = i + (k << slice_shift);
#pragma unroll
      for (int e = 0; e < E; ++e) a[k][e] = 0.f;
      if (part > ch.last) continue;
      const float* p = of(part);
      if constexpr (E == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p + lane * 4);
        a[k][0] = u.x, a[k][1] = u.y, a[k][2] = u.z, a[k][3] = u.w;
      } else {
        const float2 u = *reinterpret_cast<const float2*>(p + lane * 2);
        a[k][0] = u.x, a[k][1] = u.y;
      }
    }
    float top = s.x;
#pragma unroll
    for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(m, __shfl_sync(0xffffffffu, top, 0));
    // (A part has tokens, so m is -inf only of keys that are all NaN, and so is the sum.)
    const float w = fast_exp2(m - top), share = fast_exp2(s.x - top);
    l = l * w + share * s.y;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= w;
    m = top;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float y = __shfl_sync(0xffffffffu, share, k);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += y * a[k][e];
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (slice_shift > 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) all[warp][lane * E + e] = o[e];
    if (lane == 0) all[warp][D] = m, all[warp][D + 1] = l;
    __syncthreads();
    if (slice > 0) return;
    float top = m;
    for (int k = 1; k < 1 << slice_shift; ++k) top = fmaxf(top, all[warp + k][D]);
    float w = fast_exp2(m - top);
    l *= w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= w;
    for (int k = 1; k < 1 << slice_shift; ++k) {
      w = fast_exp2(all[warp + k][D] - top);
      l += w * all[warp + k][D + 1];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += w * all[warp + k][lane * E + e];
    }
  }
  if (ch.last < ch.first) return;
  const float inv = 1.f / kValueUnit / l;
  uint32_t* to = reinterpret_cast<uint32_t*>(x.a.out + (int64_t)ch.b * x.a.out_stride + (int64_t)h * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) to[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
}

// Map of a code array as (column, token row, kv head) with a box of one unit.
bool unit_map(CUtensorMap* map, const void* codes, const QuantCache& c, int unit) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t d = c.head_dim, heads = c.num_kv_heads;
  const cuuint64_t dims[3] = {d, (cuuint64_t)(c.num_blocks * c.block_size), heads};
  const cuuint64_t strides[2] = {heads * d, d};
  const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)unit, (cuuint32_t)heads};
  const cuuint32_t ones[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
  int ctas, most;  // most: with cuts; the workspace is sized by it
  bool by_seq, whole;
  size_t part_bytes, total_bytes;
};

// Stages (0.62 us each for a CTA alone) of the longest sequence up to which none is cut:
// the second kernel for the cut ones takes 3 us more.  With 16/8/128, a stage of 16
// tokens: one sequence of 64 tokens 5.7 us whole and 7.7 cut, of 128 8.1 and 8.6, of
// 192 10.6 and 8.7; 64 sequences of 256 14.1 and 15.1, as the SMs have their own.
constexpr int kWholeStages = 6, kWholeStagesOfMany = 16, kMany = 48;

// One CTA per SM, or as many as the bound of the lengths gives a share (64 tokens
// or a sequence each).  The workspace is that of a batch that is cut even where none
// is: it then never shrinks as sequences or the bound grow, and that of the largest
// batch serves the others.
Plan plan(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_context_len, int num_sms) {
  Plan p;
  const int stage_tokens = kPiece * (head_dim == 128 ? stage_pieces<128>() : stage_pieces<64>()) / num_kv_heads;
  p.whole = max_context_len <= stage_tokens * (num_seqs >= kMany ? kWholeStagesOfMany : kWholeStages);
  long long ctas = ((long long)num_seqs * max_context_len + 63) / 64;
  if (ctas < num_seqs) ctas = num_seqs;
  if (ctas > num_sms) ctas = num_sms;
  p.most = ctas < 1 ? 1 : (int)ctas;
  p.ctas = p.whole && num_seqs < p.most ? (num_seqs < 1 ? 1 : num_seqs) : p.most;
  p.by_seq = num_seqs <= p.ctas;
  p.part_bytes = (size_t)p.most * 2 * num_heads * (head_dim + 4) * sizeof(float);  // (a multiple of 16)
  p.total_bytes = p.part_bytes + (size_t)p.most * sizeof(Chain) + 16;
  return p;
}

template <int kFormat, int D, int G>
cudaError_t launch(const Args& x, const QuantCache& c, const Plan& p, cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!unit_map(&mk, c.k, c, x.unit) || !unit_map(&mv, c.v, c, x.unit)) return cudaErrorInvalidValue;
  constexpr size_t smem = sizeof(Smem<D, G>) + 1024;  // (the struct begins at a multiple of 1024)
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  auto split = (1 << c.scale_shift) >= kPiece && c.block_size % kPiece == 0 ? quant_split_kernel<kFormat, D, G, true>
                                                                           : quant_split_kernel<kFormat, D, G, false>;
  cudaError_t e = cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_shadow(split, dim3(p.ctas), kThreads, smem, stream, mk, mv, x);
  if (e != cudaSuccess || p.whole) return e;
  // Warps for each head of a chain: one for eight parts that it may have.
  const int chains = p.by_seq ? x.a.num_seqs : p.ctas;
  int slice_shift = 0, head_shift = 0;
  while (slice_shift < 3 && (8 << slice_shift) * chains < p.ctas) ++slice_shift;
  while (1 << head_shift < x.a.num_heads) ++head_shift;
  const int blocks = (int)((((int64_t)chains << head_shift << slice_shift) + kMergeWarps - 1) / kMergeWarps);
  return launch_shadow(quant_merge_kernel<D>, dim3(blocks), kMergeWarps * 32, 0, stream, x, chains, head_shift,
                       slice_shift);
}

template <int kFormat, int D>
cudaError_t launch(const Args& x, const QuantCache& c, const Plan& p, cudaStream_t stream) {
  switch (x.a.num_heads / c.num_kv_heads) {
    case 1: return launch<kFormat, D, 1>(x, c, p, stream);
    case 2: return launch<kFormat, D, 2>(x, c, p, stream);
    case 4: return launch<kFormat, D, 4>(x, c, p, stream);
    default: return launch<kFormat, D, 8>(x, c, p, stream);
  }
}

}  // namespace

size_t quant_decode_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_context_len,
                                    int num_sms) {
  return plan(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len, num_sms).total_bytes;
}

cudaError_t launch_quant_decode(const QuantDecodeArgs& a, const QuantCache& c, int num_sms, int* status,
                                cudaStream_t stream) {
  const Plan p = plan(a.num_seqs, a.num_heads, c.num_kv_heads, c.head_dim, a.max_context_len, num_sms);
  Args x;
  x.a = a;
  x.num_blocks = c.num_blocks;
  x.block_size = c.block_size;
  // A unit fills a stage where a page has room for that: few copies, and long ones.
  // (64 sequences of 65536 tokens, 8/1/128 e4m3: 160 us; with units of 16 tokens 220.)
  x.piece_shift = 0;
  const int pieces = c.head_dim == 128 ? stage_pieces<128>() : stage_pieces<64>();
  while (x.piece_shift < 3 && 2 * c.num_kv_heads << x.piece_shift <= pieces && c.block_size % (2 * kPiece << x.piece_shift) == 0)
    ++x.piece_shift;
  x.unit = kPiece << x.piece_shift;
  x.least = 64 / x.unit > 1 ? 64 / x.unit : 1;
  x.page_units = (c.block_size + x.unit - 1) / x.unit;
  x.by_block = divisor(c.block_size);
  x.by_page_units = divisor(x.page_units);
  x.scale_shift = c.scale_shift;
  x.num_kv_heads = c.num_kv_heads;
  x.head_shift = 0;
  while (1 << x.head_shift < c.num_kv_heads) ++x.head_shift;
  x.k_scales = c.k_scales;
  x.v_scales = c.v_scales;
  x.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  x.part = static_cast<float*>(a.workspace);
  x.chains = reinterpret_cast<Chain*>(static_cast<uint8_t*>(a.workspace) + p.part_bytes);
  x.by_seq = p.by_seq;
  x.whole = p.whole;
  x.status = status;
  if (c.format == KVP_E4M3)
    return c.head_dim == 128 ? launch<KVP_E4M3, 128>(x, c, p, stream) : launch<KVP_E4M3, 64>(x, c, p, stream);
  return c.head_dim == 128 ? launch<KVP_INT8, 128>(x, c, p, stream) : launch<KVP_INT8, 64>(x, c, p, stream);
}

}  // namespace kvp
