// kv_quant_store: a step's new K/V rows quantised into the 8-bit paged cache.
//
// A scale serves the scale_tokens tokens of a block of the page and one kv
// head.  The rows of one call that fall into the same block stand next to one
// another in slot_mapping, in ascending slots: a run.  The scale becomes
//   max(the least power of two that holds the run's largest number,
//       the block's present scale)
// the latter only where the run does not begin the block (offset 0).  Where a
// block's scale grows, the codes of its other tokens are rounded anew.
//
// Memory bound: a row is read once (bf16) and its codes are written once, so
// the numbers of a run are held in registers between the search for the largest
// one and the rounding.  A team of head_dim / 16 lanes has a row of one head,
// two 16-byte chunks per lane, and four rows (of one run, or of four runs where
// blocks have one or two tokens); a run is shared by as many teams as its block
// needs.  A CTA has some rows of slot_mapping, one of K and V, and some of the
// heads: few enough that its warps hold a full block's runs in one or two rounds.
// Eight prompts of 256 .. 2048 tokens (9216 rows of 32/8/128, int8, blocks of 64):
// 12.5 us, 4.5 TB/s of the 6.7 that a copy reaches; 40000 rows 44 us, 5.6 TB/s.
// What remains is the start and two dependent trips, to the slots and to the rows.
// 64 decode rows: 3.3 us, a launch.
// The comparisons below, where they name rows alone, are of one prompt stored again and
// again to the same blocks of a cache, which L2 holds: 1 to 2 us less than with two
// sets of rows and blocks in turn, as above (9216 rows, blocks of 64: 10.6 and 11.5).
#include <type_traits>

#include "rope_device.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 256, kMostThreads = 512;  // of a CTA: more where a run needs them
constexpr int kTile = 256;   // most rows of slot_mapping that a CTA looks through
constexpr int kRotatedTile = 64;  // where their cosines are kept
constexpr int kWords = (kTile + 256) / 32;  // of the rows that its runs may reach

struct StoreShape {
  int tile;        // rows of slot_mapping per CTA
  int teams;       // per run
  int heads;       // per CTA
  int groups;      // of that many heads
  unsigned ctas;   // that store; the others rotate q
  Divisor by_heads, by_pairs;
};

__device__ __forceinline__ float magnitude_of(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;  // infinities and NaN do not count
}

// The two largest |x| of four words of bf16, each among the words' lower or upper
// halves, as bits.
__device__ __forceinline__ uint32_t top_bits(uint32_t top, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  return top;
}

// A lane's numbers of one row (chunks li and li + D / 16 of a head, at src), rotated
// by the row's cosines and sines, in fp32: what is quantised is not rounded to bf16
// before.
template <int D>
__device__ __forceinline__ void rotate_row(const uint4 (&raw)[2], const uint16_t* src, int li, const RopeArgs& r,
                                           const float2* turns, float (&x)[2][8]) {
  bf16_floats(raw[0], x[0]);
  bf16_floats(raw[1], x[1]);
  const int half = r.rotary_dim / 2;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int pair = (li + i * (D / 16)) * 4 + p;
        if (pair >= half) continue;
        const float2 cs = turns[pair];
        const float a = x[i][2 * p], b = x[i][2 * p + 1];
        x[i][2 * p] = a * cs.x - b * cs.y;
        x[i][2 * p + 1] = b * cs.x + a * cs.y;
      }
    }
  } else if (half == D / 2) {  // both numbers of a pair are this lane's
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float2 cs = turns[li * 8 + p];
      const float a = x[0][p], b = x[1][p];
      x[0][p] = a * cs.x - b * cs.y;
      x[1][p] = b * cs.x + a * cs.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int e = (li + i * (D / 16)) * 8 + p;
        if (e >= r.rotary_dim) continue;
        const bool first = e < half;
        const float2 cs = turns[first ? e : e - half];
        const float other = bf16lo(src[first ? e + half : e - half]);
        x[i][p] = x[i][p] * cs.x + (first ? -other : other) * cs.y;
      }
    }
  }
}

// Registers for four CTAs of 256 threads per SM (9216 rows of 32/8/128: 10.1 us; with as
// many registers as the compiler likes, and three CTAs, 12.7), for three where runs are
// one or two rows (16 us; 18.5 with two, and four make 2300 rows 8.3 for 6.7), for two where rows are rotated.
__host__ __device__ constexpr int most_threads(int rows) { return rows < 4 ? kThreads : kMostThreads; }
__host__ __device__ constexpr int least_ctas(bool rope, int rows) {
  return rows < 4 ? (rope ? 2 : 3) : (rope ? 1 : 2);
}

// kRows rows of a team's run, kRuns runs at once.
template <int kFormat, int D, bool kRope, int kRows>
__global__ void __launch_bounds__(most_threads(kRows), least_ctas(kRope, kRows))
    quant_store_kernel(const QuantStoreRows a, const QuantCache c, const RopeArgs r, const RopeRows q,
                       const RopeShape qs, const StoreShape s, int* status) {
  constexpr int TL = D / 16;  // lanes of a team
  constexpr int kRuns = 4 / kRows;
  out_of_shadow();
  if constexpr (kRope) {
    if (blockIdx.x >= s.ctas) {
      rope_thread(r, q, RopeRows{}, qs, (int64_t)(blockIdx.x - s.ctas) * blockDim.x + threadIdx.x);
      return;
    }
  }
  __shared__ int slots[kTile], leaders[kTile];
  __shared__ uint32_t begins[kWords + 1];  // bit i: row first + i continues no run
  __shared__ int count, end;  // runs that begin in the tile; the row behind the last of them
  __shared__ float tops[2][kMostThreads / 32];
  __shared__ int64_t positions[kRope ? kWords * 32 : 1];
  __shared__ uint64_t freqs[kRope ? D / 2 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_v = blockIdx.x & 1;
  const unsigned cta = blockIdx.x >> 1;
  const int64_t first = (int64_t)(cta / s.groups) * s.tile;
  const int head0 = (int)(cta % s.groups) * s.heads;
  const int heads = c.num_kv_heads - head0 < s.heads ? c.num_kv_heads - head0 : s.heads;
  const int tokens = 1 << c.scale_shift;
  const int64_t pool = c.num_blocks * c.block_size;

  const bool turns = kRope && !is_v;
  const int pairs = kRope ? r.rotary_dim / 2 : 0;
  if (turns && threadIdx.x < pairs) freqs[kRope ? threadIdx.x : 0] = r.freqs[threadIdx.x];
  // The tile's rows and those that its runs may reach: which of them go on where the
  // row before left off, in the same block.
  const int words = (s.tile + tokens + 31) / 32;
  for (int w = warp; w < words; w += (int)blockDim.x / 32) {
    const int i = w * 32 + lane;
    const int64_t row = first + i;
    const int64_t slot = row < a.num_tokens ? a.slots[row] : -1;
    const int64_t before = row > 0 && row < a.num_tokens ? a.slots[row - 1] : -2;
    const bool follows = slot > 0 && slot < pool && (slot & (tokens - 1)) && before == slot - 1;
    const unsigned mask = __ballot_sync(0xffffffffu, !follows);
    if (lane == 0) begins[w] = mask;
    if (turns && row < a.num_tokens) positions[kRope ? i : 0] = r.positions[row];
    if (i < s.tile) {
      slots[i] = slot >= 0 && slot < pool ? (int)slot : -1;
      if (slot >= pool) record_error(status, KVP_ERR_DEVICE_DATA);
    }
  }
  __syncthreads();
  // Where the run of row i ends: the next row that continues none.
  auto run_end = [&](int i) {
    int w = (i + 1) / 32;
    uint32_t rest = w < words ? begins[w] & (0xffffffffu << ((i + 1) & 31)) : 1u;
    while (!rest && ++w < words) rest = begins[w];
    return w * 32 + (rest ? __ffs(rest) - 1 : 0);
  };
  if (warp == 0) {
    int n = 0;
    for (int at = 0; at < s.tile; at += 32) {
      const int i = at + lane;
      const bool leads = i < s.tile && slots[i] >= 0 && (begins[i / 32] >> lane & 1);
      const unsigned mask = __ballot_sync(0xffffffffu, leads);
      if (leads) leaders[n + __popc(mask & ((1u << lane) - 1))] = i;
      n += __popc(mask);
    }
    __syncwarp();
    if (lane == 0) {
      count = n;
      end = n ? run_end(leaders[n - 1]) : 0;
    }
  }
  __syncthreads();
  if (count == 0) return;

  // Cosines and sines of the runs' rows, for all heads.
  extern __shared__ float2 table[];
  const int table_row = pairs + 1, row0 = leaders[0];

  const int units = count * heads;                 // (run, head)
  const int lanes = s.teams * TL;                  // of a unit, a power of two
  const int unit_lane = threadIdx.x & (lanes - 1);
  const int team = unit_lane / TL, li = unit_lane % TL;
  const int per_round = (int)blockDim.x / lanes;
  const uint16_t* src = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  uint8_t* codes = is_v ? c.v : c.k;
  float* scales = is_v ? c.v_scales : c.k_scales;
  const int warps = lanes > 32 ? lanes / 32 : 1;
  const int in_warp = lanes < 32 ? lanes : 32;
  const int wl = threadIdx.x & (in_warp - 1);

  for (int base = 0, round = 0; base < units; base += per_round * kRuns, ++round) {
    bool active[kRuns];
    int64_t row[kRuns], slot[kRuns];
    int n[kRuns], head[kRuns];
    float old[kRuns];
    uint4 raw[kRuns][kRows][2];
    auto at = [&](int m) { return src + row[m] * stride + (int64_t)head[m] * D; };
    auto group = [&](int m) { return (slot[m] >> c.scale_shift) * c.num_kv_heads + head[m]; };
#pragma unroll
    for (int m = 0; m < kRuns; ++m) {
      const int u = base + m * per_round + (int)threadIdx.x / lanes;
      active[m] = u < units;
      row[m] = slot[m] = 0;
      n[m] = head[m] = 0;
      if (active[m]) {
        const int lead = heads == s.heads ? quotient(u, s.by_heads) : u / heads, i = leaders[lead];
        head[m] = head0 + u - lead * heads;
        row[m] = first + i;
        slot[m] = slots[i];
        n[m] = run_end(i) - i;
      }
      old[m] = 0.f;
      if (active[m] && wl == 0 && (slot[m] & (tokens - 1))) old[m] = scales[group(m)];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int i = team + j * s.teams;
        raw[m][j][0] = raw[m][j][1] = make_uint4(0, 0, 0, 0);
        if (i >= n[m]) continue;
        raw[m][j][0] = load_once(at(m) + i * stride + li * 8);
        raw[m][j][1] = load_once(at(m) + i * stride + (li + TL) * 8);
      }
    }
    if (turns && round == 0) {  // while the first rows are on their way
      for (int i = threadIdx.x; i < (end - row0) * pairs; i += blockDim.x) {
        const int j = quotient(i, s.by_pairs), p = i - j * pairs;
        table[j * table_row + p] = rope_turn<false>(positions[row0 + j], freqs[p], r.magnitude);
      }
      __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < kRuns; ++m) {
      float x[kRope ? kRows : 1][2][8];  // rotated rows
      float top = 0.f;
      bool finite = false;
      if (turns) {
        const float2* row_turns = table + ((int)(row[m] - first) - row0) * table_row;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const int i = team + j * s.teams;
          if (i >= n[m]) continue;
          float(&y)[2][8] = x[kRope ? j : 0];
          rotate_row<D>(raw[m][j], at(m) + i * stride, li, r, row_turns + i * table_row, y);
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, magnitude_of(y[e >> 3][e & 7]));
        }
      } else {
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < kRows; ++j) bits = top_bits(top_bits(bits, raw[m][j][0]), raw[m][j][1]);
        const uint32_t most = max(bits & 0xffffu, bits >> 16);
        if (most < 0x7f80u) {
          top = __uint_as_float(most << 16);
          finite = true;
        } else {  // infinities or NaN among them
#pragma unroll
          for (int j = 0; j < 2 * kRows; ++j) {
            float y[8];
            bf16_floats(raw[m][j >> 1][j & 1], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, magnitude_of(y[e]));
          }
        }
      }
      for (int o = in_warp / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      float before = __shfl_sync(0xffffffffu, old[m], lane & ~(in_warp - 1));
      if (!(before > 0.f && before < INFINITY)) before = 0.f;  // no scale: its codes mean nothing
      if (warps > 1) {
        const int turn = (round * kRuns + m) & 1;
        if (lane == 0) tops[turn][warp] = top;
        named_barrier_sync(1 + warp / warps, warps * 32);
        for (int w = 0; w < warps; ++w) top = fmaxf(top, tops[turn][(warp & ~(warps - 1)) + w]);
      }
      if (!active[m]) continue;
      const bool fresh = (slot[m] & (tokens - 1)) == 0;
      const float need = scale_for<kFormat>(top);
      const float scale = fresh ? need : fmaxf(before, need);
      const float inv = 1.f / scale;
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int i = team + j * s.teams;
        if (i >= n[m]) continue;
        uint8_t* dst = codes + ((slot[m] + i) * c.num_kv_heads + head[m]) * D;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y[8];
          if (turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[kRope ? j : 0][h][e];
          } else {
            bf16_floats(raw[m][j][h], y);
          }
          *reinterpret_cast<uint2*>(dst + (li + h * TL) * 8) = encode8<kFormat>(y, inv, finite);
        }
      }
      if (scale == before) continue;
      if (unit_lane == 0) scales[group(m)] = scale;
      if (fresh) continue;
      // The block's other tokens, at the new scale (codes without a scale: zero, NaN too).
      const float ratio = before / scale;
      const int from = (int)(slot[m] & (tokens - 1));
      for (int i = team; i < tokens; i += s.teams) {
        if (i >= from && i < from + n[m]) continue;
        uint8_t* dst = codes + ((slot[m] - from + i) * c.num_kv_heads + head[m]) * D;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint2* p = reinterpret_cast<uint2*>(dst + (li + h * TL) * 8);
          const uint2 w = before > 0.f ? *p : make_uint2(0, 0);
          const float2 f[4] = {decode2<kFormat>(w.x), decode2<kFormat>(w.x >> 16), decode2<kFormat>(w.y),
                               decode2<kFormat>(w.y >> 16)};
          const float y[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
          *p = encode8<kFormat>(y, ratio);
        }
      }
    }
  }
}

template <int kFormat, int D, bool kRope, int kRows>
cudaError_t launch(const QuantStoreRows& rows, const QuantCache& c, const RopeArgs& r, const RopeRows& q,
                   int num_sms, int* status, cudaStream_t stream) {
  StoreShape s;
  // A run's teams: few rows for each, so that its numbers fit the registers.
  const int tokens = 1 << c.scale_shift;
  s.teams = tokens / kRows < 1 ? 1 : tokens / kRows;
  const int threads = s.teams * (D / 16) > kThreads ? s.teams * (D / 16) : kThreads;
  const int slots = threads / (s.teams * (D / 16)) * (4 / kRows);  // runs of one head that a CTA holds at once
  s.heads = slots < c.num_kv_heads ? slots : c.num_kv_heads;
  auto groups = [&] { return (c.num_kv_heads + s.heads - 1) / s.heads; };
  // Two rounds of heads for a CTA where full blocks leave each SM its four CTAs all the same
  // (the eight prompts above: 12.5 us; with one round 13.4, with four 19.5).
  if (2 * groups() * (rows.num_tokens / tokens) >= (int64_t)num_sms * 7)
    s.heads = 2 * s.heads < c.num_kv_heads ? 2 * s.heads : c.num_kv_heads;
  s.groups = groups();
  s.by_heads = divisor(s.heads);
  // Rows of slot_mapping per CTA: a block's, or as many as fill the CTA where
  // blocks are short, but few where that leaves SMs without any.  (A window shorter
  // than a block leaves CTAs without a run's start: 9216 rows, blocks of 256 13.6 us, in
  // windows of 60 rows 21.2.)
  int64_t tile = slots > c.num_kv_heads ? (int64_t)tokens * (slots / c.num_kv_heads) : tokens;
  const int64_t few = rows.num_tokens * (s.groups > 2 ? s.groups : 2) / (2 * num_sms);
  if (tile > few) tile = few;
  const int most = kRope ? kRotatedTile : kTile;
  s.tile = (int)(tile < 1 ? 1 : tile > most ? most : tile);
  int64_t ctas = 2 * s.groups * ((rows.num_tokens + s.tile - 1) / s.tile);
  RopeShape qs{};
  const int64_t store_ctas = ctas;
  if (kRope) {
    // Fewer threads for q than attn_rope's: the stores' fill the SMs already (five chunks
    // of up to 900 tokens, 16/8/128: 17.6 us with the load behind; 18.2 with twice as
    // many, 20.4 with four times).
    qs = rope_shape(r, q, RopeRows{}, rows.num_tokens, c.head_dim, (int64_t)num_sms * 256);
    ctas += (rows.num_tokens * qs.units * qs.slices + threads - 1) / threads;
  }
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  s.ctas = (unsigned)store_ctas;
  size_t table = 0;
  if (kRope) {
    s.by_pairs = divisor(r.rotary_dim / 2);
    table = (size_t)(s.tile + tokens) * (r.rotary_dim / 2 + 1) * sizeof(float2);  // at most 166 KB
    const cudaError_t e = cudaFuncSetAttribute(quant_store_kernel<kFormat, D, kRope, kRows>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_shadow(quant_store_kernel<kFormat, D, kRope, kRows>, dim3((unsigned)ctas), threads, table, stream, rows, c,
                       r, q, qs, s, status);
}

template <int kFormat, int D>
cudaError_t launch(const QuantStoreRows& rows, const QuantCache& c, const RopeArgs* rope, const RopeRows* q,
                   int num_sms, int* status, cudaStream_t stream) {
  // Four rows for a team: of one run, or of four or two where runs are of one or two
  // (9216 rows of 32/8/128: 16.3 us for 21.0 with one run of one row, 11.9 for 15.4 with
  // one run of two).
  auto with = [&](auto rows_of_run) {
    constexpr int R = decltype(rows_of_run)::value;
    return rope ? launch<kFormat, D, true, R>(rows, c, *rope, *q, num_sms, status, stream)
                : launch<kFormat, D, false, R>(rows, c, RopeArgs{}, RopeRows{}, num_sms, status, stream);
  };
  if (c.scale_shift == 0) return with(std::integral_constant<int, 1>());
  if (c.scale_shift == 1) return with(std::integral_constant<int, 2>());
  return with(std::integral_constant<int, 4>());
}

}  // namespace

cudaError_t launch_quant_store(const QuantStoreRows& rows, const QuantCache& c, const RopeArgs* rope,
                               const RopeRows* q, int num_sms, int* status, cudaStream_t stream) {
  if (c.format == KVP_E4M3)
    return c.head_dim == 128 ? launch<KVP_E4M3, 128>(rows, c, rope, q, num_sms, status, stream)
                             : launch<KVP_E4M3, 64>(rows, c, rope, q, num_sms, status, stream);
  return c.head_dim == 128 ? launch<KVP_INT8, 128>(rows, c, rope, q, num_sms, status, stream)
                           : launch<KVP_INT8, 64>(rows, c, rope, q, num_sms, status, stream);
}

}  // namespace kvp
