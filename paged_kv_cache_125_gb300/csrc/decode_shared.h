// Internal interface of the shared-prefix decode (decode_shared.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kvp_internal.h"

namespace kvp {

// The plan buffer of attn_shared_plan: what the attention calls of one step
// need to know about the batch, for num_seqs = B sequences.
struct SharedPlanHead {
  int magic, num_seqs, group, num_kv_heads;  // the shape the plan was made for
  int block_size, max_blocks, num_tiles;
  int sms;                 // SMs of the device it was made on
  int gap, pad;            // positions before each sequence's own tokens (see own_gap)
  long long prefix_chunk;  // steps of a prefix CTA of the first wave, of prefix_total
  long long prefix_total;
  long long own_chunk;     // positions per CTA of the own-part kernel, of own_total
  long long own_total;
  long long prefix_chunk2;  // steps of a prefix CTA of the second wave
};
static_assert(sizeof(SharedPlanHead) == 80, "the records after it are 16-byte aligned");

// What a CTA needs to begin, in one load.
struct alignas(16) SharedOwnStart {
  int seq, ctx, own, pad;  // the sequence that holds its first position; its lengths
  long long seq_end;       // cum_tokens[seq + 1]
  long long pad2;
};
struct alignas(16) SharedPrefixStart {
  int tile, seq0, nseq, prefix;  // the tile that holds its first step
  long long step0, step1;        // cum_steps[tile], cum_steps[tile + 1]
};

struct SharedPlan {
  SharedPlanHead* head;
  long long* cum_tokens;  // [B + 1] positions (gap + own tokens) of the sequences before b
  long long* cum_steps;   // [B + 1] prefix steps of the tiles before t, all kv heads
  SharedOwnStart* own_start;        // [sms] where own-part CTA c starts
  SharedPrefixStart* prefix_start;  // [2 * sms] where prefix CTA c starts
  int* ctx;               // [B] context length (0: no row)
  int* prefix;            // [B] keys read with the group, [0, prefix)
  int* tile_of;           // [B] tile of sequence b, or -1 (prefix 0)
  int* tile_seq;          // [B + 1] first sequence of tile t
  int* cum_rows;          // [B + 1] sequences in the tiles before t
  int* same;              // [B] plan kernel: leading pages shared with sequence b - 1
  int* group_min;         // [B] plan kernel: fewest of them in a group
  int* group_seq;         // [B] plan kernel: first sequence of a group
};

size_t shared_plan_bytes(int num_seqs, int num_sms);
SharedPlan shared_plan_view(void* base, int num_seqs, int num_sms);

cudaError_t launch_shared_plan(const int32_t* block_tables, int max_blocks, const int32_t* ctx,
                               int num_seqs, int64_t num_blocks, int block_size, int group,
                               int num_kv_heads, int min_shared_len, const SharedPlan& plan,
                               int num_sms, int* status, cudaStream_t stream);

size_t shared_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                              int num_sms);

struct SharedCall {
  const uint16_t* q;
  int64_t q_stride;
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  int64_t num_blocks;
  int block_size;
  const int32_t* block_tables;
  int max_blocks;
  int num_seqs, num_heads, num_kv_heads, head_dim;
  float softmax_scale;
  void* workspace;
  uint16_t* out;
  int64_t out_stride;
};
// app: the step's new rows, stored by the same call (or null).
cudaError_t launch_decode_shared(const SharedCall& c, const SharedPlan& plan,
                                 const DecodeAppend* app, int num_sms, int* status,
                                 cudaStream_t stream);

}  // namespace kvp
