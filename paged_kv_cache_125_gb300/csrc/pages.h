// Internal interface of the page operators (pages.cu) to the C-ABI layer.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kvp {

struct PagesHead {
  int copies;  // pages to copy (fork, compact); pages asked for (extend)
  int tokens;  // extend: new tokens over all rows
};

// One page copy: the first `tokens` rows of page src go to page dst.
struct PagePair {
  int src, dst, tokens, pad;
};

// What a row asks of kv_pages_extend.
struct alignas(16) RowGrowth {
  int page0, token0;  // new pages / asked tokens of the rows before it
  int len, add;       // its length; the tokens it can take (if the pool has the pages)
};

struct PagesWorkspace {
  PagesHead* head;
  int* team_counts;         // one count per CTA of the plan kernel
  PagePair* pairs;          // [max(num_blocks, rows)]
  RowGrowth* grow;          // [rows]
  int* page;                // [num_blocks]
};

struct PagesArgs {
  const int32_t* block_tables;  // [num_rows, max_blocks]
  const int32_t* context_lens;  // [num_rows]
  const int32_t* ref_counts;    // [num_blocks]
  int num_rows;
  int max_blocks;
  int64_t num_blocks;
  int block_size;
  const int32_t* parents;     // fork: [num_out]
  int num_out;                // fork: rows of the outputs (else 0)
  const int32_t* new_tokens;  // extend: [num_rows]
  int64_t num_slots;          // extend: entries of slot_mapping
  int32_t* slot_mapping;
  int32_t* places;  // compact: [num_blocks]
  int32_t* out_tables;
  int32_t* out_lens;
  int32_t* out_counts;
  PagesWorkspace ws;
  int* status;
};

struct PagesCache {
  uint16_t* cache;
  int64_t num_planes, plane_stride, row_elems;
};

size_t pages_workspace_bytes(int64_t num_blocks, int64_t rows);
PagesWorkspace pages_workspace(void* base, int64_t num_blocks, int64_t rows);
cudaError_t launch_pages_fork(const PagesArgs& a, const PagesCache& c, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_pages_extend(const PagesArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesArgs& a, const PagesCache& c, int num_sms,
                                 cudaStream_t stream);

}  // namespace kvp
