// Internal declarations of the page operators (pages.cu, pages_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "nsv_common.cuh"

namespace nsv {

// Words at the workspace's start: cluster sums and totals.
constexpr int kPageWords = 64;

// Workspace bytes that serve every page operator on this shape.  fork: two
// int2 per row and the free blocks (at most one per row); extend: two int2 per
// row and the free blocks; compact: the map of the blocks, the holes and the
// moving blocks (at most half of the blocks each).
inline uint64_t page_ws_bytes(int rows, long long num_blocks) {
  const uint64_t most = num_blocks > rows ? num_blocks : rows;
  const uint64_t lists = (uint64_t)rows * 16 + most * 4;
  const uint64_t compact = (uint64_t)num_blocks * 4 + 2 * ((uint64_t)num_blocks / 2 + 1) * 4;
  return kPageWords * 4 + (lists > compact ? lists : compact);
}

struct PageParams {
  const int32_t* parents;   // fork: parents; copy: sources; free: rows
  const int32_t* children;  // fork: children; copy: destinations
  int32_t* block_tables;
  int32_t* context_lens;
  int32_t* refs;            // [num_blocks]
  const int32_t* chunk_starts;
  int64_t* write_slots;
  void* k_pool;
  void* v_pool;
  int32_t* ws;
  uint32_t* status;
  long long num_blocks, tokens;
  int rows, max_blocks, count;
  int block_vecs;       // 16-byte vectors of one block of one pool
  int units_per_block;  // warp units of one block of one pool
  int num_sms;
};

int page_units(int block_vecs);
cudaError_t launch_blocks_copy(const PageParams& p, cudaStream_t stream);
cudaError_t launch_rows_fork(const PageParams& p, cudaStream_t stream);
cudaError_t launch_rows_extend(const PageParams& p, cudaStream_t stream);
cudaError_t launch_rows_free(const PageParams& p, cudaStream_t stream);
cudaError_t launch_blocks_compact(const PageParams& p, cudaStream_t stream);

}  // namespace nsv
