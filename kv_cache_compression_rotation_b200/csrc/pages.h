// Launch parameters of the page pool's kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tq.h"

namespace tq {

constexpr int kPageChunk = 4096;             // reference counts a block
constexpr int kCopySlice = 16384;            // bytes of a page that a block moves at a time
constexpr int kCheckBlocks = 256;            // blocks that look through the source rows of a fork

struct PoolCopy {                            // the arrays whose pages move together
  char* data[TQ_MAX_POOL_ARRAYS];
  int64_t page_bytes[TQ_MAX_POOL_ARRAYS];
  int slice0[TQ_MAX_POOL_ARRAYS + 1];        // slices of a page before each array
  int n;
};

struct PagesParams {
  tq_page_pool pool;
  const int32_t* src;                        // fork: rows copied from
  const int32_t* rows;                       // fork: rows made; reserve, free: the rows
  const int32_t* old_lens;                   // reserve
  const int32_t* lens;
  int n;                                     // requests
  int32_t* shortfall;
  int32_t* page_map;                         // compact
  int32_t* live;
  PoolCopy copy;
  // scratch
  int32_t* chunk_free;                       // [chunks] free pages of each chunk
  int32_t* prefix;                           // [n + 1] pages wanted before each request; [n] = -1: refused
  uint32_t* marks;                           // [2][(rows + 31) / 32]
  int32_t* bad;                              // [kCheckBlocks] fork: a source row lacks pages
  int32_t* from;                             // page copies: pairs
  int32_t* to;
  int chunks;
  int* status;
};

cudaError_t launch_pages_free(const PagesParams& p, cudaStream_t s);
cudaError_t launch_pages_fork(const PagesParams& p, int sms, cudaStream_t s);
cudaError_t launch_pages_reserve(const PagesParams& p, cudaStream_t s);
cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t s);
cudaError_t launch_pages_copy(const PagesParams& p, int sms, cudaStream_t s);

}  // namespace tq
