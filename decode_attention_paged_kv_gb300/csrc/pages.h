// pages.h -- arguments of the kernels that manage a paged cache's blocks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dkv {

constexpr int kMaxPools = 16;
constexpr int kMaxTableRows = 16384;

struct PoolView {
  char* p;
  int64_t stride, bytes;
  int wide;  // 16-byte accesses fit
};

struct PagesArgs {
  int rows, cols, block, nb, npools;
  int32_t* table;
  int64_t ts;
  int32_t* refs;
  PoolView pool[kMaxPools];
  uint32_t* status;  // workspace header
};

// What one row becomes (dkv_kv_pages_fork).
struct RowPlan {
  int parent;  // -1: none
  int whole;   // pages shared with the parent
  int pages;   // with the last one, where it is not whole
  int end;     // pages of the new row
  int fresh;   // the row's first place in the list of blocks taken
  int copied;  // its last page is a copy
  int pad[2];
};

struct ForkArgs {
  PagesArgs g;
  const int32_t *lens, *parents, *news;
  int32_t* snap;   // the table as it was [rows, cols]
  RowPlan* plan;   // [rows]
  int32_t* taken;  // the lowest free blocks
  int slices;      // CTAs a row
};

struct CompactArgs {
  PagesArgs g;
  int32_t* table_out;
  int64_t ts_out;
  int32_t *refs_out, *map;
  int32_t* totals;             // [0]: blocks in use, [1]: moves
  int32_t* counts;             // blocks in use of every chunk of refs
  int32_t *src, *dst, *count;  // of every move: from, to, references
  int32_t* rank;               // the move of a block
  int items;                   // pieces of one move, over all pools
};

constexpr int kCompactChunk = 1024;   // refs a CTA counts
constexpr int kCompactPiece = 16384;  // bytes of a block that a CTA moves at a time

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s);
cudaError_t launch_compact(const CompactArgs& a, int num_sms, cudaStream_t s);

}  // namespace dkv
