// The tensor-core kernel for many queries over one shared prefix, and its work line.
#pragma once

#include "attn.h"

namespace coli {

constexpr int kPrefixRows = 128, kPrefixKeys = 128;  // of a block's tile

// Parts that the values' channels of a head are cut in, a segment each.
inline int prefix_halves(int head_dim) { return head_dim > 128 ? 2 : 1; }

struct PrefixArgs {
  KvView c;
  const void* q;
  size_t q_stride;
  const int32_t* pages;
  int len;             // tokens of the prefix
  int group;           // query heads of a key head
  int rows;            // B * group
  int pair;            // 1: a segment is 256 rows of a key head, else 128
  int row_tiles;       // of a key head: segment = (head * row_tiles + tile) * halves + half
  int tiles;           // 128-key tiles of a segment
  int64_t total, per;  // tiles in all, of a block
  int box;             // rows of a TMA box: the power of two that divides page_size, to 128
  int pool_rows;       // n_pages * n_kv_heads * page_size
  float scale;
  float* mean;         // [blocks + segments][128 or 256][head_dim]
  float2* ml;          // [blocks + segments][128 or 256]
  int* status;
};
cudaError_t launch_prefix(const PrefixArgs& p, int grid, cudaStream_t st);

}  // namespace coli
