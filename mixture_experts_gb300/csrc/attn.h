// Host-side launchers of the attention-side operators (rotary positions,
// paged key-value cache, decode attention).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace coli {

constexpr int kMaxHeadDim = 256;
constexpr int kMxBlock = 32;

// ---- rotary positions ---------------------------------------------------------
struct RopeFreq {
  int scaling;
  // YARN: w_i is kept where turns_per_w w_i passes ramp_from + ramp_span; YARN_INDEX:
  // divided where i does
  double base, factor, turns_per_w, ramp_from, ramp_span, amplitude;
};
cudaError_t launch_rope_table(const RopeFreq& f, int rot_dim, int n_positions, float* table,
                              cudaStream_t st);

// Rows of heads: [T][n_heads][head_dim], `stride` elements between tokens.
struct HeadRows {
  const void* in;
  void* out;  // nullptr: the rows go to the cache
  size_t in_stride, out_stride;
  int n_heads;
};

struct RotaryView {
  const float* table;  // nullptr: no rotation
  const int32_t* positions;
  int n_positions, rot_dim, interleaved;
  float sine_sign;  // -1: inverse
};

// The cache with what the kernels derive from its shape. Byte strides: a row
// is one token's key (or value) of one head.
struct KvView {
  char* k;
  char* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int dtype;
  int n_pages, page_size, n_heads, head_dim;
  int row_bytes, scale_stride;  // scale_stride: bytes of a row's scales (padded to 4)
};

// q (and k) rotated into their outputs; cache.k != nullptr: k rows rotated
// (when r.table is set) and v rows stored at slots instead.
cudaError_t launch_rotate(const HeadRows& q, const HeadRows& k, const RotaryView& r, int T,
                          int head_dim, int act, int* status, cudaStream_t st);
cudaError_t launch_kv_append(const KvView& c, const HeadRows& q, const HeadRows& k,
                             const HeadRows& v, const RotaryView& r, const int32_t* slots, int T,
                             int* status, cudaStream_t st);
cudaError_t launch_kv_read(const KvView& c, const int32_t* slots, int N, void* k_out,
                           size_t k_stride, void* v_out, size_t v_stride, int* status,
                           cudaStream_t st);

// ---- decode attention -----------------------------------------------------------
struct PagedArgs {
  KvView c;
  const void* q;
  void* out;
  float* lse;  // may be nullptr
  size_t q_stride, out_stride;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int B, max_pages, n_q_heads, window;
  float scale;
  float* scratch;
  int* status;
};
size_t paged_scratch_bytes(const KvView& c, int B, int n_q_heads);
bool paged_direct(const KvView& c, int max_pages);  // needs no scratch
cudaError_t launch_paged_attention(const PagedArgs& a, cudaStream_t st);

}  // namespace coli
