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
  // ---- other calls than the plain decode attention; read where ext is 1
  int ext;
  int head_tables;  // 1: block_table is [B][n_kv_heads][max_pages], pages for each key head
  int fixed_len;    // > 0: every sequence's length, seq_lens unused
  int fold;         // > 0: one sequence (B = 1) stands for several, whose queries' key heads
                    // have `fold` heads each: q, out and lse are [..][n_kv_heads * fold]
  int raw;          // 1: out is fp32 and lse float2 pairs (m, l): the row's weights are
                    // 2^(x - m) and sum to l, out is their mean
  int may_cut;      // 1: scratch is there whatever paged_direct says
  int overlap;      // 1: the kernel before in the stream lets this one start beside it
};
size_t paged_scratch_bytes(const KvView& c, int B, int n_q_heads);
bool paged_direct(const KvView& c, int max_pages);  // needs no scratch
cudaError_t launch_paged_attention(const PagedArgs& a, cudaStream_t st);
int sm_count();  // of the current device
// Launches a kernel whose blocks may be placed while the one before in the stream drains: it
// has to wait for its end (griddepcontrol.wait) before it reads anything of it.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                         cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
// Raises a kernel's dynamic shared memory limit once per device; `ready` is the kernel's own.
template <class K>
cudaError_t raise_shared(K* kernel, int bytes, bool (&ready)[128]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 128 && ready[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 128) ready[dev] = true;
  return e;
}

// ---- attention behind a shared prefix ------------------------------------------------
struct SharedArgs {
  PagedArgs own;  // the sequences' own tokens; q, out, lse of the whole call
  const int32_t* prefix_pages;
  int prefix_len;
  void* scratch;
};
size_t shared_scratch_bytes(const KvView& c, int B, int n_q_heads);
cudaError_t launch_shared_attention(const SharedArgs& a, cudaStream_t st);

// ---- pages chosen by a cheap score --------------------------------------------------------
cudaError_t launch_page_bounds(const KvView& c, const int32_t* pages, const int32_t* fills, int N,
                               void* bounds, int* status, cudaStream_t st);
struct SelectArgs {
  KvView c;
  const void* bounds;  // [n_pages][n_kv_heads][2][head_dim] act dtype
  const void* q;
  size_t q_stride;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int B, max_pages, n_q_heads, keep, first, last;
  int32_t* pages;  // [B][n_kv_heads][keep]
  int32_t* lens;   // [B]
  float2* scores;  // [B][n_kv_heads][max_pages]: score, how far off it may be
  int* status;
};
cudaError_t launch_select_pages(const SelectArgs& a, cudaStream_t st);

// ---- eviction by accumulated attention weight ----------------------------------------------
struct MassArgs {
  KvView c;
  const void* q;
  size_t q_stride;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* lse;       // [B][n_q_heads]
  const int32_t* known;   // [B], or nullptr
  float* mass;            // [n_pages][n_kv_heads][page_size]
  int B, max_pages, n_q_heads, window;
  float scale;
  int* status;
};
cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t st);
struct EvictArgs {
  KvView c;
  float* mass;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* into;  // [B][into_pages]; block_table: in place
  int B, max_pages, into_pages, keep, first, recent;
  int32_t* kept;        // [B][n_kv_heads][keep]
  int32_t* new_lens;    // [B]
  int* status;
};
cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st);

}  // namespace coli
