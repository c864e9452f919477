// Argument checks of the attention-side entry points: each returns COLI_OK, or
// records a message and returns the code of the error.
#pragma once

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/coli_moe.h"
#include "attn.h"

namespace coli {

inline int reject(int code, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return record_error(code, msg);
}

inline bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

inline int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return COLI_OK;
  return reject(COLI_ECUDA, "%s failed: %s", what, cudaGetErrorString(e));
}

inline int elem_size(int act) { return act == COLI_F32 ? 4 : 2; }

// A batch of head rows: pointer set and aligned, rows 16-byte aligned and
// not overlapping.
inline int check_rows(const char* name, const void* p, size_t stride, int n_heads, int head_dim, int act) {
  if (p == nullptr) return reject(COLI_EINVAL, "%s must be set", name);
  if (misaligned(p, 16) || stride * elem_size(act) % 16)
    return reject(COLI_EINVAL, "%s: pointer and token stride must be 16-byte aligned", name);
  if (stride < static_cast<size_t>(n_heads) * head_dim)
    return reject(COLI_EINVAL, "%s: token stride %zu is less than n_heads * head_dim = %d", name,
                  stride, n_heads * head_dim);
  if (stride > static_cast<size_t>(INT32_MAX))
    return reject(COLI_EINVAL, "%s: token stride %zu is above 2^31 - 1", name, stride);
  return COLI_OK;
}

// A vector of 32-bit ids, lengths or results.
inline int check_words(const char* name, const void* p) {
  if (p == nullptr) return reject(COLI_EINVAL, "%s must be set", name);
  if (misaligned(p, 4)) return reject(COLI_EINVAL, "%s must be 4-byte aligned", name);
  return COLI_OK;
}

inline int check_heads(const char* name, int n) {
  return n >= 1 && n <= 1024 ? COLI_OK : reject(COLI_EINVAL, "%s=%d outside 1..1024", name, n);
}

inline int check_head_dim(int head_dim) {
  if (head_dim < 8 || head_dim > kMaxHeadDim || head_dim % 8)
    return reject(COLI_EINVAL, "head_dim=%d is not a multiple of 8 in 8..%d", head_dim,
                  kMaxHeadDim);
  return COLI_OK;
}

inline int check_rotary(const coli_rotary* r, const int32_t* positions, int head_dim, RotaryView* out) {
  if (r->table == nullptr || positions == nullptr || misaligned(r->table, 16))
    return reject(COLI_EINVAL, "rotary table (16-byte aligned) and positions must be set");
  if (int rc = check_words("positions", positions)) return rc;
  if (r->rot_dim < 2 || r->rot_dim > head_dim || r->rot_dim % 2)
    return reject(COLI_EINVAL, "rot_dim=%d is not even in 2..head_dim=%d", r->rot_dim, head_dim);
  if (r->layout != COLI_ROPE_HALF && r->layout != COLI_ROPE_INTERLEAVED)
    return reject(COLI_EINVAL, "bad rotary layout %d", r->layout);
  if (r->n_positions < 1) return reject(COLI_EINVAL, "n_positions=%d < 1", r->n_positions);
  if (r->inverse != 0 && r->inverse != 1)
    return reject(COLI_EINVAL, "inverse=%d is not 0 or 1", r->inverse);
  *out = RotaryView{r->table, positions, r->n_positions, r->rot_dim,
                    r->layout == COLI_ROPE_INTERLEAVED, r->inverse ? -1.f : 1.f};
  return COLI_OK;
}

inline int check_cache(const coli_kv_cache* c, KvView* out) {
  if (c == nullptr) return reject(COLI_EINVAL, "cache is NULL");
  const bool mx = c->dtype == COLI_MXFP8 || c->dtype == COLI_MXFP4;
  if (!mx && c->dtype != COLI_F32 && c->dtype != COLI_BF16)
    return reject(COLI_EINVAL, "cache dtype %d is not F32, BF16, MXFP8 or MXFP4", c->dtype);
  if (int rc = check_head_dim(c->head_dim)) return rc;
  if (mx && c->head_dim % kMxBlock)
    return reject(COLI_EINVAL, "an MX cache needs head_dim (%d) a multiple of 32", c->head_dim);
  if (c->page_size < 16 || c->page_size > 4096 || c->page_size % 16)
    return reject(COLI_EINVAL, "page_size=%d is not a multiple of 16 in 16..4096", c->page_size);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 256)
    return reject(COLI_EINVAL, "n_kv_heads=%d outside 1..256", c->n_kv_heads);
  if (c->n_pages < 1 || static_cast<int64_t>(c->n_pages) * c->page_size > INT32_MAX)
    return reject(COLI_EINVAL, "n_pages=%d: need at least 1 and n_pages * page_size < 2^31",
                  c->n_pages);
  // tiles of 16 rows are numbered in 32 bits (2^36 rows of at least 16 bytes: over a TiB)
  if (static_cast<int64_t>(c->n_pages) * c->page_size / 16 * c->n_kv_heads >= UINT32_MAX)
    return reject(COLI_EINVAL, "cache of %d pages of %d tokens and %d heads is too large",
                  c->n_pages, c->page_size, c->n_kv_heads);
  if (!c->k || !c->v || misaligned(c->k, 16) || misaligned(c->v, 16))
    return reject(COLI_EINVAL, "cache k and v must be set and 16-byte aligned");
  if (mx && (!c->k_scale || !c->v_scale || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4)))
    return reject(COLI_EINVAL, "cache k_scale and v_scale must be set and 4-byte aligned");
  *out = KvView{};
  out->k = static_cast<char*>(c->k);
  out->v = static_cast<char*>(c->v);
  out->k_scale = mx ? c->k_scale : nullptr;
  out->v_scale = mx ? c->v_scale : nullptr;
  out->dtype = c->dtype;
  out->n_pages = c->n_pages;
  out->page_size = c->page_size;
  out->n_heads = c->n_kv_heads;
  out->head_dim = c->head_dim;
  out->row_bytes = c->dtype == COLI_F32     ? c->head_dim * 4
                   : c->dtype == COLI_BF16  ? c->head_dim * 2
                   : c->dtype == COLI_MXFP8 ? c->head_dim
                                            : c->head_dim / 2;
  out->scale_stride = mx ? (c->head_dim / kMxBlock + 3) / 4 * 4 : 0;
  return COLI_OK;
}

inline int act_of(const KvView& c) { return c.dtype == COLI_F32 ? COLI_F32 : COLI_BF16; }

inline int check_tokens(const char* name, int T) {
  if (T < 0 || T > (1 << 24)) return reject(COLI_EINVAL, "%s=%d outside [0, 2^24]", name, T);
  return COLI_OK;
}

// Tokens or entries of a list that the calls for long contexts take: their kernels count up to
// a block's stride or a look-ahead past the last one, in 32 bits.
constexpr int64_t kMostPlaces = (int64_t{1} << 31) - (1 << 16);

// One call's sequences: their number, the query heads and the tables of their pages.
inline int check_sequences(const KvView& c, int B, int n_q_heads, const int32_t* block_table,
                           int max_pages, const int32_t* seq_lens) {
  if (B < 0 || B > 65535) return reject(COLI_EINVAL, "B=%d outside [0, 65535]", B);
  if (int rc = check_heads("n_q_heads", n_q_heads)) return rc;
  if (n_q_heads % c.n_heads)
    return reject(COLI_EINVAL, "n_q_heads=%d is not a multiple of n_kv_heads=%d", n_q_heads,
                  c.n_heads);
  if (B == 0) return COLI_OK;
  if (static_cast<int64_t>(B) * n_q_heads > INT32_MAX / 2)
    return reject(COLI_EINVAL, "B=%d sequences of %d heads are too many", B, n_q_heads);
  if (int rc = check_words("block_table", block_table)) return rc;
  if (int rc = check_words("seq_lens", seq_lens)) return rc;
  if (max_pages < 1 || static_cast<int64_t>(max_pages) * c.page_size > kMostPlaces)
    return reject(COLI_EINVAL, "max_pages=%d: need 1 or more and max_pages * page_size up to "
                  "2^31 - 2^16", max_pages);
  return COLI_OK;
}

inline int check_scratch(const void* scratch, size_t bytes, size_t need) {
  if (bytes < need || (need > 0 && (scratch == nullptr || misaligned(scratch, 16))))
    return reject(COLI_EINVAL, "scratch: need %zu bytes, 16-byte aligned, got %zu", need, bytes);
  return COLI_OK;
}

}  // namespace coli
