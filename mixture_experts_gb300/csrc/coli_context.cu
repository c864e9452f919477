// C ABI of what keeps long contexts affordable: attention behind a shared prefix,
// attention over chosen pages, eviction. Argument checks, then the launches.
#include "attn_checks.h"

using namespace coli;

namespace {

// The arguments that the attention calls here share.
int check_attention(const KvView& c, const coli_attn_config* cfg, const void* q, size_t q_stride,
                    int B, const int32_t* block_table, int max_pages, const int32_t* seq_lens) {
  if (cfg == nullptr) return reject(COLI_EINVAL, "cfg is NULL");
  if (int rc = check_sequences(c, B, cfg->n_q_heads, block_table, max_pages, seq_lens)) return rc;
  if (cfg->window < 0) return reject(COLI_EINVAL, "window=%d is negative", cfg->window);
  if (!isfinite(cfg->scale)) return reject(COLI_EINVAL, "scale must be finite");
  if (B == 0) return COLI_OK;
  return check_rows("q", q, q_stride, cfg->n_q_heads, c.head_dim, act_of(c));
}

PagedArgs attention_args(const KvView& c, const coli_attn_config* cfg, const void* q,
                         size_t q_stride, int B, const int32_t* block_table, int max_pages,
                         const int32_t* seq_lens, void* out, size_t out_stride, float* lse) {
  PagedArgs a{};
  a.c = c;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.B = B;
  a.max_pages = max_pages;
  a.n_q_heads = cfg->n_q_heads;
  a.window = cfg->window;
  a.scale = cfg->scale;
  a.status = device_status_ptr();
  return a;
}

int check_out(const KvView& c, const coli_attn_config* cfg, const void* q, const void* out,
              size_t out_stride, const float* lse) {
  if (cfg->window != 0) return reject(COLI_EINVAL, "window=%d: there is none here", cfg->window);
  if (int rc = check_rows("out", out, out_stride, cfg->n_q_heads, c.head_dim, act_of(c)))
    return rc;
  if (q == out) return reject(COLI_EINVAL, "out must not be q");
  return lse != nullptr ? check_words("lse", lse) : COLI_OK;
}

// A list of `keep` entries for each sequence and key head.
int check_list(const char* name, int keep, int B, const KvView& c) {
  if (keep > kMostPlaces)
    return reject(COLI_EINVAL, "%s=%d is above 2^31 - 2^16", name, keep);
  if (static_cast<int64_t>(keep) * B * c.n_heads > INT32_MAX)
    return reject(COLI_EINVAL, "%s=%d for %d sequences of %d key heads: 2^31 entries or more", name,
                  keep, B, c.n_heads);
  return COLI_OK;
}

}  // namespace

extern "C" {

size_t coli_shared_attention_scratch_bytes(const coli_kv_cache* cache, int32_t B,
                                           int32_t n_q_heads) {
  KvView c;
  if (check_cache(cache, &c) || B < 1 || B > 65535 || n_q_heads < 1 || n_q_heads > 1024 ||
      n_q_heads % c.n_heads || static_cast<int64_t>(B) * n_q_heads > INT32_MAX / 2)
    return 0;
  return shared_scratch_bytes(c, B, n_q_heads);
}

int coli_shared_attention(const coli_kv_cache* cache, const coli_attn_config* cfg, const void* q,
                          size_t q_stride, int32_t B, const int32_t* prefix_pages,
                          int32_t prefix_len, const int32_t* block_table, int32_t max_pages,
                          const int32_t* seq_lens, void* out, size_t out_stride, float* lse,
                          void* scratch, size_t scratch_bytes, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_attention(c, cfg, q, q_stride, B, block_table, max_pages, seq_lens))
    return rc;
  if (prefix_len < 0 || prefix_len > kMostPlaces)
    return reject(COLI_EINVAL, "prefix_len=%d outside [0, 2^31 - 2^16]", prefix_len);
  if (B == 0) return COLI_OK;
  if (prefix_len > 0)
    if (int rc = check_words("prefix_pages", prefix_pages)) return rc;
  if (int rc = check_out(c, cfg, q, out, out_stride, lse)) return rc;
  if (int rc = check_scratch(scratch, scratch_bytes, shared_scratch_bytes(c, B, cfg->n_q_heads)))
    return rc;
  SharedArgs a{};
  a.own = attention_args(c, cfg, q, q_stride, B, block_table, max_pages, seq_lens, out, out_stride,
                         lse);
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.scratch = scratch;
  return launched(launch_shared_attention(a, static_cast<cudaStream_t>(stream)),
                  "shared attention");
}

int coli_page_bounds(const coli_kv_cache* cache, const int32_t* pages, const int32_t* fills,
                     int32_t N, void* bounds, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_tokens("N", N)) return rc;
  if (N == 0) return COLI_OK;
  if (int rc = check_words("pages", pages)) return rc;
  if (int rc = check_words("fills", fills)) return rc;
  if (bounds == nullptr || misaligned(bounds, 16))
    return reject(COLI_EINVAL, "bounds must be set and 16-byte aligned");
  return launched(launch_page_bounds(c, pages, fills, N, bounds, device_status_ptr(),
                                     static_cast<cudaStream_t>(stream)),
                  "page bounds");
}

size_t coli_select_pages_scratch_bytes(const coli_kv_cache* cache, int32_t B, int32_t max_pages) {
  KvView c;
  if (check_cache(cache, &c) || B < 1 || B > 65535 || max_pages < 1 ||
      static_cast<int64_t>(max_pages) * c.page_size > kMostPlaces)
    return 0;
  return static_cast<size_t>(B) * c.n_heads * max_pages * sizeof(float2);
}

int coli_select_pages(const coli_kv_cache* cache, const void* bounds, const void* q,
                      size_t q_stride, int32_t n_q_heads, int32_t B, const int32_t* block_table,
                      int32_t max_pages, const int32_t* seq_lens, int32_t keep, int32_t first,
                      int32_t last, int32_t* pages, int32_t* lens, void* scratch,
                      size_t scratch_bytes, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_sequences(c, B, n_q_heads, block_table, max_pages, seq_lens)) return rc;
  if (first < 0 || last < 1 || keep < 1 ||
      static_cast<int64_t>(first) + last > keep)
    return reject(COLI_EINVAL, "keep=%d, first=%d, last=%d: need first >= 0, last >= 1 and "
                  "first + last <= keep", keep, first, last);
  if (B == 0) return COLI_OK;
  if (int rc = check_list("keep", keep, B, c)) return rc;
  if (int rc = check_rows("q", q, q_stride, n_q_heads, c.head_dim, act_of(c))) return rc;
  if (bounds == nullptr || misaligned(bounds, 16))
    return reject(COLI_EINVAL, "bounds must be set and 16-byte aligned");
  if (int rc = check_words("pages", pages)) return rc;
  if (int rc = check_words("lens", lens)) return rc;
  if (lens == seq_lens) return reject(COLI_EINVAL, "lens must not be seq_lens");
  if (int rc = check_scratch(scratch, scratch_bytes,
                             static_cast<size_t>(B) * c.n_heads * max_pages * sizeof(float2)))
    return rc;
  SelectArgs a{};
  a.c = c;
  a.bounds = bounds;
  a.q = q;
  a.q_stride = q_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.B = B;
  a.max_pages = max_pages;
  a.n_q_heads = n_q_heads;
  a.keep = keep;
  a.first = first;
  a.last = last;
  a.pages = pages;
  a.lens = lens;
  a.scores = static_cast<float2*>(scratch);
  a.status = device_status_ptr();
  return launched(launch_select_pages(a, static_cast<cudaStream_t>(stream)), "choice of pages");
}

int coli_selected_attention(const coli_kv_cache* cache, const coli_attn_config* cfg,
                            const void* q, size_t q_stride, int32_t B, const int32_t* pages,
                            int32_t max_pages, const int32_t* lens, void* out, size_t out_stride,
                            float* lse, void* scratch, size_t scratch_bytes, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_attention(c, cfg, q, q_stride, B, pages, max_pages, lens)) return rc;
  if (B == 0) return COLI_OK;
  if (int rc = check_out(c, cfg, q, out, out_stride, lse)) return rc;
  if (int rc = check_scratch(scratch, scratch_bytes,
                             paged_direct(c, max_pages) ? 0
                                                        : paged_scratch_bytes(c, B, cfg->n_q_heads)))
    return rc;
  PagedArgs a = attention_args(c, cfg, q, q_stride, B, pages, max_pages, lens, out, out_stride,
                               lse);
  a.scratch = static_cast<float*>(scratch);
  a.head_tables = 1;
  a.ext = 1;
  return launched(launch_paged_attention(a, static_cast<cudaStream_t>(stream)),
                  "attention over chosen pages");
}

int coli_attention_mass(const coli_kv_cache* cache, const coli_attn_config* cfg, const void* q,
                        size_t q_stride, int32_t B, const int32_t* block_table,
                        int32_t max_pages, const int32_t* seq_lens, const float* lse,
                        const int32_t* known, float* mass, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_attention(c, cfg, q, q_stride, B, block_table, max_pages, seq_lens))
    return rc;
  if (B == 0) return COLI_OK;
  if (int rc = check_words("lse", lse)) return rc;
  if (known != nullptr)
    if (int rc = check_words("known", known)) return rc;
  if (int rc = check_words("mass", mass)) return rc;
  MassArgs a{c,     q, q_stride,  block_table,    seq_lens,    lse,        known,
             mass,  B, max_pages, cfg->n_q_heads, cfg->window, cfg->scale, device_status_ptr()};
  return launched(launch_attention_mass(a, static_cast<cudaStream_t>(stream)), "attention mass");
}

int coli_kv_evict(const coli_kv_cache* cache, float* mass, int32_t B, const int32_t* block_table,
                  int32_t max_pages, const int32_t* seq_lens, int32_t keep, int32_t first,
                  int32_t recent, const int32_t* into, int32_t into_pages, int32_t* kept,
                  int32_t* new_lens, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_sequences(c, B, c.n_heads, block_table, max_pages, seq_lens)) return rc;
  if (first < 0 || recent < 0 || keep < 1 ||
      static_cast<int64_t>(first) + recent > keep)
    return reject(COLI_EINVAL, "keep=%d, first=%d, recent=%d: need keep >= 1, the others >= 0 and "
                  "first + recent <= keep", keep, first, recent);
  if (into == nullptr || into == block_table) {
    into = block_table;
    into_pages = max_pages;
  } else {
    if (int rc = check_words("into", into)) return rc;
    if (into_pages < 1 || static_cast<int64_t>(into_pages) * c.page_size > kMostPlaces ||
        static_cast<int64_t>(into_pages) * c.page_size < keep)
      return reject(COLI_EINVAL, "into_pages=%d pages of %d tokens: need room for keep=%d and "
                    "2^31 - 2^16 at most", into_pages, c.page_size, keep);
  }
  if (B == 0) return COLI_OK;
  if (int rc = check_list("keep", keep, B, c)) return rc;
  if (int rc = check_words("mass", mass)) return rc;
  if (int rc = check_words("kept", kept)) return rc;
  if (int rc = check_words("new_lens", new_lens)) return rc;
  if (new_lens == seq_lens) return reject(COLI_EINVAL, "new_lens must not be seq_lens");
  EvictArgs a{c,    mass, block_table, seq_lens, into,   B,    max_pages,
              into_pages, keep, first, recent, kept, new_lens, device_status_ptr()};
  return launched(launch_kv_evict(a, static_cast<cudaStream_t>(stream)), "eviction");
}

}  // extern "C"
