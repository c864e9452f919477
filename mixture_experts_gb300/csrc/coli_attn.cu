// C ABI of the attention-side operators: argument checks, then the launches.
// Rotary positions, the paged key-value cache and its decode attention sit
// beside the layer the pages centre on (the overview page keeps a KV cache
// next to the experts, section 3.4).
#include "attn_checks.h"

using namespace coli;

extern "C" {

int coli_rope_table(const coli_rope_config* cfg, int32_t n_positions, float* table, void* stream) {
  if (cfg == nullptr || table == nullptr)
    return reject(COLI_EINVAL, "cfg and table must be set");
  if (cfg->rot_dim < 2 || cfg->rot_dim > kMaxHeadDim || cfg->rot_dim % 2)
    return reject(COLI_EINVAL, "rot_dim=%d is not even in 2..%d", cfg->rot_dim, kMaxHeadDim);
  if (n_positions < 1 || static_cast<int64_t>(n_positions) * cfg->rot_dim > INT32_MAX)
    return reject(COLI_EINVAL, "n_positions=%d: need 1 or more and n_positions * rot_dim < 2^31",
                  n_positions);
  if (misaligned(table, 16)) return reject(COLI_EINVAL, "table must be 16-byte aligned");
  const int s = cfg->scaling;
  const bool by_index = s == COLI_ROPE_YARN_INDEX;
  if ((s < COLI_ROPE_NONE || s > COLI_ROPE_YARN) && !by_index)
    return reject(COLI_EINVAL, "bad scaling %d", s);
  if (!(cfg->base > 0) || !isfinite(cfg->base) || !isfinite(cfg->amplitude))
    return reject(COLI_EINVAL, "base must be positive and finite, amplitude finite");
  if (s != COLI_ROPE_NONE && (!(cfg->factor > 0) || !isfinite(cfg->factor)))
    return reject(COLI_EINVAL, "factor must be positive and finite");
  if (s == COLI_ROPE_NTK && cfg->rot_dim == 2)
    return reject(COLI_EINVAL, "NTK scaling needs rot_dim above 2");
  if ((s == COLI_ROPE_YARN || by_index) &&
      (cfg->original_positions < 1 || !(cfg->beta_fast > cfg->beta_slow) ||
       !isfinite(cfg->beta_fast) || !isfinite(cfg->beta_slow)))
    return reject(COLI_EINVAL, "YaRN needs original_positions >= 1 and beta_fast > beta_slow");
  if (by_index && (!(cfg->base > 1) || !(cfg->beta_slow > 0)))
    return reject(COLI_EINVAL, "YaRN by index needs base > 1 and beta_slow > 0");
  RopeFreq f{};
  f.scaling = s;
  f.base = s == COLI_ROPE_NTK
               ? cfg->base * pow(cfg->factor, double(cfg->rot_dim) / (cfg->rot_dim - 2))
               : cfg->base;
  f.factor = cfg->factor;
  f.turns_per_w = cfg->original_positions / 6.283185307179586476925;
  f.ramp_from = cfg->beta_slow;
  f.ramp_span = cfg->beta_fast - cfg->beta_slow;
  if (by_index) {
    auto at = [&](double turns) {
      return cfg->rot_dim * log(f.turns_per_w / turns) / (2 * log(cfg->base));
    };
    const double lo = fmax(floor(at(cfg->beta_fast)), 0.0);
    const double hi = fmin(ceil(at(cfg->beta_slow)), cfg->rot_dim - 1.0);
    f.ramp_from = lo;
    f.ramp_span = hi == lo ? 0.001 : hi - lo;
  }
  f.amplitude = cfg->amplitude;
  return launched(launch_rope_table(f, cfg->rot_dim, n_positions, table,
                                    static_cast<cudaStream_t>(stream)),
                  "rotary table");
}

int coli_rope_apply(const coli_rotary* rotary, const int32_t* positions, int32_t T,
                    int32_t head_dim, int32_t act, const void* q, size_t q_stride,
                    int32_t n_q_heads, void* q_out, size_t q_out_stride, const void* k,
                    size_t k_stride, int32_t n_kv_heads, void* k_out, size_t k_out_stride,
                    void* stream) {
  if (rotary == nullptr) return reject(COLI_EINVAL, "rotary is NULL");
  if (act != COLI_F32 && act != COLI_BF16) return reject(COLI_EINVAL, "bad act dtype %d", act);
  if (int rc = check_tokens("T", T)) return rc;
  if (int rc = check_head_dim(head_dim)) return rc;
  if (T == 0) return COLI_OK;
  RotaryView r;
  if (int rc = check_rotary(rotary, positions, head_dim, &r)) return rc;
  HeadRows rows[2] = {};
  struct {
    const char *name, *out_name;
    const void* in;
    size_t stride;
    int n;
    void* out;
    size_t out_stride;
  } arg[2] = {{"q", "q_out", q, q_stride, n_q_heads, q_out, q_out_stride},
              {"k", "k_out", k, k_stride, n_kv_heads, k_out, k_out_stride}};
  for (int i = 0; i < (k != nullptr ? 2 : 1); ++i) {
    if (int rc = check_heads(i ? "n_kv_heads" : "n_q_heads", arg[i].n)) return rc;
    if (int rc = check_rows(arg[i].name, arg[i].in, arg[i].stride, arg[i].n, head_dim, act))
      return rc;
    if (int rc = check_rows(arg[i].out_name, arg[i].out, arg[i].out_stride, arg[i].n, head_dim,
                            act))
      return rc;
    if (arg[i].in == arg[i].out && arg[i].stride != arg[i].out_stride)
      return reject(COLI_EINVAL, "%s in place needs one stride", arg[i].name);
    rows[i] = HeadRows{arg[i].in, arg[i].out, arg[i].stride, arg[i].out_stride, arg[i].n};
  }
  return launched(launch_rotate(rows[0], rows[1], r, T, head_dim, act, device_status_ptr(),
                                static_cast<cudaStream_t>(stream)),
                  "rotation");
}

int coli_kv_append(const coli_kv_cache* cache, const void* k, size_t k_stride, const void* v,
                   size_t v_stride, const int32_t* slots, int32_t T, const coli_rotary* rotary,
                   const int32_t* positions, const void* q, size_t q_stride, int32_t n_q_heads,
                   void* q_out, size_t q_out_stride, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_tokens("T", T)) return rc;
  if (T == 0) return COLI_OK;
  const int act = act_of(c);
  if (int rc = check_words("slots", slots)) return rc;
  if (int rc = check_rows("k", k, k_stride, c.n_heads, c.head_dim, act)) return rc;
  if (int rc = check_rows("v", v, v_stride, c.n_heads, c.head_dim, act)) return rc;
  RotaryView r{};
  if (rotary != nullptr)
    if (int rc = check_rotary(rotary, positions, c.head_dim, &r)) return rc;
  HeadRows qr{};
  if (q != nullptr) {
    if (rotary == nullptr) return reject(COLI_EINVAL, "q is only rotated: rotary must be set");
    if (int rc = check_heads("n_q_heads", n_q_heads)) return rc;
    if (int rc = check_rows("q", q, q_stride, n_q_heads, c.head_dim, act)) return rc;
    if (int rc = check_rows("q_out", q_out, q_out_stride, n_q_heads, c.head_dim, act)) return rc;
    if (q == q_out && q_stride != q_out_stride)
      return reject(COLI_EINVAL, "q in place needs one stride");
    qr = HeadRows{q, q_out, q_stride, q_out_stride, n_q_heads};
  }
  return launched(launch_kv_append(c, qr, HeadRows{k, nullptr, k_stride, 0, c.n_heads},
                                   HeadRows{v, nullptr, v_stride, 0, c.n_heads}, r, slots, T,
                                   device_status_ptr(), static_cast<cudaStream_t>(stream)),
                  "cache write");
}

int coli_kv_read(const coli_kv_cache* cache, const int32_t* slots, int32_t N, void* k_out,
                 size_t k_out_stride, void* v_out, size_t v_out_stride, void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (int rc = check_tokens("N", N)) return rc;
  if (N == 0) return COLI_OK;
  if (int rc = check_words("slots", slots)) return rc;
  if (k_out == nullptr && v_out == nullptr)
    return reject(COLI_EINVAL, "k_out or v_out must be set");
  const int act = act_of(c);
  if (k_out != nullptr)
    if (int rc = check_rows("k_out", k_out, k_out_stride, c.n_heads, c.head_dim, act)) return rc;
  if (v_out != nullptr)
    if (int rc = check_rows("v_out", v_out, v_out_stride, c.n_heads, c.head_dim, act)) return rc;
  return launched(launch_kv_read(c, slots, N, k_out, k_out_stride, v_out, v_out_stride,
                                 device_status_ptr(), static_cast<cudaStream_t>(stream)),
                  "cache read");
}

size_t coli_paged_attention_scratch_bytes(const coli_kv_cache* cache, int32_t B,
                                          int32_t n_q_heads) {
  KvView c;
  if (check_cache(cache, &c) || B < 1 || n_q_heads < 1 || n_q_heads > 1024 ||
      n_q_heads % c.n_heads)
    return 0;
  return paged_scratch_bytes(c, B, n_q_heads);
}

int coli_paged_attention(const coli_kv_cache* cache, const coli_attn_config* cfg, const void* q,
                         size_t q_stride, int32_t B, const int32_t* block_table,
                         int32_t max_pages, const int32_t* seq_lens, void* out,
                         size_t out_stride, float* lse, void* scratch, size_t scratch_bytes,
                         void* stream) {
  KvView c;
  if (int rc = check_cache(cache, &c)) return rc;
  if (cfg == nullptr) return reject(COLI_EINVAL, "cfg is NULL");
  if (B < 0 || B > 65535) return reject(COLI_EINVAL, "B=%d outside [0, 65535]", B);
  if (int rc = check_heads("n_q_heads", cfg->n_q_heads)) return rc;
  if (cfg->n_q_heads % c.n_heads)
    return reject(COLI_EINVAL, "n_q_heads=%d is not a multiple of n_kv_heads=%d", cfg->n_q_heads,
                  c.n_heads);
  if (cfg->window < 0) return reject(COLI_EINVAL, "window=%d is negative", cfg->window);
  if (!isfinite(cfg->scale)) return reject(COLI_EINVAL, "scale must be finite");
  if (B == 0) return COLI_OK;
  if (static_cast<int64_t>(B) * cfg->n_q_heads > INT32_MAX / 2)
    return reject(COLI_EINVAL, "B=%d sequences of %d heads are too many", B, cfg->n_q_heads);
  const int act = act_of(c);
  if (int rc = check_rows("q", q, q_stride, cfg->n_q_heads, c.head_dim, act)) return rc;
  if (int rc = check_rows("out", out, out_stride, cfg->n_q_heads, c.head_dim, act)) return rc;
  if (q == out) return reject(COLI_EINVAL, "out must not be q");
  if (int rc = check_words("block_table", block_table)) return rc;
  if (int rc = check_words("seq_lens", seq_lens)) return rc;
  if (lse != nullptr)
    if (int rc = check_words("lse", lse)) return rc;
  if (max_pages < 1 || static_cast<int64_t>(max_pages) * c.page_size > INT32_MAX)
    return reject(COLI_EINVAL, "max_pages=%d: need 1 or more and max_pages * page_size < 2^31",
                  max_pages);
  const size_t need =
      paged_direct(c, max_pages) ? 0 : paged_scratch_bytes(c, B, cfg->n_q_heads);
  if (scratch_bytes < need || (need > 0 && (scratch == nullptr || misaligned(scratch, 16))))
    return reject(COLI_EINVAL, "scratch: need %zu bytes, 16-byte aligned, got %zu", need,
                  scratch_bytes);
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
  a.scratch = static_cast<float*>(scratch);
  a.status = device_status_ptr();
  return launched(launch_paged_attention(a, static_cast<cudaStream_t>(stream)),
                  "paged attention");
}

}  // extern "C"
