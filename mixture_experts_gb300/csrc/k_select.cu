// Pages to attend to: those where a query may score highest.
//
// score(p) = max over the key head's query heads of sum_d (q_d > 0 ? q_d largest_d : q_d
// least_d), two plain products, of q's positive part with the largest keys and of its
// negative part with the least.
//
// k_page_scores: 16 pages a warp and step on the warp MMA (pages are its 16 rows, 8 query
// heads its columns, the bounds come from memory straight into the operand's registers: a lane's
// 16 bytes are elements 8t .. + 7 of every 32 on both operands). A third product, |q| with
// the larger magnitude, says how far the fp32 sums may be off: 8 x 2^-24 of the sum
// of magnitudes an instruction, DP / 8 of them a score. fp32 caches: plain FMAs, chains of at
// most 24 roundings: 2^-18.
// k_page_pick: a block a (sequence, key head) finds the keep-th largest score T. Scores further
// than twice the largest error from T are settled; where the others are not just as many
// as are still wanted, they are computed again in fp64 and ranked by that (two to four pages of
// thousands, by themselves; all of a list where more than kFew are open, as with equal pages).
//
// 32 contexts of up to 65536 tokens in pages of 32, 8 heads of 128 (134 MB of bounds): scores 27
// us (4.8 TB/s, 16 warps an SM: 126 registers), choice of 64 pages 15 us. One context of 7813 pages: 10
// and 14 us; a block's choice is a chain of short steps between barriers.
#include "mx.cuh"
#include "paged.cuh"
#include "pick.cuh"

namespace coli {
namespace {

constexpr int kScoreWarps = 4;

struct ScoreArgs {
  SelectArgs s;
  int chunks;  // blocks of a (sequence, key head)
};

// (2^-116: what sums below fp32's normal range lose, 512 products of 2^-126 at most)
COLI_DEV float score_error(float score, float sum, float unit) {
  return score != score || fabsf(score) == INFINITY ? INFINITY : fmaf(sum, unit, 0x1p-116f);
}

template <int DP>
__global__ void __launch_bounds__(kScoreWarps * 32) k_page_scores(const ScoreArgs a) {
  constexpr int kJ = DP / 32;
  const SelectArgs& p = a.s;
  const int bh = blockIdx.x / a.chunks, chunk = blockIdx.x - bh * a.chunks;
  const int b = bh / p.c.n_heads, h = bh - b * p.c.n_heads;
  const int lane = lane_id(), w = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const int D = p.c.head_dim, group = p.n_q_heads / p.c.n_heads, tiles = (group + 7) / 8;
  const int len = context_len(p.seq_lens, b, p.max_pages, p.c.page_size, p.status,
                              h == 0 && chunk == 0 && threadIdx.x == 0);
  const int n = (len + p.c.page_size - 1) / p.c.page_size;
  if (n <= p.keep) return;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride +
                           static_cast<size_t>(h) * group * D;
  const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  float2* out = p.scores + static_cast<size_t>(bh) * p.max_pages;
  const int step = a.chunks * kScoreWarps * 16;
  for (int p0 = (chunk * kScoreWarps + w) * 16; p0 < n; p0 += step) {
    uint4 lo[kJ][2], hi[kJ][2];  // of pages g, g + 8
    bool in[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = p0 + g + 8 * r, at = i < n ? __ldg(table + i) : 0;
      in[r] = at >= 0 && at < p.c.n_pages;
      if (!in[r]) latch_error(p.status, kErrDevice);
      const __nv_bfloat16* src =
          static_cast<const __nv_bfloat16*>(p.bounds) +
          (static_cast<size_t>(in[r] ? at : 0) * p.c.n_heads + h) * 2 * D + t * 8;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const bool live = i < n && in[r] && j * 32 + t * 8 < D;
        lo[j][r] = live ? ldg_stream(src + j * 32) : make_uint4(0, 0, 0, 0);
        hi[j][r] = live ? ldg_stream(src + D + j * 32) : make_uint4(0, 0, 0, 0);
      }
    }
    float best[2] = {-INFINITY, -INFINITY}, off[2] = {0.f, 0.f};
    for (int nt = 0; nt < tiles; ++nt) {
      const bool head = nt * 8 + g < group;
      const __nv_bfloat16* qh = q + static_cast<size_t>(nt * 8 + g) * D + t * 8;
      float x[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const uint4 u = head && j * 32 + t * 8 < D ? ldg_keep(qh + j * 32) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t b0 = word_of(u, 2 * k), b1 = word_of(u, 2 * k + 1);
          uint32_t v[2][4];  // rows g and g + 8, both words: largest, least
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              v[0][2 * e + r] = word_of(hi[j][r], 2 * k + e);
              v[1][2 * e + r] = word_of(lo[j][r], 2 * k + e);
            }
          mma_bf16_16816(x, v[0][0], v[0][1], v[0][2], v[0][3], __vmaxs2(b0, 0u),
                         __vmaxs2(b1, 0u));
          mma_bf16_16816(x, v[1][0], v[1][1], v[1][2], v[1][3], __vmins2(b0, 0u),
                         __vmins2(b1, 0u));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[0][e] = __vmaxu2(v[0][e] & 0x7fff7fffu, v[1][e] & 0x7fff7fffu);
          mma_bf16_16816(m, v[0][0], v[0][1], v[0][2], v[0][3], b0 & 0x7fff7fffu,
                         b1 & 0x7fff7fffu);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (nt * 8 + 2 * t + (c & 1) >= group) continue;
        best[c >> 1] = fmaxf(best[c >> 1], x[c]);
        off[c >> 1] = fmaxf(off[c >> 1], score_error(x[c], m[c], DP / 8 * 0x1p-21f));
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int k = 1; k < 4; k <<= 1) {
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], k));
        off[r] = fmaxf(off[r], __shfl_xor_sync(0xffffffffu, off[r], k));
      }
      const int i = p0 + g + 8 * r;
      if (t == 0 && i < n) out[i] = in[r] ? make_float2(best[r], off[r]) : make_float2(-INFINITY, 0.f);
    }
  }
}

// fp32 bounds: a page a warp, its lanes along the channels.
__global__ void __launch_bounds__(kScoreWarps * 32) k_page_scores_f32(const ScoreArgs a) {
  const SelectArgs& p = a.s;
  const int bh = blockIdx.x / a.chunks, chunk = blockIdx.x - bh * a.chunks;
  const int b = bh / p.c.n_heads, h = bh - b * p.c.n_heads;
  const int lane = lane_id(), w = threadIdx.x / 32;
  const int D = p.c.head_dim, group = p.n_q_heads / p.c.n_heads;
  const int len = context_len(p.seq_lens, b, p.max_pages, p.c.page_size, p.status,
                              h == 0 && chunk == 0 && threadIdx.x == 0);
  const int n = (len + p.c.page_size - 1) / p.c.page_size;
  if (n <= p.keep) return;
  const float* q = static_cast<const float*>(p.q) + b * p.q_stride +
                   static_cast<size_t>(h) * group * D;
  float2* out = p.scores + static_cast<size_t>(bh) * p.max_pages;
  for (int i = chunk * kScoreWarps + w; i < n; i += a.chunks * kScoreWarps) {
    const int at = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + i);
    if (at < 0 || at >= p.c.n_pages) {
      latch_error(p.status, kErrDevice);
      if (lane == 0) out[i] = make_float2(-INFINITY, 0.f);
      continue;
    }
    const float* src = static_cast<const float*>(p.bounds) +
                       (static_cast<size_t>(at) * p.c.n_heads + h) * 2 * D;
    float lo[8], hi[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int d = k * 32 + lane;
      lo[k] = d < D ? __ldg(src + d) : 0.f;
      hi[k] = d < D ? __ldg(src + D + d) : 0.f;
    }
    float best = -INFINITY, off = 0.f;
    for (int r = 0; r < group; ++r) {
      float x = 0.f, m = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = k * 32 + lane;
        const float v = d < D ? __ldg(q + static_cast<size_t>(r) * D + d) : 0.f;
        if (v != 0.f) {
          x = fmaf(v, v > 0.f ? hi[k] : lo[k], x);
          m = fmaf(fabsf(v), fmaxf(fabsf(lo[k]), fabsf(hi[k])), m);
        }
      }
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, k);
        m += __shfl_xor_sync(0xffffffffu, m, k);
      }
      best = fmaxf(best, x);
      off = fmaxf(off, score_error(x, m, 0x1p-18f));
    }
    if (lane == 0) out[i] = make_float2(best, off);
  }
}

constexpr int kFew = 256;  // pages ranked at once
constexpr int kMostCached = 160 * 1024;  // bytes of keys that shared memory holds

// The score of head r of the group in a page, in fp64 (a warp; every lane gets it).
template <class T>
COLI_DEV double score64(const SelectArgs& p, int b, int h, int r, int page) {
  const int D = p.c.head_dim, group = p.n_q_heads / p.c.n_heads;
  if (page < 0 || page >= p.c.n_pages) return -INFINITY;
  const T* box =
      static_cast<const T*>(p.bounds) + (static_cast<size_t>(page) * p.c.n_heads + h) * 2 * D;
  const T* q = static_cast<const T*>(p.q) + b * p.q_stride + static_cast<size_t>(h * group + r) * D;
  float v[8], to[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int d = k * 32 + static_cast<int>(lane_id());
    v[k] = d < D ? to_f32(q[d]) : 0.f;
    const float lo = d < D ? to_f32(box[d]) : 0.f, hi = d < D ? to_f32(box[D + d]) : 0.f;
    to[k] = v[k] > 0.f ? hi : lo;
  }
  double x = 0.;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k * 32 < D && v[k] != 0.f) x = fma(double(v[k]), double(to[k]), x);
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
  return x;
}

// The listed pages' scores as ordered keys, a warp a page and head; those with a NaN: -infinity.
template <class T, int THREADS>
COLI_DEV void exact_scores(const SelectArgs& p, int b, int h, const int32_t* table,
                           const int* list, int m, unsigned long long* keys, int* nan) {
  const int group = p.n_q_heads / p.c.n_heads;
  for (int e = threadIdx.x; e < m; e += THREADS) keys[e] = 0, nan[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x / 32; i < m * group; i += THREADS / 32) {
    const int e = i / group;
    const double x = score64<T>(p, b, h, i - e * group, __ldg(table + list[e]));
    if (lane_id() != 0) continue;
    if (x != x) {
      nan[e] = 1;
      latch_error(p.status, kErrDevice);
    } else {
      atomicMax(&keys[e], static_cast<unsigned long long>(order_key(x)));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < m; e += THREADS)
    if (nan[e]) keys[e] = order_key(-double(INFINITY));
  __syncthreads();
}

template <class T, int kPickThreads, bool CACHED>
__global__ void __launch_bounds__(kPickThreads) k_page_pick(const SelectArgs p) {
  extern __shared__ uint32_t s_keys[];
  __shared__ PickShared s;
  __shared__ int s_list[kFew], s_n;
  __shared__ unsigned long long s_exact[kFew];
  __shared__ int s_nan[kFew];
  __shared__ float s_off[kPickThreads / 32];
  const int b = blockIdx.x / p.c.n_heads, h = blockIdx.x - b * p.c.n_heads;
  const int lane = lane_id(), w = threadIdx.x / 32, page = p.c.page_size;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = context_len(p.seq_lens, b, p.max_pages, page, p.status,
                              h == 0 && threadIdx.x == 0);
  const int n = (len + page - 1) / page;
  const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  int32_t* out = p.pages + static_cast<size_t>(blockIdx.x) * p.keep;
  if (h == 0 && threadIdx.x == 0) p.lens[b] = n > p.keep ? len - (n - p.keep) * page : len;
  if (n <= p.keep) {
    for (int i = threadIdx.x; i < p.keep; i += kPickThreads) out[i] = i < n ? __ldg(table + i) : -1;
    return;
  }
  float2* row = p.scores + static_cast<size_t>(blockIdx.x) * p.max_pages;
  auto forced = [&](int i) { return i < p.first || i >= n - p.last; };
  auto put = [&](int r, int i) { out[r] = __ldg(table + i); };
  // ordered scores, four loads in flight, and the largest error
  float off = 0.f;
  constexpr int kDeep = 4;
  for (int i0 = threadIdx.x; i0 < n; i0 += kPickThreads * kDeep) {
    float2 v[kDeep];
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int i = i0 + e * kPickThreads;
      v[e] = i < n ? row[i] : make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int i = i0 + e * kPickThreads;
      if (i >= n) break;
      if (!forced(i)) off = fmaxf(off, v[e].y);
      if constexpr (CACHED) s_keys[i] = forced(i) ? 0xffffffffu : order_key(v[e].x);
    }
  }
  auto key = [&](int i) {
    if constexpr (CACHED) return s_keys[i];
    return forced(i) ? 0xffffffffu : order_key(row[i].x);
  };
  auto score = [&](int i) {  // of a page that is not forced (NaN: -infinity; all are open then)
    const uint32_t k = key(i);
    return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
  };
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) off = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, k));
  if (lane == 0) s_off[w] = off;
  __syncthreads();
  const Cut<uint32_t> cut = radix_cut<kPickThreads, false, uint32_t>(n, p.keep, key, s);
#pragma unroll
  for (int k = 0; k < kPickThreads / 32; ++k) off = fmaxf(off, s_off[k]);
  if (cut.from == 0xffffffffu) {  // nothing but the first and last pages
    chosen<kPickThreads, uint32_t>(n, cut, key, put, s);
    return;
  }
  const float at = __uint_as_float(cut.from >> 31 ? cut.from ^ 0x80000000u : ~cut.from);
  const float over = __fadd_ru(at, 2.f * off), under = __fadd_rd(at, -2.f * off);
  // scores that are neither surely chosen nor surely not
  auto open = [&](int i) {
    return !forced(i) && !(score(i) > over) && !(score(i) < under);
  };
  int mine = 0;  // all but the surely left out
  for (int i = threadIdx.x; i < n; i += kPickThreads) mine += forced(i) || !(score(i) < under);
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, k);
  if (lane == 0) s.warp[0][w] = mine;
  __syncthreads();
  int within = 0;
#pragma unroll
  for (int k = 0; k < kPickThreads / 32; ++k) within += s.warp[0][k];
  __syncthreads();
  if (within == p.keep) {
    chosen<kPickThreads, uint32_t>(n, Cut<uint32_t>{order_key(under), n}, key, put, s);
    return;
  }
  // Few are open: they are ranked in fp64 by themselves, and their keys say who is chosen.
  if constexpr (CACHED) {
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPickThreads)
      if (open(i)) {
        const int e = atomicAdd(&s_n, 1);
        if (e < kFew) s_list[e] = i;
      }
    __syncthreads();
    const int m = s_n;
    __syncthreads();  // (every warp has read it before the loop below starts it again)
    if (m <= kFew) {
      exact_scores<T, kPickThreads>(p, b, h, table, s_list, m, s_exact, s_nan);
      const int left = p.keep - (within - m);  // places for them
      for (int e = threadIdx.x; e < m; e += kPickThreads) {
        int better = 0;
        for (int k = 0; k < m; ++k)
          better += s_exact[k] > s_exact[e] || (s_exact[k] == s_exact[e] && s_list[k] < s_list[e]);
        s_keys[s_list[e]] = better < left ? 0xffffffffu : 0u;
      }
      __syncthreads();
      chosen<kPickThreads, uint32_t>(n, Cut<uint32_t>{order_key(over), 0}, key, put, s);
      return;
    }
  }
  // Else the open ones' keys go in the scores' place, +-infinity for the others, and all are ranked.
  unsigned long long* exact = reinterpret_cast<unsigned long long*>(row);
  for (int i0 = 0; i0 < n; i0 += kFew) {
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    for (int i = i0 + threadIdx.x; i < min(n, i0 + kFew); i += kPickThreads) {
      if (open(i))
        s_list[atomicAdd(&s_n, 1)] = i;
      else
        exact[i] = order_key(forced(i) || score(i) > over ? double(INFINITY) : -double(INFINITY));
    }
    __syncthreads();
    exact_scores<T, kPickThreads>(p, b, h, table, s_list, s_n, s_exact, s_nan);
    for (int e = threadIdx.x; e < s_n; e += kPickThreads) exact[s_list[e]] = s_exact[e];
    __syncthreads();
  }
  auto key64 = [&](int i) { return forced(i) ? ~0ull : static_cast<uint64_t>(exact[i]); };
  const Cut<uint64_t> cut64 = radix_cut<kPickThreads, true, uint64_t>(n, p.keep, key64, s);
  chosen<kPickThreads, uint64_t>(n, cut64, key64, put, s);
}

template <class T, int THREADS, bool CACHED>
cudaError_t pick_with(const SelectArgs& a, size_t smem, cudaStream_t st) {
  static bool ready[128] = {};
  if (CACHED && smem > 32 * 1024) {
    const cudaError_t e = raise_shared(k_page_pick<T, THREADS, CACHED>, kMostCached, ready);
    if (e != cudaSuccess) return e;
  }
  // few rows are bound by the host, for which the plain launch is cheaper (8 rows 43 against 46
  // us, with the attention after it; 256 rows 94 against 91.5)
  const int rows = a.B * a.c.n_heads;
  if (rows >= 64)
    return launch_after(k_page_pick<T, THREADS, CACHED>, rows, THREADS, smem, st, a);
  k_page_pick<T, THREADS, CACHED><<<rows, THREADS, smem, st>>>(a);
  return cudaGetLastError();
}
// Long lists by 1024 threads; what shared memory does not hold is read again from memory.
template <class T>
cudaError_t launch_pick(const SelectArgs& a, cudaStream_t st) {
  const size_t keys = static_cast<size_t>(a.max_pages) * 4;
  if (keys > kMostCached) return pick_with<T, 1024, false>(a, 0, st);
  if (a.max_pages > 4096) return pick_with<T, 1024, true>(a, keys, st);
  return pick_with<T, 256, true>(a, keys, st);
}

}  // namespace

cudaError_t launch_select_pages(const SelectArgs& a, cudaStream_t st) {
  const int rows = a.B * a.c.n_heads;
  if (a.max_pages > a.keep) {
    // blocks of 64 pages, unless there are many more of them than the GPU takes at once
    const int most = (a.max_pages + kScoreWarps * 16 - 1) / (kScoreWarps * 16);
    const int fill = (sm_count() * 16 + rows - 1) / rows;
    const ScoreArgs p{a, most < fill ? most : fill};
    const unsigned grid = static_cast<unsigned>(rows) * p.chunks;
    const int dp = a.c.head_dim <= 64 ? 64 : (a.c.head_dim <= 128 ? 128 : 256);
    if (a.c.dtype == DT_F32) {
      k_page_scores_f32<<<grid, kScoreWarps * 32, 0, st>>>(p);
    } else {
      auto kernel = dp == 64    ? k_page_scores<64>
                    : dp == 128 ? k_page_scores<128>
                                : k_page_scores<256>;
      kernel<<<grid, kScoreWarps * 32, 0, st>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return a.c.dtype == DT_F32 ? launch_pick<float>(a, st) : launch_pick<__nv_bfloat16>(a, st);
}

}  // namespace coli
