// Eviction by accumulated weight: each key head of a sequence keeps its first and
// last tokens and those of the largest mass, whose rows are then copied together.
//
// k_evict_pick: a block a (sequence, key head); the masses come through the page table into
// shared memory as ordered keys (tokens that are kept anyway: the largest key), and
// pick.cuh finds the keep-th largest and lists the kept places in rising order.
// A block's choice takes 14 us of 2176 tokens and 25 of 32768: loads of pages and masses, a pass
// for the range, up to three over the digits, two to list.
// k_evict_copy: into other pages, a block takes 64 kept tokens of a (sequence, key head),
// keys and values and their scales and masses, 16 bytes a thread and step (64 sequences of 2048
// bf16 tokens, 8 heads of 128, 1.1 GB read and written: 164 us, 6.6 TB/s).
// k_evict_pack: in place. A kept row moves to an earlier place or stays, so rows copied
// in order, each batch read before it is written, never overwrite one that is still to be
// read. A block takes 128 bytes of all of a head's rows (or its scales, or masses):
// blocks share no byte. The same sequences in place: 222 us with the choice, against 180.
#include "mx.cuh"
#include "pick.cuh"

namespace coli {
namespace {

constexpr int kMostCached = 200 * 1024;  // bytes of keys that shared memory holds

template <int THREADS, bool CACHED>
__global__ void __launch_bounds__(THREADS) k_evict_pick(const EvictArgs p) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ PickShared s;
  const int b = blockIdx.x / p.c.n_heads, h = blockIdx.x - b * p.c.n_heads;
  const int page = p.c.page_size;
  const int n = context_len(p.seq_lens, b, p.max_pages, page, p.status, threadIdx.x == 0);
  int32_t* out = p.kept + static_cast<size_t>(blockIdx.x) * p.keep;
  if (h == 0 && threadIdx.x == 0) p.new_lens[b] = min(n, p.keep);
  const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  if (n <= p.keep) {
    for (int i = threadIdx.x; i < p.keep; i += THREADS) out[i] = i < n ? i : -1;
    return;
  }
  auto load = [&](int i) {
    if (i < p.first || i >= n - p.recent) return 0xffffffffu;
    const int pi = i / page, at = __ldg(table + pi);
    if (at < 0 || at >= p.c.n_pages) {
      latch_error(p.status, kErrDevice);
      return order_key(-INFINITY);
    }
    return order_key(__ldg(p.mass + kv_row(p.c, at, h, i - pi * page)));
  };
  if constexpr (CACHED) {  // four tokens of a page at once, eight such loads in flight
    constexpr int kDeep = THREADS == 1024 ? 8 : 4;
    const uint32_t per = 0xffffffffu / page + 1;  // i * per / 2^32 is i / page, or one more
    const bool whole = (reinterpret_cast<uintptr_t>(p.mass) & 15) == 0;
    for (int i0 = threadIdx.x * 4; i0 < n; i0 += THREADS * 4 * kDeep) {
      int at[kDeep], off[kDeep];
      float4 m[kDeep];
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        const int i = i0 + e * THREADS * 4;
        int pi = __umulhi(i, per);
        if (pi * page > i) --pi;
        off[e] = i - pi * page;
        at[e] = i < n ? __ldg(table + pi) : 0;
      }
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        const bool in = at[e] >= 0 && at[e] < p.c.n_pages;
        if (!in) latch_error(p.status, kErrDevice);
        m[e] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (!in || i0 + e * THREADS * 4 >= n) continue;
        const float* src = p.mass + kv_row(p.c, at[e], h, off[e]);
        if (whole)
          m[e] = __ldg(reinterpret_cast<const float4*>(src));
        else
          m[e] = make_float4(__ldg(src), __ldg(src + 1), __ldg(src + 2), __ldg(src + 3));
      }
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        const int i = i0 + e * THREADS * 4;
        if (i >= n) break;
        uint4 k = make_uint4(order_key(m[e].x), order_key(m[e].y), order_key(m[e].z),
                             order_key(m[e].w));
        if (i < p.first || i + 4 > n - p.recent) {  // kept anyway
          auto forced = [&](int t) { return t < p.first || t >= n - p.recent; };
          k.x = forced(i) ? 0xffffffffu : k.x;
          k.y = forced(i + 1) ? 0xffffffffu : k.y;
          k.z = forced(i + 2) ? 0xffffffffu : k.z;
          k.w = forced(i + 3) ? 0xffffffffu : k.w;
        }
        *reinterpret_cast<uint4*>(s_keys + i) = k;  // past the last token: room, never read
      }
    }
    __syncthreads();
  }
  auto key = [&](int i) {
    if constexpr (CACHED) return s_keys[i];
    return load(i);
  };
  const Cut<uint32_t> cut = radix_cut<THREADS, true, uint32_t>(n, p.keep, key, s);
  chosen<THREADS, uint32_t>(n, cut, key, [&](int r, int i) { out[r] = i; }, s);
}

// Row of the kept token of rank r, and the one it goes to; false where either page is none
// of the pool's.
COLI_DEV bool rows_of(const EvictArgs& p, int b, int h, int from, int r, size_t* src,
                      size_t* dst) {
  const int page = p.c.page_size;
  const int sp = from / page, dp = r / page;
  const int sa = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + sp);
  const int da = __ldg(p.into + static_cast<size_t>(b) * p.into_pages + dp);
  if (sa < 0 || sa >= p.c.n_pages || da < 0 || da >= p.c.n_pages) {
    latch_error(p.status, kErrDevice);
    return false;
  }
  *src = kv_row(p.c, sa, h, from - sp * page);
  *dst = kv_row(p.c, da, h, r - dp * page);
  return true;
}

constexpr int kCopyThreads = 256, kRanks = 64, kUnits = 4;

__global__ void __launch_bounds__(kCopyThreads) k_evict_copy(const EvictArgs p, int chunks) {
  __shared__ size_t s_src[kRanks], s_dst[kRanks];
  __shared__ int s_in[kRanks];
  const int bh = blockIdx.x / chunks, r0 = (blockIdx.x - bh * chunks) * kRanks;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = bh / p.c.n_heads, h = bh - b * p.c.n_heads;
  const int32_t* kept = p.kept + static_cast<size_t>(bh) * p.keep;
  if (threadIdx.x < kRanks) {
    const int r = r0 + threadIdx.x, from = r < p.keep ? kept[r] : -1;
    s_in[threadIdx.x] =
        from >= 0 && rows_of(p, b, h, from, r, &s_src[threadIdx.x], &s_dst[threadIdx.x]);
    if (s_in[threadIdx.x]) p.mass[s_dst[threadIdx.x]] = p.mass[s_src[threadIdx.x]];
  }
  __syncthreads();
  if (kept[r0] < 0) return;
  const int U = p.c.row_bytes / 16, n = kRanks * U;
#pragma unroll
  for (int pool = 0; pool < 2; ++pool) {
    char* base = pool ? p.c.v : p.c.k;
    for (int i0 = threadIdx.x; i0 < n; i0 += kCopyThreads * kUnits) {
      uint4 v[kUnits];
      size_t to[kUnits];
#pragma unroll
      for (int e = 0; e < kUnits; ++e) {
        const int i = i0 + e * kCopyThreads, r = i / U, u = i - r * U;
        to[e] = ~size_t(0);
        if (i < n && s_in[r]) {
          v[e] = *reinterpret_cast<const uint4*>(base + s_src[r] * p.c.row_bytes + u * 16);
          to[e] = s_dst[r] * p.c.row_bytes + u * 16;
        }
      }
#pragma unroll
      for (int e = 0; e < kUnits; ++e)
        if (to[e] != ~size_t(0)) *reinterpret_cast<uint4*>(base + to[e]) = v[e];
    }
    if (p.c.scale_stride) {
      uint8_t* sc = pool ? p.c.v_scale : p.c.k_scale;
      const int words = p.c.scale_stride / 4;
      for (int i = threadIdx.x; i < kRanks * words; i += kCopyThreads) {
        const int r = i / words, u = i - r * words;
        if (s_in[r])
          *reinterpret_cast<uint32_t*>(sc + s_dst[r] * p.c.scale_stride + u * 4) =
              *reinterpret_cast<const uint32_t*>(sc + s_src[r] * p.c.scale_stride + u * 4);
      }
    }
  }
}

// Pieces of sizeof(T) bytes, `units` (a power of two up to 8) side by side from byte `off` of
// each row of `base`, kPackRanks rows at a time: their places come a batch ahead through shared
// memory, all pieces of a batch are read before one is written.
constexpr int kPackRanks = 128, kSlice = 128;

template <class T>
COLI_DEV void pack_rows(const EvictArgs& p, int b, int h, char* base, int row, int off, int units) {
  __shared__ size_t s_src[2][kPackRanks], s_dst[2][kPackRanks];
  constexpr size_t kStay = ~size_t(0);
  constexpr int kDeep = kPackRanks * 8 / kCopyThreads;
  const int32_t* kept = p.kept + (static_cast<size_t>(b) * p.c.n_heads + h) * p.keep;
  auto places = [&](int r0, int buf) {
    if (threadIdx.x >= kPackRanks) return;
    const int r = r0 + threadIdx.x, from = r < p.keep ? kept[r] : -1;
    size_t src, dst;
    // (a row that stays is not touched)
    const bool move = from > r && rows_of(p, b, h, from, r, &src, &dst);
    s_src[buf][threadIdx.x] = move ? src : kStay;
    s_dst[buf][threadIdx.x] = move ? dst : 0;
  };
  places(0, 0);
  __syncthreads();
  int buf = 0;
  const int shift = __ffs(units) - 1, each = kPackRanks << shift;
  for (int r0 = 0; r0 < p.keep; r0 += kPackRanks, buf ^= 1) {
    T v[kDeep];
    size_t to[kDeep];
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int i = threadIdx.x + e * kCopyThreads, r = i >> shift, u = i & (units - 1);
      const size_t src = i < each ? s_src[buf][r] : kStay;
      to[e] = kStay;
      if (src != kStay) {
        v[e] = *reinterpret_cast<const T*>(base + src * row + off + u * sizeof(T));
        to[e] = s_dst[buf][r] * row + off + u * sizeof(T);
      }
    }
    places(r0 + kPackRanks, buf ^ 1);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kDeep; ++e)
      if (to[e] != kStay) *reinterpret_cast<T*>(base + to[e]) = v[e];
  }
}

// Slices of kSlice bytes of the keys' rows, then of the values'; masses; scales.
__global__ void __launch_bounds__(kCopyThreads) k_evict_pack(const EvictArgs p, int slices) {
  const int kinds = 2 * slices + 1 + (p.c.scale_stride ? 2 : 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int bh = blockIdx.x / kinds, x = blockIdx.x - bh * kinds;
  const int b = bh / p.c.n_heads, h = bh - b * p.c.n_heads;
  // a sequence that is kept whole stays where it is
  if (context_len(p.seq_lens, b, p.max_pages, p.c.page_size, p.status, false) <= p.keep) return;
  if (x < 2 * slices) {
    // the row's last slice may be narrower: a row is a multiple of 16 bytes
    char* base = x < slices ? p.c.k : p.c.v;
    int off = x % slices * kSlice, left = min(kSlice, p.c.row_bytes - off);
    for (int width = kSlice; width >= 16; width /= 2)
      if (left & width) {
        pack_rows<uint4>(p, b, h, base, p.c.row_bytes, off, width / 16);
        off += width;
        __syncthreads();
      }
  } else if (x == 2 * slices) {
    pack_rows<uint32_t>(p, b, h, reinterpret_cast<char*>(p.mass), 4, 0, 1);
  } else {
    pack_rows<uint32_t>(p, b, h,
                        reinterpret_cast<char*>(x == 2 * slices + 1 ? p.c.k_scale : p.c.v_scale),
                        p.c.scale_stride, 0, p.c.scale_stride / 4);
  }
}

template <int THREADS, bool CACHED>
cudaError_t launch_pick(const EvictArgs& a, size_t smem, cudaStream_t st) {
  static bool ready[128] = {};
  if (CACHED && smem > 32 * 1024) {
    const cudaError_t e = raise_shared(k_evict_pick<THREADS, CACHED>, kMostCached, ready);
    if (e != cudaSuccess) return e;
  }
  k_evict_pick<THREADS, CACHED><<<a.B * a.c.n_heads, THREADS, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st) {
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.c.page_size;
  cudaError_t e;
  if (most * 4 > kMostCached)
    e = launch_pick<1024, false>(a, 0, st);
  else if (most > 8192)
    e = launch_pick<1024, true>(a, most * 4, st);
  else
    e = launch_pick<256, true>(a, most * 4, st);
  if (e != cudaSuccess) return e;
  const int rows = a.B * a.c.n_heads;
  if (a.into != a.block_table) {
    const int chunks = (a.keep + kRanks - 1) / kRanks;
    return launch_after(k_evict_copy, static_cast<unsigned>(static_cast<int64_t>(rows) * chunks),
                        kCopyThreads, 0, st, a, chunks);
  } else {
    const int slices = (a.c.row_bytes + kSlice - 1) / kSlice;
    const int kinds = 2 * slices + 1 + (a.c.scale_stride ? 2 : 0);
    return launch_after(k_evict_pack, static_cast<unsigned>(static_cast<int64_t>(rows) * kinds),
                        kCopyThreads, 0, st, a, slices);
  }
}

}  // namespace coli
