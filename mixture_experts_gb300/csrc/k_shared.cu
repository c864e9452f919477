// Attention behind a shared prefix: the prefix once for the queries of all sequences (k_prefix,
// or the decode kernel with all queries as one group), each sequence's own tokens by the decode
// kernel, whose first blocks start under k_prefix's last, and a join. 64 sequences behind
// 32768 bf16 tokens with up to 512 of their own: 76 us, of which k_prefix 54; 128 behind 40009
// MXFP8 ones with up to 1000: 266 us, 201 of them k_prefix.
#include "paged.cuh"
#include "prefix.h"

namespace coli {
namespace {

using namespace paged;

// The parts of a row: its sequence's own tokens, and those of the prefix. The prefix's lie
// in one array of rows like the own ones (n_parts 1) or in the slots of k_prefix's pieces.
struct JoinArgs {
  const float* own;      // [rows][D] means
  const float2* own_ml;  // (m, l): weights are 2^(x - m), their sum l
  const float* mean;     // of the prefix
  const float2* ml;
  int64_t tiles, per;    // of a segment and a block on k_prefix's line; 0: rows as above
  int row_tiles, seg_rows, halves;
  int group;
  void* out;
  float* lse;
  size_t out_stride;
  int rows, heads, D;    // rows = B * heads
};

constexpr int kJoinWarps = 8;

// A warp a row (and half of its channels, blockIdx.y, where those have segments of their own),
// its lanes along the channels. Every factor is a part's share of the weights, so
// a mean stays one; parts are added in their order.
template <class T>
__global__ void __launch_bounds__(kJoinWarps * 32) k_shared_join(const JoinArgs p) {
  const int row = blockIdx.x * kJoinWarps + threadIdx.x / 32, lane = lane_id();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= p.rows) return;
  const int b = row / p.heads, hq = row - b * p.heads;
  size_t first = row;  // part i: row first + i * step
  int n = 1, step = 0;
  if (p.per > 0) {
    const int h = hq / p.group, r = b * p.group + hq - h * p.group;
    const int64_t seg =
        (static_cast<int64_t>(h) * p.row_tiles + r / p.seg_rows) * p.halves + blockIdx.y;
    const int64_t c0 = seg * p.tiles / p.per, c1 = ((seg + 1) * p.tiles - 1) / p.per;
    first = static_cast<size_t>(c0 + seg) * p.seg_rows + r % p.seg_rows;
    n = static_cast<int>(c1 - c0) + 1;
    step = p.seg_rows;
  }
  const float2 own = p.own_ml[row];
  float top = own.x, l = 0.f;
  // (m, l) of up to 32 parts at once, a part a lane
  auto part = [&](int i) {
    return i < n ? p.ml[first + static_cast<size_t>(i) * step] : make_float2(-FLT_MAX, 0.f);
  };
  const float2 mine = part(lane);
  top = fmaxf(top, mine.x);
  for (int i = lane + 32; i < n; i += 32) top = fmaxf(top, part(i).x);
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  const float w0 = own.y * ex2(own.x - top);
  l = mine.y * ex2(mine.x - top);
  for (int i = lane + 32; i < n; i += 32) {
    const float2 v = part(i);
    l += v.y * ex2(v.x - top);
  }
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  l += w0;
  T* out = static_cast<T*>(p.out) + b * p.out_stride + static_cast<size_t>(hq) * p.D;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int d0 = blockIdx.y * 128; d0 < p.D; d0 += gridDim.y * 128) {
    const int d = d0 + lane * 4;
    const bool in = d < p.D;
    float4 o = zero;
    auto add = [&](const float4& v, float w) {
      const float f = w / l;
      o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
    };
    const float4 last =
        in ? *reinterpret_cast<const float4*>(p.own + static_cast<size_t>(row) * p.D + d) : zero;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const float2 ml = i0 == 0 ? mine : part(i0 + lane);
      const float w = ml.y * ex2(ml.x - top);
      constexpr int kDeep = 8;  // loads in flight
      const int i1 = min(n - i0, 32);
      for (int i = 0; i < i1; i += kDeep) {
        float4 v[kDeep];
#pragma unroll
        for (int e = 0; e < kDeep; ++e)
          v[e] = in && i + e < i1
                     ? *reinterpret_cast<const float4*>(
                           p.mean + (first + static_cast<size_t>(i0 + i + e) * step) * p.D + d)
                     : zero;
#pragma unroll
        for (int e = 0; e < kDeep; ++e) {
          // (a part without weight may hold anything)
          const float f = i + e < i1 ? __shfl_sync(0xffffffffu, w, i + e) : 0.f;
          if (f != 0.f) add(v[e], f);
        }
      }
    }
    if (w0 != 0.f) add(last, w0);
    if (!in) continue;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(out + d) = o;
    else
      *reinterpret_cast<uint2*>(out + d) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
  if (p.lse != nullptr && blockIdx.y == 0 && lane == 0)
    p.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

// Of means and (m, l) pairs.
size_t mean_bytes(const KvView& c, int64_t rows) { return align16(rows * c.head_dim * 4); }
size_t part_bytes(const KvView& c, int64_t rows) { return mean_bytes(c, rows) + align16(rows * 8); }

// Whether k_prefix takes the prefix: 128 queries of a key head cost it as much as one, the decode
// kernel reads the prefix once for every 8 or 16. The call replayed, us, k_prefix / decode
// kernel at 8, 9, 16, 24, 64 queries of a key head, 8 key heads:
//   behind 32768  bf16, heads of 128  40 / 39  41 / 50  40 / 51  39 / 53   41 / 74
//                 bf16, 256           76 / 62  76 / 82  76 / 82  77 / 121  79 / 193
//                 MXFP8, 128          42 / 36  47 / 47  47 / 49  47 / 68   48 / 109
//                 MXFP8, 64           40 / 29  40 / 35  41 / 36  41 / 48   41 / 68
//                 MXFP4, 64           40 / 27  40 / 31  40 / 31  40 / 38   41 / 52
//   behind 4096   bf16, 128           15 / 19  15 / 25  15 / 25  15 / 26   20 / 32
//                 MXFP8, 64           15 / 19  15 / 24  15 / 24  15 / 25   21 / 32
//                 MXFP4, 64           14 / 18  14 / 22  15 / 22  15 / 23   20 / 29
// One threshold for all lengths: the scratch is sized before the prefix's is known. It costs MX
// heads of 64 with 9 to 16 queries 5 to 9 us behind the longest prefixes and saves them 7 to 9
// behind short ones. MX heads above 128, whose codes would not fit beside what they are
// widened to, stay with the decode kernel. (k_prefix numbers the pool's rows in 31 bits.)
bool on_tensor_cores(const KvView& c, int rows_of_head) {
  return c.dtype != DT_F32 && (c.head_dim <= 128 || c.dtype == DT_BF16) && rows_of_head > 8 &&
         static_cast<int64_t>(c.n_pages) * c.n_heads * c.page_size < INT32_MAX;
}

// Rows of a segment of k_prefix: 256, two 128-row tiles that share the loads of keys and values, or
// 128, whose two streams take the tiles by turns. Of an odd number of tiles the last pair is
// half idle. The call behind 32768 tokens with 8 key heads, us, in pairs / alone:
//   tiles of a head     2        3         4         5         6         11         13
//   bf16, heads of 128  68 / 71  98 / 83   111 / 116 144 / 130 151 / 162 269 / 255  305 / 312
//   bf16, 64            50 / 47  78 / 64   86 / 82   115 / 100 120 / 116 219 / 203  255 / 237
//   MXFP8, 128          75 / 81  106 / 111 118 / 141 154 / 171 163 / 200 293 / 355  339 / 409
//   MXFP8, 64           60 / 70  94 / 99   103 / 128 139 / 156 145 / 178 266 / 316  310 / 370
//   MXFP4, 128          74 / 74  103 / 100 115 / 129 151 / 157 157 / 185 284 / 329  328 / 381
//   MXFP4, 64           60 / 68  94 / 96   103 / 124 139 / 152 145 / 178 266 / 314  310 / 368
// A pair saves bf16 tiles, whose loads both halves share, 1 to 2 us a tile, and MX ones, which are
// widened once for both, 2 to 7; an idle half costs what a tile does. bf16 heads to 64 lose in pairs
// throughout (40 tiles: 719 / 707). (Two tiles' queries of heads above 128 leave no room for keys.)
int segment_rows(const KvView& c, int rows_of_head) {
  const int tiles = (rows_of_head + kPrefixRows - 1) / kPrefixRows;
  const bool even = tiles % 2 == 0;
  const bool pair = c.dtype == DT_BF16 ? c.head_dim > 64 && c.head_dim <= 128 && (even || tiles >= 13)
                                       : even || tiles >= 5;
  return pair ? 2 * kPrefixRows : kPrefixRows;
}

// Rows of the prefix's partial results.
int64_t prefix_rows(const KvView& c, int B, int n_q_heads) {
  const int rows = B * (n_q_heads / c.n_heads);
  if (!on_tensor_cores(c, rows)) return static_cast<int64_t>(B) * n_q_heads;
  const int seg_rows = segment_rows(c, rows);
  const int64_t segments = static_cast<int64_t>(c.n_heads) *
                           ((rows + seg_rows - 1) / seg_rows) * prefix_halves(c.head_dim);
  return (segments + sm_count()) * seg_rows;
}

}  // namespace

size_t shared_scratch_bytes(const KvView& c, int B, int n_q_heads) {
  const int64_t rows = static_cast<int64_t>(B) * n_q_heads;
  const size_t one = paged_scratch_bytes(c, 1, static_cast<int>(rows));
  const size_t own = paged_scratch_bytes(c, B, n_q_heads);
  return part_bytes(c, rows) + part_bytes(c, prefix_rows(c, B, n_q_heads)) +
         align16(one > own ? one : own);
}

cudaError_t launch_shared_attention(const SharedArgs& s, cudaStream_t st) {
  const KvView& c = s.own.c;
  const int B = s.own.B, heads = s.own.n_q_heads, rows = B * heads, group = heads / c.n_heads;
  const int64_t parts = prefix_rows(c, B, heads);
  char* own = static_cast<char*>(s.scratch);
  char* prefix = own + part_bytes(c, rows);
  float* own_mean = reinterpret_cast<float*>(own);
  float2* own_ml = reinterpret_cast<float2*>(own + mean_bytes(c, rows));
  float* mean = reinterpret_cast<float*>(prefix);
  float2* ml = reinterpret_cast<float2*>(prefix + mean_bytes(c, parts));
  PagedArgs a = s.own;
  a.scratch = reinterpret_cast<float*>(prefix + part_bytes(c, parts));
  if (s.prefix_len == 0) return launch_paged_attention(a, st);

  JoinArgs j{own_mean, own_ml, mean, ml, 0, 0, 0, 0, 1, group, a.out, a.lse, a.out_stride, rows,
             heads, c.head_dim};
  a.raw = 1;
  a.ext = 1;
  a.may_cut = 1;
  a.out_stride = static_cast<size_t>(heads) * c.head_dim;
  cudaError_t e;
  if (on_tensor_cores(c, B * group)) {
    PrefixArgs p{};
    p.c = c;
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.pages = s.prefix_pages;
    p.len = s.prefix_len;
    p.group = group;
    p.rows = B * group;
    const int seg_rows = segment_rows(c, p.rows);
    p.pair = seg_rows == 2 * kPrefixRows;
    p.row_tiles = (p.rows + seg_rows - 1) / seg_rows;
    p.tiles = (p.len + kPrefixKeys - 1) / kPrefixKeys;
    p.total = static_cast<int64_t>(c.n_heads) * p.row_tiles * prefix_halves(c.head_dim) * p.tiles;
    const int grid = p.total < sm_count() ? static_cast<int>(p.total) : sm_count();
    p.per = (p.total + grid - 1) / grid;
    p.box = c.page_size & -c.page_size;
    p.box = p.box > kPrefixKeys ? kPrefixKeys : p.box;
    p.pool_rows = c.n_pages * c.n_heads * c.page_size;
    p.scale = a.scale;
    p.mean = mean;
    p.ml = ml;
    p.status = a.status;
    j.tiles = p.tiles;
    j.per = p.per;
    j.row_tiles = p.row_tiles;
    j.seg_rows = seg_rows;
    j.halves = prefix_halves(c.head_dim);
    e = launch_prefix(p, grid, st);
    a.overlap = 1;  // the own tokens need none of its results
  } else {
    PagedArgs f = a;
    f.out = mean;
    f.lse = reinterpret_cast<float*>(ml);
    f.block_table = s.prefix_pages;
    f.max_pages = (s.prefix_len + c.page_size - 1) / c.page_size;
    f.fixed_len = s.prefix_len;
    f.fold = group;
    f.n_q_heads = rows;
    f.B = 1;
    e = launch_paged_attention(f, st);
  }
  if (e != cudaSuccess) return e;
  a.out = own_mean;
  a.lse = reinterpret_cast<float*>(own_ml);
  e = launch_paged_attention(a, st);
  if (e != cudaSuccess) return e;
  const dim3 grid((rows + kJoinWarps - 1) / kJoinWarps, j.halves);
  return c.dtype == DT_F32
             ? launch_after(k_shared_join<float>, grid, kJoinWarps * 32, 0, st, j)
             : launch_after(k_shared_join<__nv_bfloat16>, grid, kJoinWarps * 32, 0, st, j);
}

}  // namespace coli
