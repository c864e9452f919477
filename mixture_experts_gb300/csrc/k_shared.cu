// Attention behind a shared prefix: the prefix once for the queries of all sequences, each
// sequence's own tokens as ever, and a join.
#include "paged.cuh"

namespace coli {
namespace {

using namespace paged;

struct JoinArgs {
  const float* mean[2];   // prefix, own: [rows][head_dim] fp32
  const float2* ml[2];    // (m, l): weights are 2^(x - m), their sum l
  void* out;
  float* lse;
  size_t out_stride;
  int rows, heads, D;     // rows = B * heads
};

constexpr int kJoinWarps = 8;

template <class T>
__global__ void __launch_bounds__(kJoinWarps * 32) k_shared_join(const JoinArgs p) {
  const int row = blockIdx.x * kJoinWarps + threadIdx.x / 32, lane = lane_id();
  if (row >= p.rows) return;
  float w[2], l = 0.f, top = -FLT_MAX;
  float2 ml[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ml[i] = p.ml[i][row];
    top = fmaxf(top, ml[i].x);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = ml[i].y * ex2(ml[i].x - top);
    l += w[i];
  }
  const int b = row / p.heads, h = row - b * p.heads;
  T* out = static_cast<T*>(p.out) + b * p.out_stride + static_cast<size_t>(h) * p.D;
  for (int d = lane * 4; d < p.D; d += 128) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (ml[i].y == 0.f) continue;
      const float4 v =
          *reinterpret_cast<const float4*>(p.mean[i] + static_cast<size_t>(row) * p.D + d);
      const float f = w[i] / l;
      o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
    }
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(out + d) = o;
    else
      *reinterpret_cast<uint2*>(out + d) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

// Of one side's means and (m, l) pairs.
size_t side_bytes(const KvView& c, int64_t rows) {
  return align16(rows * c.head_dim * sizeof(float)) + align16(rows * sizeof(float2));
}

}  // namespace

size_t shared_scratch_bytes(const KvView& c, int B, int n_q_heads) {
  const int64_t rows = static_cast<int64_t>(B) * n_q_heads;
  const size_t one = paged_scratch_bytes(c, 1, static_cast<int>(rows));
  const size_t own = paged_scratch_bytes(c, B, n_q_heads);
  return 2 * side_bytes(c, rows) + align16(one > own ? one : own);
}

cudaError_t launch_shared_attention(const SharedArgs& s, cudaStream_t st) {
  const KvView& c = s.own.c;
  const int rows = s.own.B * s.own.n_q_heads;
  const size_t side = side_bytes(c, rows);
  char* at = static_cast<char*>(s.scratch);
  JoinArgs j{};
  for (int i = 0; i < 2; ++i) {
    j.mean[i] = reinterpret_cast<float*>(at + i * side);
    j.ml[i] = reinterpret_cast<float2*>(at + i * side + align16(size_t(rows) * c.head_dim * 4));
  }
  PagedArgs a = s.own;
  a.scratch = reinterpret_cast<float*>(at + 2 * side);
  if (s.prefix_len == 0) return launch_paged_attention(a, st);
  a.out_stride = static_cast<size_t>(a.n_q_heads) * c.head_dim;
  a.raw = 1;
  {
    PagedArgs f = a;
    f.out = const_cast<float*>(j.mean[0]);
    f.lse = reinterpret_cast<float*>(const_cast<float2*>(j.ml[0]));
    f.block_table = s.prefix_pages;
    f.max_pages = (s.prefix_len + c.page_size - 1) / c.page_size;
    f.fixed_len = s.prefix_len;
    f.fold = a.n_q_heads / c.n_heads;
    f.n_q_heads = rows;
    f.B = 1;
    const cudaError_t e = launch_paged_attention(f, st);
    if (e != cudaSuccess) return e;
  }
  a.out = const_cast<float*>(j.mean[1]);
  a.lse = reinterpret_cast<float*>(const_cast<float2*>(j.ml[1]));
  const cudaError_t e = launch_paged_attention(a, st);
  if (e != cudaSuccess) return e;
  j.out = s.own.out;
  j.lse = s.own.lse;
  j.out_stride = s.own.out_stride;
  j.rows = rows;
  j.heads = a.n_q_heads;
  j.D = c.head_dim;
  const unsigned grid = (rows + kJoinWarps - 1) / kJoinWarps;
  if (c.dtype == DT_F32)
    k_shared_join<float><<<grid, kJoinWarps * 32, 0, st>>>(j);
  else
    k_shared_join<__nv_bfloat16><<<grid, kJoinWarps * 32, 0, st>>>(j);
  return cudaGetLastError();
}

}  // namespace coli
