// Attention of one new token a sequence over its paged context.
//
// One block per (sequence, query head); its warps take the keys in turn. A
// warp holds its query in registers (lane l: elements l, l + 32, ...), keeps
// the running maximum m and sum l of the softmax over its keys and the
// weighted values o, and rescales them when the maximum grows; the block joins
// its warps at the end:  m = max m_w,  l = sum l_w 2^(m_w - m),  o likewise.
#include <math.h>

#include "attn.h"
#include "common.cuh"
#include "mx.cuh"

namespace coli {
namespace {

constexpr int kWarps = 8;

template <int FMT>
COLI_DEV float element(const char* row, const uint8_t* scales, int d) {
  if constexpr (FMT == DT_F32) return reinterpret_cast<const float*>(row)[d];
  if constexpr (FMT == DT_BF16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
  uint32_t h[4];
  if constexpr (FMT == DT_MXFP8) {
    e4m3x8_f16(static_cast<uint8_t>(row[d]), 0, h);
  } else {
    const uint32_t byte = static_cast<uint8_t>(row[d / 2]);
    e2m1x8_f16(d % 2 ? byte >> 4 : byte & 15u, h);
  }
  float x[8];
  f16x8_f32(h, x);
  return x[0] * e8m0_f32(scales[d / kMxBlock]);
}

template <int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_paged(const PagedArgs a) {
  constexpr int kPer = kMaxHeadDim / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kMaxHeadDim];
  const int b = blockIdx.y, hq = blockIdx.x, D = a.c.head_dim;
  const int h = hq / (a.n_q_heads / a.c.n_heads);
  const int w = threadIdx.x / 32, lane = lane_id();
  int len = a.seq_lens[b];
  const int most = a.max_pages * a.c.page_size;
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) latch_error(a.status, kErrDevice);
    len = len < 0 ? 0 : most;
  }
  const int start = a.window > 0 && len > a.window ? len - a.window : 0;
  const size_t qo = b * a.q_stride + static_cast<size_t>(hq) * D;
  float q[kPer], o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = lane + 32 * i;
    o[i] = q[i] = 0.f;
    if (d < D)
      q[i] = FMT == DT_F32 ? static_cast<const float*>(a.q)[qo + d]
                           : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[qo + d]);
  }
  float m = -INFINITY, l = 0.f;
  for (int j = start + w; j < len; j += kWarps) {
    const int pi = j / a.c.page_size;
    const int page = a.block_table[static_cast<size_t>(b) * a.max_pages + pi];
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) latch_error(a.status, kErrDevice);
      continue;
    }
    const size_t row = kv_row(a.c, page, h, j - pi * a.c.page_size);
    const char* kr = a.c.k + row * a.c.row_bytes;
    const char* vr = a.c.v + row * a.c.row_bytes;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = lane + 32 * i;
      if (d < D) s += q[i] * element<FMT>(kr, a.c.k_scale + row * a.c.scale_stride, d);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale;
    const float mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float old = expf(m - base), p = expf(s - base);
    l = l * old + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = lane + 32 * i;
      if (d < D) o[i] = o[i] * old + p * element<FMT>(vr, a.c.v_scale + row * a.c.scale_stride, d);
    }
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < D) so[w][lane + 32 * i] = o[i];
  if (lane == 0) sm[w] = m, sl[w] = l;
  __syncthreads();
  float mm = -INFINITY;
  for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, sm[i]);
  const float base = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  for (int i = 0; i < kWarps; ++i) ll += sl[i] * expf(sm[i] - base);
  const size_t oo = b * a.out_stride + static_cast<size_t>(hq) * D;
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float x = 0.f;
    for (int i = 0; i < kWarps; ++i) x += so[i][d] * expf(sm[i] - base);
    x = ll == 0.f ? 0.f : x / ll;
    if constexpr (FMT == DT_F32)
      static_cast<float*>(a.out)[oo + d] = x;
    else
      static_cast<__nv_bfloat16*>(a.out)[oo + d] = __float2bfloat16_rn(x);
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[static_cast<size_t>(b) * a.n_q_heads + hq] = ll == 0.f ? -INFINITY : logf(ll) + base;
}

}  // namespace

size_t paged_scratch_bytes(const KvView& c, int B, int n_q_heads) { return 0; }

cudaError_t launch_paged_attention(const PagedArgs& a, cudaStream_t st) {
  const dim3 grid(a.n_q_heads, a.B);
  switch (a.c.dtype) {
    case DT_F32: k_paged<DT_F32><<<grid, kWarps * 32, 0, st>>>(a); break;
    case DT_BF16: k_paged<DT_BF16><<<grid, kWarps * 32, 0, st>>>(a); break;
    case DT_MXFP8: k_paged<DT_MXFP8><<<grid, kWarps * 32, 0, st>>>(a); break;
    default: k_paged<DT_MXFP4><<<grid, kWarps * 32, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace coli
