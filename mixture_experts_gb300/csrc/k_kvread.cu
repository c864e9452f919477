// Reading the paged key-value cache back: slots -> rows in the activation
// type. One thread writes the same 16 bytes of the key and the value row (from
// 16, 8 or 4 stored ones each) for up to four tokens, whose loads it has in
// flight together; its head and place in the row stay the same over them. HBM
// bound: 65536 MXFP8 tokens of 8 heads of 128 (407 MB) in 65.5 us, 6.2 TB/s. Blocks
// an SM, 5 / 6, in us of back-to-back reads: MXFP8 71 / 67, MXFP4 65 / 61, BF16 84 / 87
// and F32 160 / 166 (these have 16 bytes a load and then spill). Evict-first stores
// took 64 for MXFP8, but the rows are read next. An MX value is formed in fp32
// (exact) and rounded once.
#include "attn.h"
#include "common.cuh"
#include "mx.cuh"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;

struct ReadArgs {
  KvView c;
  const int32_t* slots;
  char* out[2];      // k, v (either may be nullptr)
  size_t stride[2];  // bytes between tokens
  int N;
  int units;         // 16-byte pieces of a token's key rows
  int per_block;     // tokens a block takes at once (units <= kThreads), else 1
  int page_shift;    // log2(page_size), or -1
  int* status;
};

template <int FMT>
__global__ void __launch_bounds__(kThreads, FMT == DT_MXFP8 || FMT == DT_MXFP4 ? 6 : 5)
    k_kv_read(const ReadArgs p) {
  // bytes a piece of 16 comes from
  constexpr int kSrc = FMT == DT_MXFP8 ? 8 : (FMT == DT_MXFP4 ? 4 : 16);
  const int out_row = p.c.head_dim * (FMT == DT_F32 ? 4 : 2);
  int local = 0, unit = blockIdx.y * kThreads + threadIdx.x;
  if (p.units <= kThreads) {
    local = threadIdx.x / p.units;
    unit = threadIdx.x - local * p.units;
    if (local >= p.per_block) return;
  }
  if (unit >= p.units) return;
  const int h = unit / (out_row / 16), c = unit - h * (out_row / 16);
  const int base = blockIdx.x * (p.per_block * kTokens) + local;
  int slot[kTokens];
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    const int tok = base + n * p.per_block;
    slot[n] = tok < p.N ? __ldg(p.slots + tok) : -1;
  }
  uint4 raw[kTokens][2];
  uint32_t scale[kTokens][2];
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    raw[n][0] = raw[n][1] = make_uint4(0, 0, 0, 0);
    scale[n][0] = scale[n][1] = 127;
    if (slot[n] < 0 || slot[n] >= p.c.n_pages * p.c.page_size) {
      if (slot[n] != -1 && unit == 0) latch_error(p.status, kErrDevice);
      continue;
    }
    const int page = p.page_shift >= 0 ? slot[n] >> p.page_shift : slot[n] / p.c.page_size;
    const size_t row = kv_row(p.c, page, h, slot[n] - page * p.c.page_size);
    const size_t at = row * p.c.row_bytes + c * kSrc;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (p.out[s] == nullptr) continue;
      const char* src = (s ? p.c.v : p.c.k) + at;
      if constexpr (kSrc == 16) {
        raw[n][s] = *reinterpret_cast<const uint4*>(src);
      } else {
        if constexpr (kSrc == 8) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          raw[n][s].x = u.x, raw[n][s].y = u.y;
        } else {
          raw[n][s].x = *reinterpret_cast<const uint32_t*>(src);
        }
        scale[n][s] = (s ? p.c.v_scale : p.c.k_scale)[row * p.c.scale_stride + c / 4];
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    const int tok = base + n * p.per_block;
    if (tok >= p.N) break;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (p.out[s] == nullptr) continue;
      uint4 o = raw[n][s];
      if constexpr (kSrc != 16) {
        uint32_t hf[4];
        if constexpr (kSrc == 8)
          e4m3x8_f16(raw[n][s].x, raw[n][s].y, hf);
        else
          e2m1x8_f16(raw[n][s].x, hf);
        float x[8];
        f16x8_f32(hf, x);
        const float f = e8m0_f32(scale[n][s]);
        o = make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                       pack_bf16x2(x[4] * f, x[5] * f), pack_bf16x2(x[6] * f, x[7] * f));
      }
      *reinterpret_cast<uint4*>(p.out[s] + tok * p.stride[s] + static_cast<size_t>(h) * out_row +
                                c * 16) = o;
    }
  }
}

}  // namespace

cudaError_t launch_kv_read(const KvView& c, const int32_t* slots, int N, void* k_out,
                           size_t k_stride, void* v_out, size_t v_stride, int* status,
                           cudaStream_t st) {
  const int e = c.dtype == DT_F32 ? 4 : 2;
  ReadArgs p{};
  p.c = c;
  p.slots = slots;
  p.out[0] = static_cast<char*>(k_out);
  p.out[1] = static_cast<char*>(v_out);
  p.stride[0] = k_stride * e;
  p.stride[1] = v_stride * e;
  p.N = N;
  p.units = c.n_heads * (c.head_dim * e / 16);
  p.per_block = p.units <= kThreads ? kThreads / p.units : 1;
  p.page_shift = -1;
  for (int i = 0; i < 13; ++i)
    if (c.page_size == 1 << i) p.page_shift = i;
  p.status = status;
  const dim3 grid((N + p.per_block * kTokens - 1) / (p.per_block * kTokens),
                  p.units <= kThreads ? 1 : (p.units + kThreads - 1) / kThreads);
  switch (c.dtype) {
    case DT_F32: k_kv_read<DT_F32><<<grid, kThreads, 0, st>>>(p); break;
    case DT_BF16: k_kv_read<DT_BF16><<<grid, kThreads, 0, st>>>(p); break;
    case DT_MXFP8: k_kv_read<DT_MXFP8><<<grid, kThreads, 0, st>>>(p); break;
    default: k_kv_read<DT_MXFP4><<<grid, kThreads, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace coli
