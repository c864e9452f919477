// Reading the paged key-value cache back: slots -> rows in the activation
// type. One thread writes 16 bytes of a row (from 16, 8 or 4 stored ones) for
// each of four rows, whose loads it has in flight together.
#include "attn.h"
#include "common.cuh"
#include "mx.cuh"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 4;

struct ReadArgs {
  KvView c;
  const int32_t* slots;
  char* out[2];  // k, v (either may be nullptr)
  size_t stride[2];  // bytes between tokens
  uint32_t rows;     // N * sides * n_heads
  int sides, first;  // sides: 1 or 2 outputs; first: 1 when only v is read
  int* status;
};

template <int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_read(const ReadArgs p) {
  constexpr int kSrc = FMT == DT_MXFP8 ? 8 : (FMT == DT_MXFP4 ? 4 : 16);  // bytes a thread loads
  const int out_row = p.c.head_dim * (FMT == DT_F32 ? 4 : 2);
  const int cpr = out_row / 16, rows = kThreads / cpr;
  const int local = threadIdx.x / cpr, c = threadIdx.x % cpr;
  if (local >= rows) return;
  const uint32_t base = blockIdx.x * static_cast<uint32_t>(rows * kRowsPerThread) + local;
  uint4 raw[kRowsPerThread];
  uint32_t scale[kRowsPerThread];
  char* dst[kRowsPerThread];
#pragma unroll
  for (int n = 0; n < kRowsPerThread; ++n) {
    const uint32_t r = base + n * rows;
    dst[n] = nullptr;
    raw[n] = make_uint4(0, 0, 0, 0);
    scale[n] = 127;
    if (r >= p.rows) continue;
    const uint32_t tok = r / (p.sides * p.c.n_heads);
    const int rest = r - tok * (p.sides * p.c.n_heads);
    const int side = p.first + rest / p.c.n_heads, h = rest % p.c.n_heads;
    dst[n] = p.out[side] + tok * p.stride[side] + static_cast<size_t>(h) * out_row + c * 16;
    const int slot = p.slots[tok];
    if (slot < 0 || slot >= p.c.n_pages * p.c.page_size) {
      if (slot != -1 && rest == 0 && c == 0) latch_error(p.status, kErrDevice);
      continue;
    }
    const int page = slot / p.c.page_size;
    const size_t row = kv_row(p.c, page, h, slot - page * p.c.page_size);
    const char* src = (side ? p.c.v : p.c.k) + row * p.c.row_bytes + c * kSrc;
    if constexpr (kSrc == 16) {
      raw[n] = *reinterpret_cast<const uint4*>(src);
    } else {
      if constexpr (kSrc == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(src);
        raw[n].x = u.x, raw[n].y = u.y;
      } else {
        raw[n].x = *reinterpret_cast<const uint32_t*>(src);
      }
      scale[n] = (side ? p.c.v_scale : p.c.k_scale)[row * p.c.scale_stride + c / 4];
    }
  }
#pragma unroll
  for (int n = 0; n < kRowsPerThread; ++n) {
    if (dst[n] == nullptr) continue;
    uint4 o = raw[n];
    if constexpr (kSrc != 16) {
      uint32_t h[4];
      if constexpr (kSrc == 8)
        e4m3x8_f16(raw[n].x, raw[n].y, h);
      else
        e2m1x8_f16(raw[n].x, h);
      float x[8];
      f16x8_f32(h, x);
      const float s = e8m0_f32(scale[n]);
      o = make_uint4(pack_bf16x2(x[0] * s, x[1] * s), pack_bf16x2(x[2] * s, x[3] * s),
                     pack_bf16x2(x[4] * s, x[5] * s), pack_bf16x2(x[6] * s, x[7] * s));
    }
    *reinterpret_cast<uint4*>(dst[n]) = o;
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
  p.sides = (k_out != nullptr) + (v_out != nullptr);
  p.first = k_out == nullptr;
  const int64_t rows = static_cast<int64_t>(N) * p.sides * c.n_heads;
  const int per_block = kThreads / (c.head_dim * e / 16) * kRowsPerThread;
  if (rows + per_block > INT32_MAX) return cudaErrorInvalidValue;
  p.rows = static_cast<uint32_t>(rows);
  p.status = status;
  const unsigned grid = static_cast<unsigned>((rows + per_block - 1) / per_block);
  switch (c.dtype) {
    case DT_F32: k_kv_read<DT_F32><<<grid, kThreads, 0, st>>>(p); break;
    case DT_BF16: k_kv_read<DT_BF16><<<grid, kThreads, 0, st>>>(p); break;
    case DT_MXFP8: k_kv_read<DT_MXFP8><<<grid, kThreads, 0, st>>>(p); break;
    default: k_kv_read<DT_MXFP4><<<grid, kThreads, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace coli
