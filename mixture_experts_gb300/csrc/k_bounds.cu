// Bounds of pages: the least and largest key of each channel among a page's tokens,
// from which a query's largest possible score in the page follows.
//
// A warp takes one head of one listed page. The head's rows of a page are contiguous:
// lane l reads 16-byte unit l % U of rows l / U, l / U + S, ... (U units a row, S = 32 / U
// rows at once), four rows in flight, keeps minima and maxima of its unit's channels in
// packed bf16 (exact: they are keys; MX ones are formed in fp32 and rounded once, as the
// cache's read does) and the S lanes of a unit are joined by a shuffle tree.
//
// 4099 pages of 64 MXFP8 tokens, 8 heads of 128 (292 MB): 62 us, 4.7 TB/s, bound by the integer
// pipe (71% busy: conversions, packing, minima and maxima). In fp16, codes times a scale
// relative to the page's largest, the steps are half as many, but the scales have to be read
// first: 75 us.
#include "attn.h"
#include "common.cuh"
#include "mx.cuh"

namespace coli {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 4;  // rows a lane has in flight

struct BoundsArgs {
  KvView c;
  const int32_t* pages;
  const int32_t* fills;
  char* bounds;
  int N;
  int* status;
};

COLI_DEV uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
COLI_DEV uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
COLI_DEV uint32_t min_f32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
COLI_DEV uint32_t max_f32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_page_bounds(const BoundsArgs p) {
  constexpr int W = words16<FMT>();
  constexpr bool kF32 = FMT == DT_F32, kMx = FMT == DT_MXFP8 || FMT == DT_MXFP4;
  const int lane = lane_id();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  const int i = static_cast<int>(item / p.c.n_heads), head = static_cast<int>(item % p.c.n_heads);
  if (i >= p.N) return;
  const int page = __ldg(p.pages + i), fill = __ldg(p.fills + i);
  if (page == -1) return;
  if (page < 0 || page >= p.c.n_pages || fill < 1 || fill > p.c.page_size) {
    if (lane == 0) latch_error(p.status, kErrDevice);
    return;
  }
  const size_t row0 = kv_row(p.c, page, head, 0);
  const int units = p.c.row_bytes / 16, D = p.c.head_dim;
  const int U = units < 32 ? units : 32, S = 32 / U;
  const int slice = lane / U;
  for (int u0 = 0; u0 < units; u0 += 32) {
    const int unit = u0 + lane - slice * U;
    const bool mine = slice < S && unit < units;
    uint32_t lo[W], hi[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      lo[k] = kF32 ? 0x7f800000u : 0x7f807f80u;
      hi[k] = kF32 ? 0xff800000u : 0xff80ff80u;
    }
    if (mine) {
      const char* src = p.c.k + row0 * p.c.row_bytes + unit * 16;
      // MXFP8: 16 codes a unit, half a block
      const uint8_t* sc = kMx ? p.c.k_scale + row0 * p.c.scale_stride +
                                    (FMT == DT_MXFP8 ? unit / 2 : unit)
                              : nullptr;
      for (int r = slice; r < fill; r += S * kBatch) {
        uint4 raw[kBatch];
        uint32_t s[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int at = min(r + e * S, fill - 1);  // past the end: the last row again
          raw[e] = ldg_stream(src + static_cast<uint32_t>(at * p.c.row_bytes));
          s[e] = kMx ? __ldg(sc + static_cast<uint32_t>(at * p.c.scale_stride)) : 0;
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          uint32_t w[W];
          decode16<FMT>(raw[e], s[e], w);
#pragma unroll
          for (int k = 0; k < W; ++k) {
            lo[k] = kF32 ? min_f32(lo[k], w[k]) : min_bf16x2(lo[k], w[k]);
            hi[k] = kF32 ? max_f32(hi[k], w[k]) : max_bf16x2(hi[k], w[k]);
          }
        }
      }
    }
    // slices k apart, halving k
    int k0 = 1;
    while (k0 < S) k0 *= 2;
    for (int k = k0 / 2; k >= 1; k /= 2) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t a = __shfl_down_sync(0xffffffffu, lo[j], U * k);
        const uint32_t b = __shfl_down_sync(0xffffffffu, hi[j], U * k);
        if (slice + k < S) {
          lo[j] = kF32 ? min_f32(lo[j], a) : min_bf16x2(lo[j], a);
          hi[j] = kF32 ? max_f32(hi[j], b) : max_bf16x2(hi[j], b);
        }
      }
    }
    if (slice == 0 && mine) {
      const int row = D * (kF32 ? 4 : 2);
      char* out = p.bounds + (row0 / p.c.page_size) * 2 * row + unit * (W * 4);
#pragma unroll
      for (int k = 0; k < W; k += 4) {
        *reinterpret_cast<uint4*>(out + k * 4) = make_uint4(lo[k], lo[k + 1], lo[k + 2], lo[k + 3]);
        *reinterpret_cast<uint4*>(out + row + k * 4) =
            make_uint4(hi[k], hi[k + 1], hi[k + 2], hi[k + 3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_page_bounds(const KvView& c, const int32_t* pages, const int32_t* fills, int N,
                               void* bounds, int* status, cudaStream_t st) {
  const BoundsArgs p{c, pages, fills, static_cast<char*>(bounds), N, status};
  const int64_t items = static_cast<int64_t>(N) * c.n_heads;
  const unsigned grid = static_cast<unsigned>((items + kWarps - 1) / kWarps);
  switch (c.dtype) {
    case DT_F32: k_page_bounds<DT_F32><<<grid, kWarps * 32, 0, st>>>(p); break;
    case DT_BF16: k_page_bounds<DT_BF16><<<grid, kWarps * 32, 0, st>>>(p); break;
    case DT_MXFP8: k_page_bounds<DT_MXFP8><<<grid, kWarps * 32, 0, st>>>(p); break;
    default: k_page_bounds<DT_MXFP4><<<grid, kWarps * 32, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace coli
