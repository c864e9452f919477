// What each cached token weighed in a decode step, added to its mass.
//
// mass(j) += sum over the key head's query heads of exp(scale q.k_j - lse): with the
// log-sum-exp known the weights need no maximum and no second pass, only the keys.
//
// A warp takes 16 tokens of a (sequence, key head) at once on the warp MMA: tokens are its 16
// rows, 8 query heads its columns (NT column tiles, more heads in further passes over the
// keys). The keys come from memory straight into the operand's registers: of every 32
// channels lane 4g + t has 8t .. + 7 of rows g and g + 8, on both operands. bf16 queries
// and keys are operands as they are; MX codes are widened to fp16, against fp16 queries, and a
// block's scale goes on its sum (queries that fp16 does not hold, or far from 1, meet bf16 keys);
// fp32 runs in three tf32 products of operands in two parts.
//
// 32 bf16 contexts of up to 8192 tokens, 32 heads on 8 of 128 (302 MB): 51 us, 5.9 TB/s, HBM
// bound. 16 MXFP4 contexts of up to 60000, 64 heads on 4 (145 MB): 64 us, 2.3 TB/s: a quarter of
// the bytes at twice the heads, bound by the steps' instructions and their latency with 16
// warps an SM (128 registers; a second tile fetched ahead leaves 12 warps: 79 us).
#include "mx.cuh"
#include "paged.cuh"
#include "pick.cuh"

namespace coli {
namespace {

using namespace paged;

constexpr int kMassWarps = 4;

struct MassGrid {
  MassArgs m;
  int chunks;  // blocks of a (sequence, key head)
};

// Bytes of 8 channels in the cache.
template <int FMT>
constexpr int bytes8() {
  return FMT == DT_F32 ? 32 : FMT == DT_BF16 ? 16 : FMT == DT_MXFP8 ? 8 : 4;
}
template <int FMT>
struct Raw8 {
  uint32_t w[bytes8<FMT>() / 4];
};
template <int FMT>
COLI_DEV Raw8<FMT> load8(const char* p) {
  Raw8<FMT> r;
  if constexpr (FMT == DT_F32) {
    const uint4 a = ldg_stream(p), b = ldg_stream(p + 16);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
  } else if constexpr (FMT == DT_BF16) {
    const uint4 a = ldg_stream(p);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
  } else if constexpr (FMT == DT_MXFP8) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = a.x, r.w[1] = a.y;
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
  return r;
}
// An fp32 score by itself: where infinities met the parts of the split products.
__device__ __noinline__ float plain_score(const float* q, const float* k, int D) {
  float x = 0.f;
  for (int d = 0; d < D; ++d) x = fmaf(q[d], k[d], x);
  return x;
}

template <int FMT, int DP, int NT>
__global__ void __launch_bounds__(kMassWarps * 32) k_mass(const MassGrid a) {
  constexpr int kJ = DP / 32;
  constexpr bool kF32 = FMT == DT_F32, kMx = FMT == DT_MXFP8 || FMT == DT_MXFP4;
  const MassArgs& p = a.m;
  const int bh = blockIdx.x / a.chunks, chunk = blockIdx.x - bh * a.chunks;
  const int b = bh / p.c.n_heads, h = bh - b * p.c.n_heads;
  const int lane = lane_id(), w = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const int D = p.c.head_dim, group = p.n_q_heads / p.c.n_heads, page_size = p.c.page_size;
  const int len = context_len(p.seq_lens, b, p.max_pages, page_size, p.status,
                              h == 0 && chunk == 0 && threadIdx.x == 0);
  const int start = p.window > 0 && len > p.window ? len - p.window : 0;
  const int known = p.known == nullptr ? INT32_MAX : __ldg(p.known + b);
  const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  const int tiles = (len + kTile - 1) / kTile, per_page = page_size / kTile;
  const int t0 = start / kTile + chunk * kMassWarps + w, step = a.chunks * kMassWarps;
  if (t0 >= tiles) return;  // (tile numbers stay below 2^28, and steps far below that)

  for (int r0 = 0; r0 < group; r0 += 8 * NT) {
    // head r0 + 8 nt + g's elements; scales and lse of heads 2t, 2t + 1
    uint32_t q[NT][kJ][kF32 ? 8 : 4];
    float lse[NT][2];
    bool live[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + g;
      const size_t at =
          static_cast<size_t>(b) * p.q_stride + static_cast<size_t>(h * group + r) * D + t * 8;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const bool in = r < group && j * 32 + t * 8 < D;
        const char* src = static_cast<const char*>(p.q) + (at + j * 32) * (kF32 ? 4 : 2);
#pragma unroll
        for (int e = 0; e < (kF32 ? 2 : 1); ++e) {
          const uint4 u = in ? ldg_keep(src + 16 * e) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < 4; ++k) q[nt][j][4 * e + k] = word_of(u, k);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int head = r0 + nt * 8 + 2 * t + c;
        lse[nt][c] = head < group
                         ? __ldg(p.lse + static_cast<size_t>(b) * p.n_q_heads + h * group + head)
                         : -INFINITY;
        live[nt][c] = lse[nt][c] != -INFINITY;
      }
    }
    // MX: queries in fp16, the head's largest element at 2^14, where that is exact (no element
    // but 0 below 2^-31 of it): codes are fp16 numbers, and their scale goes on a block's sum.
    // For heads of 2^-24 to 2^40 and scales of 2^-24 to 2^24: a block's sum, up to 2^29, passes
    // fp32's range then only where scores are 2^(96 - 24 - 24) and more, and the least block
    // scale, which counts as 0, is worth 2^(41 + 24 - 127 + 9 + 8) at most.
    float scale[NT][2];
    const float size = fabsf(p.scale);
    bool half = kMx && size >= 0x1p-24f && size <= 0x1p24f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) scale[nt][0] = scale[nt][1] = p.scale;
    if constexpr (kMx) {
      int e[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) most = __vmaxu2(most, q[nt][j][i] & 0x7fff7fffu);
        uint32_t top = max(most << 16, most & 0x7fff0000u);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        e[nt] = top == 0 ? 0 : static_cast<int>(top >> 23) - 127;
        half = half && e[nt] <= 40 && e[nt] >= -24;
        const uint32_t least = static_cast<uint32_t>(max(e[nt], -24) - 31 + 127) << 23;
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = q[nt][j][i] << 16 & 0x7fffffffu, a1 = q[nt][j][i] & 0x7fff0000u;
            half = half && a0 - 1 >= least - 1 && a1 - 1 >= least - 1;  // 0 wraps round
          }
      }
      half = __all_sync(0xffffffffu, half);
      if (half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float up = __uint_as_float(static_cast<uint32_t>(14 - e[nt] + 127) << 23);
#pragma unroll
          for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              q[nt][j][i] = pack_f16x2(bf16_lo(q[nt][j][i]) * up, bf16_hi(q[nt][j][i]) * up);
          const float down = __uint_as_float(static_cast<uint32_t>(e[nt] - 14 + 127) << 23);
          // block scales below carry a factor 1 + 2^-23
#pragma unroll
          for (int c = 0; c < 2; ++c)
            scale[nt][c] = p.scale * __shfl_sync(0xffffffffu, down, 8 * t + 4 * c) * (1.f - 0x1p-23f);
        }
      } else {
        // keys below bf16's normal range, which show against large heads or scales, go in times 2^64
        bool large = size > 0x1p24f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) large = large || e[nt] > 40;
        if (__any_sync(0xffffffffu, large) && size >= 0x1p-24f) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) scale[nt][0] = scale[nt][1] = p.scale * 0x1p-64f;
        }
      }
    }

    // a tile's keys, MX ones a tile ahead: 1 or 2 KB a warp are too few in flight
    struct Keys {
      Raw8<FMT> raw[kJ][2];
      uint32_t sc[2][2];
      size_t row;
      bool in;
    };
    // the tile whose page is looked up next: its number, page in the table, place in it
    int next = t0, next_pi = t0 / per_page, next_sub = t0 - next_pi * per_page;
    const int step_pi = step / per_page, step_sub = step - step_pi * per_page;
    struct Spot {
      int tile, page, sub;
    };
    auto look_up = [&]() {
      const Spot s{next, next < tiles ? __ldg(table + next_pi) : 0, next_sub};
      next = next < tiles ? next + step : next;
      next_pi += step_pi;
      next_sub += step_sub;
      if (next_sub >= per_page) next_sub -= per_page, ++next_pi;
      return s;
    };
    auto fetch = [&](Keys& k, const Spot& s) {
      k.in = s.tile < tiles && s.page >= 0 && s.page < p.c.n_pages;
      if (!k.in) {
        if (s.tile < tiles && lane == 0) latch_error(p.status, kErrDevice);
        return;
      }
      k.row = kv_row(p.c, s.page, h, s.sub * kTile);
      const char* src = p.c.k + (k.row + g) * p.c.row_bytes + t * bytes8<FMT>();
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          k.raw[j][e] = Raw8<FMT>{};
          if (j * 32 + t * 8 < D)
            k.raw[j][e] = load8<FMT>(src + static_cast<size_t>(e) * 8 * p.c.row_bytes +
                                     j * 4 * bytes8<FMT>());
        }
      if constexpr (kMx) {
        const uint8_t* s = p.c.k_scale + (k.row + g) * p.c.scale_stride;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          k.sc[e][0] = __ldg(reinterpret_cast<const uint32_t*>(s + e * 8 * p.c.scale_stride));
          k.sc[e][1] = 0;
          if (DP > 128 && p.c.scale_stride > 4)
            k.sc[e][1] = __ldg(reinterpret_cast<const uint32_t*>(s + e * 8 * p.c.scale_stride + 4));
        }
      }
    };
    Keys ahead;
    Spot spot = look_up();
    if constexpr (kMx) {
      fetch(ahead, spot);
      spot = look_up();
    }
    for (int tile = t0; tile < tiles; tile += step) {
      Keys now;
      if constexpr (kMx) {
        now = ahead;
        fetch(ahead, spot);
      } else {
        fetch(now, spot);
      }
      spot = look_up();
      if (!now.in) continue;
      auto& raw = now.raw;
      auto& sc = now.sc;
      const size_t row = now.row;
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[nt][c] = 0.f;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        if constexpr (kF32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float hi[4], lo[4];
            split_tf32(__uint_as_float(raw[j][0].w[2 * e]), &hi[0], &lo[0]);
            split_tf32(__uint_as_float(raw[j][1].w[2 * e]), &hi[1], &lo[1]);
            split_tf32(__uint_as_float(raw[j][0].w[2 * e + 1]), &hi[2], &lo[2]);
            split_tf32(__uint_as_float(raw[j][1].w[2 * e + 1]), &hi[3], &lo[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float qh[2], ql[2];
              split_tf32(__uint_as_float(q[nt][j][2 * e]), &qh[0], &ql[0]);
              split_tf32(__uint_as_float(q[nt][j][2 * e + 1]), &qh[1], &ql[1]);
              mma_tf32_1688(x[nt], lo, qh);
              mma_tf32_1688(x[nt], hi, ql);
              mma_tf32_1688(x[nt], hi, qh);
            }
          }
        } else if constexpr (FMT == DT_BF16) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(x[nt], raw[j][0].w[0], raw[j][1].w[0], raw[j][0].w[1], raw[j][1].w[1],
                           q[nt][j][0], q[nt][j][1]);
            mma_bf16_16816(x[nt], raw[j][0].w[2], raw[j][1].w[2], raw[j][0].w[3], raw[j][1].w[3],
                           q[nt][j][2], q[nt][j][3]);
          }
        }
      }
      if constexpr (kMx) {
        // bytes past the head's blocks may hold anything
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < (DP > 128 ? 2 : 1); ++i) {
            const int n = D / kMxBlock - 4 * i;
            sc[e][i] &= n >= 4 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
          }
        if (half) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            // as fp32 bits with the last one set: byte 255 is then NaN by itself (and byte 0,
            // 2^-127, counts as 0)
            const int up = 23 - 8 * (j % 4);
            const float f0 = __uint_as_float(
                ((up > 0 ? sc[0][j / 4] << (up & 31) : sc[0][j / 4] >> 1) & 0x7f800000u) | 1u);
            const float f1 = __uint_as_float(
                ((up > 0 ? sc[1][j / 4] << (up & 31) : sc[1][j / 4] >> 1) & 0x7f800000u) | 1u);
            uint32_t k0[4], k1[4];
            if constexpr (FMT == DT_MXFP8) {
              e4m3x8_f16(raw[j][0].w[0], raw[j][0].w[1], k0);
              e4m3x8_f16(raw[j][1].w[0], raw[j][1].w[1], k1);
            } else {
              e2m1x8_f16(raw[j][0].w[0], k0);
              e2m1x8_f16(raw[j][1].w[0], k1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float d[4];
              mma_f16_16816_z(d, k0[0], k1[0], k0[1], k1[1], q[nt][j][0], q[nt][j][1]);
              mma_f16_16816(d, k0[2], k1[2], k0[3], k1[3], q[nt][j][2], q[nt][j][3]);
#pragma unroll
              for (int c = 0; c < 4; ++c) x[nt][c] = fmaf(d[c], c < 2 ? f0 : f1, x[nt][c]);
            }
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < kJ; ++j) {  // rare: widened to bf16 with their scale
            const float up = scale[0][0] == p.scale ? 1.f : 0x1p64f;
            uint32_t w[2][2], k0[4], k1[4], qj[NT][4];
            const int last = bytes8<FMT>() / 4 - 1;
            float f[2];
#pragma unroll
            for (int i = 0; i < kJ; ++i) {
              if (i != j) continue;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                w[e][0] = raw[i][e].w[0], w[e][1] = raw[i][e].w[last];
                f[e] = e8m0_f32(sc[e][i / 4] >> 8 * (i % 4) & 0xffu) * up;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) qj[nt][k] = q[nt][i][k];
            }
            mx8_bf16<FMT>(w[0][0], w[0][1], f[0], k0);
            mx8_bf16<FMT>(w[1][0], w[1][1], f[1], k1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16_16816(x[nt], k0[0], k1[0], k0[1], k1[1], qj[nt][0], qj[nt][1]);
              mma_bf16_16816(x[nt], k0[2], k1[2], k0[3], k1[3], qj[nt][2], qj[nt][3]);
            }
          }
        }
      }
      if constexpr (kF32) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (x[nt][c] != x[nt][c] && live[nt][c & 1])
              x[nt][c] = plain_score(
                  static_cast<const float*>(p.q) + static_cast<size_t>(b) * p.q_stride +
                      static_cast<size_t>(h * group + r0 + nt * 8 + 2 * t + (c & 1)) * D,
                  reinterpret_cast<const float*>(p.c.k) + (row + g + (c >> 1) * 8) * D, D);
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float y = fmaf(x[nt][c], scale[nt][c & 1], -lse[nt][c & 1]) * 1.4426950408889634f;
          sum[c >> 1] += live[nt][c & 1] ? ex2(y) : 0.f;
        }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 1; k < 4; k <<= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], k);
      const int at = g + (t & 1) * 8, j = tile * kTile + at;
      if (t < 2 && j >= start && j < len) {
        float* m = p.mass + row + at;
        const float v = t ? sum[1] : sum[0];
        if (j >= known && r0 == 0)
          *m = v;
        else
          atomicAdd(m, v);
      }
    }
  }
}

template <int FMT, int DP>
void launch_group(const MassGrid& p, unsigned grid, cudaStream_t st) {
  // two column tiles where there are heads for them and registers (fp32 heads of 256 spill)
  constexpr bool kTwo = FMT != DT_F32 || DP < 256;
  if constexpr (kTwo)
    if (p.m.n_q_heads / p.m.c.n_heads > 8) {
      k_mass<FMT, DP, 2><<<grid, kMassWarps * 32, 0, st>>>(p);
      return;
    }
  k_mass<FMT, DP, 1><<<grid, kMassWarps * 32, 0, st>>>(p);
}
template <int FMT>
void launch_heads(const MassGrid& p, unsigned grid, cudaStream_t st) {
  if (p.m.c.head_dim <= 64)
    launch_group<FMT, 64>(p, grid, st);
  else if (p.m.c.head_dim <= 128)
    launch_group<FMT, 128>(p, grid, st);
  else
    launch_group<FMT, 256>(p, grid, st);
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t st) {
  const int rows = a.B * a.c.n_heads;
  const int64_t tiles = static_cast<int64_t>(a.max_pages) * (a.c.page_size / kTile);
  const int64_t most = (tiles + kMassWarps - 1) / kMassWarps;
  const int fill = (sm_count() * 16 + rows - 1) / rows;
  const MassGrid p{a, static_cast<int>(most < fill ? most : fill)};
  const unsigned grid = static_cast<unsigned>(rows) * p.chunks;
  switch (a.c.dtype) {
    case DT_F32: launch_heads<DT_F32>(p, grid, st); break;
    case DT_BF16: launch_heads<DT_BF16>(p, grid, st); break;
    case DT_MXFP8: launch_heads<DT_MXFP8>(p, grid, st); break;
    default: launch_heads<DT_MXFP4>(p, grid, st);
  }
  return cudaGetLastError();
}

}  // namespace coli
