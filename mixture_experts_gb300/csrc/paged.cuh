// Attention of one new token a sequence over its paged context, on the warp
// tensor-core MMA (the query heads of one key head are at most a few rows: a
// 128-row tcgen05 tile would be 90% padding, and the kernel streams the cache
// from HBM far below either pipe's rate).
//
// Mathematics. For the G query heads of a key head, x_j = scale log2(e) q.k_j
// and o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m), one pass over the keys
// with a running maximum m. Both products are taken transposed, keys and value
// channels on the MMA's 16 rows and 8 query heads on its columns:
//   S^T[16 keys][8 heads] = K[16 x D] Q^T,     O^T[D][8 heads] += V^T[D x 16] P^T,
// so a group of up to 8 heads fills its tile, and the tile of S^T becomes the
// other product's operand by two 8x8 register transposes. m is only raised
// when a score passes it by kSlack: one vote a tile instead of a reduction.
//
// Work split. The tiles of 16 keys of every (sequence, key head, block of
// heads) lie on one line that is cut into equal pieces, one per block, so
// ragged lengths load every SM alike. A block that covers a whole segment
// writes its output; a segment cut by block borders leaves partial sums that
// k_join adds in order of the blocks (no atomics: the same bits every time).
// Within a block warp w takes tiles w, w + W, ... with its own ring of
// shared-memory slots filled by cp.async (rows past the context zero-filled),
// so no warp waits for another before the segment's end.
#pragma once

#include <float.h>

#include "attn.h"
#include "common.cuh"
#include "mx.cuh"

namespace coli {
namespace paged {

constexpr int kTile = 16;  // keys a warp takes at once

struct Params {
  PagedArgs a;
  int group;       // query heads of a key head
  int blocks;      // blocks of 8 * NT heads a group is cut into
  float* part;     // partial sums, two slots a block
  int4* span;      // per block: the cut segment that starts in it
};

template <int FMT, int DP, int NT>
struct Cfg {
  static constexpr bool kMx = FMT == DT_MXFP8 || FMT == DT_MXFP4;
  static constexpr int kBits = FMT == DT_F32 ? 32 : FMT == DT_BF16 ? 16 : FMT == DT_MXFP8 ? 8 : 4;
  static constexpr int kRow = DP * kBits / 8;          // bytes of a row in shared memory
  static constexpr int kScaleRow = kMx ? (DP > 128 ? 8 : 4) : 0;
  // whole 128-byte lines: addresses within a line are XORed
  static constexpr int kSlot = (kTile * (kRow + kScaleRow) + 127) / 128 * 128;
  static constexpr int kRegs = DP / 16 * 4 * NT;       // O^T registers of a lane
  static constexpr int kWarps = kSlot > 8192 + 256 || NT * DP == 256 && NT == 2 ? 4 : 8;
  static constexpr int kPerSm =
      DP * NT <= 128 && kSlot <= 4096 + 256 ? 2 : (NT == 2 && DP * NT == 256 ? 3 : 1);
  static constexpr int kBudget = (kPerSm == 3 ? 74 : (kPerSm == 2 ? 112 : 224)) * 1024;
  static constexpr int kFit = kBudget / (kWarps * kSlot);
  // odd, so key and value slots alternate through the ring with one lead
  static constexpr int kRing = kFit >= 7 ? 7 : (kFit >= 5 ? 5 : 3);
  static constexpr int kRingBytes = kRing * kWarps * kSlot;
  static constexpr int kMergeBytes = kWarps * kRegs * 128;
  static constexpr int kMain = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  static constexpr int kSmem = kMain + kWarps * 8 * NT * 8;
  static_assert(kRing * kWarps * kSlot <= kBudget, "ring does not fit");
  static constexpr int kPart = kRegs * 32 + 16 * NT;   // floats of a partial slot
};

// ---- small pieces --------------------------------------------------------------------
COLI_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
COLI_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
COLI_DEV uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 8x8 transpose of 16-bit elements over the warp (lane 4g + t: row g, columns 2t, 2t + 1).
COLI_DEV uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
COLI_DEV void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
COLI_DEV void mma_tf32_1688(float (&d)[4], const float (&a)[4], const float (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
        "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])));
}
// x = hi + lo with hi on the 11 bits a tf32 operand keeps, lo the exact rest
// rounded to as many (22 bits together; the truncated hi cannot overflow).
COLI_DEV void split_tf32(float x, float* hi, float* lo) {
  *hi = __uint_as_float(__float_as_uint(x) & 0xffffe000u);
  const float r = fabsf(x) == INFINITY ? 0.f : x - *hi;
  uint32_t u;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(u) : "f"(r));
  *lo = __uint_as_float(u);
}
COLI_DEV void cp_async16_n(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
COLI_DEV void cp_async4_n(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
COLI_DEV uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
COLI_DEV uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Where 16-byte piece c of row r lies in a tile: the piece's place XORed, within
// its 128 bytes, with a number of the row chosen so that the lanes of one
// shared-memory phase meet 8 different pieces: rows g = 0..7 when keys are read
// (lane 4g + t holds 8 elements from 8t on of every 32), rows 2t when values
// are (8 elements from 8g on of every 64).
template <int FMT, int ROW, bool KEYS>
COLI_DEV constexpr uint32_t row_xor(int r) {
  if (KEYS) {
    if (FMT == DT_F32) return r & 1;
    if (FMT == DT_BF16) return (r & 1) << 2;
    if (FMT == DT_MXFP8) return ROW >= 128 ? (r & 3) << 1 : ((r >> 1) & 1) << 1;
    return ROW >= 128 ? r & 7 : (ROW >= 64 ? (r >> 1) & 3 : (r >> 2) & 1);
  }
  if (FMT == DT_F32) return ((r >> 1) & 1) | (((r >> 2) & 1) << 2);
  return ROW >= 64 ? r & 6 : ((r >> 2) & 1) << 1;
}
template <int FMT, int ROW, bool KEYS>
COLI_DEV uint32_t piece(int r, int c) {
  return ((r * (ROW / 16) + c) ^ row_xor<FMT, ROW, KEYS>(r)) * 16;
}
// Address `off` bytes further on in a tile, for offsets whose bits the lane's
// own place leaves clear: within a 128-byte line they are XORed too.
COLI_DEV uint32_t further(uint32_t at, uint32_t off) { return (at ^ (off & 127u)) + (off & ~127u); }

// Starts the copy of one tile's keys or values into a slot (a multiple of 128).
// Lane l takes the pieces l, l + 32, ... of the tile's memory: `place` is its
// first piece's place, src its address. Rows outside [r0, r1) and bytes past
// row_bytes become zeros.
template <class C, int FMT, bool KEYS>
COLI_DEV void copy_tile(uint32_t slot, uint32_t place, const char* src, int row_bytes, int r0,
                        int r1, int lane) {
  constexpr int kPieces = C::kRow / 16;
  constexpr int kIters = kTile * kPieces / 32;
  const uint32_t dst = slot + place;
  if (r0 <= 0 && r1 >= kTile && row_bytes == C::kRow) {
#pragma unroll
    for (int i = 0; i < kIters; ++i)
      cp_async16_n((dst ^ (row_xor<FMT, C::kRow, KEYS>(i * 32 / kPieces) * 16)) + i * 512,
                   src + i * 512, 16);
  } else {
    const char* tile = src - lane * 16;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int p = i * 32 + lane, r = p / kPieces, c = p % kPieces;
      const bool in = r >= r0 && r < r1 && c * 16 < row_bytes;
      cp_async16_n((dst ^ (row_xor<FMT, C::kRow, KEYS>(i * 32 / kPieces) * 16)) + i * 512,
                   in ? tile + r * row_bytes + c * 16 : src, in ? 16 : 0);
    }
  }
}

// And of its scales, one word a lane.
template <class C>
COLI_DEV void copy_scales(uint32_t slot, const uint8_t* src, int r0, int r1, int lane) {
  constexpr int kWords = C::kScaleRow / 4;
  if (lane < kTile * kWords) {
    const int r = lane / kWords;
    cp_async4_n(slot + kTile * C::kRow + lane * 4, src + lane * 4, r >= r0 && r < r1 ? 4 : 0);
  }
}

// Bytes equal to 0 or 255 in a word of scales (2^-127 and NaN need care).
COLI_DEV bool odd_scales(uint32_t w) {
  const uint32_t n = ~w;
  return (((w - 0x01010101u) & n) | ((n - 0x01010101u) & w)) & 0x80808080u;
}

// The line of work: tiles of sequence b, in tiles of 16 keys counted from the
// context's start.
struct Seq {
  int len, first, n;  // length, first tile, number of tiles
};
COLI_DEV Seq seq_of(const PagedArgs& a, int b, bool latch) {
  int len = __ldg(a.seq_lens + b);
  const int most = a.max_pages * a.c.page_size;
  if (len < 0 || len > most) {
    if (latch) latch_error(a.status, kErrDevice);
    len = len < 0 ? 0 : most;
  }
  const int start = a.window > 0 && len > a.window ? len - a.window : 0;
  const int first = start / kTile;
  return {len, first, (len + kTile - 1) / kTile - first};
}

template <int FMT, int DP, int NT>
__global__ void __launch_bounds__(Cfg<FMT, DP, NT>::kWarps * 32, Cfg<FMT, DP, NT>::kPerSm)
    k_paged(const Params p) {
  using C = Cfg<FMT, DP, NT>;
  constexpr int W = C::kWarps, kJ = DP / 32, kV = DP / 64;
  constexpr bool kF32 = FMT == DT_F32, kMx = C::kMx;
  // Weights rise to 2^kSlack over the running maximum before it is raised;
  // fp16 weights (MX caches) are held 2^kLift higher, up to 2^15, so that they
  // keep 9 bits or more down to 2^-30 of the largest.
  constexpr float kSlack = kMx ? 1.f : 8.f, kLift = kMx ? 14.f : 0.f;
  extern __shared__ __align__(128) char smem[];
  __shared__ long long s_scan[W + 2];
  const PagedArgs& a = p.a;
  const int lane = lane_id(), w = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const int hr_n = a.c.n_heads * p.blocks;  // segments of a sequence

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) p.span[blockIdx.x] = make_int4(0, 0, 0, 0);

  // ---- this block's piece of the line --------------------------------------------------
  int b = 0;
  long long before = 0, total = 0;  // tiles before sequence b, tiles in all
  long long u0 = 0, u1 = 0, per = 0;
  if (a.B <= 32) {  // every warp scans the lengths itself
    const int n = lane < a.B ? seq_of(a, lane, blockIdx.x == 0 && w == 0).n : 0;
    long long s = n;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, s, i);
      if (lane >= i) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31) * hr_n;
    per = (total + gridDim.x - 1) / gridDim.x;
    per = per < W ? W : per;
    u0 = blockIdx.x * per;
    u1 = u0 + per < total ? u0 + per : total;
    const uint32_t past = __ballot_sync(0xffffffffu, s * hr_n > u0);
    b = past ? __ffs(past) - 1 : 0;
    before = __shfl_sync(0xffffffffu, s - n, b);
  } else {
    // chunks of W * 32 lengths: once for the total, once to find the piece's start
    for (int pass = 0; pass < 2; ++pass) {
      long long sum = 0;
      for (int base = 0; base < a.B; base += W * 32) {
        const int i = base + threadIdx.x;
        const int n = i < a.B ? seq_of(a, i, blockIdx.x == 0 && pass == 0).n : 0;
        long long s = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, s, k);
          if (lane >= k) s += o;
        }
        if (lane == 31) s_scan[w] = s;
        __syncthreads();
        long long mine = sum;
        for (int k = 0; k < W; ++k) {
          if (k < w) mine += s_scan[k];
          sum += s_scan[k];
        }
        if (pass == 1) {
          const long long end = mine + s, start = end - n;
          if (n > 0 && start * hr_n <= u0 && u0 < end * hr_n) {
            s_scan[W] = i;
            s_scan[W + 1] = start;
          }
        }
        __syncthreads();
        if (pass == 1 && sum * hr_n > u0) break;
      }
      if (pass == 0) {
        total = sum * hr_n;
        per = (total + gridDim.x - 1) / gridDim.x;
        per = per < W ? W : per;
        u0 = blockIdx.x * per;
        u1 = u0 + per < total ? u0 + per : total;
        if (u0 >= total) break;
      } else {
        b = static_cast<int>(s_scan[W]);
        before = s_scan[W + 1];
      }
    }
  }
  // sequences with nothing to see: zeros, lse -inf
  for (int e = blockIdx.x; e < a.B; e += gridDim.x) {
    if (seq_of(a, e, false).n > 0) continue;
    const int bytes = a.n_q_heads * a.c.head_dim * (kF32 ? 4 : 2);
    char* o = static_cast<char*>(a.out) + static_cast<size_t>(e) * a.out_stride * (kF32 ? 4 : 2);
    for (int i = threadIdx.x * 16; i < bytes; i += W * 32 * 16)
      *reinterpret_cast<uint4*>(o + i) = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr)
      for (int i = threadIdx.x; i < a.n_q_heads; i += W * 32)
        a.lse[static_cast<size_t>(e) * a.n_q_heads + i] = -INFINITY;
  }
  if (u0 >= total) return;

  const int D = a.c.head_dim;
  const uint32_t ring = smem_u32(smem) + w * (C::kRing * C::kSlot);
  float* s_m = reinterpret_cast<float*>(smem + C::kMain);  // [W][8 NT] maxima, then sums
  float* s_l = s_m + W * 8 * NT;
  const float sl = a.scale * 1.4426950408889634f;
  const int tiles_per_page = a.c.page_size / kTile;
  // bytes of a page, of a head in it and of a tile (all below 2^31)
  const uint32_t head_bytes = a.c.page_size * a.c.row_bytes;
  const uint32_t page_bytes = head_bytes * a.c.n_heads, tile_bytes = kTile * a.c.row_bytes;
  const uint32_t head_scales = a.c.page_size * C::kScaleRow;
  const uint32_t page_scales = head_scales * a.c.n_heads;
  // this lane's places in a tile: where its copies go, where its reads start
  constexpr int kPieces = C::kRow / 16;
  const uint32_t put_k = piece<FMT, C::kRow, true>(lane / kPieces, lane % kPieces);
  const uint32_t put_v = piece<FMT, C::kRow, false>(lane / kPieces, lane % kPieces);
  const uint32_t get_k =
      FMT == DT_BF16    ? piece<FMT, C::kRow, true>(g, t)
      : FMT == DT_F32   ? piece<FMT, C::kRow, true>(g, t * 2)
      : FMT == DT_MXFP8 ? piece<FMT, C::kRow, true>(g, t >> 1) + (t & 1) * 8
                        : piece<FMT, C::kRow, true>(g, 0) + t * 4;
  const uint32_t get_v =
      FMT == DT_BF16    ? piece<FMT, C::kRow, false>(2 * t, g)
      : FMT == DT_F32   ? piece<FMT, C::kRow, false>(2 * t, g * 2)
      : FMT == DT_MXFP8 ? piece<FMT, C::kRow, false>(2 * t, g >> 1) + (g & 1) * 8
                        : piece<FMT, C::kRow, false>(2 * t, g >> 2) + (g & 3) * 4;
  // MX: of two rows' scale words, the bytes of this lane's blocks 2v + g/4
  const uint32_t pick = (g >> 2) * 0x1111u + 0x6420u;
  uint32_t live[2];  // the scale bytes of the head's blocks
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = D / kMxBlock - 4 * i;
    live[i] = n >= 4 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
  }

  Seq sq = seq_of(a, b, false);
  long long into = u0 - before * hr_n;
  int hr = static_cast<int>(into / sq.n), t0 = static_cast<int>(into - static_cast<long long>(hr) * sq.n);
  long long u = u0;
  bool first_seg = true;
  while (u < u1) {
    const int t1 = sq.n - t0 < u1 - u ? sq.n : t0 + static_cast<int>(u1 - u);
    const int h = hr / p.blocks, row0 = (hr - h * p.blocks) * 8 * NT;

    // ---- the queries: lane 4g + t holds elements 32j + 8t .. + 7 of head g --------------
    uint4 q[NT][kJ];
    float qf[kF32 ? NT : 1][kF32 ? kJ : 1][8];
    float xs[NT][2];  // scale of the scores of this lane's columns (heads 2t, 2t + 1)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      const size_t at = static_cast<size_t>(b) * a.q_stride +
                        static_cast<size_t>(h * p.group + r) * D;
      xs[nt][0] = xs[nt][1] = sl;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int d = j * 32 + t * 8;
        const bool in = r < p.group && d < D;
        if constexpr (kF32) {
          const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + d);
          const float4 lo = in ? __ldg(src) : make_float4(0, 0, 0, 0);
          const float4 hi = in ? __ldg(src + 1) : make_float4(0, 0, 0, 0);
          qf[nt][j][0] = lo.x, qf[nt][j][1] = lo.y, qf[nt][j][2] = lo.z, qf[nt][j][3] = lo.w;
          qf[nt][j][4] = hi.x, qf[nt][j][5] = hi.y, qf[nt][j][6] = hi.z, qf[nt][j][7] = hi.w;
        } else {
          q[nt][j] = in ? ldg_keep(static_cast<const __nv_bfloat16*>(a.q) + at + d)
                        : make_uint4(0, 0, 0, 0);
        }
      }
      if constexpr (kMx) {
        // fp16 queries: the head's largest element is brought to [2^14, 2^15),
        // an exact power of two that goes into the scores' scale
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = word_of(q[nt][j], i);
            top = max(top, max((v << 16) & 0x7fff0000u, v & 0x7fff0000u));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = static_cast<int>(top >> 23) - 127;
        e = e < -112 ? -112 : e;
        const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const uint4 v = q[nt][j];
          q[nt][j] = make_uint4(pack_f16x2(bf16_lo(v.x) * up, bf16_hi(v.x) * up),
                                pack_f16x2(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                                pack_f16x2(bf16_lo(v.z) * up, bf16_hi(v.z) * up),
                                pack_f16x2(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
        }
        const float down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
        xs[nt][0] = sl * __shfl_sync(0xffffffffu, down, 8 * t);
        xs[nt][1] = sl * __shfl_sync(0xffffffffu, down, 8 * t + 4);
      }
    }

    float acc[DP / 16][NT][4], m[NT][2], l[NT][2];
    // MX: acc holds O^T / 2^(ref - 127) of the lane's value block 2v + g/4; bias
    // is 0x1000 - ref in both halves. Blocks past the head read scale 0 = ref.
    int ref[kMx ? kV : 1];
    uint32_t bias[kMx ? kV : 1], mine[kMx ? kV : 1], hot = 0;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][nt][c] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -FLT_MAX, l[nt][0] = l[nt][1] = 0.f;
    if constexpr (kMx) {
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const bool in = (v * 2 + (g >> 2)) * kMxBlock < D;
        ref[v] = in ? -1000 : 0;
        bias[v] = (0x1000 - ref[v]) * 0x10001;
        mine[v] = in ? 0x00ff00ffu : 0u;
      }
    }

    // ---- this warp's tiles ---------------------------------------------------------------
    const int n_it = (t1 - t0 - w + W - 1) / W;  // <= 0: none
    const int start = a.window > 0 && sq.len > a.window ? sq.len - a.window : 0;
    int page_of = 0, off_of = 0;  // lane i: page, and tile in it, of the warp's tile batch + i
    int batch = -32;
    auto pages = [&](int it) {  // loads the pages of tiles it .. it + 31
      batch = it;
      const int k = it + lane;
      page_of = -1;
      if (k < n_it) {
        const int tile = sq.first + t0 + w + k * W, pi = tile / tiles_per_page;
        off_of = tile - pi * tiles_per_page;
        page_of = __ldg(a.block_table + static_cast<size_t>(b) * a.max_pages + pi);
        if (page_of < 0 || page_of >= a.c.n_pages) {
          latch_error(a.status, kErrDevice);
          page_of = -1;
        }
      }
    };
    uint32_t fill = ring;  // slot the next copy goes to
    auto next = [&](uint32_t s) {
      s += C::kSlot;
      return s == ring + C::kRing * C::kSlot ? ring : s;
    };
    // the tile being fetched: offsets of its keys (and values) and scales, rows in sight
    uint64_t lead = 0, lead_sc = 0;
    int lead_r0 = 0, lead_r1 = 0;
    uint32_t hidden = 0;  // bit it % 32: tile `it` lies in a page that is left out
    auto issue_k = [&](int it) {
      __syncwarp();
      if (it < n_it) {
        if (it >= batch + 32) pages(it);
        const int page = __shfl_sync(0xffffffffu, page_of, it - batch);
        const uint32_t off = __shfl_sync(0xffffffffu, off_of, it - batch);
        const uint32_t pg = page < 0 ? 0 : page;
        lead = static_cast<uint64_t>(pg) * page_bytes + (h * head_bytes + off * tile_bytes + lane * 16);
        const int key = (sq.first + t0 + w + it * W) * kTile;
        lead_r0 = start - key;
        lead_r1 = page < 0 ? 0 : sq.len - key;
        hidden = (hidden & ~(1u << (it & 31))) | (page < 0 ? 1u : 0u) << (it & 31);
        copy_tile<C, FMT, true>(fill, put_k, a.c.k + lead, a.c.row_bytes, lead_r0, lead_r1, lane);
        if constexpr (kMx) {
          lead_sc = static_cast<uint64_t>(pg) * page_scales +
                    (h * head_scales + off * (kTile * C::kScaleRow));
          copy_scales<C>(fill, a.c.k_scale + lead_sc, lead_r0, lead_r1, lane);
        }
      }
      cp_async_commit();
      fill = next(fill);
    };
    auto issue_v = [&](int it) {
      __syncwarp();
      if (it < n_it) {
        copy_tile<C, FMT, false>(fill, put_v, a.c.v + lead, a.c.row_bytes, lead_r0, lead_r1, lane);
        if constexpr (kMx)
          copy_scales<C>(fill, a.c.v_scale + lead_sc, lead_r0, lead_r1, lane);
      }
      cp_async_commit();
      fill = next(fill);
    };
    // Scores of 32 elements in three tf32 products (hi hi + hi lo + lo hi). An
    // infinity times a part that is 0 would be NaN: `careful` leaves such
    // operands out of the cross products.
    auto score_f32 = [&](float(&d)[NT][4], uint32_t at0, int j, bool careful) {
      if constexpr (kF32) {
        float ka[8], kb[8];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t at = further(at0 + get_k, j * 128 + hf * 16);
          const uint4 va = lds128(at), vb = lds128(at + 8 * C::kRow);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ka[hf * 4 + i] = __uint_as_float(word_of(va, i));
            kb[hf * 4 + i] = __uint_as_float(word_of(vb, i));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float hi[4], lo[4];
          split_tf32(ka[2 * i], &hi[0], &lo[0]);
          split_tf32(kb[2 * i], &hi[1], &lo[1]);
          split_tf32(ka[2 * i + 1], &hi[2], &lo[2]);
          split_tf32(kb[2 * i + 1], &hi[3], &lo[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float qh[2], ql[2];
            split_tf32(qf[nt][j][2 * i], &qh[0], &ql[0]);
            split_tf32(qf[nt][j][2 * i + 1], &qh[1], &ql[1]);
            mma_tf32_1688(d[nt], hi, qh);
            if (careful) {
#pragma unroll
              for (int k = 0; k < 4; ++k) hi[k] = fabsf(hi[k]) == INFINITY ? 0.f : hi[k];
#pragma unroll
              for (int k = 0; k < 2; ++k) qh[k] = fabsf(qh[k]) == INFINITY ? 0.f : qh[k];
            }
            mma_tf32_1688(d[nt], lo, qh);
            mma_tf32_1688(d[nt], hi, ql);
          }
        }
      }
    };
    constexpr int kLead = (C::kRing - 1) / 2;
#pragma unroll
    for (int i = 0; i < kLead; ++i) {
      issue_k(i);
      issue_v(i);
    }
    uint32_t slot = ring;
    for (int it = 0; it < n_it; ++it) {
      // ---- scores ----------------------------------------------------------------------
      issue_k(it + kLead);
      cp_async_wait<C::kRing - 1>();
      __syncwarp();
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
      float f0[kMx ? kJ : 1], f1[kMx ? kJ : 1];  // the blocks' scales of keys g and g + 8
      if constexpr (kMx) {
        const uint32_t at = slot + kTile * C::kRow + g * C::kScaleRow;
        uint32_t sc0[2], sc1[2];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < C::kScaleRow / 4; ++i) {
          // bytes past the head's blocks may hold anything: 1
          sc0[i] = (lds32(at + 4 * i) & live[i]) | (0x7f7f7f7fu & ~live[i]);
          sc1[i] = (lds32(at + 8 * C::kScaleRow + 4 * i) & live[i]) | (0x7f7f7f7fu & ~live[i]);
          odd = odd || odd_scales(sc0[i]) || odd_scales(sc1[i]);
        }
        if (!__any_sync(0xffffffffu, odd)) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            constexpr uint32_t kExp = 0x7f800000u;
            const int up = 23 - 8 * (j % 4);
            f0[j] = __uint_as_float((up > 0 ? sc0[j / 4] << (up & 31) : sc0[j / 4] >> 1) & kExp);
            f1[j] = __uint_as_float((up > 0 ? sc1[j / 4] << (up & 31) : sc1[j / 4] >> 1) & kExp);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            f0[j] = e8m0_f32((sc0[j / 4] >> (8 * (j % 4))) & 255u);
            f1[j] = e8m0_f32((sc1[j / 4] >> (8 * (j % 4))) & 255u);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        if constexpr (FMT == DT_BF16) {
          const uint32_t at = further(slot + get_k, j * 64);
          const uint4 ka = lds128(at), kb = lds128(at + 8 * C::kRow);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(x[nt], ka.x, kb.x, ka.y, kb.y, q[nt][j].x, q[nt][j].y);
            mma_bf16_16816(x[nt], ka.z, kb.z, ka.w, kb.w, q[nt][j].z, q[nt][j].w);
          }
        } else if (kMx && j * 32 < D) {
          uint32_t ka[4], kb[4];
          if constexpr (FMT == DT_MXFP8) {
            const uint32_t at = further(slot + get_k, j * 32);
            const uint2 va = lds64(at), vb = lds64(at + 8 * C::kRow);
            e4m3x8_f16(va.x, va.y, ka);
            e4m3x8_f16(vb.x, vb.y, kb);
          } else {
            const uint32_t at = further(slot + get_k, j * 16);
            e2m1x8_f16(lds32(at), ka);
            e2m1x8_f16(lds32(at + 8 * C::kRow), kb);
          }
          // the block's scale goes on its partial score: codes are exact in fp16
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16_16816(d, ka[0], kb[0], ka[1], kb[1], q[nt][j].x, q[nt][j].y);
            mma_f16_16816(d, ka[2], kb[2], ka[3], kb[3], q[nt][j].z, q[nt][j].w);
            x[nt][0] = fmaf(d[0], f0[j], x[nt][0]);
            x[nt][1] = fmaf(d[1], f0[j], x[nt][1]);
            x[nt][2] = fmaf(d[2], f1[j], x[nt][2]);
            x[nt][3] = fmaf(d[3], f1[j], x[nt][3]);
          }
        }
      }
      if constexpr (kF32) {
#pragma unroll 1
        for (int careful = 0; careful < 2; ++careful) {
          bool nan = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
          for (int j = 0; j < kJ; ++j) score_f32(x, slot, j, careful != 0);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) nan |= x[nt][c] != x[nt][c];
          if (!__any_sync(0xffffffffu, nan)) break;
        }
      }
      const int tile_key = (sq.first + t0 + w + it * W) * kTile;
      // rows in sight of this tile
      const int r0 = start - tile_key, r1 = hidden >> (it & 31) & 1u ? 0 : sq.len - tile_key;
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[nt][c] *= xs[nt][c & 1];
      if (r0 > 0 || r1 < kTile) {
        const bool in0 = g >= r0 && g < r1, in1 = g + 8 >= r0 && g + 8 < r1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (!in0) x[nt][0] = x[nt][1] = -INFINITY;
          if (!in1) x[nt][2] = x[nt][3] = -INFINITY;
        }
      }
      // ---- weights ---------------------------------------------------------------------
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) up |= fmaxf(x[nt][c], x[nt][c + 2]) > m[nt][c] + kSlack;
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(x[nt][c], x[nt][c + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(top, m[nt][c]);
            const float f = ex2(m[nt][c] - top);
            m[nt][c] = top;
            l[nt][c] *= f;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) acc[i][nt][c] *= f, acc[i][nt][c + 2] *= f;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[nt][c] = ex2(x[nt][c] - (m[nt][c & 1] - kLift));
          l[nt][c & 1] += x[nt][c];
        }
      slot = next(slot);

      // ---- values ------------------------------------------------------------------------
      // the weights as the other product's operand: keys 2t, 2t + 1 (and + 8) of head g
      uint32_t pb[NT][2], pl[NT][2];
      float pf[kF32 ? NT : 1][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (FMT == DT_BF16) {
          // bf16 weights and, beside them, what the rounding left: 16 bits together
          const uint32_t h0 = pack_bf16x2(x[nt][0], x[nt][1]);
          const uint32_t h1 = pack_bf16x2(x[nt][2], x[nt][3]);
          pb[nt][0] = transpose8(h0);
          pb[nt][1] = transpose8(h1);
          pl[nt][0] = transpose8(pack_bf16x2(x[nt][0] - bf16_lo(h0), x[nt][1] - bf16_hi(h0)));
          pl[nt][1] = transpose8(pack_bf16x2(x[nt][2] - bf16_lo(h1), x[nt][3] - bf16_hi(h1)));
        } else if constexpr (kF32) {
          const int src = 8 * t + (g >> 1);  // lane of key 2t, head g
#pragma unroll
          for (int k = 0; k < 4; ++k) {      // keys 2t, 2t + 1, 2t + 8, 2t + 9
            const float e0 = __shfl_sync(0xffffffffu, x[nt][(k >> 1) * 2], src + (k & 1) * 4);
            const float e1 = __shfl_sync(0xffffffffu, x[nt][(k >> 1) * 2 + 1], src + (k & 1) * 4);
            pf[nt][k] = g & 1 ? e1 : e0;
          }
        }
      }
      issue_v(it + kLead);
      cp_async_wait<C::kRing - 1>();
      __syncwarp();
      if constexpr (FMT == DT_BF16) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
          const uint32_t at = slot + get_v;
          const uint4 r_0 = lds128(further(at, v * 128));
          const uint4 r_1 = lds128(further(at, v * 128 + C::kRow));
          const uint4 r_2 = lds128(further(at, v * 128 + C::kRow * 8));
          const uint4 r_3 = lds128(further(at, v * 128 + C::kRow * 9));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w0 = word_of(r_0, i), w1 = word_of(r_1, i), w2 = word_of(r_2, i),
                           w3 = word_of(r_3, i);
            const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
            const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16_16816(acc[v * 4 + i][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
              mma_bf16_16816(acc[v * 4 + i][nt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
            }
          }
        }
      } else if constexpr (kF32) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint4 r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              r[k] = lds128(further(slot + get_v, v * 256 + hf * 16 +
                                                      ((k & 1) + (k >> 1) * 8) * C::kRow));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int s = 0; s < 2; ++s) {  // keys 2t, 2t + 1; then 2t + 8, 2t + 9
                float hi[4], lo[4];
                split_tf32(__uint_as_float(word_of(r[2 * s], 2 * i)), &hi[0], &lo[0]);
                split_tf32(__uint_as_float(word_of(r[2 * s], 2 * i + 1)), &hi[1], &lo[1]);
                split_tf32(__uint_as_float(word_of(r[2 * s + 1], 2 * i)), &hi[2], &lo[2]);
                split_tf32(__uint_as_float(word_of(r[2 * s + 1], 2 * i + 1)), &hi[3], &lo[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float ph[2], plo[2];
                  split_tf32(pf[nt][2 * s], &ph[0], &plo[0]);
                  split_tf32(pf[nt][2 * s + 1], &ph[1], &plo[1]);
                  float(&d)[4] = acc[v * 4 + hf * 2 + i][nt];
                  mma_tf32_1688(d, lo, ph);
                  mma_tf32_1688(d, hi, plo);
                  mma_tf32_1688(d, hi, ph);
                }
              }
            }
          }
        }
      } else {
        // Value codes are exact in fp16, and so is a code times 2^(s - ref) for
        // scales s in [ref - 14, ref + 7]: ref follows the largest scale of the
        // lane's block (the four lanes of a g share it). sd holds s - ref + 0x1000
        // for the keys of a pair in its halves. A tile with a scale out of that
        // range, a NaN one or a weight too small for fp16 takes the careful way.
        uint32_t sd[kV][2];
        uint32_t bad = 0;
        const bool part = r0 > 0 || r1 < kTile;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t at = slot + kTile * C::kRow + (2 * t + 8 * k) * C::kScaleRow;
#pragma unroll
          for (int i = 0; i < C::kScaleRow / 4; ++i) {
            uint32_t w0, w1;
            if constexpr (C::kScaleRow == 4) {
              const uint2 v = lds64(at);
              w0 = v.x, w1 = v.y;
            } else {
              w0 = lds32(at + 4 * i), w1 = lds32(at + 8 + 4 * i);
            }
            const uint32_t by = __byte_perm(w0, w1, pick);
            sd[2 * i][k] = (by & mine[2 * i]) + bias[2 * i];
            if constexpr (kV > 1) sd[2 * i + 1][k] = (by >> 8 & mine[2 * i + 1]) + bias[2 * i + 1];
          }
          if (part) {  // rows out of sight hold zeros, whatever their scale
            const int row = 2 * t + 8 * k;
            const uint32_t lo = row < r0 || row >= r1 ? 0xffffu : 0u;
            const uint32_t hi = row + 1 < r0 || row + 1 >= r1 ? 0xffff0000u : 0u;
#pragma unroll
            for (int v = 0; v < kV; ++v)
              sd[v][k] = (sd[v][k] & ~(lo | hi)) | (0x10001000u & (lo | hi));
          }
#pragma unroll
          for (int v = 0; v < kV; ++v) bad |= (sd[v][k] - 0x0ff20ff2u) | (0x10071007u - sd[v][k]);
        }
        bad = (bad & 0x80008000u) | hot;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)  // 0 < weight < 2^-16
            bad |= __float_as_uint(x[nt][c]) - 1u < 0x377fffffu ? 1u : 0u;
        bool wide = false;
        float fw[kV][4];  // the careful way's factors
        if (__any_sync(0xffffffffu, bad != 0)) {
          int s[kV][4];
          hot = 0;
#pragma unroll
          for (int v = 0; v < kV; ++v) {
            int top = -1000;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              s[v][k] = static_cast<int>(sd[v][k >> 1] >> (16 * (k & 1)) & 0xffffu) - 0x1000 + ref[v];
              if (s[v][k] != 255) top = max(top, s[v][k]);
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > ref[v] + 7) {
              const float f = ex2(static_cast<float>(ref[v] - top));
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 4; ++c) acc[v * 4 + i][nt][c] *= f;
              ref[v] = top;
              bias[v] = (0x1000 - top) * 0x10001;
            }
            if (ref[v] > 247) hot = 1;  // a NaN scale would pass for 2^128
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = 2 * t + (k & 1) + (k >> 1) * 8;
              if (row < r0 || row >= r1) s[v][k] = ref[v];
              const int e = s[v][k] - ref[v];
              wide |= e < -14 || e > 7 || s[v][k] == 255;
              fw[v][k] = s[v][k] == 255 ? __uint_as_float(0x7fc00000u)
                                        : __uint_as_float(static_cast<uint32_t>(e < -127 ? 0 : e + 127) << 23);
            }
            sd[v][0] = (s[v][0] - ref[v] + 0x1000) | (s[v][1] - ref[v] + 0x1000) << 16;
            sd[v][1] = (s[v][2] - ref[v] + 0x1000) | (s[v][3] - ref[v] + 0x1000) << 16;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) wide |= __float_as_uint(x[nt][c]) - 1u < 0x377fffffu;
          wide = __any_sync(0xffffffffu, wide);
        }
        if (!wide) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            pb[nt][0] = transpose8(pack_f16x2(x[nt][0], x[nt][1]));
            pb[nt][1] = transpose8(pack_f16x2(x[nt][2], x[nt][3]));
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            pb[nt][0] = transpose8(pack_bf16x2(x[nt][0], x[nt][1]));
            pb[nt][1] = transpose8(pack_bf16x2(x[nt][2], x[nt][3]));
          }
        }
#pragma unroll
        for (int v = 0; v < kV; ++v) {
          uint32_t op[2][8];  // [keys 2t, 2t + 1 or + 8][element]: the two keys' codes in fp16
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t off = v * (C::kBits * 8) + k * 8 * C::kRow;
            uint32_t h4[4];
            if constexpr (FMT == DT_MXFP8) {
              const uint2 e0 = lds64(further(slot + get_v, off));
              const uint2 e1 = lds64(further(slot + get_v, off + C::kRow));
              e4m3x8_f16(__byte_perm(e0.x, e1.x, 0x5140), __byte_perm(e0.x, e1.x, 0x7362), h4);
#pragma unroll
              for (int i = 0; i < 4; ++i) op[k][i] = h4[i];
              e4m3x8_f16(__byte_perm(e0.y, e1.y, 0x5140), __byte_perm(e0.y, e1.y, 0x7362), h4);
#pragma unroll
              for (int i = 0; i < 4; ++i) op[k][4 + i] = h4[i];
            } else {
              const uint32_t e0 = lds32(further(slot + get_v, off));
              const uint32_t e1 = lds32(further(slot + get_v, off + C::kRow));
              e2m1x8_f16((e0 & 0x0f0f0f0fu) | ((e1 & 0x0f0f0f0fu) << 4), h4);
#pragma unroll
              for (int i = 0; i < 4; ++i) op[k][2 * i] = h4[i];
              e2m1x8_f16(((e0 >> 4) & 0x0f0f0f0fu) | (e1 & 0xf0f0f0f0u), h4);
#pragma unroll
              for (int i = 0; i < 4; ++i) op[k][2 * i + 1] = h4[i];
            }
          }
          if (!wide) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t f = (sd[v][k] - 0x0ff10ff1u) << 10;  // 2^(s - ref), both keys
#pragma unroll
              for (int i = 0; i < 8; ++i) op[k][i] = mul_f16x2(op[k][i], f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(acc[v * 4 + i][nt], op[0][2 * i], op[0][2 * i + 1], op[1][2 * i],
                              op[1][2 * i + 1], pb[nt][0], pb[nt][1]);
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float lo, hi;
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                    "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                    : "=f"(lo), "=f"(hi)
                    : "r"(op[k][i]));
                op[k][i] = pack_bf16x2(lo * fw[v][2 * k], hi * fw[v][2 * k + 1]);
              }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_bf16_16816(acc[v * 4 + i][nt], op[0][2 * i], op[0][2 * i + 1], op[1][2 * i],
                               op[1][2 * i + 1], pb[nt][0], pb[nt][1]);
          }
        }
      }
      slot = next(slot);
    }
    cp_async_wait<0>();

    // ---- join the warps ------------------------------------------------------------------
    if constexpr (kMx) {
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const float f = ref[v] == -1000 ? 0.f : e8m0_f32(ref[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[v * 4 + i][nt][c] *= f;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], i);
        m[nt][c] = m[nt][c] == -FLT_MAX ? m[nt][c] : m[nt][c] - kLift;
      }
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) s_m[w * 8 * NT + nt * 8 + 2 * t + c] = m[nt][c];
    }
    __syncthreads();  // maxima in place, every ring drained
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[nt][c] = -FLT_MAX;
#pragma unroll
        for (int k = 0; k < W; ++k)
          top[nt][c] = fmaxf(top[nt][c], s_m[k * 8 * NT + nt * 8 + 2 * t + c]);
        const float f = ex2(m[nt][c] - top[nt][c]);
        l[nt][c] *= f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) acc[i][nt][c] *= f, acc[i][nt][c + 2] *= f;
        if (g == 0) s_l[w * 8 * NT + nt * 8 + 2 * t + c] = l[nt][c];
      }
    float* buf = reinterpret_cast<float*>(smem) + w * C::kRegs * 32 + lane;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) buf[((i * NT + nt) * 4 + c) * 32] = acc[i][nt][c];
    __syncthreads();
    const bool whole = t0 == 0 && t1 == sq.n;
    float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (first_seg ? 0 : 1)) * C::kPart;
    // warp w adds the register groups w, w + W, ... (one MMA tile of 16 x 8) of all warps
    for (int gr = w; gr < DP / 16 * NT; gr += W) {
      const int i = gr / NT, nt = gr - i * NT;
      float o[4] = {0.f, 0.f, 0.f, 0.f}, sum[2] = {0.f, 0.f}, mx[2] = {-FLT_MAX, -FLT_MAX};
      for (int k = 0; k < W; ++k) {
        const float* src = reinterpret_cast<const float*>(smem) + k * C::kRegs * 32 + gr * 128 + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] += src[c * 32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sum[c] += s_l[k * 8 * NT + nt * 8 + 2 * t + c];
          mx[c] = fmaxf(mx[c], s_m[k * 8 * NT + nt * 8 + 2 * t + c]);
        }
      }
      if (!whole) {
#pragma unroll
        for (int c = 0; c < 4; ++c) part[gr * 128 + c * 32 + lane] = o[c];
        if (i == 0 && g == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            part[C::kRegs * 32 + nt * 8 + 2 * t + c] = mx[c];
            part[C::kRegs * 32 + 8 * NT + nt * 8 + 2 * t + c] = sum[c];
          }
        }
      } else {
        const int d = (i / 4) * 64 + g * 8 + (i % 4) * 2;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = row0 + nt * 8 + 2 * t + c;
          if (r >= p.group) continue;
          const int hq = h * p.group + r;
          const float inv = sum[c] == 0.f ? 0.f : 1.f / sum[c];
          if (d < D) {
            const size_t at = static_cast<size_t>(b) * a.out_stride + static_cast<size_t>(hq) * D + d;
            const float y0 = sum[c] == 0.f ? 0.f : o[c] * inv;
            const float y1 = sum[c] == 0.f ? 0.f : o[c + 2] * inv;
            if constexpr (kF32)
              *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(y0, y1);
            else
              *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at) =
                  pack_bf16x2(y0, y1);
          }
          if (a.lse != nullptr && i == 0 && g == 0)
            a.lse[static_cast<size_t>(b) * a.n_q_heads + hq] =
                sum[c] == 0.f ? -INFINITY : (mx[c] + log2f(sum[c])) * 0.6931471805599453f;
        }
      }
    }
    if (t0 == 0 && !whole && threadIdx.x == 0) {
      // the segment starts here and ends in a later block
      const long long end = u + sq.n;
      p.span[blockIdx.x] = make_int4(b, hr, first_seg ? 0 : 1,
                                     static_cast<int>((end - 1) / per) - blockIdx.x + 1);
    }
    __syncthreads();  // the buffers become rings again

    // ---- the next segment -----------------------------------------------------------------
    u += t1 - t0;
    first_seg = false;
    t0 = 0;
    if (u < u1 && ++hr == hr_n) {
      hr = 0;
      do {
        sq = seq_of(a, ++b, false);
      } while (sq.n == 0);
    }
  }
}

}  // namespace paged
}  // namespace coli
