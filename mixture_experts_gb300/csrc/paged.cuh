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
// so a group of up to 8 heads fills its tile, the 16-row operands come out of
// shared memory in the MMA's own order (ldmatrix, transposed for bf16 values),
// and the tile of S^T becomes the other product's operand by two 8x8 register
// transposes. m is only raised when a score passes it by kSlack: one vote a step
// instead of a reduction.
//
// Work split. The tiles of 16 keys of every (sequence, key head, block of
// heads) lie on one line, each such segment behind kOpen empty places for what
// its start and join cost, and the line is cut into equal pieces, one per block,
// so ragged lengths load every SM alike and tiny segments do not queue up. A
// block that covers a whole segment writes its output; a segment cut by block
// borders leaves partial means and weights that k_join joins in the order of the blocks (no
// atomics: the same bits every time). Within a block warp w takes steps w, w + W,
// ... with its own ring of shared-memory slots filled by cp.async (rows past the
// context zero-filled), so no warp waits for another before the segment's end,
// and the next segment's first copies fly while the warps' sums are joined.
//
// Precision. Scores, softmax statistics and sums are fp32; the products' operands are not:
//   scores  bf16 as it is; fp32 in two tf32 parts, low x low left out (21 bits); MX codes
//           and queries as they are, in as many parts as that takes;
//   values  weights in two tf32 parts (fp32, so are the values), in a bf16 number and one
//           for its rounding (16 bits), in fp16 (MX: 11 bits, 9 at 2^-30 of the largest;
//           bf16 in two parts below); the normaliser adds the unrounded ones. 11 bits lie
//           below what the bf16 output rounds away (8), and fp16 takes half the products.
// MX numbers further apart than these operands hold (scales, queries) take plain_tiles.
//
// What bounds it (GB300, 32 query and 8 key heads of 128 unless said, against the
// 6.8 TB/s of a copy): bf16 HBM: 6.9 TB/s on one context of 500009 tokens, 6.1 TB/s
// on 32 ragged ones (586 MB, 96 us). fp32 HBM (6.6 TB/s, 8 heads, 7 x 26157 tokens).
// MXFP8 5.5 TB/s on 64 contexts (1168 MB, 212 us): 480 instructions a tile, issue 56%
// and the ALU pipe 50% busy (widening value codes to fp16, their scales), with three
// warps a scheduler to cover the steps' own latency. MXFP4, 64 query heads on 4:
// 2.0 TB/s (282 MB, 140 us): 636 instructions a tile, the same work at half the bytes
// and twice the heads. A group of more than 16 query heads (fp32: 8) is cut in segments
// that read the keys and values once each: 640000 keys, 16 / 32 / 64 heads on one key
// head, bf16 67 / 113 / 186 us, MXFP8 66 / 115 / 197; fp32, 8 / 16 / 32: 108 / 197 / 375.

#pragma once

#include <float.h>

#include <type_traits>

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
  float* part;     // partial means with their weights, two slots a block
  int4* span;      // per block: the cut segment that starts in it
  int direct;      // one block a segment: nothing is cut, nothing joined
};

template <int FMT, int DP, int NT>
struct Cfg {
  static constexpr bool kMx = FMT == DT_MXFP8 || FMT == DT_MXFP4;
  static constexpr int kBits = FMT == DT_F32 ? 32 : FMT == DT_BF16 ? 16 : FMT == DT_MXFP8 ? 8 : 4;
  static constexpr int kRow = DP * kBits / 8;          // bytes of a row in shared memory
  static constexpr int kScaleRow = kMx ? (DP > 128 ? 8 : 4) : 0;
  // Tiles a warp takes in one step: two of an MX cache, whose small tiles leave
  // the step's fixed work (pages, waits, votes) as long as the tile's own (64 MXFP8
  // contexts: two 212 us, one 225 us; groups of 16 heads: two spill, 148 against 140 us).
  static constexpr int kStep = kMx && DP <= 128 && DP * NT <= 128 ? 2 : 1;
  static constexpr int kTileBytes = kTile * kRow, kTileScales = kTile * kScaleRow;
  // whole 128-byte lines: addresses within a line are XORed
  static constexpr int kSlot = (kStep * (kTileBytes + 2 * kTileScales) + 127) / 128 * 128;
  static constexpr int kRegs = DP / 16 * 4 * NT;       // O^T registers of a lane
  static constexpr int kOpen = 8;  // a segment's fixed cost, in tiles (3 us at 2.7 tiles a us)
  // Warps of a block and blocks of an SM: what the registers of the widest step allow
  // without many spills. MXFP8 heads of 128, 64 contexts: 12 warps of 168 registers
  // 212 us, 8 of 255 240 us (16 warps: no room for their rings); MXFP4 groups of 16
  // heads, 160 windowed contexts: 12 warps 140 us, 8 warps 148 us, 16 warps 203 us.
  static constexpr int kAcc = DP * NT;
  static constexpr int kWarps = kAcc == 512 ? (kMx ? 8 : 6)
                                : kSlot > 8448 || (kMx && kAcc >= 128 && DP <= 128) ||
                                          (NT == 2 && kAcc == 256)
                                    ? 4
                                    : 8;
  static constexpr int kPerSm = kMx && DP <= 128 ? (kAcc >= 128 ? 3 : 2)
                                : kAcc <= 128 && kSlot <= 4096 ? 2
                                : NT == 2 && kAcc == 256       ? 3
                                                               : 1;
  // Queries in shared memory, 16 bytes a lane: fp32 ones in two parts; those of two
  // column tiles of MX heads, whose registers are worth more warps
  static constexpr bool kQShared = FMT == DT_F32 || (NT == 2 && (kMx || DP == 256));
  static constexpr int kQBytes = FMT == DT_F32 ? DP / 8 * 512 : (kQShared ? NT * DP / 32 * 512 : 0);
  // MXFP8: query elements that its two terms do not hold, in fp16
  static constexpr int kFineBytes = FMT == DT_MXFP8 ? NT * DP / 32 * 512 : 0;
  // The warps' sums are joined half the registers at a time, beside the rings: the
  // next segment's copies are in flight meanwhile.
  static constexpr int kMergeBytes = kWarps * kRegs * 64;
  static constexpr int kState = kWarps * 8 * NT * 8;  // maxima and sums
  // shared memory of a block less the system's 1 KB and the static part
  static constexpr int kBudget =
      228 * 1024 / kPerSm - 1280 - kMergeBytes - kQBytes - kFineBytes - kState;
  static constexpr int kFit = kBudget / (kWarps * kSlot);
  // odd, so key and value slots alternate through the ring with one lead
  static constexpr int kRing = kFit >= 7 ? 7 : (kFit >= 5 ? 5 : 3);
  static constexpr int kRingBytes = kRing * kWarps * kSlot;
  static constexpr int kMain = kRingBytes + kMergeBytes;
  static constexpr int kSmem = kMain + kQBytes + kFineBytes + kState;
  static_assert(kRingBytes <= kBudget, "ring does not fit");
  static constexpr int kPart = kRegs * 32 + 16 * NT;   // floats of a partial slot
};

// ---- small pieces --------------------------------------------------------------------
COLI_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Of a sum of weights: 2^-8 or more.
COLI_DEV float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
// Four 8x8 matrices of 16-bit elements (lane l: the row address of row l % 8 of
// matrix l / 8) -> lane 4g + t: row g, elements 2t, 2t + 1 of each; or, transposed,
// elements g of rows 2t, 2t + 1.
COLI_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
COLI_DEV void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
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
// d = A x B (a zero accumulator input).
COLI_DEV void mma_f16_16816_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// e4m3 x e4m3 (or e5m2), 32 indices: twice the f16 form's work an instruction, summed
// as exactly: off by at most 10 x 2^-24 of the largest term (e5m2: 8; f16 and bf16: 7;
// tf32: 8), over 38400 random and one-signed sums a form.
COLI_DEV void mma_e4m3_16832(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
COLI_DEV void mma_e4m3_e5m2_16832_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e5m2.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// Where 16-byte piece c of row r lies in a tile: the piece's place XORed, within
// its 128 bytes, with a number of the row chosen so that the lanes of one
// shared-memory phase meet 8 different pieces. ldmatrix reads one piece of rows
// 0-7 (or 8-15) at once; the other reads take rows g = 0..7 of MXFP4 keys (lane
// 4g + t: 4 bytes) and, of values, rows 2t (8 elements from 8g on of every 64).
template <int FMT, int ROW, bool KEYS>
COLI_DEV constexpr uint32_t row_xor(int r) {
  if (KEYS || FMT == DT_BF16) return ROW >= 128 ? r & 7 : (ROW >= 64 ? (r >> 1) & 3 : (r >> 2) & 1);
  if (FMT == DT_F32) return ((r >> 1) & 1) | (((r >> 2) & 1) << 2);
  return ROW >= 64 ? r & 6 : ((r >> 2) & 1) << 1;
}
// Channel of register c (0-3) of accumulator tile i: bf16 values come transposed
// in order, the others as pairs out of the lane's 8 elements.
template <bool IN_ORDER>
COLI_DEV int channel(int i, int g, int c) {
  return IN_ORDER ? i * 16 + g + (c >> 1) * 8 : (i >> 2) * 64 + g * 8 + (i & 3) * 2 + (c >> 1);
}
// EXT: the forms that other calls than the plain decode attention use (page lists for each key
// head, many sequences' queries as one group, means and (m, l) pairs for a later join, a start
// beside the kernel before). They are instantiations of their own: as branches they cost
// the plain call 1%.
//
// Place of query row r of key head h of sequence b in rows of heads `width` apart, tokens
// `stride` apart: head h group + r of the sequence, or, where a.fold heads of each sequence
// follow each other as one group, head h fold + r % fold of sequence r / fold.
template <bool EXT>
COLI_DEV size_t row_at(const PagedArgs& a, int group, int b, int h, int r, size_t stride,
                       int width) {
  if (EXT && a.fold > 0) {
    const int s = r / a.fold;
    return s * stride + static_cast<size_t>(h * a.fold + r - s * a.fold) * width;
  }
  return b * stride + static_cast<size_t>(h * group + r) * width;
}
// log sum of a row's weights 2^(x - m), or with a.raw the pair (m, sum) for a later join.
template <bool EXT>
COLI_DEV void store_lse(const PagedArgs& a, int group, int b, int h, int r, float m, float sum) {
  const int n = EXT && a.fold > 0 ? a.fold * a.c.n_heads : a.n_q_heads;
  const size_t at = row_at<EXT>(a, group, b, h, r, n, 1);
  if (EXT && a.raw)
    reinterpret_cast<float2*>(a.lse)[at] = make_float2(m, sum);
  else
    a.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}
// Two outputs (channels of c and c + 2) of one head.
template <bool IN_ORDER, bool F32, bool EXT>
COLI_DEV void store_out(const PagedArgs& a, size_t row, int i, int g, float y0, float y1) {
  const int d = channel<IN_ORDER>(i, g, 0), e = channel<IN_ORDER>(i, g, 2), D = a.c.head_dim;
  if (EXT && !F32 && a.raw) {  // fp32 means, for a later join
    float* o = static_cast<float*>(a.out) + row;
    if (d < D) o[d] = y0;
    if (e < D) o[e] = y1;
  } else if constexpr (IN_ORDER) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + row;
    if (d < D) o[d] = __float2bfloat16_rn(y0);
    if (e < D) o[e] = __float2bfloat16_rn(y1);
  } else if (d < D) {
    if constexpr (F32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row + d) = make_float2(y0, y1);
    else
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row + d) =
          pack_bf16x2(y0, y1);
  }
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
// first piece's place, src its address.
template <class C, int FMT, bool KEYS>
COLI_DEV void copy_tile(uint32_t slot, uint32_t place, const char* src) {
  constexpr int kPieces = C::kRow / 16;
#pragma unroll
  for (int i = 0; i < kTile * kPieces / 32; ++i)
    cp_async16_n(((slot + place) ^ (row_xor<FMT, C::kRow, KEYS>(i * 32 / kPieces) * 16)) + i * 512,
                 src + i * 512, 16);
}

// The same for rows of row_bytes < kRow bytes, with zeros after them: src is the
// address of the lane's first piece (of its row, where the piece lies past the row).
template <class C, int FMT, bool KEYS>
COLI_DEV void copy_narrow(uint32_t slot, uint32_t place, const char* src, int row_bytes, int lane) {
  constexpr int kPieces = C::kRow / 16;
#pragma unroll
  for (int i = 0; i < kTile * kPieces / 32; ++i) {
    const bool in = (i * 32 + lane) % kPieces * 16 < row_bytes;
    const int more = kPieces > 32 && in ? i * 32 % kPieces * 16 : 0;
    cp_async16_n(((slot + place) ^ (row_xor<FMT, C::kRow, KEYS>(i * 32 / kPieces) * 16)) + i * 512,
                 src + (i * 32 / kPieces) * row_bytes + more, in ? 16 : 0);
  }
}

// And with zeros for rows outside [r0, r1) too; src as for whole rows.
template <class C, int FMT, bool KEYS>
COLI_DEV void copy_part(uint32_t slot, uint32_t place, const char* src, int row_bytes, int r0,
                        int r1, int lane) {
  constexpr int kPieces = C::kRow / 16;
  const char* tile = src - lane * 16;
#pragma unroll
  for (int i = 0; i < kTile * kPieces / 32; ++i) {
    const int p = i * 32 + lane, r = p / kPieces, c = p % kPieces;
    const bool in = r >= r0 && r < r1 && c * 16 < row_bytes;
    cp_async16_n(((slot + place) ^ (row_xor<FMT, C::kRow, KEYS>(i * 32 / kPieces) * 16)) + i * 512,
                 in ? tile + r * row_bytes + c * 16 : src, in ? 16 : 0);
  }
}

// a / b, both positive; the line is rarely longer than 32 bits.
COLI_DEV long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Where the pages of a sequence's key head are listed: the sequence's row, or its own.
template <bool EXT>
COLI_DEV size_t table_at(const PagedArgs& a, int b, int h) {
  const size_t row = EXT && a.head_tables ? static_cast<size_t>(b) * a.c.n_heads + h : b;
  return row * a.max_pages;
}

// The line of work: tiles of sequence b, in tiles of 16 keys counted from the
// context's start.
struct Seq {
  int len, first, n;  // length, first tile, number of tiles
};
template <bool EXT>
COLI_DEV Seq seq_of(const PagedArgs& a, int b, bool latch) {
  int len = EXT && a.fixed_len > 0 ? a.fixed_len : __ldg(a.seq_lens + b);
  const int most = a.max_pages * a.c.page_size;
  if (len < 0 || len > most) {
    if (latch) latch_error(a.status, kErrDevice);
    len = len < 0 ? 0 : most;
  }
  const int start = a.window > 0 && len > a.window ? len - a.window : 0;
  const int first = start / kTile;
  return {len, first, (len + kTile - 1) / kTile - first};
}

// One warp's tiles of an MX cache once more, in fp32 straight from memory: lane 4g + t takes
// the channels 64 v + 8 g .. + 7 of heads 2t, 2t + 1 (+ 8 nt), one key after the other. For
// numbers further apart than the operands of k_paged hold, which no trained model's are: sums
// and products overflow where plain fp32 ones would. 25 times the steps' time (64 MXFP8
// contexts: 5.3 ms). Called or inlined, the steps themselves take the same (212 us).
template <int DP, int NT>
struct PlainSums {
  float acc[DP / 16][NT][4], m[NT][2], l[NT][2];
};
template <int FMT>
COLI_DEV void decode8(const KvView& c, const char* pool, const uint8_t* scales, size_t row, int ch,
                      float (&x)[8]) {
  uint32_t h4[4];
  if constexpr (FMT == DT_MXFP8) {
    const uint2 u = *reinterpret_cast<const uint2*>(pool + row * c.row_bytes + ch);
    e4m3x8_f16(u.x, u.y, h4);
  } else {
    e2m1x8_f16(*reinterpret_cast<const uint32_t*>(pool + row * c.row_bytes + ch / 2), h4);
  }
  f16x8_f32(h4, x);
  const float f = e8m0_f32(scales[row * c.scale_stride + ch / kMxBlock]);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= f;
}
template <int FMT, int DP, int NT, bool EXT>
__device__ __noinline__ void plain_tiles(const PagedArgs a, int group, int b, int h, int row0,
                                         int start, int key_end, int tile0, int tile_end, float sl,
                                         PlainSums<DP, NT>* out) {
  constexpr int S = Cfg<FMT, DP, NT>::kStep, W = Cfg<FMT, DP, NT>::kWarps;
  const int g = lane_id() >> 2, t = lane_id() & 3, D = a.c.head_dim;
  const int tiles_per_page = a.c.page_size / kTile;
  float acc[DP / 16][NT][4] = {}, m[NT][2], l[NT][2] = {};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -FLT_MAX;
#pragma unroll 1
  for (int n = 0;; ++n) {
    const int tile = tile0 + n / S * (W * S) + n % S;
    if (tile >= tile_end) break;
    const int pi = tile / tiles_per_page;
    const int page = __ldg(a.block_table + table_at<EXT>(a, b, h) + pi);
    if (page < 0 || page >= a.c.n_pages) continue;
    const size_t at = kv_row(a.c, page, h, (tile - pi * tiles_per_page) * kTile);
    const int r1 = min(kTile, key_end - tile * kTile);
#pragma unroll 1
    for (int r = max(start - tile * kTile, 0); r < r1; ++r) {
      float s[NT][2] = {}, x[8];
#pragma unroll 1
      for (int ch = g * 8; ch < D; ch += 64) {
        decode8<FMT>(a.c, a.c.k, a.c.k_scale, at + r, ch, x);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int hd = row0 + nt * 8 + 2 * t + c;
            if (hd >= group) continue;
            const uint4 u = ldg_keep(static_cast<const __nv_bfloat16*>(a.q) +
                                     row_at<EXT>(a, group, b, h, hd, a.q_stride, D) + ch);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              s[nt][c] = fmaf(bf16_lo(word_of(u, k)), x[2 * k], s[nt][c]);
              s[nt][c] = fmaf(bf16_hi(word_of(u, k)), x[2 * k + 1], s[nt][c]);
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) s[nt][c] += __shfl_xor_sync(0xffffffffu, s[nt][c], k);
          const float y = s[nt][c] * sl, top = fmaxf(m[nt][c], y), f = ex2(m[nt][c] - top);
          m[nt][c] = top;
          s[nt][c] = ex2(y - top);
          l[nt][c] = l[nt][c] * f + (g == 0 ? s[nt][c] : 0.f);
#pragma unroll
          for (int i = 0; i < DP / 16; ++i) acc[i][nt][c] *= f, acc[i][nt][c + 2] *= f;
        }
#pragma unroll
      for (int v = 0; v < DP / 64; ++v) {
        if (v * 64 + g * 8 >= D) continue;
        decode8<FMT>(a.c, a.c.v, a.c.v_scale, at + r, v * 64 + g * 8, x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              acc[v * 4 + i][nt][c] =
                  fmaf(s[nt][c & 1], x[2 * i + (c >> 1)], acc[v * 4 + i][nt][c]);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) out->acc[i][nt][c] = acc[i][nt][c];
      if (c < 2) out->m[nt][c] = m[nt][c], out->l[nt][c] = l[nt][c];
    }
}

// EXT with fp32: the tensor core's sums, which it cuts to 24 bits at every step, are short ones
// that are added up in fp32 as it should be (kFine): four times as exact.
template <int FMT, int DP, int NT, bool EXT = false>
__global__ void __launch_bounds__(Cfg<FMT, DP, NT>::kWarps * 32, Cfg<FMT, DP, NT>::kPerSm)
    k_paged(const Params p) {
  using C = Cfg<FMT, DP, NT>;
  constexpr int W = C::kWarps, kJ = DP / 32, kV = DP / 64;
  constexpr bool kF32 = FMT == DT_F32, kMx = C::kMx, kFine = EXT && kF32;
  // Weights are 2^kLift at a head's running maximum (m: the maximum - kLift) and rise to
  // 2^kSlack times that before it is raised: to 1, so that sums overflow no sooner than plain
  // ones; or, in fp16 (MX caches, whose sums are relative to a scale), to 2^15, which keeps
  // 9 bits or more down to 2^-30 of the largest.
  constexpr float kSlack = kMx ? 1.f : 8.f, kLift = kMx ? 14.f : -8.f;
  extern __shared__ __align__(128) char smem[];
  __shared__ long long s_scan[W + 2];
  const PagedArgs& a = p.a;
  const int lane = lane_id(), w = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const int hr_n = a.c.n_heads * p.blocks;  // segments of a sequence

  if (!p.direct) {
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) p.span[blockIdx.x] = make_int4(0, 0, 0, 0);
  }

  auto places = [](int n) { return n > 0 ? n + C::kOpen : 0; };  // of a segment of n tiles
  // ---- this block's piece of the line --------------------------------------------------
  int b = 0;
  long long before = 0, total = 0;  // tiles before sequence b, tiles in all
  long long u0 = 0, u1 = 0, per = 0;
  if (p.direct) {
    b = blockIdx.x / hr_n;
    const int n = places(seq_of<EXT>(a, b, threadIdx.x == 0 && blockIdx.x % hr_n == 0).n);
    u0 = static_cast<long long>(blockIdx.x - b * hr_n) * n;  // counted from the sequence's start
    u1 = total = u0 + n;
    per = n;
  } else if (a.B <= 32) {  // every warp scans the lengths itself
    const int n = lane < a.B ? places(seq_of<EXT>(a, lane, blockIdx.x == 0 && w == 0).n) : 0;
    long long s = n;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, s, i);
      if (lane >= i) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31) * hr_n;
    per = quotient(total + gridDim.x - 1, gridDim.x);
    per = per < W * C::kStep ? W * C::kStep : per;
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
        const int n = i < a.B ? places(seq_of<EXT>(a, i, blockIdx.x == 0 && pass == 0).n) : 0;
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
        per = quotient(total + gridDim.x - 1, gridDim.x);
        per = per < W * C::kStep ? W * C::kStep : per;
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
    if (seq_of<EXT>(a, e, false).n > 0) continue;
    const int wide = kF32 || (EXT && a.raw) ? 4 : 2, bytes = a.n_q_heads * a.c.head_dim * wide;
    char* o = static_cast<char*>(a.out) + static_cast<size_t>(e) * a.out_stride * wide;
    for (int i = threadIdx.x * 16; i < bytes; i += W * 32 * 16)
      *reinterpret_cast<uint4*>(o + i) = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr)
      for (int i = threadIdx.x; i < a.n_q_heads; i += W * 32)
        store_lse<EXT>(a, a.n_q_heads, e, 0, i, -FLT_MAX, 0.f);
  }
  // launched while the kernel before still runs: this one's end has to imply that one's
  auto end = [&]() {
    if (EXT && a.overlap) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (u0 >= total) return end();

  const int D = a.c.head_dim;
  const uint32_t ring = smem_u32(smem) + w * (C::kRing * C::kSlot);
  uint4* s_q = reinterpret_cast<uint4*>(smem + C::kMain) + lane;  // kQShared: piece f at s_q[32 f]
  uint4* s_fine = s_q + C::kQBytes / 16;                          // MXFP8: the same
  // [W][8 NT] maxima, sums
  float* s_m = reinterpret_cast<float*>(smem + C::kMain + C::kQBytes + C::kFineBytes);
  float* s_l = s_m + W * 8 * NT;
  const float sl = a.scale * 1.4426950408889634f;
  const int tiles_per_page = a.c.page_size / kTile;
  const uint32_t tile_bytes = kTile * a.c.row_bytes;
  // this lane's places in a tile: where its copies go, where its reads start
  constexpr int kPieces = C::kRow / 16;
  // where rows are shorter: from lane * 16 to the lane's piece
  const int narrow = (lane / kPieces) * (a.c.row_bytes - C::kRow) -
                     (lane % kPieces * 16 < a.c.row_bytes ? 0 : lane % kPieces * 16);
  const uint32_t put_k = piece<FMT, C::kRow, true>(lane / kPieces, lane % kPieces);
  const uint32_t put_v = piece<FMT, C::kRow, false>(lane / kPieces, lane % kPieces);
  // keys: rows l % 8 (+ 8) of ldmatrix's four parts, two pieces; or row g's words
  const uint32_t get_k = FMT == DT_MXFP4 ? piece<FMT, C::kRow, true>(g, 0) + t * 4
                                         : piece<FMT, C::kRow, true>(lane & 15, lane >> 4);
  const uint32_t get_v =
      FMT == DT_BF16    ? piece<FMT, C::kRow, false>((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1)
      : FMT == DT_F32   ? piece<FMT, C::kRow, false>(2 * t, g * 2)
      : FMT == DT_MXFP8 ? piece<FMT, C::kRow, false>(2 * t, g >> 1) + (g & 1) * 8
                        : piece<FMT, C::kRow, false>(2 * t, g >> 2) + (g & 3) * 4;
  // MX: of two rows' scale words, the bytes of this lane's blocks 2v + g/4
  const uint32_t pick = (g >> 2) * 0x1111u + 0x6420u;
  // MX: a lane copies one word of the keys' scales (lanes 0-15) or the values'
  // (two, of rows of 8 bytes)
  const uint8_t* scale_src = (lane < 16 ? a.c.k_scale : a.c.v_scale) + (lane & 15) * 4;
  uint32_t live[2];  // the scale bytes of the head's blocks
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = D / kMxBlock - 4 * i;
    live[i] = n >= 4 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
  }

  Seq sq = seq_of<EXT>(a, b, false);
  long long into = u0 - before * hr_n;
  int hr = static_cast<int>(quotient(into, places(sq.n)));
  // place of the segment at hand where this block starts (tile + kOpen)
  int x0 = static_cast<int>(into - static_cast<long long>(hr) * places(sq.n));
  long long u = u0;
  bool first_seg = true;
  // the segment at hand: tiles [t0, t1) of sequence b, key head h, query heads from row0 on
  int t0 = 0, t1 = 0, h = 0, row0 = 0;
  constexpr int S = C::kStep, kScales = S * C::kTileBytes;  // scales' place in a slot
  constexpr int kLead = (C::kRing - 1) / 2;
  constexpr uint32_t kNone = 0xffffffffu;
  int n_it = 0, start = 0, tile0 = 0, tile_end = 0, key0 = 0, key_end = 0, batch = 0, whole_a = 0;
  unsigned whole_n = 0;
  uint32_t tile_of = 0, hidden = 0, fill = ring;

  // ---- a warp's steps of kStep tiles -------------------------------------------------
  // n_it steps (<= 0: none), step `it` takes the tiles tile0 + it W S ...; keys of the piece
  // end at key_end. Lane S k + i keeps the pool's tile (16 rows) of tile i of step batch + k.
  auto pages = [&](int it) {  // looks up the tiles of the next 32 / S steps
    batch = it;
    const int tile = tile0 + (it + lane / S) * (W * S) + lane % S;
    tile_of = kNone;
    if (tile < tile_end) {
      const int pi = tile / tiles_per_page;
      const int page = __ldg(a.block_table + table_at<EXT>(a, b, h) + pi);
      if (page < 0 || page >= a.c.n_pages)
        latch_error(a.status, kErrDevice);
      else
        tile_of = (static_cast<uint32_t>(page) * a.c.n_heads + h) * tiles_per_page +
                  (tile - pi * tiles_per_page);
    }
  };
  auto next = [&](uint32_t s) {
    s += C::kSlot;
    return s == ring + C::kRing * C::kSlot ? ring : s;
  };
  // Both scales of a tile go into its keys' slot: the keys' rows, then the values'.
  auto copy_scales = [&](int it, int i, uint32_t tile, int r0, int r1) {
    const uint32_t dst = fill + kScales + i * 2 * C::kTileScales;
    const uint8_t* src = scale_src + static_cast<uint64_t>(tile) * C::kTileScales;
    if constexpr (C::kScaleRow == 4) {
      const int r = lane & 15;
      cp_async4_n(dst + lane * 4, src, r >= r0 && r < r1 ? 4 : 0);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = (lane & 15) / 2 + 8 * e;
        cp_async4_n(dst + (lane >> 4) * C::kTileScales + (lane & 15) * 4 + e * 64, src + e * 64,
                    r >= r0 && r < r1 ? 4 : 0);
      }
    }
  };
  // whole_n steps from whole_a on are tiles in sight from end to end; once a page is left
  // out none is, and bit (it S + i) % 32 of `hidden` says which tiles are.
  auto issue = [&](int it, auto keys) {
    constexpr bool K = decltype(keys)::value;
    __syncwarp();
    if (it < n_it) {
      if (K && it >= batch + 32 / S) pages(it);
      const char* pool = (K ? a.c.k : a.c.v) + lane * 16;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const uint32_t tile = __shfl_sync(0xffffffffu, tile_of, (it - batch) * S + i);
        if (K && tile == kNone) {
          whole_n = 0;
          hidden |= 1u << ((it * S + i) & 31);
        } else if (K && hidden != 0) {
          hidden &= ~(1u << ((it * S + i) & 31));
        }
        const uint32_t dst = fill + i * C::kTileBytes;
        if (static_cast<unsigned>(it - whole_a) < whole_n) {
          const char* src = pool + static_cast<uint64_t>(tile) * tile_bytes;
          if (a.c.row_bytes == C::kRow)
            copy_tile<C, FMT, K>(dst, K ? put_k : put_v, src);
          else
            copy_narrow<C, FMT, K>(dst, K ? put_k : put_v, src + narrow, a.c.row_bytes, lane);
          if (K && kMx) copy_scales(it, i, tile, 0, kTile);
        } else {
          const uint32_t at = tile == kNone ? 0 : tile;
          const int key = key0 + (it * (W * S) + i) * kTile;
          const int r0 = start - key, r1 = tile == kNone ? 0 : key_end - key;
          copy_part<C, FMT, K>(dst, K ? put_k : put_v,
                               pool + static_cast<uint64_t>(at) * tile_bytes, a.c.row_bytes, r0,
                               r1, lane);
          if (K && kMx) copy_scales(it, i, at, r0, r1);
        }
      }
    }
    cp_async_commit();
    fill = next(fill);
  };
  using Keys = std::integral_constant<bool, true>;
  using Values = std::integral_constant<bool, false>;
  // sets a segment up and starts its first copies
  auto begin = [&]() {
    const int x1 = places(sq.n) - x0 < u1 - u ? places(sq.n) : x0 + static_cast<int>(u1 - u);
    t0 = max(x0 - C::kOpen, 0);
    t1 = max(x1 - C::kOpen, 0);
    h = hr / p.blocks;
    row0 = (hr - h * p.blocks) * 8 * NT;
    n_it = ((t1 - t0 + S - 1) / S - w + W - 1) / W;
    start = a.window > 0 && sq.len > a.window ? sq.len - a.window : 0;
    tile0 = sq.first + t0 + w * S;
    tile_end = sq.first + t1;
    key0 = tile0 * kTile;
    key_end = min(sq.len, (sq.first + t1) * kTile);
    whole_a = start > key0 ? 1 : 0;
    whole_n = key_end - key0 >= S * kTile
                  ? (key_end - key0 - S * kTile) / (W * S * kTile) + 1 - whole_a
                  : 0;
    batch = -32;
    hidden = 0;
    fill = ring;
#pragma unroll
    for (int i = 0; i < kLead; ++i) {
      issue(i, Keys());
      issue(i, Values());
    }
  };
  if (x0 + (u1 - u) <= C::kOpen) return end();  // nothing but empty places
  begin();
  while (true) {
    float acc[DP / 16][NT][4], m[NT][2], l[NT][2];
    // MX: acc holds O^T / 2^(ref - 127) of the lane's value block 2v + g/4; bias
    // is 14 - ref in both halves, byte v of ref0 the first ref. Blocks past the head
    // read scale 0 = ref.
    int ref[kMx ? kV : 1];
    uint32_t bias[kMx ? kV : 1], mine[kMx ? kV : 1], hot = 0, ref0 = 0;
    bool odd = false;  // MX: numbers too far apart for these operands (plain_tiles)
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
        bias[v] = (14 - ref[v]) * 0x10001;
        mine[v] = in ? 0x00ff00ffu : 0u;
      }
    }

    // ---- the queries, head g's (+ 8 nt) elements in the order of the keys' reads ---------
    uint4 q[kF32 ? 1 : NT][kJ];
    float xs[NT][2];  // scale of the scores of this lane's columns (heads 2t, 2t + 1)
    uint32_t fine = 0;  // MXFP8: bit j NT + nt: some of elements 32j .. + 31 are in s_fine
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      const size_t at = row_at<EXT>(a, p.group, b, h, r, a.q_stride, D);
      xs[nt][0] = xs[nt][1] = sl;
      if constexpr (kF32) {
        // in shared memory, once a block: per 8 elements t and t + 4 in two tf32 parts
        if (w == 0) {
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            const float* src = static_cast<const float*>(a.q) + at + i * 8 + t;
            const bool in = r < p.group && i * 8 < D;
            float hi[2], lo[2];
            split_tf32(in ? __ldg(src) : 0.f, &hi[0], &lo[0]);
            split_tf32(in ? __ldg(src + 4) : 0.f, &hi[1], &lo[1]);
            s_q[32 * i] = make_uint4(__float_as_uint(hi[0]), __float_as_uint(hi[1]),
                                     __float_as_uint(lo[0]), __float_as_uint(lo[1]));
          }
        }
      } else {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + at;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          q[nt][j] = make_uint4(0, 0, 0, 0);
          if (r >= p.group || j * 32 >= D) continue;
          if constexpr (FMT == DT_BF16) {  // elements 2t, 2t + 1 of every 8
            const uint32_t* u = reinterpret_cast<const uint32_t*>(src + j * 32) + t;
            q[nt][j].x = __ldg(u);
            if (j * 32 + 8 < D) q[nt][j].y = __ldg(u + 4);
            if (j * 32 + 16 < D) q[nt][j].z = __ldg(u + 8);
            if (j * 32 + 24 < D) q[nt][j].w = __ldg(u + 12);
          } else if constexpr (FMT == DT_MXFP8) {  // 4t .. + 3 of every 16
            const uint2* u = reinterpret_cast<const uint2*>(src + j * 32) + t;
            const uint2 lo = __ldg(u), hi = __ldg(u + 4);
            q[nt][j] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else {  // 8t .. + 7 of every 32
            q[nt][j] = ldg_keep(src + j * 32 + t * 8);
          }
        }
      }
      if constexpr (kMx) {
        // The head's largest element is brought to [2^kTop, 2^(kTop + 1)), an exact
        // power of two that goes into the scores' scale. MXFP4 keys meet fp16
        // queries. MXFP8 keys are an operand as they are: the query is cut in an e4m3 term and
        // an e5m2 one, what the first leaves (at most half its last place: three bits).
        // bf16's 8 bits fit the two exactly down to 2^-13 of the largest element, and fp16 down
        // to 2^-31. Smaller elements, few if any, meet MXFP8 keys in fp16 (`fine`), 2^7 larger;
        // queries with elements below 2^-31 of the largest take the plain pass.
        constexpr int kTop = FMT == DT_MXFP8 ? 7 : 14, kFit = FMT == DT_MXFP8 ? 13 : 31;
        uint32_t most = 0, least = 0x7fff7fffu;
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = word_of(q[nt][j], i) & 0x7fff7fffu;
            most = __vmaxu2(most, v);
            if (j * 32 < D) least = __vminu2(least, v);
          }
        uint32_t top = max(most << 16, most & 0x7fff0000u);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = static_cast<int>(top >> 23) - 127;
        e = e < -112 ? -112 : e;
        // Against such queries (or such a scale) key scales of 2^-127, which count as 0 below, or
        // scores near the smallest numbers would show
        odd |= top != 0 && (max(e, e + static_cast<int>(__float_as_uint(sl) >> 23 & 255u) - 127) > 80 ||
                            e < -80);
        const float up = __uint_as_float(static_cast<uint32_t>(kTop - e + 127) << 23);
        const uint32_t fit = static_cast<uint32_t>(e - kFit + 127) << 23;
        if (__any_sync(0xffffffffu, r < p.group && min(least << 16, least & 0x7fff0000u) < fit)) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            uint32_t keep[4], rest[4];
            bool some = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v = word_of(q[nt][j], i), v0 = v << 16, v1 = v & 0xffff0000u;
              const uint32_t a0 = v0 & 0x7fffffffu, a1 = v1 & 0x7fffffffu;
              odd |= a0 - 1 < (fit - (31 - kFit) * 0x800000u) - 1 ||
                     a1 - 1 < (fit - (31 - kFit) * 0x800000u) - 1;
              const bool s0 = a0 < fit, s1 = a1 < fit;
              some |= (s0 && a0 != 0) || (s1 && a1 != 0);
              keep[i] = (s0 ? 0u : v0 >> 16) | (s1 ? 0u : v1);
              rest[i] = pack_f16x2(s0 ? __uint_as_float(v0) * up * 0x1p7f : 0.f,
                                   s1 ? __uint_as_float(v1) * up * 0x1p7f : 0.f);
            }
            if constexpr (FMT == DT_MXFP8) {
              q[nt][j] = make_uint4(keep[0], keep[1], keep[2], keep[3]);
              // every warp of the block writes the same values, and reads its own
              s_fine[32 * (j * NT + nt)] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
              fine |= (__any_sync(0xffffffffu, some) ? 1u : 0u) << (j * NT + nt);
            }
          }
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const uint4 v = q[nt][j];
          const float y[8] = {bf16_lo(v.x) * up, bf16_hi(v.x) * up, bf16_lo(v.y) * up,
                              bf16_hi(v.y) * up, bf16_lo(v.z) * up, bf16_hi(v.z) * up,
                              bf16_lo(v.w) * up, bf16_hi(v.w) * up};
          if constexpr (FMT == DT_MXFP8) {
            const uint2 hi = pack_e4m3x8(y);
            uint32_t h4[4];
            float z[8];
            e4m3x8_f16(hi.x, hi.y, h4);
            f16x8_f32(h4, z);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = y[i] - z[i];
            const uint2 lo = pack_e5m2x8(z);
            q[nt][j] = make_uint4(hi.x, hi.y, lo.x, lo.y);
          } else {
            q[nt][j] = make_uint4(pack_f16x2(y[0], y[1]), pack_f16x2(y[2], y[3]),
                                  pack_f16x2(y[4], y[5]), pack_f16x2(y[6], y[7]));
          }
        }
        // (an infinite or NaN query: NaN scores)
        const float down = e > 127 ? __uint_as_float(0x7fc00000u)
                                   : __uint_as_float(static_cast<uint32_t>(e - kTop + 127) << 23);
        // scales below carry a factor 1 + 2^-23
        xs[nt][0] = sl * __shfl_sync(0xffffffffu, down, 8 * t) * (1.f - 0x1p-23f);
        xs[nt][1] = sl * __shfl_sync(0xffffffffu, down, 8 * t + 4) * (1.f - 0x1p-23f);
      }
      if constexpr (!kF32 && C::kQShared) {
        // every warp of the block writes the same values, and reads its own
#pragma unroll
        for (int j = 0; j < kJ; ++j) s_q[32 * (j * NT + nt)] = q[nt][j];
        __syncwarp();
      }
    }
    if constexpr (kF32) __syncthreads();

    uint32_t slot = ring;
    for (int it = 0; it < n_it; ++it) {
      // ---- scores: lane 4g + t gets keys g, g + 8 of heads 2t, 2t + 1 --------------------
      issue(it + kLead, Keys());
      cp_async_wait<C::kRing - 1>();
      __syncwarp();
      float x[S][NT][4];
      // MX: bytes of the values' scales, of keys 2t, 2t + 1 (+ 8 k) and this lane's blocks
      uint32_t vs[S][2][2];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const uint32_t tile = slot + i * C::kTileBytes;
        if constexpr (FMT == DT_BF16) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[i][nt][c] = 0.f;
#pragma unroll
          for (int j = 0; j < DP / 16; ++j) {
            uint32_t k4[4];
            ldsm4(k4, further(tile + get_k, j * 32));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 u = C::kQShared ? s_q[32 * (j / 2 * NT + nt)] : q[nt][j / 2];
              mma_bf16_16816(x[i][nt], k4[0], k4[1], k4[2], k4[3], j % 2 ? u.z : u.x,
                             j % 2 ? u.w : u.y);
            }
          }
        } else if constexpr (kF32) {
          // Three tf32 products, hi hi + lo hi + hi lo. An infinity times a part that is 0
          // would be NaN: where a score is NaN it is formed again with such operands left
          // out of the cross products.
#pragma unroll 1
          for (int careful = 0; careful < 2; ++careful) {
            bool nan = false;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) {
              uint32_t k4[4];
              ldsm4(k4, further(tile + get_k, j * 32));
              const uint4 qv = s_q[32 * j];
              float hi[4], lo[4];
              float qh[2] = {__uint_as_float(qv.x), __uint_as_float(qv.y)};
              const float ql[2] = {__uint_as_float(qv.z), __uint_as_float(qv.w)};
#pragma unroll
              for (int k = 0; k < 4; ++k) split_tf32(__uint_as_float(k4[k]), &hi[k], &lo[k]);
              mma_tf32_1688(d, hi, qh);
              if (careful) {
#pragma unroll
                for (int k = 0; k < 4; ++k) hi[k] = fabsf(hi[k]) == INFINITY ? 0.f : hi[k];
#pragma unroll
                for (int k = 0; k < 2; ++k) qh[k] = fabsf(qh[k]) == INFINITY ? 0.f : qh[k];
              }
              mma_tf32_1688(d, lo, qh);
              mma_tf32_1688(d, hi, ql);
              if constexpr (kFine) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  x[i][0][c] = j == 0 ? d[c] : x[i][0][c] + d[c];
                  d[c] = 0.f;
                }
              }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if constexpr (!kFine) x[i][0][c] = d[c];
              nan |= x[i][0][c] != x[i][0][c];
            }
            if (!__any_sync(0xffffffffu, nan)) break;
          }
        } else {
          // The blocks' scales of keys g and g + 8, as fp32 bits with the last bit set: byte
          // 255 is then NaN by itself (and byte 0, 2^-127, counts as 0). A scale goes on its
          // block's partial score: codes are exact operands.
          const uint32_t sat = slot + kScales + i * 2 * C::kTileScales + g * C::kScaleRow;
          uint32_t sc0[2], sc1[2];
#pragma unroll
          for (int k = 0; k < C::kScaleRow / 4; ++k) {
            // bytes past the head's blocks may hold anything: 1
            sc0[k] = (lds32(sat + 4 * k) & live[k]) | (0x7f7f7f7fu & ~live[k]);
            sc1[k] = (lds32(sat + 8 * C::kScaleRow + 4 * k) & live[k]) | (0x7f7f7f7fu & ~live[k]);
          }
          // the values' scales too: this slot is filled again before they are needed
          const uint32_t vat = slot + kScales + (2 * i + 1) * C::kTileScales + 2 * t * C::kScaleRow;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if constexpr (C::kScaleRow == 4) {
              const uint2 v = lds64(vat + 8 * k * C::kScaleRow);
              vs[i][k][0] = __byte_perm(v.x, v.y, pick);
            } else {
              const uint4 v = lds128(vat + 8 * k * C::kScaleRow);
              vs[i][k][0] = __byte_perm(v.x, v.z, pick);
              vs[i][k][1] = __byte_perm(v.y, v.w, pick);
            }
          }
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const int up = 23 - 8 * (j % 4);
            const float f0 = __uint_as_float(
                ((up > 0 ? sc0[j / 4] << (up & 31) : sc0[j / 4] >> 1) & 0x7f800000u) | 1u);
            const float f1 = __uint_as_float(
                ((up > 0 ? sc1[j / 4] << (up & 31) : sc1[j / 4] >> 1) & 0x7f800000u) | 1u);
            uint32_t k4[4], ka[4], kb[4];
            if constexpr (FMT == DT_MXFP8) {
              ldsm4(k4, further(tile + get_k, j * 32));
            } else {
              const uint32_t at = further(tile + get_k, j * 16);
              e2m1x8_f16(lds32(at), ka);
              e2m1x8_f16(lds32(at + 8 * C::kRow), kb);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float d[4];
              const uint4 u = C::kQShared ? s_q[32 * (j * NT + nt)] : q[nt][j];
              if constexpr (FMT == DT_MXFP8) {
                mma_e4m3_e5m2_16832_z(d, k4[0], k4[1], k4[2], k4[3], u.z, u.w);
                mma_e4m3_16832(d, k4[0], k4[1], k4[2], k4[3], u.x, u.y);
              } else {
                mma_f16_16816_z(d, ka[0], kb[0], ka[1], kb[1], u.x, u.y);
                mma_f16_16816(d, ka[2], kb[2], ka[3], kb[3], u.z, u.w);
              }
#pragma unroll
              for (int c = 0; c < 4; ++c)
                x[i][nt][c] = j == 0 ? d[c] * (c < 2 ? f0 : f1)
                                     : fmaf(d[c], c < 2 ? f0 : f1, x[i][nt][c]);
            }
          }
          if constexpr (FMT == DT_MXFP8) {
#pragma unroll 1
            for (uint32_t todo = fine; todo != 0; todo &= todo - 1) {
              const int f = __ffs(todo) - 1, j = f / NT;
              const uint32_t s0 = DP > 128 && j >= 4 ? sc0[1] : sc0[0];
              const uint32_t s1 = DP > 128 && j >= 4 ? sc1[1] : sc1[0];
              const float f0 = __uint_as_float((s0 >> 8 * (j % 4) << 23 & 0x7f800000u) | 1u);
              const float f1 = __uint_as_float((s1 >> 8 * (j % 4) << 23 & 0x7f800000u) | 1u);
              uint32_t k4[4], h[4];
              float d[4];
              const uint4 u = s_fine[32 * f];
              ldsm4(k4, further(tile + get_k, j * 32));
              // a word of four codes: the product's indices 2t, 2t + 1 and 2t + 8, 2t + 9
              e4m3x8_f16(k4[0], k4[1], h);
              mma_f16_16816_z(d, h[0], h[2], h[1], h[3], u.x, u.y);
              e4m3x8_f16(k4[2], k4[3], h);
              mma_f16_16816(d, h[0], h[2], h[1], h[3], u.z, u.w);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (nt != f % NT) continue;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  x[i][nt][c] = fmaf(d[c] * 0x1p-7f, c < 2 ? f0 : f1, x[i][nt][c]);
              }
            }
          }
        }
      }
      const bool part = static_cast<unsigned>(it - whole_a) >= whole_n;
      // first and last row of a tile in sight
      auto rows = [&](int i, int* r0, int* r1) {
        const int key = key0 + (it * (W * S) + i) * kTile;
        *r0 = start - key;
        *r1 = hidden >> ((it * S + i) & 31) & 1u ? 0 : key_end - key;
      };
      // scores of keys out of sight
      auto hide = [&](float(&s)[S][NT][4]) {
        if (!part) return;
#pragma unroll
        for (int i = 0; i < S; ++i) {
          int r0, r1;
          rows(i, &r0, &r1);
          const bool in0 = g >= r0 && g < r1, in1 = g + 8 >= r0 && g + 8 < r1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (!in0) s[i][nt][0] = s[i][nt][1] = kMx ? -FLT_MAX : -INFINITY;
            if (!in1) s[i][nt][2] = s[i][nt][3] = kMx ? -FLT_MAX : -INFINITY;
          }
        }
      };
      // ---- weights: 2^y, y = scaled score - m ------------------------------------------
      float y[S][NT][4];
      auto exponents = [&]() {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              y[i][nt][c] = fmaf(x[i][nt][c], xs[nt][c & 1], -m[nt][c & 1]);
        hide(y);
      };
      exponents();
      float top = y[0][0][0];
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) top = fmaxf(top, y[i][nt][c]);
      if (__any_sync(0xffffffffu, top > kLift + kSlack)) {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) y[i][nt][c] = x[i][nt][c] * xs[nt][c & 1];
        hide(y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = fmaxf(y[0][nt][c], y[0][nt][c + 2]);
#pragma unroll
            for (int i = 1; i < S; ++i) v = fmaxf(v, fmaxf(y[i][nt][c], y[i][nt][c + 2]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            v = fmaxf(v - kLift, m[nt][c]);
            const float f = ex2(m[nt][c] - v);
            m[nt][c] = v;
            l[nt][c] *= f;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) acc[i][nt][c] *= f, acc[i][nt][c + 2] *= f;
          }
        exponents();
      }
      // MX: a weight below 2^-30 of the largest that is not 0. Keys out of sight weigh 0, which
      // fp16 holds (counted, they sent every first and last step the wide way: 160 windows of 300
      // MXFP8 tokens 80 us instead of 64, 64 contexts up to 900 28.8 instead of 26.8).
      bool wide = false;
      if constexpr (kMx) {
        float low = 0.f;
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) low = fminf(low, y[i][nt][c]);
        // a score of -inf: plain_tiles (keys out of sight of MX caches have the lowest finite one)
        if (__any_sync(0xffffffffu, low == -INFINITY)) odd = true;
        if (part) {
          low = 0.f;
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (y[i][nt][c] > -128.f) low = fminf(low, y[i][nt][c]);
        }
        wide = low < -16.f;
      }
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            x[i][nt][c] = ex2(y[i][nt][c]);
            l[nt][c & 1] += x[i][nt][c];
          }
      slot = next(slot);

      // ---- values: O^T += V^T P^T ----------------------------------------------------------
      issue(it + kLead, Values());
      // the weights as the product's operand: keys 2t, 2t + 1 (and + 8) of head g
      if constexpr (FMT == DT_BF16) {
        uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // bf16 weights and, beside them, what the rounding left: 16 bits together
          const float(&y)[4] = x[0][nt];
          const uint32_t h0 = pack_bf16x2(y[0], y[1]), h1 = pack_bf16x2(y[2], y[3]);
          pb[nt][0] = transpose8(h0);
          pb[nt][1] = transpose8(h1);
          pl[nt][0] = transpose8(pack_bf16x2(y[0] - bf16_lo(h0), y[1] - bf16_hi(h0)));
          pl[nt][1] = transpose8(pack_bf16x2(y[2] - bf16_lo(h1), y[3] - bf16_hi(h1)));
        }
        cp_async_wait<C::kRing - 1>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          uint32_t v4[4];
          ldsm4_t(v4, further(slot + get_v, i * 32));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(acc[i][nt], v4[0], v4[1], v4[2], v4[3], pb[nt][0], pb[nt][1]);
            mma_bf16_16816(acc[i][nt], v4[0], v4[1], v4[2], v4[3], pl[nt][0], pl[nt][1]);
          }
        }
      } else if constexpr (kF32) {
        float pf[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int src = 8 * t + (g >> 1);  // lane of key 2t, head g
#pragma unroll
          for (int k = 0; k < 4; ++k) {      // keys 2t, 2t + 1, 2t + 8, 2t + 9
            const float e0 = __shfl_sync(0xffffffffu, x[0][nt][(k >> 1) * 2], src + (k & 1) * 4);
            const float e1 =
                __shfl_sync(0xffffffffu, x[0][nt][(k >> 1) * 2 + 1], src + (k & 1) * 4);
            pf[nt][k] = g & 1 ? e1 : e0;
          }
        }
        cp_async_wait<C::kRing - 1>();
        __syncwarp();
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
                  float(&sum)[4] = acc[v * 4 + hf * 2 + i][nt];
                  float part[4] = {0.f, 0.f, 0.f, 0.f};
                  float(&d)[4] = kFine ? part : sum;
                  mma_tf32_1688(d, lo, ph);
                  mma_tf32_1688(d, hi, plo);
                  mma_tf32_1688(d, hi, ph);
                  if constexpr (kFine) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum[c] += part[c];
                  }
                }
              }
            }
          }
        }
      } else {
        cp_async_wait<C::kRing - 1>();
        __syncwarp();
        // Value codes are exact in fp16, and so is a code times 2^(s - ref) for
        // scales s in [ref - 14, ref + 1]: ref follows the largest scale of the
        // lane's block (the four lanes of a g share it). sd holds s - ref + 14
        // for the keys of a pair in its halves: four bits, or the scale is out of that
        // range (a borrow or carry between the halves only comes with such a one).
        // A step with a scale below it, a NaN one or a weight too small for fp16 is
        // done with bf16 operands. Values and earlier sums stay exact there for scales less than
        // kFar below ref, and ref within kFar of the first one. Further off the smaller values
        // may still be what counts, where the larger ones have no weight: such a warp
        // takes its tiles again, in plain fp32.
        constexpr int kFar = 48;
        uint32_t sd[S][kV][2];
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < S; ++i) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int e = 0; e < C::kScaleRow / 4; ++e) {
              const uint32_t by = vs[i][k][e];
              sd[i][2 * e][k] = (by & mine[2 * e]) + bias[2 * e];
              if constexpr (kV > 1)
                sd[i][2 * e + 1][k] = (by >> 8 & mine[2 * e + 1]) + bias[2 * e + 1];
            }
            if (part) {  // rows out of sight hold zeros, whatever their scale
              int r0, r1;
              rows(i, &r0, &r1);
              const int row = 2 * t + 8 * k;
              const uint32_t lo = row < r0 || row >= r1 ? 0xffffu : 0u;
              const uint32_t hi = row + 1 < r0 || row + 1 >= r1 ? 0xffff0000u : 0u;
#pragma unroll
              for (int v = 0; v < kV; ++v)
                sd[i][v][k] = (sd[i][v][k] & ~(lo | hi)) | (0x000e000eu & (lo | hi));
            }
#pragma unroll
            for (int v = 0; v < kV; ++v)
              bad |= sd[i][v][k] & 0xfff0fff0u;
          }
        }
        bad |= hot;
        if (__any_sync(0xffffffffu, bad != 0)) {
          // raise ref where a scale is above its range; is everything in range then?
          hot = 0;
#pragma unroll
          for (int v = 0; v < kV; ++v) {
            int sv[S][4], most = -1;
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                sv[i][k] = (vs[i][k >> 1][v / 2] >> 8 * (v & 1) & mine[v]) >> 16 * (k & 1) & 0xffu;
                int r0, r1;
                rows(i, &r0, &r1);
                const int row = 2 * t + (k & 1) + (k >> 1) * 8;
                if (row < r0 || row >= r1) sv[i][k] = -1;  // zeros, whatever the scale
                if (sv[i][k] != 255) most = max(most, sv[i][k]);
              }
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
            if (most >= 0 && most > ref[v] + 1) {
              if (ref[v] == -1000) ref0 |= most << 8 * v;
              odd |= most > static_cast<int>(ref0 >> 8 * v & 0xffu) + kFar;
              const float f = ex2(static_cast<float>(ref[v] - most));
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 4; ++c) acc[v * 4 + i][nt][c] *= f;
              ref[v] = most;
              bias[v] = (14 - most) * 0x10001;
            }
            if (ref[v] > 247) hot = 1;  // a NaN scale would pass for 2^128
#pragma unroll
            for (int i = 0; i < S; ++i) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (sv[i][k] < 0) sv[i][k] = ref[v];
                const int e = max(sv[i][k] - ref[v], -kFar);
                wide |= e < -14 || sv[i][k] == 255;
                sv[i][k] = (sv[i][k] == 255 ? 255 : e) + 14;  // 255: NaN (e is at most 1)
              }
              sd[i][v][0] = (sv[i][0] & 0xffffu) | sv[i][1] << 16;
              sd[i][v][1] = (sv[i][2] & 0xffffu) | sv[i][3] << 16;
            }
          }
        }
        auto product = [&](auto way) {
          constexpr bool kWide = decltype(way)::value;
#pragma unroll
          for (int i = 0; i < S; ++i) {
            uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float(&y)[4] = x[i][nt];
              if constexpr (!kWide) {
                pb[nt][0] = transpose8(pack_f16x2(y[0], y[1]));
                pb[nt][1] = transpose8(pack_f16x2(y[2], y[3]));
              } else {
                const uint32_t h0 = pack_bf16x2(y[0], y[1]), h1 = pack_bf16x2(y[2], y[3]);
                pb[nt][0] = transpose8(h0);
                pb[nt][1] = transpose8(h1);
                pl[nt][0] = transpose8(pack_bf16x2(y[0] - bf16_lo(h0), y[1] - bf16_hi(h0)));
                pl[nt][1] = transpose8(pack_bf16x2(y[2] - bf16_lo(h1), y[3] - bf16_hi(h1)));
              }
            }
            const uint32_t at = slot + i * C::kTileBytes + get_v;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
              uint32_t op[2][8];  // [keys 2t, 2t + 1 or + 8][element]: the two keys' codes in fp16
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t off = v * (C::kBits * 8) + k * 8 * C::kRow;
                uint32_t h4[4];
                if constexpr (FMT == DT_MXFP8) {
                  const uint2 e0 = lds64(further(at, off)), e1 = lds64(further(at, off + C::kRow));
                  e4m3x8_f16(__byte_perm(e0.x, e1.x, 0x5140), __byte_perm(e0.x, e1.x, 0x7362), h4);
#pragma unroll
                  for (int c = 0; c < 4; ++c) op[k][c] = h4[c];
                  e4m3x8_f16(__byte_perm(e0.y, e1.y, 0x5140), __byte_perm(e0.y, e1.y, 0x7362), h4);
#pragma unroll
                  for (int c = 0; c < 4; ++c) op[k][4 + c] = h4[c];
                } else {
                  const uint32_t e0 = lds32(further(at, off));
                  const uint32_t e1 = lds32(further(at, off + C::kRow));
                  e2m1x8_f16((e0 & 0x0f0f0f0fu) | ((e1 & 0x0f0f0f0fu) << 4), h4);
#pragma unroll
                  for (int c = 0; c < 4; ++c) op[k][2 * c] = h4[c];
                  e2m1x8_f16(((e0 >> 4) & 0x0f0f0f0fu) | (e1 & 0xf0f0f0f0u), h4);
#pragma unroll
                  for (int c = 0; c < 4; ++c) op[k][2 * c + 1] = h4[c];
                }
                if constexpr (!kWide) {
                  const uint32_t f = sd[i][v][k] * 1024u + 0x04000400u;  // 2^(s - ref), both keys
#pragma unroll
                  for (int c = 0; c < 8; ++c) op[k][c] = mul_f16x2(op[k][c], f);
                } else {
                  const int e0 = static_cast<int16_t>(sd[i][v][k] & 0xffffu) - 14;
                  const int e1 = static_cast<int16_t>(sd[i][v][k] >> 16) - 14;
                  uint32_t any = 0;  // zeros lie at no distance
#pragma unroll
                  for (int c = 0; c < 8; ++c) any |= op[k][c];
                  odd |= (e0 == -kFar && (any & 0x7fffu)) || (e1 == -kFar && (any & 0x7fff0000u));
                  const float f0 = __uint_as_float(e0 == 255 ? 0x7fc00000u : (e0 + 127u) << 23);
                  const float f1 = __uint_as_float(e1 == 255 ? 0x7fc00000u : (e1 + 127u) << 23);
#pragma unroll
                  for (int c = 0; c < 8; ++c) {
                    float lo, hi;
                    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                        : "=f"(lo), "=f"(hi)
                        : "r"(op[k][c]));
                    op[k][c] = pack_bf16x2(lo * f0, hi * f1);
                  }
                }
              }
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float(&d)[4] = acc[v * 4 + c][nt];
                  const uint32_t a0 = op[0][2 * c], a1 = op[0][2 * c + 1], a2 = op[1][2 * c],
                                 a3 = op[1][2 * c + 1];
                  if constexpr (!kWide) {
                    mma_f16_16816(d, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                  } else {
                    mma_bf16_16816(d, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    mma_bf16_16816(d, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                  }
                }
            }
          }
        };
        if (__any_sync(0xffffffffu, wide))
          product(std::integral_constant<bool, true>());
        else
          product(std::integral_constant<bool, false>());
      }
      slot = next(slot);
    }

    if constexpr (kMx) {
      // A block's partial score times its scale may overflow where the score itself does not:
      // a score of infinity was seen above, or left NaN in the sums.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) odd |= l[nt][0] != l[nt][0] || l[nt][1] != l[nt][1];
      if (__any_sync(0xffffffffu, odd)) {
        PlainSums<DP, NT> sums;
        plain_tiles<FMT, DP, NT, EXT>(a, p.group, b, h, row0, start, key_end, tile0, tile_end, sl, &sums);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) acc[i][nt][c] = sums.acc[i][nt][c];
            if (c < 2) m[nt][c] = sums.m[nt][c], l[nt][c] = sums.l[nt][c];
          }
#pragma unroll
        for (int v = 0; v < kV; ++v) ref[v] = 127;
      }
    }

    // ---- the next segment's first copies fly while this one is joined ------------------
    const int ob = b, ohr = hr, oh = h, orow0 = row0, on = sq.n;
    const bool whole = t0 == 0 && t1 == sq.n, opens = t0 == 0 && !whole, slot1 = !first_seg;
    const long long oend = u - x0 + places(on);  // the segment's end on the line
    u = oend;
    first_seg = false;
    x0 = 0;
    // another segment, unless only its empty places are left
    const bool more = u + C::kOpen < u1;
    if (more) {
      if (++hr == hr_n) {
        hr = 0;
        do {
          sq = seq_of<EXT>(a, ++b, false);
        } while (sq.n == 0);
      }
      begin();
    }

    // ---- join the warps ------------------------------------------------------------------
    // Each warp's sums over its weights' sum first: means of values, which cannot overflow.
    // MX: on a value scale of 1 or more the reciprocal goes on the scale, so that neither
    // product leaves the range before the result does.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], i);
    float inv[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) inv[nt][c] = l[nt][c] == 0.f ? 0.f : reciprocal(l[nt][c]);
#pragma unroll
    for (int v = 0; v < DP / 64; ++v) {
      const float f = !kMx ? 1.f : ref[v] == -1000 ? 0.f : e8m0_f32(ref[v]);
      const float f0 = f < 1.f ? 1.f : f, f1 = f < 1.f ? f : 1.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float by = inv[nt][c] * f0;
#pragma unroll
          for (int i = v * 4; i < v * 4 + 4; ++i) {
            acc[i][nt][c] = acc[i][nt][c] * by * f1;
            acc[i][nt][c + 2] = acc[i][nt][c + 2] * by * f1;
          }
        }
    }
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) s_m[w * 8 * NT + nt * 8 + 2 * t + c] = m[nt][c];
    }
    __syncthreads();  // maxima in place
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = -FLT_MAX;
#pragma unroll
        for (int k = 0; k < W; ++k) top = fmaxf(top, s_m[k * 8 * NT + nt * 8 + 2 * t + c]);
        if (g == 0) s_l[w * 8 * NT + nt * 8 + 2 * t + c] = l[nt][c] * ex2(m[nt][c] - top);
      }
    float* merge = reinterpret_cast<float*>(smem + C::kRingBytes) + lane;
    float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (slot1 ? 1 : 0)) * C::kPart;
    constexpr int kHalf = DP / 32 * NT;  // groups (MMA tiles of 16 x 8) of half the registers
#pragma unroll
    for (int rd = 0; rd < 2; ++rd) {
#pragma unroll
      for (int i = 0; i < DP / 32; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            merge[(w * kHalf + i * NT + nt) * 128 + c * 32] = acc[rd * (DP / 32) + i][nt][c];
      __syncthreads();
      // warp w joins the groups w, w + W, ... of all warps
      for (int k0 = w; k0 < kHalf; k0 += W) {
        const int gr = rd * kHalf + k0;
        const int i = gr / NT, nt = gr - i * NT;
        float o[4] = {0.f, 0.f, 0.f, 0.f}, sum[2] = {0.f, 0.f}, mx[2] = {-FLT_MAX, -FLT_MAX}, by[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          for (int k = 0; k < W; ++k) {
            sum[c] += s_l[k * 8 * NT + nt * 8 + 2 * t + c];
            mx[c] = fmaxf(mx[c], s_m[k * 8 * NT + nt * 8 + 2 * t + c]);
          }
          by[c] = sum[c] == 0.f ? 0.f : reciprocal(sum[c]);
        }
        for (int k = 0; k < W; ++k) {
          const float* src = merge + (k * kHalf + k0) * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            o[c] = fmaf(src[c * 32], s_l[k * 8 * NT + nt * 8 + 2 * t + (c & 1)] * by[c & 1], o[c]);
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
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = orow0 + nt * 8 + 2 * t + c;
            if (r >= p.group) continue;
            store_out<FMT == DT_BF16, kF32, EXT>(a, row_at<EXT>(a, p.group, ob, oh, r, a.out_stride, D), i, g,
                                            sum[c] == 0.f ? 0.f : o[c],
                                            sum[c] == 0.f ? 0.f : o[c + 2]);
            if (a.lse != nullptr && i == 0 && g == 0)
              store_lse<EXT>(a, p.group, ob, oh, r, mx[c], sum[c]);
          }
        }
      }
      __syncthreads();
    }
    if (opens && threadIdx.x == 0) {
      // the segment starts here and ends in a later block
      p.span[blockIdx.x] = make_int4(ob, ohr, slot1 ? 1 : 0,
                                     static_cast<int>(quotient(oend - 1, per)) - blockIdx.x + 1);
    }
    if (!more) break;
  }
  end();
}

}  // namespace paged
}  // namespace coli
