// Attention of many sequences' queries over one shared prefix, on the tcgen05 tensor cores.
//
// Mathematics. The queries of all sequences that share a key head are the rows of one matrix
// (R = B * heads of a group), so the prefix is attention with R queries: S = Q K^T,
// P = 2^(s x - m), O += P V with a running maximum m, the prefix read once for 128 rows
// instead of once for each sequence.
//
// A block takes 128 or (PAIR) 256 rows of a key head and a run of 128-key tiles. It has two
// streams, each with its own S, O, m and l in tensor memory and registers of its own warpgroup
// (columns 0-127 and 128-255 S, 256-511 O), so one stream's softmax runs under the other's
// products: the MMA warp issues S(0) S(1) PV(0) S(2) PV(1) ... in order. The streams take the
// tiles by turns, and their sums are joined at the end; or, with 256 rows, 128 rows each and
// every tile, so that a tile is loaded (and widened) for twice the products. P goes back
// over S's columns as two bf16 terms, the weight and what its rounding left (16 bits together),
// and is the second product's A operand from tensor memory; V is its B operand as it lies
// (keys by channels, "transposed"). m is raised only where a score passes it (weights are
// 2^-8 at a new maximum and rise to 1), so O is rarely rescaled.
//
// Loader warps bring K and V tiles to 128-byte swizzled shared memory: bf16 by TMA, a box a
// page or the part of it that the tile has (rows past the pool read as zeros, which stands for
// pages that are left out; the 16 rows that the prefix ends in are copied by hand, zeros behind
// it); MX codes by TMA as they are, then widened to bf16 with their scale by eight warps (exact
// within bf16's range, which is fp32's). Scores of keys out of sight are set to -inf.
//
// Heads above 128 (bf16): two accumulators of 256 columns and the scores are more than tensor
// memory holds, so a segment has half of the values' channels and forms the scores for itself.
//
// Work split: the tiles of all (key head, 128 rows) segments lie on one line that is cut into
// equal pieces, one a block; a piece's part of a segment gives a partial mean with (m, l), in
// slot (block + segment), which k_shared_join joins in the line's order with each sequence's
// own tokens.
//
// What bounds it (GB300, heads of 128): the products, 24 instructions of 128 x 128 x 16 a unit
// (128 rows by 128 keys). By the SM's clock a unit of paired bf16 rows takes 2330 cycles, of which
// the warp that issues the products waits 220 for weights and 250 for tiles; in the rest the tensor
// cores take an instruction every 78, where the pipe's rate is 64. A stream goes from
// its scores to its weights in 2130 cycles and then waits 1900 for the next scores. MXFP8: 2640 a
// unit, 190 and 300 of them waits, 2440 from scores to weights. 128 rows alone load a tile for half the
// products: 2850, 920 of them waits for tiles. 64 sequences of 32 heads on 8 behind 32768 bf16 tokens
// 54 us, 128 of 64 on 8 behind 40009 MXFP8 ones 201 us (835 TFLOP/s, 1250 with the second
// weight term); ncu has the tensor pipe at 43% to 50%, starts and ends included. The
// second term costs a third of the products; without it the output's error would be 1.2 times
// the rounding's own. What a block does once (queries, first tiles, the last means) takes 8 us.
// Heads of 256: 64 instructions for 128 rows by 128 keys, a quarter of them the scores formed
// twice, and keys loaded for 128 rows and half of the values: 4060 cycles a unit, 1740 of them waits
// for tiles; the call of 64 sequences of 32 heads on 8 behind 32768 tokens 161 us.
#include <limits.h>

#include "tcgen05.cuh"

#include "mx.cuh"
#include "paged.cuh"
#include "prefix.h"

namespace coli {
namespace {

using paged::ex2;

constexpr int kSub = kPrefixRows * 128;  // bytes of 128 rows of 64 channels
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoad0 = 9;
constexpr int kConv0 = 12, kConvWarps = 8;  // MX: the warps that widen
constexpr uint32_t kOCol = 256;          // O of the streams; S at 0 and 128
constexpr uint32_t kNone = 0xffffffffu;

constexpr int kMost = 3, kRaw = 3;

// Heads above 128 (DP 256): a segment has all of them for its scores and half of the values'
// channels, and keys come in two parts of 128.
template <int DP>
constexpr int halves() {
  return DP > 128 ? 2 : 1;
}
template <int DP>
constexpr int part_bytes() {  // of a stage: 128 rows of up to 128 channels
  return DP / 64 * kSub / halves<DP>();
}
template <int FMT, int DP, bool PAIR>
constexpr int stages_k() {
  return FMT == DT_BF16 && !PAIR ? 3 : 2;
}
template <int FMT, int DP, bool PAIR>
constexpr int stages_v() {
  return DP > 128 ? 2 : stages_k<FMT, DP, PAIR>();
}
template <bool PAIR>
constexpr int raw_stages() {
  return PAIR ? 2 : kRaw;
}
template <int FMT>
constexpr int threads() {  // a multiple of four warps: what a scheduler's share of registers goes by
  return (FMT == DT_BF16 ? kConv0 : kConv0 + kConvWarps) * 32;
}
// MX: a tile as it is stored, 128 rows of codes and of scale words
template <int FMT, int DP>
constexpr int raw_bytes() {
  return FMT == DT_BF16 ? 0 : kPrefixKeys * (DP * (FMT == DT_MXFP8 ? 8 : 4) / 8 + 4);
}

struct PrefixMaps {  // the pools as rows: boxes of a page's rows (p.box); bf16: also of 16 rows
  CUtensorMap k, v, k16, v16;
};

template <bool PAIR>
struct Ctrl {
  uint64_t kfull[kMost], kfree[kMost], vfull[kMost], vfree[kMost];
  uint64_t raw_full[kRaw], raw_free[kRaw];
  uint64_t q_full, q_free, s_full[2], p_full[2], o_full, o_free, ml_full;
  uint32_t tmem;
  int abort;
  float2 ml[PAIR ? 1 : 2][PAIR ? 1 : kPrefixRows];  // of the streams, where they are joined
};

template <int FMT, int DP, bool PAIR>
constexpr int smem_bytes() {
  return DP / 64 * kSub * (PAIR ? 2 : 1) +
         part_bytes<DP>() * (stages_k<FMT, DP, PAIR>() + stages_v<FMT, DP, PAIR>()) +
         raw_stages<PAIR>() * raw_bytes<FMT, DP>() + static_cast<int>(sizeof(Ctrl<PAIR>));
}

// B operand as it lies: 16-bit elements, reduction rows of 128 bytes (64 columns), 8 rows 1024
// bytes apart, the next 64 columns a sub-tile further; 128-byte swizzle.
COLI_DEV uint64_t sw128_desc_mn(uint32_t addr) {
  uint64_t d = static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kSub >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Waits for a phase; gives up, and has the block do so, after about kWaitTimeoutNs. By the SM's
// clock: reading the global timer, as waits of milliseconds may, costs a microsecond.
COLI_DEV bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long begin = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - begin > static_cast<long long>(2 * kWaitTimeoutNs)) {
      *abort = 1;
      return false;
    }
  }
}

// The products, issued by one lane of a converged warp: with the operands in uniform registers an
// instruction takes less to issue than to run (a single lane's code needs 110 cycles an
// instruction to move them there, the product of 128 x 128 x 16 takes 64).
COLI_DEV void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
COLI_DEV void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
COLI_DEV void mma_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
COLI_DEV bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort));
}

COLI_DEV void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

COLI_DEV void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Place of 16-byte chunk c of row r in a tile of 64-channel sub-tiles, 128-byte swizzle.
COLI_DEV uint32_t place(int r, int c) {
  return (c >> 3) * kSub + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

COLI_DEV float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits i: keys 16 i .. of the tile are in sight (lanes 0-7 look their pages up).
COLI_DEV uint32_t groups_in_sight(const PrefixArgs& p, int key0) {
  const int key = key0 + (lane_id() & 7) * 16;
  bool in = key < p.len;
  if (in) {
    const int page = __ldg(p.pages + key / p.c.page_size);
    in = page >= 0 && page < p.c.n_pages;
  }
  return __ballot_sync(0xffffffffu, in) & 0xffu;
}

// A block's pieces: segment by segment along its part of the line.
struct Walk {
  int64_t pos, end;
  int seg, t0, n;
  COLI_DEV Walk(const PrefixArgs& p) {
    pos = blockIdx.x * p.per;
    end = pos + p.per < p.total ? pos + p.per : p.total;
  }
  COLI_DEV bool next(const PrefixArgs& p) {
    if (pos >= end) return false;
    seg = static_cast<int>(pos / p.tiles);
    t0 = static_cast<int>(pos - static_cast<int64_t>(seg) * p.tiles);
    const int64_t left = end - pos;
    n = left < p.tiles - t0 ? static_cast<int>(left) : p.tiles - t0;
    pos += n;
    return true;
  }
};

template <int FMT, int DP, bool PAIR>
__global__ void __launch_bounds__(threads<FMT>(), 1) k_prefix(const PrefixArgs p, const __grid_constant__ PrefixMaps maps) {
  constexpr int kTileBytes = part_bytes<DP>(), kQBytes = DP / 64 * kSub;
  constexpr int kHalves = halves<DP>(), DV = DP / kHalves;  // channels of a stage
  constexpr int kStagesK = stages_k<FMT, DP, PAIR>(), kStagesV = stages_v<FMT, DP, PAIR>();
  constexpr int kRaws = raw_stages<PAIR>();
  constexpr int kQTiles = PAIR ? 2 : 1, kSegRows = kQTiles * kPrefixRows;
  extern __shared__ __align__(1024) char smem_raw[];  // there is no room to align it by hand
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {
    if (threadIdx.x == 0) latch_error(p.status, kErrDevice);
    return;
  }
  const uint32_t s_q = base, s_k = base + kQTiles * kQBytes, s_v = s_k + kStagesK * kTileBytes;
  const uint32_t s_raw = s_v + kStagesV * kTileBytes;
  Ctrl<PAIR>& C = *reinterpret_cast<Ctrl<PAIR>*>(smem_raw + (s_raw - base) +
                                                 kRaws * raw_bytes<FMT, DP>());
  volatile int* abort = &C.abort;
  const int warp = threadIdx.x / 32, lane = lane_id();
  const int D = p.c.head_dim;
  // a segment's key head, row tile and half of the values
  auto head_of = [&](const Walk& w) { return w.seg / (p.row_tiles * kHalves); };
  auto tile_of = [&](const Walk& w) { return w.seg / kHalves % p.row_tiles; };
  auto half_of = [&](const Walk& w) { return w.seg % kHalves; };

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    // TMA: the bytes announced, the edge by hand; MX: the warps that widen
    constexpr int kFull = FMT == DT_BF16 ? 2 : kConvWarps;
    for (int i = 0; i < kRaws; ++i) {
      mbar_init(smem_u32(&C.raw_full[i]), 33);  // the bytes announced, each lane's scales
      mbar_init(smem_u32(&C.raw_free[i]), kConvWarps);
    }
    for (int i = 0; i < kStagesK; ++i) {
      mbar_init(smem_u32(&C.kfull[i]), kFull);
      mbar_init(smem_u32(&C.kfree[i]), 1);
    }
    for (int i = 0; i < kStagesV; ++i) {
      mbar_init(smem_u32(&C.vfull[i]), kFull);
      mbar_init(smem_u32(&C.vfree[i]), 1);
    }
    mbar_init(smem_u32(&C.q_full), kSoftWarps * 32);
    mbar_init(smem_u32(&C.q_free), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&C.s_full[i]), 1);
      mbar_init(smem_u32(&C.p_full[i]), kSoftWarps / 2);
    }
    mbar_init(smem_u32(&C.o_full), 1);
    mbar_init(smem_u32(&C.o_free), kSoftWarps);
    mbar_init(smem_u32(&C.ml_full), kSoftWarps);
    C.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&C.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;

  if (warp < kSoftWarps) {
    // ---- softmax: warpgroup X has stream X, thread (warp % 4, lane) row 32 (warp % 4) + lane
    const int X = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = lanes + X * 128, t_o = lanes + kOCol + X * 128;
    // the sign went into Q; never 0, which times a hidden score's -inf is NaN (2^-149 times any
    // finite score is below 2^-21, which weights do not show)
    const float sl = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 0x1p-149f);
    // the piece's queries: 128 rows by all softmax warps, their sign that of the scale
    auto load_queries = [&](const Walk& w) {
      const int h = head_of(w), r0 = tile_of(w) * kSegRows;
      const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
      constexpr int kQ = kPrefixRows * (DV / 8) / (kSoftWarps * 32);  // loads in flight
#pragma unroll 1
      for (int t = 0; t < kQTiles * kHalves; ++t) {  // a row tile, or half of one
        uint4 v[kQ];
#pragma unroll
        for (int e = 0; e < kQ; ++e) {
          const int i = threadIdx.x + e * kSoftWarps * 32, r = i / (DV / 8);
          const int c = i - r * (DV / 8) + (PAIR ? 0 : t * (DV / 8));
          const int at = r0 + (PAIR ? t * kPrefixRows : 0) + r;
          v[e] = make_uint4(0, 0, 0, 0);
          if (at < p.rows && c * 8 < D) {
            const int b = at / p.group, g = at - b * p.group;
            v[e] = ldg_keep(static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride +
                            static_cast<size_t>(h * p.group + g) * D + c * 8);
          }
        }
#pragma unroll
        for (int e = 0; e < kQ; ++e) {
          const int i = threadIdx.x + e * kSoftWarps * 32, r = i / (DV / 8);
          const int c = i - r * (DV / 8) + (PAIR ? 0 : t * (DV / 8));
          v[e].x ^= flip, v[e].y ^= flip, v[e].z ^= flip, v[e].w ^= flip;
          sts128(s_q + (PAIR ? t * kQBytes : 0) + place(r, c), v[e]);
        }
      }
      proxy_fence();
      mbar_arrive(smem_u32(&C.q_full));
    };
    uint32_t s_phase = 0;
    int piece = 0;
    Walk walk(p), ahead(p);
    if (ahead.next(p)) load_queries(ahead);
    for (; walk.next(p) && !*abort; ++piece) {
      float m = -FLT_MAX, l = 0.f;
      bool ok = true;
      for (int j = PAIR ? 0 : X; j < walk.n; j += PAIR ? 1 : 2) {
        const int key0 = (walk.t0 + j) * kPrefixKeys;
        const uint32_t groups = groups_in_sight(p, key0);
        const bool part = groups != 0xffu || key0 + kPrefixKeys > p.len;
        ok = __all_sync(0xffffffffu, wait_for(smem_u32(&C.s_full[X]), s_phase, abort));
        if (!ok) break;
        s_phase ^= 1u;
        tc_fence_after();
        if (part) {  // scores out of sight: -inf
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(t_s + 32 * c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(groups >> (2 * c + (i >> 4)) & 1u) || key0 + 32 * c + i >= p.len)
                v[i] = 0xff800000u;
            tmem_st32(t_s + 32 * c, v);
          }
          tmem_st_wait();
        }
        // (Loops of 32 keys: unrolled, the roles' code together is more than the instruction
        // caches hold, and every warp waited for instructions.)
        float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(t_s + 32 * c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            tops[i & 1] = max3(tops[i & 1], __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        }
        const float top = fmaxf(tops[0], tops[1]);
        const bool raise = fmaf(top, sl, -m) > 0.f;
        if (__any_sync(0xffffffffu, raise)) {
          const float to = raise ? fmaf(top, sl, 8.f) : m;
          const float f = raise ? ex2(m - to) : 1.f;
          m = to;
          l *= f;
          if (j >= (PAIR ? 1 : 2)) {  // its stream's first product overwrites O
#pragma unroll 1
            for (int c = 0; c < DV / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(t_o + 32 * c, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              tmem_st32(t_o + 32 * c, v);
            }
          }
        }
        const uint64_t sl2 = f32x2(sl, sl), neg_m = f32x2(-m, -m), minus = f32x2(-1.f, -1.f);
        uint64_t l2 = 0;  // of even and odd keys
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(t_s + 32 * c, v);
          // columns 32 c ..: 16 of the weights in bf16, 16 of what the rounding left
          uint32_t o[32];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t y = fma_f32x2(
                f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sl2, neg_m);
            const float x0 = ex2(f32x2_lo(y)), x1 = ex2(f32x2_hi(y));
            const uint64_t x = f32x2(x0, x1);
            l2 = add_f32x2(l2, x);
            const uint32_t h = pack_bf16x2(x0, x1);
            const uint64_t rest = fma_f32x2(f32x2(bf16_lo(h), bf16_hi(h)), minus, x);
            o[i] = h;
            o[16 + i] = pack_bf16x2(f32x2_lo(rest), f32x2_hi(rest));
          }
          tmem_st32(t_s + 32 * c, o);
        }
        l += f32x2_lo(l2) + f32x2_hi(l2);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&C.p_full[X]));
      }
      if (!ok) break;
      // ---- the piece's end: the next one's queries once the last scores are formed, then both
      // streams' means joined, half of the channels each
      if (ahead.next(p)) {
        if (!__all_sync(0xffffffffu, wait_for(smem_u32(&C.q_free), piece & 1, abort))) break;
        load_queries(ahead);
      }
      const int r = tile_of(walk) * kSegRows + (PAIR ? X * kPrefixRows : 0) + row;
      const size_t slot = (static_cast<size_t>(blockIdx.x) + walk.seg) * kSegRows +
                          (PAIR ? X * kPrefixRows : 0) + row;
      float* out = p.mean + slot * D;
      if constexpr (PAIR) {
        // the streams are rows of their own
        if (!warp_wait(smem_u32(&C.o_full), piece & 1, abort)) break;
        tc_fence_after();
        const float by = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(t_o + c * 32, v);
          if (r < p.rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              if (c * 32 + i >= D) break;
              float o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] = l == 0.f ? 0.f : __uint_as_float(v[i + k]) * by;
              *reinterpret_cast<float4*>(out + c * 32 + i) = make_float4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        if (r < p.rows) p.ml[slot] = make_float2(m, l);
      } else {
      // (the piece before has been read out of it, as it has out of O)
      if (!warp_wait(smem_u32(&C.o_free), (piece & 1) ^ 1u, abort)) break;
      C.ml[X][row] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&C.ml_full));
      ok = __all_sync(0xffffffffu, wait_for(smem_u32(&C.ml_full), piece & 1, abort) &&
                                       wait_for(smem_u32(&C.o_full), piece & 1, abort));
      if (!ok) break;
      tc_fence_after();
      const float2 a = C.ml[0][row], b = C.ml[1][row];
      const float mm = fmaxf(a.x, b.x);
      const float wa = a.y * ex2(a.x - mm), wb = b.y * ex2(b.x - mm), sum = wa + wb;
      // sums over their own weights first: means cannot overflow
      const float fa = wa == 0.f ? 0.f : wa / sum, ia = wa == 0.f ? 0.f : 1.f / a.y;
      const float fb = wb == 0.f ? 0.f : wb / sum, ib = wb == 0.f ? 0.f : 1.f / b.y;
#pragma unroll 1
      for (int c = 0; c < DV / 64; ++c) {
        const int col = (X * (DV / 64) + c) * 32, to = half_of(walk) * DV + col;
        uint32_t v[32], u[32];
        tmem_ld32(lanes + kOCol + col, v);
        tmem_ld32(lanes + kOCol + 128 + col, u);
        if (r < p.rows) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            if (to + i >= D) break;
            float o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // a stream without weight may have no sums at all
              const float oa = wa == 0.f ? 0.f : __uint_as_float(v[i + k]) * ia * fa;
              const float ob = wb == 0.f ? 0.f : __uint_as_float(u[i + k]) * ib * fb;
              o[k] = oa + ob;
            }
            *reinterpret_cast<float4*>(out + to + i) = make_float4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      if (X == 0 && r < p.rows) p.ml[slot] = make_float2(mm, sum);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&C.o_free));
    }
  } else if (warp == kMmaWarp) {
    // ---- products
    constexpr uint32_t kIdS = idesc_bf16(kPrefixRows, kPrefixKeys);
    constexpr uint32_t kIdO = idesc_bf16(kPrefixRows, DV) | 1u << 16;  // B as it lies
    int ks = 0, vs = 0, piece = 0;
    uint32_t kp = 0, vp = 0, p_phase = 0;  // bit X: of stream X
    bool ok = true;
    Walk walk(p);
    for (; ok && walk.next(p); ++piece) {
      if (!warp_wait(smem_u32(&C.q_full), piece & 1, abort)) break;
      tc_fence_after();
      // unit u: stream u % 2; its tile is the u-th, or (PAIR) the streams take each in turn
      const int units = PAIR ? 2 * walk.n : walk.n;
      for (int u = 0; u <= units; ++u) {
        if (u < units) {
          const uint32_t q0 = s_q + (PAIR ? (u & 1) * kQBytes : 0);
#pragma unroll
          for (int part = 0; part < kHalves; ++part) {
            if (!PAIR || u % 2 == 0)
              if (!(ok = warp_wait(smem_u32(&C.kfull[ks]), kp, abort))) break;
            tc_fence_after();
            const uint32_t k0 = s_k + ks * kTileBytes;
#pragma unroll
            for (int k = 0; k < DV / 16; ++k) {
              const uint32_t off = k / 4 * kSub + k % 4 * 32;
              mma_ss(tmem + (u & 1) * 128, sw128_desc(q0 + part * kTileBytes + off),
                     sw128_desc(k0 + off), kIdS, part != 0 || k != 0 ? 1u : 0u);
            }
            if (part == kHalves - 1) {
              mma_commit(smem_u32(&C.s_full[u & 1]));
              if (u == units - 1) mma_commit(smem_u32(&C.q_free));
            }
            if (!PAIR || u % 2 == 1) {
              mma_commit(smem_u32(&C.kfree[ks]));
              if (++ks == kStagesK) ks = 0, kp ^= 1u;
            }
          }
          if (!ok) break;
        }
        if (u == 0) continue;
        const int X = (u - 1) & 1;
        // the piece before has been read out of O
        if (u == 1 && !(ok = warp_wait(smem_u32(&C.o_free), (piece & 1) ^ 1u, abort))) break;
        if (!PAIR || X == 0)
          if (!(ok = warp_wait(smem_u32(&C.vfull[vs]), vp, abort))) break;
        if (!(ok = warp_wait(smem_u32(&C.p_full[X]), p_phase >> X & 1u, abort))) break;
        p_phase ^= 1u << X;
        tc_fence_after();
        const uint32_t v0 = s_v + vs * kTileBytes;
#pragma unroll
        for (int k = 0; k < kPrefixKeys / 16; ++k) {
          const uint64_t b = sw128_desc_mn(v0 + k * 16 * 128);
          const uint32_t a = tmem + X * 128 + k / 2 * 32 + k % 2 * 8;
          mma_ts(tmem + kOCol + X * 128, a, b, kIdO, u > 2 || k > 0 ? 1u : 0u);
          mma_ts(tmem + kOCol + X * 128, a + 16, b, kIdO, 1u);
        }
        if (!PAIR || X == 1) {
          mma_commit(smem_u32(&C.vfree[vs]));
          if (++vs == kStagesV) vs = 0, vp ^= 1u;
        }
      }
      if (ok) mma_commit(smem_u32(&C.o_full));
    }
  } else if (warp < kLoad0 + (FMT == DT_BF16 ? 2 : 1)) {
    // ---- loaders
    const int tiles_per_page = p.c.page_size / 16;
    int piece = 0;
    bool ok = true;
    // Pages are looked up for four tiles at once, lane l for their keys 16 l .., a batch ahead:
    // the table's latency is half a tile's time. (Bringing tiles to the L2 ahead as well costs the
    // loaders more than it saves: 128 sequences of 32 heads, 32768 tokens 140 against 127 us.)
    // `cur`: the pool's tiles (16 rows) of the batch at hand, `raw`: the pages of the next.
    constexpr int kBatch = 32 * 16;  // keys
    uint32_t cur = kNone;
    int raw = -1;
    auto page_of = [&](int key) {
      return key < p.len ? __ldg(p.pages + key / p.c.page_size) : INT_MIN;
    };
    auto pool_tile = [&](int h, int key, int page) {
      if (key >= p.len) return kNone;
      if (page < 0 || page >= p.c.n_pages) {
        latch_error(p.status, kErrDevice);
        return kNone;
      }
      return (static_cast<uint32_t>(page) * p.c.n_heads + h) * tiles_per_page +
             key % p.c.page_size / 16;
    };
    auto start = [&](int h, int key0) {
      const int key = key0 + lane * 16;
      const int page = page_of(key);
      raw = page_of(key + kBatch);
      cur = pool_tile(h, key, page);
    };
    auto advance = [&](int h, int key0) {  // to the batch from key0 on
      const int key = key0 + lane * 16;
      cur = pool_tile(h, key, raw);
      raw = page_of(key + kBatch);
    };
    // the row of the pool where lane i's box of tile j starts; past the pool (zeros) for none
    auto box_row = [&](int j, int box) {
      const uint32_t at = __shfl_sync(0xffffffffu, cur, (j & 3) * 8 + (lane * box / 16 & 7));
      return at == kNone ? p.pool_rows : static_cast<int>(at) * 16;
    };
    int stage = 0;
    uint32_t phase = 0;
    Walk walk(p);
    if constexpr (FMT == DT_BF16) {
      // warp 0 of the loaders brings the keys, warp 1 the values, lane i the i-th box of rows
      const bool keys = warp == kLoad0;
      const char* pool = keys ? p.c.k : p.c.v;
      const int parts = keys ? kHalves : 1;
      for (; ok && walk.next(p) && !*abort; ++piece) {
        const int h = head_of(walk);
        start(h, walk.t0 * kPrefixKeys);
        for (int i = 0; i < walk.n * parts; ++i) {
          const int j = keys ? i / kHalves : i;
          const int ch0 = (keys ? i % kHalves : half_of(walk)) * DV;  // first channel
          const int key0 = (walk.t0 + j) * kPrefixKeys;
          if (i > 0 && i % (4 * parts) == 0) advance(h, key0);
          const uint32_t full = smem_u32(keys ? &C.kfull[stage] : &C.vfull[stage]);
          const uint32_t dst = (keys ? s_k : s_v) + stage * kTileBytes;
          ok = warp_wait(smem_u32(keys ? &C.kfree[stage] : &C.vfree[stage]), phase ^ 1u, abort);
          if (!ok) break;
          // a tile that the prefix ends in: boxes of 16 rows, the one it ends in by hand
          const bool part = key0 + kPrefixKeys > p.len;
          const int box = part ? 16 : p.box, edge = part ? (p.len - key0) / 16 : kPrefixKeys;
          const bool by_hand = part && p.len % 16 != 0;
          if (lane == 0)
            mbar_arrive_expect_tx(full, kTileBytes - (by_hand ? DV / 64 * 16 * 128 : 0));
          __syncwarp();
          const CUtensorMap* map = part ? (keys ? &maps.k16 : &maps.v16) : (keys ? &maps.k : &maps.v);
          const int row = box_row(j, box);
          if (lane < kPrefixKeys / box && !(by_hand && lane == edge)) {
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
              tma_load_2d(dst + c * kSub + lane * box * 128, map, full, ch0 + c * 64, row);
          }
          if (by_hand) {
            const uint32_t last = __shfl_sync(0xffffffffu, cur, (j & 3) * 8 + edge);
#pragma unroll 4
            for (int e = lane; e < 16 * (DV / 8); e += 32) {
              const int r = e / (DV / 8), c = e - r * (DV / 8);
              uint4 v = make_uint4(0, 0, 0, 0);
              if (last != kNone && ch0 + c * 8 < D && r < p.len % 16)
                v = ldg_keep(pool + (static_cast<size_t>(last) * 16 + r) * p.c.row_bytes +
                             ch0 * 2 + c * 16);
              sts128(dst + place(edge * 16 + r, c), v);
            }
            proxy_fence();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(full);
          if (++stage == (keys ? kStagesK : kStagesV)) stage = 0, phase ^= 1u;
        }
      }
    } else {
      // codes by TMA, lane i the i-th box; scale words by the lanes
      for (; ok && walk.next(p) && !*abort; ++piece) {
        const int h = head_of(walk);
        start(h, walk.t0 * kPrefixKeys);
        for (int j = 0; ok && j < walk.n; ++j) {
          if (j > 0 && j % 4 == 0) advance(h, (walk.t0 + j) * kPrefixKeys);
          const int row = box_row(j, p.box);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = warp_wait(smem_u32(&C.raw_free[stage]), phase ^ 1u, abort);
            if (!ok) break;
            const uint32_t full = smem_u32(&C.raw_full[stage]);
            const uint32_t dst = s_raw + stage * raw_bytes<FMT, DP>();
            const uint32_t scales = dst + raw_bytes<FMT, DP>() - kPrefixKeys * 4;
            if (lane == 0) mbar_arrive_expect_tx(full, kPrefixKeys * p.c.row_bytes);
            __syncwarp();
            if (lane < kPrefixKeys / p.box)
              tma_load_2d(dst + lane * p.box * p.c.row_bytes, kv ? &maps.v : &maps.k, full, 0, row);
            const uint8_t* sc = kv ? p.c.v_scale : p.c.k_scale;
#pragma unroll
            for (int i = 0; i < kPrefixKeys / 32; ++i) {
              const int r = i * 32 + lane;
              const uint32_t at = __shfl_sync(0xffffffffu, cur, (j & 3) * 8 + r / 16);
              const size_t from = at == kNone ? 0 : static_cast<size_t>(at) * 16 + r % 16;
              paged::cp_async4_n(scales + r * 4, sc + from * 4, at == kNone ? 0 : 4);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full)
                         : "memory");
            if (++stage == kRaws) stage = 0, phase ^= 1u;
          }
        }
      }
      cp_async_wait<0>();
    }
  } else if (warp >= kConv0) {
    if constexpr (FMT != DT_BF16) {
      // ---- codes to bf16: 16 bytes, CH channels, CH / 8 chunks of an operand's row at a time
      constexpr int CH = FMT == DT_MXFP8 ? 16 : 32, kU = DP / CH;
      constexpr int kStep = kConvWarps * 32 / kU, kN = kPrefixKeys / kStep;
      static_assert(kStep % 8 == 0, "rows of a thread share r % 8");
      const int ct = threadIdx.x - kConv0 * 32, u = ct % kU, r0 = ct / kU;
      const bool in_row = u * CH < D;
      // the units of a row's second 64 channels start with their second half: no bank is met
      // twice by the eight lanes that store together
      const bool swap = u * CH >= 64;
      int raw = 0, at[2] = {0, 0};
      uint32_t raw_phase = 0, phases = 0;  // bit 0: of the keys' stages, 1: of the values'
      bool ok = true;
      // where the unit's chunks go in row r0: rows kStep apart keep their swizzle, 8 divides it
      uint32_t to[CH / 8];
#pragma unroll
      for (int k = 0; k < CH / 8; ++k)
        to[k] = place(r0, u * (CH / 8) + (swap ? k ^ (CH / 16) : k));
      const uint32_t from = r0 * p.c.row_bytes + u * 16, half = swap ? 8 : 0;
      const uint32_t scale_at = raw_bytes<FMT, DP>() - kPrefixKeys * 4 + r0 * 4 + u * CH / kMxBlock;
      auto widen = [&](uint32_t dst, uint32_t full, int valid) {
        uint32_t src = s_raw + raw * raw_bytes<FMT, DP>() + from;
        uint32_t sc_src = s_raw + raw * raw_bytes<FMT, DP>() + scale_at;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          uint32_t w[CH / 2];
          uint2 a = make_uint2(0, 0), b = make_uint2(0, 0);
          uint32_t sc = 0;
          if (in_row && r0 + i * kStep < valid) {
            a = lds64(src + half);
            b = lds64(src + 8 - half);
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sc) : "r"(sc_src));
          }
          decode16<FMT>(make_uint4(a.x, a.y, b.x, b.y), sc, w);
#pragma unroll
          for (int k = 0; k < CH / 8; ++k)
            sts128(dst + to[k], make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
          src += kStep * p.c.row_bytes;
          sc_src += kStep * 4;
          dst += kStep * 128;
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full);
          mbar_arrive(smem_u32(&C.raw_free[raw]));
        }
        if (++raw == kRaws) raw = 0, raw_phase ^= 1u;
      };
      Walk walk(p);
      while (ok && walk.next(p) && !*abort) {
#pragma unroll 1
        for (int i = 0; ok && i < 2 * walk.n; ++i) {
          const int kv = i & 1, stage = kv ? at[1] : at[0];
          ok = warp_wait(smem_u32(&C.raw_full[raw]), raw_phase, abort) &&
               warp_wait(smem_u32(kv ? &C.vfree[stage] : &C.kfree[stage]),
                         (phases >> kv & 1u) ^ 1u, abort);
          if (!ok) break;
          widen((kv ? s_v : s_k) + stage * kTileBytes,
                smem_u32(kv ? &C.vfull[stage] : &C.kfull[stage]),
                p.len - (walk.t0 + i / 2) * kPrefixKeys);
          const bool round = stage + 1 == (kv ? kStagesV : kStagesK);
          if (kv)
            at[1] = round ? 0 : stage + 1;
          else
            at[0] = round ? 0 : stage + 1;
          phases ^= (round ? 1u : 0u) << kv;
        }
      }
    }
  }

  __syncthreads();
  if (C.abort && threadIdx.x == 0) {
    latch_error(p.status, kErrTimeout);
    const uint64_t t0 = global_timer_ns();  // let products in flight end
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int FMT, int DP, bool PAIR>
cudaError_t launch(const PrefixArgs& p, int grid, cudaStream_t st) {
  static bool ready[128] = {};
  cudaError_t e = raise_shared(k_prefix<FMT, DP, PAIR>, smem_bytes<FMT, DP, PAIR>(), ready);
  if (e != cudaSuccess) return e;
  PrefixMaps maps{};
  auto encode = [&](CUtensorMap* m, const void* pool, int rows) {
    if (e != cudaSuccess) return;
    if (FMT == DT_BF16)
      e = encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, p.pool_rows, p.c.head_dim,
                         64, rows, CU_TENSOR_MAP_SWIZZLE_128B);
    else
      e = encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, pool, p.pool_rows, p.c.row_bytes,
                         p.c.row_bytes, rows, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  encode(&maps.k, p.c.k, p.box);
  encode(&maps.v, p.c.v, p.box);
  if (FMT == DT_BF16) {
    encode(&maps.k16, p.c.k, 16);
    encode(&maps.v16, p.c.v, 16);
  }
  if (e != cudaSuccess) return e;
  k_prefix<FMT, DP, PAIR><<<grid, threads<FMT>(), smem_bytes<FMT, DP, PAIR>(), st>>>(p, maps);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_heads(const PrefixArgs& p, int grid, cudaStream_t st) {
  if constexpr (FMT == DT_BF16)
    if (p.c.head_dim > 128) return launch<FMT, 256, false>(p, grid, st);
  if (p.pair) {
    if constexpr (FMT != DT_BF16)  // (bf16 heads to 64 are never paired)
      if (p.c.head_dim <= 64) return launch<FMT, 64, true>(p, grid, st);
    return launch<FMT, 128, true>(p, grid, st);
  }
  return p.c.head_dim <= 64 ? launch<FMT, 64, false>(p, grid, st)
                            : launch<FMT, 128, false>(p, grid, st);
}

}  // namespace

cudaError_t launch_prefix(const PrefixArgs& p, int grid, cudaStream_t st) {
  switch (p.c.dtype) {
    case DT_BF16: return launch_heads<DT_BF16>(p, grid, st);
    case DT_MXFP8: return launch_heads<DT_MXFP8>(p, grid, st);
    default: return launch_heads<DT_MXFP4>(p, grid, st);
  }
}

}  // namespace coli
