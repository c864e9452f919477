// Rotary positions and the write into the paged key-value cache.
//
// The rotation turns pairs of a head's elements by the token's angles:
// (a, b) -> (a c - b s, b c + a s). Both products and their sum are rounded
// separately in fp32 (no fused multiply-add), so the result does not depend
// on how a caller's own fp32 check is compiled, and an MX block's scale and
// codes follow from it bit for bit.
//
// A row's threads are in one block, which reads all its rows before it stores
// any, so q_out may be q. A thread takes HPT heads of its token, whose loads it
// has in flight together, and keeps the token's cosines and sines in registers
// over them. Three ways to share a row among threads:
//   kInter  16 bytes a thread (pairs are neighbours);
//   kPair   16 bytes of the first half and their partners in the second, where
//           both are whole vectors (and, for an MX cache, whole blocks lie in
//           four neighbouring lanes);
//   kHalf   16 bytes a thread, partners read one by one: any other rot_dim (16384
//           tokens of 40 heads of 80, a quarter rotated: 90.1 us for 211 MB).
// A block holds rows of q, of k or of v only, so what it does with them is known
// to all its threads.
//
// What bounds it: HBM for prompts (16384 tokens of 32 + 8 heads of 128: rotation
// 340 MB in 55.6 us, 6.1 TB/s; rotated and stored as MXFP8 379 MB in 68.3 us,
// 5.5 TB/s, where the quantiser's shuffles and conversions also show); the chain
// position -> table row -> store for a decode batch (32 tokens: 4 us).
#include "../../include/coli_moe.h"
#include "attn.h"
#include "common.cuh"
#include "mx.cuh"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsOnly = -1;  // no cache: both outputs are rows
enum { kInter = 0, kPair = 1, kHalf = 2 };

struct RotateArgs {
  HeadRows rows[3];     // q, k, v
  RotaryView r;
  KvView c;
  const int32_t* slots;
  int T, head_dim;
  int groups[3];        // threads' heads of each kind: n * groups + g, n < HPT
  unsigned blocks[3];   // as many of k as of v, or none of v
  int page_shift;       // log2(page_size), or -1
  int* status;
};

template <typename A>
struct Chunk {
  static constexpr int N = 16 / sizeof(A);
};

template <typename A>
COLI_DEV void unpack(const uint4& u, float (&x)[Chunk<A>::N]) {
  if constexpr (sizeof(A) == 4) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  } else {
    x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x);
    x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z);
    x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
  }
}

template <typename A>
COLI_DEV uint4 pack(const float (&x)[Chunk<A>::N]) {
  if constexpr (sizeof(A) == 4) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  } else {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
}

// 16 bytes that this kernel touches once (evict-first).
COLI_DEV uint4 ld_once(const void* p) { return __ldcs(static_cast<const uint4*>(p)); }
COLI_DEV void st_once(void* p, const uint4& v) { __stcs(static_cast<uint4*>(p), v); }

// max(|a|, |b|), NaN if either is (the sign is not used).
COLI_DEV float max_abs(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// One block's rows of kind KIND (0 q, 1 k, 2 v).
template <typename A, int FMT, int MODE, int HPT, int KIND>
COLI_DEV void rotate_rows(const RotateArgs& p, unsigned block) {
  constexpr int N = Chunk<A>::N, CH = MODE == kPair ? 2 : 1;
  constexpr bool kStore = FMT != kRowsOnly && KIND > 0;  // rows go to the cache
  constexpr bool kMx = kStore && (FMT == DT_MXFP8 || FMT == DT_MXFP4);
  const int tpr = p.head_dim / (N * CH);  // threads per row
  const int rows = kThreads / tpr;        // rows a block holds at once
  const int local = threadIdx.x / tpr, u = threadIdx.x - local * tpr;
  const int groups = p.groups[KIND];
  const uint32_t id = block * static_cast<uint32_t>(rows) + local;
  const uint32_t t = id / groups;
  const int g = id - t * groups;
  const bool live = local < rows && t < static_cast<uint32_t>(p.T);
  const HeadRows& hr = p.rows[KIND];
  const int rot = p.r.rot_dim, half = rot / 2;
  // elements from d0 on, and `apart` further (kPair: partners, or two pieces past rot_dim)
  int d0 = u * N, apart = 0;
  if constexpr (MODE == kPair) {
    const bool in = d0 < half;
    d0 = in ? d0 : d0 + half;
    apart = in ? half : (p.head_dim - rot) / 2;
  }
  const int n_in = live ? (hr.n_heads - g + groups - 1) / groups : 0;  // heads of this thread
  const int step = groups * p.head_dim;  // elements between them

  const A* src = static_cast<const A*>(hr.in) + (live ? t * hr.in_stride : 0) + g * p.head_dim + d0;
  uint4 own[HPT][CH];
#pragma unroll
  for (int n = 0; n < HPT; ++n)
    if (n < n_in) {
      own[n][0] = ld_once(src + n * step);
      if constexpr (CH == 2) own[n][1] = ld_once(src + n * step + apart);
    }

  // the cosine and sine of each pair; kHalf: of each element's, signed
  constexpr int kAngles = MODE == kInter ? N / 2 : N;
  float cs[kAngles], sn[kAngles];
  uint4 other[MODE == kHalf ? HPT : 1];
  bool turn = false, bad_pos = false;
  if (KIND < 2 && live && p.r.table != nullptr) {
    const int pos = p.r.positions[t];
    bad_pos = static_cast<uint32_t>(pos) >= static_cast<uint32_t>(p.r.n_positions);
    if (bad_pos && u == 0 && g == 0) latch_error(p.status, kErrDevice);
    turn = !bad_pos && d0 < rot;
    if (turn) {
      const float2* row =
          reinterpret_cast<const float2*>(p.r.table) + static_cast<size_t>(pos) * half;
      if constexpr (MODE == kInter) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 v = d0 + 2 * i < rot ? __ldg(row + d0 / 2 + i) : make_float2(1, 0);
          cs[i] = v.x, sn[i] = v.y * p.r.sine_sign;
        }
      } else if constexpr (MODE == kPair) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(row + d0 + i));
          cs[i] = v.x, sn[i] = v.y * p.r.sine_sign;
          cs[i + 1] = v.z, sn[i + 1] = v.w * p.r.sine_sign;
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int d = d0 + i;
          const float2 v = d < rot ? __ldg(row + (d < half ? d : d - half)) : make_float2(1, 0);
          cs[i] = v.x;
          sn[i] = v.y * (d < half ? -p.r.sine_sign : p.r.sine_sign);
        }
#pragma unroll
        for (int n = 0; n < HPT; ++n) {
          if (n >= n_in) continue;
          A e[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int d = d0 + i;
            e[i] = src[n * step + i + (d >= rot ? 0 : (d < half ? half : -half))];
          }
          other[n] = *reinterpret_cast<const uint4*>(e);
        }
      }
    }
  }
  // where the rows go
  A* dst = nullptr;
  size_t row = 0;
  bool put = live;
  if constexpr (!kStore) {
    dst = static_cast<A*>(hr.out) + (live ? t * hr.out_stride : 0) + g * p.head_dim + d0;
  } else if (live) {
    const int slot = p.slots[t];
    const bool bad = slot < -1 || slot >= p.c.n_pages * p.c.page_size;
    if (bad && u == 0 && g == 0) latch_error(p.status, kErrDevice);
    if (KIND == 2 && p.r.table != nullptr)
      bad_pos = static_cast<uint32_t>(p.r.positions[t]) >= static_cast<uint32_t>(p.r.n_positions);
    put = slot >= 0 && !bad && !bad_pos;
    const int page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.c.page_size;
    if (put) row = kv_row(p.c, page, g, slot - page * p.c.page_size);
  }
  if constexpr (!kStore) __syncthreads();  // q_out may be q: all rows are read before any is stored
  const int row_step = groups * p.c.page_size;
#pragma unroll
  for (int n = 0; n < HPT; ++n) {
    float x[CH][N];
    if (n < n_in) {
#pragma unroll
      for (int k = 0; k < CH; ++k) unpack<A>(own[n][k], x[k]);
      if (turn) {
        if constexpr (MODE == kPair) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float a = x[0][i], b = x[CH - 1][i];
            x[0][i] = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(b, sn[i]));
            x[CH - 1][i] = __fadd_rn(__fmul_rn(b, cs[i]), __fmul_rn(a, sn[i]));
          }
        } else {
          float v[N];
          if constexpr (MODE == kInter) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
              const float a = x[0][2 * i], b = x[0][2 * i + 1];
              v[2 * i] = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(b, sn[i]));
              v[2 * i + 1] = __fadd_rn(__fmul_rn(b, cs[i]), __fmul_rn(a, sn[i]));
            }
          } else {
            unpack<A>(other[n], v);
#pragma unroll
            for (int i = 0; i < N; ++i)
              v[i] = __fadd_rn(__fmul_rn(x[0][i], cs[i]), __fmul_rn(v[i], sn[i]));
          }
          if (d0 + N <= rot) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[0][i] = v[i];
          } else {  // elements past rot_dim keep their bits
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (d0 + i < rot) x[0][i] = v[i];
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) x[k][i] = 0.f;
    }
    if constexpr (!kStore) {
      if (n < n_in) {
        st_once(dst + n * step, pack<A>(x[0]));
        if constexpr (CH == 2) st_once(dst + n * step + apart, pack<A>(x[CH - 1]));
      }
    } else {
      const size_t r = row + static_cast<size_t>(n) * row_step;
      char* to = (KIND == 1 ? p.c.k : p.c.v) + r * p.c.row_bytes;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (d0 + k * apart) / N;  // piece of the row
        if constexpr (!kMx) {
          if (n < n_in && put) *reinterpret_cast<uint4*>(to + c * 16) = pack<A>(x[k]);
        } else {
          // a block's 32 elements are in four neighbouring lanes
          float top = max_abs(max_abs(max_abs(x[k][0], x[k][1]), max_abs(x[k][2], x[k][3])),
                              max_abs(max_abs(x[k][4], x[k][5]), max_abs(x[k][6], x[k][7])));
          top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const uint32_t amax = __float_as_uint(top) & 0x7fffffffu;
          float inv;
          const uint32_t s = mx_scale<FMT == DT_MXFP8 ? 8 : 2>(amax, &inv);
#pragma unroll
          for (int i = 0; i < N; ++i) x[k][i] *= inv;
          if (n < n_in && put) {
            if constexpr (FMT == DT_MXFP8) {
              const uint2 code = pack_e4m3x8(x[k]);
              *reinterpret_cast<uint2*>(to + c * 8) = s == 255u ? make_uint2(0, 0) : code;
            } else {
              const uint32_t code = pack_e2m1x8(x[k]);
              *reinterpret_cast<uint32_t*>(to + c * 4) = s == 255u ? 0u : code;
            }
            if (c % 4 == 0)
              (KIND == 1 ? p.c.k_scale : p.c.v_scale)[r * p.c.scale_stride + c / 4] =
                  static_cast<uint8_t>(s);
          }
        }
      }
    }
  }
}

template <typename A, int FMT, int MODE, int HPT>
__global__ void __launch_bounds__(kThreads, HPT > 1 && MODE != kHalf ? 4 : 1)
    k_rotate(const RotateArgs p) {
  if constexpr (FMT == kRowsOnly) {
    if (blockIdx.x < p.blocks[0])
      rotate_rows<A, FMT, MODE, HPT, 0>(p, blockIdx.x);
    else
      rotate_rows<A, FMT, MODE, HPT, 1>(p, blockIdx.x - p.blocks[0]);
  } else {
    // the blocks of k and v, with the quantiser's work, lie evenly among q's
    const uint64_t i = blockIdx.x, others = p.blocks[1] + p.blocks[2], all = p.blocks[0] + others;
    const unsigned j = static_cast<unsigned>(i * others / all);
    if (j == static_cast<unsigned>((i + 1) * others / all))
      rotate_rows<A, FMT, MODE, HPT, 0>(p, blockIdx.x - j);
    else if (j % 2 == 0)
      rotate_rows<A, FMT, MODE, HPT, 1>(p, j / 2);
    else
      rotate_rows<A, FMT, MODE, HPT, 2>(p, j / 2);
  }
}

template <typename A, int FMT, int MODE>
cudaError_t launch_hpt(RotateArgs& p, cudaStream_t st) {
  constexpr int CH = MODE == kPair ? 2 : 1;
  // measured at 16384 tokens of 40 (stored: 48) heads of 128, us: pairs rotated and
  // stored as MXFP8 2 / 3 / 4 heads a thread 75.4 / 71.6 / 67.8, neighbours 4 / 6 / 8
  // heads 77.4 / 75.8 / 67.3. All with 4 blocks an SM, for which some spill a few
  // registers; without spills at 3 blocks pairs take 69.4 and neighbours 73.4
  constexpr int kMany = MODE == kInter ? 8 : 4;
  const int rows = kThreads / (p.head_dim / (Chunk<A>::N * CH));
  int heads = 0;
  for (const HeadRows& h : p.rows) heads += h.n_heads;
  // few rows: one head a thread, for the shortest chain of loads; many: the
  // heads of a thread share the token's table row
  const int hpt = static_cast<int64_t>(p.T) * heads <= 152 * 8 * rows ? 1 : kMany;
  int64_t blocks = 0;
  for (int k = 0; k < 3; ++k) {
    p.groups[k] = (p.rows[k].n_heads + hpt - 1) / hpt;
    const int64_t ids = static_cast<int64_t>(p.T) * p.groups[k];
    if (ids + rows > INT32_MAX) return cudaErrorInvalidValue;
    p.blocks[k] = static_cast<unsigned>((ids + rows - 1) / rows);
    if (p.groups[k] == 0) p.groups[k] = 1, p.blocks[k] = 0;  // no heads: no blocks
    blocks += p.blocks[k];
  }
  p.page_shift = -1;
  for (int i = 0; i < 13; ++i)
    if (p.c.page_size == 1 << i) p.page_shift = i;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (hpt == 1)
    k_rotate<A, FMT, MODE, 1><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
  else
    k_rotate<A, FMT, MODE, kMany><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename A, int FMT>
cudaError_t launch_layout(RotateArgs& p, cudaStream_t st) {
  constexpr bool kMx = FMT == DT_MXFP8 || FMT == DT_MXFP4;
  constexpr int kUnit = kMx ? kMxBlock : Chunk<A>::N;
  if (p.r.interleaved) return launch_hpt<A, FMT, kInter>(p, st);
  // without a rotation any split in two will do: rot_dim is 0 then
  const int half = p.r.rot_dim / 2, rest = p.head_dim - p.r.rot_dim;
  if (half % kUnit == 0 && rest % (2 * kUnit) == 0) return launch_hpt<A, FMT, kPair>(p, st);
  return launch_hpt<A, FMT, kHalf>(p, st);
}

// w_i evaluated per entry in fp64: one table serves every layer and step of a
// run, so the 2 fp64 transcendentals an entry costs are paid once.
__global__ void k_rope_table(RopeFreq f, int half, int n, float2* __restrict__ table) {
  const uint32_t e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= static_cast<uint32_t>(n) * half) return;
  const int pos = e / half, i = e % half;
  double w = pow(f.base, -static_cast<double>(i) / half);
  if (f.scaling == COLI_ROPE_LINEAR) w /= f.factor;
  if (f.scaling == COLI_ROPE_YARN || f.scaling == COLI_ROPE_YARN_INDEX) {
    const bool by_index = f.scaling == COLI_ROPE_YARN_INDEX;
    double keep = ((by_index ? i : f.turns_per_w * w) - f.ramp_from) / f.ramp_span;
    keep = fmin(fmax(keep, 0.0), 1.0);
    if (by_index) keep = 1.0 - keep;
    w = w * keep + w / f.factor * (1.0 - keep);
  }
  double s, c;
  sincos(pos * w, &s, &c);
  table[e] = make_float2(static_cast<float>(c * f.amplitude), static_cast<float>(s * f.amplitude));
}

}  // namespace

cudaError_t launch_rope_table(const RopeFreq& f, int rot_dim, int n_positions, float* table,
                              cudaStream_t st) {
  const int half = rot_dim / 2;
  const uint32_t n = static_cast<uint32_t>(n_positions) * half;
  k_rope_table<<<(n + 255) / 256, 256, 0, st>>>(f, half, n_positions,
                                                reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

cudaError_t launch_rotate(const HeadRows& q, const HeadRows& k, const RotaryView& r, int T,
                          int head_dim, int act, int* status, cudaStream_t st) {
  RotateArgs p{};
  p.rows[0] = q;
  p.rows[1] = k;
  p.r = r;
  p.T = T;
  p.head_dim = head_dim;
  p.status = status;
  return act == DT_F32 ? launch_layout<float, kRowsOnly>(p, st)
                       : launch_layout<__nv_bfloat16, kRowsOnly>(p, st);
}

cudaError_t launch_kv_append(const KvView& c, const HeadRows& q, const HeadRows& k,
                             const HeadRows& v, const RotaryView& r, const int32_t* slots, int T,
                             int* status, cudaStream_t st) {
  RotateArgs p{};
  p.rows[0] = q;
  p.rows[1] = k;
  p.rows[2] = v;
  p.r = r;
  p.c = c;
  p.slots = slots;
  p.T = T;
  p.head_dim = c.head_dim;
  p.status = status;
  switch (c.dtype) {
    case DT_F32: return launch_layout<float, DT_F32>(p, st);
    case DT_BF16: return launch_layout<__nv_bfloat16, DT_BF16>(p, st);
    case DT_MXFP8: return launch_layout<__nv_bfloat16, DT_MXFP8>(p, st);
    default: return launch_layout<__nv_bfloat16, DT_MXFP4>(p, st);
  }
}

}  // namespace coli
