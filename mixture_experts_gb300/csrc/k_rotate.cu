// Rotary positions and the write into the paged key-value cache.
//
// The rotation turns pairs of a head's elements by the token's angles:
// (a, b) -> (a c - b s, b c + a s). Both products and their sum are rounded
// separately in fp32 (no fused multiply-add), so the result does not depend
// on how a caller's own fp32 check is compiled, and an MX block's scale and
// codes follow from it bit for bit.
//
// One thread holds 16 bytes of one head row and reads the pair partners it
// needs from the same row (the other half of the head, in L1); a row's threads
// are in one block, which reads all its rows before it stores any, so q_out may
// be q. The token's cosines and sines stay in registers over HPT heads.
#include "attn.h"
#include "common.cuh"
#include "mx.cuh"

namespace coli {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsOnly = -1;  // no cache: both outputs are rows

struct RotateArgs {
  HeadRows q, k, v;
  RotaryView r;
  KvView c;
  const int32_t* slots;
  int T, head_dim, heads;  // heads: q + k (+ v)
  int groups;              // threads' heads: n * groups + g
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

template <typename A, int FMT, bool INTER, int HPT>
__global__ void __launch_bounds__(kThreads) k_rotate(const RotateArgs p) {
  constexpr int N = Chunk<A>::N;
  const int cpr = p.head_dim / N;        // chunks (threads) per row
  const int rows = kThreads / cpr;       // rows a block holds at once
  const int local = threadIdx.x / cpr, c = threadIdx.x % cpr;
  const uint32_t slot_id = blockIdx.x * static_cast<uint32_t>(rows) + local;
  const uint32_t t = slot_id / p.groups;
  const int g = slot_id % p.groups;
  const bool live = local < rows && t < static_cast<uint32_t>(p.T);
  const int d0 = c * N, half = p.r.rot_dim / 2;

  bool turn = live && p.r.table != nullptr && d0 < p.r.rot_dim, bad_pos = false;
  int pos = 0;
  if (live && p.r.table != nullptr) {
    pos = p.r.positions[t];
    bad_pos = static_cast<uint32_t>(pos) >= static_cast<uint32_t>(p.r.n_positions);
    if (bad_pos) {
      turn = false;
      if (c == 0 && g == 0) latch_error(p.status, kErrDevice);
    }
  }
  // the cosine and signed sine of each element's pair; (1, 0) past rot_dim
  float cs[N], sn[N];
#pragma unroll
  for (int i = 0; i < N; ++i) cs[i] = 1.f, sn[i] = 0.f;
  const bool aligned = half % N == 0;  // partner chunk and table rows are whole vectors
  if (turn) {
    const float2* row = reinterpret_cast<const float2*>(p.r.table) + static_cast<size_t>(pos) * half;
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (d0 + 2 * i < p.r.rot_dim) {
          const float2 v = __ldg(row + d0 / 2 + i);
          cs[2 * i] = cs[2 * i + 1] = v.x;
          sn[2 * i + 1] = v.y * p.r.sine_sign;
          sn[2 * i] = -sn[2 * i + 1];
        }
      }
    } else if (aligned) {
      const int i0 = d0 < half ? d0 : d0 - half;
      const float sgn = d0 < half ? -p.r.sine_sign : p.r.sine_sign;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
        cs[i] = v.x, sn[i] = v.y * sgn, cs[i + 1] = v.z, sn[i + 1] = v.w * sgn;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int d = d0 + i;
        if (d < p.r.rot_dim) {
          const float2 v = __ldg(row + (d < half ? d : d - half));
          cs[i] = v.x;
          sn[i] = v.y * (d < half ? -p.r.sine_sign : p.r.sine_sign);
        }
      }
    }
  }
  // where the keys and values go
  int page = 0, off = 0;
  bool store = false;
  if constexpr (FMT != kRowsOnly) {
    if (live) {
      const int slot = p.slots[t];
      const bool bad = slot < -1 || slot >= p.c.n_pages * p.c.page_size;
      if (bad && c == 0 && g == 0) latch_error(p.status, kErrDevice);
      store = slot >= 0 && !bad && !bad_pos;
      page = store ? slot / p.c.page_size : 0;
      off = store ? slot - page * p.c.page_size : 0;
    }
  }

  uint4 own[HPT], other[HPT];
  const int hq = p.q.n_heads, hk = hq + p.k.n_heads;
#pragma unroll
  for (int n = 0; n < HPT; ++n) {
    const int h = n * p.groups + g;
    if (!live || h >= p.heads) continue;
    const HeadRows& src = h < hq ? p.q : (h < hk ? p.k : p.v);
    const int hh = h < hq ? h : (h < hk ? h - hq : h - hk);
    const A* row = static_cast<const A*>(src.in) + t * src.in_stride +
                   static_cast<size_t>(hh) * p.head_dim;
    own[n] = *reinterpret_cast<const uint4*>(row + d0);
    if constexpr (!INTER) {
      if (turn && h < hk) {
        if (aligned) {
          other[n] = *reinterpret_cast<const uint4*>(row + (d0 < half ? d0 + half : d0 - half));
        } else {
          A e[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int d = d0 + i;
            e[i] = row[d >= p.r.rot_dim ? d : (d < half ? d + half : d - half)];
          }
          other[n] = *reinterpret_cast<const uint4*>(e);
        }
      }
    }
  }
  __syncthreads();  // q_out may be q: every row is read before any is stored
#pragma unroll
  for (int n = 0; n < HPT; ++n) {
    const int h = n * p.groups + g;
    const bool here = live && h < p.heads;
    float x[N];
    if (here) {
      unpack<A>(own[n], x);
      if (turn && h < hk) {
        float y[N];
        if constexpr (INTER) {
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] = x[i ^ 1];
        } else {
          unpack<A>(other[n], y);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          // elements past rot_dim keep their value (and their sign of zero)
          if (d0 + i < p.r.rot_dim)
            x[i] = __fadd_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(y[i], sn[i]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = 0.f;
    }
    if (here && (FMT == kRowsOnly || h < hq)) {
      const HeadRows& dst = h < hq ? p.q : p.k;
      const int hh = h < hq ? h : h - hq;
      A* row = static_cast<A*>(dst.out) + t * dst.out_stride + static_cast<size_t>(hh) * p.head_dim;
      *reinterpret_cast<uint4*>(row + d0) = pack<A>(x);
    }
    if constexpr (FMT != kRowsOnly) {
      const bool is_k = h < hk;
      const bool put = here && h >= hq && store;
      const size_t row = put ? kv_row(p.c, page, is_k ? h - hq : h - hk, off) : 0;
      char* dst = (is_k ? p.c.k : p.c.v) + row * p.c.row_bytes;
      if constexpr (FMT == DT_F32 || FMT == DT_BF16) {
        if (put) *reinterpret_cast<uint4*>(dst + c * 16) = pack<A>(x);
      } else {
        // a block's 32 elements are in four neighbouring lanes
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float inv;
        const uint32_t s = mx_scale<FMT == DT_MXFP8 ? 8 : 2>(amax, &inv);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = inv == 0.f ? 0.f : x[i] * inv;
        if (put) {
          if constexpr (FMT == DT_MXFP8)
            *reinterpret_cast<uint2*>(dst + c * 8) = pack_e4m3x8(x);
          else
            *reinterpret_cast<uint32_t*>(dst + c * 4) = pack_e2m1x8(x);
          if (c % 4 == 0)
            (is_k ? p.c.k_scale : p.c.v_scale)[row * p.c.scale_stride + c / 4] =
                static_cast<uint8_t>(s);
        }
      }
    }
  }
}

template <typename A, int FMT, bool INTER>
cudaError_t launch_hpt(RotateArgs& p, cudaStream_t st) {
  const int rows = kThreads / (p.head_dim / Chunk<A>::N);
  // few rows: one head a thread, for the shortest chain of loads; many: four
  // heads a thread share the token's table row
  const int hpt = static_cast<int64_t>(p.T) * p.heads <= 152 * 8 * rows ? 1 : 4;
  p.groups = (p.heads + hpt - 1) / hpt;
  const int64_t slots = static_cast<int64_t>(p.T) * p.groups;
  const int64_t blocks = (slots + rows - 1) / rows;
  if (slots + rows > INT32_MAX) return cudaErrorInvalidValue;
  if (hpt == 1)
    k_rotate<A, FMT, INTER, 1><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
  else
    k_rotate<A, FMT, INTER, 4><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename A, int FMT>
cudaError_t launch_layout(RotateArgs& p, cudaStream_t st) {
  return p.r.interleaved ? launch_hpt<A, FMT, true>(p, st) : launch_hpt<A, FMT, false>(p, st);
}

// w_i evaluated per entry in fp64: one table serves every layer and step of a
// run, so the 2 fp64 transcendentals an entry costs are paid once.
__global__ void k_rope_table(RopeFreq f, int half, int n, float2* __restrict__ table) {
  const uint32_t e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= static_cast<uint32_t>(n) * half) return;
  const int pos = e / half, i = e % half;
  double w = pow(f.base, -static_cast<double>(i) / half);
  if (f.scaling == 1) w /= f.factor;
  if (f.scaling == 3) {
    double keep = (f.turns_per_w * w - f.beta_slow) / f.beta_span;
    keep = fmin(fmax(keep, 0.0), 1.0);
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
  p.q = q;
  p.k = k;
  p.r = r;
  p.T = T;
  p.head_dim = head_dim;
  p.heads = q.n_heads + k.n_heads;
  p.status = status;
  return act == DT_F32 ? launch_layout<float, kRowsOnly>(p, st)
                       : launch_layout<__nv_bfloat16, kRowsOnly>(p, st);
}

cudaError_t launch_kv_append(const KvView& c, const HeadRows& q, const HeadRows& k,
                             const HeadRows& v, const RotaryView& r, const int32_t* slots, int T,
                             int* status, cudaStream_t st) {
  RotateArgs p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.r = r;
  p.c = c;
  p.slots = slots;
  p.T = T;
  p.head_dim = c.head_dim;
  p.heads = q.n_heads + 2 * c.n_heads;
  p.status = status;
  switch (c.dtype) {
    case DT_F32: return launch_layout<float, DT_F32>(p, st);
    case DT_BF16: return launch_layout<__nv_bfloat16, DT_BF16>(p, st);
    case DT_MXFP8: return launch_layout<__nv_bfloat16, DT_MXFP8>(p, st);
    default: return launch_layout<__nv_bfloat16, DT_MXFP4>(p, st);
  }
}

}  // namespace coli
