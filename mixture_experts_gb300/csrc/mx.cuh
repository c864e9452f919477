// Microscaling blocks in registers: 32 elements under one E8M0 scale byte,
// quantised and decoded by the lanes that hold them.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace coli {

// 2^(s - 127); byte 255 is NaN, byte 0 the subnormal 2^-127.
COLI_DEV float e8m0_f32(uint32_t s) {
  const uint32_t bits = s == 255u ? 0x7fc00000u : (s == 0u ? 0x00400000u : s << 23);
  return __uint_as_float(bits);
}

// The scale byte of a block whose largest magnitude has the fp32 bits `amax`,
// and the factor 2^-(exponent) its elements are multiplied by (exact: the
// exponent is at most 127 - emax). A NaN or infinity in the block (amax bits
// from 0x7f800000 on) gives byte 255 and factor 0.
template <int EMAX>
COLI_DEV uint32_t mx_scale(uint32_t amax, float* inv) {
  if (amax >= 0x7f800000u) {
    *inv = 0.f;
    return 255u;
  }
  int ex = amax == 0u ? 0 : static_cast<int>(amax >> 23) - 127 - EMAX;
  ex = ex < -127 ? -127 : ex;
  *inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
  return static_cast<uint32_t>(ex + 127);
}

// 8 fp32 values -> 8 E4M3 bytes / 8 E2M1 nibbles (element 0 lowest), round to
// nearest even, saturated.
COLI_DEV uint2 pack_e4m3x8(const float (&x)[8]) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 c, %7, %6;\n\tcvt.rn.satfinite.e4m3x2.f32 d, %9, %8;\n\t"
      "mov.b32 %0, {a, b};\n\tmov.b32 %1, {c, d};\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

COLI_DEV uint2 pack_e5m2x8(const float (&x)[8]) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 a, %3, %2;\n\tcvt.rn.satfinite.e5m2x2.f32 b, %5, %4;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 c, %7, %6;\n\tcvt.rn.satfinite.e5m2x2.f32 d, %9, %8;\n\t"
      "mov.b32 %0, {a, b};\n\tmov.b32 %1, {c, d};\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

COLI_DEV uint32_t pack_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// fp16 pairs -> fp32 (exact).
COLI_DEV void f16x8_f32(const uint32_t (&h)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
        : "r"(h[i]));
  }
}

// ---- stored rows to bf16 pairs, for products and comparisons in bf16 ------------
// 8 codes (MXFP8: both words, MXFP4: w0) times their scale, element 0 lowest: exact in bf16
// within its range (fp32's) and rounded once to it beyond, as the cache's read rounds them.
// Through fp32: the fp16 forms' bits moved to bf16's places and multiplied there take fewer
// steps, but of the integer pipe, which is what such kernels run out of (bounds of 4099 pages
// 78 against 65 us), and no NaN codes.
template <int FMT>
COLI_DEV void mx8_bf16(uint32_t w0, uint32_t w1, float scale, uint32_t (&o)[4]) {
  uint32_t h[4];
  float x[8];
  if constexpr (FMT == DT_MXFP8)
    e4m3x8_f16(w0, w1, h);
  else
    e2m1x8_f16(w0, h);
  f16x8_f32(h, x);
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(x[2 * k] * scale, x[2 * k + 1] * scale);
}

// Words that 16 stored bytes make: bf16 pairs, or fp32 as it is.
template <int FMT>
constexpr int words16() {
  return FMT == DT_MXFP8 ? 8 : (FMT == DT_MXFP4 ? 16 : 4);
}
template <int FMT>
COLI_DEV void decode16(const uint4& raw, uint32_t scale, uint32_t (&w)[words16<FMT>()]) {
  if constexpr (FMT == DT_F32 || FMT == DT_BF16) {
    w[0] = raw.x, w[1] = raw.y, w[2] = raw.z, w[3] = raw.w;
  } else {
    const float f = e8m0_f32(scale);
#pragma unroll
    for (int i = 0; i < words16<FMT>() / 4; ++i) {
      uint32_t o[4];
      if constexpr (FMT == DT_MXFP8)
        mx8_bf16<FMT>(word_of(raw, 2 * i), word_of(raw, 2 * i + 1), f, o);
      else
        mx8_bf16<FMT>(word_of(raw, i), 0, f, o);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = o[k];
    }
  }
}

// Number of the row (page, head, offset in the page) in a pool.
COLI_DEV size_t kv_row(const KvView& c, int page, int head, int off) {
  return (static_cast<size_t>(page) * c.n_heads + head) * c.page_size + off;
}

}  // namespace coli
