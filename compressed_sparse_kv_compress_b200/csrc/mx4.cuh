// MXFP4 vectors and 4-bit main-KV rows (OCP microscaling formats).
//
// [SW] shareware.cn/news/167317 §六.1 / §十三.4: the indexer's QK path may run in FP4, the main KV
// in few bits, while the dimensions most sensitive to position keep a higher precision.
//
// A block of 32 values shares one E8M0 scale 2^(e - 127) (e = 0xFF is NaN).  Elements are E2M1
// (sign, two exponent bits with bias 1, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a byte
// with element 2j in the low nibble, or E4M3 bytes.  The shared exponent is
// floor(log2 amax) - emax, emax = 2 (E2M1) or 8 (E4M3), at least -127; a block of zeros takes
// e = 0, a block that holds an infinity or a NaN e = 0xFF and zero codes.  Dividing by a power
// of two is exact, so an element is rounded once: to nearest, ties to even, saturating.
//
// A 4-bit main-KV row holds K (128 dims) then V (128 dims) of one compressed entry, 176 bytes:
//   [  0,  32) K dims 0..63, E2M1                 [ 96, 160) V dims 0..127, E2M1
//   [ 32,  96) K dims 64..127 (the RoPE dims), E4M3
//   [160, 168) E8M0 scales of the eight 32-value blocks;  [168, 176) zero
// Every decoded value is a power of two times a 2- or 4-bit significand: exact in bf16 (down to
// bf16's subnormals), so attention over bf16 copies of the rows loses nothing.
#pragma once

#include "common.cuh"

namespace cskv {

constexpr int kMxBlock = 32;
constexpr int kKv4RowBytes = CSKV_KV4_ROW_BYTES;
constexpr int kKv4Rope = 32, kKv4V = 96, kKv4Scales = 160;  // byte offsets inside a row
constexpr int kE2m1Emax = 2, kE4m3Emax = 8;

// E8M0 code of a block whose largest magnitude has the bits `amax` (a non-negative fp32):
// the biased exponent of 2^(floor(log2 amax) - emax), 0 at least.
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax, int emax) {
  const int e = (int)(amax >> 23) - emax;  // a subnormal amax: exponent field 0
  return amax >= 0x7F800000u ? 0xFFu : (uint32_t)max(e, 0);
}

// 2^(127 - e), the reciprocal of the scale (exact; 2^127 .. 2^-126 for e = 0 .. 253).  A block
// without a finite scale gets 0: finite elements become zero codes (the others are masked).
__device__ __forceinline__ float mx_inv_scale(uint32_t e) {
  return e == 0xFFu ? 0.f : __uint_as_float((254u - e) << 23);
}

// 2^(e - 127) as fp32 (2^-127 is a subnormal; e = 0xFF is NaN).
__device__ __forceinline__ float mx_scale(uint32_t e) {
  return e == 0xFFu ? __uint_as_float(0x7FC00000u) : e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}

// max(m, |x|) that keeps a NaN.
__device__ __forceinline__ float amax_nan(float m, float x) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(x)));
  return d;
}

// Eight fp32 values -> eight E2M1 codes, element i in nibble i.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

// Eight fp32 values -> eight E4M3 codes.
__device__ __forceinline__ uint2 e4m3x8(const float (&y)[8]) {
  uint2 w;
  asm("{\n\t.reg .b16 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 c, %7, %6;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 d, %9, %8;\n\t"
      "mov.b32 %0, {a, b};\n\tmov.b32 %1, {c, d};\n\t}"
      : "=r"(w.x), "=r"(w.y)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

// Value of an E2M1 code without its scale: the code's exponent and mantissa bits moved into
// fp32's fields give value * 2^-126 (the 0.5 as a subnormal), so one exact product restores it.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  return __uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)) * __uint_as_float(0x7E800000u);
}
// The same for an E4M3 code (value * 2^-120).  0x7F and 0xFF, NaN in E4M3, are never written by
// the quantiser and read as +-480.
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  return __uint_as_float(((c & 0x7Fu) << 20) | ((c & 0x80u) << 24)) * __uint_as_float(0x7B800000u);
}

// ---------------------------------------------------------------- decoding to bf16, pairs at a time
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 2^(e - 127) twice, as bf16 (2^-127 is a subnormal; 0xFF is NaN).
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t e) {
  const uint32_t b = e == 0xFFu ? 0x7FC0u : e == 0 ? 0x0040u : e << 7;
  return b * 0x00010001u;
}
// Four E2M1 codes (16 bits of w) -> two words of bf16 pairs: the high and low byte of each
// magnitude come from 8-byte tables by byte permute; a selector nibble's top bit (the sign) turns
// the selected 0x80 into 0xFF, whose low bit moves to the sign place.
__device__ __forceinline__ void e2m1x4_bf16(uint32_t w, uint32_t wm, uint32_t s, uint32_t& o0, uint32_t& o1) {
  const uint32_t hi = prmt(0x3F3F3F00u, 0x40404040u, wm), lo = prmt(0xC0800000u, 0xC0804000u, wm);
  const uint32_t sg = prmt(0x80808080u, 0x80808080u, w);
  const uint32_t hs = hi | ((sg << 7) & 0x80808080u);
  o0 = mul_bf16x2(prmt(lo, hs, 0x5140u), s);
  o1 = mul_bf16x2(prmt(lo, hs, 0x7362u), s);
}
__device__ __forceinline__ uint4 e2m1x8_bf16(uint32_t w, uint32_t s) {
  uint4 o;
  const uint32_t wm = w & 0x77777777u;
  e2m1x4_bf16(w, wm, s, o.x, o.y);
  e2m1x4_bf16(w >> 16, wm >> 16, s, o.z, o.w);
  return o;
}
// Two E4M3 codes in the high bytes of h's halves -> bf16: exponent and mantissa moved into place
// (value * 2^-120), then two exact products (one would overflow the factor for large scales).
__device__ __forceinline__ uint32_t e4m3x2_bf16(uint32_t h, uint32_t s) {
  const uint32_t b = ((h >> 4) & 0x07F007F0u) | (h & 0x80008000u);
  return mul_bf16x2(mul_bf16x2(b, 0x7B807B80u), s);
}
__device__ __forceinline__ uint4 e4m3x8_bf16(uint32_t w0, uint32_t w1, uint32_t s) {
  return make_uint4(e4m3x2_bf16(prmt(w0, 0u, 0x1404u), s), e4m3x2_bf16(prmt(w0, 0u, 0x3424u), s),
                    e4m3x2_bf16(prmt(w1, 0u, 0x1404u), s), e4m3x2_bf16(prmt(w1, 0u, 0x3424u), s));
}

// Values 8 * part .. 8 * part + 7 (part 0..31 over the 256 K||V values) of a 4-bit row, as fp32.
__device__ __forceinline__ void kv4_load8(const uint8_t* row, int part, float (&f)[8]) {
  const float s = mx_scale(__ldg(row + kKv4Scales + (part >> 2)));
  if (part >= 8 && part < 16) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + kKv4Rope) + (part - 8));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = e4m3_value((i < 4 ? w.x : w.y) >> (8 * (i & 3))) * s;
    return;
  }
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(row + (part < 8 ? 4 * part : kKv4V + 4 * (part - 16))));
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = e2m1_value(w >> (4 * i)) * s;
}

// Values 32 * part .. 32 * part + 31 (part 0..7) of a 4-bit row.
__device__ __forceinline__ void kv4_load_part(const uint8_t* row, int part, float (&f)[32]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    float g[8];
    kv4_load8(row, 4 * part + v, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[8 * v + i] = g[i];
  }
}

}  // namespace cskv
