// kv4.cuh -- the 4-bit cache format: where each code and scale of a page lies, and its conversions.
//
// A value is code * scale.  The code is e2m1 (sign, magnitudes 0 0.5 1 1.5 2 3 4 6); the scale of 16
// neighbouring channels of one position is one byte, ue5m3: 5 exponent bits (bias 15), 3 mantissa bits.  That
// byte shifted left by 7 is the scale as an fp16 (subnormals and NaN included), so a scale costs one shift.  A
// code times a scale has at most 6 significant bits: exact in fp16 and bf16, so a product of dequantised
// operands on the tensor cores carries no rounding of the cache's values.
//
// The bytes of one (page, KV head) block of 64 positions lie in the order in which the m16n8k16 fragments
// want them, so a warp reads its operands with 16-byte loads and without shuffles.  With h = dh / 64,
// g = lane / 4, t = lane % 4:
//   K codes   [tile of 16 positions][h][lane][j 4] words; byte 0/2: position g, byte 1/3: position g + 8;
//             channels dh/4 t + 16 h + 4 j + {0,1 | 2,3} (low, high nibble of byte 0/1 | byte 2/3)
//   V codes   [tile][h][lane][j 4] words; byte 0/1: positions 2t, 2t+1 (low, high nibble) of channels
//             dh/8 g + 8 h + 2 j + {0 | 1}, byte 2/3: positions 2t+8, 2t+9 of the same
//   K scales  [position % 8][t][position / 8][h] bytes: block h-th of the lane's channels
//   V scales  [block of 16 channels][t][tile][4] bytes: positions 2t, 2t+1, 2t+8, 2t+9
#pragma once

#include <cuda_fp16.h>

#include "dg_device.cuh"

namespace dg {

constexpr int kPage = 64;

template <int DH>
struct Kv4 {
  static constexpr int kH = DH / 64;
  static constexpr int kCodes = kPage * DH / 2;    // bytes of K's (or V's) codes
  static constexpr int kScales = kPage * DH / 16;  // bytes of K's (or V's) scales
  static constexpr int kBytes = 2 * (kCodes + kScales);
  static constexpr int kV = kCodes, kSk = 2 * kCodes, kSv = 2 * kCodes + kScales;   // offsets; K at 0
};

// the four e2m1 pairs of a word as fp16 pairs (low nibble first)
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// bytes A and B of w as a pair of fp16 scales (A in the low half)
template <int A, int B>
__device__ __forceinline__ uint32_t scale_pair(uint32_t w) {
  return __byte_perm(w, 0, 0x4040 | A | (B << 8)) << 7;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float ue5m3_to_f32(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// The largest scale: 6 * 10240 is the largest multiple that fp16 still holds, so larger values saturate.
constexpr float kMaxScale = 10240.f;

// Scale byte of a block whose largest magnitude is amax (NaN if one of its values is): amax / 6 to the
// nearest ue5m3, ties to even.  amax has at most 11 significant bits, so amax / 6 is either on a rounding border (at most
// 5 bits) or off it by 2^-12 of itself: a product with 1 / 6, rounded to 16 bits, decides as the exact quotient does.
__device__ __forceinline__ uint32_t ue5m3_scale(float amax) {
  const float q = fminf(amax * 0.16666667f, kMaxScale);
  uint32_t u = (__float_as_uint(q) + 0x80u) & ~0xffu;
  // below 2^-14 steps of 2^-17: the sum's last bit is that step
  const uint32_t small = __float_as_uint(__fadd_rn(__uint_as_float(u), 64.f)) & 15u;
  u = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
  u = q < 6.103515625e-05f ? small : u;
  return amax != amax ? 255u : u;
}

// Quotient x / s on the grid of 2^-16, from r = 1 / s to 2^-22.  The product errs by less than 2^-18 and an exact
// quotient of an 11-bit value by a 4-bit scale is either on a border between two codes (a multiple of 1/4) or at
// least 2^-13 away from it: on the grid every border case is met exactly, and ties go to the even code.
// (two at once)
__device__ __forceinline__ uint64_t on_grid2(uint64_t x, uint64_t r) {
  return fadd_f32x2(ffma_f32x2(x, r, pack_f32x2(192.f, 192.f)), pack_f32x2(-192.f, -192.f));
}

// four pairs of quotients as the e2m1 bytes of a word (first of a pair in the low nibble), nearest, ties to even,
// beyond 6 saturating
__device__ __forceinline__ uint32_t to_e2m1_word(float a0, float a1, float b0, float b1, float c0, float c1, float d0,
                                                 float d1) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(w)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1), "f"(d0), "f"(d1));
  return w;
}

// 1 / s, to 2^-23 (s a positive scale)
__device__ __forceinline__ float fast_rcp(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 16-bit element pairs <-> float
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
  static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
};
template <>
struct Half<__half> {
  static __device__ __forceinline__ float lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)w)); }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) { return Half<__half>::pack(lo, hi); }

}  // namespace dg
