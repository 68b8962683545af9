// MXFP4 (OCP Microscaling, block of 32): E2M1 elements (0, 0.5, 1, 1.5, 2, 3,
// 4, 6 and their negatives) that share one E8M0 scale 2^(byte - 127).
//
// Quantisation of a block x_0..x_31 with a = max |x_i|:
//   byte = clamp(floor(log2 a) - 2 + 127, 0, 254)   (0 where a = 0)
//   code_i = nearest E2M1 to x_i * 2^(127 - byte), ties to the even mantissa,
//            saturated to 6; the sign is kept, also of a zero
// (2 is the exponent of the format's largest element, 6 = 1.5 * 2^2). The
// product by a power of two is exact or far below 0.25 in a subnormal's last
// bit, so no element is decided by a rounding other than its own. A block
// that holds a NaN or an infinity gets byte 255 (NaN) and zero codes.
#pragma once

#include "moe_common.cuh"

namespace moe {

constexpr int MX_BLOCK = 32;

// Bytes of one row of scales: K / 32, rounded up to whole 32-bit words.
__host__ __device__ constexpr int64_t mx_scale_pitch(int64_t K) { return (K + 127) / 128 * 4; }

// The E8M0 byte of a block from the FP32 bits of its largest magnitude
// (integer order puts infinities and NaNs above every finite value).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t ex = amax_bits >> 23;  // floor(log2 a) + 127; 0 for zero and FP32 subnormals
  if (ex == 255u) return 255u;
  return ex > 2u ? ex - 2u : 0u;
}

// 2^(127 - byte), the factor that brings the block onto the E2M1 grid
// (byte <= 252 here: a finite FP32 has ex <= 254); 0 for a NaN block.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); 2^-127 is an FP32 subnormal; NaN for byte 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  if (byte == 255u) return __int_as_float(0x7FC00000);
  return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// Eight scaled values -> eight E2M1 codes, v[0] in the lowest four bits.
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight E2M1 codes -> four pairs of FP16 (every E2M1 value is an FP16).
__device__ __forceinline__ void mx_unpack8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

}  // namespace moe
