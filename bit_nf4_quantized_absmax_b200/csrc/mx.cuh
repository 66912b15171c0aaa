// Microscaled (MX) formats: 32 consecutive elements of a row share a scale 2^e
// stored as the byte e + 127 (255: NaN). Elements are e4m3 or e2m1.
//
// For a block with largest magnitude amax, e = max(floor(log2 amax) - emax,
// -127) with emax the exponent of the element type's largest value (8 for
// e4m3's 448, 2 for e2m1's 6). With f the exponent field of amax as fp32 or
// bf16 (both have a bias of 127) the byte is max(f - emax, 0): no logarithm is
// taken, f = 0 (zero and subnormals) gives byte 0, and f = 255 (an infinity or
// a NaN in the block) gives byte 255. Multiplying by 2^-e is exact, so the
// only rounding of an element is the conversion to its type.
#pragma once

#include "common.cuh"

namespace qlora {

constexpr int kMxE4M3 = 0;
constexpr int kMxE2M1 = 1;

template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t exp_field) {
  constexpr int emax = FMT == kMxE4M3 ? 8 : 2;
  return exp_field == 255u ? 255u : static_cast<uint32_t>(max(static_cast<int>(exp_field) - emax, 0));
}

// 2^-e of a scale byte 0..252 (a normal fp32); 0 for byte 255, which makes every
// finite element code 0 (the caller clears the others).
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^e of a scale byte: byte 0 is 2^-127, an fp32 subnormal.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7FC00000u);
  return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Two values to two e4m3 codes (lo in the low byte), nearest even, saturated.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Eight values to eight e2m1 codes, element i in nibble i, nearest even, saturated.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}

// One block of 32 bf16 values (two a word) to its codes (8 words of e4m3, 4 of e2m1);
// returns the scale byte. The maximum is taken on the magnitude bits, two at a time,
// which order like the values and place NaN above infinity.
template <int FMT>
__device__ __forceinline__ uint32_t mx_quantize_block(const uint32_t (&v)[16], uint32_t (&o)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  const uint32_t byte = mx_scale_byte<FMT>(m >> 7);
  const float inv = mx_inverse_scale(byte);
  const bool bad = byte == 255u;
  float f[32];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const f32x2 a = mul_f32x2({bf16lo_to_f32(v[i]), bf16hi_to_f32(v[i])}, {inv, inv});
    f[2 * i] = a.x;
    f[2 * i + 1] = a.y;
  }
  if (FMT == kMxE4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = bad ? 0u : cvt_e4m3x2(f[4 * i], f[4 * i + 1]) | (cvt_e4m3x2(f[4 * i + 2], f[4 * i + 3]) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g[8] = {f[8 * i],     f[8 * i + 1], f[8 * i + 2], f[8 * i + 3],
                          f[8 * i + 4], f[8 * i + 5], f[8 * i + 6], f[8 * i + 7]};
      o[i] = bad ? 0u : cvt_e2m1x8(g);
    }
  }
  return byte;
}

// Two e4m3 codes (low 16 bits) to two fp32 values (exact).
__device__ __forceinline__ f32x2 e4m3x2_to_f32x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  f32x2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

}  // namespace qlora
