// kv4.cuh -- the 4-bit cache's format (include/diffattn.h, "Key/value cache in 4 bits"): device
// helpers shared by the kernels that write it, read it back and attend over it.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace da {

constexpr int kKv4Tokens = 16;            // tokens of one record
constexpr int kKv4PlaneCodes = 1024;      // 16 tokens x 128 channels x 4 bits
constexpr int kKv4Plane = 1024 + 128;     // and 16 x 8 scales

// Where token `key` (0..15) of a record has its data in a plane. K: channels 32t .. 32t+31 are
// 16 bytes at k_code(key, t), their two scales 2 bytes at k_scale(key, t). V: channels
// 16g .. 16g+15 are 8 bytes at v_code(key, g), their scale one byte at v_scale(key, g).
// Both orders are those in which a lane of the attention's matrix products needs them: lane
// 4g + t takes K's rows 4(g/2) + g%2 and that + 2 at channels 32t .., and V's rows 4t .. 4t+3 at
// channels 16g .., as whole 16-byte pieces that lie side by side over the lanes of a warp.
__host__ __device__ constexpr int kv4_k_code(int key, int t) {
  return ((key >> 1) & 1) * 512 + (key >> 2) * 128 + (key & 1) * 64 + t * 16;
}
__host__ __device__ constexpr int kv4_k_scale(int key, int t) {
  return kKv4PlaneCodes + (key >> 2) * 32 + (key & 1) * 16 + t * 4 + ((key >> 1) & 1) * 2;
}
__host__ __device__ constexpr int kv4_v_code(int key, int g) {
  return ((key >> 1) & 1) * 512 + g * 64 + (key >> 2) * 16 + (key & 1) * 8;
}
__host__ __device__ constexpr int kv4_v_scale(int key, int g) {
  return kKv4PlaneCodes + g * 16 + (key >> 2) * 4 + (key & 3);
}

// Eight e2m1 codes (low nibble first) as four half2, exactly.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Two e4m3 values (low byte first) as a half2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t d;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(two));
  return d;
}
// Four e4m3 values (low byte first) as two half2, exactly.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 h0, h1;\n\tmov.b32 {h0, h1}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h0;\n\tcvt.rn.f16x2.e4m3x2 %1, h1;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  const uint32_t h = e4m3x2_to_half2(byte);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}
// x (not negative, NaN not special here) rounded to e4m3, at most 448.
__device__ __forceinline__ uint32_t float_to_e4m3(float x) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(x));
  return d & 0xffu;
}
// Four half2 rounded to eight e2m1 codes (ties to the even code, at most 6), the first in the lowest
// nibble.
__device__ __forceinline__ uint32_t half2x4_to_e2m1x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b0, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b1, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b2, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b3, %4;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "r"(a), "r"(b), "r"(c), "r"(d));
  return w;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace da
