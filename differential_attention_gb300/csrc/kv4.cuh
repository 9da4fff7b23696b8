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

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

struct Kv4Block {  // 16 channels as they are stored
  uint32_t lo, hi, scale;
};

// s = e4m3(amax / 6), c = e2m1(x / s) of 16 bf16 values.
// x has 8 significant bits, s 4 and a border b of e2m1 (0.25, 0.75, .. 5) 3, so x / s is either b or
// some 2^-8 b away from it. x times the rounded 1 / s, rounded once more to fp16's 11 bits, is then b
// where the quotient is, and on its side of b where it is not: the decision of the exact quotient
// without a division.
__device__ __forceinline__ Kv4Block kv4_round_block(const uint4& w0, const uint4& w1, float exp_inv) {
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t top2 = 0;  // the largest magnitudes' bits, ordered as the values are
#pragma unroll
  for (int j = 0; j < 8; ++j) top2 = __vmaxu2(top2, w[j] & 0x7fff7fffu);
  const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  Kv4Block b{0, 0, 0x7fu};
  if (top >= 0x7f80u) return b;  // an Inf or NaN: the block reads as NaN
  b.scale = float_to_e4m3(__fdiv_rn(__uint_as_float(top << 16) * exp_inv, 6.f));
  if (b.scale == 0) return b;
  const float r = __frcp_rn(e4m3_to_float(b.scale)) * exp_inv;
  uint32_t y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = bf16x2_to_float2(w[j]);
    y[j] = pack_half2(x.x * r, x.y * r);
  }
  b.lo = half2x4_to_e2m1x8(y[0], y[1], y[2], y[3]);
  b.hi = half2x4_to_e2m1x8(y[4], y[5], y[6], y[7]);
  return b;
}

}  // namespace da
