// kv4_mma.cuh -- records of the 4-bit cache as operands of m16n8k16, straight from shared memory: shared by
// the kernels for few query rows (decode_kv4.cu, chunk_kv4_few.cu).
#pragma once
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
// the first product of a sum
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// S^T of one record: rows g (key 4 (g/2) + g%2) and g + 8 (that + 2), columns 2t and 2t + 1. `at`: the
// K plane's codes for this lane.
__device__ __forceinline__ void scores(float (&c)[4], uint32_t at, int lane, const uint4 (&qf)[4]) {
  const uint4 lo4 = lds128(at), hi4 = lds128(at + 512);
  const uint32_t sc = lds32(at - lane * 12 + kKv4PlaneCodes);
  uint32_t slo, shi;
  e4m3x4_to_half2(sc, slo, shi);
  const uint32_t wl[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, wh[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // the scale of channels 32t + 8k .. of row g, and of row g + 8, in both halves
    const uint32_t sl = __byte_perm(slo, 0, k < 2 ? 0x1010 : 0x3232);
    const uint32_t sh = __byte_perm(shi, 0, k < 2 ? 0x1010 : 0x3232);
    uint32_t x[4], y[4];
    e2m1x8_to_half2(wl[k], x);
    e2m1x8_to_half2(wh[k], y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = half2_mul(x[i], sl), y[i] = half2_mul(y[i], sh);
    if (k == 0) mma_first(c, x[0], y[0], x[1], y[1], qf[k].x, qf[k].y);
    else mma(c, x[0], y[0], x[1], y[1], qf[k].x, qf[k].y);
    mma(c, x[2], y[2], x[3], y[3], qf[k].z, qf[k].w);
  }
}

}  // namespace da
