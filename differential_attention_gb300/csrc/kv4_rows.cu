// kv4_rows.cu -- rows into and out of the 4-bit cache: diffattn_kv4_append rounds new K and V rows
// and writes them at their slots, diffattn_kv4_gather reads cached rows back as packed bf16.
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// One thread rounds one block of 16 channels: s = e4m3(amax / 6), c = e2m1(x / s). x has 8
// significant bits, s 4 and a border of e2m1 3: a quotient that is not on a border is off by more
// than 2^-9 of it, so the 32-bit quotient decides as the exact one would.
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  const int blocks = (a.kp + a.vp) * 8;  // of one (token, head)
  const long long i = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= static_cast<long long>(a.total) * a.H * blocks) return;
  const int blk = static_cast<int>(i % blocks);
  const int h = static_cast<int>(i / blocks % a.H);
  const long long token = i / blocks / a.H;
  const int slot = a.slot_map[token];
  if (slot < 0 || slot >= a.num_pages * a.page_size) {
    if (slot != -1) flag_device_error(DEV_BAD_INDEX);
    return;
  }
  const bool is_k = blk < a.kp * 8;
  const int plane = blk >> 3, b8 = blk & 7;
  const __nv_bfloat16* src =
      is_k ? a.k + token * a.k_token + h * a.k_head + blk * 16
           : a.v + token * a.v_token + h * a.v_head + (blk - a.kp * 8) * 16;
  const uint4 w0 = *reinterpret_cast<const uint4*>(src), w1 = *reinterpret_cast<const uint4*>(src + 8);
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  const float f = is_k ? a.k_inv : a.v_inv;
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = bf16x2_to_float2(w[j]);
    odd = odd || !(fabsf(x.x) < INFINITY) || !(fabsf(x.y) < INFINITY);
    amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
  }
  const uint32_t s8 = odd ? 0x7fu : float_to_e4m3(__fdiv_rn(amax * f, 6.f));
  const float s = e4m3_to_float(s8);
  uint32_t c[2] = {0, 0};
  if (s > 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 x = bf16x2_to_float2(w[j]);
      c[j >> 2] |= float2_to_e2m1x2(__fdiv_rn(x.x * f, s), __fdiv_rn(x.y * f, s)) << (8 * (j & 3));
    }
  }
  const int page = slot / a.page_size, off = slot - page * a.page_size, key = off & 15;
  uint8_t* rec = a.pool + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                              static_cast<size_t>((a.kp + a.vp) * kKv4Plane);
  uint8_t* p = rec + plane * kKv4Plane;
  const int t = b8 >> 1, u = b8 & 1;
  const int at = is_k ? kv4_k_code(key, t) + u * 8 : kv4_v_code(key, b8);
  *reinterpret_cast<uint2*>(p + at) = make_uint2(c[0], c[1]);
  p[is_k ? kv4_k_scale(key, t) + u : kv4_v_scale(key, b8)] = static_cast<uint8_t>(s8);
}

// One thread reads back one block of 16 channels of one (row, head).
__global__ void __launch_bounds__(kRowThreads) kv4_gather_kernel(const Kv4GatherArgs a) {
  const int blocks = (a.kp + a.vp) * 8;
  const long long i = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= static_cast<long long>(a.total) * a.H * blocks) return;
  const int blk = static_cast<int>(i % blocks);
  const int h = static_cast<int>(i / blocks % a.H);
  const int row = static_cast<int>(i / blocks / a.H);
  // the sequence that owns this row: the last b with cu[b] <= row
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_seqlens[mid] <= row) lo = mid; else hi = mid;
  }
  const int c0 = a.cu_seqlens[lo], c1 = a.cu_seqlens[lo + 1];
  if (row < c0 || row >= c1) return;  // behind the last sequence (or offsets that do not ascend)
  const long long pos = (a.starts ? a.starts[lo] : 0) + static_cast<long long>(row - c0);
  if (pos < 0 || pos >= static_cast<long long>(a.max_pages) * a.page_size) {
    flag_device_error(DEV_BAD_INDEX);
    return;
  }
  const int pi = static_cast<int>(pos / a.page_size), off = static_cast<int>(pos % a.page_size), key = off & 15;
  int page = a.block_table[static_cast<size_t>(lo) * a.max_pages + pi];
  if (page < 0 || page >= a.num_pages) {
    flag_device_error(DEV_BAD_INDEX);
    page = 0;
  }
  const uint8_t* rec = a.pool + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                                    static_cast<size_t>((a.kp + a.vp) * kKv4Plane);
  const int plane = blk >> 3, b8 = blk & 7;
  const bool is_k = plane < a.kp;
  const uint8_t* p = rec + plane * kKv4Plane;
  const int t = b8 >> 1, u = b8 & 1;
  const uint2 c = *reinterpret_cast<const uint2*>(p + (is_k ? kv4_k_code(key, t) + u * 8 : kv4_v_code(key, b8)));
  const float s = e4m3_to_float(p[is_k ? kv4_k_scale(key, t) + u : kv4_v_scale(key, b8)]) * (is_k ? a.k_mul : a.v_mul);
  uint32_t half[8];
  {
    uint32_t x[4], y[4];
    e2m1x8_to_half2(c.x, x);
    e2m1x8_to_half2(c.y, y);
    for (int j = 0; j < 4; ++j) half[j] = x[j], half[4 + j] = y[j];
  }
  uint32_t out[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&half[j]));
    const __nv_bfloat162 o = __floats2bfloat162_rn(v.x * s, v.y * s);
    out[j] = *reinterpret_cast<const uint32_t*>(&o);
  }
  const size_t at = static_cast<size_t>(row) * a.H + h;
  __nv_bfloat16* dst = is_k ? a.k_out + at * (a.kp * 128) + blk * 16
                            : a.v_out + at * (a.vp * 128) + (blk - a.kp * 8) * 16;
  *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
  *reinterpret_cast<uint4*>(dst + 8) = make_uint4(out[4], out[5], out[6], out[7]);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
  const long long n = static_cast<long long>(a.total) * a.H * (a.kp + a.vp) * 8;
  if (n == 0) return cudaSuccess;
  kv4_append_kernel<<<static_cast<unsigned>((n + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t st) {
  const long long n = static_cast<long long>(a.total) * a.H * (a.kp + a.vp) * 8;
  if (n == 0) return cudaSuccess;
  kv4_gather_kernel<<<static_cast<unsigned>((n + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t status_kv4_rows(int* v) { return read_clear_status(v); }

}  // namespace da
