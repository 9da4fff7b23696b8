// decode_kv4.cu -- decode attention over the 4-bit cache: one query token per sequence.
//
// For one (sequence, KV head) the kernel keeps COLS running softmaxes (V1: the two maps of one
// head; V2: the G query heads of the group) over the same keys and one output row of V's width for
// each: o = sum_j 2^(s_j - m) v_j, l = sum_j 2^(s_j - m), rescaled where the maximum m grows.
// Then V1: o1/l1 - lambda o2/l2, the norm and the scale; V2: o_2p/l_2p - sigmoid(lam) o_2p+1/l_2p+1.
// This first form is the plain one: a block for each (sequence, KV head), 16 keys at a time unpacked
// into shared memory as fp32, and CUDA-core products.
#include <cmath>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int KP, int G>  // KP: planes of K (2: V1, 1: V2); G: query heads per KV head (V1: 1)
__global__ void __launch_bounds__(KP * 128) kv4_decode_kernel(const Kv4DecodeArgs a) {
  constexpr int W = KP * 128;             // row width of K and of V
  constexpr int COLS = KP == 2 ? 2 : G;
  __shared__ float sq[COLS][128];         // the queries, times log2(e) / sqrt(d) 2^k_exp
  __shared__ float sk[16][W + 1], sv[16][W];
  __shared__ float ss[COLS][16], sm[COLS], sl[COLS], sc[COLS];
  __shared__ float red[W / 32];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  for (int i = tid; i < COLS * 128; i += W) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    sq[i >> 7][i & 127] = __bfloat162float(q[(static_cast<size_t>(b) * a.H + h) * COLS * 128 + i]) * a.qk_scale;
  }
  if (tid < COLS) sm[tid] = -INFINITY, sl[tid] = 0.f;
  const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
  int len = a.seqlens[b];
  len = len < 0 ? 0 : len > cap ? static_cast<int>(cap) : len;
  float o[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) o[c] = 0.f;
  __syncthreads();
  for (int k0 = 0; k0 < len; k0 += 16) {
    const int pi = k0 / a.page_size, off = k0 - pi * a.page_size;
    int page = a.block_table[static_cast<size_t>(b) * a.max_pages + pi];
    if (page < 0 || page >= a.num_pages) {
      if (tid == 0) flag_device_error(DEV_BAD_INDEX);
      page = 0;
    }
    const uint8_t* rec = a.pool + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                                      static_cast<size_t>(2 * KP * kKv4Plane);
    const int n = min(16, len - k0);
    // 16 keys x 2 KP planes x 8 blocks of 16 channels
    for (int i = tid; i < 16 * 2 * KP * 8; i += W) {
      const int key = i / (2 * KP * 8), blk = i % (2 * KP * 8), plane = blk >> 3, b8 = blk & 7;
      const bool is_k = plane < KP;
      const uint8_t* p = rec + plane * kKv4Plane;
      const int t = b8 >> 1, u = b8 & 1;
      const uint2 c = *reinterpret_cast<const uint2*>(p + (is_k ? kv4_k_code(key, t) + u * 8 : kv4_v_code(key, b8)));
      float s = e4m3_to_float(p[is_k ? kv4_k_scale(key, t) + u : kv4_v_scale(key, b8)]);
      if (key >= n) s = 0.f;  // rows past the end may hold anything
      float* dst = is_k ? &sk[key][blk * 16] : &sv[key][(blk - KP * 8) * 16];
      uint32_t x[4], y[4];
      e2m1x8_to_half2(c.x, x);
      e2m1x8_to_half2(c.y, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&y[j]));
        dst[2 * j] = f.x * s;
        dst[2 * j + 1] = f.y * s;
        dst[8 + 2 * j] = g.x * s;
        dst[8 + 2 * j + 1] = g.y * s;
      }
    }
    __syncthreads();
    if (tid < COLS * 16) {
      const int c = tid >> 4, key = tid & 15;
      float s = 0.f;
      for (int d = 0; d < 128; ++d) s = fmaf(sq[c][d], sk[key][(KP == 2 ? c * 128 : 0) + d], s);
      ss[c][key] = key < n ? s : -INFINITY;
    }
    __syncthreads();
    if (tid < COLS) {
      float m = sm[tid];
      for (int j = 0; j < n; ++j) m = ss[tid][j] > m ? ss[tid][j] : m;
      const float ref = m == -INFINITY ? 0.f : m;
      const float corr = exp2f(sm[tid] - ref);
      float l = sl[tid] * corr;
      for (int j = 0; j < 16; ++j) {
        const float pj = exp2f(ss[tid][j] - ref);
        ss[tid][j] = pj;
        l += pj;
      }
      sm[tid] = m;
      sl[tid] = l;
      sc[tid] = corr;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      float x = o[c] * sc[c];
      for (int j = 0; j < 16; ++j) x = fmaf(ss[c][j], sv[j][tid], x);
      o[c] = x;
    }
    __syncthreads();
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  const bool none = len == 0;
  if constexpr (KP == 2) {
    float y = none ? 0.f : (o[0] / sl[0] - a.lambda[h] * (o[1] / sl[1])) * a.v_mul;
    if (a.flags & 2) {
      float t = y * y;
      for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
      if ((tid & 31) == 0) red[tid >> 5] = t;
      __syncthreads();
      float sum = 0.f;
      for (int i = 0; i < W / 32; ++i) sum += red[i];
      y *= (1.f / sqrtf(sum / static_cast<float>(W) + a.eps)) * (a.norm_w ? a.norm_w[tid] : 1.f);
    }
    if (a.flags & 4) y *= 1.f - a.lambda_init;
    out[(static_cast<size_t>(b) * a.H + h) * W + tid] = __float2bfloat16_rn(y);
  } else {
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
      const size_t pair = (static_cast<size_t>(b) * a.H + h) * (COLS / 2) + c / 2;
      const float sig = 1.f / (1.f + expf(-a.lam_logit[pair]));
      const float y = none ? 0.f : (o[c] / sl[c] - sig * (o[c + 1] / sl[c + 1])) * a.v_mul;
      out[pair * W + tid] = __float2bfloat16_rn(y);
    }
  }
}

}  // namespace

size_t kv4_decode_workspace_bytes(int B, int H, int cols, int width) {
  (void)B, (void)H, (void)cols, (void)width;
  return 256;
}

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t st) {
  const dim3 grid(a.H, a.B);
  if (a.group == 0) kv4_decode_kernel<2, 1><<<grid, 256, 0, st>>>(a);
  else if (a.group == 2) kv4_decode_kernel<1, 2><<<grid, 128, 0, st>>>(a);
  else if (a.group == 4) kv4_decode_kernel<1, 4><<<grid, 128, 0, st>>>(a);
  else kv4_decode_kernel<1, 8><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t status_decode_kv4(int* v) { return read_clear_status(v); }

}  // namespace da
