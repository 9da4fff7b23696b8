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

struct Block {  // 16 channels as they are stored
  uint32_t lo, hi, scale;
};

// s = e4m3(amax / 6), c = e2m1(x / s) of 16 bf16 values.
// x has 8 significant bits, s 4 and a border b of e2m1 (0.25, 0.75, .. 5) 3, so x / s is either b or at
// least b / 512 >= 2^-11 from it. fma(|x|, 1/s, 6144) rounds |x| / s (but for the 2^-24 of 1/s) to a
// multiple of 2^-11, as all borders are: a quotient on a border lands on it, any other stays on its
// side. Three instructions instead of a division, and the decision of the exact quotient; the sign is
// put back last, so that a code of 0 has it too.
__device__ __forceinline__ Block round_block(const uint4& w0, const uint4& w1, float exp_inv) {
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t top = 0;  // the largest magnitude's bits, ordered as the values are
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
  Block b{0, 0, 0x7fu};
  if (top >= 0x7f80u) return b;  // an Inf or NaN: the block reads as NaN
  b.scale = float_to_e4m3(__fdiv_rn(__uint_as_float(top << 16) * exp_inv, 6.f));
  if (b.scale == 0) return b;
  const float r = __frcp_rn(e4m3_to_float(b.scale)) * exp_inv;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = bf16x2_to_float2(w[j] & 0x7fff7fffu);
    const float y0 = __uint_as_float(__float_as_uint(fmaf(x.x, r, 6144.f) - 6144.f) | ((w[j] << 16) & 0x80000000u));
    const float y1 = __uint_as_float(__float_as_uint(fmaf(x.y, r, 6144.f) - 6144.f) | (w[j] & 0x80000000u));
    const uint32_t c = float2_to_e2m1x2(y0, y1) << (8 * (j & 3));
    if (j < 4) b.lo |= c; else b.hi |= c;
  }
  return b;
}

// A warp rounds 8 rows of one head and plane: a lane 32 channels of a row of K (two blocks, one
// 16-byte piece of the record), or the same 16 channels of two rows of V, which are one piece too where
// the rows' slots are the two of a pair. What bounds it: the bytes (2 read, 9/16 written a channel).
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  const int planes = a.kp + a.vp, lane = threadIdx.x & 31;
  const long long u = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int plane = static_cast<int>(u % planes), h = static_cast<int>(u / planes % a.H);
  const long long row0 = u / planes / a.H * 8;
  if (row0 >= a.total) return;
  const bool is_k = plane < a.kp;
  auto slot_of = [&](long long row) {
    if (row >= a.total) return -1;
    const int s = __ldg(a.slot_map + row);
    if (s >= 0 && s < a.num_pages * a.page_size) return s;
    if (s != -1) flag_device_error(DEV_BAD_INDEX);
    return -1;
  };
  auto place = [&](int slot) {
    const int page = slot / a.page_size, off = slot - page * a.page_size;
    return a.pool + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                        static_cast<size_t>(planes * kKv4Plane) + plane * kKv4Plane;
  };
  if (is_k) {
    const long long row = row0 + (lane >> 2);
    const int t = lane & 3, slot = slot_of(row);
    if (slot < 0) return;
    const uint4* src = reinterpret_cast<const uint4*>(a.k + row * a.k_token + h * a.k_head + plane * 128 + t * 32);
    const uint4 w0 = __ldg(src), w1 = __ldg(src + 1), w2 = __ldg(src + 2), w3 = __ldg(src + 3);
    const Block x = round_block(w0, w1, a.k_inv), y = round_block(w2, w3, a.k_inv);
    uint8_t* p = place(slot);
    *reinterpret_cast<uint4*>(p + kv4_k_code(slot & 15, t)) = make_uint4(x.lo, x.hi, y.lo, y.hi);
    *reinterpret_cast<uint16_t*>(p + kv4_k_scale(slot & 15, t)) = static_cast<uint16_t>(x.scale | (y.scale << 8));
  } else {
    const long long row = row0 + 2 * (lane >> 3);
    const int g = lane & 7, s0 = slot_of(row), s1 = slot_of(row + 1);
    const __nv_bfloat16* src = a.v + row * a.v_token + h * a.v_head + (plane - a.kp) * 128 + g * 16;
    uint4 w[4];
    if (s0 >= 0) w[0] = __ldg(reinterpret_cast<const uint4*>(src)), w[1] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    src += a.v_token;
    if (s1 >= 0) w[2] = __ldg(reinterpret_cast<const uint4*>(src)), w[3] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    Block x{}, y{};
    if (s0 >= 0) x = round_block(w[0], w[1], a.v_inv);
    if (s1 >= 0) y = round_block(w[2], w[3], a.v_inv);
    if (s0 >= 0 && s1 == s0 + 1 && (s0 & 1) == 0) {
      uint8_t* p = place(s0);
      *reinterpret_cast<uint4*>(p + kv4_v_code(s0 & 15, g)) = make_uint4(x.lo, x.hi, y.lo, y.hi);
      *reinterpret_cast<uint16_t*>(p + kv4_v_scale(s0 & 15, g)) = static_cast<uint16_t>(x.scale | (y.scale << 8));
      return;
    }
    if (s0 >= 0) {
      uint8_t* p = place(s0);
      *reinterpret_cast<uint2*>(p + kv4_v_code(s0 & 15, g)) = make_uint2(x.lo, x.hi);
      p[kv4_v_scale(s0 & 15, g)] = static_cast<uint8_t>(x.scale);
    }
    if (s1 >= 0) {
      uint8_t* p = place(s1);
      *reinterpret_cast<uint2*>(p + kv4_v_code(s1 & 15, g)) = make_uint2(y.lo, y.hi);
      p[kv4_v_scale(s1 & 15, g)] = static_cast<uint8_t>(y.scale);
    }
  }
}

__device__ __forceinline__ uint32_t half2_to_bf16x2(uint32_t h, float f) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 o = __floats2bfloat162_rn(v.x * f, v.y * f);
  return *reinterpret_cast<const uint32_t*>(&o);
}

// A warp reads one record of one head of one sequence, in the order in which it lies in memory, and
// writes its rows: a lane 32 channels of two rows of K, and 16 channels of four rows of V. What bounds
// it: the bytes (9/16 read, 2 written a channel).
//
// Sequence b's records have the warps from cu[b] / 16 + 2 b on: n rows touch at most n / 16 + 2 records,
// so that the ranges do not overlap, whatever the sequences' first tokens are.
__global__ void __launch_bounds__(kRowThreads) kv4_gather_kernel(const Kv4GatherArgs a) {
  const int lane = threadIdx.x & 31;
  const long long i = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int h = static_cast<int>(i % a.H);
  const long long u = i / a.H;
  if (u >= a.total / 16 + 2LL * a.B) return;
  // the last b whose first warp is not behind this one: 32 candidates at a time
  int lo = 0, n = a.B;
  while (n > 1) {
    const int step = (n + 31) >> 5, b = lo + lane * step;
    const bool at = lane * step < n && __ldg(a.cu_seqlens + b) / 16 + 2LL * b <= u;
    const unsigned hit = __ballot_sync(0xffffffffu, at);
    const int last = hit ? 31 - __clz(hit) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const int c0 = __ldg(a.cu_seqlens + lo), c1 = __ldg(a.cu_seqlens + lo + 1);
  if (c0 < 0 || c1 > a.total || c0 >= c1) {
    if (c0 < 0 || c1 > a.total || c0 > c1) flag_device_error(DEV_BAD_INDEX);
    return;
  }
  const long long first = a.starts ? __ldg(a.starts + lo) : 0, end = first + (c1 - c0);
  // token of this record's first row (its record counted from the sequence's first one, towards
  // minus infinity where the first token is negative)
  const long long tok = (((first - (first & 15)) >> 4) + (u - c0 / 16 - 2LL * lo)) * 16;
  if (tok >= end) return;
  const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
  if (tok < 0 || tok >= cap) {
    flag_device_error(DEV_BAD_INDEX);
    return;
  }
  const int pi = static_cast<int>(tok / a.page_size), off = static_cast<int>(tok - static_cast<long long>(pi) * a.page_size);
  int page = __ldg(a.block_table + static_cast<size_t>(lo) * a.max_pages + pi);
  if (page < 0 || page >= a.num_pages) {
    flag_device_error(DEV_BAD_INDEX);
    page = 0;
  }
  const uint8_t* rec = a.pool + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                                    static_cast<size_t>((a.kp + a.vp) * kKv4Plane);
  const int g = lane >> 2, t = lane & 3;
  const long long row0 = c0 + (tok - first);  // output row of the record's token 0 (it may not be wanted)
  auto wanted = [&](int key) { return tok + key >= first && tok + key < end; };
  for (int pl = 0; pl < a.kp + a.vp; ++pl) {
    const uint8_t* p = rec + pl * kKv4Plane;
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p) + lane), y = __ldg(reinterpret_cast<const uint4*>(p + 512) + lane);
    uint32_t s01, s23;
    e4m3x4_to_half2(__ldg(reinterpret_cast<const uint32_t*>(p + kKv4PlaneCodes) + lane), s01, s23);
    const float2 s0 = __half22float2(*reinterpret_cast<const __half2*>(&s01));
    const float2 s1 = __half22float2(*reinterpret_cast<const __half2*>(&s23));
    // 8 codes, scale, 8 channels from `ch` of a token
    auto put = [&](__nv_bfloat16* out, int w, int key, int ch, uint32_t codes, float s) {
      if (!wanted(key)) return;
      uint32_t v[4];
      e2m1x8_to_half2(codes, v);
      *reinterpret_cast<uint4*>(out + (static_cast<size_t>(row0 + key) * a.H + h) * w + ch) =
          make_uint4(half2_to_bf16x2(v[0], s), half2_to_bf16x2(v[1], s), half2_to_bf16x2(v[2], s), half2_to_bf16x2(v[3], s));
    };
    if (pl < a.kp) {
      const int key = (g >> 1) * 4 + (g & 1), ch = pl * 128 + 32 * t, w = a.kp * 128;
      const float f[4] = {s0.x * a.k_mul, s0.y * a.k_mul, s1.x * a.k_mul, s1.y * a.k_mul};
      put(a.k_out, w, key, ch, x.x, f[0]), put(a.k_out, w, key, ch + 8, x.y, f[0]);
      put(a.k_out, w, key, ch + 16, x.z, f[1]), put(a.k_out, w, key, ch + 24, x.w, f[1]);
      put(a.k_out, w, key + 2, ch, y.x, f[2]), put(a.k_out, w, key + 2, ch + 8, y.y, f[2]);
      put(a.k_out, w, key + 2, ch + 16, y.z, f[3]), put(a.k_out, w, key + 2, ch + 24, y.w, f[3]);
    } else {
      const int key = 4 * t, ch = (pl - a.kp) * 128 + 16 * g, w = a.vp * 128;
      const float f[4] = {s0.x * a.v_mul, s0.y * a.v_mul, s1.x * a.v_mul, s1.y * a.v_mul};
      put(a.v_out, w, key, ch, x.x, f[0]), put(a.v_out, w, key, ch + 8, x.y, f[0]);
      put(a.v_out, w, key + 1, ch, x.z, f[1]), put(a.v_out, w, key + 1, ch + 8, x.w, f[1]);
      put(a.v_out, w, key + 2, ch, y.x, f[2]), put(a.v_out, w, key + 2, ch + 8, y.y, f[2]);
      put(a.v_out, w, key + 3, ch, y.z, f[3]), put(a.v_out, w, key + 3, ch + 8, y.w, f[3]);
    }
  }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  const long long warps = (static_cast<long long>(a.total) + 7) / 8 * a.H * (a.kp + a.vp);
  kv4_append_kernel<<<static_cast<unsigned>((warps * 32 + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  const long long warps = (a.total / 16 + 2LL * a.B) * a.H;
  kv4_gather_kernel<<<static_cast<unsigned>((warps * 32 + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t status_kv4_rows(int* v) { return read_clear_status(v); }

}  // namespace da
