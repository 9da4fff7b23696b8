// kv4_rows.cu -- rows into and out of the 4-bit cache: diffattn_kv4_append rounds new K and V rows
// and writes them at their slots, diffattn_kv4_gather reads cached rows back as packed bf16.
#include "early.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {
namespace {

// (Append of 16K rows of 12 V1 heads and their read-out: 87.3 us with 256 and 256 threads, 86.0 so; the
// read-out alone is 0.3 slower with 64.)
constexpr int kAppendThreads = 64, kGatherThreads = 256;

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

struct Block {  // 16 channels as they are stored
  uint32_t lo, hi, scale;
};

// s = e4m3(amax / 6), c = e2m1(x / s) of 16 bf16 values.
// x has 8 significant bits, s 4 and a border b of e2m1 (0.25, 0.75, .. 5) 3, so x / s is either b or
// some 2^-8 b away from it. x times the rounded 1 / s, rounded once more to fp16's 11 bits, is then b
// where the quotient is, and on its side of b where it is not: the decision of the exact quotient
// without a division.
__device__ __forceinline__ Block round_block(const uint4& w0, const uint4& w1, float exp_inv) {
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t top2 = 0;  // the largest magnitudes' bits, ordered as the values are
#pragma unroll
  for (int j = 0; j < 8; ++j) top2 = __vmaxu2(top2, w[j] & 0x7fff7fffu);
  const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  Block b{0, 0, 0x7fu};
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

// A warp rounds 8 rows of one head, plane after plane: a lane 32 channels of a row of K (two blocks, one
// 16-byte piece of the record), then the same 16 channels of two rows of V, which are one piece too
// where the rows' slots are the two of a pair. The next plane is loaded while one is rounded. What
// bounds it: the bytes (2 read, 9/16 written a channel): 64K rows of 12 V1 heads, 1.03 GB, take 153.5 us,
// 6.72 TB/s of a copy's 6.78, with 55 % of the ALU pipe and 63 % of the issue slots in use; 16K rows 43.9,
// 5.9 TB/s. (With a division for each value 16K rows took about 100.)
template <int KP>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  grid_wait();
  grid_release();
  const int lane = threadIdx.x & 31;
  const long long u = static_cast<long long>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int h = static_cast<int>(u % a.H);
  const long long row0 = u / a.H * 8;
  if (row0 >= a.total) return;
  auto slot_of = [&](long long row) {
    if (row >= a.total) return -1;
    const int s = *(a.slot_map + row);
    if (s >= 0 && s < a.num_pages * a.page_size) return s;
    if (s != -1) flag_device_error(DEV_BAD_INDEX);
    return -1;
  };
  auto place = [&](int slot) {
    const int page = slot / a.page_size, off = slot - page * a.page_size;
    return a.pool + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                        static_cast<size_t>(2 * KP * kKv4Plane);
  };
  const int t = lane & 3, g = lane & 7;
  const long long krow = row0 + (lane >> 2), vrow = row0 + 2 * (lane >> 3);
  const int ks = slot_of(krow), s0 = slot_of(vrow), s1 = slot_of(vrow + 1);
  const uint4* ksrc = reinterpret_cast<const uint4*>(a.k + krow * a.k_token + h * a.k_head + t * 32);
  const uint4* vsrc0 = reinterpret_cast<const uint4*>(a.v + vrow * a.v_token + h * a.v_head + g * 16);
  const uint4* vsrc1 = reinterpret_cast<const uint4*>(a.v + (vrow + 1) * a.v_token + h * a.v_head + g * 16);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](int plane, uint4 (&w)[4]) {
    if (plane < KP) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = ks >= 0 ? *(ksrc + plane * 16 + i) : zero;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = s0 >= 0 ? *(vsrc0 + (plane - KP) * 16 + i) : zero;
        w[2 + i] = s1 >= 0 ? *(vsrc1 + (plane - KP) * 16 + i) : zero;
      }
    }
  };
  uint8_t* kdst = place(max(ks, 0));
  uint8_t* vdst0 = place(max(s0, 0)) + KP * kKv4Plane;
  uint8_t* vdst1 = place(max(s1, 0)) + KP * kKv4Plane;
  const bool joined = s0 >= 0 && s1 == s0 + 1 && (s0 & 1) == 0;
  uint4 w[2][4];
  load(0, w[0]);
#pragma unroll
  for (int plane = 0; plane < 2 * KP; ++plane) {
    if (plane + 1 < 2 * KP) load(plane + 1, w[(plane + 1) & 1]);
    const uint4(&c)[4] = w[plane & 1];
    const float inv = plane < KP ? a.k_inv : a.v_inv;
    const Block x = round_block(c[0], c[1], inv), y = round_block(c[2], c[3], inv);
    if (plane < KP) {
      if (ks >= 0) {
        uint8_t* p = kdst + plane * kKv4Plane;
        *reinterpret_cast<uint4*>(p + kv4_k_code(ks & 15, t)) = make_uint4(x.lo, x.hi, y.lo, y.hi);
        *reinterpret_cast<uint16_t*>(p + kv4_k_scale(ks & 15, t)) = static_cast<uint16_t>(x.scale | (y.scale << 8));
      }
    } else if (joined) {
      uint8_t* p = vdst0 + (plane - KP) * kKv4Plane;
      *reinterpret_cast<uint4*>(p + kv4_v_code(s0 & 15, g)) = make_uint4(x.lo, x.hi, y.lo, y.hi);
      *reinterpret_cast<uint16_t*>(p + kv4_v_scale(s0 & 15, g)) = static_cast<uint16_t>(x.scale | (y.scale << 8));
    } else {
      if (s0 >= 0) {
        uint8_t* p = vdst0 + (plane - KP) * kKv4Plane;
        *reinterpret_cast<uint2*>(p + kv4_v_code(s0 & 15, g)) = make_uint2(x.lo, x.hi);
        p[kv4_v_scale(s0 & 15, g)] = static_cast<uint8_t>(x.scale);
      }
      if (s1 >= 0) {
        uint8_t* p = vdst1 + (plane - KP) * kKv4Plane;
        *reinterpret_cast<uint2*>(p + kv4_v_code(s1 & 15, g)) = make_uint2(y.lo, y.hi);
        p[kv4_v_scale(s1 & 15, g)] = static_cast<uint8_t>(y.scale);
      }
    }
  }
}

__device__ __forceinline__ uint32_t half2_to_bf16x2(uint32_t h, float f) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 o = __floats2bfloat162_rn(v.x * f, v.y * f);
  return *reinterpret_cast<const uint32_t*>(&o);
}

// A warp reads a record of one sequence and head, plane after plane with the next one's loads under way,
// and writes its rows, two at a time: a lane 8 channels, so that each store of the warp is whole rows of
// 128 channels (16 bytes a lane, side by side). What bounds it: the bytes (9/16 read, 2 written a channel,
// so four fifths of them writes): 6 x 8160 tokens of 8 V2 heads, 257 MB, take 41.4 us, 6.2 TB/s of a
// copy's 6.78, 4 x 4080 of 12 V1 heads 42.5, 4 x 16384 of them 157.0, 6.6 TB/s. (Two or four heads a warp, which share one look-up of the
// sequence and the page: 42.3 and 42.3 us, 43.8 and 43.7. Streaming stores: no difference.)
//
// Sequence b's records have the warps from cu[b] / 16 + 2 b on: n rows touch at most n / 16 + 2 records,
// so that the ranges do not overlap, whatever the sequences' first tokens are.
template <int KP>
__global__ void __launch_bounds__(kGatherThreads) kv4_gather_kernel(const Kv4GatherArgs a) {
  grid_wait();
  grid_release();
  const int lane = threadIdx.x & 31;
  const long long i = static_cast<long long>(blockIdx.x) * (kGatherThreads / 32) + (threadIdx.x >> 5);
  const int h = static_cast<int>(i % a.H);
  const long long u = i / a.H;
  if (u >= a.total / 16 + 2LL * a.B) return;
  // the last b whose first warp is not behind this one: 32 candidates at a time
  int lo = 0, n = a.B;
  while (n > 1) {
    const int step = (n + 31) >> 5, b = lo + lane * step;
    const bool at = lane * step < n && *(a.cu_seqlens + b) / 16 + 2LL * b <= u;
    const unsigned hit = __ballot_sync(0xffffffffu, at);
    const int last = hit ? 31 - __clz(hit) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const int c0 = *(a.cu_seqlens + lo), c1 = *(a.cu_seqlens + lo + 1);
  if (c0 < 0 || c1 > a.total || c0 >= c1) {
    if (c0 < 0 || c1 > a.total || c0 > c1) flag_device_error(DEV_BAD_INDEX);
    return;
  }
  const long long first = a.starts ? *(a.starts + lo) : 0, end = first + (c1 - c0);
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
  int page = *(a.block_table + static_cast<size_t>(lo) * a.max_pages + pi);
  if (page < 0 || page >= a.num_pages) {
    flag_device_error(DEV_BAD_INDEX);
    page = 0;
  }
  const uint8_t* rec = a.pool + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                                    static_cast<size_t>(2 * KP * kKv4Plane);
  const long long row0 = c0 + (tok - first);  // output row of the record's token 0 (it may not be wanted)
  // lane: rows 2 i + hi, 8 channels from 8 c
  const int c = lane & 15, hi = lane >> 4;
  const int k_at = kv4_k_code(hi, c >> 2) + (c & 3) * 4, v_at = kv4_v_code(hi, c >> 1) + (c & 1) * 4;
  const int k_sc = kv4_k_scale(hi, c >> 2), v_sc = kv4_v_scale(0, c >> 1);
  const int k_sh = ((c >> 1) & 1) * 8, v_sh = hi * 8;
  struct Plane {
    uint32_t codes[8], scales[4];
  };
  auto load = [&](int pl, Plane& x) {
    const bool is_k = pl < KP;
    const uint8_t* p = rec + pl * kKv4Plane;
#pragma unroll
    for (int i = 0; i < 8; ++i)  // tokens 2 i + hi: a quad of tokens is 128 (K) or 16 (V) bytes on, its second half 512
      x.codes[i] = *reinterpret_cast<const uint32_t*>(p + (is_k ? k_at + (i >> 1) * 128 : v_at + (i >> 1) * 16) + (i & 1) * 512);
#pragma unroll
    for (int i = 0; i < 4; ++i)  // a quad's scales: K's two rows by two blocks, V's four rows
      x.scales[i] = *reinterpret_cast<const uint32_t*>(p + (is_k ? k_sc + i * 32 : v_sc + i * 4));
  };
  auto store = [&](int pl, const Plane& x) {
    const bool is_k = pl < KP;
    const float mul = is_k ? a.k_mul : a.v_mul;
    const int shift = is_k ? k_sh : v_sh;
    __nv_bfloat16* out = (is_k ? a.k_out + pl * 128 : a.v_out + (pl - KP) * 128) + c * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int key = 2 * i + hi;
      if (tok + key < first || tok + key >= end || !dbg_index_ok(row0 + key, a.total)) continue;
      const float s = e4m3_to_float((x.scales[i >> 1] >> (shift + 16 * (i & 1))) & 0xffu) * mul;
      uint32_t v[4];
      e2m1x8_to_half2(x.codes[i], v);
      *reinterpret_cast<uint4*>(out + (static_cast<size_t>(row0 + key) * a.H + h) * (KP * 128)) =
          make_uint4(half2_to_bf16x2(v[0], s), half2_to_bf16x2(v[1], s), half2_to_bf16x2(v[2], s), half2_to_bf16x2(v[3], s));
    }
  };
  Plane x[2];
  load(0, x[0]);
#pragma unroll
  for (int pl = 0; pl < 2 * KP; ++pl) {
    if (pl + 1 < 2 * KP) load(pl + 1, x[(pl + 1) & 1]);
    store(pl, x[pl & 1]);
  }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  const long long warps = (static_cast<long long>(a.total) + 7) / 8 * a.H;
  const unsigned blocks = static_cast<unsigned>((warps * 32 + kAppendThreads - 1) / kAppendThreads);
  return launch_early(a.kp == 1 ? kv4_append_kernel<1> : kv4_append_kernel<2>, blocks, kAppendThreads, 0, st, 1, a);
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  const long long warps = (a.total / 16 + 2LL * a.B) * a.H;
  const unsigned blocks = static_cast<unsigned>((warps * 32 + kGatherThreads - 1) / kGatherThreads);
  return launch_early(a.kp == 1 ? kv4_gather_kernel<1> : kv4_gather_kernel<2>, blocks, kGatherThreads, 0, st, 1, a);
}

cudaError_t status_kv4_rows(int* v) { return launched_status(v); }

}  // namespace da
