// rope.cu -- rotary positions: diffattn_rope turns queries and keys (and, backward, their gradients),
// diffattn_rope_append and diffattn_rope_kv4_append write turned keys and values into pages on the way.
//
// A row of a head is made of parts of d channels, whose first 2 P are P pairs:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,   (c, s) = table[position on the pair's axis][pair].
//
// What bounds it: the rows' bytes, read and written once (and 8 P bytes of table a token, shared by all
// heads). A warp takes a token: its lanes hold the cosines and sines of 8 pairs each in registers, for all
// heads that the warp goes through, and 16 channels of a part, so that a load or store of the warp is whole
// pieces of 128 bytes. Where the tokens are few, a token's parts are dealt out over several warps.
//
// A bf16 result is the fp64 sum of the two products (which are exact in fp64) rounded to bf16, so that the three
// calls agree in every bit, and the 4-bit codes, which have borders too, are those of these keys' bf16. In fp32 a
// value is off by at most t = 2^-24 (|x2 s| + |y|); where y - 2t and y + 2t round to the same bf16 (all but one in
// some 2^12), that is the fp64 sum's; else the sum is formed.
#include <type_traits>

#include "early.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {
namespace {

// Parts that a lane has under way, and blocks an SM. More parts take registers from warps, whose chains of position,
// table and rows are what is waited for. (16384 tokens of 24 heads of 256 channels, backward / 16400 of 64 + 8 heads
// into bf16 pages / 16384 of 12 + 12 of 256 into 4-bit pages and read back, us: 4 parts and 5 blocks 102, 140, 190;
// 3 and 6 91, 136, 177; 2 and 7 77, 124, 153; 2 and 8, which spills, 79, 127, 155; 1 and 8 85, 135, 151. The same
// bytes at a copy's rate: 60, 99, 105. Streaming hints change nothing.)
constexpr int kThreads = 128, kBlocks = 7;
constexpr int kAhead = 2;

// fp64 to bf16 in one rounding: cut to fp32 with the last bit set where anything was cut off ("round to
// odd"), which the second rounding then takes the right way.
__device__ __forceinline__ uint32_t bf16_of(double x) {
  float f = __double2float_rz(x);
  if (static_cast<double>(f) != x) f = __uint_as_float(__float_as_uint(f) | 1u);
  return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}
__device__ __noinline__ uint32_t turn_exact(float x1, float x2, float c, float s) {
  const double a = x1, b = x2, dc = c, ds = s;
  return bf16_of(a * dc - b * ds) | bf16_of(b * dc + a * ds) << 16;
}
// (y1, y2) of one pair, packed; `unsure` gets bits where it may not be the fp64 sum's rounding
__device__ __forceinline__ uint32_t turn_fast(float x1, float x2, float c, float s, uint32_t& unsure) {
  constexpr float kTwo = 1.f / (1 << 23);
  const float p1 = x2 * s, p2 = x2 * c;
  const float y1 = fmaf(x1, c, -p1), y2 = fmaf(x1, s, p2);
  const float t1 = fabsf(p1) + fabsf(y1), t2 = fabsf(p2) + fabsf(y2);
  const uint32_t lo = pack_bf16x2(fmaf(t1, -kTwo, y1), fmaf(t2, -kTwo, y2));
  const uint32_t hi = pack_bf16x2(fmaf(t1, kTwo, y1), fmaf(t2, kTwo, y2));
  unsure |= lo ^ hi;
  return lo;
}
// x1 c - x2 s to within 1.5 steps, whatever cancels (the first product's rounding error is put back: of an
// infinite product there is none, and Inf - Inf would make a NaN of the infinity that the formula gives)
__device__ __forceinline__ float turn_f32(float x1, float x2, float c, float s) {
  const float p = x2 * s, e = fmaf(-x2, s, p);
  return fmaf(x1, c, -p) + (fabsf(p) < INFINITY ? e : 0.f);
}

// 16 channels of a part as a lane holds them: two runs of 8 (bf16: one uint4 each, fp32: two)
template <typename T>
struct Item {
  static constexpr int kWords = 8 * sizeof(T) / 16;
  uint4 run[2][kWords];
};

// (One test for all eight pairs: a branch for each is more instructions than the turning.)
template <bool kInter>
__device__ __forceinline__ void turn(Item<__nv_bfloat16>& x, const float2 (&cs)[8]) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&x.run[0][0]);
  uint32_t* b = reinterpret_cast<uint32_t*>(&x.run[1][0]);
  // pair i of the item
  auto first = [&](int i) {
    if constexpr (kInter) return __uint_as_float((i < 4 ? a : b)[i & 3] << 16);  // a word is a pair
    else return __uint_as_float(i & 1 ? a[i >> 1] & 0xffff0000u : a[i >> 1] << 16);
  };
  auto second = [&](int i) {
    if constexpr (kInter) return __uint_as_float((i < 4 ? a : b)[i & 3] & 0xffff0000u);
    else return __uint_as_float(i & 1 ? b[i >> 1] & 0xffff0000u : b[i >> 1] << 16);
  };
  uint32_t y[8], unsure = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = turn_fast(first(i), second(i), cs[i].x, cs[i].y, unsure);
  if (unsure) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t mine = 0;
      turn_fast(first(i), second(i), cs[i].x, cs[i].y, mine);
      if (mine) y[i] = turn_exact(first(i), second(i), cs[i].x, cs[i].y);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = kInter ? y[i] : __byte_perm(y[2 * i], y[2 * i + 1], 0x5410);
    b[i] = kInter ? y[4 + i] : __byte_perm(y[2 * i], y[2 * i + 1], 0x7632);
  }
}
template <bool kInter>
__device__ __forceinline__ void turn(Item<float>& x, const float2 (&cs)[8]) {
  float* a = reinterpret_cast<float*>(&x.run[0][0]);
  float* b = reinterpret_cast<float*>(&x.run[1][0]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x1 = kInter ? (i < 4 ? a : b)[2 * (i & 3)] : a[i];
    float& x2 = kInter ? (i < 4 ? a : b)[2 * (i & 3) + 1] : b[i];
    const float y1 = turn_f32(x1, x2, cs[i].x, cs[i].y), y2 = turn_f32(x2, x1, cs[i].x, -cs[i].y);
    x1 = y1, x2 = y2;
  }
}

// Where a tensor's rows lie: part `r` of a token's row (head h = r / parts) from its first channel
template <typename T>
__device__ __forceinline__ T* part_of(const RopeRows& t, long long token, int r, int h, int parts, int d) {
  return static_cast<T*>(t.data) + token * t.token + h * t.head + (r - h * parts) * d;
}
__device__ __forceinline__ int quotient(int j, uint32_t magic, uint32_t shift) { return (__umulhi(j, magic) + j) >> shift; }

// kPages 0: rows to rows; 1: keys and values to bf16 pages; 2: to 4-bit pages (the values by warps of
// their own, 8 rows of a head each).
template <typename T, bool kInter, int kPages>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const RopeArgs a) {
  grid_wait();
  grid_release();
  const int lane = threadIdx.x & 31;
  long long w = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const long long rope_warps = static_cast<long long>(a.total) * a.split;

  // (`s` is loaded with the position, not behind it)
  auto raw_slot = [&](long long row) { return row < a.total ? *(a.slot_map + row) : -1; };
  auto slot_of = [&](int s) {
    if (s >= 0 && s < a.num_pages * a.page_size) return s;
    if (s != -1) flag_device_error(DEV_BAD_INDEX);
    return -1;
  };
  // whether a token has its places on all axes; one at -1 is left out
  auto placed = [&](long long row) {
    if (row >= a.total) return false;
    for (int x = 0; x < a.n_axes; ++x) {
      const int p = *(a.positions + x * static_cast<long long>(a.total) + row);
      if (p < 0 || p >= a.top) {
        if (p != -1) flag_device_error(DEV_BAD_INDEX);
        return false;
      }
    }
    return true;
  };

  if constexpr (kPages == 2) {
    if (w >= rope_warps) {
      // Values: lane (2 rows of 4, block g of 16 channels). Two rows whose slots are the two of a pair are
      // one 16-byte piece of the record.
      w -= rope_warps;
      const int h = static_cast<int>(w % a.H), g = lane & 7;
      const long long row = w / a.H * 8 + 2 * (lane >> 3);
      const int raw0 = raw_slot(row), raw1 = raw_slot(row + 1);
      const int s0 = placed(row) ? slot_of(raw0) : -1, s1 = placed(row + 1) ? slot_of(raw1) : -1;
      const int vp = a.vw >> 7;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.v.data) + row * a.v.token + h * a.v.head + g * 16;
      auto place = [&](int slot) {
        const int page = slot / a.page_size, off = slot - page * a.page_size;
        return static_cast<uint8_t*>(a.k_dst) +
               ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) *
                   static_cast<size_t>((a.kw + a.vw) / 128 * kKv4Plane) + (a.kw >> 7) * kKv4Plane;
      };
      const bool joined = s0 >= 0 && s1 == s0 + 1 && (s0 & 1) == 0;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint8_t *d0 = place(max(s0, 0)), *d1 = place(max(s1, 0));
      for (int pl = 0; pl < vp; ++pl, d0 += kKv4Plane, d1 += kKv4Plane, src += 128) {
        uint4 c[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          c[i] = s0 >= 0 ? *(reinterpret_cast<const uint4*>(src) + i) : zero;
          c[2 + i] = s1 >= 0 ? *(reinterpret_cast<const uint4*>(src + a.v.token) + i) : zero;
        }
        const Kv4Block x = kv4_round_block(c[0], c[1], a.v_inv), y = kv4_round_block(c[2], c[3], a.v_inv);
        if (joined) {
          *reinterpret_cast<uint4*>(d0 + kv4_v_code(s0 & 15, g)) = make_uint4(x.lo, x.hi, y.lo, y.hi);
          *reinterpret_cast<uint16_t*>(d0 + kv4_v_scale(s0 & 15, g)) = static_cast<uint16_t>(x.scale | (y.scale << 8));
        } else {
          if (s0 >= 0) {
            *reinterpret_cast<uint2*>(d0 + kv4_v_code(s0 & 15, g)) = make_uint2(x.lo, x.hi);
            d0[kv4_v_scale(s0 & 15, g)] = static_cast<uint8_t>(x.scale);
          }
          if (s1 >= 0) {
            *reinterpret_cast<uint2*>(d1 + kv4_v_code(s1 & 15, g)) = make_uint2(y.lo, y.hi);
            d1[kv4_v_scale(s1 & 15, g)] = static_cast<uint8_t>(y.scale);
          }
        }
      }
      return;
    }
  }
  if (w >= rope_warps) return;
  const long long token = w / a.split;
  const int share = static_cast<int>(w - token * a.split);
  int raw = -1;
  if constexpr (kPages != 0) raw = raw_slot(token);
  if (!placed(token)) return;

  // lane: item `it` (16 channels) of slot `sl` of the parts that the warp has in hand
  const int items = a.d >> 4, slots = 32 / items, it = lane & (items - 1), sl = lane / items;
  const bool turns = it * 8 < a.pairs;
  // its two runs of 8 channels: of pairs 8 it .. 8 it + 7, or of what stays as it is
  const int run0 = kInter || !turns ? it * 16 : it * 8, run1 = kInter || !turns ? run0 + 8 : run0 + a.pairs;
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = make_float2(1.f, 0.f);
  if (turns) {
    if (a.n_axes == 1) {  // 64 bytes on end
      const float4* row = reinterpret_cast<const float4*>(a.table + static_cast<size_t>(*(a.positions + token)) * a.pairs + it * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *(row + i);
        cs[2 * i] = make_float2(v.x, v.y), cs[2 * i + 1] = make_float2(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int x = *(a.axes + it * 8 + i);
        if (x < 0 || x >= a.n_axes) {
          flag_device_error(DEV_BAD_INDEX);
          x = 0;
        }
        const int p = *(a.positions + x * static_cast<long long>(a.total) + token);
        cs[i] = *(a.table + static_cast<size_t>(p) * a.pairs + it * 8 + i);
      }
    }
    if (a.inverse) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i].y = -cs[i].y;
    }
  }

  // n parts, kAhead of them at a time, from where `source` says
  auto rows = [&](int n, bool rotate, auto&& source, auto&& store) {
    const int step = slots * a.split;
    for (int r0 = share * slots + sl; r0 - sl < n; r0 += step * kAhead) {
      Item<T> x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int r = r0 + u * step;
        if (r < n) {
          const T* src = source(r);
#pragma unroll
          for (int i = 0; i < Item<T>::kWords; ++i) {
            x[u].run[0][i] = *(reinterpret_cast<const uint4*>(src + run0) + i);
            x[u].run[1][i] = *(reinterpret_cast<const uint4*>(src + run1) + i);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int r = r0 + u * step;
        if (rotate && turns && r < n) turn<kInter>(x[u], cs);
        store(x[u], r, r < n);
      }
    }
  };
  auto put = [&](T* dst, const Item<T>& x) {
#pragma unroll
    for (int i = 0; i < Item<T>::kWords; ++i) {
      *(reinterpret_cast<uint4*>(dst + run0) + i) = x.run[0][i];
      *(reinterpret_cast<uint4*>(dst + run1) + i) = x.run[1][i];
    }
  };
  const int parts = a.kw / a.d, nq = a.hq * parts, nk = a.H * parts;
  auto head = [&](int r) { return quotient(r, a.kw_magic, a.kw_shift); };
  auto q_or_k = [&](const RopeRows& q, const RopeRows& k, int r) {
    const bool is_k = r >= nq;
    const int i = is_k ? r - nq : r;
    return part_of<T>(is_k ? k : q, token, i, head(i), parts, a.d);
  };
  if constexpr (kPages == 0) {
    rows(nq + nk, true, [&](int r) { return q_or_k(a.q, a.k, r); },
         [&](const Item<T>& x, int r, bool live) {
           if (live) put(q_or_k(a.q_out, a.k_out, r), x);
         });
  } else {
    const int slot = slot_of(raw);
    if constexpr (kPages == 1) {
      const RopeRows k_out{static_cast<T*>(a.k_dst) + static_cast<size_t>(max(slot, 0)) * a.H * a.kw, 0, a.kw};
      rows(slot < 0 ? nq : nq + nk, true, [&](int r) { return q_or_k(a.q, a.k, r); },
           [&](const Item<T>& x, int r, bool live) {
             if (live) put(q_or_k(a.q_out, k_out, r), x);
           });
      if (slot < 0) return;
      const int vparts = a.vw / a.d;
      rows(a.H * vparts, false,
           [&](int r) { return part_of<T>(a.v, token, r, quotient(r, a.vw_magic, a.vw_shift), vparts, a.d); },
           [&](const Item<T>& x, int r, bool live) {
             if (live) put(static_cast<T*>(a.v_dst) + static_cast<size_t>(slot) * a.H * a.vw + static_cast<size_t>(r) * a.d, x);
           });
    } else {
      rows(nq, true, [&](int r) { return part_of<T>(a.q, token, r, head(r), parts, a.d); },
           [&](const Item<T>& x, int r, bool live) {
             if (live) put(part_of<T>(a.q_out, token, r, head(r), parts, a.d), x);
           });
      if (slot < 0) return;
      const int page = slot / a.page_size, off = slot - page * a.page_size, key = off & 15;
      const size_t rec = static_cast<size_t>((a.kw + a.vw) / 128 * kKv4Plane);
      rows(nk, true, [&](int r) { return part_of<T>(a.k, token, r, head(r), parts, a.d); },
           [&](const Item<T>& x, int r, bool live) {
        // a lane wants 16 channels on end: where its runs are of two blocks, it trades one with its neighbour
        uint4 lo = x.run[0][0], hi = x.run[1][0];
        int blk = it;
        if (!kInter) {
          const bool odd = it & 1;
          const uint4 give = odd ? lo : hi;
          uint4 got;
          got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
          got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
          got.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
          got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
          if (turns) {
            if (odd) lo = got;
            else hi = got;
            blk = (it >> 1) + (odd ? a.pairs >> 4 : 0);
          }
        }
        const Kv4Block b = kv4_round_block(lo, hi, a.k_inv);
        if (!live) return;
        const int h = head(r);
        uint8_t* p = static_cast<uint8_t*>(a.k_dst) + ((static_cast<size_t>(page) * a.H + h) * (a.page_size >> 4) + (off >> 4)) * rec +
                     (r - h * parts) * kKv4Plane;
        *reinterpret_cast<uint2*>(p + kv4_k_code(key, blk >> 1) + 8 * (blk & 1)) = make_uint2(b.lo, b.hi);
        p[kv4_k_scale(key, blk >> 1) + (blk & 1)] = static_cast<uint8_t>(b.scale);
      });
    }
  }
}

// cos and sin of position * frequency, in fp64 and rounded once
__global__ void __launch_bounds__(256) rope_table_kernel(const RopeTableArgs a) {
  grid_wait();
  grid_release();
  const long long n = static_cast<long long>(a.top) * a.pairs;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const int p = static_cast<int>(i / a.pairs);
    double c, s;
    sincos(static_cast<double>(p) * *(a.freq + (i - static_cast<long long>(p) * a.pairs)), &s, &c);
    a.table[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
  }
}

}  // namespace

template <typename T, int kPages>
static cudaError_t launch(const RopeArgs& a, bool interleaved, unsigned blocks, cudaStream_t st) {
  return launch_early(interleaved ? rope_kernel<T, true, kPages> : rope_kernel<T, false, kPages>, blocks, kThreads, 0, st, 1, a);
}

cudaError_t launch_rope(RopeArgs a, int pages, bool fp32, bool interleaved, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  // warps of a token: as many as give each of the 152 SMs 16, but not more than its rows have work for
  const int slots = 512 / a.d;
  const int heads = pages == 2 ? (a.hq > a.H ? a.hq : a.H) : a.hq + a.H;
  const int most = (heads * (a.kw / a.d) + slots - 1) / slots;
  page_magic(a.kw / a.d, &a.kw_magic, &a.kw_shift);
  page_magic(pages ? a.vw / a.d : 1, &a.vw_magic, &a.vw_shift);
  const long long want = (152 * 16 + a.total - 1) / a.total;
  a.split = static_cast<int>(want < 1 ? 1 : want > most ? most : want);
  if (a.split < 1) a.split = 1;
  long long warps = static_cast<long long>(a.total) * a.split;
  if (pages == 2) warps += (static_cast<long long>(a.total) + 7) / 8 * a.H;
  const unsigned blocks = static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads);
  if (fp32) return launch<float, 0>(a, interleaved, blocks, st);
  return pages == 0   ? launch<__nv_bfloat16, 0>(a, interleaved, blocks, st)
         : pages == 1 ? launch<__nv_bfloat16, 1>(a, interleaved, blocks, st)
                      : launch<__nv_bfloat16, 2>(a, interleaved, blocks, st);
}

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t st) {
  const long long n = static_cast<long long>(a.top) * a.pairs;
  if (n == 0) return cudaSuccess;
  const long long blocks = (n + 255) / 256;
  return launch_early(rope_table_kernel, static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, st, 1, a);
}

cudaError_t status_rope(int* v) { return launched_status(v); }

}  // namespace da
