// kv4_chunk.cuh -- chunks over the 4-bit cache: the batch's units (a KV head, a sequence and a tile of its new
// tokens each), one behind the other, cut into ranges of equal cost. Shared by the kernels that attend
// (chunk_kv4.cu, chunk_kv4_few.cu) and the one that joins the pieces of units that are cut.
#pragma once
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {

constexpr int kChunkSms = 152;
constexpr int kMinCost = 2;  // the smallest range, in tiles of keys

struct Walk {  // place in the walk over units: sequences, heads, tiles of tokens
  int b, h, rt, q0, Lq, Lk, nrt;
  int tile, tiles;
  long long todo;  // tiles of the range, and the costs of the units that begin in it, from here on
};

// ---- the batch's units -------------------------------------------------------------------------
struct Seq {
  int q0, Lq, Lk;
};
// kEarly: before grid_wait(), in a kernel that knows of the write by the release of the one before it
template <bool kEarly>
__device__ __forceinline__ int ld(const int* p) {
  return kEarly ? __ldcg(p) : *p;
}
template <bool kEarly>
__device__ __forceinline__ Seq sequence(const Kv4ChunkArgs& a, int b, bool report = false) {
  Seq s{ld<kEarly>(a.cu_seqlens + b), 0, 0};
  const int end = ld<kEarly>(a.cu_seqlens + b + 1), n = ld<kEarly>(a.seqlens + b), cap = a.max_pages * a.page_size;
  if (s.q0 < 0 || end < s.q0 || end > a.total) {
    if (report) flag_device_error(DEV_BAD_INDEX);
    return s;
  }
  s.Lq = end - s.q0;
  s.Lk = n < 0 ? 0 : n > cap ? cap : n;
  return s;
}
// leading tokens that see no key
__device__ __forceinline__ int hidden(const Kv4ChunkArgs& a, const Seq& s) {
  return s.Lk == 0 ? s.Lq : a.causal ? max(0, s.Lq - s.Lk) : 0;
}
__device__ __forceinline__ int tiles_of(const Kv4ChunkArgs& a, int Lq, int Lk, int rt) {
  const int end = a.causal ? Lk - Lq + min(Lq, (rt + 1) << a.tok_log2) : Lk;
  return (end + (1 << a.tile_log2) - 1) >> a.tile_log2;
}
// of one head
template <bool kEarly>
__device__ __forceinline__ long long cost_of(const Kv4ChunkArgs& a, int b, bool report) {
  const Seq s = sequence<kEarly>(a, b, report);
  const int z = hidden(a, s), n = (s.Lq + a.tokens - 1) >> a.tok_log2;
  if (z >= s.Lq) return 0;
  long long sum = 0;
#pragma unroll 1
  for (int rt = z >> a.tok_log2; rt < n; ++rt) sum += tiles_of(a, s.Lq, s.Lk, rt) + a.unit_cost;
  return sum;
}
// the first unit of sequence w.b, head w.h; false: it has none
template <bool kEarly>
__device__ __forceinline__ bool enter(const Kv4ChunkArgs& a, Walk& w) {
  const Seq s = sequence<kEarly>(a, w.b);
  const int z = hidden(a, s);
  w.q0 = s.q0, w.Lq = s.Lq, w.Lk = s.Lk;
  w.nrt = (s.Lq + a.tokens - 1) >> a.tok_log2;
  w.rt = z >> a.tok_log2;
  w.tile = 0;
  if (z >= s.Lq) return false;
  w.tiles = tiles_of(a, s.Lq, s.Lk, w.rt);
  return true;
}
__device__ __forceinline__ void next_unit(const Kv4ChunkArgs& a, Walk& w) {
  w.todo -= a.unit_cost;
  if (w.todo <= 0) return;
  if (++w.rt < w.nrt) {
    w.tile = 0;
    w.tiles = tiles_of(a, w.Lq, w.Lk, w.rt);
    return;
  }
  if (++w.h < a.H) {
    enter<false>(a, w);
    return;
  }
  w.h = 0;
  do {
    if (++w.b >= a.B) {
      w.todo = 0;
      return;
    }
  } while (!enter<false>(a, w));
}
// `n` tiles of the unit are done
__device__ __forceinline__ void advance(const Kv4ChunkArgs& a, Walk& w, int n) {
  w.tile += n;
  w.todo -= n;
  if (w.tile == w.tiles) next_unit(a, w);
}

// x / y for 0 <= x, 0 < y: one copy of the code, and nearly always both have 32 bits. (All of this is run once a
// launch or unit, cold: what counts is that it is short.)
static __device__ __noinline__ long long quotient64(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
__device__ __forceinline__ int range_count(long long total, int grid) {
  const long long want = total / kMinCost;
  return static_cast<int>(want < 1 ? 1 : want > grid ? grid : want);
}
__device__ __forceinline__ long long range_start(long long total, int n, int i) {
  const long long each = quotient64(total, n);
  return each * i + quotient64((total - each * n) * i, n);
}
// the range that holds x < total: the largest i with total i / n < x + 1
__device__ __forceinline__ int range_of(long long total, int n, long long x) {
  return static_cast<int>(quotient64((x + 1) * n - 1, total));
}

// The costs before each thread's share of the sequences; a whole block of NT threads. Returns their sum.
template <int NT, bool kEarly>
__device__ __forceinline__ long long fill(const Kv4ChunkArgs& a, long long* pre, long long* sum, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (a.B + NT - 1) / NT;
  const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
  long long incl = 0;
#pragma unroll 1
  for (int b = lo; b < hi; ++b) incl += cost_of<kEarly>(a, b, report);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sum[warp] = incl;
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < warp; ++w) incl += sum[w];
  pre[tid + 1] = incl;
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  return pre[NT] * a.H;
}
// The unit that holds place t0 of all costs (a whole warp). w.tile: the first tile at or behind t0; `first`:
// where the unit's tiles begin.
template <int NT, bool kEarly>
__device__ __forceinline__ void locate(const Kv4ChunkArgs& a, const long long* pre, long long t0, Walk& w, long long& first) {
  const int lane = threadIdx.x & 31, per = (a.B + NT - 1) / NT;
  w = Walk{};
  int share = 0;
#pragma unroll 1
  for (int i = 0; i < NT; i += 32)
    if (const unsigned hit = __ballot_sync(0xffffffffu, pre[i + lane] * a.H <= t0 && t0 < pre[i + lane + 1] * a.H)) {
      share = i + __ffs(hit) - 1;
      break;
    }
  long long at = pre[share], cost = 0;
  const int end = min(a.B, (share + 1) * per);
#pragma unroll 1
  for (int b = share * per; b < end; ++b) {
    cost = per == 1 ? pre[share + 1] - pre[share] : cost_of<kEarly>(a, b, false);
    w.b = b;
    if (t0 < (at + cost) * a.H) break;
    at += cost;
  }
  long long left = t0 - at * a.H;  // in the sequence
  w.h = static_cast<int>(quotient64(left, cost));
  left -= w.h * cost;
  enter<kEarly>(a, w);
#pragma unroll 1
  for (int rt = w.rt;; rt += 32) {  // 32 tiles of tokens at a time
    const int mine = rt + lane < w.nrt ? tiles_of(a, w.Lq, w.Lk, rt + lane) + a.unit_cost : 0;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, left < incl);
    if (hit || rt + 32 >= w.nrt) {
      const int l = hit ? __ffs(hit) - 1 : 0;
      w.rt = rt + l;
      w.tiles = __shfl_sync(0xffffffffu, mine, l) - a.unit_cost;
      left -= __shfl_sync(0xffffffffu, incl - mine, l);
      break;
    }
    left -= __shfl_sync(0xffffffffu, incl, 31);
  }
  first = t0 - left + a.unit_cost;
  w.tile = static_cast<int>(max(0LL, left - a.unit_cost));
}

// Joins the pieces of units that are cut: behind the kernel that attends, with the same `a`.
cudaError_t launch_kv4_chunk_join(const Kv4ChunkArgs& a, cudaStream_t st);
// Whether the kernel for few new tokens takes the call, and its launch, with the join.
bool kv4_chunk_few(const Kv4ChunkArgs& a);
cudaError_t launch_kv4_chunk_few(Kv4ChunkArgs a, cudaStream_t st);

}  // namespace da
