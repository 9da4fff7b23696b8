// chunk_kv4.cu -- attention of chunks over the 4-bit cache: each sequence's new tokens, the last of its
// positions, over all its cached keys (V1: both maps of a head; V2: the query heads of a KV head's group).
//
// A unit is a KV head, a sequence and a tile of its new tokens: R columns (64 or 128), a column being one
// softmax (V2: column G t + g is query head g of token t; V1: column m T + t is map m of token t). Over the
// keys, 128 at a time, everything is held transposed, keys or channels on the 128 lanes of tensor memory:
//   S^T [128 keys x R] = K Q^T              (V1: map m's columns by the K plane of map m)
//   P = 2^(s c - m),  l += P                (column by column: m a reference, c the scale)
//   O^T [128 channels x R] += V^T P         (V1: two planes of channels)
// so that a product costs what its columns cost: few new tokens leave the machine to the loads, and V1's
// maps multiply no zeros, which rows of both maps over one K of 256 channels would. At the end V1:
// o1/l1 - lambda o2/l2, the norm and the scale, V2: o_2p/l_2p - sigmoid(lam) o_2p+1/l_2p+1.
//
// Warps. 8 for the softmax: warpgroup w has half of the columns (w R/2 ..), thread `key` one key of the
// tile, so its P go to shared memory as whole pieces of 16 bytes, over the K plane that S came from. 4
// unpack: they read records into registers, four planes ahead, and write K and V as fp16 (exact: an e2m1
// times an e4m3 has 6 significant bits) in the products' 128-byte swizzle. One issues the products: S of
// the next tile before P V of this one.
//
// Numerics, as in the decode over the same cache: the query enters as fp16 after a power of two of its own
// for each column, P is rounded to fp16 at 2^10 times its value against m, which moves only where a score
// passes it by 2^4 (the whole warpgroup then finds the columns' new references and rescales O and l).
// Sums and statistics are fp32. Keys that a column may not see have P = 0, and a V block that is NaN is held
// as zeros and its first key noted: the columns that see that key get NaN at the end, the others nothing.
//
// Work. All units one behind the other are cut into equal ranges of tiles, one for each SM; pieces of units
// that are cut go to the workspace, at most two a range, and a second kernel joins them in the order of the
// ranges, so that equal inputs give equal bits.
#include <cfloat>
#include <cmath>

#include "early.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kSms = 152;
constexpr int kSoftmaxWarps = 8, kUnpackWarps = 4, kMmaWarp = kSoftmaxWarps + kUnpackWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;
// Registers a thread: the launch's 128, dealt out anew to the warpgroups (2 x 160 + 120 + 72 of 4 x 128).
constexpr int kSoftmaxRegs = 160, kUnpackRegs = 120, kMmaRegs = 72;
static_assert(2 * kSoftmaxRegs + kUnpackRegs + kMmaRegs <= 4 * 128, "more registers than the launch has");
constexpr int kTile = 128;                       // keys
constexpr int kSlot = kTile * 128 * 2;           // one plane of a tile in fp16
constexpr int kSlots = 6;
constexpr int kHalf = kSlot / 2;                 // 64 of its channels (or columns of P)
constexpr int kUnitCost = 3;                     // what a unit costs besides its tiles, in tiles
constexpr int kMinCost = 2;                      // the smallest range
constexpr float kPScale = 10.f, kMoveRef = 14.f;
constexpr int kNanSets = 4;

template <int KP, int R>
struct Cfg {
  static constexpr int kHalfCols = R / 2;
  static constexpr int kQRows = KP == 1 ? R : R / 2;  // rows of one product's Q
  static constexpr int kQBytes = R * 256;
  static constexpr int kWidth = KP * 128;
  static constexpr int kO = 2 * R;                    // tensor memory: S twice, then O's planes
  static constexpr int kPiece = 2 * R + R * kWidth;   // floats: m, l, o
  static_assert(2 * R + KP * R <= 512, "tensor memory");
};

struct Small {  // behind the slots and Q
  float4 cm[64];       // columns 2i and 2i + 1: scales, and the references (less kPScale) negated
  int lim[128];        // keys that a column sees; 0 where there is no such token
  int top[128];        // a move: the columns' largest exponents (ordered), then the factors
  uint64_t full[kSlots], free[kSlots], s_full[2], p_full[2], pv_done[2], q_full, teardown;
  int nan_key[kNanSets][16];
  uint32_t tmem;
  int abort, seg;      // seg: tiles of the unit whose Q is there, 0 behind the last
};

struct Walk {  // place in the walk over units: sequences, heads, tiles of tokens
  int b, h, rt, q0, Lq, Lk, nrt;
  int tile, tiles;
  long long todo;  // tiles of the range, and the costs of the units that begin in it, from here on
};
// at startup, in Q's place
struct Scan {
  long long pre[kThreads + 1], sum[kThreads / 32];
  Walk walk;
  int ranges;
};
static_assert(sizeof(Scan) <= 64 * 256, "fits in the smaller Q");

template <int R>
constexpr int smem_bytes() {
  return kSlots * kSlot + R * 256 + static_cast<int>(sizeof(Small));
}
static_assert(smem_bytes<128>() <= 232448, "shared memory");

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
  const int end = ld<kEarly>(a.cu_seqlens + b + 1);
  if (s.q0 < 0 || end < s.q0 || end > a.total) {
    if (report) flag_device_error(DEV_BAD_INDEX);
    return s;
  }
  const int cap = a.max_pages * a.page_size, n = ld<kEarly>(a.seqlens + b);
  s.Lq = end - s.q0;
  s.Lk = n < 0 ? 0 : n > cap ? cap : n;
  return s;
}
// leading tokens that see no key
__device__ __forceinline__ int hidden(const Kv4ChunkArgs& a, const Seq& s) {
  return s.Lk == 0 ? s.Lq : a.causal ? max(0, s.Lq - s.Lk) : 0;
}
__device__ __forceinline__ int tiles_of(const Kv4ChunkArgs& a, int Lq, int Lk, int rt) {
  const int end = a.causal ? Lk - Lq + min(Lq, (rt + 1) * a.tokens) : Lk;
  return (end + kTile - 1) / kTile;
}
// of one head
template <bool kEarly>
__device__ __forceinline__ long long cost_of(const Kv4ChunkArgs& a, int b, bool report) {
  const Seq s = sequence<kEarly>(a, b, report);
  const int z = hidden(a, s), n = (s.Lq + a.tokens - 1) / a.tokens;
  if (z >= s.Lq) return 0;
  long long sum = 0;
  for (int rt = z / a.tokens; rt < n; ++rt) sum += tiles_of(a, s.Lq, s.Lk, rt) + kUnitCost;
  return sum;
}
// the first unit of sequence w.b, head w.h; false: it has none
template <bool kEarly>
__device__ __forceinline__ bool enter(const Kv4ChunkArgs& a, Walk& w) {
  const Seq s = sequence<kEarly>(a, w.b);
  const int z = hidden(a, s);
  w.q0 = s.q0, w.Lq = s.Lq, w.Lk = s.Lk;
  w.nrt = (s.Lq + a.tokens - 1) / a.tokens;
  w.rt = z / a.tokens;
  w.tile = 0;
  if (z >= s.Lq) return false;
  w.tiles = tiles_of(a, s.Lq, s.Lk, w.rt);
  return true;
}
__device__ __forceinline__ void next_unit(const Kv4ChunkArgs& a, Walk& w) {
  w.todo -= kUnitCost;
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

__device__ __forceinline__ int range_count(long long total, int grid) {
  const long long want = total / kMinCost;
  return static_cast<int>(want < 1 ? 1 : want > grid ? grid : want);
}
__device__ __forceinline__ long long range_start(long long total, int n, int i) {
  return total / n * i + total % n * i / n;
}
// the range that holds x < total: the largest i with total i / n < x + 1
__device__ __forceinline__ int range_of(long long total, int n, long long x) { return static_cast<int>(((x + 1) * n - 1) / total); }

// The costs before each thread's share of the sequences; a whole block of NT threads. Returns their sum.
template <int NT, bool kEarly>
__device__ __forceinline__ long long fill(const Kv4ChunkArgs& a, long long* pre, long long* sum, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (a.B + NT - 1) / NT;
  const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
  long long incl = 0;
  for (int b = lo; b < hi; ++b) incl += cost_of<kEarly>(a, b, report);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sum[warp] = incl;
  __syncthreads();
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
  for (int i = 0; i < NT; i += 32)
    if (const unsigned hit = __ballot_sync(0xffffffffu, pre[i + lane] * a.H <= t0 && t0 < pre[i + lane + 1] * a.H)) {
      share = i + __ffs(hit) - 1;
      break;
    }
  long long at = pre[share], cost = 0;
  const int end = min(a.B, (share + 1) * per);
  for (int b = share * per; b < end; ++b) {
    cost = per == 1 ? pre[share + 1] - pre[share] : cost_of<kEarly>(a, b, false);
    w.b = b;
    if (t0 < (at + cost) * a.H) break;
    at += cost;
  }
  long long left = t0 - at * a.H;  // in the sequence
  w.h = static_cast<int>(left / cost);
  left -= w.h * cost;
  enter<kEarly>(a, w);
  for (int rt = w.rt;; rt += 32) {  // 32 tiles of tokens at a time
    const int mine = rt + lane < w.nrt ? tiles_of(a, w.Lq, w.Lk, rt + lane) + kUnitCost : 0;
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
      w.tiles = __shfl_sync(0xffffffffu, mine, l) - kUnitCost;
      left -= __shfl_sync(0xffffffffu, incl - mine, l);
      break;
    }
    left -= __shfl_sync(0xffffffffu, incl, 31);
  }
  first = t0 - left + kUnitCost;
  w.tile = static_cast<int>(max(0LL, left - kUnitCost));
}

template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- small parts -------------------------------------------------------------------------------
__device__ __forceinline__ uint4 ldg128(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
// whether any of `count` threads of the block's barrier `id` has p
__device__ __forceinline__ bool barrier_any(uint32_t id, uint32_t count, bool p) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(p))
      : "memory");
  return any != 0;
}
// an order-preserving map of floats to ints; a NaN counts as the least
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return x != x ? INT_MIN : i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int i) {
  return i == INT_MIN ? -INFINITY : __int_as_float(i >= 0 ? i : i ^ 0x7fffffff);
}
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return umma_idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

// where a tile's planes lie, and the phase of their slot's use; j counts the block's tiles. V2: three stages
// of two slots. V1: two stages of three; P takes K1's slot and V2 takes K2's, so that of a stage's slots
// 0 and 1 the one that held K1 and P goes to V1 the next time.
template <int KP>
struct Place {
  int slot, phase;
};
template <int KP>
__device__ __forceinline__ Place<KP> place_k(int j, int map) {
  if constexpr (KP == 1) return {2 * (j % 3), (j / 3) & 1};
  if (map == 0) return {3 * (j & 1) + ((j >> 1) & 1), (j >> 1) & 1};
  return {3 * (j & 1) + 2, 0};
}
template <int KP>
__device__ __forceinline__ Place<KP> place_v(int j, int half) {
  if constexpr (KP == 1) return {2 * (j % 3) + 1, (j / 3) & 1};
  if (half == 0) return {3 * (j & 1) + 1 - ((j >> 1) & 1), (j >> 1) & 1};
  return {3 * (j & 1) + 2, 1};
}

template <int KP, int R>
__global__ void __launch_bounds__(kThreads, 1) kv4_chunk_kernel(const Kv4ChunkArgs a) {
  using C = Cfg<KP, R>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const s_q = smem + kSlots * kSlot;
  Small& sm = *reinterpret_cast<Small*>(s_q + C::kQBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t slots = smem_u32(smem), q_at = smem_u32(s_q);
  auto bar = [](uint64_t& x) { return smem_u32(&x); };

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(sm.full[i]), kUnpackWarps);
      mbar_init(bar(sm.free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sm.s_full[i]), 1);
      mbar_init(bar(sm.p_full[i]), kSoftmaxWarps);
      mbar_init(bar(sm.pv_done[i]), 1);
    }
    mbar_init(bar(sm.q_full), kSoftmaxWarps);
    mbar_init(bar(sm.teardown), 1);
    sm.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  for (int i = tid; i < kNanSets * 16; i += kThreads) sm.nan_key[i >> 4][i & 15] = INT_MAX;
  for (int i = tid; i < 128; i += kThreads) sm.top[i] = INT_MIN;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm.tmem), 512);
    tmem_relinquish();
  }
  grid_wait();
  grid_release();

  Walk w{};
  Scan& scan = *reinterpret_cast<Scan*>(s_q);
  {
    const long long total = fill<kThreads, false>(a, scan.pre, scan.sum, blockIdx.x == 0);
    const int n = range_count(total, a.grid), r = blockIdx.x;
    if (warp == 0) {
      long long first = 0;
      const long long t0 = range_start(total, n, r), t1 = r < n ? range_start(total, n, r + 1) : t0;
      if (t0 < t1) {
        locate<kThreads, false>(a, scan.pre, t0, w, first);
        w.todo = t1 - max(t0, first);
      }
      if (lane == 0) scan.walk = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    w = scan.walk;
    __syncthreads();  // Q's place is free
  }
  const uint32_t tmem = sm.tmem;
  volatile int* abrt = &sm.abort;

  if (warp >= kMmaWarp) {
    // ================================ products ================================
    registers_down<kMmaRegs>();
    if (warp == kMmaWarp && lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16(kTile, C::kQRows, 0, 0), idesc_o = idesc_f16(128, R, 1, 1);
      const uint64_t dk = umma_smem_desc(slots, 16, 1024), dq = umma_smem_desc(q_at, 16, 1024);
      const uint64_t dmn = umma_smem_desc(slots, kHalf, 1024);  // V and P: 64 channels or columns a half
      int j = 0;
      bool ok = true;
      auto scores = [&](int t) {
#pragma unroll
        for (int map = 0; map < KP; ++map) {
          const Place<KP> k = place_k<KP>(t, map);
          if (!(ok = ok && mbar_wait(bar(sm.full[k.slot]), k.phase, abrt))) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ss(tmem + (t & 1) * R + map * C::kQRows, desc_add(dk, k.slot * kSlot + (kk >> 2) * kHalf + (kk & 3) * 32),
                        desc_add(dq, map * C::kQRows * 256 + (kk >> 2) * C::kQRows * 128 + (kk & 3) * 32), idesc_s, kk > 0);
          if (map == 1) tc_commit(bar(sm.free[k.slot]));  // V1: K2's slot goes to V2
        }
        tc_commit(bar(sm.s_full[t & 1]));
      };
      for (int unit = 0; ok; ++unit) {
        if (!(ok = mbar_wait(bar(sm.q_full), unit & 1, abrt))) break;
        tc_fence_after();
        const int seg = *static_cast<volatile int*>(&sm.seg);
        if (seg == 0) break;
        scores(j);
        for (int i = 0; ok && i < seg; ++i, ++j) {
          if (i + 1 < seg) scores(j + 1);
          if (!ok) break;
          const Place<KP> p = place_k<KP>(j, 0);
          if (!(ok = mbar_wait(bar(sm.p_full[j & 1]), (j >> 1) & 1, abrt))) break;
#pragma unroll
          for (int half = 0; half < KP; ++half) {
            const Place<KP> v = place_v<KP>(j, half);
            if (!(ok = ok && mbar_wait(bar(sm.full[v.slot]), v.phase, abrt))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(tmem + C::kO + half * R, desc_add(dmn, v.slot * kSlot + kk * 2048),
                          desc_add(dmn, p.slot * kSlot + kk * 2048), idesc_o, i > 0 || kk > 0);
            tc_commit(bar(sm.free[v.slot]));
          }
          if (!ok) break;
          tc_commit(bar(sm.free[p.slot]));
          tc_commit(bar(sm.pv_done[j & 1]));
        }
      }
      // every product that was issued ends before tensor memory is given back
      tc_commit(bar(sm.teardown));
      mbar_wait(bar(sm.teardown), 0, nullptr);
    }
  } else if (warp >= kSoftmaxWarps) {
    // ================================ unpack ================================
    registers_down<kUnpackRegs>();
    // Warp u takes records u and u + 4 of each plane of a tile; a step is a plane.
    constexpr int kSteps = 4, kPerTile = 2 * KP;
    const int u = warp - kSoftmaxWarps;
    struct Step {
      uint4 lo[2], hi[2];
      uint32_t sc[2];
      int key0, left, unit;  // of the tile: its first key, keys from there on (0 or less: the stream has ended)
    };
    Step st[kSteps];
    const int recs = a.page_size >> 4;
    const size_t rec_bytes = static_cast<size_t>(2 * KP) * kKv4Plane;
    int unit = 0, page[2];
    const uint8_t* src[2];
    // the pages of this warp's records of the tile at w
    auto look_up = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = w.tile * kTile + (u + 4 * i) * 16;
        page[i] = w.todo > 0 && key < w.Lk && dbg_index_ok(key / a.page_size, a.max_pages)
                      ? *(a.block_table + static_cast<size_t>(w.b) * a.max_pages + key / a.page_size) : 0;
      }
    };
    auto issue = [&](Step& s, int plane) {
      if (plane == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rec = w.tile * 8 + u + 4 * i;
          if (page[i] < 0 || page[i] >= a.num_pages) {
            if (lane == 0) flag_device_error(DEV_BAD_INDEX);
            page[i] = 0;
          }
          src[i] = a.pool + ((static_cast<size_t>(page[i]) * a.H + w.h) * recs + rec % recs) * rec_bytes + lane * 16;
        }
      }
      s.key0 = w.tile * kTile;
      s.left = w.todo > 0 ? w.Lk - s.key0 : 0;
      s.unit = unit;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (s.left > (u + 4 * i) * 16) {
          const uint8_t* p = src[i] + plane * kKv4Plane;
          s.lo[i] = ldg128(p);
          s.hi[i] = ldg128(p + 512);
          s.sc[i] = *reinterpret_cast<const uint32_t*>(p - lane * 12 + kKv4PlaneCodes);
        } else {
          s.lo[i] = s.hi[i] = make_uint4(0, 0, 0, 0);
          s.sc[i] = 0;
        }
      }
      if (plane == kPerTile - 1 && w.todo > 0) {
        if (w.tile + 1 == w.tiles) ++unit;
        advance(a, w, 1);
        look_up();
      }
    };
    auto dup = [](uint32_t two, int high) { return __byte_perm(two, 0, high ? 0x3232 : 0x1010); };
    auto put = [](uint32_t at, uint32_t word, uint32_t scale) {
      uint32_t v[4];
      e2m1x8_to_half2(word, v);
      st_shared_v4(at, half2_mul(v[0], scale), half2_mul(v[1], scale), half2_mul(v[2], scale), half2_mul(v[3], scale));
    };
    auto unpack_k = [&](const Step& s, uint32_t slot) {
      const int ka = lane >> 3, r = (lane >> 2) & 1, t = lane & 3;
      const bool far = t & 2;  // its channels lie in the upper half: the pieces in another order, for the banks
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t s0, s1;
        e4m3x4_to_half2(s.sc[i], s0, s1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 w4 = h ? s.hi[i] : s.lo[i];
          const int in_rec = 4 * ka + 2 * h + r, row = (u + 4 * i) * 16 + in_rec;
          const bool live = row < s.left;
          const uint32_t sc = live ? (h ? s1 : s0) : 0u;
          const uint32_t a0 = dup(sc, far), a1 = dup(sc, !far);
          const uint32_t x0 = far ? w4.z : w4.x, x1 = far ? w4.w : w4.y, x2 = far ? w4.x : w4.z, x3 = far ? w4.y : w4.w;
          const uint32_t base = slot + (t >> 1) * kHalf + row * 128;
          const int c = ((t & 1) * 4 + (t & 2)) ^ (row & 7);
          put(base + (c << 4), x0, a0);
          put(base + ((c ^ 1) << 4), x1, a0);
          put(base + ((c ^ 2) << 4), x2, a1);
          put(base + ((c ^ 3) << 4), x3, a1);
        }
      }
    };
    auto unpack_v = [&](const Step& s, uint32_t slot, int half) {
      const int g = lane >> 2, t = lane & 3;
      const bool far = t & 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row0 = (u + 4 * i) * 16 + 4 * t;  // this lane's four tokens
        uint32_t sc = s.sc[i];
        const int live = s.left - row0;
        if (live < 4) sc = live <= 0 ? 0u : sc & (0xffffffffu >> (32 - 8 * live));
        const uint32_t odd = (((sc & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u);  // scales that are NaN
        if (odd) {
          atomicMin(&sm.nan_key[s.unit & (kNanSets - 1)][half * 8 + g], s.key0 + row0 + ((__ffs(odd) - 1) >> 3));
          sc &= ~((odd >> 7) * 0xffu);
        }
        uint32_t s01, s23;
        e4m3x4_to_half2(sc, s01, s23);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w4 = p ? s.hi[i] : s.lo[i];
          const uint32_t s2 = p ? s23 : s01;
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int row = row0 + 2 * p + jj;
            const uint32_t x0 = jj ? w4.z : w4.x, x1 = jj ? w4.w : w4.y, f = dup(s2, jj);
            const uint32_t base = slot + (g >> 2) * kHalf + row * 128;
            const int c = (((g & 3) * 2) ^ (row & 7)) ^ (far ? 1 : 0);
            put(base + (c << 4), far ? x1 : x0, f);
            put(base + ((c ^ 1) << 4), far ? x0 : x1, f);
          }
        }
      }
    };
    int j = 0;
    bool ok = true;
    look_up();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) issue(st[s], s % kPerTile);
    while (ok) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        constexpr int kTilesHere = kSteps / kPerTile;
        const int plane = s % kPerTile, t = j + s / kPerTile;
        static_assert(kTilesHere * kPerTile == kSteps, "whole tiles");
        if (st[s].left <= 0) {
          ok = false;
          break;
        }
        const Place<KP> d = plane < KP ? place_k<KP>(t, plane) : place_v<KP>(t, plane - KP);
        if (!__all_sync(0xffffffffu, mbar_wait(bar(sm.free[d.slot]), d.phase ^ 1, abrt))) {
          ok = false;
          break;
        }
        if (plane < KP) unpack_k(st[s], slots + d.slot * kSlot);
        else unpack_v(st[s], slots + d.slot * kSlot, plane - KP);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.full[d.slot]));
        issue(st[s], plane);
      }
      j += kSteps / kPerTile;
    }
  } else {
    // ================================ softmax ================================
    registers_up<kSoftmaxRegs>();
    const int wg = warp >> 2, quarter = warp & 3, key = quarter * 32 + lane, wtid = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    constexpr int NC = C::kHalfCols;
    const int col0 = wg * NC;
    const uint32_t cm_at = smem_u32(sm.cm) + wg * NC * 8;
    bool ok = true;
    int j = 0, unit = 0;
    // tokens that see no key get zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const Seq s = sequence<false>(a, b);
      const int z = hidden(a, s);
      const size_t row = static_cast<size_t>(a.H) * (KP == 2 ? 256 : a.group * 64);
      uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + s.q0 * row);
      for (size_t i = tid; i < z * row / 8; i += kSoftmaxWarps * 32) out[i] = make_uint4(0, 0, 0, 0);
    }
    while (w.todo > 0) {
      const int seg = static_cast<int>(min(static_cast<long long>(w.tiles - w.tile), w.todo));
      const bool starts = w.tile == 0, whole = starts && seg == w.tiles;
      const int tok0 = w.rt * a.tokens, toks = min(a.tokens, w.Lq - tok0);  // tokens of the unit
      const int edge = a.causal ? w.Lk - w.Lq + tok0 + 1 : w.Lk;            // keys that its first token sees
      // Q, with 256 / R threads for a column
      {
        constexpr int TPR = 256 / R, kPieces = 16 / TPR;  // 16-byte pieces for a thread
        const int col = tid / TPR, part = tid % TPR;
        const int t = KP == 2 ? col % C::kQRows : col / a.group, sub = KP == 2 ? col / C::kQRows : col % a.group;
        const bool live = t < toks;
        const size_t row = KP == 2 ? (static_cast<size_t>(w.q0 + tok0 + t) * a.H + w.h) * 2 + sub
                                   : static_cast<size_t>(w.q0 + tok0 + t) * a.H * a.group + w.h * a.group + sub;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + row * 128) + part * kPieces;
        uint4 x[kPieces];
        uint32_t top = 0;  // the largest magnitude's bits (ordered as the values are)
#pragma unroll
        for (int i = 0; i < kPieces; ++i) x[i] = live ? *(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const uint32_t m2 = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                       __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
          top = max(top, max(m2 & 0xffffu, m2 >> 16));
        }
#pragma unroll
        for (int d = 1; d < TPR; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = max(static_cast<int>(top >> 7) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);  // 2^(14 - e)
        // (never 0 or Inf, which a score of 0 or a masked one's Inf would turn into NaN)
        const float down = fminf(fmaxf(ldexpf(a.qk_scale, e - 14), FLT_MIN), FLT_MAX);
        auto two = [&](uint32_t v) { return pack_half2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up); };
        const int qrow = KP == 2 ? t : col;
        const uint32_t base = q_at + (KP == 2 ? sub * C::kQRows * 256 : 0) + qrow * 128;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int p = part * kPieces + i;  // of 16: 8 in each half of the channels
          st_shared_v4(base + (p >> 3) * C::kQRows * 128 + (((p & 7) ^ (qrow & 7)) << 4), two(x[i].x), two(x[i].y), two(x[i].z),
                       two(x[i].w));
        }
        if (part == 0) {
          float* cm = reinterpret_cast<float*>(&sm.cm[col >> 1]) + (col & 1);
          cm[0] = live ? down : 0.f;
          cm[2] = live ? FLT_MAX : 0.f;
          sm.lim[col] = !live ? 0 : a.causal ? max(0, w.Lk - w.Lq + tok0 + t + 1) : w.Lk;
        }
        if (tid == 0) sm.seg = seg;
        fence_proxy_async_smem();
        named_barrier_sync(1, kSoftmaxWarps * 32);
        if (lane == 0) mbar_arrive(bar(sm.q_full));
      }
      uint64_t l2[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l2[i] = 0;

      for (int i = 0; i < seg; ++i, ++j) {
        const int key0 = (w.tile + i) * kTile;
        ok = ok && mbar_wait(bar(sm.s_full[j & 1]), (j >> 1) & 1, abrt);
        __syncwarp();
        tc_fence_after();
        float e[NC];
        const uint32_t s_at = tmem + lanes + (j & 1) * R + col0;
        auto load = [&]() {
          uint32_t raw[NC / 32][32];
#pragma unroll
          for (int c = 0; c < NC / 32; ++c) tmem_ld32(s_at + 32 * c, raw[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NC; ++c) e[c] = __uint_as_float(raw[c >> 5][c & 31]);
        };
        auto mask = [&]() {
          if (key0 + kTile <= edge) return;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (key0 + key >= sm.lim[col0 + c]) e[c] = -INFINITY;
        };
        auto exponents = [&]() {  // s c - m; the largest
          float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float4 cm = lds_f4(cm_at + c * 8);
            const uint64_t x = f2fma(f2pack(e[c], e[c + 1]), f2pack(cm.x, cm.y), f2pack(cm.z, cm.w));
            f2unpack(x, e[c], e[c + 1]);
          }
          mask();
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            top0 = fmax3(top0, e[c], e[c + 1]);
            top1 = fmax3(top1, e[c + 2], e[c + 3]);
          }
          return fmaxf(top0, top1);
        };
        load();
        if (barrier_any(2 + wg, 128, exponents() > kMoveRef)) {
          // New references. The columns' largest y = s c over the tile's keys:
          load();
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float4 cm = lds_f4(cm_at + c * 8);
            e[c] *= cm.x, e[c + 1] *= cm.y;
          }
          mask();
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 32) {
            int mine = INT_MIN;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int v = __reduce_max_sync(0xffffffffu, ordered(e[c0 + c]));
              if (lane == c) mine = v;
            }
            atomicMax(&sm.top[col0 + c0 + lane], mine);
          }
          named_barrier_sync(2 + wg, 128);
          if (wtid < NC) {
            float* m = reinterpret_cast<float*>(&sm.cm[(col0 + wtid) >> 1]) + (wtid & 1) + 2;
            const float old = -*m, next = fmaxf(old, unordered(sm.top[col0 + wtid]) - kPScale);
            *m = -next;
            sm.top[col0 + wtid] = __float_as_int(ex2_approx(old - next));
          }
          named_barrier_sync(2 + wg, 128);
#pragma unroll
          for (int c = 0; c < NC / 2; ++c) {
            const uint64_t f = f2pack(__int_as_float(sm.top[col0 + 2 * c]), __int_as_float(sm.top[col0 + 2 * c + 1]));
            l2[c] = f2fma(l2[c], f, 0ull);
          }
          if (i > 0) {  // O holds the tiles before this one
            ok = ok && mbar_wait(bar(sm.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, abrt);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < KP * NC; c += 32) {
              const int col = c % NC, at = tmem + lanes + C::kO + (c / NC) * R + col0 + col;
              uint32_t o[32];
              tmem_ld32(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x)
                o[x] = __float_as_uint(__uint_as_float(o[x]) * __int_as_float(sm.top[col0 + col + x]));
              tmem_st32(at, o);
            }
            tmem_wait_st();
          }
          named_barrier_sync(2 + wg, 128);
          if (wtid < NC) sm.top[col0 + wtid] = INT_MIN;
          load();
          exponents();
        }
        const uint32_t p_at = slots + place_k<KP>(j, 0).slot * kSlot + (R == 128 ? wg * kHalf : 0) + key * 128;
#pragma unroll
        for (int c = 0; c < NC; c += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float p0 = ex2_approx(e[c + 2 * x]), p1 = ex2_approx(e[c + 2 * x + 1]);
            l2[c / 2 + x] = f2add(l2[c / 2 + x], f2pack(p0, p1));
            pk[x] = pack_half2(p0, p1);
          }
          const int piece = c / 8 + (R == 64 ? wg * 4 : 0);
          st_shared_v4(p_at + ((piece ^ (key & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.p_full[j & 1]));
      }

      // ---- the unit's end ----
      ok = ok && mbar_wait(bar(sm.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, abrt);
      __syncwarp();
      tc_fence_after();
      // Q's place is free: all scores are done
      float* s_part = reinterpret_cast<float*>(s_q);         // [8 warps][64]
      float* s_fac = s_part + 8 * 64;                        // [R]
      float* s_norm = s_fac + 128;                           // [8 warps][32], then [64]
      {
        float l[NC];
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) f2unpack(l2[c], l[2 * c], l[2 * c + 1]);
        int at = 0;
#pragma unroll
        for (int d = 16, n = NC / 2; d >= 1; d >>= 1, n >>= 1) {  // halves of the columns to halves of the lanes
          const bool up = lane & d;
          at += up ? n : 0;
#pragma unroll
          for (int c = 0; c < n; ++c) {
            const float give = up ? l[c] : l[c + n], keep = up ? l[c + n] : l[c];
            l[c] = keep + __shfl_xor_sync(0xffffffffu, give, d);
          }
        }
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) s_part[warp * 64 + at + c] = l[c];
      }
      named_barrier_sync(1, kSoftmaxWarps * 32);
      float* rec = a.pieces + static_cast<size_t>(2 * blockIdx.x + (starts ? 1 : 0)) * C::kPiece;
      if (tid < R) {
        const int g = tid / NC, c = tid % NC;
        const float* p = s_part + g * 4 * 64 + c;
        const float l = (p[0] + p[64]) + (p[128] + p[192]);
        if (whole) {
          const int t = KP == 2 ? tid % C::kQRows : tid / a.group;
          float f = 0.f;
          if (t < toks && sm.lim[tid] > 0) {
            f = 1.f / l;
            if constexpr (KP == 2) {
              f *= tid < C::kQRows ? a.v_mul : *(a.lambda + w.h) * a.v_mul;
            } else {
              const int sub = tid - t * a.group;
              f *= a.v_mul;
              if (sub & 1)
                f *= 1.f / (1.f + __expf(-*(a.lam_logit + static_cast<size_t>(w.q0 + tok0 + t) * (a.H * a.group / 2) +
                                            (w.h * a.group + sub) / 2)));
            }
          }
          s_fac[tid] = f;
        } else {
          rec[tid] = -*(reinterpret_cast<const float*>(&sm.cm[tid >> 1]) + (tid & 1) + 2);
          rec[R + tid] = l;
        }
      }
      named_barrier_sync(1, kSoftmaxWarps * 32);
      int* nan = sm.nan_key[unit & (kNanSets - 1)];
      // channel `key` of each plane, and the first key whose value there is NaN
      int bad[KP];
#pragma unroll
      for (int p = 0; p < KP; ++p) bad[p] = nan[p * 8 + (key >> 4)];
      const float kNan = __int_as_float(0x7fffffff);
      const uint32_t o_at = tmem + lanes + C::kO;
      if (!whole) {
        const int cols = KP == 2 ? R : toks * a.group;
#pragma unroll 1
        for (int c = 0; c < KP * NC; c += 32) {
          const int p = c / NC, col = col0 + c % NC;
          uint32_t o[32];
          tmem_ld32(o_at + p * R + col, o);
          tmem_wait_ld();
          const int first_bad = KP == 2 && p == 1 ? bad[KP - 1] : bad[0];
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (col + x < cols && (KP == 1 || (col + x) % C::kQRows < toks))
              rec[2 * R + static_cast<size_t>(col + x) * C::kWidth + p * 128 + key] =
                  first_bad < sm.lim[col + x] ? kNan : __uint_as_float(o[x]);
        }
      } else if constexpr (KP == 1) {
        const int pairs = a.H * a.group / 2;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + static_cast<size_t>(w.q0 + tok0) * pairs * 128 + key;
#pragma unroll 1
        for (int c = 0; c < NC; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_at + col0 + c, o);
          tmem_wait_ld();
          if ((col0 + c) / a.group >= toks) continue;
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const int col = col0 + c + x, t = col / a.group, sub = col - t * a.group;
            float y = __uint_as_float(o[x]) * s_fac[col] - __uint_as_float(o[x + 1]) * s_fac[col + 1];
            if (bad[0] < sm.lim[col]) y = kNan;
            if (sm.lim[col] <= 0) y = 0.f;
            if (t < toks && dbg_index_ok(w.q0 + tok0 + t, a.total))
              out[(static_cast<size_t>(t) * pairs + (w.h * a.group + sub) / 2) * 128] = __float2bfloat16_rn(y);
          }
        }
      } else {
        constexpr int T = C::kQRows, TN = T / 2;  // the warpgroup's tokens
        const int t0 = wg * TN;
        float y[2][TN], ss[TN];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t o1[TN], o2[TN];
          if constexpr (TN == 32) {
            tmem_ld32(o_at + p * R + t0, o1);
            tmem_ld32(o_at + p * R + T + t0, o2);
          } else {
            tmem_ld16(o_at + p * R + t0, o1);
            tmem_ld16(o_at + p * R + T + t0, o2);
          }
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            const int lim = sm.lim[t0 + t];
            float v = __uint_as_float(o1[t]) * s_fac[t0 + t] - __uint_as_float(o2[t]) * s_fac[T + t0 + t];
            if (bad[p] < lim) v = kNan;
            y[p][t] = v;
          }
        }
        float f = 1.f;
        if (a.flags & 2) {
#pragma unroll
          for (int t = 0; t < TN; ++t) ss[t] = fmaf(y[0][t], y[0][t], y[1][t] * y[1][t]);
          int at = 0;
#pragma unroll
          for (int d = 16, n = TN / 2; d >= 1; d >>= 1, n >>= 1) {
            const bool up = lane & d;
            if (n >= 1) {
              at += up ? n : 0;
#pragma unroll
              for (int c = 0; c < n; ++c) {
                const float give = up ? ss[c] : ss[c + n], keep = up ? ss[c + n] : ss[c];
                ss[c] = keep + __shfl_xor_sync(0xffffffffu, give, d);
              }
            } else {
              ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], d);
            }
          }
          s_norm[warp * 32 + at] = ss[0];
          named_barrier_sync(2 + wg, 128);
          if (wtid < TN) {
            const float* q = s_norm + wg * 4 * 32 + wtid;
            const float sum = (q[0] + q[32]) + (q[64] + q[96]);
            s_part[t0 + wtid] = 1.f / sqrtf(sum / 256.f + a.eps);
          }
          named_barrier_sync(2 + wg, 128);
        }
        if (a.flags & 4) f = 1.f - a.lambda_init;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(w.q0 + tok0) * a.H + w.h) * 256 + key;
        float wgt[2] = {1.f, 1.f};
        if ((a.flags & 2) && a.norm_w) wgt[0] = *(a.norm_w + key), wgt[1] = *(a.norm_w + 128 + key);
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          if (t0 + t >= toks || !dbg_index_ok(w.q0 + tok0 + t0 + t, a.total)) continue;
          const float n = (a.flags & 2) ? s_part[t0 + t] * f : f;
          const bool none = sm.lim[t0 + t] <= 0;  // (zeros, whatever the weight and the scale hold)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            out[static_cast<size_t>(t0 + t) * a.H * 256 + p * 128] = __float2bfloat16_rn(none ? 0.f : y[p][t] * n * wgt[p]);
        }
      }
      tc_fence_before();
      named_barrier_sync(1, kSoftmaxWarps * 32);
      if (tid < 16) nan[tid] = INT_MAX;
      ++unit;
      advance(a, w, seg);
    }
    if (tid == 0) sm.seg = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(sm.q_full));
  }

  // ---- teardown ----
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins, of each unit whose tiles lie in more than one range, its pieces: that of the range that begins it and
// of the ranges that begin inside it, in this order. Block (i, y): the unit that range i + 1 begins inside,
// if no earlier range does, and every gridDim.y-th of its tokens (V1) or pairs (V2) from y on; a thread a channel.
template <int KP, int R>
__global__ void __launch_bounds__(KP * 128) kv4_chunk_join_kernel(const Kv4ChunkArgs a) {
  using C = Cfg<KP, R>;
  constexpr int NT = KP * 128;
  __shared__ long long s_pre[NT + 1], s_sum[NT / 32], s_first;
  __shared__ Walk s_walk;
  __shared__ float s_red[NT / 32];
  const int tid = threadIdx.x;
  // All but the pieces is known before the first kernel ends: it released this one after its own wait.
  const long long total = fill<NT, true>(a, s_pre, s_sum, false);
  const int n = range_count(total, a.grid), i = blockIdx.x;
  bool mine = i + 1 < n;
  if (mine) {
    if (tid < 32) {
      Walk w;
      long long first;
      locate<NT, true>(a, s_pre, range_start(total, n, i + 1), w, first);
      if (tid == 0) s_walk = w, s_first = first;
    }
    __syncthreads();
  }
  const Walk w = mine ? s_walk : Walk{};
  const long long first = mine ? s_first : 0;
  // range i + 1 begins with the unit, or is not the first to begin inside it
  mine = mine && w.tile > 0 && range_start(total, n, i) <= first;
  grid_wait();
  grid_release();
  if (!mine) return;
  const int i0 = range_of(total, n, first), pieces = range_of(total, n, first + w.tiles - 1) - i0 + 1;
  const int tok0 = w.rt * a.tokens, toks = min(a.tokens, w.Lq - tok0);
  const int outs = KP == 2 ? toks : toks * a.group / 2;  // of the unit
  float wgt = 1.f;
  if (KP == 2 && (a.flags & 2) && a.norm_w) wgt = *(a.norm_w + tid);
  for (int o = blockIdx.y; o < outs; o += gridDim.y) {
    const int c[2] = {KP == 2 ? o : 2 * o, KP == 2 ? C::kQRows + o : 2 * o + 1};
    float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f}, v[2] = {0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < pieces; ++k) {
      const float* r = a.pieces + static_cast<size_t>(2 * (i0 + k) + (k == 0 ? 1 : 0)) * C::kPiece;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mk = r[c[e]], lk = r[R + c[e]], vk = r[2 * R + static_cast<size_t>(c[e]) * C::kWidth + tid];
        const float top = fmaxf(m[e], mk), f = ex2_approx(m[e] - top), fk = ex2_approx(mk - top);
        m[e] = top;
        l[e] = l[e] * f + lk * fk;
        v[e] = v[e] * f + vk * fk;
      }
    }
    const int t = KP == 2 ? o : 2 * o / a.group;
    const size_t token = static_cast<size_t>(w.q0) + tok0 + t;
    const bool none = a.causal && w.Lk - w.Lq + tok0 + t < 0;  // it sees no key
    if constexpr (KP == 1) {
      const int pairs = a.H * a.group / 2, pair = w.h * (a.group / 2) + o - t * (a.group / 2);
      const float sig = 1.f / (1.f + __expf(-*(a.lam_logit + token * pairs + pair)));
      const float y = (v[0] / l[0] - sig * (v[1] / l[1])) * a.v_mul;
      static_cast<__nv_bfloat16*>(a.out)[(token * pairs + pair) * 128 + tid] = __float2bfloat16_rn(none ? 0.f : y);
    } else {
      float y = (v[0] / l[0] - *(a.lambda + w.h) * (v[1] / l[1])) * a.v_mul;
      if (a.flags & 2) {
        float ss = y * y;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
        __syncthreads();
        if ((tid & 31) == 0) s_red[tid >> 5] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < NT / 32; ++k) ss += s_red[k];
        y *= 1.f / sqrtf(ss / 256.f + a.eps) * wgt;
      }
      if (a.flags & 4) y *= 1.f - a.lambda_init;
      static_cast<__nv_bfloat16*>(a.out)[(token * a.H + w.h) * 256 + tid] = __float2bfloat16_rn(none ? 0.f : y);
    }
  }
}

template <int KP, int R>
cudaError_t launch(Kv4ChunkArgs a, cudaStream_t st) {
  static std::atomic<uint64_t> raised{};
  a.tokens = KP == 2 ? R / 2 : R / a.group;
  // no more blocks than the tables' capacity can give ranges: a sequence's tiles of tokens overlap the total's
  const long long tiles = (static_cast<long long>(a.max_pages) * a.page_size + kTile - 1) / kTile;
  const long long units = (static_cast<long long>(a.total) / a.tokens + a.B) * a.H;
  const long long most = units >= kSms ? kSms : (tiles + kUnitCost) * units / kMinCost;
  a.grid = static_cast<int>(most < 1 ? 1 : most > kSms ? kSms : most);
  cudaError_t e = launch_early_large(kv4_chunk_kernel<KP, R>, a.grid, kThreads, smem_bytes<R>(), smem_bytes<R>(), st, 1, a, raised);
  if (e != cudaSuccess || a.grid == 1) return e;
  g_launched.store(true, std::memory_order_relaxed);
  cudaLaunchAttribute at[1] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.grid - 1, R / 16);
  cfg.blockDim = dim3(KP * 128);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_chunk_join_kernel<KP, R>, a);
}

}  // namespace

// Columns of a unit: 64 where the longest chunk fits in them, which halves a tile's products and softmax.
int kv4_chunk_cols(int group, int max_seqlen_q) {
  return static_cast<long long>(max_seqlen_q) * (group == 0 ? 2 : group) <= 64 ? 64 : 128;
}
size_t kv4_chunk_workspace_bytes(int group, int max_seqlen_q) {
  const size_t cols = kv4_chunk_cols(group, max_seqlen_q), width = group == 0 ? 256 : 128;
  return 2 * static_cast<size_t>(kSms) * (2 * cols + cols * width) * sizeof(float);
}

cudaError_t launch_kv4_chunk(const Kv4ChunkArgs& a, int cols, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  if (a.group == 0) return cols == 64 ? launch<2, 64>(a, st) : launch<2, 128>(a, st);
  return cols == 64 ? launch<1, 64>(a, st) : launch<1, 128>(a, st);
}

cudaError_t status_chunk_kv4(int* v) { return launched_status(v); }

}  // namespace da
