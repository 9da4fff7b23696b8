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
// tile, so its P go to shared memory as whole pieces of 16 bytes, over the K plane that S came from. 8
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
// warps: softmax 0 .. 7, K 8 .. 11, V 12 .. 15, products 16, addresses 17
constexpr int kKWarp = 8, kVWarp = 12, kMmaWarp = 16, kAddressWarp = 17;
constexpr int kSoftmaxWarps = 8, kThreads = 20 * 32;
constexpr int kTile = 128;                       // keys
constexpr int kSlot = kTile * 128 * 2;           // one plane of a tile in fp16
constexpr int kHalf = kSlot / 2;                 // 64 of its channels (or columns of P)
constexpr int kUnitCost = 3;                     // what a unit costs besides its tiles, in tiles
constexpr int kMinCost = 2;                      // the smallest range
constexpr float kPScale = 6.f, kMoveRef = 15.f;  // log2 of P's scale, and of the P at which the reference moves
constexpr int kNanSets = 4;
constexpr int kRing = 4;                         // tiles whose records' addresses are known

template <int KP, int R>
struct Cfg {
  static constexpr int kHalfCols = R / 2;
  static constexpr int kQRows = KP == 1 ? R : R / 2;  // rows of one product's Q
  static constexpr int kQBytes = R * 256;
  static constexpr int kWidth = KP * 128;
  static constexpr int kVSlots = KP == 1 ? 3 : 4;     // V: stages of a plane (V2), of two planes (V1)
  static constexpr int kP = kVSlots * kSlot;          // shared memory: V, P twice, Q
  static constexpr int kQ = kP + 2 * R * 256;
  static constexpr int kSmall = kQ + kQBytes;
  static constexpr int kO = 2 * R;                    // tensor memory: S twice, O's planes, K twice
  static constexpr int kK = kO + KP * R;
  static constexpr int kPiece = 2 * R + R * kWidth;   // floats: m, l, o
  // Registers a thread: the launch's 96, dealt out anew to the warpgroups (2 of softmax, K, V, the rest).
  static constexpr int kSoftmaxRegs = R == 64 ? 128 : 152, kUnpackRegs = R == 64 ? 96 : 72, kRestRegs = 32;
  static_assert(2 * kSoftmaxRegs + 2 * kUnpackRegs + kRestRegs <= 5 * 96, "more registers than the launch has");
  static_assert(kK + 2 * KP * 64 <= 512, "tensor memory");
};

struct TileAt {
  const uint8_t* rec[8];
  int key0, left, unit, pad;  // its first key, keys from there on (0: the stream has ended), its unit's number
};
struct Small {  // behind Q
  float ref[128];      // the columns' references (less kPScale), negated
  float fac[128];      // where the columns' queries have powers of two of their own: what S is to be multiplied with
  int lim[128];        // keys that a column sees; 0 where there is no such token
  int top[128];        // a move: the columns' largest exponents (ordered), then the factors
  uint64_t v_full[4], v_free[4], k_full[2], k_free[2], s_full[2], p_full[2], pv_done[2], q_full, teardown;
  uint64_t tile_full[kRing], tile_free[kRing];
  TileAt tile[kRing];
  int nan_key[kNanSets][16];
  int exp_max, exp_min;  // exponents of the unit's queries
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

template <int KP, int R>
constexpr int smem_bytes() {
  return Cfg<KP, R>::kSmall + static_cast<int>(sizeof(Small));
}
static_assert(smem_bytes<1, 128>() <= 232448 && smem_bytes<2, 64>() <= 232448, "shared memory");

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

// one lane of a converged warp; the compiler knows that it is one, and keeps what it computes in uniform
// registers, which the products' descriptors have to be in
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// ---- small parts -------------------------------------------------------------------------------
__device__ __forceinline__ uint4 ldg128(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ldg32(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
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

// where V's plane `half` of the block's tile j lies, and the phase of its slot's use
struct Place {
  int slot, phase;
};
template <int KP>
__device__ __forceinline__ Place place_v(int j, int half) {
  if constexpr (KP == 1) return {j % 3, (j / 3) & 1};
  return {2 * (j & 1) + half, (j >> 1) & 1};
}

template <int KP, int R>
__global__ void __launch_bounds__(kThreads, 1) kv4_chunk_kernel(const Kv4ChunkArgs a) {
  using C = Cfg<KP, R>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const s_q = smem + C::kQ;
  Small& sm = *reinterpret_cast<Small*>(smem + C::kSmall);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t slots = smem_u32(smem), p_slots = slots + C::kP, q_at = smem_u32(s_q);
  auto bar = [](uint64_t& x) { return smem_u32(&x); };

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(sm.v_full[i]), 4);
      mbar_init(bar(sm.v_free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sm.k_full[i]), 4);
      mbar_init(bar(sm.k_free[i]), 1);
      mbar_init(bar(sm.s_full[i]), 1);
      mbar_init(bar(sm.p_full[i]), kSoftmaxWarps);
      mbar_init(bar(sm.pv_done[i]), 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar(sm.tile_full[i]), 1);
      mbar_init(bar(sm.tile_free[i]), 8);
    }
    mbar_init(bar(sm.q_full), kSoftmaxWarps);
    mbar_init(bar(sm.teardown), 1);
    sm.abort = 0;
    sm.exp_max = INT_MIN, sm.exp_min = INT_MAX;
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
    registers_down<C::kRestRegs>();
    if (warp == kMmaWarp && elect_one()) {
      // ================================ products ================================
      constexpr uint32_t idesc_s = idesc_f16(kTile, C::kQRows, 0, 0), idesc_o = idesc_f16(128, R, 1, 1);
      const uint64_t dq = umma_smem_desc(q_at, 16, 1024);
      const uint64_t dv = umma_smem_desc(slots, kHalf, 1024), dp = umma_smem_desc(p_slots, kHalf, 1024);
      int j = 0;
      bool ok = true;
      auto scores = [&](int t) {
        if (!(ok = mbar_wait(bar(sm.k_full[t & 1]), (t >> 1) & 1, abrt))) return;
        tc_fence_after();
#pragma unroll 1
        for (int map = 0; map < KP; ++map)
#pragma unroll 2
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(tmem + (t & 1) * R + map * C::kQRows, tmem + C::kK + ((t & 1) * KP + map) * 64 + kk * 8,
                        desc_add(dq, map * C::kQRows * 256 + (kk >> 2) * C::kQRows * 128 + (kk & 3) * 32), idesc_s, kk > 0);
        tc_commit(bar(sm.s_full[t & 1]));
        tc_commit(bar(sm.k_free[t & 1]));
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
          if (!(ok = mbar_wait(bar(sm.p_full[j & 1]), (j >> 1) & 1, abrt))) break;
#pragma unroll 1
          for (int half = 0; half < KP; ++half) {
            const Place v = place_v<KP>(j, half);
            if (!(ok = ok && mbar_wait(bar(sm.v_full[v.slot]), v.phase, abrt))) break;
            tc_fence_after();
#pragma unroll 2
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(tmem + C::kO + half * R, desc_add(dv, v.slot * kSlot + kk * 2048),
                          desc_add(dp, (j & 1) * R * 256 + kk * 2048), idesc_o, i > 0 || kk > 0);
            tc_commit(bar(sm.v_free[v.slot]));
          }
          if (!ok) break;
          tc_commit(bar(sm.pv_done[j & 1]));
        }
      }
      // every product that was issued ends before tensor memory is given back
      tc_commit(bar(sm.teardown));
      mbar_wait(bar(sm.teardown), 0, nullptr);
    } else if (warp == kAddressWarp) {
      // ================================ addresses ================================
      // Lane 8 i + r looks up record r of tile i of a batch: up to four tiles of a unit. The next batch's pages
      // are looked up before this one is passed on, tile by tile, as the ring has room.
      const int recs = a.page_size >> 4, i4 = lane >> 3, r8 = lane & 7;
      struct Batch {
        int n, h, page, off, key0, left, unit;  // tiles; this lane's page and record of the page; the first tile's
        bool used;
      };
      auto look_up = [&](int unit) {
        Batch x;
        x.n = static_cast<int>(min(min(4LL, static_cast<long long>(w.tiles - w.tile)), max(w.todo, 0LL)));
        const int rec = min((w.tile + i4) * 8 + r8, max(0, (w.Lk - 1) >> 4)), pi = (__umulhi(rec, a.rec_magic) + rec) >> a.rec_shift;
        x.used = i4 < x.n && ((w.tile + i4) * 8 + r8) * 16 < w.Lk && dbg_index_ok(pi, a.max_pages);
        x.page = x.used ? *(a.block_table + static_cast<size_t>(w.b) * a.max_pages + pi) : 0;
        x.off = rec - pi * recs;
        x.h = w.h, x.key0 = w.tile * kTile, x.left = w.Lk - x.key0, x.unit = unit;
        return x;
      };
      int t = 0, unit = 0;
      bool ok = true;
      Batch next = look_up(0);
      while (ok) {
        Batch x = next;
        if (x.n > 0) {
          if (w.tile + x.n == w.tiles) ++unit;
          advance(a, w, x.n);
          next = look_up(unit);
        }
        if (x.used && (x.page < 0 || x.page >= a.num_pages)) {
          flag_device_error(DEV_BAD_INDEX);
          x.page = 0;
        }
        const uint8_t* src = a.pool + ((static_cast<size_t>(x.page) * a.H + x.h) * recs + x.off) * (2 * KP * kKv4Plane);
        for (int i = 0; ok && i < max(x.n, 1); ++i, ++t) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(sm.tile_free[t % kRing]), ((t / kRing) & 1) ^ 1, abrt));
          TileAt& at = sm.tile[t % kRing];
          if (i4 == i) {
            at.rec[r8] = src;
            if (x.used) prefetch_l2(src, 2 * KP * kKv4Plane);
          }
          if (lane == 0) at.key0 = x.key0 + i * kTile, at.left = x.n > 0 ? x.left - i * kTile : 0, at.unit = x.unit;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sm.tile_full[t % kRing]));
        }
        if (x.n == 0) break;
      }
    }
  } else if (warp >= kKWarp) {
    // ================================ unpack ================================
    // Both kinds of warps load a tile's bytes into registers one or two tiles before they unpack them (also
    // where the sequence has no such record, from page 0: no branch comes between loads in flight).
    registers_down<C::kUnpackRegs>();
    const int q4 = warp & 3;
    int next = 0, end = INT_MAX;  // the next tile to load; behind the stream's last its end stays, and is read again
    bool ok = true;
    struct Tile {
      int key0, left, unit;
    };
    auto tile_at = [&](Tile& t) -> const TileAt& {
      const int i = min(next, end);
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(sm.tile_full[i % kRing]), (i / kRing) & 1, abrt));
      const TileAt& at = sm.tile[i % kRing];
      t.key0 = at.key0, t.left = ok ? at.left : 0, t.unit = at.unit;
      if (t.left <= 0) end = i;
      ++next;
      return at;
    };
    auto tile_read = [&](const Tile& t) {  // (its addresses are in registers)
      __syncwarp();
      if (lane == 0 && t.left > 0) mbar_arrive(bar(sm.tile_free[(next - 1) % kRing]));
    };
    auto dup = [](uint32_t two, int high) { return __byte_perm(two, 0, high ? 0x3232 : 0x1010); };
    if (warp < kVWarp) {
      // K: lane `key` takes a key of the tile, tensor memory's lane of that number: its 64 bytes of codes are
      // on end, its scales two bytes of each word of 16.
      constexpr int kAhead = 1;
      struct Data {
        uint4 w[4], sc;
      };
      Data d[kAhead][KP];
      Tile tl[kAhead], tile;
      const int key = lane & 15, h = (key >> 1) & 1, row = 32 * q4 + lane;
      const int code = kv4_k_code(key, 0), scale = kKv4PlaneCodes + (key >> 2) * 32 + (key & 1) * 16;
      const uint32_t to = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + C::kK;
      const uint8_t* src = nullptr;
      auto load = [&](Data& x, int plane) {
        const uint8_t* p = src + plane * kKv4Plane;
#pragma unroll
        for (int i = 0; i < 4; ++i) x.w[i] = ldg128(p + code + 16 * i);
        x.sc = ldg128(p + scale);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        src = tile_at(tl[i]).rec[2 * q4 + (lane >> 4)];
        tile_read(tl[i]);
#pragma unroll
        for (int p = 0; p < KP; ++p) load(d[i][p], p);
      }
      for (int j = 0; ok; j += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          tile = tl[i];
          if (tile.left <= 0) {
            ok = false;
            break;
          }
          const int t = j + i;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(sm.k_free[t & 1]), ((t >> 1) & 1) ^ 1, abrt));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int p = 0; p < KP; ++p) {
            const uint32_t sc4[4] = {d[i][p].sc.x, d[i][p].sc.y, d[i][p].sc.z, d[i][p].sc.w};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t v[32];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint4 w4 = d[i][p].w[2 * half + x];
                const uint32_t word[4] = {w4.x, w4.y, w4.z, w4.w};
                const uint32_t two = row < tile.left ? e4m3x2_to_half2(sc4[2 * half + x] >> (16 * h)) : 0u;
                const uint32_t f0 = dup(two, 0), f1 = dup(two, 1);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  uint32_t o[4];
                  e2m1x8_to_half2(word[y], o);
#pragma unroll
                  for (int z = 0; z < 4; ++z) v[x * 16 + y * 4 + z] = half2_mul(o[z], y < 2 ? f0 : f1);
                }
              }
              tmem_st32(to + ((t & 1) * KP + p) * 64 + half * 32, v);
            }
            if (p == 0) {
              src = tile_at(tl[i]).rec[2 * q4 + (lane >> 4)];
              tile_read(tl[i]);
            }
            load(d[i][p], p);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sm.k_full[t & 1]));
        }
      }
    } else {
      // V: warp v takes records v and v + 4, to shared memory. A piece of 8 channels lies at its number XOR the
      // row's; lanes of a quarter-warp whose places would meet in the banks (t4 of 0 and 2, 1 and 3) take
      // their pieces in another order.
      constexpr int kAhead = 1;
      struct Data {
        uint4 lo[2], hi[2];
        uint32_t sc[2];
      };
      Data d[kAhead][KP];
      Tile tl[kAhead], tile;
      const int t4 = lane & 3, g8 = lane >> 2;  // tokens 4 t4 .., channels 16 g8 ..
      const bool far = t4 & 2;
      const uint32_t at0 = slots + (g8 >> 2) * kHalf + (q4 * 16 + 4 * t4) * 128;
      const int c0 = ((g8 & 3) * 2) ^ (4 * (t4 & 1)) ^ (far ? 1 : 0);
      const uint8_t* src[2] = {nullptr, nullptr};
      auto load = [&](Data& x, int half) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* p = src[i] + (KP + half) * kKv4Plane;
          x.lo[i] = ldg128(p + lane * 16);
          x.hi[i] = ldg128(p + lane * 16 + 512);
          x.sc[i] = ldg32(p + lane * 4 + kKv4PlaneCodes);
        }
      };
      auto fetch = [&](Tile& t) {
        const TileAt& at = tile_at(t);
        src[0] = at.rec[q4], src[1] = at.rec[q4 + 4];
        tile_read(t);
      };
      auto put = [](uint32_t at, uint32_t word, uint32_t f) {
        uint32_t v[4];
        e2m1x8_to_half2(word, v);
        st_shared_v4(at, half2_mul(v[0], f), half2_mul(v[1], f), half2_mul(v[2], f), half2_mul(v[3], f));
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        fetch(tl[i]);
#pragma unroll
        for (int p = 0; p < KP; ++p) load(d[i][p], p);
      }
      for (int j = 0; ok; j += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          tile = tl[i];
          if (tile.left <= 0) {
            ok = false;
            break;
          }
#pragma unroll
          for (int half = 0; half < KP; ++half) {
            const Place to = place_v<KP>(j + i, half);
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(sm.v_free[to.slot]), to.phase ^ 1, abrt));
            if (!ok) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const Data& y = d[i][half];
              uint32_t sc = y.sc[x];
              const int token = (q4 + 4 * x) * 16 + 4 * t4, live = tile.left - token;
              if (live < 4) sc = live <= 0 ? 0u : sc & (0xffffffffu >> (32 - 8 * live));
              const uint32_t odd = ((sc & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // scales that are NaN
              if (odd) {
                atomicMin(&sm.nan_key[tile.unit & (kNanSets - 1)][half * 8 + g8], tile.key0 + token + ((__ffs(odd) - 1) >> 3));
                sc &= ~((odd >> 7) * 0xffu);
              }
              uint32_t s01, s23;
              e4m3x4_to_half2(sc, s01, s23);
              const uint32_t base = at0 + to.slot * kSlot + x * 64 * 128;
              const uint32_t a0 = base + (c0 << 4), a1 = base + ((c0 ^ 1) << 4), a2 = base + ((c0 ^ 2) << 4), a3 = base + ((c0 ^ 3) << 4);
              const uint32_t f0 = dup(s01, 0), f1 = dup(s01, 1), f2 = dup(s23, 0), f3 = dup(s23, 1);
              put(a0, far ? y.lo[x].y : y.lo[x].x, f0);
              put(a1, far ? y.lo[x].x : y.lo[x].y, f0);
              put(a1 + 128, far ? y.lo[x].w : y.lo[x].z, f1);
              put(a0 + 128, far ? y.lo[x].z : y.lo[x].w, f1);
              put(a2 + 256, far ? y.hi[x].y : y.hi[x].x, f2);
              put(a3 + 256, far ? y.hi[x].x : y.hi[x].y, f2);
              put(a3 + 384, far ? y.hi[x].w : y.hi[x].z, f3);
              put(a2 + 384, far ? y.hi[x].z : y.hi[x].w, f3);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sm.v_full[to.slot]));
            if (half == 0) fetch(tl[i]);
            load(d[i][half], half);
          }
          if (!ok) break;
        }
      }
    }
  } else {
    // ================================ softmax ================================
    registers_up<C::kSoftmaxRegs>();
    const int wg = warp >> 2, quarter = warp & 3, key = quarter * 32 + lane, wtid = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    constexpr int NC = C::kHalfCols, NH = NC / 32;  // columns, 32 at a time
    const int col0 = wg * NC;
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
      float scale;  // what S is to be multiplied with
      bool mixed;   // and with the column's factor
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
        // One power of two for all columns where their largest channels lie within 2^12 of each other (zeros
        // lie anywhere), else one for each column.
        const int own = max(static_cast<int>(top >> 7) - 127, -100);
        const int hi = __reduce_max_sync(0xffffffffu, top ? own : INT_MIN), lo = __reduce_min_sync(0xffffffffu, top ? own : INT_MAX);
        if (lane == 0) atomicMax(&sm.exp_max, hi), atomicMin(&sm.exp_min, lo);
        named_barrier_sync(1, kSoftmaxWarps * 32);
        const int all = max(sm.exp_max, -100);
        mixed = sm.exp_max != INT_MIN && sm.exp_max - sm.exp_min > 12;
        const int e = mixed ? own : all;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);  // 2^(14 - e)
        // (never 0 or Inf, which a score of 0 or a masked one's Inf would turn into NaN)
        auto down = [&](int x) { return fminf(fmaxf(ldexpf(a.qk_scale, x - 14), FLT_MIN), FLT_MAX); };
        scale = mixed ? 1.f : down(all);
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
          sm.ref[col] = live ? FLT_MAX : 0.f;
          sm.fac[col] = down(own);
          sm.lim[col] = !live ? 0 : a.causal ? max(0, w.Lk - w.Lq + tok0 + t + 1) : w.Lk;
        }
        if (tid == 0) sm.seg = seg;
        fence_proxy_async_smem();
        named_barrier_sync(1, kSoftmaxWarps * 32);
        if (tid == 0) sm.exp_max = INT_MIN, sm.exp_min = INT_MAX;
        if (lane == 0) mbar_arrive(bar(sm.q_full));
      }
      uint64_t l2[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l2[i] = 0;
      const uint64_t scale2 = f2pack(scale, scale);

      for (int i = 0; i < seg; ++i, ++j) {
        const int key0 = (w.tile + i) * kTile;
        const uint32_t p_at = p_slots + (j & 1) * R * 256 + (R == 128 ? wg * kHalf : 0) + key * 128;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const int c0 = col0 + 32 * h;
          float4 ref[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) ref[x] = *reinterpret_cast<const float4*>(&sm.ref[c0 + 4 * x]);
          if (h == 0) {
            ok = ok && mbar_wait(bar(sm.s_full[j & 1]), (j >> 1) & 1, abrt);
            __syncwarp();
            tc_fence_after();
          }
          float e[32];
          auto load = [&]() {
            uint32_t raw[32];
            tmem_ld32(tmem + lanes + (j & 1) * R + c0, raw);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) e[c] = __uint_as_float(raw[c]);
            if (mixed) {
#pragma unroll
              for (int c = 0; c < 32; ++c) e[c] *= sm.fac[c0 + c];
            }
          };
          auto mask = [&]() {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (key0 + key >= sm.lim[c0 + c]) e[c] = -INFINITY;
          };
          for (bool moved = false;; moved = true) {  // exponents s c - m; once more where a column needs a new reference
            load();
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              f2unpack(f2fma(f2pack(e[4 * x], e[4 * x + 1]), scale2, f2pack(ref[x].x, ref[x].y)), e[4 * x], e[4 * x + 1]);
              f2unpack(f2fma(f2pack(e[4 * x + 2], e[4 * x + 3]), scale2, f2pack(ref[x].z, ref[x].w)), e[4 * x + 2], e[4 * x + 3]);
            }
            if (key0 + kTile > edge) mask();
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              top0 = fmax3(top0, e[c], e[c + 1]);
              top1 = fmax3(top1, e[c + 2], e[c + 3]);
            }
            if (__builtin_expect(!barrier_any(2 + wg, 128, fmaxf(top0, top1) > kMoveRef) || moved, 1)) break;
            // New references. The columns' largest y = s c over the tile's keys:
            load();
#pragma unroll
            for (int c = 0; c < 32; ++c) e[c] *= scale;
            if (key0 + kTile > edge) mask();
            int mine = INT_MIN;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int v = __reduce_max_sync(0xffffffffu, ordered(e[c]));
              if (lane == c) mine = v;
            }
            atomicMax(&sm.top[c0 + lane], mine);
            named_barrier_sync(2 + wg, 128);
            if (wtid < 32) {
              const float old = -sm.ref[c0 + wtid], to = fmaxf(old, __fsub_ru(unordered(sm.top[c0 + wtid]), kPScale));
              sm.ref[c0 + wtid] = -to;
              sm.top[c0 + wtid] = __float_as_int(ex2_approx(old - to));
            }
            named_barrier_sync(2 + wg, 128);
#pragma unroll
            for (int x = 0; x < 8; ++x) ref[x] = *reinterpret_cast<const float4*>(&sm.ref[c0 + 4 * x]);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const uint64_t f = f2pack(__int_as_float(sm.top[c0 + 2 * c]), __int_as_float(sm.top[c0 + 2 * c + 1]));
              l2[16 * h + c] = f2fma(l2[16 * h + c], f, 0ull);
            }
            if (i > 0) {  // O holds the tiles before this one
              ok = ok && mbar_wait(bar(sm.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, abrt);
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int p = 0; p < KP; ++p) {
                const uint32_t at = tmem + lanes + C::kO + p * R + c0;
                uint32_t o[32];
                tmem_ld32(at, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * __int_as_float(sm.top[c0 + x]));
                tmem_st32(at, o);
              }
              tmem_wait_st();
            }
            named_barrier_sync(2 + wg, 128);
            if (wtid < 32) sm.top[c0 + wtid] = INT_MIN;
          }
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float p0 = ex2_approx(e[c + 2 * x]), p1 = ex2_approx(e[c + 2 * x + 1]);
              l2[16 * h + c / 2 + x] = f2add(l2[16 * h + c / 2 + x], f2pack(p0, p1));
              pk[x] = pack_half2(p0, p1);
            }
            const int piece = 4 * (R == 64 ? wg : h) + c / 8;
            st_shared_v4(p_at + ((piece ^ (key & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
          }
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
          rec[tid] = -sm.ref[tid];
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
        constexpr int T = C::kQRows, TN = 16;  // the warpgroup's tokens, 16 at a time
        float wgt[2] = {1.f, 1.f};
        if ((a.flags & 2) && a.norm_w) wgt[0] = *(a.norm_w + key), wgt[1] = *(a.norm_w + 128 + key);
        const float f = (a.flags & 4) ? 1.f - a.lambda_init : 1.f;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(w.q0 + tok0) * a.H + w.h) * 256 + key;
#pragma unroll 1
        for (int t0 = wg * (T / 2); t0 < (wg + 1) * (T / 2); t0 += TN) {
          float y[2][TN];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t o1[TN], o2[TN];
            tmem_ld16(o_at + p * R + t0, o1);
            tmem_ld16(o_at + p * R + T + t0, o2);
            tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < TN; ++t) {
              const float v = __uint_as_float(o1[t]) * s_fac[t0 + t] - __uint_as_float(o2[t]) * s_fac[T + t0 + t];
              y[p][t] = bad[p] < sm.lim[t0 + t] ? kNan : v;
            }
          }
          if (a.flags & 2) {
            float ss[TN];
#pragma unroll
            for (int t = 0; t < TN; ++t) ss[t] = fmaf(y[0][t], y[0][t], y[1][t] * y[1][t]);
            int at = 0;
#pragma unroll
            for (int d = 16, n = TN / 2; d >= 2; d >>= 1, n >>= 1) {
              const bool up = lane & d;
              at += up ? n : 0;
#pragma unroll
              for (int c = 0; c < n; ++c) {
                const float give = up ? ss[c] : ss[c + n], keep = up ? ss[c + n] : ss[c];
                ss[c] = keep + __shfl_xor_sync(0xffffffffu, give, d);
              }
            }
            s_norm[warp * TN + at] = ss[0] + __shfl_xor_sync(0xffffffffu, ss[0], 1);
            named_barrier_sync(2 + wg, 128);
            if (wtid < TN) {
              const float* q = s_norm + wg * 4 * TN + wtid;
              const float sum = (q[0] + q[TN]) + (q[2 * TN] + q[3 * TN]);
              s_part[t0 + wtid] = f / sqrtf(sum / 256.f + a.eps);
            }
            named_barrier_sync(2 + wg, 128);
          }
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            if (t0 + t >= toks || !dbg_index_ok(w.q0 + tok0 + t0 + t, a.total)) continue;
            const float n = (a.flags & 2) ? s_part[t0 + t] : f;
            const bool none = sm.lim[t0 + t] <= 0;  // (zeros, whatever the weight and the scale hold)
#pragma unroll
            for (int p = 0; p < 2; ++p)
              out[static_cast<size_t>(t0 + t) * a.H * 256 + p * 128] = __float2bfloat16_rn(none ? 0.f : y[p][t] * n * wgt[p]);
          }
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
  page_magic(a.page_size >> 4, &a.rec_magic, &a.rec_shift);
  // no more blocks than the tables' capacity can give ranges: a sequence's tiles of tokens overlap the total's
  const long long tiles = (static_cast<long long>(a.max_pages) * a.page_size + kTile - 1) / kTile;
  const long long units = (static_cast<long long>(a.total) / a.tokens + a.B) * a.H;
  const long long most = units >= kSms ? kSms : (tiles + kUnitCost) * units / kMinCost;
  a.grid = static_cast<int>(most < 1 ? 1 : most > kSms ? kSms : most);
  cudaError_t e = launch_early_large(kv4_chunk_kernel<KP, R>, a.grid, kThreads, smem_bytes<KP, R>(), smem_bytes<KP, R>(), st, 1, a, raised);
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

// Columns of a unit. V2: 64 where the longest chunk fits in them, which halves a tile's products and softmax.
// V1: 64, as tensor memory holds both planes of O.
int kv4_chunk_cols(int group, int max_seqlen_q) {
  return group == 0 || static_cast<long long>(max_seqlen_q) * group <= 64 ? 64 : 128;
}
size_t kv4_chunk_workspace_bytes(int group, int max_seqlen_q) {
  const size_t cols = kv4_chunk_cols(group, max_seqlen_q), width = group == 0 ? 256 : 128;
  return 2 * static_cast<size_t>(kSms) * (2 * cols + cols * width) * sizeof(float);
}

cudaError_t launch_kv4_chunk(const Kv4ChunkArgs& a, int cols, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  if (a.group == 0) return launch<2, 64>(a, st);
  return cols == 64 ? launch<1, 64>(a, st) : launch<1, 128>(a, st);
}

cudaError_t status_chunk_kv4(int* v) { return launched_status(v); }

}  // namespace da
