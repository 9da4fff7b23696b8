// chunk_kv4.cu -- attention of chunks over the 4-bit cache: each sequence's new tokens, the last of its
// positions, over all its cached keys (V1: both maps of a head; V2: the query heads of a KV head's group).
//
// A unit is a KV head, a sequence and a tile of its new tokens: 128 rows, a row being one softmax (V2: row
// G t + g is query head g of token t; V1: row 2 t + m is map m of token t, its query in the m-th half of 256
// channels whose other half is 0). Over the keys, 128 at a time:
//   S [128 x 128] = Q K^T,   P = 2^(s c - m),   l += P,   O [128 x 128 or 256] += P V
// with S, P and O in tensor memory, a row a lane. At the end V1: o1/l1 - lambda o2/l2, the norm and the
// scale, V2: o_2p/l_2p - sigmoid(lam) o_2p+1/l_2p+1: the two rows of a pair are neighbouring lanes.
//
// Warps. Softmax: a thread a row. V2 has two warpgroups, which take tiles in turn and have an O, m and l of
// their own each, joined at the unit's end; V1, whose products take twice as long a tile, has one. K and V:
// four warps each read records into registers, a tile ahead, and write fp16 (exact: an e2m1 times an e4m3 has
// 6 significant bits) in the products' 128-byte swizzle, into a ring of planes. One warp looks the records'
// addresses up and has L2 fetch them; one issues the products: S of the next tile before P V of this one. At a unit's
// end the next unit's queries go in first, so that its first scores are there when the output is written.
//
// Numerics, as in the decode over the same cache: the query enters as fp16 after a power of two of its own
// for each row, P is rounded to fp16 at 2^6 times its value against m, which moves only where a score passes
// it by 2^9 (the row's l and O are then rescaled). Sums and statistics are fp32. Keys that a row may not see
// have P = 0, and a V block that is NaN is held as zeros and its first key noted: the rows that see that key
// get NaN at the end, the others nothing.
//
// Work. All units one behind the other are cut into equal ranges of tiles, one for each SM; pieces of units
// that are cut go to the workspace, at most two a range, and a second kernel joins them in the order of the
// ranges, so that equal inputs give equal bits.
//
// What bounds it: the products, and shared memory beside them. A V2 tile is 8 products S (103 cycles each, both
// operands from shared memory) and 8 of P V (70, P in tensor memory): 1380 cycles; what the unpacking writes (64 KB,
// 512 cycles) and the products read (768) comes on top, as it uses the same port, and a tile takes 2150. V1: 3150, of
// which 2750 are its 32 products, a half of S's by zeros. Measured (calls one by one, each after a write of 256 MB):
// 20 ragged prompts of up to 2048 new tokens over up to 16384, G = 8 (V2) 1222 us, 930 TFLOP/s; 4 x 1024 over 4096, V1,
// 337 us, 800; 24 x 8 tokens over 32768, V2, where half of the 128 rows are empty, 394 us. Measured on the way:
// everything transposed, keys and channels on the 128 lanes and 64 queries as columns, 360 for the last and 2950 for the
// first; one O for both streams, its m handed on, slower for all; 8 unpacking warps for V1, and V in front of the next
// tile's K, 444 where 4 x 1024 took 353.
#include <cfloat>
#include <cmath>

#include "early.cuh"
#include "internal.h"
#include "kv4_chunk.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kRows = 128;
constexpr int kTile = 128;                       // keys (2^7)
constexpr int kSlot = kTile * 128 * 2;           // one plane of a tile in fp16
constexpr int kHalf = kSlot / 2;                 // 64 of its channels
constexpr float kPScale = 6.f, kMoveRef = 15.f;  // log2 of P's scale, and of the P at which the reference moves
constexpr int kNanSets = 8;
constexpr int kRing = 4;                         // tiles whose records' addresses are known

template <int KP>
struct Cfg {
  // What a unit costs besides its tiles, in tiles: its query, the wait for its first scores, the join and the output,
  // 9 to 12 thousand cycles with V2 (a tile 2150) and 13 with V1 (3150). (With 5 and 8, us: V2, 20 ragged prompts of up
  // to 2048 new and 16384 cached tokens 1406 and 1241, 100 of up to 300 and 1000 200 and 218, 64 of up to 64 and 30000
  // with G = 4 206 and 198; V1, 40 of up to 512 and 4096 161 and 181, 64 of up to 64 and 8000 134 and 151.)
  static constexpr int kUnitCost = KP == 1 ? 8 : 5;
  static constexpr int kStreams = KP == 1 ? 2 : 1;  // softmax warpgroups
  static constexpr int kRecs = KP == 1 ? 2 : 1, kUnpackWarps = 8 / kRecs;  // K's, and V's: records of a plane for each
  static constexpr int kKWarp = 4 * kStreams, kVWarp = kKWarp + kUnpackWarps, kMmaWarp = kVWarp + kUnpackWarps;
  static constexpr int kAddressWarp = kMmaWarp + 1;
  static constexpr int kThreads = (kMmaWarp + 4) * 32;
  static constexpr int kWidth = KP * 128;
  static constexpr int kSlots = KP == 1 ? 6 : 5;    // the ring of planes: of each tile K's, then V's
  static constexpr int kQ = kSlots * kSlot;         // Q: 64 channels of 128 rows at a time
  static constexpr int kSmall = kQ + kRows * kWidth * 2;
  static constexpr int kO = 2 * kTile;              // tensor memory: S (P in its place) twice, O of each stream
  static constexpr int kPiece = 2 * kRows + kRows * kWidth;  // floats: m, l, o
  // Registers a thread: the launch's (96 or 80) dealt out anew to the warpgroups
  static constexpr int kLaunchRegs = KP == 1 ? 96 : 80;
  static constexpr int kSoftmaxRegs = KP == 1 ? 128 : 152, kUnpackRegs = KP == 1 ? 88 : 64, kRestRegs = KP == 1 ? 48 : 64;
  static_assert(kSoftmaxRegs >= kLaunchRegs && kUnpackRegs <= kLaunchRegs && kRestRegs <= kLaunchRegs, "raised and lowered");
  static_assert(kStreams * kSoftmaxRegs + kUnpackWarps / 2 * kUnpackRegs + kRestRegs <= (kThreads / 128) * kLaunchRegs, "more registers than the launch has");
  static_assert(kThreads <= 768, "Scan");
  static_assert(kO + kStreams * kWidth <= 512, "tensor memory");
};

struct TileAt {
  const uint8_t* rec[8];
  int key0, left, unit, pad;  // its first key, keys from there on (0: the stream has ended), its unit's number
};
struct Small {  // behind Q
  int top[kRows];      // the exponent of the rows' largest query channel
  float2 join[kRows];  // V2, at a unit's end: the second stream's m and l, then both streams' weights
  uint64_t full[6], free[6], s_full[2], p_full[2], pv_done[2], q_full, teardown;
  uint64_t tile_full[kRing], tile_free[kRing];
  TileAt tile[kRing];
  int nan_key[kNanSets][16];
  uint32_t tmem;
  int abort, seg;      // seg: tiles of the unit whose Q is there, 0 behind the last
};

constexpr int kMaxThreads = 768;
struct Scan {  // at startup, in Q's place
  long long pre[kMaxThreads + 1], sum[kMaxThreads / 32];
  Walk walk;
};
template <int KP>
constexpr int smem_bytes() {
  return Cfg<KP>::kSmall + static_cast<int>(sizeof(Small));
}
static_assert(smem_bytes<1>() <= 232448 && smem_bytes<2>() <= 232448, "shared memory");

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
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return umma_idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

// Where plane p of the block's tile j lies in the ring (0 .. KP - 1: K's, then V's), and the phase of its slot's
// use. The ring's order is K(0), K(1), V(0), K(2), V(1), ..: V is needed a softmax later than K.
struct Place {
  int slot, phase;
};
template <int KP>
__device__ __forceinline__ Place place(int j, int p) {
  const uint32_t n = p >= KP ? 2 * KP * j + KP + p : j == 0 ? p : 2 * KP * j - KP + p, use = n / Cfg<KP>::kSlots;
  return {static_cast<int>(n - use * Cfg<KP>::kSlots), static_cast<int>(use & 1)};
}

template <int KP>
__global__ void __launch_bounds__(Cfg<KP>::kThreads, 1) kv4_chunk_kernel(const Kv4ChunkArgs a) {
  using C = Cfg<KP>;
  constexpr int kThreads = C::kThreads, kStreams = C::kStreams;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const s_q = smem + C::kQ;
  Small& sm = *reinterpret_cast<Small*>(smem + C::kSmall);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t slots = smem_u32(smem), q_at = smem_u32(s_q);
  auto bar = [](uint64_t& x) { return smem_u32(&x); };

  if (tid == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(bar(sm.full[i]), C::kUnpackWarps);
      mbar_init(bar(sm.free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sm.s_full[i]), 1);
      mbar_init(bar(sm.p_full[i]), 4);
      mbar_init(bar(sm.pv_done[i]), 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar(sm.tile_full[i]), 1);
      mbar_init(bar(sm.tile_free[i]), 2 * C::kUnpackWarps);
    }
    mbar_init(bar(sm.q_full), 4 * kStreams);
    mbar_init(bar(sm.teardown), 1);
    sm.abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  for (int i = tid; i < kNanSets * 16; i += kThreads) sm.nan_key[i >> 4][i & 15] = INT_MAX;
  if (warp == C::kMmaWarp) {
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

  if (warp >= C::kMmaWarp) {
    registers_down<C::kRestRegs>();
    if (warp == C::kMmaWarp && elect_one()) {
      // ================================ products ================================
      constexpr uint32_t idesc_s = idesc_f16(kRows, kTile, 0, 0), idesc_v = idesc_f16(kRows, 128, 0, 1);
      const uint64_t dq = umma_smem_desc(q_at, 16, 1024), dk = umma_smem_desc(slots, 16, 1024);
      const uint64_t dv = umma_smem_desc(slots, kHalf, 1024);
      int j = 0;
      bool ok = true;
      auto scores = [&](int t) {
        // (P of tile t - 2 lay where S goes)
        if (t >= 2 && !(ok = mbar_wait(bar(sm.pv_done[t & 1]), ((t - 2) >> 1) & 1, abrt))) return;
#pragma unroll 1
        for (int p = 0; p < KP; ++p) {
          const Place k = place<KP>(t, p);
          if (!(ok = mbar_wait(bar(sm.full[k.slot]), k.phase, abrt))) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
            mma_bf16_ss(tmem + (t & 1) * kTile, desc_add(dq, p * 2 * kHalf + off), desc_add(dk, k.slot * kSlot + off), idesc_s,
                        p > 0 || kk > 0);
          }
          tc_commit(bar(sm.free[k.slot]));
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
          if (!(ok = mbar_wait(bar(sm.p_full[j & 1]), (j >> 1) & 1, abrt))) break;
          const uint32_t o = tmem + C::kO + (kStreams == 2 ? (j & 1) * 128 : 0);
#pragma unroll 1
          for (int p = 0; p < KP; ++p) {
            const Place v = place<KP>(j, KP + p);
            if (!(ok = mbar_wait(bar(sm.full[v.slot]), v.phase, abrt))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts(o + p * 128, tmem + (j & 1) * kTile + kk * 8, desc_add(dv, v.slot * kSlot + kk * 2048), idesc_v,
                          i >= kStreams || kk > 0);
            tc_commit(bar(sm.free[v.slot]));
          }
          if (!ok) break;
          tc_commit(bar(sm.pv_done[j & 1]));
        }
      }
      // every product that was issued ends before tensor memory is given back
      tc_commit(bar(sm.teardown));
      mbar_wait(bar(sm.teardown), 0, nullptr);
    } else if (warp == C::kAddressWarp) {
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
  } else if (warp >= C::kKWarp) {
    // ================================ unpack ================================
    // A tile's bytes are loaded into registers before the tile before it is waited for (also where the
    // sequence has no such record, from page 0: no branch comes between loads in flight). Warp q of K's or
    // V's takes record q (V2: and q + 4) of each plane. A piece of 8 channels lies at its number XOR the
    // row's; lanes of a quarter-warp whose places would meet in the banks (t4 of 0 and 2, 1 and 3) take their
    // pieces in another order.
    registers_down<C::kUnpackRegs>();
    constexpr int kRecs = C::kRecs;
    const bool is_k = warp < C::kVWarp;
    const int q = warp - (is_k ? C::kKWarp : C::kVWarp), t4 = lane & 3, hi8 = lane >> 2;
    const bool far = t4 & 2;
    struct Tile {
      int key0, left, unit;
    };
    struct Data {
      uint4 lo[kRecs], hi[kRecs];
      uint32_t sc[kRecs];
    };
    Data d[KP];
    Tile next{}, tile;
    const uint8_t* src[kRecs] = {};
    int loaded = 0;
    bool ok = true;
    auto fetch = [&]() {  // the next tile's addresses; behind the stream's end they stay
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(sm.tile_full[loaded % kRing]), (loaded / kRing) & 1, abrt));
      const TileAt& at = sm.tile[loaded % kRing];
#pragma unroll
      for (int x = 0; x < kRecs; ++x) src[x] = at.rec[q + 4 * x] + (is_k ? 0 : KP * kKv4Plane);
      next.key0 = at.key0, next.left = ok ? at.left : 0, next.unit = at.unit;
      __syncwarp();
      if (next.left > 0) {
        if (lane == 0) mbar_arrive(bar(sm.tile_free[loaded % kRing]));
        ++loaded;
      }
    };
    auto load = [&](Data& x, int p) {
#pragma unroll
      for (int i = 0; i < kRecs; ++i) {
        const uint8_t* from = src[i] + p * kKv4Plane;
        x.lo[i] = ldg128(from + lane * 16);
        x.hi[i] = ldg128(from + lane * 16 + 512);
        x.sc[i] = ldg32(from + lane * 4 + kKv4PlaneCodes);
      }
    };
    auto dup = [](uint32_t two, int high) { return __byte_perm(two, 0, high ? 0x3232 : 0x1010); };
    auto put = [](uint32_t at, uint32_t word, uint32_t f) {
      uint32_t v[4];
      e2m1x8_to_half2(word, v);
      st_shared_v4(at, half2_mul(v[0], f), half2_mul(v[1], f), half2_mul(v[2], f), half2_mul(v[3], f));
    };
    // K: key 4 (hi8 / 2) + hi8 % 2 and that + 2, channels 32 t4 ..; V: tokens 4 t4 .., channels 16 hi8 ..
    const int row = q * 16 + (is_k ? 4 * (hi8 >> 1) + (hi8 & 1) : 4 * t4);
    const int c0 = is_k ? ((t4 & 1) * 4 + (t4 & 2)) ^ (row & 7) : ((hi8 & 3) * 2) ^ (row & 7) ^ (far ? 1 : 0);
    const uint32_t at0 = slots + (is_k ? t4 >> 1 : hi8 >> 2) * kHalf + row * 128;
    auto loop = [&](auto&& unpack) {
      fetch();
#pragma unroll
      for (int p = 0; p < KP; ++p) load(d[p], p);
      for (int j = 0; ok; ++j) {
        tile = next;
        if (tile.left <= 0) break;
#pragma unroll
        for (int p = 0; p < KP; ++p) {
          const Place to = place<KP>(j, (is_k ? 0 : KP) + p);
          ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(sm.free[to.slot]), to.phase ^ 1, abrt));
          if (!ok) break;
#pragma unroll
          for (int x = 0; x < kRecs; ++x) {
            const uint32_t base = at0 + to.slot * kSlot + x * 64 * 128;
            unpack(d[p].lo[x], d[p].hi[x], d[p].sc[x], p, tile.left - x * 64, x * 64, base + (c0 << 4), base + ((c0 ^ 1) << 4),
                   base + ((c0 ^ 2) << 4), base + ((c0 ^ 3) << 4));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sm.full[to.slot]));
          if (p == 0) fetch();
          load(d[p], p);
        }
      }
    };
    if (is_k) {
      loop([&](const uint4& lo, const uint4& hi, uint32_t sc, int, int left, int, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        uint32_t s0, s1;
        e4m3x4_to_half2(sc, s0, s1);
        if (left <= row) s0 = 0;
        if (left <= row + 2) s1 = 0;
        const uint32_t f0 = dup(s0, far), f1 = dup(s0, !far), g0 = dup(s1, far), g1 = dup(s1, !far);
        put(a0, far ? lo.z : lo.x, f0);
        put(a1, far ? lo.w : lo.y, f0);
        put(a2, far ? lo.x : lo.z, f1);
        put(a3, far ? lo.y : lo.w, f1);
        put(a2 + 256, far ? hi.z : hi.x, g0);  // two rows on
        put(a3 + 256, far ? hi.w : hi.y, g0);
        put(a0 + 256, far ? hi.x : hi.z, g1);
        put(a1 + 256, far ? hi.y : hi.w, g1);
      });
    } else {
      loop([&](const uint4& lo, const uint4& hi, uint32_t sc, int p, int left, int key, uint32_t a0, uint32_t a1, uint32_t a2,
               uint32_t a3) {
        const int live = left - row;
        if (live < 4) sc = live <= 0 ? 0u : sc & (0xffffffffu >> (32 - 8 * live));
        const uint32_t odd = ((sc & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // scales that are NaN
        if (odd) {
          atomicMin(&sm.nan_key[tile.unit & (kNanSets - 1)][p * 8 + hi8], tile.key0 + key + row + ((__ffs(odd) - 1) >> 3));
          sc &= ~((odd >> 7) * 0xffu);
        }
        uint32_t s01, s23;
        e4m3x4_to_half2(sc, s01, s23);
        const uint32_t f0 = dup(s01, 0), f1 = dup(s01, 1), f2 = dup(s23, 0), f3 = dup(s23, 1);
        put(a0, far ? lo.y : lo.x, f0);
        put(a1, far ? lo.x : lo.y, f0);
        put(a1 + 128, far ? lo.w : lo.z, f1);
        put(a0 + 128, far ? lo.z : lo.w, f1);
        put(a2 + 256, far ? hi.y : hi.x, f2);
        put(a3 + 256, far ? hi.x : hi.y, f2);
        put(a3 + 384, far ? hi.w : hi.z, f3);
        put(a2 + 384, far ? hi.z : hi.w, f3);
      });
    }
  } else {
    // ================================ softmax ================================
    registers_up<C::kSoftmaxRegs>();
    constexpr int kAll = kStreams * 128;
    const int wg = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    bool ok = true;
    int j = 0, unit = 0;
    // tokens that see no key get zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const Seq s = sequence<false>(a, b);
      const int z = hidden(a, s);
      const size_t width = static_cast<size_t>(a.H) * (KP == 2 ? 256 : a.group * 64);
      uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + s.q0 * width);
      for (size_t i = tid; i < z * width / 8; i += kAll) out[i] = make_uint4(0, 0, 0, 0);
    }
    const int per = KP == 2 ? 2 : a.group;  // rows of a token
    auto tiles_here = [](const Walk& x) { return static_cast<int>(max(0LL, min(static_cast<long long>(x.tiles - x.tile), x.todo))); };
    // A unit's queries: a half-warp a row, two rows at a time, kRounds times in batches of 8
    constexpr int kQWarps = 4 * kStreams, kBatches = kRows / 2 / kQWarps / 8;
    auto row_of = [&](int i) { return (i * kQWarps + warp) * 2 + (lane >> 4); };
    const int part = lane & 15;  // of 16 bytes: 8 in each 64 channels
    auto fetch = [&](uint4 (&x)[8], const Walk& u, int batch) {
      const int tok0 = u.rt * a.tokens, rows = min(a.tokens, u.Lq - tok0) * per;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = row_of(batch * 8 + i), t = r / per, sub = r - t * per;
        const size_t from = (static_cast<size_t>(u.q0 + tok0 + t) * a.H + u.h) * per + sub;
        x[i] = u.todo > 0 && r < rows ? *(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + from * 128) + part)
                                      : make_uint4(0, 0, 0, 0);
      }
    };
    auto write = [&](const uint4 (&x)[8], int batch) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = row_of(batch * 8 + i);
        const uint32_t m2 = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
        uint32_t top = max(m2 & 0xffffu, m2 >> 16);  // the largest magnitude's bits (ordered as the values are)
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = max(static_cast<int>(top >> 7) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);  // 2^(14 - e)
        if (part == 0) sm.top[r] = e;
        auto two = [&](uint32_t v) { return pack_half2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up); };
        const uint32_t at = q_at + r * 128 + (part >> 3) * kHalf + (((part & 7) ^ (r & 7)) << 4);
        const uint32_t mine = KP == 2 ? (r & 1) * 2 * kHalf : 0;
        st_shared_v4(at + mine, two(x[i].x), two(x[i].y), two(x[i].z), two(x[i].w));
        if (KP == 2) st_shared_v4(at + (2 * kHalf - mine), 0u, 0u, 0u, 0u);  // the other map's channels
      }
    };
    // The unit `u` (tiles_here of 0: the range's end) to the products, whose place for Q is free; `x`: its first batch.
    auto present = [&](uint4 (&x)[8], const Walk& u) {
      if (u.todo > 0) {
#pragma unroll
        for (int b = 0; b < kBatches; ++b) {
          if (b > 0) fetch(x, u, b);
          write(x, b);
        }
      }
      if (tid == 0) sm.seg = tiles_here(u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.q_full));
    };
    {
      uint4 x[8];
      fetch(x, w, 0);
      present(x, w);
      named_barrier_sync(1, kAll);
    }
    while (w.todo > 0) {
      const int seg = tiles_here(w);
      const bool starts = w.tile == 0, whole = starts && seg == w.tiles;
      const int tok0 = w.rt * a.tokens, toks = min(a.tokens, w.Lq - tok0), rows = toks * per;  // tokens and rows of the unit
      // what the row's S is to be multiplied with (never 0 or Inf, which a score of 0 or a masked one's Inf would
      // turn into NaN)
      const float scale = fminf(fmaxf(ldexpf(a.qk_scale, sm.top[row] - 14), FLT_MIN), FLT_MAX);
      // keys that the row sees (none where there is no such token)
      const int lim = row >= rows ? 0 : a.causal ? max(0, w.Lk - w.Lq + tok0 + row / per + 1) : w.Lk;
      const bool busy = quarter * 32 < rows;  // the warp has rows in use
      const int edge = __reduce_min_sync(0xffffffffu, row < rows ? lim : INT_MAX);
      float m = -FLT_MAX, l = 0.f;
      Walk next = w;  // (here its loads are not waited for)
      advance(a, next, seg);

      for (int i = 0; i < seg; ++i, ++j) {
        if (kStreams == 2 && (j & 1) != wg) continue;
        const int key0 = (w.tile + i) * kTile;
        ok = ok && mbar_wait(bar(sm.s_full[j & 1]), (j >> 1) & 1, abrt);
        __syncwarp();
        tc_fence_after();
        if (busy) {
          const uint32_t s_at = tmem + lanes + (j & 1) * kTile;
          const bool cut = key0 + kTile > edge;
          auto load = [&](float (&e)[32], int c) {
            uint32_t raw[32];
            tmem_ld32(s_at + c, raw);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) e[x] = __uint_as_float(raw[x]);
            if (cut) {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (key0 + c + x >= lim) e[x] = -INFINITY;
            }
            __syncwarp();
          };
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kTile; c += 32) {
            float e[32], t1 = -INFINITY;
            load(e, c);
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              top = fmax3(top, e[x], e[x + 1]);
              t1 = fmax3(t1, e[x + 2], e[x + 3]);
            }
            top = fmaxf(top, t1);
          }
          top *= scale;
          const bool move = top - m > kMoveRef;
          if (__any_sync(0xffffffffu, move)) {
            const float to = move ? fmaxf(m, __fsub_ru(top, kPScale)) : m, f = ex2_approx(m - to);
            m = to;
            l *= f;
            if (i >= kStreams) {  // O holds earlier tiles (V2: S of this one came behind their product)
              if (kStreams == 1) {
                ok = ok && mbar_wait(bar(sm.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, abrt);
                __syncwarp();
                tc_fence_after();
              }
#pragma unroll 1
              for (int c = 0; c < C::kWidth; c += 32) {
                const uint32_t at = tmem + lanes + C::kO + wg * 128 + c;
                uint32_t o[32];
                tmem_ld32(at, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                tmem_st32(at, o);
              }
            }
          }
          const uint64_t scale2 = f2pack(scale, scale), ref2 = f2pack(-m, -m);
          uint64_t sum = f2pack(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < kTile; c += 32) {
            float e[32];
            load(e, c);
            uint32_t pk[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float e0, e1;
              f2unpack(f2fma(f2pack(e[2 * x], e[2 * x + 1]), scale2, ref2), e0, e1);
              const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
              sum = f2add(sum, f2pack(p0, p1));
              pk[x] = pack_half2(p0, p1);
            }
            tmem_st16(s_at + c / 2, pk);
          }
          float l0, l1;
          f2unpack(sum, l0, l1);
          l += l0 + l1;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.p_full[j & 1]));
      }

      // ---- the unit's end ----
      // The next unit's queries first: their products run meanwhile. Q's place is free once the last scores are there.
      const int t = row / per, sub = row - t * per;
      const size_t token = static_cast<size_t>(w.q0) + tok0 + t;
      float lam = 0.f;
      {
        uint4 x[8];
        fetch(x, next, 0);
        if (whole && (row & 1) && row < rows)
          lam = KP == 2 ? *(a.lambda + w.h) : *(a.lam_logit + token * (a.H * per / 2) + (w.h * per + sub) / 2);
        if (kStreams == 2) ok = ok && mbar_wait(bar(sm.s_full[(j - 1) & 1]), ((j - 1) >> 1) & 1, abrt);
        if (kStreams == 2 && wg == 1) sm.join[row] = make_float2(m, l);
        named_barrier_sync(1, kAll);  // (nor does a warp still want this unit's exponents)
        present(x, next);
      }
      float w0 = 1.f, w1 = 0.f;  // what the streams' O are to be multiplied with
      if constexpr (kStreams == 2) {
        if (wg == 0) {
          const float2 other = sm.join[row];
          const float m0 = m, m1 = other.x;
          m = fmaxf(m0, m1);
          w0 = ex2_approx(m0 - m), w1 = ex2_approx(m1 - m);
          l = fmaf(l, w0, other.y * w1);
          const float f = whole ? 1.f / l : 1.f;
          w0 *= f, w1 *= f;
          sm.join[row] = make_float2(w0, w1);
        }
        named_barrier_sync(1, kAll);
        if (wg == 1) w0 = sm.join[row].x, w1 = sm.join[row].y;
      } else if (whole) {
        w0 = 1.f / l;
      }
      if (kStreams == 2 && seg > 1) ok = ok && mbar_wait(bar(sm.pv_done[(j - 2) & 1]), ((j - 2) >> 1) & 1, abrt);
      ok = ok && mbar_wait(bar(sm.pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1, abrt);
      __syncwarp();
      tc_fence_after();
      // (an O that no tile of this unit went to is left out)
      const bool use0 = kStreams == 1 || seg > 1 || ((j - 1) & 1) == 0, use1 = kStreams == 2 && (seg > 1 || ((j - 1) & 1) == 1);
      const int* nan = sm.nan_key[unit & (kNanSets - 1)];
      const uint32_t o_at = tmem + lanes + C::kO;
      const float kNan = __int_as_float(0x7fffffff);
      auto load_o = [&](float (&y)[32], int c, float f) {  // channels c .. c + 31
        uint32_t o[32];
        if (use0) {
          tmem_ld32(o_at + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) y[x] = __uint_as_float(o[x]) * (w0 * f);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) y[x] = 0.f;
        }
        if (use1) {
          tmem_ld32(o_at + 128 + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) y[x] = fmaf(__uint_as_float(o[x]), w1 * f, y[x]);
        }
        const bool bad0 = nan[c >> 4] < lim, bad1 = nan[(c >> 4) + 1] < lim;
        if (__any_sync(0xffffffffu, bad0 || bad1)) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x < 16 ? bad0 : bad1) y[x] = kNan;
        }
      };
      if (!busy) {
      } else if (!whole) {
        // a piece: m, l, and o by fours of channels, so that a warp's stores lie side by side
        float* rec = a.pieces + static_cast<size_t>(2 * blockIdx.x + (starts ? 1 : 0)) * C::kPiece;
        if (wg == 0) rec[row] = m, rec[kRows + row] = l;
#pragma unroll 1
        for (int c = wg * 32; c < C::kWidth; c += 32 * kStreams) {
          float y[32];
          load_o(y, c, 1.f);
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *reinterpret_cast<float4*>(rec + 2 * kRows + ((c + x) / 4 * kRows + row) * 4) = make_float4(y[x], y[x + 1], y[x + 2], y[x + 3]);
        }
      } else {
        // this row's share of its pair's output: f times o (the odd row with its lambda, negative)
        float f = 0.f;
        if (lim > 0) {
          f = a.v_mul;
          if (row & 1) f *= KP == 2 ? -lam : -1.f / (1.f + __expf(-lam));
        }
        float g = 1.f;  // V1: the norm's factor and the scale
        // 32 channels of the pair's output, 16 for each of its two lanes
        auto pair = [&](float (&z)[16], int c) {
          float y[32];
          load_o(y, c, f);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float give = row & 1 ? y[x] : y[x + 16], keep = row & 1 ? y[x + 16] : y[x];
            z[x] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
          }
        };
        if (KP == 2) {
          // into O's place on the way, for the second pass
          float ss = 0.f;
#pragma unroll 1
          for (int c = 0; c < C::kWidth; c += 32) {
            float z[16];
            pair(z, c);
            uint32_t raw[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) ss = fmaf(z[x], z[x], ss), raw[x] = __float_as_uint(z[x]);
            tmem_st16(o_at + c, raw);
          }
          tmem_wait_st();
          if (a.flags & 2) {
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            g = 1.f / sqrtf(ss / 256.f + a.eps);
          }
          if (a.flags & 4) g *= 1.f - a.lambda_init;
        }
        const size_t at = KP == 2 ? (token * a.H + w.h) * 256 : (token * (a.H * per / 2) + (w.h * per + sub) / 2) * 128;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at + (row & 1) * 16;
        const bool weights = KP == 2 && (a.flags & 2) && a.norm_w;
        const bool store = row < rows && dbg_index_ok(static_cast<long long>(token), a.total);
#pragma unroll 1
        for (int c = wg * 32; c < C::kWidth; c += 32 * kStreams) {
          float z[16];
          if constexpr (KP == 2) {
            uint32_t raw[16];
            tmem_ld16(o_at + c, raw);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) z[x] = __uint_as_float(raw[x]) * g;
            if (weights) {
              const float4* wgt = reinterpret_cast<const float4*>(a.norm_w + c + (row & 1) * 16);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float4 v = wgt[x];
                z[4 * x] *= v.x, z[4 * x + 1] *= v.y, z[4 * x + 2] *= v.z, z[4 * x + 3] *= v.w;
              }
            }
          } else {
            pair(z, c);
          }
          uint32_t o[8];
#pragma unroll
          for (int x = 0; x < 16; x += 2)  // (zeros where no key is seen, whatever the weight and the scale hold)
            o[x / 2] = lim > 0 ? pack_bf16x2(z[x], z[x + 1]) : 0u;
          if (store) {
            *reinterpret_cast<uint4*>(out + c) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      __syncwarp();
      tc_fence_before();
      named_barrier_sync(1, kAll);
      if (tid < 16) sm.nan_key[unit & (kNanSets - 1)][tid] = INT_MAX;
      ++unit;
      w = next;
    }
  }

  // ---- teardown ----
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins, of each unit whose tiles lie in more than one range, its pieces: that of the range that begins it and
// of the ranges that begin inside it, in this order. Block (i, y): the unit that range i + 1 begins inside,
// if no earlier range does, and every gridDim.y-th of its tokens (V1) or pairs (V2) from y on; a thread a channel.
template <int KP>
__global__ void __launch_bounds__(KP * 128) kv4_chunk_join_kernel(const Kv4ChunkArgs a) {
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
  const size_t piece = static_cast<size_t>(a.rows) * (2 + NT);
  float wgt = 1.f;
  if (KP == 2 && (a.flags & 2) && a.norm_w) wgt = *(a.norm_w + tid);
  for (int o = blockIdx.y; o < outs; o += gridDim.y) {
    const int c[2] = {2 * o, 2 * o + 1};  // its rows
    float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f}, v[2] = {0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < pieces; ++k) {
      const float* r = a.pieces + static_cast<size_t>(2 * (i0 + k) + (k == 0 ? 1 : 0)) * piece;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mk = r[c[e]], lk = r[a.rows + c[e]], vk = r[2 * a.rows + (tid / 4 * a.rows + c[e]) * 4 + tid % 4];
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

template <int KP>
cudaError_t launch_join(const Kv4ChunkArgs& a, cudaStream_t st) {
  g_launched.store(true, std::memory_order_relaxed);
  cudaLaunchAttribute at[1] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.grid - 1, a.rows < kRows ? a.rows / 4 : 8);
  cfg.blockDim = dim3(KP * 128);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_chunk_join_kernel<KP>, a);
}

template <int KP>
cudaError_t launch(Kv4ChunkArgs a, cudaStream_t st) {
  static std::atomic<uint64_t> raised{};
  a.rows = kRows;
  a.tokens = kRows / (KP == 2 ? 2 : a.group);
  a.tok_log2 = KP == 2 ? 6 : a.group == 2 ? 6 : a.group == 4 ? 5 : 4;
  a.tile_log2 = 7;
  a.unit_cost = Cfg<KP>::kUnitCost;
  page_magic(a.page_size >> 4, &a.rec_magic, &a.rec_shift);
  // no more blocks than the tables' capacity can give ranges: a sequence's tiles of tokens overlap the total's
  const long long tiles = (static_cast<long long>(a.max_pages) * a.page_size + kTile - 1) / kTile;
  const long long units = (static_cast<long long>(a.total) / a.tokens + a.B) * a.H;
  const long long most = units >= kChunkSms ? kChunkSms : (tiles + a.unit_cost) * units / kMinCost;
  a.grid = static_cast<int>(most < 1 ? 1 : most > kChunkSms ? kChunkSms : most);
  cudaError_t e = launch_early_large(kv4_chunk_kernel<KP>, a.grid, Cfg<KP>::kThreads, smem_bytes<KP>(), smem_bytes<KP>(), st, 1, a, raised);
  if (e != cudaSuccess || a.grid == 1) return e;
  return launch_kv4_chunk_join(a, st);
}

}  // namespace

size_t kv4_chunk_workspace_bytes(int group) {
  return 2 * static_cast<size_t>(kChunkSms) * (group == 0 ? Cfg<2>::kPiece : Cfg<1>::kPiece) * sizeof(float);
}

cudaError_t launch_kv4_chunk(const Kv4ChunkArgs& a, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  if (kv4_chunk_few(a)) return launch_kv4_chunk_few(a, st);
  return a.group == 0 ? launch<2>(a, st) : launch<1>(a, st);
}

cudaError_t launch_kv4_chunk_join(const Kv4ChunkArgs& a, cudaStream_t st) {
  return a.group == 0 ? launch_join<2>(a, st) : launch_join<1>(a, st);
}

cudaError_t status_chunk_kv4(int* v) { return launched_status(v); }

}  // namespace da
