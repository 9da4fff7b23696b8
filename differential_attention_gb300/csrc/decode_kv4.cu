// decode_kv4.cu -- decode attention over the 4-bit cache: one query token per sequence.
//
// For one (sequence, KV head), a "row" here, there are up to 8 softmaxes over the same keys (V1: the two
// maps of a head; V2: the G query heads of a group), each with an output of V's width:
//   o = sum_j 2^(s_j - m) v_j,   l = sum_j 2^(s_j - m),   s_j = log2(e) / sqrt(d) q . k_j,
// and then V1: o1/l1 - lambda o2/l2, the norm and the scale; V2: o_2p/l_2p - sigmoid(lam) o_2p+1/l_2p+1.
//
// What bounds it: the cache's bytes, 144 (V2) or 288 (V1) a key, read once. At 6.8 TB/s an SM gets
// 23.5 bytes a cycle, a key of 256 channels every 6.1 cycles, so unpacking and both products have
// to stay under that: some 24 instructions a key over all four schedulers.
//
// Products. Both run as m16n8k16 with the keys or V's channels on the 16 rows and the query heads
// on the 8 columns, which is where G = 8 fits exactly:
//   S^T [16 keys x 8] = K [16 keys x 128] Q^T,    O^T [channels x 8] += V^T [channels x 16 keys] P^T.
// The operands come straight from registers: a record (16 tokens) holds its bytes in the order in
// which the lanes need them, so one 16-byte shared-memory load gives a lane the codes of four
// products, one cvt turns a byte into two fp16 values (exact: an e2m1 times an e4m3 has at most 6
// significant bits), and one multiply puts the scale on. A tensor-memory product would want the
// unpacked tile written to shared memory first, 512 bytes a key at 128 bytes a cycle: 4 of the 6.1
// cycles for the writes alone. P^T's fragment is S^T's transposed, by movmatrix.
//
// Numerics. Q enters as fp16 after a power of two of its own for each head (its largest channel at
// 2^14 .. 2^15; a channel at 2^-17 still has bf16's 8 bits, below that it is rounded to multiples of
// 2^-24: off by 2^-39 of the largest at most, whatever the keys hold there). P is rounded to fp16 at 2^10 times its value against the reference m, so that its absolute
// error is 2^-35 of the largest probability; m follows the running maximum only where a score
// passes it by 2^4, which leaves every P below 2^14. Sums and statistics are fp32.
//
// Work. The rows, one after the other, are cut into equal ranges, one for each resident block, whatever
// the sequences' lengths; a row counts its tiles and a fixed cost. A block walks its range: a row that
// lies in it whole is finished there; the pieces of one that does not go to the workspace, at most
// two a block, and the second kernel merges them, in the order of the ranges. Where the tables hold few
// keys for each resident block, a row is cut over the blocks of a cluster instead, which join through
// each other's shared memory: one launch, no workspace. (Tried and dropped, V2 with lengths of 1 to 16K, 52
// us at the time: two ranges a block, the second taken over by cluster launch control, 58 us, as each
// range adds pieces; the last block of a row merging it, without a second kernel, 60 us, as the blocks
// wait for their fence and their count; shares by a block's age on its SM, whose schedulers serve the
// older first, 52 us, and 400 instead of 388 for 64 x 32768 keys.)
//
// Where it stands: 64 x 32768 keys, 8 KV heads, G = 8 (2.42 GB): 360 us, 6.71 TB/s, where a copy reaches
// 6.78; with all pages in L2 the same work takes as long, so that the unpacking (116 of 245 instructions a
// record go to the ALU pipe, most of them the 64 conversions) is as near its limit as the memory. 96
// sequences of 1 to 16K keys, G = 4 (235 MB): 49 us, of which the loads alone take 39 and the second kernel
// 3. V1, 24 x 32768 keys, 12 heads (2.72 GB): 405 us, 6.71 TB/s. While all blocks run, tiles arrive at 7.1
// TB/s; what is lost is the end, as the SMs, and the blocks of one SM, get unequal shares of it (the first
// are done after 85 % of the time). Ranges that the blocks take late, by a counter, even that out (the last
// tile of the 32768 keys arrives after 345 instead of 355 us), but their pieces cost as much: the call took
// 365 to 368.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "early.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kSms = 152;
constexpr int kFewTiles = 4;
constexpr float kPScale = 10.f;                  // log2 of P's scale
constexpr float kMoveRef = 14.f;                 // log2 P at which the reference moves

template <int KP>
struct Cfg {
  // Measured, V2, 64 x 32768 keys, 367 us so: 4 blocks an SM at 96 registers 375; 1 record a warp and 4
  // blocks 415; 4 records and 2 blocks 384; 6 warps and 2 blocks 446 (they lie unevenly on the four
  // schedulers); 8 warps and 2 blocks 421, 12 and 1 523 (more of them wait for each tile). V1, 24 x 32768
  // keys x 12, 405 us so: 1 record a warp and 3 blocks 412.
  static constexpr int kWarps = 4;               // consumer warps (an even number, at least 4)
  static constexpr int kThreads = (kWarps + 1) * 32;  // and a producer
  static constexpr int kRecs = 2;                // records of a tile for each of them
  static constexpr int kTileRecs = kWarps * kRecs;
  static constexpr int kTileKeys = 16 * kTileRecs;
  static constexpr int kCtas = KP == 1 ? 3 : 2;  // blocks of an SM
  static constexpr int kGrid = kSms * kCtas;
  static constexpr int kRowCost = 2;             // what a row costs besides its tiles, in tiles
  static constexpr int kMinCost = KP == 1 ? 3 : 2;  // the smallest range
  static constexpr int kRecord = 2 * KP * kKv4Plane;
  static constexpr int kWidth = KP * 128;
  static constexpr int kMaxCols = KP == 1 ? 8 : 2;
  static constexpr int kQBytes = kMaxCols * 256;
  static constexpr int kStage = kTileRecs * kRecord + kQBytes;
  static constexpr int kStages = KP == 1 ? 3 : 2;
  static constexpr int kPitch = kWidth + 4;      // floats of one column's row in the exchange
  static constexpr int kSmem = kStages * kStage + kWarps / 2 * kMaxCols * kPitch * 4;
  // Threads of the second kernel, with few rows and else. Small blocks find room beside the first kernel's
  // last ones, large ones have more pieces under way (V2, 96 sequences of 1 to 16K keys: 48.8 us with 256,
  // 50.0 with 512; V1, 48 of 1 to 9001: 41.6 and 41.2. Few rows: a V1 row of 65000 keys 19.8 with 1024, 29.1
  // with 512; a V2 row of 200000 20.5 and 27.9).
  static constexpr int kMergeFew = 1024, kMerge = KP == 1 ? 256 : 512;
};

struct Params {
  Kv4DecodeArgs a;
  int cols, grid;  // grid: by rows, the blocks of a cluster
  float* rec;  // [2 * grid][2 cols + cols * width]: m, l, o of a piece
};

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
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float a;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a) : "r"(addr) : "memory");
  return a;
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
// place in the walk over rows (sequence-major, heads inner)
struct Walk {
  int b, h, tile, tiles, len;
  int todo;         // tiles of the range, and the costs of the rows that begin in it, from here on
  long long first;  // where the row's tiles begin among all costs
};
// kEarly: before grid_wait(), in a kernel that knows of the write by the release of the one before it; from
// L2, so that no line an SM kept from an earlier kernel is read.
template <bool kEarly = false>
__device__ __forceinline__ int clamp_len(const Kv4DecodeArgs& a, int b) {
  const int cap = a.max_pages * a.page_size;
  const int n = kEarly ? __ldcg(a.seqlens + b) : *(a.seqlens + b);
  return n < 0 ? 0 : n > cap ? cap : n;
}
template <int KP>
__device__ __forceinline__ int tiles_of(int len) {
  return (len + Cfg<KP>::kTileKeys - 1) / Cfg<KP>::kTileKeys;
}
// what a row takes of a range: its tiles, and kRowCost for its query, its join and its output
template <int KP>
__device__ __forceinline__ int cost_of(int len) {
  return len == 0 ? 0 : tiles_of<KP>(len) + Cfg<KP>::kRowCost;
}
template <int KP>
__device__ __forceinline__ void next_row(const Kv4DecodeArgs& a, Walk& w) {
  w.first += w.tiles + Cfg<KP>::kRowCost;
  w.todo -= Cfg<KP>::kRowCost;
  w.tile = 0;
  if (++w.h < a.H) return;
  w.h = 0;
  do {
    if (++w.b >= a.B) return;  // the range ends here
    w.len = clamp_len(a, w.b);
  } while (w.len == 0);
  w.tiles = tiles_of<KP>(w.len);
}

// x / y for 0 <= x, 0 < y; nearly always both have 32 bits
__device__ __forceinline__ long long div(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
// 0 .. total cut in n equal parts
struct Cut {
  long long total;
  int n;
  __device__ __forceinline__ Cut(long long total_, int n_) : total(total_), n(n_) {}
  __device__ __forceinline__ long long start(int i) const { return div(total * i, n); }
  // the last part that begins at or before x < total: the largest i with total i / n < x + 1
  __device__ __forceinline__ int owner(long long x) const { return static_cast<int>(div((x + 1) * n - 1, total)); }
};

// The batch's rows one behind the other, cut in n equal parts. pre[i]: the costs (of one head) before
// thread i's share of the sequences. A whole block of NT threads.
template <int KP, int NT, bool kEarly>
struct Ranges {
  long long pre[NT + 1];
  long long sum[NT / 32];

  __device__ __forceinline__ void fill(const Kv4DecodeArgs& a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (a.B + NT - 1) / NT;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    long long incl = 0;
    for (int b = lo; b < hi; ++b) incl += cost_of<KP>(clamp_len<kEarly>(a, b));
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
  }
  __device__ __forceinline__ long long total(const Kv4DecodeArgs& a) const { return pre[NT] * a.H; }
  static __device__ __forceinline__ int count(long long total, int grid) {
    const long long want = total / Cfg<KP>::kMinCost;
    return static_cast<int>(want < 1 ? 1 : want > grid ? grid : want);
  }
  // where range r of n begins (a whole warp)
  __device__ __forceinline__ void locate(const Kv4DecodeArgs& a, const Cut& cut, int r, Walk& w) const {
    const int lane = threadIdx.x & 31, per = (a.B + NT - 1) / NT;
    const long long t0 = cut.start(r), t1 = cut.start(r + 1);
    w = Walk{};
    if (t1 <= t0) return;
    int share = 0;
    for (int i = 0; i < NT; i += 32)
      if (const unsigned hit = __ballot_sync(0xffffffffu, pre[i + lane] * a.H <= t0 && t0 < pre[i + lane + 1] * a.H)) {
        share = i + __ffs(hit) - 1;
        break;
      }
    long long at = pre[share];
    const int end = min(a.B, (share + 1) * per);
    for (int b0 = share * per; b0 < end; b0 += 32) {
      const int b = b0 + lane, len = b < end ? clamp_len<kEarly>(a, b) : 0, cost = cost_of<KP>(len);
      int incl = cost;
      if (per > 1) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
      }
      if (const unsigned hit = __ballot_sync(0xffffffffu, t0 < (at + incl) * a.H)) {
        const int l = __ffs(hit) - 1;
        at += __shfl_sync(0xffffffffu, incl - cost, l);
        w.b = b0 + l;
        w.len = __shfl_sync(0xffffffffu, len, l);
        break;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    w.tiles = tiles_of<KP>(w.len);
    const int cost = w.tiles + Cfg<KP>::kRowCost;
    w.h = static_cast<int>(div(t0 - at * a.H, cost));
    w.first = at * a.H + static_cast<long long>(w.h) * cost + Cfg<KP>::kRowCost;
    w.tile = static_cast<int>(max(t0 - w.first, 0LL));
    w.todo = static_cast<int>(t1 - max(t0, w.first));
  }
};

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

// O^T += V^T P^T of one record and plane: rows g and g + 8 of product j are channels 16g + 2j and + 1.
// `keep`: a byte of ones for each of this lane's tokens 4t .. 4t + 3 that counts; the others' scale is 0.
__device__ __forceinline__ void outputs(float (*o)[4], uint32_t at, int lane, uint32_t keep, uint32_t b0, uint32_t b1) {
  const uint4 va = lds128(at), vb = lds128(at + 512);
  const uint32_t sc = lds32(at - lane * 12 + kKv4PlaneCodes);
  uint32_t s01, s23;
  e4m3x4_to_half2(sc & keep, s01, s23);
  // pairs of tokens side by side: the low nibbles of two rows' bytes, then the high ones
  const uint32_t r0[2] = {va.x, va.y}, r1[2] = {va.z, va.w}, r2[2] = {vb.x, vb.y}, r3[2] = {vb.z, vb.w};
  constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t e01[4], d01[4], e23[4], d23[4];
    e2m1x8_to_half2((r0[k] & kLow) | ((r1[k] << 4) & ~kLow), e01);
    e2m1x8_to_half2(((r0[k] >> 4) & kLow) | (r1[k] & ~kLow), d01);
    e2m1x8_to_half2((r2[k] & kLow) | ((r3[k] << 4) & ~kLow), e23);
    e2m1x8_to_half2(((r2[k] >> 4) & kLow) | (r3[k] & ~kLow), d23);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mma(o[4 * k + i], half2_mul(e01[i], s01), half2_mul(d01[i], s01), half2_mul(e23[i], s23),
          half2_mul(d23[i], s23), b0, b1);
  }
}

// V1's factor for a whole row of 256 channels: the norm's 1 / rms and the fixed scale. ss: the squares of
// this thread's two channels. The first four warps.
__device__ __forceinline__ float norm_scale(const Kv4DecodeArgs& a, float ss, float* s_red) {
  float f = 1.f;
  if (a.flags & 2) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = ss;
    named_barrier_sync(2, 128);
    ss = (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
    f = 1.f / sqrtf(ss / 256.f + a.eps);
  }
  return (a.flags & 4) ? f * (1.f - a.lambda_init) : f;
}

// kByRow: one row for each cluster of p.grid blocks
template <int KP, bool kByRow>
__global__ void __launch_bounds__(Cfg<KP>::kThreads, Cfg<KP>::kCtas) kv4_decode_kernel(const Params p) {
  using C = Cfg<KP>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * C::kStages];
  __shared__ Ranges<KP, kThreads, false> s_ranges;
  __shared__ int s_abort;
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  __shared__ float s_red[kWarps];
  const Kv4DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t ring = smem_u32(smem), bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (C::kStages + s); };
  float* s_o = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
  float* s_x = reinterpret_cast<float*>(smem);  // by rows: the block's piece, m, l, o

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);
    }
    fence_barrier_init();
    s_abort = 0;
  }

  grid_wait();
  grid_release();
  Walk w{};
  int n = 0;
  const int range = blockIdx.x;
  if constexpr (kByRow) {
    const int row = blockIdx.x / p.grid, rank = blockIdx.x - row * p.grid;
    w.b = row / a.H;
    w.h = row - w.b * a.H;
    w.len = clamp_len(a, w.b);
    w.tiles = tiles_of<KP>(w.len);
    const int per = (w.tiles + p.grid - 1) / p.grid;
    w.tile = min(rank * per, w.tiles);
    w.todo = min(per, w.tiles - w.tile);
    __syncthreads();
  } else {
    s_ranges.fill(a);
    const long long total = s_ranges.total(a);
    n = s_ranges.count(total, p.grid);
    if (range >= n) return;
    s_ranges.locate(a, Cut(total, n), range, w);
  }

  if (warp == kWarps) {
    // Producer. Lane i looks up the page of record i of the next tiles of the row (32 records); the
    // lanes of a tile's records then copy one each, and lane 0 the row's query with its first tile.
    // The next batch's pages are looked up before the copies of this one.
    constexpr int kBatch = 32 / C::kTileRecs;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool alive = true, first = true;
    const int lane_rec = min(lane, kBatch * C::kTileRecs - 1);
    auto look_up = [&](int tile) {  // the page of record tile * kTileRecs + lane, if the row has it
      const int key = (tile * C::kTileRecs + lane_rec) * 16;
      if (key >= w.len || !dbg_index_ok(key / a.page_size, a.max_pages)) return 0;
      return *(a.block_table + static_cast<size_t>(w.b) * a.max_pages + key / a.page_size);
    };
    int page = w.todo > 0 ? look_up(w.tile) : 0;
    while (w.todo > 0 && alive) {
      const int batch = min(min(kBatch, w.tiles - w.tile), w.todo);
      const int r = w.tile * C::kTileRecs + lane, records = (w.len + 15) >> 4;
      const bool mine_ok = lane < batch * C::kTileRecs && r < records;
      if (mine_ok && (page < 0 || page >= a.num_pages)) {
        flag_device_error(DEV_BAD_INDEX);
        page = 0;
      }
      const int off = r * 16 % a.page_size;
      const uint8_t* src =
          a.pool + ((static_cast<size_t>(page) * a.H + w.h) * (a.page_size >> 4) + (off >> 4)) * C::kRecord;
      if (w.tile + batch < w.tiles) page = look_up(w.tile + batch);
      for (int i = 0; i < batch; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty(stage), phase ^ 1, &s_abort))) {
          alive = false;
          break;
        }
        const uint32_t dst = ring + stage * C::kStage;
        if (lane == 0) {
          const int here = min(C::kTileRecs, records - (w.tile + i) * C::kTileRecs);
          const uint32_t q_bytes = first ? p.cols * 256 : 0;
          mbar_arrive_expect_tx(full(stage), here * C::kRecord + q_bytes);
          if (first)
            bulk_load(dst + C::kTileRecs * C::kRecord,
                      static_cast<const uint8_t*>(a.q) + (static_cast<size_t>(w.b) * a.H + w.h) * (p.cols * 256), q_bytes,
                      full(stage));
        }
        __syncwarp();
        if (mine_ok && lane / C::kTileRecs == i)
          bulk_load(dst + (lane % C::kTileRecs) * C::kRecord, src, C::kRecord, full(stage));
        first = false;
        ++issued;
        if (++stage == C::kStages) stage = 0, phase ^= 1;
      }
      w.todo -= batch;
      w.tile += batch;
      if (!kByRow && w.tile == w.tiles) {
        next_row<KP>(a, w);
        first = true;
        if (w.todo > 0) page = look_up(w.tile);
      }
    }
    if (!alive) {
      // a wait ran out: the copies in flight still land in this block's memory
      for (int back = 0; back < min(issued, C::kStages); ++back) {
        if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
        mbar_wait_limit(full(stage), phase, nullptr, kWaitLimitNs);
      }
    }
    if constexpr (!kByRow) return;
  }

  // Consumers.
  if (warp < kWarps) {
    const int g = lane >> 2, t = lane & 3;
    const int cols = p.cols;
    uint4 qf[4];                 // Q^T fragments: channels 32t + 8k .. + 7 of column g
    float cs0 = 0.f, cs1 = 0.f;  // what a sum of columns 2t and 2t + 1 is to be multiplied with
    float o[KP * 8][4];
    float m0, m1, l0, l1;        // references (less kPScale) and sums of columns 2t, 2t + 1
    int stage = 0;
    uint32_t phase = 0;
    bool alive = true;

    auto load_q = [&](uint32_t at) {
      uint32_t raw[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) raw[i] = 0;
      if (g < cols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = lds128(at + g * 256 + t * 64 + i * 16);
          raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
        }
      }
      uint32_t top = 0;  // the largest magnitude's bits (ordered as the values are)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, max(raw[i] & 0x7fffu, (raw[i] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max(static_cast<int>(top >> 7) - 127, -100);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);     // 2^(14 - e)
      // (never 0 or Inf, which a masked score's Inf or a score of 0 would turn into NaN)
      const float down = fminf(fmaxf(ldexpf(a.qk_scale, e - 14), FLT_MIN), FLT_MAX);
      auto two = [&](uint32_t x) { return pack_half2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up); };
#pragma unroll
      for (int k = 0; k < 4; ++k) qf[k] = make_uint4(two(raw[4 * k]), two(raw[4 * k + 1]), two(raw[4 * k + 2]), two(raw[4 * k + 3]));
      cs0 = __shfl_sync(0xffffffffu, down, 8 * t);
      cs1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
    };
    auto wait = [&]() {
      if (__all_sync(0xffffffffu, mbar_try_wait(full(stage), phase))) return;
      alive = __all_sync(0xffffffffu, alive && mbar_wait(full(stage), phase, &s_abort));
    };

    // empty places in the batch get zeros
    for (int b = range; !kByRow && b < a.B; b += n)
      if (clamp_len(a, b) == 0) {
        const size_t size = static_cast<size_t>(a.H) * (cols / 2) * C::kWidth;
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + b * size);
        for (size_t i = tid; i < size / 8; i += kWarps * 32) out[i] = make_uint4(0, 0, 0, 0);
      }
    if (kByRow && w.todo <= 0)  // a piece of no keys
      for (int i = tid; i < C::kMaxCols * (2 + C::kWidth); i += kWarps * 32) s_x[i] = i < C::kMaxCols ? -FLT_MAX : 0.f;
    while (w.todo > 0) {
      const int seg = min(w.tiles - w.tile, w.todo);  // tiles of this row in the range
      const bool starts = w.tile == 0, whole = !kByRow && starts && seg == w.tiles;
      wait();
      load_q(ring + stage * C::kStage + C::kTileRecs * C::kRecord);
#pragma unroll
      for (int j = 0; j < KP * 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      m0 = m1 = -FLT_MAX;
      l0 = l1 = 0.f;
      // One tile; `last`: it may be the row's last one, and short.
      auto take = [&](int i, auto last) {
        constexpr int R = C::kRecs;
        // record w + kWarps r of the tile is warp w's; `left`: keys from its first one on
        const int left = last ? w.len - ((w.tile + i) * C::kTileRecs + warp) * 16 : 0;
        if (alive && !(last && left <= 0)) {
          const uint32_t rec = ring + stage * C::kStage + warp * C::kRecord + lane * 16;
          float y[R][4];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t at = rec + r * kWarps * C::kRecord;
            if constexpr (KP == 1) {
              scores(y[r], at, lane, qf);
            } else {  // V1: column 0 from the first plane, column 1 from the second
              float s1[4], s2[4];
              scores(s1, at, lane, qf);
              scores(s2, at + kKv4Plane, lane, qf);
              y[r][0] = s1[0], y[r][1] = s2[1], y[r][2] = s1[2], y[r][3] = s2[3];
            }
          }
          uint32_t keep[R];
#pragma unroll
          for (int r = 0; r < R; ++r) keep[r] = 0xffffffffu;
          if (last && left < 16 * (1 + (R - 1) * kWarps)) {  // keys past the end
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const int live = left - r * kWarps * 16 - 4 * t;
              keep[r] = live >= 4 ? 0xffffffffu : live <= 0 ? 0u : 0xffffffffu >> (32 - 8 * live);
              const int key = r * kWarps * 16 + (g >> 1) * 4 + (g & 1);
              if (key >= left) y[r][0] = y[r][1] = -INFINITY;
              if (key + 2 >= left) y[r][2] = y[r][3] = -INFINITY;
            }
          }
          // exponents against the reference; it moves where one passes kMoveRef
          float e[R][4], top = -INFINITY;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            e[r][0] = fmaf(y[r][0], cs0, -m0), e[r][1] = fmaf(y[r][1], cs1, -m1);
            e[r][2] = fmaf(y[r][2], cs0, -m0), e[r][3] = fmaf(y[r][3], cs1, -m1);
            top = fmaxf(top, fmaxf(fmaxf(e[r][0], e[r][1]), fmaxf(e[r][2], e[r][3])));
          }
          if (__any_sync(0xffffffffu, top > kMoveRef)) {
            float n0 = -FLT_MAX, n1 = -FLT_MAX;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              n0 = fmaxf(n0, fmaxf(y[r][0] * cs0, y[r][2] * cs0));
              n1 = fmaxf(n1, fmaxf(y[r][1] * cs1, y[r][3] * cs1));
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
              n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
            }
            n0 = fmaxf(m0, n0 - kPScale), n1 = fmaxf(m1, n1 - kPScale);
            const float f0 = ex2_approx(m0 - n0), f1 = ex2_approx(m1 - n1);
            m0 = n0, m1 = n1;
            l0 *= f0, l1 *= f1;
#pragma unroll
            for (int j = 0; j < KP * 8; ++j) o[j][0] *= f0, o[j][1] *= f1, o[j][2] *= f0, o[j][3] *= f1;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              e[r][0] = fmaf(y[r][0], cs0, -m0), e[r][1] = fmaf(y[r][1], cs1, -m1);
              e[r][2] = fmaf(y[r][2], cs0, -m0), e[r][3] = fmaf(y[r][3], cs1, -m1);
            }
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float p00 = ex2_approx(e[r][0]), p01 = ex2_approx(e[r][1]);
            const float p10 = ex2_approx(e[r][2]), p11 = ex2_approx(e[r][3]);
            l0 += p00 + p10;
            l1 += p01 + p11;
            // lane (g, t) now wants column g at keys 4t .. 4t + 3
            const uint32_t b0 = transpose8x8(pack_half2(p00, p01)), b1 = transpose8x8(pack_half2(p10, p11));
#pragma unroll
            for (int pl = 0; pl < KP; ++pl)
              outputs(o + pl * 8, rec + r * kWarps * C::kRecord + (KP + pl) * kKv4Plane, lane, keep[r], b0, b1);
          }
        }
        __syncwarp();
        if (alive && lane == 0) mbar_arrive(empty(stage));
        if (++stage == C::kStages) stage = 0, phase ^= 1;
      };
      if constexpr (KP == 1) {
        // V2: whole tiles without the tests (367 -> 361 us for 64 x 32768 keys). V1's code is twice as long,
        // and a second copy of it costs more than the tests do (24 x 32768 x 12: 401 and 403 us).
        const int whole_tiles = min(seg, w.len / C::kTileKeys - w.tile);
        for (int i = 0; i < whole_tiles; ++i) {
          if (i > 0) wait();
          take(i, std::false_type{});
        }
        if (whole_tiles < seg) {
          if (seg > 1) wait();
          take(seg - 1, std::true_type{});
        }
      } else {
        for (int i = 0; i < seg; ++i) {
          if (i > 0) wait();
          take(i, std::true_type{});
        }
      }

      // Join the warps' pieces. (What the row's end needs of global memory is loaded first.)
      const size_t row = static_cast<size_t>(w.b) * a.H + w.h;
      const bool out_thread = tid < 128;
      float lam[C::kMaxCols / 2], wgt[KP];
#pragma unroll
      for (int c = 0; c < C::kMaxCols / 2; ++c)
        lam[c] = !whole || 2 * c >= cols ? 0.f : KP == 2 ? *(a.lambda + w.h) : *(a.lam_logit + row * (cols / 2) + c);
#pragma unroll
      for (int k = 0; k < KP; ++k)
        wgt[k] = KP == 2 && whole && out_thread && (a.flags & 2) && a.norm_w ? *(a.norm_w + k * 128 + tid) : 1.f;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      if (g == 0) {
        s_m[warp][2 * t] = m0, s_m[warp][2 * t + 1] = m1;
        s_l[warp][2 * t] = l0, s_l[warp][2 * t + 1] = l1;
      }
      named_barrier_sync(1, kWarps * 32);
      float top0 = m0, top1 = m1;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        top0 = fmaxf(top0, s_m[i][2 * t]);
        top1 = fmaxf(top1, s_m[i][2 * t + 1]);
      }
      l0 = l1 = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        l0 = fmaf(s_l[i][2 * t], ex2_approx(s_m[i][2 * t] - top0), l0);
        l1 = fmaf(s_l[i][2 * t + 1], ex2_approx(s_m[i][2 * t + 1] - top1), l1);
      }
      float* rec = kByRow ? s_x : p.rec + static_cast<size_t>(2 * range + (starts ? 1 : 0)) * (2 * cols + cols * C::kWidth);
      const int rec_cols = kByRow ? C::kMaxCols : cols;
      float f0 = ex2_approx(m0 - top0), f1 = ex2_approx(m1 - top1);
      if (whole) {
        f0 *= 1.f / l0, f1 *= 1.f / l1;
      } else if (warp == 0 && g == 0 && 2 * t < rec_cols) {  // a piece: m, l of each column, and o below
        rec[2 * t] = top0, rec[2 * t + 1] = top1;
        rec[rec_cols + 2 * t] = l0, rec[rec_cols + 2 * t + 1] = l1;
      }
      // the upper half of the warps hand their sums to the lower half
      auto exchange = [&](auto&& step) {
        if (2 * t < C::kMaxCols) {
          float* at = s_o + (warp % (kWarps / 2) * C::kMaxCols + 2 * t) * C::kPitch;
#pragma unroll
          for (int j = 0; j < KP * 8; ++j) {
            const int ch = (j >> 3) * 128 + 16 * g + 2 * (j & 7);
            step(reinterpret_cast<float2*>(at + ch), o[j][0] * f0, o[j][2] * f0);
            step(reinterpret_cast<float2*>(at + C::kPitch + ch), o[j][1] * f1, o[j][3] * f1);
          }
        }
      };
      if (warp >= kWarps / 2) exchange([](float2* at, float x, float y) { *at = make_float2(x, y); });
      named_barrier_sync(1, kWarps * 32);
      if (warp < kWarps / 2)
        exchange([](float2* at, float x, float y) {
          const float2 v = *at;
          *at = make_float2(v.x + x, v.y + y);
        });
      named_barrier_sync(1, kWarps * 32);
      // thread `tid` < 128 takes channel tid (V1: and tid + 128) of every column
      if (out_thread) {
        float sum[C::kMaxCols][KP];
#pragma unroll
        for (int c = 0; c < C::kMaxCols; ++c)
#pragma unroll
          for (int k = 0; k < KP; ++k) {
            sum[c][k] = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps / 2; ++i) sum[c][k] += s_o[(i * C::kMaxCols + c) * C::kPitch + k * 128 + tid];
          }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < C::kMaxCols; ++c) {
            if (c >= rec_cols) break;
#pragma unroll
            for (int k = 0; k < KP; ++k) rec[2 * rec_cols + c * C::kWidth + k * 128 + tid] = sum[c][k];
          }
        } else if constexpr (KP == 1) {
#pragma unroll
          for (int c = 0; c < C::kMaxCols; c += 2) {
            if (c >= cols) break;
            const float sig = 1.f / (1.f + __expf(-lam[c / 2]));
            const float y = (sum[c][0] - sig * sum[c + 1][0]) * a.v_mul;
            static_cast<__nv_bfloat16*>(a.out)[(row * (cols / 2) + c / 2) * 128 + tid] = __float2bfloat16_rn(y);
          }
        } else {
          float y[KP], ss = 0.f;
#pragma unroll
          for (int k = 0; k < KP; ++k) {
            y[k] = (sum[0][k] - lam[0] * sum[1][k]) * a.v_mul;
            ss = fmaf(y[k], y[k], ss);
          }
          const float f = norm_scale(a, ss, s_red);
#pragma unroll
          for (int k = 0; k < KP; ++k)
            static_cast<__nv_bfloat16*>(a.out)[row * C::kWidth + k * 128 + tid] = __float2bfloat16_rn(y[k] * f * wgt[k]);
        }
      }
      w.todo -= seg;
      w.tile += seg;
      if (!kByRow && w.tile == w.tiles) next_row<KP>(a, w);
    }
  }

  if constexpr (kByRow) {
    // Every block's piece lies in its ring, which nothing uses any more. The columns' pairs are dealt out
    // over the blocks; thread `tid` takes channel tid (V1: and tid + 128).
    const int parts = p.grid, rank = blockIdx.x % parts;
    const size_t row = static_cast<size_t>(w.b) * a.H + w.h;
    auto lambda_of = [&](int pair) { return KP == 2 ? *(a.lambda + w.h) : *(a.lam_logit + row * (p.cols / 2) + pair); };
    float raw = KP == 1 && rank < p.cols / 2 ? lambda_of(rank) : 0.f;  // (V2: on its way over the barrier)
    cluster_sync_all();
    for (int pair = rank; pair < p.cols / 2 && tid < 128; pair += parts) {
      float top[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f}, sum[2][KP] = {};
      const uint32_t x = smem_u32(s_x);
      for (int i = 0; i < parts; ++i) {
        const uint32_t from = mapa_shared(x, i);
#pragma unroll
        for (int e = 0; e < 2; ++e) top[e] = fmaxf(top[e], ld_cluster_f32(from + 4 * (2 * pair + e)));
      }
      for (int i = 0; i < parts; ++i) {
        const uint32_t from = mapa_shared(x, i);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * pair + e;
          const float f = ex2_approx(ld_cluster_f32(from + 4 * c) - top[e]);
          l[e] = fmaf(ld_cluster_f32(from + 4 * (C::kMaxCols + c)), f, l[e]);
#pragma unroll
          for (int k = 0; k < KP; ++k)
            sum[e][k] = fmaf(ld_cluster_f32(from + 4 * (2 * C::kMaxCols + c * C::kWidth + k * 128 + tid)), f, sum[e][k]);
        }
      }
      if (KP == 2 || pair != rank) raw = lambda_of(pair);
      const float lam = KP == 2 ? raw : 1.f / (1.f + __expf(-raw));
      float y[KP], ss = 0.f, f = 1.f;
#pragma unroll
      for (int k = 0; k < KP; ++k) {
        y[k] = (sum[0][k] / l[0] - lam * (sum[1][k] / l[1])) * a.v_mul;
        ss = fmaf(y[k], y[k], ss);
      }
      if constexpr (KP == 2) f = norm_scale(a, ss, s_red);
#pragma unroll
      for (int k = 0; k < KP; ++k) {
        const float wgt = KP == 2 && (a.flags & 2) && a.norm_w ? *(a.norm_w + k * 128 + tid) : 1.f;
        const float o = w.len == 0 ? 0.f : y[k] * f * wgt;  // (zeros, whatever the weight and the scale hold)
        static_cast<__nv_bfloat16*>(a.out)[(row * (p.cols / 2) + pair) * C::kWidth + k * 128 + tid] = __float2bfloat16_rn(o);
      }
    }
    cluster_sync_all();  // no block leaves while another reads its piece
  }
}

// Merge, of each row whose tiles lie in more than one range: its pieces are that of the range that begins it
// and of the ranges that begin inside it, always in this order; groups of threads take every n-th piece,
// and join. Few rows: a block for each pair of columns of each row. Else: block i for the row that range
// i + 1 begins inside, if no earlier range does, with all its columns.
template <int KP, bool kFewRows>
__global__ void __launch_bounds__(kFewRows ? Cfg<KP>::kMergeFew : Cfg<KP>::kMerge) kv4_merge_kernel(const Params p) {
  constexpr int W = KP * 128, NT = kFewRows ? Cfg<KP>::kMergeFew : Cfg<KP>::kMerge;
  __shared__ float s_m[NT / (W / 4)], s_l[NT / (W / 4)];  // a column of a group each
  __shared__ float4 s_o[NT];
  __shared__ float s_red[W / 32];
  const Kv4DecodeArgs& a = p.a;
  const int tid = threadIdx.x, cols = p.cols;
  // All but the pieces is known before the first kernel ends: it released this one after its own wait, so
  // the lengths, the lambdas and the weights are there.
  __shared__ Ranges<KP, NT, true> s_ranges;
  __shared__ Walk s_walk;
  s_ranges.fill(a);
  const long long total = s_ranges.total(a);
  const int n = s_ranges.count(total, p.grid);
  const Cut cut(total, n);
  const int c0 = kFewRows ? 2 * static_cast<int>(blockIdx.x % (cols / 2)) : 0, nc = kFewRows ? 2 : cols;  // the columns
  if (tid < 32) {
    Walk w{};
    if constexpr (kFewRows) {  // B <= NT: a share of one sequence a thread
      const int row = blockIdx.x / (cols / 2);
      w.b = row / a.H;
      w.h = row - w.b * a.H;
      w.len = clamp_len<true>(a, w.b);
      w.tiles = tiles_of<KP>(w.len);
      w.first = s_ranges.pre[w.b] * a.H + static_cast<long long>(w.h) * cost_of<KP>(w.len) + Cfg<KP>::kRowCost;
    } else if (static_cast<int>(blockIdx.x) + 1 < n) {
      s_ranges.locate(a, cut, blockIdx.x + 1, w);
      // no row is this block's: range i + 1 begins with one, or is not the first to begin inside its row
      if (w.tile == 0 || cut.start(blockIdx.x) > w.first) w.tiles = 0;
    }
    if (tid == 0) s_walk = w;
  }
  __syncthreads();
  const Walk d = s_walk;
  const int i0 = d.tiles > 0 ? cut.owner(d.first) : 0;
  const int pieces = d.tiles > 0 ? cut.owner(d.first + d.tiles - 1) - i0 + 1 : 0;
  if (pieces < 2) {
    grid_wait();
    grid_release();
    return;
  }
  const int lanes = nc * (W / 4), groups = NT / lanes;  // a float4 of all its columns' outputs each
  const size_t rec = 2 * cols + cols * W;
  const int grp = tid / lanes, ln = tid % lanes, c = ln / (W / 4);
  const size_t row = static_cast<size_t>(d.b) * a.H + d.h;
  // the output channels of the end: `tid` and every NT-th on (V1: the row's 256)
  constexpr int kOuts = KP == 2 || kFewRows ? 1 : 512 / NT;
  float lam[kOuts];
#pragma unroll
  for (int i = 0; i < kOuts; ++i) {
    const int pair = (tid + i * NT) / W;
    lam[i] = 2 * pair >= nc ? 0.f
             : KP == 2      ? __ldcg(a.lambda + d.h)
                            : 1.f / (1.f + __expf(-__ldcg(a.lam_logit + row * (cols / 2) + c0 / 2 + pair)));
  }
  const float wgt = KP == 2 && tid < W && (a.flags & 2) && a.norm_w ? __ldcg(a.norm_w + tid) : 1.f;
  grid_wait();
  grid_release();
  float m = -FLT_MAX, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = grp; k < pieces; k += groups) {
    const float* r = p.rec + static_cast<size_t>(2 * (i0 + k) + (k == 0 ? 1 : 0)) * rec;
    const float mk = r[c0 + c], lk = r[cols + c0 + c];
    const float4 ok = *reinterpret_cast<const float4*>(r + 2 * cols + c0 * W + ln * 4);
    const float top = fmaxf(m, mk), f = ex2_approx(m - top), fk = ex2_approx(mk - top);
    m = top;
    l = l * f + lk * fk;
    o.x = o.x * f + ok.x * fk;
    o.y = o.y * f + ok.y * fk;
    o.z = o.z * f + ok.z * fk;
    o.w = o.w * f + ok.w * fk;
  }
  s_o[tid] = o;
  if (ln % (W / 4) == 0) s_m[grp * nc + c] = m, s_l[grp * nc + c] = l;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOuts; ++i) {
    const int pair = (tid + i * NT) / W, ch = (tid + i * NT) % W;
    if (2 * pair >= nc) return;
    float q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 2 * pair + e;
      float top = s_m[col];
      for (int k = 1; k < groups; ++k) top = fmaxf(top, s_m[k * nc + col]);
      float sum = 0.f, ls = 0.f;
      for (int k = 0; k < groups; ++k) {
        const float f = ex2_approx(s_m[k * nc + col] - top);
        ls = fmaf(s_l[k * nc + col], f, ls);
        sum = fmaf(reinterpret_cast<const float*>(s_o + k * lanes)[col * W + ch], f, sum);
      }
      q[e] = sum / ls;
    }
    float y = (q[0] - lam[i] * q[1]) * a.v_mul;
    if constexpr (KP == 2) {
      if (a.flags & 2) {
        float ss = y * y;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
        if ((tid & 31) == 0) s_red[tid >> 5] = ss;
        named_barrier_sync(1, W);
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < W / 32; ++k) ss += s_red[k];
        y *= 1.f / sqrtf(ss / static_cast<float>(W) + a.eps) * wgt;
      }
      if (a.flags & 4) y *= 1.f - a.lambda_init;
    }
    static_cast<__nv_bfloat16*>(a.out)[(row * (cols / 2) + c0 / 2 + pair) * W + ch] = __float2bfloat16_rn(y);
  }
}

template <int KP>
cudaError_t launch(const Kv4DecodeArgs& a, cudaStream_t st) {
  using C = Cfg<KP>;
  Params p{};
  p.a = a;
  p.cols = KP == 2 ? 2 : a.group;
  p.rec = static_cast<float*>(a.ws);
  static std::atomic<uint64_t> raised[2] = {};
  const long long tiles = (static_cast<long long>(a.max_pages) * a.page_size + C::kTileKeys - 1) / C::kTileKeys;
  const long long rows = static_cast<long long>(a.B) * a.H;
  // Few keys: a row over a cluster, of as many blocks as leave it two tiles each and are resident at once;
  // where the rows' blocks then have at most kFewTiles more tiles than an equal share: the second kernel
  // and the ranges cost about that. (GPU time of a call so and by ranges: 8 rows of 777 keys, V2, 5.6 and
  // 8.7 us; 400 rows of 1000, 15.6 and 19.2; 48 rows of 1500, V1, 10.1 and 12.9; 240 of 800, 15.3 and 18.7;
  // 96 of 3000, V1, where clusters of two would leave a third of the machine idle, 23.6 and 21.2. The host
  // has one launch less as well. Only up to 8 tiles a block: the tables' capacity, which is all the host
  // knows, is not the sequences' length.)
  int parts = 1;
  while (parts < 8 && parts * 2 < tiles && rows * parts * 2 <= C::kGrid) parts *= 2;
  if (rows <= C::kGrid && rows * tiles <= 8LL * C::kGrid &&
      (tiles + parts - 1) / parts <= rows * tiles / C::kGrid + kFewTiles) {
    p.grid = parts;
    return launch_early_large(kv4_decode_kernel<KP, true>, static_cast<unsigned>(rows * p.grid), C::kThreads, C::kSmem,
                              C::kSmem, st, p.grid, p, raised[1]);
  }
  // no more blocks than the tables' capacity can give ranges
  const long long most = (tiles + C::kRowCost) * rows / C::kMinCost;
  p.grid = static_cast<int>(most < 1 ? 1 : most > C::kGrid ? C::kGrid : most);
  cudaError_t e = launch_early_large(kv4_decode_kernel<KP, false>, p.grid, C::kThreads, C::kSmem, C::kSmem, st, 1, p, raised[0]);
  if (e != cudaSuccess || p.grid == 1) return e;
  // A block for each pair of columns of each row, where those are fewer: the rows are long then, and their
  // many pieces are read by more threads (8 rows of 16K keys, V2: 12.9 us the whole call, 18.4 the other way).
  if (rows * (p.cols / 2) < p.grid && a.B <= C::kMergeFew)
    return launch_early(kv4_merge_kernel<KP, true>, static_cast<unsigned>(rows * (p.cols / 2)), C::kMergeFew, 0, st, 1, p);
  return launch_early(kv4_merge_kernel<KP, false>, p.grid - 1, C::kMerge, 0, st, 1, p);
}

}  // namespace

size_t kv4_decode_workspace_bytes(int cols, int width) {
  const size_t grid = width == 128 ? Cfg<1>::kGrid : Cfg<2>::kGrid;
  return 2 * grid * (2 * cols + static_cast<size_t>(cols) * width) * sizeof(float);
}

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t st) {
  return a.group == 0 ? launch<2>(a, st) : launch<1>(a, st);
}

cudaError_t status_decode_kv4(int* v) { return launched_status(v); }

}  // namespace da
