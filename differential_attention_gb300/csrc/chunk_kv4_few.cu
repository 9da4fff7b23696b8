// chunk_kv4_few.cu -- V1 attention of short chunks over the 4-bit cache: a few new tokens of each sequence, as a
// server checks drafted ones, over all its cached keys.
//
// The mathematics and the units are chunk_kv4.cu's; a unit here is both maps of up to 8 tokens. So few rows would
// leave most of a 128-row product in tensor memory empty, and its operands would still have to be unpacked to shared
// memory, 1024 bytes a key. Here they go from the records to m16n8k16 in registers, as in decode_kv4.cu: keys, or
// V's channels, are the 16 rows of a product, 8 tokens its columns. K's planes meet a column tile each (map m's
// queries), V's planes both.
//
// Warps. One copies records into a ring of tiles, two prepare the queries of the next unit; two sets of four attend,
// a tile of 128 keys in turn, two records of 16 keys a warp at a time, so that there are independent instructions to
// issue. Each warp has a running maximum, sum and O of its own, joined through shared memory at the unit's end.
//
// Numerics as in decode_kv4.cu: the query as fp16 after a power of two of its own for each row, P rounded to fp16
// at 2^10 times its value against a reference that moves where a score passes it by 2^4, sums and statistics in fp32.
// Keys that a row may not see have P = 0; a NaN block of V is held as zeros, its first key noted, and the rows that
// see that key get NaN at the end.
//
// What bounds it: issue. A record takes some 590 instructions, 147 cycles of the SM's four schedulers where its bytes
// take 196 at the memory's rate, but the accumulators (16 x 256 floats a warp) leave room for only two warps a
// scheduler, and those issue in about half of the cycles. 16 sequences of 16384 keys, 6 new tokens, 12 heads (907 MB):
// 184 us, 4.9 TB/s (calls one by one, each after a write of 256 MB; in a row 173, 5.2); the kernel for 128 rows takes
// 307. Measured on the way, same case: a record at a time 206, two records and tiles of 256 keys 191 (whose two stages
// are both in use while no copy runs), a record at a time with the next tile's scores among this one's outputs 204. The
// same with V2 (four column tiles a warp, 32 rows) took 335 us
// for 24 x 32768 keys, where 128 rows take 386, and more than those with mixed lengths (104 and 87 us) or 64 rows
// (645); so V2 has no such kernel.
#include <cfloat>
#include <cmath>

#include "early.cuh"
#include "kv4_chunk.cuh"
#include "kv4_mma.cuh"

namespace da {
namespace {

constexpr float kPScale = 10.f;   // log2 of P's scale
constexpr float kMoveRef = 14.f;  // log2 P at which the reference moves
// What a unit costs besides its tiles, in tiles: the join of the warps, and its first and last tile, which one set of
// warps takes while the other has none. (48 sequences of 1 to 16384 keys, 6 new tokens, 12 heads: 128 us with 2, 99
// with 4, 91 with 5, 93 with 6, 104 with 10.)
constexpr int kUnitCost = 5;
constexpr int kWarps = 8;         // consumers
constexpr int kThreads = (kWarps + 4) * 32;  // and the producer's warpgroup
// Registers a thread: the launch's dealt out anew to the warpgroups
constexpr int kLaunchRegs = 168, kConsumerRegs = 224, kProducerRegs = 56;
static_assert(2 * kConsumerRegs + kProducerRegs <= 3 * kLaunchRegs, "more registers than the launch has");

constexpr int kTileRecs = 8, kTileLog2 = 7;       // a tile's records
constexpr int kSet = kWarps / 2;                  // warps that share a tile, each its records `warp` and `warp` + 4
constexpr int kTokens = 8, kRows = 2 * kTokens;   // of a unit: column tile m holds map m of its tokens
// The exchange, floats: 32 channels of a column take 36, so that the 16-byte accesses of a quarter of a warp (two of
// g, four of t) meet all banks once
constexpr int kPitch = 8 * 36 + 4;
__device__ __forceinline__ int place_of(int ch) { return (ch >> 5) * 36 + (ch & 31) + (ch >> 4 & 1) * 4; }
constexpr int kRecord = 4 * kKv4Plane, kStage = kTileRecs * kRecord, kStages = 4;
constexpr int kBufs = kWarps / 2;                 // exchange buffers
constexpr int kO = kStages * kStage;
constexpr int kFrag = kO + kBufs * kRows * kPitch * 4, kFragBytes = 2 * 4 * 512;  // Q's fragments, of two units
constexpr int kSmall = kFrag + 2 * kFragBytes;
struct Small {
  uint64_t full[kStages], empty[kStages], q_full[2], q_free[2];
  float m[kWarps][kRows], l[kWarps][kRows], scale[2][kRows];
  int nan_key[2][16];  // by the unit's parity: the first key with a NaN block in 16 of V's channels
  int abort;
};
constexpr int kSmem = kSmall + static_cast<int>(sizeof(Small));
static_assert(kSmem <= 232448, "shared memory");
struct Scan {  // at startup, in the exchange's place
  long long pre[kThreads + 1], sum[kThreads / 32];
  Walk walk;
};
static_assert(sizeof(Scan) <= kFrag - kO, "the exchange's place");

// One column's query, its channels 32t .. 32t + 31 in `raw` of the four lanes t: as fp16 fragments, and what its
// sums are to be multiplied with (never 0 or Inf, which a masked score's Inf or a score of 0 would turn into NaN).
__device__ __forceinline__ float query(const Kv4ChunkArgs& a, const uint32_t (&raw)[16], uint4 (&qf)[4]) {
  uint32_t top = 0;  // the largest magnitude's bits (ordered as the values are)
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, max(raw[i] & 0x7fffu, (raw[i] >> 16) & 0x7fffu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int e = max(static_cast<int>(top >> 7) - 127, -100);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);  // 2^(14 - e)
  auto two = [&](uint32_t x) { return pack_half2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up); };
#pragma unroll
  for (int k = 0; k < 4; ++k) qf[k] = make_uint4(two(raw[4 * k]), two(raw[4 * k + 1]), two(raw[4 * k + 2]), two(raw[4 * k + 3]));
  return fminf(fmaxf(ldexpf(a.qk_scale, e - 14), FLT_MIN), FLT_MAX);
}
__device__ __forceinline__ void load_row(const Kv4ChunkArgs& a, size_t from, int t, bool used, uint32_t (&raw)[16]) {
  const uint4* at = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + from * 128 + t * 32);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = used ? at[i] : make_uint4(0, 0, 0, 0);
    raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
  }
}

// S^T of two records, `apart` bytes from one to the next: column tile p against K's plane p, whose fragments lie at
// `frag`; as scores().
__device__ __forceinline__ void scores_maps(float (&y)[2][2][4], uint32_t at, int apart, int lane, uint32_t frag) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint4 lo[2], hi[2];
    uint32_t slo[2], shi[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t from = at + r * apart + p * kKv4Plane;
      lo[r] = lds128(from), hi[r] = lds128(from + 512);
      e4m3x4_to_half2(lds32(from - lane * 12 + kKv4PlaneCodes), slo[r], shi[r]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 q = lds128(frag + (p * 4 + k) * 512);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t sl = __byte_perm(slo[r], 0, k < 2 ? 0x1010 : 0x3232), sh = __byte_perm(shi[r], 0, k < 2 ? 0x1010 : 0x3232);
        uint32_t x[4], z[4];
        e2m1x8_to_half2(k == 0 ? lo[r].x : k == 1 ? lo[r].y : k == 2 ? lo[r].z : lo[r].w, x);
        e2m1x8_to_half2(k == 0 ? hi[r].x : k == 1 ? hi[r].y : k == 2 ? hi[r].z : hi[r].w, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = half2_mul(x[i], sl), z[i] = half2_mul(z[i], sh);
        if (k == 0) mma_first(y[r][p], x[0], z[0], x[1], z[1], q.x, q.y);
        else mma(y[r][p], x[0], z[0], x[1], z[1], q.x, q.y);
        mma(y[r][p], x[2], z[2], x[3], z[3], q.z, q.w);
      }
    }
  }
}

// O^T += V^T P^T of one record and plane: rows g and g + 8 of product j are channels 16g + 2j and + 1. sc: the scales
// of this lane's tokens 4t .. 4t + 3, 0 where one is not to count.
__device__ __forceinline__ void outputs(float (&o)[2][16][4], int j0, uint32_t at, uint32_t sc, const uint32_t (&b)[2][2]) {
  const uint4 va = lds128(at), vb = lds128(at + 512);
  uint32_t s01, s23;
  e4m3x4_to_half2(sc, s01, s23);
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
    for (int i = 0; i < 4; ++i) {
      const uint32_t x0 = half2_mul(e01[i], s01), x1 = half2_mul(d01[i], s01), x2 = half2_mul(e23[i], s23), x3 = half2_mul(d23[i], s23);
#pragma unroll
      for (int n = 0; n < 2; ++n) mma(o[n][j0 + 4 * k + i], x0, x1, x2, x3, b[n][0], b[n][1]);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) kv4_chunk_few_kernel(const Kv4ChunkArgs a) {
  constexpr int kAll = kWarps * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  Small& sm = *reinterpret_cast<Small*>(smem + kSmall);
  float* const s_o = reinterpret_cast<float*>(smem + kO);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t ring = smem_u32(smem);
  auto full = [&](int s) { return smem_u32(&sm.full[s]); };
  auto empty = [&](int s) { return smem_u32(&sm.empty[s]); };

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kSet);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), 2);
      mbar_init(smem_u32(&sm.q_free[i]), kWarps);
    }
    fence_barrier_init();
    sm.abort = 0;
  }
  if (tid < 32) sm.nan_key[tid >> 4][tid & 15] = INT_MAX;
  grid_wait();
  grid_release();
  Walk w{};
  {
    Scan& scan = *reinterpret_cast<Scan*>(s_o);
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
    __syncthreads();
    w = scan.walk;
    __syncthreads();  // the exchange's place is free
  }

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp == kWarps + 3) return;
    if (warp > kWarps) {
      // Queries: map `warp - kWarps - 1` of the units' tokens, a unit ahead
      const int map = warp - kWarps - 1, g = lane >> 2, t = lane & 3;
      for (int unit = 0; w.todo > 0; ++unit) {
        const int seg = static_cast<int>(min(static_cast<long long>(w.tiles - w.tile), w.todo));
        const int tok0 = w.rt * a.tokens, toks = min(a.tokens, w.Lq - tok0), b = unit & 1;
        uint32_t raw[16];
        uint4 qf[4];
        load_row(a, ((static_cast<size_t>(w.q0) + tok0 + g) * a.H + w.h) * 2 + map, t, g < toks, raw);
        const float s = query(a, raw, qf);
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.q_free[b]), (unit >> 1 & 1) ^ 1, &sm.abort))) return;
        if (t == 0) sm.scale[b][8 * map + g] = s;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          st_shared_v4(ring + kFrag + b * kFragBytes + (map * 4 + k) * 512 + lane * 16, qf[k].x, qf[k].y, qf[k].z, qf[k].w);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[b]));
        advance(a, w, seg);
      }
      return;
    }
    // Producer. Lane i looks up the page of record i of the next tiles of the unit (32 records at most); the lanes
    // of a tile's records then copy one each. The next batch's pages are looked up before the copies of this one.
    constexpr int kBatch = 32 / kTileRecs;
    const int recs = a.page_size >> 4;
    struct Batch {
      int n, h, page, off, records;  // tiles; this lane's page and record of it; the unit's records from the first tile on
      bool used;
    };
    auto look_up = [&]() {
      Batch x;
      x.n = static_cast<int>(min(min(static_cast<long long>(kBatch), static_cast<long long>(w.tiles - w.tile)), max(w.todo, 0LL)));
      const int all = (w.Lk + 15) >> 4, rec = min(w.tile * kTileRecs + lane, max(0, all - 1));
      const int pi = (__umulhi(rec, a.rec_magic) + rec) >> a.rec_shift;
      x.records = all - w.tile * kTileRecs;
      x.used = lane < x.n * kTileRecs && lane < x.records && dbg_index_ok(pi, a.max_pages);
      x.page = x.used ? *(a.block_table + static_cast<size_t>(w.b) * a.max_pages + pi) : 0;
      x.off = rec - pi * recs;
      x.h = w.h;
      return x;
    };
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool alive = true;
    Batch next = look_up();
    while (alive && next.n > 0) {
      Batch x = next;
      advance(a, w, x.n);
      next = look_up();
      if (x.used && (x.page < 0 || x.page >= a.num_pages)) {
        flag_device_error(DEV_BAD_INDEX);
        x.page = 0;
      }
      const uint8_t* src = a.pool + ((static_cast<size_t>(x.page) * a.H + x.h) * recs + x.off) * kRecord;
      for (int i = 0; i < x.n; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty(stage), phase ^ 1, &sm.abort))) {
          alive = false;
          break;
        }
        // (a debug build leaves out a copy from outside the table, and its bytes)
        const unsigned copies = __ballot_sync(0xffffffffu, x.used && lane / kTileRecs == i);
        if (lane == 0) mbar_arrive_expect_tx(full(stage), __popc(copies) * kRecord);
        __syncwarp();
        if (copies >> lane & 1)
          bulk_load(ring + stage * kStage + lane % kTileRecs * kRecord, src, kRecord, full(stage));
        ++issued;
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
    if (!alive) {
      // a wait ran out: the copies in flight still land in this block's memory
      for (int back = 0; back < min(issued, kStages); ++back) {
        if (--stage < 0) stage = kStages - 1, phase ^= 1;
        mbar_wait_limit(full(stage), phase, nullptr, kWaitLimitNs);
      }
    }
    return;
  }

  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  // Consumers. Lane (g, t) has S^T's rows g and g + 8 (keys 4 (g / 2) + g % 2 and that + 2 of a record) and columns
  // 2t and 2t + 1 (tokens) of both maps' tiles.
  const int g = lane >> 2, t = lane & 3;
  bool alive = true;
  int stage = 0, unit = 0, j = 0;
  uint32_t phase = 0;
  auto wait = [&](int s, uint32_t ph) {
    if (__all_sync(0xffffffffu, mbar_try_wait(full(s), ph))) return;
    alive = __all_sync(0xffffffffu, alive && mbar_wait(full(s), ph, &sm.abort));
  };
  // tokens that see no key get zeros
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const Seq s = sequence<false>(a, b);
    const int z = hidden(a, s);
    const size_t width = static_cast<size_t>(a.H) * 256;
    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + s.q0 * width);
    for (size_t i = tid; i < z * width / 8; i += kAll) out[i] = make_uint4(0, 0, 0, 0);
  }
  while (w.todo > 0) {
    const int seg = static_cast<int>(min(static_cast<long long>(w.tiles - w.tile), w.todo));
    const bool starts = w.tile == 0, whole = starts && seg == w.tiles;
    const int tok0 = w.rt * a.tokens, toks = min(a.tokens, w.Lq - tok0);  // tokens of the unit
    const size_t first = static_cast<size_t>(w.q0) + tok0;
    float cs[2][2], m[2][2], l[2][2], o[2][16][4];
    const int qb = unit & 1;
    alive = __all_sync(0xffffffffu, alive && mbar_wait(smem_u32(&sm.q_full[qb]), unit >> 1 & 1, &sm.abort));
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) cs[n][e] = sm.scale[qb][8 * n + 2 * t + e];
    const uint32_t frag = ring + kFrag + qb * kFragBytes + lane * 16;
    const float lam = *(a.lambda + w.h);
    // keys that a token sees: the first one's, and any
    const int edge = a.causal ? max(0, w.Lk - w.Lq + tok0 + 1) : w.Lk;
    auto limit = [&](int tok) { return tok >= toks ? 0 : a.causal ? max(0, w.Lk - w.Lq + tok0 + tok + 1) : w.Lk; };
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      m[n][0] = m[n][1] = -FLT_MAX;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
    }
#pragma unroll 1
    for (int i = 0; i < seg; ++i, ++j) {
      const int from = stage;
      const uint32_t ph = phase;
      if (++stage == kStages) stage = 0, phase ^= 1;
      if ((j & 1) != warp / kSet) continue;
      wait(from, ph);
      constexpr int kApart = kSet * kRecord;
      const int key0 = ((w.tile + i) * kTileRecs + warp % kSet) * 16;
      const uint32_t rec = ring + from * kStage + warp % kSet * kRecord + lane * 16;
      // (a record that the sequence does not have holds an earlier tile's: none of it is seen)
      float y[2][2][4];
      scores_maps(y, rec, kApart, lane, frag);
      uint32_t sc[2][2], odd = 0;  // of V, by record and plane; whether one is NaN
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int p = 0; p < 2; ++p) sc[r][p] = lds32(rec + r * kApart - lane * 12 + (2 + p) * kKv4Plane + kKv4PlaneCodes);
      if (key0 + kSet * 16 + 16 > edge) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int first_key = key0 + r * kSet * 16, live = w.Lk - first_key - 4 * t, key = first_key + (g >> 1) * 4 + (g & 1);
          const uint32_t keep = live >= 4 ? 0xffffffffu : live <= 0 ? 0u : 0xffffffffu >> (32 - 8 * live);
          sc[r][0] &= keep, sc[r][1] &= keep;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lim = limit(2 * t + e);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              if (key >= lim) y[r][n][e] = -INFINITY;
              if (key + 2 >= lim) y[r][n][2 + e] = -INFINITY;
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int p = 0; p < 2; ++p) odd |= ((sc[r][p] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
      if (odd) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            if ((odd = ((sc[r][p] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0) {
              atomicMin(&sm.nan_key[unit & 1][p * 8 + g], key0 + r * kSet * 16 + 4 * t + ((__ffs(odd) - 1) >> 3));
              sc[r][p] &= ~((odd >> 7) * 0xffu);
            }
      }
      // exponents against the reference; it moves where one passes kMoveRef
      float top = -INFINITY;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          top = fmaxf(top, fmaxf(fmaxf(fmaf(y[r][n][0], cs[n][0], -m[n][0]), fmaf(y[r][n][2], cs[n][0], -m[n][0])),
                                 fmaxf(fmaf(y[r][n][1], cs[n][1], -m[n][1]), fmaf(y[r][n][3], cs[n][1], -m[n][1]))));
      if (__any_sync(0xffffffffu, top > kMoveRef)) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float to = -FLT_MAX;
#pragma unroll
            for (int r = 0; r < 2; ++r) to = fmaxf(to, fmaxf(y[r][n][e] * cs[n][e], y[r][n][2 + e] * cs[n][e]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
            to = fmaxf(m[n][e], __fsub_ru(to, kPScale));
            const float f = ex2_approx(m[n][e] - to);
            m[n][e] = to;
            l[n][e] *= f;
#pragma unroll
            for (int c = 0; c < 16; ++c) o[n][c][e] *= f, o[n][c][2 + e] *= f;
          }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t b[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p00 = ex2_approx(fmaf(y[r][n][0], cs[n][0], -m[n][0])), p01 = ex2_approx(fmaf(y[r][n][1], cs[n][1], -m[n][1]));
          const float p10 = ex2_approx(fmaf(y[r][n][2], cs[n][0], -m[n][0])), p11 = ex2_approx(fmaf(y[r][n][3], cs[n][1], -m[n][1]));
          l[n][0] += p00 + p10;
          l[n][1] += p01 + p11;
          // lane (g, t) now wants column g at keys 4t .. 4t + 3
          b[n][0] = transpose8x8(pack_half2(p00, p01)), b[n][1] = transpose8x8(pack_half2(p10, p11));
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) outputs(o, p * 8, rec + r * kApart + (2 + p) * kKv4Plane, sc[r][p], b);
      }
      __syncwarp();
      if (alive && lane == 0) mbar_arrive(empty(from));
    }

    // ---- the unit's end ----
    if (lane == 0) mbar_arrive(smem_u32(&sm.q_free[qb]));
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
        if (g == 0) sm.m[warp][8 * n + 2 * t + e] = m[n][e], sm.l[warp][8 * n + 2 * t + e] = l[n][e];
      }
    named_barrier_sync(1, kAll);
    if (tid < 16) sm.nan_key[(unit + 1) & 1][tid] = INT_MAX;  // (every warp has left the unit before this one)
    float* piece = a.pieces + static_cast<size_t>(2 * blockIdx.x + (starts ? 1 : 0)) * (kRows * (2 + 256));
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 8 * n + 2 * t + e;
        float top = m[n][e], sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sm.m[i][c]);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum = fmaf(sm.l[i][c], ex2_approx(sm.m[i][c] - top), sum);
        float f = ex2_approx(m[n][e] - top);
        if (whole) {
          f *= 1.f / sum;
        } else if (warp == 0 && g == 0) {
          const int row = 2 * (2 * t + e) + n;
          piece[row] = top, piece[kRows + row] = sum;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) o[n][j][e] *= f, o[n][j][2 + e] *= f;
      }
    // the upper half of the warps hand their sums to the lower half: 16 channels of a column side by side
    auto exchange = [&](auto&& step) {
      float* at = s_o + warp % kBufs * (kRows * kPitch) + 2 * t * kPitch + place_of(16 * g);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int c = 0; c < 16; c += 2)
            step(reinterpret_cast<float4*>(at + (8 * n + e) * kPitch + (c >> 3) * 144 + 2 * (c & 7)),
                 make_float4(o[n][c][e], o[n][c][2 + e], o[n][c + 1][e], o[n][c + 1][2 + e]));
    };
    if (warp >= kBufs) exchange([](float4* at, float4 x) { *at = x; });
    named_barrier_sync(1, kAll);
    if (warp < kBufs)
      exchange([](float4* at, float4 x) {
        const float4 v = *at;
        *at = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
      });
    named_barrier_sync(1, kAll);
    // a token a warp, four channels of each half a lane
    const int* nan = sm.nan_key[unit & 1];
    if (warp < toks) {
      const size_t token = first + warp;
      const int lim = limit(warp);
      float z[2][2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float* at = s_o + (8 * e + warp) * kPitch + place_of(p * 128 + 4 * lane);
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kBufs; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(at + k * kRows * kPitch);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
          }
          if (nan[p * 8 + (lane >> 2)] < lim) v.x = v.y = v.z = v.w = __int_as_float(0x7fffffff);
          z[e][p][0] = v.x, z[e][p][1] = v.y, z[e][p][2] = v.z, z[e][p][3] = v.w;
          if (!whole) *reinterpret_cast<float4*>(piece + 2 * kRows + ((p * 32 + lane) * kRows + 2 * warp + e) * 4) = v;
        }
      if (whole && dbg_index_ok(static_cast<long long>(token), a.total)) {
        float ss = 0.f, f = 1.f;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            z[0][p][x] = (z[0][p][x] - lam * z[1][p][x]) * a.v_mul;
            ss = fmaf(z[0][p][x], z[0][p][x], ss);
          }
        if (a.flags & 2) {
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
          f = 1.f / sqrtf(ss / 256.f + a.eps);
        }
        if (a.flags & 4) f *= 1.f - a.lambda_init;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float4 wgt = make_float4(1.f, 1.f, 1.f, 1.f);
          if ((a.flags & 2) && a.norm_w) wgt = *reinterpret_cast<const float4*>(a.norm_w + p * 128 + 4 * lane);
          const float* x = z[0][p];
          // (zeros where no key is seen, whatever the weight and the scale hold)
          const uint32_t lo = lim > 0 ? pack_bf16x2(x[0] * f * wgt.x, x[1] * f * wgt.y) : 0u;
          const uint32_t hi = lim > 0 ? pack_bf16x2(x[2] * f * wgt.z, x[3] * f * wgt.w) : 0u;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (token * a.H + w.h) * 256 + p * 128 + 4 * lane) = make_uint2(lo, hi);
        }
      }
    }
    ++unit;
    advance(a, w, seg);
  }
}

}  // namespace

// One unit's tokens: with more, the cache is read once more for every 8 (16 x 16384 keys: 187 us for 8 tokens, twice
// that for 9 to 16; the kernel for 128 rows 317 for any up to 64).
bool kv4_chunk_few(const Kv4ChunkArgs& a) { return a.group == 0 && a.longest <= kTokens; }

cudaError_t launch_kv4_chunk_few(Kv4ChunkArgs a, cudaStream_t st) {
  static std::atomic<uint64_t> raised{};
  a.rows = kRows;
  a.tokens = kTokens;
  a.tok_log2 = 3;
  a.tile_log2 = kTileLog2;
  a.unit_cost = kUnitCost;
  page_magic(a.page_size >> 4, &a.rec_magic, &a.rec_shift);
  // no more blocks than the tables' capacity can give ranges
  const long long tiles = (static_cast<long long>(a.max_pages) * a.page_size + (1 << kTileLog2) - 1) >> kTileLog2;
  const long long units = (static_cast<long long>(a.total) / a.tokens + a.B) * a.H;
  const long long most = units >= kChunkSms ? kChunkSms : (tiles + kUnitCost) * units / kMinCost;
  a.grid = static_cast<int>(most < 1 ? 1 : most > kChunkSms ? kChunkSms : most);
  cudaError_t e = launch_early_large(kv4_chunk_few_kernel, a.grid, kThreads, kSmem, kSmem, st, 1, a, raised);
  if (e != cudaSuccess || a.grid == 1) return e;
  return launch_kv4_chunk_join(a, st);
}

cudaError_t status_chunk_kv4_few(int* v) { return launched_status(v); }

}  // namespace da
