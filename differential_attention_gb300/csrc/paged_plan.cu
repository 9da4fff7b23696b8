// paged_plan.cu -- a step's page plan: block tables, slot maps, positions and offsets from the
// lengths of its requests.
//
// Every output follows from four prefix sums over the requests (new tokens, keys of the requests
// that have new tokens, pages they grow into, pages of ended requests): token i of the step belongs
// to the request whose range of the first sum holds i, and the a-th page taken from the ring to the
// request whose range of the third holds a. The sums sit in shared memory and each token and page
// finds its request by a binary search there, so that one long prompt costs no more than many
// short ones.
//
// What bounds it is latency: a step moves a few hundred kilobytes at most. So it is one launch of one
// cluster of up to 8 blocks. Every block forms all the sums (for 1024 requests one pass of its
// threads), then the cluster meets once, and each block writes its share. The one meeting is what
// lets the lengths and the ring's state be updated in place: all blocks have read them by then. 256
// requests of one new token take 5.1 us, 48 with 33K new tokens 8.5 (GPU time of a call).
#include "early.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int DEV_NO_FIT = 8;  // beside ptx.cuh's codes: a step that does not fit
constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;

struct PlanParams {
  const int* seqlens;
  const int* new_tokens;
  int* seqlens_out;
  int* block_table;
  int* ring;
  const int* state;
  int* state_out;
  int* cu_q;
  int* cu_k;
  int* slots;
  int* positions;
  int B, max_pages, num_pages, page_size, total_max;
};

struct Four {
  long long q, k, take, back;
};
__device__ __forceinline__ Four operator+(const Four& a, const Four& b) {
  return {a.q + b.q, a.k + b.k, a.take + b.take, a.back + b.back};
}
__device__ __forceinline__ Four shfl_up(const Four& a, int d) {
  return {__shfl_up_sync(0xffffffffu, a.q, d), __shfl_up_sync(0xffffffffu, a.k, d),
          __shfl_up_sync(0xffffffffu, a.take, d), __shfl_up_sync(0xffffffffu, a.back, d)};
}

// the largest i in [0, n) with first[i] <= x (first ascending, first[0] <= x)
__device__ __forceinline__ int owner(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p) {
  extern __shared__ int sm[];
  int* s_len = sm;                     // [B] cached tokens
  int* s_q = s_len + p.B;              // [B + 1] new tokens before each request
  int* s_take = s_q + p.B + 1;         // [B + 1] pages taken before it
  int* s_back = s_take + p.B + 1;      // [B + 1] pages returned before it
  __shared__ Four warp_sum[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int all = static_cast<int>(gridDim.x) * kPlanThreads, gid = static_cast<int>(blockIdx.x) * kPlanThreads + tid;
  const bool lead = blockIdx.x == 0;
  const int ps = p.page_size;
  const long long cap = static_cast<long long>(p.max_pages) * ps;
  grid_wait();
  grid_release();
  const int head = p.state[0], count = p.state[1];
  bool bad = head < 0 || head >= p.num_pages || count < 0 || count > p.num_pages;

  Four carry = {0, 0, 0, 0};
  for (int i0 = 0; i0 < p.B; i0 += kPlanThreads) {
    const int i = i0 + tid;
    Four v = {0, 0, 0, 0};
    int s = 0;
    if (i < p.B) {
      s = p.seqlens[i];
      const int n = p.new_tokens[i];
      if (s < 0 || s > cap || n < -1 || (n > 0 && static_cast<long long>(s) + n > cap)) {
        bad = true;
        s = 0;
      } else {
        const int have = (s + ps - 1) / ps;
        if (n < 0) {
          v.back = have;
        } else if (n > 0) {
          v.q = n;
          v.k = static_cast<long long>(s) + n;
          v.take = (s + n + ps - 1) / ps - have;
        }
      }
    }
    Four in = v;  // inclusive sum over the warp
    for (int d = 1; d < 32; d <<= 1) {
      const Four o = shfl_up(in, d);
      if (lane >= d) in = in + o;
    }
    if (lane == 31) warp_sum[warp] = in;
    __syncthreads();
    if (warp == 0) {
      Four w = warp_sum[lane];
      for (int d = 1; d < 32; d <<= 1) {
        const Four o = shfl_up(w, d);
        if (lane >= d) w = w + o;
      }
      warp_sum[lane] = w;
    }
    __syncthreads();
    Four before = carry;
    if (warp > 0) before = before + warp_sum[warp - 1];
    const Four incl = before + in;
    if (i < p.B) {
      s_len[i] = s;
      s_q[i] = static_cast<int>(incl.q - v.q);
      s_take[i] = static_cast<int>(incl.take - v.take);
      s_back[i] = static_cast<int>(incl.back - v.back);
      if (lead) p.cu_k[i] = static_cast<int>(incl.k - v.k);
    }
    carry = carry + warp_sum[kPlanThreads / 32 - 1];
    __syncthreads();
  }
  bad = bad || carry.q > p.total_max || carry.k > 0x7fffffffLL ||
        carry.take > count + carry.back || count + carry.back > p.num_pages;
  bad = __syncthreads_or(bad);  // every block finds the same
  // every input that the outputs may overlay (lengths, ring state) has been read by now
  if (gridDim.x > 1) cluster_sync_all();
  if (bad) {
    // the step does not fit: nothing is taken or returned, and no row has a slot
    if (lead && tid == 0) flag_device_error(DEV_NO_FIT);
    for (int i = gid; i < p.B; i += all)
      if (p.seqlens_out != p.seqlens) p.seqlens_out[i] = p.seqlens[i];
    for (int i = tid; lead && i <= p.B; i += kPlanThreads) p.cu_q[i] = p.cu_k[i] = 0;
    for (int i = gid; i < p.total_max; i += all) {
      p.slots[i] = -1;
      if (p.positions) p.positions[i] = -1;
    }
    if (lead && tid == 0) {
      p.state_out[0] = head;
      p.state_out[1] = count;
    }
    return;
  }
  const int total = static_cast<int>(carry.q), take = static_cast<int>(carry.take);
  const int back = static_cast<int>(carry.back);
  if (tid == 0) {
    s_q[p.B] = total;
    s_take[p.B] = take;
    s_back[p.B] = back;
  }
  if (lead && tid == 0) {
    p.cu_k[p.B] = static_cast<int>(carry.k);
    p.state_out[0] = static_cast<int>((static_cast<long long>(head) + take) % p.num_pages);
    p.state_out[1] = count + back - take;
  }
  __syncthreads();

  // the f-th page of the ended requests, and the a-th page taken: the ring's free pages first, then
  // the pages returned in this step (read where they come from, so that nothing waits for a write)
  auto returned = [&](int f) {
    const int b = owner(s_back, p.B, f);
    return p.block_table[static_cast<size_t>(b) * p.max_pages + (f - s_back[b])];
  };
  auto taken = [&](int a) {
    if (a >= count) return returned(a - count);
    int at = head + a - (p.num_pages - head <= a ? p.num_pages : 0);
    return p.ring[at];
  };
  bool odd = false;
  for (int f = gid; f < back; f += all) {
    const long long at = static_cast<long long>(head) + count + f;
    p.ring[at % p.num_pages] = returned(f);
  }
  for (int a = gid; a < take; a += all) {
    const int b = owner(s_take, p.B, a);
    const int have = (s_len[b] + ps - 1) / ps;
    p.block_table[static_cast<size_t>(b) * p.max_pages + have + (a - s_take[b])] = taken(a);
  }
  for (int i = gid; i < p.B; i += all) {
    const int n = s_q[i + 1] - s_q[i];
    const bool ended = s_back[i + 1] > s_back[i];
    p.seqlens_out[i] = ended ? 0 : s_len[i] + n;
  }
  for (int i = gid; i <= p.B; i += all) p.cu_q[i] = s_q[i];
  for (int i = gid; i < p.total_max; i += all) {
    int slot = -1, pos = -1;
    if (i < total) {
      const int b = owner(s_q, p.B, i);
      pos = s_len[b] + (i - s_q[b]);
      const int pi = pos / ps, have = (s_len[b] + ps - 1) / ps;
      const int page = pi < have ? p.block_table[static_cast<size_t>(b) * p.max_pages + pi]
                                 : taken(s_take[b] + pi - have);
      if (page >= 0 && page < p.num_pages) slot = page * ps + (pos - pi * ps);
      else odd = true;
    }
    p.slots[i] = slot;
    if (p.positions) p.positions[i] = pos;
  }
  if (odd) flag_device_error(DEV_BAD_INDEX);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  PlanParams p{a.seqlens, a.new_tokens, a.seqlens_out, a.block_table, a.free_ring, a.ring_state,
               a.ring_state_out, a.cu_seqlens_q, a.cu_seqlens_k, a.slot_map, a.positions,
               a.B, a.max_pages, a.num_pages, a.page_size, a.total_max};
  const int smem = (4 * a.B + 3) * static_cast<int>(sizeof(int));
  static_assert((4 * kPlanMaxRequests + 3) * 4 <= 200 * 1024, "shared memory");
  // Blocks for the slots and the requests, about two rounds of their threads each. (GPU time of 1, 2, 4 and
  // 8 blocks for 33K new tokens: 31.3, 18.3, 11.7, 8.5 us; for 256 requests of one token one block takes
  // 5.1 and 8 take 5.5.)
  const int work = a.total_max > a.B ? a.total_max : a.B;
  int blocks = 1;
  while (blocks < kPlanCluster && blocks * 2 * kPlanThreads < work) blocks *= 2;
  static std::atomic<uint64_t> raised{0};
  return launch_early_large(paged_plan_kernel, blocks, kPlanThreads, smem, (4 * kPlanMaxRequests + 3) * 4, st, blocks, p, raised);
}

cudaError_t status_paged_plan(int* v) { return launched_status(v); }

}  // namespace da
