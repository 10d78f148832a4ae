// kv_plan.cuh -- what a batch of requests needs before its layers run, from
// the request lengths alone: row offsets, positions, cache slots, total lengths
// and the block-table entries of the pages that the new tokens open.
//
// Request b brings q_b tokens behind the n_b that it has cached; with pages of
// P tokens it opens ceil((n_b + q_b) / P) - ceil(n_b / P) new pages, taken from
// the free list in request order.  Its token t sits at position n_b + t and in
// slot table[b][position / P] * P + position % P.
//
// One launch: every CTA scans all request lengths itself (two block scans in
// shared memory, about a microsecond for a thousand requests), which needs no
// exchange between CTAs, then writes its own share of the rows and of the new
// table entries.  Entries that hold cached pages are only read and new ones only
// written (a token in a new page takes its page from the free list, not from the
// table), so the CTAs do not race.  The launch and the scans bound it, not its few
// hundred kilobytes: 4.4 us for 64 requests of one token, 7.3 us for 1000 requests
// and 30000 rows (back to back in a graph).
#pragma once

#include <cstdint>

#include "kv_common.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

constexpr int kPlanThreads = 512;
constexpr int kPlanRows = 1024;            // rows of positions and slots per CTA
constexpr int kPlanRequests = 64;          // requests whose results a CTA writes, a warp each
constexpr int kPlanMaxRequests = 16384;    // 8 bytes of shared memory each

struct PlanParams {
  const int* q_lens;
  const int* kv_lens;
  int* table;
  long long table_stride;
  int width;
  const int* free_pages;
  int free_count;
  int batch, rows, page_log2;
  int* cu_q;
  int* total;
  int* positions;
  long long* slots;
  int* used;
};

// Inclusive sum over the block of one value per thread; `warp_sums` is shared.
__device__ __forceinline__ long long block_inclusive_sum(long long v, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();                          // warp_sums may still be read from the previous scan
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) before += w < warp ? warp_sums[w] : 0;
  return v + before;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
  extern __shared__ int plan_smem[];
  int* cu = plan_smem;                      // [batch + 1] first row of each request
  int* first = plan_smem + p.batch + 1;     // [batch] its first page of the free list
  __shared__ long long warp_sums[kPlanThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  const int mask = (1 << p.page_log2) - 1;
  bool bad = false;

  // new tokens of request b: a negative length, or a total past 31 bits, counts as none
  auto lengths = [&](int b, int& q, int& n) {
    q = p.q_lens[b];
    n = p.kv_lens[b];
    if (q < 0 || n < 0 || static_cast<long long>(q) + n > 0x7fffffffLL) {
      bad = true;
      q = 0;
      n = max(n, 0);
    }
  };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    int q, n;
    lengths(b, q, n);
    mine += q;
  }
  long long run = block_inclusive_sum(mine, warp_sums) - mine;
  if (tid == 0) cu[0] = 0;
  for (int b = b0; b < b1; ++b) {
    int q, n;
    lengths(b, q, n);
    run += q;
    if (run > p.rows) bad = true;           // tokens past the last row are dropped
    cu[b + 1] = static_cast<int>(min(run, static_cast<long long>(p.rows)));
  }
  __syncthreads();

  // pages: a request's table row ends at `width`
  auto pages = [&](int b, int& held, int& need) {
    int q, n;
    lengths(b, q, n);
    q = cu[b + 1] - cu[b];
    const long long total = static_cast<long long>(n) + q;
    held = static_cast<int>((static_cast<long long>(n) + mask) >> p.page_log2);
    const long long want = (total + mask) >> p.page_log2;
    if (want > p.width) bad = true;
    need = static_cast<int>(min(want, static_cast<long long>(p.width)));
    need = max(need, held);
  };
  mine = 0;
  for (int b = b0; b < b1; ++b) {
    int held, need;
    pages(b, held, need);
    mine += need - held;
  }
  const long long upto = block_inclusive_sum(mine, warp_sums);
  run = upto - mine;
  for (int b = b0; b < b1; ++b) {
    int held, need;
    pages(b, held, need);
    first[b] = static_cast<int>(min(run, 0x7fffffffLL));
    run += need - held;
  }
  if (tid == kPlanThreads - 1) {
    if (upto > p.free_count) bad = true;
    if (blockIdx.x == 0) *p.used = static_cast<int>(min(upto, static_cast<long long>(p.free_count)));
  }
  __syncthreads();

  // this CTA's requests (every gridDim.x-th): offsets, totals, new table entries
  const int lane = tid & 31;
  if (blockIdx.x == 0 && tid == 0) p.cu_q[0] = 0;
  for (int b = blockIdx.x + (tid >> 5) * gridDim.x; b < p.batch; b += gridDim.x * (kPlanThreads / 32)) {
    int held, need, q, n;
    pages(b, held, need);
    lengths(b, q, n);
    if (lane == 0) {
      p.cu_q[b + 1] = cu[b + 1];
      p.total[b] = n + cu[b + 1] - cu[b];
    }
    for (int j = lane; j < need - held; j += 32) {
      const long long f = static_cast<long long>(first[b]) + j;
      p.table[b * p.table_stride + held + j] = f < p.free_count ? p.free_pages[f] : -1;
    }
  }

  // this CTA's rows
  const int r_end = min((static_cast<int>(blockIdx.x) + 1) * kPlanRows, p.rows);
  for (int r = blockIdx.x * kPlanRows + tid; r < r_end; r += kPlanThreads) {
    int pos = -1;
    long long slot = -1;
    if (r < cu[p.batch]) {
      int lo = 0, hi = p.batch;             // the last request that starts at or before row r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid;
      }
      int held, need, q, n;
      pages(lo, held, need);
      lengths(lo, q, n);
      pos = n + r - cu[lo];
      const int col = pos >> p.page_log2;
      int page = -1;
      if (col < held) {
        if (col < p.width) page = p.table[lo * p.table_stride + col];
      } else if (col < need) {
        const long long f = static_cast<long long>(first[lo]) + (col - held);
        if (f < p.free_count) page = p.free_pages[f];
      }
      if (page >= 0)
        slot = (static_cast<long long>(page) << p.page_log2) + (pos & mask);
      else
        bad = true;
    }
    p.positions[r] = pos;
    p.slots[r] = slot;
  }
  if (bad) raise_error(kErrIndex);
}

}  // namespace svdq
