// kv_sched.cuh -- how the attention kernels share their work.
//
// An item is one tile of RT query rows (a row is a token and one of the query
// heads that share a key head) of one request and key head; its keys, cut into
// units of KT, are the work.  The units of all items, in the order request, key
// head, row tile, key, form one line that the CTAs cut into equal contiguous
// shares, whatever the lengths: a CTA finishes whole items by itself, and an item
// that spans CTAs is joined by the last of them to arrive.  Lengths stay on the
// GPU: each CTA finds its share by itself, 32 requests at a time per warp.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "kv_cache.cuh"
#include "kv_common.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): m = ceil(2^(31 + s) / d), s = ceil(log2 d).
struct FastDiv {
  uint32_t m;
  int shift, d;
};
__host__ inline FastDiv fast_div(int d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  FastDiv f;
  f.d = d;
  f.shift = 31 + s;
  f.m = static_cast<uint32_t>(((1ull << f.shift) + d - 1) / d);
  return f;
}
__device__ __forceinline__ int operator/(int n, const FastDiv& f) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(n)) * f.m) >> f.shift);
}

struct AttnParams {
  KvGeom g;
  const __nv_bfloat16* q;
  long long q_stride;            // elements between rows
  __nv_bfloat16* out;
  long long out_stride;
  float* lse;                    // [rows][q_heads], or null
  const int* cu_q;               // [batch + 1]
  const int* kv_lens;            // [batch]
  const int* table;
  long long table_stride;
  int width;
  int batch, rows, q_heads;
  FastDiv rep;                   // query heads per key head; rows * rep < 2^31
  int causal, window;
  float scale;
  float* partials;               // workspace: 2 slots per CTA of RT x D sums and RT (max, sum) pairs
  unsigned long long* counters;  // workspace: one word per CTA
  unsigned long long nonce;      // of this launch, in the upper 48 bits
  int min_units;                 // units that make a CTA worth its share
  long long budget;              // of a bounded wait, in cycles
};

// Keys of a request; rows and windows are cut to it too, so that positions stay far inside 32 bits.
constexpr long long kMaxKeys = (1ll << 30) - 65536;

struct Request {
  int row0, n, kv;               // first row, new tokens, keys
};

// Lengths as the caller gives them, cut to what the rows and the table hold.
__device__ __forceinline__ Request load_request(const AttnParams& p, int b) {
  const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], kv = p.kv_lens[b];
  const long long cap = min(static_cast<long long>(p.width) << p.g.page_log2, kMaxKeys);
  Request r;
  r.row0 = min(max(c0, 0), p.rows);
  r.n = min(max(c1, r.row0), p.rows) - r.row0;
  r.kv = static_cast<int>(min(static_cast<long long>(max(kv, 0)), cap));
  if (c0 != r.row0 || c1 != r.row0 + r.n || kv != r.kv) raise_error(kErrIndex);
  return r;
}

// Keys [low, k1) that any row of tile rt sees; k0 is low cut down to a multiple of KT.  What lies between k0 and low
// is in front of every row's window: its pages may be gone and its bytes anything, so it is neither looked up nor used.
template <int RT, int KT>
__device__ __forceinline__ void tile_keys(const AttnParams& p, const Request& r, int rt, int& k0, int& k1, int& low) {
  const int rows = r.n * p.rep.d;
  k1 = p.causal ? max(0, min(r.kv, r.kv - r.n + (min((rt + 1) * RT, rows) - 1) / p.rep + 1)) : r.kv;
  low = min(k1, p.window > 0 ? max(0, r.kv - r.n + (rt * RT) / p.rep - p.window + 1) : 0);
  k0 = low / KT * KT;
}

// Units of a tile: at least one, so that rows without keys are written too.
template <int RT, int KT>
__device__ __forceinline__ int tile_units(const AttnParams& p, const Request& r, int rt) {
  int k0, k1, low;
  tile_keys<RT, KT>(p, r, rt, k0, k1, low);
  return max(1, (k1 - k0 + KT - 1) / KT);
}

template <int RT>
__device__ __forceinline__ int row_tiles(const AttnParams& p, const Request& r) {
  return (r.n * p.rep.d + RT - 1) / RT;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Units of one key head of the requests base .. base + 31, one per lane: a lane adds
// up a few tiles by itself, and the warp goes over a long request's tiles together.
template <int RT, int KT>
__device__ __forceinline__ long long group_units(const AttnParams& p, int base, Request& r) {
  const int lane = threadIdx.x & 31, b = base + lane;
  r = Request{0, 0, 0};
  if (b < p.batch) r = load_request(p, b);
  const int tiles = row_tiles<RT>(p, r);
  constexpr int kFew = 4;
  long long mine = 0;
  if (tiles <= kFew)
    for (int rt = 0; rt < tiles; ++rt) mine += tile_units<RT, KT>(p, r, rt);
  unsigned many = __ballot_sync(0xffffffffu, tiles > kFew);
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    Request o;
    o.row0 = 0;
    o.n = __shfl_sync(0xffffffffu, r.n, src);
    o.kv = __shfl_sync(0xffffffffu, r.kv, src);
    const int n = __shfl_sync(0xffffffffu, tiles, src);
    long long s = 0;
    for (int rt = lane; rt < n; rt += 32) s += tile_units<RT, KT>(p, o, rt);
    s = warp_sum(s);
    if (lane == src) mine = s;
  }
  return mine;
}

__device__ __forceinline__ long long warp_inclusive(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Where a CTA's share begins, and its size.  In shared memory.
struct Share {
  long long base;                // units of a CTA's share; the first `rem` CTAs have one more
  long long begin;               // first unit of this CTA
  int rem;
  int snap;                      // see find_share
  int count;                     // units of this CTA (0: none)
  int b, h, rt, unit;            // the item of the first unit, and the unit inside it
};

// n / d, in 32 bits where they hold it (the usual case; 64-bit division is a long subroutine).
__device__ __forceinline__ long long div_units(long long n, long long d) {
  if (((n | d) >> 32) == 0) return static_cast<long long>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d));
  return n / d;
}
__device__ __forceinline__ long long share_begin(long long base, int rem, int c) { return base * c + min(c, rem); }
// The CTA whose share holds unit u.
__device__ __forceinline__ int share_of(long long base, int rem, long long u) {
  const long long head = (base + 1) * rem;
  return static_cast<int>(u < head ? div_units(u, base + 1) : rem + div_units(u - head, base));
}

// Where unit u lies, found by one warp from the 32 requests in its lanes' `one` and `r` (groups == 1) or from
// the sums of 32 requests each.
struct Place {
  int b, h, rt, unit, units;     // the item, the unit inside it, its units
};
template <int RT, int KT>
__device__ __forceinline__ Place find_unit(const AttnParams& p, const long long* sums, int groups, Request r, long long one, long long left) {
  const int lane = threadIdx.x & 31;
  int g = 0;
  if (groups > 1) {
    // the group of 32 requests that holds it
    for (int base = 0;; base += 32) {
      const long long v = base + lane < groups ? sums[base + lane] : 0;
      const long long inc = warp_inclusive(v);
      const unsigned over = __ballot_sync(0xffffffffu, inc > left);
      if (over) {
        const int k = __ffs(over) - 1;
        left -= __shfl_sync(0xffffffffu, inc - v, k);
        g = base + k;
        break;
      }
      left -= __shfl_sync(0xffffffffu, inc, 31);
      if (base + 32 >= groups) break;         // not reached: u < total
    }
    one = group_units<RT, KT>(p, 32 * g, r);
  }
  // the request, the key head, the row tile
  const long long v = one * p.g.heads, inc = warp_inclusive(v);
  const unsigned over = __ballot_sync(0xffffffffu, inc > left);
  const int k = over ? __ffs(over) - 1 : 0;
  left -= __shfl_sync(0xffffffffu, inc - v, k);
  const long long per_head = max(1LL, __shfl_sync(0xffffffffu, one, k));
  Request o;
  o.row0 = 0;
  o.n = __shfl_sync(0xffffffffu, r.n, k);
  o.kv = __shfl_sync(0xffffffffu, r.kv, k);
  Place at;
  at.b = 32 * g + k;
  at.h = static_cast<int>(div_units(left, per_head));
  left -= at.h * per_head;
  const int tiles = row_tiles<RT>(p, o);
  at.rt = 0;
  if (tiles > 1) {
    for (int base = 0; base < tiles; base += 32) {
      const long long w = base + lane < tiles ? tile_units<RT, KT>(p, o, base + lane) : 0;
      const long long winc = warp_inclusive(w);
      const unsigned past = __ballot_sync(0xffffffffu, winc > left);
      if (past) {
        const int j = __ffs(past) - 1;
        left -= __shfl_sync(0xffffffffu, winc - w, j);
        at.rt = base + j;
        break;
      }
      left -= __shfl_sync(0xffffffffu, winc, 31);
    }
  }
  at.unit = static_cast<int>(left);
  at.units = tiles > 0 ? tile_units<RT, KT>(p, o, at.rt) : 1;
  return at;
}

// A cut costs the many-row kernel one more end of an item, 13 to 20 thousand cycles where a unit takes 3700.
constexpr int kCutUnits = 5;

// Called by all threads.  `sums` holds (batch + 31) / 32 words of shared memory.
// SNAP: a boundary between shares that lies within share.snap units of an item's end moves there: by what a cut costs,
// kCutUnits, at most, so that no share pays more for the longer way than the cut would have cost it (and by a sixth of
// a share, so that boundaries keep their order).  A prompt of 4096 tokens, 32 query and 8 key heads: 209 us, 227 if none
// moves, 204 if all within a sixth of a share do; 2500 tokens over 6000 keys: 208, 209 and 235.
// Items of one length are not cut at all where whole ones make the largest share no more than kCutUnits longer than
// equal shares.  Tokens attending to each other, uncut and cut: 2048 of 18 heads (144 items of 16 units) 47 and 61 us;
// 2304 of 32 heads (288 of 18) 92 and 107; 4608 of 24 heads (432 of 36) 240 and 257; but 4096 of 24 heads (384 of 32, in
// the largest share 96, in equal ones 83) 220 and 214.
template <int RT, int KT, bool SNAP>
__device__ __forceinline__ void find_share(const AttnParams& p, long long* sums, Share* s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int groups = (p.batch + 31) / 32;
  Request r;
  long long one = 0;                          // units of one key head of this lane's request
  for (int g = warp; g < groups; g += warps) {
    one = group_units<RT, KT>(p, 32 * g, r);
    const long long t = warp_sum(one);
    if (lane == 0) sums[g] = t * p.g.heads;
  }
  if (groups > 1) __syncthreads();
  if (warp == 0) {
    __syncwarp();
    long long total = 0;
    for (int g = lane; g < groups; g += 32) total += sums[g];
    total = warp_sum(total);
    const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), div_units(total + p.min_units - 1, p.min_units)));
    const int c = blockIdx.x;
    if (c >= ctas) {                          // also when there is no work at all
      if (lane == 0) s->count = 0;
    } else {
      const long long each = div_units(total, ctas);
      const int rem = static_cast<int>(total - each * ctas);
      int snap = 0;
      if (SNAP) {
        snap = static_cast<int>(min(each / 6, static_cast<long long>(kCutUnits)));
        if (groups == 1 && !p.causal && p.window == 0) {         // the tiles of a request are alike
          const int len = row_tiles<RT>(p, r) > 0 ? tile_units<RT, KT>(p, r, 0) : 0;
          const int most = __reduce_max_sync(0xffffffffu, len);
          if (__all_sync(0xffffffffu, len == 0 || len == most)) {
            const long long items = div_units(total, most), whole = div_units(items + ctas - 1, ctas) * most;
            if (whole <= each + kCutUnits) snap = max(snap, most / 2);   // every boundary is as near to an end
          }
        }
      }
      long long begin = share_begin(each, rem, c), end = share_begin(each, rem, c + 1);
      Place at = find_unit<RT, KT>(p, sums, groups, r, one, begin);
      if (SNAP) {
        auto moved = [&](const Place& w) {    // by how much the boundary at w moves
          const int back = w.unit, on = w.units - w.unit;
          return min(back, on) > snap || back == 0 ? 0 : back <= on ? -back : on;
        };
        const int d = moved(at);
        begin += d;
        if (d < 0) at.unit = 0;
        if (d > 0) at = find_unit<RT, KT>(p, sums, groups, r, one, min(begin, total - 1));
        if (c + 1 < ctas) end += moved(find_unit<RT, KT>(p, sums, groups, r, one, end));
      }
      if (lane == 0) {
        s->base = each;
        s->begin = begin;
        s->rem = rem;
        s->snap = snap;
        s->count = static_cast<int>(max(0LL, min(end - begin, 0x7fffffffLL)));
        s->b = at.b;
        s->h = at.h;
        s->rt = at.rt;
        s->unit = at.unit;
      }
    }
  }
  __syncthreads();
}

// The CTAs c0 .. c1 that an item of `units` units from unit number `item` is cut between.
__device__ __forceinline__ void item_parts(const Share& s, long long item, int units, int& c0, int& c1) {
  c0 = share_of(s.base, s.rem, item + s.snap);
  c1 = max(c0, share_of(s.base, s.rem, item + max(0, units - 1 - s.snap)));
}

// ------------------------------------------------------------- split items ---
// An item cut between CTAs c0 .. c1 leaves a partial result per CTA: its first part in
// slot 2 c0 + 1 (it is the last of c0's share), the others in slot 2c of theirs.  Counter word c0 counts arrivals.  The words need no initial value: one
// that does not carry the launch's 48-bit nonce counts as zero, and the last CTA
// to arrive leaves zero behind, so a graph that replays the launch starts from
// zero too.  Sums are taken in the order of the CTAs, whoever arrives last.

// One thread.  True if this is the last of `parts` arrivals.
__device__ __forceinline__ bool arrive_last(unsigned long long* word, unsigned long long nonce, int parts) {
  unsigned long long old = 0;                 // what a workspace in use holds between launches
  while (true) {
    const unsigned long long count = (old & ~0xFFFFull) == nonce ? (old & 0xFFFFull) : 0ull;
    const bool last = count + 1 == static_cast<unsigned long long>(parts);
    const unsigned long long seen = atomicCAS(word, old, last ? 0ull : (nonce | (count + 1)));
    if (seen == old) return last;
    old = seen;
  }
}

}  // namespace svdq
