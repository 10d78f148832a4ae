// kv_attn_rows.cuh -- attention over the paged 4-bit cache for many query rows
// per key head (prompts, chunks of prompts, whole images), on tcgen05.
//
// A tile is 256 rows (a row is a token and one query head of the key head's
// group) as two halves of 128, walked over the keys 128 at a time:
//   S_w = Q_w K^T   (128 x 128 x D, operands in shared memory, TMEM columns 128 w)
//   P_w = exp2(S_w f - m), fp16, written over the first half of S_w in TMEM
//   O_w += P_w V    (128 x D x 128, P from TMEM, V from shared memory, columns 256 + 128 w)
// Sixteen warps: two groups of four keep the softmax of a half each (a thread per
// row: maximum, sum and row factor are private to it), four turn codes into fp16
// tiles, one issues the MMAs.  While a half's softmax runs, the tensor core works
// for the other half.
//
// 4608 tokens of 24 heads attending to each other, NVFP4: 240 us, 1090 TFLOP/s; 3
// prompts of up to 1500 tokens over up to 6000 keys, FP4 g32: 195 us, 690 TFLOP/s;
// INT4, with its second product for the keys: 337 us, and 3 such prompts of other lengths 238 us, 480
// TFLOP/s (561 and 317 with its tiles worked out in fp32 instead of fp16 pairs).  A tile of 128 keys takes 3700 cycles,
// 2048 of them on the tensor core; the chain scores - softmax -
// values - scores of a half (2000 + 1100 + hand-offs) bounds it, and 13 to 20 thousand
// cycles at each end of an item.
//
// Numbers.  FP4 values (code * scale) are exact in fp16.  INT4 values need up to 14
// bits: keys enter as a pair hi + lo of fp16 values (two MMAs), values are rounded once
// to fp16 (2^-11, as the weights); both are multiplied by a power of two that brings
// the largest scale (of the tile's keys, of the values so far) to 2^10 .. 2^11, so
// that what fp16 keeps reaches down to scales 2^-24 of it: keys are exact to there.
// The power goes into the scores' factor and the sums' scale.  Queries are divided
// by a power of two per row, as in the decode kernel.  The maximum is followed
// lazily: it moves when a row's scores pass it by more than 2^5, so most tiles leave O
// alone; weights are exp2(x - m + 10) <= 2^15 and keep 2^-11 relative down to
// 2^-24 of the largest, 2^-35 absolute.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv_attn.cuh"
#include "kv_cache.cuh"
#include "kv_common.cuh"
#include "kv_sched.cuh"
#include "svdq_formats.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

constexpr int kRowsThreads = 512;
constexpr int kRowsTile = 256;
constexpr int kRowsKeys = 128;
constexpr int kRowsRing = 4;                        // tiles whose masks and exponents are kept
constexpr float kRowsLazy = 5.f, kRowsShift = 10.f;
constexpr int kRowsInt4Up = 10;                     // INT4: the largest scale is brought to 2^10 .. 2^11 (times 8: below 2^14)

// Shared memory: Q (two halves), K stages (hi, and lo for INT4), V stages.
template <int FMT, int D>
struct RowsSmem {
  static constexpr int kPanel = 128 * 128;          // 128 rows of 64 fp16 values, 128-byte swizzle
  static constexpr int kTile = kPanel * (D / 64);
  static constexpr int kParts = FMT == kFmtInt4 ? 2 : 1;
  static constexpr int kKStages = (FMT == kFmtInt4 && D == 128) ? 1 : 2;
  static constexpr int kVStages = 2;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kTile;
  static constexpr int kV = kK + kKStages * kParts * kTile;
  static constexpr int kBars = kV + kVStages * kTile;
  static constexpr int kMisc = kBars + 256;
  static constexpr int kBytes = kMisc + 512 + 1024 /* alignment */;
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[smem] * B[smem], fp16 -> fp32; and with A in TMEM.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, P;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, P;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// fp16 x fp16 -> fp32; B K-major, or (transposed) with its N side contiguous.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_transposed) {
  return (1u << 4) | (b_transposed ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Byte offset of 16-byte chunk c (8 values) of row r in a tile of 64-value panels.
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// A CTA's walk over the items of its share; every role keeps its own.
struct Walk {
  int b, h, rt, unit, count;
  long long at;                  // unit number of the segment's first unit
  Request req;
  int k0, k1, low, units, here, first;
};
template <int RT, int KT>
__device__ __forceinline__ void walk_segment(const AttnParams& p, Walk& w) {
  tile_keys<RT, KT>(p, w.req, w.rt, w.k0, w.k1, w.low);
  w.units = max(1, (w.k1 - w.k0 + KT - 1) / KT);
  w.here = min(w.units - w.unit, w.count);
  w.first = w.k0 + w.unit * KT;
}
template <int RT, int KT>
__device__ __forceinline__ Walk walk_start(const AttnParams& p, const Share& s) {
  Walk w;
  w.b = s.b, w.h = s.h, w.rt = s.rt, w.unit = s.unit, w.count = s.count, w.at = s.begin;
  if (w.count > 0) {
    w.req = load_request(p, w.b);
    walk_segment<RT, KT>(p, w);
  }
  return w;
}
// To the next item; false at the end of the share.
template <int RT, int KT>
__device__ __forceinline__ bool walk_next(const AttnParams& p, Walk& w) {
  w.count -= w.here;
  w.at += w.here;
  if (w.count <= 0) return false;
  w.unit = 0;
  if (++w.rt >= row_tiles<RT>(p, w.req)) {
    w.rt = 0;
    if (++w.h >= p.g.heads) {
      w.h = 0;
      do {
        if (++w.b >= p.batch) return false;         // not reached: the share ends inside the batch
        w.req = load_request(p, w.b);
      } while (w.req.n == 0);
    }
  }
  walk_segment<RT, KT>(p, w);
  return true;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kRowsThreads, 1) kv_attn_rows_kernel(const AttnParams p) {
  using L = RowsSmem<FMT, D>;
  constexpr int RT = kRowsTile, KT = kRowsKeys;
  constexpr int SB = kv_scale_bytes(FMT, D);
  constexpr int SLOT = RT * (D + 2);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* q_full = bars;                            // [2] softmax -> MMA
  uint64_t* s_full = bars + 2;                        // [2] MMA -> softmax
  uint64_t* p_full = bars + 4;                        // [2] softmax -> MMA
  uint64_t* o_full = bars + 6;                        // [2] MMA -> softmax, last tile of a segment
  uint64_t* k_full = bars + 8;                        // [2] codes -> MMA
  uint64_t* k_empty = bars + 10;                      // [2]
  uint64_t* v_full = bars + 12;                       // [2]
  uint64_t* v_empty = bars + 14;                      // [2]
  uint64_t* join = bars + 16;                         // [2] the warps of a half, at a split item
  uint64_t* exps = bars + 18;                         // the code warps, at a tile's exponents (INT4)
  uint64_t* mma_done = bars + 19;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 20);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + L::kMisc);        // [ring][4]: a bit per key of a tile that counts
  int* kexp = reinterpret_cast<int*>(masks + 4 * kRowsRing);             // [ring]
  int* vexp = kexp + kRowsRing;                                          // [ring]
  int* last_flag = vexp + kRowsRing;                                     // [2]
  int* scratch = last_flag + 2;                                          // [2][8]
  __shared__ Share share;
  const int warp = static_cast<int>(warp_id()), lane = threadIdx.x & 31;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
      mbar_init(&join[i], 4);
    }
    mbar_init(exps, 4);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  griddep_wait();
  find_share<RT, KT, true>(p, reinterpret_cast<long long*>(smem), &share);
  fence_proxy_async_smem();                           // the scan's words lie under Q
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const long long budget = p.budget;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (warp_wait(bar, parity, budget, const_cast<int*>(abort_flag))) return true;
    if (lane == 0) {
      if (!*abort_flag) raise_error(kErrWaitAttn);
      *abort_flag = 1;
    }
    return false;
  };
  // A barrier of the warps that arrive on `bar`, bounded like every other wait.
  auto meet = [&](uint64_t* bar, uint32_t parity) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    return wait(bar, parity);
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int half = warp >> 2;
    const int lrow = (warp & 3) * 32 + lane;          // row of the half = TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);   // lanes 32 (warp % 4) ..
    const uint32_t s_cols = lane_base + 128 * half, o_cols = lane_base + 256 + 128 * half;
    const uint32_t q_addr = smem_u32(smem + L::kQ + half * L::kTile);
    uint32_t n_tiles = 0;                             // tiles of this half so far: phase of s_full
    uint32_t n_seg = 0, tile = 0;                     // segments of this half; tiles of the CTA (ring index)
    Walk w = walk_start<RT, KT>(p, share);
    bool more = w.count > 0;
    while (more) {
      const int rows = w.req.n * p.rep.d;
      const int row = w.rt * RT + half * 128 + lrow;
      if (w.rt * RT + half * 128 >= rows) {           // nothing in this half
        tile += w.here;
        more = walk_next<RT, KT>(p, w);
        continue;
      }
      const bool live = row < rows;
      const int tok = min(row, rows - 1) / p.rep;
      const int hq = w.h * p.rep.d + (min(row, rows - 1) - tok * p.rep.d);
      const int pos = w.req.kv - w.req.n + tok;
      const int hi = p.causal ? min(w.req.kv, pos + 1) : w.req.kv;
      const int lo = p.window > 0 ? pos - p.window + 1 : 0;
      // Queries: bf16 -> fp16 / 2^e, into the swizzled tile.  The warp loads its 32 rows D / 8 lanes a row, so a
      // load covers whole lines; a row's exponent goes to the lane that keeps the row.
      int e_row = 0;
      {
        constexpr int LPR = D / 8, RPL = 32 / LPR;    // lanes of a row, rows of a load
        const int c = lane % LPR;
        uint4 v[32 / RPL];
#pragma unroll
        for (int i = 0; i < 32 / RPL; ++i) {
          const int gr = w.rt * RT + half * 128 + (warp & 3) * 32 + i * RPL + lane / LPR;
          const int tk = min(gr, rows - 1) / p.rep;
          const __nv_bfloat16* src = p.q + (w.req.row0 + tk) * p.q_stride + (w.h * p.rep.d + (min(gr, rows - 1) - tk * p.rep.d)) * D;
          v[i] = gr < rows ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 32 / RPL; ++i) {
          const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          float amax = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) amax = fmax3(amax, fabsf(bf16_lo(u[j])), fabsf(bf16_hi(u[j])));
#pragma unroll
          for (int x = 1; x < LPR; x *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
          const int e = min(max(static_cast<int>((__float_as_uint(amax) >> 23) & 255u) - 127 - 12, -120), 120);
          const float inv = p.scale < 0.f ? -pow2(-e) : pow2(-e);     // a negative scale turns the queries round
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = pack_f16x2(bf16_lo(u[j]) * inv, bf16_hi(u[j]) * inv);
          sts128(q_addr + tile_chunk((warp & 3) * 32 + i * RPL + lane / LPR, c), h[0], h[1], h[2], h[3]);
          const int from = __shfl_sync(0xffffffffu, e, (lane % RPL) * LPR);
          if (lane / RPL == i) e_row = from;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[half]);
      }
      const float f = fmaxf(fabsf(p.scale) * 1.4426950408889634f * pow2(e_row), 1.17549435e-38f);
      float m = -INFINITY, l = 0.f;
      int ev = 0;
      bool ok = true;
      for (int j = 0; j < w.here; ++j, ++tile, ++n_tiles) {
        ok = wait(&s_full[half], n_tiles & 1);
        if (!ok) break;
        tc_fence_after();
        const uint4 mask = *reinterpret_cast<const uint4*>(masks + 4 * (tile % kRowsRing));
        float ft = f;
        float grow = 1.f;                             // change of the values' power of two
        if constexpr (FMT == kFmtInt4) {
          ft = fmaxf(f * pow2(kexp[tile % kRowsRing]), 1.17549435e-38f);
          const int e2 = vexp[tile % kRowsRing];
          if (j > 0) grow = pow2(max(ev - e2, -126));
          ev = e2;
        }
        const int base = w.first + j * KT;
        const bool cut = base < lo || base + KT > hi;
        const bool masked = __any_sync(0xffffffffu, cut || (mask.x & mask.y & mask.z & mask.w) != 0xffffffffu);
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_cols + 32 * c, sr[c]);
        tmem_wait_ld();
        if (masked) {
          const uint32_t mw[4] = {mask.x, mask.y, mask.z, mask.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t see = mw[c];                     // columns that this row sees
            const int b0 = base + 32 * c, under = lo - b0, over = hi - b0;
            if (under > 0) see &= under >= 32 ? 0u : 0xffffffffu << under;
            if (over < 32) see &= over <= 0 ? 0u : 0xffffffffu >> (32 - over);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((see >> i) & 1)) sr[c][i] = 0xff800000u;
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) top[k] = fmax3(top[k], __uint_as_float(sr[c][i + k]), __uint_as_float(sr[c][i + k + 4]));
        const float x = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * ft;
        const bool move = x > m + kRowsLazy;          // also from -inf
        float shrink = grow;
        if (move) {
          const float c = ex2(m - x);
          l *= c;
          shrink *= c;
          m = x;
        }
        const float sub = m == -INFINITY ? 0.f : kRowsShift - m;
        const float2 f2 = make_float2(ft, ft), b2 = make_float2(sub, sub);
        float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 v = ffma2(make_float2(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1])), f2, b2);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            sum2[i & 1] = fadd2(sum2[i & 1], v);
            pk[i] = pack_f16x2(v.x, v.y);
          }
          tmem_st16(s_cols + 16 * c, pk);
        }
        const float2 sum = fadd2(sum2[0], sum2[1]);
        l += sum.x + sum.y;
        if (__any_sync(0xffffffffu, shrink != 1.f) && j > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_cols + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
            tmem_st32(o_cols + c, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[half]);
      }
      if (!ok || !wait(&o_full[half], n_seg & 1)) break;
      ++n_seg;
      tc_fence_after();
      const bool split = w.unit > 0 || w.here < w.units;
      float unscale = 1.f;
      if constexpr (FMT == kFmtInt4) unscale = pow2(ev);
      // The finished rows leave through the half's query tile (its MMAs are done): a lane writes its row as
      // 16-byte chunks, and the warp copies its 32 rows out D / 8 lanes a row.  A row lies where its query lay: the
      // warps of a half do not wait for each other here, and a warp whose next queries are already in the tile must
      // find no other warp's rows in its own, nor leave its rows in theirs.
      auto put = [&](int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        sts128(q_addr + tile_chunk((warp & 3) * 32 + lane, chunk), a, b, c, d);
      };
      auto copy_out = [&]() {
        __syncwarp();
        constexpr int LPR = D / 8, RPL = 32 / LPR;
#pragma unroll 4
        for (int i = 0; i < 32 / RPL; ++i) {
          const int lr = i * RPL + lane / LPR, c = lane % LPR;
          const int gr = w.rt * RT + half * 128 + (warp & 3) * 32 + lr;
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(q_addr + tile_chunk((warp & 3) * 32 + lr, c)) : "memory");
          if (gr < rows) {
            const int tk = gr / p.rep;
            *reinterpret_cast<uint4*>(p.out + (w.req.row0 + tk) * p.out_stride + (w.h * p.rep.d + (gr - tk * p.rep.d)) * D + 8 * c) = v;
          }
        }
        __syncwarp();
      };
      // a partial result: [D / 4][256] float4, so that the lanes of a store are neighbours; then [256] (max, sum)
      float4* slot = reinterpret_cast<float4*>(p.partials + (2ll * blockIdx.x + (w.unit == 0 ? 1 : 0)) * SLOT);
      const int srow = half * 128 + lrow;
      const float inv = l == 0.f ? 0.f : unscale / l;    // a row without keys; a sum that is NaN stays NaN
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_cols + c, o);
        tmem_wait_ld();
        if (!split) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t pk[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pk[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
            put(c / 8 + i, pk[0], pk[1], pk[2], pk[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(slot + (c / 4 + i) * RT + srow,
                   make_float4(__uint_as_float(o[4 * i]) * unscale, __uint_as_float(o[4 * i + 1]) * unscale,
                               __uint_as_float(o[4 * i + 2]) * unscale, __uint_as_float(o[4 * i + 3]) * unscale));
        }
      }
      tc_fence_before();                              // O is read before the next segment's MMAs
      float* lse = p.lse == nullptr || !live ? nullptr : p.lse + static_cast<long long>(w.req.row0 + tok) * p.q_heads + hq;
      if (!split) {
        copy_out();
        if (lse != nullptr) *lse = l == 0.f ? -INFINITY : (m - kRowsShift + log2f(l)) * 0.6931471805599453f;
      } else {
        __stcg(reinterpret_cast<float2*>(slot + RT * (D / 4)) + srow, make_float2(m, l));
        // each half of an item is joined by itself, by the CTA whose four warps arrive last
        const long long item = w.at - w.unit;
        int c0, c1;
        item_parts(share, item, w.units, c0, c1);
        __threadfence();
        if (!meet(&join[half], 0)) break;
        if ((warp & 3) == 0 && lane == 0) {
          last_flag[half] = arrive_last(&p.counters[2 * c0 + half], p.nonce, c1 - c0 + 1);
          __threadfence();
        }
        if (!meet(&join[half], 1)) break;
        if (last_flag[half]) {
          const float* part0 = p.partials + (2ll * c0 + 1) * SLOT;
          auto part = [&](int c) { return reinterpret_cast<const float4*>(c == c0 ? part0 : p.partials + 2ll * c * SLOT); };
          float top = -INFINITY, total = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float2 ms = __ldcg(reinterpret_cast<const float2*>(part(c) + RT * (D / 4)) + srow);
            const float m2 = fmaxf(top, ms.x);
            total = m2 > -INFINITY ? total * ex2(top - m2) + ms.y * ex2(ms.x - m2) : total + ms.y;   // 0 or NaN
            top = m2;
          }
          const float each = total == 0.f ? 0.f : 1.f / total;
#pragma unroll 1
          for (int d = 0; d < D / 4; d += 8) {
            float4 acc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = c0; c <= c1; ++c) {
              const float mc = __ldcg(reinterpret_cast<const float2*>(part(c) + RT * (D / 4)) + srow).x;
              const float fc = mc > -INFINITY ? ex2(mc - top) * each : 0.f;
              float4 v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = __ldcg(part(c) + (d + i) * RT + srow);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                acc[i].x = fmaf(v[i].x, fc, acc[i].x), acc[i].y = fmaf(v[i].y, fc, acc[i].y);
                acc[i].z = fmaf(v[i].z, fc, acc[i].z), acc[i].w = fmaf(v[i].w, fc, acc[i].w);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              put(d / 2 + i, pack_bf16x2(acc[2 * i].x, acc[2 * i].y), pack_bf16x2(acc[2 * i].z, acc[2 * i].w),
                  pack_bf16x2(acc[2 * i + 1].x, acc[2 * i + 1].y), pack_bf16x2(acc[2 * i + 1].z, acc[2 * i + 1].w));
          }
          copy_out();
          if (lse != nullptr) *lse = total == 0.f ? -INFINITY : (top - kRowsShift + log2f(total)) * 0.6931471805599453f;
        }
      }
      more = walk_next<RT, KT>(p, w);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------- codes -> fp16 tiles
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const int key = threadIdx.x - 256;                // key of a tile
    constexpr int CW = D / 32;                        // 16-byte words of codes of a key
    uint32_t tile = 0;
    int run_ev = -1000;                               // largest value exponent of the segment so far
    Walk w = walk_start<RT, KT>(p, share);
    bool more = w.count > 0;
    // A tile's key codes are loaded while the values of the tile before are turned over, and its value codes while
    // its keys are; its page is looked up a tile ahead.  A key that no row of the item sees or in a bad page reads as zeros.
    struct Raw {
      uint4 c[CW];
      uint2 s;
    };
    auto page_of = [&](const Walk& w, int j) {
      const int t = w.first + j * KT + key;
      if (t >= w.k1 || t < w.low) return -1;
      const int page = p.table[w.b * p.table_stride + (t >> p.g.page_log2)];
      if (page < 0 || page >= p.g.num_pages) {
        raise_error(kErrIndex);
        return -1;
      }
      return page;
    };
    auto fetch = [&](int t, int page, int h, bool value) {
      Raw r;
      r.s = make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < CW; ++i) r.c[i] = make_uint4(0u, 0u, 0u, 0u);
      if (page >= 0) {
        const int off = t & (p.g.page - 1);
        const uint8_t* blk = p.g.pool + kv_block(p.g, page, h) + (value ? p.g.vc : 0);
        const uint4* c = reinterpret_cast<const uint4*>(blk + off * (D / 2));
#pragma unroll
        for (int i = 0; i < CW; ++i) r.c[i] = c[i];
        const uint8_t* sc = blk + p.g.ks + off * SB;
        if constexpr (SB == 8) {
          r.s = *reinterpret_cast<const uint2*>(sc);
        } else if constexpr (SB == 4) {
          r.s.x = *reinterpret_cast<const uint32_t*>(sc);
        } else {
          r.s.x = *reinterpret_cast<const uint16_t*>(sc);
        }
      }
      return r;
    };
    // FP4: scale pair of the 8 codes of chunk c
    auto fp4_tile = [&](uint32_t addr, const uint4 (&codes)[CW], const uint2& sc) {
      constexpr int NS = SB;                          // scales of the key
      uint32_t s2[NS];
#pragma unroll
      for (int i = 0; i < NS; i += 2) {
        const uint32_t word = i < 4 ? sc.x : sc.y;
        const uint32_t two = e4m3x2_to_f16((word >> (8 * (i & 3))) & 0xffffu);
        s2[i] = __byte_perm(two, two, 0x1010);
        if (i + 1 < NS) s2[i + 1] = __byte_perm(two, two, 0x3232);
      }
#pragma unroll
      for (int i = 0; i < CW; ++i) {
        const uint32_t u[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = 4 * i + k;
          const uint32_t s = s2[c * 8 / kv_group(FMT)];
          uint32_t h[4];
          e2m1x8_to_f16(u[k], h);
          sts128(addr + tile_chunk(key, c), hmul2_u(h[0], s), hmul2_u(h[1], s), hmul2_u(h[2], s), hmul2_u(h[3], s));
        }
      }
    };
    // INT4: code * scale * 2^e, rounded to fp16, and what the rounding left (LO; exact by the fused multiply-add)
    auto int4_tile = [&](uint32_t addr, uint32_t addr_lo, const uint4 (&codes)[CW], const uint2& sc, float up, bool lo) {
      uint32_t s2[D / 64];
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        const float s = int4_scale(sc.x, g) * up;
        s2[g] = pack_f16x2(s, s);
      }
#pragma unroll
      for (int i = 0; i < CW; ++i) {
        const uint32_t u[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = 4 * i + k;
          uint32_t h[4], hi[4], rest[4];
          int4x8_to_f16(u[k], h);                     // pairs (0, 4), (1, 5), (2, 6), (3, 7)
          const uint32_t v[4] = {__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410), __byte_perm(h[0], h[1], 0x7632),
                                 __byte_perm(h[2], h[3], 0x7632)};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            hi[x] = hmul2_u(v[x], s2[c / 8]);
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(rest[x]) : "r"(v[x]), "r"(s2[c / 8]), "r"(hi[x] ^ 0x80008000u));
          }
          sts128(addr + tile_chunk(key, c), hi[0], hi[1], hi[2], hi[3]);
          if (lo) sts128(addr_lo + tile_chunk(key, c), rest[0], rest[1], rest[2], rest[3]);
        }
      }
    };
    // exponent of the largest of a key's scales (fp16, at least 2^-24), over the warp
    auto warp_exponent = [&](uint32_t two) {
      int e = -24;
#pragma unroll
      for (int i = 0; i < SB / 2; ++i) {
        const float s = fabsf(__half2float(__ushort_as_half(static_cast<uint16_t>(i ? two >> 16 : two & 0xffffu))));
        e = max(e, static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127);
      }
      return __reduce_max_sync(0xffffffffu, min(e, 16));
    };

    Raw k, v;
    int page = -1, page_next = -1, at = 0;            // of the tile in k and v, of the one after; the tile's key
    if (more) {
      page = page_of(w, 0);
      at = w.first + key;
      k = fetch(at, page, w.h, false);
      v = fetch(at, page, w.h, true);
    }
    int j = 0, next_at = 0, next_h = 0;
    for (; more; ++tile) {
      // the tile after this one, maybe of the next segment
      const bool end = j + 1 == w.here, fresh = j == 0;
      if (end) {
        more = walk_next<RT, KT>(p, w);
        j = 0;
      } else {
        ++j;
      }
      if (more) {
        page_next = page_of(w, j);
        next_at = w.first + j * KT + key;
        next_h = w.h;
      } else {
        page_next = -1;
      }
      const unsigned good = __ballot_sync(0xffffffffu, page >= 0);
      const uint32_t ks = tile % L::kKStages, vs = tile % L::kVStages;
      const uint32_t kaddr = smem_u32(smem + L::kK + ks * L::kParts * L::kTile), vaddr = smem_u32(smem + L::kV + vs * L::kTile);
      int ek = 0;
      if constexpr (FMT == kFmtInt4) {
        if (fresh) run_ev = -1000;
        int* sc = scratch + 8 * (tile & 1);           // written again two tiles on, behind the next tile's barrier
        const int wk = warp_exponent(k.s.x), wv = warp_exponent(v.s.x);
        if (lane == 0) {
          sc[warp - 8] = wk;
          sc[warp - 4] = wv;
        }
        if (!meet(exps, tile & 1)) break;
        ek = max(max(sc[0], sc[1]), max(sc[2], sc[3]));
        run_ev = max(run_ev, max(max(sc[4], sc[5]), max(sc[6], sc[7])));
      }
      if (!wait(&k_empty[ks], ((tile / L::kKStages) & 1) ^ 1)) break;
      if (lane == 0) masks[4 * (tile % kRowsRing) + warp - 8] = good;
      if constexpr (FMT == kFmtInt4) {
        if (threadIdx.x == 256) {
          kexp[tile % kRowsRing] = ek - kRowsInt4Up;
          vexp[tile % kRowsRing] = run_ev - kRowsInt4Up;
        }
        int4_tile(kaddr, kaddr + L::kTile, k.c, k.s, pow2(kRowsInt4Up - ek), true);
      } else {
        fp4_tile(kaddr, k.c, k.s);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[ks]);
      k = fetch(next_at, page_next, next_h, false);
      if (!wait(&v_empty[vs], ((tile / L::kVStages) & 1) ^ 1)) break;
      if constexpr (FMT == kFmtInt4)
        int4_tile(vaddr, 0u, v.c, v.s, pow2(kRowsInt4Up - run_ev), false);
      else
        fp4_tile(vaddr, v.c, v.s);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[vs]);
      v = fetch(next_at, page_next, next_h, true);
      page = page_next;
      at = next_at;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 12) {
      // ---------------------------------------------------------------- MMA
      // The whole warp waits, one lane issues: descriptors then live in uniform registers (with one lane in the whole
      // loop an MMA took 80 to 120 cycles to issue, against 64 on the tensor core).
      {
        constexpr uint32_t id_s = idesc_f16_f32(128, KT, false), id_o = idesc_f16_f32(128, D, true);
        uint32_t tile = 0, pf[2] = {0, 0}, qf[2] = {0, 0};
        Walk w = walk_start<RT, KT>(p, share);
        bool more = w.count > 0, ok = true;
        const uint64_t qd = make_kmajor_desc(smem_u32(smem + L::kQ), 128), kd = make_kmajor_desc(smem_u32(smem + L::kK), 128);
        const uint64_t vd = make_sdesc(smem_u32(smem + L::kV), L::kPanel, 1024, kSwizzle128B);
        auto commit = [&](uint64_t* bar) {
          if (elect_one()) tc_commit(bar);
          __syncwarp();
        };
        // descriptors count addresses in 16 bytes: offsets are added to the low word's field
        auto scores = [&](int half, uint32_t stage) {
          if (elect_one()) {
#pragma unroll
          for (int part = 0; part < L::kParts; ++part)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k / 4) * L::kPanel + (k % 4) * 32;
              mma_f16_ss(tmem + 128 * half, qd + ((half * L::kTile + off) >> 4), kd + (((stage * L::kParts + part) * L::kTile + off) >> 4), id_s,
                         part > 0 || k > 0);
            }
          tc_commit(&s_full[half]);
          }
          __syncwarp();
        };
        auto values = [&](int half, uint32_t stage, bool first) {
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < KT / 16; ++k)
              mma_f16_ts(tmem + 256 + 128 * half, tmem + 128 * half + 8 * k, vd + ((stage * L::kTile + k * 2048) >> 4), id_o, !first || k > 0);
          }
          __syncwarp();
        };
        while (more && ok) {
          const int halves = w.rt * RT + 128 < w.req.n * p.rep.d ? 2 : 1;
          ok = wait(&k_full[tile % L::kKStages], (tile / L::kKStages) & 1);
          for (int i = 0; i < halves && ok; ++i) {
            ok = wait(&q_full[i], qf[i]++ & 1);
            if (!ok) break;
            tc_fence_after();
            scores(i, tile % L::kKStages);
          }
          if (!ok) break;
          commit(&k_empty[tile % L::kKStages]);
          for (int j = 0; j < w.here && ok; ++j, ++tile) {
            const bool next = j + 1 < w.here;
            const uint32_t ks = (tile + 1) % L::kKStages, vs = tile % L::kVStages;
            // what the code warps bring is there long before the weights
            ok = wait(&v_full[vs], (tile / L::kVStages) & 1) &&
                 (!next || L::kKStages == 1 || wait(&k_full[ks], ((tile + 1) / L::kKStages) & 1));
            for (int i = 0; i < halves && ok; ++i) {
              ok = wait(&p_full[i], pf[i]++ & 1);
              if (!ok) break;
              tc_fence_after();
              values(i, vs, j == 0);
              if (L::kKStages == 1 && next && i == 0) {   // a single stage is filled behind the scores before it
                ok = wait(&k_full[ks], ((tile + 1) / L::kKStages) & 1);
                if (!ok) break;
                tc_fence_after();
              }
              if (next)
                scores(i, ks);
              else
                commit(&o_full[i]);
            }
            if (!ok) break;
            commit(&v_empty[vs]);
            if (next) commit(&k_empty[ks]);
          }
          more = ok && walk_next<RT, KT>(p, w);
        }
        if (elect_one()) tc_commit(mma_done);
        __syncwarp();
      }
      // everything issued has retired before TMEM is released
      if (!warp_wait(mma_done, 0, drain_budget(budget), nullptr) && lane == 0) raise_error(kErrWaitAttn);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace svdq
