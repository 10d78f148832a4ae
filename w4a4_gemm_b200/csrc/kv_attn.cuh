// kv_attn.cuh -- attention over the paged 4-bit cache:
//
//   o_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(scale q_i . k_t - max),
//   lse_i = log sum_t exp(scale q_i . k_t)
//
// over the keys t that query i sees: t < kv_len, with `causal` t <= pos_i, with a
// window t > pos_i - window, where pos_i = kv_len - q_len + i.  A query that sees
// no key gives o = 0 and lse = -inf.
//
// The kernel of this file is for few query rows per key head (decode), which read the
// cache once: 64 requests of 2048 to 8192 keys, 8 key heads of 128, NVFP4: 84 us, 4.7 TB/s (FP4 g32
// 78, INT4 85); 3 requests of 131000 keys, INT4: 102 us, 4.2 TB/s; one of 1000 keys: 11 us.
// Latency at low occupancy bounds it: 157 registers and 74 KB per CTA leave three warps to a scheduler,
// each in one serial chain per 64 keys (wait, convert, scores, maximum, exp2, transpose, values).  Of the
// first case's cycles the schedulers issue in 53 % (46 million instructions, about 270 per 16 keys and key
// head), DRAM is busy in 54 %, the ALUs in 45 %; copies alone take 70 us.  Then the ends of the
// items.  A warp takes 64 keys at a time, all D, from a ring of bulk copies of its own, turns the codes into operand fragments in registers, and
// keeps a running maximum and sum per row; the warps of a CTA take turns along the
// keys and join at the end of an item.  The products run transposed,
//   S^T = K q^T,   O^T += V^T P^T,
// so that the keys (16 at a time) fill the 16-row side of mma.sync.m16n8k16 and
// the few query rows its 8-column side.
//   * FP4 formats: code * scale is exact in fp16 (2 + 4 significant bits), both for
//     keys and values.
//   * INT4: the codes are exact in fp16.  A key group's scale multiplies its partial
//     scores in fp32; a value group's scale, divided by the power of two of the largest
//     so far (a running exponent, like the running maximum), multiplies the weights
//     before they are rounded to fp16.
//   * Queries are bf16 and scores are products with fp16 keys: a row is divided by
//     the power of two of its largest element, which leaves an exact fp16 value for
//     every element down to 2^-17 of the largest and an error below 2^-36 of it
//     for the rest.  The factor goes into the scores' scale.
//   * Weights are exp2(x - max + 15) (14 for INT4), so that they, times a scale
//     below 2, end at 2^15 and fp16 holds them to 2^-11 relative down to 2^-29 of the
//     largest (2^-28), to 2^-40 (2^-39) absolute.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv_cache.cuh"
#include "kv_common.cuh"
#include "kv_sched.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

constexpr int kDecChunk = 64;                       // keys of a warp's step
constexpr int kDecBlocks = kDecChunk / 16;
constexpr int kDecStages = 2;
// CTAs of 4 warps, three to an SM, or one CTA of 12 (see kv_api.cuh).  A unit of work is a step of every warp.
constexpr int kDecWide = 12, kDecNarrow = 4;
// The weights are exp2(x - max + shift).
__host__ __device__ constexpr float dec_shift(int fmt) { return fmt == kFmtInt4 ? 14.f : 15.f; }

__host__ __device__ constexpr int dec_stage_bytes(int fmt, int D) {
  return 2 * kDecChunk * (D / 2 + kv_scale_bytes(fmt, D));
}
__host__ __device__ constexpr uint32_t dec_smem_bytes(int fmt, int D, int NB, int warps) {
  return static_cast<uint32_t>(warps * kDecStages * (dec_stage_bytes(fmt, D) + 8 /* barriers */ + 8 /* what was loaded */) +
                               2 * warps * 8 * NB * 4 /* max, sum */ + 128);
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight E2M1 codes -> four fp16 pairs, code 2i in the low half of pair i.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// (a & b) ^ c and the bits of a where m is set, of b elsewhere, in one instruction each.
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t bit_select(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(d) : "r"(a), "r"(b), "r"(m));
  return d;
}

// Four 4-bit two's complement codes of each half word -> four fp16 pairs, pair i from bits 4i of both halves: u =
// code ^ 8 under the exponent of 1024 is 1024 + u (or 1024 + 16 u), minus 1032 (or / 16, minus 72).
__device__ __forceinline__ void int4x8_to_f16(uint32_t x, uint32_t* h) {
  const uint32_t y = x >> 8;
  const uint32_t p[4] = {and_xor(x, 0x000F000Fu, 0x64086408u), and_xor(x, 0x00F000F0u, 0x64806480u), and_xor(y, 0x000F000Fu, 0x64086408u),
                         and_xor(y, 0x00F000F0u, 0x64806480u)};
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(p[i]), "r"(0x64086408u));                               // 1032
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[i + 1]) : "r"(p[i + 1]), "r"(0x2C002C00u), "r"(0xD480D480u));  // 1/16, -72
  }
}

// Key of row m (0..15) of a 16-key block: pairs (2t, 2t + 1) are keys t and 4 + (t ^ 1), so that the rows
// of a fragment load lie in both halves of the 32 banks.
__device__ __forceinline__ int key_of_row(int m) {
  const int t = (m & 7) >> 1;
  return (m & 8) + ((m & 1) ? 4 + (t ^ 1) : t);
}

// Queries of one 8-row block as B fragments of K q^T.  Lane (r, t) holds elements of row r; pair k of
// register kk matches the key fragments below.  `f` receives 2^e of the row; `negate`: for a
// negative scale, which turns the queries round.
template <int FMT, int D>
__device__ __forceinline__ void load_queries(const __nv_bfloat16* row, bool live, int t, bool negate, uint32_t (&qf)[D / 8], float& f) {
  constexpr int N = D / 4;                            // elements of this lane
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  if (live) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      // FP4 at D = 128: 32 neighbouring elements per lane; else 16 of each group of 64
      const int d = (FMT != kFmtInt4 && D == 128) ? 32 * t + i : 64 * (i / 16) + 16 * t + i % 16;
      const uint4 w = *reinterpret_cast<const uint4*>(row + d);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i + 2 * j] = bf16_lo(u[j]);
        v[i + 2 * j + 1] = bf16_hi(u[j]);
      }
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // 2^e with 2^12 <= amax / 2^e < 2^13; both factors stay normal
  const int e = min(max(static_cast<int>((__float_as_uint(amax) >> 23) & 255u) - 127 - 12, -120), 120);
  f = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  const float inv = __uint_as_float((static_cast<uint32_t>(127 - e) << 23) | (negate ? 0x80000000u : 0u));
#pragma unroll
  for (int i = 0; i < N; i += 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // FP4 pairs are neighbours (2j, 2j + 1); INT4 pairs are (j, j + 4)
      const float a = FMT == kFmtInt4 ? v[i + j] : v[i + 2 * j];
      const float b = FMT == kFmtInt4 ? v[i + j + 4] : v[i + 2 * j + 1];
      qf[i / 2 + j] = pack_f16x2(a * inv, b * inv);
    }
  }
}

// Scores of 16 keys (rows `key`, `key + 8` of this lane) against NB blocks of 8 rows, before the rows' factors.
template <int FMT, int D, int NB>
__device__ __forceinline__ void key_scores(const uint8_t* codes, const uint8_t* scales, int key, int t, const uint32_t (&qf)[NB][D / 8],
                                           float (&s)[NB][4]) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[nb][i] = 0.f;
  if constexpr (FMT == kFmtInt4) {
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      const uint2 lo = *reinterpret_cast<const uint2*>(codes + key * (D / 2) + 32 * g + 8 * t);
      const uint2 hi = *reinterpret_cast<const uint2*>(codes + (key + 8) * (D / 2) + 32 * g + 8 * t);
      float part[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[nb][i] = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t x[4], y[4];
        int4x8_to_f16(w ? lo.y : lo.x, x);
        int4x8_to_f16(w ? hi.y : hi.x, y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a[4] = {x[2 * h], y[2 * h], x[2 * h + 1], y[2 * h + 1]};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_f16_16816(part[nb], a, qf[nb][8 * g + 4 * w + 2 * h], qf[nb][8 * g + 4 * w + 2 * h + 1]);
        }
      }
      const float s0 = __half2float(*reinterpret_cast<const __half*>(scales + key * (D / 32) + 2 * g));
      const float s1 = __half2float(*reinterpret_cast<const __half*>(scales + (key + 8) * (D / 32) + 2 * g));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        s[nb][0] = fmaf(part[nb][0], s0, s[nb][0]);
        s[nb][1] = fmaf(part[nb][1], s0, s[nb][1]);
        s[nb][2] = fmaf(part[nb][2], s1, s[nb][2]);
        s[nb][3] = fmaf(part[nb][3], s1, s[nb][3]);
      }
    }
  } else {
    constexpr int W = D / 32;                         // words (8 codes) of this lane per key
    uint32_t lo[W], hi[W];
    const uint8_t* at = codes + key * (D / 2) + 4 * W * t;
    if constexpr (W == 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(at), b = *reinterpret_cast<const uint4*>(at + 8 * (D / 2));
      lo[0] = a.x, lo[1] = a.y, lo[2] = a.z, lo[3] = a.w;
      hi[0] = b.x, hi[1] = b.y, hi[2] = b.z, hi[3] = b.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(at), b = *reinterpret_cast<const uint2*>(at + 8 * (D / 2));
      lo[0] = a.x, lo[1] = a.y;
      hi[0] = b.x, hi[1] = b.y;
    }
    // scale pairs (s, s): of word w's group, for the keys `key` (lo) and `key + 8` (hi)
    constexpr int SB = kv_scale_bytes(FMT, D);
    constexpr int PER = FMT == kFmtNvfp4 ? 2 : 4;     // words of a group
    constexpr int GL = W / PER > 0 ? W / PER : 1;     // groups that this lane touches
    uint32_t sl[GL], sh[GL];
    if constexpr (GL == 2) {
      const uint32_t a = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(scales + key * SB + 2 * t));
      const uint32_t b = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(scales + (key + 8) * SB + 2 * t));
      sl[0] = __byte_perm(a, a, 0x1010), sl[1] = __byte_perm(a, a, 0x3232);
      sh[0] = __byte_perm(b, b, 0x1010), sh[1] = __byte_perm(b, b, 0x3232);
    } else {
      const int g = t * W / PER;
      sl[0] = e4m3x2_to_f16(scales[key * SB + g] * 0x101u);
      sh[0] = e4m3x2_to_f16(scales[(key + 8) * SB + g] * 0x101u);
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint32_t x[4], y[4];
      e2m1x8_to_f16(lo[w], x);
      e2m1x8_to_f16(hi[w], y);
      const uint32_t s0 = sl[GL == 2 ? w / 2 : 0], s1 = sh[GL == 2 ? w / 2 : 0];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = hmul2_u(x[i], s0);
        y[i] = hmul2_u(y[i], s1);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a[4] = {x[2 * h], y[2 * h], x[2 * h + 1], y[2 * h + 1]};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_f16_16816(s[nb], a, qf[nb][4 * w + 2 * h], qf[nb][4 * w + 2 * h + 1]);
      }
    }
  }
}

// O^T += V^T P^T for 16 keys.  w[nb][0..3]: the weights of this lane's score elements (keys of rows r and
// r + 8, columns 2t and 2t + 1).  Scales of keys outside `from` .. `usable` - 1 count as zero (FP4).
// INT4: `sc` holds the fp16 scales of the keys of rows r and r + 8, `down` the power of two that they are
// divided by.
__device__ __forceinline__ float int4_scale(uint32_t two, int g) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(g ? two >> 16 : two & 0xffffu)));
}
template <int FMT, int D, int NB, bool WHOLE>
__device__ __forceinline__ void add_values(const uint8_t* codes, const uint8_t* scales, int r, int t, int from, int usable, const uint32_t (&sc)[2],
                                           float down, const float (&w)[NB][4], float (&o)[NB][D / 16][4]) {
  int key[4];                                         // keys of contraction indices 2t, 2t + 1, 2t + 8, 2t + 9
  key[0] = t, key[1] = 4 + (t ^ 1), key[2] = 8 + t, key[3] = 12 + (t ^ 1);
  if constexpr (FMT == kFmtInt4) {
    // words 8 r' .. of each group of 64: m-tile j of a group has row r = element 8 r + 2j, row r + 8 the next
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      const float s0 = int4_scale(sc[0], g) * down, s1 = int4_scale(sc[1], g) * down;
      uint32_t b[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        b[nb][0] = movmatrix(pack_f16x2(w[nb][0] * s0, w[nb][1] * s0));
        b[nb][1] = movmatrix(pack_f16x2(w[nb][2] * s1, w[nb][3] * s1));
      }
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = *reinterpret_cast<const uint32_t*>(codes + key[i] * (D / 2) + 32 * g + 4 * r);
#pragma unroll
      for (int half = 0; half < 2; ++half) {          // codes 0..3, 4..7 of the words: (key a, key b) pairs
        uint32_t ux[4], uy[4];
        int4x8_to_f16(__byte_perm(c[0], c[1], half ? 0x7632 : 0x5410), ux);
        int4x8_to_f16(__byte_perm(c[2], c[3], half ? 0x7632 : 0x5410), uy);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a[4] = {ux[2 * j], ux[2 * j + 1], uy[2 * j], uy[2 * j + 1]};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_f16_16816(o[nb][4 * g + 2 * half + j], a, b[nb][0], b[nb][1]);
        }
      }
    }
  } else {
    uint32_t b[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      b[nb][0] = movmatrix(pack_f16x2(w[nb][0], w[nb][1]));
      b[nb][1] = movmatrix(pack_f16x2(w[nb][2], w[nb][3]));
    }
    // row r holds D / 8 neighbouring elements from D / 8 * r; m-tile j: row r = element 2j of them, row r + 8 the next
    constexpr int W = D / 64;                         // words per key
    constexpr int SB = kv_scale_bytes(FMT, D);
    const int g = r * (D / 8) / kv_group(FMT);
    uint32_t c[4][W], sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* at = codes + key[i] * (D / 2) + (D / 16) * r;
      if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        c[i][0] = v.x, c[i][1] = v.y;
      } else {
        c[i][0] = *reinterpret_cast<const uint32_t*>(at);
      }
      sc[i] = WHOLE || (key[i] >= from && key[i] < usable) ? scales[key[i] * SB + g] : 0u;
    }
    const uint32_t s01 = e4m3x2_to_f16(sc[0] | (sc[1] << 8)), s23 = e4m3x2_to_f16(sc[2] | (sc[3] << 8));
#pragma unroll
    for (int v = 0; v < W; ++v) {
      // bytes (key a's code, key b's code) of the even and the odd elements
      const uint32_t m = 0x0F0F0F0Fu;
      const uint32_t e01 = bit_select(c[0][v], c[1][v] << 4, m), o01 = bit_select(c[0][v] >> 4, c[1][v], m);
      const uint32_t e23 = bit_select(c[2][v], c[3][v] << 4, m), o23 = bit_select(c[2][v] >> 4, c[3][v], m);
      uint32_t f[4][4];
      e2m1x8_to_f16(e01, f[0]);
      e2m1x8_to_f16(o01, f[1]);
      e2m1x8_to_f16(e23, f[2]);
      e2m1x8_to_f16(o23, f[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a[4] = {hmul2_u(f[0][j], s01), hmul2_u(f[1][j], s01), hmul2_u(f[2][j], s23), hmul2_u(f[3][j], s23)};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_f16_16816(o[nb][4 * v + j], a, b[nb][0], b[nb][1]);
      }
    }
  }
}

// First of the two neighbouring elements of row r (and row r + 8) of accumulator tile j.
template <int FMT, int D>
__device__ __forceinline__ int value_element(int r, int j) {
  if (FMT == kFmtInt4) return 64 * (j / 4) + 8 * r + 2 * (j % 4);
  return (D / 8) * r + 2 * j;
}

// Weights and values of one step: kDecBlocks blocks of 16 keys from `kc`.  WHOLE: every row sees every key.
// `base` is the first key, `have` a bit per block that was loaded, `low` .. `limit` - 1 the keys that count.
template <int FMT, int D, int NB, bool WHOLE>
__device__ __forceinline__ void dec_step(const uint8_t* kc, int r, int t, int base, int have, int low, int limit, const uint32_t (&qf)[NB][D / 8],
                                         const float (&factor)[NB][2], const int (&lo_key)[NB][2], const int (&hi_key)[NB][2],
                                         float (&m)[NB][2], float (&l)[NB][2], float (&o)[NB][D / 16][4], int& vexp) {
  constexpr int SB = kv_scale_bytes(FMT, D);
  const uint8_t* ks = kc + kDecChunk * (D / 2);
  const uint8_t* vc = kc + kDecChunk * (D / 2 + SB);
  const uint8_t* vs = vc + kDecChunk * (D / 2);
  const int kr = key_of_row(r);
  // INT4: the value scales of this lane's keys, and the running power of two that they are divided by, so that
  // the weights times scales, at most 2^14 * 2, fit fp16
  uint32_t sv[kDecBlocks][2];
  if constexpr (FMT == kFmtInt4) {
    uint32_t big = 0u;
#pragma unroll
    for (int u = 0; u < kDecBlocks; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint8_t* at = vs + (16 * u + kr + 8 * k) * SB;
        uint32_t two = D == 128 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
        const int key = base + 16 * u + kr + 8 * k;
        if (!WHOLE && (!((have >> u) & 1) || key < low || key >= limit)) two = 0u;
        sv[u][k] = two;
        big = __vmaxu2(big, two);                     // fp16 of one sign order like integers
      }
    big = max(big & 0xffffu, big >> 16);
    const int e = max(static_cast<int>((__float_as_uint(int4_scale(big, 0)) >> 23) & 255u) - 127, -24);
    if (__any_sync(0xffffffffu, e > vexp)) {
      const int e2 = max(vexp, static_cast<int>(__reduce_max_sync(0xffffffffu, e)));
      const float f = vexp > -100 ? __uint_as_float(static_cast<uint32_t>(vexp - e2 + 127) << 23) : 1.f;   // the sums are 0 at first
      vexp = e2;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nb][d][i] *= f;
    }
  }
  const float down = FMT == kFmtInt4 ? __uint_as_float(static_cast<uint32_t>(127 - vexp) << 23) : 1.f;
  float s[kDecBlocks][NB][4];
#pragma unroll
  for (int u = 0; u < kDecBlocks; ++u) {
    key_scores<FMT, D, NB>(kc + u * 16 * (D / 2), ks + u * 16 * SB, kr, t, qf, s[u]);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!WHOLE) {
          const int key = base + 16 * u + kr + (i & 2 ? 8 : 0);
          const bool see = ((have >> u) & 1) && key < limit && key < hi_key[nb][i & 1] && key >= lo_key[nb][i & 1];
          if (!see) s[u][nb][i] = -INFINITY;
        }
      }
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float top[2];                                       // the factors are positive
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      top[j] = fmaxf(s[0][nb][j], s[0][nb][j + 2]);
#pragma unroll
      for (int u = 1; u < kDecBlocks; ++u) top[j] = fmax3(top[j], s[u][nb][j], s[u][nb][j + 2]);
      top[j] *= factor[nb][j];
    }
    // a lane whose own maximum passes the running one makes the warp look for the new one
    if (__any_sync(0xffffffffu, top[0] > m[nb][0] || top[1] > m[nb][1])) {
      float c2[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], x));
        const float m2 = fmaxf(m[nb][j], top[j]);
        c2[j] = m2 == -INFINITY ? 1.f : ex2(m[nb][j] - m2);
        m[nb][j] = m2;
        l[nb][j] *= c2[j];
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][d][i] *= c2[i & 1];
    }
    const float2 f2 = make_float2(factor[nb][0], factor[nb][1]);
    const float2 b2 = make_float2(m[nb][0] == -INFINITY ? 0.f : dec_shift(FMT) - m[nb][0], m[nb][1] == -INFINITY ? 0.f : dec_shift(FMT) - m[nb][1]);
    float2 sum = make_float2(l[nb][0], l[nb][1]);
#pragma unroll
    for (int u = 0; u < kDecBlocks; ++u)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float2 x = ffma2(make_float2(s[u][nb][i], s[u][nb][i + 1]), f2, b2);
        s[u][nb][i] = ex2(x.x);
        s[u][nb][i + 1] = ex2(x.y);
        sum = fadd2(sum, make_float2(s[u][nb][i], s[u][nb][i + 1]));
      }
    l[nb][0] = sum.x;
    l[nb][1] = sum.y;
  }
#pragma unroll
  for (int u = 0; u < kDecBlocks; ++u) {
    const int usable = WHOLE ? 16 : (((have >> u) & 1) ? limit - base - 16 * u : 0);
    add_values<FMT, D, NB, WHOLE>(vc + u * 16 * (D / 2), vs + u * 16 * SB, r, t, low - base - 16 * u, usable, sv[u], down, s[u], o);
  }
}

// Writes four elements of a finished row, and its lse.  A sum of 0 is a row without keys; one that is NaN stays NaN.
template <int FMT>
__device__ __forceinline__ void write_row(const AttnParams& p, int row0, int h, int row, int d, int D, float4 acc, float top, float sum) {
  const int i = row / p.rep, hq = h * p.rep.d + row - i * p.rep.d;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(p.out + (row0 + i) * p.out_stride + hq * D + d) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse != nullptr && d == 0)
    p.lse[static_cast<long long>(row0 + i) * p.q_heads + hq] = sum == 0.f ? -INFINITY : (top - dec_shift(FMT) + log2f(sum)) * 0.6931471805599453f;
}

template <int FMT, int D, int NB, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == kDecWide ? 1 : 3) kv_attn_decode_kernel(const AttnParams p) {
  constexpr int RT = 8 * NB;
  constexpr int UNIT = kDecChunk * WARPS;
  constexpr int STAGE = dec_stage_bytes(FMT, D);
  constexpr int SB = kv_scale_bytes(FMT, D);
  constexpr int PITCH = D + 4;                        // floats of a row of the joined sums
  static_assert(RT * PITCH * 4 <= kDecStages * STAGE, "a warp's sums fit its ring");
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int warp = static_cast<int>(warp_id()), lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  uint8_t* ring = dec_smem + warp * kDecStages * STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(dec_smem + WARPS * kDecStages * STAGE) + warp * kDecStages;
  int2* loaded = reinterpret_cast<int2*>(dec_smem + WARPS * kDecStages * (STAGE + 8)) + warp * kDecStages;   // blocks, first key
  float* row_max = reinterpret_cast<float*>(dec_smem + WARPS * kDecStages * (STAGE + 16));   // [warps][RT]
  float* row_sum = row_max + WARPS * RT;
  __shared__ Share share;
  __shared__ int last_flag;

  griddep_launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < kDecStages; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  griddep_wait();
  find_share<RT, UNIT, false>(p, reinterpret_cast<long long*>(dec_smem), &share);
  fence_proxy_async_smem();                           // the scan's words lie under the rings
  int count = share.count;
  if (count == 0) return;
  int b = share.b, h = share.h, rt = share.rt, unit = share.unit;
  long long at = share.begin;                         // unit number of the current segment's first unit
  Request req = load_request(p, b);
  uint32_t phase = 0;                                 // bit s: parity of stage s
  bool dead = false;                                  // a wait ran out

  // Pieces of a step that lie in one page are copied by lanes 0 .. pieces - 1.
  const int piece_log2 = min(p.g.page_log2, 6);
  static_assert(kDecChunk == 64, "the copies' steps");
  const int piece = 1 << piece_log2;
  const bool copier = (lane << piece_log2) < kDecChunk;

  while (true) {
    int k0, k1, low;
    tile_keys<RT, UNIT>(p, req, rt, k0, k1, low);
    const int units = max(1, (k1 - k0 + UNIT - 1) / UNIT);
    const int here = min(units - unit, count);
    const int first = k0 + unit * UNIT;           // keys of this segment
    const int limit = here >= units - unit ? k1 : first + here * UNIT;
    const int* table = p.table + b * p.table_stride;
    // The warps take turns along the keys, in an order that does not change from run to run: nor do the sums.
    int key = first + warp * kDecChunk;
    auto claim = [&]() {
      const int c = key < limit ? key : -1;           // first key of the step, or none left
      key += UNIT;
      return c;
    };
    // The page of this lane's piece of the step at `key0`: -1 where no row sees a key of it, or outside the pool.
    auto page_of = [&](int key0) {
      const int key = key0 + (lane << piece_log2);
      int page = -1;
      if (copier && key0 >= 0 && key < limit && key + piece > low) {
        page = table[key >> p.g.page_log2];
        if (page >= p.g.num_pages) page = -2;
        if (page < 0) raise_error(kErrIndex);
      }
      return page;
    };
    auto issue = [&](int st, int key0, int page) {
      const unsigned good = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0) {
        // a bit per piece becomes a bit per 16 keys
        const unsigned spread = piece_log2 == 4 ? good : piece_log2 == 5 ? (good & 1) * 3 + (good >> 1) * 12 : good * 15;
        loaded[st] = make_int2(static_cast<int>(spread), key0);
        mbar_arrive_expect_tx(&bars[st], (__popc(good) << piece_log2) * 2 * (D / 2 + SB));
      }
      __syncwarp();
      if (page >= 0) {
        const int k = lane << piece_log2, off = (key0 + k) & (p.g.page - 1);
        const uint8_t* blk = p.g.pool + kv_block(p.g, page, h);
        uint8_t* dst = ring + st * STAGE;
        if (p.g.page_log2 == 6) {                     // a page of 64 keys lies in the order of a stage
          bulk_load(dst, blk, STAGE, &bars[st]);
          return;
        }
        bulk_load(dst + k * (D / 2), blk + off * (D / 2), piece * (D / 2), &bars[st]);
        bulk_load(dst + kDecChunk * (D / 2) + k * SB, blk + p.g.ks + off * SB, piece * SB, &bars[st]);
        bulk_load(dst + STAGE / 2 + k * (D / 2), blk + p.g.vc + off * (D / 2), piece * (D / 2), &bars[st]);
        bulk_load(dst + STAGE / 2 + kDecChunk * (D / 2) + k * SB, blk + p.g.vs + off * SB, piece * SB, &bars[st]);
      }
    };
    int flying = 0;                                   // stages filled or on their way
    int next = -1;                                    // the step after those
    if (!dead) {
      int keys[kDecStages], pages[kDecStages];
#pragma unroll
      for (int s = 0; s < kDecStages; ++s) {
        keys[s] = s == 0 || keys[s ? s - 1 : 0] >= 0 ? claim() : -1;
        pages[s] = page_of(keys[s]);
      }
#pragma unroll
      for (int s = 0; s < kDecStages; ++s)
        if (keys[s] >= 0) {
          issue(s, keys[s], pages[s]);
          ++flying;
        }
      if (flying == kDecStages) next = claim();
    }

    // this lane's score columns: rows 2t, 2t + 1 of each block
    const int rows = req.n * p.rep.d;
    uint32_t qf[NB][D / 8];
    float factor[NB][2];
    int lo_key[NB][2], hi_key[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = rt * RT + nb * 8 + r;
      const bool live = row < rows;
      const int i = live ? row / p.rep : 0, hq = h * p.rep.d + (live ? row - i * p.rep.d : 0);
      float f;
      load_queries<FMT, D>(p.q + (req.row0 + i) * p.q_stride + hq * D, live, t, p.scale < 0.f, qf[nb], f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        factor[nb][j] = fmaxf(__shfl_sync(0xffffffffu, f, (2 * t + j) * 4) * (fabsf(p.scale) * 1.4426950408889634f), 1.17549435e-38f);
        const int pos = req.kv - req.n + min(rt * RT + nb * 8 + 2 * t + j, rows - 1) / p.rep;
        hi_key[nb][j] = p.causal ? min(req.kv, pos + 1) : req.kv;
        lo_key[nb][j] = p.window > 0 ? pos - p.window + 1 : 0;
      }
    }
    // keys that every row of the tile sees
    const int all_hi = min(limit, p.causal ? req.kv - req.n + (rt * RT) / p.rep + 1 : req.kv);
    const int all_lo = p.window > 0 ? req.kv - req.n + (min((rt + 1) * RT, rows) - 1) / p.rep - p.window + 1 : 0;

    float m[NB][2], l[NB][2], o[NB][D / 16][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nb][j] = -INFINITY;
        l[nb][j] = 0.f;
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][d][i] = 0.f;
    }

    int st = 0, vexp = -1000;
    while (flying > 0) {
      const int page = page_of(next);                 // looked up a step ahead of its copy
      if (!warp_wait(&bars[st], (phase >> st) & 1, p.budget, nullptr)) {
        if (lane == 0) raise_error(kErrWaitAttn);
        dead = true;                                  // copies in flight land before the ring is given up
        for (; flying > 0; --flying) {
          warp_wait(&bars[st], (phase >> st) & 1, drain_budget(p.budget), nullptr);
          phase ^= 1u << st;
          st = st + 1 == kDecStages ? 0 : st + 1;
        }
        break;
      }
      const uint8_t* kc = ring + st * STAGE;
      const int have = loaded[st].x, base = loaded[st].y;
      if (have == (1 << kDecBlocks) - 1 && base >= all_lo && base + kDecChunk <= all_hi)
        dec_step<FMT, D, NB, true>(kc, r, t, base, have, low, limit, qf, factor, lo_key, hi_key, m, l, o, vexp);
      else
        dec_step<FMT, D, NB, false>(kc, r, t, base, have, low, limit, qf, factor, lo_key, hi_key, m, l, o, vexp);
      phase ^= 1u << st;
      --flying;
      __syncwarp();                                   // every lane has left the stage
      if (next >= 0) {
        issue(st, next, page);
        ++flying;
        next = claim();
      }
      st = st + 1 == kDecStages ? 0 : st + 1;
    }

    // ------------------------------------------------ join the warps of the CTA
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], x);
        if (r == 0) {
          row_max[warp * RT + nb * 8 + 2 * t + j] = m[nb][j];
          row_sum[warp * RT + nb * 8 + 2 * t + j] = l[nb][j];
        }
      }
    __syncthreads();                                  // every warp has left its ring, too
    float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = nb * 8 + 2 * t + j;
        float top = row_max[row];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) top = fmaxf(top, row_max[w * RT + row]);
        float c = m[nb][j] == -INFINITY ? 0.f : ex2(m[nb][j] - top);
        if (FMT == kFmtInt4) c *= __uint_as_float(static_cast<uint32_t>(max(vexp, -24) + 127) << 23);
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
          *reinterpret_cast<float2*>(sums + row * PITCH + value_element<FMT, D>(r, d)) =
              make_float2(o[nb][d][j] * c, o[nb][d][j + 2] * c);
      }
    __syncthreads();
    const int live_rows = min(RT, rows - rt * RT);
    const bool split = unit > 0 || here < units;
    constexpr int Q = D / 4;
    constexpr int SLOT = RT * (D + 2);
    const float* all = reinterpret_cast<const float*>(dec_smem);
    constexpr int kWarpFloats = kDecStages * STAGE / 4;
    float* slot = p.partials + (2ll * blockIdx.x + (unit == 0 ? 1 : 0)) * SLOT;
    for (int e = threadIdx.x; e < live_rows * Q; e += (32 * WARPS)) {
      const int row = e / Q, d = e % Q * 4;
      float top = row_max[row];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) top = fmaxf(top, row_max[w * RT + row]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float mw = row_max[w * RT + row];
        sum += row_sum[w * RT + row] * (mw == -INFINITY ? 0.f : ex2(mw - top));
        const float4 v = *reinterpret_cast<const float4*>(all + w * kWarpFloats + row * PITCH + d);
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      }
      if (!split) {
        write_row<FMT>(p, req.row0, h, rt * RT + row, d, D, acc, top, sum);
      } else {
        __stcg(reinterpret_cast<float4*>(slot + row * D + d), acc);
        if (d == 0) __stcg(reinterpret_cast<float2*>(slot + RT * D + 2 * row), make_float2(top, sum));
      }
    }
    if (split) {
      const long long item = at - unit;               // unit number of the item's first unit
      int c0, c1;
      item_parts(share, item, units, c0, c1);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        last_flag = arrive_last(&p.counters[c0], p.nonce, c1 - c0 + 1);
        __threadfence();
      }
      __syncthreads();
      if (last_flag) {
        const float* part0 = p.partials + (2ll * c0 + 1) * SLOT;
        for (int e = threadIdx.x; e < live_rows * Q; e += (32 * WARPS)) {
          const int row = e / Q, d = e % Q * 4;
          float top = -INFINITY, sum = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const float* sl = c == c0 ? part0 : p.partials + 2ll * c * SLOT;
            const float2 ms = __ldcg(reinterpret_cast<const float2*>(sl + RT * D + 2 * row));
            const float4 v = __ldcg(reinterpret_cast<const float4*>(sl + row * D + d));
            const float m2 = fmaxf(top, ms.x);
            const float f0 = m2 == -INFINITY ? 0.f : ex2(top - m2), f1 = m2 == -INFINITY ? 0.f : ex2(ms.x - m2);
            sum = sum * f0 + ms.y * f1;
            acc.x = acc.x * f0 + v.x * f1, acc.y = acc.y * f0 + v.y * f1;
            acc.z = acc.z * f0 + v.z * f1, acc.w = acc.w * f0 + v.w * f1;
            top = m2;
          }
          write_row<FMT>(p, req.row0, h, rt * RT + row, d, D, acc, top, sum);
        }
      }
    }

    // ------------------------------------------------ the next item of the share
    count -= here;
    at += here;
    if (count <= 0) break;
    __syncthreads();                                  // the sums have been read: the rings may be filled again
    fence_proxy_async_smem();
    unit = 0;
    if (++rt >= row_tiles<RT>(p, req)) {
      rt = 0;
      if (++h >= p.g.heads) {
        h = 0;
        do {
          if (++b >= p.batch) return;                 // not reached: the share ends inside the batch
          req = load_request(p, b);
        } while (req.n == 0);
      }
    }
  }
}

}  // namespace svdq
