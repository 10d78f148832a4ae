// qk_norm_rope.cuh -- RMS norm of every query and key head and the rotation of
// their leading `rot` elements by the row's position, in one pass over the rows
// that the QKV projection writes.
//
//   y = x * rsqrt(mean(x^2) + eps) * w
//   (a, b) -> (a cos - b sin, b cos + a sin)
//   pairs: (2i, 2i + 1) interleaved, else (i, i + rot / 2), i < rot / 2
//
// fp32 from the load to the one rounding to bf16 at the store.
// A head belongs to L = 2 to 32 neighbouring lanes (8 elements = 16 bytes each; L is the
// power of two that holds them, the lanes past D / 8 idle), so a warp's loads and stores are whole lines, the mean is log2(L)
// shuffles, and the half-split partner of an element sits in another lane at the
// same place.  A lane group keeps its cosines, sines and weights in registers
// over the heads of a row that it walks.
// HBM bounds it at many rows (2 bytes in and out per element): 16383 rows of 40 heads
// of 128, 69 us, 4.9 TB/s; 4608 rows of 48 heads, 21.7 us, 5.3 TB/s; the launch at
// few: 16 rows 2.0 us.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "kv_common.cuh"
#include "svdq_formats.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

constexpr int kNormThreads = 128;
constexpr int kNormBatch = 4;

struct NormRopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;   // elements between rows
  const __nv_bfloat16* q_weight;   // D, or null: ones
  const __nv_bfloat16* k_weight;
  const float* table;              // [table_rows][rot]: rot / 2 cosines, rot / 2 sines
  const int* positions;            // null: the row's own number
  int table_rows;
  int rows, q_heads, k_heads, D, rot;
  int norm, interleaved;
  float eps;
  int chunk;                       // heads that a lane group walks
  int chunks;                      // lane groups per row
};

__device__ __forceinline__ void bf16x8_to_f32(const uint4& a, float2* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
}

// out = r (x A + x' B): x' the partner of x in its pair, A = w cos, B = -+ w' sin, r the head's 1 / rms.
// A and B do not depend on the head, only on the row and on whether it is a query or a key.  The next BATCH heads
// are on their way while a batch is worked on, the first ones before the row's position is known.
template <int LANES, bool INTERLEAVED, int BATCH>
__global__ void __launch_bounds__(kNormThreads, 4) qk_norm_rope_kernel(const NormRopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int group = static_cast<int>(blockIdx.x * kNormThreads + threadIdx.x) / LANES;
  const int l = threadIdx.x & (LANES - 1);
  const int row = group / p.chunks;
  const int h0 = (group - row * p.chunks) * p.chunk, h1 = min(h0 + p.chunk, p.q_heads + p.k_heads);
  const bool there = row < p.rows && 8 * l < p.D;
  const __nv_bfloat16* qrow = p.q + row * p.q_stride + 8 * l;
  const __nv_bfloat16* krow = p.k + row * p.k_stride - static_cast<long long>(p.q_heads) * p.D + 8 * l;   // as if the keys followed the queries
  uint4 ahead[BATCH];
  auto load = [&](int h) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
      ahead[b] = there && h + b < h1 ? *reinterpret_cast<const uint4*>((h + b < p.q_heads ? qrow : krow) + (h + b) * p.D) : make_uint4(0u, 0u, 0u, 0u);
  };
  load(h0);
  // A padded row (position below 0) is left as it is; every lane stays for the shuffles.
  bool mine = there;
  int pos = row;
  if (row < p.rows && p.positions != nullptr) pos = p.positions[row];
  if (row < p.rows && pos >= p.table_rows && p.rot > 0) {
    if (l == 0) raise_error(kErrIndex);
    mine = false;
  }
  if (pos < 0) mine = false;

  const int half = p.rot / 2;
  const bool rotated = 8 * l < p.rot;
  const int partner = (rotated && !INTERLEAVED) ? (8 * l < half ? l + half / 8 : l - half / 8) : l;
  float2 cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = make_float2(1.f, 1.f);
    sn[i] = make_float2(0.f, 0.f);
  }
  if (mine && rotated) {
    const float* t = p.table + static_cast<long long>(pos) * p.rot;
    if (INTERLEAVED) {                       // 4 pairs of this lane
      const float4 c = __ldg(reinterpret_cast<const float4*>(t + 4 * l)), s = __ldg(reinterpret_cast<const float4*>(t + half + 4 * l));
      const float cc[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = make_float2(cc[i], cc[i]);
        sn[i] = make_float2(-s4[i], s4[i]);
      }
    } else {                                 // 8 pairs, their other halves in the partner lane
      const bool second = 8 * l >= half;
      const float* t0 = t + 8 * l - (second ? half : 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(t0 + 4 * i)), s = __ldg(reinterpret_cast<const float4*>(t0 + half + 4 * i));
        cs[2 * i] = make_float2(c.x, c.y);
        cs[2 * i + 1] = make_float2(c.z, c.w);
        sn[2 * i] = second ? make_float2(s.x, s.y) : make_float2(-s.x, -s.y);
        sn[2 * i + 1] = second ? make_float2(s.z, s.w) : make_float2(-s.z, -s.w);
      }
    }
  }
  const float inv_d = 1.f / static_cast<float>(p.D);
  __nv_bfloat16* qout = p.q_out + row * p.q_out_stride + 8 * l;
  __nv_bfloat16* kout = p.k_out + row * p.k_out_stride - static_cast<long long>(p.q_heads) * p.D + 8 * l;
  float2 A[4], B[4];
  int kind = -1;                             // of A and B: 0 queries, 1 keys
  for (int j = 0; j < p.chunk; j += BATCH) { // the same count for every lane of a warp
    uint4 raw[BATCH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) raw[b] = ahead[b];
    if (j + BATCH < p.chunk) load(h0 + j + BATCH);
    float ss[BATCH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      float2 x[4];
      bf16x8_to_f32(raw[b], x);
      float2 s2 = fmul2_rn(x[0], x[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) s2 = ffma2(x[i], x[i], s2);
      ss[b] = s2.x + s2.y;
    }
#pragma unroll
    for (int o = 1; o < LANES; o *= 2)
#pragma unroll
      for (int b = 0; b < BATCH; ++b) ss[b] += __shfl_xor_sync(0xffffffffu, ss[b], o);
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int h = h0 + j + b;
      if (kind != (h < p.q_heads ? 0 : 1)) {
        kind = h < p.q_heads ? 0 : 1;
        const __nv_bfloat16* w = kind == 0 ? p.q_weight : p.k_weight;
#pragma unroll
        for (int i = 0; i < 4; ++i) A[i] = B[i] = make_float2(1.f, 1.f);
        if (p.norm && w != nullptr && mine) {
          bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(w + 8 * l)), A);
          bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(w + 8 * partner)), B);
          if (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) B[i] = make_float2(B[i].y, B[i].x);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          A[i] = fmul2_rn(A[i], cs[i]);
          B[i] = fmul2_rn(B[i], sn[i]);
        }
      }
      uint4 other;
      if (INTERLEAVED) {
        other = make_uint4(__byte_perm(raw[b].x, 0, 0x1032), __byte_perm(raw[b].y, 0, 0x1032), __byte_perm(raw[b].z, 0, 0x1032),
                           __byte_perm(raw[b].w, 0, 0x1032));
      } else {
        other.x = __shfl_sync(0xffffffffu, raw[b].x, partner, LANES);
        other.y = __shfl_sync(0xffffffffu, raw[b].y, partner, LANES);
        other.z = __shfl_sync(0xffffffffu, raw[b].z, partner, LANES);
        other.w = __shfl_sync(0xffffffffu, raw[b].w, partner, LANES);
      }
      if (!rotated) other = make_uint4(0u, 0u, 0u, 0u);     // those elements keep their values, infinities included
      const float r = p.norm ? rsqrtf(ss[b] * inv_d + p.eps) : 1.f;
      const float2 r2 = make_float2(r, r);
      float2 x[4], y[4];
      bf16x8_to_f32(raw[b], x);
      bf16x8_to_f32(other, y);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = fmul2_rn(ffma2(x[i], A[i], fmul2_rn(y[i], B[i])), r2);
        o[i] = pack_bf16x2(t.x, t.y);
      }
      if (mine && h < h1) *reinterpret_cast<uint4*>((kind == 0 ? qout : kout) + h * p.D) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace svdq
