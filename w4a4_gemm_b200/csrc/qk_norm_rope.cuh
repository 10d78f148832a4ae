// qk_norm_rope.cuh -- RMS norm of every query and key head and the rotation of
// their leading `rot` elements by the row's position, in one pass over the rows
// that the QKV projection writes.
//
//   y = x * rsqrt(mean(x^2) + eps) * w
//   (a, b) -> (a cos - b sin, b cos + a sin)
//   pairs: (2i, 2i + 1) interleaved, else (i, i + rot / 2), i < rot / 2
//
// fp32 from the load to the one rounding to bf16 at the store.
// A head belongs to L = 4, 8, 16 or 32 neighbouring lanes (8 elements = 16 bytes
// each), so a warp's loads and stores are whole lines, the mean is log2(L)
// shuffles, and the half-split partner of an element sits in another lane at the
// same place.  A lane group keeps its cosines, sines and weights in registers
// over the heads of a row that it walks.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "svdq_formats.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

constexpr int kNormThreads = 128;

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
  int lanes_log2;                  // log2 of the lanes of a head
  int chunk;                       // heads that a lane group walks
  int chunks;                      // lane groups per row
};

__device__ __forceinline__ void bf16x8_to_f32(const uint4& a, float* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_kernel(const NormRopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int L = 1 << p.lanes_log2;
  const long long group = (static_cast<long long>(blockIdx.x) * kNormThreads + threadIdx.x) >> p.lanes_log2;
  const int l = threadIdx.x & (L - 1);
  const long long row = group / p.chunks;
  const int h0 = static_cast<int>(group % p.chunks) * p.chunk;
  const int heads = p.q_heads + p.k_heads;
  // A padded row (position below 0) is left as it is; every lane stays for the shuffles.
  bool ok = row < p.rows;
  long long pos = row;
  if (ok && p.positions != nullptr) pos = p.positions[row];
  if (ok && pos >= p.table_rows && p.rot > 0) {
    if (l == 0) raise_error(kErrIndex);
    ok = false;
  }
  if (pos < 0) ok = false;
  const bool mine = ok && 8 * l < p.D;

  const int half = p.rot / 2;
  const bool rotated = 8 * l < p.rot;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (mine && rotated) {
    const float* t = p.table + pos * p.rot;
    if (p.interleaved) {                     // 4 pairs of this lane
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[2 * i] = cs[2 * i + 1] = __ldg(t + 4 * l + i);
        const float s = __ldg(t + half + 4 * l + i);
        sn[2 * i] = -s;
        sn[2 * i + 1] = s;
      }
    } else {                                 // 8 pairs, their other halves in the partner lane
      const int i0 = (8 * l) % half;
      const bool second = 8 * l >= half;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = __ldg(t + i0 + i);
        const float s = __ldg(t + half + i0 + i);
        sn[i] = second ? s : -s;
      }
    }
  }
  const int partner = (rotated && !p.interleaved) ? (8 * l < half ? l + half / 8 : l - half / 8) : l;
  const float inv_d = 1.f / static_cast<float>(p.D);

  for (int j = 0; j < p.chunk; ++j) {
    const int h = h0 + j;
    const bool is_q = h < p.q_heads;
    const int hh = is_q ? h : h - p.q_heads;
    const bool act = mine && h < heads;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (act) {
      const __nv_bfloat16* src = (is_q ? p.q + row * p.q_stride : p.k + row * p.k_stride) + hh * p.D + 8 * l;
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(src), x);
    }
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      for (int o = 1; o < L; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss * inv_d + p.eps);
      const __nv_bfloat16* w = is_q ? p.q_weight : p.k_weight;
      float wf[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) wf[i] = 1.f;
      if (act && w != nullptr) bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(w + 8 * l)), wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * wf[i];
    }
    float y[8];
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner, L);
    }
    if (act) {
      if (rotated) {                         // the others keep their values, infinities included
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(y[i], sn[i], x[i] * cs[i]);
      }
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      __nv_bfloat16* dst = (is_q ? p.q_out + row * p.q_out_stride : p.k_out + row * p.k_out_stride) + hh * p.D + 8 * l;
      *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace svdq
