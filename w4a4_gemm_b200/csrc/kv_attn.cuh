// kv_attn.cuh -- attention over the paged 4-bit cache:
//
//   o_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(scale q_i . k_t - max),
//   lse_i = log sum_t exp(scale q_i . k_t)
//
// over the keys t that query i sees: t < kv_len, with `causal` t <= pos_i, with a
// window t > pos_i - window, where pos_i = kv_len - q_len + i.  A query that sees
// no key gives o = 0 and lse = -inf.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv_cache.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

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
  int causal, window;
  float scale;
};

// One warp per (row, query head), D / 32 neighbouring elements per lane, one key at a time.
template <int FMT, int D>
__global__ void __launch_bounds__(128) kv_attn_rows_kernel(const AttnParams p) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int row = static_cast<int>(unit / p.q_heads), h = static_cast<int>(unit % p.q_heads);
  if (row >= p.rows) return;
  int lo = 0, hi = p.batch;
  if (row < p.cu_q[0] || row >= p.cu_q[p.batch]) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid] <= row) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int n = p.cu_q[b + 1] - p.cu_q[b];
  long long kv = p.kv_lens[b];
  if (kv < 0 || kv > static_cast<long long>(p.width) * p.g.page) {
    if (lane == 0) raise_error(kErrIndex);
    kv = kv < 0 ? 0 : static_cast<long long>(p.width) * p.g.page;
  }
  const long long pos = kv - n + (row - p.cu_q[b]);
  const long long end = p.causal ? (pos + 1 < kv ? pos + 1 : kv) : kv;
  long long begin = p.window > 0 ? pos - p.window + 1 : 0;
  if (begin < 0) begin = 0;
  const int kvh = h / (p.q_heads / p.g.heads);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[row * p.q_stride + h * D + lane * E + e]) * p.scale;
    o[e] = 0.f;
  }
  for (long long t = begin; t < end; ++t) {
    const int page = p.table[b * p.table_stride + (t >> p.g.page_log2)];
    if (page < 0 || page >= p.g.num_pages) {
      if (lane == 0) raise_error(kErrIndex);
      continue;
    }
    const int off = static_cast<int>(t & (p.g.page - 1));
    const uint8_t* blk = p.g.pool + kv_block(p.g, page, kvh);
    float kvv[2][E];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint8_t* at = blk + (side ? p.g.vc : 0);
      const uint8_t* sc = at + p.g.ks + off * kv_scale_bytes(FMT, D);
      const int grp = lane * E / kv_group(FMT);
      float s;
      if (FMT == kFmtInt4)
        s = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(sc + 2 * grp)));
      else
        s = e4m3_value(sc[grp]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t byte = at[off * (D / 2) + (lane * E + e) / 2];
        const uint32_t nib = (e & 1) ? byte >> 4 : byte & 15u;
        kvv[side][e] = s * (FMT == kFmtInt4 ? static_cast<float>(static_cast<int>(nib << 28) >> 28) : e2m1_value(nib));
      }
    }
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) d = fmaf(q[e], kvv[0][e], d);
#pragma unroll
    for (int x = 16; x > 0; x /= 2) d += __shfl_xor_sync(0xffffffffu, d, x);
    const float m2 = fmaxf(m, d);
    const float c = expf(m - m2), w = expf(d - m2);
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, kvv[1][e], o[e] * c);
    m = m2;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out[row * p.out_stride + h * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
  if (p.lse != nullptr && lane == 0) p.lse[static_cast<long long>(row) * p.q_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace svdq
