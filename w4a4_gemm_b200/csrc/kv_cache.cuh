// kv_cache.cuh -- geometry of the paged 4-bit key/value cache and the kernels
// that write it (quantize and append) and read it back.
//
// Pool: [num_pages][kv_heads] blocks of `head_bytes` bytes, each
//   key codes   [page][D / 2]    element 2i in the low nibble of byte i
//   key scales  [page][D / g]    E4M3 bytes (g = 16, 32) or fp16 (g = 64)
//   value codes [page][D / 2]
//   value scales[page][D / g]
// so that the tokens of one head and page are contiguous: a run of tokens of a
// page is four contiguous pieces, each a multiple of 16 bytes for every 16
// tokens (D = 64 or 128), which is what bulk copies want.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv_common.cuh"
#include "svdq_formats.cuh"
#include "svdq_ptx.cuh"

namespace svdq {

constexpr int kFmtNvfp4 = 0, kFmtInt4 = 1, kFmtFp4g32 = 2;

__host__ __device__ constexpr int kv_group(int fmt) { return fmt == kFmtNvfp4 ? 16 : (fmt == kFmtInt4 ? 64 : 32); }
// bytes of the scales of one head's key (or value) of one token
__host__ __device__ constexpr int kv_scale_bytes(int fmt, int D) {
  return D / kv_group(fmt) * (fmt == kFmtInt4 ? 2 : 1);
}

struct KvGeom {
  uint8_t* pool;
  long long num_pages;
  int heads, D, page, page_log2;
  int ks, vc, vs;         // byte offsets inside a block: key scales, value codes, value scales
  int head_bytes;
};

// Byte offset of block (page, head).  64-bit: a long cache passes 2^32 bytes.
__device__ __forceinline__ size_t kv_block(const KvGeom& g, long long page, int head) {
  return (static_cast<size_t>(page) * g.heads + head) * static_cast<size_t>(g.head_bytes);
}

// 8 bf16 (a 16-byte word) -> fp32
__device__ __forceinline__ void bf16x8_to_floats(const uint4& a, float* v) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// ------------------------------------------------------------------ append ---
// A thread quantizes pieces of 8 values (16 bytes of one head's row, 4 code
// bytes), so that a warp's loads and stores are whole lines; the 16, 32 or 64 values
// of a scale meet their maximum over 2, 4 or 8 neighbouring lanes.  The quantizer is
// the activation kernel's, decision for decision:
// scale = rounded amax / q_max, code = round(v * RN(1 / scale)).
// Bound by HBM at many rows (2 D bytes in, D / 2 + scales out, per head and
// side) and by the launch at few: 8191 rows of 8 heads of 128 take 14.5 us to append in
// INT4 and 12.3 in the FP4 formats (6.5 by their bytes), and to read 10.4 us as bf16 and
// 17.0 as fp32 in INT4, 21.2 and 27.1 in the FP4 formats (6.5 and 11.7), whose codes the read
// decodes by their bit fields; 64 rows 1.8 and 2.0 us.  With 16 values a thread, whose
// stores interleave, and the row found per piece append and read of INT4 took 34.4 us.  A slot below 0 is a padded row and is
// skipped; one at or past the pool's end is skipped and raises kErrIndex.
// UNITS pieces per thread, a CTA's threads apart: their loads are issued together.
constexpr int kAppendThreads = 256;
constexpr int kAppendUnits = 4;

// A row has 2 heads D / VALUES pieces (keys, then values).  A thread has the same piece in UNITS rows, `step` rows
// apart: a CTA covers 256 pieces of a row (blockIdx.y says which), or several whole rows where a row has fewer, and
// only the slot differs from one unit to the next.
struct Piece {
  int row, step;                 // first row, and the rows between units; row < 0: none
  int side, head, part;          // 0 keys, 1 values; the head; which piece of its values
};
template <int VALUES, int UNITS>
__device__ __forceinline__ Piece piece_of_thread(const KvGeom& g) {
  const int per_head = g.D / VALUES, per_row = 2 * g.heads * per_head;
  Piece p;
  int at = threadIdx.x, sub = 0;
  p.step = 1;
  if (per_row < kAppendThreads) {
    p.step = kAppendThreads / per_row;
    sub = at / per_row;
    at -= sub * per_row;
  } else {
    at += blockIdx.y * kAppendThreads;
  }
  p.row = sub < p.step && at < per_row ? static_cast<int>(blockIdx.x) * p.step * UNITS + sub : -1;
  const int head2 = at / per_head;
  p.part = at - head2 * per_head;
  p.side = head2 >= g.heads;
  p.head = p.side ? head2 - g.heads : head2;
  return p;
}

template <int FMT, int UNITS>
__global__ void __launch_bounds__(kAppendThreads)
    kv_append_kernel(const KvGeom g, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                     long long k_stride, long long v_stride, const long long* __restrict__ slots, int M) {
  griddep_launch_dependents();
  griddep_wait();
  const Piece pc = piece_of_thread<8, UNITS>(g);
  // the lanes that share a group have their rows in common: they are in or out together
  const __nv_bfloat16* src = (pc.side ? v : k) + pc.head * g.D + pc.part * 8;
  const long long stride = pc.side ? v_stride : k_stride;
  uint4 raw[UNITS];
  long long slot[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int row = pc.row + u * pc.step;
    slot[u] = -1;
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    if (pc.row >= 0 && row < M) {
      raw[u] = __ldg(reinterpret_cast<const uint4*>(src + row * stride));
      slot[u] = slots[row];
    }
  }
  const size_t page_bytes = static_cast<size_t>(g.heads) * g.head_bytes;
  uint8_t* base = g.pool + static_cast<size_t>(pc.head) * g.head_bytes + (pc.side ? g.vc : 0);
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const bool past = slot[u] >= g.num_pages * g.page;
    if (past && pc.part == 0 && pc.head == 0) raise_error(kErrIndex);
    float x[8];
    bf16x8_to_floats(raw[u], x);
    float amax = fmax3(fmax3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])), fmax3(fabsf(x[3]), fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7])));
    amax = fminf(fmaxf(amax, 0.f), 3.402823466e+38f);  // not infinite: a NaN scale would reach rows that mask the key
    constexpr int kLanes = kv_group(FMT) / 8;          // lanes that share a scale
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    uint32_t codes = 0u;
    uint32_t scale;
    if (FMT == kFmtInt4) {
      scale = int4_scale_bits(amax);
      const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(scale)));
      const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) codes |= (static_cast<uint32_t>(int4_code(x[i], inv)) & 15u) << (4 * i);
    } else {
      scale = e4m3_code(div6_rn(amax));
      if (scale != 0u) {
        const float inv = __frcp_rn(e4m3_value(scale));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], inv);
        codes = e2m1_pack8(x);
      }
    }
    if (slot[u] >= 0 && !past) {
      const int off = static_cast<int>(slot[u] & (g.page - 1));
      uint8_t* blk = base + static_cast<size_t>(slot[u] >> g.page_log2) * page_bytes;
      *reinterpret_cast<uint32_t*>(blk + off * (g.D / 2) + pc.part * 4) = codes;
      uint8_t* sc = blk + g.ks + off * kv_scale_bytes(FMT, g.D);
      if (pc.part % kLanes == 0) {
        if (FMT == kFmtInt4)
          *reinterpret_cast<uint16_t*>(sc + pc.part / kLanes * 2) = static_cast<uint16_t>(scale);
        else
          sc[pc.part / kLanes] = static_cast<uint8_t>(scale);
      }
    }
  }
}

// -------------------------------------------------------------------- read ---
// A thread reads the codes of 16 output bytes (4 fp32 or 8 bf16 values) and
// their scale and writes the values they stand for: code * scale, exact in fp32 (at
// most 3 + 11 bits) and, for the E2M1 formats (2 + 4 bits), in bf16; INT4 in bf16 is
// rounded once.  A row with a slot below 0 or past the end is written as zeros.
template <int FMT, typename Out, int UNITS>
__global__ void __launch_bounds__(kAppendThreads)
    kv_read_kernel(const KvGeom g, const long long* __restrict__ slots, int M, Out* __restrict__ k,
                   Out* __restrict__ v) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int VALUES = 16 / sizeof(Out);
  const Piece pc = piece_of_thread<VALUES, UNITS>(g);
  long long slot[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int row = pc.row + u * pc.step;
    slot[u] = pc.row >= 0 && row < M ? slots[row] : -1;
  }
  const size_t page_bytes = static_cast<size_t>(g.heads) * g.head_bytes;
  const uint8_t* base = g.pool + static_cast<size_t>(pc.head) * g.head_bytes + (pc.side ? g.vc : 0);
  uint32_t c[UNITS];
  float s[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const bool past = slot[u] >= g.num_pages * g.page;
    if (past && pc.part == 0 && pc.head == 0) raise_error(kErrIndex);
    c[u] = 0u;
    s[u] = 0.f;
    if (slot[u] >= 0 && !past) {
      const int off = static_cast<int>(slot[u] & (g.page - 1));
      const uint8_t* blk = base + static_cast<size_t>(slot[u] >> g.page_log2) * page_bytes;
      const uint8_t* at = blk + off * (g.D / 2) + pc.part * (VALUES / 2);
      c[u] = VALUES == 8 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
      const uint8_t* sc = blk + g.ks + off * kv_scale_bytes(FMT, g.D);
      const int group = pc.part * VALUES / kv_group(FMT);
      if (FMT == kFmtInt4)
        s[u] = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(sc + group * 2)));
      else
        s[u] = e4m3_value(sc[group]);
    }
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int row = pc.row + u * pc.step;
    if (pc.row < 0 || row >= M) break;
    float x[VALUES];
#pragma unroll
    for (int i = 0; i < VALUES; ++i) {
      const uint32_t nib = (c[u] >> (4 * i)) & 15u;
      const float val = FMT == kFmtInt4 ? static_cast<float>(static_cast<int>(nib << 28) >> 28) : e2m1_value(nib);
      x[i] = __fmul_rn(val, s[u]);
    }
    Out* dst = (pc.side ? v : k) + (static_cast<long long>(row) * g.heads + pc.head) * g.D + pc.part * VALUES;
    if constexpr (VALUES == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

}  // namespace svdq
