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

// 16 bf16 (two 16-byte words) -> fp32
__device__ __forceinline__ void bf16x16_to_f32(const uint4& a, const uint4& b, float* v) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// ------------------------------------------------------------------ append ---
// One thread quantizes 16 values (32 bytes of one head's row, 8 code bytes); a
// group of 32 or 64 meets its maximum over 2 or 4 neighbouring lanes.  The
// quantizer is the activation kernel's, decision for decision:
// scale = rounded amax / q_max, code = round(v * RN(1 / scale)).
// Bound by HBM at many rows (2 D bytes in, D / 2 + scales out, per head and
// side) and by the launch at few.  A slot below 0 is a padded row and is
// skipped; one at or past the pool's end is skipped and raises kErrIndex.
constexpr int kAppendThreads = 256;

template <int FMT>
__global__ void __launch_bounds__(kAppendThreads)
    kv_append_kernel(const KvGeom g, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                     long long k_stride, long long v_stride, const long long* __restrict__ slots, int M) {
  griddep_launch_dependents();
  griddep_wait();
  const int per_head = g.D / 16;                       // threads of one head's row: 4 or 8
  const long long n = static_cast<long long>(M) * 2 * g.heads * per_head;
  const long long idx = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x;
  // n is a multiple of 4 or 8 threads, so the lanes that share a group leave together
  const bool live = idx < n;
  const int part = static_cast<int>(idx % per_head);
  const long long hr = idx / per_head;
  const int head2 = static_cast<int>(hr % (2 * g.heads));
  const long long row = hr / (2 * g.heads);
  const int side = head2 >= g.heads;                   // 0 keys, 1 values
  const int head = side ? head2 - g.heads : head2;
  const long long slot = live ? slots[row] : -1;
  const bool past = slot >= g.num_pages * g.page;
  const bool ok = slot >= 0 && !past;
  if (past && part == 0 && head2 == 0) raise_error(kErrIndex);
  float x[16];
  if (ok) {
    const __nv_bfloat16* src = (side ? v + row * v_stride : k + row * k_stride) + head * g.D + part * 16;
    const uint4* s4 = reinterpret_cast<const uint4*>(src);
    bf16x16_to_f32(__ldg(s4), __ldg(s4 + 1), x);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  }
  float amax = absmax16(x);
  constexpr int kLanes = kv_group(FMT) / 16;           // lanes that share a scale
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!ok) return;
  uint32_t codes[2] = {0u, 0u};
  uint32_t scale;
  if (FMT == kFmtInt4) {
    scale = int4_scale_bits(amax);
    const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(scale)));
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) codes[i / 8] |= (static_cast<uint32_t>(int4_code(x[i], inv)) & 15u) << (4 * (i % 8));
  } else {
    scale = e4m3_code(div6_rn(amax));
    if (scale != 0u) {
      const float inv = __frcp_rn(e4m3_value(scale));
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], inv);
      codes[0] = e2m1_pack8(x);
      codes[1] = e2m1_pack8(x + 8);
    }
  }
  const long long page = slot >> g.page_log2;
  const int off = static_cast<int>(slot & (g.page - 1));
  uint8_t* blk = g.pool + kv_block(g, page, head) + (side ? g.vc : 0);
  *reinterpret_cast<uint2*>(blk + off * (g.D / 2) + part * 8) = make_uint2(codes[0], codes[1]);
  uint8_t* sc = blk + g.ks + off * kv_scale_bytes(FMT, g.D);
  if (part % kLanes == 0) {
    if (FMT == kFmtInt4)
      *reinterpret_cast<uint16_t*>(sc + part / kLanes * 2) = static_cast<uint16_t>(scale);
    else
      sc[part / kLanes] = static_cast<uint8_t>(scale);
  }
}

// -------------------------------------------------------------------- read ---
// One thread reads 16 codes (8 bytes) and their scale and writes the values
// they stand for: code * scale, exact in fp32 (at most 3 + 11 bits) and, for
// the E2M1 formats (2 + 4 bits), in bf16; INT4 in bf16 is rounded once.
// A row with a slot below 0 or past the end is written as zeros.
template <int FMT, typename Out>
__global__ void __launch_bounds__(kAppendThreads)
    kv_read_kernel(const KvGeom g, const long long* __restrict__ slots, int M, Out* __restrict__ k,
                   Out* __restrict__ v) {
  griddep_launch_dependents();
  griddep_wait();
  const int per_head = g.D / 16;
  const long long n = static_cast<long long>(M) * 2 * g.heads * per_head;
  const long long idx = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x;
  if (idx >= n) return;
  const int part = static_cast<int>(idx % per_head);
  const long long hr = idx / per_head;
  const int head2 = static_cast<int>(hr % (2 * g.heads));
  const long long row = hr / (2 * g.heads);
  const int side = head2 >= g.heads;
  const int head = side ? head2 - g.heads : head2;
  const long long slot = slots[row];
  const bool past = slot >= g.num_pages * g.page;
  if (past && part == 0 && head2 == 0) raise_error(kErrIndex);
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (slot >= 0 && !past) {
    const long long page = slot >> g.page_log2;
    const int off = static_cast<int>(slot & (g.page - 1));
    const uint8_t* blk = g.pool + kv_block(g, page, head) + (side ? g.vc : 0);
    const uint2 c = *reinterpret_cast<const uint2*>(blk + off * (g.D / 2) + part * 8);
    const uint8_t* sc = blk + g.ks + off * kv_scale_bytes(FMT, g.D);
    constexpr int kLanes = kv_group(FMT) / 16;
    float s;
    if (FMT == kFmtInt4)
      s = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(sc + part / kLanes * 2)));
    else
      s = e4m3_value(sc[part / kLanes]);
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t nib = (w[i / 8] >> (4 * (i % 8))) & 15u;
      const float val = FMT == kFmtInt4 ? static_cast<float>(static_cast<int>(nib << 28) >> 28) : e2m1_value(nib);
      x[i] = __fmul_rn(val, s);
    }
  }
  Out* dst = (side ? v : k) + (row * g.heads + head) * g.D + part * 16;
  if constexpr (sizeof(Out) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace svdq
