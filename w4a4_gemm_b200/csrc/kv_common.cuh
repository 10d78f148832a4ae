// kv_common.cuh -- what the cache operators' kernels share beside svdq_ptx.cuh and
// svdq_formats.cuh.
#pragma once

#include <cuda_runtime.h>

#include "svdq_ptx.cuh"

namespace svdq {

// Further bits of the sticky device error word (bits 0 to 2: svdq_ptx.cuh).
enum : unsigned {
  kErrIndex = 1u << 3,      // an index or a length out of range: that element was left out
  kErrWaitAttn = 1u << 4,   // a bounded wait ran out in an attention kernel
};

// Two fp32 operations in one instruction (IEEE round-to-nearest per lane).
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  unsigned long long x, y, z, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(w) : "l"(x), "l"(y), "l"(z));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(w));
  return r;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  unsigned long long x, y, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(w) : "l"(x), "l"(y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(w));
  return r;
}

}  // namespace svdq
