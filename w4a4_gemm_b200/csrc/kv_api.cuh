// kv_api.cuh -- host side of the cache operators of include/svdq.h (batch plan,
// query/key norm and rotation, append, read, attention): argument checks and
// launches.  Included by svdq_api.cu, whose error macros, device table and
// launch helper it uses.
#pragma once

#include "kv_attn.cuh"
#include "kv_attn_rows.cuh"
#include "kv_cache.cuh"
#include "kv_plan.cuh"
#include "qk_norm_rope.cuh"

namespace {

inline int log2_exact(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// ------------------------------------------------------------- attention ---
constexpr int kMaxAttnCtas = 148 * 3;      // the most CTAs of a launch: words and slots of the workspace
constexpr int kAttnMaxBatch = 65536;       // the sums of 32 requests each are scanned in shared memory (16 KB)
constexpr size_t kAttnCounterBytes = (kMaxAttnCtas * sizeof(unsigned long long) + 255) & ~static_cast<size_t>(255);

// Blocks of 8 query rows that a decode tile has: two where a key head has more than 8 rows per request on average.
int dec_blocks(const svdq_kv_attention_desc* d) {
  const long long rep = d->q_heads / d->cache.kv_heads;
  return d->batch > 0 && static_cast<long long>(d->rows) * rep > 8LL * d->batch ? 2 : 1;
}
// One CTA of 12 warps per SM where the items (key heads of requests) are no more than the SMs: an SM then works on
// one or two items, whose steps all its warps share.  With more items the ends of the items cost more than that
// gives, and three CTAs of 4 warps cover for one another.
bool dec_wide(const svdq_kv_attention_desc* d, int nb, int sms) {
  const long long rep = d->q_heads / d->cache.kv_heads;
  const long long tiles = std::min<long long>(d->rows, (static_cast<long long>(d->rows) * rep + 8 * nb - 1) / (8 * nb) + d->batch);
  return tiles * d->cache.kv_heads <= sms;
}

// The tcgen05 kernel takes the call where a key head has more than this many query rows per request on average: its
// tiles have 256 rows.  16 requests over 8192 keys, 8 key heads: at 24 rows 64 us against 101, at 48 rows 96 against 98.
// The rule looks at the call, whose lengths are not known here, not at each request: a call that mixes a long prompt with
// single tokens is slower than one call for each (1500 tokens beside 64 single ones over up to 8192 keys: 452 us, apart
// 56 and 81).
constexpr int kRowsFrom = 48;
bool many_rows(const svdq_kv_attention_desc* d) {
  return d->batch > 0 && static_cast<long long>(d->rows) * (d->q_heads / d->cache.kv_heads) > static_cast<long long>(kRowsFrom) * d->batch;
}

using AttnKernel = void (*)(AttnParams);

template <int FMT, int D, int NB>
AttnKernel dec_kernel_for(bool wide) {
  return wide ? kv_attn_decode_kernel<FMT, D, NB, kDecWide> : kv_attn_decode_kernel<FMT, D, NB, kDecNarrow>;
}
template <int FMT>
AttnKernel dec_kernel_of(int D, int nb, bool wide) {
  if (D == 64) return nb == 1 ? dec_kernel_for<FMT, 64, 1>(wide) : dec_kernel_for<FMT, 64, 2>(wide);
  return nb == 1 ? dec_kernel_for<FMT, 128, 1>(wide) : dec_kernel_for<FMT, 128, 2>(wide);
}
AttnKernel dec_kernel(int fmt, int D, int nb, bool wide) {
  return fmt == SVDQ_NVFP4 ? dec_kernel_of<kFmtNvfp4>(D, nb, wide)
         : fmt == SVDQ_INT4 ? dec_kernel_of<kFmtInt4>(D, nb, wide) : dec_kernel_of<kFmtFp4g32>(D, nb, wide);
}

template <int FMT>
AttnKernel rows_kernel_of(int D, int* smem) {
  *smem = D == 64 ? RowsSmem<FMT, 64>::kBytes : RowsSmem<FMT, 128>::kBytes;
  return D == 64 ? kv_attn_rows_kernel<FMT, 64> : kv_attn_rows_kernel<FMT, 128>;
}
AttnKernel rows_kernel(int fmt, int D, int* smem) {
  return fmt == SVDQ_NVFP4 ? rows_kernel_of<kFmtNvfp4>(D, smem) : fmt == SVDQ_INT4 ? rows_kernel_of<kFmtInt4>(D, smem) : rows_kernel_of<kFmtFp4g32>(D, smem);
}

// 48 bits that differ from launch to launch (a counter spread by an odd multiplier and
// the shifts of splitmix64's finalizer), above 16 zero bits.
unsigned long long launch_nonce() {
  static std::atomic<unsigned long long> count{0};
  unsigned long long z = (count.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  z ^= z >> 31;
  return (z | 0x10000ull) & ~0xFFFFull;
}

// Kernel attributes of the cache operators, once per device.
std::atomic<bool> g_kv_set[kMaxDevices];

int kv_device(int* dev) {
  const int rc = current_device(dev);
  if (rc) return rc;
  if (g_kv_set[*dev].load(std::memory_order_acquire)) return SVDQ_OK;
  std::lock_guard<std::mutex> lk(g_mutex);
  if (g_kv_set[*dev].load(std::memory_order_relaxed)) return SVDQ_OK;
  SVDQ_CUDA(cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (2 * kPlanMaxRequests + 1) * static_cast<int>(sizeof(int))));
  if (g_dev[*dev].sms * 3 > kMaxAttnCtas) return SVDQ_ERR_CUDA;   // the workspace is laid out for 148 SMs
  for (int fmt : {SVDQ_NVFP4, SVDQ_INT4, SVDQ_FP4G32})
    for (int D : {64, 128})
      for (int nb : {1, 2})
        for (int wide : {0, 1})
          SVDQ_CUDA(cudaFuncSetAttribute(dec_kernel(fmt, D, nb, wide), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(dec_smem_bytes(fmt, D, nb, wide ? kDecWide : kDecNarrow))));
  for (int fmt : {SVDQ_NVFP4, SVDQ_INT4, SVDQ_FP4G32})
    for (int D : {64, 128}) {
      int smem = 0;
      AttnKernel k = rows_kernel(fmt, D, &smem);
      SVDQ_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
      cudaFuncAttributes at;
      SVDQ_CUDA(cudaFuncGetAttributes(&at, k));
      // its warp groups raise their registers to 184 out of what the block starts with: all of 65536, or they would wait
      if (at.numRegs * kRowsThreads < 2 * 128 * 184 + 128 * 80 + 128 * 64) return SVDQ_ERR_CUDA;
    }
  g_kv_set[*dev].store(true, std::memory_order_release);
  return SVDQ_OK;
}

// SVDQ_OK and the geometry of a cache description, or why it is refused.
int kv_geometry(const svdq_kv_cache* c, KvGeom* g, bool need_pool) {
  if (c == nullptr || (c->fmt != SVDQ_NVFP4 && c->fmt != SVDQ_INT4 && c->fmt != SVDQ_FP4G32)) return SVDQ_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->kv_heads < 1 || c->kv_heads > 1024 || c->page_size < 16 ||
      c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (c->num_pages < 0 || c->num_pages > 0x7fffffffLL) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (need_pool && (c->pool == nullptr || !aligned16(c->pool))) return SVDQ_ERR_INVALID_ARG;
  const int codes = c->page_size * c->head_dim / 2, scales = c->page_size * kv_scale_bytes(c->fmt, c->head_dim);
  g->pool = static_cast<uint8_t*>(c->pool);
  g->num_pages = c->num_pages;
  g->heads = c->kv_heads;
  g->D = c->head_dim;
  g->page = c->page_size;
  g->page_log2 = log2_exact(c->page_size);
  g->ks = codes;
  g->vc = codes + scales;
  g->vs = 2 * codes + scales;
  g->head_bytes = 2 * (codes + scales);
  return SVDQ_OK;
}

// Rows that plan, append and read take: the kernels count rows, and CTAs of up to 1024 rows, in 32 bits.
constexpr int kMaxRows = 1 << 30;

// The grid of append or read, `values` to a piece, and the rows of a thread: several where there are enough pieces for
// every thread that the SMs hold, so that more loads are in flight; one where latency counts.
int append_grid(int M, const KvGeom& g, int values, int sms, dim3* grid) {
  const int per_row = 2 * g.heads * (g.D / values);
  const int units = static_cast<long long>(M) * per_row >= static_cast<long long>(sms) * 2048 * kAppendUnits ? kAppendUnits : 1;
  const int rows = units * std::max(1, kAppendThreads / per_row);      // of a CTA
  *grid = dim3((M + rows - 1) / rows, std::max(1, (per_row + kAppendThreads - 1) / kAppendThreads));
  return units;
}

template <typename Out>
using ReadKernel = void (*)(KvGeom, const long long*, int, Out*, Out*);

template <typename Out>
ReadKernel<Out> read_kernel(int fmt, bool many) {
  if (fmt == SVDQ_NVFP4) return many ? kv_read_kernel<0, Out, kAppendUnits> : kv_read_kernel<0, Out, 1>;
  if (fmt == SVDQ_INT4) return many ? kv_read_kernel<1, Out, kAppendUnits> : kv_read_kernel<1, Out, 1>;
  return many ? kv_read_kernel<2, Out, kAppendUnits> : kv_read_kernel<2, Out, 1>;
}

using NormKernel = void (*)(NormRopeParams);

template <int LANES>
NormKernel norm_kernel_of(bool interleaved, bool batched) {
  if (interleaved) return batched ? qk_norm_rope_kernel<LANES, true, kNormBatch> : qk_norm_rope_kernel<LANES, true, 1>;
  return batched ? qk_norm_rope_kernel<LANES, false, kNormBatch> : qk_norm_rope_kernel<LANES, false, 1>;
}
NormKernel norm_kernel(int lanes_log2, bool interleaved, bool batched) {
  switch (lanes_log2) {
    case 1: return norm_kernel_of<2>(interleaved, batched);
    case 2: return norm_kernel_of<4>(interleaved, batched);
    case 3: return norm_kernel_of<8>(interleaved, batched);
    case 4: return norm_kernel_of<16>(interleaved, batched);
    default: return norm_kernel_of<32>(interleaved, batched);
  }
}

// rows of heads x D bf16 values whose loads are whole 16-byte words
bool rows_ok(const void* p, long long stride) { return p != nullptr && aligned16(p) && stride % 8 == 0 && stride >= 0; }

}  // namespace

extern "C" {

SVDQ_API int svdq_kv_page_bytes(const svdq_kv_cache* cache, size_t* bytes) {
  KvGeom g;
  const int rc = kv_geometry(cache, &g, false);
  if (rc) return rc;
  if (bytes == nullptr) return SVDQ_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(g.head_bytes) * g.heads;
  return SVDQ_OK;
}

SVDQ_API int svdq_kv_plan(const svdq_kv_plan_desc* d, void* stream) {
  if (d == nullptr || d->batch < 0 || d->rows < 0 || d->table_width < 0 || d->free_count < 0 || d->table_stride < d->table_width)
    return SVDQ_ERR_INVALID_ARG;
  if (d->batch > kPlanMaxRequests || d->rows > kMaxRows || d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)) != 0)
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (d->cu_q == nullptr || d->used == nullptr || (d->batch > 0 && (d->q_lens == nullptr || d->kv_lens == nullptr || d->total_lens == nullptr)) ||
      (d->batch > 0 && d->table_width > 0 && d->block_table == nullptr) || (d->free_count > 0 && d->free_pages == nullptr) ||
      (d->rows > 0 && (d->positions == nullptr || d->slots == nullptr)))
    return SVDQ_ERR_INVALID_ARG;
  int dev;
  const int rc = kv_device(&dev);
  if (rc) return rc;
  PlanParams p;
  p.q_lens = d->q_lens;
  p.kv_lens = d->kv_lens;
  p.table = d->block_table;
  p.table_stride = d->table_stride;
  p.width = d->table_width;
  p.free_pages = d->free_pages;
  p.free_count = d->free_count;
  p.batch = d->batch;
  p.rows = d->rows;
  p.page_log2 = log2_exact(d->page_size);
  p.cu_q = d->cu_q;
  p.total = d->total_lens;
  p.positions = d->positions;
  p.slots = reinterpret_cast<long long*>(d->slots);
  p.used = d->used;
  const int ctas = std::max({1, (d->rows + kPlanRows - 1) / kPlanRows, (d->batch + kPlanRequests - 1) / kPlanRequests});
  const size_t smem = (2 * static_cast<size_t>(d->batch) + 1) * sizeof(int);
  SVDQ_CUDA(launch_pdl(kv_plan_kernel, dim3(ctas), dim3(kPlanThreads), smem, static_cast<cudaStream_t>(stream), 0u, p));
  return SVDQ_OK;
}

SVDQ_API int svdq_qk_norm_rope(const svdq_qk_norm_rope_desc* d, void* stream) {
  if (d == nullptr || d->rows < 0 || d->q_heads < 0 || d->k_heads < 0) return SVDQ_ERR_INVALID_ARG;
  if (d->head_dim < 16 || d->head_dim > 256 || d->head_dim % 16 != 0 || d->rot_dim < 0 || d->rot_dim > d->head_dim ||
      d->rot_dim % 16 != 0 || d->q_heads > 65536 || d->k_heads > 65536)
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (d->rows == 0 || d->q_heads + d->k_heads == 0) return SVDQ_OK;
  const long long qn = static_cast<long long>(d->q_heads) * d->head_dim, kn = static_cast<long long>(d->k_heads) * d->head_dim;
  if (d->q_heads > 0 && (!rows_ok(d->q, d->q_stride) || !rows_ok(d->q_out, d->q_out_stride) || (d->rows > 1 && d->q_out_stride < qn)))
    return SVDQ_ERR_INVALID_ARG;
  if (d->k_heads > 0 && (!rows_ok(d->k, d->k_stride) || !rows_ok(d->k_out, d->k_out_stride) || (d->rows > 1 && d->k_out_stride < kn)))
    return SVDQ_ERR_INVALID_ARG;
  if (d->rot_dim > 0 && (d->table == nullptr || !aligned16(d->table) || d->table_rows < 0)) return SVDQ_ERR_INVALID_ARG;
  if (d->rot_dim > 0 && d->positions == nullptr && d->table_rows < d->rows) return SVDQ_ERR_INVALID_ARG;
  if ((d->q_weight != nullptr && !aligned16(d->q_weight)) || (d->k_weight != nullptr && !aligned16(d->k_weight))) return SVDQ_ERR_INVALID_ARG;
  if (d->norm && !(d->eps >= 0.f)) return SVDQ_ERR_INVALID_ARG;
  int dev;
  const int rc = kv_device(&dev);
  if (rc) return rc;
  NormRopeParams p;
  p.q = static_cast<const __nv_bfloat16*>(d->q);
  p.k = static_cast<const __nv_bfloat16*>(d->k);
  p.q_out = static_cast<__nv_bfloat16*>(d->q_out);
  p.k_out = static_cast<__nv_bfloat16*>(d->k_out);
  p.q_stride = d->q_stride;
  p.k_stride = d->k_stride;
  p.q_out_stride = d->q_out_stride;
  p.k_out_stride = d->k_out_stride;
  p.q_weight = static_cast<const __nv_bfloat16*>(d->q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(d->k_weight);
  p.table = d->table;
  p.positions = d->positions;
  p.table_rows = d->table_rows;
  p.rows = d->rows;
  p.q_heads = d->q_heads;
  p.k_heads = d->k_heads;
  p.D = d->head_dim;
  p.rot = d->rot_dim;
  p.norm = d->norm != 0;
  p.interleaved = d->interleaved != 0;
  p.eps = d->eps;
  const int lanes_log2 = log2_exact((d->head_dim + 7) / 8);   // of a head
  const int heads = d->q_heads + d->k_heads;
  // Heads that a lane group walks: as many as leave two waves of the 512 threads that an SM holds, at most 16; each
  // row's cosines and sines are then loaded once per chunk (4608 x 48 heads: 21.6 us, with chunks of 8 24 us).  Few
  // rows take a head per group: latency counts there.
  const long long lanes = static_cast<long long>(d->rows) << lanes_log2;
  const long long want = static_cast<long long>(g_dev[dev].sms) * 512 * 2;
  p.chunk = static_cast<int>(std::max<long long>(1, std::min<long long>(16, lanes * heads / want)));
  if (p.chunk >= kNormBatch) p.chunk = p.chunk / kNormBatch * kNormBatch;
  p.chunks = (heads + p.chunk - 1) / p.chunk;
  const long long ctas = (lanes * p.chunks + kNormThreads - 1) / kNormThreads;
  if (ctas * kNormThreads > 0x7fffffffLL) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  SVDQ_CUDA(launch_pdl(norm_kernel(lanes_log2, p.interleaved, p.chunk >= kNormBatch), dim3(static_cast<unsigned>(ctas)),
                       dim3(kNormThreads), 0, static_cast<cudaStream_t>(stream), 0u, p));
  return SVDQ_OK;
}

SVDQ_API int svdq_kv_append(const svdq_kv_cache* cache, const void* k, const void* v, long long k_stride,
                            long long v_stride, const int64_t* slots, int M, void* stream) {
  KvGeom g;
  int rc = kv_geometry(cache, &g, M > 0);
  if (rc) return rc;
  if (M < 0) return SVDQ_ERR_INVALID_ARG;
  if (M == 0) return SVDQ_OK;
  if (M > kMaxRows) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (slots == nullptr || !rows_ok(k, k_stride) || !rows_ok(v, v_stride)) return SVDQ_ERR_INVALID_ARG;
  int dev;
  if ((rc = kv_device(&dev))) return rc;
  dim3 grid;
  const bool many = append_grid(M, g, 8, g_dev[dev].sms, &grid) > 1;
  auto* kernel = cache->fmt == SVDQ_NVFP4 ? (many ? kv_append_kernel<0, kAppendUnits> : kv_append_kernel<0, 1>)
                 : cache->fmt == SVDQ_INT4 ? (many ? kv_append_kernel<1, kAppendUnits> : kv_append_kernel<1, 1>)
                                           : (many ? kv_append_kernel<2, kAppendUnits> : kv_append_kernel<2, 1>);
  SVDQ_CUDA(launch_pdl(kernel, grid, dim3(kAppendThreads), 0, static_cast<cudaStream_t>(stream), 0u, g, static_cast<const __nv_bfloat16*>(k),
                       static_cast<const __nv_bfloat16*>(v), k_stride, v_stride, reinterpret_cast<const long long*>(slots), M));
  return SVDQ_OK;
}

SVDQ_API int svdq_kv_read(const svdq_kv_cache* cache, const int64_t* slots, int M, int out_fp32, void* k, void* v,
                          void* stream) {
  KvGeom g;
  int rc = kv_geometry(cache, &g, M > 0);
  if (rc) return rc;
  if (M < 0) return SVDQ_ERR_INVALID_ARG;
  if (M == 0) return SVDQ_OK;
  if (M > kMaxRows) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (slots == nullptr || k == nullptr || v == nullptr || !aligned16(k) || !aligned16(v)) return SVDQ_ERR_INVALID_ARG;
  int dev;
  if ((rc = kv_device(&dev))) return rc;
  dim3 grid;
  const bool many = append_grid(M, g, out_fp32 ? 4 : 8, g_dev[dev].sms, &grid) > 1;
  const long long* sl = reinterpret_cast<const long long*>(slots);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (out_fp32) {
    SVDQ_CUDA(launch_pdl(read_kernel<float>(cache->fmt, many), grid, dim3(kAppendThreads), 0, st, 0u, g, sl, M, static_cast<float*>(k),
                         static_cast<float*>(v)));
  } else {
    SVDQ_CUDA(launch_pdl(read_kernel<__nv_bfloat16>(cache->fmt, many), grid, dim3(kAppendThreads), 0, st, 0u, g, sl, M,
                         static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v)));
  }
  return SVDQ_OK;
}

SVDQ_API int svdq_kv_attention_workspace_bytes(const svdq_kv_attention_desc* d, size_t* bytes) {
  if (d == nullptr || bytes == nullptr || d->rows < 0 || d->batch < 0) return SVDQ_ERR_INVALID_ARG;
  KvGeom g;
  const int rc = kv_geometry(&d->cache, &g, false);
  if (rc) return rc;
  if (d->q_heads < 1 || d->q_heads % g.heads != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  const size_t rows = many_rows(d) ? static_cast<size_t>(kMaxAttnCtas / 3) * 2 * kRowsTile * (g.D + 2) * sizeof(float) : 0;
  const size_t few = static_cast<size_t>(kMaxAttnCtas) * 2 * 8 * dec_blocks(d) * (g.D + 2) * sizeof(float);
  *bytes = kAttnCounterBytes + std::max(rows, few);
  return SVDQ_OK;
}

SVDQ_API int svdq_kv_attention(const svdq_kv_attention_desc* d, void* stream) {
  if (d == nullptr) return SVDQ_ERR_INVALID_ARG;
  AttnParams p;
  int rc = kv_geometry(&d->cache, &p.g, d->rows > 0);
  if (rc) return rc;
  if (d->rows < 0 || d->batch < 0 || d->window < 0 || d->table_width < 0 || d->table_stride < d->table_width) return SVDQ_ERR_INVALID_ARG;
  if (d->q_heads < 1 || d->q_heads % p.g.heads != 0 || d->q_heads > 65536) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!(d->scale == d->scale) || std::isinf(d->scale)) return SVDQ_ERR_INVALID_ARG;
  if (d->rows == 0 || d->batch == 0) return SVDQ_OK;
  if (!rows_ok(d->q, d->q_stride) || !rows_ok(d->out, d->out_stride) || d->out == d->q || d->cu_q == nullptr || d->kv_lens == nullptr ||
      (d->table_width > 0 && d->block_table == nullptr) ||
      (d->rows > 1 && d->out_stride < static_cast<long long>(d->q_heads) * p.g.D))
    return SVDQ_ERR_INVALID_ARG;
  if (d->batch > kAttnMaxBatch || static_cast<long long>(d->rows) * (d->q_heads / p.g.heads) > kMaxKeys) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (d->workspace == nullptr || (reinterpret_cast<uintptr_t>(d->workspace) & 255u)) return SVDQ_ERR_INVALID_ARG;
  int dev;
  if ((rc = kv_device(&dev))) return rc;
  p.q = static_cast<const __nv_bfloat16*>(d->q);
  p.q_stride = d->q_stride;
  p.out = static_cast<__nv_bfloat16*>(d->out);
  p.out_stride = d->out_stride;
  p.lse = d->lse;
  p.cu_q = d->cu_q;
  p.kv_lens = d->kv_lens;
  p.table = d->block_table;
  p.table_stride = d->table_stride;
  p.width = d->table_width;
  p.batch = d->batch;
  p.rows = d->rows;
  p.q_heads = d->q_heads;
  p.rep = fast_div(d->q_heads / p.g.heads);
  p.causal = d->causal != 0;
  p.window = static_cast<int>(std::min<long long>(d->window, kMaxKeys + 1));   // longer windows see every key alike
  p.scale = d->scale;
  p.budget = wait_budget();
  p.nonce = launch_nonce();
  p.counters = static_cast<unsigned long long*>(d->workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(d->workspace) + kAttnCounterBytes);
  p.min_units = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (many_rows(d)) {
    p.min_units = 2;
    int smem = 0;
    AttnKernel k = rows_kernel(d->cache.fmt, p.g.D, &smem);
    SVDQ_CUDA(launch_pdl(k, dim3(g_dev[dev].sms), dim3(kRowsThreads), static_cast<size_t>(smem), st, 0u, p));
    return SVDQ_OK;
  }
  const int nb = dec_blocks(d);
  const bool wide = dec_wide(d, nb, g_dev[dev].sms);
  const int warps = wide ? kDecWide : kDecNarrow, unit = warps * kDecChunk;
  // enough CTAs for the most units that these rows and this table can hold
  const long long tiles = std::min<long long>((static_cast<long long>(d->rows) * p.rep.d + 8 * nb - 1) / (8 * nb) + d->batch,
                                              static_cast<long long>(d->rows) * p.rep.d);
  const long long units = tiles * p.g.heads * std::max<long long>(1, ((static_cast<long long>(p.width) << p.g.page_log2) + unit - 1) / unit + 1);
  const int ctas = static_cast<int>(std::min<long long>(units, static_cast<long long>(g_dev[dev].sms) * (wide ? 1 : 3)));
  SVDQ_CUDA(launch_pdl(dec_kernel(d->cache.fmt, p.g.D, nb, wide), dim3(ctas), dim3(32 * warps), dec_smem_bytes(d->cache.fmt, p.g.D, nb, warps), st,
                       0u, p));
  return SVDQ_OK;
}

}  // extern "C"
