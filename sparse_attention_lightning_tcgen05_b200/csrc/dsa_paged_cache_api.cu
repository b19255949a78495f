// dsa_paged_cache_api.cu -- C ABI of the paged cache's writers (the
// operations, layouts and error rules are stated in
// include/dsa_paged_cache.h): argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "dsa_launch.h"
#include "dsa_paged_cache.h"
#include "paged_cache.cuh"
#include "paged_geom.h"

namespace dsa_host {

dsa_status_t check_paged_cache(const dsa_paged_cache_t *c) {
  if (c->num_seqs < 1 || c->H_kv < 1 || c->pages_per_seq < 1 || c->num_pages < 1)
    return DSA_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) != 0)
    return DSA_ERR_INVALID_ARG;
  if (c->dtype != DSA_KV_BF16 && c->dtype != DSA_KV_FP8_E4M3_E8M0_B32) return DSA_ERR_INVALID_ARG;
  if (c->D != 128 || c->H_kv > 128) return DSA_ERR_UNSUPPORTED;
  for (const int64_t s : {c->page_stride, c->slot_stride, c->head_stride})
    if (s < 128 || s % 128 != 0) return DSA_ERR_INVALID_ARG;
  if (!c->block_table || !aligned(c->block_table, 4)) return DSA_ERR_INVALID_ARG;
  // slots of a sequence and of the pool are 32-bit; a page's offset is 64-bit
  const int64_t ps = c->page_size;
  if (c->pages_per_seq * ps > INT32_MAX || c->num_pages * ps > INT32_MAX)
    return DSA_ERR_UNSUPPORTED;
  const int64_t most = (int64_t{1} << 56) / std::max<int64_t>(c->num_pages, ps);
  if (c->page_stride > most || c->slot_stride > most || c->head_stride > most)
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

dsa::PagedGeom paged_geom(const dsa_paged_cache_t *c) {
  dsa::PagedGeom g{};
  g.num_seqs = c->num_seqs;
  g.H_kv = c->H_kv;
  g.page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
  g.pages_per_seq = c->pages_per_seq;
  g.num_pages = c->num_pages;
  g.page_stride = c->page_stride;
  g.slot_stride = c->slot_stride;
  g.head_stride = c->head_stride;
  g.table = c->block_table;
  return g;
}

dsa_status_t check_pool(const dsa_paged_cache_t *c, const void *data, const uint8_t *scale) {
  if (!data || !aligned(data, 16)) return DSA_ERR_INVALID_ARG;
  if (c->dtype == DSA_KV_BF16) return scale ? DSA_ERR_INVALID_ARG : DSA_OK;
  return scale && aligned(scale, 4) ? DSA_OK : DSA_ERR_INVALID_ARG;
}

namespace {

using AppendFn = void (*)(const dsa::AppendParams);

template <bool kQ, bool kKv>
AppendFn append_fn(bool halves) {
  return halves ? dsa::cache_append_kernel<kQ, kKv, true> : dsa::cache_append_kernel<kQ, kKv, false>;
}

using PoolFn = void (*)(const dsa::PoolParams);

template <bool kFp8>
PoolFn pool_fn(bool pow2, int block_size) {
  if (!pow2) return dsa::block_pool_kernel<kFp8, 0>;
  switch (block_size) {
    case 1: return dsa::block_pool_kernel<kFp8, 1>;
    case 2: return dsa::block_pool_kernel<kFp8, 2>;
    case 4: return dsa::block_pool_kernel<kFp8, 4>;
    case 8: return dsa::block_pool_kernel<kFp8, 8>;
    default: return dsa::block_pool_kernel<kFp8, 16>;
  }
}

dsa_status_t check_append(const dsa_append_desc_t *d) {
  if (!d) return DSA_ERR_INVALID_ARG;
  dsa_status_t st = check_paged_cache(&d->cache);
  if (st != DSA_OK) return st;
  if (d->T < 1 || d->H < 0) return DSA_ERR_INVALID_ARG;
  if (d->H > 256) return DSA_ERR_UNSUPPORTED;
  if (d->rope != DSA_ROPE_INTERLEAVED && d->rope != DSA_ROPE_HALVES) return DSA_ERR_INVALID_ARG;
  if (d->rope_dim < 0 || d->rope_dim > 128 || d->rope_dim % 2 != 0) return DSA_ERR_INVALID_ARG;
  if (d->rope == DSA_ROPE_HALVES && d->rope_dim % 16 != 0) return DSA_ERR_UNSUPPORTED;
  if (d->q_dtype != DSA_KV_BF16 && d->q_dtype != DSA_KV_FP8_E4M3_E8M0_B32)
    return DSA_ERR_INVALID_ARG;
  const int64_t kv_row = static_cast<int64_t>(d->cache.H_kv) * 128;
  if (d->H > 0 && (d->q_stride % 8 != 0 || d->q_stride < static_cast<int64_t>(d->H) * 128))
    return DSA_ERR_INVALID_ARG;
  if (d->k_stride % 8 != 0 || d->k_stride < kv_row) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

dsa_status_t check_block_pool(const dsa_block_pool_desc_t *d) {
  if (!d) return DSA_ERR_INVALID_ARG;
  const dsa_status_t st = check_paged_cache(&d->cache);
  if (st != DSA_OK) return st;
  if (d->block_size < 1 || d->S_pool < 1) return DSA_ERR_INVALID_ARG;
  if (d->block_size > 65536) return DSA_ERR_UNSUPPORTED;
  if (d->seq_stride < 0 || d->head_stride < 0 || d->seq_stride % 128 != 0 ||
      d->head_stride % 128 != 0)
    return DSA_ERR_INVALID_ARG;
  if (d->S_pool > INT32_MAX || d->seq_stride > (int64_t{1} << 56) / d->cache.num_seqs ||
      d->head_stride > (int64_t{1} << 48))
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa_host

using namespace dsa_host;

extern "C" {

dsa_status_t dsa_cache_append(const dsa_append_desc_t *desc, const void *q, const void *k,
                              const void *v, const float *cos, const float *sin,
                              const int32_t *positions, const int32_t *seq_ids, void *q_out,
                              uint8_t *q_scale, void *k_cache, uint8_t *k_scale, void *v_cache,
                              uint8_t *v_scale, dsa_stream_t stream) {
  dsa_status_t st = check_append(desc);
  if (st != DSA_OK) return st;
  const dsa_paged_cache_t &c = desc->cache;
  const bool q_fp8 = desc->q_dtype != DSA_KV_BF16, kv_fp8 = c.dtype != DSA_KV_BF16;
  if (!k || !positions || !aligned(k, 16) || !aligned(positions, 4) || !aligned(seq_ids, 4))
    return DSA_ERR_INVALID_ARG;
  if (desc->H > 0) {
    if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return DSA_ERR_INVALID_ARG;
    if (q_fp8 ? (!q_scale || !aligned(q_scale, 4)) : q_scale != nullptr) return DSA_ERR_INVALID_ARG;
    // in place only where a row is written where it was read
    if (q_out == q && (q_fp8 || desc->q_stride != static_cast<int64_t>(desc->H) * 128))
      return DSA_ERR_INVALID_ARG;
  } else if (q || q_out || q_scale) {
    return DSA_ERR_INVALID_ARG;
  }
  if (desc->rope_dim > 0 && (!cos || !sin || !aligned(cos, 4) || !aligned(sin, 4)))
    return DSA_ERR_INVALID_ARG;
  st = check_pool(&c, k_cache, k_scale);
  if (st != DSA_OK) return st;
  if (v) {
    if (!aligned(v, 16) || desc->v_stride % 8 != 0 ||
        desc->v_stride < static_cast<int64_t>(c.H_kv) * 128)
      return DSA_ERR_INVALID_ARG;
    st = check_pool(&c, v_cache, v_scale);
    if (st != DSA_OK) return st;
  } else if (v_cache || v_scale) {
    return DSA_ERR_INVALID_ARG;
  }
  DeviceInfo *dev = nullptr;
  st = device_info(&dev);
  if (st != DSA_OK) return st;

  dsa::AppendParams p{};
  p.g = paged_geom(&c);
  p.T = desc->T;
  p.H = desc->H;
  p.rows = desc->H + c.H_kv * (v ? 2 : 1);
  p.units = (p.rows + dsa::kAppendRows - 1) / dsa::kAppendRows;
  p.half = desc->rope_dim / 2;
  p.vec = p.half % 4 == 0 && aligned(cos, 16) && aligned(sin, 16);
  p.minus_zero = -0.f;
  p.q_stride = desc->q_stride;
  p.k_stride = desc->k_stride;
  p.v_stride = desc->v_stride;
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.cos = cos;
  p.sin = sin;
  p.positions = positions;
  p.seq_ids = seq_ids;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.q_scale = q_scale;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const bool halves = desc->rope == DSA_ROPE_HALVES;
  // without queries one instance per cache type serves both query types
  const bool qf = desc->H > 0 ? q_fp8 : kv_fp8;
  const AppendFn fn = qf ? (kv_fp8 ? append_fn<true, true>(halves) : append_fn<true, false>(halves))
                         : (kv_fp8 ? append_fn<false, true>(halves) : append_fn<false, false>(halves));
  const int lanes = qf || kv_fp8 ? dsa::kAppendLanes<true> : dsa::kAppendLanes<false>;
  const int per_block = dsa::kAppendThreads / lanes;
  const int64_t blocks = (static_cast<int64_t>(p.T) * p.units + per_block - 1) / per_block;
  // the kernel numbers its threads in 32 bits
  if (blocks * dsa::kAppendThreads > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (launch_pdl(fn, static_cast<int>(blocks), dsa::kAppendThreads, 0,
                 reinterpret_cast<cudaStream_t>(stream), 0, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  return DSA_OK;
}

dsa_status_t dsa_block_pool(const dsa_block_pool_desc_t *desc, const void *k_cache,
                            const uint8_t *k_scale, const int32_t *start,
                            const int32_t *positions, void *pooled, uint8_t *pooled_scale,
                            int32_t *last_block, dsa_stream_t stream) {
  dsa_status_t st = check_block_pool(desc);
  if (st != DSA_OK) return st;
  const dsa_paged_cache_t &c = desc->cache;
  if (!positions || !aligned(positions, 4) || !aligned(start, 4) || !aligned(last_block, 4))
    return DSA_ERR_INVALID_ARG;
  st = check_pool(&c, k_cache, k_scale);
  if (st != DSA_OK) return st;
  st = check_pool(&c, pooled, pooled_scale);
  if (st != DSA_OK) return st;
  DeviceInfo *dev = nullptr;
  st = device_info(&dev);
  if (st != DSA_OK) return st;

  dsa::PoolParams p{};
  p.g = paged_geom(&c);
  p.block_size = desc->block_size;
  // a run of 16 slots a half warp
  const bool pow2 = (p.block_size & (p.block_size - 1)) == 0;
  p.share = 1;
  while (p.share < dsa::kPoolGroups && p.share * dsa::kPoolRun < p.block_size) p.share *= 2;
  p.block_shift = __builtin_ctz(static_cast<unsigned>(p.block_size));
  const int together = pow2 ? std::max(1, dsa::kPoolRun / p.block_size) : 1;   // blocks of an item
  const int per_cta = dsa::kPoolGroups / p.share;
  const int64_t sets = (p.g.capacity() / p.block_size + together - 1) / together;
  // the kernel numbers up to kPoolSeqs sequences' items in 32 bits
  if (sets * c.H_kv > INT32_MAX / std::min(c.num_seqs, dsa::kPoolSeqs)) return DSA_ERR_UNSUPPORTED;
  const bool fp8 = c.dtype != DSA_KV_BF16;
  // (blocks larger than the table are never complete: last_block is still due)
  const int64_t most = std::max<int64_t>(1, (sets * c.H_kv * c.num_seqs + per_cta - 1) / per_cta);
  const int wave = dev->num_sms * (fp8 ? dsa::kPoolCtasPerSm<true> : dsa::kPoolCtasPerSm<false>);
  const int blocks = static_cast<int>(std::min<int64_t>(most, wave));
  p.S_pool = desc->S_pool;
  p.seq_stride = desc->seq_stride;
  p.head_stride = desc->head_stride;
  p.k = k_cache;
  p.k_scale = k_scale;
  p.start = start;
  p.positions = positions;
  p.pooled = pooled;
  p.pooled_scale = pooled_scale;
  p.last_block = last_block;
  const PoolFn fn = fp8 ? pool_fn<true>(pow2, p.block_size) : pool_fn<false>(pow2, p.block_size);
  if (launch_pdl(fn, blocks, dsa::kPoolThreads, 0,
                 reinterpret_cast<cudaStream_t>(stream), 0, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  return DSA_OK;
}

}  // extern "C"
