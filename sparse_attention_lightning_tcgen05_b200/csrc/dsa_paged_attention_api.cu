// dsa_paged_attention_api.cu -- C ABI of attention over a paged cache (the
// operation, layouts and error rules are stated in
// include/dsa_paged_attention.h): argument checks, the workspace and the
// launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dsa_launch.h"
#include "dsa_paged_attention.h"
#include "paged_attention.cuh"
#include "paged_geom.h"

namespace dsa_host {
namespace {

// The partial results' room is sized for the 148 SMs of a B200, so that the
// workspace size depends on the descriptor alone.
constexpr int kPaCtasPerSm = 2;
constexpr int kPaGrid = 148 * kPaCtasPerSm;

dsa_status_t check_attn(const dsa_paged_attention_desc_t *d, bool list) {
  if (!d) return DSA_ERR_INVALID_ARG;
  const dsa_status_t st = check_paged_cache(&d->cache);
  if (st != DSA_OK) return st;
  if (d->T < 1 || d->H < 1 || d->H % d->cache.H_kv != 0 || d->window < 0 ||
      !std::isfinite(d->sm_scale))
    return DSA_ERR_INVALID_ARG;
  if (d->H / d->cache.H_kv > 128) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->T) * d->H > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (list) {
    if (d->block_size < 1 || d->block_size > 65536 || (d->block_size & (d->block_size - 1)) != 0)
      return DSA_ERR_INVALID_ARG;
    if (d->num_blocks < 1) return DSA_ERR_INVALID_ARG;
    if (d->block_heads != 1 && d->block_heads != d->cache.H_kv) return DSA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(d->num_blocks) * d->block_size + d->window >= (1 << 30))
      return DSA_ERR_UNSUPPORTED;
  }
  return DSA_OK;
}

size_t part_floats() { return static_cast<size_t>(kPaGrid) * 2 * dsa::kPaRows * dsa::kRowD; }

size_t workspace_bytes_needed() {
  return kWorkspaceHeader + part_floats() * 4 + static_cast<size_t>(kPaGrid) * 2 * dsa::kPaRows * 8 +
         static_cast<size_t>(kPaGrid) * 16;
}

template <bool kFp8, bool kList>
dsa_status_t launch(const dsa::PagedAttnParams &p, int grid, DeviceInfo *dev, uint32_t bit,
                    cudaStream_t s) {
  const int smem = dsa::PaSmem<kFp8>::kTotal;
  const dsa_status_t st = ensure_smem_attr(dev, bit, dsa::paged_attention_kernel<kFp8, kList>, smem);
  if (st != DSA_OK) return st;
  if (launch_pdl(dsa::paged_attention_kernel<kFp8, kList>, grid, dsa::kPaThreads,
                 static_cast<size_t>(smem), s, 0, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (launch_pdl(dsa::paged_attention_join_kernel, grid * (dsa::kPaRows / 2), dsa::kPaJoinThreads, 0,
                 s, 0, p, grid) != cudaSuccess)
    return DSA_ERR_CUDA;
  return DSA_OK;
}

dsa_status_t attend(const dsa_paged_attention_desc_t *d, bool list, const void *q, const void *k,
                    const uint8_t *k_scale, const void *v, const uint8_t *v_scale,
                    const float *sinks, const int32_t *positions, const int32_t *seq_ids,
                    const int32_t *blocks, void *out, float *lse, void *workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  dsa_status_t st = check_attn(d, list);
  if (st != DSA_OK) return st;
  if (!q || !positions || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(positions, 4) ||
      !aligned(sinks, 4) || !aligned(seq_ids, 4) || !aligned(lse, 4))
    return DSA_ERR_INVALID_ARG;
  if (list && (!blocks || !aligned(blocks, 4))) return DSA_ERR_INVALID_ARG;
  st = check_pool(&d->cache, k, k_scale);
  if (st != DSA_OK) return st;
  st = check_pool(&d->cache, v, v_scale);
  if (st != DSA_OK) return st;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < workspace_bytes_needed())
    return DSA_ERR_WORKSPACE;
  DeviceInfo *dev = nullptr;
  st = device_info(&dev);
  if (st != DSA_OK) return st;

  dsa::PagedAttnParams p{};
  p.g = paged_geom(&d->cache);
  p.T = d->T;
  p.H = d->H;
  p.G = d->H / d->cache.H_kv;
  p.head_tiles = (p.G + dsa::kPaRows - 1) / dsa::kPaRows;
  p.window = d->window;
  p.gran_shift = 4;
  int64_t most_chunks = (p.g.capacity() + dsa::kPaChunk - 1) / dsa::kPaChunk;
  if (d->window > 0 || list)       // a window may begin inside a step
    most_chunks = std::min<int64_t>(most_chunks, (static_cast<int64_t>(d->window) + 15) / 16 + 1);
  if (list) {
    p.block_shift = __builtin_ctz(static_cast<unsigned>(d->block_size));
    p.num_blocks = d->num_blocks;
    p.block_heads = d->block_heads;
    p.gran_shift = std::min(4, p.block_shift);
    p.list_chunks = static_cast<int>(
        (static_cast<int64_t>(d->num_blocks) * d->block_size + dsa::kPaChunk - 1) / dsa::kPaChunk);
    most_chunks += p.list_chunks;
  }
  p.scale_log2 = d->sm_scale * dsa::kPaLog2e;
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint8_t *>(k);
  p.v = static_cast<const uint8_t *>(v);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.sinks = sinks;
  p.positions = positions;
  p.seq_ids = seq_ids;
  p.blocks = blocks;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kWorkspaceHeader);
  p.part_ml = reinterpret_cast<float2 *>(p.part_o + part_floats());
  p.chain = reinterpret_cast<int4 *>(p.part_ml + static_cast<size_t>(kPaGrid) * 2 * dsa::kPaRows);
  // no more CTAs than tiles
  const int64_t most_tiles = std::max<int64_t>(1, (most_chunks + dsa::kPaWarps - 1) / dsa::kPaWarps);
  const int64_t rows = static_cast<int64_t>(p.T) * p.g.H_kv * p.head_tiles;
  const int grid = static_cast<int>(std::min<int64_t>(
      std::min(kPaGrid, dev->num_sms * kPaCtasPerSm),
      rows > kPaGrid ? rows : rows * most_tiles));
  const bool fp8 = d->cache.dtype != DSA_KV_BF16;
  if (list)
    return fp8 ? launch<true, true>(p, grid, dev, kAttrPagedAttn + 3, stream)
               : launch<false, true>(p, grid, dev, kAttrPagedAttn + 2, stream);
  return fp8 ? launch<true, false>(p, grid, dev, kAttrPagedAttn + 1, stream)
             : launch<false, false>(p, grid, dev, kAttrPagedAttn, stream);
}

}  // namespace
}  // namespace dsa_host

using namespace dsa_host;

extern "C" {

dsa_status_t dsa_paged_attention_workspace_size(const dsa_paged_attention_desc_t *desc,
                                                size_t *bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  const dsa_status_t st = check_attn(desc, desc && desc->num_blocks != 0);
  if (st != DSA_OK) return st;
  *bytes = workspace_bytes_needed();
  return DSA_OK;
}

dsa_status_t dsa_paged_attention_forward(const dsa_paged_attention_desc_t *desc, const void *q,
                                         const void *k, const uint8_t *k_scale, const void *v,
                                         const uint8_t *v_scale, const float *sinks,
                                         const int32_t *positions, const int32_t *seq_ids,
                                         void *out, float *lse, void *workspace,
                                         size_t workspace_bytes, dsa_stream_t stream) {
  return attend(desc, false, q, k, k_scale, v, v_scale, sinks, positions, seq_ids, nullptr, out,
                lse, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_block_attention_forward(const dsa_paged_attention_desc_t *desc, const void *q,
                                         const void *k, const uint8_t *k_scale, const void *v,
                                         const uint8_t *v_scale, const float *sinks,
                                         const int32_t *positions, const int32_t *seq_ids,
                                         const int32_t *blocks, void *out, float *lse,
                                         void *workspace, size_t workspace_bytes,
                                         dsa_stream_t stream) {
  return attend(desc, true, q, k, k_scale, v, v_scale, sinks, positions, seq_ids, blocks, out, lse,
                workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
