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
#include "paged_attention_wide.cuh"
#include "paged_geom.h"

namespace dsa_host {
namespace {

// The partial results' room is sized for the 148 SMs of a B200, so that the
// workspace size depends on the descriptor alone.
constexpr int kPaCtasPerSm = 2;
constexpr int kSizingSms = 148;
constexpr uint64_t kPaWaitLimitNs = 4000000000ull;
constexpr uint64_t kPaDrainLimitNs = 4000000000ull;

dsa_status_t check_attn(const dsa_paged_attention_desc_t *d, bool list) {
  if (!d) return DSA_ERR_INVALID_ARG;
  const dsa_status_t st = check_paged_cache(&d->cache);
  if (st != DSA_OK) return st;
  if (d->T < 1 || d->H < 1 || d->H % d->cache.H_kv != 0 || d->window < 0 ||
      !std::isfinite(d->sm_scale * dsa::kPaLog2e))
    return DSA_ERR_INVALID_ARG;
  if (d->flags & ~DSA_FLAG_SELFTEST_STALL) return DSA_ERR_INVALID_ARG;
  if (d->H / d->cache.H_kv > 128) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->T) * d->H > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  // a tensor map's strides are below 2^40 bytes
  for (const int64_t s : {d->cache.page_stride, d->cache.slot_stride, d->cache.head_stride})
    if (s >= int64_t{1} << 39) return DSA_ERR_UNSUPPORTED;
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

// The kernel of a call. Wide: all query heads of a key-value head as the rows of
// one tcgen05 tile, from more than 16 of them on (the other kernel takes 16 at a
// time, each time with all the slots), for an fp8 cache from more than 48 on:
// there the conversion bounds the wide kernel whatever the heads. Contexts with
// one key head, us (graph replays, three inputs in turn), other kernel / wide:
//   heads               16         32         48         64        128
//   bf16 4 x 65,536  32 / 35    37 / 35    68 / 36    60 / 37   109 / 39
//        16 x 4,096  16 / 24    21 / 25    23 / 27    26 / 29    35 / 34
//        16 x 1,024  10 / 13    15 / 13    15 / 13    16 / 14    18 / 14
//   fp8  4 x 65,536  25 / 53    35 / 54    49 / 55    61 / 55   111 / 55
//        16 x 4,096  15 / 30    21 / 32    24 / 33    26 / 34    38 / 40
//        16 x 1,024  14 / 16    16 / 16    16 / 17    17 / 17    21 / 18
// Of the lengths the host knows the table's capacity alone; what the wide kernel
// loses between short and long ones is a few us, what it gains on many long ones is
// the larger part (64 contexts of 1,024 to 32,768 slots, 2 key heads of 32 heads,
// bf16: 315 / 195).
struct Plan {
  bool fp8, wide;
  int rows, head_tiles, step, grid;      // grid: CTAs at most
};

Plan plan_of(const dsa_paged_attention_desc_t *d) {
  Plan p{};
  const int G = d->H / d->cache.H_kv;
  p.fp8 = d->cache.dtype != DSA_KV_BF16;
  p.wide = G > (p.fp8 ? 3 : 1) * dsa::kPaRows;
  p.rows = p.wide ? dsa::kPwRows : dsa::kPaRows;
  p.head_tiles = (G + p.rows - 1) / p.rows;
  p.step = p.wide ? dsa::kPwTile : p.fp8 ? dsa::PaSmem<true>::kStep : dsa::PaSmem<false>::kStep;
  p.grid = p.wide ? kSizingSms : kSizingSms * kPaCtasPerSm;
  return p;
}

size_t part_rows(const Plan &p) { return static_cast<size_t>(p.grid) * 2 * p.rows; }

size_t workspace_bytes_needed(const Plan &p) {
  return kWorkspaceHeader + part_rows(p) * (dsa::kRowD * 4 + 8) + static_cast<size_t>(p.grid) * 16;
}

using AttnFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap,
                        const dsa::PagedAttnParams);

// A pool as [page][head][half of a row][slot][128 bytes] (an fp8 row is one
// half), in boxes of `rows` slots: both halves of them where they are a whole
// stage of the kernel (`both`), one after the other in shared memory.
dsa_status_t pool_map(CUtensorMap *m, const dsa_paged_cache_t *c, const void *base, int rows,
                      bool both) {
  const bool fp8 = c->dtype != DSA_KV_BF16;
  const cuuint64_t elt = fp8 ? 1 : 2, halves = fp8 ? 1 : 2;
  const cuuint64_t dims[5] = {128 / halves, static_cast<cuuint64_t>(c->page_size), halves,
                              static_cast<cuuint64_t>(c->H_kv), static_cast<cuuint64_t>(c->num_pages)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(c->slot_stride) * elt, 128,
                                 static_cast<cuuint64_t>(c->head_stride) * elt,
                                 static_cast<cuuint64_t>(c->page_stride) * elt};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(dims[0]), static_cast<cuuint32_t>(rows),
                             both ? static_cast<cuuint32_t>(halves) : 1, 1, 1};
  // no more of a line than the box's 128 bytes of an fp8 row: the next 128 are
  // another head's
  return make_map(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base,
                  dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                  fp8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
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
  const Plan plan = plan_of(d);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < workspace_bytes_needed(plan))
    return DSA_ERR_WORKSPACE;
  DeviceInfo *dev = nullptr;
  st = device_info(&dev);
  if (st != DSA_OK) return st;

  dsa::PagedAttnParams p{};
  p.g = paged_geom(&d->cache);
  p.T = d->T;
  p.H = d->H;
  p.G = d->H / d->cache.H_kv;
  p.rows = plan.rows;
  p.head_tiles = plan.head_tiles;
  p.window = d->window;
  const int unit = std::min(plan.step, 32);
  int unit_shift = unit == 32 ? 5 : 4;
  int64_t most_steps = (p.g.capacity() + plan.step - 1) / plan.step;
  if (d->window > 0 || list)       // a window may begin inside a step
    most_steps = std::min<int64_t>(most_steps, (static_cast<int64_t>(d->window) + 31) / plan.step + 2);
  p.gran_shift = std::min(unit_shift, p.g.page_shift);
  if (list) {
    p.block_shift = __builtin_ctz(static_cast<unsigned>(d->block_size));
    p.num_blocks = d->num_blocks;
    p.block_heads = d->block_heads;
    p.gran_shift = std::min(p.gran_shift, p.block_shift);
    p.list_steps = static_cast<int>(
        (static_cast<int64_t>(d->num_blocks) * d->block_size + plan.step - 1) / plan.step);
    most_steps += p.list_steps;
  }
  p.scale_log2 = d->sm_scale * dsa::kPaLog2e;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.sinks = sinks;
  p.positions = positions;
  p.seq_ids = seq_ids;
  p.blocks = blocks;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kWorkspaceHeader);
  p.part_ml = reinterpret_cast<float2 *>(p.part_o + part_rows(plan) * dsa::kRowD);
  p.chain = reinterpret_cast<int4 *>(p.part_ml + part_rows(plan));
  p.err = static_cast<unsigned int *>(workspace);
  p.err_info = p.err + 1;
  p.selftest_stall = (d->flags & DSA_FLAG_SELFTEST_STALL) != 0;
  p.wait_limit_ns = d->wait_limit_ns ? d->wait_limit_ns : kPaWaitLimitNs;
  p.drain_limit_ns = kPaDrainLimitNs;
  CUtensorMap tq, tk, tv;
  {
    const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(p.T) * p.H};
    const cuuint64_t strides[1] = {256};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(plan.wide ? p.G : plan.rows)};
    const int rows = 1 << p.gran_shift;
    st = make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q, dims, strides, box);
    if (st == DSA_OK) st = pool_map(&tk, &d->cache, k, rows, rows == plan.step);
    if (st == DSA_OK) st = pool_map(&tv, &d->cache, v, rows, rows == plan.step);
    if (st != DSA_OK) return st;
  }
  // no more CTAs than have enough steps
  const int least = plan.wide  ? dsa::kPwLeast
                    : plan.fp8 ? dsa::PaSmem<true>::kLeast
                               : dsa::PaSmem<false>::kLeast;
  const int64_t items = static_cast<int64_t>(p.T) * p.g.H_kv * p.head_tiles;
  const int64_t most = std::min(plan.grid, dev->num_sms * (plan.wide ? 1 : kPaCtasPerSm));
  const int64_t want = items > most * least
                           ? most
                           : (items * std::max<int64_t>(1, most_steps) + least - 1) / least;
  int grid = static_cast<int>(std::min(most, want));
  // A multiple of the key heads, where that idles less than a sixteenth of the
  // CTAs: the heads' shares then begin alike, and what lies side by side in
  // memory (a slot's rows and scales of all heads) is read at the same time. (2, 4
  // and 8 key heads divide the 296 CTAs anyhow.) 16 contexts of 2,048 to 32,768 slots,
  // 8 query heads a key head, us otherwise and so: bf16 with 3, 6, 7, 12, 16 key
  // heads 84 and 84, 144 and 144, 165 and 163, 267 and 263, 355 and 340; fp8 63 and
  // 63, 102 and 101, 118 and 114, 180 and 182, 230 and 237.
  if (grid % p.g.H_kv * 16 < grid) grid -= grid % p.g.H_kv;
  p.chain_by_item = items <= grid;
  p.ctas = grid;
  const int entries = static_cast<int>(std::min<int64_t>(items, grid));
  const int variant = (plan.wide ? 4 : 0) + (plan.fp8 ? 2 : 0) + (list ? 1 : 0);
  static const AttnFn fns[8] = {
      dsa::paged_attention_kernel<false, false>,      dsa::paged_attention_kernel<false, true>,
      dsa::paged_attention_kernel<true, false>,       dsa::paged_attention_kernel<true, true>,
      dsa::paged_attention_wide_kernel<false, false>, dsa::paged_attention_wide_kernel<false, true>,
      dsa::paged_attention_wide_kernel<true, false>,  dsa::paged_attention_wide_kernel<true, true>};
  static const int smems[4] = {dsa::PaSmem<false>::kTotal, dsa::PaSmem<true>::kTotal,
                               dsa::PwSmem<false>::kTotal, dsa::PwSmem<true>::kTotal};
  static const int threads_of[4] = {dsa::PaSmem<false>::kThreads, dsa::PaSmem<true>::kThreads,
                                    dsa::PwSmem<false>::kThreads, dsa::PwSmem<true>::kThreads};
  const int smem = smems[variant >> 1], threads = threads_of[variant >> 1];
  st = ensure_smem_attr(dev, kAttrPagedAttn + variant, fns[variant], smem);
  if (st != DSA_OK) return st;
  if (launch_pdl(fns[variant], grid, threads, static_cast<size_t>(smem), stream, 0, tq, tk, tv, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  const bool long_chains = 8 * items <= grid;
  const auto join = long_chains ? dsa::paged_attention_join_kernel<8> : dsa::paged_attention_join_kernel<1>;
  const int join_blocks =
      entries * (plan.rows / (long_chains ? dsa::kPaJoinHeads<8> : dsa::kPaJoinHeads<1>));
  if (launch_pdl(join, join_blocks, dsa::kPaJoinThreads, 0, stream, 0, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  return DSA_OK;
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
  *bytes = workspace_bytes_needed(plan_of(desc));
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
