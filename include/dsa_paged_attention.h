/*
 * dsa_paged_attention.h -- C ABI of attention over a paged key-value cache in
 * libdsa_indexer, for NVIDIA B200 (sm_100a): each query token over all slots
 * of its sequence (decoding), or over the blocks of slots listed for it.
 *
 * For query token t at position p = positions[t] of sequence i = seq_ids[t],
 * head h and its key-value head g = h / (H / H_kv):
 *     l_s = sm_scale * q[t, h, :] . k(i, s, g)          for every kept slot s
 *                      (the product of q and k in fp32, within its range)
 *     lse[t, h]    = ln sum_s e^{l_s}
 *     out[t, h, :] = sum_s e^{l_s} v(i, s, g) / (sum_s e^{l_s} + e^{sinks[h]})
 * The kept slots:
 *   dsa_paged_attention_forward: 0 <= s <= p, and s > p - window where
 *     window > 0;
 *   dsa_block_attention_forward: the slots s <= p - window of every listed
 *     block b, s in [b * block_size, (b + 1) * block_size), and the last
 *     window slots p - window < s <= p. A listed block that is negative is
 *     masked, and so are slots past p; a block listed twice counts twice. The
 *     recent slots are there besides the list, and never counted twice: an
 *     indexer over pooled keys lists complete blocks, and a window of at
 *     least block_size covers the open one.
 * A slot past the block table, or in a page outside the pool, is not kept. A
 * token with no kept slot (a negative position, a sequence outside
 * [0, num_seqs), a list of -1) gets out = 0 and lse = -infinity, as does one
 * whose kept slots all have the logit -infinity. What masked slots hold, NaN
 * and infinities among it, has no effect; a NaN that is kept gives NaN, and beside
 * other slots so may an infinite value whose weight is 0. A weight
 * e^{l_s} takes part as a bf16 number relative to its row's largest (one below
 * 2^-126 of that may count as 0), and over an fp8 cache under up to 48 heads so
 * does its product with the value's scale, so that scales below 2^-107 lose bits
 * of small weights; sums are fp32, of weights up to 2^8 times the final largest
 * one: values of 2^100 and more may make them overflow.
 *
 * Where the operation is defined (page titles and sections):
 *  - NeMo AutoModel optimized_kernels, sparse_attention_torch and
 *    dense_attention_topk_torch: per-head sink logits, -1 masks an index;
 *    build_dsv4_sparse_topk_indices: a window of recent tokens beside the
 *    selected compressed ones.
 *  - tokamax Supported Ops, lightning_indexer: a paged KV cache.
 *  - Sparse Attention Indexer MX BF16Score Kernel API Reference: e4m3 caches
 *    with block-32 e8m0 scales.
 *
 * Conventions are those of dsa_indexer.h (device pointers of the current
 * device, no allocation, host-side checks before any launch, asynchronous on
 * `stream`, a workspace of one call at a time, bounded device-side waits
 * reported by dsa_indexer_get_error; after a reported timeout `out` and `lse`
 * are unspecified and the workspace can be used again). Results do not depend
 * on the order in which blocks of the GPU finish: the same call gives the same
 * bits.
 */
#ifndef DSA_PAGED_ATTENTION_H
#define DSA_PAGED_ATTENTION_H

#include "dsa_paged_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  dsa_paged_cache_t cache;
  int32_t T;               /* query tokens, >= 1                                */
  int32_t H;               /* query heads: a multiple of H_kv, with
                              H / H_kv <= 128 and T * H < 2^31                  */
  float sm_scale;          /* logit scale, |sm_scale| < 2^127                   */
  int32_t window;          /* recent slots, >= 0 (see above)                    */
  int32_t block_size;      /* block attention: slots a block, a power of two in
                              [1, 65536]; otherwise unused                      */
  int32_t num_blocks;      /* block attention: list entries, >= 1, with
                              num_blocks * block_size + window < 2^30; 0 where
                              the descriptor serves attention over all slots    */
  int32_t block_heads;     /* block attention: 1 (one list for every head) or
                              H_kv (one for each key-value head)                */
  uint32_t flags;          /* 0, or DSA_FLAG_SELFTEST_STALL (dsa_indexer.h): a
                              warp keeps back an arrival that others wait for, so
                              that the wait limit runs out and is reported       */
  uint64_t wait_limit_ns;  /* device-side wait limit; 0 = the default, 4 s      */
} dsa_paged_attention_desc_t;

/*
 * Layouts (row-major, innermost index last):
 *  q          [T, H, D] bf16                               (16-byte aligned)
 *  k, v       the pools of the cache (v may be k)          (16-byte aligned)
 *  k_scale, v_scale   the scale pools (fp8 only, else NULL; 4-byte aligned)
 *  sinks      [H] fp32, or NULL: none
 *  positions  [T] int32
 *  seq_ids    [T] int32, or NULL: token t belongs to sequence t
 *  blocks     [T, block_heads, num_blocks] int32 (e.g. the indexer's top-k)
 *  out        [T, H, D] bf16                               (16-byte aligned)
 *  lse        [T, H] fp32, or NULL
 */

/* Bytes of workspace a call needs (host only): the 256-byte header and the
 * partial results of rows whose slots are split over the GPU. 256-byte
 * aligned, zero-filled once before first use, reused freely by attention calls
 * (of any descriptor that it is large enough for) ordered on one stream. A
 * descriptor with num_blocks = 0 is checked as one of attention over all
 * slots. */
dsa_status_t dsa_paged_attention_workspace_size(const dsa_paged_attention_desc_t *desc,
                                                size_t *bytes);

/* Attention over all slots of each token's sequence (the last `window` ones
 * where window > 0). */
dsa_status_t dsa_paged_attention_forward(const dsa_paged_attention_desc_t *desc, const void *q,
                                         const void *k, const uint8_t *k_scale, const void *v,
                                         const uint8_t *v_scale, const float *sinks,
                                         const int32_t *positions, const int32_t *seq_ids,
                                         void *out, float *lse, void *workspace,
                                         size_t workspace_bytes, dsa_stream_t stream);

/* Attention over each token's listed blocks and its last `window` slots. */
dsa_status_t dsa_block_attention_forward(const dsa_paged_attention_desc_t *desc, const void *q,
                                         const void *k, const uint8_t *k_scale, const void *v,
                                         const uint8_t *v_scale, const float *sinks,
                                         const int32_t *positions, const int32_t *seq_ids,
                                         const int32_t *blocks, void *out, float *lse,
                                         void *workspace, size_t workspace_bytes,
                                         dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_PAGED_ATTENTION_H */
