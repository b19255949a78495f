/*
 * dsa_paged_cache.h -- C ABI of the paged key-value cache of libdsa_indexer,
 * for NVIDIA B200 (sm_100a): appending a step's keys and values (rotated by
 * their positions, bf16 or fp8) to the pages a block table names, and pooling
 * completed blocks of keys for the compressed indexer.
 *
 * dsa_cache_append, per token t with position p = positions[t] and sequence
 * i = seq_ids[t]:
 *     q_out[t, h, :]        = rope(q[t, h, :], t)
 *     k cache (i, p, g)     = rope(k[t, g, :], t)
 *     v cache (i, p, g)     = v[t, g, :]
 * where cache (i, p, g) is the row of head g at slot p % page_size of page
 * block_table[i, p / page_size]. rope(x, t) turns rope_dim leading features
 * in pairs, by the angle whose cosine and sine are cos[t, j], sin[t, j],
 * j < rope_dim/2: (a, b) -> (a cos - b sin, a sin + b cos), computed in fp32
 * (each product and the sum rounded), where (a, b) is (x[2j], x[2j+1])
 * (DSA_ROPE_INTERLEAVED) or (x[j], x[j + rope_dim/2]) (DSA_ROPE_HALVES).
 * An fp8 row holds, per 32 features, the byte e + 127 of the least power of
 * two 2^e (e >= -127) with max|x| <= 448 * 2^e, and x * 2^-e rounded to the
 * nearest e4m3, ties to even; 32 features that hold a NaN or an infinity get
 * the scale byte 255, which stands for NaN, and zero data. An fp8 cache that
 * other code wrote has to keep to that: NaN by the scale byte and zero data,
 * not by e4m3's NaN codes (0x7f, 0xff). A scale byte 0 (2^-127) may be read as 0.
 *
 * dsa_block_pool, per sequence i with last position p = positions[i] and
 * first new position s = start[i], for every block b of block_size slots that
 * the new tokens completed, s / block_size <= b < (p + 1) / block_size:
 *     pooled[i, g, b, :] = (1 / block_size) sum over its slots of k cache
 * rounded once to the cache's type, and last_block[i, g] = (p + 1) /
 * block_size - 1, the last complete block (-1: none). The pooled rows are a
 * key cache that dsa_indexer_forward scores: with one row per (sequence,
 * head), positions = last_block (DSA_MASK_POSITIONS, k_seq_stride =
 * head_stride where the rows are evenly spaced, for an fp8 cache a multiple of
 * 512 as the indexer has it); for one sequence's prefill,
 * DSA_MASK_COMPRESSED with compress_ratio = block_size. Its index sets are
 * block lists of dsa_block_attention_forward (dsa_paged_attention.h).
 *
 * Where the operations are defined (page titles and sections):
 *  - tokamax Supported Ops, lightning_indexer: the scores run over a paged KV
 *    cache; deepseek_rope: DeepSeek's RoPE is interleaved.
 *  - DeepSeek-V3.2 Sparse Indexer Kernel API Reference,
 *    deepseek_v32_sparse_indexer, Parameters: key_cache written in place at
 *    each token's current position; cos / sin [n_tokens, rope_dim // 2].
 *  - Sparse Attention Indexer MX BF16Score Kernel API Reference: e4m3 data
 *    with block-32 e8m0 scales; k_cache and k_scale_cache.
 *  - NeMo AutoModel optimized_kernels, dsv4_indexer_scores: pooled keys, each
 *    of compress_ratio raw tokens.
 *
 * Conventions are those of dsa_indexer.h (device pointers of the current
 * device, no allocation, host-side checks before any launch, asynchronous on
 * `stream`). These calls have no device-side waits and need no workspace:
 * calls on different streams may overlap unless they write the same rows.
 */
#ifndef DSA_PAGED_CACHE_H
#define DSA_PAGED_CACHE_H

#include "dsa_indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Where a paged cache keeps head g's row of slot p of sequence i: with page
 * = block_table[i * pages_per_seq + p / page_size] and slot = p % page_size,
 * at element page * page_stride + slot * slot_stride + g * head_stride of the
 * pool. The key and the value pool share the strides. fp8: the scale pools
 * hold the row's D/32 bytes at 1/32 of that element offset. A table entry
 * outside [0, num_pages) names no page: nothing is written to its slots, and
 * they take no part in what is read. */
typedef struct {
  int32_t num_seqs;        /* rows of block_table, >= 1                         */
  int32_t H_kv;            /* key-value heads, 1 .. 128                         */
  int32_t D;               /* head dim; must be 128                             */
  int32_t page_size;       /* slots a page, a power of two in [16, 65536]       */
  int32_t pages_per_seq;   /* block-table entries a sequence, >= 1, with
                              pages_per_seq * page_size < 2^31                  */
  int32_t num_pages;       /* pages of the pools, >= 1, with
                              num_pages * page_size < 2^31                      */
  dsa_kv_dtype_t dtype;    /* of the key and value pools                        */
  int64_t page_stride;     /* elements, multiples of 128, > 0: between pages,   */
  int64_t slot_stride;     /* between the slots of a page                       */
  int64_t head_stride;     /* and between the heads of a slot (for attention
                              below 2^39)                                       */
  const int32_t *block_table; /* device [num_seqs, pages_per_seq]               */
} dsa_paged_cache_t;

typedef enum {
  DSA_ROPE_INTERLEAVED = 0,  /* pairs (x[2j], x[2j+1])                          */
  DSA_ROPE_HALVES = 1        /* pairs (x[j], x[j + rope_dim/2])                 */
} dsa_rope_t;

typedef struct {
  dsa_paged_cache_t cache;
  int32_t T;               /* tokens, >= 1, with T * (H + 2 H_kv + 3) < 2^29    */
  int32_t H;               /* query heads to rotate, 0 .. 256 (0: none)         */
  int32_t rope_dim;        /* leading features turned, 0 .. D: even
                              (INTERLEAVED) or a multiple of 16 (HALVES)        */
  dsa_rope_t rope;
  dsa_kv_dtype_t q_dtype;  /* of q_out                                          */
  int64_t q_stride;        /* elements between consecutive tokens' inputs,      */
  int64_t k_stride;        /* multiples of 8, at least heads * D                */
  int64_t v_stride;
} dsa_append_desc_t;

/*
 * Layouts (innermost index last):
 *  q, k, v    token t's heads [heads, D] at element t * stride, bf16
 *                                                          (16-byte aligned)
 *  cos, sin   [T, rope_dim/2] fp32 (may be NULL when rope_dim = 0)
 *  positions  [T] int32; a negative position marks a padded token, of which
 *             nothing is written
 *  seq_ids    [T] int32, or NULL: token t belongs to sequence t
 *  q_out      [T, H, D] bf16, or e4m3 with q_scale [T, H, D/32] e8m0
 *                                                          (16-byte aligned)
 *  k_cache, v_cache    the pools                           (16-byte aligned)
 *  k_scale, v_scale    the scale pools (fp8 only, else NULL; 4-byte aligned)
 * q = NULL exactly when H = 0; v = NULL with v_cache = NULL appends keys
 * only. q_out may be q itself when q_dtype is bf16 and q_stride = H * D.
 * A position past the block table's slots, a sequence outside [0, num_seqs)
 * or a page outside the pool writes no key and no value (the token's query
 * is written all the same). Tokens of one call that name the same slot leave
 * one of their rows there, or parts of several: give each its own slot. The
 * inputs overlap no output but for that q_out.
 */
dsa_status_t dsa_cache_append(const dsa_append_desc_t *desc, const void *q, const void *k,
                              const void *v, const float *cos, const float *sin,
                              const int32_t *positions, const int32_t *seq_ids, void *q_out,
                              uint8_t *q_scale, void *k_cache, uint8_t *k_scale, void *v_cache,
                              uint8_t *v_scale, dsa_stream_t stream);

typedef struct {
  dsa_paged_cache_t cache;
  int32_t block_size;      /* slots a block, 1 .. 65536                         */
  int64_t S_pool;          /* pooled rows per (sequence, head), 1 .. 2^31 - 1:
                              a block at or past it writes nothing              */
  int64_t seq_stride;      /* elements between sequences' pooled rows and       */
  int64_t head_stride;     /* between heads'; multiples of 128, >= 0            */
} dsa_block_pool_desc_t;

/*
 *  k_cache, k_scale     as in dsa_cache_append
 *  start      [num_seqs] int32, or NULL: from the first block on; a negative
 *             start is 0
 *  positions  [num_seqs] int32: each sequence's last position (negative: no
 *             block); one past the block table's slots counts as the last slot
 *  pooled     block b of (sequence i, head g) at element i * seq_stride +
 *             g * head_stride + b * D, the cache's type    (16-byte aligned)
 *  pooled_scale  fp8: the rows' D/32 bytes at 1/32 of that offset (4-byte
 *             aligned); NULL for bf16
 *  last_block [num_seqs, H_kv] int32, or NULL
 * A slot of a page outside the pool counts as a zero key.
 */
dsa_status_t dsa_block_pool(const dsa_block_pool_desc_t *desc, const void *k_cache,
                            const uint8_t *k_scale, const int32_t *start,
                            const int32_t *positions, void *pooled, uint8_t *pooled_scale,
                            int32_t *last_block, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_PAGED_CACHE_H */
