"""fp64 oracle of the paged key-value cache: append, block pooling, attention.

TEST INFRASTRUCTURE. Only the tests use this module; the CUDA library never
calls it. Definitions: include/dsa_paged_cache.h and
include/dsa_paged_attention.h; the pages they cite name the parts (tokamax
Supported Ops, lightning_indexer over a paged KV cache and deepseek_rope; Sparse
Attention Indexer MX BF16Score Kernel API Reference, e4m3 data with block-32
e8m0 scales; NeMo AutoModel optimized_kernels, sparse_attention_torch,
dsv4_indexer_scores and build_dsv4_sparse_topk_indices).

A cache is float64 rows [num_pages, page_size, H_kv, D] (whatever its layout
in memory) and a block table [num_seqs, pages_per_seq].
"""
from __future__ import annotations

import numpy as np


def rope(x, cos, sin, rope_dim, halves):
    """x [..., D] with its leading rope_dim features turned in pairs; cos and
    sin [..., rope_dim/2] broadcast against x without its last axis."""
    out = np.array(x, np.float64)
    half = rope_dim // 2
    for j in range(half):
        a, b = (j, j + half) if halves else (2 * j, 2 * j + 1)
        out[..., a] = x[..., a] * cos[..., j] - x[..., b] * sin[..., j]
        out[..., b] = x[..., a] * sin[..., j] + x[..., b] * cos[..., j]
    return out


def mx_exponents(x):
    """The least e >= -127 with max|block| <= 448 * 2^e, per 32 features (by
    trying: starting low enough, doubling until it fits)."""
    top = np.abs(x).reshape(*x.shape[:-1], -1, 32).max(axis=-1)
    e = np.full(top.shape, -127)
    for _ in range(256):
        e = np.where(top > 448.0 * 2.0 ** e, e + 1, e)
    return e


def lookup(table, num_pages, page_size, seq, slot):
    """(page, slot in page) or None where the slot has no page."""
    if not (0 <= seq < table.shape[0]) or not (0 <= slot < table.shape[1] * page_size):
        return None
    page = int(table[seq, slot // page_size])
    return (page, slot % page_size) if 0 <= page < num_pages else None


def pool_blocks(k, table, start, positions, block_size, S_pool):
    """{(seq, block): mean key rows [H_kv, D]} of the completed blocks, and
    last_block per sequence. A slot without a page counts as zeros."""
    num_pages, ps = k.shape[:2]
    cap = table.shape[1] * ps
    rows, last = {}, []
    for i, p in enumerate(positions):
        n = min(int(p) + 1, cap)
        done = n // block_size if n > 0 else 0
        last.append(done - 1)
        first = 0 if start is None else max(0, int(start[i])) // block_size
        for b in range(first, min(done, S_pool)):
            total = np.zeros(k.shape[2:])
            for s in range(b * block_size, (b + 1) * block_size):
                at = lookup(table, num_pages, ps, i, s)
                if at is not None:
                    total += k[at]
            rows[i, b] = total / block_size
    return rows, last


def kept_slots(pos, capacity, window, blocks=None, block_size=1):
    """The slots a token attends to, repeated ones repeated. blocks None: all
    slots up to pos (the last `window` where window > 0)."""
    if pos < 0:
        return []
    if blocks is None:
        lo = max(0, pos - window + 1) if window > 0 else 0
        return [s for s in range(lo, pos + 1) if s < capacity]
    got = []
    for b in blocks:
        if b >= 0:
            got += [s for s in range(b * block_size, (b + 1) * block_size)
                    if s <= pos - window and s < capacity]
    return got + [s for s in range(max(0, pos - window + 1), pos + 1) if s < capacity]


def attention(q, k, v, table, positions, seq_ids, sm_scale, *, window=0, sinks=None, blocks=None,
              block_size=1):
    """q [T, H, D], k and v [num_pages, page_size, H_kv, D], blocks [T, Hb,
    n] -> out [T, H, D], lse [T, H], and what the tolerances need: the largest
    sum over features of |q k| * sm_scale and the mean |v| under the same
    weights [T, H, D]."""
    T, H, D = q.shape
    num_pages, ps, Hkv = k.shape[:3]
    G = H // Hkv
    out, wabs = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, reach = np.full((T, H), -np.inf), np.zeros((T, H))
    for t in range(T):
        seq = t if seq_ids is None else int(seq_ids[t])
        if not 0 <= seq < table.shape[0]:
            continue
        for g in range(Hkv):
            mine = None if blocks is None else [int(b) for b in blocks[t, g if blocks.shape[1] > 1 else 0]]
            slots = kept_slots(int(positions[t]), table.shape[1] * ps, window, mine, block_size)
            at = [lookup(table, num_pages, ps, seq, s) for s in slots]
            at = [a for a in at if a is not None]
            if not at:
                continue
            pg, sl = np.array(at).T
            kk, vv = k[pg, sl, g], v[pg, sl, g]
            for h in range(g * G, (g + 1) * G):
                x = kk @ q[t, h] * sm_scale
                m = x.max()
                e = np.exp(x - m)
                den = e.sum()
                lse[t, h] = m + np.log(den)
                full = den + (np.exp(sinks[h] - m) if sinks is not None else 0.0)
                out[t, h] = e @ vv / full
                wabs[t, h] = e @ np.abs(vv) / full
                reach[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * abs(sm_scale)
    return out, lse, reach, wabs
