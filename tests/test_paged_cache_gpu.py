"""The paged cache's writers (append, block pooling) vs the fp64 oracle, and
the operators run together as a decoding step uses them (GPU only).

Tolerances. A rotated feature is two products and a sum, each rounded to fp32
(half a step: 2^-24): off by at most 2^-22 (|a| + |b|); then one rounding to
bf16 (2^-8 of the value) or to e4m3 (2^-4 of the value, or half the least
subnormal step, 2^-10, under its scale). A mean of n keys: n additions of 2^-24
each of at most sum |k|, a division, and the same rounding. The scale byte is
the oracle's wherever the largest magnitude is not within that fp32 error of a
border.
"""
import numpy as np
import pytest
import torch

import oracle.paged as orc
from paged_util import D, Cache, attend, bf16_bits, check_attention, decode_mx, dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_attention_lightning_tcgen05_b200 as m
    return m


def check_rows(got, ref, slack):
    """bf16 rows against float64 ones; slack: the fp32 error."""
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + slack)


def check_mx_rows(data, scale, ref, slack):
    """e4m3 rows and their scale bytes (numpy uint8) against float64 ones."""
    e = orc.mx_exponents(ref)
    top = np.abs(ref).reshape(*ref.shape[:-1], -1, 32).max(axis=-1)
    err = slack.reshape(*ref.shape[:-1], -1, 32).max(axis=-1)
    got_e = scale.astype(np.int64) - 127
    lo, hi = top - err, top + err
    assert np.all((got_e == -127) | (hi > 448.0 * 2.0 ** (got_e - 1.0)))
    assert np.all(lo <= 448.0 * 2.0 ** got_e.astype(np.float64))
    assert np.mean(got_e != e) <= 0.01
    val = decode_mx(torch.from_numpy(data), torch.from_numpy(scale))
    step = np.repeat(2.0 ** (got_e - 10.0), 32, axis=-1)
    assert np.all(np.abs(val - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), step) + 2 * slack)


class Append:
    """One append's inputs (host) and its oracle."""

    def __init__(self, rng, cache, T, H, rope_dim, halves, positions, seq_ids=None, values=True):
        Hkv = cache.Hkv
        self.c, self.T, self.H, self.rope, self.halves = cache, T, H, rope_dim, halves
        self.pos, self.seq, self.values = np.asarray(positions), seq_ids, values
        self.q, self.k, self.v = (bf16_bits(rng.standard_normal((T, n, D))) for n in (H, Hkv, Hkv))
        ang = rng.uniform(-7, 7, (T, rope_dim // 2))
        self.cos, self.sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)

    def rotated(self, x):
        """Rotated rows and the fp32 error of each feature."""
        x = x.double().numpy()
        c, s = self.cos[:, None].astype(np.float64), self.sin[:, None].astype(np.float64)
        r = orc.rope(x, c, s, self.rope, self.halves)
        slack = np.zeros_like(x)
        half = self.rope // 2
        for j in range(half):
            a, b = (j, j + half) if self.halves else (2 * j, 2 * j + 1)
            slack[..., a] = slack[..., b] = 2.0 ** -22 * (np.abs(x[..., a]) + np.abs(x[..., b]))
        return r, slack

    def run(self, m, q_fp8=False, stream=None, packed=False):
        c, T, H, Hkv = self.c, self.T, self.H, self.c.Hkv
        self.dev, table = c.to("cuda")
        if packed:                        # one buffer of q, k and v rows with a gap
            width = (H + 2 * Hkv) * D + 8
            buf = torch.zeros((T, width), dtype=torch.bfloat16)
            for x, n, o in ((self.q, H, 0), (self.k, Hkv, H * D), (self.v, Hkv, (H + Hkv) * D)):
                buf[:, o:o + n * D] = x.reshape(T, n * D)
            buf = buf.cuda()
            q, k, v = buf, buf[:, H * D:], buf[:, (H + Hkv) * D:]
            strides = dict(q_stride=width, k_stride=width, v_stride=width)
        else:
            q, k, v, strides = self.q.cuda(), self.k.cuda(), self.v.cuda(), {}
        desc = m.make_append_desc(c.desc(m, table), T, H, self.rope, q_dtype=int(q_fp8),
                                  rope_style=m.DSA_ROPE_HALVES if self.halves else m.DSA_ROPE_INTERLEAVED,
                                  **strides)
        self.q_out = torch.full((T, H, D), 3, dtype=torch.uint8 if q_fp8 else torch.bfloat16, device="cuda")
        self.q_scale = torch.full((T, H, D // 32), 3, dtype=torch.uint8, device="cuda") if q_fp8 else None
        cos, sin = (torch.from_numpy(x).cuda() if self.rope else None for x in (self.cos, self.sin))
        kc, vc = self.dev["k"], self.dev["v"] if self.values else (None, None)
        m.dsa_cache_append(desc, q if H else None, k, v if self.values else None, cos, sin, dev_i32(self.pos),
                           None if self.seq is None else dev_i32(self.seq), self.q_out if H else None,
                           self.q_scale if H else None, kc[0], kc[1], vc[0], vc[1],
                           torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()

    def check(self, q_fp8=False):
        c = self.c
        rq, sq = self.rotated(self.q)
        rk, sk = self.rotated(self.k)
        rv = self.v.double().numpy()
        live = self.pos >= 0
        if self.H:
            if q_fp8:
                d, s = self.q_out.cpu().numpy(), self.q_scale.cpu().numpy()
                check_mx_rows(d[live], s[live], rq[live], sq[live])
                assert np.all(d[~live] == 3) and np.all(s[~live] == 3)
            else:
                got = self.q_out.double().cpu().numpy()
                check_rows(got[live], rq[live], sq[live])
                assert np.all(got[~live] == 3)
        for name, ref, slack in (("k", rk, sk), ("v", rv, np.zeros_like(rv))):
            if name == "v" and not self.values:
                continue
            data, scale = (x.cpu() if x is not None else None for x in self.dev[name])
            data = data.view(torch.uint8) if c.fp8 else data
            left_d, left_s = c.pools[name][0].clone(), c.pools[name][1]
            left_s = left_s.clone() if left_s is not None else None
            for t in range(self.T):
                at = orc.lookup(c.table, c.num_pages, c.ps, t if self.seq is None else int(self.seq[t]),
                                int(self.pos[t])) if self.pos[t] >= 0 else None
                if at is None:
                    continue
                for g in range(c.Hkv):
                    o = int(c.at[at[0], at[1], g])
                    row = slice(o, o + D)
                    if c.fp8:
                        sr = slice(o // 32, o // 32 + 4)
                        check_mx_rows(data[row].numpy(), scale[sr].numpy(), ref[t, g], slack[t, g])
                        left_s[sr] = scale[sr]
                    else:
                        check_rows(data[row].double().numpy(), ref[t, g], slack[t, g])
                    left_d[row] = data[row]
            # everything else is as it was
            assert torch.equal(left_d.view(torch.uint8), data.view(torch.uint8))
            assert left_s is None or torch.equal(left_s, scale)


def spread(rng, T, num_seqs, cap):
    """Distinct (sequence, position) of T tokens."""
    pick = rng.permutation(num_seqs * cap)[:T]
    return pick // cap, pick % cap


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_fp8", [False, True])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("rope_dim", [0, 16, 64, 96, 128])
def test_append(dsa, rope_dim, halves, q_fp8, fp8):
    rng = np.random.default_rng(rope_dim)
    c = Cache(rng, 3, 3, 16, 2, fp8, layout="heads" if halves else "slots")
    seq, pos = spread(rng, 37, 3, 48)
    pos[5], pos[36] = -1, -7
    a = Append(rng, c, 37, 5, rope_dim, halves, pos, seq)
    a.run(dsa, q_fp8, packed=rope_dim == 64)
    a.check(q_fp8)


@pytest.mark.parametrize("rope_dim", [2, 6, 30, 126])
def test_append_odd_pair_counts(dsa, rope_dim):
    """Interleaved pairs whose count is no multiple of 4."""
    rng = np.random.default_rng(rope_dim)
    c = Cache(rng, 2, 2, 32, 1)
    seq, pos = spread(rng, 9, 2, 64)
    a = Append(rng, c, 9, 3, rope_dim, False, pos, seq)
    a.run(dsa)
    a.check()


@pytest.mark.parametrize("T,H,Hkv,values", [(1, 0, 1, False), (1, 64, 8, True), (3, 1, 1, True),
                                            (300, 0, 1, False), (33, 128, 1, False), (5, 0, 7, True)])
def test_append_head_counts(dsa, T, H, Hkv, values):
    """Keys only, no queries, one token, many heads; token t of sequence t
    where there are as many sequences."""
    rng = np.random.default_rng(T)
    own = T <= 5
    c = Cache(rng, T if own else 4, 2, 128, Hkv, layout="gaps")
    seq, pos = (None, rng.integers(0, 256, T)) if own else spread(rng, T, 4, 256)
    a = Append(rng, c, T, H, 64, False, pos, seq, values)
    a.run(dsa)
    a.check()


def test_append_without_a_place(dsa):
    """Positions past the table, sequences outside it and pages outside the
    pool write no key; the token's query is written."""
    rng = np.random.default_rng(21)
    c = Cache(rng, 2, 2, 16, 1, True)
    c.table[1, 1] = -1
    c.table[0, 0] = c.num_pages
    a = Append(rng, c, 6, 2, 64, False, [31, 32, 3, 20, 20, 2 ** 31 - 1], np.array([0, 0, 0, 1, 2, -1]))
    a.run(dsa)
    a.check()


def test_append_special_values_in_fp8(dsa):
    """Zeros, the largest bf16, subnormals, and blocks with a NaN or an
    infinity, which become a NaN scale over zero data."""
    c = Cache(np.random.default_rng(0), 6, 1, 16, 1, True)
    a = Append(np.random.default_rng(22), c, 6, 0, 0, False, [3] * 6)
    x = a.k.float()
    x[0] = 0.0
    x[1] = float(torch.finfo(torch.bfloat16).max)
    x[2] = 2.0 ** -130
    x[3, :, 40] = float("nan")
    x[4, :, 100] = float("inf")
    x[5, :, :32], x[5, :, 32:64] = 448.0, 450.0          # on and just past a border
    a.k = x.to(torch.bfloat16)
    a.run(dsa)
    data, scale = a.dev["k"][0].cpu().view(torch.uint8), a.dev["k"][1].cpu()
    rows = [int(c.at[c.table[t, 0], 3, 0]) for t in range(6)]
    sc = np.stack([scale[o // 32:o // 32 + 4].numpy() for o in rows])
    val = np.stack([decode_mx(data[o:o + D], scale[o // 32:o // 32 + 4]) for o in rows])
    assert np.all(sc[0] == 0) and np.all(val[0] == 0)
    top = float(torch.finfo(torch.bfloat16).max)
    assert np.all(np.abs(val[1] - top) <= 2.0 ** -4 * top)
    assert np.all(np.abs(val[2] - 2.0 ** -130) <= 2.0 ** -137)      # half the least step under 2^-127
    assert sc[3].tolist().index(255) == 1 and np.isnan(val[3, 32:64]).all() and np.isfinite(val[3, 64:]).all()
    assert sc[4, 3] == 255 and np.isnan(val[4, 96:]).all()
    assert sc[5, 0] == 127 and np.all(val[5, :32] == 448.0)
    assert sc[5, 1] == 128 and np.all(np.abs(val[5, 32:64] - 450.0) <= 2.0 ** -4 * 450)


def test_append_in_place_queries_and_other_stream(dsa):
    rng = np.random.default_rng(23)
    c = Cache(rng, 4, 1, 16, 1)
    a = Append(rng, c, 4, 6, 128, True, [0, 5, 15, -1])
    dev, table = c.to("cuda")
    q = a.q.cuda()
    desc = dsa.make_append_desc(c.desc(dsa, table), 4, 6, 128, rope_style=dsa.DSA_ROPE_HALVES)
    cos, sin, k, v, pos = torch.from_numpy(a.cos).cuda(), torch.from_numpy(a.sin).cuda(), a.k.cuda(), \
        a.v.cuda(), dev_i32(a.pos)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    dsa.dsa_cache_append(desc, q, k, v, cos, sin, pos, None, q, None, dev["k"][0], None, dev["v"][0], None,
                         s.cuda_stream)
    s.synchronize()
    a.dev, a.q_out = dev, q.clone()
    a.q_out[3] = 3                                        # the padded token's query is as it was
    assert torch.equal(q[3], a.q.cuda()[3])
    a.check()


# ---- block pooling --------------------------------------------------------------

def run_pool(m, c, bs, S_pool, start, pos, gap=0):
    dev, table = c.to("cuda")
    head = S_pool * D + gap
    desc = m.make_block_pool_desc(c.desc(m, table), bs, S_pool, head_stride=head)
    n = c.num_seqs * c.Hkv * head
    pooled = torch.full((n,), 3, dtype=torch.uint8 if c.fp8 else torch.bfloat16, device="cuda")
    scale = torch.full((n // 32,), 3, dtype=torch.uint8, device="cuda") if c.fp8 else None
    last = torch.full((c.num_seqs, c.Hkv), -9, dtype=torch.int32, device="cuda")
    m.dsa_block_pool(desc, dev["k"][0], dev["k"][1], None if start is None else dev_i32(start), dev_i32(pos),
                     pooled, scale, last, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    rows, done = orc.pool_blocks(c.rows("k"), c.table, start, pos, bs, S_pool)
    assert np.array_equal(last.cpu().numpy(), np.repeat(np.array(done)[:, None], c.Hkv, axis=1))
    pooled, scale = pooled.cpu(), scale.cpu() if scale is not None else None
    touched = torch.zeros(n, dtype=torch.bool)
    size = np.abs(np.nan_to_num(c.rows("k"))).max()
    for (i, b), ref in rows.items():
        for g in range(c.Hkv):
            o = (i * c.Hkv + g) * head + b * D
            slack = np.full(D, (bs + 1) * 2.0 ** -24 * size)
            if c.fp8:
                check_mx_rows(pooled[o:o + D].numpy(), scale[o // 32:o // 32 + 4].numpy(), ref[g], slack)
            else:
                check_rows(pooled[o:o + D].double().numpy(), ref[g], slack)
            touched[o:o + D] = True
    assert torch.all(pooled[~touched] == 3)
    assert scale is None or torch.all(scale[~touched[::32]] == 3)
    return len(rows)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [1, 2, 3, 4, 7, 16, 32, 60, 64, 100])
def test_pool(dsa, bs, fp8):
    """Whole sequences, the blocks one step completed, empty ones; block sizes
    that divide a page, span pages and do neither."""
    rng = np.random.default_rng(bs)
    pos = np.array([191, 0, -1, 100, 63, 64, 500, 130])
    c = Cache(rng, len(pos), 6, 32, 3, fp8, layout="heads" if bs % 2 else "gaps", values=False)
    assert run_pool(dsa, c, bs, 192 // bs + 1, None, pos, gap=D) > 0
    run_pool(dsa, c, bs, max(1, 192 // bs - 1), np.array([191, 0, 5, 96, -3, 64, 180, 200]), pos)


def test_pool_one_large_block(dsa):
    rng = np.random.default_rng(31)
    c = Cache(rng, 2, 9, 256, 1, values=False)
    run_pool(dsa, c, 2048, 1, None, np.array([2303, 2046]))


@pytest.mark.parametrize("bs", [33, 64, 65536])
def test_pool_blocks_larger_than_the_table(dsa, bs):
    """No block is ever complete; the last one is still told: -1."""
    rng = np.random.default_rng(33)
    c = Cache(rng, 3, 2, 16, 2, values=False)
    assert run_pool(dsa, c, bs, 1, None, np.array([31, -1, 100])) == 0


def test_pool_pages_outside_the_pool_count_as_zeros(dsa):
    rng = np.random.default_rng(32)
    c = Cache(rng, 2, 4, 16, 2, values=False)
    c.table[0, 1], c.table[1, 3] = -1, c.num_pages
    run_pool(dsa, c, 8, 8, None, np.array([63, 63]))
    run_pool(dsa, c, 64, 1, None, np.array([63, 63]))


# ---- run together ------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
def test_a_step_from_append_to_block_attention(dsa, fp8):
    """Two steps of a batch as a server runs them: the new tokens' queries are
    rotated and their keys and values appended; the keys' blocks of 16 pooled
    (bf16 caches); the indexer scores the pooled keys with the step's queries
    and picks 4 blocks for every key head; attention runs over them and the
    last 16 slots, and over everything. Each stage is checked against the
    oracle on what the stage before left on the device."""
    rng = np.random.default_rng(41)
    B, Hkv, G, bs, n = 4, 2, 8, 16, 4
    c = Cache(rng, B, 8, 32, Hkv, fp8)
    dev, table = c.to("cuda")
    for n_ in dev:
        c.pools[n_] = dev[n_]                              # the oracle reads the device's rows
    S_pool = 256 // bs
    pooled = torch.zeros((B, Hkv, S_pool, D), dtype=torch.bfloat16, device="cuda")
    last = torch.zeros((B, Hkv), dtype=torch.int32, device="cuda")
    start = np.zeros(B, np.int64)
    for pos in (np.array([200, 63, 10, 127]), np.array([201, 64, 11, 128])):
        H = Hkv * G
        q, k, v = (bf16_bits(rng.standard_normal((B, h, D))).cuda() for h in (H, Hkv, Hkv))
        ang = pos[:, None] * 10000.0 ** (-np.arange(32) / 32)
        cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).cuda() for f in (np.cos, np.sin))
        dpos = dev_i32(pos)
        stream = torch.cuda.current_stream().cuda_stream
        ad = dsa.make_append_desc(c.desc(dsa, table), B, H, 64)
        dsa.dsa_cache_append(ad, q, k, v, cos, sin, dpos, None, q, None, *dev["k"], *dev["v"], stream)
        kr = c.rows("k")
        ref_k = orc.rope(k.double().cpu().numpy(), np.cos(ang).astype(np.float32)[:, None],
                         np.sin(ang).astype(np.float32)[:, None], 64, False)
        for i in range(B):
            got = kr[c.table[i, pos[i] // 32], pos[i] % 32]
            assert np.all(np.abs(got - ref_k[i]) <= (2.0 ** -4 if fp8 else 2.0 ** -8) * np.abs(ref_k[i]).max())
        if not fp8:
            pd = dsa.make_block_pool_desc(c.desc(dsa, table), bs, S_pool)
            dsa.dsa_block_pool(pd, *dev["k"], dev_i32(start), dpos, pooled, None, last, stream)
            start = pos + 1
            # the indexer over one row per (sequence, key head)
            w = torch.full((B * Hkv, G), 1.0 / G, device="cuda")
            idesc = dsa.make_desc(B * Hkv, G, n, S=S_pool, k_seq_stride=S_pool * D)
            scores = torch.zeros((B * Hkv, S_pool), device="cuda")
            top = torch.full((B * Hkv, n), -7, dtype=torch.int32, device="cuda")
            iws = torch.zeros(dsa.dsa_indexer_workspace_size(idesc), dtype=torch.uint8, device="cuda")
            dsa.dsa_indexer_forward(idesc, q, None, w, pooled, None, last, scores, top, iws, iws.numel(), stream)
            assert dsa.dsa_indexer_get_error(iws) == dsa.DSA_OK
            rows, _ = orc.pool_blocks(kr, c.table, None, pos, bs, S_pool)
            lists = top.cpu().numpy().reshape(B, Hkv, n)
            qn = q.double().cpu().numpy().reshape(B, Hkv, G, D)
            for i in range(B):
                done = (pos[i] + 1) // bs
                for g in range(Hkv):
                    s = np.array([np.maximum(qn[i, g] @ rows[i, b][g], 0).mean() for b in range(done)])
                    mine = [b for b in lists[i, g] if b >= 0]
                    assert len(set(mine)) == len(mine) == min(n, done)
                    tol = 2e-2 * (np.abs(s).max() if done else 0)
                    rest = [s[b] for b in range(done) if b not in mine]
                    assert not rest or min(s[b] for b in mine) >= max(rest) - tol
        else:
            lists = np.stack([[rng.permutation(max(n, p // bs + 1))[:n] for _ in range(Hkv)] for p in pos])
        out, lse = attend(dsa, c, dev, table, q, dpos, D ** -0.5, blocks=lists, block_size=bs, window=bs)
        qn = q.double().cpu().numpy()
        check_attention(out, lse, orc.attention(qn, kr, c.rows("v"), c.table, pos, None, D ** -0.5,
                                                window=bs, blocks=lists, block_size=bs))
        out, lse = attend(dsa, c, dev, table, q, dpos, D ** -0.5)
        check_attention(out, lse, orc.attention(qn, kr, c.rows("v"), c.table, pos, None, D ** -0.5))


def test_the_indexer_reads_appended_fp8_pages(dsa):
    """The front end's queries and keys, quantised by the append into e4m3
    queries and the indexer's paged fp8 cache, scored and selected there."""
    rng = np.random.default_rng(42)
    T, H, L, k_top = 3, 8, 100, 16
    c = Cache(rng, T, 2, 64, 1, True, values=False)
    dev, table = c.to("cuda")
    seq = np.repeat(np.arange(T), L)
    pos = np.tile(np.arange(L), T)
    keys = bf16_bits(rng.standard_normal((T * L, 1, D))).cuda()
    stream = torch.cuda.current_stream().cuda_stream
    kd = dsa.make_append_desc(c.desc(dsa, table), T * L, 0, 0)
    dsa.dsa_cache_append(kd, None, keys, None, None, None, dev_i32(pos), dev_i32(seq), None, None,
                         *dev["k"], None, None, stream)
    # the step's own token: its key at slot L, its query quantised
    q, k1 = bf16_bits(rng.standard_normal((T, H, D))).cuda(), bf16_bits(rng.standard_normal((T, 1, D))).cuda()
    q8 = torch.zeros((T, H, D), dtype=torch.uint8, device="cuda")
    qs = torch.zeros((T, H, D // 32), dtype=torch.uint8, device="cuda")
    last = dev_i32([L] * T)
    sd = dsa.make_append_desc(c.desc(dsa, table), T, H, 0, q_dtype=dsa.DSA_KV_FP8_E4M3_E8M0_B32)
    dsa.dsa_cache_append(sd, q, k1, None, None, None, last, None, q8, qs, *dev["k"], None, None, stream)
    w = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    idesc = dsa.make_desc(T, H, k_top, S=128, dtype=dsa.DSA_KV_FP8_E4M3_E8M0_B32, page_size=64,
                          pages_per_seq=2, num_pages=c.num_pages, block_table=table)
    scores = torch.zeros((T, 128), device="cuda")
    top = torch.zeros((T, k_top), dtype=torch.int32, device="cuda")
    ws = torch.zeros(dsa.dsa_indexer_workspace_size(idesc), dtype=torch.uint8, device="cuda")
    dsa.dsa_indexer_forward(idesc, q8, qs, w, dev["k"][0], dev["k"][1], last, scores, top, ws, ws.numel(), stream)
    assert dsa.dsa_indexer_get_error(ws) == dsa.DSA_OK
    qv = decode_mx(q8.cpu(), qs.cpu())
    kv = c.rows("k", dev)
    for t in range(T):
        mine = kv[c.table[t]].reshape(-1, D)[:L + 1]
        ref = (np.maximum(qv[t] @ mine.T, 0) * w[t].cpu().double().numpy()[:, None]).sum(axis=0)
        got = scores[t, :L + 1].double().cpu().numpy()
        assert np.abs(got - ref).max() <= 6e-2 * np.abs(ref).max()
        exact = np.maximum(q[t].double().cpu().numpy() @ np.concatenate(
            [keys[t * L:(t + 1) * L, 0].double().cpu().numpy(), k1[t].double().cpu().numpy()]).T, 0)
        exact = (exact * w[t].cpu().double().numpy()[:, None]).sum(axis=0)
        assert np.abs(ref - exact).max() <= 0.2 * np.abs(exact).max()       # quantisation alone
        assert set(top[t].cpu().tolist()) == set(np.argsort(-got, kind="stable")[:k_top].tolist())


# ---- many items, many sequences, far offsets, one graph ------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [3, 4])
def test_pool_more_sequences_than_are_counted_at_once(dsa, bs, fp8):
    """2,500 sequences of up to 32 slots."""
    rng = np.random.default_rng(34)
    c = Cache(rng, 2500, 2, 16, 1, fp8, values=False)
    pos = rng.integers(-1, 32, 2500)
    assert run_pool(dsa, c, bs, 32 // bs, np.maximum(0, pos - rng.integers(0, 9, 2500)), pos) > 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [64, 100, 512])
def test_pool_many_turns_a_block_of_threads(dsa, bs, fp8):
    """More shared items than the GPU takes at once, twice to the same bits."""
    rng = np.random.default_rng(35)
    n, pages, ps, Hkv = 2, 1024, 128, 2
    g = torch.Generator(device="cuda").manual_seed(35)
    x = torch.randn((n * pages, ps, Hkv, D), generator=g, device="cuda")
    table = torch.from_numpy(rng.permutation(n * pages).astype(np.int32).reshape(n, pages)).cuda()
    if fp8:
        data = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        scale = torch.randint(119, 122, data.shape[:-1] + (D // 32,), generator=g, device="cuda", dtype=torch.uint8)
        rows = data.double() * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=-1)
    else:
        data, scale = x.bfloat16(), None
        rows = data.double()
    cache = dsa.make_paged_cache(ps, pages, n * pages, table, num_seqs=n, H_kv=Hkv,
                                 dtype=dsa.DSA_KV_FP8_E4M3_E8M0_B32 if fp8 else dsa.DSA_KV_BF16)
    S_pool = pages * ps // bs
    last = [pages * ps - 1, 100001]
    desc = dsa.make_block_pool_desc(cache, bs, S_pool)
    got = []
    for _ in range(2):
        pooled = torch.zeros((n, Hkv, S_pool, D), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
        ps_ = torch.zeros((n, Hkv, S_pool, D // 32), dtype=torch.uint8, device="cuda") if fp8 else None
        dsa.dsa_block_pool(desc, data, scale, None, dev_i32(last), pooled, ps_, None,
                           torch.cuda.current_stream().cuda_stream)
        got.append((pooled, ps_))
    assert torch.equal(got[0][0], got[1][0]) and (not fp8 or torch.equal(got[0][1], got[1][1]))
    for i, p in enumerate(last):
        done = (p + 1) // bs
        mine = rows[table[i].long()].flatten(0, 1)[:done * bs].unflatten(0, (done, bs))
        ref = mine.mean(dim=1).transpose(0, 1).cpu().numpy()
        slack = np.full(ref.shape, (bs + 1) * 2.0 ** -24 * float(mine.abs().max()))
        if fp8:
            check_mx_rows(got[0][0][i, :, :done].cpu().numpy(), got[0][1][i, :, :done].cpu().numpy(), ref, slack)
        else:
            check_rows(got[0][0][i, :, :done].double().cpu().numpy(), ref, slack)
        assert not got[0][0][i, :, done:].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_append_and_pool_past_32_bit_offsets(dsa, fp8):
    """Pages 2^31 elements apart: keys appended there, and their blocks pooled."""
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    rng = np.random.default_rng(36)
    ps, far, L = 16, 2 ** 31, 45
    size = 2 * far + ps * D
    kp = torch.zeros(size, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    ks = torch.zeros(size // 32, dtype=torch.uint8, device="cuda") if fp8 else None
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    cache = dsa.make_paged_cache(ps, 3, 3, table, num_seqs=1, page_stride=far,
                                 dtype=dsa.DSA_KV_FP8_E4M3_E8M0_B32 if fp8 else dsa.DSA_KV_BF16)
    k = bf16_bits(rng.standard_normal((L, 1, D)))
    stream = torch.cuda.current_stream().cuda_stream
    dsa.dsa_cache_append(dsa.make_append_desc(cache, L, 0, 0), None, k.cuda(), None, None, None,
                         dev_i32(np.arange(L)), dev_i32(np.zeros(L)), None, None, kp, ks, None, None, stream)
    at = [([2, 0, 1][p // ps]) * far + p % ps * D for p in range(L)]
    ref = k[:, 0].double().numpy()
    data = torch.stack([kp[o:o + D] for o in at]).cpu()
    if fp8:
        scale = torch.stack([ks[o // 32:o // 32 + 4] for o in at]).cpu()
        check_mx_rows(data.numpy(), scale.numpy(), ref, np.zeros_like(ref))
        rows = decode_mx(data, scale)
    else:
        assert torch.equal(data, k[:, 0])
        rows = ref
    pooled = torch.zeros((11, D), dtype=kp.dtype, device="cuda")
    pscale = torch.zeros((11, D // 32), dtype=torch.uint8, device="cuda") if fp8 else None
    dsa.dsa_block_pool(dsa.make_block_pool_desc(cache, 4, 11), kp, ks, None, dev_i32([L - 1]), pooled, pscale,
                       None, stream)
    mean = rows[:44].reshape(11, 4, D).mean(axis=1)
    slack = np.full(mean.shape, 5 * 2.0 ** -24 * np.abs(rows).max())
    if fp8:
        check_mx_rows(pooled.cpu().numpy(), pscale.cpu().numpy(), mean, slack)
    else:
        check_rows(pooled.double().cpu().numpy(), mean, slack)


def test_a_whole_step_in_one_graph(dsa):
    """Append, pooling, the indexer, attention over its blocks and over all
    slots captured once, replayed for the next steps' positions, queries and
    keys: each attention against the oracle on the rows then in the cache."""
    rng = np.random.default_rng(43)
    B, Hkv, G, bs, n, ps = 4, 2, 8, 16, 4, 32
    H, S_pool = Hkv * G, 256 // bs
    c = Cache(rng, B, 8, ps, Hkv)
    dev, table = c.to("cuda")
    for name in dev:
        c.pools[name] = dev[name]
    q, k, v = (torch.zeros((B, h, D), dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    qr = torch.zeros_like(q)
    cos, sin = torch.zeros((B, 32), device="cuda"), torch.zeros((B, 32), device="cuda")
    pos, start = dev_i32([0] * B), dev_i32([0] * B)
    pooled = torch.zeros((B, Hkv, S_pool, D), dtype=torch.bfloat16, device="cuda")
    last = torch.zeros((B, Hkv), dtype=torch.int32, device="cuda")
    w = torch.full((B * Hkv, G), 1.0 / G, device="cuda")
    scores = torch.zeros((B * Hkv, S_pool), device="cuda")
    top = torch.full((B, Hkv, n), -1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    lses = [torch.zeros((B, H), device="cuda") for _ in range(2)]
    cache = c.desc(dsa, table)
    ad = dsa.make_append_desc(cache, B, H, 64)
    pd = dsa.make_block_pool_desc(cache, bs, S_pool)
    idesc = dsa.make_desc(B * Hkv, G, n, S=S_pool, k_seq_stride=S_pool * D)
    iws = torch.zeros(dsa.dsa_indexer_workspace_size(idesc), dtype=torch.uint8, device="cuda")
    bd = dsa.make_paged_attention_desc(cache, B, H, D ** -0.5, window=bs, block_size=bs, num_blocks=n,
                                       block_heads=Hkv)
    dd = dsa.make_paged_attention_desc(cache, B, H, D ** -0.5)
    ws_bytes = max(dsa.dsa_paged_attention_workspace_size(x) for x in (bd, dd))
    ws = torch.zeros(ws_bytes, dtype=torch.uint8, device="cuda")

    def step():
        s = torch.cuda.current_stream().cuda_stream
        dsa.dsa_cache_append(ad, q, k, v, cos, sin, pos, None, qr, None, *dev["k"], *dev["v"], s)
        dsa.dsa_block_pool(pd, *dev["k"], start, pos, pooled, None, last, s)
        dsa.dsa_indexer_forward(idesc, qr, None, w, pooled, None, last, scores, top, iws, iws.numel(), s)
        dsa.dsa_block_attention_forward(bd, qr, *dev["k"], *dev["v"], None, pos, None, top, outs[0], lses[0],
                                        ws, ws_bytes, s)
        dsa.dsa_paged_attention_forward(dd, qr, *dev["k"], *dev["v"], None, pos, None, outs[1], lses[1],
                                        ws, ws_bytes, s)

    def fill(at):
        for x in (q, k, v):
            x.copy_(bf16_bits(rng.standard_normal(tuple(x.shape))))
        ang = at[:, None] * 10000.0 ** (-np.arange(32) / 32)
        cos.copy_(torch.from_numpy(np.cos(ang).astype(np.float32)))
        sin.copy_(torch.from_numpy(np.sin(ang).astype(np.float32)))
        pos.copy_(dev_i32(at))

    at = np.array([200, 63, 10, 127])
    fill(at)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        start.copy_(dev_i32(at + 1))
        at = at + 1
        fill(at)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert dsa.dsa_indexer_get_error(ws) == dsa.DSA_OK and dsa.dsa_indexer_get_error(iws) == dsa.DSA_OK
        kr, vr, qn = c.rows("k"), c.rows("v"), qr.double().cpu().numpy()
        for i in range(B):
            assert torch.equal(torch.from_numpy(vr[c.table[i, at[i] // ps], at[i] % ps]), v[i].double().cpu())
        done = (at + 1) // bs
        assert np.array_equal(last.cpu().numpy(), np.repeat(done[:, None] - 1, Hkv, axis=1))
        lists = top.cpu().numpy()
        for i in range(B):
            for g in range(Hkv):
                mine = [b for b in lists[i, g] if b >= 0]
                assert len(set(mine)) == len(mine) == min(n, done[i]) and all(b < done[i] for b in mine)
        check_attention(outs[0], lses[0], orc.attention(qn, kr, vr, c.table, at, None, D ** -0.5, window=bs,
                                                        blocks=lists, block_size=bs))
        check_attention(outs[1], lses[1], orc.attention(qn, kr, vr, c.table, at, None, D ** -0.5))
