"""Attention over a paged cache (all slots, or listed blocks) vs the fp64
oracle, through the C ABI (GPU only). Tolerances: paged_util.check_attention.
"""
import numpy as np
import pytest
import torch

import oracle.paged as orc
from paged_util import D, Cache, attend, bf16_bits, check_attention, dev_i32

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


@pytest.fixture(scope="module")
def dsa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_attention_lightning_tcgen05_b200 as m
    return m


def queries(rng, T, H, amp=1.0):
    return bf16_bits(rng.standard_normal((T, H, D)) * amp)


def run(dsa, cache, q, positions, *, amp=SCALE, **kw):
    """A call and its check; returns the device outputs."""
    dev, table = cache.to("cuda")
    out, lse = attend(dsa, cache, dev, table, q.cuda(), positions, amp, **kw)
    kw = {k: v for k, v in kw.items() if k in ("window", "sinks", "blocks", "block_size")} | \
        dict(seq_ids=kw.get("seq_ids"))
    ref = orc.attention(q.double().numpy(), cache.rows("k"), cache.rows("v"), cache.table,
                        positions, kw.pop("seq_ids"), amp, **kw)
    check_attention(out, lse, ref)
    return out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (5, 1), (16, 1), (17, 1), (33, 1), (64, 1),
                                   (100, 1), (128, 1), (8, 8), (64, 8), (24, 3), (96, 2)])
def test_heads(dsa, H, Hkv, fp8):
    """Every grouping of query heads over key heads; lengths that end inside
    a 16-slot step, a 64-slot tile and a page; one empty row."""
    rng = np.random.default_rng(H * 10 + Hkv)
    c = Cache(rng, 5, 3, 64, Hkv, fp8)
    run(dsa, c, queries(rng, 5, H), np.array([0, 191, -1, 70, 128]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ps", [16, 32, 64, 256])
@pytest.mark.parametrize("layout", ["slots", "heads", "gaps"])
def test_layouts_and_lengths(dsa, ps, layout, fp8):
    """Lengths 1, 15 .. 17, 63 .. 65 and past a page, one row each; a position
    past the block table sees every slot of it."""
    rng = np.random.default_rng(ps)
    pos = np.array([0, 14, 15, 16, 62, 63, 64, ps - 1, ps, 2 * ps + 3, 3 * ps - 1, 3 * ps + 500, -1, -5])
    c = Cache(rng, len(pos), 3, ps, 2, fp8, layout)
    run(dsa, c, queries(rng, len(pos), 8), pos)


@pytest.mark.parametrize("fp8", [False, True])
def test_split_rows(dsa, fp8):
    """Few long rows: every item is shared by many CTAs and joined; a short
    and an empty row between long ones."""
    rng = np.random.default_rng(3)
    c = Cache(rng, 4, 16, 256, 1, fp8)
    run(dsa, c, queries(rng, 4, 20), np.array([4095, -1, 3, 4000]),
        sinks=rng.standard_normal(20))


def test_many_rows(dsa):
    """More items than CTAs, several tokens a sequence (seq_ids), ragged."""
    rng = np.random.default_rng(4)
    c = Cache(rng, 7, 8, 16, 2)
    T = 700
    seq = rng.integers(0, 7, T)
    pos = rng.integers(-1, 128, T)
    run(dsa, c, queries(rng, T, 4), pos, seq_ids=seq)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 15, 16, 33, 100, 10 ** 9])
def test_window(dsa, window, fp8):
    rng = np.random.default_rng(window % 1000)
    pos = np.array([0, 15, 16, 31, 100, 191, 250, -1])
    c = Cache(rng, len(pos), 3, 64, 2, fp8)
    run(dsa, c, queries(rng, len(pos), 6), pos, window=window)


def test_sinks_and_growing_maximum(dsa):
    """Very large and very small sinks; logits that grow along the slots by
    far more than the lazy rescaling's 2^8."""
    rng = np.random.default_rng(5)
    c = Cache(rng, 2, 8, 64, 1)
    q = queries(rng, 2, 8)
    rows = c.rows("k")
    for i in range(2):
        flat = rows[c.table[i]].reshape(-1, D)
        order = np.argsort(flat @ q[i, 0].double().numpy())
        rows[c.table[i]] = flat[order].reshape(8, 64, 1, D)
    c.set_rows("k", rows)
    sinks = np.array([60.0, -60.0, 0.0, 5.0, -5.0, 20.0, 1.0, -1.0])
    run(dsa, c, q, np.array([511, 300]), amp=1.0, sinks=sinks)
    run(dsa, c, q, np.array([511, 300]), amp=-1.0)
    run(dsa, c, q, np.array([511, 300]), amp=0.0, sinks=sinks)


def test_large_and_tiny_queries_over_fp8(dsa):
    """The query is brought to f16's range and back: rows of 2^100, of 2^-60,
    of zeros and rows whose features span 2^24."""
    rng = np.random.default_rng(6)
    c = Cache(rng, 4, 2, 64, 1, True)
    q = rng.standard_normal((4, 4, D))
    q[1] *= 2.0 ** -60
    q[2] = 0.0
    q[3, :, ::2] *= 2.0 ** -24
    run(dsa, c, bf16_bits(q), np.array([127, 90, 100, 60]))
    big = bf16_bits(q * 2.0 ** 100)
    run(dsa, c, big, np.array([127, -1, 100, 60]), amp=SCALE * 2.0 ** -100)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool_are_masked(dsa, fp8):
    rng = np.random.default_rng(7)
    c = Cache(rng, 5, 4, 16, 2, fp8)
    c.table[0, 1] = -1
    c.table[1, :] = c.num_pages
    c.table[2, 3] = 2 ** 31 - 1
    c.table[3, 0] = -2 ** 31
    run(dsa, c, queries(rng, 5, 4), np.array([63, 63, 63, 20, 63]))
    blocks = np.array([[[0, 1, 3]]] * 5)
    run(dsa, c, queries(rng, 5, 4), np.array([63, 63, 63, 20, 63]), blocks=blocks, block_size=16)


def test_sequences_outside_the_table_are_empty(dsa):
    rng = np.random.default_rng(8)
    c = Cache(rng, 3, 2, 32, 1)
    run(dsa, c, queries(rng, 5, 3), np.array([40, 40, 40, 40, 40]),
        seq_ids=np.array([2, 3, -1, 0, 2 ** 31 - 1]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_masked_slots_hold_has_no_effect(dsa, bad):
    """Every slot that no row keeps holds NaN or an infinity, in k and v."""
    rng = np.random.default_rng(9)
    c = Cache(rng, 3, 3, 32, 2)
    pos = np.array([40, 0, 69])
    for n in ("k", "v"):
        rows = np.full((c.num_pages, 32, 2, D), bad)
        good = c.rows(n)
        for i, p in enumerate(pos):
            for s in range(p + 1):
                rows[c.table[i, s // 32], s % 32] = good[c.table[i, s // 32], s % 32]
        c.set_rows(n, rows)
    run(dsa, c, queries(rng, 3, 4), pos)
    run(dsa, c, queries(rng, 3, 4), pos, blocks=np.array([[[0, 2, 1]], [[0, 1, 2]], [[2, 0, -1]]]),
        block_size=32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [1, 2, 4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("each", [False, True])
def test_blocks(dsa, bs, each, fp8):
    """Lists of random distinct blocks in any order, -1 among them, with and
    without the recent window; blocks past the position are masked."""
    rng = np.random.default_rng(bs)
    Hkv, n = 3, max(1, 96 // bs)
    pos = np.array([255, 0, 17, -1, 130, 200])
    c = Cache(rng, len(pos), 4, 64, Hkv, fp8)
    total = 256 // bs
    blocks = np.stack([[rng.permutation(total + 2)[:n] if total + 2 >= n else
                        np.resize(rng.permutation(total + 2), n) for _ in range(Hkv if each else 1)]
                       for _ in pos]).astype(np.int64)
    blocks[rng.random(blocks.shape) < 0.15] = -1
    q = queries(rng, len(pos), 6)
    for window in (0, 1, bs, 50):
        run(dsa, c, q, pos, blocks=blocks, block_size=bs, window=window)


def test_a_block_listed_twice_counts_twice(dsa):
    rng = np.random.default_rng(11)
    c = Cache(rng, 2, 2, 64, 1)
    run(dsa, c, queries(rng, 2, 4), np.array([127, 80]), blocks=np.array([[[1, 1, 3, 1]], [[0, 4, 0, 0]]]),
        block_size=16)


def test_list_entries_out_of_range(dsa):
    """Entries far past the table, where block * block_size leaves 32 bits."""
    rng = np.random.default_rng(12)
    c = Cache(rng, 2, 2, 64, 1)
    far = 2 ** 31 - 1
    run(dsa, c, queries(rng, 2, 4), np.array([127, 2 ** 31 - 1]),
        blocks=np.array([[[far, 1, 2 ** 25]], [[0, far - 1, -far]]]), block_size=64)
    out, lse = run(dsa, c, queries(rng, 2, 4), np.array([127, 127]),
                   blocks=np.array([[[-1, -1]], [[2, 3]]]), block_size=64)
    assert torch.all(out == 0) and torch.all(lse == float("-inf"))


def test_one_list_is_the_dense_window_form(dsa):
    """Every block listed once = all slots; no block = the sliding window."""
    rng = np.random.default_rng(13)
    c = Cache(rng, 3, 4, 32, 2)
    dev, table = c.to("cuda")
    q = queries(rng, 3, 8).cuda()
    pos = np.array([127, 5, 77])
    dense = attend(dsa, c, dev, table, q, pos, SCALE)
    every = np.tile(np.arange(4), (3, 1, 1))
    a = attend(dsa, c, dev, table, q, pos, SCALE, blocks=every, block_size=32)
    assert torch.allclose(a[0].float(), dense[0].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    assert torch.allclose(a[1], dense[1], rtol=2.0 ** -16, atol=2.0 ** -16)
    b = attend(dsa, c, dev, table, q, pos, SCALE, blocks=-np.ones((3, 1, 1), np.int64), block_size=32,
               window=40)
    w = attend(dsa, c, dev, table, q, pos, SCALE, window=40)
    assert torch.allclose(b[0].float(), w[0].float(), rtol=2.0 ** -7, atol=2.0 ** -7)


def test_offsets_past_32_bits(dsa):
    """Pages 2^31 elements apart, keys and values in one buffer."""
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    rng = np.random.default_rng(14)
    c = Cache(rng, 1, 3, 16, 1, spare=0)
    c.table[:] = [[2, 0, 1]]
    buf = torch.zeros(2 * 2 ** 31 + 2 * 16 * D, dtype=torch.bfloat16, device="cuda")
    kr, vr = c.rows("k"), c.rows("v")
    for p in range(3):
        buf[p * 2 ** 31:][:16 * D] = bf16_bits(kr[p].reshape(-1)).cuda()
        buf[p * 2 ** 31 + 16 * D:][:16 * D] = bf16_bits(vr[p].reshape(-1)).cuda()
    c.strides = (2 ** 31, D, D)
    q = queries(rng, 1, 4)
    table = torch.from_numpy(c.table).cuda()
    dev = {"k": [buf, None], "v": [buf[16 * D:], None]}
    out, lse = attend(dsa, c, dev, table, q.cuda(), np.array([44]), SCALE)
    ref = orc.attention(q.double().numpy(), kr, vr, c.table, [44], None, SCALE)
    check_attention(out, lse, ref)


def test_same_bits_again_and_without_lse(dsa):
    rng = np.random.default_rng(15)
    c = Cache(rng, 3, 32, 64, 1)
    dev, table = c.to("cuda")
    q = queries(rng, 3, 64).cuda()
    pos = np.array([2047, 1500, 9])
    first = attend(dsa, c, dev, table, q, pos, SCALE)
    for _ in range(3):
        again = attend(dsa, c, dev, table, q, pos, SCALE)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    out, _ = attend(dsa, c, dev, table, q, pos, SCALE, want_lse=False)
    assert torch.equal(out, first[0])


def test_two_streams_at_once(dsa):
    """Two calls in flight on two streams, each with its own workspace."""
    rng = np.random.default_rng(16)
    c = Cache(rng, 4, 32, 64, 2)
    dev, table = c.to("cuda")
    q = queries(rng, 4, 16).cuda()
    pos = [dev_i32([2047, 1, 900, 1200]), dev_i32([100, 2000, -1, 64])]
    want = [attend(dsa, c, dev, table, q, p, SCALE) for p in pos]
    desc = dsa.make_paged_attention_desc(c.desc(dsa, table), 4, 16, SCALE)
    n = dsa.dsa_paged_attention_workspace_size(desc)
    ws = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in pos]
    got = [(torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])) for _ in pos]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            dsa.dsa_paged_attention_forward(desc, q, dev["k"][0], None, dev["v"][0], None, None, pos[i],
                                            None, got[i][0], got[i][1], ws[i], n, s.cuda_stream)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_captured_and_replayed(dsa):
    """A captured call replayed on changed positions, queries and lists."""
    rng = np.random.default_rng(17)
    c = Cache(rng, 3, 16, 64, 2)
    dev, table = c.to("cuda")
    q = queries(rng, 3, 8).cuda()
    pos, blocks = dev_i32([1000, 3, 500]), dev_i32(rng.integers(0, 16, (3, 2, 4)))
    desc = dsa.make_paged_attention_desc(c.desc(dsa, table), 3, 8, SCALE, window=8, block_size=64,
                                         num_blocks=4, block_heads=2)
    n = dsa.dsa_paged_attention_workspace_size(desc)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros((3, 8, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 8), device="cuda")

    def call():
        dsa.dsa_block_attention_forward(desc, q, dev["k"][0], None, dev["v"][0], None, None, pos, None,
                                        blocks, out, lse, ws, n, torch.cuda.current_stream().cuda_stream)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new in ([900, 1023, -1], [0, 64, 777]):
        pos.copy_(dev_i32(new))
        q.copy_(queries(rng, 3, 8).cuda())
        blocks.copy_(dev_i32(rng.integers(-1, 16, (3, 2, 4))))
        g.replay()
        torch.cuda.synchronize()
        ref = orc.attention(q.cpu().double().numpy(), c.rows("k"), c.rows("v"), c.table, new, None, SCALE,
                            window=8, blocks=blocks.cpu().numpy(), block_size=64)
        check_attention(out, lse, ref)


def test_keys_as_values(dsa):
    """One pool that is both key and value (multi-query over a latent head)."""
    rng = np.random.default_rng(18)
    c = Cache(rng, 2, 4, 64, 1)
    dev, table = c.to("cuda")
    dev["v"] = dev["k"]
    q = queries(rng, 2, 64)
    out, lse = attend(dsa, c, dev, table, q.cuda(), np.array([255, 99]), SCALE)
    ref = orc.attention(q.double().numpy(), c.rows("k"), c.rows("k"), c.table, [255, 99], None, SCALE)
    check_attention(out, lse, ref)


# ---- many query heads on a key-value head: the other kernel -------------------------
# (more than 16 over bf16, more than 48 over fp8)

@pytest.mark.parametrize("fp8,G", [(False, 17), (False, 40), (False, 128), (True, 49), (True, 128)])
@pytest.mark.parametrize("ps,layout", [(16, "slots"), (32, "gaps"), (64, "heads"), (256, "slots")])
def test_wide_layouts_and_lengths(dsa, ps, layout, fp8, G):
    """Lengths around the 32-slot units and the 128-slot tiles; empty rows; a
    position past the block table."""
    rng = np.random.default_rng(ps + G)
    pos = np.array([0, 15, 31, 32, 63, 127, 128, 129, 255, 3 * ps - 1, 3 * ps + 500, -1])
    c = Cache(rng, len(pos), max(3, 320 // ps), ps, 1 if G > 64 else 2, fp8, layout)
    run(dsa, c, queries(rng, len(pos), G * c.Hkv), pos)


@pytest.mark.parametrize("fp8,G", [(False, 20), (True, 64)])
@pytest.mark.parametrize("bs", [1, 2, 4, 8, 16, 32, 64, 256])
def test_wide_blocks(dsa, bs, fp8, G):
    rng = np.random.default_rng(bs + G)
    pos = np.array([255, 0, 17, -1, 130, 200])
    c = Cache(rng, len(pos), 4, 64, 2, fp8)
    total, n = max(1, 256 // bs), max(1, 160 // bs)
    for each in (False, True):
        blocks = np.stack([[np.resize(rng.permutation(total + 2), n) for _ in range(2 if each else 1)]
                           for _ in pos]).astype(np.int64)
        blocks[rng.random(blocks.shape) < 0.15] = -1
        for window in (0, 1, 50):
            run(dsa, c, queries(rng, len(pos), 2 * G), pos, blocks=blocks, block_size=bs, window=window)


@pytest.mark.parametrize("fp8,G", [(False, 64), (True, 64)])
def test_wide_split_rows_windows_and_sinks(dsa, fp8, G):
    """Long rows shared by many CTAs, one stream or both of them without a
    tile, short and empty rows between; windows."""
    rng = np.random.default_rng(G)
    c = Cache(rng, 5, 16, 256, 1, fp8)
    pos = np.array([4095, -1, 3, 4000, 127])
    sinks = rng.standard_normal(G)
    q = queries(rng, 5, G)
    run(dsa, c, q, pos, sinks=sinks)
    for window in (1, 100, 1000):
        run(dsa, c, q, pos, sinks=sinks, window=window)


@pytest.mark.parametrize("fp8", [False, True])
def test_wide_many_rows(dsa, fp8):
    """More items than CTAs, several tokens a sequence."""
    rng = np.random.default_rng(41)
    c = Cache(rng, 5, 16, 32, 2, fp8)
    T = 300
    run(dsa, c, queries(rng, T, 2 * 50), rng.integers(-1, 512, T), seq_ids=rng.integers(0, 5, T))


@pytest.mark.parametrize("G", [8, 64])
@pytest.mark.parametrize("amp", [1.0, -1.0, 0.0])
def test_growing_maximum(dsa, G, amp):
    """Logits that grow along the slots by far more than 2^8, over several
    tiles; a negative and a zero scale."""
    rng = np.random.default_rng(42)
    c = Cache(rng, 1, 16, 64, 1)
    q = queries(rng, 1, G)
    rows = c.rows("k")
    flat = rows[c.table[0]].reshape(-1, D)
    order = np.argsort((amp or 1.0) * (flat @ q[0, 0].double().numpy()))
    rows[c.table[0]] = flat[order].reshape(16, 64, 1, D)
    c.set_rows("k", rows)
    run(dsa, c, q, np.array([1000]), amp=amp)


@pytest.mark.parametrize("G", [8, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_masked_slots_of_a_shared_page(dsa, G, bad):
    """The rest of a token's last page, pages of nobody and blocks not listed
    hold NaN or infinities."""
    rng = np.random.default_rng(43)
    c = Cache(rng, 2, 6, 64, 1)
    pos = np.array([200, 5])
    for n in ("k", "v"):
        good, rows = c.rows(n), np.full((c.num_pages, 64, 1, D), bad)
        for i, p in enumerate(pos):
            for s in range(p + 1):
                rows[c.table[i, s // 64], s % 64] = good[c.table[i, s // 64], s % 64]
        c.set_rows(n, rows)
    run(dsa, c, queries(rng, 2, G), pos)
    run(dsa, c, queries(rng, 2, G), pos, window=70)
    run(dsa, c, queries(rng, 2, G), pos, blocks=np.array([[[3, 0, 5]], [[0, 1, -1]]]), block_size=64)


@pytest.mark.parametrize("G", [8, 64])
def test_fp8_scales_of_every_size(dsa, G):
    """Scale bytes from 1 to 254 in the values (with weights that keep the
    sums finite), zero blocks, and a NaN scale, which reaches the rows that keep
    its slot and no others."""
    rng = np.random.default_rng(44)
    c = Cache(rng, 3, 2, 64, 1, True)
    data, scale = c.pools["v"]
    per_row = scale.view(-1, 4)
    for i, s in enumerate((1, 60, 110, 134, 135, 140, 200, 240)):
        per_row[i::16] = s
    per_row[8] = 0
    data.view(-1, D)[8] = 0
    pos = np.array([127, 100, 64])
    q = queries(rng, 3, G)
    run(dsa, c, q, pos)
    # one slot of sequence 1 becomes NaN, in v and in k of another feature block
    row = int(c.at[c.table[1, 0], 7, 0]) // D
    data.view(-1, D)[row, 32:64] = 0
    per_row[row, 1] = 255
    dev, table = c.to("cuda")
    out, lse = attend(dsa, c, dev, table, q.cuda(), pos, SCALE)
    assert torch.isnan(out[1, :, 32:64]).all() and torch.isfinite(lse).all()
    other = torch.ones(D, dtype=torch.bool)
    other[32:64] = False
    assert torch.isfinite(out[1][:, other.cuda()]).all() and torch.isfinite(out[[0, 2]]).all()
    kd, ks = c.pools["k"]
    kd.view(-1, D)[row, :32] = 0
    ks.view(-1, 4)[row, 0] = 255
    dev, table = c.to("cuda")
    out, lse = attend(dsa, c, dev, table, q.cuda(), pos, SCALE)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()
    out, _ = attend(dsa, c, dev, table, q.cuda(), np.array([127, 6, 64]), SCALE)
    assert torch.isfinite(out).all()                     # slot 7 not kept


@pytest.mark.parametrize("H,fp8", [(4, False), (40, False), (4, True), (64, True)])
def test_again_and_again_between_other_calls(dsa, H, fp8):
    """Many short items a CTA, so that every buffer is filled many times over;
    between the runs a call whose keys and values are NaN goes through the same
    shared memory. The same bits every time, and right."""
    rng = np.random.default_rng(45)
    c = Cache(rng, 7, 8, 16, 2, fp8)
    T = 500
    seq, pos = rng.integers(0, 7, T), rng.integers(-1, 128, T)
    q = queries(rng, T, 2 * H)
    first = run(dsa, c, q, pos, seq_ids=seq)
    nan = Cache(rng, 40, 4, 64, 2, fill=float("nan"))
    ndev, ntable = nan.to("cuda")
    nq = queries(rng, 40, 2 * H).cuda()
    dev, table = c.to("cuda")
    qc = q.cuda()
    desc = dsa.make_paged_attention_desc(c.desc(dsa, table), T, 2 * H, SCALE)
    ndesc = dsa.make_paged_attention_desc(nan.desc(dsa, ntable), 40, 2 * H, SCALE)
    n = max(dsa.dsa_paged_attention_workspace_size(d) for d in (desc, ndesc))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out, lse, nout = torch.zeros_like(first[0]), torch.zeros_like(first[1]), torch.zeros_like(nq)
    dpos, dseq, npos = dev_i32(pos), dev_i32(seq), dev_i32([255] * 40)
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(60):
        dsa.dsa_paged_attention_forward(ndesc, nq, ndev["k"][0], None, ndev["v"][0], None, None, npos, None,
                                        nout, None, ws, n, stream)
        out.zero_()
        dsa.dsa_paged_attention_forward(desc, qc, *dev["k"], *dev["v"], None, dpos, dseq, out, lse, ws, n, stream)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert dsa.dsa_indexer_get_error(ws) == dsa.DSA_OK


@pytest.mark.parametrize("H,fp8", [(8, False), (8, True), (64, False), (64, True)])
def test_a_wait_that_runs_out_is_reported(dsa, H, fp8):
    """With a wait limit of a nanosecond some device-side wait runs out: the
    kernel records the timeout and exits; the next call is right."""
    rng = np.random.default_rng(46)
    c = Cache(rng, 4, 32, 64, 1, fp8)
    dev, table = c.to("cuda")
    q, pos = queries(rng, 4, H), np.array([2047, 2000, 1500, 900])
    desc = dsa.make_paged_attention_desc(c.desc(dsa, table), 4, H, SCALE, wait_limit_ns=1)
    n = dsa.dsa_paged_attention_workspace_size(desc)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.zeros((4, H, D), dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    dsa.dsa_paged_attention_forward(desc, q.cuda(), *dev["k"], *dev["v"], None, dev_i32(pos), None, out, None,
                                    ws, n, stream)
    status = dsa.dsa_indexer_get_error(ws, stream)
    assert status in (dsa.DSA_OK, dsa.DSA_ERR_TIMEOUT)     # OK only if nothing had to wait
    assert dsa.dsa_indexer_get_error(ws, stream) == dsa.DSA_OK
    out, lse = attend(dsa, c, dev, table, q.cuda(), pos, SCALE, workspace=ws)
    ref = orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, pos, None, SCALE)
    check_attention(out, lse, ref)


@pytest.mark.parametrize("G,fp8", [(8, False), (64, False), (8, True), (64, True)])
def test_a_kept_nan_gives_nan(dsa, G, fp8):
    """Rows whose logits are all NaN (the query, or every kept key) are not
    taken for rows without a slot, whether one CTA has them or many."""
    rng = np.random.default_rng(47)
    c = Cache(rng, 3, 80, 64, 1, fp8)
    if fp8:
        data, scale = c.pools["k"]
        idx = c.at[c.table[1, 0], 0, 0]
        data[idx:idx + 32], scale[idx // 32] = 0, 255
    else:
        rows = c.rows("k")
        rows[c.table[1, 0], 0, 0, 5] = np.nan
        c.set_rows("k", rows)
    dev, table = c.to("cuda")
    q = queries(rng, 3, G)
    q[2, 1::2, 7] = float("nan")
    out, lse = attend(dsa, c, dev, table, q.cuda(), np.array([100, 0, 5100]), SCALE)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isnan(out[2, 1::2]).all() and torch.isnan(lse[2, 1::2]).all()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2, ::2]).all() and torch.isfinite(lse[2, ::2]).all()
    out, lse = attend(dsa, c, dev, table, q.cuda(), np.array([100, 0, 5100]), SCALE,
                      blocks=np.array([[[0]], [[0]], [[1]]]), block_size=64)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all() and torch.isnan(lse[2, 1::2]).all()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2, ::2]).all()


@pytest.mark.parametrize("H", [8, 64])
def test_a_timeout_writes_no_row_of_another_call(dsa, H):
    """Where waits run out, what an earlier and larger call left in the
    workspace leads to no write past this call's rows."""
    rng = np.random.default_rng(48)
    c = Cache(rng, 4, 32, 64, 1)
    dev, table = c.to("cuda")
    q, pos = queries(rng, 4, H).cuda(), dev_i32([2047, 2000, 1500, 900])
    desc = dsa.make_paged_attention_desc(c.desc(dsa, table), 4, H, SCALE, wait_limit_ns=1)
    n = dsa.dsa_paged_attention_workspace_size(desc)
    stream = torch.cuda.current_stream().cuda_stream
    for fill in (1, 5, 0x70):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        out = torch.full((64, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        dsa.dsa_paged_attention_forward(desc, q, *dev["k"], *dev["v"], None, pos, None, out, None, ws, n, stream)
        assert dsa.dsa_indexer_get_error(ws, stream) in (dsa.DSA_OK, dsa.DSA_ERR_TIMEOUT)
        assert torch.all(out[4:] == 7.0)
