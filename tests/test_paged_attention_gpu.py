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
