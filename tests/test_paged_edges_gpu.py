"""Edges of attention over a paged cache and of the cache's writers, each
against the fp64 oracle (GPU only). Tolerances: paged_util.check_attention, and
what a test derives beside it.
"""
import numpy as np
import pytest
import torch

import oracle.paged as orc
from paged_scales import POSITIONS, scaled_cache
from paged_util import D, Cache, attend, bf16_bits, check_attention, decode_mx, dev_i32

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


@pytest.fixture(scope="module")
def dsa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_attention_lightning_tcgen05_b200 as m
    return m


def queries(rng, T, H, amp=1.0):
    return bf16_bits(rng.standard_normal((T, H, D)) * amp)


@pytest.mark.parametrize("H,fp8,ps", [(128, False, 64), (64, True, 32), (8, True, 16), (8, False, 16)])
def test_the_last_slots_of_the_longest_sequence(dsa, H, fp8, ps):
    """A sequence of as many slots as are accepted, 2^31 less a page, of which
    only the last pages lie in the pool: its last token sees exactly those, over
    all slots, in a window and in listed blocks."""
    rng = np.random.default_rng(61)
    pages = 2 ** 31 // ps - 1
    cap = pages * ps
    c = Cache(rng, 1, 4, ps, 1, fp8)
    dev, _ = c.to("cuda")
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, -4:] = torch.from_numpy(c.table[0]).cuda()
    small = 4 * ps                              # the oracle's sequence: the last four pages
    c.pps = pages
    q = queries(rng, 1, H)
    for pos in (cap - 1, cap - 3, 2 ** 31 - 1):
        at = min(pos, cap - 1) - (cap - small)
        for window in (0, ps + 5):
            w = max(0, window - (pos - min(pos, cap - 1)))
            out, lse = attend(dsa, c, dev, table, q.cuda(), np.array([pos]), SCALE, window=window)
            ref = orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, [at], None, SCALE, window=w)
            if window and not w:
                assert torch.all(out == 0) and torch.all(lse == float("-inf"))
            else:
                check_attention(out, lse, ref)
    blocks = np.array([[[pages - 1, pages - 3, 5]]])
    out, lse = attend(dsa, c, dev, table, q.cuda(), np.array([cap - 1]), SCALE, blocks=blocks, block_size=ps, window=7)
    ref = orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, [small - 1], None, SCALE,
                        blocks=np.array([[[3, 1, -1]]]), block_size=ps, window=7)
    check_attention(out, lse, ref)


@pytest.mark.parametrize("T", [1, 64])
@pytest.mark.parametrize("top", [2.0 ** 12, 2.0 ** 24, 2.0 ** 28, 2.0 ** 31, 2.0 ** 33, 1e10, 1e30])
@pytest.mark.parametrize("G,fp8", [(8, False), (8, True), (64, False), (64, True)])
def test_large_finite_logits(dsa, G, fp8, top, T):
    """Logits up to `top` that grow along the slots, the largest three times, for
    every other head the smallest three times (a negative query). Keys and queries
    have one feature, so that logits are exact products; neighbouring ones are a
    sixteenth apart at least, hundreds of the largest logit's rounding steps, so
    that only the three count, with the same weight: out is their values' mean,
    off by its rounding (2^-8) and the fp32 sums' (2^-20 covers three terms and the
    division), lse the largest logit + ln 3 by relative 2^-21 (a scale, a product,
    a sum and the factor ln 2 in fp32, half a step each). One token, whose steps lie
    in as many warps, or 64 equal ones, where a warp has several."""
    rng = np.random.default_rng(62)
    c = Cache(rng, 1, 16, 64, 1, fp8)
    n = 1000
    order = np.sort(rng.integers(0x31, 0x77, n)).astype(np.uint8)
    order[:3], order[3:] = 0x30, np.maximum(order[3:], 0x31)
    order[-3:], order[:-3] = 0x77, np.minimum(order[:-3], 0x76)
    last, first = [400, 700, n - 1], [0, 333, 800]
    for a, b in zip(last + first, [n - 1, n - 2, n - 3, 0, 1, 2]):
        order[a], order[b] = order[b], order[a]
    value = torch.from_numpy(order).view(torch.float8_e4m3fn).double().numpy()
    last, first = np.flatnonzero(order == 0x77), np.flatnonzero(order == 0x30)
    assert len(last) == len(first) == 3
    page, slot = c.table[0][np.arange(n) // 64], np.arange(n) % 64
    if fp8:
        data, scale = c.pools["k"]
        data.zero_()
        scale.fill_(127)
        data[c.at[page, slot, 0]] = torch.from_numpy(order)
    else:
        rows = np.zeros((c.num_pages, 64, 1, D))
        rows[page, slot, 0, 0] = value
        c.set_rows("k", rows)
    q = torch.zeros((T, G, D), dtype=torch.bfloat16)
    q[:, ::2, 0], q[:, 1::2, 0] = 1.0, -1.0
    dev, table = c.to("cuda")
    amp = float(np.float32(top / value.max()))
    out, lse = attend(dsa, c, dev, table, q.cuda(), np.full(T, n - 1), amp, seq_ids=np.zeros(T))
    v = c.rows("v")[page, slot, 0]
    for h in range(G):
        mine, sign = (first, -1.0) if h % 2 else (last, 1.0)
        if h % 2 and amp * value.min() / 16 < 40:           # the smallest are not far enough apart
            continue
        ref, size = v[mine].mean(axis=0), np.abs(v[mine]).mean(axis=0)
        got = out[:, h].double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size), h
        x = sign * amp * value[mine[0]] + np.log(3.0)
        assert np.all(np.abs(lse[:, h].double().cpu().numpy() - x) <= 2.0 ** -21 * abs(x)), h


def mx_rows(x):
    """e4m3 bytes and e8m0 bytes of float32 rows (the format's rule, on the host)."""
    e = orc.mx_exponents(x.astype(np.float64))
    y = x.astype(np.float64) * np.repeat(2.0 ** -e.astype(np.float64), 32, axis=-1)       # exact
    data = torch.from_numpy(y.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    return data.numpy(), (e + 127).astype(np.uint8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("rope_dim", [30, 64, 128])
def test_append_rounds_every_product_and_the_sum(dsa, rope_dim, halves, fp8):
    """The rotation is the stated fp32 formula to the last bit: two products, each
    rounded, and their rounded sum. Half of the pairs cancel (equal features under
    equal factors), where a product that is not rounded leaves a remainder."""
    if halves and rope_dim % 16:
        rope_dim = 48
    rng = np.random.default_rng(63)
    T, H, half = 300, 5, rope_dim // 2
    c = Cache(rng, T, 1, 16, 2, fp8, values=False)
    x = rng.standard_normal((T, H + 2, D))
    cos, sin = rng.standard_normal((2, T, half)).astype(np.float32)
    first = np.arange(half) if halves else 2 * np.arange(half)
    second = first + (half if halves else 1)
    same = rng.random((T, half)) < 0.5
    sin = np.where(same, cos, sin)
    x[:, :, second] = np.where(same[:, None], x[:, :, first], x[:, :, second])
    x = bf16_bits(x)
    a, b = x.float().numpy()[..., first], x.float().numpy()[..., second]
    want = x.float().numpy().copy()
    want[..., first] = a * cos[:, None] - b * sin[:, None]          # float32, each operation rounded
    want[..., second] = a * sin[:, None] + b * cos[:, None]
    dev, table = c.to("cuda")
    kd, ks = dev["k"]
    q_out = torch.zeros((T, H, D), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    q_scale = torch.zeros((T, H, D // 32), dtype=torch.uint8, device="cuda") if fp8 else None
    desc = dsa.make_append_desc(c.desc(dsa, table), T, H, rope_dim, q_dtype=int(fp8),
                                rope_style=dsa.DSA_ROPE_HALVES if halves else dsa.DSA_ROPE_INTERLEAVED)
    pos = rng.integers(0, 16, T)
    dsa.dsa_cache_append(desc, x[:, :H].contiguous().cuda(), x[:, H:].contiguous().cuda(), None,
                         torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(), dev_i32(pos), None, q_out,
                         q_scale, kd, ks, None, None, torch.cuda.current_stream().cuda_stream)
    at = c.at[c.table[:, 0], pos]                                   # [T, 2]
    rows = kd.cpu().view(torch.uint8 if fp8 else torch.bfloat16)[at[..., None] + torch.arange(D)]
    if fp8:
        scales = ks.cpu()[at[..., None] // 32 + torch.arange(D // 32)]
        for got, got_s, ref in ((q_out.cpu(), q_scale.cpu(), want[:, :H]), (rows, scales, want[:, H:])):
            data, e = mx_rows(ref)
            assert np.array_equal(got_s.numpy(), e)
            assert np.array_equal(decode_mx(got, got_s), decode_mx(torch.from_numpy(data), torch.from_numpy(e)))
    else:
        ref = torch.from_numpy(want).to(torch.bfloat16)
        assert torch.equal(q_out.cpu(), ref[:, :H]) and torch.equal(rows, ref[:, H:])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("G", [8, 64])
def test_rows_of_infinitely_small_logits_are_empty(dsa, G, bad):
    """Every kept slot's logit is -infinity, its value infinite or NaN: out = 0 and
    lse = -infinity, in one CTA and in many, beside rows that are as ever."""
    rng = np.random.default_rng(64)
    c = Cache(rng, 3, 80, 64, 1)
    for name, x in (("k", -np.inf), ("v", bad)):
        rows = c.rows(name)
        for i, n in ((0, 5), (1, 5000)):
            s = np.arange(n)
            rows[c.table[i, s // 64], s % 64, 0, 3] = x
        c.set_rows(name, rows)
    dev, table = c.to("cuda")
    q = queries(rng, 3, G)
    q[:2, :, 3] = q[:2, :, 3].abs() + 1
    pos = np.array([4, 4999, 100])
    out, lse = attend(dsa, c, dev, table, q.cuda(), pos, SCALE)
    assert torch.all(out[:2] == 0) and torch.all(lse[:2] == float("-inf"))
    ref = orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, [-1, -1, 100], None, SCALE)
    check_attention(out, lse, ref)
    out, lse = attend(dsa, c, dev, table, q.cuda(), pos, SCALE, blocks=np.array([[[0, -1]], [[3, 60]], [[-1, 0]]]),
                      block_size=64)
    assert torch.all(out[:2] == 0) and torch.all(lse[:2] == float("-inf")) and torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("T", [4, 400])
@pytest.mark.parametrize("H,fp8", [(8, False), (8, True), (64, False), (64, True)])
def test_a_stalled_call_reports_the_timeout(dsa, H, fp8, T, listed):
    """A warp keeps an arrival back, others wait for it and give up after a
    millisecond: the status is reported once, nothing past the call's rows is
    written (whatever an earlier call left in the workspace), and the next call on
    the same workspace is right. Few long items, which many CTAs share, and many
    short ones."""
    rng = np.random.default_rng(65)
    c = Cache(rng, 4, 32, 64, 1, fp8)
    dev, table = c.to("cuda")
    q, seq = queries(rng, T, H), np.arange(T) % 4
    pos = rng.integers(1000, 2048, T) if T == 4 else rng.integers(-1, 300, T)
    blocks = rng.integers(-1, 32, (T, 1, 3)) if listed else None
    more = dict(block_size=64, num_blocks=3, window=20) if listed else {}
    desc = dsa.make_paged_attention_desc(c.desc(dsa, table), T, H, SCALE, wait_limit_ns=1_000_000,
                                         flags=dsa.DSA_FLAG_SELFTEST_STALL, **more)
    n = dsa.dsa_paged_attention_workspace_size(desc)
    stream = torch.cuda.current_stream().cuda_stream
    lists = [dev_i32(blocks)] if listed else []
    call = dsa.dsa_block_attention_forward if listed else dsa.dsa_paged_attention_forward
    qc, dpos, dseq = q.cuda(), dev_i32(pos), dev_i32(seq)
    for fill in (0, 1, 0x70):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        out = torch.full((T + 60, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T + 60, H), 7.0, device="cuda")
        call(desc, qc, *dev["k"], *dev["v"], None, dpos, dseq, *lists, out, lse, ws, n, stream)
        assert dsa.dsa_indexer_get_error(ws, stream) == dsa.DSA_ERR_TIMEOUT
        assert dsa.dsa_indexer_get_error(ws, stream) == dsa.DSA_OK
        assert torch.all(out[T:] == 7.0) and torch.all(lse[T:] == 7.0)
        kw = dict(blocks=blocks, block_size=64, window=20) if listed else {}
        got = attend(dsa, c, dev, table, qc, pos, SCALE, seq_ids=seq, workspace=ws, **kw)
    ref = orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, pos, seq, SCALE, **kw)
    check_attention(*got, ref)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("G", [8, 40, 64, 128])
def test_fp8_value_scales_one_by_one(dsa, G, listed):
    """Scale bytes from 20 to 218, each deciding outputs of its own (a CPU test
    shows that the check sees every one): one byte a feature block, blocks that differ
    by up to 2^198, and slots around the border of the two-step conversion."""
    rng = np.random.default_rng(66)
    c, _ = scaled_cache(rng)
    dev, table = c.to("cuda")
    q = queries(rng, c.num_seqs, G)
    kw = {}
    if listed:
        kw = dict(blocks=np.tile(np.array([2, 0, 5, -1, 1, 7]), (c.num_seqs, 1, 1)), block_size=16, window=16)
    out, lse = attend(dsa, c, dev, table, q.cuda(), POSITIONS, SCALE, **kw)
    check_attention(out, lse, orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, POSITIONS, None,
                                            SCALE, **kw))


@pytest.mark.parametrize("G", [8, 64])
@pytest.mark.parametrize("byte", [20, 60, 110, 132, 133, 134, 135, 160, 200])
def test_fp8_key_scales(dsa, G, byte):
    """Keys under two neighbouring scale bytes, the logit scale the other way round,
    so that the logits are ordinary ones."""
    rng = np.random.default_rng(67 + byte)
    c = Cache(rng, 4, 3, 64, 1, True)
    scale = c.pools["k"][1]
    scale[:] = torch.from_numpy(rng.integers(byte, byte + 2, len(scale)).astype(np.uint8))
    dev, table = c.to("cuda")
    q, pos, amp = queries(rng, 4, G), np.array([191, 60, 100, 127]), SCALE * 2.0 ** (121 - byte)
    out, lse = attend(dsa, c, dev, table, q.cuda(), pos, amp)
    check_attention(out, lse, orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, pos, None, amp))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [1, 2, 3, 4, 7, 16, 32, 63, 64])
def test_pooling_keys_near_the_largest_number(dsa, bs, fp8):
    """The mean of keys of up to bf16's largest number is as finite as they are:
    within the fp32 sum's rounding (bs + 1 half steps of the largest) and its own
    (2^-8, or 2^-4 for e4m3)."""
    rng = np.random.default_rng(68)
    c = Cache(rng, 2, 2, 64, 1, fp8, values=False)
    if fp8:
        data, scale = c.pools["k"]
        data[:] = torch.from_numpy(rng.integers(0x70, 0x7f, len(data)).astype(np.uint8))    # 128 .. 448
        scale[:] = 246                                                                        # 2^119
    else:
        top = float(torch.finfo(torch.bfloat16).max)
        c.set_rows("k", rng.uniform(0.3, 1.0, (c.num_pages, 64, 1, D)) * top)
    dev, table = c.to("cuda")
    n, pos = 128 // bs, [127, 100]
    pooled = torch.zeros((2, n, D), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    pscale = torch.zeros((2, n, D // 32), dtype=torch.uint8, device="cuda") if fp8 else None
    dsa.dsa_block_pool(dsa.make_block_pool_desc(c.desc(dsa, table), bs, n), *dev["k"], None, dev_i32(pos), pooled,
                       pscale, None, torch.cuda.current_stream().cuda_stream)
    got = decode_mx(pooled.cpu(), pscale.cpu()) if fp8 else pooled.double().cpu().numpy()
    rows, _ = orc.pool_blocks(c.rows("k"), c.table, None, pos, bs, n)
    assert len(rows) == 128 // bs + 101 // bs
    for (i, b), ref in rows.items():
        slack = (bs + 1) * 2.0 ** -24 * np.abs(ref).max()
        assert np.all(np.abs(got[i, b] - ref[0]) <= (2.0 ** -4 if fp8 else 2.0 ** -8) * np.abs(ref[0]) + 2 * slack)


@pytest.mark.parametrize("amp", [2.0 ** -127, -2.0 ** -127, 2.0 ** -126])
@pytest.mark.parametrize("G,fp8", [(8, False), (8, True), (64, False), (64, True)])
def test_logit_scales_below_the_normal_numbers(dsa, G, fp8, amp):
    """Products of query and key near fp32's largest number under a logit scale
    near its smallest: ordinary logits."""
    rng = np.random.default_rng(69)
    c = Cache(rng, 3, 2, 64, 1, fp8)
    if fp8:
        c.pools["k"][1] += 58
    else:
        c.set_rows("k", c.rows("k") * 2.0 ** 60)
    dev, table = c.to("cuda")
    q, pos = queries(rng, 3, G, 2.0 ** 60), np.array([127, 70, 20])
    largest = np.abs(c.rows("k")).reshape(-1, D) @ np.abs(q.double().numpy()).reshape(-1, D).T
    assert largest.max() < torch.finfo(torch.float32).max      # no partial sum overflows
    out, lse = attend(dsa, c, dev, table, q.cuda(), pos, amp)
    check_attention(out, lse, orc.attention(q.double().numpy(), c.rows("k"), c.rows("v"), c.table, pos, None, amp))
