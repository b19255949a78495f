"""Edges of attention over a paged cache and of the cache's writers, each
against the fp64 oracle (GPU only). Tolerances: paged_util.check_attention, and
what a test derives beside it.
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
