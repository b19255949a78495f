"""Values under chosen scale bytes: an fp8 cache in which every scale byte decides
outputs of its own, so that one that is read wrongly cannot hide behind larger
ones."""
from __future__ import annotations

import numpy as np
import torch

from paged_util import D, Cache

# Scale bytes of a sequence's four blocks of 32 features (all its slots'), or of
# its slots in turn (all features'). 134 is the largest that one multiplication of
# the bf16 conversion takes.
BY_BLOCK = [(20, 21, 30, 40), (60, 60, 60, 60), (100, 110, 111, 112), (117, 120, 126, 127), (133, 134, 135, 136),
            (134, 134, 134, 134), (135, 135, 135, 135), (140, 150, 160, 170), (200, 201, 210, 218),
            (60, 134, 135, 200), (200, 20, 134, 60), (135, 134, 20, 136), (218, 20, 218, 20)]
BY_SLOT = [(133, 134, 135, 136), (134, 135, 134, 135), (119, 120, 121, 122)]
POSITIONS = np.array([150, 31, 191, 7, 100, 130, 64, 127, 190, 63, 180, 99, 16] + [191, 150, 77])


def scaled_cache(rng):
    """A cache of 16 sequences of three pages of 64 slots, one key head, with the
    value scales above, and the byte of every value [pages, slots, 1, D]."""
    n = len(BY_BLOCK) + len(BY_SLOT)
    c = Cache(rng, n, 3, 64, 1, True)
    data, scale = c.pools["v"]
    # codes of a column keep one sign, so that no block's outputs cancel
    codes = torch.from_numpy(rng.integers(0x30, 0x70, (c.num_pages, 64, 1, D)).astype(np.uint8))
    codes |= torch.from_numpy((rng.integers(0, 2, D) << 7).astype(np.uint8))
    data[c.at[..., None] + torch.arange(D)] = codes
    byte = np.full((c.num_pages, 64, 1, D // 32), 127, np.uint8)
    for i, four in enumerate(BY_BLOCK):
        byte[c.table[i]] = np.array(four)
    for i, turn in enumerate(BY_SLOT):
        byte[c.table[len(BY_BLOCK) + i]] = np.array(turn)[np.arange(64) % len(turn)][:, None, None]
    scale[c.at[..., None] // 32 + torch.arange(D // 32)] = torch.from_numpy(byte)
    return c, np.repeat(byte, 32, axis=-1)
