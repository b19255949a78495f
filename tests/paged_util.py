"""Paged caches for the tests: random ones in any layout, on the device and as
the float64 rows they stand for."""
from __future__ import annotations

import numpy as np
import torch

D = 128


def bf16_bits(x):
    """Nearest bf16 of float64 / float32 values, as torch.bfloat16."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def decode_mx(data, scale):
    """float64 values of e4m3 data (uint8 tensor [.., D]) under e8m0 bytes
    [.., D/32]; byte 255 is NaN."""
    x = data.view(torch.float8_e4m3fn).float().double().numpy()
    s = scale.numpy().astype(np.int64)
    f = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return x * np.repeat(f, 32, axis=-1)


class Cache:
    """num_seqs sequences of pages_per_seq pages over a pool with `spare`
    pages more than the tables use. layout: "slots" [page, slot, head, D],
    "heads" [page, head, slot, D], "gaps" (slots order with unused rows between
    heads, slots and pages)."""

    def __init__(self, rng, num_seqs, pages_per_seq, page_size, Hkv, fp8=False, layout="slots",
                 spare=2, values=True, fill=None):
        self.num_seqs, self.pps, self.ps, self.Hkv, self.fp8 = num_seqs, pages_per_seq, page_size, Hkv, fp8
        self.num_pages = num_seqs * pages_per_seq + spare
        self.table = rng.permutation(self.num_pages)[:num_seqs * pages_per_seq].astype(np.int32) \
            .reshape(num_seqs, pages_per_seq)
        if layout == "heads":
            self.strides = (Hkv * page_size * D, D, page_size * D)
        elif layout == "gaps":
            head = 2 * D
            slot = Hkv * head + 3 * D
            self.strides = (page_size * slot + 5 * D, slot, head)
        else:
            self.strides = (page_size * Hkv * D, Hkv * D, D)
        page, slot, head = self.strides
        self.size = (self.num_pages - 1) * page + (page_size - 1) * slot + (Hkv - 1) * head + D
        at = (np.arange(self.num_pages)[:, None, None] * page + np.arange(page_size)[:, None] * slot +
              np.arange(Hkv) * head)
        self.at = torch.from_numpy(at)                       # element offset of each row
        self.pools = {}
        for n in ("k", "v") if values else ("k",):
            rows = rng.standard_normal((self.num_pages, page_size, Hkv, D)) if fill is None else \
                np.full((self.num_pages, page_size, Hkv, D), fill)
            self.set_rows(n, rows, rng)

    def set_rows(self, name, rows, rng=None):
        """Fill a pool: bf16 of the rows, or e4m3 codes under random scales."""
        idx = self.at[..., None] + torch.arange(D)
        if self.fp8:
            s = torch.from_numpy(rng.integers(117, 124, rows.shape[:-1] + (D // 32,)).astype(np.uint8))
            y = torch.from_numpy(np.clip(np.nan_to_num(rows) * 100, -448, 448).astype(np.float32))
            codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
            data, scale = torch.zeros(self.size, dtype=torch.uint8), torch.zeros(self.size // 32, dtype=torch.uint8)
            data[idx] = codes
            scale[self.at[..., None] // 32 + torch.arange(D // 32)] = s
            self.pools[name] = [data, scale]
        else:
            data = torch.zeros(self.size, dtype=torch.bfloat16)
            data[idx] = bf16_bits(rows)
            self.pools[name] = [data, None]

    def rows(self, name, pools=None):
        """float64 rows [num_pages, page_size, H_kv, D] of a pool on the host."""
        data, scale = (pools or self.pools)[name]
        data = data.cpu()
        idx = self.at[..., None] + torch.arange(D)
        if not self.fp8:
            return data[idx].double().numpy()
        return decode_mx(data[idx], scale.cpu()[self.at[..., None] // 32 + torch.arange(D // 32)])

    def to(self, device):
        """Device copies {name: [data, scale]} and the block table."""
        dev = {n: [x.to(device) if x is not None else None for x in p] for n, p in self.pools.items()}
        return dev, torch.from_numpy(self.table).to(device)

    def desc(self, m, table):
        page, slot, head = self.strides
        return m.make_paged_cache(self.ps, self.pps, self.num_pages, table, num_seqs=self.num_seqs,
                                  H_kv=self.Hkv, page_stride=page, slot_stride=slot, head_stride=head,
                                  dtype=m.DSA_KV_FP8_E4M3_E8M0_B32 if self.fp8 else m.DSA_KV_BF16)


def dev_i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def attend(m, cache, dev, table, q, positions, sm_scale, *, seq_ids=None, window=0, sinks=None,
           blocks=None, block_size=0, want_lse=True, stream=None, workspace=None):
    """One call on device tensors; numpy index arrays are copied over. Returns
    out, lse (device) after checking the device status."""
    T, H, _ = q.shape
    more = {} if blocks is None else dict(block_size=block_size, num_blocks=blocks.shape[2],
                                          block_heads=blocks.shape[1])
    desc = m.make_paged_attention_desc(cache.desc(m, table), T, H, sm_scale, window=window, **more)
    nbytes = m.dsa_paged_attention_workspace_size(desc)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda") if want_lse else None
    pos = positions if isinstance(positions, torch.Tensor) else dev_i32(positions)
    seq = None if seq_ids is None else dev_i32(seq_ids)
    snk = None if sinks is None else torch.from_numpy(np.ascontiguousarray(sinks, np.float32)).cuda()
    (kd, ks), (vd, vs) = dev["k"], dev["v"]
    stream = torch.cuda.current_stream().cuda_stream if stream is None else stream
    if blocks is None:
        m.dsa_paged_attention_forward(desc, q, kd, ks, vd, vs, snk, pos, seq, out, lse, ws, nbytes, stream)
    else:
        m.dsa_block_attention_forward(desc, q, kd, ks, vd, vs, snk, pos, seq, dev_i32(blocks), out, lse, ws,
                                      nbytes, stream)
    assert m.dsa_indexer_get_error(ws, stream) == m.DSA_OK
    return out, lse


def check_attention(out, lse, ref):
    """out and lse (torch) against the oracle's, within the kernel's
    arithmetic. Logits: 128 products exact in fp32 added in fp32, error at
    most 128 * 2^-24 = 2^-17 of sum |q k| * scale, twice that covers the
    scalings. A weight is then off by that, by the exponential's
    approximation (2^-22) and by its rounding to bf16 (2^-8); the output by
    its own rounding (2^-8). fp32 sums of the weights and of O: 2^-16 covers
    4096 slots."""
    o, l, reach, wabs = ref
    out = out.double().cpu().numpy()
    dl = 2.0 ** -16 * reach
    bound = (2.0 ** -8 + 2.0 ** -16 + 2 * dl)[..., None] * wabs + 2.0 ** -8 * np.abs(o)
    err = np.abs(out - o)
    assert np.all(err <= bound), float(np.max(err - bound))
    if lse is not None:
        lse = lse.double().cpu().numpy()
        empty = ~np.isfinite(l)
        assert np.all(lse[empty] == -np.inf)
        e = np.abs(lse[~empty] - l[~empty])
        # the running sum in fp32, ln by log2f and a product: 2^-16 absolute, 2^-22 relative
        assert np.all(e <= dl[~empty] + 2.0 ** -16 + 2.0 ** -22 * np.abs(l[~empty])), float(e.max())
