"""The paged cache's entry points refuse bad arguments on the host before any
device work, their descriptors sit as a C compiler puts them, and the fp64
oracle they are tested against is pinned (CPU only)."""
import ctypes
import pathlib
import subprocess

import numpy as np
import pytest

import oracle.paged as orc
import sparse_attention_lightning_tcgen05_b200 as dsa

ROOT = pathlib.Path(__file__).resolve().parent.parent
FAKE = 1 << 20                      # never dereferenced: checks fail first
BF16, FP8 = dsa.DSA_KV_BF16, dsa.DSA_KV_FP8_E4M3_E8M0_B32
INV, UNS, WS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE


def cache(**kw):
    d = dict(page_size=64, pages_per_seq=16, num_pages=40, block_table=FAKE, num_seqs=2, H_kv=2)
    d.update(kw)
    return dsa.make_paged_cache(**d)


def refused(code, call):
    with pytest.raises(dsa.DsaError) as e:
        call()
    assert e.value.status == code, e.value


BAD_CACHES = [
    (dict(page_size=8), INV), (dict(page_size=48), INV), (dict(page_size=1 << 17), INV),
    (dict(pages_per_seq=0), INV), (dict(num_pages=0), INV), (dict(num_seqs=0), INV),
    (dict(H_kv=0), INV), (dict(H_kv=129), UNS), (dict(D=64), UNS), (dict(dtype=5), INV),
    (dict(block_table=None), INV), (dict(block_table=FAKE + 2), INV),
    (dict(page_stride=-128), INV), (dict(slot_stride=130), INV), (dict(head_stride=64), INV),
    (dict(num_pages=1 << 26), UNS), (dict(pages_per_seq=1 << 26), UNS),
    (dict(page_stride=1 << 60), UNS),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(kw, code):
    c = cache(**kw)
    refused(code, lambda: dsa.dsa_cache_append(dsa.make_append_desc(c, 2, 0, 0), None, FAKE, None, None, None,
                                               FAKE, None, None, None, FAKE, None, None, None))
    refused(code, lambda: dsa.dsa_block_pool(dsa.make_block_pool_desc(c, 4, 8), FAKE, None, None, FAKE, FAKE,
                                             None))
    refused(code, lambda: dsa.dsa_paged_attention_workspace_size(dsa.make_paged_attention_desc(c, 2, 4, 0.1)))


def append(desc=None, ckw=None, dkw=None, **over):
    """An append call on fake pointers, some of them replaced."""
    c = cache(**(ckw or {}))
    kw = dict(T=3, H=4, rope_dim=64)
    kw.update(dkw or {})
    fp8, q_fp8 = c.dtype == FP8, kw.get("q_dtype", BF16) == FP8
    args = dict(q=FAKE, k=FAKE, v=FAKE, cos=FAKE, sin=FAKE, positions=FAKE, seq_ids=None, q_out=2 * FAKE,
                q_scale=FAKE if q_fp8 else None, k_cache=FAKE, k_scale=FAKE if fp8 else None, v_cache=FAKE,
                v_scale=FAKE if fp8 else None)
    args.update(over)
    return lambda: dsa.dsa_cache_append(dsa.make_append_desc(c, **kw), *args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dkw=dict(T=0)), INV), (dict(dkw=dict(H=-1)), INV), (dict(dkw=dict(H=257)), UNS),
    (dict(dkw=dict(rope_dim=63)), INV), (dict(dkw=dict(rope_dim=130)), INV), (dict(dkw=dict(rope_dim=-2)), INV),
    (dict(dkw=dict(rope_dim=24, rope_style=1)), UNS), (dict(dkw=dict(rope_style=2)), INV),
    (dict(dkw=dict(q_dtype=9)), INV),
    (dict(dkw=dict(q_stride=511)), INV), (dict(dkw=dict(q_stride=504)), INV), (dict(dkw=dict(k_stride=248)), INV),
    (dict(dkw=dict(v_stride=260)), INV),
    (dict(k=None), INV), (dict(positions=None), INV), (dict(positions=FAKE + 1), INV), (dict(k=FAKE + 8), INV),
    (dict(v=FAKE + 8), INV), (dict(q=None), INV), (dict(q_out=None), INV), (dict(q_out=FAKE + 8), INV),
    (dict(q_scale=FAKE), INV), (dict(cos=None), INV), (dict(sin=None), INV), (dict(seq_ids=FAKE + 2), INV),
    (dict(k_cache=None), INV), (dict(k_cache=FAKE + 8), INV), (dict(k_scale=FAKE), INV),
    (dict(v=None), INV), (dict(v_cache=None), INV), (dict(v_scale=FAKE), INV),
    (dict(dkw=dict(H=0)), INV),                                  # queries given without heads
    (dict(ckw=dict(dtype=FP8), k_scale=None), INV), (dict(ckw=dict(dtype=FP8), v_scale=None), INV),
    (dict(ckw=dict(dtype=FP8), k_scale=FAKE + 2), INV),
    (dict(dkw=dict(q_dtype=FP8), q_scale=None), INV),
    (dict(dkw=dict(q_dtype=FP8), q_out=FAKE), INV),              # fp8 rows over the bf16 ones
    (dict(dkw=dict(q_stride=1024), q_out=FAKE), INV),            # in place over spread rows
])
def test_append_refusals(kw, code):
    refused(code, append(**kw))


def pool(ckw=None, dkw=None, **over):
    c = cache(**(ckw or {}))
    kw = dict(block_size=4, S_pool=256)
    kw.update(dkw or {})
    fp8 = c.dtype == FP8
    args = dict(k=FAKE, ks=FAKE if fp8 else None, start=None, positions=FAKE, pooled=FAKE,
                pooled_scale=FAKE if fp8 else None, last=None)
    args.update(over)
    return lambda: dsa.dsa_block_pool(dsa.make_block_pool_desc(c, **kw), *args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dkw=dict(block_size=0)), INV), (dict(dkw=dict(block_size=65537)), UNS), (dict(dkw=dict(S_pool=0)), INV),
    (dict(dkw=dict(S_pool=1 << 32)), UNS), (dict(dkw=dict(seq_stride=100)), INV),
    (dict(dkw=dict(head_stride=-128)), INV), (dict(dkw=dict(head_stride=1 << 50)), UNS),
    (dict(k=None), INV), (dict(k=FAKE + 8), INV), (dict(ks=FAKE), INV), (dict(positions=None), INV),
    (dict(positions=FAKE + 1), INV), (dict(start=FAKE + 2), INV), (dict(pooled=None), INV),
    (dict(pooled=FAKE + 8), INV), (dict(pooled_scale=FAKE), INV), (dict(last=FAKE + 1), INV),
    (dict(ckw=dict(dtype=FP8), ks=None), INV), (dict(ckw=dict(dtype=FP8), pooled_scale=None), INV),
])
def test_pool_refusals(kw, code):
    refused(code, pool(**kw))


def attention(ckw=None, dkw=None, blocks=None, ws_bytes=1 << 30, **over):
    c = cache(**(ckw or {}))
    kw = dict(T=3, H=4, sm_scale=0.1)
    if blocks is not None:
        kw.update(block_size=64, num_blocks=4)
    kw.update(dkw or {})
    fp8 = c.dtype == FP8
    a = dict(q=FAKE, k=FAKE, ks=FAKE if fp8 else None, v=FAKE, vs=FAKE if fp8 else None, sinks=None,
             positions=FAKE, seq_ids=None, out=FAKE, lse=None, ws=FAKE)
    a.update(over)
    d = dsa.make_paged_attention_desc(c, **kw)
    head = [a["q"], a["k"], a["ks"], a["v"], a["vs"], a["sinks"], a["positions"], a["seq_ids"]]
    tail = [a["out"], a["lse"], a["ws"], ws_bytes]
    if blocks is None:
        return lambda: dsa.dsa_paged_attention_forward(d, *head, *tail)
    return lambda: dsa.dsa_block_attention_forward(d, *head, None if blocks == 0 else blocks, *tail)


@pytest.mark.parametrize("kw,code", [
    (dict(dkw=dict(T=0)), INV), (dict(dkw=dict(H=0)), INV), (dict(dkw=dict(H=3)), INV),
    (dict(dkw=dict(H=258)), UNS), (dict(dkw=dict(T=1 << 30)), UNS), (dict(dkw=dict(sm_scale=float("inf"))), INV),
    (dict(dkw=dict(sm_scale=float("nan"))), INV), (dict(dkw=dict(sm_scale=3e38)), INV),
    (dict(dkw=dict(window=-1)), INV),
    (dict(q=None), INV), (dict(q=FAKE + 8), INV), (dict(out=None), INV), (dict(out=FAKE + 4), INV),
    (dict(positions=None), INV), (dict(positions=FAKE + 2), INV), (dict(sinks=FAKE + 2), INV),
    (dict(seq_ids=FAKE + 1), INV), (dict(lse=FAKE + 2), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(k=FAKE + 8), INV), (dict(ks=FAKE), INV), (dict(vs=FAKE), INV),
    (dict(ckw=dict(dtype=FP8), ks=None), INV), (dict(ckw=dict(dtype=FP8), vs=FAKE + 1), INV),
    (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(ws_bytes=256), WS),
])
def test_attention_refusals(kw, code):
    refused(code, attention(**kw))
    refused(code, attention(blocks=FAKE, **kw))


@pytest.mark.parametrize("kw,code", [
    (dict(blocks=0), INV), (dict(blocks=FAKE + 2), INV),
    (dict(blocks=FAKE, dkw=dict(block_size=0)), INV), (dict(blocks=FAKE, dkw=dict(block_size=12)), INV),
    (dict(blocks=FAKE, dkw=dict(block_size=1 << 17)), INV), (dict(blocks=FAKE, dkw=dict(num_blocks=0)), INV),
    (dict(blocks=FAKE, dkw=dict(block_heads=3)), INV), (dict(blocks=FAKE, dkw=dict(num_blocks=1 << 25)), UNS),
    (dict(blocks=FAKE, dkw=dict(window=(1 << 30) - 1)), UNS),
])
def test_block_attention_refusals(kw, code):
    refused(code, attention(**kw))


def test_valid_calls_without_a_gpu_fail_cleanly():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    refused(dsa.DSA_ERR_CUDA, append())
    refused(dsa.DSA_ERR_CUDA, append(v=None, v_cache=None))
    refused(dsa.DSA_ERR_CUDA, pool())
    refused(dsa.DSA_ERR_CUDA, attention())
    refused(dsa.DSA_ERR_CUDA, attention(blocks=FAKE))
    n = dsa.dsa_paged_attention_workspace_size(dsa.make_paged_attention_desc(cache(), 3, 4, 0.1))
    refused(dsa.DSA_ERR_CUDA, attention(ws_bytes=n))
    refused(WS, attention(ws_bytes=n - 1))
    refused(INV, lambda: dsa.dsa_paged_attention_workspace_size(
        dsa.make_paged_attention_desc(cache(), 3, 4, 0.1, num_blocks=4, block_size=5)))


def test_tensors_of_another_device_are_refused():
    import torch
    if torch.cuda.is_available():
        pytest.skip("without a GPU every tensor is on another device")
    host = torch.zeros(4096, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dsa_block_pool"):
        dsa.dsa_block_pool(dsa.make_block_pool_desc(cache(), 4, 8), host, None, None, FAKE, FAKE, None)


_LAYOUT = r"""
#include <stddef.h>
#include <stdio.h>
#include "dsa_paged_attention.h"
int main(void) {
%s
  return 0;
}
"""


def test_descriptors_match_the_c_headers():
    out_dir = ROOT / "_build" / "paged_layout"
    out_dir.mkdir(parents=True, exist_ok=True)
    types = [dsa.dsa_paged_cache_t, dsa.dsa_append_desc_t, dsa.dsa_block_pool_desc_t,
             dsa.dsa_paged_attention_desc_t]
    lines = [f'printf("{t.__name__} {f[0]} %zu\\n", offsetof({t.__name__}, {f[0]}));'
             for t in types for f in t._fields_]
    lines += [f'printf("{t.__name__} sizeof %zu\\n", sizeof({t.__name__}));' for t in types]
    (out_dir / "layout.c").write_text(_LAYOUT.replace("%s", "\n".join(lines), 1))
    subprocess.run(["gcc", "-O0", "-I", str(ROOT / "include"), str(out_dir / "layout.c"), "-o",
                    str(out_dir / "layout")], check=True)
    got = subprocess.run([str(out_dir / "layout")], capture_output=True, text=True, check=True).stdout
    by_name = {t.__name__: t for t in types}
    rows = [line.split() for line in got.strip().splitlines()]
    assert len(rows) == len(lines)
    for name, field, off in rows:
        t = by_name[name]
        assert int(off) == (ctypes.sizeof(t) if field == "sizeof" else getattr(t, field).offset), (name, field)


# ---- pins of the oracle --------------------------------------------------------------

def test_rope_turns_the_stated_pairs():
    x = np.arange(1.0, 129.0)[None]
    c, s = np.zeros((1, 2)), np.ones((1, 2))                 # a quarter turn
    a = orc.rope(x, c, s, 4, False)[0]
    assert a[:6].tolist() == [-2, 1, -4, 3, 5, 6]
    b = orc.rope(x, c, s, 4, True)[0]
    assert b[:6].tolist() == [-3, -4, 1, 2, 5, 6]


def test_rope_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 128))
    w = rng.uniform(0, 1, 32)

    def at(x, p, halves):
        return orc.rope(x, np.cos(p * w), np.sin(p * w), 64, halves)
    for halves in (False, True):
        assert np.isclose(np.linalg.norm(at(q, 9, halves)), np.linalg.norm(q))
        assert np.isclose(at(q, 9, halves) @ at(k, 4, halves), at(q, 105, halves) @ at(k, 100, halves))


def test_mx_exponents_are_the_least_that_fit():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 128)) * 2.0 ** rng.integers(-140, 120, (50, 1))
    x[0, :32], x[1, :32], x[2, :32] = 448.0, np.nextafter(448.0, 500), 0.0
    e = orc.mx_exponents(x)
    top = np.abs(x).reshape(50, 4, 32).max(-1)
    assert np.all(top <= 448.0 * 2.0 ** e) and np.all((e == -127) | (top > 448.0 * 2.0 ** (e - 1)))
    assert (e[0, 0], e[1, 0], e[2, 0]) == (0, 1, -127)


def test_kept_slots_by_enumeration():
    """Every small case against the statement read literally, slot by slot."""
    for cap in (1, 4, 9):
        for pos in range(-1, cap + 3):
            for w in range(0, 6):
                dense = [s for s in range(cap) if s <= pos and (w == 0 or s > pos - w)]
                assert orc.kept_slots(pos, cap, w) == (dense if pos >= 0 else [])
                for bs in (1, 2, 4):
                    lists = [[-1], [0], [1, 0], [0, 0], [2, -3, 1]]
                    for blocks in lists:
                        want = [s for b in blocks if b >= 0 for s in range(cap)
                                if b * bs <= s < (b + 1) * bs and s <= pos - w]
                        want += [s for s in range(cap) if pos - w < s <= pos]
                        assert orc.kept_slots(pos, cap, w, blocks, bs) == (want if pos >= 0 else [])


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 4, 16, 1, 128))
    table = np.array([[2, 0]], np.int32)
    q = rng.standard_normal((1, 2, 128))
    out, lse, _, _ = orc.attention(q, k, v, table, [0], None, 0.3)           # one slot
    assert np.allclose(out[0], v[2, 0, 0]) and np.allclose(lse[0], 0.3 * q[0] @ k[2, 0, 0])
    out, lse, _, _ = orc.attention(q * 0, k, v, table, [20], None, 0.3)      # the mean
    rows = np.concatenate([v[2, :, 0], v[0, :5, 0]])
    assert np.allclose(out[0], rows.mean(axis=0)) and np.allclose(lse[0], np.log(21))
    out, lse, _, _ = orc.attention(q * 0, k, v, table, [20], None, 0.3, sinks=np.array([0.0, 50.0]))
    assert np.allclose(out[0, 0], rows.sum(axis=0) / 22) and np.all(np.abs(out[0, 1]) < 1e-18)
    out, lse, _, _ = orc.attention(q, k, v, table, [-1], None, 0.3)
    assert np.all(out == 0) and np.all(lse == -np.inf)
    every = np.array([[[1, 0]]])
    a = orc.attention(q, k, v, table, [25], None, 0.3)
    b = orc.attention(q, k, v, table, [25], None, 0.3, blocks=every, block_size=16)
    c = orc.attention(q, k, v, table, [25], None, 0.3, blocks=every, block_size=16, window=7)
    assert np.allclose(a[0], b[0]) and np.allclose(a[0], c[0]) and np.allclose(a[1], c[1])


def test_pooled_blocks_are_the_completed_ones():
    k = np.arange(3 * 16 * 1 * 128, dtype=np.float64).reshape(3, 16, 1, 128)
    table = np.array([[1, 0], [2, 5]], np.int32)
    rows, last = orc.pool_blocks(k, table, [6, 0], [21, 40], 4, 100)
    assert sorted(b for i, b in rows if i == 0) == [1, 2, 3, 4] and last == [4, 7]
    assert np.allclose(rows[0, 4][0], k[0, 0:4, 0].mean(axis=0))             # slots 16 .. 19: page 0
    assert np.allclose(rows[1, 0][0], k[2, 0:4, 0].mean(axis=0))
    assert np.all(rows[1, 4][0] == 0)                                        # page 5 is outside
