"""Edges of the paged operators that need no GPU: the kernels' row arithmetic
at the ends of its range."""
import pathlib
import subprocess

import pytest

ROOT = pathlib.Path(__file__).resolve().parent.parent
CSRC = ROOT / "sparse_attention_lightning_tcgen05_b200" / "csrc"

_ROWS = r"""
#include <cstdio>
#include "paged_rows.h"
int main() {
  long long cap;
  int num_seqs, window, list, list_steps, step, seq, at;
  while (std::scanf("%lld %d %d %d %d %d %d %d", &cap, &num_seqs, &window, &list, &list_steps, &step,
                    &seq, &at) == 8) {
    const dsa::PaRow r = dsa::pa_row_at(cap, num_seqs, window, list != 0, list_steps, step, seq, at);
    std::printf("%d %d %d %d %d\n", r.seq, r.last, r.lo, r.wbase, r.steps);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def rows_of():
    out = ROOT / "_build" / "paged_rows"
    out.mkdir(parents=True, exist_ok=True)
    (out / "rows.cpp").write_text(_ROWS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I", str(CSRC), str(out / "rows.cpp"), "-o",
                    str(out / "rows")], check=True)

    def run(cases):
        text = "\n".join(" ".join(str(int(x)) for x in c) for c in cases)
        got = subprocess.run([str(out / "rows")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(x) for x in line.split()) for line in got.splitlines()]
    return run


def expected_row(cap, num_seqs, window, is_list, list_steps, step, seq, at):
    """The kept slots [lo, last] and the steps from wbase on, in whole numbers."""
    if not 0 <= seq < num_seqs or at < 0:
        return 0, -1, 0, 0, 1
    last = min(at, cap - 1)
    lo = min(max(0, at + 1 - window) if is_list or window > 0 else 0, last + 1)
    unit = min(step, 32)
    wbase = lo // unit * unit
    steps = -(-(last + 1 - wbase) // step) if lo <= last else 0
    return seq, last, lo, wbase, max(1, steps + (list_steps if is_list else 0))


def test_rows_at_the_ends_of_the_range(rows_of):
    """Sequences of up to 2^31 - 16 slots, the most that is accepted: the steps of
    16, 32 and 128 slots to the last of them, with and without a window or a
    list; and every small row."""
    cases = []
    for cap in (2 ** 31 - 16, 2 ** 31 - 32, 2 ** 31 - 64, 2 ** 31 - 128, 2 ** 31 - 65536):
        for step in (16, 32, 128):
            for window in (0, 1, 17, 128, 2 ** 31 - 1):
                for is_list, list_steps in ((0, 0), (1, 5)):
                    for at in (cap - 200, cap - 128, cap - 127, cap - 33, cap - 2, cap - 1, cap, 2 ** 31 - 1):
                        if at < 2 ** 31:
                            cases.append((cap, 1, window, is_list, list_steps, step, 0, at))
    for cap in (16, 48):
        for step in (16, 32, 128):
            for window in (0, 1, 16, 20, 100):
                for is_list in (0, 1):
                    for seq in (-1, 0, 1, 2):
                        for at in range(-2, 60):
                            cases.append((cap, 2, window, is_list, 3, step, seq, at))
    got = rows_of(cases)
    assert len(got) == len(cases)
    for c, row in zip(cases, got):
        assert row == expected_row(*c), (c, row, expected_row(*c))


def test_attention_flags():
    """The self-test flag is accepted, any other one refused; the field lies where
    the descriptor had a gap, so that its size and its other offsets are as they were."""
    import ctypes

    import sparse_attention_lightning_tcgen05_b200 as dsa
    cache = dsa.make_paged_cache(64, 16, 40, 1 << 20, num_seqs=2, H_kv=2)

    def size(flags):
        return dsa.dsa_paged_attention_workspace_size(
            dsa.make_paged_attention_desc(cache, 3, 4, 0.1, flags=flags))
    assert size(dsa.DSA_FLAG_SELFTEST_STALL) == size(0)
    for flags in (1, 3, 4, 1 << 31):
        with pytest.raises(dsa.DsaError) as e:
            size(flags)
        assert e.value.status == dsa.DSA_ERR_INVALID_ARG
    t = dsa.dsa_paged_attention_desc_t
    assert t.flags.offset == t.block_heads.offset + 4 and t.wait_limit_ns.offset == t.block_heads.offset + 8
    assert ctypes.sizeof(t) == t.wait_limit_ns.offset + 8


def _calls(dsa, cache):
    """Every call of the paged operators on fake pointers that fail no check."""
    f = 1 << 20
    attn = dsa.make_paged_attention_desc(cache, 3, 4, 0.1)
    listed = dsa.make_paged_attention_desc(cache, 3, 4, 0.1, block_size=64, num_blocks=4)
    return {
        "dsa_cache_append": lambda: dsa.dsa_cache_append(
            dsa.make_append_desc(cache, 3, 4, 0), f, f, f, None, None, f, None, 2 * f, None, f, None, f, None),
        "dsa_block_pool": lambda: dsa.dsa_block_pool(
            dsa.make_block_pool_desc(cache, 4, 8), f, None, None, f, f, None),
        "dsa_paged_attention_forward": lambda: dsa.dsa_paged_attention_forward(
            attn, f, f, None, f, None, None, f, None, f, None, f, 1 << 30),
        "dsa_block_attention_forward": lambda: dsa.dsa_block_attention_forward(
            listed, f, f, None, f, None, None, f, None, f, f, None, f, 1 << 30)}


@pytest.mark.parametrize("current,where", [(0, "host"), (1, "cuda0"), (None, "host")])
def test_a_block_table_of_another_device_is_refused(monkeypatch, current, where):
    """The descriptors remember where their table lies: a call on another device
    (or on none) is refused before anything else is looked at."""
    import torch

    import sparse_attention_lightning_tcgen05_b200 as dsa

    class OnDevice0:                                # stands in for a CUDA tensor
        def get_device(self):
            return 0

        def data_ptr(self):
            return 1 << 20

    def device():
        if current is None:
            raise RuntimeError("no CUDA device")
        return current
    monkeypatch.setattr(dsa, "_current_device", device)
    table = torch.zeros((2, 16), dtype=torch.int32) if where == "host" else OnDevice0()
    cache = dsa.make_paged_cache(64, 16, 40, table, num_seqs=2, H_kv=2)
    for name, call in _calls(dsa, cache).items():
        with pytest.raises(ValueError, match=name + ".*block table"):
            call()


def test_a_block_table_of_the_current_device_or_a_pointer_is_taken(monkeypatch):
    import torch

    import sparse_attention_lightning_tcgen05_b200 as dsa
    if torch.cuda.is_available():
        pytest.skip("the pointers are fake")
    monkeypatch.setattr(dsa, "_current_device", lambda: 0)

    class OnDevice0:
        def get_device(self):
            return 0

        def data_ptr(self):
            return 1 << 20
    for table in (OnDevice0(), 1 << 20):
        cache = dsa.make_paged_cache(64, 16, 40, table, num_seqs=2, H_kv=2)
        for call in _calls(dsa, cache).values():
            with pytest.raises(dsa.DsaError) as e:  # past every check: no device
                call()
            assert e.value.status == dsa.DSA_ERR_CUDA


def test_pointers_as_numpy_integers():
    """They reach the library like Python's; what is no pointer is a TypeError."""
    import numpy as np

    import sparse_attention_lightning_tcgen05_b200 as dsa
    f = np.int64(1 << 20)
    cache = dsa.make_paged_cache(64, 16, 40, f, num_seqs=2, H_kv=2)
    assert cache.block_table == 1 << 20
    desc = dsa.make_block_pool_desc(cache, 4, 8)
    with pytest.raises(dsa.DsaError) as e:          # pooled is misaligned, and seen to be
        dsa.dsa_block_pool(desc, f, None, None, np.uint64(1 << 20), np.int64((1 << 20) + 8), None)
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG
    for bad in (1.5, "pool"):
        with pytest.raises(TypeError):
            dsa.dsa_block_pool(desc, bad, None, None, f, f, None)


def test_what_only_looks_like_a_tensor_ends_with_an_error(monkeypatch):
    import sparse_attention_lightning_tcgen05_b200 as dsa

    class NoPointer:
        def get_device(self):
            return 0
    monkeypatch.setattr(dsa, "_current_device", lambda: 0)
    cache = dsa.make_paged_cache(64, 16, 40, 1 << 20, num_seqs=2, H_kv=2)
    with pytest.raises(AttributeError):
        dsa.dsa_block_pool(dsa.make_block_pool_desc(cache, 4, 8), NoPointer(), None, None, 1 << 20, 1 << 20, None)


def test_every_scale_byte_decides_outputs():
    """The check of attention over the chosen scales sees each of them: with the
    values of any one byte of a sequence left out of the oracle, or off by a step of
    the scale, the exact outputs fail it."""
    import numpy as np
    import torch

    import oracle.paged as orc
    from paged_scales import BY_BLOCK, BY_SLOT, POSITIONS, scaled_cache
    from paged_util import bf16_bits, check_attention
    rng = np.random.default_rng(66)
    c, byte = scaled_cache(rng)
    q = rng.standard_normal((c.num_seqs, 2, 128))
    k, v = c.rows("k"), c.rows("v")
    assert np.isfinite(v).all()

    def attention(values, i):
        return orc.attention(q[i:i + 1], k, values, c.table[i:i + 1], POSITIONS[i:i + 1], None, 128 ** -0.5)
    tried = 0
    for i, bytes_ in enumerate(BY_BLOCK + BY_SLOT):
        exact = attention(v, i)
        out, lse = bf16_bits(exact[0]), torch.from_numpy(exact[1]).float()
        check_attention(out, lse, exact)
        for b in set(bytes_):
            for wrong in (0.0, 0.5, 2.0):
                with pytest.raises(AssertionError):
                    check_attention(out, lse, attention(np.where(byte == b, wrong * v, v), i))
                tried += 1
    assert tried > 100
