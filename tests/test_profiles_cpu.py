"""Every committed profile was taken on the sources as they are, the kernel's
device code and the host code that launches it, or says in a line "stale: .."
what changed since (CPU only)."""
import pathlib
import re

import pytest

import bench

ROOT = pathlib.Path(__file__).resolve().parent.parent
CSRC = ROOT / "sparse_attention_lightning_tcgen05_b200" / "csrc"
PROFILES = sorted((ROOT / "profiles").glob("*.md"))
PAGED = ("cache_append_kernel", "block_pool_kernel", "paged_attention_")


@pytest.mark.parametrize("path", PROFILES, ids=lambda p: p.stem)
def test_profiles_are_current(path):
    text = path.read_text()
    got = re.search(r"src_hash:\s*`([0-9a-f]{16})`", text).group(1)
    files = bench.PAGED_SOURCES if path.name.startswith(PAGED) else bench.KERNEL_SOURCES
    stale = re.search(r"^stale: \S", text, re.M) is not None
    assert (got == bench.source_hash(files)) != stale


def closure(*files):
    """The files beside the kernels that these include, and themselves."""
    seen, todo = set(), list(files)
    while todo:
        f = todo.pop()
        if f in seen or not (CSRC / f).exists():        # (public headers lie elsewhere)
            continue
        seen.add(f)
        todo += re.findall(r'#include "([^"]+)"', (CSRC / f).read_text())
    return seen


@pytest.mark.parametrize("files,entries", [
    (bench.KERNEL_SOURCES, ("dsa_indexer_api.cu", "dsa_sparse_mqa_api.cu", "dsa_prepare_api.cu")),
    (bench.PAGED_SOURCES, ("dsa_paged_attention_api.cu", "dsa_paged_cache_api.cu"))])
def test_the_hashed_files_are_all_that_a_call_is_made_of(files, entries):
    assert set(files) == closure(*entries) and list(files) == sorted(files)
