"""Kernels that launch while the kernel before them drains (launch_early) may be resident before that
kernel's writes are visible: each waits for it, and none reads through the read-only path (__ldg,
ld.global.nc, a __restrict__ pointer to constant data), which is neither ordered behind the wait nor
meant for memory that another kernel still writes. Shown on the source text (CPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_long_moba_b200", "csrc")


def _code(path):
    """The file without its comments."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


EARLY = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "launch_early(" in _code(p))


def test_there_are_such_files():
    assert {os.path.basename(p) for p in EARLY} >= {"paged.cu", "kv_cache.cu", "qk_norm.cu"}


@pytest.mark.parametrize("path", EARLY, ids=os.path.basename)
def test_no_read_only_loads(path):
    code = _code(path)
    for word in ("__ldg", "ld.global.nc", "__restrict__", "__restrict"):
        assert not re.search(re.escape(word) + r"\b", code), word


@pytest.mark.parametrize("path", EARLY, ids=os.path.basename)
def test_every_kernel_waits(path):
    kernels = _code(path).split("__global__")[1:]
    assert kernels
    for k in kernels:
        assert "wait_previous_kernel()" in k, k[:200]
