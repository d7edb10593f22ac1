"""The library loads and builds without _bind.so, the native argument marshalling of the norm and
paged-cache calls, which none of the other calls uses (CPU)."""
import os
import subprocess
import sys

import pytest

from block_sparse_long_moba_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, text=True, timeout=300,
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    assert r.returncode == 0, r.stdout
    return r.stdout


def test_the_binding_is_loaded_where_it_is_built():
    _run("import warnings; warnings.simplefilter('error')\n"
         "from block_sparse_long_moba_b200 import moba\n"
         "moba.load_library()\n"
         "assert moba._bind is not None")


@pytest.mark.parametrize("fault", ["missing", "another torch", "without a version"])
def test_library_loads_without_the_binding(fault):
    """With a warning; calls are checked (and refused) by the Python side."""
    stand_in = {"missing": "None", "another torch": "M('1.0')", "without a version": "object()"}
    _run("import sys, warnings, torch\n"
         "class M:\n"
         "    def __init__(self, v): self.torch_version = v\n"
         "import block_sparse_long_moba_b200 as package\n"
         f"m = {stand_in[fault]}\n"
         "sys.modules['block_sparse_long_moba_b200._bind'] = m\n"
         "if m is not None: package._bind = m\n"
         "from block_sparse_long_moba_b200 import moba\n"
         "with warnings.catch_warnings(record=True) as w:\n"
         "    warnings.simplefilter('always')\n"
         "    lib = moba.load_library()\n"
         "assert any('_bind.so' in str(x.message) for x in w)\n"
         "assert moba._bind is None and lib.moba_version() > 0\n"
         "assert moba.load_library() is lib\n"
         "try:\n"
         "    moba.moba_qk_norm_rope(*[torch.zeros(2, 3)] * 6)\n"
         "except (moba.MobaError, ValueError, TypeError) as e:\n"
         "    assert '3-D' in str(e)\n"
         "else:\n"
         "    raise SystemExit('accepted')\n")


def test_a_binding_of_another_torch_is_built_again(monkeypatch):
    import torch
    assert not build.bind_needs_build()
    monkeypatch.setattr(torch, "__version__", "0.1.0")
    assert build.bind_needs_build()


def test_no_binding_beside_a_torch_without_cuda(monkeypatch):
    import torch
    monkeypatch.setattr(torch.version, "cuda", None)
    monkeypatch.setattr(subprocess, "run", lambda *a, **k: pytest.fail("ran a compiler"))
    assert build.build_bind(force=True) is None
    assert build.build() == build.LIB
