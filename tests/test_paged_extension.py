"""The extension of the paged entries is loaded by them alone, and only if it was built for this torch."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from compressive_memory_long_b200 import build


def run_copy(tmp_path, code, **env):
    """``code`` in a process of its own, over a copy of the package with the CUDA library alone."""
    pkg = tmp_path / "compressive_memory_long_b200"
    pkg.mkdir()
    for name in os.listdir(build.PKG):
        if name.endswith(".py"):
            shutil.copy(os.path.join(build.PKG, name), pkg)
    shutil.copy(build.LIB, pkg)
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                          env={**os.environ, "PYTHONPATH": str(tmp_path), **env})


def test_other_entries_need_no_extension(tmp_path):
    """The binding loads and answers without the paged entries' extension; a paged call names it."""
    got = run_copy(tmp_path, """
import torch
from compressive_memory_long_b200 import binding
assert binding.infini_attn_version() > 0
x = torch.zeros(1, 1, 4, 32)
try:
    binding.rotary(x, None, torch.ones(16, dtype=torch.float64))
except ImportError as e:
    assert "_paged" in str(e)
    print("refused")
""", INFINI_NO_AUTOBUILD="1")
    assert got.returncode == 0 and got.stdout.strip() == "refused", got.stderr


def test_the_extension_of_another_torch_is_not_loaded(tmp_path, monkeypatch):
    here = build.ext_path()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert build.ext_path() != here
    monkeypatch.setenv("INFINI_NO_AUTOBUILD", "1")
    with pytest.raises(ImportError):
        build.load_ext()
