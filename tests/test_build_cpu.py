"""What the build and the binding do where the C++ side of the binding (_native.so) is not there."""
import os
import subprocess
import sys

import pytest

from long_context_compressed_06_b200 import build as csa_build

WITHOUT = """
import sys, types
{block}
import torch
import long_context_compressed_06_b200 as csa
from long_context_compressed_06_b200 import binding
L = csa.load()
assert binding._native is binding._Unbound
assert csa.strerror(-2) and L.csa_version() >= 0
assert csa.attend_workspace_bytes(2, 1, 128, 512, 4096) >= 0
i = torch.zeros(4, dtype=torch.int32)
for call in (lambda: csa.csa_plan_pages(i, i, i, i.view(2, 2), 4, 16, 16, 9, 9), lambda: csa.csa_paged_write(i, i, i),
             lambda: csa.hca_attend_paged(i, i, i, 4, i, i, 16, 1.0)):
    try:
        call()
    except TypeError:   # the long way's check: not a CUDA tensor
        continue
    raise SystemExit("no refusal")
"""


@pytest.mark.parametrize("block", [
    "sys.modules['long_context_compressed_06_b200._native'] = None",                       # not built
    "m = types.ModuleType('x'); m.torch_version = '1.0'; m.bind = None; "
    "sys.modules['long_context_compressed_06_b200._native'] = m"])                        # built for another torch
def test_binding_without_native(block):
    csa_build.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT.format(block=block)], cwd=csa_build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_library_is_built_without_a_host_compiler(monkeypatch, capsys):
    monkeypatch.setenv("CXX", "/nowhere/g++")
    monkeypatch.setattr(csa_build, "NATIVE", csa_build.NATIVE + ".test")
    assert csa_build.build() == csa_build.LIB and os.path.exists(csa_build.LIB)
    assert "_native.so is not built" in capsys.readouterr().err


def test_native_is_built_with_nvcc_by_name(monkeypatch, tmp_path):
    """NVCC may be a name that the shell finds."""
    monkeypatch.setattr(csa_build, "NVCC", "nvcc")
    monkeypatch.setattr(csa_build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(csa_build, "BUILD", str(tmp_path))
    monkeypatch.setenv("PATH", "/usr/local/cuda/bin" + os.pathsep + os.environ["PATH"])
    assert os.path.exists(csa_build.build_native(force=True))


def test_row_tiles_whose_units_pass_32_bits_are_not_taken():
    """A row tile of 128 rows meets three requests of 65 heads; its units are numbered in 32 bits with those of the
    others.  Past that the call goes query by query (no workspace: one split)."""
    import long_context_compressed_06_b200 as csa
    csa_build.build()
    batch = 2 ** 29 // 65  # 2^22 row tiles, 511 units each fit
    for keys, fits in ((160 * 128, True), (172 * 128, False), (253 * 128, False)):
        pages = (keys - 16) // 16  # own entries, and a ring of 16 rows
        need = csa.attend_paged_workspace_bytes(batch, 1, 65, 512, 16, pages, 0, 16, 16, False, True)
        assert (need > 0) == fits, keys
