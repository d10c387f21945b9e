"""CPU: the 4-bit store compiles without a warning (its codes are built from
the bits of floats, in unsigned arithmetic)."""
import os
import shutil
import subprocess

import pytest

from medusa_head_speculative_02_b200 import build


@pytest.mark.skipif(not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")), reason="no nvcc")
def test_store_compiles_without_warnings(tmp_path):
    r = subprocess.run([build.nvcc()] + build.NVCC_FLAGS +
                       ["-Werror", "all-warnings", "-c", os.path.join(build.CSRC, "kv_pack.cu"),
                        "-o", str(tmp_path / "kv_pack.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stderr.strip() == ""
