"""The debug build's check of the direct stores of a block's feed-forward
half, in a child process that loads only the debug library."""
import os
import subprocess
import sys

import pytest
import torch

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi
from tests import block_bounds_cases

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_build(tmp_path):
    libbuild.build()
    capi.load()
    want = {n: x.cpu() for n, x in block_bounds_cases.results().items()}
    torch.save(want, tmp_path / "want.pt")
    r = subprocess.run([sys.executable, os.path.join(HERE, "block_bounds_cases.py"), str(tmp_path / "want.pt")],
                       capture_output=True, text=True, timeout=900, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert "clean in every mode" in r.stdout
