"""Workspaces of cross attention's backward where a key head has few queries."""
import os
import shutil

import pytest
import torch

import flashattention_backward_fa_gb300 as fa
from flashattention_backward_fa_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("no nvcc to build the library")
        from flashattention_backward_fa_gb300.build import build_library
        build_library()
    return fa.load_library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("Nq", [1, 3, 16, 127])
def test_few_queries(Nq, dtype):
    """Three fp32 values a query at most (four queries at least, then whole tiles: less than twice as many as there
    are) beside 256 bytes and more of padding, where no axis is cut: not 128 queries a head."""
    B = Hq = 4096
    assert fa.fa_cross_bwd_workspace_size(B, Nq, 32, Hq, Hq, 64, dtype) < \
        B * Hq * (3 * 4 * max(4, 2 * Nq) + 16) + 4 * 256
