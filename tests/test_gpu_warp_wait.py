"""A warp's bounded wait gives all of its lanes one answer (tfk::mbar_warp_wait_or_abort).

`tests/warp_wait_check.cu` is built here (nvcc, sm_103a) and called through ctypes.
"""

import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
BLOCKS = 8192


@pytest.fixture(scope="module")
def lib():
    out = os.path.join(tempfile.mkdtemp(prefix="warpwait_"), "warp_wait.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-o", out, os.path.join(HERE, "warp_wait_check.cu")], check=True)
    so = ctypes.CDLL(out)
    so.warp_wait_check.argtypes = [ctypes.c_uint] * 3 + [ctypes.c_void_p] * 2
    return so


@pytest.mark.parametrize("gap", [0, 1, 8, 64])
@pytest.mark.parametrize("what,allowed", [(0, {0}), (1, {0, 2 ** 32 - 1}), (2, {0, 2 ** 32 - 1}), (3, {2 ** 32 - 1})])
def test_one_answer_a_warp(lib, what, allowed, gap):
    torch.cuda.set_device(0)
    answers = torch.full((BLOCKS,), 5, dtype=torch.int32, device="cuda")
    sink = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert lib.warp_wait_check(what, gap, BLOCKS, answers.data_ptr(), sink.data_ptr()) == 0
    assert {int(a) & 0xFFFFFFFF for a in answers.unique().tolist()} <= allowed
