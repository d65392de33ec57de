"""The report of a wait that ran out in the matrix kernel, on the host: a flag as the kernel sets it
makes the next launch's check fail, once. No GPU; the kernel's side is not made to fail."""
import os
import subprocess

import pytest

import rmsnorm_row_b200 as fn
from rmsnorm_row_b200 import _abi, _block_abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "host_checks.h"
int main() {
  int word = 0;
  std::printf("%d ", block_ops::wait_status(&word));
  for (int round = 0; round < 2; ++round) {
    word = 1;
    std::printf("%d ", block_ops::wait_status(&word));
    std::printf("%d %d ", block_ops::wait_status(&word), word);
  }
  std::printf("%d\n", block_ops_last_cuda_error());
}
"""


def test_a_wait_that_ran_out_is_reported_once(tmp_path):
    _block_abi.load()
    exe = str(tmp_path / "waits")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-x", "c++", "-", "-x", "none", "-I", os.path.join(ROOT, "rmsnorm_row_b200", "csrc", "block"),
                    _abi.LIB_PATH, "-Wl,-rpath," + os.path.dirname(_abi.LIB_PATH), "-o", exe], input=PROGRAM, text=True, check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    OK, CUDA = fn.FN_OK, fn.FN_ERR_CUDA
    assert got == [OK, CUDA, OK, 0, CUDA, OK, 0, 702]


@pytest.mark.gpu
def test_timeouts_are_counted_per_device():
    import torch

    x, w = torch.randn(1, 300, 512, device="cuda").bfloat16(), torch.randn(256, 512, device="cuda").bfloat16()
    fn.linear_gate_residual(x, w)
    assert fn.linear_gate_timeouts() == 0 and fn.linear_gate_timeouts(x.device) == 0
