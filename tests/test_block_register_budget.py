"""Registers and spills of the hot instances of the operators of include/block_ops.h (host-only: nvcc
and ptxas, no GPU). Some spill, as their comments say; the bounds below are what they were timed
with, so that a change that adds to it is seen here and timed."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rmsnorm_row_b200", "csrc")

NORM_QUANT = {  # <vectors, RMS, shared operands, modulation per token, bias or shift>: spill stores, registers
    (5, 0, 1, 0, 1): (0, 128),   # LayerNorm, D = 5120, modulation per frame or batch
    (5, 1, 1, 0, 0): (0, 128),   # RMSNorm with a weight
    (5, 1, 0, 1, 1): (0, 128),   # RMSNorm, modulation per token
    (5, 0, 0, 1, 1): (104, 128),  # LayerNorm, modulation per token
    (5, 0, 0, 0, 1): (0, 128),   # LayerNorm, a few rows
}
ROPE = {  # <heads of a lane, norm over all (2) or per head (1), half pairs, passing pairs>
    (10, 2, 0, 0): (56, 168),    # 40 heads of 128
    (10, 2, 1, 0): (72, 168),
    (4, 1, 0, 0): (0, 168),
    (4, 1, 1, 0): (0, 168),
    (2, 2, 0, 0): (0, 168),      # the same heads, a few rows
}
GRADIENT = {  # <heads of a thread, norm, half pairs, dweight, passing pairs>
    (2, 2, 0, 1, 0): (8, 128),
    (2, 2, 1, 1, 0): (8, 128),
    (2, 1, 0, 1, 0): (0, 128),
    (2, 1, 1, 1, 0): (0, 128),
}
TILES = {(2, 256, 0, 0): (0, 168), (2, 256, 1, 0): (0, 168), (2, 192, 0, 0): (0, 168), (1, 64, 0, 0): (0, 168)}  # <CTAs, columns, e4m3, fp16>
SPLIT = {(2, 256, 0, 0): (0, 168), (1, 128, 0, 0): (0, 168), (1, 64, 0, 0): (0, 168)}


def flags(values, ints):
    return ", ".join(str(v) if i < ints else ("true" if v else "false") for i, v in enumerate(values))


def rope_source():
    lines = ['#include "block/rope_norm_kernel.cuh"', "namespace block_ops {"]
    lines += [f"template __global__ void rope_norm_rows<false, {flags(k, 2)}>(const __grid_constant__ RopeParams);" for k in ROPE]
    lines += [f"template __global__ void rope_norm_gradient<false, {flags(k, 2)}>(const __grid_constant__ RopeParams);" for k in GRADIENT]
    return "\n".join(lines + ["}"])


def linear_source():
    lines = ['#include "block/linear_gate_kernel.cuh"', "namespace block_ops {"]
    m = "const __grid_constant__ CUtensorMap"
    lines += [f"template __global__ void linear_gate_tiles<{flags(k, 2)}>(const __grid_constant__ LinearParams, {m}, {m}, {m}, {m});" for k in TILES]
    lines += [f"template __global__ void linear_gate_split<{flags(k, 2)}>(const __grid_constant__ LinearParams, {m}, {m});" for k in SPLIT]
    return "\n".join(lines + ["}"])


def report(tmp_path, source):
    """{(kernel, template arguments): (spill stores, registers)}"""
    src = tmp_path / "budget.cu"
    src.write_text(source + "\n")
    out = subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                          "-Xptxas", "-v", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "budget.o")],
                         capture_output=True, text=True, timeout=900)
    assert out.returncode == 0, out.stderr[-3000:]
    got, current, spill, of = {}, None, 0, None
    for line in out.stderr.splitlines():
        if m := re.search(r"Compiling entry function '(\S+)'", line):
            current = m.group(1)
        elif m := re.search(r"Function properties for (\S+)", line):
            of = m.group(1)
        elif m := re.search(r"(\d+) bytes spill stores", line):
            spill = int(m.group(1)) if of == current else spill
        elif (m := re.search(r"Used (\d+) registers", line)) and current:
            name = re.search(r"(norm_quant_rows|rope_norm_rows|rope_norm_gradient|linear_gate_tiles|linear_gate_split)I((?:L[ib]\d+E)+)E", current)
            if name:
                args = tuple(int(v) for v in re.findall(r"L[ib](\d+)E", name.group(2)))
                got[name.group(1), args] = (spill, int(m.group(1)))
            current = None
    return got


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="needs nvcc")
@pytest.mark.parametrize("source,kernels", [
    ('#include "block/norm_quant.cu"', {"norm_quant_rows": NORM_QUANT}),
    (rope_source(), {"rope_norm_rows": {(0, *k): v for k, v in ROPE.items()}, "rope_norm_gradient": {(0, *k): v for k, v in GRADIENT.items()}}),
    (linear_source(), {"linear_gate_tiles": TILES, "linear_gate_split": SPLIT}),
], ids=["norm_quant", "rope_norm", "linear_gate"])
def test_hot_instances_keep_their_registers(tmp_path, source, kernels):
    got = report(tmp_path, source)
    for kernel, bounds in kernels.items():
        for args, (spill, registers) in bounds.items():
            stores, used = got[kernel, args]
            assert stores <= spill and used <= registers, f"{kernel}{args}: {stores} bytes of spill stores, {used} registers"
