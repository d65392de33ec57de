"""Host-side checks of include/block_ops.h: every declared function is exported, the ctypes view
has the header's layouts, and every argument rule is applied before a launch. Nothing here makes a
CUDA call; device pointers are aligned addresses that nobody reads."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import rmsnorm_row_b200 as fn
from rmsnorm_row_b200 import _abi, _block_abi
from rmsnorm_row_b200._block_abi import BO_BF16, BO_E4M3, BO_FP16, BO_FP32

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "block_ops.h")
OK, INV, UNS, MIS = fn.FN_OK, fn.FN_ERR_INVALID_ARG, fn.FN_ERR_UNSUPPORTED, fn.FN_ERR_MISALIGNED
BASE = 0x7F0000000000
GAP = 1 << 30


def at(k):
    return BASE + k * GAP


def test_header_functions_are_exported():
    text = open(HEADER).read()
    names = set(re.findall(r"^(?:fn_status|const char\*|int)\s+(\w+)\s*\(", text, re.M))
    assert names == set(_block_abi.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", _abi.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT\s+(\w+)$", out, re.M))
    lib = _block_abi.load()
    for s in range(6):
        assert lib.block_ops_status_string(s)
    assert lib.block_ops_last_cuda_error() == 0


def test_struct_layouts_match_header(tmp_path):
    names = ["nq_config", "nq_args", "rn_config", "rn_rows", "rn_args", "rn_backward_args", "lg_config", "lg_args"]
    last = {"nq_config": "eps", "nq_args": "r_stride_l", "rn_config": "eps", "rn_rows": "stride_h", "rn_args": "y",
            "rn_backward_args": "workspace_bytes", "lg_config": "has_residual", "lg_args": "out_stride_l"}
    body = "".join(f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {last[n]}));' for n in names)
    exe = str(tmp_path / "sizes")
    src = f'#include "{HEADER}"\n#include <stdio.h>\n#include <stddef.h>\nint main(){{{body}return 0;}}'
    subprocess.run(["gcc", "-Wall", "-Werror", "-x", "c", "-", "-o", exe], input=src, text=True, check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    want = []
    for n in names:
        c = getattr(_block_abi, n)
        want += [ctypes.sizeof(c), getattr(c, last[n]).offset]
    assert [int(v) for v in got] == want


def create(op, cfg):
    h = ctypes.c_void_p()
    return getattr(_block_abi.load(), f"{op}_create")(ctypes.byref(h), ctypes.byref(cfg)), h


def made(op, cfg):
    s, h = create(op, cfg)
    assert s == OK
    return h


def changed(make, **kw):
    """make()'s struct with attributes (dotted names reach into its operands) set."""
    v = make()
    for name, value in kw.items():
        at_, o = name.split("__"), v
        for part in at_[:-1]:
            o = getattr(o, part)
        setattr(o, at_[-1], value)
    return v


@pytest.mark.parametrize("op", ["norm_quant", "rope_norm", "linear_gate"])
def test_null_arguments(op):
    lib = _block_abi.load()
    assert getattr(lib, f"{op}_create")(None, None) == INV
    assert getattr(lib, f"{op}_validate")(None, None) == INV
    assert getattr(lib, f"{op}_launch")(None, None, None) == INV
    assert getattr(lib, f"{op}_destroy")(None) == OK


# ---- norm_quant ------------------------------------------------------------------------------

def nq_cfg():
    return _block_abi.nq_config(D=5120, is_rms=0, has_residual=1, has_gate=1, has_weight=1, has_bias=0, affine_fp32=0,
                                has_modulation=1, eps=1e-6)


def nq_args(B=2, L=8, D=5120):
    a = _block_abi.nq_args()
    a.B, a.L = B, L
    row = (L * D, 0, D)
    a.x, a.residual = fn.fn_operand(at(0), *row), fn.fn_operand(at(1), *row)
    a.gate, a.scale, a.shift = fn.fn_operand(at(2), 0, 0, 0), fn.fn_operand(at(3), *row), fn.fn_operand(at(4), *row)
    a.weight = at(5)
    a.q, a.q_stride_b, a.q_stride_l = at(6), L * D, D
    a.row_scale = at(7)
    a.r, a.r_stride_b, a.r_stride_l = at(8), L * D, D
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(D=16), OK), (dict(D=16384), OK), (dict(D=24), UNS), (dict(D=0), UNS), (dict(D=-16), UNS),
    (dict(D=16400), UNS), (dict(is_rms=2), INV), (dict(has_residual=0), INV), (dict(affine_fp32=1), OK),
    (dict(affine_fp32=1, has_weight=0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(eps=0.0), OK), (dict(has_modulation=3), INV),
])
def test_norm_quant_configurations(kw, want):
    assert create("norm_quant", changed(nq_cfg, **kw))[0] == want


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(B=0), OK), (dict(L=0), OK), (dict(B=-1), INV), (dict(L=1 << 40), INV),
    (dict(tokens_per_frame=3), INV), (dict(tokens_per_frame=4), OK), (dict(tokens_per_frame=4, gate__stride_f=5120), OK),
    (dict(gate__stride_f=5120), INV), (dict(x__ptr=None), INV), (dict(weight=None), INV), (dict(bias=at(9)), INV),
    (dict(gate__ptr=None), INV), (dict(shift__ptr=None), INV), (dict(row_scale=None), INV), (dict(r=None), INV),
    (dict(x__ptr=at(0) + 2), MIS), (dict(x__stride_l=5124), MIS), (dict(weight=at(5) + 8), MIS), (dict(q=at(6) + 8), MIS),
    (dict(q_stride_l=5128), INV), (dict(q_stride_l=5128, q_stride_b=1 << 16), MIS), (dict(q_stride_l=5104), INV), (dict(q_stride_b=5120), INV), (dict(row_scale=at(7) + 2), MIS),
    (dict(x__stride_l=-5120), INV), (dict(x__stride_l=0, x__stride_b=0), OK),
    (dict(q=at(0)), INV), (dict(r=at(0)), INV), (dict(r=at(1)), OK), (dict(r=at(1) + 16), INV), (dict(row_scale=at(6)), INV),
    (dict(r=at(5)), INV), (dict(r=at(6) + 5120), INV), (dict(residual__stride_b=1 << 50), INV),
])
def test_norm_quant_arguments(kw, want):
    h = made("norm_quant", nq_cfg())
    a = changed(nq_args, **kw)
    lib = _block_abi.load()
    assert lib.norm_quant_validate(h, ctypes.byref(a)) == want
    if want != OK or not (a.B and a.L):
        assert lib.norm_quant_launch(h, ctypes.byref(a), None) == want
    lib.norm_quant_destroy(h)


# ---- rope_norm -------------------------------------------------------------------------------

def rn_cfg():
    return _block_abi.rn_config(dtype=BO_BF16, heads=40, head_dim=128, axes=3, section=(22, 21, 21, 0), norm=2, has_weight=1,
                                weight_fp32=0, half_pairs=0, shared_frequencies=0, index64=0, theta=1e4, eps=1e-6)


def rows(k, B=2, L=8, H=40, hd=128):
    return _block_abi.rn_rows(at(k), L * H * hd, H * hd, hd)


def rn_args():
    return _block_abi.rn_args(2, 8, rows(0), at(1), 0, 3, at(2), rows(3))


def rn_back():
    return _block_abi.rn_backward_args(2, 8, rows(0), rows(4), at(1), 0, 3, at(2), rows(3), at(5), at(6), 1 << 28)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(dtype=BO_FP16), OK), (dict(dtype=BO_E4M3), UNS), (dict(dtype=BO_FP32), UNS), (dict(heads=0), INV),
    (dict(heads=128), OK), (dict(heads=129), UNS), (dict(head_dim=120), INV), (dict(head_dim=136), UNS), (dict(head_dim=528, heads=1), UNS),
    (dict(head_dim=512, heads=32), OK), (dict(axes=0), INV), (dict(axes=5), INV), (dict(axes=4), INV), (dict(axes=1), OK),
    (dict(axes=1, half_pairs=1), UNS), (dict(half_pairs=1), OK), (dict(norm=0), INV), (dict(norm=0, has_weight=0), OK),
    (dict(norm=3), INV), (dict(weight_fp32=1), OK), (dict(weight_fp32=1, has_weight=0), INV), (dict(theta=0.0), INV),
    (dict(theta=float("nan")), INV), (dict(eps=-1.0), INV), (dict(eps=0.0), OK),
])
def test_rope_configurations(kw, want):
    assert create("rope_norm", changed(rn_cfg, **kw))[0] == want


def test_rope_every_shape_has_a_launch():
    """Any number of heads that fits has its kernels (the host settles launch shapes at creation)."""
    for hd in range(16, 513, 16):
        for H in {1, 2, 3, 5, 7, 16, 37, 16384 // hd // 2 + 1, 16384 // hd}:
            if H * hd > 16384:
                continue
            for norm in (0, 1, 2):
                c = changed(rn_cfg, heads=H, head_dim=hd, axes=1, norm=norm, has_weight=int(norm > 0))
                c.section[0] = hd // 2
                h = made("rope_norm", c)
                n = ctypes.c_uint64()
                assert _block_abi.load().rope_norm_backward_workspace(h, 1, 5000, ctypes.byref(n)) == OK
                assert n.value <= 1024 * 4 * (H * hd if norm == 2 else hd) and (n.value > 0) == (norm > 0)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(B=0), OK), (dict(B=-1), INV), (dict(L=1 << 31), INV), (dict(x__ptr=None), INV), (dict(positions=None), INV),
    (dict(weight=None), INV), (dict(y__ptr=None), INV), (dict(x__ptr=at(0) + 8), MIS), (dict(x__stride_h=132), MIS),
    (dict(x__stride_l=-8), INV), (dict(positions=at(1) + 2), MIS), (dict(pos_stride_l=-3), INV), (dict(pos_stride_l=0), OK),
    (dict(weight=at(2) + 4), MIS), (dict(y__stride_h=64), INV), (dict(y__stride_l=5112), INV), (dict(y__ptr=at(0)), OK),
    (dict(y__ptr=at(0) + 16), INV), (dict(y__ptr=at(2)), INV), (dict(y__ptr=at(1)), INV), (dict(x__stride_h=0), OK),
    (dict(y__stride_l=128, y__stride_h=1024), OK), (dict(y__stride_l=128, y__stride_h=1016), INV),
])
def test_rope_arguments(kw, want):
    h = made("rope_norm", rn_cfg())
    a = changed(rn_args, **kw)
    if "y__stride_h" in kw and "y__stride_l" in kw:  # heads outside tokens
        a.y.stride_b = 40 * 1024
    lib = _block_abi.load()
    assert lib.rope_norm_validate(h, ctypes.byref(a)) == want
    if want != OK or not a.B:
        assert lib.rope_norm_launch(h, ctypes.byref(a), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(grad__ptr=None), INV), (dict(x__ptr=None), INV), (dict(dweight=None), INV), (dict(dweight=at(5) + 2), MIS),
    (dict(workspace=None), INV), (dict(workspace_bytes=16), INV), (dict(workspace=at(6) + 8), MIS), (dict(dx__ptr=at(0)), OK),
    (dict(dx__ptr=at(4)), OK), (dict(dx__ptr=at(0) + 16), INV), (dict(dweight=at(0)), INV), (dict(workspace=at(4)), INV),
    (dict(dweight=at(6)), INV), (dict(workspace=at(3)), INV), (dict(L=-1), INV), (dict(grad__stride_h=0), OK),
])
def test_rope_backward_arguments(kw, want):
    h = made("rope_norm", rn_cfg())
    a = changed(rn_back, **kw)
    lib = _block_abi.load()
    assert lib.rope_norm_backward_validate(h, ctypes.byref(a)) == want
    if want != OK:
        assert lib.rope_norm_backward_launch(h, ctypes.byref(a), None) == want


def test_rope_backward_without_norm_takes_no_x():
    h = made("rope_norm", changed(rn_cfg, norm=0, has_weight=0))
    lib = _block_abi.load()
    plain = dict(weight=None, dweight=None, workspace=None, workspace_bytes=0)
    assert lib.rope_norm_backward_validate(h, ctypes.byref(changed(rn_back, x__ptr=None, **plain))) == OK
    assert lib.rope_norm_backward_validate(h, ctypes.byref(changed(rn_back, **plain))) == INV
    n = ctypes.c_uint64(7)
    assert lib.rope_norm_backward_workspace(h, 2, 8, ctypes.byref(n)) == OK and n.value == 0
    assert lib.rope_norm_backward_workspace(h, -1, 8, ctypes.byref(n)) == INV
    assert lib.rope_norm_backward_workspace(h, 2, 8, None) == INV


# ---- linear_gate -----------------------------------------------------------------------------

def lg_cfg():
    return _block_abi.lg_config(dtype=BO_BF16, K=512, N=768, act=1, has_bias=1, has_gate=1, has_residual=1)


def lg_args(B=2, L=8, K=512, N=768):
    a = _block_abi.lg_args()
    a.B, a.L = B, L
    a.x = fn.fn_operand(at(0), L * K, 0, K)
    a.weight, a.weight_stride = at(1), K
    a.bias = at(2)
    a.gate, a.residual = fn.fn_operand(at(3), 0, 0, 0), fn.fn_operand(at(4), L * N, 0, N)
    a.out, a.out_stride_b, a.out_stride_l = at(5), L * N, N
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(dtype=BO_E4M3), OK), (dict(dtype=BO_FP32), UNS), (dict(K=8, N=8), OK), (dict(K=4), UNS), (dict(K=12), UNS),
    (dict(N=12), UNS), (dict(dtype=BO_E4M3, K=520), UNS), (dict(K=1 << 21), UNS), (dict(act=4), INV), (dict(act=-1), INV),
    (dict(has_gate=2), INV),
])
def test_linear_configurations(kw, want):
    assert create("linear_gate", changed(lg_cfg, **kw))[0] == want


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(B=0), OK), (dict(L=-1), INV), (dict(L=0x7FFFFFFF), INV), (dict(x__ptr=None), INV), (dict(weight=None), INV),
    (dict(bias=None), INV), (dict(gate__ptr=None), INV), (dict(residual__ptr=None), INV), (dict(out=None), INV),
    (dict(x_scale=at(8)), INV), (dict(weight_scale=at(8)), INV), (dict(x__ptr=at(0) + 8), MIS), (dict(x__stride_l=516), MIS),
    (dict(weight_stride=504), INV), (dict(weight_stride=516), MIS), (dict(bias=at(2) + 2), MIS), (dict(x__stride_f=8), INV),
    (dict(tokens_per_frame=3), INV), (dict(tokens_per_frame=4, gate__stride_f=768), OK), (dict(residual__stride_l=0), INV),
    (dict(out_stride_l=760), INV), (dict(out=at(5) + 8), MIS), (dict(out=at(4)), OK), (dict(out=at(4) + 16), INV),
    (dict(out=at(0)), INV), (dict(out=at(1)), INV), (dict(out=at(2)), INV), (dict(out=at(3)), INV),
    (dict(x__stride_l=0, x__stride_b=0), UNS), (dict(B=1, L=4, x__stride_l=0), OK), (dict(x__stride_b=1 << 44), INV),
])
def test_linear_arguments(kw, want):
    h = made("linear_gate", lg_cfg())
    a = changed(lg_args, **kw)
    lib = _block_abi.load()
    assert lib.linear_gate_validate(h, ctypes.byref(a)) == want
    if want != OK or not a.B:
        assert lib.linear_gate_launch(h, ctypes.byref(a), None) == want


def test_linear_scales_come_with_e4m3():
    h = made("linear_gate", changed(lg_cfg, dtype=BO_E4M3))
    lib = _block_abi.load()
    for kw, want in ((dict(x_scale=at(8), weight_scale=at(9)), OK), (dict(x_scale=at(8)), INV), (dict(), INV),
                     (dict(x_scale=at(8) + 2, weight_scale=at(9)), MIS), (dict(x_scale=at(8), weight_scale=at(9) + 4), MIS),
                     (dict(x_scale=at(5), weight_scale=at(9)), INV)):
        assert lib.linear_gate_validate(h, ctypes.byref(changed(lg_args, **kw))) == want


# ---- the tensor-level functions, as far as they come without a GPU ------------------------------

def test_tensor_functions_refuse_what_is_not_a_cuda_tensor():
    bf = torch.bfloat16
    x, w = torch.zeros(1, 4, 64, dtype=bf), torch.zeros(32, 64, dtype=bf)
    q, pos = torch.zeros(1, 4, 2, 32, dtype=bf), torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: fn.norm_scale_shift_quant(x, None, None, None, None),
                 lambda: fn.fused_residual_norm_scale_shift_quant(x, x, None, None, None, None, None),
                 lambda: fn.rope_norm(q, pos, (16,)), lambda: fn.rope_norm_backward(q, q, pos, (16,)),
                 lambda: fn.linear_gate_residual(x, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: fn.norm_scale_shift_quant([1.0], None, None, None, None), lambda: fn.rope_norm(None, pos, (16,)),
                 lambda: fn.linear_gate_residual(x, 3), lambda: fn.linear_gate_residual(x.float(), w.float())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="B, L, D"):
        fn.norm_scale_shift_quant(x[0], None, None, None, None)
    with pytest.raises(ValueError, match="H, hd"):
        fn.rope_norm(x, pos, (16,))
    with pytest.raises(ValueError, match="residual is required"):
        fn.fused_residual_norm_scale_shift_quant(None, x, None, None, None, None, None)
