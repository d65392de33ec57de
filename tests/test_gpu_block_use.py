"""The operators of include/block_ops.h as a program uses them side by side: on several streams at
once, in captured graphs, with operands of every mix of layouts. Results are compared bit for bit
with the same call made alone."""
import subprocess
import sys

import pytest
import torch

import rmsnorm_row_b200 as fn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rand(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.empty(shape, device="cuda").normal_(generator=g).to(BF)


def same(a, b):
    if isinstance(a, torch.Tensor):
        a, b = (a,), (b,)
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def streams():
    out = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in out:
        s.wait_stream(torch.cuda.current_stream())
    return out


def calls():
    rows = dict(residual=rand(1, 9000, 5120), x=rand(1, 9000, 5120, seed=1))
    g, sc, sh = (rand(1, 1, 5120, seed=k) for k in (2, 3, 4))
    x, w = rand(1, 64, 5120), rand(5120, 5120, seed=5)
    big, wide = rand(1, 20000, 1024), rand(4096, 1024, seed=6)
    q, dq, wq = rand(1, 3000, 40, 128), rand(1, 3000, 40, 128, seed=7), rand(5120, seed=8)
    pos = torch.arange(9000, device="cuda", dtype=torch.int32).view(3000, 3)
    return {
        "rows": lambda **kw: fn.fused_residual_norm_scale_shift_quant(rows["residual"], rows["x"], g, None, None, sc, sh, "layer", **kw),
        "rotation": lambda **kw: fn.rope_norm(q, pos, (22, 21, 21), wq, **kw),
        "gradient": lambda **kw: fn.rope_norm_backward(dq, q, pos, (22, 21, 21), wq, **kw),
        "split product": lambda **kw: fn.linear_gate_residual(x, w, **kw),
        "product": lambda **kw: fn.linear_gate_residual(big, wide, activation="silu", **kw),
        "token": lambda **kw: fn.linear_gate_residual(x[:, :1], w, **kw),
    }


def test_two_streams_at_once():
    every = calls()
    alone = {k: f() for k, f in every.items()}
    pair = streams()
    got = [(k, f(stream=pair[(i + j) % 2])) for j in range(4) for i, (k, f) in enumerate(every.items())]
    torch.cuda.synchronize()
    for k, out in got:
        assert same(out, alone[k]), k


def test_captured_side_by_side_and_replayed():
    every = calls()
    alone = {k: f() for k, f in every.items()}
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append({k: f() for k, f in every.items()})
    pair = streams()
    for _ in range(3):
        for g, s in zip(graphs, pair):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        for k in every:
            assert same(out[k], alone[k]), k


def test_first_call_may_be_captured():
    """In a process of its own: no call has loaded a kernel before the capture."""
    code = """
import torch, rmsnorm_row_b200 as fn
r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
x, w, q, pos, wq = r(1, 64, 512), r(512, 512), r(1, 700, 6, 64), torch.zeros(700, 1, device="cuda", dtype=torch.int32), r(64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = fn.norm_scale_shift_quant(x, None, None, None, None, "rms")
    b = fn.rope_norm_backward(fn.rope_norm(q, pos, (32,), wq, norm="head"), q, pos, (32,), wq, norm="head")
    c = fn.linear_gate_residual(x, w)
g.replay()
torch.cuda.synchronize()
assert torch.equal(c, fn.linear_gate_residual(x, w))
assert torch.equal(a[1], fn.norm_scale_shift_quant(x, None, None, None, None, "rms")[1])
print("captured")
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]


def test_layouts_that_mix():
    # batches of one row, each with modulation of its own
    x, w = rand(7000, 1, 512), rand(512, seed=1)
    sc, sh = rand(7000, 1, 512, seed=2), rand(7000, 1, 512, seed=3)
    flat = [t.view(1, 7000, 512) for t in (x, sc, sh)]
    a, b = fn.norm_scale_shift_quant(x, w, None, sc, sh, "rms"), fn.norm_scale_shift_quant(flat[0], w, None, flat[1], flat[2], "rms")
    assert same(a, [t.view(s.shape) for t, s in zip(b, a)])
    # a broadcast scale with a shift per frame, many rows; the same with every operand per token
    x, sc, sh = rand(2, 4200, 1024), rand(1024, seed=1), rand(1, 3, 1, 1024, seed=2)
    each = [t.expand(2, 4200, 1024).contiguous() for t in (sc, sh.repeat_interleave(1400, 1).squeeze(2))]
    assert same(fn.norm_scale_shift_quant(x, None, None, sc, sh), fn.norm_scale_shift_quant(x, None, None, *each))
    # one head read by all, positions shared by the batch
    x, w = rand(2, 300, 1, 64).expand(2, 300, 6, 64), rand(384, seed=1)
    pos = torch.arange(600, device="cuda", dtype=torch.int32).view(1, 300, 2)
    assert same(fn.rope_norm(x, pos, (16, 16), w), fn.rope_norm(x.contiguous(), pos.expand(2, 300, 2), (16, 16), w))
    # a weight that is a slice of columns
    both = rand(512, 1024)
    assert same(fn.linear_gate_residual(rand(1, 40, 512), both[:, 512:]), fn.linear_gate_residual(rand(1, 40, 512), both[:, 512:].contiguous()))


def test_refusals():
    x, w = rand(1, 40, 512), rand(64, 512)
    with pytest.raises(fn.FusedNormError, match="MISALIGNED"):
        fn.linear_gate_residual(x, w, rand(72)[1:65])
    with pytest.raises(fn.FusedNormError, match="UNSUPPORTED"):
        fn.linear_gate_residual(x.expand(3, 40, 512), w)
    with pytest.raises(ValueError, match="contiguous"):
        fn.linear_gate_residual(x, rand(512, 64).t())
    with pytest.raises(ValueError, match="x_scale"):
        fn.linear_gate_residual(x, w, x_scale=torch.ones(1, 40, device="cuda"))
    with pytest.raises(ValueError, match="activation"):
        fn.linear_gate_residual(x, w, activation="relu")
    with pytest.raises(fn.FusedNormError):
        fn.linear_gate_residual(rand(1, 40, 64), rand(64, 64), out=rand(1, 40, 72)[:, :, 1:65])
    with pytest.raises(ValueError, match="together"):
        fn.norm_scale_shift_quant(x, None, None, rand(512), None)
    with pytest.raises(ValueError, match="broadcast"):
        fn.norm_scale_shift_quant(x, None, None, rand(1, 39, 512), rand(1, 39, 512))
    q, pos = rand(1, 40, 2, 64), torch.zeros(40, 2, device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError, match="positions"):
        fn.rope_norm(q, pos, (16,))
    with pytest.raises(ValueError, match="sections"):
        fn.rope_norm(q, pos, (20, 20))
    with pytest.raises(TypeError, match="int32"):
        fn.rope_norm(q, pos.float(), (16, 16))
    with pytest.raises(ValueError, match="weight"):
        fn.rope_norm(q, pos, (16, 16), rand(64), norm="all")
    with pytest.raises(ValueError, match="on cpu"):
        fn.rope_norm(q, pos.cpu(), (16, 16))


def test_offsets_beyond_32_bits():
    """More than 2^32 elements: the last rows are those of a call on them alone."""
    L, D = 270000, 16384
    tail = slice(L - 70, L)
    x, w = rand(1, 1, D).expand(1, L, D).contiguous(), rand(D, seed=1)
    x[:, tail] = rand(1, 70, D, seed=2)
    q, s = fn.norm_scale_shift_quant(x, w, None, None, None, "rms")
    q2, s2 = fn.norm_scale_shift_quant(x[:, tail], w, None, None, None, "rms")
    assert same((q[:, tail], s[:, tail]), (q2, s2)) and torch.all(s[:, :-70] == s[0, 0])
    del q, s
    heads, pos = x.view(1, L, 128, 128), torch.arange(L, device="cuda", dtype=torch.int32)[:, None]
    want = fn.rope_norm(heads[:, tail], pos[tail], (64,), w)
    back = fn.rope_norm_backward(heads[:, tail], heads[:, tail], pos[tail], (64,), w)[0]
    got = fn.rope_norm_backward(heads, heads, pos, (64,), w)[0]
    assert same(got[:, tail], back)
    del got
    assert same(fn.rope_norm(heads, pos, (64,), w, out=heads)[:, tail], want)
    small, weight = rand(1, L, 64), rand(D, 64, seed=3)
    out = fn.linear_gate_residual(small, weight, residual=x, out=x)
    again = fn.linear_gate_residual(small[:, tail], weight, residual=want.view(1, 70, D))
    # one step of K in both: the same sums, whatever the tiles
    assert same(out[:, tail], again)
