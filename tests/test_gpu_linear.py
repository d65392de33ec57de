"""GPU checks of the matrix product with its epilogue against the formula in 64 bits.

Tolerances, with u = 2^-24 and S = sum |x w| of an element:

* the sum: products of 16-bit and e4m3 numbers are exact in fp32. One tensor-core product adds
  16 of them (32 e4m3) with an error of at most 2^-23 of their magnitudes and the accumulator's,
  and there are K / 16 of them at most; lanes of a token's dot product have chains of
  K / 32 + 5. Ez = (K / 16 + 4) 2^-23 S covers both, and the scales and bias add 4 u (|z| + |bias|).
* activations have slopes of at most 1.13. Their own error: the quotients by 1 + e^-t are within
  (4 + 2 |t|) 2^-23 relative, 2^-17 where the value exceeds 1e-12; erff is within 2^-22 of |z|.
* gate and residual: one fused multiply-add, u of the result; the output half a step
  (bf16 2^-8, fp16 2^-11, or 2^-25 below its normal numbers).
"""
import math

import pytest
import torch

import rmsnorm_row_b200 as fn
from rmsnorm_row_b200 import _block_abi

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def rand(shape, seed, sd=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0, sd, generator=g).to(dtype)


def rows(t, B, L):
    """An operand as (B, L, N) in 64 bits."""
    t = t.double()
    if t.dim() == 4:
        t = t.repeat_interleave(L // t.shape[1], 1)[:, :, 0]
    elif t.dim() == 2 and t.shape[0] == B and B > 1:
        t = t[:, None]
    elif t.dim() < 3:
        t = t.reshape(1, 1, -1)
    return t.expand(B, L, t.shape[-1])


def act64(z, kind):
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def check(out, t, act="none"):
    x, w = t["x"], t["weight"]
    B, L, K = x.shape
    X, W = x.double(), w.double()
    if x.dtype == F8:
        X, W = X * t["x_scale"].double()[..., None], W * t["weight_scale"].double()[:, None]
    z = X @ W.T
    S = X.abs() @ W.abs().T
    Ez = (K / 16 + 4) * 2 * U * S
    if t["bias"] is not None:
        Ez = Ez + 4 * U * t["bias"].double().abs()
        z = z + t["bias"].double()
    Ez = Ez + 4 * U * z.abs()
    v = act64(z, act)
    E = 1.13 * Ez
    if act == "gelu":
        E = E + 4 * U * z.abs()
    elif act != "none":
        E = E + 2.0 ** -17 * v.abs() + 1e-12
    if t["gate"] is not None:
        g = rows(t["gate"], B, L)
        v, E = v * g, E * g.abs() + 2 * U * (v * g).abs()
    if t["residual"] is not None:
        v = v + t["residual"].double()
        E = E + U * v.abs()
    dtype = BF if x.dtype == F8 else x.dtype
    assert out.dtype == dtype and out.shape == (B, L, w.shape[0])
    half, tiny = torch.finfo(dtype).eps / 2, 2.0 ** -25 if dtype == HF else 0.0
    # (a code drawn beyond 448 is NaN in e4m3, and so is its row in both)
    bad = ~((out.double() - v).abs() <= half * (v.abs() + E) + E + tiny) & ~(out.isnan() & v.isnan())
    assert not bad.any(), f"{bad.sum().item()} of {bad.numel()} outside the bound, first at {bad.nonzero()[0].tolist()}"


def make(B, L, K, N, dtype=BF, F=0, bias=True, gate="none", residual=False, seed=0):
    out = BF if dtype == F8 else dtype
    shape = {"none": None, "vec": (N,), "bcast": (1, 1, N), "batch": (B, 1, N), "flat": (B, N), "row": (B, L, N), "frame": (B, F, 1, N)}[gate]
    fp8 = dtype == F8
    t = dict(x=rand((B, L, K), seed + 1, 100.0 if fp8 else 1.0, dtype),
             weight=rand((N, K), seed + 2, 100.0 if fp8 else 1 / math.sqrt(K), dtype),
             bias=rand((N,), seed + 3, 0.1, out) if bias else None,
             gate=None if shape is None else rand(shape, seed + 4, 0.5, out),
             residual=rand((B, L, N), seed + 5, 1.0, out) if residual else None,
             x_scale=None, weight_scale=None)
    if fp8:
        t["x_scale"] = rand((B, L), seed + 6, 0.002, torch.float32).abs() + 0.005
        t["weight_scale"] = (rand((N,), seed + 7, 0.2, torch.float32).abs() + 0.5) * 0.01 / math.sqrt(K)
    return t


def call(t, act="none", **kw):
    return fn.linear_gate_residual(t["x"], t["weight"], t["bias"], t["gate"], t["residual"], activation=act,
                                   x_scale=t["x_scale"], weight_scale=t["weight_scale"], **kw)


def timeouts():
    import ctypes
    n = ctypes.c_int(-1)
    _block_abi.check(_block_abi.load().linear_gate_timeouts(ctypes.byref(n)), "linear_gate_timeouts")
    return n.value


CASES = [
    # B, L, K, N, dtype, F, act, bias, gate, residual
    (1, 5, 64, 64, BF, 0, "none", False, "none", False),
    (1, 128, 64, 256, BF, 0, "none", False, "none", False),
    (1, 129, 72, 8, BF, 0, "silu", True, "vec", True),
    (1, 333, 2056, 1288, HF, 0, "silu", True, "none", False),
    (3, 333, 264, 520, HF, 0, "gelu", True, "batch", True),
    (2, 42, 512, 96, F8, 21, "gelu_tanh", True, "frame", True),
    (1, 300, 16, 72, F8, 0, "none", False, "none", False),
    (1, 1000, 5120, 5120, BF, 0, "gelu", True, "bcast", True),
    (1, 2100, 5120, 5120, F8, 21, "none", True, "frame", True),
    (2, 1111, 1000, 2600, HF, 0, "gelu_tanh", True, "row", False),
    (5, 700, 8, 6000, BF, 7, "none", True, "frame", True),
    (1, 5000, 4096, 2048, BF, 0, "silu", False, "none", True),
    (1, 70000, 64, 64, BF, 0, "none", True, "none", True),
    (1, 1, 5120, 30720, BF, 0, "none", True, "none", False),
    (1, 1, 8, 8, HF, 0, "gelu", True, "bcast", True),
    (2, 1, 264, 40, BF, 0, "silu", True, "flat", True),
    (1, 3, 5128, 1288, HF, 0, "none", False, "row", False),
    (2, 2, 6160, 520, F8, 2, "gelu_tanh", True, "frame", True),
    (1, 4, 16, 24, F8, 0, "none", False, "none", False),
    (7, 1, 512, 512, BF, 0, "none", True, "none", False),
    (1, 16, 12288, 512, BF, 0, "none", True, "none", True),
    (1, 64, 5120, 5120, HF, 0, "silu", True, "bcast", True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_against_the_formula(case):
    B, L, K, N, dtype, F, act, bias, gate, residual = case
    t = make(B, L, K, N, dtype, F, bias, gate, residual)
    check(call(t, act), t, act)
    assert timeouts() == 0


# Few tiles, where K is split over a cluster: two to eight parts, pairs of CTAs, parts that own one
# chunk of columns or none, K that does not divide; rows of batches apart. And the sizes between,
# which take pairs of CTAs on 192 or 128 columns.
SPLIT = [
    (1, 999, 2056, 1288, HF, 0, "silu", True, "none", False),
    (3, 333, 2056, 1288, BF, 0, "none", True, "batch", True),
    (1, 64, 5120, 5120, BF, 0, "none", True, "bcast", True),
    (1, 5, 12288, 512, HF, 0, "gelu", True, "vec", True),
    (1, 130, 1000, 64, BF, 0, "none", False, "row", True),
    (1, 100, 4096, 8, BF, 0, "none", True, "none", True),
    (1, 512, 11000, 264, HF, 0, "silu", False, "none", False),
    (2, 300, 2048, 2048, F8, 3, "gelu_tanh", True, "frame", True),
    (1, 31, 16384, 1032, F8, 0, "none", True, "none", True),
    (1, 700, 256, 600, F8, 0, "none", True, "row", False),
    (1, 1500, 3000, 1000, BF, 0, "gelu_tanh", True, "none", True),
    (1, 9, 520, 520, HF, 0, "none", True, "none", False),
    (1, 37800, 4096, 512, BF, 21, "silu", True, "frame", True),
    (1, 1024, 1024, 5120, BF, 0, "none", True, "row", True),
    (1, 512, 5120, 5120, F8, 0, "silu", True, "none", True),
    (5, 420, 1000, 2504, HF, 21, "gelu", True, "frame", True),
    (1, 4096, 1536, 1544, BF, 0, "none", False, "bcast", True),
    # a few tokens: a warp or four to the columns, K shorter than their reach, columns that end inside a CTA
    (1, 4, 520, 16392, BF, 0, "silu", True, "row", True),
    (3, 1, 1040, 16384, F8, 0, "none", True, "batch", True),
    (1, 3, 1032, 16384, HF, 0, "gelu", True, "bcast", True),
    (1, 2, 13824, 520, HF, 2, "gelu_tanh", True, "frame", True),
    (1, 4, 4104, 8, BF, 0, "none", True, "none", True),
    (1, 1, 16, 24, F8, 0, "none", True, "none", False),
    (2, 1, 264, 30728, BF, 0, "none", False, "vec", True),
    (1, 37800, 4104, 520, HF, 0, "none", False, "none", False),
]


@pytest.mark.parametrize("case", SPLIT, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_split_sums_and_pairs(case):
    B, L, K, N, dtype, F, act, bias, gate, residual = case
    before = timeouts()
    t = make(B, L, K, N, dtype, F, bias, gate, residual, seed=300)
    out = call(t, act)
    check(out, t, act)
    bits = out.view(torch.int16)  # a NaN's too
    assert torch.equal(bits, call(t, act).view(torch.int16))
    if residual:  # in place
        assert torch.equal(call(t, act, out=t["residual"]).view(torch.int16), bits)
    assert timeouts() == before


@pytest.mark.parametrize("L", [3, 200])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_strided_rows_outputs_and_in_place(L, dtype):
    B, K, N = 2, 160, 264
    t = make(B, L, K, N, dtype, residual=True)
    wide = rand((B, L + 3, 3, K), 21, 100.0 if dtype == F8 else 1.0, dtype)
    t["x"] = wide[:, 1:L + 1, 1]           # batches apart, rows apart
    t["weight"] = rand((N, 2 * K), 22, 100.0 if dtype == F8 else 0.1, dtype)[:, K:]
    want = call(t)
    check(want, t)
    buf = torch.full((B, L + 2, 2 * N), 7.0, device="cuda", dtype=BF)
    out = call(t, out=buf[:, :L, N:])
    assert torch.equal(out, want) and (buf[:, L:] == 7).all() and (buf[:, :, :N] == 7).all()
    res = rand((B, L, 2 * N), 23)
    t["residual"] = res[:, :, :N]
    want, keep = call(t), res[:, :, N:].clone()
    assert call(t, out=t["residual"]) is t["residual"]
    assert torch.equal(res[:, :, :N], want) and torch.equal(res[:, :, N:], keep)


def test_rows_do_not_depend_on_the_batch_and_twice_the_same():
    t = make(1, 3000, 512, 768, residual=True, gate="row")
    out = call(t)
    assert torch.equal(out, call(t))
    check(out, t)
    half = {k: (v[:, 1000:] if v is not None and k in ("x", "gate", "residual") else v) for k, v in t.items()}
    check(call(half), half)


@pytest.mark.parametrize("L", [2, 300])
def test_special_values_stay_in_their_rows(L):
    t = make(1, L, 256, 128)
    t["x"][0, 1, 5] = float("nan")
    t["weight"][7, 3] = float("inf")
    out = call(t)
    assert torch.isnan(out[0, 1]).all() and not torch.isfinite(out[0, :, 7]).any()
    good = torch.isfinite(out)
    good[0, 1], good[0, :, 7] = True, True
    assert good.all()
    big = make(1, L, 256, 128, HF)
    big["x"][0, 0] = 60000.0
    big["weight"][0] = 1.0
    assert call(big)[0, 0, 0] == float("inf")  # beyond fp16, as a rounding of the sum gives
    x = make(1, L, 64, 64, bias=True)
    x["x"].zero_()
    x["bias"][:] = torch.tensor([-200.0, -30.0, 0.0, 30.0] * 16, device="cuda", dtype=BF)
    for act in ("silu", "gelu", "gelu_tanh"):
        check(call(x, act), x, act)


def test_empty_other_stream_and_graphs():
    t = make(2, 0, 64, 64, residual=True)
    assert call(t).shape == (2, 0, 64)
    for L in (2, 300):
        t = make(1, L, 320, 264, gate="bcast", residual=True)
        want = call(t)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = call(t, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
        for g in graphs:
            with torch.cuda.graph(g):
                outs.append(call(t, "silu"))
        t["x"].copy_(rand(t["x"].shape, 40))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            check(out, t, "silu")


def test_two_streams_at_once():
    a, b = make(1, 3000, 1024, 1024, gate="bcast", residual=True), make(1, 2500, 768, 1536, dtype=HF, seed=50)
    wa, wb = call(a), call(b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [(call(a, stream=streams[0]), call(b, stream=streams[1])) for _ in range(8)]
    torch.cuda.synchronize()
    for oa, ob in outs:
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_quantised_rows_into_the_product():
    """norm -> e4m3 -> product -> gate and residual, as a block runs them."""
    B, F, tokens, D, N = 1, 3, 50, 512, 1024
    L = F * tokens
    res, x, gate = rand((B, L, D), 1), rand((B, L, D), 2), rand((B, F, 1, D), 3, 0.5)
    scale, shift = rand((B, F, 1, D), 4, 0.1), rand((B, F, 1, D), 5, 0.1)
    q, s, r = fn.fused_residual_norm_scale_shift_quant(res, x, gate, None, None, scale, shift, "layer")
    w, ws, _ = fn.fused_residual_norm_scale_shift_quant(  # a quantiser for W's rows too
        torch.zeros(1, N, D, device="cuda", dtype=BF), rand((1, N, D), 6, 1 / math.sqrt(D)), None, None, None, None, None, "rms")
    t = dict(x=q, weight=w[0], bias=rand((N,), 7, 0.1), gate=None, residual=None, x_scale=s, weight_scale=ws[0])
    h = call(t, "gelu_tanh")
    check(h, t, "gelu_tanh")
    t = dict(x=h, weight=rand((D, N), 8, 1 / math.sqrt(N)), bias=None, gate=gate, residual=r, x_scale=None, weight_scale=None)
    y = call(t)
    check(y, t)
    heads = y.view(B, L, 8, 64)
    pos = torch.stack([torch.arange(L, device="cuda") // tokens, torch.arange(L, device="cuda") % tokens], -1).int()
    out = fn.rope_norm(heads, pos, (16, 16), norm="head")
    from test_gpu_rope import check_forward
    check_forward(out, heads, pos, (16, 16), None, norm="head")
