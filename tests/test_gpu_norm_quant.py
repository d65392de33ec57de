"""GPU checks of the norm rows with an e4m3 output against the formula in 64 bits.

r is compared bit for bit (an exact sum rounded once). For q and row_scale the tolerance is
the rounding of the kernel's fp32 steps, u = 2^-24. With n = (r - mu) rho:

* a thread's fp32 sums have chains of at most 10 terms and 3 joining sums: 13 u of sum |r|
  and of sum r^2 at most, so rho is within 7 u + u (its own rounding) = 8 u, and mu within
  13 u mean|r|;
* the two subtractions, the products with rho and weight, the bias sum, 1 + scale, the last
  fma: 7 u of P = |1 + scale| (|n w| + |b|) + |shift|;
* the product with 448 / max: 2 u, and the maximum carries the error of its own element.

E = u (32 P + 16 |w (1 + scale)| rho mean|r|) covers one element's error before the scale;
the scale's relative error is that of the row's largest element, at most max E / max |y|. A
code is right when it lies between the codes of the two ends of that interval.
"""
import pytest
import torch

import rmsnorm_row_b200 as fn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


def rand(shape, seed, sd=1.0, mean=0.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.empty(shape, device="cuda").normal_(mean, sd, generator=g)).to(dtype)


def operand(layout, B, L, F, D, seed, sd):
    shape = {"none": None, "vec": (D,), "bcast": (1, 1, D), "batch": (B, 1, D), "row": (B, L, D), "frame": (B, F, 1, D)}[layout]
    return None if shape is None else rand(shape, seed, sd)


def per_token(t, B, L):
    if t is None:
        return None
    if t.dim() == 4:
        t = t.repeat_interleave(L // t.shape[1], 1)[:, :, 0]
    if t.dim() == 1:
        t = t[None, None]
    return t.double().expand(B, L, t.shape[-1])


def e4m3(v):
    return v.clamp(-448, 448).float().to(torch.float8_e4m3fn).float()


def check(q, s, r, residual, x, gate, weight, bias, scale, shift, norm, eps):
    B, L, D = x.shape
    v = x.double()
    if residual is not None:
        g = per_token(gate, B, L)
        exact = residual.double() + (v if g is None else g * v)
        # one rounding of the exact sum: to odd into fp32, then to nearest even
        near = exact.float()
        odd = torch.where(near.double() == exact, near, _to_odd(exact, near))
        assert torch.equal(r.view(torch.int16), odd.to(BF).view(torch.int16))
        v = r.double()
    mu = v.mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(v[..., :1])
    rho = 1 / ((v - mu).square().mean(-1, keepdim=True) + eps).sqrt()
    n = (v - mu) * rho
    w = weight.double() if weight is not None else torch.ones(D, dtype=torch.float64, device=x.device)
    b = bias.double() if bias is not None else torch.zeros_like(w)
    sc = per_token(scale, B, L) if scale is not None else torch.zeros_like(v)
    sh = per_token(shift, B, L) if shift is not None else torch.zeros_like(v)
    y = (n * w + b) * (1 + sc) + sh
    P = (1 + sc).abs() * ((n * w).abs() + b.abs()) + sh.abs()
    E = U * (32 * P + 16 * (w * (1 + sc)).abs() * rho * v.abs().mean(-1, keepdim=True))
    a = y.abs().amax(-1)
    zero = a == 0
    err = E.amax(-1)
    assert torch.all(s[zero] == 1) and torch.all(q.float()[zero] == 0)
    assert torch.all((s.double() * 448 - a).abs()[~zero] <= (err + 2 * U * a)[~zero])
    at = a.clamp_min(1e-300)[..., None]
    widen = E + y.abs() * (err / a.clamp_min(1e-300))[..., None]
    lo, hi = e4m3((y - widen) * 448 / at), e4m3((y + widen) * 448 / at)
    got = q.float()
    assert torch.all(torch.isfinite(got))
    ok = (lo <= got) & (got <= hi)
    assert torch.all(ok | zero[..., None]), f"{(~ok).sum().item()} codes outside their interval"


def _to_odd(exact, near):
    """exact in fp32, towards zero with the last bit set (it is not representable)."""
    bits = near.view(torch.int32)
    away = near.double().abs() > exact.abs()
    return ((bits - away.int()) | 1).view(torch.float32)


CASES = [
    # B, L, D, F, norm, residual, gate, mod, weight, bias, affine
    (1, 1, 5120, 0, "rms", True, "none", "none", True, False, BF),
    (1, 1, 16, 0, "layer", False, "none", "none", False, False, BF),
    (2, 7, 32, 0, "rms", True, "bcast", "row", True, True, torch.float32),
    (3, 5, 256, 5, "layer", True, "frame", "frame", True, True, BF),
    (1, 9, 272, 0, "layer", True, "row", "batch", False, True, BF),
    (2, 11, 768, 0, "rms", False, "none", "bcast", True, False, BF),
    (1, 13, 1008, 13, "layer", True, "batch", "frame", False, False, BF),
    (1, 17, 1024, 0, "rms", True, "bcast", "vec", True, False, torch.float32),
    (5, 3, 1040, 0, "layer", True, "row", "row", True, True, BF),
    (2, 33, 2320, 0, "layer", False, "none", "batch", True, True, torch.float32),
    (1, 16, 5120, 0, "rms", True, "bcast", "bcast", True, False, BF),
    (1, 42, 5120, 21, "layer", True, "frame", "frame", True, False, BF),
    (2, 19, 5136, 0, "rms", True, "none", "row", False, True, BF),
    (1, 12, 10240, 0, "layer", True, "bcast", "row", True, False, BF),
    (1, 3, 16384, 0, "layer", True, "none", "row", True, True, torch.float32),
    (1, 4, 16368, 0, "rms", False, "none", "none", True, False, BF),
]


def make(case, seed=0):
    B, L, D, F, norm, residual, gate, mod, weight, bias, affine = case
    return dict(
        residual=rand((B, L, D), seed + 1) if residual else None, x=rand((B, L, D), seed + 2),
        gate=operand(gate, B, L, F, D, seed + 3, 0.5),
        weight=rand((D,), seed + 4, 0.1, 1.0, affine) if weight else None,
        bias=rand((D,), seed + 5, 0.1, 0.0, affine) if bias else None,
        scale=operand(mod, B, L, F, D, seed + 6, 0.1), shift=operand(mod, B, L, F, D, seed + 7, 0.1))


def call(t, norm, eps=1e-6, **kw):
    if t["residual"] is None:
        q, s = fn.norm_scale_shift_quant(t["x"], t["weight"], t["bias"], t["scale"], t["shift"], norm, eps, **kw)
        return q, s, None
    return fn.fused_residual_norm_scale_shift_quant(t["residual"], t["x"], t["gate"], t["weight"], t["bias"],
                                                    t["scale"], t["shift"], norm, eps, **kw)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_rows_against_the_formula(case):
    t = make(case)
    check(*call(t, case[4]), **t, norm=case[4], eps=1e-6)


# Many rows that share their operands: a row for every width of a thread's part, segments that
# end inside a CTA's rows, rows that do not divide evenly.
MANY = [
    (1, 21000, 5120, 21, "layer", True, "frame", "frame", True, False, BF),
    (3, 7001, 2320, 0, "layer", False, "none", "batch", True, True, torch.float32),
    (1, 5003, 5136, 0, "rms", True, "bcast", "none", True, False, BF),
    (2, 2600, 16368, 0, "rms", True, "batch", "bcast", False, True, BF),
    (1, 2500, 10240, 2, "layer", True, "none", "frame", False, False, BF),
    (1, 40001, 256, 0, "layer", True, "vec", "vec", True, True, BF),
    (4, 12000, 512, 3, "rms", False, "none", "frame", False, False, BF),
    (1, 30011, 752, 0, "layer", False, "none", "none", False, False, BF),
    (1, 20011, 1008, 0, "rms", True, "bcast", "bcast", True, False, torch.float32),
    (1, 19003, 1296, 0, "rms", True, "none", "none", False, True, BF),
    (1, 6001, 3856, 0, "layer", True, "bcast", "bcast", True, True, torch.float32),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_many_rows(case):
    B, L, D, F, norm = case[:5]
    t = make(case, 200)
    q, s, r = call(t, norm)
    for at in {0, L - 300, max(0, L // max(F, 1) - 150)}:  # rows around the first operands' change too
        rows = slice(at, at + 300)
        part = {k: per_token(v, B, L)[:, rows].to(BF) if k in ("gate", "scale", "shift") and v is not None
                else v[:, rows] if k in ("x", "residual") and v is not None else v for k, v in t.items()}
        check(q[:, rows], s[:, rows], r[:, rows] if r is not None else None, **part, norm=norm, eps=1e-6)
        q2, s2, r2 = call(part, norm)  # few rows, with operands of their own: the same bits
        assert torch.equal(q2.view(torch.uint8), q[:, rows].view(torch.uint8)) and torch.equal(s2, s[:, rows])
        assert r is None or torch.equal(r2, r[:, rows])
    # in place, and a row that fp32 sums do not serve among the others
    if t["residual"] is not None:
        t["x"][0, 5] = 0.0
        t["residual"][0, 5] = 0.0
        t["residual"][0, 6] *= 1e25
        q, s, r = call(t, norm)
        q2, s2, r2 = call(t, norm, residual_out=t["residual"])
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s) and torch.equal(r2, r)


@pytest.mark.parametrize("D", [128, 5120])
@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_rows_that_fp32_sums_do_not_serve(norm, D):
    """Offset rows, huge and tiny magnitudes, constant rows and zeros go through fp64 sums."""
    x = rand((1, 9, D), 3)
    x[0, 1] = (x[0, 1].float() * 0.01 + 100).to(BF)   # 100 in bf16: no spread is left
    x[0, 8] = (x[0, 8].float() + 100).to(BF)          # mean far above the spread
    x[0, 2] = (x[0, 2].float() * 1e25).to(BF)         # squares overflow fp32
    x[0, 3] = (x[0, 3].float() * 1e-30).to(BF)        # squares underflow fp32
    x[0, 4] = 3.0                                     # no spread
    x[0, 5] = 0.0
    x[0, 6, 1:] = 0.0                                 # one element carries the row
    t = dict(residual=None, x=x, gate=None, weight=None, bias=None, scale=None, shift=None)
    q, s, r = call(t, norm)
    check(q, s, None, **t, norm=norm, eps=1e-6)
    if norm == "layer":  # a constant row is its mean: y = 0
        for flat in (1, 4):
            assert torch.all(q[0, flat].float() == 0) and s[0, flat].item() == 1.0
    q, s, r = call(t, norm, eps=0.0)
    # 0 / 0 without eps: a NaN row, as in the 16-bit ops; the others follow the formula
    undefined = [1, 4, 5] if norm == "layer" else [5]
    assert torch.all(torch.isnan(s[0, undefined])) and torch.all(torch.isnan(q[0, undefined].float()))
    rest = [k for k in range(9) if k not in undefined]
    check(q[:, rest], s[:, rest], None, **dict(t, x=x[:, rest]), norm=norm, eps=0.0)


def test_special_values_stay_visible():
    x = rand((1, 4, 5120), 5)
    x[0, 1, 7] = float("nan")
    x[0, 2, 9] = float("inf")
    for norm in ("rms", "layer"):
        q, s = fn.norm_scale_shift_quant(x, None, None, None, None, norm)
        assert torch.isnan(s[0, 1]) and torch.all(torch.isnan(q[0, 1].float()))
        assert not torch.isfinite(s[0, 2]) and torch.isnan(q[0, 2, 9].float())
        assert torch.isfinite(s[0, 0]) and torch.all(torch.isfinite(q[0, 3].float()))


def test_tiny_rows_have_a_floor():
    x = rand((1, 2, 64), 6)
    w = torch.full((64,), 2.0 ** -110, device="cuda")
    q, s = fn.norm_scale_shift_quant(x, w, None, None, None, "rms")
    assert torch.all(s == 2.0 ** -100 / 448) and torch.all(torch.isfinite(q.float()))


def test_strided_inputs_outputs_and_in_place():
    B, L, D = 2, 9, 2064
    wide = rand((B, L, 3, D), 11)
    t = dict(residual=wide[:, :, 0], x=rand((B, L, 2 * D), 12)[:, :, D:], gate=None, weight=None, bias=None,
             scale=None, shift=None)
    keep = wide.clone()
    q0, s0, r0 = call(t, "rms")
    check(q0, s0, r0, **t, norm="rms", eps=1e-6)
    buf = torch.full((B, L + 2, 2 * D), 1.0, device="cuda").to(torch.float8_e4m3fn)
    q, s, r = call(t, "rms", out=buf[:, :L, D:], residual_out=t["residual"])
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0) and torch.equal(r, r0)
    assert torch.all(buf[:, L:].float() == 1) and torch.all(buf[:, :, :D].float() == 1)
    assert torch.equal(wide[:, :, 1:], keep[:, :, 1:])
    # an output whose byte range holds an input is refused, as in the 16-bit ops
    with pytest.raises(fn.FusedNormError):
        call(dict(t, x=wide[:, :, 2]), "rms", residual_out=t["residual"])


def test_same_rows_whatever_the_batch_and_twice():
    t = make(CASES[12])
    q, s, r = call(t, "rms")
    q2, s2, r2 = call(t, "rms")
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2) and torch.equal(r, r2)
    one = {k: (v[:1, 3:4] if v is not None and v.dim() == 3 else v) for k, v in t.items()}
    q1, s1, r1 = call(one, "rms")
    assert torch.equal(q1.view(torch.uint8), q[:1, 3:4].view(torch.uint8)) and torch.equal(s1, s[:1, 3:4])


def test_empty_and_other_stream_and_graph():
    x = rand((2, 0, 64), 1)
    q, s = fn.norm_scale_shift_quant(x, None, None, None, None, "rms")
    assert q.shape == (2, 0, 64) and s.shape == (2, 0)
    t = make(CASES[10])
    q0, s0, r0 = call(t, "rms")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s, r = call(t, "rms", stream=side)
    side.synchronize()
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(r, r0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, s, r = call(t, "rms")
    t["x"].copy_(rand(t["x"].shape, 99))
    g.replay()
    torch.cuda.synchronize()
    check(q, s, r, **t, norm="rms", eps=1e-6)
