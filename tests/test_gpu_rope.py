"""GPU checks of q/k norm with rotary positions against the formula in 64 bits.

Tolerances, with u = 2^-24 and h = half a step of the 16-bit type (bf16 2^-8, fp16 2^-11,
and 2^-25 absolute below fp16's normal numbers):

* rho: sums of squares have chains of 8 + 1 + 4 terms in a thread, 5 shuffles and at most 16
  warps: 34 u, halved by the root; 1 / n and the sum with eps 2 u; rsqrtf 4 u: 23 u in all.
* cos and sin: 2 u of their own, and the angle's turn rounded to fp32: 2 pi * u / 2 <= 3.2 u,
  absolute; the fp64 product adds |turns| 2^-52 <= 0.1 u here. 6 u in all.
* forward: y = n0 c - n1 s from n = x rho w (25 u): |n0| + |n1| times (25 + 6 + 2) u. E = 40 u
  of it; the output is within h |y| + E.
* dn = grad turned back: 8 u of S = |g0| + |g1|. dx = rho (w dn - n m), n = x rho,
  m = rho mean(w dn x): the first term 23 + 10 u, the second 23 (outer) + 23 (n) + 23 (m) + 34
  (the sum's chain) + 10 + 4 = 117 u of |n| rho mean(|w| S |x|). E = 128 u of both.
* dweight: terms dn x rho, 33 u; chains of at most 40 rows and heads in a thread, 5 shuffles, 16
  warps: 100 u of the sum of S |x| rho.
"""
import math

import pytest
import torch

import rmsnorm_row_b200 as fn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
I32, I64 = torch.int32, torch.int64


def rand(shape, seed, sd=1.0, mean=0.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(mean, sd, generator=g).to(dtype)


def rotation(x, positions, sections, theta, pairing, shared):
    """(index of first, index of second, cos, sin) of the pairs, in 64 bits; cos (.., L, 1, P)."""
    P = sum(sections)
    i = torch.arange(P, device=x.device)
    lo, hi = (i, i + P) if pairing == "half" else (2 * i, 2 * i + 1)
    freq, axis = [], []
    for a, n in enumerate(sections):
        for k in range(n):
            freq.append(theta ** -(len(freq) / P if shared else k / n))
            axis.append(a)
    angle = positions.double()[..., axis] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    angle = angle[..., None, :]
    return lo, hi, angle.cos(), angle.sin()


def turned(n, lo, hi, c, s):
    a, b = n[..., lo], n[..., hi]
    out = n.clone()
    out[..., lo] = a * c - b * s
    out[..., hi] = a * s + b * c
    return out


def pair_magnitude(v, lo, hi):
    m = v.abs().clone()
    both = m[..., lo] + m[..., hi]
    m[..., lo] = both
    m[..., hi] = both
    return m


def normed(x, w, norm, eps):
    if norm == "none":
        return x, torch.ones_like(x[..., :1])
    dims = (-2, -1) if norm == "all" else (-1,)
    rho = 1 / (x.square().mean(dims, keepdim=True) + eps).sqrt()
    n = x * rho
    if w is not None:
        n = n * w.double().view(-1, x.shape[-1])
    return n, rho


def half_step(dtype):
    return torch.finfo(dtype).eps / 2, 2.0 ** -25 if dtype == HF else 0.0


def check_forward(y, x, positions, sections, w, theta=10000.0, pairing="interleaved", shared_frequencies=False, norm="all", eps=1e-6):
    n, _ = normed(x.double(), w, norm, eps)
    lo, hi, c, s = rotation(x, positions, sections, theta, pairing, shared_frequencies)
    want = turned(n, lo, hi, c, s)
    h, tiny = half_step(x.dtype)
    E = 40 * U * pair_magnitude(n, lo, hi)
    assert y.shape == x.shape and y.dtype == x.dtype
    bad = (y.double() - want).abs() > h * (want.abs() + E) + E + tiny
    assert not bad.any(), f"{bad.sum().item()} values outside the bound"


def check_backward(dx, dw, dy, x, positions, sections, w, theta=10000.0, pairing="interleaved", shared_frequencies=False, norm="all", eps=1e-6):
    x64 = x.double().requires_grad_()
    w64 = w.double().requires_grad_() if w is not None else None
    n, rho = normed(x64, w64, norm, eps)
    lo, hi, c, s = rotation(x, positions, sections, theta, pairing, shared_frequencies)
    a, b = n[..., lo], n[..., hi]
    out = n.index_copy(-1, lo, a * c - b * s).index_copy(-1, hi, a * s + b * c)
    grads = torch.autograd.grad((out * dy.double()).sum(), [x64] + ([w64] if w is not None else []))
    h, tiny = half_step(x.dtype)
    rho, X = rho.detach(), x.double().abs()
    S = pair_magnitude(dy.double(), lo, hi)
    wS = S * w.double().abs().view(-1, x.shape[-1]) if w is not None else S
    if norm == "none":
        E = 8 * U * S
    else:
        dims = (-2, -1) if norm == "all" else (-1,)
        E = 128 * U * rho * (wS + X * rho * rho * (wS * X).mean(dims, keepdim=True))
    assert dx.shape == x.shape and dx.dtype == x.dtype
    bad = (dx.double() - grads[0]).abs() > h * (grads[0].abs() + E) + E + tiny
    assert not bad.any(), f"{bad.sum().item()} of dx outside the bound"
    if w is None:
        assert dw is None
        return grads[0], E
    dims = (0, 1) if norm == "all" else (0, 1, 2)
    T = (S * X * rho).sum(dims).flatten()
    assert dw.dtype == F32 and dw.shape == w.shape
    bad = (dw.double() - grads[1]).abs().flatten() > 100 * U * T + U * grads[1].abs().flatten()
    assert not bad.any(), f"{bad.sum().item()} of dweight outside the bound"
    return grads[0], E


CASES = [
    # B, L, H, hd, sections, dtype, norm, weight, pairing, shared, index, first
    (1, 1, 40, 128, (22, 21, 21), BF, "all", BF, "interleaved", False, I32, 8399),
    (1, 1, 1, 16, (8,), BF, "head", F32, "half", False, I64, 0),
    (2, 3, 1, 32, (5, 6), HF, "all", HF, "interleaved", True, I32, 17),
    (1, 77, 2, 64, (11, 10, 11), BF, "head", BF, "interleaved", False, I32, 0),
    (3, 37, 12, 96, (24, 12, 12), HF, "head", F32, "half", True, I64, 1000000),
    (2, 19, 5, 80, (40,), BF, "none", None, "half", False, I64, 5000),
    (2, 19, 5, 80, (3, 1, 1, 2), BF, "none", None, "interleaved", False, I32, 5000),
    (1, 50, 40, 128, (8, 28, 28), BF, "all", BF, "half", False, I32, 0),
    (1, 50, 40, 128, (16, 8, 8), BF, "all", F32, "half", False, I32, 0),
    (1, 33, 3, 48, (8, 8), HF, "all", None, "half", False, I32, 3),
    (2, 9, 7, 144, (30, 20, 3), BF, "head", None, "interleaved", True, I64, 12),
    (1, 9, 64, 256, (64, 32, 32), BF, "all", BF, "interleaved", False, I32, 0),
    (1, 9, 64, 256, (64, 32, 24), HF, "head", F32, "half", False, I32, 0),
    (1, 5, 32, 512, (128, 128), BF, "all", F32, "half", False, I32, 9),
    (1, 260, 1, 512, (200, 3), BF, "head", BF, "interleaved", False, I32, 9),
    (1, 400, 24, 64, (32,), HF, "all", HF, "interleaved", False, I64, 0),
    (5, 7, 9, 16, (1,), BF, "none", None, "interleaved", False, I32, -40),
]


def make(case, seed=0):
    B, L, H, hd, sections, dtype, norm, wt, pairing, shared, index, first = case
    x = rand((B, L, H, hd), seed + 1, dtype=dtype)
    dy = rand((B, L, H, hd), seed + 2, dtype=dtype)
    n = H * hd if norm == "all" else hd
    w = None if wt is None else rand((n,), seed + 3, 0.1, 1.0, wt)
    g = torch.Generator(device="cuda").manual_seed(seed + 4)
    pos = (torch.randint(0, 100, (L, len(sections)), generator=g, device="cuda") + first).to(index)
    return dy, x, pos, sections, w, dict(norm=norm, pairing=pairing, shared_frequencies=shared)


ids = lambda c: "-".join(str(v).replace("torch.", "") for v in c)


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward_against_the_formula(case):
    dy, x, pos, sections, w, kw = make(case)
    check_forward(fn.rope_norm(x, pos, sections, w, **kw), x, pos, sections, w, **kw)


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_gradient_against_the_formula(case):
    dy, x, pos, sections, w, kw = make(case)
    dx, dw = fn.rope_norm_backward(dy, x, pos, sections, w, **kw)
    check_backward(dx, dw, dy, x, pos, sections, w, **kw)


# Every number of heads per thread and warps per row of both directions; rows whose stages fill
# shared memory (48, 144, 432); two heads to a thread of a row that has one warp (6, 16).
SHAPES = [
    (2, 11, 6, 128, (22, 21, 21), BF, "all", F32, "interleaved", True, I32, 0),
    (1, 700, 6, 128, (22, 21, 21), BF, "all", BF, "half", False, I32, 0),
    (1, 9, 16, 64, (32,), BF, "all", HF, "half", False, I32, 0),
    (1, 650, 16, 64, (30,), BF, "all", F32, "interleaved", False, I32, 0),
    (1, 650, 24, 128, (22, 21, 21), BF, "all", BF, "interleaved", False, I32, 0),
    (1, 600, 14, 128, (64,), HF, "all", HF, "half", False, I32, 0),
    (2, 301, 30, 96, (16, 16, 16), HF, "all", F32, "half", True, I64, 7),
    (1, 650, 48, 128, (64,), BF, "all", BF, "interleaved", False, I32, 0),
    (1, 650, 128, 128, (56,), BF, "all", BF, "interleaved", False, I32, 0),
    (1, 9, 289, 48, (24,), BF, "all", BF, "interleaved", False, I32, 0),
    (1, 700, 105, 144, (40, 32), HF, "all", HF, "half", False, I32, 0),
    (1, 9, 37, 432, (100, 100), BF, "all", F32, "interleaved", False, I32, 0),
    (1, 650, 37, 432, (100, 108), BF, "head", F32, "half", False, I32, 0),
    (1, 1000, 341, 48, (3,), BF, "head", BF, "interleaved", False, I32, 0),
    (1, 650, 204, 80, (40,), HF, "none", None, "half", False, I32, 0),
    (1, 650, 9, 64, (32,), BF, "head", BF, "interleaved", False, I32, 0),
    (1, 650, 1024, 16, (8,), BF, "all", BF, "half", False, I32, 0),
]


@pytest.mark.parametrize("case", SHAPES, ids=ids)
def test_launch_shapes(case):
    dy, x, pos, sections, w, kw = make(case, 100)
    if w is not None and w.dtype not in (x.dtype, F32):
        w = w.to(x.dtype)
    y = fn.rope_norm(x, pos, sections, w, **kw)
    check_forward(y, x, pos, sections, w, **kw)
    few = slice(x.shape[1] // 2, x.shape[1] // 2 + 3)  # few rows, in other launch shapes: the same bits
    assert torch.equal(fn.rope_norm(x[:, few], pos[few], sections, w, **kw), y[:, few])
    dx, dw = fn.rope_norm_backward(dy, x, pos, sections, w, **kw)
    check_backward(dx, dw, dy, x, pos, sections, w, **kw)


@pytest.mark.parametrize("case", [CASES[3], CASES[7], CASES[5]], ids=ids)
def test_gradient_against_differences(case):
    """<dx, v> against central differences of the formula along v (an error of delta^2)."""
    dy, x, pos, sections, w, kw = make(case)
    dx, dw = fn.rope_norm_backward(dy, x, pos, sections, w, **kw)
    grad, E = check_backward(dx, dw, dy, x, pos, sections, w, **kw)
    v = rand(x.shape, 77, dtype=F32).double()
    lo, hi, c, s = rotation(x, pos, sections, 10000.0, kw["pairing"], kw["shared_frequencies"])

    def loss(at):
        return (turned(normed(at, w, kw["norm"], 1e-6)[0], lo, hi, c, s) * dy.double()).sum()

    d = 1e-5
    numeric = (loss(x.double() + d * v) - loss(x.double() - d * v)) / (2 * d)
    bound = ((half_step(x.dtype)[0] * (grad.abs() + E) + E) * v.abs()).sum()
    slack = 1e-6 * (grad.abs() * v.abs()).sum()  # the differences' own error
    assert (numeric - (dx.double() * v).sum()).abs() <= bound + slack
    if w is not None:
        wv = rand(w.shape, 78, dtype=F32).double()

        def wloss(sign):
            n, _ = normed(x.double(), w.double() + sign * d * wv, kw["norm"], 1e-6)
            return (turned(n, lo, hi, c, s) * dy.double()).sum()

        numeric = (wloss(1) - wloss(-1)) / (2 * d)
        T = (pair_magnitude(dy.double(), lo, hi) * normed(x.double(), None, kw["norm"], 1e-6)[0].abs()).sum()
        assert (numeric - (dw.double() * wv).sum()).abs() <= (100 * U + 1e-6) * T * wv.abs().max()


@pytest.mark.parametrize("norm", ["head", "all"])
@pytest.mark.parametrize("H,hd", [(2, 64), (40, 128)])
def test_magnitudes_that_fp32_sums_do_not_serve(norm, H, hd):
    x = rand((1, 6, H, hd), 5)
    dy = rand((1, 6, H, hd), 6)
    for row, f in ((0, 1e25), (1, 1e-30), (2, 0.0), (4, 1e-12)):
        x[0, row] = (x[0, row].float() * f).to(BF)
    dy[0, 5] = (dy[0, 5].float() * 1e30).to(BF)  # the sum of w dn x leaves the range kept in fp32
    pos = torch.arange(6, device="cuda", dtype=I32)[:, None]
    w = rand((H * hd if norm == "all" else hd,), 7, 0.1, 1.0)
    sections = (hd // 2,)
    check_forward(fn.rope_norm(x, pos, sections, w, norm=norm), x, pos, sections, w, norm=norm)
    # rows apart: one dweight over all of them would be row 5's alone
    for row in range(6):
        one = (dy[:, row:row + 1], x[:, row:row + 1], pos[row:row + 1], sections, w)
        check_backward(*fn.rope_norm_backward(*one, norm=norm), *one, norm=norm)
    zero = torch.zeros(1, 1, H, hd, device="cuda", dtype=BF)
    assert torch.isnan(fn.rope_norm(zero, pos[:1], sections, None, norm=norm, eps=0.0)).all()  # 0 / 0


def test_special_values_stay_in_their_place():
    x = rand((1, 4, 2, 64), 8)
    x[0, 1, 0, 63] = float("nan")
    x[0, 2, 1, 62] = float("inf")
    pos = torch.zeros(4, 1, device="cuda", dtype=I32)
    y = fn.rope_norm(x, pos, (4,), None, norm="none")  # channels 8.. pass
    assert torch.equal(y.view(torch.int16)[..., 8:], x.view(torch.int16)[..., 8:])
    assert torch.equal(y[..., :8], x[..., :8])  # position 0 turns by nothing
    y = fn.rope_norm(x, pos, (4,), None, norm="head")
    bad = ~torch.isfinite(y)
    assert bad[0, 1, 0].all() and torch.isnan(y[0, 2, 1, 62])
    assert not bad[0, 0].any() and not bad[0, 1, 1].any() and not bad[0, 2, 0].any() and not bad[0, 3].any()


def test_far_positions():
    """Angles stay exact far out: the product in fp64 loses |turns| 2^-52."""
    x = rand((1, 8, 2, 64), 9)
    pos = torch.tensor([[0], [1], [-1], [2 ** 20 + 1], [-(2 ** 24) - 1], [2 ** 31 - 1], [-2 ** 31], [123456789]],
                       device="cuda", dtype=I64)
    y = fn.rope_norm(x, pos, (32,), None, norm="none")
    # at 2^31 the formula's own fp64 angle is known to 2^31 2^-53: 2^-22 = 4 u more
    n = x.double()
    lo, hi, c, s = rotation(x, pos, (32,), 10000.0, "interleaved", False)
    want, E = turned(n, lo, hi, c, s), 48 * U * pair_magnitude(n, lo, hi)
    assert torch.all((y.double() - want).abs() <= 2.0 ** -8 * (want.abs() + E) + E)
    assert torch.equal(y[:, :3], fn.rope_norm(x[:, :3], pos[:3].int(), (32,), None, norm="none"))


def test_strides_batched_positions_and_in_place():
    B, L, H, hd = 3, 21, 6, 64
    qkv = rand((B, L, 3, H, hd), 10)
    keep = qkv.clone()
    pos = torch.randint(0, 50, (B, L, 3), device="cuda", dtype=I32)
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    w = rand((H * hd,), 11, 0.1, 1.0)
    y = fn.rope_norm(q, pos, (12, 10, 10), w)
    check_forward(y, q, pos, (12, 10, 10), w)
    by_head = rand((B, H, L, hd), 12).transpose(1, 2)  # heads outside tokens
    check_forward(fn.rope_norm(by_head, pos, (12, 10, 10), w), by_head, pos, (12, 10, 10), w)
    out = torch.empty(B, H, L, hd, device="cuda", dtype=BF).transpose(1, 2)
    assert fn.rope_norm(q, pos, (12, 10, 10), w, out=out) is out and torch.equal(out, y)
    shared = fn.rope_norm(q, pos[:1], (12, 10, 10), w)
    assert torch.equal(shared, fn.rope_norm(q, pos[0], (12, 10, 10), w))
    dy = rand((B, L, 1, hd), 13).expand(B, L, H, hd)  # the same gradient for every head
    dx, dw = fn.rope_norm_backward(dy, q, pos, (12, 10, 10), w)
    check_backward(dx, dw, dy, q, pos, (12, 10, 10), w)
    dx2, dw2 = fn.rope_norm_backward(dy, q, pos, (12, 10, 10), w, out=q)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and dx2 is q
    assert torch.equal(qkv[:, :, 1:], keep[:, :, 1:])
    qkv.copy_(keep)
    assert torch.equal(fn.rope_norm(k, pos, (12, 10, 10), w, out=k), fn.rope_norm(keep[:, :, 1], pos, (12, 10, 10), w))
    assert torch.equal(qkv[:, :, 0], keep[:, :, 0]) and torch.equal(qkv[:, :, 2], keep[:, :, 2])


def test_same_rows_whatever_the_batch_and_twice():
    dy, x, pos, sections, w, kw = make((1, 3000, 40, 128, (22, 21, 21), BF, "all", BF, "interleaved", False, I32, 0))
    y = fn.rope_norm(x, pos, sections, w, **kw)
    assert torch.equal(y[:, 2000:2003], fn.rope_norm(x[:, 2000:2003], pos[2000:2003], sections, w, **kw))
    dx, dw = fn.rope_norm_backward(dy, x, pos, sections, w, **kw)
    dx2, dw2 = fn.rope_norm_backward(dy, x, pos, sections, w, **kw)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    check_backward(dx, dw, dy, x, pos, sections, w, **kw)
    one, _ = fn.rope_norm_backward(dy[:, 7:8], x[:, 7:8], pos[7:8], sections, w, **kw)
    assert torch.equal(one, dx[:, 7:8])


def test_empty_other_stream_and_graphs():
    x = torch.empty(2, 0, 3, 32, device="cuda", dtype=BF)
    pos = torch.empty(0, 2, device="cuda", dtype=I32)
    w = torch.ones(32, device="cuda", dtype=BF)
    assert fn.rope_norm(x, pos, (8, 8), w, norm="head").shape == x.shape
    dx, dw = fn.rope_norm_backward(x, x, pos, (8, 8), w, norm="head")
    assert dx.shape == x.shape and torch.equal(dw, torch.zeros(32, device="cuda"))

    dy, x, pos, sections, w, kw = make(CASES[7])
    y0 = fn.rope_norm(x, pos, sections, w, **kw)
    dx0, dw0 = fn.rope_norm_backward(dy, x, pos, sections, w, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = fn.rope_norm(x, pos, sections, w, stream=side, **kw)
    dx, dw = fn.rope_norm_backward(dy, x, pos, sections, w, stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, y0) and torch.equal(dx, dx0) and torch.equal(dw, dw0)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]  # both live, replayed in turn
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append((fn.rope_norm(x, pos, sections, w, **kw),) + fn.rope_norm_backward(dy, x, pos, sections, w, **kw))
    x.copy_(rand(x.shape, 55))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for y, dx, dw in outs:
        check_forward(y, x, pos, sections, w, **kw)
        check_backward(dx, dw, dy, x, pos, sections, w, **kw)
