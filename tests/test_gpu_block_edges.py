"""GPU tests of the operators of include/block_ops.h at the edges of their calls: row slots
without a row, long sums, rare values, calls from several host threads, autograd."""
import ctypes
import threading

import pytest
import torch

import rmsnorm_row_b200 as fn
from rmsnorm_row_b200 import _block_abi

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def rand(*shape, seed=0, dtype=BF, sd=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.empty(shape, device="cuda").normal_(mean, sd, generator=g).to(dtype)


def leave_nan_in_shared_memory():
    """Rows of 1024 heads keep their 16384 weights in shared memory, here NaN."""
    x = rand(1, 2000, 1024, 16)
    pos = torch.zeros(2000, 1, device="cuda", dtype=torch.int32)
    y = fn.rope_norm(x, pos, (8,), torch.full((16384,), float("nan"), device="cuda"))
    assert torch.isnan(y).all()


@pytest.mark.parametrize("norm", ["head", "all"])
@pytest.mark.parametrize("H,hd,L", [(1, 16, 5), (1, 16, 200), (2, 16, 300), (1, 64, 3), (4, 128, 9), (3, 48, 1)])
def test_slots_without_a_row_add_nothing_to_dweight(H, hd, L, norm):
    """Several rows share a CTA; what shared memory holds where it has none does not count.

    dweight is a sum of L H (or L) terms dn x rho, each within 40 u of (|g0| + |g1|) |x| rho, in
    chains of at most L H: (40 + L H) u of the terms' magnitudes."""
    x, g = rand(1, L, H, hd), rand(1, L, H, hd, seed=1)
    w = rand(hd if norm == "head" else H * hd, seed=2)
    pos = torch.arange(L, device="cuda", dtype=torch.int32)[:, None]
    leave_nan_in_shared_memory()
    dx, dw = fn.rope_norm_backward(g, x, pos, (hd // 2,), w, norm=norm)
    x64 = x.double()
    dims = (-1,) if norm == "head" else (-2, -1)
    n = x64 / (x64.square().mean(dims, keepdim=True) + 1e-6).sqrt()
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    a = (pos.double() * 10000.0 ** (-i / (hd // 2)))[None, :, None, :]
    g0, g1 = g.double()[..., 0::2], g.double()[..., 1::2]
    dn = torch.stack((g0 * a.cos() + g1 * a.sin(), g1 * a.cos() - g0 * a.sin()), -1).flatten(-2)
    size = (g0.abs() + g1.abs()).repeat_interleave(2, -1)
    over = (0, 1, 2) if norm == "head" else (0, 1)
    want, bound = (dn * n).sum(over).flatten(), (size * n.abs()).sum(over).flatten()
    assert torch.all((dw.double() - want).abs() <= (40 + L * H) * 2.0 ** -24 * bound)
    assert not torch.isnan(dx).any()


# ---- norm_quant --------------------------------------------------------------------------------

def codes(q):
    return q.view(torch.uint8)


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("D,affine,mod", [(512, BF, False), (5120, BF, False), (5120, F32, True), (512, None, True), (512, None, False)])
def test_zeros_keep_their_sign_in_one_row_and_in_many(D, affine, mod, norm):
    """Many rows and the same rows a few at a time give the same bytes, zeros' signs included;
    without bias and modulation a zero's sign is that of n w."""
    rows = 4000
    x = rand(1, rows, D)
    x[:, :, ::7] = -0.0
    w = None
    if affine is not None:
        w = rand(D, seed=1, dtype=affine)
        w[::5] = 0.0
        w[1::5] = -0.0
    sc = sh = None
    if mod:
        sc, sh = rand(D, seed=2), rand(D, seed=3)
        sh[::3] = -0.0
        sh[1::3] = 0.0
    q, s = fn.norm_scale_shift_quant(x, w, None, sc, sh, norm)
    for at in range(0, rows, 1000):
        part = slice(at, at + 3)
        q1, s1 = fn.norm_scale_shift_quant(x[:, part], w, None, sc, sh, norm)
        assert torch.equal(codes(q1), codes(q[:, part])) and torch.equal(s1, s[:, part])
    if norm == "rms" and not mod:
        y = x.double() * (1.0 if w is None else w.double())
        zero = y == 0
        assert zero.any() and torch.equal(codes(q)[zero] == 0x80, torch.signbit(y)[zero])


# ---- long sums of dweight ------------------------------------------------------------------------

@pytest.mark.parametrize("H,hd,L,norm,step,terms", [(40, 128, 1800000, "all", 13, 1), (40, 128, 1800000, "head", 12, 2), (40, 128, 90000, "head", 12, 2),
                                                    (2, 64, 3000000, "all", 13, 1), (1, 16, 5000000, "head", 13, 1), (24, 48, 300000, "head", 13, 4)])
def test_dweight_of_many_tokens(H, hd, L, norm, step, terms):
    """x and grad are 1, nothing turns, and eps makes every term rho = 1 - 1.1 * 2^-step: an fp32 sum
    of 2^(step - 2) and more loses almost half of its last place with each term.

    rho is off by 23 u. A thread sums 512 tokens of `terms` heads in fp32: 512 terms u; the runs of a
    CTA are added in fp32, L / (512 * 444) of them at the least 148 * 3 CTAs: 8 u. Joining in fp64
    and the roundings to fp32 add 3 u."""
    rho = 1 - 1.1 * 2.0 ** -step
    one = torch.ones(1, 1, 1, 1, device="cuda", dtype=BF).expand(1, 1, H, hd).contiguous().expand(1, L, H, hd)
    w = torch.ones(hd if norm == "head" else H * hd, device="cuda", dtype=BF)
    pos = torch.zeros(1, 1, device="cuda", dtype=torch.int32).expand(L, 1)
    dw = fn.rope_norm_backward(one, one, pos, (hd // 2,), w, norm=norm, eps=rho ** -2 - 1)[1].double()
    want = rho * L * (H if norm == "head" else 1)
    assert (dw - want).abs().max().item() <= (23 + 512 * terms + 8 + 3) * 2.0 ** -24 * want


def test_runs_of_dweight_add_up():
    """Tokens beyond a launch's: dx is that of the tokens alone, dweight the sum over the parts."""
    H, hd, L = 40, 128, 600000
    x, g, w = rand(1, 1000, H, hd), rand(1, 1000, H, hd, seed=1), rand(H * hd, seed=2)
    pos = torch.arange(1000, device="cuda", dtype=torch.int32)[:, None]
    dx1, dw1 = fn.rope_norm_backward(g, x, pos, (hd // 2,), w)
    again = lambda t: t.expand(L // 1000, *t.shape[1:])
    dx, dw = fn.rope_norm_backward(again(g), again(x), pos, (hd // 2,), w)
    assert torch.equal(dx, again(dx1))
    # 552 u (sums) and 40 u (terms) of the terms' magnitudes
    x64 = x.double()
    n = x64 / (x64.square().mean((-2, -1), keepdim=True) + 1e-6).sqrt()
    size = (g.double().abs()[..., 0::2] + g.double().abs()[..., 1::2]).repeat_interleave(2, -1)
    bound = (size * n.abs()).sum((0, 1)).flatten() * (L // 1000)
    assert torch.all((dw.double() - dw1.double() * (L // 1000)).abs() <= 600 * 2.0 ** -24 * bound)


# ---- several host threads --------------------------------------------------------------------------

def launches_of_rows(D):
    """(a launch of norm_quant for rows of D channels through the C ABI, the tensors it needs)"""
    lib, rows = _block_abi.load(), 1300
    x, q = rand(1, rows, D), torch.empty(1, rows, D, device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty(1, rows, device="cuda")
    h = ctypes.c_void_p()
    assert lib.norm_quant_create(ctypes.byref(h), ctypes.byref(_block_abi.nq_config(D=D, is_rms=1, eps=1e-6))) == fn.FN_OK
    a = _block_abi.nq_args()
    a.B, a.L, a.x = 1, rows, fn.fn_operand(x.data_ptr(), 0, 0, D)
    a.q, a.q_stride_b, a.q_stride_l, a.row_scale = q.data_ptr(), rows * D, D, s.data_ptr()
    return (lambda stream: lib.norm_quant_launch(h, ctypes.byref(a), stream)), (x, q, s, a)


def launches_of_rotation(H, backward):
    lib, rows, D = _block_abi.load(), 700, H * 128
    x, y, w = rand(1, rows, H, 128), torch.empty(1, rows, H, 128, device="cuda", dtype=BF), rand(D)
    pos = torch.zeros(rows, 1, device="cuda", dtype=torch.int32)
    h = ctypes.c_void_p()
    c = _block_abi.rn_config(dtype=0, heads=H, head_dim=128, axes=1, section=(64, 0, 0, 0), norm=2, has_weight=1, theta=1e4, eps=1e-6)
    assert lib.rope_norm_create(ctypes.byref(h), ctypes.byref(c)) == fn.FN_OK
    r = lambda t: _block_abi.rn_rows(t.data_ptr(), rows * D, D, 128)
    if not backward:
        a = _block_abi.rn_args(1, rows, r(x), pos.data_ptr(), 0, 1, w.data_ptr(), r(y))
        return (lambda stream: lib.rope_norm_launch(h, ctypes.byref(a), stream)), (x, y, w, pos, a)
    n = ctypes.c_uint64()
    assert lib.rope_norm_backward_workspace(h, 1, rows, ctypes.byref(n)) == fn.FN_OK
    work, dw = torch.empty(n.value, device="cuda", dtype=torch.uint8), torch.empty(D, device="cuda")
    a = _block_abi.rn_backward_args(1, rows, r(x), r(x), pos.data_ptr(), 0, 1, w.data_ptr(), r(y), dw.data_ptr(), work.data_ptr(), n.value)
    return (lambda stream: lib.rope_norm_backward_launch(h, ctypes.byref(a), stream)), (x, y, w, pos, work, dw, a)


@pytest.mark.parametrize("make,sizes", [(launches_of_rows, [(5120,), (10240,)]), (launches_of_rotation, [(128, False), (100, False)]),
                                        (launches_of_rotation, [(128, True), (100, True)])])
def test_two_host_threads_launch_different_sizes(make, sizes):
    """Two handles whose sizes share a kernel, launched by two host threads at once: every call is valid."""
    calls = [make(*size) for size in sizes]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    status = [set(), set()]

    def run(i):
        for _ in range(20000):
            status[i].add(calls[i][0](streams[i].cuda_stream))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{fn.FN_OK}, {fn.FN_OK}]


# ---- linear_gate -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [2, 64, 5000])
@pytest.mark.parametrize("activation", ["gelu", "silu"])
def test_activations_far_below_zero(activation, rows, dtype):
    """x W^T is the bias alone, so z is exact. z Phi(z) = z erfc(-z / sqrt 2) / 2: the argument is off by
    one rounding and the product by another, 2 u of it, which erfc's exponent turns into at most
    2 (z^2 / 2 + 1) 2 u, and erfcf is good to 6 ulp: (2 z^2 + 16) u. SiLU: e^-z is off by (2 + 2 |z|) ulp
    (__expf), the quotient by 2 ulp: (2 |z| + 8) 2 u. Then half a step of the type; below its normal
    numbers half of its smallest."""
    z = torch.arange(-12, 4, 0.125, device="cuda").to(dtype)
    x, w = torch.zeros(1, rows, 64, device="cuda", dtype=dtype), torch.zeros(z.numel(), 64, device="cuda", dtype=dtype)
    out = fn.linear_gate_residual(x, w, z, activation=activation)
    v = z.double()
    if activation == "gelu":
        want, u = 0.5 * v * torch.special.erfc(-v / 2 ** 0.5), 2 * v * v + 16
    else:
        want, u = v / (1 + (-v).exp()), 4 * v.abs() + 16
    info = torch.finfo(dtype)
    bound = want.abs() * (info.eps / 2 + u * 2.0 ** -24) + info.smallest_normal * info.eps / 2
    assert torch.all((out.double() - want).abs() <= bound)


# ---- autograd ------------------------------------------------------------------------------------------

def written():
    """Every call with tensors of the caller's for its results: (name, call, those tensors)."""
    x, w, res = rand(1, 40, 64), rand(64, 64, seed=1), rand(1, 40, 64, seed=2)
    q, s, r = torch.empty(1, 40, 64, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(1, 40, device="cuda"), torch.empty_like(x)
    h, pos = x.view(1, 40, 2, 32), torch.zeros(40, 1, device="cuda", dtype=torch.int32)
    y, dx = torch.empty_like(h), torch.empty_like(h)
    return [
        ("rows", lambda: fn.norm_scale_shift_quant(x, None, None, None, None, out=q, row_scale_out=s), [q, s]),
        ("residual rows", lambda: fn.fused_residual_norm_scale_shift_quant(res, x, None, None, None, None, None, residual_out=r), [r]),
        ("residual in place", lambda: fn.fused_residual_norm_scale_shift_quant(res, x, None, None, None, None, None, residual_out=res), [res]),
        ("rotation", lambda: fn.rope_norm(h, pos, (16,), out=y), [y]),
        ("gradient", lambda: fn.rope_norm_backward(h, h, pos, (16,), out=dx), [dx]),
        ("product", lambda: fn.linear_gate_residual(x, w, residual=res, out=res), [res]),
    ]


def test_written_tensors_count_as_changed():
    """A tensor that autograd has saved and that a call then writes fails the backward pass, as with any in-place op."""
    for name, call, outs in written():
        before = [t._version for t in outs]
        call()
        assert [t._version for t in outs] == [v + 1 for v in before], name
    a = torch.ones(1, 40, 64, device="cuda", dtype=BF, requires_grad=True)
    res = rand(1, 40, 64)
    loss = (a * res).sum()
    fn.linear_gate_residual(rand(1, 40, 64), rand(64, 64), residual=res, out=res)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        for name, call, outs in written():
            call()


def test_results_require_no_gradient():
    x, w = rand(1, 40, 64).requires_grad_(), rand(64, 64).requires_grad_()
    h, pos = x.view(1, 40, 2, 32), torch.zeros(40, 1, device="cuda", dtype=torch.int32)
    for out in (fn.linear_gate_residual(x, w), fn.norm_scale_shift_quant(x, None, None, None, None)[1], fn.rope_norm(h, pos, (16,))):
        assert not out.requires_grad and out.grad_fn is None


# ---- handles -------------------------------------------------------------------------------------------

def test_configurations_that_change_with_each_call_do_not_pile_up():
    """20000 thetas and epsilons: the process keeps a bounded number of handles (2.4 KB each), and calls
    with a configuration given up long ago, or just now, are right."""
    x, pos = rand(1, 3, 2, 32), torch.arange(3, device="cuda", dtype=torch.int32)[:, None]
    call = lambda i: fn.rope_norm(x, pos, (16,), norm="head", theta=1000.0 + i, eps=1e-6 * (1 + i))
    first, last = call(0), call(20000)
    resident = lambda: int(open("/proc/self/statm").read().split()[1]) * 4096
    for i in range(1, 200):
        call(i)
    torch.cuda.synchronize()
    before = resident()
    for i in range(200, 20001):
        out = call(i)
    torch.cuda.synchronize()
    assert resident() - before < 16 << 20
    assert torch.equal(out, last) and torch.equal(call(0), first) and not torch.equal(first, last)


# ---- what runs -----------------------------------------------------------------------------------------

def test_every_call_runs_its_own_kernel_and_nothing_else():
    """A CUDA activity trace of each call: one kernel of the library, two for a gradient with a weight."""
    from torch.profiler import ProfilerActivity, profile

    x, w, many = rand(1, 300, 512), rand(256, 512), rand(1, 4000, 512)
    h, pos, wq = rand(1, 300, 4, 64), torch.zeros(300, 1, device="cuda", dtype=torch.int32), rand(256)
    long, wide = rand(1, 64, 5120), rand(512, 5120)
    q, s = fn.norm_scale_shift_quant(rand(1, 256, 512), None, None, None, None)
    calls = [
        (lambda: fn.norm_scale_shift_quant(x, None, None, None, None), ["norm_quant_rows"]),
        (lambda: fn.norm_scale_shift_quant(many, None, None, None, None, "rms"), ["norm_quant_rows"]),
        (lambda: fn.fused_residual_norm_scale_shift_quant(x, x, None, None, None, None, None), ["norm_quant_rows"]),
        (lambda: fn.rope_norm(h, pos, (32,), wq), ["rope_norm_rows"]),
        (lambda: fn.rope_norm_backward(h, h, pos, (32,), wq), ["rope_norm_gradient", "sum_partials"]),
        (lambda: fn.rope_norm_backward(h, h, pos, (32,), norm="none"), ["rope_norm_rows"]),
        (lambda: fn.linear_gate_residual(many, w), ["linear_gate_tiles"]),
        (lambda: fn.linear_gate_residual(long, wide), ["linear_gate_split"]),
        (lambda: fn.linear_gate_residual(x[:, :2], w), ["linear_gate_tokens"]),
        (lambda: fn.linear_gate_residual(q, q[0], x_scale=s, weight_scale=s[0]), ["linear_gate"]),
    ]
    for call, _ in calls:
        call()
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        for call, _ in calls:
            call()
        torch.cuda.synchronize()
    ran = [e.name for e in sorted(prof.events(), key=lambda e: e.time_range.start) if e.device_type == torch.autograd.DeviceType.CUDA]
    if not ran:
        pytest.skip("no CUDA activity recorded (tracing unavailable)")
    want = [name for _, names in calls for name in names]
    assert len(ran) == len(want) and all(w in r for w, r in zip(want, ran)), ran


# ---- layouts that the documents name -------------------------------------------------------------------

def product64(x, w):
    return x.double() @ w.double().T


@pytest.mark.parametrize("L", [2, 3, 8])
def test_many_short_batches_that_lie_apart(L):
    """A part of longer rows: each batch has tiles of its own, and the result is that of the tokens together
    within the sums' K u (|x| |W|) and half a step."""
    x, w = rand(2000, 16, 128)[:, 2:2 + L], rand(264, 128, seed=1)
    out = fn.linear_gate_residual(x, w)
    want, size = product64(x, w), x.double().abs() @ w.double().abs().T
    assert torch.all((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * 128 * 2.0 ** -24 * size)


def test_x_that_repeats_rows():
    x, w = rand(1, 2, 128), rand(264, 128, seed=1)
    assert torch.equal(fn.linear_gate_residual(x.expand(2, 2, 128), w), fn.linear_gate_residual(x.repeat(2, 1, 1), w))
    one = x[:, :1].expand(1, 4, 128)
    assert torch.equal(fn.linear_gate_residual(one, w), fn.linear_gate_residual(one.contiguous(), w))
    for apart in (x.expand(3, 2, 128), x[:, :1].expand(1, 5, 128)):
        with pytest.raises(fn.FusedNormError, match="UNSUPPORTED"):
            fn.linear_gate_residual(apart, w)


@pytest.mark.parametrize("B,L", [(1, 7), (7, 1), (1, 1)])
def test_strides_along_extents_of_one_mean_nothing(B, L):
    def odd(t):
        size, stride = t.shape, [s if n > 1 else 1 for n, s in zip(t.shape, t.stride())]
        return t.as_strided(size, stride)

    x, res, w = rand(B, L, 64), rand(B, L, 64, seed=1), rand(64, 64, seed=2)
    q, r, out = (odd(torch.empty(B, L, 64, device="cuda", dtype=t)) for t in (torch.float8_e4m3fn, BF, BF))
    want = fn.fused_residual_norm_scale_shift_quant(res, x, None, None, None, None, None)
    got = fn.fused_residual_norm_scale_shift_quant(odd(res), odd(x), None, None, None, None, None, out=q, residual_out=r)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((t.contiguous() for t in got), want))
    assert torch.equal(fn.linear_gate_residual(odd(x), w, residual=odd(res), out=out), fn.linear_gate_residual(x, w, residual=res))
    h, pos = x.view(B, L, 2, 32), torch.arange(L, device="cuda", dtype=torch.int32)[:, None]
    y = odd(torch.empty_like(h))
    assert torch.equal(fn.rope_norm(odd(h), pos, (16,), out=y), fn.rope_norm(h, pos, (16,)))


@pytest.mark.parametrize("rows", [3, 3000])
@pytest.mark.parametrize("D", [16, 48, 80, 784, 2320, 5120, 5136, 10256, 16384])
def test_rows_of_one_value_are_zero_under_layernorm(D, rows):
    """r - mean is 0 throughout, so y is the bias, or a row of zeros with row_scale 1."""
    values = torch.tensor([1.0, -3.0, 300.0, 1e38, -1e-30, 0.1, 7e20, 0.0], device="cuda").to(BF)
    x = values[torch.arange(rows, device="cuda") % 8][None, :, None].expand(1, rows, D).contiguous()
    q, s = fn.norm_scale_shift_quant(x, None, None, None, None, "layer", 1e-6)
    assert (s == 1).all() and (q.float() == 0).all()
    bias = rand(D, seed=1)
    q, s = fn.norm_scale_shift_quant(x, None, bias, None, None, "layer", 1e-6)
    top = bias.float().abs().max()
    assert torch.equal(s, (top.double() / 448).float().expand_as(s))  # (a float by a scalar is a product in torch)
    near = (bias.double() * 448 / top.double()).float()
    lo, hi = ((near * (1 + e * 2.0 ** -22)).to(torch.float8_e4m3fn).float() for e in (-1, 1))
    got = q.float()
    assert torch.all((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi)))
