"""The dense product with its epilogue and its backward against plain binary64 forms, at
the sizes, types and epilogues where they can go wrong; their refusals."""
import ctypes
import math

import pytest
import torch

import expert_ref as X

gpu_only = pytest.mark.gpu
NONE, RELU, SILU, GELU, GELU_TANH, SWIGLU = range(6)
ACTS = [NONE, RELU, SILU, GELU, GELU_TANH, SWIGLU]
F = torch.nn.functional


def act64(act, v):
    if act == SWIGLU:
        g, u = v.chunk(2, dim=1)
        return F.silu(g) * u
    return {NONE: lambda t: t, RELU: F.relu, SILU: F.silu, GELU: F.gelu, GELU_TANH: lambda t: F.gelu(t, approximate="tanh")}[act](v)


def context(moe):
    return moe.Context(moe.make_config(1, 8, 1, 1, 1))


def randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def pre_bound(x, w, bias):
    """The sums with their bias in binary64, and how far binary32 may be off them."""
    v, mag = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    if bias is not None:
        v, mag = v + bias.double(), mag + bias.double().abs()
    return v, (x.shape[1] + 64) * X.F32_STEP * mag + 2.0 ** -120


def act_bound(act, v, off):
    """What an activation makes of sums off by `off` (its slope is at most 1.13), and a few dozen steps of its own."""
    if act == SWIGLU:
        g, u = v.chunk(2, dim=1)
        dg, du = off.chunk(2, dim=1)
        s = F.silu(g).abs()
        return 1.13 * dg * (u.abs() + du) + s * du + 64 * X.F32_STEP * (s * u.abs() + g.abs() * u.abs() * X.F32_STEP)
    # a gate's relative error grows with the size of its exponent; where that is large the value is small beside |v|
    return 1.13 * off + 64 * X.F32_STEP * act64(act, v).abs() + 64 * X.F32_STEP * v.abs() * torch.exp(-v.abs())


def check_forward(moe, ctx, T, K, N, act, bias, residual, dtype, seed=0, alias=False):
    g = generator(seed + T + K + N)
    M = 2 * N if act == SWIGLU else N
    x, w = randn(g, T, K), randn(g, M, K, scale=1.5 * K ** -0.5)
    b = randn(g, M) if bias else None
    r = randn(g, T, N) if residual else None
    out = torch.full((T + 1, N), 7.0, dtype=dtype, device="cuda")
    pre = torch.full((T + 1, M), 7.0, dtype=torch.bfloat16, device="cuda")
    if alias:
        out[:T] = r
    got = moe.moe_linear(ctx, x, w, bias=b, act=act, residual=out[:T] if alias else r, out=out[:T], pre=pre[:T])
    v, off = pre_bound(x, w, b)
    ref, tol = act64(act, v), act_bound(act, v, off)
    if r is not None:
        ref = ref + r.double()
        tol = tol + X.F32_STEP * (ref.abs() + r.double().abs())
    half = X.BF16_HALF if dtype is torch.bfloat16 else X.F32_STEP / 2
    X.check(got, ref, tol + half * (ref.abs() + tol), "out")
    X.check(pre[:T], v, off + X.BF16_HALF * (v.abs() + off), "pre")
    assert (out[T:] == 7.0).all() and (pre[T:] == 7.0).all()
    plain = moe.moe_linear(ctx, x, w, bias=b, act=act, residual=r, out_dtype=dtype)   # without pre, into memory of its own
    assert torch.equal(plain, got)


SIZES = [(1, 8, 8), (1, 1032, 264), (2, 64, 40), (15, 72, 520), (16, 256, 128), (17, 1000, 24), (33, 200, 72), (64, 448, 256), (65, 64, 136),
         (77, 520, 88), (130, 264, 2056), (300, 2048, 64)]


@gpu_only
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear(gpu, T, K, N, act):
    ctx = context(gpu)
    for bias, residual, dtype in ((False, False, torch.bfloat16), (True, True, torch.bfloat16), (True, False, torch.float32), (False, True, torch.float32)):
        check_forward(gpu, ctx, T, K, N, act, bias, residual, dtype)
    check_forward(gpu, ctx, T, K, N, act, True, True, torch.bfloat16, alias=True)
    assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
    ctx.close()


@gpu_only
def test_gelu_keeps_its_lower_tail(gpu):
    """v times the normal distribution below v, relative to its own size, down to where binary32 ends."""
    from scipy.special import log_ndtr
    ctx = context(gpu)
    v = torch.cat((torch.linspace(-12.5, 4.0, 60001), -torch.logspace(-6, 1.09, 20000), torch.logspace(-6, 0.6, 9999))).float()
    rows = (v.numel() + 7) // 8
    v = torch.nn.functional.pad(v, (0, rows * 8 - v.numel()), value=1.0).reshape(rows, 8)
    # sums that are exactly v: its 24 bits in three numbers of eight, times one
    x, rest = torch.zeros(rows, 24), v.clone()
    for part in range(3):
        x[:, part::3] = rest.bfloat16().float()
        rest -= x[:, part::3]
    assert (rest == 0).all()
    w = torch.eye(8).repeat_interleave(3, dim=1)
    xd, wd = x.bfloat16().cuda(), w.bfloat16().cuda()
    assert torch.equal(gpu.moe_linear(ctx, xd, wd, out_dtype=torch.float32).cpu(), v)
    got = gpu.moe_linear(ctx, xd, wd, act=GELU, out_dtype=torch.float32).double().cpu()
    below = torch.from_numpy(log_ndtr(v.double().numpy())).exp()
    # half steps: the exponent v^2 / 2 is rounded twice and its factor log2(e) once, each worth v^2 / 2; the fit 8; the hardware's
    # reciprocal one more than a rounding, which enters up to 3.8 times; its exponential two; three products
    tol = (1.5 * v.double().pow(2) + 20) * (X.F32_STEP / 2)
    off = (got / (v.double() * below) - 1).abs()
    assert (off <= tol).all(), (float((off / tol).max()), float(v.flatten()[(off / tol).argmax()]))
    ctx.close()


# products whose contraction is shared out, in each kind of tile, and tiles of 128 x 128 that are not
@gpu_only
@pytest.mark.parametrize("act", [NONE, SILU, SWIGLU])
@pytest.mark.parametrize("T,K,N", [(24, 7168, 256), (3, 5000, 72), (13, 1032, 264), (64, 4096, 1032), (100, 2056, 520), (520, 4104, 4096), (700, 72, 3000), (2000, 4160, 264)])
def test_linear_in_parts(gpu, T, K, N, act):
    ctx = context(gpu)
    for bias, residual, dtype in ((True, True, torch.bfloat16), (False, False, torch.float32)):
        check_forward(gpu, ctx, T, K, N, act, bias, residual, dtype)
    ctx.close()


# rows and columns around whole tiles of the large kernel, and lengths of a step's ends
@gpu_only
@pytest.mark.parametrize("act", [GELU, SWIGLU])
@pytest.mark.parametrize("T,K,N", [(4096, 64, 2048), (4097, 72, 2056), (4000, 136, 2040), (2177, 200, 4104), (2100, 8, 4096), (3968, 328, 2200), (8200, 64, 1032)])
def test_linear_of_many_tiles(gpu, T, K, N, act):
    ctx = context(gpu)
    for bias, residual, dtype in ((True, True, torch.bfloat16), (False, False, torch.float32)):
        check_forward(gpu, ctx, T, K, N, act, bias, residual, dtype)
    ctx.close()


@gpu_only
def test_long_rows(gpu):
    """The longest contraction and the most columns, products whose sums are whole numbers."""
    ctx, most = context(gpu), gpu.MOE_MAX_FEATURES
    g = generator(1)
    for T, K, N in ((3, most, 16), (20, most, 72), (2, 16, most), (70, 64, most)):
        x = torch.randint(-2, 3, (T, K), generator=g, device="cuda").bfloat16()
        w = torch.randint(-2, 3, (N, K), generator=g, device="cuda").bfloat16()
        out = gpu.moe_linear(ctx, x, w, out_dtype=torch.float32)
        assert torch.equal(out.double(), x.double() @ w.double().t())   # below 2^24: every partial sum is exact
    ctx.close()


@gpu_only
def test_outputs_past_32_bits(gpu):
    """More than 2^32 bytes of output, and rows of x beyond 2^32 bytes."""
    ctx = context(gpu)
    T, K, N = 40000, 64, 65536
    x, w = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 16400, 32768, 39999], device="cuda")
    x[at, 3] = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda").bfloat16()
    w[:, 3] = (torch.arange(N, device="cuda") % 128).bfloat16()
    out = gpu.moe_linear(ctx, x, w)
    assert torch.equal(out[at], (x[at, 3].float()[:, None] * w[:, 3].float()[None]).bfloat16())   # one exact product each, rounded
    assert int(out.count_nonzero()) == int(out[at].count_nonzero())
    del out
    T, K, N = 70000, 32768, 8
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[69999, 32767], x[65540, 0] = 3.0, 5.0
    w = torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    out = gpu.moe_linear(ctx, x, w)
    assert (out[69999] == 3).all() and (out[65540] == 5).all() and int(out.count_nonzero()) == 2 * N
    ctx.close()


@gpu_only
def test_a_billion_rows(gpu):
    """More tiles of 128 rows than a launch has workgroups for (2^32 threads)."""
    ctx = context(gpu)
    T = 2 ** 30 + 5
    if torch.cuda.mem_get_info()[0] < 3 * T * 16:
        pytest.skip("needs 52 GB")
    x = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 2] = torch.arange(1, 9, device="cuda").bfloat16()
    at = [0, 127, 2 ** 29 - 1, 2 ** 29, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 4]
    for i, r in enumerate(at):
        x[r, 2] = float(i + 1)
    out = gpu.moe_linear(ctx, x, w)
    for i, r in enumerate(at):
        assert torch.equal(out[r], w[:, 2] * (i + 1)), r
    out[torch.tensor(at, device="cuda")] = 0
    assert not out.view(torch.int64).any()
    ctx.close()


@gpu_only
@pytest.mark.parametrize("act", ACTS)
def test_extreme_sums(gpu, act):
    """Sums up to the ends of bf16's range stay finite where the function is, and NaN and infinities stay in their rows."""
    ctx = context(gpu)
    v = torch.tensor([0.0, 1e-30, -1e-30, 3e38, -3e38, 1e20, -1e20, 90.0, -90.0, -1000.0, 12.0, -12.0, -5.5, 1.0, -1.0, 60.0]).bfloat16()
    N = 16
    M = 2 * N if act == SWIGLU else N
    w = torch.zeros(M, 8, dtype=torch.bfloat16)
    w[:N, 0] = v
    w[N:, 0] = 0.5
    x = torch.zeros(3, 8, dtype=torch.bfloat16)
    x[0, 0] = 1.0
    x[1, 0] = float("nan")
    out = gpu.moe_linear(ctx, x.cuda(), w.cuda(), act=act, out_dtype=torch.float32).double().cpu()
    sums = w[:, 0].double()[None]
    ref = act64(act, sums)[0]
    assert torch.isfinite(out[0]).all()
    # exponents up to 100 are off by their own rounding; further out the function is 0 or its argument
    assert ((out[0] - ref).abs() <= 300 * X.F32_STEP * ref.abs() + 2.0 ** -100).all()
    assert torch.isnan(out[1]).all() and (out[2] == 0).all()
    # and the slopes there
    pre = sums.bfloat16().cuda()
    d = torch.ones(1, N, dtype=torch.bfloat16, device="cuda")
    eye = torch.eye(M, dtype=torch.bfloat16, device="cuda")
    grad = gpu.moe_linear_backward(ctx, d, torch.zeros(1, M, dtype=torch.bfloat16, device="cuda"), eye, act=act, pre=pre if act else None)[0].double().cpu()
    p = sums.clone().requires_grad_()
    slope = torch.autograd.grad(act64(act, p).sum(), p)[0]
    slope = torch.nan_to_num(slope, nan=0.0)   # the reference's own inf * 0
    assert torch.isfinite(grad).all()
    finite = sums[0].abs() < 1e19
    assert ((grad - slope)[0, finite].abs() <= X.BF16_HALF * slope[0, finite].abs() + 300 * X.F32_STEP * (1 + slope[0, finite].abs())).all()
    ctx.close()


# ---------------------------------------------------------------- backward
def check_backward(moe, ctx, T, K, N, act, grad_dtype, weights_dtype, accumulate, seed=0):
    g = generator(seed + T + K + N)
    M = 2 * N if act == SWIGLU else N
    x, w, d = randn(g, T, K), randn(g, M, K, scale=M ** -0.5), randn(g, T, N, dtype=grad_dtype)
    pre = randn(g, T, M, scale=2.0) if act != NONE else None
    gx = torch.full((T + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    held_w, held_b = randn(g, M, K, dtype=weights_dtype), randn(g, M, dtype=torch.float32)
    gw, gb = held_w.clone(), held_b.clone()
    ws = torch.full((moe.moe_linear_backward_workspace(T, K, N, act, grad_dtype, True) + 16,), 255, dtype=torch.uint8, device="cuda")
    got = moe.moe_linear_backward(ctx, d, x, w, act=act, pre=pre, bias=True, grad_x=gx[:T], grad_weights=gw, grad_bias=gb, accumulate=accumulate, workspace=ws)
    assert got[1] is gw and got[2] is gb and (ws[-16:] == 255).all()
    d64 = d.double()
    slip = torch.zeros(T, M, dtype=torch.float64, device="cuda")   # of the gradient before the activation
    if act != NONE:
        p = pre.double().requires_grad_()
        d64 = torch.autograd.grad(act64(act, p), p, d.double())[0]
        big = d.double().abs() * (1 + pre.double().abs()[:, :N]) if act != SWIGLU else torch.cat([d.double().abs()] * 2, 1) * (
            1 + torch.cat([pre.double()[:, N:].abs()] * 2, 1)) * (1 + torch.cat([pre.double()[:, :N].abs()] * 2, 1))
        slip = 64 * X.F32_STEP * big
    bias_ref = d64.sum(0)
    bias_tol = (slip + (T + 8) * X.F32_STEP * (d64.abs() + slip)).sum(0) + 2.0 ** -120
    if accumulate:
        bias_ref = bias_ref + held_b.double()
    X.check(gb, bias_ref, bias_tol + X.F32_STEP * bias_ref.abs(), "grad_bias")
    if act != NONE or grad_dtype is torch.float32:
        slip = slip + X.BF16_HALF * (d64.abs() + slip)   # rounded for the products
    mag = d64.abs() + slip
    ref = d64 @ w.double()
    tol = slip @ w.double().abs() + (M + 64) * X.F32_STEP * (mag @ w.double().abs()) + 2.0 ** -120
    X.check(gx[:T], ref, tol + X.BF16_HALF * (ref.abs() + tol), "grad_x")
    assert (gx[T:] == 7.0).all()
    ref = d64.t() @ x.double()
    tol = slip.t() @ x.double().abs() + (T + 64) * X.F32_STEP * (mag.t() @ x.double().abs()) + 2.0 ** -120
    if accumulate:
        ref = ref + held_w.double()
        tol = tol + X.F32_STEP * ref.abs()
    half = X.BF16_HALF if weights_dtype is torch.bfloat16 else X.F32_STEP / 2
    X.check(gw, ref, tol + half * (ref.abs() + tol), "grad_weights")
    # parts of it alone, and by the defaults, give the same
    if not accumulate and weights_dtype is torch.bfloat16:
        args = dict(act=act, pre=pre)
        assert torch.equal(moe.moe_linear_backward(ctx, d, x, w, need_weights=False, **args)[0], gx[:T])
        only = moe.moe_linear_backward(ctx, d, x, w, need_x=False, **args)
        assert only[0] is None and only[2] is None and torch.equal(only[1], gw)
        assert torch.equal(moe.moe_linear_backward(ctx, d, x, w, need_x=False, need_weights=False, bias=True, **args)[2], gb)


@gpu_only
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_backward(gpu, T, K, N, act):
    ctx = context(gpu)
    for grad_dtype, weights_dtype, accumulate in ((torch.bfloat16, torch.bfloat16, False), (torch.float32, torch.bfloat16, True),
                                                  (torch.float32, torch.float32, False), (torch.bfloat16, torch.float32, True)):
        check_backward(gpu, ctx, T, K, N, act, grad_dtype, weights_dtype, accumulate)
    assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
    ctx.close()


@gpu_only
@pytest.mark.parametrize("act,T,K,N", [(GELU, 100, 72, 8192), (RELU, 4100, 264, 136), (SWIGLU, 520, 1368, 2560), (NONE, 4000, 1024, 1032), (SILU, 1, 4096, 4096), (NONE, 3000, 40, 24)])
def test_backward_in_parts(gpu, act, T, K, N):
    ctx = context(gpu)
    check_backward(gpu, ctx, T, K, N, act, torch.bfloat16, torch.bfloat16, False)
    check_backward(gpu, ctx, T, K, N, act, torch.float32, torch.float32, True)
    check_backward(gpu, ctx, T, K, N, act, torch.bfloat16, torch.bfloat16, True)
    ctx.close()


@gpu_only
@pytest.mark.parametrize("act,T,K,N", [(GELU, 2000, 2056, 1032), (SWIGLU, 1100, 1096, 2056), (NONE, 4099, 1024, 1032), (SILU, 2048, 4104, 520)])
def test_backward_of_many_tiles(gpu, act, T, K, N):
    ctx = context(gpu)
    check_backward(gpu, ctx, T, K, N, act, torch.bfloat16, torch.bfloat16, False)
    check_backward(gpu, ctx, T, K, N, act, torch.float32, torch.float32, True)
    ctx.close()


@gpu_only
@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(gpu, act):
    """Small whole numbers, so that the sums are kept exactly: the gradients along random directions against central
    differences of the binary64 forward."""
    ctx = context(gpu)
    g = torch.Generator().manual_seed(3 + act)
    T, K, N = 5, 16, 8
    M = 2 * N if act == SWIGLU else N
    x, w = (torch.randint(-1, 2, (r, K), generator=g).bfloat16() for r in (T, M))
    b = torch.randint(1, 3, (M,), generator=g).bfloat16() - 0.5   # no sum is 0, where the rectifier bends
    d = torch.randn(T, N, generator=g).bfloat16()
    pre = torch.empty(T, M, dtype=torch.bfloat16, device="cuda")
    gpu.moe_linear(ctx, x.cuda(), w.cuda(), bias=b.cuda(), act=act, pre=pre)
    assert torch.equal(pre.double().cpu(), x.double() @ w.double().t() + b.double())
    gx, gw, gb = gpu.moe_linear_backward(ctx, d.cuda(), x.cuda(), w.cuda(), act=act, pre=pre, bias=True)

    def loss(x, w, b):
        return (act64(act, x @ w.t() + b) * d.double()).sum()
    start = [t.double() for t in (x, w, b)]
    for n, grad in enumerate((gx, gw, gb)):
        for _ in range(4):
            v = torch.randn(start[n].shape, generator=g, dtype=torch.float64)
            h = 1e-5
            up, down = ([t + s * h * v if i == n else t for i, t in enumerate(start)] for s in (1, -1))
            slope = float(loss(*up) - loss(*down)) / (2 * h)
            along = grad.double().cpu() * v
            # each entry is off by its own rounding and by those of the at most 16 terms it adds, each of size under 20
            tol = float((v.abs() * (X.BF16_HALF * (grad.double().cpu().abs() + 16 * 20))).sum())
            assert abs(float(along.sum()) - slope) <= tol
    ctx.close()


@gpu_only
def test_no_rows(gpu):
    ctx = context(gpu)
    x, w = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(24, 16, dtype=torch.bfloat16, device="cuda")
    assert gpu.moe_linear(ctx, x, w).shape == (0, 24)
    d = torch.zeros(0, 24, dtype=torch.bfloat16, device="cuda")
    gw, gb = torch.full_like(w, 7.0), torch.full((24,), 7.0, device="cuda")
    gpu.moe_linear_backward(ctx, d, x, w, bias=True, grad_weights=gw, grad_bias=gb, accumulate=True)
    assert (gw == 7.0).all() and (gb == 7.0).all()
    gx, _, _ = gpu.moe_linear_backward(ctx, d, x, w, bias=True, grad_weights=gw, grad_bias=gb)
    assert gx.shape == (0, 16) and (gw == 0).all() and (gb == 0).all()
    ctx.close()


@gpu_only
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_rows_of_a_large_matrix(gpu, dtype):
    """Gradients of no rows where the matrix has more tiles than the dense product's own kernels take: zeros, or left."""
    ctx = context(gpu)
    K, M = 5128, 4112
    x, w = torch.zeros(0, K, dtype=torch.bfloat16, device="cuda"), torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    for act, N in ((NONE, M), (SWIGLU, M // 2)):
        d, pre = torch.zeros(0, N, dtype=dtype, device="cuda"), torch.zeros(0, M, dtype=torch.bfloat16, device="cuda")
        gw, gb = torch.full((M, K), 7.0, dtype=dtype, device="cuda"), torch.full((M,), 7.0, device="cuda")
        gpu.moe_linear_backward(ctx, d, x, w, act=act, pre=pre, bias=True, grad_weights=gw, grad_bias=gb, accumulate=True)
        assert (gw == 7.0).all() and (gb == 7.0).all()
        gx, _, _ = gpu.moe_linear_backward(ctx, d, x, w, act=act, pre=pre, bias=True, grad_weights=gw, grad_bias=gb)
        assert gx.shape == (0, K) and (gw == 0).all() and (gb == 0).all()
    assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
    ctx.close()


@gpu_only
def test_streams_and_capture(gpu):
    """Forward and backward on a side stream, and captured with the workspace that the binding makes, replayed on new inputs
    beside eager calls of the same context."""
    ctx = context(gpu)
    g = generator(5)
    T, K, N = 200, 264, 136
    x, w, b, d = randn(g, T, K), randn(g, 2 * N, K, scale=K ** -0.5), randn(g, 2 * N), randn(g, T, N)
    pre = torch.empty(T, 2 * N, dtype=torch.bfloat16, device="cuda")

    def step():
        out = gpu.moe_linear(ctx, x, w, bias=b, act=SWIGLU, pre=pre)
        return (out,) + gpu.moe_linear_backward(ctx, d, x, w, act=SWIGLU, pre=pre, bias=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first, step()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for _ in range(4):
        x.copy_(randn(g, T, K))
        d.copy_(randn(g, T, N))
        graph.replay()
        got = [t.clone() for t in kept]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, eager))
    ctx.close()


@gpu_only
@pytest.mark.parametrize("act,T,K,N", [(NONE, 24, 7168, 256), (SWIGLU, 100, 2056, 264), (GELU, 129, 72, 8200), (RELU, 300, 1024, 24)])
def test_workspace_is_not_left(gpu, act, T, K, N):
    """Workspaces of exactly the bytes that are asked for; what lies behind stays, and results are the same."""
    ctx = context(gpu)
    g = generator(T)
    M = 2 * N if act == SWIGLU else N
    x, w, d = randn(g, T, K), randn(g, M, K, scale=K ** -0.5), randn(g, T, N)
    pre = torch.empty(T, M, dtype=torch.bfloat16, device="cuda")
    sizes = gpu.moe_linear_workspace(T, K, N, act), gpu.moe_linear_backward_workspace(T, K, N, act, bias=True)
    ws = [torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    out = gpu.moe_linear(ctx, x, w, act=act, pre=pre, workspace=ws[0])
    grads = gpu.moe_linear_backward(ctx, d, x, w, act=act, pre=pre, bias=True, workspace=ws[1])
    assert all((a[n:] == 255).all() for a, n in zip(ws, sizes))
    assert torch.equal(out, gpu.moe_linear(ctx, x, w, act=act))
    assert all(torch.equal(a, b) for a, b in zip(grads, gpu.moe_linear_backward(ctx, d, x, w, act=act, pre=pre, bias=True)))
    ctx.close()


# ---------------------------------------------------------------- refusals
def test_null_arguments_rejected():
    import combine_moe_dispatch_layout_amd as moe
    lib, n = moe.load_library(), ctypes.c_size_t(0)
    bad = moe.MOE_ERR_INVALID_ARG
    assert lib.moe_linear(None, None, 1, None, 8, 8, None, 0, None, None, 0, None, None, None) == bad
    assert lib.moe_linear_backward(None, None, 0, 1, None, None, 8, 8, 0, None, None, None, 0, 0, None, None, None) == bad
    assert lib.moe_linear_backward_workspace(4, 8, 8, 0, 0, 1, None) == bad
    assert lib.moe_linear_workspace(4, 8, 8, 0, None) == bad
    for args, status in [((-1, 8, 8, 0, 0, 0), 1), ((4, 8, 0, 0, 0, 0), 1), ((4, 0, 8, 0, 0, 0), 1), ((4, 8, 8, 6, 0, 0), 1), ((4, 8, 8, -1, 0, 0), 1),
                         ((4, 8, 8, 0, 2, 0), 1), ((4, 8, 8, 0, 0, 2), 1), ((4, 8, 12, 0, 0, 0), 2), ((4, 12, 8, 0, 0, 0), 2), ((4, 8, 65536, 5, 0, 0), 2),
                         ((4, 8, 65536, 0, 0, 0), 0)]:
        assert lib.moe_linear_backward_workspace(*args, ctypes.byref(n)) == status, args
        if args[4:] == (0, 0):
            assert lib.moe_linear_workspace(*args[:4], ctypes.byref(n)) == status, args


def test_workspace_sizes():
    import combine_moe_dispatch_layout_amd as moe
    back = moe.moe_linear_backward_workspace
    assert back(100, 64, 64) == 0
    assert back(100, 64, 64, act=GELU) >= 100 * 64 * 2
    assert back(100, 64, 64, act=SWIGLU) >= 100 * 128 * 2
    assert back(100, 64, 64, out_dtype=torch.float32) >= 100 * 64 * 2
    assert back(1000, 64, 64, bias=True) >= 64 * 4
    assert back(100, 64, 8192) >= 2 * 100 * 64 * 4   # a long contraction for few results is shared out
    assert back(0, 64, 64, act=GELU, bias=True) == 0
    assert moe.moe_linear_workspace(0, 64, 64) == moe.moe_linear_workspace(1, 512, 64) == moe.moe_linear_workspace(8192, 4096, 4096) == 0
    assert moe.moe_linear_workspace(24, 7168, 256) >= 2 * 24 * 256 * 4
    # more tiles than a launch has workgroups for
    assert moe.moe_linear_workspace(2 ** 31 - 65536, 8, 256) == 0 and back(2 ** 29 - 16384, 8, 128, act=SWIGLU) > 0
    for query in (lambda: moe.moe_linear_workspace(2 ** 31 - 65535, 8, 256), lambda: moe.moe_linear_workspace(2 ** 30, 8, 264),
                  lambda: back(2 ** 29 - 16383, 8, 128, act=SWIGLU), lambda: back(2 ** 28, 8, 136)):
        with pytest.raises(moe.MoeError) as e:
            query()
        assert e.value.status == moe.MOE_ERR_UNSUPPORTED


def moe_bytes(moe):
    return moe.moe_linear_workspace(24, 7168, 256)


@gpu_only
def test_refusals(gpu):
    ctx = context(gpu)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w, out, pre = torch.zeros(4, 16, **bf), torch.zeros(24, 16, **bf), torch.zeros(4, 24, **bf), torch.zeros(4, 24, **bf)
    unsupported = [(torch.zeros(4, 12, **bf), torch.zeros(24, 12, **bf), 0), (x, torch.zeros(20, 16, **bf), 0), (x, w, 5),
                   (torch.zeros(1, 65544, **bf), torch.zeros(8, 65544, **bf), 0), (torch.zeros(1, 8, **bf), torch.zeros(65544, 8, **bf), 0)]
    for a, b, act in unsupported:
        with pytest.raises(gpu.MoeError) as e:
            gpu.moe_linear(ctx, a, b, act=act)
        assert e.value.status == gpu.MOE_ERR_UNSUPPORTED
    for act in (6, -1):
        with pytest.raises(gpu.MoeError):
            gpu.moe_linear(ctx, x, w, act=act)
    for kwargs in (dict(bias=torch.zeros(23, **bf)), dict(residual=torch.zeros(4, 16, **bf)), dict(out=torch.zeros(5, 24, **bf)), dict(pre=torch.zeros(4, 16, **bf))):
        with pytest.raises(ValueError):
            gpu.moe_linear(ctx, x, w, **kwargs)
    for kwargs in (dict(bias=torch.zeros(24, device="cuda")), dict(out_dtype=torch.float16), dict(residual=torch.zeros(24, 4, **bf).t())):
        with pytest.raises(TypeError):
            gpu.moe_linear(ctx, x, w, **kwargs)
    with pytest.raises(TypeError):
        gpu.moe_linear(ctx, x.cpu(), w)
    lib, p = gpu.load_library(), lambda t: t.data_ptr()
    f32 = torch.zeros(4, 24, device="cuda")
    bad = [(None, p(w), None, None, p(out), 0, None), (p(x) + 2, p(w), None, None, p(out), 0, None), (p(x), None, None, None, p(out), 0, None),
           (p(x), p(w) + 8, None, None, p(out), 0, None), (p(x), p(w), p(x) + 2, None, p(out), 0, None), (p(x), p(w), None, None, None, 0, None),
           (p(x), p(w), None, None, p(x), 0, None), (p(x), p(w), None, None, p(w), 0, None), (p(x), p(w), None, p(f32), p(f32), 1, None),
           (p(x), p(w), None, None, p(out), 0, p(out)), (p(x), p(w), None, None, p(out), 2, None)]
    for a in bad:
        assert lib.moe_linear(ctx.handle, a[0], 4, a[1], 16, 24, a[2], 0, a[3], a[4], a[5], a[6], None, None) == gpu.MOE_ERR_INVALID_ARG, a
    lx, lw = torch.zeros(24, 7168, **bf), torch.zeros(256, 7168, **bf)   # a product that needs its workspace
    lo, ls = torch.zeros(24, 256, **bf), torch.zeros(moe_bytes(gpu), dtype=torch.uint8, device="cuda")
    long = lambda ws: lib.moe_linear(ctx.handle, p(lx), 24, p(lw), 7168, 256, None, 0, None, p(lo), 0, None, ws, None)
    assert [long(ws) for ws in (None, p(ls) + 8, p(lx), p(lo))] == [gpu.MOE_ERR_INVALID_ARG] * 4 and long(p(ls)) == gpu.MOE_OK
    with pytest.raises(ValueError):
        gpu.moe_linear(ctx, lx, lw, workspace=ls[:-16])
    d = torch.zeros(4, 24, **bf)
    gx, gw, gb = torch.zeros(4, 16, **bf), torch.zeros(24, 16, **bf), torch.zeros(24, device="cuda")
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")

    def back(grad=p(d), out_type=0, rows=4, x_=p(x), w_=p(w), act=GELU, pre_=p(pre), gx_=p(gx), gw_=p(gw), kind=0, acc=0, gb_=p(gb), ws_=p(ws)):
        return lib.moe_linear_backward(ctx.handle, grad, out_type, rows, x_, w_, 16, 24, act, pre_, gx_, gw_, kind, acc, gb_, ws_, None)
    assert back() == gpu.MOE_OK
    for kwargs in (dict(grad=None), dict(out_type=3), dict(rows=-1), dict(x_=None), dict(w_=None), dict(act=7), dict(pre_=None), dict(gx_=p(d)), dict(gw_=p(x)),
                   dict(kind=2), dict(acc=2), dict(ws_=None), dict(ws_=p(ws) + 8), dict(gb_=p(gb) + 4), dict(gx_=p(gw)), dict(gx_=p(pre)), dict(ws_=p(gx))):
        assert back(**kwargs) == gpu.MOE_ERR_INVALID_ARG, kwargs
    assert back(act=NONE, pre_=None) == back(gx_=None, w_=None) == back(gw_=None, x_=None) == gpu.MOE_OK
    with pytest.raises(ValueError):
        gpu.moe_linear_backward(ctx, d, x, w, accumulate=True)
    with pytest.raises(ValueError):
        gpu.moe_linear_backward(ctx, d, x, w, act=GELU, pre=pre, workspace=ws[:64])
    with pytest.raises(ValueError):
        gpu.moe_linear_backward(ctx, d[:3], x, w)
    with pytest.raises(TypeError):
        gpu.moe_linear_backward(ctx, d.half(), x, w)
    torch.cuda.synchronize()
    ctx.close()
