"""The expert products and the gated activation: against plain binary64 forms at
the sizes, orders and routings where they can go wrong; their refusals; and a run
of them together between dispatch and combine."""
import ctypes
import itertools

import pytest
import torch

import expert_ref as X

RECV, PACKED = 0, 1
gpu_only = pytest.mark.gpu


# ---------------------------------------------------------------- refusals on the CPU
@pytest.fixture(scope="module")
def lib():
    import combine_moe_dispatch_layout_amd as moe
    return moe.load_library()


def test_null_arguments_rejected(lib):
    bad = 1   # MOE_ERR_INVALID_ARG
    assert lib.moe_expert_gemm(None, None, 0, None, 8, 8, None, None, 0, None) == bad
    assert lib.moe_expert_gemm_fp8(None, None, None, 0, None, None, 128, 8, None, None, 0, None) == bad
    assert lib.moe_expert_gemm_backward_rows(None, None, 0, None, 8, 8, None, None, 0, None) == bad
    assert lib.moe_expert_gemm_backward_weights(None, None, 0, None, 0, 8, 8, None, None, 0, 0, None) == bad
    assert lib.moe_swiglu(None, None, 8, 0, None, None, None) == bad
    assert lib.moe_swiglu_fp8(None, None, 128, 0, None, None, None, None) == bad
    assert lib.moe_swiglu_backward(None, None, None, 8, 0, None, None, None) == bad


def test_binding_rejects_cpu_tensors_without_a_gpu():
    import combine_moe_dispatch_layout_amd as moe

    class Ctx:
        cfg, device = moe.make_config(4, 128, 2, 1, 1), 0
        handle = None
    t = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        moe._binding._expert_rows(Ctx, t, torch.bfloat16, 8, RECV, "rows")
    with pytest.raises(ValueError):
        moe._binding._mats_shape(Ctx, torch.zeros(3, 8, 8))
    with pytest.raises(ValueError):
        moe._binding._gate_up_features(torch.zeros(4, 7))


# ---------------------------------------------------------------- products
ROUTINGS = {
    # name: Case arguments
    "one token": dict(T=1, k=2, E=4),
    "ragged": dict(T=77, k=2, E=8, R=2, empty=0.05),
    "no valid slot": dict(T=9, k=2, E=4, empty=1.1),
    "hot": dict(T=300, k=3, E=9, R=3, hot=0),
    "one expert": dict(T=515, k=1, E=1),
    "padded": dict(T=70, k=3, E=6, R=2, layout=1, src=1, empty=0.1, max_tokens=80),
    "padded, one token": dict(T=1, k=2, E=66, R=2, layout=1),
    "many experts": dict(T=40, k=4, E=1000, R=4),
    "a repeated expert": dict(T=5, k=3, E=4, idx=torch.tensor([[1, 1, 1], [2, -1, 2], [1, 0, 1], [-1, -1, -1], [3, 3, 0]])),
    "a window that overflows": dict(T=3, k=3, E=4, R=2, layout=1, src=1,
                                    idx=torch.tensor([[1, 1, 1], [1, 0, 1], [2, -1, 2]])),
}


def orders_of(routing):
    both = [RECV, PACKED]
    return list(itertools.product(both, both)) if ROUTINGS[routing].get("layout") else [(RECV, PACKED)]


SIZES = [(64, 64), (8, 8), (72, 264), (520, 40), (256, 1032)]


@gpu_only
@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("routing", ROUTINGS)
def test_gemm(gpu, routing, K, N):
    c = X.Case(gpu, **ROUTINGS[routing])
    w = c.randn(c.E, N, K, scale=K ** -0.5)
    x = c.randn(c.n, K)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    for ro, oo in orders_of(routing):
        rows = c.buffer(ro, x, float("nan"))
        out = torch.full((c.size[oo], N), 7.0, dtype=torch.bfloat16, device="cuda")
        assert gpu.moe_expert_gemm(c.ctx, rows, w.cuda(), c.handle, out=out, rows_order=ro, out_order=oo) is out
        got, rest = c.rows_of(out, oo)
        X.check(got, ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
        assert (rest == 7.0).all()
    gpu.moe_poll_error(c.ctx)   # clears the window overflow that the dispatch reports
    c.close()


@gpu_only
@pytest.mark.parametrize("K,N", [(128, 64), (256, 8), (384, 264), (128, 1032)])
@pytest.mark.parametrize("routing", ROUTINGS)
def test_gemm_fp8(gpu, routing, K, N):
    c = X.Case(gpu, **ROUTINGS[routing])
    wq = (c.randn(c.E, N, K, scale=112.0).float().clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.rand(c.E, -(-N // 128), K // 128, generator=c.gen) * 0.01 + 1e-4
    xq, xs = X.quantise(c.randn(c.n, K).float()) if c.n else (torch.zeros(0, K, dtype=torch.uint8), torch.zeros(0, K // 128))
    w = X.e4m3(wq) * X.expand(ws, N, K)
    x = X.e4m3(xq) * xs.double().repeat_interleave(128, 1)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    for ro, oo in orders_of(routing):
        rows, scales = c.buffer(ro, xq, 0x7F), c.buffer(ro, xs, float("nan"))
        out = torch.full((c.size[oo], N), 7.0, dtype=torch.bfloat16, device="cuda")
        gpu.moe_expert_gemm_fp8(c.ctx, rows, scales, wq.cuda(), ws.cuda(), c.handle, out=out, rows_order=ro, out_order=oo)
        got, rest = c.rows_of(out, oo)
        X.check(got, ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
        assert (rest == 7.0).all()
    c.close()


@gpu_only
@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("routing", ROUTINGS)
def test_gemm_backward_rows(gpu, routing, K, N):
    c = X.Case(gpu, **ROUTINGS[routing])
    w, dy = c.randn(c.E, N, K, scale=N ** -0.5), c.randn(c.n, N)
    wt = w.transpose(1, 2).contiguous()
    ref, mag = X.per_expert(c, dy, wt), X.per_expert(c, dy.abs(), wt.abs())
    for ro, oo in orders_of(routing):
        grad = torch.full((c.size[ro], K), 7.0, dtype=torch.bfloat16, device="cuda")
        gpu.moe_expert_gemm_backward_rows(c.ctx, c.buffer(oo, dy, float("nan")), w.cuda(), c.handle, grad_rows=grad,
                                          out_order=oo, rows_order=ro)
        got, rest = c.rows_of(grad, ro)
        X.check(got, ref, X.sum_bound(ref, mag, N, X.BF16_HALF), "grad_rows")
        assert (rest == 7.0).all()
    c.close()


@gpu_only
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("routing", ROUTINGS)
def test_gemm_backward_weights(gpu, routing, K, N, accumulate, dtype):
    c = X.Case(gpu, **ROUTINGS[routing])
    x, dy = c.randn(c.n, K), c.randn(c.n, N)
    half = X.BF16_HALF if dtype is torch.bfloat16 else X.F32_STEP / 2
    before = c.randn(c.E, N, K).to(dtype) if accumulate else torch.full((c.E, N, K), float("nan"), dtype=dtype)
    ref, mag = X.outer(c, dy, x, c.E), X.outer(c, dy.abs(), x.abs(), c.E)
    if accumulate:
        ref, mag = ref + before.double(), mag + before.double().abs()
    longest = int(torch.bincount(c.expert, minlength=c.E).max())
    for ro, oo in orders_of(routing):
        grad = before.cuda()
        gpu.moe_expert_gemm_backward_weights(c.ctx, c.buffer(oo, dy, float("nan")), c.buffer(ro, x, float("nan")), c.handle,
                                             grad_weights=grad, out_order=oo, rows_order=ro, accumulate=accumulate)
        X.check(grad.cpu(), ref, X.sum_bound(ref, mag, longest, half), "grad_weights")
        if not accumulate:
            assert (grad.cpu()[torch.bincount(c.expert, minlength=c.E) == 0] == 0).all()
    c.close()


# ---------------------------------------------------------------- activation
# |g| <= 32 here: e^-g in binary32 is off by at most |g| + 4 half steps, the
# reciprocal, products and differences by a few more: under 64 steps in all, of
# the terms' magnitudes.
ACT = 64 * X.F32_STEP
TINY = 2.0 ** -120


@gpu_only
@pytest.mark.parametrize("features", [8, 504, 512, 520, 2048])
@pytest.mark.parametrize("routing", ROUTINGS)
def test_swiglu_and_backward(gpu, routing, features):
    c = X.Case(gpu, **ROUTINGS[routing])
    gu, da = c.randn(c.n, 2 * features, scale=4).clamp(-32, 32), c.randn(c.n, features)
    ref = X.swiglu64(gu)
    g, u = gu.double().chunk(2, dim=1)
    s = torch.sigmoid(g)
    d = da.double()
    gref = torch.cat((d * u * s * (1 + g * torch.sigmoid(-g)), d * g * s), 1)
    gmag = torch.cat(((d * u * s).abs() * (1 + g.abs()), (d * g * s).abs()), 1)
    for order in {a for a, _ in orders_of(routing)}:
        out = torch.full((c.size[order], features), 7.0, dtype=torch.bfloat16, device="cuda")
        gate_up = c.buffer(order, gu, float("nan"))
        gpu.moe_swiglu(c.ctx, gate_up, c.handle, out=out, order=order)
        got, rest = c.rows_of(out, order)
        X.check(got, ref, (X.BF16_HALF + 2 * ACT) * ref.abs() + TINY, "act")
        assert (rest == 7.0).all()
        grad = torch.full((c.size[order], 2 * features), 7.0, dtype=torch.bfloat16, device="cuda")
        gpu.moe_swiglu_backward(c.ctx, c.buffer(order, da, float("nan")), gate_up, c.handle, grad_gate_up=grad, order=order)
        got, rest = c.rows_of(grad, order)
        X.check(got, gref, X.BF16_HALF * gref.abs() + 2 * ACT * gmag + TINY, "grad")
        assert (rest == 7.0).all()
        # in place
        gpu.moe_swiglu_backward(c.ctx, c.buffer(order, da, float("nan")), gate_up, c.handle, grad_gate_up=gate_up, order=order)
        assert torch.equal(c.rows_of(gate_up, order)[0].view(torch.int16), got.view(torch.int16))
    c.close()


@gpu_only
@pytest.mark.parametrize("features", [128, 640, 2048])
@pytest.mark.parametrize("routing", ROUTINGS)
def test_swiglu_fp8(gpu, routing, features):
    c = X.Case(gpu, **ROUTINGS[routing])
    gpu.moe_poll_error(c.ctx)
    gu = c.randn(c.n, 2 * features, scale=4).clamp(-32, 32)
    if c.n:
        gu[0, :128] = 0          # an all-zero block: the floor of the scale
    ref = X.swiglu64(gu)
    amax = ref.unflatten(1, (-1, 128)).abs().amax(2).clamp(min=1e-4)
    for order in {a for a, _ in orders_of(routing)}:
        out = torch.full((c.size[order], features), 7, dtype=torch.uint8, device="cuda")
        scales = torch.full((c.size[order], features // 128), 7.0, device="cuda")
        gpu.moe_swiglu_fp8(c.ctx, c.buffer(order, gu, float("nan")), c.handle, out=out, scales=scales, order=order)
        codes, rest = c.rows_of(out, order)
        sc, srest = c.rows_of(scales, order)
        assert (rest == 7).all() and (srest == 7.0).all()
        X.check(sc, amax / 448, 4 * ACT * amax / 448, "scales")
        step = sc.double().repeat_interleave(128, 1)
        # half a step of the code (2^-4 relative, 2^-10 in the subnormal range), and the value's own error
        X.check(X.e4m3(codes) * step, ref, (2.0 ** -4 + 4 * ACT) * ref.abs() + (2.0 ** -10 + 4 * ACT) * step, "codes")
        assert int((codes & 0x7F).max() if c.n else 0x7E) == 0x7E   # each row's largest block reaches the format's end
    assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_OK
    c.close()


@gpu_only
def test_swiglu_extremes(gpu):
    """Saturated gates, infinities and NaN: as the formula gives them; the quantising form reports them."""
    c = X.Case(gpu, T=1, k=1, E=1)
    g = torch.tensor([0.0, -0.0, 200.0, -200.0, 3e38, float("inf"), float("nan"), 1.0])
    gu = torch.cat((g, torch.ones(8))).bfloat16().reshape(1, 16)
    out = gpu.moe_swiglu(c.ctx, gu.cuda(), c.handle)[0].float().cpu()
    assert out[0] == 0 and out[1] == 0 and out[2] == 200 and out[3] == 0 and out[4] > 2.9e38
    assert out[5] == float("inf") and torch.isnan(out[6])
    assert abs(float(out[7]) - 0.7310585786300049) <= 0.7311 * X.BF16_HALF * 1.01
    gu8 = torch.zeros(1, 512, dtype=torch.bfloat16)
    gu8[0, 130] = float("nan")
    gu8[0, :128] = 1.0
    gu8[0, 256:] = 1.0
    codes, scales = gpu.moe_swiglu_fp8(c.ctx, gu8.cuda(), c.handle)
    assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_ERR_NONFINITE
    assert (codes[0, :128] == 0x7E).all()
    c.close()


# ---------------------------------------------------------------- special values
@gpu_only
def test_nan_and_inf_stay_in_their_rows_and_columns(gpu):
    c = X.Case(gpu, T=130, k=2, E=3)
    K, N = 72, 136
    w, x = c.randn(3, N, K), c.randn(c.n, K)
    x[5, 3] = float("nan")
    x[7, 71] = float("inf")
    w[1, 9, 0] = float("nan")
    out = gpu.moe_expert_gemm(c.ctx, c.buffer(RECV, x, float("nan")), w.cuda(), c.handle)
    got = c.rows_of(out, RECV)[0]
    bad = torch.zeros(c.n, N, dtype=torch.bool)
    bad[5] = True
    bad[7] = True
    bad[:, 9] |= c.expert == 1
    assert (~torch.isfinite(got) == bad).all()
    c.close()


# ---------------------------------------------------------------- gradients against differences
@gpu_only
def test_gradients_against_exact_differences(gpu):
    """Small whole numbers, where every product, sum and rounding is exact: the loss
    sum(go * out) moves by exactly <gradient, direction>."""
    c = X.Case(gpu, T=37, k=2, E=5, empty=0.1)
    K, N = 16, 24
    ints = lambda *s: torch.randint(-2, 3, s, generator=c.gen).bfloat16()   # noqa: E731
    x, dx, w, dw, go = ints(c.n, K), ints(c.n, K), ints(5, N, K), ints(5, N, K), ints(c.n, N)

    def loss(x, w):
        out = gpu.moe_expert_gemm(c.ctx, c.buffer(RECV, x, 0.0), w.cuda(), c.handle)
        return (c.rows_of(out, RECV)[0].double() * go.double()).sum()
    gr = c.rows_of(gpu.moe_expert_gemm_backward_rows(c.ctx, c.buffer(RECV, go, 0.0), w.cuda(), c.handle), RECV)[0]
    gw = gpu.moe_expert_gemm_backward_weights(c.ctx, c.buffer(RECV, go, 0.0), c.buffer(RECV, x, 0.0), c.handle).cpu()
    assert float((loss(x + dx, w) - loss(x - dx, w)) / 2) == float((gr.double() * dx.double()).sum())
    assert float((loss(x, w + dw) - loss(x, w - dw)) / 2) == float((gw.double() * dw.double()).sum())
    c.close()


@gpu_only
def test_swiglu_gradient_against_differences(gpu):
    c = X.Case(gpu, T=16, k=1, E=2)
    I, h = 64, 2.0 ** -12
    gu, da = c.randn(c.n, 2 * I, scale=2).clamp(-8, 8), c.randn(c.n, I)
    got = c.rows_of(gpu.moe_swiglu_backward(c.ctx, c.buffer(RECV, da, 0.0), c.buffer(RECV, gu, 0.0), c.handle), RECV)[0].double()
    x = gu.double()
    for part in (0, 1):
        step = torch.zeros_like(x)
        step[:, part * I:(part + 1) * I] = h
        diff = (X.swiglu64(x + step) - X.swiglu64(x - step)) / (2 * h) * da.double()
        # the third derivative of silu is below 1: the difference is off by at most h^2 / 6 |u da|
        mag = (da.double() * (x[:, I:] if part == 0 else torch.ones_like(da).double())).abs()
        bound = X.BF16_HALF * diff.abs() + h * h * mag + 4 * ACT * mag * (1 + x[:, :I].abs()) + 1e-9
        X.check(got[:, part * I:(part + 1) * I], diff, bound, "part %d" % part)
    c.close()


# ---------------------------------------------------------------- together
@gpu_only
@pytest.mark.parametrize("layout", [0, 1])
def test_expert_mlp_forward_and_backward(gpu, layout):
    """dispatch -> gate-and-up product -> activation -> down product -> combine, and back to the gradients of x,
    both matrices and the routing weights, in the order a training step makes the calls."""
    T, k, E, H, I = 100, 2, 6, 256, 192
    c = X.Case(gpu, T=T, k=k, E=E, R=2, layout=layout, src=1, empty=0.05, hidden=H)
    mid = PACKED
    w1, w2 = c.randn(E, 2 * I, H, scale=H ** -0.5), c.randn(E, H, I, scale=I ** -0.5)
    tw = torch.rand(T, k, generator=c.gen).float()
    go = c.randn(T, H)
    m = gpu
    rows = c.bufs.recv_rows
    gu = m.moe_expert_gemm(c.ctx, rows, w1.cuda(), c.handle, out_order=mid)
    act = m.moe_swiglu(c.ctx, gu, c.handle, order=mid)
    y = m.moe_expert_gemm(c.ctx, act, w2.cuda(), c.handle, rows_order=mid)
    out = m.moe_combine(c.ctx, y, tw.cuda(), c.handle)
    gy, gtw = m.moe_combine_backward(c.ctx, go.cuda(), tw.cuda(), y, c.handle)
    gact = m.moe_expert_gemm_backward_rows(c.ctx, gy, w2.cuda(), c.handle, rows_order=mid)
    gw2 = m.moe_expert_gemm_backward_weights(c.ctx, gy, act, c.handle, rows_order=mid)
    ggu = m.moe_swiglu_backward(c.ctx, gact, gu, c.handle, order=mid)
    grows = m.moe_expert_gemm_backward_rows(c.ctx, ggu, w1.cuda(), c.handle, out_order=mid)
    gw1 = m.moe_expert_gemm_backward_weights(c.ctx, ggu, rows, c.handle, out_order=mid)
    gx = m.moe_dispatch_backward(c.ctx, grows, c.handle)
    assert m.moe_poll_error(c.ctx)[0] == m.MOE_OK
    # the same step in binary64 with autograd
    x64, w1r, w2r, twr = (t.detach().cpu().double().requires_grad_() for t in (c.x, w1, w2, tw))
    total = torch.zeros(T, H, dtype=torch.float64)
    idx = c.idx.cpu()
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if e >= 0:
                g, u = (w1r[e] @ x64[t]).chunk(2)
                total[t] = total[t] + twr[t, j] * (w2r[e] @ (g * torch.sigmoid(g) * u))
    (total * go.double()).sum().backward()
    # Every stage rounds its result to bf16 once (half a step, 2^-8).  The longest chain
    # (x's gradient) has eight roundings before it, whose errors are independent and enter
    # the norm of the result with factors of order one: 16 half steps bound the norm.
    for name, got, ref in (("out", out, total), ("x", gx, x64.grad), ("w1", gw1, w1r.grad), ("w2", gw2, w2r.grad),
                           ("topk_weights", gtw, twr.grad)):
        far = (got.cpu().double() - ref.detach()).norm() / ref.detach().norm()
        assert far <= 16 * X.BF16_HALF, (name, float(far))
    c.close()


@gpu_only
def test_expert_mlp_fp8_decode(gpu):
    """The decode path: low-latency fp8 dispatch, fp8 products with a quantising activation in between, combine."""
    T, k, E, H, I = 12, 3, 16, 512, 256
    c = X.Case(gpu, T=T, k=k, E=E, R=4, layout=1, src=2, hidden=H, quant=1)
    m = gpu

    def mats(n, kk):
        q = (c.randn(E, n, kk, scale=112.0).float().clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
        s = (torch.rand(E, -(-n // 128), kk // 128, generator=c.gen) + 0.5) / 112 * kk ** -0.5
        return q, s, X.e4m3(q) * X.expand(s, n, kk)
    q1, s1, w1 = mats(2 * I, H)
    q2, s2, w2 = mats(H, I)
    tw = torch.rand(T, k, generator=c.gen).float()
    gu = m.moe_expert_gemm_fp8(c.ctx, c.bufs.recv_rows, c.bufs.recv_scales, q1.cuda(), s1.cuda(), c.handle, out_order=PACKED)
    a, sa = m.moe_swiglu_fp8(c.ctx, gu, c.handle, order=PACKED)
    y = m.moe_expert_gemm_fp8(c.ctx, a, sa, q2.cuda(), s2.cuda(), c.handle, rows_order=PACKED)
    out = m.moe_combine(c.ctx, y, tw.cuda(), c.handle)
    assert m.moe_poll_error(c.ctx)[0] == m.MOE_OK
    # each stage against its plain form on the values it really got
    xq, xs = c.rows_of(c.bufs.recv_rows, RECV)[0], c.rows_of(c.bufs.recv_scales, RECV)[0]
    x = X.e4m3(xq) * xs.double().repeat_interleave(128, 1)
    ref = X.per_expert(c, x, w1)
    got = c.rows_of(gu, PACKED)[0]
    X.check(got, ref, X.sum_bound(ref, X.per_expert(c, x.abs(), w1.abs()), H, X.BF16_HALF), "gate_up")
    av = X.e4m3(c.rows_of(a, PACKED)[0]) * c.rows_of(sa, PACKED)[0].double().repeat_interleave(128, 1)
    act = X.swiglu64(got)
    step = c.rows_of(sa, PACKED)[0].double().repeat_interleave(128, 1)
    X.check(av, act, (2.0 ** -4 + 4 * ACT) * act.abs() + (2.0 ** -10 + 4 * ACT) * step, "act")
    ref = X.per_expert(c, av, w2)
    got = c.rows_of(y, RECV)[0]
    X.check(got, ref, X.sum_bound(ref, X.per_expert(c, av.abs(), w2.abs()), I, X.BF16_HALF), "y")
    assert torch.isfinite(out).all()
    c.close()


# ---------------------------------------------------------------- refusals on the GPU
@gpu_only
def test_refusals(gpu):
    m = gpu
    c = X.Case(m, T=20, k=2, E=4, R=2, layout=1)
    lib, h, ctx = m.load_library(), c.handle, c.ctx
    K, N = 64, 72
    w, x = c.randn(4, N, K).cuda(), c.buffer(RECV, c.randn(c.n, K), 0.0)
    out = torch.empty(c.size[RECV], N, dtype=torch.bfloat16, device="cuda")

    def call(rows=x.data_ptr(), ro=0, weights=w.data_ptr(), k=K, n=N, hc=ctypes.byref(h.c), o=out.data_ptr(), oo=0):
        return lib.moe_expert_gemm(ctx.handle, rows, ro, weights, k, n, hc, o, oo, 0)
    assert call() == m.MOE_OK
    assert call(rows=None) == call(weights=None) == call(o=None) == call(hc=None) == m.MOE_ERR_INVALID_ARG
    assert call(rows=x.data_ptr() + 2) == call(o=out.data_ptr() + 8) == m.MOE_ERR_INVALID_ARG
    assert call(o=x.data_ptr()) == call(ro=2) == call(oo=-1) == call(k=0) == call(n=-8) == m.MOE_ERR_INVALID_ARG
    assert call(k=60) == call(n=68) == call(n=65544) == m.MOE_ERR_UNSUPPORTED
    other = m.Context(m.make_config(20, 128, 4, 2, 2, 0, 0, 0))
    assert lib.moe_expert_gemm(other.handle, x.data_ptr(), 0, w.data_ptr(), K, N, ctypes.byref(h.c), out.data_ptr(), 0,
                               0) == m.MOE_ERR_HANDLE
    other.close()
    w8 = torch.zeros(4, N, 128, dtype=torch.uint8, device="cuda")
    x8 = torch.zeros(c.size[RECV], 128, dtype=torch.uint8, device="cuda")
    s8, ws8 = torch.zeros(c.size[RECV], 1, device="cuda"), torch.zeros(4, 1, 1, device="cuda")

    def call8(xs=s8.data_ptr(), ws=ws8.data_ptr(), k=128):
        return lib.moe_expert_gemm_fp8(ctx.handle, x8.data_ptr(), xs, 0, w8.data_ptr(), ws, k, N, ctypes.byref(h.c),
                                       out.data_ptr(), 0, 0)
    assert call8() == m.MOE_OK
    assert call8(xs=None) == call8(ws=None) == call8(xs=s8.data_ptr() + 1) == m.MOE_ERR_INVALID_ARG
    assert call8(k=64) == m.MOE_ERR_UNSUPPORTED
    gw = torch.empty(4, N, K, device="cuda")
    wcall = lambda t, acc: lib.moe_expert_gemm_backward_weights(   # noqa: E731
        ctx.handle, out.data_ptr(), 0, x.data_ptr(), 0, K, N, ctypes.byref(h.c), gw.data_ptr(), t, acc, 0)
    assert wcall(2, 0) == wcall(0, 2) == m.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        m.moe_expert_gemm(ctx, x[:-1], w, h)                 # too few rows for the receive layout
    with pytest.raises(ValueError):
        m.moe_expert_gemm(ctx, x, w[:3], h)
    with pytest.raises(TypeError):
        m.moe_expert_gemm(ctx, x.float(), w, h)
    with pytest.raises(TypeError):
        m.moe_expert_gemm(ctx, x, w.transpose(1, 2), h)      # not contiguous
    with pytest.raises(ValueError):
        m.moe_expert_gemm(ctx, x, w, h, rows_order=5)
    with pytest.raises(m.MoeError):
        m.moe_swiglu_fp8(ctx, torch.zeros(c.size[RECV], 16, dtype=torch.bfloat16, device="cuda"), h)
    with pytest.raises(ValueError):
        m.moe_expert_gemm_backward_weights(ctx, out, x, h, accumulate=True)
    with pytest.raises(ValueError):
        m.moe_swiglu(ctx, out, h, out=torch.empty(c.size[RECV], 40, dtype=torch.bfloat16, device="cuda"))
    c.close()


@gpu_only
def test_no_tokens(gpu):
    m = gpu
    ctx = m.Context(m.make_config(4, 128, 3, 1, 2))
    bufs, h = m.moe_dispatch(ctx, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"),
                             torch.empty(0, 2, dtype=torch.int64, device="cuda"))
    w = torch.ones(3, 16, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full((8, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_expert_gemm(ctx, bufs.recv_rows, w, h, out=out)
    assert (out == 7.0).all()
    gw = torch.full((3, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_expert_gemm_backward_weights(ctx, out, bufs.recv_rows, h, grad_weights=gw, accumulate=True)
    assert (gw == 7.0).all()
    m.moe_expert_gemm_backward_weights(ctx, out, bufs.recv_rows, h, grad_weights=gw)
    assert (gw == 0.0).all()
    ctx.close()


@gpu_only
def test_offsets_that_cannot_be_are_reported(gpu):
    """A handle whose offset array was overwritten: the rows it would address are not touched."""
    m = gpu
    c = X.Case(m, T=20, k=2, E=4)
    good = c.handle.expert_offsets.clone()
    w, x = c.randn(4, 16, 64).cuda(), c.buffer(RECV, c.randn(c.n, 64), 0.0)
    gu = c.buffer(RECV, c.randn(c.n, 32), 0.0)
    for bad in ([0, 5, 3, 20, 40], [0, 10, 20, 30, 41], [-1, 10, 20, 30, 40]):
        c.handle.expert_offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        m.moe_expert_gemm(c.ctx, x, w, c.handle)
        assert m.moe_poll_error(c.ctx)[0] == m.MOE_ERR_DEVICE_BOUNDS
        m.moe_expert_gemm_backward_weights(c.ctx, x, x, c.handle)
        assert m.moe_poll_error(c.ctx)[0] == m.MOE_ERR_DEVICE_BOUNDS
    m.moe_swiglu(c.ctx, gu, c.handle)
    c.handle.expert_offsets.copy_(torch.tensor([0, 10, 20, 30, 41], dtype=torch.int32))
    m.moe_poll_error(c.ctx)
    m.moe_swiglu(c.ctx, gu, c.handle)
    assert m.moe_poll_error(c.ctx)[0] == m.MOE_ERR_DEVICE_BOUNDS
    c.handle.expert_offsets.copy_(good)
    m.moe_expert_gemm(c.ctx, x, w, c.handle)
    assert m.moe_poll_error(c.ctx)[0] == m.MOE_OK
    c.close()


# ---------------------------------------------------------------- streams and graphs
@gpu_only
def test_graph_replays_match_eager(gpu):
    m = gpu
    c = X.Case(m, T=60, k=2, E=8, hidden=256)
    w = c.randn(8, 512, 256, scale=0.06).cuda()
    rows = c.bufs.recv_rows
    gu, act = m._binding._expert_out(c.ctx, 512, torch.bfloat16, 0), m._binding._expert_out(c.ctx, 256, torch.bfloat16, 0)
    gr, gw = torch.empty_like(rows), torch.empty_like(w)

    def step():
        m.moe_expert_gemm(c.ctx, rows, w, c.handle, out=gu)
        m.moe_swiglu(c.ctx, gu, c.handle, out=act)
        m.moe_expert_gemm_backward_rows(c.ctx, gu, w, c.handle, grad_rows=gr)
        m.moe_expert_gemm_backward_weights(c.ctx, gu, rows, c.handle, grad_weights=gw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    want = [t[:c.n].clone() if t is not gw else t.clone() for t in (gu, act, gr, gw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        for t in (gu, act, gr, gw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t[:c.n] if t is not gw else t for t in (gu, act, gr, gw)]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        step()   # eager work between the replays
        torch.cuda.synchronize()
    c.close()


@gpu_only
def test_timing_names_the_new_kernels(gpu):
    m = gpu
    c = X.Case(m, T=20, k=2, E=4)
    x, w = c.buffer(RECV, c.randn(c.n, 64), 0.0), c.randn(4, 32, 64).cuda()
    c.ctx.timing_begin(16)
    out = m.moe_expert_gemm(c.ctx, x, w, c.handle)
    act = m.moe_swiglu(c.ctx, out, c.handle)
    m.moe_swiglu_backward(c.ctx, act, out, c.handle)
    m.moe_expert_gemm_backward_rows(c.ctx, out, w, c.handle)
    m.moe_expert_gemm_backward_weights(c.ctx, out, x, c.handle)
    t = c.ctx.timing_end()
    assert all(t[n]["launches"] == 1 for n in ("expert_gemm", "expert_bwd_rows", "expert_bwd_weights", "swiglu", "swiglu_bwd"))
    c.close()
