"""The layer of a few tokens against a plain binary64 form, at the routings and sizes where it
can go wrong; its refusals; and runs of the router, the dense products and the layer together, also
against dispatch, expert products and combine."""
import ctypes

import pytest
import torch

import expert_ref as X

gpu_only = pytest.mark.gpu
F = torch.nn.functional


def uniform(T, k, E, empty=0.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).topk(min(k, E), dim=1).indices
    idx = torch.cat((idx, torch.full((T, k - idx.shape[1]), -1)), 1)
    idx[torch.rand(T, k, generator=g) < empty] = -1
    return idx


# name: experts, topk_idx
ROUTINGS = {
    "one token, one slot": (4, torch.tensor([[2]])),
    "one token": (16, uniform(1, 6, 16)),
    "one expert": (1, torch.zeros(40, 1, dtype=torch.int64)),
    "64 slots": (8, uniform(32, 2, 8)),
    "64 slots of one expert": (3, torch.full((64, 1), 1)),
    "65 slots": (9, uniform(13, 5, 9)),
    "no valid slot": (4, torch.full((5, 3), -1)),
    "no valid slot, many": (4, torch.full((50, 3), -1)),
    "empty slots": (12, uniform(20, 3, 12, empty=0.3)),
    "empty slots, many": (12, uniform(70, 3, 12, empty=0.3)),
    "repeated experts": (4, torch.tensor([[1, 1, 1], [2, -1, 2], [1, 0, 1], [-1, -1, -1], [3, 3, 0]])),
    "repeated experts, many": (3, torch.arange(300).remainder(7).remainder(3).reshape(50, 6)),
    "hot": (40, torch.cat((torch.full((100, 1), 7), uniform(100, 2, 7, seed=1)), 1)),
    "as many as there may be": (24, uniform(128, 8, 24)),
    "1024 tokens": (5, uniform(1024, 1, 5)),
    "many experts": (1000, uniform(30, 4, 1000)),
    "fewer experts than slots": (2, uniform(6, 5, 2)),
}


class Layer:
    def __init__(self, moe, routing, H, I, fp8=False, residual=True, seed=0, max_tokens=None):
        E, self.idx = ROUTINGS[routing] if isinstance(routing, str) else routing
        self.moe, self.H, self.I, self.E, self.fp8 = moe, H, I, E, fp8
        self.T, self.k = self.idx.shape
        g = torch.Generator().manual_seed(seed + H + I)
        self.x = torch.randn(self.T, H, generator=g).bfloat16()
        self.w = torch.rand(self.T, self.k, generator=g)
        self.w[self.idx < 0] = float("nan")   # an empty slot's weight is not used
        self.residual = torch.randn(self.T, H, generator=g).bfloat16() if residual else None
        self.mats, self.scales, self.values = [], [], []
        used = set(self.idx[(self.idx >= 0) & (self.idx < E)].tolist())
        unused = [e for e in range(E) if e not in used]
        for rows, cols in ((2 * I, H), (H, I)):
            if fp8:
                m = (torch.randn(E, rows, cols, generator=g) * 112).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                s = (torch.rand(E, rows // 128, cols // 128, generator=g) + 0.5) * 0.01 * cols ** -0.5
                self.values.append(X.e4m3(m) * X.expand(s, rows, cols))
                m[unused] = 0x7F   # NaN: not read
                self.scales.append(s.cuda())
            else:
                m = (torch.randn(E, rows, cols, generator=g) * cols ** -0.5).bfloat16()
                self.values.append(m.double())
                m[unused] = float("nan")
            self.mats.append(m.cuda())
        self.ctx = moe.Context(moe.make_config(max_tokens or self.T, H, E, 1, self.k))
        self.args = [t.cuda() for t in (self.x, self.idx, self.w)]

    def __call__(self, x=None, idx=None, w=None, **kwargs):
        a, b, c = (new if new is not None else old for new, old in zip((x, idx, w), self.args))
        if self.fp8:
            return self.moe.moe_layer_fp8(self.ctx, a, b, c, self.mats[0], self.scales[0], self.mats[1], self.scales[1], **kwargs)
        return self.moe.moe_layer(self.ctx, a, b, c, self.mats[0], self.mats[1], **kwargs)

    def reference(self):
        """The outputs in binary64, and how far off they may be: the first product's sums, the rounding of the activations, the
        second product's sums with them, the sum over the slots, the output's rounding."""
        out = torch.zeros(self.T, self.H, dtype=torch.float64)
        tol = torch.zeros_like(out)
        mag = torch.zeros_like(out)
        w1, w2 = self.values
        step = X.F32_STEP
        for e in range(self.E):
            t, j = torch.nonzero(self.idx == e, as_tuple=True)
            if not t.numel():
                continue
            x = self.x[t].double()
            v, d = x @ w1[e].t(), (self.H + 192) * step * (x.abs() @ w1[e].abs().t())
            (g, u), (dg, du) = v.chunk(2, dim=1), d.chunk(2, dim=1)
            s = F.silu(g)
            a = s * u
            da = 1.13 * dg * (u.abs() + du) + s.abs() * du + 128 * step * a.abs()
            da = da + X.BF16_HALF * (a.abs() + da)
            y, size = a @ w2[e].t(), (a.abs() + da) @ w2[e].abs().t()
            dy = da @ w2[e].abs().t() + (self.I + 192) * step * size
            c = self.w[t, j].double().unsqueeze(1)
            out.index_add_(0, t, c * y)
            mag.index_add_(0, t, c * y.abs())
            tol.index_add_(0, t, c * dy)
        if self.residual is not None:
            out += self.residual.double()
            mag += self.residual.double().abs()
        tol = tol + (self.k + 4) * step * (mag + tol) + 2.0 ** -120
        return out, tol + X.BF16_HALF * (out.abs() + tol)

    def check(self):
        r = self.residual.cuda() if self.residual is not None else None
        out = torch.full((self.T + 1, self.H), 7.0, dtype=torch.bfloat16, device="cuda")
        nbytes = self.T * self.k * self.I * 2
        ws = torch.full((nbytes + 64,), 255, dtype=torch.uint8, device="cuda")
        got = self(residual=r, out=out[:self.T], workspace=ws)
        ref, tol = self.reference()
        X.check(got.cpu(), ref, tol, "out")
        assert (out[self.T:] == 7.0).all() and (ws[nbytes:] == 255).all()
        assert torch.equal(self(residual=r), got)
        if r is not None:
            assert torch.equal(self(residual=r, out=r), got)
        assert self.moe.moe_poll_error(self.ctx) == (self.moe.MOE_OK, 0)

    def close(self):
        self.ctx.close()


@gpu_only
@pytest.mark.parametrize("H,I", [(64, 64), (8, 8), (264, 72), (72, 520), (1000, 24)])
@pytest.mark.parametrize("routing", ROUTINGS)
def test_layer(gpu, routing, H, I):
    c = Layer(gpu, routing, H, I, residual=H != 72)
    c.check()
    c.close()


@gpu_only
@pytest.mark.parametrize("H,I", [(128, 128), (256, 128), (128, 384), (640, 256)])
@pytest.mark.parametrize("routing", ROUTINGS)
def test_layer_fp8(gpu, routing, H, I):
    if ROUTINGS[routing][0] > 100 and H * I > 2 ** 15:
        H, I = 128, 128
    c = Layer(gpu, routing, H, I, fp8=True, residual=H != 256)
    c.check()
    c.close()


@gpu_only
@pytest.mark.parametrize("fp8", [False, True])
def test_long_rows(gpu, fp8):
    """Rows of a model's length, and the longest the library takes."""
    for routing, H, I in (("one token", 7168, 2048), ((2, torch.tensor([[1, 0], [0, -1]])), 32768, 256), ((2, torch.tensor([[1, 0], [0, -1]])), 256, 32768)):
        c = Layer(gpu, routing, H, I, fp8=fp8)
        c.check()
        c.close()


# 1024 slots, so that a workgroup of the first product takes 1, 2, 4, 8 or 16 column tiles one after another; the last of a
# row of workgroups takes fewer, with half a tile at the end where bf16 features are no multiple of 16
@gpu_only
@pytest.mark.parametrize("E,H,I,fp8", [(40, 64, 648, False), (24, 200, 1512, False), (16, 64, 3400, False), (64, 40, 4104, False), (5, 72, 7704, False),
                                       (64, 256, 1024, True), (40, 128, 1280, True), (24, 384, 3200, True), (32, 128, 5504, True), (5, 128, 7808, True),
                                       (5, 72, 15400, False), (16, 40, 13112, False), (5, 128, 15232, True), (12, 128, 13696, True)])
def test_many_columns_a_workgroup(gpu, E, H, I, fp8):
    """Each activation and each output, with scales that differ a lot from block to block."""
    c = Layer(gpu, (E, uniform(256, 4, E, empty=0.02)), H, I, fp8=fp8)
    if fp8:
        g = torch.Generator().manual_seed(I)
        for n, (rows, cols) in enumerate(((2 * I, H), (H, I))):
            factor = 4.0 ** torch.randint(-1, 2, c.scales[n].shape, generator=g)
            c.scales[n] = c.scales[n] * factor.cuda()
            c.values[n] = c.values[n] * X.expand(factor, rows, cols)
    c.check()
    ws = torch.full((c.T * c.k, I), 7.0, dtype=torch.bfloat16, device="cuda")
    c(workspace=ws)
    act, step = ws.cpu(), X.F32_STEP
    for e in range(E):
        p = torch.nonzero(c.idx.reshape(-1) == e).flatten()
        x = c.x[p // c.k].double()
        v, d = x @ c.values[0][e].t(), (H + 192) * step * (x.abs() @ c.values[0][e].abs().t())
        (g, u), (dg, du) = v.chunk(2, dim=1), d.chunk(2, dim=1)
        s = F.silu(g)
        a = s * u
        da = 1.13 * dg * (u.abs() + du) + s.abs() * du + 128 * step * a.abs()
        X.check(act[p], a, da + X.BF16_HALF * (a.abs() + da) + 2.0 ** -120, "activations of expert %d" % e)
    assert (act[c.idx.reshape(-1) < 0] == 7.0).all()   # empty slots have none
    c.close()


@gpu_only
@pytest.mark.parametrize("many", [False, True])
def test_bad_ids_and_not_finite(gpu, many):
    """An id out of range is empty and reported; NaN and infinities of one token stay in it."""
    idx = uniform(60 if many else 6, 3, 5, seed=2)
    idx[1, 0], idx[3, 2] = 5, -2
    c = Layer(gpu, (5, idx.clone()), 64, 72)
    x, w = c.x.clone(), c.w.clone()
    x[2, 3], x[4, 5] = float("nan"), float("inf")
    w[1, 0] = w[3, 2] = float("nan")
    got = c(x=x.cuda(), w=w.cuda(), residual=c.residual.cuda()).cpu()
    assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_ERR_BAD_TOPK
    c.idx[1, 0] = c.idx[3, 2] = -1
    ref, tol = c.reference()
    rest = torch.tensor([t for t in range(c.T) if t not in (2, 4)])
    X.check(got[rest], ref[rest], tol[rest], "out")
    assert torch.isnan(got[2]).all()
    c.close()


@gpu_only
def test_matrices_past_32_bits(gpu):
    """Experts whose matrices lie beyond 2^32 bytes and 2^31 elements, and few rows of them read."""
    E, H, I = 40, 4096, 8192
    ctx = gpu.Context(gpu.make_config(2, H, E, 1, 2))
    g = torch.Generator().manual_seed(1)
    w1 = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(2, H, generator=g).bfloat16()
    for e in (33, 39):
        w1[e] = (torch.randn(2 * I, H, generator=g) * H ** -0.5).bfloat16().cuda()
        w2[e] = (torch.randn(H, I, generator=g) * I ** -0.5).bfloat16().cuda()
    idx, w = torch.tensor([[39, 33], [33, -1]]), torch.tensor([[0.5, 0.25], [2.0, 1.0]])
    got = gpu.moe_layer(ctx, x.cuda(), idx.cuda(), w.cuda(), w1, w2).double().cpu()
    ref = torch.zeros(2, H, dtype=torch.float64)
    for t, j in ((0, 0), (0, 1), (1, 0)):
        v = w1[idx[t, j]].double() @ x[t].cuda().double()
        ref[t] += float(w[t, j]) * (w2[idx[t, j]].double() @ (F.silu(v[:I]) * v[I:])).cpu()
    # activations and outputs are rounded to bf16; 8 rounding steps of the rows' size are far more than their sums give
    assert ((got - ref).abs() <= 8 * X.BF16_HALF * ref.pow(2).mean(1, keepdim=True).sqrt() + X.BF16_HALF * ref.abs()).all()
    ctx.close()


@gpu_only
@pytest.mark.parametrize("fp8", [False, True])
def test_streams_and_capture(gpu, fp8):
    """The layer on a side stream, and two graphs of it with workspaces of their own, replayed in turn on new routings."""
    c = Layer(gpu, (16, uniform(40, 3, 16)), 256, 128, fp8=fp8, residual=False)
    few = [t[:4].clone() for t in c.args]
    want = c()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    graphs = []
    for args in (c.args, few):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = c(*args)
        graphs.append((graph, args, out))
    for n in range(4):
        for graph, args, out in graphs:
            args[1].copy_(uniform(args[1].shape[0], 3, 16, empty=0.2, seed=n))
            args[2].copy_(torch.rand(args[2].shape))
            graph.replay()
        for graph, args, out in graphs:
            kept = out.clone()
            assert torch.equal(kept, c(*args))
    c.close()


@gpu_only
def test_two_at_once(gpu):
    """Two contexts on two streams, a router, a product in parts and a layer each, over the same matrices: as one after the other."""
    m = gpu
    E, k, H, I = 16, 3, 1024, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def mat(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()
    router, w1, w2 = mat(E, H), mat(E, 2 * I, H), mat(E, H, I)
    ctxs = [m.Context(m.make_config(T, H, E, 1, k)) for T in (24, 100)]
    xs = [torch.randn(T, H, generator=g, device="cuda").bfloat16() for T in (24, 100)]

    def run(ctx, x):
        logits = m.moe_linear(ctx, x, router, out_dtype=torch.float32)
        idx, w = m.moe_route(ctx, logits, m.MOE_SCORE_SIGMOID, groups=4, topk_groups=2, group_top=2)
        return logits, idx, w, m.moe_layer(ctx, x, idx, w, w1, w2, residual=x)
    want = [[t.clone() for t in run(c, x)] for c, x in zip(ctxs, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ctxs]
    got = [[], []]
    for _ in range(20):
        for i, (c, x, s) in enumerate(zip(ctxs, xs, streams)):
            with torch.cuda.stream(s):
                got[i].append(run(c, x))
    torch.cuda.synchronize()
    for i in range(2):
        for result in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(result, want[i]))
        assert m.moe_poll_error(ctxs[i]) == (m.MOE_OK, 0)
        ctxs[i].close()


# ---------------------------------------------------------------- together
@gpu_only
@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_whole_layer(gpu, T):
    """Logits, routing, the shared expert, and the routed experts with its output as their residual: against 64 bits, and the
    experts' part against dispatch, products, activation and combine."""
    m = gpu
    E, k, H, I, S = 32, 4, 512, 256, 384
    g = torch.Generator().manual_seed(T)

    def mat(*shape):
        return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).bfloat16()
    x, router, w1, w2, s1, s2 = torch.randn(T, H, generator=g).bfloat16(), mat(E, H), mat(E, 2 * I, H), mat(E, H, I), mat(2 * S, H), mat(H, S)
    ctx = m.Context(m.make_config(T, H, E, 4, k, 1))
    xd, rd, w1d, w2d, s1d, s2d = (t.cuda() for t in (x, router, w1, w2, s1, s2))
    logits = m.moe_linear(ctx, xd, rd, out_dtype=torch.float32)
    idx, w = m.moe_route(ctx, logits, scale=1.5)
    shared = m.moe_linear(ctx, m.moe_linear(ctx, xd, s1d, act=m.MOE_ACT_SWIGLU), s2d, residual=xd)
    out = m.moe_layer(ctx, xd, idx, w, w1d, w2d, residual=shared, out=shared).double().cpu()
    # the same experts the long way
    bufs, h = m.moe_dispatch(ctx, xd, idx)
    rows = m.moe_expert_gemm(ctx, m.moe_swiglu(ctx, m.moe_expert_gemm(ctx, bufs.recv_rows, w1d, h), h), w2d, h)
    long_way = m.moe_combine(ctx, rows, w, h).double().cpu()
    short = m.moe_layer(ctx, xd, idx, w, w1d, w2d).double().cpu()
    assert m.moe_poll_error(ctx) == (m.MOE_OK, 0)
    # 64 bits, with the experts that the logits chose
    v = x.double() @ router.double().t()
    X.check(logits.cpu(), v, X.sum_bound(v, x.double().abs() @ router.double().abs().t(), H, X.F32_STEP / 2), "logits")
    c = idx.cpu()
    share = torch.softmax(v.gather(1, c), 1) * 1.5
    ref = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            a = w1[c[t, j]].double() @ x[t].double()
            ref[t] += share[t, j] * (w2[c[t, j]].double() @ (F.silu(a[:I]) * a[I:]))
    a = x.double() @ s1.double().t()
    whole = ref + (F.silu(a[:, :S]) * a[:, S:]) @ s2.double().t() + x.double()
    # every rounding to bf16 on the way (up to five) is half a step of values of the rows' size; a factor of four covers their tails
    for got, want, roundings in ((out, whole, 4), (short, ref, 2), (long_way, ref, 5)):
        size = want.abs() + want.pow(2).mean(1, keepdim=True).sqrt()
        assert ((got - want).abs() <= 4 * roundings * X.BF16_HALF * size).all()
    ctx.close()


@gpu_only
def test_training_of_the_router(gpu):
    """Gradients from the combine's weights back to the router's matrix, against autograd in 64 bits."""
    m = gpu
    T, E, k, H = 50, 16, 3, 64
    g = torch.Generator().manual_seed(2)
    x, router = torch.randn(T, H, generator=g).bfloat16(), (torch.randn(E, H, generator=g) * H ** -0.5).bfloat16()
    ctx = m.Context(m.make_config(T, H, E, 1, k))
    logits = m.moe_linear(ctx, x.cuda(), router.cuda(), out_dtype=torch.float32)
    idx, w = m.moe_route(ctx, logits, m.MOE_SCORE_SIGMOID, scale=2.0)
    bufs, h = m.moe_dispatch(ctx, x.cuda(), idx)
    y = torch.randn(T * k, H, generator=g).bfloat16()   # experts' outputs
    d = torch.randn(T, H, generator=g).bfloat16()
    _, gw = m.moe_combine_backward(ctx, d.cuda(), w, y.cuda(), h)
    gl = m.moe_route_backward(ctx, gw, logits, idx, m.MOE_SCORE_SIGMOID, scale=2.0)
    gx, gr, _ = m.moe_linear_backward(ctx, gl, x.cuda(), router.cuda())
    x64, r64 = x.double().requires_grad_(), router.double().requires_grad_()
    s = torch.sigmoid(x64 @ r64.t()).gather(1, idx.cpu())
    share = 2.0 * s / s.sum(1, keepdim=True)
    out = (share.unsqueeze(2) * y.double()[h.pos[:T].cpu().long()]).sum(1)
    rx, rr = torch.autograd.grad(out, (x64, r64), d.double())
    gl64 = gl.double().cpu()
    # the logits' gradient is rounded to bf16 for the products, and those once more
    tol = 1.1 * X.BF16_HALF * gl64.abs()
    X.check(gx.cpu(), rx, tol @ router.double().abs() + X.BF16_HALF * rx.abs() + 1e-4, "grad_x")
    X.check(gr.cpu(), rr, tol.t() @ x.double().abs() + X.BF16_HALF * rr.abs() + 1e-4, "grad_router")
    ctx.close()


# ---------------------------------------------------------------- refusals
def test_null_arguments_rejected():
    import combine_moe_dispatch_layout_amd as moe
    lib = moe.load_library()
    assert lib.moe_layer(None, None, None, None, 1, None, None, 8, None, None, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_layer_fp8(None, None, None, None, 1, None, None, None, None, 128, None, None, None, None) == moe.MOE_ERR_INVALID_ARG


@gpu_only
def test_refusals(gpu):
    m = gpu
    c = Layer(m, (4, uniform(3, 2, 4)), 64, 72, max_tokens=3)
    x, idx, w = c.args
    with pytest.raises(m.MoeError) as e:   # more tokens than the context is made for
        c(torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 2, dtype=torch.int64, device="cuda"), torch.zeros(4, 2, device="cuda"))
    assert e.value.status == m.MOE_ERR_CAPACITY
    big = m.Context(m.make_config(600, 64, 4, 1, 2))
    with pytest.raises(m.MoeError) as e:   # 1026 slots
        m.moe_layer(big, torch.zeros(513, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(513, 2, dtype=torch.int64, device="cuda"),
                    torch.zeros(513, 2, device="cuda"), *c.mats)
    assert e.value.status == m.MOE_ERR_UNSUPPORTED
    big.close()
    for args in ((x.float(), idx, w), (x, idx.int(), w), (x, idx, w.double()), (x.cpu(), idx, w)):
        with pytest.raises(TypeError):
            c(*args)
    for args, kwargs in (((x[:, :56].contiguous(), idx, w), {}), ((x, idx[:2], w), {}), ((x, idx, w[:, :1].contiguous()), {}),
                         ((x, idx, w), dict(out=torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"))),
                         ((x, idx, w), dict(residual=torch.zeros(3, 72, dtype=torch.bfloat16, device="cuda"))),
                         ((x, idx, w), dict(workspace=torch.zeros(3 * 2 * 72 * 2 - 1, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(ValueError):
            c(*args, **kwargs)
    with pytest.raises(ValueError):
        m.moe_layer(c.ctx, x, idx, w, c.mats[0], c.mats[1][:3])
    assert c(x[:0], idx[:0], w[:0]).shape == (0, 64)
    lib, out, ws = m.load_library(), torch.zeros_like(x), torch.zeros(4096, dtype=torch.uint8, device="cuda")
    p = {"x": x, "idx": idx, "w": w, "w1": c.mats[0], "w2": c.mats[1], "out": out, "ws": ws}
    good = {n: t.data_ptr() for n, t in p.items()} | {"T": 3, "I": 72, "res": None}

    def call(**kwargs):
        a = good | kwargs
        return lib.moe_layer(c.ctx.handle, a["x"], a["idx"], a["w"], a["T"], a["w1"], a["w2"], a["I"], a["res"], a["out"], a["ws"], None)
    assert call() == m.MOE_OK
    for name in ("x", "idx", "w", "w1", "w2", "out", "ws"):
        assert call(**{name: None}) == m.MOE_ERR_INVALID_ARG, name
        assert call(**{name: good[name] + 2}) == m.MOE_ERR_INVALID_ARG, name
    for kwargs in (dict(out=good["x"]), dict(out=good["w1"]), dict(out=good["ws"]), dict(ws=good["x"]), dict(ws=good["w2"]), dict(ws=good["x"], res=good["x"]), dict(I=0), dict(T=-1), dict(res=good["x"] + 4)):
        assert call(**kwargs) == m.MOE_ERR_INVALID_ARG, kwargs
    assert call(I=76) == call(I=32776) == m.MOE_ERR_UNSUPPORTED
    q = Layer(m, (2, uniform(2, 1, 2)), 128, 128, fp8=True)
    args = [q.args[0].data_ptr(), q.args[1].data_ptr(), q.args[2].data_ptr(), 2, q.mats[0].data_ptr(), q.scales[0].data_ptr(), q.mats[1].data_ptr(),
            q.scales[1].data_ptr(), 128, None, torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda").data_ptr(), ws.data_ptr(), None]
    for at, value, status in ((5, None, 1), (7, None, 1), (5, args[5] + 2, 1), (8, 64, 2), (8, 136, 2)):
        assert lib.moe_layer_fp8(q.ctx.handle, *[value if i == at else a for i, a in enumerate(args)]) == status
    with pytest.raises(ValueError):
        m.moe_layer_fp8(q.ctx, *q.args, q.mats[0], q.scales[0][:, :1].contiguous(), q.mats[1], q.scales[1])
    torch.cuda.synchronize()
    q.close()
    c.close()
