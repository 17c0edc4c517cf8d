"""The expert products with many tiles: segments of every length around the tile
sizes, contractions of every number of steps, the largest features, buffers past
4 GB, other streams, and captured graphs whose inputs change."""
import pytest
import torch

import expert_ref as X

RECV, PACKED = 0, 1
pytestmark = pytest.mark.gpu

# rows of the experts, in turn: on both sides of every tile size
LENGTHS = [0, 1, 16, 17, 32, 33, 64, 65, 96, 128, 129, 144, 145, 160, 161, 192, 193, 255, 256, 257, 300, 517]
EXPERTS = 6 * len(LENGTHS)


@pytest.fixture(scope="module")
def case(gpu):
    e = torch.arange(EXPERTS).repeat_interleave(torch.tensor(LENGTHS * 6))
    idx = e[torch.randperm(e.numel(), generator=torch.Generator().manual_seed(5))].reshape(-1, 1)
    c = X.Case(gpu, T=e.numel(), k=1, E=EXPERTS, R=4, idx=idx)
    yield c
    c.close()


@pytest.mark.parametrize("K,N", [(8, 264), (64, 256), (72, 520), (128, 40), (192, 264), (256, 264), (320, 264), (512, 136),
                                 (576, 264), (1000, 8)])
def test_gemm(gpu, case, K, N):
    c = case
    w, x = c.randn(EXPERTS, N, K, scale=K ** -0.5), c.randn(c.n, K)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    out = torch.full((c.n, N), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_expert_gemm(c.ctx, c.buffer(RECV, x, float("nan")), w.cuda(), c.handle, out=out)
    X.check(c.rows_of(out, RECV)[0], ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")


@pytest.mark.parametrize("blocks,N", [(1, 264), (2, 256), (3, 136), (4, 264), (5, 8), (6, 264), (7, 264), (8, 264), (9, 136),
                                      (12, 264)])
def test_gemm_fp8(gpu, case, blocks, N):
    c, K = case, 128 * blocks
    wq = (c.randn(EXPERTS, N, K, scale=112.0).float().clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.rand(EXPERTS, -(-N // 128), blocks, generator=c.gen) * 0.01 + 1e-4
    xq, xs = X.quantise(c.randn(c.n, K).float() * torch.rand(c.n, 1, generator=c.gen) * 10)
    w = X.e4m3(wq) * X.expand(ws, N, K)
    x = X.e4m3(xq) * xs.double().repeat_interleave(128, 1)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    out = gpu.moe_expert_gemm_fp8(c.ctx, c.buffer(RECV, xq, 0x7F), c.buffer(RECV, xs, float("nan")), wq.cuda(), ws.cuda(), c.handle)
    X.check(c.rows_of(out, RECV)[0], ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")


@pytest.mark.parametrize("K,N", [(264, 8), (256, 64), (520, 72), (40, 128), (264, 192), (264, 320), (136, 520)])
def test_backward_rows(gpu, case, K, N):
    c = case
    w, dy = c.randn(EXPERTS, N, K, scale=N ** -0.5), c.randn(c.n, N)
    wt = w.transpose(1, 2).contiguous()
    ref, mag = X.per_expert(c, dy, wt), X.per_expert(c, dy.abs(), wt.abs())
    grad = gpu.moe_expert_gemm_backward_rows(c.ctx, c.buffer(RECV, dy, float("nan")), w.cuda(), c.handle)
    X.check(c.rows_of(grad, RECV)[0], ref, X.sum_bound(ref, mag, N, X.BF16_HALF), "grad_rows")


@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False), (torch.bfloat16, True),
                                              (torch.float32, True)])
@pytest.mark.parametrize("K,N", [(264, 520), (8, 8), (256, 256), (72, 264)])
def test_backward_weights(gpu, case, K, N, dtype, accumulate):
    c = case
    x, dy = c.randn(c.n, K), c.randn(c.n, N)
    before = c.randn(EXPERTS, N, K).to(dtype) if accumulate else torch.full((EXPERTS, N, K), float("nan"), dtype=dtype)
    ref, mag = X.outer(c, dy, x, EXPERTS), X.outer(c, dy.abs(), x.abs(), EXPERTS)
    if accumulate:
        ref, mag = ref + before.double(), mag + before.double().abs()
    grad = before.cuda()
    gpu.moe_expert_gemm_backward_weights(c.ctx, c.buffer(RECV, dy, float("nan")), c.buffer(RECV, x, float("nan")), c.handle,
                                         grad_weights=grad, accumulate=accumulate)
    half = X.BF16_HALF if dtype is torch.bfloat16 else X.F32_STEP / 2
    X.check(grad.cpu(), ref, X.sum_bound(ref, mag, max(LENGTHS), half), "grad_weights")


@pytest.mark.parametrize("E,T", [(2, 5), (140, 150)])    # narrow tiles, wide tiles
@pytest.mark.parametrize("K,N", [(65536, 8), (8, 65536)])
def test_largest_features(gpu, E, T, K, N):
    c = X.Case(gpu, T=T, k=1, E=E)
    w, x, dy = c.randn(E, N, K, scale=K ** -0.5), c.randn(c.n, K), c.randn(c.n, N)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    wd, xd, dyd = w.cuda(), c.buffer(RECV, x, 0.0), c.buffer(RECV, dy, 0.0)
    out = gpu.moe_expert_gemm(c.ctx, xd, wd, c.handle)
    X.check(c.rows_of(out, RECV)[0], ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
    wt = w.transpose(1, 2).contiguous()
    ref, mag = X.per_expert(c, dy, wt), X.per_expert(c, dy.abs(), wt.abs())
    grad = gpu.moe_expert_gemm_backward_rows(c.ctx, dyd, wd, c.handle)
    X.check(c.rows_of(grad, RECV)[0], ref, X.sum_bound(ref, mag, N, X.BF16_HALF), "grad_rows")
    gw = gpu.moe_expert_gemm_backward_weights(c.ctx, dyd, xd, c.handle)
    ref, mag = X.outer(c, dy, x, E), X.outer(c, dy.abs(), x.abs(), E)
    X.check(gw.cpu(), ref, X.sum_bound(ref, mag, T, X.BF16_HALF), "grad_weights")
    c.close()


def test_matrices_past_4_gb(gpu):
    """40 matrices of 8192 x 8192: the last ones start past 2^32 bytes, in the products and in fp32 gradients."""
    E, K = 40, 8192
    c = X.Case(gpu, T=2 * E, k=1, E=E)
    w = torch.zeros((E, K, K), dtype=torch.bfloat16, device="cuda")
    last = c.randn(K, K, scale=K ** -0.5)
    w[E - 1] = last.cuda()
    x = c.randn(c.n, K)
    r = c.expert == E - 1
    assert r.any()
    out = c.rows_of(gpu.moe_expert_gemm(c.ctx, c.buffer(RECV, x, 0.0), w, c.handle), RECV)[0]
    ref = x[r].double() @ last.double().t()
    X.check(out[r], ref, X.sum_bound(ref, x[r].double().abs() @ last.double().abs().t(), K, X.BF16_HALF), "out")
    assert (out[~r] == 0).all()
    grad = c.rows_of(gpu.moe_expert_gemm_backward_rows(c.ctx, c.buffer(RECV, x, 0.0), w, c.handle), RECV)[0]
    ref = x[r].double() @ last.double()
    X.check(grad[r], ref, X.sum_bound(ref, x[r].double().abs() @ last.double().abs(), K, X.BF16_HALF), "grad_rows")
    del w
    gw = torch.empty((E, K, K), dtype=torch.float32, device="cuda")
    xd = c.buffer(RECV, x, 0.0)
    gpu.moe_expert_gemm_backward_weights(c.ctx, xd, xd, c.handle, grad_weights=gw)
    ref = x[r].double().t() @ x[r].double()
    X.check(gw[E - 1].cpu(), ref, X.sum_bound(ref, x[r].double().abs().t() @ x[r].double().abs(), int(r.sum()), X.F32_STEP / 2),
            "grad_weights")
    c.close()
    del gw
    torch.cuda.empty_cache()


def test_padded_rows_past_4_gb(gpu):
    """The padded layout's windows of the last experts start past 2^32 bytes."""
    T, k, E, R, K, N = 64, 4, 256, 32, 8192, 16
    c = X.Case(gpu, T=T, k=k, E=E, R=R, layout=1, src=31)
    w, x = c.randn(E, N, K, scale=K ** -0.5), c.randn(c.n, K)
    assert int(c.at[RECV].max()) * K * 2 > 2 ** 32
    rows = torch.full((c.size[RECV], K), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[c.at[RECV].cuda()] = x.cuda()
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    out = gpu.moe_expert_gemm(c.ctx, rows, w.cuda(), c.handle)
    X.check(out[c.at[RECV].cuda()].cpu(), ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
    act = gpu.moe_swiglu(c.ctx, rows, c.handle, out=torch.zeros(c.size[RECV], K // 2, dtype=torch.bfloat16, device="cuda"))
    ref = X.swiglu64(x)
    X.check(act[c.at[RECV].cuda()].cpu(), ref, (X.BF16_HALF + 128 * X.F32_STEP) * ref.abs() + 2.0 ** -120, "act")
    c.close()
    del rows, out, act
    torch.cuda.empty_cache()


def test_contexts_on_concurrent_streams(gpu):
    """Two contexts at once on two streams, neither of them the one their tensors were made on."""
    cases = [X.Case(gpu, T=300, k=2, E=40, seed=s) for s in (1, 2)]
    data = []
    for c in cases:
        w = c.randn(40, 528, 264, scale=0.06).cuda()
        x, dy = c.buffer(RECV, c.randn(c.n, 264), 0.0), c.buffer(RECV, c.randn(c.n, 528), 0.0)

        def calls(c=c, w=w, x=x, dy=dy):
            y = gpu.moe_expert_gemm(c.ctx, x, w, c.handle)
            return (y, gpu.moe_expert_gemm_backward_rows(c.ctx, dy, w, c.handle),
                    gpu.moe_expert_gemm_backward_weights(c.ctx, dy, x, c.handle), gpu.moe_swiglu(c.ctx, y, c.handle))
        data.append((calls, calls()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(data[i][0]())
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        for g in got[i]:
            for a, b in zip(g, data[i][1]):
                n = c.n if a.dim() == 2 else a.shape[0]
                assert torch.equal(a[:n], b[:n])
        c.close()


@pytest.mark.parametrize("T", [1, 24])
def test_captured_fp8_decode_step_with_new_inputs(gpu, T):
    """dispatch, product, quantising activation, product and combine as one graph, replayed on new tokens and new
    routings, with eager work in between: every replay gives the eager bits."""
    m, k, E, H, I = gpu, 2, 12, 512, 256
    ctx = m.Context(m.make_config(T, H, E, 2, k, 1, m.MOE_QUANT_FP8_E4M3, m.MOE_LAYOUT_PADDED_LL))
    g = torch.Generator().manual_seed(T)

    def mats(n, kk):
        q = (torch.randn(E, n, kk, generator=g) * 112).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return q.cuda(), ((torch.rand(E, -(-n // 128), kk // 128, generator=g) + 0.5) / 112 * kk ** -0.5).cuda()
    (q1, s1), (q2, s2) = mats(2 * I, H), mats(H, I)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int64, device="cuda")
    tw = torch.empty(T, k, device="cuda")
    bufs, h = m.DispatchBuffers(ctx), m.Handle(ctx)
    gu = torch.empty(T * k, 2 * I, dtype=torch.bfloat16, device="cuda")
    a, sa = torch.empty(T * k, I, dtype=torch.uint8, device="cuda"), torch.empty(T * k, I // 128, device="cuda")
    y = torch.empty(E * T * 2, H, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    def new_inputs():
        x.copy_(torch.randn(T, H, generator=g))
        i = torch.rand(T, E, generator=g).topk(k, dim=1).indices
        i[torch.rand(T, k, generator=g) < 0.2] = -1
        idx.copy_(i)
        tw.copy_(torch.rand(T, k, generator=g))

    def step():
        m.moe_dispatch(ctx, x, idx, bufs=bufs, handle=h)
        m.moe_expert_gemm_fp8(ctx, bufs.recv_rows, bufs.recv_scales, q1, s1, h, out=gu, out_order=PACKED)
        m.moe_swiglu_fp8(ctx, gu, h, out=a, scales=sa, order=PACKED)
        m.moe_expert_gemm_fp8(ctx, a, sa, q2, s2, h, out=y, rows_order=PACKED)
        m.moe_combine(ctx, y, tw, h, out=out)
    side = torch.cuda.Stream()
    new_inputs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(4):
        new_inputs()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and (T == 1 or out.abs().sum() > 0)
    assert m.moe_poll_error(ctx)[0] == m.MOE_OK
    ctx.close()


def test_handle_of_the_allocation_free_dispatch(gpu):
    m = gpu
    c = X.Case(m, T=50, k=2, E=8, empty=0.1)
    scfg = m.StaticConfig(m.make_config(50, 128, 8, 1, 2))
    bufs, h = m.DispatchBuffers(scfg), m.Handle(scfg)
    m.moe_dispatch_noalloc(scfg, c.x, c.idx, bufs, h)
    w = c.randn(8, 72, 128, scale=0.1).cuda()
    a, b = m.moe_expert_gemm(c.ctx, bufs.recv_rows, w, h), m.moe_expert_gemm(c.ctx, c.bufs.recv_rows, w, c.handle)
    assert torch.equal(a[:c.n], b[:c.n])
    c.close()


def test_activation_with_more_items_than_workgroups(gpu):
    """65536 rows of 32768 channels and more: the kernel's workgroups loop."""
    T, I = 70001, 32768
    c = X.Case(gpu, T=T, k=1, E=4, hidden=8)
    probe = torch.tensor([0, 1, 65535, 65536, 69999, T - 1])
    v = c.randn(probe.numel(), 2 * I)
    gu = torch.zeros(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    gu[probe.cuda()] = v.cuda()
    out = torch.full((T, I), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_swiglu(c.ctx, gu, c.handle, out=out)
    ref = X.swiglu64(v)
    X.check(out[probe.cuda()].cpu(), ref, (X.BF16_HALF + 128 * X.F32_STEP) * ref.abs() + 2.0 ** -120, "act")
    out[probe.cuda()] = 0
    assert not out.any()
    c.close()
    del gu, out
    torch.cuda.empty_cache()


def test_grids_past_the_launch_limit_are_refused(gpu):
    """More tiles than one launch may have.  (The handle's offsets still describe four tokens.)"""
    import ctypes
    m, M, k, N = gpu, 1 << 20, 32, 65536
    ctx = m.Context(m.make_config(M, 8, 32, 1, k))
    idx = torch.arange(32, device="cuda").repeat(4, 1)
    bufs, h = m.moe_dispatch(ctx, torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"), idx)
    w = torch.zeros(32, N, 8, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(128, N, dtype=torch.bfloat16, device="cuda")

    def call():
        return m.load_library().moe_expert_gemm(ctx.handle, bufs.recv_rows.data_ptr(), 0, w.data_ptr(), 8, N,
                                                ctypes.byref(h.c), out.data_ptr(), 0, 0)
    assert call() == m.MOE_OK
    h.c.num_tokens = M
    assert call() == m.MOE_ERR_UNSUPPORTED
    ctx.close()
    del bufs, h, w, out
    torch.cuda.empty_cache()


# Few tiles.  Lengths of a mean of at most 8 (one wavefront a tile of 16 rows), of more (32 rows), and of enough rows
# and columns for the narrow tiles of a whole workgroup (64 x 64, 128 x 128), each on both sides of its tile sizes.
FEW = {
    "mean of 5": ([0, 1, 2, 16, 17, 0, 3, 5, 1, 33, 2, 0, 4, 1, 6, 0], [8, 16, 24, 40, 1000, 2056]),
    "mean of 31": ([0, 1, 15, 16, 17, 31, 32, 33, 64, 100], [8, 24, 40, 72, 1000, 3400]),
    "mean of 65": ([0, 1, 31, 32, 33, 63, 64, 65, 100, 129, 200], [1064, 1096]),
    "mean of 114": ([0, 1, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257], [1608, 2056]),
}
FEW_CASES = [(name, N) for name in FEW for N in FEW[name][1]]


def few_case(gpu, name):
    lengths = FEW[name][0]
    idx = torch.arange(len(lengths)).repeat_interleave(torch.tensor(lengths))
    idx = idx[torch.randperm(idx.numel(), generator=torch.Generator().manual_seed(3))].reshape(-1, 1)
    return X.Case(gpu, T=idx.numel(), k=1, E=len(lengths), R=1, idx=idx)


@pytest.mark.parametrize("K", [8, 40, 64, 248, 256, 264, 520, 1032, 2056])
@pytest.mark.parametrize("name,N", FEW_CASES)
def test_gemm_of_few_rows(gpu, name, N, K):
    c = few_case(gpu, name)
    w, x = c.randn(c.E, N, K, scale=K ** -0.5), c.randn(c.n, K)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    out = torch.full((c.n, N), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_expert_gemm(c.ctx, c.buffer(RECV, x, float("nan")), w.cuda(), c.handle, out=out)
    X.check(c.rows_of(out, RECV)[0], ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
    c.close()


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 8, 9, 17])
@pytest.mark.parametrize("name,N", FEW_CASES)
def test_gemm_fp8_of_few_rows(gpu, name, N, blocks):
    c, K = few_case(gpu, name), 128 * blocks
    wq = (c.randn(c.E, N, K, scale=112.0).float().clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.rand(c.E, -(-N // 128), blocks, generator=c.gen) * 0.01 + 1e-4
    xq, xs = X.quantise(c.randn(c.n, K).float() * torch.rand(c.n, 1, generator=c.gen) * 10)
    w = X.e4m3(wq) * X.expand(ws, N, K)
    x = X.e4m3(xq) * xs.double().repeat_interleave(128, 1)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    out = gpu.moe_expert_gemm_fp8(c.ctx, c.buffer(RECV, xq, 0x7F), c.buffer(RECV, xs, float("nan")), wq.cuda(), ws.cuda(), c.handle)
    X.check(c.rows_of(out, RECV)[0], ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
    c.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_largest_features_of_one_row(gpu, fp8):
    """The longest contraction and the most columns that a token can have."""
    for K, N in ((65536, 136), (128, 65536)):
        c = X.Case(gpu, T=1, k=2, E=3, hidden=128)
        if fp8:
            wq = (c.randn(c.E, N, K, scale=112.0).float().clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
            ws = torch.rand(c.E, -(-N // 128), K // 128, generator=c.gen) * 0.01 + 1e-4
            xq, xs = X.quantise(c.randn(c.n, K).float())
            w, x = X.e4m3(wq) * X.expand(ws, N, K), X.e4m3(xq) * xs.double().repeat_interleave(128, 1)
            out = gpu.moe_expert_gemm_fp8(c.ctx, c.buffer(RECV, xq, 0x7F), c.buffer(RECV, xs, float("nan")), wq.cuda(),
                                          ws.cuda(), c.handle)
        else:
            w, x = c.randn(c.E, N, K, scale=K ** -0.5), c.randn(c.n, K)
            out = gpu.moe_expert_gemm(c.ctx, c.buffer(RECV, x, float("nan")), w.cuda(), c.handle)
        ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
        X.check(c.rows_of(out, RECV)[0], ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
        c.close()


@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("E,K,N", [(3, 8, 8), (70, 136, 264), (130, 624, 1000), (1000, 72, 40)])
def test_weights_gradient_where_most_experts_have_no_rows(gpu, E, K, N, dtype, accumulate):
    """Runs of experts without rows at the start, between and at the end; matrices of more and less than one run of zeros."""
    busy = torch.tensor([1, E // 2, E // 2 + 1] if E > 3 else [1])
    idx = busy.repeat_interleave(torch.tensor([5, 300, 1][:busy.numel()])).reshape(-1, 1)
    c = X.Case(gpu, T=idx.numel(), k=1, E=E, idx=idx)
    x, dy = c.randn(c.n, K), c.randn(c.n, N)
    before = c.randn(E, N, K).to(dtype) if accumulate else torch.full((E, N, K), float("nan"), dtype=dtype)
    ref, mag = X.outer(c, dy, x, E), X.outer(c, dy.abs(), x.abs(), E)
    if accumulate:
        ref, mag = ref + before.double(), mag + before.double().abs()
    grad = before.cuda()
    gpu.moe_expert_gemm_backward_weights(c.ctx, c.buffer(RECV, dy, float("nan")), c.buffer(RECV, x, float("nan")), c.handle,
                                         grad_weights=grad, accumulate=accumulate)
    half = X.BF16_HALF if dtype is torch.bfloat16 else X.F32_STEP / 2
    X.check(grad.cpu(), ref, X.sum_bound(ref, mag, 300, half), "grad_weights")
    c.close()


@pytest.mark.parametrize("rows_order,out_order", [(RECV, RECV), (RECV, PACKED), (PACKED, RECV), (PACKED, PACKED)])
def test_padded_windows_with_many_tiles(gpu, rows_order, out_order):
    """Every product over slot windows where it has too many tiles for the narrow ones."""
    c = X.Case(gpu, T=70, k=3, E=66, R=2, layout=1, src=1, empty=0.1, max_tokens=72)
    E, K, N = 66, 1032, 1040
    orders = dict(rows_order=rows_order, out_order=out_order)
    w, x, dy = c.randn(E, N, K, scale=K ** -0.5), c.randn(c.n, K), c.randn(c.n, N)
    wt = w.transpose(1, 2).contiguous()
    rows, go = c.buffer(rows_order, x, float("nan")), c.buffer(out_order, dy, float("nan"))
    out = torch.full((c.size[out_order], N), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_expert_gemm(c.ctx, rows, w.cuda(), c.handle, out=out, **orders)
    got, rest = c.rows_of(out, out_order)
    X.check(got, X.per_expert(c, x, w), X.sum_bound(X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs()), K, X.BF16_HALF), "out")
    assert (rest == 7.0).all()
    grad = torch.full((c.size[rows_order], K), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_expert_gemm_backward_rows(c.ctx, go, w.cuda(), c.handle, grad_rows=grad, **orders)
    got, rest = c.rows_of(grad, rows_order)
    X.check(got, X.per_expert(c, dy, wt), X.sum_bound(X.per_expert(c, dy, wt), X.per_expert(c, dy.abs(), wt.abs()), N, X.BF16_HALF),
            "grad_rows")
    assert (rest == 7.0).all()
    gw = gpu.moe_expert_gemm_backward_weights(c.ctx, go, rows, c.handle, **orders)
    X.check(gw.cpu(), X.outer(c, dy, x, E), X.sum_bound(X.outer(c, dy, x, E), X.outer(c, dy.abs(), x.abs(), E), 70, X.BF16_HALF), "grad_w")
    K, N = 1024, 2056
    wq = (c.randn(E, N, K, scale=112.0).float().clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.rand(E, -(-N // 128), K // 128, generator=c.gen) * 0.01 + 1e-4
    xq, xs = X.quantise(c.randn(c.n, K).float())
    w8, x8 = X.e4m3(wq) * X.expand(ws, N, K), X.e4m3(xq) * xs.double().repeat_interleave(128, 1)
    out = gpu.moe_expert_gemm_fp8(c.ctx, c.buffer(rows_order, xq, 0x7F), c.buffer(rows_order, xs, float("nan")), wq.cuda(), ws.cuda(),
                                  c.handle, **orders)
    X.check(c.rows_of(out, out_order)[0], X.per_expert(c, x8, w8),
            X.sum_bound(X.per_expert(c, x8, w8), X.per_expert(c, x8.abs(), w8.abs()), K, X.BF16_HALF), "fp8")
    c.close()


@pytest.mark.parametrize("features", [8, 64, 120, 128, 256, 384, 504, 512, 520, 744, 1408])
@pytest.mark.parametrize("rows", [1, 7, 64, 1001])
def test_activation_of_rows_that_share_wavefronts(gpu, rows, features):
    c = X.Case(gpu, T=rows, k=1, E=3)
    size = c.size[RECV] + 3   # rows behind the last stay as they were
    gu, d = c.randn(rows, 2 * features, scale=2.0), c.randn(rows, features)
    tail = lambda v: torch.cat([c.buffer(RECV, v, 0.0), torch.full((3, v.shape[1]), float("nan"), dtype=v.dtype, device="cuda")])
    out = torch.full((size, features), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_swiglu(c.ctx, tail(gu), c.handle, out=out)
    ref = X.swiglu64(gu)
    X.check(out[:rows].cpu(), ref, (X.BF16_HALF + 128 * X.F32_STEP) * ref.abs() + 2.0 ** -120, "act")
    assert (out[rows:] == 7.0).all()
    grad = torch.full((size, 2 * features), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_swiglu_backward(c.ctx, tail(d), tail(gu), c.handle, grad_gate_up=grad)
    x = gu.double().requires_grad_()
    y = torch.nn.functional.silu(x[:, :features]) * x[:, features:]
    y.backward(d.double())
    # s (1 + g (1 - s)) cancels near its zero: errors are relative to 1 + |g|
    scale = torch.cat([(d.double() * x[:, features:]).abs() * (1 + x[:, :features].abs()), x.grad[:, features:].abs()], 1).detach()
    X.check(grad[:rows].cpu(), x.grad, X.BF16_HALF * x.grad.abs() + 128 * X.F32_STEP * scale + 2.0 ** -120, "grad")
    assert (grad[rows:] == 7.0).all()
    if features % 128 == 0:
        codes = torch.full((size, features), 3, dtype=torch.uint8, device="cuda")
        scales = torch.full((size, features // 128), 7.0, device="cuda")
        gpu.moe_swiglu_fp8(c.ctx, tail(gu), c.handle, out=codes, scales=scales)
        amax = ref.abs().reshape(rows, -1, 128).amax(2).clamp_min(1e-4)
        X.check(scales[:rows].cpu(), amax / 448, 130 * X.F32_STEP * amax / 448, "scales")
        v = X.e4m3(codes[:rows].cpu()) * scales[:rows].cpu().double().repeat_interleave(128, 1)
        # half a step of E4M3, or of its smallest numbers (2^-9), beside the binary32 error
        step = torch.maximum(ref.abs() * 2.0 ** -4, scales[:rows].cpu().double().repeat_interleave(128, 1) * 2.0 ** -10)
        X.check(v, ref, step * (1 + 1e-4) + 256 * X.F32_STEP * ref.abs(), "fp8")
        assert (codes[rows:] == 3).all() and (scales[rows:] == 7.0).all()
    c.close()


@pytest.mark.parametrize("T,K,N", [(1, 4096, 512), (64, 1024, 512), (300, 1024, 1096), (700, 512, 2056), (2000, 256, 8200)])
def test_the_same_call_gives_the_same_bits(gpu, T, K, N):
    """From one token to many, every product twice and into another buffer."""
    c = X.Case(gpu, T=T, k=2, E=8, empty=0.1)
    w, x, dy = c.randn(8, N, K, scale=K ** -0.5).cuda(), c.randn(T * 2, K).cuda(), c.randn(T * 2, N).cuda()
    xq, xs = X.quantise(x.float().cpu())
    wq = torch.randint(0, 120, (8, N, K), dtype=torch.uint8, generator=c.gen).cuda()
    ws = torch.rand(8, -(-N // 128), K // 128, generator=c.gen).cuda()
    xq, xs = xq.cuda(), xs.cuda()
    calls = [lambda: gpu.moe_expert_gemm(c.ctx, x, w, c.handle)[:c.n],
             lambda: gpu.moe_expert_gemm_fp8(c.ctx, xq, xs, wq, ws, c.handle)[:c.n],
             lambda: gpu.moe_expert_gemm_backward_rows(c.ctx, dy, w, c.handle)[:c.n],
             lambda: gpu.moe_expert_gemm_backward_weights(c.ctx, dy, x, c.handle)]
    for f in calls:
        first = f().view(torch.int16).clone()
        for _ in range(3):
            assert torch.equal(f().view(torch.int16), first)
    c.close()


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 7, 32])
@pytest.mark.parametrize("padded", [False, True])
def test_gemm_fp8_of_many_experts_with_few_rows(gpu, padded, blocks):
    c, E, K, N = X.Case(gpu, T=200, k=4, E=130, R=2, layout=int(padded), src=1, hot=3, max_tokens=200), 130, 128 * blocks, 776
    wq = (c.randn(E, N, K, scale=112.0).float().clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.rand(E, -(-N // 128), blocks, generator=c.gen) * 0.01 + 1e-4
    xq, xs = X.quantise(c.randn(c.n, K).float())
    w, x = X.e4m3(wq) * X.expand(ws, N, K), X.e4m3(xq) * xs.double().repeat_interleave(128, 1)
    ref, mag = X.per_expert(c, x, w), X.per_expert(c, x.abs(), w.abs())
    out = torch.full((c.size[PACKED], N), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu.moe_expert_gemm_fp8(c.ctx, c.buffer(RECV, xq, 0x7F), c.buffer(RECV, xs, float("nan")), wq.cuda(), ws.cuda(), c.handle,
                            out=out, out_order=PACKED)
    got, rest = c.rows_of(out, PACKED)
    X.check(got, ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "out")
    assert (rest == 7.0).all()
    c.close()
