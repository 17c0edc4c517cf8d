"""Expert offsets that cannot be: what the products and the activation report, and
which rows they leave alone."""
import pytest
import torch

import expert_ref as X

PACKED = 1
pytestmark = pytest.mark.gpu


def calls(m, c, w, x, gu, d, order):
    """Every call on the rows, and the outputs that it made."""
    size, dev = c.size[order], "cuda"

    def new(width, dtype=torch.bfloat16):
        return torch.full((size, width), 7, dtype=dtype, device=dev)
    I = gu.shape[1] // 2
    yield "swiglu", [m.moe_swiglu(c.ctx, gu, c.handle, out=new(I), order=order)]
    yield "swiglu_fp8", m.moe_swiglu_fp8(c.ctx, gu, c.handle, out=new(I, torch.uint8), scales=new(I // 128, torch.float32), order=order)
    yield "swiglu_backward", [m.moe_swiglu_backward(c.ctx, d, gu, c.handle, grad_gate_up=new(2 * I), order=order)]
    yield "gemm", [m.moe_expert_gemm(c.ctx, x, w, c.handle, out=new(w.shape[1]), rows_order=order, out_order=order)]
    yield "backward_rows", [m.moe_expert_gemm_backward_rows(c.ctx, x, w.transpose(1, 2).contiguous(), c.handle, grad_rows=new(w.shape[1]),
                                                            rows_order=order, out_order=order)]


def rows_and_calls(m, features=128, **case):
    c = X.Case(m, **case)
    order = PACKED
    w, x = c.randn(c.E, 16, 64).cuda(), c.buffer(order, c.randn(c.n, 64), 0.0)
    gu, d = c.buffer(order, c.randn(c.n, 2 * features), 0.0), c.buffer(order, c.randn(c.n, features), 0.0)
    return c, lambda: calls(m, c, w, x, gu, d, order)


def offsets(c, values):
    c.handle.expert_offsets.copy_(torch.tensor(values, dtype=torch.int32))


@pytest.mark.parametrize("features", [128, 256, 640])
@pytest.mark.parametrize("layout", [0, 1])
def test_offsets_that_descend_are_reported_by_every_call(gpu, layout, features):
    c, every = rows_and_calls(gpu, T=20, k=2, E=4, R=2, layout=layout, src=1, features=features)
    right = c.handle.expert_offsets.clone()
    for bad in ([0, 5, 3, 20, 40], [-1, 10, 20, 30, 40], [0, 10, 41, 30, 40], [0, 10, 20, 30, 41], [0, 10, 20, 30, -1]):
        offsets(c, bad)
        gen = every()
        for name, outs in gen:
            assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_ERR_DEVICE_BOUNDS, (name, bad)
            if not 0 <= bad[-1] <= 40 and name.startswith("swiglu"):
                assert all((o == 7).all() for o in outs), (name, bad)
    c.handle.expert_offsets.copy_(right)
    for name, outs in every():
        assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_OK, name
    c.close()


def test_the_last_expert_of_many_is_looked_at(gpu):
    c, every = rows_and_calls(gpu, T=20, k=2, E=1024)
    n = c.handle.expert_offsets.cpu().tolist()
    for e in (1, 255, 256, 1023):
        offsets(c, n[:e] + [41] + n[e + 1:])
        for name, _ in every():
            assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_ERR_DEVICE_BOUNDS, (name, e)
    c.close()


def test_offsets_past_the_tokens_of_the_handle(gpu):
    """20 tokens of at most 40 in two slots each: 40 rows, in buffers of 80."""
    c, every = rows_and_calls(gpu, T=20, k=2, E=4, max_tokens=40)
    for bad, kept in (([0, 10, 20, 30, 80], 30), ([0, 10, 20, 30, 41], 30), ([0, 60, 70, 75, 80], 0), ([50, 60, 70, 75, 80], 0)):
        offsets(c, bad)
        for name, outs in every():
            assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_ERR_DEVICE_BOUNDS, (name, bad)
            rows = 0 if name.startswith("swiglu") else kept
            assert all((o[rows:] == 7).all() for o in outs), (name, bad)
            assert all((o[:rows] != 7).any() for o in outs) or rows == 0, (name, bad)
        grad = torch.full((4, 16, 64), 7.0, device="cuda")
        gpu.moe_expert_gemm_backward_weights(c.ctx, torch.ones(80, 16, dtype=torch.bfloat16, device="cuda"),
                                             torch.ones(80, 64, dtype=torch.bfloat16, device="cuda"), c.handle, grad_weights=grad)
        assert gpu.moe_poll_error(c.ctx)[0] == gpu.MOE_ERR_DEVICE_BOUNDS
        assert (grad[:3] == (10.0 if kept else 0.0)).all() and (grad[3] == 0).all()
    c.close()


@pytest.mark.parametrize("layout", [0, 1])
def test_a_handle_without_tokens_has_no_rows(gpu, layout):
    m = gpu
    ctx = m.Context(m.make_config(4, 128, 3, 1, 2, 0, m.MOE_QUANT_BF16, layout))
    h = m.Handle(ctx)
    h.expert_offsets.fill_(5)   # what an earlier call left; a dispatch of no tokens writes zeros
    bufs, h = m.moe_dispatch(ctx, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"),
                             torch.empty(0, 2, dtype=torch.int64, device="cuda"), handle=h)
    gw = m.moe_expert_gemm_backward_weights(ctx, torch.ones(bufs.recv_rows.shape[0], 16, dtype=torch.bfloat16, device="cuda"),
                                            bufs.recv_rows, h)
    assert (gw == 0).all() and m.moe_poll_error(ctx)[0] == m.MOE_OK
    ctx.close()


@pytest.mark.parametrize("layout", [0, 1])
def test_after_a_stale_layout_the_other_tokens_are_right(gpu, layout):
    """Tokens whose routing changed after the layout are dropped and reported; their places stay in the segments."""
    m, T, k, E, K, N = gpu, 40, 2, 6, 128, 72
    g = torch.Generator().manual_seed(4)
    ctx = m.Context(m.make_config(T, K, E, 1, k, 0, m.MOE_QUANT_BF16, layout))
    idx = torch.rand(T, E, generator=g).topk(k, dim=1).indices
    x = torch.randn(T, K, generator=g).bfloat16()
    w = (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16()
    dev = idx.cuda()
    m.moe_dispatch_layout(ctx, dev)
    changed = torch.zeros(T, dtype=torch.bool)
    changed[3::7] = True
    dev[changed.cuda(), 0] = (dev[changed.cuda(), 0] + 1) % E
    bufs = m.DispatchBuffers(ctx)
    bufs.recv_rows.fill_(float("nan"))
    bufs, h = m.moe_dispatch(ctx, x.cuda(), dev, bufs=bufs, reuse_layout=True)
    out = m.moe_expert_gemm(ctx, bufs.recv_rows, w.cuda(), h).cpu()
    assert m.moe_poll_error(ctx)[0] == m.MOE_ERR_STALE_LAYOUT
    pos = h.pos.cpu()
    assert (pos[changed] == -1).all() and (pos[~changed] >= 0).all()
    for t in torch.nonzero(~changed).flatten().tolist():
        for j in range(k):
            e = int(idx[t, j])
            ref, mag = w[e].double() @ x[t].double(), w[e].double().abs() @ x[t].double().abs()
            X.check(out[pos[t, j]], ref, X.sum_bound(ref, mag, K, X.BF16_HALF), "token %d" % t)
    ctx.close()
