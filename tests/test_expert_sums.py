"""How exactly the expert products add.  E4M3 products: rows and matrices whose codes
spread over the whole format, against the bound that the matrix instruction keeps."""
import pytest
import torch

import expert_ref as X

RECV = 0

# The E4M3 matrix instruction adds the products of eight neighbouring channels after it has cut each, towards zero, to
# a multiple of 2^(m - 13), m the largest sum of two operands' exponents among the eight (E4M3's smallest numbers count
# with the exponent -6).  The product with that exponent has 6 bits behind its leading one and loses nothing, so at
# most seven products lose less than 2^(m - 13) each.
GROUP, LOST = 8, 7 * 2.0 ** -13


def exponents(codes):
    """Exponents of E4M3 numbers, -inf for zeros."""
    v = X.e4m3(codes).float().abs()
    return torch.where(v > 0, torch.floor(torch.log2(v)).clamp(min=-6.0), torch.full_like(v, -float("inf")))


def cut(xq, wq):
    """Most that the instruction loses in each (row, column, block of 128): [rows, columns, blocks]."""
    ex, ew = exponents(xq).unflatten(1, (-1, GROUP)), exponents(wq).unflatten(1, (-1, GROUP))
    m = torch.full((xq.shape[0], wq.shape[0], ex.shape[1]), -float("inf"))
    for j in range(GROUP):
        torch.maximum(m, ex[:, None, :, j] + ew[None, :, :, j], out=m)
    return LOST * torch.exp2(m.double()).unflatten(2, (-1, 128 // GROUP)).sum(3)


def wide(gen, *shape):
    """E4M3 codes of normal numbers times powers of two over the format's range."""
    v = torch.randn(*shape, generator=gen) * torch.exp2(torch.randint(-9, 8, shape, generator=gen).float())
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def test_bound_of_a_group():
    """The bound against the cut itself, and that numbers of one size stay below it by far."""
    g = torch.Generator().manual_seed(1)
    for draw in (wide, lambda g, *s: (torch.randn(*s, generator=g) * 112).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)):
        xq, wq = draw(g, 40, 128), draw(g, 30, 128)
        p = X.e4m3(xq)[:, None] * X.e4m3(wq)[None]
        m = (exponents(xq)[:, None] + exponents(wq)[None]).unflatten(2, (-1, GROUP)).amax(3, keepdim=True).double()
        step = torch.where(m.isinf(), torch.ones_like(m), torch.exp2(m - 13))
        kept = (torch.trunc(p.unflatten(2, (-1, GROUP)) / step) * step).sum((2, 3))
        assert ((kept - p.sum(2)).abs() <= cut(xq, wq).sum(2)).all()
        # sums of numbers of one size stay within a binary32 sum's bound, those of codes of every size do not
        inside = (kept - p.sum(2)).abs() <= X.sum_bound(p.sum(2), p.abs().sum(2), 128, 0.0)
        assert inside.all() == (draw is not wide)
        assert (p.unflatten(2, (-1, GROUP)).abs().amax(3, keepdim=True) < 4 * torch.exp2(m)).all()


# rows of the experts, columns, blocks of 128 channels: each of the kernels, from one row to tiles of 256
CASES = {
    "a row": ([1, 0, 1], 136, 5),
    "a few rows": ([40], 136, 4),
    "32-row tiles": ([1, 3, 0, 8, 1, 2, 1, 1, 5, 1] * 10, 400, 4),
    "64-row tiles": ([31, 33, 64, 65, 100, 129, 200, 0, 1], 1064, 2),
    "128-row tiles": ([64, 65, 127, 128, 129, 255, 256, 257], 1608, 2),
    "256 columns": ([0, 1, 32, 33, 64, 65, 128, 129, 160, 161, 192, 193, 256, 257] * 8, 264, 4),
    "256 columns, an odd number of blocks": ([0, 1, 32, 33, 64, 65, 128, 129, 160, 161, 192, 193, 256, 257] * 8, 264, 3),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_e4m3_codes_of_every_size(gpu, name):
    lengths, N, blocks = CASES[name]
    E, K = len(lengths), 128 * blocks
    idx = torch.arange(E).repeat_interleave(torch.tensor(lengths)).reshape(-1, 1)
    c = X.Case(gpu, T=idx.numel(), k=1, E=E, idx=idx)
    xq, wq = wide(c.gen, c.n, K), wide(c.gen, E, N, K)
    xs = torch.rand(c.n, blocks, generator=c.gen) + 0.5
    ws = torch.rand(E, -(-N // 128), blocks, generator=c.gen) + 0.5
    out = gpu.moe_expert_gemm_fp8(c.ctx, xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), c.handle)[:c.n].cpu()
    for e, r in enumerate(c.segments()):
        if r.numel() == 0:
            continue
        x, w = X.e4m3(xq[r]) * xs[r].double().repeat_interleave(128, 1), X.e4m3(wq[e]) * X.expand(ws[e], N, K)
        scales = xs[r].double()[:, None, :] * ws[e].double().repeat_interleave(128, 0)[:N][None]
        lost = (cut(xq[r], wq[e]) * scales).sum(2)
        ref = x @ w.t()
        X.check(out[r], ref, lost * (1 + X.BF16_HALF) + X.sum_bound(ref, x.abs() @ w.abs().t(), K, X.BF16_HALF), "expert %d" % e)
    c.close()
