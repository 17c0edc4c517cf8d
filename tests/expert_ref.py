"""Plain binary64 forms of the expert products and the gated activation, and the
routing and buffers their tests share.  Nothing here uses the library's kernels
but the dispatch that makes a handle."""
import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2   # a rounding is off by at most half a step, relative
F32_STEP = torch.finfo(torch.float32).eps         # one step: also covers sums that truncate
CONTIGUOUS, PADDED = 0, 1


class Case:
    """A routing on the device: its context, handle, and where every valid row stands in each order."""

    def __init__(self, moe, T, k, E, R=1, layout=CONTIGUOUS, src=0, empty=0.0, hot=None, max_tokens=None, hidden=128,
                 seed=0, idx=None, quant=0):
        self.moe, self.T, self.k, self.E, self.R, self.layout = moe, T, k, E, R, layout
        g = torch.Generator().manual_seed(seed)
        self.M = M = T if max_tokens is None else max_tokens
        if idx is None:
            keys = torch.rand(T, E, generator=g)
            if hot is not None:   # expert `hot` in every token's first slot, some experts in none
                keys[:, hot] += 2
                keys[:, hot + 1::3] -= 1
            idx = keys.topk(k, dim=1).indices
            idx[torch.rand(T, k, generator=g) < empty] = -1
        self.gen = g
        self.idx = idx.cuda()
        self.ctx = moe.Context(moe.make_config(max(M, 1), hidden, E, R, k, src, quant, layout))
        self.x = torch.randn(T, hidden, generator=g).bfloat16().cuda()
        self.bufs, self.handle = moe.moe_dispatch(self.ctx, self.x, self.idx)
        flat = idx.reshape(-1)
        valid = flat >= 0
        order = torch.sort(torch.where(valid, flat, E), stable=True).indices[:int(valid.sum())]
        self.expert = flat[order]
        self.counts = torch.bincount(self.expert, minlength=E)
        off = torch.cumsum(self.counts, 0) - self.counts
        self.n = order.numel()
        within = torch.arange(self.n) - off[self.expert]
        packed = torch.arange(self.n)
        cap = max(M, 1) * R
        placed = within < max(M, 1) if layout == PADDED else torch.ones(self.n, dtype=torch.bool)
        recv = self.expert * cap + src * max(M, 1) + within if layout == PADDED else packed
        self.placed = placed
        self.at = {moe.MOE_ROWS_RECV: recv[placed], moe.MOE_ROWS_PACKED: packed[placed]}
        self.expert = self.expert[placed]
        self.n = int(placed.sum())
        self.size = {moe.MOE_ROWS_RECV: E * cap if layout == PADDED else max(M, 1) * k, moe.MOE_ROWS_PACKED: max(M, 1) * k}

    def randn(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.gen) * scale).bfloat16()

    def buffer(self, order, values, fill):
        """A device row buffer with `values` at the valid rows and `fill` elsewhere."""
        b = torch.full((self.size[order], values.shape[1]), fill, dtype=values.dtype)
        b[self.at[order]] = values
        return b.cuda()

    def segments(self):
        return [torch.nonzero(self.expert == e).flatten() for e in range(self.E)]

    def rows_of(self, buf, order):
        """The valid rows of a buffer (cpu), and whether every other row still holds its fill value."""
        b = buf.cpu()
        other = torch.ones(b.shape[0], dtype=torch.bool)
        other[self.at[order]] = False
        return b[self.at[order]], b[other]

    def close(self):
        self.ctx.close()


def per_expert(case, rows, mats):
    """rows[r] mats[e(r)]^T in binary64."""
    out = torch.zeros(rows.shape[0], mats.shape[1], dtype=torch.float64)
    for e, r in enumerate(case.segments()):
        if r.numel():
            out[r] = rows[r].double() @ mats[e].double().t()
    return out


def outer(case, grad, rows, E):
    g = torch.zeros(E, grad.shape[1], rows.shape[1], dtype=torch.float64)
    for e, r in enumerate(case.segments()):
        if r.numel():
            g[e] = grad[r].double().t() @ rows[r].double()
    return g


def sum_bound(ref, mag, length, half):
    """Error of a binary32 sum of `length` exact products (magnitudes summing to
    mag), each addition off by at most one step, then one rounding by `half`."""
    acc = (length + 64) * F32_STEP * mag + 2.0 ** -120
    return acc + half * (ref.abs() + acc)


def check(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %g against %g" % (
        what, int(bad.sum()), bad.numel(), float((got.double() - ref).abs()[bad].max()), float(bound[bad].max()))


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float64)


def quantise(v):
    """E4M3 codes and binary32 scales of fp32 rows, one scale for each 128 channels."""
    b = v.float().unflatten(-1, (-1, 128))
    amax = b.abs().amax(-1, keepdim=True).clamp(min=1e-4)
    codes = (b * (448.0 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.flatten(-2).view(torch.uint8), (amax / 448.0).squeeze(-1)


def expand(scales, n, k):
    """Block scales [.., ceil(n/128), k/128] for every element [.., n, k]."""
    return scales.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def swiglu64(gu):
    g, u = gu.double().chunk(2, dim=1)
    return g * torch.sigmoid(g) * u
