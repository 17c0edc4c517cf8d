"""The router and its gradient against plain binary64 forms, at the sizes, masks, ties and
groups where they can go wrong; their refusals."""
import ctypes
import math

import pytest
import torch

gpu_only = pytest.mark.gpu
SOFTMAX, SIGMOID = 0, 1
INF = math.inf
STEP = torch.finfo(torch.float32).eps


# ---------------------------------------------------------------- plain forms, one token after another
def plain_scores(row, score):
    """Scores of one token's logits (float64 list, masked ones -inf)."""
    if score == SIGMOID:
        return [0.0 if v == -INF else 1 / (1 + math.exp(-v)) if v > -700 else math.exp(v) for v in row]
    m = max(row)
    if m == -INF:
        return [0.0] * len(row)
    e = [math.exp(v - m) for v in row]
    return [v / sum(e) for v in e]


def plain_choice(row, k, score, bias, groups, keep, top):
    s = plain_scores(row, score)
    if bias is None and groups == 1:
        key = list(row)
    else:
        key = [-INF if v == -INF else s[e] + (bias[e] if bias is not None else 0.0) for e, v in enumerate(row)]
    if groups > 1:
        size = len(row) // groups
        value = []
        for g in range(groups):
            best = [v for v in sorted(key[g * size:(g + 1) * size], reverse=True)[:top] if v > -INF]
            value.append(sum(best) if best else -INF)
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:keep]
        key = [v if e // size in kept else -INF for e, v in enumerate(key)]
    order = sorted(range(len(row)), key=lambda e: (-key[e], e))[:k]
    chosen = [e for e in order if key[e] > -INF]
    return chosen + [-1] * (k - len(chosen))


def plain_weights(row, chosen, score, normalize, scale):
    """Weights, and how far binary32 may be off them, relative: the exponent's rounding and a few steps for the rest."""
    s = plain_scores(row, score)
    there = [e for e in chosen if e >= 0]
    if not there:
        return [0.0] * len(chosen)
    if normalize:   # shares of a sum, from the logarithms, so that none is lost to underflow
        log = [row[e] if score == SOFTMAX else -math.log1p(math.exp(-row[e])) if row[e] > -700 else row[e] for e in there]
        share = [math.exp(v - max(log)) for v in log]
        w = dict(zip(there, [v / sum(share) for v in share]))
    else:
        w = {e: s[e] for e in there}
    return [scale * w[e] if e >= 0 else 0.0 for e in chosen]


def bound(w, row, E, k):
    """An exponential of a difference d is off by |d| + 4 half steps, a sum of n terms by n, the rest by a few."""
    finite = [v for v in row if v > -INF]
    spread = max(finite) - min(finite) if finite else 0.0
    return [abs(v) * (min(spread, 100.0) + E + k + 16) * STEP + 2.0 ** -120 for v in w]


def logits_of(g, T, E, dtype=torch.float32, masked=0.0, scale=2.0):
    v = torch.randn(T, E, generator=g) * scale
    v[torch.rand(T, E, generator=g) < masked] = -INF
    return v.to(dtype)


def run_and_check(moe, logits, k, score, normalize=True, scale=1.0, bias=None, groups=1, keep=1, top=1):
    T, E = logits.shape
    ctx = moe.Context(moe.make_config(max(T, 1), 8, E, 1, k))
    idx = torch.full((T, k), -7, dtype=torch.int64, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    got = moe.moe_route(ctx, logits.cuda(), score, bias=None if bias is None else bias.cuda(), groups=groups, topk_groups=keep,
                        group_top=top, normalize=normalize, scale=scale, topk_idx=idx, topk_weights=w)
    assert got[0] is idx and got[1] is w
    rows = logits.double().tolist()
    b = None if bias is None else bias.double().tolist()
    for t, row in enumerate(rows):
        row = [v if v < INF else -INF for v in row]   # NaN compares false
        chosen = plain_choice(row, k, score, b, groups, keep, top)
        assert idx[t].tolist() == chosen, (t, idx[t].tolist(), chosen)
        ref = plain_weights(row, chosen, score, normalize, scale)
        for x, y, d in zip(w[t].tolist(), ref, bound(ref, row, E, k)):
            assert abs(x - y) <= d, (t, x, y, d)
    return ctx, idx, w


SIZES = [(1, 1, 1), (3, 2, 2), (5, 7, 3), (17, 16, 4), (9, 17, 17), (33, 60, 6), (257, 64, 6), (4, 65, 8), (6, 128, 8), (7, 130, 32),
         (40, 256, 8), (5, 257, 5), (6, 512, 8), (3, 1000, 31), (2, 1024, 32)]


@gpu_only
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route(gpu, T, E, k, score, dtype):
    g = torch.Generator().manual_seed(E + T)
    for normalize, scale, masked, biased in ((True, 1.0, 0.0, False), (False, 2.5, 0.3, False), (True, 2.5, 0.3, True), (False, 1.0, 0.0, True)):
        # bf16 logits tie often: the lowest expert is taken
        bias = torch.randn(E, generator=g) * 0.2 if biased else None
        ctx, _, _ = run_and_check(gpu, logits_of(g, T, E, dtype, masked), k, score, normalize, scale, bias)
        assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
        ctx.close()


@gpu_only
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("E,groups,keep,top,k", [(8, 8, 3, 1, 2), (8, 2, 1, 2, 4), (12, 4, 2, 2, 6), (60, 5, 2, 2, 4), (64, 64, 7, 2, 6), (256, 8, 4, 2, 8),
                                                 (256, 8, 4, 1, 8), (256, 64, 4, 2, 8), (300, 3, 2, 2, 8), (1024, 32, 5, 2, 32), (2, 2, 2, 1, 2), (4, 2, 1, 2, 4)])
def test_groups(gpu, E, groups, keep, top, k, score):
    g = torch.Generator().manual_seed(E + groups)
    for masked, biased in ((0.0, True), (0.4, True), (0.7, False)):
        bias = torch.randn(E, generator=g) * 0.3 if biased else None
        ctx, _, _ = run_and_check(gpu, logits_of(g, 21, E, masked=masked), k, score, True, 2.5, bias, groups, keep, top)
        ctx.close()


@gpu_only
@pytest.mark.parametrize("E", [6, 64, 200, 600])
def test_masks_and_ties(gpu, E):
    """Rows with nothing, one or few experts left; equal logits; the type's lowest and highest values; bias that masks."""
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    v = torch.zeros(10, E)
    v[0] = -INF
    v[1] = -INF
    v[1, E - 1] = -3.0
    v[2] = low
    v[3, ::2] = low
    v[4] = high
    v[5, 1] = high
    v[6] = -200.0
    v[7] = -80.0
    v[7, 3] = 90.0
    v[8] = -INF
    v[8, [0, E // 2]] = low
    for score in (SOFTMAX, SIGMOID):
        for bias in (None, torch.tensor([0.0, -INF] + [0.0] * (E - 2))):
            for groups in (1, 2):
                if bias is not None or groups > 1:
                    v[6] = -20.0   # their scores in 64 bits do not vanish beside the bias
                run = dict(score=score, bias=bias, groups=groups, keep=1, top=2)
                for normalize in (True, False):
                    rows = v[[0, 1, 4, 5, 6, 7, 9]] if normalize and score == SIGMOID else v   # 0 / 0 elsewhere
                    ctx, idx, w = run_and_check(gpu, rows, 4, normalize=normalize, **run)
                    assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
                    assert (idx[0] == -1).all() and (w[0] == 0).all()
                    ctx.close()


@gpu_only
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_not_finite_is_reported_and_not_chosen(gpu, bad, dtype):
    v = torch.randn(6, 40, generator=torch.Generator().manual_seed(1)).to(dtype)
    v[2, 7] = bad
    v[3] = bad
    for bias in (None, torch.zeros(40)):
        ctx, idx, w = run_and_check(gpu, v, 5, SOFTMAX, bias=bias)
        assert (idx[3] == -1).all() and (w[3] == 0).all()
        assert gpu.moe_poll_error(ctx)[0] == gpu.MOE_ERR_NONFINITE
        ctx.close()


@gpu_only
def test_keys_are_compared_beyond_binary32(gpu):
    """Two scores that agree in binary32 with their bias added are still taken in the formula's order."""
    E, T = 32, 64
    v = torch.full((T, E), -30.0)
    v[:, 5] = -29.0   # sigmoids near 1e-13, below half a step of the bias
    v[:, 9] = -28.0
    ctx, idx, _ = run_and_check(gpu, v, 3, SIGMOID, bias=torch.ones(E))
    assert (idx[:, 0] == 9).all() and (idx[:, 1] == 5).all()
    ctx.close()


@gpu_only
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_apart(gpu, dtype):
    """Logits that are columns of a wider product, at any offset, and outputs inside larger buffers."""
    g = torch.Generator().manual_seed(3)
    T, E, k = 37, 60, 4
    wide = logits_of(g, T, 77, dtype).cuda()
    wide[:, :5], wide[:, 65:] = float("nan"), float("nan")
    ctx = gpu.Context(gpu.make_config(50, 8, E, 1, k))
    part = wide[:, 5:65]
    idx = torch.full((T + 3, k), -7, dtype=torch.int64, device="cuda")
    w = torch.full((T + 3, k), 7.0, device="cuda")
    gpu.moe_route(ctx, part, topk_idx=idx[:T], topk_weights=w[:T])
    same = gpu.moe_route(ctx, part.contiguous())
    assert torch.equal(idx[:T], same[0]) and torch.equal(w[:T], same[1])
    assert (idx[T:] == -7).all() and (w[T:] == 7.0).all()
    d = torch.randn(T, k, generator=g).cuda()
    gl = torch.full((T + 2, E), 7.0, device="cuda")
    gpu.moe_route_backward(ctx, d, part, idx[:T], grad_logits=gl[:T])
    assert torch.equal(gl[:T], gpu.moe_route_backward(ctx, d, part.contiguous(), same[0]))
    assert (gl[T:] == 7.0).all()
    assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
    ctx.close()


# ---------------------------------------------------------------- gradient
def forward64(v, idx, score, normalize, scale):
    """Weights of the given experts, binary64, differentiable.  v: [T, E] with masked logits at -inf."""
    there = idx >= 0
    at = idx.clamp(min=0)
    some = (v > -INF).any(1, keepdim=True)
    s = torch.sigmoid(v) if score == SIGMOID else torch.softmax(torch.where(some, v, 0.0), 1)
    c = torch.where(there, s.gather(1, at), 0.0)
    if normalize:
        n = c.sum(1, keepdim=True)
        c = c / torch.where(n > 0, n, 1.0)
    return c * scale


@gpu_only
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gradient(gpu, T, E, k, score, normalize):
    g = torch.Generator().manual_seed(7 * E + T)
    for masked, dtype in ((0.0, torch.float32), (0.4, torch.float32), (0.0, torch.bfloat16)):
        v = logits_of(g, T, E, dtype, masked)
        ctx = gpu.Context(gpu.make_config(T, 8, E, 1, k))
        idx, _ = gpu.moe_route(ctx, v.cuda(), score, normalize=normalize, scale=2.5)
        d = torch.randn(T, k, generator=g)
        d[idx.cpu() < 0] = float("nan")   # an empty slot's gradient is not read
        got = gpu.moe_route_backward(ctx, d.cuda(), v.cuda(), idx, score, normalize=normalize, scale=2.5).double().cpu()
        idx = idx.cpu()
        v64 = v.double().requires_grad_()
        w = forward64(v64, idx, score, normalize, 2.5)
        dd = torch.where(idx >= 0, d, 0.0).double()
        ref = torch.autograd.grad(w, v64, dd)[0]
        ref = torch.where(v64.detach() > -INF, ref, 0.0)
        # terms of size weight times gradient, each off by a few steps for its exponentials and sums, cancel
        size = (w.detach().abs() * dd.abs()).sum(1, keepdim=True) + (w.detach().abs() * dd.abs().amax(1, keepdim=True)).sum(1, keepdim=True)
        assert ((got - ref).abs() <= (40 + E + k) * STEP * size + 2.0 ** -110).all()
        # and against differences of the weights, along a direction
        if masked == 0.0:
            direction = torch.randn(T, E, generator=g, dtype=torch.float64)
            h = 1e-5
            up, down = (forward64(v64.detach() + s * h * direction, idx, score, normalize, 2.5) for s in (1, -1))
            slope = ((up - down) * dd).sum(1) / (2 * h)
            along = (got * direction).sum(1)
            # cubic terms of the difference, its rounding, and the kernel's own steps
            tol = (1e-8 + 64 * (40 + E + k) * STEP) * (1 + size.squeeze(1)) * (1 + direction.abs().amax(1)) ** 3
            assert ((along - slope).abs() <= tol).all()
        assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
        ctx.close()


@gpu_only
@pytest.mark.parametrize("score,normalize", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True), (SIGMOID, False)])
def test_gradient_of_given_experts(gpu, score, normalize):
    """An expert in two slots gets both gradients; ids out of range, and masked experts, have no part."""
    g = torch.Generator().manual_seed(5)
    v = logits_of(g, 4, 20)
    v[3, 6] = -INF
    idx = torch.tensor([[3, 3, 5], [1, -1, 1], [19, 20, 0], [6, 2, -9]])
    d = torch.randn(4, 3, generator=g)
    ctx = gpu.Context(gpu.make_config(4, 8, 20, 1, 3))
    got = gpu.moe_route_backward(ctx, d.cuda(), v.cuda(), idx.cuda(), score, normalize=normalize).double().cpu()
    assert gpu.moe_poll_error(ctx)[0] == gpu.MOE_ERR_BAD_TOPK
    right = torch.tensor([[3, 3, 5], [1, -1, 1], [19, -1, 0], [-1, 2, -1]])
    v64 = v.double().requires_grad_()
    w = forward64(v64, right, score, normalize, 1.0)
    ref = torch.autograd.grad(w, v64, torch.where(right >= 0, d, 0.0).double())[0]
    ref = torch.where(v64.detach() > -INF, ref, 0.0)
    assert ((got - ref).abs() <= 100 * STEP * (1 + d.abs().sum(1, keepdim=True))).all()
    ctx.close()


def plain_gradient(v, idx, d, score, normalize, scale):
    """The gradient of one token's weights as sums of differences, none of which cancels in binary64, and the sum of their sizes.
    v: float64 [E] without NaN or +inf; idx, d: the slots' experts and gradients."""
    E = v.numel()
    out, size = torch.zeros(E, dtype=torch.float64), torch.zeros(E, dtype=torch.float64)
    there = [j for j, e in enumerate(idx.tolist()) if e >= 0]
    e, d = idx[there], d[there].double()
    if score == SIGMOID or normalize:   # slots share the sum of their scores, or have nothing to do with each other
        x = v[e]
        s, rest = torch.sigmoid(x), torch.sigmoid(-x)
        if normalize:
            r = torch.exp(torch.log_softmax(torch.nn.functional.logsigmoid(x) if score == SIGMOID else x, 0))
            each = r[None, :] * (d[:, None] - d[None, :])
        else:
            r, each = s, torch.diag(d)
        factor = scale * r * (rest if score == SIGMOID else 1.0)
        out.index_add_(0, e, factor * each.sum(1))
        size.index_add_(0, e, factor * each.abs().sum(1))
        return out, size
    p = torch.softmax(v, 0)
    of = torch.zeros(E, dtype=torch.float64).index_add_(0, e, d)   # what each expert's slots get together
    each = p[None, :] * (of[:, None] - of[None, :])
    return scale * p * each.sum(1), scale * p * each.abs().sum(1)


@gpu_only
@pytest.mark.parametrize("score,normalize", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True), (SIGMOID, False)])
@pytest.mark.parametrize("E,k", [(8, 2), (12, 12), (64, 6), (100, 20), (256, 32), (257, 6), (1000, 32)])
def test_gradient_of_a_dominant_expert(gpu, E, k, score, normalize):
    """One expert far ahead of the others: its own gradient is a small sum over the others, and is as exact as theirs."""
    g = torch.Generator().manual_seed(E + k)
    gaps = [0.0, 2.0, 4.0, 6.0, 8.0, 10.0, 12.0, 14.0, 16.0, 18.0]
    for repeated in (False, True):
        v = torch.randn(len(gaps), E, generator=g) - (9.0 if score == SIGMOID else 0.0)
        for t, gap in enumerate(gaps):
            v[t, 3] = v[t].max() + gap
        idx = torch.stack([torch.cat((torch.tensor([3]), torch.randperm(E, generator=g)[:k - 1])) for _ in gaps])
        first = torch.stack([(row[:, None] == row[None, :]).int().argmax(1) for row in idx])
        if not repeated:   # an empty slot where the dominant expert was drawn once more
            idx = torch.where(first == torch.arange(k), idx, -1)
        else:
            idx[:, 1:] = torch.where(torch.rand(len(gaps), k - 1, generator=g) < 0.3, idx[:, :1], idx[:, 1:])
        idx = torch.gather(idx, 1, torch.stack([torch.randperm(k, generator=g) for _ in gaps]))
        # gradients of an expert's slots are added before they are compared with others': of one sign, so that this loses nothing
        d = 1.0 + torch.rand(len(gaps), k, generator=g)
        ctx = gpu.Context(gpu.make_config(len(gaps), 8, E, 1, k))
        got = gpu.moe_route_backward(ctx, d.cuda(), v.cuda(), idx.cuda(), score, normalize=normalize, scale=2.5).double().cpu()
        for t in range(len(gaps)):
            ref, size = plain_gradient(v[t].double(), idx[t], d[t], score, normalize, 2.5)
            # an exponential of a difference x is off by |x| half steps for the difference and two steps of its own, twice in a
            # product of two shares; their sums by a half step a term; a difference of gradients, products and quotients by ten
            spread = float(v[t].max() - v[t].min())
            # sums of an expert's gradients are off by as many half steps as it has slots, whatever their difference to others' is
            if repeated and score == SOFTMAX and not normalize:
                p = torch.softmax(v[t].double(), 0)
                of = torch.zeros(E, dtype=torch.float64).index_add_(0, idx[t], d[t].double())
                size = size + 2.5 * p * ((p * of).sum() - p * of + (1 - p) * of)
            tol = (2 * spread + 2 * E + 4 * k + 20) * (STEP / 2) * size + 2.0 ** -110
            assert ((got[t] - ref).abs() <= tol).all(), (gaps[t], got[t], ref)
        assert gpu.moe_poll_error(ctx) == (gpu.MOE_OK, 0)
        ctx.close()


@gpu_only
def test_captured(gpu):
    """A captured routing with its gradient, replayed on new logits."""
    T, E, k = 70, 64, 6
    g = torch.Generator().manual_seed(9)
    ctx = gpu.Context(gpu.make_config(T, 8, E, 1, k))
    v, d = torch.zeros(T, E, device="cuda"), torch.randn(T, k, generator=g).cuda()
    idx, w, gl = torch.empty(T, k, dtype=torch.int64, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")

    def step():
        gpu.moe_route(ctx, v, topk_idx=idx, topk_weights=w)
        gpu.moe_route_backward(ctx, d, v, idx, grad_logits=gl)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        v.copy_(logits_of(g, T, E))
        graph.replay()
        got = idx.clone(), w.clone(), gl.clone()
        step()
        assert torch.equal(got[0], idx) and torch.equal(got[1], w) and torch.equal(got[2], gl)
    ctx.close()


# ---------------------------------------------------------------- settings
def test_settings_are_read_at_every_call():
    """Settings that are tensors of one element, changed in place between calls: each call takes what they hold."""
    import combine_moe_dispatch_layout_amd as moe
    scale, normalize, keep = torch.tensor(2.5), torch.tensor(True), torch.tensor(2)
    for factor, norm, groups in ((2.5, 1, 2), (5.0, 0, 3), (0.25, 1, 4)):
        scale.fill_(factor)
        normalize.fill_(norm)
        keep.fill_(groups)
        r = moe._binding._router(SIGMOID, 4, keep, 1, normalize, scale)._obj
        assert (r.score, r.groups, r.topk_groups, r.group_top, r.normalize, r.scale) == (SIGMOID, 4, groups, 1, norm, factor)
    rows, flag = torch.tensor(24), torch.tensor(True)
    first = moe.moe_linear_workspace(rows, 7168, 256), moe.moe_linear_backward_workspace(rows, 7168, 256, bias=flag)
    rows.fill_(48)
    flag.fill_(False)
    second = moe.moe_linear_workspace(rows, 7168, 256), moe.moe_linear_backward_workspace(rows, 7168, 256, bias=flag)
    assert first == (moe.moe_linear_workspace(24, 7168, 256), moe.moe_linear_backward_workspace(24, 7168, 256, bias=True))
    assert second == (moe.moe_linear_workspace(48, 7168, 256), moe.moe_linear_backward_workspace(48, 7168, 256))
    assert first[0] != second[0]


@gpu_only
def test_scale_changed_in_place(gpu):
    """The factor of the weights and of their gradient as a tensor that the program changes."""
    g = torch.Generator().manual_seed(11)
    ctx = gpu.Context(gpu.make_config(9, 8, 16, 1, 3))
    v, d, scale = logits_of(g, 9, 16).cuda(), torch.randn(9, 3, generator=g).cuda(), torch.tensor(1.0)
    for factor in (1.0, 2.0, 0.5):   # powers of two: weights and gradients are exact multiples
        scale.fill_(factor)
        idx, w = gpu.moe_route(ctx, v, scale=scale)
        assert torch.equal(w, factor * gpu.moe_route(ctx, v)[1])
        assert torch.equal(gpu.moe_route_backward(ctx, d, v, idx, scale=scale), factor * gpu.moe_route_backward(ctx, d, v, idx))
    ctx.close()


# ---------------------------------------------------------------- refusals
def test_null_arguments_rejected():
    import combine_moe_dispatch_layout_amd as moe
    lib = moe.load_library()
    r = moe._binding.moe_router(0, 1, 1, 1, 1, 1.0)
    assert lib.moe_route(None, None, 0, 8, 1, ctypes.byref(r), None, None, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_route_backward(None, None, None, 0, 8, None, 1, ctypes.byref(r), None, None) == moe.MOE_ERR_INVALID_ARG


def test_binding_rejects_cpu_tensors_without_a_gpu():
    import combine_moe_dispatch_layout_amd as moe

    class Ctx:
        cfg, device, handle = moe.make_config(4, 8, 16, 1, 2), 0, None
    with pytest.raises(TypeError, match="logits must be"):
        moe.moe_route(Ctx(), torch.zeros(4, 16))
    with pytest.raises(TypeError, match="logits must be"):
        moe.moe_route_backward(Ctx(), torch.zeros(4, 2), torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int64))


@gpu_only
def test_refusals(gpu):
    ctx = gpu.Context(gpu.make_config(4, 8, 16, 1, 2))
    v = torch.zeros(4, 16, device="cuda")
    idx, w, gl = torch.zeros(4, 2, dtype=torch.int64, device="cuda"), torch.zeros(4, 2, device="cuda"), torch.zeros(4, 16, device="cuda")
    for kwargs, status in [(dict(score=2), 1), (dict(score=-1), 1), (dict(groups=0), 1), (dict(groups=3), 2), (dict(groups=4, topk_groups=5), 1),
                           (dict(groups=4, topk_groups=0), 1), (dict(groups=4, group_top=3), 1), (dict(group_top=0), 1), (dict(scale=float("nan")), 1),
                           (dict(scale=INF), 1)]:
        with pytest.raises(gpu.MoeError) as e:
            gpu.moe_route(ctx, v, **kwargs)
        assert e.value.status == status, kwargs
    with pytest.raises(gpu.MoeError) as e:
        gpu.moe_route(ctx, torch.zeros(5, 16, device="cuda"))
    assert e.value.status == gpu.MOE_ERR_CAPACITY
    for bad in (v.half(), v.double()):
        with pytest.raises(TypeError):
            gpu.moe_route(ctx, bad)
    for bad in (torch.zeros(4, 15, device="cuda"), torch.zeros(16, 4, device="cuda").t(), v[0], v[:1].expand(4, 16)):
        with pytest.raises(ValueError):
            gpu.moe_route(ctx, bad)
    with pytest.raises(ValueError):
        gpu.moe_route(ctx, v, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError):
        gpu.moe_route(ctx, v, topk_idx=idx.int())
    lib, r = gpu.load_library(), gpu._binding.moe_router(0, 1, 1, 1, 1, 1.0)
    p, call = v.data_ptr(), lambda *a: lib.moe_route(ctx.handle, a[0], a[1], a[2], 4, ctypes.byref(r), None, a[3], a[4], None)
    bad = [(None, 0, 16, idx.data_ptr(), w.data_ptr()), (p, 2, 16, idx.data_ptr(), w.data_ptr()), (p, 0, 15, idx.data_ptr(), w.data_ptr()),
           (p + 2, 0, 16, idx.data_ptr(), w.data_ptr()), (p, 0, 16, None, w.data_ptr()), (p, 0, 16, idx.data_ptr() + 4, w.data_ptr()),
           (p, 0, 16, idx.data_ptr(), None), (p, 0, 16, p, w.data_ptr()), (p, 0, 16, idx.data_ptr(), p), (p, 0, 16, idx.data_ptr(), idx.data_ptr())]
    assert [call(*a) for a in bad] == [gpu.MOE_ERR_INVALID_ARG] * len(bad)
    back = lambda *a: lib.moe_route_backward(ctx.handle, a[0], p, 0, 16, a[1], 4, ctypes.byref(r), a[2], None)
    bad = [(None, idx.data_ptr(), gl.data_ptr()), (w.data_ptr(), None, gl.data_ptr()), (w.data_ptr(), idx.data_ptr(), None), (w.data_ptr(), idx.data_ptr(), p),
           (w.data_ptr(), idx.data_ptr(), idx.data_ptr())]
    assert [back(*a) for a in bad] == [gpu.MOE_ERR_INVALID_ARG] * len(bad)
    r.normalize = 2
    assert call(p, 0, 16, idx.data_ptr(), w.data_ptr()) == gpu.MOE_ERR_INVALID_ARG
    empty = gpu.moe_route(ctx, v[:0])
    assert empty[0].shape == (0, 2) and gpu.moe_route_backward(ctx, w[:0], v[:0], idx[:0]).shape == (0, 16)
    ctx.close()
    many = gpu.Context(gpu.make_config(2 ** 26, 8, 4, 1, 1))   # more tokens than a launch has lanes for
    r.normalize = 1
    assert lib.moe_route(many.handle, p, 0, 4, 2 ** 26, ctypes.byref(r), None, idx.data_ptr(), w.data_ptr(), None) == gpu.MOE_ERR_UNSUPPORTED
    assert lib.moe_route_backward(many.handle, w.data_ptr(), p, 0, 4, idx.data_ptr(), 2 ** 26, ctypes.byref(r), gl.data_ptr(),
                                  None) == gpu.MOE_ERR_UNSUPPORTED
    many.close()
