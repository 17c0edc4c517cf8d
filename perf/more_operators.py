"""Cases of the operators around the experts: what is timed, on which inputs, and
what the results have to be.

  layer      out[t] = residual[t] + sum_j w[t, j] W2[e] (silu(g) u), (g, u) = W1[e] x[t], e = idx[t, j]:
             the experts of a few tokens in one call, matrices in bf16 or as E4M3 codes with a scale for
             each 128 x 128 block
  linear     out = act(x W^T + bias) + residual: the router's logits, the shared expert
  linear_backward
             grad_pre = grad_out act'(pre); grad_x = grad_pre W, grad_W = grad_pre^T x, grad_bias = the
             rows of grad_pre summed
  route      the experts and weights of each token from its logits, and the logits' gradient

`own` selects the framework's kernels instead of the plain form.
"""
import math

import torch

own = False

BLOCK = 128          # channels that share a scale, and columns
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def _layer(name, T, k, E, H, I, fp8=False, skew=0.0, empty=0.0, residual=True):
    """T tokens of H channels with k slots each over E experts of I features; skew: Zipf exponent of the experts'
    popularity; empty: share of slots without an expert."""
    return dict(name=name, op="layer", T=T, k=k, E=E, H=H, I=I, fp8=fp8, skew=skew, empty=empty, residual=residual)


def _linear(name, op, T, K, N, act="none", bias=False, residual=False, fp32=False):
    """T rows, K to N features (swiglu: the matrix has 2N rows, gates first); fp32: the type of the output."""
    return dict(name=name, op=op, T=T, K=K, N=N, act=act, bias=bias, residual=residual, fp32=fp32)


def _route(name, T, E, k, score, bias=False, groups=1, keep=1, top=1, norm=True, scale=1.0, masked=0.0, bf16=False, train=False):
    """T tokens choose k of E experts; groups: of experts, `keep` of them stay, those with the largest sums of their
    `top` best scores; norm: weights sum to `scale`; masked: share of logits at -inf; train: the gradient as well."""
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, bias=bias, groups=groups, keep=keep, top=top, norm=norm,
                scale=scale, masked=masked, bf16=bf16, train=train)


def listed():
    return [
        # one token answers: its six experts' matrices are read once
        _layer("layer one token", 1, 6, 64, 4096, 2048),
        # a handful of tokens through small experts of an odd size, some slots empty: latency
        _layer("layer tiny", 16, 2, 8, 256, 264, empty=0.1),
        # one token through block-quantised experts
        _layer("layer fp8 one token", 1, 8, 256, 7168, 2048, fp8=True),
        # the decode workload: nearly every expert's matrices are read, for a few rows each
        _layer("layer fp8 decode", 128, 8, 256, 7168, 2048, fp8=True),
        # the prefill workload's router: few columns, a long contraction, logits in fp32
        _linear("linear router", "linear", 4096, 7168, 256, fp32=True),
        # the shared expert's gate and up product with the activation, prefill
        _linear("linear gate-up", "linear", 4096, 7168, 2048, act="swiglu"),
        # the shared expert's down product for one token, added to what the routed experts gave
        _linear("linear one token", "linear", 1, 2048, 7168, residual=True),
        # odd sizes throughout, everything in the epilogue
        _linear("linear odd sizes", "linear", 333, 1000, 2056, act="gelu_tanh", bias=True, residual=True),
        # a training step's backward of a shared expert's layer over the skewed workload's tokens
        _linear("linear backward", "linear_backward", 8192, 4096, 4096, act="gelu", bias=True),
        # the backward of a small batch through a gated layer
        _linear("linear backward small", "linear_backward", 77, 256, 264, act="swiglu", bias=True),
        # the group-limited workload's routing
        _route("route grouped", 4096, 256, 8, "sigmoid", bias=True, groups=8, keep=4, top=2, scale=2.5),
        # a training step's routing and its gradient, as the skewed workload has it
        _route("route training", 8192, 64, 6, "softmax", train=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")


def draw(rng):
    while True:
        op = rng.choice(("layer", "layer", "layer", "linear", "linear", "linear", "linear_backward", "linear_backward", "route", "route"))
        if op == "layer":
            fp8 = rng.random() < 0.5
            E = _log_uniform(rng, 1, 256)
            k = rng.randint(1, min(8, E))
            T = _log_uniform(rng, 1, 128)
            H, I = (128 * _log_uniform(rng, 1, 56), 128 * _log_uniform(rng, 1, 32)) if fp8 else (8 * _log_uniform(rng, 8, 896), 8 * _log_uniform(rng, 8, 512))
            c = _layer("", T, k, E, H, I, fp8, rng.choice((0.0, 0.0, 1.2)), rng.choice((0.0, 0.0, 0.1)), rng.random() < 0.5)
            if E * H * I > 1.6e9:
                continue   # matrices of about ten GB at most
        elif op == "route":
            groups = rng.choice((1, 1, 2, 4, 8))
            E = groups * _log_uniform(rng, 2, 512 // groups)
            keep = rng.randint(1, groups)
            c = _route("", _log_uniform(rng, 1, 16384), E, rng.randint(1, min(8, keep * E // groups)), rng.choice(("softmax", "sigmoid")),
                       rng.random() < 0.5, groups, keep, rng.choice((1, 2)), rng.random() < 0.7, rng.choice((1.0, 2.5)),
                       rng.choice((0.0, 0.0, 0.3)), rng.random() < 0.3, rng.random() < 0.5)
        else:
            T, K, N = _log_uniform(rng, 1, 8192), 8 * _log_uniform(rng, 8, 896), 8 * _log_uniform(rng, 4, 896)
            act = rng.choice(ACTS)
            forward = op == "linear"
            c = _linear("", op, T, K, N, act, rng.random() < 0.5, forward and rng.random() < 0.5, forward and rng.random() < 0.3)
            if T * K * N * (2 if act == "swiglu" else 1) > 1.3e11:
                continue   # no more work than the largest listed case
        del c["name"]
        return c


def _active(c):
    """Experts expected to have rows, for a routing without skew."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])


def work(c):
    """Each input read once, each output written once; of the experts' matrices those of experts with rows."""
    T = c["T"]
    if c["op"] == "layer":
        pairs, values = T * c["k"] * (1 - c["empty"]), _active(c) * 3 * c["H"] * c["I"]
        size = 1 + 4 / BLOCK ** 2 if c["fp8"] else 2
        return {"bytes": values * size + T * (2 * c["H"] * (3 if c["residual"] else 2) + 12 * c["k"]), "flops": 6 * pairs * c["H"] * c["I"]}
    if c["op"] == "route":
        logits = T * c["E"] * (2 if c["bf16"] else 4)
        grad = logits + 12 * T * c["k"] + 4 * T * c["E"] if c["train"] else 0
        return {"bytes": logits + 12 * T * c["k"] + grad, "flops": T * c["E"] * (20 if c["train"] else 10)}
    K, N = c["K"], c["N"]
    M = 2 * N if c["act"] == "swiglu" else N
    if c["op"] == "linear":
        return {"bytes": 2 * (T * K + M * K + (M if c["bias"] else 0) + (T * N if c["residual"] else 0)) + T * N * (4 if c["fp32"] else 2),
                "flops": 2 * T * K * M}
    pre = 2 * T * M if c["act"] != "none" else 0
    return {"bytes": 2 * (T * N + 2 * T * K + 2 * M * K) + pre + (4 * M if c["bias"] else 0), "flops": 4 * T * K * M}


# ---------------------------------------------------------------- inputs
def _normal(g, dev, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device=dev, dtype=dtype).mul_(scale)


def _prepare_layer(c, g, dev, s):
    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    popularity = -c["skew"] * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    u = torch.rand(T, E, generator=g, device=dev).clamp_(1e-30, 1 - 1e-7)
    idx = (popularity - torch.log(-torch.log(u))).topk(k, dim=1).indices
    idx[torch.rand(T, k, generator=g, device=dev) < c["empty"]] = -1
    w = torch.rand(T, k, generator=g, device=dev) + 0.05
    s |= {"x": _normal(g, dev, (T, H), torch.bfloat16), "idx": idx, "w": w / w.sum(1, keepdim=True)}
    s["residual"] = _normal(g, dev, (T, H), torch.bfloat16) if c["residual"] else None
    for name, rows, cols in (("w1", 2 * I, H), ("w2", H, I)):
        if c["fp8"]:
            # codes spread over the format's range and a scale for each block, as a block-quantised matrix has them
            m = torch.empty((E, rows, cols), device=dev, dtype=torch.uint8)
            for e in range(0, E, 16):
                v = _normal(g, dev, (min(16, E - e), rows, cols), torch.bfloat16, E4M3_MAX / 4).clamp_(-E4M3_MAX, E4M3_MAX)
                m[e:e + 16] = v.to(torch.float8_e4m3fn).view(torch.uint8)
            scales = torch.rand((E, rows // BLOCK, cols // BLOCK), generator=g, device=dev)
            s[name + "_scales"] = scales.add_(0.5).mul_(4 / E4M3_MAX * cols ** -0.5)
        else:
            m = torch.empty((E, rows, cols), device=dev, dtype=torch.bfloat16)
            for e in range(0, E, 16):
                m[e:e + 16] = _normal(g, dev, (min(16, E - e), rows, cols), torch.bfloat16, cols ** -0.5)
        s[name] = m
    # the plain form's plan: the experts with rows, and their rows in a table padded to the longest segment
    flat = idx.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.cumsum(counts, 0) - counts
    pair = torch.sort(torch.where(flat >= 0, flat, E), stable=True).indices[:int(counts.sum())]
    expert = flat[pair]
    active = torch.nonzero(counts).flatten()
    slot = torch.zeros(E, device=dev, dtype=torch.long)
    slot[active] = torch.arange(active.numel(), device=dev)
    longest = max(int(counts.max()), 1)
    cell = slot[expert] * longest + torch.arange(pair.numel(), device=dev) - offsets[expert]
    s |= {"pair": pair, "active": active, "longest": longest, "cell": cell}


def _prepare_linear(c, g, dev, s):
    T, K, N = c["T"], c["K"], c["N"]
    M = 2 * N if c["act"] == "swiglu" else N
    s["x"] = _normal(g, dev, (T, K), torch.bfloat16)
    s["weights"] = _normal(g, dev, (M, K), torch.bfloat16, K ** -0.5)
    if c["op"] == "linear":
        s["bias"] = _normal(g, dev, (M,), torch.bfloat16) if c["bias"] else None
        s["residual"] = _normal(g, dev, (T, N), torch.bfloat16) if c["residual"] else None
    else:
        s["grad_out"] = _normal(g, dev, (T, N), torch.bfloat16)
        # what the forward pass kept
        s["pre"] = _normal(g, dev, (T, M), torch.bfloat16) if c["act"] != "none" else None


def _prepare_route(c, g, dev, s):
    T, E = c["T"], c["E"]
    v = _normal(g, dev, (T, E), torch.float32, 1.5)
    v[torch.rand(T, E, generator=g, device=dev) < c["masked"]] = -math.inf
    s["logits"] = v.bfloat16() if c["bf16"] else v
    s["bias"] = _normal(g, dev, (E,), torch.float32, 0.1) if c["bias"] else None
    if c["train"]:
        s["grad"] = _normal(g, dev, (T, c["k"]), torch.float32)


def prepare(c, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": c}
    {"layer": _prepare_layer, "route": _prepare_route}.get(c["op"], _prepare_linear)(c, g, dev, s)
    if own:
        # the context that a user's program makes once
        import combine_moe_dispatch_layout_amd as moe
        s |= {"moe": moe, "ctx": moe.Context(moe.make_config(c["T"], c.get("H", 8), c.get("E", 1), 1, c.get("k", 1)))}
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    moe, ctx, c = s["moe"], s["ctx"], s["case"]
    if c["op"] == "layer":
        if c["fp8"]:
            return moe.moe_layer_fp8(ctx, s["x"], s["idx"], s["w"], s["w1"], s["w1_scales"], s["w2"], s["w2_scales"], residual=s["residual"])
        return moe.moe_layer(ctx, s["x"], s["idx"], s["w"], s["w1"], s["w2"], residual=s["residual"])
    if c["op"] == "route":
        score = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}[c["score"]]
        idx, w = moe.moe_route(ctx, s["logits"], score, bias=s["bias"], groups=c["groups"], topk_groups=c["keep"], group_top=c["top"],
                               normalize=c["norm"], scale=c["scale"])
        if not c["train"]:
            return idx, w
        return idx, w, moe.moe_route_backward(ctx, s["grad"], s["logits"], idx, score, normalize=c["norm"], scale=c["scale"])
    act = getattr(moe, "MOE_ACT_" + c["act"].upper())
    if c["op"] == "linear":
        return moe.moe_linear(ctx, s["x"], s["weights"], bias=s["bias"], act=act, residual=s["residual"],
                              out_dtype=torch.float32 if c["fp32"] else torch.bfloat16)
    gx, gw, gb = moe.moe_linear_backward(ctx, s["grad_out"], s["x"], s["weights"], act=act, pre=s["pre"], bias=c["bias"])
    return (gx, gw, gb) if c["bias"] else (gx, gw)


def _table(s, rows):
    """fp32 rows of the valid pairs as [active experts, longest segment, width], zero where a segment has ended."""
    t = torch.zeros((s["active"].numel() * s["longest"], rows.shape[1]), device=rows.device)
    t[s["cell"]] = rows
    return t.unflatten(0, (s["active"].numel(), s["longest"]))


def _matrices(s, name):
    """The matrices of the experts with rows, in fp32."""
    w = s[name][s["active"]]
    if not s["case"]["fp8"]:
        return w.float()
    w = w.view(torch.float8_e4m3fn).float()
    b = w.view(w.shape[0], w.shape[1] // BLOCK, BLOCK, w.shape[2] // BLOCK, BLOCK)
    b *= s[name + "_scales"][s["active"]][:, :, None, :, None]
    return w


def _plain_layer(s):
    c = s["case"]
    T, k, H = c["T"], c["k"], c["H"]
    gate_up = torch.bmm(_table(s, s["x"].float()[s["pair"] // k]), _matrices(s, "w1").transpose(1, 2))
    gate, up = gate_up.chunk(2, dim=2)
    y = torch.bmm(gate / (1 + torch.exp(-gate)) * up, _matrices(s, "w2").transpose(1, 2))
    terms = torch.zeros((T * k, H), device=y.device)
    terms[s["pair"]] = y.flatten(0, 1)[s["cell"]] * s["w"].reshape(-1)[s["pair"]].unsqueeze(1)
    out = terms.view(T, k, H).sum(1)
    return (out if s["residual"] is None else out + s["residual"].float()).bfloat16()


def _activated(act, v):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "swiglu":
        g, u = v.chunk(2, dim=1)
        return g / (1 + torch.exp(-g)) * u
    return v


def _slope(act, v, d):
    """d times the activation's derivative at v."""
    if act == "relu":
        return d * (v > 0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return d * (s * (1 + v * (1 - s)))
    if act == "gelu":
        return d * (0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi)))
    if act == "gelu_tanh":
        r = math.sqrt(2 / math.pi)
        t = torch.tanh(r * (v + 0.044715 * v ** 3))
        return d * (0.5 * (1 + t) + 0.5 * v * (1 - t * t) * r * (1 + 3 * 0.044715 * v * v))
    if act == "swiglu":
        g, u = v.chunk(2, dim=1)
        s = 1 / (1 + torch.exp(-g))
        return torch.cat((d * u * (s * (1 + g * (1 - s))), d * g * s), 1)
    return d


def _plain_linear(s):
    c = s["case"]
    v = torch.mm(s["x"].float(), s["weights"].float().t())
    if s["bias"] is not None:
        v += s["bias"].float()
    v = _activated(c["act"], v)
    if s["residual"] is not None:
        v += s["residual"].float()
    return v if c["fp32"] else v.bfloat16()


def _plain_linear_backward(s):
    c = s["case"]
    d = s["grad_out"].float()
    if s["pre"] is not None:
        d = _slope(c["act"], s["pre"].float(), d)
    grads = torch.mm(d, s["weights"].float()).bfloat16(), torch.mm(d.t(), s["x"].float()).bfloat16()
    return grads + (d.sum(0),) if c["bias"] else grads


def _scores(s):
    """In 64 bits: what is chosen may lie next to what is not."""
    v = s["logits"].double()
    if s["case"]["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    e = torch.exp(v - v.amax(1, keepdim=True).clamp(min=-1e300))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _weights(c, s, chosen):
    """Weights of the chosen experts' scores, in 64 bits; 0 where none is."""
    total = chosen.sum(1, keepdim=True)
    return chosen * c["scale"] / torch.where(total > 0, total, 1) if c["norm"] else chosen * c["scale"]


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    free = s["logits"] > -math.inf
    score = _scores(s)
    key = score if s["bias"] is None else score + s["bias"].double()
    if s["bias"] is None and G == 1:
        key = s["logits"].double()   # grows with the score, and never ties where the logits do not
    key = torch.where(free, key, -math.inf)
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["top"]]
        sums = torch.where(best > -math.inf, best, 0).sum(2)
        sums = torch.where(best[:, :, 0] > -math.inf, sums, -math.inf)
        rank = sums.sort(dim=1, descending=True, stable=True).indices.argsort(1)
        key = torch.where((rank < c["keep"]).repeat_interleave(E // G, 1), key, -math.inf)
    top = key.sort(dim=1, descending=True, stable=True)
    idx = torch.where(top.values[:, :k] > -math.inf, top.indices[:, :k], -1)
    there = idx >= 0
    at = idx.clamp(min=0)
    chosen = torch.where(there, score.gather(1, at), 0)
    w = _weights(c, s, chosen)
    if not c["train"]:
        return idx, w.float()
    d = torch.where(there, s["grad"].double(), 0) * c["scale"]
    if c["norm"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1)
        d = (d - (d * (chosen / total)).sum(1, keepdim=True)) / total   # of one expert alone nothing is left
    ds = torch.zeros_like(score).scatter_add_(1, at, torch.where(there, d, 0))
    if c["score"] == "sigmoid":
        grad = ds * score * (1 - score)
    else:
        grad = score * (ds - (ds * score).sum(1, keepdim=True))
    return idx, w.float(), torch.where(free, grad, 0).float()


def _run_plain(s):
    return {"layer": _plain_layer, "linear": _plain_linear, "linear_backward": _plain_linear_backward, "route": _plain_route}[s["case"]["op"]](s)


# ---------------------------------------------------------------- in 64 bits
def _matrix64(s, name, e):
    if not s["case"]["fp8"]:
        return s[name][e].double()
    m = s[name][e].view(torch.float8_e4m3fn).double()
    return m * torch.kron(s[name + "_scales"][e].double(), torch.ones(BLOCK, BLOCK, device=m.device, dtype=torch.float64))


def _exact_layer(c, s):
    out = torch.zeros((c["T"], c["H"]), device=s["x"].device, dtype=torch.float64)
    if s["residual"] is not None:
        out += s["residual"].double()
    for e in s["active"].tolist():
        token, slot = torch.nonzero(s["idx"] == e, as_tuple=True)
        v = torch.mm(s["x"][token].double(), _matrix64(s, "w1", e).t())
        h = torch.nn.functional.silu(v[:, :c["I"]]) * v[:, c["I"]:]
        out.index_add_(0, token, torch.mm(h, _matrix64(s, "w2", e).t()) * s["w"][token, slot].double().unsqueeze(1))
    return out


def _exact_act(act, v):
    f = torch.nn.functional
    if act == "swiglu":
        return f.silu(v[:, :v.shape[1] // 2]) * v[:, v.shape[1] // 2:]
    return {"none": lambda t: t, "relu": f.relu, "silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act](v)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "layer":
        return _exact_layer(c, s)
    if c["op"] == "linear":
        v = torch.mm(s["x"].double(), s["weights"].double().t())
        v = _exact_act(c["act"], v if s["bias"] is None else v + s["bias"].double())
        return v if s["residual"] is None else v + s["residual"].double()
    if c["op"] == "linear_backward":
        d = s["grad_out"].double()
        if s["pre"] is not None:
            with torch.enable_grad():
                pre = s["pre"].double().requires_grad_()
                d = torch.autograd.grad(_exact_act(c["act"], pre), pre, d)[0]
        grads = torch.mm(d, s["weights"].double()), torch.mm(d.t(), s["x"].double())
        return grads + (d.sum(0),) if c["bias"] else grads
    # route: the chosen experts are whole numbers; what follows from them is taken on the experts that the definition chooses
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    with torch.enable_grad():
        v = s["logits"].double().requires_grad_()
        masked = torch.isneginf(v)
        p = torch.sigmoid(v) if c["score"] == "sigmoid" else torch.softmax(torch.where(masked.all(1, keepdim=True), 0.0, v), 1)
        order = p.detach() if s["bias"] is None else p.detach() + s["bias"].double()
        order = torch.where(masked, -math.inf, order)
        if G > 1:
            grouped = order.view(T, G, -1).topk(min(c["top"], E // G), 2).values
            some = grouped.amax(2) > -math.inf
            value = torch.where(some, torch.where(grouped > -math.inf, grouped, 0.0).sum(2), -math.inf)
            keep = torch.zeros(T, G, device=v.device, dtype=torch.bool).scatter_(1, value.topk(c["keep"], 1).indices, True)
            order = torch.where(keep.repeat_interleave(E // G, 1), order, -math.inf)
        best = order.topk(k, 1)
        there = best.values > -math.inf
        if c["norm"]:   # shares of a sum are a softmax of the logarithms
            log = v if c["score"] == "softmax" else -torch.nn.functional.softplus(-v)
            log = torch.where(there, log.gather(1, best.indices), -math.inf)
            w = torch.where(there, torch.softmax(torch.where(there.any(1, keepdim=True), log, 0.0), 1), 0.0) * c["scale"]
        else:
            w = torch.where(there, p.gather(1, best.indices), 0.0) * c["scale"]
        if not c["train"]:
            return None, w.detach()
        if c["bf16"]:
            return None, w.detach(), None   # bf16 logits tie: another choice among equals has its gradient elsewhere
        grad = torch.autograd.grad(w, v, s["grad"].double())[0]
        return None, w.detach(), torch.where(masked, 0.0, grad)
