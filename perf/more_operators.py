"""What the operators around the mixture-of-experts layer are measured on.

Three operators with their gradients make a block of the layer:

  select   routing from the router's logits: softmax or sigmoid scores, a bias that counts for
           the choice only, groups of experts, top-K, renormalised and scaled gates
  norm     the norms before and after a block fused with its gate and the scaled residual
  linear   product of bf16 rows with a weight kept in 8 bits, a power-of-two scale for each
           block of 128

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits (the choice
of experts in 64); with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
SOFTMAX, SIGMOID = "softmax", "sigmoid"


# ---- cases -------------------------------------------------------------------------------

def listed():
    return [
        # One decode batch of the 768-expert layer, some rows of it padding: latency.
        dict(name="select_T65_E768_padded", op="select", T=65, E=768, K=12, score=SOFTMAX, groups=1, top=1, rank=1,
             renorm=True, scale=1.0, bias=True, pad=0.1),
        # A prompt through the 768-expert layer, experts on 8 devices of which a token uses 4.
        dict(name="select_T16384_E768_groups", op="select", T=16384, E=768, K=12, score=SIGMOID, groups=8, top=4, rank=2,
             renorm=True, scale=2.5, bias=True, pad=0.0),
        # A small layer of odd sizes, the gradient of a loss on the logits beside it.
        dict(name="select_bw_T1777_E77", op="select_bw", T=1777, E=77, K=5, score=SOFTMAX, renorm=False, scale=1.0,
             aux=True, pad=0.0),
        # A training step of the 768-expert layer: the dense gradient of sparse picks.
        dict(name="select_bw_T16384_E768", op="select_bw", T=16384, E=768, K=12, score=SIGMOID, renorm=True, scale=2.5,
             aux=True, pad=0.1),
        # One decode batch: norm after the block, gate, residual, norm before the next: latency.
        dict(name="norm_T64_d6144", op="norm", T=64, d=6144, dtype=BF16, post=True, gate="channel"),
        # A prompt: memory traffic.
        dict(name="norm_T16384_d6144", op="norm", T=16384, d=6144, dtype=BF16, post=True, gate="channel"),
        # An fp32 layer of odd sizes, a gate for each token (a gated dense branch).
        dict(name="norm_bw_f32_T333_d1028", op="norm_bw", T=333, d=1028, dtype=F32, post=True, gate="token"),
        # A training step: six arrays of tokens and three sums over them.
        dict(name="norm_bw_T16384_d6144", op="norm_bw", T=16384, d=6144, dtype=BF16, post=True, gate="channel"),
        # One decode batch through a dense branch of the layer: the weight's bytes count.
        dict(name="linear_T64_d6144_n6144", op="linear", T=64, k=6144, n=6144),
        # A prompt through the same: the FP8 matrix cores.
        dict(name="linear_T16384_d6144_n6144", op="linear", T=16384, k=6144, n=6144),
        # A fine-tuning step of odd sizes.
        dict(name="linear_bw_T777_k1032_n520", op="linear_bw", T=777, k=1032, n=520),
        # A training step: both gradients, the tokens and dy quantised along both axes.
        dict(name="linear_bw_T16384_d6144_n2048", op="linear_bw", T=16384, k=6144, n=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("select", "select_bw", "norm", "norm_bw", "linear", "linear_bw"))
    T = _log(rng, 1, 16384)
    if op in ("select", "select_bw"):
        groups = rng.choice((1, 1, 2, 4, 8, 16))
        size = _log(rng, 4 if groups > 1 else 12, 768 // groups)
        top = rng.randint(1, groups)
        K = rng.randint(1, min(12, top * size))
        case = dict(op=op, T=T, E=groups * size, K=K, score=rng.choice((SOFTMAX, SIGMOID)), renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5)), pad=rng.choice((0.0, 0.3)))
        if op == "select":
            return dict(case, groups=groups, top=top, rank=rng.choice((1, 2)), bias=rng.random() < 0.7)
        return dict(case, aux=rng.random() < 0.5)
    if op in ("norm", "norm_bw"):
        dtype = rng.choice((BF16, BF16, F32))
        d = 8 * _log(rng, 4, 768) if dtype == BF16 else 4 * _log(rng, 8, 700)
        return dict(op=op, T=T, d=d, dtype=dtype, post=rng.random() < 0.6,
                    gate=rng.choice((None, "channel", "token")))
    k, n = 8 * _log(rng, 8, 768), 8 * _log(rng, 8, 768)
    if op == "linear_bw":
        n = min(n, 2048)
    return dict(op=op, T=T, k=k, n=n)


# ---- inputs ------------------------------------------------------------------------------

EPS = 2.0 ** -20
SHARE, BRANCH = 0.875, 0.5  # scales of the residual stream and of the block


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _tokens(g, T, d):
    """Rows of different sizes, as a residual stream has them."""
    return _randn(g, T, d) * torch.exp(0.5 * _randn(g, T, 1))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op, T = case["op"], case["T"]
    if op in ("select", "select_bw"):
        E = case["E"]
        s["logits"] = _randn(g, T, E)
        s["mask"] = (torch.rand(T, generator=g, device=DEV) >= case["pad"]).to(torch.uint8) if case["pad"] else None
        spread = 0.1 / E if case["score"] == SOFTMAX else 0.05
        s["bias"] = spread * (2 * torch.rand(E, generator=g, device=DEV) - 1)
        if op == "select":
            if not case["bias"]:
                s["bias"] = None
        else:  # picks of another router state; a padded token has none
            s["idx"] = torch.topk(s["logits"] + 0.3 * _randn(g, E), case["K"], dim=1).indices.to(torch.int32)
            if s["mask"] is not None:
                s["idx"][s["mask"] == 0] = -1
            s["dgate"] = _randn(g, T, case["K"])
            s["aux"] = 1e-3 * _randn(g, T, E) if case["aux"] else None
        if own:  # the router's settings, made once
            import mixture_experts_layer_router_amd as lm
            s["gating"] = lm.Gating(case["score"], case.get("groups", 1), case.get("top", 1), case.get("rank", 1),
                                    case["renorm"], case["scale"])
        return s
    if op in ("norm", "norm_bw"):
        d, dt = case["d"], DTYPES[case["dtype"]]
        s["y"] = _tokens(g, T, d).to(dt)
        s["w_pre"] = 1 + 0.1 * _randn(g, d)
        s["w_post"] = 1 + 0.1 * _randn(g, d) if case["post"] else None
        s["gate"] = {None: None, "channel": lambda: 0.5 + 0.2 * _randn(g, d),
                     "token": lambda: torch.rand((T, 1), generator=g, device=DEV)}[case["gate"]]
        s["gate"] = s["gate"] and s["gate"]()
        if op == "norm":
            s["x"] = _tokens(g, T, d).to(dt)
        else:
            s["h"] = _tokens(g, T, d).to(dt)
            s["dh"] = (1e-2 * _randn(g, T, d)).to(dt)
            s["dz"] = (1e-2 * _randn(g, T, d)).to(dt)
        return s
    k, n = case["k"], case["n"]
    s["x"] = _tokens(g, T, k).to(torch.bfloat16)
    s["w"] = (_randn(g, n, k) / math.sqrt(k)).to(torch.bfloat16)
    if op == "linear_bw":
        s["dy"] = (1e-2 * _tokens(g, T, n)).to(torch.bfloat16)
    if own:  # the weight in 8 bits, made when it is loaded
        import mixture_experts_layer_router_amd as lm
        s["wq"] = lm.quantize_matrix(s["w"], transposed=op == "linear_bw")
    else:
        s["wq"] = _block_values(s["w"])
    return s


# ---- one pass ----------------------------------------------------------------------------

def run(s):
    return {"select": _select, "select_bw": _select_bw, "norm": _norm, "norm_bw": _norm_bw, "linear": _linear,
            "linear_bw": _linear_bw}[s["case"]["op"]](s)


def _scores(logits, score):
    """Scores in 64 bits: picks next to a border depend on every digit."""
    lg = logits.double()
    if score == SIGMOID:
        return 1 / (1 + torch.exp(-lg))
    ex = torch.exp(lg - lg.amax(1, keepdim=True))
    return ex / ex.sum(1, keepdim=True)


def _select(s):
    case = s["case"]
    if own:
        import mixture_experts_layer_router_amd as lm
        idx, gate = lm.select(s["logits"], s["bias"], case["K"], s["gating"], token_mask=s["mask"])
        return dict(idx=idx, gate=gate)
    T, E, K, G = case["T"], case["E"], case["K"], case["groups"]
    p = _scores(s["logits"], case["score"])
    c = p if s["bias"] is None else p + s["bias"].double()
    if case["top"] < G:
        best = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values[:, :, :case["rank"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["top"]]
        live = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        c = torch.where(live.repeat_interleave(E // G, 1), c, -math.inf)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :K]
    gate = p.gather(1, idx).float()
    if case["renorm"]:
        gate = gate / gate.sum(1, keepdim=True)
    gate = gate * case["scale"]
    idx = idx.to(torch.int32)
    if s["mask"] is not None:
        pad = (s["mask"] == 0)[:, None]
        idx, gate = torch.where(pad, -1, idx), torch.where(pad, 0.0, gate)
    return dict(idx=idx, gate=gate)


def _select_bw(s):
    case = s["case"]
    if own:
        import mixture_experts_layer_router_amd as lm
        return lm.select_backward(s["logits"], s["idx"], s["dgate"], s["gating"], dlogits_aux=s["aux"])
    lg, dg, scale = s["logits"], s["dgate"], case["scale"]
    ok = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    dg = torch.where(ok, dg, 0.0)
    if case["score"] == SIGMOID:
        p = 1 / (1 + torch.exp(-lg))
    else:
        ex = torch.exp(lg - lg.amax(1, keepdim=True))
        p = ex / ex.sum(1, keepdim=True)
    pk = torch.where(ok, p.gather(1, at), 0.0)
    if case["renorm"]:
        tot = pk.sum(1, keepdim=True).clamp(min=2.0 ** -126)
        dpk = scale / tot * (dg - (dg * pk).sum(1, keepdim=True) / tot)
    else:
        dpk = scale * dg
    dp = torch.zeros_like(p).scatter_add_(1, at, torch.where(ok, dpk, 0.0))
    if case["score"] == SIGMOID:
        dl = dp * p * (1 - p)
    else:
        dl = p * (dp - (p * dp).sum(1, keepdim=True))
    return dl if s["aux"] is None else dl + s["aux"]


def _norm(s):
    if own:
        import mixture_experts_layer_router_amd as lm
        h, z = lm.block_norm(s["x"], s["w_pre"], y=s["y"], w_post=s["w_post"], gate=s["gate"], residual_scale=SHARE,
                             block_scale=BRANCH, eps=EPS)
        return dict(h=h, z=z)
    u = s["y"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt(u.square().mean(1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        u = u * s["gate"]
    h = SHARE * s["x"].float() + BRANCH * u
    z = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w_pre"]
    return dict(h=h.to(s["x"].dtype), z=z.to(s["x"].dtype))


def _norm_bw(s):
    case = s["case"]
    if own:
        import mixture_experts_layer_router_amd as lm
        return lm.block_norm_backward(s["h"], s["w_pre"], s["dz"], dh=s["dh"], y=s["y"], w_post=s["w_post"],
                                      gate=s["gate"], residual_scale=SHARE, block_scale=BRANCH, eps=EPS)
    dt = s["h"].dtype
    h, y, dz = s["h"].float(), s["y"].float(), s["dz"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    hn, v = h * r, dz * s["w_pre"]
    out = dict(dw_pre=(dz * hn).sum(0))
    dt_h = s["dh"].float() + r * (v - hn * (v * hn).mean(1, keepdim=True))
    out["dx"] = (SHARE * dt_h).to(dt)
    du = BRANCH * dt_h if s["gate"] is None else BRANCH * s["gate"] * dt_h
    u = yn = y
    if case["post"]:
        q = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
        yn = y * q
        u = yn * s["w_post"]
        out["dw_post"] = (du * yn).sum(0)
    if s["gate"] is not None:
        out["dgate"] = (BRANCH * u * dt_h).sum(0) if case["gate"] == "channel" else (BRANCH * u * dt_h).sum(1, keepdim=True)
    if case["post"]:
        t = du * s["w_post"]
        du = q * (t - yn * (t * yn).mean(1, keepdim=True))
    out["dy"] = du.to(dt)
    return out


def _quantised(v, dims):
    """v [R, C] (fp32) in blocks of dims, every value rounded to E4M3 over its block's power of two."""
    R, C = v.shape
    a, b = dims
    p = torch.nn.functional.pad(v, (0, -C % b, 0, -R % a))
    p = p.view(p.shape[0] // a, a, p.shape[1] // b, b)
    frac, e = torch.frexp(p.abs().amax((1, 3), keepdim=True))
    k = torch.where(frac <= 0.875, e - 9, e - 8)  # the smallest k with amax <= 448 * 2^k
    k = torch.where(frac == 0, torch.zeros_like(k), k)
    q = torch.ldexp(torch.ldexp(p, -k).to(torch.float8_e4m3fn).float(), k)
    return q.reshape(q.shape[0] * a, -1)[:R, :C]


def _block_values(w):
    return _quantised(w.float(), (128, 128))


def _linear(s):
    if own:
        import mixture_experts_layer_router_amd as lm
        return lm.linear_fp8(s["x"], s["wq"])
    return (_quantised(s["x"].float(), (1, 128)) @ s["wq"].t()).to(torch.bfloat16)


def _linear_bw(s):
    if own:
        import mixture_experts_layer_router_amd as lm
        return lm.linear_fp8_backward(s["dy"], s["x"], s["wq"])
    x, dy = s["x"].float(), s["dy"].float()
    dx = _quantised(dy, (1, 128)) @ s["wq"]
    dw = _quantised(dy, (128, 1)).t() @ _quantised(x, (128, 1))
    return dict(dx=dx.to(torch.bfloat16), dw=dw.to(torch.bfloat16))


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "select":
        return {"bytes": 4 * T * case["E"] + 8 * T * case["K"] + 4 * case["E"] * case["bias"], "flops": 8 * T * case["E"]}
    if op == "select_bw":
        E, K = case["E"], case["K"]
        whole = case["score"] == SOFTMAX and not case["renorm"]  # only then every logit counts
        return {"bytes": T * (4 * E * (1 + case["aux"] + whole) + 8 * K + (0 if whole else 4 * K)), "flops": 6 * T * E}
    if op in ("norm", "norm_bw"):
        es, d = (2 if case["dtype"] == BF16 else 4), case["d"]
        vec = 1 + case["post"] + (case["gate"] == "channel")
        if op == "norm":
            return {"bytes": 4 * T * d * es + 4 * d * vec, "flops": 12 * T * d}
        return {"bytes": 6 * T * d * es + 8 * d * vec, "flops": 24 * T * d}
    k, n = case["k"], case["n"]
    if op == "linear":
        return {"bytes": 2 * T * k + n * k + 2 * T * n, "flops": 2 * T * k * n}
    return {"bytes": 4 * T * k + 2 * T * n + 3 * n * k, "flops": 4 * T * k * n}


# ---- the definition in 64 bits -------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"select": _exact_select, "select_bw": _exact_select_bw, "norm": _exact_norm, "norm_bw": _exact_norm_bw,
            "linear": _exact_linear, "linear_bw": _exact_linear_bw}[case["op"]](s, case)


def _exact_scores(s, case):
    lg = s["logits"].double()
    return torch.sigmoid(lg) if case["score"] == SIGMOID else torch.softmax(lg, 1)


def _exact_select(s, case):
    p = _exact_scores(s, case)
    T, E = p.shape
    c = p.clone()
    if s["bias"] is not None:
        c += s["bias"].double()
    G, size = case["groups"], E // case["groups"]
    left = c.clone().view(T, G, size)
    score = torch.zeros(T, G, dtype=torch.float64, device=DEV)
    for _ in range(case["rank"]):  # take a group's largest away, one after another
        top, at = left.max(2, keepdim=True)
        score += top[..., 0]
        left.scatter_(2, at, -math.inf)
    allowed = torch.zeros(T, G, dtype=torch.bool, device=DEV)
    for _ in range(case["top"]):
        at = score.argmax(1, keepdim=True)
        allowed.scatter_(1, at, True)
        score.scatter_(1, at, -math.inf)
    c[~allowed[:, :, None].expand(T, G, size).reshape(T, E)] = -math.inf
    gate = torch.empty(T, case["K"], dtype=torch.float64, device=DEV)
    for k in range(case["K"]):
        at = c.argmax(1, keepdim=True)
        gate[:, k:k + 1] = p.gather(1, at)
        c.scatter_(1, at, -math.inf)
    if case["renorm"]:
        gate /= gate.sum(1, keepdim=True)
    gate *= case["scale"]
    if s["mask"] is not None:
        gate *= s["mask"][:, None].double()
    return dict(idx=None, gate=gate)


def _exact_select_bw(s, case):
    lg = s["logits"].double().requires_grad_()
    p = torch.sigmoid(lg) if case["score"] == SIGMOID else torch.softmax(lg, 1)
    ok = (s["idx"] >= 0).double()
    g = p.gather(1, s["idx"].clamp(min=0).long()) * ok
    if case["renorm"]:
        g = g / (g.sum(1, keepdim=True) + (1 - ok[:, :1]))
    (case["scale"] * g * s["dgate"].double() * ok).sum().backward()
    return lg.grad if s["aux"] is None else lg.grad + s["aux"].double()


def _rms(v, w):
    return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS) * w


def _branch(y, w_post, gate):
    u = y if w_post is None else _rms(y, w_post)
    return BRANCH * (u if gate is None else gate * u)


def _wide(t, grad=False):
    return None if t is None else t.double().requires_grad_(grad)


def _exact_norm(s, case):
    h = SHARE * _wide(s["x"]) + _branch(_wide(s["y"]), _wide(s["w_post"]), _wide(s["gate"]))
    return dict(h=h, z=_rms(h, _wide(s["w_pre"])))


def _exact_norm_bw(s, case):
    """Through the graph: the norm before the next block at h, then h's own inputs."""
    h, w = _wide(s["h"], True), _wide(s["w_pre"], True)
    (_rms(h, w) * s["dz"].double()).sum().backward()
    up = h.grad + s["dh"].double()
    y, wp, g = _wide(s["y"], True), _wide(s["w_post"], True), _wide(s["gate"], True)
    (_branch(y, wp, g) * up).sum().backward()
    out = dict(dw_pre=w.grad, dx=SHARE * up, dy=y.grad)
    if wp is not None:
        out["dw_post"] = wp.grad
    if g is not None:
        out["dgate"] = g.grad
    return out


def _exact_codes(v, a, b):
    """v in blocks of a x b, rounded to E4M3 steps over the block's 2^k, in 64 bits."""
    v = v.double()
    R, C = v.shape
    big = torch.zeros(-(-R // a) * a, -(-C // b) * b, dtype=torch.float64, device=DEV)
    big[:R, :C] = v
    amax = big.abs().view(big.shape[0] // a, a, -1).amax(1).view(big.shape[0] // a, big.shape[1] // b, b).amax(2)
    k = torch.ceil(torch.log2(torch.where(amax > 0, amax, 448.0) / 448.0))
    unit = torch.exp2(k).repeat_interleave(a, 0).repeat_interleave(b, 1)
    y = big / unit
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step * unit)[:R, :C]


def _exact_linear(s, case):
    return _exact_codes(s["x"], 1, 128) @ _exact_codes(s["w"], 128, 128).t()


def _exact_linear_bw(s, case):
    dx = _exact_codes(s["dy"], 1, 128) @ _exact_codes(s["w"], 128, 128)
    dw = _exact_codes(s["dy"], 128, 1).t() @ _exact_codes(s["x"], 128, 1)
    return dict(dx=dx, dw=dw)
