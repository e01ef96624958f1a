"""Cases of the operators around the experts: routing with softmax or sigmoid scores, a balance
bias and groups; the norms before and after a block with its gate and residual scale; the experts'
products with 4-bit weights for few tokens.

With ``own`` false ``run`` computes an operator from elementary torch operations in 32 bits (in 64
where the order of nearly equal scores is decided); with ``own`` true it makes the library's calls.
``exact`` gives the same outputs in 64 bits, from the definitions."""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
SCALE = 0.5  # of a block's output, before it joins the residual stream
GATES_SCALE = 2.5  # of the routing gates
NORM_OUTPUTS = ("z", "normed", "dx", "dy", "dgate", "dw_post", "dw_pre")


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding token over 896 experts in 8 groups, balance bias, sigmoid scores
        route("route_token", 1, 896, 16, groups=8, kept=4, best=2, bias=True),
        # a prefill batch of the same width without groups
        route("route_prefill", 16384, 896, 16, bias=True),
        # a training step's routing, forward and backward, groups by their best two
        route("route_train", 8192, 896, 16, groups=8, kept=4, best=2, bias=True, train=True),
        # odd sizes: 1531 tokens, 100 experts in 10 groups, softmax scores taken as they are, bf16
        route("route_odd", 1531, 100, 6, score="softmax", groups=10, kept=3, best=1, renorm=False,
              dtype="bf16", train=True),
        # one decoding token between two blocks: the norm after one, its gate, the norm before
        # the next
        norm("norm_token", 1, 4096, gated="token"),
        # a prefill batch, a learned scale for each channel
        norm("norm_prefill", 16384, 4096, gated="channel", sigmoid=False),
        # a training step: residual stream in fp32, blocks in bf16, a gate for each token
        norm("norm_train", 8192, 4096, stream="f32", gated="token", train=True),
        # odd sizes: 1531 rows of 1000, fp32, a gate for each value, columns of wider rows
        norm("norm_odd", 1531, 1000, stream="f32", dtype="f32", gated="value", fused=True,
             train=True),
        # one decoding token through 16 of 896 experts
        w4("w4_token", 1, 896, 16, 4096, 1024, 128),
        # a small model's experts, 7 tokens
        w4("w4_small", 7, 64, 4, 512, 256, 32),
        # a serving batch of 32 tokens, zero points, finer groups
        w4("w4_batch", 32, 896, 16, 2048, 512, 64, zeros=True),
        # 64 tokens that crowd on few experts
        w4("w4_hot", 64, 896, 16, 4096, 1024, 128, skew=1.0),
    ]


def route(name, n, experts, k, score="sigmoid", groups=1, kept=1, best=1, bias=False, renorm=True,
          dtype="f32", train=False):
    return dict(name=name, op="route", n=n, experts=experts, k=k, score=score, groups=groups,
                kept=kept, best=best, bias=bias, renorm=renorm, dtype=dtype, train=train)


def norm(name, n, d, stream="bf16", dtype="bf16", gated="none", sigmoid=True, post=True,
         fused=False, train=False):
    return dict(name=name, op="norm", n=n, d=d, stream=stream, dtype=dtype, gated=gated,
                sigmoid=sigmoid, post=post, fused=fused, train=train)


def w4(name, n, experts, k, d, f, group, zeros=False, skew=0.0):
    return dict(name=name, op="w4", n=n, experts=experts, k=k, d=d, f=f, group=group, zeros=zeros,
                skew=skew)


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["route", "route", "norm", "norm", "w4", "w4"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 7, 8, 10, 16])
        size = between(max(2, 8 // groups), 1024 // groups)
        experts = groups * size
        kept = rng.randint(max(1, groups // 2), groups)
        c = route("", min(between(1, 16384), 16384 * 896 // (2 * experts)), experts,
                  rng.randint(1, min(32, kept * size)), score=rng.choice(["sigmoid", "softmax"]),
                  groups=groups, kept=kept, best=rng.choice([1, 2]), bias=flip(), renorm=flip(),
                  dtype=rng.choice(["f32", "f32", "bf16"]), train=flip())
    elif kind == "norm":
        d = between(8, 1024) * 8
        train = flip()
        n = min(65536, between(1, max(2, 8192 * 4096 // (2 * d))))
        stream, dtype = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        c = norm("", n, d, stream=stream, dtype=dtype,
                 gated=rng.choice(["none", "channel", "token", "value"]), sigmoid=flip(),
                 post=flip(), fused=flip(), train=train)
    else:
        experts = between(8, 896)
        k = rng.randint(1, min(16, experts))
        group = rng.choice([32, 64, 128])
        step = max(group, 64)
        d, f = between(2, 4096 // step) * step, between(1, 1024 // step) * step
        skew = rng.choice([0.0, 1.0])
        c = w4("", between(1, 64 if skew else 24), experts, k, d, f, group, zeros=flip(),
               skew=skew)
    del c["name"]
    return c


# ------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"route": prepare_route, "norm": prepare_norm, "w4": prepare_w4}[case["op"]](
        dict(case), gen)


def randn(gen, shape, dtype=torch.float32, mean=0.0, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)


def empty(shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare_route(c, gen):
    n, e, k = c["n"], c["experts"], c["k"]
    s = dict(c, logits=randn(gen, (n, e), DTYPES[c["dtype"]]))
    # what a balancing rule that adds small steps arrives at, on the scale of the scores
    std = 0.05 if c["score"] == "sigmoid" else 0.5 / e
    s["b"] = randn(gen, (e,), std=std) if c["bias"] else None
    s["idx"], s["gate"] = empty((n, k), torch.int32), empty((n, k))
    s["partials"] = empty(((n + 7) // 8, e))
    if c["train"]:
        s["dgate"] = randn(gen, (n, k))
        s["dlogits"] = torch.empty_like(s["logits"])
    if own:
        from top_routing_grouped_gemm_gb300 import moe
        score = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        s["rule"] = moe.RouteRule(score, c["groups"], c["kept"], c["best"], c["renorm"],
                                  GATES_SCALE)
    return s


def prepare_norm(c, gen):
    n, d, st, dt = c["n"], c["d"], DTYPES[c["stream"]], DTYPES[c["dtype"]]
    s = dict(c)
    if c["fused"]:  # the block's output and its gates as columns of one projection
        both = randn(gen, (n, 2 * d + 8), dt)
        s["y"], gates = both[:, :d], both[:, d:2 * d]
    else:
        s["y"], gates = randn(gen, (n, d), dt), None
    s["x"] = randn(gen, (n, d), st, std=2.0)
    s["gate"] = {"none": lambda: None, "channel": lambda: randn(gen, (d,), mean=0.5, std=0.2),
                 "token": lambda: randn(gen, (n,)),
                 "value": lambda: randn(gen, (n, d), dt) if gates is None else gates}[c["gated"]]()
    s["w_post"] = randn(gen, (d,), mean=1.0, std=0.2) if c["post"] else None
    s["w_pre"] = randn(gen, (d,), mean=1.0, std=0.2)
    s["z"], s["normed"] = empty((n, d), st), empty((n, d), dt)
    if c["train"]:
        s["dz"], s["dn"] = randn(gen, (n, d), st), randn(gen, (n, d), dt)
        s["dx"], s["dy"] = empty((n, d), st), empty((n, d), dt)
        s["dgate"] = None if s["gate"] is None else empty(s["gate"].shape, s["gate"].dtype)
        s["dw_post"], s["dw_pre"] = empty((d,)) if c["post"] else None, empty((d,))
    return s


def popularity(c):
    """ln of the experts' weights: a power law of their rank."""
    return -c["skew"] * np.log(np.arange(1, c["experts"] + 1))


def prepare_w4(c, gen):
    n, e, k, d, f, group = (c[i] for i in ("n", "experts", "k", "d", "f", "group"))
    s = dict(c, x=randn(gen, (n, d), torch.bfloat16), y=empty((n, d), torch.bfloat16))
    # k distinct experts a token, by their popularity
    u = torch.rand((n, e), generator=gen, device="cuda", dtype=torch.float64).clamp_(1e-12)
    score = torch.from_numpy(popularity(c)).cuda() - torch.log(-torch.log(u))
    score, s["idx"] = score.sort(descending=True)
    s["idx"] = s["idx"][:, :k].to(torch.int32).contiguous()
    s["gate"] = torch.softmax(randn(gen, (n, k)), -1)
    s["w"] = {}
    for name, rows, cols in (("gate", f, d), ("up", f, d), ("down", d, f)):
        codes = torch.randint(0, 256, (e, rows, cols // 2), generator=gen, device="cuda",
                              dtype=torch.uint8)
        scales = torch.rand((e, rows, cols // group), generator=gen, device="cuda").add_(0.5).mul_(
            0.2 * cols ** -0.5).to(torch.bfloat16)
        zeros = torch.randint(6, 11, scales.shape, generator=gen, device="cuda",
                              dtype=torch.uint8) if c["zeros"] else None
        s["w"][name] = codes, scales, zeros
    if own:  # a serving program lays its weights out once
        from top_routing_grouped_gemm_gb300 import moe
        s["problem"] = moe.Problem(n, d, e, k, f)
        s["packed"] = {name: moe.W4Weights(*w) for name, w in s["w"].items()}
        s["ws"] = empty((moe.moe_w4_expert_ffn_workspace_size(s["problem"]),), torch.uint8)
    return s


# ------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return {"route": own_route, "norm": own_norm, "w4": own_w4}[s["op"]](s)
    return {"route": plain_route, "norm": plain_norm, "w4": plain_w4}[s["op"]](s)


def own_route(s):
    from top_routing_grouped_gemm_gb300 import moe
    dt = moe.MOE_BF16 if s["dtype"] == "bf16" else moe.MOE_F32
    head = (s["n"], s["experts"], s["k"], s["rule"], dt, s["logits"])
    moe.moe_route_select(*head, s["b"], s["idx"], s["gate"], s["partials"])
    if not s["train"]:
        return s["idx"], s["gate"], s["partials"]
    moe.moe_route_select_backward(*head, s["idx"], s["dgate"], s["dlogits"], None)
    return s["idx"], s["gate"], s["partials"], s["dlogits"]


def own_norm(s):
    from top_routing_grouped_gemm_gb300 import moe
    code = {"bf16": moe.MOE_BF16, "f32": moe.MOE_F32}
    kind = {"none": moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL,
            "token": moe.MOE_GATE_TOKEN, "value": moe.MOE_GATE_VALUE}[s["gated"]]
    n, d = s["n"], s["d"]
    head = (n, d, code[s["stream"]], code[s["dtype"]], EPS, SCALE, s["x"], s["y"], kind,
            s["sigmoid"], s["gate"], s["post"], s["w_post"], s["w_pre"])
    moe.moe_block_norm(*head, s["z"], s["normed"])
    if not s["train"]:
        return s["z"], s["normed"]
    if "ws" not in s:  # kept by a training program from its first step on
        s["ws"] = empty((moe.moe_block_norm_backward_workspace_size(n, d, kind),), torch.uint8)
    moe.moe_block_norm_backward(*head, s["dz"], code[s["dtype"]], s["dn"], s["dx"], s["dy"],
                                s["dgate"], s["dw_post"], s["dw_pre"], s["ws"])
    return {i: s[i] for i in NORM_OUTPUTS}


def own_w4(s):
    from top_routing_grouped_gemm_gb300 import moe
    w = s["packed"]
    moe.moe_w4_expert_ffn(s["problem"], s["x"], s["idx"], s["gate"], w["gate"], w["up"], w["down"],
                          s["y"], s["ws"])
    return s["y"]


# ---- routing: the k largest scores + bias in the groups kept, gates from the scores alone

def stable(t):
    """Indices in descending order; equal values keep theirs."""
    return t.sort(dim=-1, descending=True, stable=True).indices


def plain_route(s):
    n, e, k, groups = s["n"], s["experts"], s["k"], s["groups"]
    logits = s["logits"].float()
    score = torch.sigmoid if s["score"] == "sigmoid" else (lambda t: torch.softmax(t, -1))
    # nearly equal scores are told apart in 64 bits; without a bias the logits have the order
    wide = score(logits.double())
    choice = wide if s["b"] is None else wide + s["b"]
    key = logits.double() if s["b"] is None else choice
    if groups > 1:
        best = choice.view(n, groups, -1).sort(dim=-1, descending=True).values
        kept = stable(best[..., :s["best"]].sum(-1))[:, :s["kept"]]
        out = torch.ones((n, groups), dtype=torch.bool, device="cuda").scatter_(1, kept, False)
        key = key.view(n, groups, -1).masked_fill(out[..., None], -math.inf).view(n, e)
    idx = stable(key)[:, :k]
    p = score(logits)
    g = p.gather(1, idx)
    total = g.sum(-1, keepdim=True)
    gate = GATES_SCALE * (g / total if s["renorm"] else g)
    share = p / p.sum(-1, keepdim=True)  # summed over blocks of eight tokens
    share = torch.cat([share, share.new_zeros((-n % 8, e))]).view(-1, 8, e).sum(1)
    out = idx.to(torch.int32), gate, share
    if not s["train"]:
        return out
    d = GATES_SCALE * s["dgate"]
    if s["renorm"]:
        d = (d - (d * g / total).sum(-1, keepdim=True)) / total
    dp = torch.zeros_like(p).scatter_(1, idx, d)
    if s["score"] == "sigmoid":
        dl = dp * p * (1 - p)
    else:
        dl = p * (dp - (dp * p).sum(-1, keepdim=True))
    return *out, dl.to(s["dlogits"].dtype)


# ---- z = x + scale a(gate) u,  u = w_post y / rms(y) or y;  normed = w_pre z / rms(z)

def rstd(t):
    return torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)


def plain_norm(s):
    x, y = s["x"].float(), s["y"].float()
    a = torch.ones((), device="cuda") if s["gate"] is None else s["gate"].float()
    a = a[:, None] if s["gated"] == "token" else a
    act = torch.sigmoid(a) if s["sigmoid"] and s["gate"] is not None else a
    ry = rstd(y) if s["post"] else None
    u = s["w_post"] * (y * ry) if s["post"] else y
    z = x + SCALE * act * u
    rz = rstd(z)
    out = z.to(s["z"].dtype), (s["w_pre"] * (z * rz)).to(s["normed"].dtype)
    if not s["train"]:
        return out

    def through(d, t, r, w):
        """Gradients of w t / rms(t) with respect to t and w."""
        th = t * r
        dw, d = (d * th).sum(0), d * w
        return r * (d - th * (d * th).mean(-1, keepdim=True)), dw

    dz, dw_pre = through(s["dn"].float(), z, rz, s["w_pre"])
    dz = dz + s["dz"].float()
    du, dw_post = SCALE * act * dz, None
    da = SCALE * dz * u
    da = {"none": lambda: None, "channel": lambda: da.sum(0),
          "token": lambda: da.sum(-1, keepdim=True), "value": lambda: da}[s["gated"]]()
    if da is not None:
        da = da * act * (1 - act) if s["sigmoid"] else da
        da = da.reshape(s["gate"].shape).to(s["gate"].dtype)
    dy = du
    if s["post"]:
        dy, dw_post = through(du, y, ry, s["w_post"])
    got = *out, dz.to(s["dx"].dtype), dy.to(s["dy"].dtype), da, dw_post, dw_pre
    return dict(zip(NORM_OUTPUTS, got))


# ---- y = sum_j gate_j W_down (silu(W_gate x) * (W_up x)), with the weights of expert idx_j

def plain_w4(s):
    group = s["group"]

    def weights(name, e):
        codes, scales, zeros = (None if t is None else t[e][0] for t in s["w"][name])
        v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
        v = v.view(v.shape[0], -1, group) - (8.0 if zeros is None else zeros.float()[..., None])
        return (v * scales.float()[..., None]).flatten(1)

    x, y = s["x"].float(), torch.zeros(s["y"].shape, device="cuda")
    for t in range(s["n"]):
        for j in range(s["k"]):
            e = s["idx"][t, j:j + 1]
            a, b = ((weights(name, e) * x[t]).sum(-1) for name in ("gate", "up"))
            h = a * torch.sigmoid(a) * b
            y[t] += s["gate"][t, j] * (weights("down", e) * h).sum(-1)
    return y.to(s["y"].dtype)


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return {"route": exact_route, "norm": exact_norm, "w4": exact_w4}[case["op"]](
        prepare(case, seed))


def exact_route(s):
    """Expert after expert taken from those that are left; gradients by differentiating."""
    n, e, k, groups = s["n"], s["experts"], s["k"], s["groups"]
    logits = s["logits"].double().requires_grad_()
    if s["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-logits))
    else:
        p = torch.exp(logits - torch.logsumexp(logits, -1, keepdim=True))
    with torch.no_grad():
        c = p.clone() if s["b"] is None else p + s["b"].double()

        def take(t):
            """The first of the largest values, as a column, which is then taken out."""
            top = (t == t.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)
            value = t.gather(-1, top)
            t.scatter_(-1, top, -math.inf)
            return top, value

        left = (logits if s["b"] is None else c).detach().clone()
        if groups > 1:
            inside = c.view(n, groups, -1).clone()
            worth = sum(take(inside)[1][..., 0] for _ in range(s["best"]))
            keep = torch.zeros((n, groups), dtype=torch.bool, device="cuda")
            for _ in range(s["kept"]):
                keep.scatter_(1, take(worth)[0], True)
            left[~keep.repeat_interleave(e // groups, 1)] = -math.inf
        idx = torch.cat([take(left)[0] for _ in range(k)], 1)
    g = p.gather(1, idx)
    gate = GATES_SCALE * (g / g.sum(-1, keepdim=True) if s["renorm"] else g)
    share = (p / p.sum(-1, keepdim=True)).detach()
    block = torch.arange(n, device="cuda") // 8
    partials = torch.zeros(s["partials"].shape, dtype=torch.float64,
                           device="cuda").index_add_(0, block, share)
    out = idx.to(torch.int32), gate.detach(), partials
    if not s["train"]:
        return out
    return *out, torch.autograd.grad((gate * s["dgate"].double()).sum(), logits)[0]


def exact_norm(s):
    """By differentiating the definition."""
    leaf = {i: s[i].double().requires_grad_() for i in ("x", "y", "gate", "w_post", "w_pre")
            if s[i] is not None}

    def rms_norm(t, w):
        return t / (t.square().mean(-1, keepdim=True) + EPS).sqrt() * w

    u = rms_norm(leaf["y"], leaf["w_post"]) if s["post"] else leaf["y"]
    if s["gated"] != "none":
        a = leaf["gate"].unsqueeze(-1) if s["gated"] == "token" else leaf["gate"]
        u = u / (1 + torch.exp(-a)) if s["sigmoid"] else u * a
    z = leaf["x"] + SCALE * u
    normed = rms_norm(z, leaf["w_pre"])
    if not s["train"]:
        return z.detach(), normed.detach()
    back = (z * s["dz"].double()).sum() + (normed * s["dn"].double()).sum()
    d = dict(zip(leaf, torch.autograd.grad(back, list(leaf.values()))))
    got = z.detach(), normed.detach(), *(d.get(i) for i in ("x", "y", "gate", "w_post", "w_pre"))
    return dict(zip(NORM_OUTPUTS, got))


def exact_w4(s):
    """Expert after expert, with all of its tokens."""
    group, idx = s["group"], s["idx"].long()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for e in idx.unique().tolist():
        w = {}
        for name, (codes, scales, zeros) in s["w"].items():
            low, high = codes[e] % 16, codes[e] // 16
            v = torch.empty((codes.shape[1], codes.shape[2] * 2), dtype=torch.float64,
                            device="cuda")
            v[:, 0::2], v[:, 1::2] = low, high
            v -= 8 if zeros is None else zeros[e].double().repeat_interleave(group, 1)
            w[name] = v * scales[e].double().repeat_interleave(group, 1)
        t, j = (idx == e).nonzero(as_tuple=True)
        x = s["x"][t].double()
        a = x @ w["gate"].T
        h = a / (1 + torch.exp(-a)) * (x @ w["up"].T)
        y.index_add_(0, t, s["gate"][t, j].double()[:, None] * (h @ w["down"].T))
    return y


# ------------------------------------------------------------------------------- the work

def work(case):
    c = case
    size = lambda dtype: 2 if dtype == "bf16" else 4  # noqa: E731
    if c["op"] == "route":
        cells, slots = c["n"] * c["experts"], c["n"] * c["k"]
        nbytes = cells * size(c["dtype"]) + c["experts"] * 4 * (c["bias"] + (c["n"] + 7) // 8)
        nbytes += slots * 8
        if c["train"]:
            nbytes += slots * 4 + cells * size(c["dtype"])
        return {"bytes": nbytes, "flops": cells * (8 if c["train"] else 6)}
    if c["op"] == "norm":
        cells, st, dt = c["n"] * c["d"], size(c["stream"]), size(c["dtype"])
        gates = {"none": 0, "channel": c["d"] * 4, "token": c["n"] * 4,
                 "value": cells * dt}[c["gated"]]
        weights = c["d"] * 4 * (1 + c["post"])
        nbytes = cells * (2 * st + 2 * dt) + gates + weights
        if c["train"]:  # dz, dn read; dx, dy and the other gradients written
            nbytes += cells * (2 * st + 2 * dt) + gates + weights
        return {"bytes": nbytes, "flops": cells * (34 if c["train"] else 10)}
    # the experts that a batch reaches, of random choices like those of the inputs
    draw = np.random.default_rng(0).gumbel(size=(c["n"], c["experts"])) + popularity(c)
    reached = len(np.unique(np.argsort(-draw, axis=1)[:, :c["k"]]))
    values = 3 * c["d"] * c["f"]
    per_group = 3 if c["zeros"] else 2
    return {"bytes": reached * (values // 2 + values // c["group"] * per_group) + c["n"] * (
        4 * c["d"] + 8 * c["k"]), "flops": 2 * c["n"] * c["k"] * values}
