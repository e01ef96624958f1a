"""Cases of the sequence-mixing operators that stand beside the gated delta rule: the per-head
norm and position rotation of queries and keys, the gated linear recurrence over packed
sequences, and the single-token forms that a decoding program calls.

With ``own`` false ``run`` computes an operator from elementary torch operations in 32 bits
(angles of positions in 64); with ``own`` true it makes the library's calls.  ``exact`` gives
the same outputs in 64 bits, from the definitions."""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of 16 requests at far positions: 16 query and 16 key heads of 128,
        # read out of a fused projection row
        rope("rope_decode", 16, 16, 16, 128, 128, dtype="bf16", far=True, fused=True),
        # the linear-attention workload's sequence: 32768 tokens, 16 + 16 heads of 128
        rope("rope_prefill", 32768, 16, 16, 128, 128, dtype="bf16", fused=True),
        # odd sizes: 1531 tokens, 10 query heads on 2 key heads of 80, 64 of them rotated in
        # neighbouring pairs, a weight row for each head, fp32
        rope("rope_odd", 1531, 10, 2, 80, 64, interleaved=True, per_head=True, dtype="f32",
             far=True),
        # the backward of the same sequence as rope_prefill, from the fp32 gradients that the
        # delta rule's backward writes
        rope("rope_backward", 32768, 16, 16, 128, 128, backward=True, dtype="bf16", fused=True),
        # the recurrence over one long sequence (prefill), 2048 channels
        glr("glr_long", 32768, 2048, 1, dtype="bf16"),
        # packed prompts of many lengths, empty ones among them, with states carried in and out,
        # gates and inputs as columns of one projection, 1000 channels, padding rows at the end
        glr("glr_packed", 9001, 1000, 37, dtype="f32", mix=True, state=True, fused=True, tail=7),
        # a training pass, forward and backward, over packed sequences: 8192 tokens, 4096 channels
        glr("glr_train", 8192, 4096, 6, dtype="bf16", train=True, mix=True, state=True),
        # a training pass over one narrow sequence: few channels, so the time axis is the work
        glr("glr_train_narrow", 4099, 320, 1, dtype="f32", train=True),
        # one token for each of 64 requests of a pool, 4096 channels
        glr_step("glr_step", 64, 4096, 96, dtype="bf16"),
        # one token of a single request, 16 heads, 128 x 128 states
        gdr_step("gdr_step_one", 1, 16, 128, 128, 1),
        # one token for each of 256 requests, 16 heads, 128 x 128 states out of a larger pool
        gdr_step("gdr_step_batch", 256, 16, 128, 128, 300),
    ]


def rope(name, n, hq, hk, d, rot, interleaved=False, per_head=False, backward=False,
         dtype="bf16", far=False, fused=False):
    return dict(name=name, op="rope", n=n, hq=hq, hk=hk, d=d, rot=rot, interleaved=interleaved,
                per_head=per_head, backward=backward, dtype=dtype, far=far, fused=fused)


def glr(name, n, d, seqs, dtype="bf16", mix=False, state=False, fused=False, tail=0, train=False):
    return dict(name=name, op="glr", n=n, d=d, seqs=seqs, dtype=dtype, mix=mix, state=state,
                fused=fused, tail=tail, train=train)


def glr_step(name, batch, d, slots, dtype="bf16", mix=False):
    return dict(name=name, op="glr_step", batch=batch, d=d, slots=slots, dtype=dtype, mix=mix)


def gdr_step(name, batch, heads, dk, dv, slots):
    return dict(name=name, op="gdr_step", batch=batch, heads=heads, dk=dk, dv=dv, slots=slots)


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["rope", "rope_backward", "glr", "glr_train", "glr_step", "gdr_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if kind.startswith("rope"):
        d = rng.choice([48, 64, 80, 96, 128, 192, 256])
        hq = between(1, 40)
        hk = between(1, hq)
        n = between(1, max(2, 32768 * 32 * 128 * 2 // ((hq + hk) * d * size)))
        c = rope("", min(n, 65536), hq, hk, d, rng.choice([d // 16 * 16, d // 2 // 16 * 16]),
                 interleaved=flip(), per_head=flip(), backward=kind == "rope_backward",
                 dtype=dtype, far=flip(), fused=flip())
    elif kind.startswith("glr") and kind != "glr_step":
        d = between(8, 1024) * 8
        n = between(1, max(2, 32768 * 2048 * 2 // (d * size * (2 if kind == "glr_train" else 1))))
        n = min(n, 65536)
        c = glr("", n, d, rng.choice([1, 1, between(1, 64)]), dtype=dtype, mix=flip(),
                state=flip(), fused=flip(), tail=rng.choice([0, 0, 3]), train=kind == "glr_train")
    elif kind == "glr_step":
        b = between(1, 512)
        c = glr_step("", b, between(8, 1024) * 8, b + rng.randrange(0, 40), dtype=dtype,
                     mix=flip())
    else:
        b = between(1, 256)
        c = gdr_step("", b, between(1, 16), rng.choice([64, 128]), rng.choice([64, 128]),
                     b + rng.randrange(0, 40))
    del c["name"]
    return c


# ------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": prepare_rope, "glr": prepare_glr, "glr_step": prepare_glr_step,
            "gdr_step": prepare_gdr_step}[case["op"]](dict(case), seed, gen)


def randn(gen, shape, dtype=torch.float32, mean=0.0, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)


def log_decay(gen, shape, dtype=torch.float32):
    """ln of forget gates sigmoid(N(4, 1)): most of the state lives on."""
    return torch.nn.functional.logsigmoid(randn(gen, shape, mean=4.0)).to(dtype)


def prepare_rope(c, seed, gen):
    n, hq, hk, d, dt = c["n"], c["hq"], c["hk"], c["d"], DTYPES[c["dtype"]]
    s = dict(c)
    if c["fused"]:  # rows of a fused projection: queries, keys, values
        row = randn(gen, (n, hq + 2 * hk, d), dt)
        s["q"], s["k"] = row[:, :hq], row[:, hq:hq + hk]
    else:
        s["q"], s["k"] = randn(gen, (n, hq, d), dt), randn(gen, (n, hk, d), dt)
    heads = (lambda h: (h, d)) if c["per_head"] else (lambda h: (d,))
    s["wq"], s["wk"] = (randn(gen, heads(h), mean=1.0, std=0.2) for h in (hq, hk))
    s["inv_freq"] = THETA ** (-torch.arange(0, c["rot"], 2, device="cuda",
                                            dtype=torch.float64) / c["rot"])
    if c["far"]:
        s["pos"] = torch.randint(0, 1 << 20, (n,), generator=gen, device="cuda",
                                 dtype=torch.int32)
    else:
        s["pos"] = torch.arange(n, device="cuda", dtype=torch.int32)
    if c["backward"]:
        s["dyq"], s["dyk"] = randn(gen, (n, hq, d)), randn(gen, (n, hk, d))
        s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
    s["yq"] = torch.empty((n, hq, d), dtype=dt, device="cuda")
    s["yk"] = torch.empty((n, hk, d), dtype=dt, device="cuda")
    return s


def prepare_glr(c, seed, gen):
    n, d, seqs, dt = c["n"], c["d"], c["seqs"], DTYPES[c["dtype"]]
    rows = n + c["tail"]
    s = dict(c, rows=rows)
    g, x = log_decay(gen, (rows, d), dt), randn(gen, (rows, d), dt)
    if c["fused"]:
        both = torch.cat([g, x], 1)
        g, x = both[:, :d], both[:, d:]
    s["g"], s["x"] = g, x
    cuts = np.sort(np.random.default_rng(seed).integers(0, n + 1, seqs - 1))
    off = np.concatenate([[0], cuts, [n]]).astype(np.int32)
    s["off"] = torch.from_numpy(off).cuda()
    s["h0"] = randn(gen, (seqs, d)) if c["state"] else None
    s["h"] = torch.zeros((rows, d), dtype=dt, device="cuda")
    s["h_T"] = torch.empty((seqs, d), device="cuda")
    if c["train"]:
        s["dh"] = randn(gen, (rows, d), dt)
        s["dh_T"] = randn(gen, (seqs, d)) if c["state"] else None
        s["h_chunks"] = torch.empty(((rows + 63) // 64, d), device="cuda")
        grads = torch.zeros((rows, 2 * d), dtype=dt, device="cuda")
        if c["fused"]:
            s["dg"], s["dx"] = grads[:, :d], grads[:, d:]
        else:
            s["dg"], s["dx"] = torch.zeros_like(s["h"]), torch.zeros_like(s["h"])
        s["dh0"] = torch.empty((seqs, d), device="cuda") if c["state"] else None
    return s


def a_choice(gen, batch, slots):
    return torch.randperm(slots, generator=gen, device="cuda")[:batch].to(torch.int32)


def prepare_glr_step(c, seed, gen):
    b, d, dt = c["batch"], c["d"], DTYPES[c["dtype"]]
    return dict(c, g=log_decay(gen, (b, d), dt), x=randn(gen, (b, d), dt),
                slot=a_choice(gen, b, c["slots"]), state=randn(gen, (c["slots"], d)),
                h=torch.empty((b, d), dtype=dt, device="cuda"))


def prepare_gdr_step(c, seed, gen):
    b, h, dk, dv = c["batch"], c["heads"], c["dk"], c["dv"]
    bf = torch.bfloat16
    return dict(c, q=randn(gen, (b, h, dk), bf), k=randn(gen, (b, h, dk), bf),
                v=randn(gen, (b, h, dv), bf), beta=torch.sigmoid(randn(gen, (b, h))),
                g=log_decay(gen, (b, h)), slot=a_choice(gen, b, c["slots"]),
                S=randn(gen, (c["slots"], h, dv, dk), std=0.2),
                o=torch.empty((b, h, dv), dtype=bf, device="cuda"))


# ------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return run_own(s)
    return {"rope": plain_rope, "glr": plain_glr, "glr_step": plain_glr_step,
            "gdr_step": plain_gdr_step}[s["op"]](s)


def run_own(s):
    from top_routing_grouped_gemm_gb300 import moe
    dt = moe.MOE_BF16 if s.get("dtype", "bf16") == "bf16" else moe.MOE_F32
    if s["op"] == "rope":
        head = (s["n"], s["d"], s["rot"], s["interleaved"], dt)
        if not s["backward"]:
            moe.moe_qk_norm_rope(*head, EPS, s["pos"], s["inv_freq"],
                                 dict(x=s["q"], y=s["yq"], weight=s["wq"]),
                                 dict(x=s["k"], y=s["yk"], weight=s["wk"]))
            return s["yq"], s["yk"]
        if "ws" not in s:  # kept by a training program from its first step on
            s["ws"] = torch.empty(moe.moe_qk_norm_rope_backward_workspace_size(
                s["n"], s["d"], s["hq"], s["hk"]), dtype=torch.uint8, device="cuda")
        moe.moe_qk_norm_rope_backward(
            *head, moe.MOE_F32, EPS, s["pos"], s["inv_freq"],
            dict(x=s["q"], dy=s["dyq"], dx=s["yq"], weight=s["wq"], dweight=s["dwq"]),
            dict(x=s["k"], dy=s["dyk"], dx=s["yk"], weight=s["wk"], dweight=s["dwk"]), s["ws"])
        return s["yq"], s["yk"], s["dwq"], s["dwk"]
    if s["op"] == "glr":
        mode = moe.MOE_GLR_MIX if s["mix"] else moe.MOE_GLR_ADD
        head = (s["rows"], s["d"], s["seqs"], s["off"], mode, dt, s["g"], s["x"], s["h0"])
        if not s["train"]:
            moe.moe_glr_forward(*head, s["h"], s["h_T"], None)
            return s["h"], s["h_T"]
        moe.moe_glr_forward(*head, s["h"], s["h_T"], s["h_chunks"])
        moe.moe_glr_backward(*head, s["h_chunks"], s["dh"], s["dh_T"], s["dg"], s["dx"],
                             s["dh0"])
        return {"h": s["h"], "h_T": s["h_T"], "dg": s["dg"], "dx": s["dx"], "dh0": s["dh0"]}
    if s["op"] == "glr_step":
        moe.moe_glr_step(s["batch"], s["d"], moe.MOE_GLR_MIX if s["mix"] else moe.MOE_GLR_ADD, dt,
                         s["g"], s["x"], s["slot"], s["slots"], s["state"], s["h"])
        return s["h"], s["state"]
    moe.moe_gdr_step(s["batch"], s["heads"], s["dk"], s["dv"], s["q"], s["k"], s["v"], s["beta"],
                     s["g"], s["slot"], s["slots"], s["dk"] ** -0.5, s["S"], s["o"])
    return s["o"], s["S"]


# ---- norm and rotation: y = R(pos) (w * x / sqrt(mean(x^2) + eps)) for each head

def cos_sin(s):
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def pairs(t, rot, interleaved):
    """The two members of each rotated pair, and what is not rotated."""
    r, rest = t[..., :rot], t[..., rot:]
    if interleaved:
        return r[..., 0::2], r[..., 1::2], rest
    return r[..., :rot // 2], r[..., rot // 2:], rest


def joined(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def plain_rope(s):
    cos, sin = cos_sin(s)

    def forward(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        a, b, rest = pairs(y, s["rot"], s["interleaved"])
        return joined(a * cos - b * sin, b * cos + a * sin, rest, s["interleaved"])

    def backward(x, w, dy):
        x = x.float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        a, b, rest = pairs(dy, s["rot"], s["interleaved"])
        dn = joined(a * cos + b * sin, b * cos - a * sin, rest, s["interleaved"])
        xh = x * rstd
        dw = (dn * xh).sum(0 if w.dim() == 2 else (0, 1))
        dn = dn * w
        return rstd * (dn - xh * (dn * xh).mean(-1, keepdim=True)), dw

    dt = s["q"].dtype
    if not s["backward"]:
        return forward(s["q"], s["wq"]).to(dt), forward(s["k"], s["wk"]).to(dt)
    (dq, dwq), (dk, dwk) = backward(s["q"], s["wq"], s["dyq"]), backward(s["k"], s["wk"], s["dyk"])
    return dq.to(dt), dk.to(dt), dwq, dwk


# ---- recurrence: h_t = exp(g_t) h_{t-1} + x_t, or exp(g_t) h_{t-1} + (1 - exp(g_t)) x_t

def scan(a, b):
    """h_t = a_t h_{t-1} + b_t from h = 0, by doubling the span that each row covers."""
    a, b, span = a.clone(), b.clone(), 1
    while span < a.shape[0]:
        b[span:] += a[span:] * b[:-span]
        a[span:] = a[span:] * a[:-span]
        span *= 2
    return b


def plain_glr(s):
    n, off = s["n"], s["off"].long()
    used = off[1:] > off[:-1]  # sequences that have rows
    first, last = off[:-1][used], off[1:][used] - 1
    g, x = s["g"][:n].float(), s["x"][:n].float()
    a = torch.exp(g)
    within = a.clone()  # the decay, zero where a sequence begins
    within[first] = 0
    b = -torch.expm1(g) * x if s["mix"] else x.clone()
    h0 = s["h0"] if s["state"] else torch.zeros_like(s["h_T"])
    b[first] += a[first] * h0[used]
    h = scan(within, b)
    h_T = h0.clone()
    h_T[used] = h[last]
    out = torch.zeros_like(s["h"])
    out[:n] = h.to(out.dtype)
    if not s["train"]:
        return out, h_T
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])  # h_{t-1}
    before[first] = h0[used]
    after = torch.cat([within[1:], torch.zeros_like(a[:1])])  # the decay of row t + 1
    d = s["dh"][:n].float()
    if s["state"]:
        d[last] += s["dh_T"][used]
    d = scan(after.flip(0), d.flip(0)).flip(0)
    dg, dx = torch.zeros_like(out), torch.zeros_like(out)
    dg[:n] = (d * a * (before - x if s["mix"] else before)).to(out.dtype)
    dx[:n] = (d * -torch.expm1(g) if s["mix"] else d).to(out.dtype)
    dh0 = None
    if s["state"]:
        dh0 = s["dh_T"].clone()
        dh0[used] = a[first] * d[first]
    return {"h": out, "h_T": h_T, "dg": dg, "dx": dx, "dh0": dh0}


def plain_glr_step(s):
    g, x, slot = s["g"].float(), s["x"].float(), s["slot"].long()
    h = torch.exp(g) * s["state"][slot] + (-torch.expm1(g) * x if s["mix"] else x)
    s["state"][slot] = h
    return h.to(s["h"].dtype), s["state"]


# ---- one token of the gated delta rule: S <- exp(g) S (I - beta k^ k^T) + beta v k^T

def plain_gdr_step(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    q = q / q.square().sum(-1, keepdim=True).sqrt()
    k = k / k.square().sum(-1, keepdim=True).sqrt()
    slot = s["slot"].long()
    S = torch.exp(s["g"])[..., None, None] * s["S"][slot]
    delta = s["beta"][..., None] * (v - (S * k[:, :, None]).sum(-1))
    S = S + delta[..., None] * k[:, :, None]
    s["S"][slot] = S
    o = (S * q[:, :, None]).sum(-1) * s["dk"] ** -0.5
    return o.to(s["o"].dtype), s["S"]


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return {"rope": exact_rope, "glr": exact_glr, "glr_step": exact_glr_step,
            "gdr_step": exact_gdr_step}[case["op"]](prepare(case, seed))


def exact_rope(s):
    """The rotation as a product of complex numbers; the gradients by differentiating it."""
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None] * s["inv_freq"])[:, None]
    rot, half = s["rot"], s["rot"] // 2

    def forward(x, w):
        y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        if s["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], half, 2).contiguous())
            r = torch.view_as_real(z * turn).flatten(-2)
        else:
            z = torch.complex(y[..., :half], y[..., half:rot]) * turn
            r = torch.cat([z.real, z.imag], -1)
        return torch.cat([r, y[..., rot:]], -1)

    if not s["backward"]:
        return forward(s["q"].double(), s["wq"].double()), forward(s["k"].double(),
                                                                   s["wk"].double())
    got = []
    for x, w, dy in ((s["q"], s["wq"], s["dyq"]), (s["k"], s["wk"], s["dyk"])):
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        got.append(torch.autograd.grad((forward(x, w) * dy.double()).sum(), (x, w)))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def exact_glr(s):
    """Row after row, as the recurrence is written."""
    off, n = s["off"].tolist(), s["n"]
    g, x = s["g"][:n].double(), s["x"][:n].double()
    a = torch.exp(g)
    b = (1 - a) * x if s["mix"] else x
    h0 = s["h0"].double() if s["state"] else torch.zeros_like(s["h_T"], dtype=torch.float64)
    h = torch.zeros(s["h"].shape, dtype=torch.float64, device="cuda")
    before, h_T = torch.zeros_like(a), h0.clone()
    for i in range(len(off) - 1):
        now = h0[i]
        for t in range(off[i], off[i + 1]):
            before[t] = now
            torch.addcmul(b[t], a[t], now, out=h[t])
            now = h[t]
        h_T[i] = now
    if not s["train"]:
        return h, h_T
    d = torch.zeros_like(h)
    d[:n] = s["dh"][:n]
    dh0 = s["dh_T"].double() if s["state"] else torch.zeros_like(h0)
    for i in range(len(off) - 1):
        back = dh0[i].clone()
        for t in range(off[i + 1] - 1, off[i] - 1, -1):
            d[t] += back
            back = a[t] * d[t]
        dh0[i] = back
    dg, dx = torch.zeros_like(d), torch.zeros_like(d)
    dg[:n] = d[:n] * a * (before - x if s["mix"] else before)
    dx[:n] = d[:n] * (1 - a) if s["mix"] else d[:n]
    return {"h": h, "h_T": h_T, "dg": dg, "dx": dx, "dh0": dh0 if s["state"] else None}


def exact_glr_step(s):
    g, slot, state = s["g"].double(), s["slot"].long(), s["state"].double()
    x = s["x"].double()
    h = g.exp() * state[slot] + ((1 - g.exp()) * x if s["mix"] else x)
    state[slot] = h
    return h, state


def exact_gdr_step(s):
    """With the transition matrix written out."""
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    slot, S = s["slot"].long(), s["S"].double()
    beta = s["beta"].double()[..., None, None]
    move = torch.eye(s["dk"], dtype=torch.float64, device="cuda") - beta * k[..., :, None] * k[
        ..., None, :]
    new = s["g"].double().exp()[..., None, None] * (S[slot] @ move) + beta * v[..., :, None] * k[
        ..., None, :]
    S[slot] = new
    return (new @ q[..., None])[..., 0] * s["dk"] ** -0.5, S


# ------------------------------------------------------------------------------- the work

def work(case):
    c = case
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        heads = c["hq"] + c["hk"]
        values, weights = c["n"] * heads * c["d"], (heads if c["per_head"] else 2) * c["d"] * 4
        nbytes = values * 2 * size + weights + c["n"] * 4 + c["rot"] * 4
        if c["backward"]:
            return {"bytes": nbytes + values * 4 + weights, "flops": 14 * values}
        return {"bytes": nbytes, "flops": 7 * values}
    if c["op"] == "glr":
        size = 2 if c["dtype"] == "bf16" else 4
        values, states = c["n"] * c["d"], c["seqs"] * c["d"] * 4
        nbytes = (6 if c["train"] else 3) * values * size + states * (2 if c["state"] else 1)
        if c["train"] and c["state"]:
            nbytes += 2 * states
        return {"bytes": nbytes + (c["seqs"] + 1) * 4, "flops": (10 if c["train"] else 3) * values}
    if c["op"] == "glr_step":
        values = c["batch"] * c["d"]
        return {"bytes": values * (8 + 3 * (2 if c["dtype"] == "bf16" else 4)) + c["batch"] * 4,
                "flops": 3 * values}
    rows = c["batch"] * c["heads"]
    return {"bytes": rows * (c["dk"] * c["dv"] * 8 + (2 * c["dk"] + 2 * c["dv"]) * 2 + 8) + c[
        "batch"] * 4, "flops": rows * c["dk"] * c["dv"] * 8}
