"""What stands around the experts, as it is used: the layer with a rule for its routing, a training step
from norm to norm, the 4-bit experts over their whole range, calls side by side and in graphs.

Tolerances as in test_gpu_moe_block.py; those of the layer's own products as in test_gpu_backward.py."""

import numpy as np
import pytest
import torch

import oracle
from oracle import moe_block as MB
from parity_util import RTOL_FP, f64, relerr
from rounding import Rounded, U
from test_gpu_moe_block import (BF, EPS, F32, LAST, SCALE, SIG, SOFT, check_w4, formed, grads_of, randn,
                                run_w4, w4_case, w4_weights)
from top_routing_grouped_gemm_gb300 import moe

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------ the layer with a rule

class Layer:
    """A layer's weights and buffers, and its 64-bit form on the logits that the GPU formed."""

    def __init__(self, T, d, E, k, F, rule, biased, cap=(0, 0), seed=0):
        gen = torch.Generator().manual_seed(seed + T + E)
        self.p = moe.Problem(T, d, E, k, F, cap_num=cap[0], cap_den=cap[1])
        self.rule, self.k = rule, k
        self.router = (randn(gen, E, d) * d ** -0.5).cuda()
        self.bias = (randn(gen, E) * 0.1).cuda()
        self.select_bias = (randn(gen, E) * 0.05).cuda() if biased else None
        self.w = [(randn(gen, E, *s) * s[1] ** -0.5).to(BF).cuda() for s in ((F, d), (F, d), (d, F))]
        self.buf = moe.LayerBuffers(self.p, "cuda", train=True)
        self.x = randn(gen, T, d).to(BF).cuda()
        self.dy = randn(gen, T, d).to(BF).cuda()

    def forward(self, x):
        return moe.layer_forward(self.buf, x, self.router, self.bias, *self.w, gather=False,
                                 rule=self.rule, select_bias=self.select_bias)

    def backward(self, dy, x):
        return moe.layer_backward(self.buf, dy, x, self.router, *self.w, rule=self.rule)

    def check(self, x, dy):
        b, r, k = self.buf, self.rule, self.k
        logits, x, dy = f64(b.logits), f64(x), f64(dy)
        T, E = logits.shape
        how = (r.score == SIG, r.groups, r.groups_kept, r.group_best, r.renormalise, r.scale)
        idx, gate, partials = MB.select(logits, f64(self.select_bias), k, *how)
        assert np.array_equal(b.topk_idx.cpu().numpy(), idx)
        assert relerr(f64(b.topk_gate), gate) <= 1e-5 and relerr(f64(b.partials), partials) <= 1e-5
        kept = b.slot_row.view(T, k).cpu().numpy() >= 0
        w = [f64(m) for m in self.w]
        y, dx, dgate = np.zeros_like(x), np.zeros_like(x), np.zeros((T, k))
        for e in range(E):
            t, j = np.nonzero((idx == e) & kept)
            if not len(t):
                continue
            out = oracle.expert_forward(x[t], *(m[e] for m in w))[3]
            g = gate[t, j][:, None]
            dX, _ = oracle.expert_backward(x[t], g * dy[t], *(m[e] for m in w))
            np.add.at(y, t, g * out)
            np.add.at(dx, t, dX)
            dgate[t, j] = (dy[t] * out).sum(-1)
        dlogits = MB.select_backward(logits, idx, dgate, how[0], r.renormalise, r.scale)
        counts = np.bincount(idx.ravel(), minlength=E)
        share = partials.sum(0) / T
        assert abs(float(b.aux.item()) - oracle.aux_loss(counts, np.tile(share, (T, 1)), T, k, E)) <= (
            1e-4 * abs(float(b.aux.item())))
        assert relerr(f64(b.y), y) <= RTOL_FP
        assert relerr(f64(b.dgate), dgate) <= RTOL_FP
        assert relerr(f64(b.dlogits_topk), np.take_along_axis(dlogits, idx, 1)) <= 2 * RTOL_FP
        assert relerr(f64(b.dx), dx + dlogits @ f64(self.router)) <= RTOL_FP
        assert int(b.dev_status.item()) == 0


LAYERS = [
    (1, 128, 8, 2, 64, moe.RouteRule(SIG), True, (0, 0)),
    (300, 192, 16, 4, 128, moe.RouteRule(SIG, 4, 2, 2, True, 2.5), True, (0, 0)),
    (257, 128, 12, 3, 192, moe.RouteRule(SIG, 1, 1, 1, False, 1.5), True, (5, 4)),
    (130, 256, 40, 6, 64, moe.RouteRule(SOFT, 8, 4, 1, True, 1.0), False, (0, 0)),
    (200, 128, 9, 2, 64, moe.RouteRule(SOFT, 3, 2, 2, True, 3.0), True, (1, 1)),
]


@pytest.mark.parametrize("case", LAYERS, ids=[str(i) for i in range(len(LAYERS))])
def test_layer_with_a_rule(case):
    layer = Layer(*case)
    layer.forward(layer.x)
    layer.backward(layer.dy, layer.x)
    layer.check(layer.x, layer.dy)


def test_rule_of_the_plain_router():
    """Softmax scores, renormalised, without groups or bias: the experts that the layer takes without a
    rule; the same logits, to the bit."""
    layer = Layer(333, 192, 24, 5, 64, moe.RouteRule(SOFT), False)
    layer.forward(layer.x)
    b = layer.buf
    idx, gate, logits, partials, aux = (t.clone() for t in (b.topk_idx, b.topk_gate, b.logits, b.partials,
                                                           b.aux))
    moe.layer_forward(b, layer.x, layer.router, layer.bias, *layer.w, gather=False)
    assert torch.equal(idx, b.topk_idx) and torch.equal(logits, b.logits)
    # both formed from k exponentials and their sum, and 8 tokens' shares of E
    assert torch.allclose(gate, b.topk_gate, rtol=32 * U, atol=0)
    assert torch.allclose(partials, b.partials, rtol=96 * U, atol=0)
    assert torch.allclose(aux, b.aux, rtol=256 * U, atol=0)


@pytest.mark.parametrize("T, d, E, k, biased", [(1, 64, 1, 1, False), (7, 128, 20, 2, True),
                                                (300, 320, 130, 8, True), (1030, 192, 896, 16, False)])
def test_route_logits_are_the_routers(T, d, E, k, biased):
    gen = torch.Generator().manual_seed(T)
    p = moe.Problem(T, d, E, k, 64)
    x, w = randn(gen, T, d).to(BF).cuda(), (randn(gen, E, d) * d ** -0.5).cuda()
    bias = randn(gen, E).cuda() if biased else None
    ws = torch.empty(moe.moe_route_workspace_size(p), dtype=torch.uint8, device="cuda")
    idx, gate = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    partials = torch.empty((moe.moe_route_num_partials(p), E), device="cuda")
    want, got = (torch.full((T, E), np.nan, device="cuda") for _ in range(2))
    moe.moe_route(p, x, w, bias, idx, gate, partials, want, ws)
    moe.moe_route_logits(p, x, w, bias, got, ws)
    assert torch.equal(want, got)


def test_dispatch_logits_backward():
    """Against sums in 64 bits: 2 k terms to a value, with dropped slots and bad experts."""
    T, d, E, k = 70, 192, 11, 4
    gen = torch.Generator().manual_seed(4)
    p = moe.Problem(T, d, E, k, 64)
    rows = randn(gen, T * k, d).to(BF)
    slot_row = torch.randperm(T * k, generator=gen).to(torch.int32)
    slot_row[::7] = -1
    idx = torch.randint(0, E, (T, k), generator=gen).to(torch.int32)
    idx[3, 1], idx[4, 0] = -1, E
    dl, w = randn(gen, T, k), randn(gen, E, d)
    dx = torch.full((T, d), np.nan, device="cuda")
    moe.moe_dispatch_logits_bwd(p, rows.cuda(), slot_row.cuda(), idx.cuda(), dl.cuda(), w.cuda(), dx)
    good = ((idx >= 0) & (idx < E)).numpy()
    terms = f64(dl * torch.from_numpy(good))[:, :, None] * f64(w)[np.where(good, idx.numpy(), 0)]
    from_rows = np.where((slot_row >= 0).numpy()[:, None], f64(rows)[slot_row.clamp(min=0).numpy()], 0)
    all_terms = np.concatenate([from_rows.reshape(T, k, d), terms], 1)
    Rounded(all_terms, U * np.abs(all_terms)).sum(1).close(f64(dx), what="dx")


def test_layer_refuses_rules():
    layer = Layer(5, 64, 4, 2, 64, moe.RouteRule(SOFT, renormalise=False), False)
    layer.forward(layer.x)
    with pytest.raises(ValueError, match="renormalised"):
        layer.backward(layer.dy, layer.x)
    layer.rule = moe.RouteRule(SIG, scale=-1.0)
    with pytest.raises(ValueError, match="scale"):
        layer.backward(layer.dy, layer.x)
    args = (layer.x, layer.router, layer.bias, *layer.w)
    with pytest.raises(ValueError, match="logits"):
        moe.layer_forward(moe.LayerBuffers(layer.p, "cuda", keep_logits=False), *args, rule=layer.rule)
    with pytest.raises(ValueError, match="remapping"):
        moe.layer_forward(moe.LayerBuffers(layer.p, "cuda", remap_rounds=1), *args, rule=layer.rule)
    with pytest.raises(ValueError, match="wants a rule"):
        moe.layer_forward(layer.buf, *args, select_bias=layer.bias)


# ------------------------------------------------------------------------ a training step

def test_training_step_from_norm_to_norm():
    """n = norm(x); y = layer(n); z, m = x + a norm(y), norm(z), and back: every stage against its form
    in 64 bits on what the stage before left; then as one captured step, replayed to the same bits."""
    T, d, E, k = 260, 256, 16, 4
    layer = Layer(T, d, E, k, 128, moe.RouteRule(SIG, 4, 2, 2, True, 2.5), True)
    gen = torch.Generator().manual_seed(1)
    x = (randn(gen, T, d) * 2).cuda()
    wn, wp, wm = ((1 + 0.2 * randn(gen, d)).cuda() for _ in range(3))
    a = randn(gen, d).cuda()
    dz, dm = randn(gen, T, d).cuda(), randn(gen, T, d).to(BF).cuda()
    new = lambda *s, t=F32: torch.full(s, np.nan, dtype=t, device="cuda")  # noqa: E731
    n, z, m = new(T, d, t=BF), new(T, d), new(T, d, t=BF)
    dy, dx1, dx = new(T, d, t=BF), new(T, d), new(T, d)
    da, dwp, dwm, dwn = (new(d) for _ in range(4))
    kind = moe.MOE_GATE_CHANNEL
    ws = [torch.empty(moe.moe_block_norm_backward_workspace_size(T, d, g), dtype=torch.uint8, device="cuda")
          for g in (kind, moe.MOE_GATE_NONE)]
    before = (T, d, moe.MOE_F32, moe.MOE_BF16, EPS, 1.0, x, None, 0, False, None, False, None, wn)

    def step():
        moe.moe_block_norm(*before, None, n)
        y = layer.forward(n)
        after = (T, d, moe.MOE_F32, moe.MOE_BF16, EPS, SCALE, x, y, kind, True, a, True, wp, wm)
        moe.moe_block_norm(*after, z, m)
        moe.moe_block_norm_backward(*after, dz, moe.MOE_BF16, dm, dx1, dy, da, dwp, dwm, ws[0])
        dn = layer.backward(dy, n)
        moe.moe_block_norm_backward(*before, dx1, moe.MOE_F32, dn, dx, None, None, None, dwn, ws[1])

    step()
    torch.cuda.synchronize()
    outs = (n, layer.buf.y, z, m, dx1, dy, da, dwp, dwm, layer.buf.dx, dx, dwn)
    want = [o.clone() for o in outs]
    X = Rounded(f64(x))
    r = (((X * X).sum(-1, True)) * (1.0 / d) + EPS).rsqrt()
    (X * r * f64(wn)).close(f64(n), LAST[BF], "n")
    layer.check(n, dy)
    case = (T, d, F32, BF, "channel", True, True)
    _, _, _, zz, _, mm = formed(case, x, layer.buf.y, a, wp, wm)
    zz.close(f64(z), U, "z")
    mm.close(f64(m), LAST[BF], "m")
    g = grads_of(case, x, layer.buf.y, a, wp, wm, dz, dm)
    for name, got, last in (("dx", dx1, U), ("dy", dy, LAST[BF]), ("dgate", da, U), ("dw_post", dwp, U),
                            ("dw_pre", dwm, U)):
        g[name].close(f64(got), last, name)
    dn = Rounded(f64(layer.buf.dx))
    mean = (dn * f64(wn) * X).sum(-1, True) * (1.0 / d) * r * r
    (Rounded(f64(dx1)) + r * (dn * f64(wn) - mean * X)).close(f64(dx), U, "dx")
    (dn * (X * r)).sum(0).close(f64(dwn), U, "dw_pre")

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


# ------------------------------------------------------------------------ 4-bit experts

# T, d, E, k, F, group, zeros, experts used (None: any)
W4 = [(1, d, 6, 3, F, group, zeros, None)
      for group in (32, 64, 128) for zeros in (False, True)
      for d, F in ((128, 1152), (2560, 128), (1152, 640))] + [
    (1, 64, 2, 2, 64, 32, True, 1),       # the same expert twice
    (4, 128, 7, 6, 192, 64, True, 3),     # 8 tokens and fewer, experts more than once in a token
    (8, 2560, 3, 3, 64, 32, False, 2),
    (8, 64, 200, 32, 704, 64, False, None),
    (9, 128, 1024, 32, 64, 32, True, None),   # few rows to an expert
    (40, 192, 64, 6, 128, 64, True, 3),       # ... of many, on three of them
    (41, 128, 64, 6, 256, 128, False, 5),
    (300, 64, 7, 3, 64, 32, False, None),
]


@pytest.mark.parametrize("case", W4, ids=[str(i) for i in range(len(W4))])
def test_w4_expert_ffn(case):
    w, x, idx, gate = w4_case(case, 7)
    check_w4(case, w, x, idx, gate, run_w4(case, w, x, idx, gate))


def test_w4_most_slots():
    case = (512, 64, 33, 32, 64, 32, True, None)
    w, x, idx, gate = w4_case(case)
    check_w4(case, w, x, idx, gate, run_w4(case, w, x, idx, gate))


@pytest.mark.parametrize("T", [1, 5, 20, 100])
def test_w4_values_of_all_sizes(T):
    """Rows of zeros, of small values and of all sizes, and single large ones among small; a row with a
    value that is not finite leaves the others as they are."""
    case = (T, 256, 6, 2, 128, 64, True, None)
    w, x, idx, gate = w4_case(case)
    for t in range(T):
        if t % 5 == 1:
            x[t, 100] = 3000.0
        elif t % 5 == 2:
            x[t] = 0
        elif t % 5 == 3:
            x[t] *= 2.0 ** -100
        elif t % 5 == 4:
            x[t] *= 2.0 ** torch.randint(-40, 1, (256,), generator=torch.Generator().manual_seed(t))
    y = run_w4(case, w, x, idx, gate)
    check_w4(case, w, x, idx, gate, y)
    for bad in (np.nan, np.inf, -np.inf):
        broken = x.clone()
        broken[T // 2, 17] = bad
        got = run_w4(case, w, broken, idx, gate)
        assert got[T // 2].isnan().all()
        rest = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(got[rest], y[rest])


def test_w4_sizes_one_after_another_in_one_workspace():
    """A workspace that calls of other sizes left as it is; every call gives the same bits again."""
    cases = [(1, 128, 20, 8, 192, 64, True, None), (6, 128, 20, 3, 192, 64, True, None),
             (30, 128, 20, 2, 192, 64, True, None), (100, 128, 20, 4, 192, 64, True, 5)]
    w = w4_case(cases[0])[0]
    packed = [moe.W4Weights(*(t.cuda() for t in m)) for m in w]
    inputs = [[t.cuda() for t in w4_case(c)[1:]] for c in cases]
    problems = [moe.Problem(*c[:5]) for c in cases]
    ws = torch.full((max(moe.moe_w4_expert_ffn_workspace_size(p) for p in problems),), 255,
                    dtype=torch.uint8, device="cuda")
    ys = [torch.empty(c[:2], dtype=BF, device="cuda") for c in cases]
    first = None
    for _ in range(20):
        for p, (x, idx, gate), y in zip(problems, inputs, ys):
            moe.moe_w4_expert_ffn(p, x, idx, gate, *packed, y, ws)
        if first is None:
            first = [y.clone() for y in ys]
            for c, x, y in zip(cases, inputs, first):
                check_w4(c, w, *(t.cpu() for t in x), y)
        assert all(torch.equal(a, b) for a, b in zip(first, ys))


def test_calls_side_by_side():
    """Two streams with what is theirs, and two graphs that share a workspace, one after the other."""
    cases = [(1, 512, 40, 8, 256, 64, True, None), (12, 512, 40, 8, 256, 64, True, None)]
    w = w4_case(cases[0])[0]
    packed = [moe.W4Weights(*(t.cuda() for t in m)) for m in w]
    inputs = [[t.cuda() for t in w4_case(c)[1:]] for c in cases]
    problems = [moe.Problem(*c[:5]) for c in cases]
    size = [moe.moe_w4_expert_ffn_workspace_size(p) for p in problems]
    ys = [torch.empty(c[:2], dtype=BF, device="cuda") for c in cases]
    own = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in size]

    def call(i, ws):
        moe.moe_w4_expert_ffn(problems[i], *inputs[i], *packed, ys[i], ws)

    for i in range(2):
        call(i, own[i])
    torch.cuda.synchronize()
    want = [y.clone() for y in ys]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    call(i, own[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, ys))
    shared = torch.empty(max(size), dtype=torch.uint8, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            call(i, shared)
    for _ in range(5):
        for y in ys:
            y.zero_()
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, ys))


def test_routing_and_norms_on_streams_of_their_own():
    """The same bits, whichever stream and however many times."""
    T, E, k, D = 500, 896, 16, 1024
    gen = torch.Generator().manual_seed(3)
    logits, bias = randn(gen, T, E).cuda(), (randn(gen, E) * 0.05).cuda()
    x, y, dz = (randn(gen, T, D).to(BF).cuda() for _ in range(3))
    wp, wn = ((1 + 0.2 * randn(gen, D)).cuda() for _ in range(2))
    dgate = randn(gen, T, k).cuda()
    rule = moe.RouteRule(SIG, 8, 4, 2, True, 2.5)
    new = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    size = moe.moe_block_norm_backward_workspace_size(T, D, 0)
    torch.cuda.synchronize()

    def all_of():
        idx, gate, partials, dl = new(T, k, t=torch.int32), new(T, k), new((T + 7) // 8, E), new(T, E)
        moe.moe_route_select(T, E, k, rule, 1, logits, bias, idx, gate, partials)
        moe.moe_route_select_backward(T, E, k, rule, 1, logits, idx, dgate, dl, None)
        z, n, dx, dy = (new(T, D, t=BF) for _ in range(4))
        dwp, dwn, ws = new(D), new(D), new(size, t=torch.uint8)
        head = (T, D, 0, 0, EPS, SCALE, x, y, 0, False, None, True, wp, wn)
        moe.moe_block_norm(*head, z, n)
        moe.moe_block_norm_backward(*head, dz, 0, n, dx, dy, None, dwp, dwn, ws)
        return idx, gate, partials, dl, z, n, dx, dy, dwp, dwn

    want = all_of()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams * 5:
        with torch.cuda.stream(s):
            got.append(all_of())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
