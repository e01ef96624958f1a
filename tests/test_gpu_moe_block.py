"""GPU parity of what stands around the experts against the fp64 oracle: routing by scores, the norms
around a block, the experts with 4-bit weights, and a run of them together.

Tolerances: selected experts are equal; values are within the bound of rounding.Rounded, carried
through the kernels' formulas, and the last rounding to their type."""

import numpy as np
import pytest
import torch

from oracle import moe_block as MB
from parity_util import f64
from rounding import Rounded, U
from top_routing_grouped_gemm_gb300 import moe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CODE = {BF: moe.MOE_BF16, F32: moe.MOE_F32}
LAST = {BF: 2.0 ** -8, F32: U}
SIG, SOFT = moe.MOE_SCORE_SIGMOID, moe.MOE_SCORE_SOFTMAX


def randn(gen, *shape):
    return torch.randn(shape, generator=gen)


# ------------------------------------------------------------------------ routing

# T, E, k, score, groups, kept, best, renormalise, bias, dtype
ROUTES = [
    (1, 1, 1, SIG, 1, 1, 1, True, False, F32),
    (1, 896, 16, SIG, 8, 4, 2, True, True, F32),
    (1, 1024, 32, SOFT, 32, 17, 1, False, True, F32),
    (7, 5, 5, SOFT, 5, 5, 1, True, False, BF),
    (8, 64, 4, SOFT, 1, 1, 1, True, False, F32),
    (9, 100, 6, SOFT, 10, 3, 1, False, False, BF),
    (17, 60, 8, SIG, 3, 2, 2, False, True, F32),
    (33, 1020, 31, SIG, 17, 9, 2, True, True, BF),
    (40, 33, 32, SIG, 1, 1, 1, True, True, F32),
    (65, 1005, 10, SOFT, 5, 2, 2, True, False, F32),
    (129, 896, 16, SOFT, 1, 1, 1, True, True, F32),
    (130, 9, 2, SIG, 9, 4, 1, True, True, BF),
    (1000, 256, 8, SIG, 8, 4, 2, True, True, F32),
    (300, 896, 16, SIG, 8, 4, 2, True, False, BF),
    (64, 128, 8, SIG, 16, 16, 2, True, False, F32),
    (70, 1023, 3, SIG, 31, 5, 2, False, True, F32),
]


def rule_of(case):
    return moe.RouteRule(case[3], case[4], case[5], case[6], case[7], 2.5)


def run_select(case, logits, bias, rule=None):
    T, E, k = case[:3]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    gate, partials = (torch.full(s, np.nan, device="cuda") for s in ((T, k), ((T + 7) // 8, E)))
    moe.moe_route_select(T, E, k, rule or rule_of(case), CODE[case[-1]], logits, bias, idx, gate,
                         partials)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), f64(gate), f64(partials)


def gates_of(case, logits, idx, renormalise=True):
    """Gates and shares of all experts as the kernel forms them, with their errors."""
    sigmoid = case[3] == SIG
    l = Rounded(logits)
    if sigmoid:
        s = l.sigmoid()
    else:
        s = (l - logits.max(-1, keepdims=True)).exp()
    total = s.sum(-1, keepdims=True)
    share = s / total
    if not sigmoid:
        s = share
    pick = lambda r: Rounded(np.take_along_axis(r.v, idx, 1),  # noqa: E731
                             np.take_along_axis(r.e, idx, 1))
    if renormalise:
        if not sigmoid:  # from the selected logits alone
            chosen = np.take_along_axis(logits, idx, 1)
            picked = (Rounded(chosen) - chosen.max(-1, keepdims=True)).exp()
        else:
            picked = pick(s)
        w = picked / picked.sum(-1, keepdims=True)
    else:
        w = pick(s)
    return w, share, pick(s)


@pytest.mark.parametrize("case", ROUTES, ids=[str(i) for i in range(len(ROUTES))])
@pytest.mark.parametrize("layout", ["dense", "columns", "shared"])
def test_route_select(case, layout):
    T, E, k, score, groups, kept, best, renormalise, with_bias, dtype = case
    gen = torch.Generator().manual_seed(T * 1000 + E)
    if layout == "columns":
        logits = randn(gen, T, E + 3).to(dtype).cuda()[:, 1:E + 1]
    elif layout == "shared":
        logits = randn(gen, 1, E).to(dtype).cuda().expand(T, E)
    else:
        logits = randn(gen, T, E).to(dtype).cuda()
    std = 0.05 if score == SIG else 0.3 / E
    bias = (randn(gen, E) * std).cuda() if with_bias else None
    idx, gate, partials = run_select(case, logits, bias)
    l = f64(logits)
    ref_idx, ref_gate, ref_partials = MB.select(l, f64(bias), k, score == SIG, groups, kept, best,
                                                renormalise, 2.5)
    assert np.array_equal(idx, ref_idx)
    w, share, _ = gates_of(case, l, ref_idx, renormalise)
    (w * 2.5).close(gate, what="gate")
    assert np.allclose((w * 2.5).v, ref_gate, rtol=1e-12)
    for b in range(len(partials)):
        rows = slice(8 * b, 8 * b + 8)
        Rounded(share.v[rows], share.e[rows]).sum(0).close(partials[b], what="partials")
    assert np.allclose(ref_partials.sum(-1), np.minimum(8, T - 8 * np.arange(len(partials))))


def test_route_select_without_partials_and_repeated():
    case = ROUTES[12]
    gen = torch.Generator().manual_seed(5)
    logits, bias = randn(gen, *case[:2]).cuda(), (randn(gen, case[1]) * 0.05).cuda()
    want = run_select(case, logits, bias)
    T, E, k = case[:3]
    idx, gate = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    for _ in range(3):
        moe.moe_route_select(T, E, k, rule_of(case), moe.MOE_F32, logits, bias, idx, gate, None)
    assert np.array_equal(idx.cpu().numpy(), want[0]) and np.array_equal(f64(gate), want[1])


def near_ties(score, T, E, gen):
    """Logits and a bias whose sums with the scores are nearly, but not quite, all equal: the order is
    decided far behind the 24 bits of fp32, and is known from sums in 64 bits."""
    l = randn(gen, T, E)
    bias = randn(gen, E) * 0.01
    for _ in range(4):  # logits that take score + bias to one value, as near as fp32 logits do
        if score == SIG:
            l = torch.logit((0.6 - bias.double()).clamp(0.05, 0.95)).float().expand(T, E).clone()
    step = torch.randint(-2, 3, (T, E), generator=gen)
    return (l.view(torch.int32) + step.to(torch.int32)).view(torch.float32), bias


@pytest.mark.parametrize("groups, kept, best", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_route_select_of_nearly_equal_scores(groups, kept, best):
    """Order beyond fp32.  What is closer than 2^-40 may be in either order: such pairs are left out of
    the comparison, and there are few."""
    T, E, k = 64, 256, 16
    case = (T, E, k, SIG, groups, kept, best, True, True, F32)
    gen = torch.Generator().manual_seed(11)
    l, bias = near_ties(SIG, T, E, gen)
    idx, _, _ = run_select(case, l.cuda(), bias.cuda())
    import decimal
    decimal.getcontext().prec = 40
    D = decimal.Decimal
    tie = 2.0 ** -40
    skipped = 0
    for t in range(T):
        c = [1 / (1 + (-D(v)).exp()) + D(b) for v, b in zip(l[t].tolist(), bias.tolist())]
        spread = float(max(c) - min(c))
        assert spread < 1e-6  # all within a few fp32 steps
        gs = E // groups
        worth = [sum(sorted(c[g * gs:(g + 1) * gs])[::-1][:best]) for g in range(groups)]
        order = sorted(range(groups), key=lambda g: (-worth[g], g))
        if groups > 1 and kept < groups and worth[order[kept - 1]] - worth[order[kept]] < D(tie):
            skipped += 1
            continue
        may = [e for e in range(E) if groups == 1 or e // gs in order[:kept]]
        want = sorted(may, key=lambda e: (-c[e], e))
        near = any(0 < c[want[j]] - c[want[j + 1]] < D(tie) for j in range(k))
        if near:
            skipped += 1
            continue
        assert idx[t].tolist() == want[:k], t
    assert skipped <= T // 4


def test_route_select_of_equal_logits():
    """Ties go to the lower index, of experts and of groups, with and without a bias."""
    T, E, k = 5, 96, 8
    for bias in (None, torch.zeros(E), torch.full((E,), 0.125)):
        for groups, kept in ((1, 1), (8, 2)):
            for score in (SIG, SOFT):
                case = (T, E, k, score, groups, kept, 2, True, True, F32)
                l = torch.zeros((T, E))
                l[1, 50:] = 1
                l[2, ::7] = -1
                idx, gate, _ = run_select(case, l.cuda(), None if bias is None else bias.cuda())
                want, ref, _ = MB.select(f64(l), f64(bias), k, score == SIG, groups, kept, 2, True, 2.5)
                assert np.array_equal(idx, want)
                assert np.allclose(gate, ref, rtol=1e-6)


def test_route_select_masked_and_extreme():
    inf, nan = float("inf"), float("nan")
    E, k = 40, 4
    l = torch.full((8, E), -inf)
    l[1, 7] = 0.5                    # one expert left
    l[2] = torch.linspace(-200, -100, E)   # scores that vanish in fp32
    l[3] = nan
    l[3, 5], l[3, 6] = 1.0, 2.0
    l[4] = torch.linspace(-3e38, 3e38, E)
    l[5, 3], l[5, 9] = inf, 1.0
    l[6] = torch.linspace(30, 34, E)  # scores within 1e-13 of 1
    l[7] = -88.0 - torch.arange(E) / 4
    for bias in (None, torch.linspace(-0.1, 0.1, E)):
        if bias is not None:
            bias[2], bias[30], bias[31] = -inf, inf, nan
        for score in (SIG, SOFT):
            for renormalise in (True, False):
                case = (8, E, k, score, 1, 1, 1, renormalise, True, F32)
                idx, gate, partials = run_select(case, l.cuda(), None if bias is None else bias.cuda())
                # +inf makes a row's softmax scores NaN (the differences of row 4's limits overflow
                # too: it has infinities)
                rows = [r for r in range(8) if score == SIG or not (l[r] == inf).any()]
                if bias is not None and score == SIG:
                    rows.remove(6)  # closer than 2^-40
                want, ref, part = MB.select(f64(l), f64(bias), k, score == SIG, 1, 1, 1, renormalise, 2.5)
                assert np.array_equal(idx[rows], want[rows]), (score, bias)
                for row in idx:
                    assert len(set(row.tolist())) == k and row.min() >= 0 and row.max() < E
                # exp(l - max): the difference's own rounding, |l - max| 2^-24, and a few more
                # (nothing of it below fp32's normal numbers)
                assert np.allclose(gate[rows], ref[rows], rtol=200 * U, atol=2.0 ** -126 * 2.5)
                if score == SIG:
                    assert np.allclose(partials, part, rtol=1e-5)


@pytest.mark.parametrize("case", ROUTES, ids=[str(i) for i in range(len(ROUTES))])
def test_route_select_backward(case):
    T, E, k, score, groups, kept, best, renormalise, with_bias, dtype = case
    gen = torch.Generator().manual_seed(T * 1000 + E + 1)
    logits = randn(gen, T, E + 5).to(dtype).cuda()[:, 2:E + 2]
    dgate = randn(gen, T, k).cuda()
    idx = torch.rand((T, E), generator=gen).argsort(1)[:, :k].to(torch.int32).cuda()
    dl = torch.full((T, E), np.nan, dtype=dtype, device="cuda")
    sparse = None
    if score == SIG or renormalise:
        sparse = torch.full((T, k), np.nan, device="cuda")
    moe.moe_route_select_backward(T, E, k, rule_of(case), CODE[dtype], logits, idx, dgate, dl, sparse)
    l, i, d = f64(logits), idx.cpu().numpy().astype(np.int64), Rounded(f64(dgate)) * 2.5
    w, share, s = gates_of(case, l, i, renormalise)
    one_less = Rounded(-np.take_along_axis(l, i, 1)).sigmoid()
    full = Rounded(np.zeros((T, E)))
    if renormalise:
        v = w * (d - (w * d).sum(-1, keepdims=True))
        v = v * one_less if score == SIG else v
    elif score == SIG:
        v = s * one_less * d
    else:
        dot = (s * d).sum(-1, keepdims=True)
        full = -(share * dot)
        v = s * (d - dot) + s * dot * 0.0  # formed as s d - s dot: both of their sizes
        v = Rounded(v.v, v.e + U * 4 * (np.abs((s * d).v) + np.abs((s * dot).v)))
    value, error = full.v.copy(), full.e.copy()
    np.put_along_axis(value, i, v.v, 1)
    np.put_along_axis(error, i, v.e, 1)
    Rounded(value, error).close(f64(dl), LAST[dtype], "dlogits")
    if sparse is not None:
        v.close(f64(sparse), what="dlogits_topk")
    ref = MB.select_backward(l, i, f64(dgate), score == SIG, renormalise, 2.5)
    assert np.allclose(value, ref, rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("score, renormalise", [(SIG, True), (SIG, False), (SOFT, True), (SOFT, False)])
def test_route_select_backward_of_repeated_and_bad_experts(score, renormalise):
    T, E, k = 11, 50, 6
    gen = torch.Generator().manual_seed(3)
    logits, dgate = randn(gen, T, E).cuda(), randn(gen, T, k).cuda()
    idx = torch.randint(0, 4, (T, k), generator=gen).to(torch.int32)
    idx[2, 3], idx[4, 0], idx[5] = -1, E, 2 ** 31 - 1
    dl, status = torch.empty((T, E), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rule = moe.RouteRule(score, renormalise=renormalise, scale=2.5)
    moe.moe_route_select_backward(T, E, k, rule, moe.MOE_F32, logits, idx.cuda(), dgate, dl, None, status)
    ref = MB.select_backward(f64(logits), idx.numpy().astype(np.int64), f64(dgate), score == SIG,
                             renormalise, 2.5)
    # sums of k terms of up to 2.5 x 4, each formed in a handful of roundings
    assert np.abs(f64(dl) - ref).max() < 64 * U * 10 * k
    assert int(status.item()) == 6


# ------------------------------------------------------------------------ norms around a block

# N, D, stream, dtype, gate, sigmoid, post, w_post, w_pre, layout
NORMS = [
    (1, 8, BF, BF, "none", False, True, True, True, "dense"),
    (1, 4096, BF, BF, "token", True, True, True, True, "dense"),
    (3, 256, F32, F32, "value", True, True, True, True, "columns"),
    (5, 264, F32, BF, "channel", False, True, False, True, "columns"),
    (9, 512, BF, BF, "channel", True, False, False, False, "dense"),
    (17, 1000, F32, F32, "value", False, True, True, False, "columns"),
    (2, 1032, F32, BF, "token", False, True, True, True, "dense"),
    (33, 2048, BF, BF, "value", True, True, True, True, "columns"),
    (4, 2056, F32, BF, "none", False, False, False, True, "columns"),
    (700, 72, F32, F32, "channel", True, True, True, True, "dense"),
    (1300, 1024, BF, BF, "token", True, True, True, True, "columns"),
    (7, 4104, F32, BF, "channel", True, True, True, True, "dense"),
    (6, 8192, BF, BF, "token", True, True, True, True, "dense"),
    (300, 5000, F32, BF, "value", True, True, True, True, "columns"),
    (310, 6144, BF, BF, "channel", True, True, True, True, "dense"),
    (2, 6152, F32, F32, "token", True, True, True, True, "dense"),
    (3, 8200, F32, F32, "value", True, True, True, True, "dense"),
    (5, 16384, F32, BF, "channel", True, True, True, True, "columns"),
    (400, 4096, F32, BF, "token", True, True, True, True, "shared"),
]
KIND = {"none": moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL, "token": moe.MOE_GATE_TOKEN,
        "value": moe.MOE_GATE_VALUE}
EPS, SCALE = 1e-5, 0.7


def matrix(gen, N, D, dtype, layout, std=1.0):
    t = (randn(gen, N, D + 16) * std).to(dtype).cuda()
    if layout == "columns":
        return t[:, 8:D + 8]
    if layout == "shared":
        return t[:1, :D].contiguous().expand(N, D)
    return t[:, :D].contiguous()


def out_matrix(N, D, dtype, layout):
    t = torch.full((N, D + 16), np.nan, dtype=dtype, device="cuda")
    return t[:, 8:D + 8] if layout == "columns" else t[:, :D].contiguous()


def norm_inputs(case, seed=0):
    N, D, st, dt, gate, sigmoid, post, w_post, w_pre, layout = case
    gen = torch.Generator().manual_seed(seed + N + D)
    x, y = matrix(gen, N, D, st, layout, 2.0), matrix(gen, N, D, dt, layout)
    if N > 4:
        if layout == "dense":
            y[1], x[2] = 0, 0
            y[3] *= 1000
    a = {"none": lambda: None, "channel": lambda: randn(gen, D).cuda(),
         "token": lambda: randn(gen, N).cuda(),
         "value": lambda: matrix(gen, N, D, dt, layout)}[gate]()
    wp = (1 + 0.2 * randn(gen, D)).cuda() if w_post else None
    wn = (1 + 0.2 * randn(gen, D)).cuda() if w_pre else None
    return x, y, a, wp, wn, gen


def formed(case, x, y, a, wp, wn):
    """The forward as the kernel forms it: y's rstd, u, a, z, z's rstd, n."""
    gate, sigmoid, post = case[4:7]
    X, Y = Rounded(f64(x)), Rounded(f64(y))
    ry = (((Y * Y).sum(-1, True)) * (1.0 / case[1]) + EPS).rsqrt() if post else None
    u = Y * ry if post else Y
    u = u * f64(wp) if wp is not None else u
    A = None
    if a is not None:
        A = Rounded(f64(a))
        A = A.sigmoid() if sigmoid else A
        if gate == "token":
            A = Rounded(A.v[:, None], A.e[:, None])
    f = u * SCALE if A is None else A * SCALE * u
    z = X + f
    rz = (((z * z).sum(-1, True)) * (1.0 / case[1]) + EPS).rsqrt()
    n = z * rz
    return ry, u, A, z, rz, n * f64(wn) if wn is not None else n


@pytest.mark.parametrize("case", NORMS, ids=[str(i) for i in range(len(NORMS))])
def test_block_norm(case):
    N, D, st, dt, gate, sigmoid, post = case[:7]
    layout = case[-1]
    x, y, a, wp, wn, _ = norm_inputs(case)
    z, n = out_matrix(N, D, st, layout), out_matrix(N, D, dt, layout)
    moe.moe_block_norm(N, D, CODE[st], CODE[dt], EPS, SCALE, x, y, KIND[gate], sigmoid, a, post, wp,
                       wn, z, n)
    _, _, _, Z, _, M = formed(case, x, y, a, wp, wn)
    Z.close(f64(z), LAST[st], "z")
    M.close(f64(n), LAST[dt], "n")
    spread = a if gate != "token" else a[:, None]
    ref = MB.block_norm(f64(x), f64(y), f64(spread), sigmoid, post, f64(wp), f64(wn), SCALE, EPS)
    assert np.allclose(Z.v, ref[0], rtol=1e-12) and np.allclose(M.v, ref[1], rtol=1e-12)


@pytest.mark.parametrize("st, dt", [(BF, BF), (F32, BF), (F32, F32)])
def test_block_norm_in_place_and_in_parts(st, dt):
    """z over x and n over y; no norm before the next block; no block before."""
    case = (37, 512, st, dt, "token", True, True, True, True, "dense")
    N, D = case[:2]
    x, y, a, wp, wn, _ = norm_inputs(case)
    z, n = torch.empty_like(x), torch.empty_like(y)
    args = (N, D, CODE[st], CODE[dt], EPS, SCALE)
    moe.moe_block_norm(*args, x, y, KIND["token"], True, a, True, wp, wn, z, n)
    only_z = torch.empty_like(x)
    moe.moe_block_norm(*args, x, y, KIND["token"], True, a, True, wp, None, only_z, None)
    assert torch.equal(only_z, z)
    only_n, copy = torch.empty_like(y), torch.empty_like(x)
    moe.moe_block_norm(*args, x, None, 0, False, None, False, None, wn, None, only_n)
    moe.moe_block_norm(*args, x, None, 0, False, None, False, None, wn, copy, n2 := torch.empty_like(y))
    assert torch.equal(only_n, n2) and torch.equal(copy, x)
    X = Rounded(f64(x))
    r = (((X * X).sum(-1, True)) * (1.0 / D) + EPS).rsqrt()
    (X * r * f64(wn)).close(f64(only_n), LAST[dt], "n of x")
    moe.moe_block_norm(*args, x, y, KIND["token"], True, a, True, wp, wn, x, y)
    assert torch.equal(x, z) and torch.equal(y, n)


def grads_of(case, x, y, a, wp, wn, dz, dn):
    """The backward as the kernel forms it."""
    gate, sigmoid, post = case[4:7]
    D = case[1]
    ry, u, A, z, rz, _ = formed(case, x, y, a, wp, wn)
    total = Rounded(np.zeros(z.v.shape) if dz is None else f64(dz))
    out = {}
    if dn is not None:
        d = Rounded(f64(dn))
        out["dw_pre"] = (d * (z * rz)).sum(0)
        wd = d * f64(wn) if wn is not None else d
        m = (wd * z).sum(-1, True) * (1.0 / D) * rz * rz
        total = total + rz * (wd - m * z)
    out["dx"] = total
    d = total * SCALE
    da = d * u
    t = d if A is None else d * A
    if A is not None:
        if gate == "token":
            da = da.sum(-1, True)
        da = da * (A * (1.0 - A)) if sigmoid else da
        if gate == "channel":
            da = da.sum(0)
        out["dgate"] = da
    Y = Rounded(f64(y))
    if post:
        out["dw_post"] = (t * (Y * ry)).sum(0)
        wt = t * f64(wp) if wp is not None else t
        m = (wt * Y).sum(-1, True) * (1.0 / D) * ry * ry
        out["dy"] = ry * (wt - m * Y)
    else:
        out["dy"] = t
    return out


@pytest.mark.parametrize("which", ["both", "dz", "dn", "dn_f32"])
@pytest.mark.parametrize("case", NORMS, ids=[str(i) for i in range(len(NORMS))])
def test_block_norm_backward(case, which):
    N, D, st, dt, gate, sigmoid, post, w_post, w_pre, layout = case
    x, y, a, wp, wn, gen = norm_inputs(case)
    gt = F32 if which == "dn_f32" else dt
    lay = "dense" if layout == "shared" else layout
    dz = None if which == "dn" else matrix(gen, N, D, st, lay)
    dn = None if which == "dz" else matrix(gen, N, D, gt, lay)
    dx, dy = out_matrix(N, D, st, lay), out_matrix(N, D, dt, lay)
    dg = None
    if a is not None:
        dg = out_matrix(N, D, dt, lay) if gate == "value" else torch.full_like(a, np.nan)
    dwp = torch.full((D,), np.nan, device="cuda") if post else None
    dwn = torch.full((D,), np.nan, device="cuda")
    ws = torch.empty(moe.moe_block_norm_backward_workspace_size(N, D, KIND[gate]), dtype=torch.uint8,
                     device="cuda")
    head = (N, D, CODE[st], CODE[dt], EPS, SCALE, x, y, KIND[gate], sigmoid, a, post, wp, wn)
    moe.moe_block_norm_backward(*head, dz, CODE[gt], dn, dx, dy, dg, dwp, dwn, ws)
    got = dict(dx=dx, dy=dy, dgate=dg, dw_post=dwp, dw_pre=dwn)
    want = grads_of(case, x, y, a, wp, wn, dz, dn)
    types = dict(dx=st, dy=dt, dgate=dt if gate == "value" else F32, dw_post=F32, dw_pre=F32)
    for name, w in want.items():
        w.close(f64(got[name]).reshape(w.v.shape), LAST[types[name]], name)
    if dn is None:
        assert not dwn.any()
    spread = a if gate != "token" else a[:, None]
    ref = MB.block_norm_backward(f64(x), f64(y), f64(spread), sigmoid, post, f64(wp), f64(wn), SCALE,
                                 EPS, f64(dz), f64(dn))
    if a is not None:
        axis = {"token": (1,), "channel": (0,), "value": ()}[gate]
        ref["dgate"] = ref["da"].sum(axis, keepdims=True)
    for name, w in want.items():
        r = ref[name].reshape(w.v.shape)
        assert np.allclose(w.v, r, rtol=1e-9, atol=1e-9 * np.abs(r).max()), name
    # over the gradients that came in, without the workspace where no sum over rows is wanted
    dz2 = None if dz is None else dz.clone()
    into = dx.clone() if dz2 is None else dz2
    yy = y.clone() if layout != "shared" else torch.empty_like(dy)
    if layout != "shared":
        dg2 = None if gate == "channel" or dg is None else torch.empty_like(dg)
        moe.moe_block_norm_backward(N, D, CODE[st], CODE[dt], EPS, SCALE, x, yy, KIND[gate], sigmoid,
                                    a, post, wp, wn, dz2, CODE[gt], dn, into, yy, dg2, None, None, None)
        assert torch.equal(into, dx) and torch.equal(yy, dy)
        if dg2 is not None:
            assert torch.equal(dg2, dg)


def test_block_norm_backward_without_a_block():
    N, D = 19, 1000
    gen = torch.Generator().manual_seed(2)
    x, dz, dn = (randn(gen, N, D).cuda() for _ in range(3))
    wn = (1 + 0.2 * randn(gen, D)).cuda()
    dx, dwn = torch.empty_like(x), torch.empty(D, device="cuda")
    ws = torch.empty(moe.moe_block_norm_backward_workspace_size(N, D, 0), dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_backward(N, D, 1, 1, EPS, 1.0, x, None, 0, False, None, False, None, wn, dz, 1, dn,
                                dx, None, None, None, dwn, ws)
    X, d = Rounded(f64(x)), Rounded(f64(dn))
    r = (((X * X).sum(-1, True)) * (1.0 / D) + EPS).rsqrt()
    m = (d * f64(wn) * X).sum(-1, True) * (1.0 / D) * r * r
    (Rounded(f64(dz)) + r * (d * f64(wn) - m * X)).close(f64(dx), U, "dx")
    (d * (X * r)).sum(0).close(f64(dwn), U, "dw_pre")


# ------------------------------------------------------------------------ 4-bit experts

def w4_weights(gen, E, rows, cols, group, zeros):
    codes = torch.randint(0, 256, (E, rows, cols // 2), generator=gen).to(torch.uint8)
    scales = ((torch.rand((E, rows, cols // group), generator=gen) + 0.5) * 0.3 * cols ** -0.5).to(BF)
    z = torch.randint(0, 16, scales.shape, generator=gen).to(torch.uint8) if zeros else None
    return codes, scales, z


# T, d, E, k, F, group, zeros, experts used (None: any)
W4 = [
    (1, 64, 1, 1, 64, 32, False, None),
    (1, 128, 8, 8, 128, 128, True, None),
    (1, 448, 20, 3, 64, 64, False, None),
    (2, 64, 3, 2, 192, 32, True, None),
    (7, 512, 16, 4, 256, 32, False, None),
    (8, 192, 4, 3, 128, 64, True, None),
    (9, 256, 5, 2, 64, 64, False, None),
    (16, 128, 2, 2, 128, 128, True, None),
    (17, 320, 6, 6, 192, 64, True, None),
    (33, 128, 3, 2, 256, 128, False, 2),
    (70, 192, 2, 2, 64, 32, True, None),
    (150, 64, 12, 5, 128, 64, False, 3),
]


def w4_case(case, seed=0):
    T, d, E, k, F, group, zeros, used = case
    gen = torch.Generator().manual_seed(seed + T + d)
    w = [w4_weights(gen, E, *s, group, zeros) for s in ((F, d), (F, d), (d, F))]
    x = randn(gen, T, d).to(BF)
    if used:
        idx = torch.randint(0, used, (T, k), generator=gen).to(torch.int32)
    else:
        idx = torch.rand((T, E), generator=gen).argsort(1)[:, :k].to(torch.int32)
    return w, x, idx, torch.rand((T, k), generator=gen) + 0.1


def run_w4(case, w, x, idx, gate, status=None):
    T, d, E, k, F = case[:5]
    p = moe.Problem(T, d, E, k, F)
    packed = [moe.W4Weights(*(None if t is None else t.cuda() for t in m)) for m in w]
    ws = torch.full((moe.moe_w4_expert_ffn_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    y = torch.full((T, d), np.nan, dtype=BF, device="cuda")
    moe.moe_w4_expert_ffn(p, x.cuda(), idx.cuda(), gate.cuda(), *packed, y, ws, status)
    torch.cuda.synchronize()
    return y


# Sums on the tensor cores: exact products of a group are added in group / 16 steps of a few roundings
# each (counted as 4 of half a step, whether they round or cut off), times the scale, over cols / 512
# or so tiles a warp and 8 warps.  The products are those of the codes, zero times the sum of the values
# being taken off afterwards: the sizes of both count, not that of their difference.
def product_count(cols, group):
    return 4 * group / 16 + 2 * cols / 512 + 16


def w4_sizes(codes, scales, zeros):
    """(16 + code + 16 + zero) scale: what the sums of a product are made of."""
    code = MB.w4_values(codes, np.ones(scales.shape), np.zeros(scales.shape, np.uint8))
    group = code.shape[-1] // scales.shape[-1]
    zero = 8.0 if zeros is None else np.repeat(zeros.astype(float), group, -1)
    return (32 + code + zero) * np.repeat(scales, group, -1)


def check_w4(case, w, x, idx, gate, y):
    T, d, E, k, F, group = case[:6]
    W = [MB.w4_values(m[0].numpy(), f64(m[1]), None if m[2] is None else m[2].numpy()) for m in w]
    sizes = [w4_sizes(m[0].numpy(), f64(m[1]), None if m[2] is None else m[2].numpy()) for m in w]
    x, g, idx = f64(x), f64(gate), idx.numpy()
    value, error = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            a, b = (Rounded(W[i][e] @ x[t], product_count(d, group) * U * (sizes[i][e] @ np.abs(x[t])))
                    for i in (0, 1))
            h = a * a.sigmoid() * b
            h = Rounded(h.v, h.e + 2.0 ** -16 * np.abs(h.v))  # two pieces
            out = Rounded(W[2][e] @ h.v, np.abs(W[2][e]) @ h.e + 2 * product_count(F, group) * U * (
                np.abs(W[2][e]) @ np.abs(h.v)))
            part = out * g[t, j]
            value[t] += part.v
            error[t] += part.e + k * U * np.abs(part.v)
    Rounded(value, error).close(f64(y), LAST[BF], "y")
    assert np.allclose(value, MB.w4_expert_ffn(x, idx, g, *W), rtol=1e-9, atol=1e-9)


@pytest.mark.parametrize("case", W4, ids=[str(i) for i in range(len(W4))])
def test_w4_expert_ffn(case):
    w, x, idx, gate = w4_case(case)
    check_w4(case, w, x, idx, gate, run_w4(case, w, x, idx, gate))


def test_w4_bad_experts_and_repeated_ones():
    case = (10, 128, 6, 4, 64, 32, True, None)
    w, x, idx, gate = w4_case(case)
    idx[0] = -1                      # nothing left of a token
    idx[1, 2], idx[2, 0] = 6, 2 ** 31 - 1
    idx[3] = 4                       # the same expert four times
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = run_w4(case, w, x, idx, gate, status)
    assert int(status.item()) == 6 and not y[0].any()
    check_w4(case, w, x, idx, gate, y)


def test_w4_packed_in_columns_order():
    """One weight at a time: each code, row and column arrives where it belongs."""
    E, d, F, group = 2, 128, 64, 64
    case = (1, d, E, 1, F, group, True, None)
    gen = torch.Generator().manual_seed(1)
    w = [w4_weights(gen, E, *s, group, True) for s in ((F, d), (F, d), (d, F))]
    for e in range(E):
        for col in (0, 1, 7, 8, 31, 32, 63, 64, 101, 127):
            x = torch.zeros((1, d), dtype=BF)
            x[0, col] = 2
            idx = torch.tensor([[e]], dtype=torch.int32)
            gate = torch.ones((1, 1))
            check_w4(case, w, x, idx, gate, run_w4(case, w, x, idx, gate))


# ------------------------------------------------------------------------ together

def test_graph_of_a_serving_step_replayed():
    """Norm, router, selection, 4-bit experts and the norm after as one captured step: replays on new
    inputs give the bits of plain calls, on a stream of its own."""
    T, d, E, k, F = 3, 256, 32, 4, 128
    gen = torch.Generator().manual_seed(9)
    p = moe.Problem(T, d, E, k, F)
    w = [moe.W4Weights(*(t.cuda() for t in w4_weights(gen, E, *s, 64, True)))
         for s in ((F, d), (F, d), (d, F))]
    router, bias = (randn(gen, E, d) * 0.05).cuda(), (randn(gen, E) * 0.02).cuda()
    wn, wp, wn2 = ((1 + 0.2 * randn(gen, d)).cuda() for _ in range(3))
    new = lambda *s, t=BF: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    x, n, y, z, n2 = (new(T, d) for _ in range(5))
    logits, idx, gate = new(T, E, t=F32), new(T, k, t=torch.int32), new(T, k, t=F32)
    token = randn(gen, T).cuda()
    ws_r = new(moe.moe_route_workspace_size(p), t=torch.uint8)
    ws = new(moe.moe_w4_expert_ffn_workspace_size(p), t=torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rule = moe.RouteRule(SIG, 4, 2, 2, True, 2.5)

    def step():
        moe.moe_block_norm(T, d, 0, 0, EPS, 1.0, x, None, 0, False, None, False, None, wn, None, n)
        moe.moe_route_logits(p, n, router, None, logits, ws_r, status)
        moe.moe_route_select(T, E, k, rule, moe.MOE_F32, logits, bias, idx, gate, None)
        moe.moe_w4_expert_ffn(p, n, idx, gate, *w, y, ws, status)
        moe.moe_block_norm(T, d, 0, 0, EPS, SCALE, x, y, moe.MOE_GATE_TOKEN, True, token, True, wp, wn2,
                           z, n2)

    outs = (n, logits, idx, gate, y, z, n2)
    inputs = [randn(gen, T, d).to(BF).cuda() for _ in range(3)]
    plain = []
    for i in inputs:
        x.copy_(i)
        step()
        plain.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i, want in zip(inputs * 2, plain * 2):
        x.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert int(status.item()) == 0
    # and the values: each operator against the oracle on what went into it
    ref_idx, ref_gate, _ = MB.select(f64(logits), f64(bias), k, True, 4, 2, 2, True, 2.5)
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    assert np.allclose(f64(gate), ref_gate, rtol=1e-5)
