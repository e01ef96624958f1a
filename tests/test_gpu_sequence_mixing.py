"""GPU parity of the operators beside the gated delta rule against the fp64 oracle: norm and
rotation of queries and keys, the gated linear recurrence, the single-token steps, and a run of
them together as a model uses them.

Tolerances.  U = 2^-24 is half an fp32 step; a result rounded to bf16 is off by at most 2^-8 of
itself.  Each check bounds the fp32 error of every value by U times a count of the roundings
that reach it, weighted with the sizes of the terms they act on (sums of absolute values, formed
in 64 bits beside the oracle), plus the last rounding."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import linear_attention as LA
from oracle import sequence_mixing as SM
from top_routing_grouped_gemm_gb300 import moe
from parity_util import f64, relerr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
CODE = {BF: moe.MOE_BF16, F32: moe.MOE_F32}
LAST = {BF: 2.0 ** -8, F32: U}  # the last rounding, relative


def close(got, ref, terms, dtype, what=""):
    """|got - ref| <= U terms + the last rounding, value by value."""
    got = f64(got)
    bound = U * terms * (1 + LAST[dtype]) + LAST[dtype] * np.abs(ref) + 1e-37
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - ref) / bound).max()))


# ---------------------------------------------------------------- norm and rotation

def heads_of(layout, N, H, D, dtype, gen, extra=2):
    """An [N, H, D] view of the given layout with N(0, 1) values."""
    if layout == "fused":      # columns of a wider row
        return torch.randn((N, H + extra, D), generator=gen).to(dtype).cuda()[:, 1:H + 1]
    if layout == "head_major":
        return torch.randn((H, N, D), generator=gen).to(dtype).cuda().transpose(0, 1)
    return torch.randn((N, H, D), generator=gen).to(dtype).cuda()


# N, q heads, k heads, D, rotary_dim, interleaved, weight, dtype, layout
ROPE = [
    (1, 1, 0, 8, 0, False, None, F32, "dense"),
    (1, 1, 1, 16, 16, True, "shared", BF, "dense"),
    (3, 5, 2, 64, 64, False, "shared", BF, "fused"),
    (17, 3, 3, 128, 128, False, "per_head", BF, "head_major"),
    (130, 4, 1, 80, 64, True, "per_head", F32, "fused"),
    (65, 2, 1, 72, 48, False, "shared", F32, "head_major"),
    (64, 9, 7, 256, 256, False, "shared", F32, "dense"),
    (33, 1, 1, 256, 16, True, "per_head", BF, "fused"),
    (300, 16, 16, 128, 64, False, "shared", BF, "fused"),
    (1025, 33, 1, 24, 16, False, "per_head", BF, "dense"),
    (4500, 2, 1, 96, 96, True, "shared", F32, "fused"),
]


# every width of a head: rows take as many lanes as they have values for, several rows to a warp,
# with other heads and layouts beside them
WIDTHS = [(41 + D // 8, 1 + D // 8 % 5, D // 8 % 4, D, D // 16 * 16 if D % 3 else D // 32 * 16,
           D // 8 % 2 == 0, ("shared", "per_head", None)[D // 8 % 3], (BF, F32)[D // 24 % 2],
           ("fused", "dense", "head_major")[D // 16 % 3]) for D in range(8, 257, 8)]


def rope_inputs(case, seed=0):
    N, hq, hk, D, rot, inter, weight, dtype, layout = case
    gen = torch.Generator().manual_seed(seed)
    freq = (1e6 ** -(torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).cuda()
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (N,), generator=gen).to(torch.int32)
    pos[0] = -(1 << 31)
    pos[N // 2] = 3
    sides = []
    for H in (hq, hk):
        if H == 0:
            sides.append(None)
            continue
        w = None
        if weight:
            w = torch.randn((H, D) if weight == "per_head" else (D,), generator=gen).cuda()
        x = heads_of(layout, N, H, D, dtype, gen)
        x[0] = 0  # a zero row
        x[N // 2] *= 1000
        sides.append(dict(x=x, weight=w, H=H))
    return sides, pos.cuda(), freq, gen


def pair_sums(n, rot, inter):
    """|n_a| + |n_b| of each value's pair."""
    n = np.abs(n)
    out = n.copy()
    if rot:
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        out[..., a] = out[..., b] = n[..., a] + n[..., b]
    return out


# Roundings on the way to a value of y: the mean (D + 1 at most, halved by the root), rsqrt (4),
# the products with rstd and w (2), the angle (its fraction of a turn is off by 2^-26, 2 pi 2^-26
# = 1.6 * 2^-24 ... counted as 2), sine and cosine (4), the rotation itself (2)
def rope_count(D):
    return (D + 1) / 2 + 4 + 2 + 2 + 4 + 2


@pytest.mark.parametrize("case", ROPE, ids=[str(i) for i in range(len(ROPE))])
def test_norm_rope(case):
    N, hq, hk, D, rot, inter, weight, dtype, layout = case
    sides, pos, freq, gen = rope_inputs(case)
    for s in sides:
        if s:
            s["y"] = torch.empty((N, s["H"], D), dtype=dtype, device="cuda")
    moe.moe_qk_norm_rope(N, D, rot, inter, CODE[dtype], 1e-6, pos if rot else None,
                         freq if rot else None, *sides)
    torch.cuda.synchronize()
    for s in sides:
        if s:
            w = None if s["weight"] is None else f64(s["weight"])
            args = (f64(s["x"]), w, f64(pos), f64(freq), rot, inter, 1e-6)
            n = SM.qk_norm_rope(args[0], w, f64(pos), f64(freq), 0, inter, 1e-6)
            close(s["y"], SM.qk_norm_rope(*args), rope_count(D) * pair_sums(n, rot, inter), dtype)


@pytest.mark.parametrize("dy32", [True, False])
@pytest.mark.parametrize("case", ROPE, ids=[str(i) for i in range(len(ROPE))])
def test_norm_rope_backward(case, dy32):
    N, hq, hk, D, rot, inter, weight, dtype, layout = case
    gtype = F32 if dy32 else dtype
    sides, pos, freq, gen = rope_inputs(case, seed=1)
    for s in sides:
        if s:
            s["dy"] = heads_of(layout, N, s["H"], D, gtype, gen, extra=1)
            s["dx"] = torch.empty((N, s["H"], D), dtype=dtype, device="cuda")
            if s["weight"] is not None:
                s["dweight"] = torch.full_like(s["weight"], float("nan"))
    ws = torch.empty(moe.moe_qk_norm_rope_backward_workspace_size(N, D, hq, hk),
                     dtype=torch.uint8, device="cuda")
    moe.moe_qk_norm_rope_backward(N, D, rot, inter, CODE[dtype], CODE[gtype], 1e-6,
                                  pos if rot else None, freq if rot else None, *sides, ws)
    torch.cuda.synchronize()
    for s in sides:
        if not s:
            continue
        w = None if s["weight"] is None else f64(s["weight"])
        x, dy = f64(s["x"]), f64(s["dy"])
        dx, dw = SM.qk_norm_rope_backward(x, w, f64(pos), f64(freq), rot, inter, 1e-6, dy)
        rstd = 1 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + 1e-6)
        xh = np.abs(x) * rstd
        u = pair_sums(dy, rot, inter) * (1 if w is None else np.abs(w))
        count = rope_count(D)
        # dx = rstd (u - xh mean(u xh)): the mean's own D roundings, and those of its factors
        terms = rstd * (2 * count * u + (3 * count + D) * xh * np.mean(u * xh, -1, keepdims=True))
        close(s["dx"], dx, terms, dtype, "dx")
        if w is None:
            continue
        each = np.sum(pair_sums(dy, rot, inter) * xh, axis=0)  # [H, D]
        rows = N if weight == "per_head" else N * s["H"]
        ref, each = (dw, each) if weight == "per_head" else (dw.sum(0), each.sum(0))
        close(s["dweight"], ref, (2 * count + rows) * each, F32, "dweight")
        # the sum itself is split over blocks and warps, so far fewer roundings reach it
        assert relerr(f64(s["dweight"]), ref) <= 2e-5


@pytest.mark.parametrize("case", WIDTHS, ids=[str(c[3]) for c in WIDTHS])
def test_norm_rope_of_every_width(case):
    test_norm_rope(case)
    test_norm_rope_backward(case, case[3] % 16 == 0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_rope_in_place_broadcast_and_determinism(dtype):
    """y over x; one row broadcast to all tokens and heads by zero strides; the same bits
    again."""
    N, H, D = 77, 3, 128
    sides, pos, freq, gen = rope_inputs((N, H, 0, D, 64, False, "shared", dtype, "fused"))
    x, w = sides[0]["x"], sides[0]["weight"]
    y, y2 = (torch.empty((N, H, D), dtype=dtype, device="cuda") for _ in range(2))
    run = lambda q: moe.moe_qk_norm_rope(N, D, 64, False, CODE[dtype], 1e-6, pos, freq, q, None)  # noqa: E731
    run(dict(x=x, y=y, weight=w))
    run(dict(x=x, y=x, weight=w))
    assert torch.equal(x, y)
    row = torch.randn((1, 1, D)).to(dtype).cuda()
    run(dict(x=row.expand(N, H, D), y=y, weight=w))
    run(dict(x=row.expand(N, H, D).contiguous(), y=y2, weight=w))
    assert torch.equal(y, y2)


def test_norm_rope_backward_in_place_and_determinism():
    N, hq, hk, D = 500, 3, 2, 64
    case = (N, hq, hk, D, 64, False, "per_head", F32, "dense")
    outs = []
    for run in range(3):
        sides, pos, freq, gen = rope_inputs(case, seed=2)
        for s in sides:
            s["dy"] = torch.randn((N, s["H"], D), generator=gen).cuda()
            s["dx"] = (torch.empty_like(s["dy"]), s["x"], s["dy"])[run]
            s["dweight"] = torch.empty_like(s["weight"])
        ws = torch.empty(moe.moe_qk_norm_rope_backward_workspace_size(N, D, hq, hk),
                         dtype=torch.uint8, device="cuda")
        moe.moe_qk_norm_rope_backward(N, D, 64, False, moe.MOE_F32, moe.MOE_F32, 1e-6, pos, freq,
                                      *sides, ws)
        outs.append([t for s in sides for t in (s["dx"].clone(), s["dweight"])])
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))


def test_norm_rope_weight_gradients_are_optional():
    """No workspace is needed without them; one side's alone is right."""
    N, D = 40, 32
    sides, pos, freq, gen = rope_inputs((N, 2, 3, D, 32, True, "shared", F32, "dense"), seed=3)
    for s in sides:
        s["dy"] = torch.randn((N, s["H"], D), generator=gen).cuda()
        s["dx"] = torch.empty_like(s["dy"])
    args = (N, D, 32, True, moe.MOE_F32, moe.MOE_F32, 1e-6, pos, freq)
    moe.moe_qk_norm_rope_backward(*args, *sides, None)
    dx = [s["dx"].clone() for s in sides]
    ws = torch.empty(moe.moe_qk_norm_rope_backward_workspace_size(N, D, 2, 3), dtype=torch.uint8,
                     device="cuda")
    sides[1]["dweight"] = torch.empty(D, device="cuda")
    moe.moe_qk_norm_rope_backward(*args, *sides, ws)
    assert all(torch.equal(a, s["dx"]) for a, s in zip(dx, sides))
    ref = SM.qk_norm_rope_backward(f64(sides[1]["x"]), f64(sides[1]["weight"]), f64(pos),
                                   f64(freq), 32, True, 1e-6, f64(sides[1]["dy"]))[1].sum(0)
    assert relerr(f64(sides[1]["dweight"]), ref) <= 2e-5


# ---------------------------------------------------------------- gated linear recurrence

def offsets(N, lengths):
    """Packed offsets of the given lengths (None: the rest), N rows in all."""
    off = [0]
    rest = N - sum(n for n in lengths if n is not None)
    for n in lengths:
        off.append(off[-1] + (rest if n is None else n))
    return off


# N, D, lengths (None: what is left; a number alone: that many equal sequences), mix, dtype, h0
GLR = [
    (1, 1, 1, False, F32, False),
    (1, 7, [0, 1, 0], True, BF, True),
    (2, 64, 2, False, BF, True),
    (63, 33, 1, True, F32, True),
    (64, 2, 1, False, BF, False),
    (65, 130, 5, True, BF, True),
    (128, 66, [64, None], False, F32, True),
    (129, 65, [0, 0, 128, 0, None, 0], True, F32, False),
    (777, 96, [1, 15, 16, 17, 0, 31, None, 1, 1], False, BF, True),
    (1000, 70, [None, 200], True, F32, True),
    (1024, 128, 64, False, BF, True),
    (2051, 34, [3, None, 3], False, F32, True),
    (5000, 200, 1, True, BF, True),
    (9000, 10, [4000, 0, None], False, F32, True),
    (700, 1030, 7, False, BF, True),
    (1300, 2050, [600, None], True, BF, False),
    (100, 8, [30, None], True, BF, True),
    (200, 4, 1, False, F32, True),
    (4100, 328, [2000, None, 0], True, BF, True),
    (3001, 100, 1, True, F32, False),
    # sequences of one and three rows; runs of empty ones; more of them than a block keeps bounds of
    (300, 72, 300, True, BF, True),
    (303, 72, 101, False, F32, True),
    (200, 72, [0] * 40 + [5] + [0] * 70 + [None] + [0] * 33 + [3], True, BF, True),
    (2000, 68, [n % 4 for n in range(900)] + [None, 0], False, F32, True),
    (5000, 64, [n % 7 for n in range(1300)] + [None, 0], True, BF, True),
]


def glr_inputs(case, seed=0, pad=0, wide=0):
    N, D, lengths, mix, dtype, with_h0 = case
    gen = torch.Generator().manual_seed(seed)
    rows = N + pad
    g = torch.nn.functional.logsigmoid(torch.randn((rows, D + wide), generator=gen) + 3)
    g[torch.rand(g.shape, generator=gen) < 0.02] = 0.0            # no decay
    g[torch.rand(g.shape, generator=gen) < 0.01] = -float("inf")  # forgets
    g[torch.rand(g.shape, generator=gen) < 0.01] = -60.0
    x = torch.randn((rows, D + wide), generator=gen)
    off = offsets(N, [N // lengths] * lengths if isinstance(lengths, int) else lengths)
    S = len(off) - 1
    h0 = torch.randn((S, D), generator=gen).cuda() if with_h0 else None
    return dict(g=g.to(dtype).cuda()[:, :D], x=x.to(dtype).cuda()[:, :D], off=off, S=S, h0=h0,
                uniform=isinstance(lengths, int), gen=gen, rows=rows)


def offsets_arg(i):
    return None if i["uniform"] else torch.tensor(i["off"], dtype=torch.int32).cuda()


def run_glr(case, i, h_T=None):
    N, D, lengths, mix, dtype, _ = case
    h = torch.full((i["rows"], D), 7.0, dtype=dtype, device="cuda")
    h_T = torch.empty((i["S"], D), device="cuda") if h_T is None else h_T
    chunks = torch.full(((i["rows"] + 63) // 64, D), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_glr_forward(i["rows"], D, i["S"], offsets_arg(i), int(mix), CODE[dtype], i["g"],
                        i["x"], i["h0"], h, h_T, chunks, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    return h, h_T, chunks


# Roundings that a step adds, relative to everything summed so far: a = exp(g) by a product with
# log2(e) (|g| log2(e) roundings of a), the exponential (4), its product into the decay of a span
# and into the state (2 and 2), the sum (2), and the input's own in the mixed form, 1 - a to a few
# roundings of itself (8)
def majorants(g, x, off, h0, mix):
    """M: the recurrence of absolute values; E: its accumulated count of roundings."""
    a = np.exp(g)
    b = -np.expm1(g) * np.abs(x) if mix else np.abs(x)
    c = 10 + 1.5 * np.abs(np.where(np.isfinite(g), g, 0.0)) + (8 if mix else 0)
    M, E = np.zeros_like(a), np.zeros_like(a)
    for s in range(len(off) - 1):
        m = np.zeros(a.shape[1]) if h0 is None else np.abs(h0[s])
        e = np.zeros(a.shape[1])
        for t in range(off[s], off[s + 1]):
            m = a[t] * m + b[t]
            e = a[t] * e + c[t] * m
            M[t], E[t] = m, e
    return M, E


# values between the end of a row of g and x and the next: rows on 16-byte boundaries where D
# allows it, dense, and rows on the boundaries of a value alone
@pytest.mark.parametrize("wide", [8, 0, 5])
@pytest.mark.parametrize("case", GLR, ids=[f"{c[0]}x{c[1]}" for c in GLR])
def test_recurrence(case, wide):
    N, D, lengths, mix, dtype, _ = case
    pad = 0 if isinstance(lengths, int) else 3
    i = glr_inputs(case, pad=pad, wide=wide)
    h, h_T, chunks = run_glr(case, i)
    g, x, h0 = f64(i["g"])[:N], f64(i["x"])[:N], f64(i["h0"])
    ref, ref_T = SM.gated_recurrence(g, x, i["off"], h0, mix)
    _, E = majorants(g, x, i["off"], h0, mix)
    close(h[:N], ref, E, dtype, "h")
    assert (h[N:] == 7.0).all()  # padding rows as they were
    for s in range(i["S"]):
        lo, hi = i["off"][s], i["off"][s + 1]
        close(h_T[s], ref_T[s], E[hi - 1] if hi > lo else 0 * ref_T[s], F32, f"h_T {s}")
    starts = {lo for lo, hi in zip(i["off"], i["off"][1:]) if hi > lo}
    for c in range(0, N, 64):
        if c in starts:
            assert (chunks[c // 64] == 0).all()
        else:
            close(chunks[c // 64], ref[c - 1], E[c - 1], F32, f"chunk {c}")


@pytest.mark.parametrize("wide", [8, 0, 5])
@pytest.mark.parametrize("case", GLR, ids=[f"{c[0]}x{c[1]}" for c in GLR])
def test_recurrence_backward(case, wide):
    N, D, lengths, mix, dtype, with_h0 = case
    pad = 0 if isinstance(lengths, int) else 3
    i = glr_inputs(case, seed=1, pad=pad, wide=wide)
    _, _, chunks = run_glr(case, i)
    dh = torch.randn((i["rows"], D), generator=i["gen"]).to(dtype).cuda()
    dh_T = torch.randn((i["S"], D), generator=i["gen"]).cuda() if with_h0 else None
    wide = i["g"].stride(0)
    both = [torch.full((i["rows"], wide), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    dg, dx = (t[:, :D] for t in both)
    dh0 = torch.empty((i["S"], D), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_glr_backward(i["rows"], D, i["S"], offsets_arg(i), int(mix), CODE[dtype], i["g"],
                         i["x"], i["h0"], chunks, dh, dh_T, dg, dx, dh0, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for t in both:  # padding rows and columns as they were
        assert (t[N:] == 7.0).all() and (t[:, D:] == 7.0).all()
    g, x, h0 = f64(i["g"])[:N], f64(i["x"])[:N], f64(i["h0"])
    dh, dh_T = f64(dh)[:N], f64(dh_T)
    ref = SM.gated_recurrence_backward(g, x, i["off"], dh, h0, dh_T, mix)
    M, E = majorants(g, x, i["off"], h0, mix)
    # lam runs the same recurrence backwards, each row's decay being the next row's
    a = np.exp(g)
    c = 10 + 1.5 * np.abs(np.where(np.isfinite(g), g, 0.0))
    L, F = np.zeros_like(a), np.zeros_like(a)   # sums of absolute values, roundings
    dg_terms, dx_terms = np.zeros_like(a), np.zeros_like(a)
    for s in range(i["S"]):
        lo, hi = i["off"][s], i["off"][s + 1]
        m = np.zeros(D) if dh_T is None else np.abs(dh_T[s])
        e = np.zeros(D)
        for t in range(hi - 1, lo - 1, -1):
            m = m + np.abs(dh[t])
            e = e + 2 * m
            if t > lo:
                before, roundings = M[t - 1], E[t - 1]
            else:
                before = np.zeros(D) if h0 is None else np.abs(h0[s])
                roundings = 0
            if mix:
                before = before + np.abs(x[t])
            gate = -np.expm1(g[t]) if mix else 1.0
            dx_terms[t] = gate * (e + 8 * m)
            dg_terms[t] = a[t] * (before * (e + (c[t] + 3) * m) + m * roundings)
            e = a[t] * (e + c[t] * m)
            m = a[t] * m
        close(dh0[s], ref["dh0"][s], e, F32, f"dh0 {s}")
    close(dx[:N], ref["dx"], dx_terms, dtype, "dx")
    close(dg[:N], ref["dg"], dg_terms, dtype, "dg")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_recurrence_states_in_place_and_prefill_in_parts(dtype):
    """h_T over h0, a long prompt in three calls, against one call; then the same bits again."""
    N, D = 900, 136
    whole = (N, D, 1, False, dtype, True)
    i = glr_inputs(whole, seed=2)
    h, h_T, _ = run_glr(whole, i)
    state, parts = i["h0"].clone(), []
    for lo, hi in ((0, 100), (100, 612), (612, 900)):
        part = dict(i, g=i["g"][lo:hi], x=i["x"][lo:hi], h0=state, rows=hi - lo)
        parts.append(run_glr((hi - lo, D, 1, False, dtype, True), part, h_T=state)[0])
    # the parts are cut elsewhere, so they round elsewhere
    E = majorants(f64(i["g"]), f64(i["x"]), [0, N], f64(i["h0"]), False)[1]
    close(torch.cat(parts), f64(h), 2 * E + LAST[dtype] / U * np.abs(f64(h)), dtype)
    close(state, f64(h_T), 2 * E[-1:], F32)
    again = run_glr(whole, i)
    assert torch.equal(again[0], h) and torch.equal(again[1], h_T)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_recurrence_sequences_do_not_see_each_other(dtype, bad):
    """A NaN or infinity in one sequence (its inputs, decays, state, padding) leaves the values
    and gradients of the others as they are without it."""
    case = (700, 72, [130, 200, 0, 70, None], True, dtype, True)
    N, D = case[0], case[1]
    outs = []
    for poisoned in (False, True):
        i = glr_inputs(case, seed=3, pad=4)
        dh = torch.randn((i["rows"], D), generator=i["gen"]).to(dtype).cuda()
        dh_T = torch.randn((i["S"], D), generator=i["gen"]).cuda()
        if poisoned:
            for t in (i["x"], dh, i["g"]):
                t[131:330] = bad
                t[N:] = bad
            i["h0"][1] = bad
            dh_T[1] = bad
        h, h_T, chunks = run_glr(case, i)
        dg, dx = (torch.zeros((i["rows"], D), dtype=dtype, device="cuda") for _ in range(2))
        dh0 = torch.empty((i["S"], D), device="cuda")
        moe.moe_glr_backward(i["rows"], D, i["S"], offsets_arg(i), 1, CODE[dtype], i["g"], i["x"],
                             i["h0"], chunks, dh, dh_T, dg, dx, dh0)
        outs.append((h, dg, dx, h_T, dh0))
    for a, b in zip(outs[0][:3], outs[1][:3]):
        assert torch.equal(a[:130], b[:130]) and torch.equal(a[330:], b[330:])
    for a, b in zip(outs[0][3:], outs[1][3:]):
        keep = [0, 2, 3, 4]
        assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(outs[1][0][131:330].float()).any()


def test_recurrence_reports_bad_offsets():
    """Offsets that decrease, pass N or do not begin at 0 are reported; rows of the buffers stay
    the only memory touched."""
    N, D = 100, 64
    g, x = -torch.rand((N, D)).cuda(), torch.randn((N, D)).cuda()
    guard = torch.full((N + 2, D), 3.0).cuda()
    h = guard[1:-1]
    for off in ([0, 50, 40, 100], [0, 50, 60, 101], [1, 50, 60, 100], [0, -3, 60, 100],
                [0, 200, 300, 100]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.moe_glr_forward(N, D, 3, torch.tensor(off, dtype=torch.int32).cuda(), 0, moe.MOE_F32,
                            g, x, None, h, torch.empty((3, D)).cuda(), None, status)
        assert int(status) == 6, off
        assert (guard[0] == 3).all() and (guard[-1] == 3).all()


def test_recurrence_past_2_to_31_values():
    """300000 x 8192 values: the last rows, states and gradients of the last of three sequences
    (what is 600 steps back has decayed by e^-60 or more)."""
    N, D, tail = 300000, 8192, 600
    assert N * D > 1 << 31
    torch.manual_seed(12)
    row = lambda n: torch.randn((n, D), device="cuda").to(BF)  # noqa: E731
    g = -0.1 - torch.rand((1, D), device="cuda").to(BF)
    x, dh = (row(1000).repeat(N // 1000, 1) for _ in range(2))
    off = torch.tensor([0, 1000, 150001, N - 5], dtype=torch.int32).cuda()
    h, dg, dx = (torch.full((N, D), 7.0, dtype=BF, device="cuda") for _ in range(3))
    h_T, chunks = torch.empty((3, D), device="cuda"), torch.empty(((N + 63) // 64, D), device="cuda")
    gs = g.expand(N, D).contiguous()
    args = (N, D, 3, off, moe.MOE_GLR_ADD, moe.MOE_BF16, gs, x)
    moe.moe_glr_forward(*args, None, h, h_T, chunks)
    moe.moe_glr_backward(*args, None, chunks, dh, None, dg, dx, None)
    torch.cuda.synchronize()
    lo, hi = N - 5 - tail, N - 5
    gt, xt, dt = f64(gs[lo:hi]), f64(x[lo:hi]), f64(dh[lo:hi])
    ref, ref_T = SM.gated_recurrence(gt, xt, [0, tail], None)
    _, E = majorants(gt, xt, [0, tail], None, False)
    keep = slice(tail - 50, tail)
    close(h[lo:hi][keep], ref[keep], E[keep], BF, "h")
    close(h_T[2], ref_T[0], E[-1], F32, "h_T")
    back = SM.gated_recurrence_backward(gt, xt, [0, tail], dt)
    for got, want in ((dx, back["dx"]), (dg, back["dg"])):
        # sums of at most ~10 terms that matter, each through at most 30 roundings of its step
        size = np.abs(want[keep]) + 30.0
        close(got[lo:hi][keep], want[keep], 400 * size, BF)
    for t in (h, dg, dx):
        assert (t[hi:] == 7.0).all()


def test_norm_rope_past_2_to_31_values():
    N, H, D = 40000, 512, 128
    assert N * H * D > 1 << 31
    gen = torch.Generator().manual_seed(13)
    x = torch.randn((N, 1, D), generator=gen).to(BF).cuda().expand(N, H, D)
    y = torch.empty((N, H, D), dtype=BF, device="cuda")
    freq = (1e6 ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()
    w = torch.rand(D, generator=gen).cuda()
    moe.moe_qk_norm_rope(N, D, D, False, moe.MOE_BF16, 1e-6, pos, freq,
                         dict(x=x, y=y, weight=w), None)
    torch.cuda.synchronize()
    t = [0, N // 2, N - 1]
    n = SM.qk_norm_rope(f64(x[t, :1]), f64(w), None, None, 0, False, 1e-6)
    ref = SM.qk_norm_rope(f64(x[t, :1]), f64(w), f64(pos[t]), f64(freq), D, False, 1e-6)
    for head in (0, 255, H - 1):
        close(y[t, head:head + 1], ref, rope_count(D) * pair_sums(n, D, False), BF)


# ---------------------------------------------------------------- single tokens

@pytest.mark.parametrize("D, few, dtype", [(1 << 20, 64, BF), ((1 << 20) - 1, 63, BF),
                                           ((1 << 20) - 3, 63, F32)])
def test_recurrence_of_the_most_channels(D, few, dtype):
    """More strips of channels than the GPU has places for, so blocks come in many rounds.  Channels
    do not see each other: the first and the last of them have the bits that a call with these few
    alone gives, which the tests above check value by value."""
    N = 67
    gen = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    g = torch.nn.functional.logsigmoid(r(N, D) + 3).to(dtype)
    x, dh, h0, dh_T = r(N, D).to(dtype), r(N, D).to(dtype), r(2, D), r(2, D)
    off = torch.tensor([0, 30, N], dtype=torch.int32, device="cuda")

    def run(part):
        i = [t[:, part].contiguous() for t in (g, x, dh, h0, dh_T)]
        d = i[0].shape[1]
        h, dg, dx = (torch.empty((N, d), dtype=dtype, device="cuda") for _ in range(3))
        h_T, dh0, chunks = (torch.empty((2, d), device="cuda") for _ in range(3))
        moe.moe_glr_forward(N, d, 2, off, 1, CODE[dtype], i[0], i[1], i[3], h, h_T, chunks)
        moe.moe_glr_backward(N, d, 2, off, 1, CODE[dtype], i[0], i[1], i[3], chunks, i[2], i[4], dg,
                             dx, dh0)
        return h, h_T, chunks, dg, dx, dh0

    every = run(slice(0, D))
    for part in (slice(0, few), slice(D - few, D)):
        for got, want in zip(every, run(part)):
            assert torch.equal(got[:, part], want)


@pytest.mark.parametrize("case", [(3, 4096, 0, 8, 0, False, "per_head", BF, "dense"),
                                  (2, 4000, 96, 24, 16, True, "shared", F32, "fused"),
                                  (5, 1000, 1000, 64, 64, False, "per_head", BF, "head_major")],
                         ids=["8", "24", "64"])
def test_norm_rope_of_many_heads(case):
    test_norm_rope(case)
    test_norm_rope_backward(case, True)


@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B, D, n_slots, slots", [(1, 1, 1, False), (5, 33, 5, False),
                                                  (7, 512, 20, True), (130, 130, 200, True)])
def test_recurrence_step(B, D, n_slots, slots, dtype, mix):
    gen = torch.Generator().manual_seed(5)
    g = torch.nn.functional.logsigmoid(torch.randn((B, D + 2), generator=gen) + 3)
    g[0] = -float("inf")
    g, x = g.to(dtype).cuda()[:, :D], torch.randn((B, D + 1), generator=gen).to(dtype).cuda()[:, :D]
    slot = torch.randperm(n_slots, generator=gen)[:B].to(torch.int32) if slots else torch.arange(B)
    state = torch.randn((n_slots, D), generator=gen).cuda()
    old = f64(state)
    h = torch.empty((B, D), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_glr_step(B, D, int(mix), CODE[dtype], g, x, slot.cuda() if slots else None, n_slots,
                     state, h, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    s = slot.long().numpy()
    off = list(range(B + 1))
    ref, _ = SM.gated_recurrence(f64(g), f64(x), off, old[s], mix)
    _, E = majorants(f64(g), f64(x), off, old[s], mix)
    close(h, ref, E, dtype, "h")
    close(state[s], ref, E, F32, "state")
    rest = np.setdiff1d(np.arange(n_slots), s)
    assert np.array_equal(f64(state)[rest], old[rest])


def gdr_step_inputs(B, H, dk, dv, n_slots, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    i = dict(q=r(B, H, dk).to(BF), k=r(B, H, dk).to(BF), v=r(B, H, dv).to(BF),
             beta=torch.sigmoid(r(B, H)), g=torch.nn.functional.logsigmoid(r(B, H) + 4),
             S=r(n_slots, H, dv, dk))
    return {n: t.cuda() for n, t in i.items()}, gen


def gdr_step_check(i, slot, S, o):
    """One step from i["S"] rows `slot`: S and o against the oracle."""
    B, H, dk = i["q"].shape
    one = lambda n: f64(i[n])[:, None]  # noqa: E731
    old = f64(i["S"])[slot]
    o_ref, S_ref = LA.gated_delta_rule(one("q"), one("k"), one("v"), one("beta"), one("g"), S0=old)
    unit = lambda x: np.abs(x) / np.maximum(np.sqrt((x * x).sum(-1, keepdims=True)), 1e-300)  # noqa: E731
    qh, kh = unit(f64(i["q"]))[:, :, None], unit(f64(i["k"]))[:, :, None]
    A = np.exp(f64(i["g"]))[..., None, None] * np.abs(old)
    # the unit vectors (dk/2 + 8 each), the decay (8), the products and the sum over dk
    c = 2 * dk + 40
    r = np.abs(f64(i["v"]))[..., None] + (A * kh).sum(-1, keepdims=True)
    S_terms = c * (A + f64(i["beta"])[..., None, None] * r * kh)
    o_terms = dk ** -0.5 * ((S_terms + c * (A + r * kh)) * qh).sum(-1)
    close(S[slot], S_ref, S_terms, F32, "S")
    close(o, o_ref[:, 0], o_terms, BF, "o")


@pytest.mark.parametrize("B, H, dk, dv, n_slots, slots", [
    (1, 1, 64, 64, 1, False), (3, 2, 128, 64, 3, False), (2, 3, 64, 128, 9, True),
    (33, 4, 128, 128, 40, True)])
def test_delta_rule_step(B, H, dk, dv, n_slots, slots):
    i, gen = gdr_step_inputs(B, H, dk, dv, n_slots)
    slot = torch.randperm(n_slots, generator=gen)[:B].to(torch.int32) if slots else None
    S, o = i["S"].clone(), torch.empty((B, H, dv), dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_gdr_step(B, H, dk, dv, i["q"], i["k"], i["v"], i["beta"], i["g"],
                     None if slot is None else slot.cuda(), n_slots, dk ** -0.5, S, o, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    s = np.arange(B) if slot is None else slot.numpy()
    gdr_step_check(i, s, S, o)
    rest = np.setdiff1d(np.arange(n_slots), s)
    assert np.array_equal(f64(S)[rest], f64(i["S"])[rest])


def test_delta_rule_step_zero_rows():
    """A zero key writes nothing, a zero query reads nothing (as in the forward)."""
    i, _ = gdr_step_inputs(2, 1, 64, 64, 2)
    i["k"][0] = 0
    i["q"][1] = 0
    S, o = i["S"].clone(), torch.empty((2, 1, 64), dtype=BF, device="cuda")
    moe.moe_gdr_step(2, 1, 64, 64, i["q"], i["k"], i["v"], i["beta"], i["g"], None, 2, 0.125, S, o)
    want = torch.exp(i["g"][0, 0].double()).cpu() * i["S"][0].double().cpu()
    close(S[0], want.numpy(), 8 * np.abs(want.numpy()), F32)
    assert (o[1] == 0).all() and torch.isfinite(S).all()


def steps(kind, slot, n_slots, B):
    """Runs one step on distinct states and returns (old state, new state, output, status)."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor(slot, dtype=torch.int32).cuda()
    if kind == "gdr":
        i, _ = gdr_step_inputs(B, 2, 64, 64, n_slots)
        new, out = i["S"].clone(), torch.full((B, 2, 64), 9.0, dtype=BF, device="cuda")
        moe.moe_gdr_step(B, 2, 64, 64, i["q"], i["k"], i["v"], i["beta"], i["g"], slot, n_slots,
                         0.125, new, out, status)
        return i["S"], new, out, int(status)
    gen = torch.Generator().manual_seed(8)
    old = torch.randn((n_slots, 200), generator=gen).cuda()
    g, x = -torch.rand((B, 200), generator=gen).cuda(), torch.randn((B, 200), generator=gen).cuda()
    new, out = old.clone(), torch.full((B, 200), 9.0, device="cuda")
    moe.moe_glr_step(B, 200, moe.MOE_GLR_ADD, moe.MOE_F32, g, x, slot, n_slots, new, out, status)
    return old, new, out, int(status)


@pytest.mark.parametrize("kind", ["gdr", "glr"])
@pytest.mark.parametrize("slot, status, skipped", [
    ([3, -1, 0, -1], 0, [1, 3]),         # padding rows
    ([3, 3, 0, 3], 6, [1, 3]),           # the first of equal slots is the one that runs
    ([5, 1, -2, 1 << 30], 6, [0, 2, 3]),  # out of range
])
def test_steps_skip_padding_and_report_bad_slots(kind, slot, status, skipped):
    old, new, out, got = steps(kind, slot, 5, 4)
    assert got == status
    ran = [b for b in range(4) if b not in skipped]
    assert all((out[b] == 9).all() for b in skipped)
    assert all((out[b] != 9).any() for b in ran)
    touched = {slot[b] for b in ran}
    for s in range(5):
        assert torch.equal(old[s], new[s]) == (s not in touched)
    alone = steps(kind, [s if b in ran else -1 for b, s in enumerate(slot)], 5, 4)
    assert torch.equal(alone[1], new)


# ---------------------------------------------------------------- together

def test_prefill_then_decode():
    """A mixer as it is served: norm and rotation out of a fused projection, the delta rule over
    the prompt, then tokens one at a time, against the oracle over the whole sequence; beside it
    the recurrence, prefilled and continued."""
    T, steps, H, D = 150, 3, 2, 64
    N = T + steps
    gen = torch.Generator().manual_seed(9)
    row = torch.randn((N, 3 * H, D), generator=gen).to(BF).cuda()
    w = [torch.rand(D, generator=gen).cuda() + 0.5 for _ in range(2)]
    freq = (1e4 ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda() + 100000
    beta = torch.sigmoid(torch.randn((N, H), generator=gen)).cuda()
    g = torch.nn.functional.logsigmoid(torch.randn((N, H), generator=gen) + 4).cuda()
    gl = torch.nn.functional.logsigmoid(torch.randn((N, H * D), generator=gen) + 4).to(BF).cuda()

    def norm_rope(lo, hi):
        qk = [torch.empty((hi - lo, H, D), dtype=BF, device="cuda") for _ in range(2)]
        moe.moe_qk_norm_rope(hi - lo, D, D, False, moe.MOE_BF16, 1e-6, pos[lo:hi], freq,
                             dict(x=row[lo:hi, :H], y=qk[0], weight=w[0]),
                             dict(x=row[lo:hi, H:2 * H], y=qk[1], weight=w[1]))
        return qk

    v = row[:, 2 * H:].contiguous()
    q, k = norm_rope(0, T)
    o = torch.empty((N, H, D), dtype=BF, device="cuda")
    S = torch.empty((1, H, D, D), device="cuda")
    ws = torch.empty(moe.moe_gdr_workspace_size(1, T, H, D, D), dtype=torch.uint8, device="cuda")
    moe.moe_gdr_forward(1, T, H, D, D, q, k, v[:T], beta[:T], g[:T], None, D ** -0.5, o[:T], S,
                        None, ws)
    h = torch.empty((N, H * D), dtype=BF, device="cuda")
    state = torch.empty((1, H * D), device="cuda")
    ov = v.view(N, H * D)
    moe.moe_glr_forward(T, H * D, 1, None, moe.MOE_GLR_MIX, moe.MOE_BF16, gl[:T], ov[:T], None,
                        h[:T], state, None)
    qs, ks = [q], [k]
    for t in range(T, N):
        q1, k1 = norm_rope(t, t + 1)
        qs.append(q1)
        ks.append(k1)
        moe.moe_gdr_step(1, H, D, D, q1, k1, v[t:t + 1], beta[t:t + 1], g[t:t + 1], None, 1,
                         D ** -0.5, S, o[t:t + 1])
        moe.moe_glr_step(1, H * D, moe.MOE_GLR_MIX, moe.MOE_BF16, gl[t:t + 1], ov[t:t + 1], None,
                         1, state, h[t:t + 1])
    assert moe.moe_gdr_device_status() == moe.MOE_OK
    seq = lambda t: f64(t)[None]  # noqa: E731
    o_ref, S_ref = LA.gated_delta_rule(seq(torch.cat(qs)), seq(torch.cat(ks)), seq(v), seq(beta),
                                       seq(g))
    # the bars of the delta rule's own tests: o is rounded to bf16, the state is fp32 with the
    # scan's two-piece products
    assert relerr(f64(o), o_ref[0]) <= 5e-3
    assert relerr(f64(S), S_ref) <= 1e-4
    h_ref, T_ref = SM.gated_recurrence(f64(gl), f64(ov), [0, N], None, True)
    E = majorants(f64(gl), f64(ov), [0, N], None, True)[1]
    close(h, h_ref, E, BF)
    close(state, T_ref, E[-1:], F32)


def test_training_pass_through_norm_rotation_and_delta_rule():
    """q, k through the norm and rotation into the delta rule and back: the gradients of the
    projections' outputs against the oracle's chain on the same rounded q, k."""
    T, H, D = 130, 2, 64
    gen = torch.Generator().manual_seed(10)
    row = torch.randn((T, 3 * H, D), generator=gen).to(BF).cuda()
    w = [torch.rand(D, generator=gen).cuda() + 0.5 for _ in range(2)]
    freq = (1e4 ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = torch.arange(T, dtype=torch.int32).cuda()
    beta = torch.sigmoid(torch.randn((T, H), generator=gen)).cuda()
    g = torch.nn.functional.logsigmoid(torch.randn((T, H), generator=gen) + 4).cuda()
    d_o = torch.randn((T, H, D), generator=gen).to(BF).cuda()
    xs = [row[:, :H], row[:, H:2 * H]]
    v = row[:, 2 * H:].contiguous()
    q, k = (torch.empty((T, H, D), dtype=BF, device="cuda") for _ in range(2))
    args = (T, D, D, False, moe.MOE_BF16)
    moe.moe_qk_norm_rope(*args, 1e-6, pos, freq, dict(x=xs[0], y=q, weight=w[0]),
                         dict(x=xs[1], y=k, weight=w[1]))
    o = torch.empty((T, H, D), dtype=BF, device="cuda")
    chunks = torch.empty((1, H, (T + 63) // 64, D, D), device="cuda")
    ws = torch.empty(max(moe.moe_gdr_workspace_size(1, T, H, D, D),
                         moe.moe_gdr_backward_workspace_size(1, T, H, D, D),
                         moe.moe_qk_norm_rope_backward_workspace_size(T, D, H, H)),
                     dtype=torch.uint8, device="cuda")
    moe.moe_gdr_forward(1, T, H, D, D, q, k, v, beta, g, None, D ** -0.5, o, None, chunks, ws)
    dq, dk, dv = (torch.empty((T, H, D), device="cuda") for _ in range(3))
    dbeta, dg = (torch.empty((T, H), device="cuda") for _ in range(2))
    moe.moe_gdr_backward(1, T, H, D, D, q, k, v, beta, g, D ** -0.5, d_o, None, chunks, dq, dk, dv,
                         dbeta, dg, None, ws)
    dxs = [torch.empty((T, H, D), dtype=BF, device="cuda") for _ in range(2)]
    dws = [torch.empty(D, device="cuda") for _ in range(2)]
    moe.moe_qk_norm_rope_backward(
        *args, moe.MOE_F32, 1e-6, pos, freq,
        dict(x=xs[0], dy=dq, dx=dxs[0], weight=w[0], dweight=dws[0]),
        dict(x=xs[1], dy=dk, dx=dxs[1], weight=w[1], dweight=dws[1]), ws)
    torch.cuda.synchronize()
    assert moe.moe_gdr_device_status() == moe.MOE_OK
    seq = lambda t: f64(t)[None]  # noqa: E731
    ref = LA.gated_delta_rule_backward(seq(q), seq(k), seq(v), seq(beta), seq(g), seq(d_o))
    for x, wi, dy, dx, dw in zip(xs, w, (ref["dq"][0], ref["dk"][0]), dxs, dws):
        dx_ref, dw_ref = SM.qk_norm_rope_backward(f64(x), f64(wi), f64(pos), f64(freq), D, False,
                                                  1e-6, dy)
        # 5e-3: the bar of the delta rule's own gradients, which are the input here
        assert relerr(f64(dx), dx_ref) <= 5e-3
        assert relerr(f64(dw), dw_ref.sum(0)) <= 5e-3


def test_captured_and_replayed_on_another_stream():
    """The calls captured into graphs on a side stream and replayed with new inputs: each graph
    has its own buffers, so two of them may run at once."""
    N, H, D = 200, 2, 64
    gen = torch.Generator().manual_seed(11)
    freq = (1e4 ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()
    weight = torch.ones(D, device="cuda")

    def buffers():
        r = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
        e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
        return dict(x=r(N, H, D), y=e(N, H, D), g=-r(N, H * D).abs(), h=e(N, H * D), h_T=e(1, H * D),
                    chunks=e((N + 63) // 64, H * D), dh=r(N, H * D), dg=e(N, H * D),
                    dx=e(N, H * D), dy=e(N, H, D), dw=e(D), state=r(4, H * D), hs=e(2, H * D),
                    slot=torch.tensor([2, 0], dtype=torch.int32).cuda(),
                    ws=torch.empty(moe.moe_qk_norm_rope_backward_workspace_size(N, D, H, 0),
                                   dtype=torch.uint8, device="cuda"))

    def chain(b):
        f = moe.MOE_F32
        moe.moe_qk_norm_rope(N, D, D, False, f, 1e-6, pos, freq,
                             dict(x=b["x"], y=b["y"], weight=weight), None)
        y = b["y"].view(N, H * D)
        moe.moe_glr_forward(N, H * D, 1, None, 1, f, b["g"], y, None, b["h"], b["h_T"],
                            b["chunks"])
        moe.moe_glr_backward(N, H * D, 1, None, 1, f, b["g"], y, None, b["chunks"], b["dh"], None,
                             b["dg"], b["dx"], None)
        moe.moe_qk_norm_rope_backward(N, D, D, False, f, f, 1e-6, pos, freq,
                                      dict(x=b["x"], dy=b["dx"].view(N, H, D), dx=b["dy"],
                                           weight=weight, dweight=b["dw"]), None, b["ws"])
        moe.moe_glr_step(2, H * D, 1, f, b["g"][:2], y[:2], b["slot"], 4, b["state"], b["hs"])

    outs = ("y", "h", "h_T", "chunks", "dg", "dx", "dy", "dw", "state", "hs")
    both, eager, graphs, streams = [buffers(), buffers()], [], [], []
    for b in both:
        kept = {n: t.clone() for n, t in b.items()}
        chain(b)
        eager.append({n: b[n].clone() for n in outs})
        for n, t in kept.items():
            b[n].copy_(t)
        torch.cuda.synchronize()
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            chain(b)
        graphs.append(graph)
        streams.append(s)
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for b, e in zip(both, eager):
        for n in outs:
            assert torch.equal(b[n], e[n]), n
    new = torch.randn((N, H, D), generator=gen).cuda()
    for b, graph in zip(both, graphs):
        b["x"].copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in outs if n not in ("state", "hs")}
        chain(b)
        torch.cuda.synchronize()
        assert all(torch.equal(b[n], t) for n, t in got.items())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, D, lengths", [(4, 392, [4]), (700, 136, [300, 0, 395]),
                                           (4099, 320, [4099])])
def test_training_passes_back_to_back_on_two_states(N, D, lengths, dtype):
    """Passes that follow one another without a wait, on two states in turn: every pass of a state
    has the bits of its first one, and the inputs stay as they were."""
    i, other = (glr_inputs((N, D, lengths, True, dtype, True), seed=s) for s in (3, 4))
    states = []
    for v in (i, other):
        gen = torch.Generator().manual_seed(5)
        states.append(dict(v, dh=torch.randn((N, D), generator=gen).to(dtype).cuda(),
                           dh_T=torch.randn((len(lengths), D), generator=gen).cuda()))

    def run(s):
        e = lambda *n, dt=F32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
        n_seq = len(lengths)
        out = dict(h=e(N, D, dt=dtype), h_T=e(n_seq, D), chunks=e((N + 63) // 64, D),
                   dg=e(N, D, dt=dtype), dx=e(N, D, dt=dtype), dh0=e(n_seq, D))
        off, head = offsets_arg(s), (moe.MOE_GLR_MIX, CODE[dtype])
        g, x = s["g"][:, :D].contiguous(), s["x"][:, :D].contiguous()
        h0 = s["h0"]

        def call():
            moe.moe_glr_forward(N, D, n_seq, off, *head, g, x, h0, out["h"], out["h_T"],
                                out["chunks"])
            moe.moe_glr_backward(N, D, n_seq, off, *head, g, x, h0, out["chunks"], s["dh"],
                                 s["dh_T"], out["dg"], out["dx"], out["dh0"])

        return call, out, dict(g=g, x=x, h0=h0, dh=s["dh"], dh_T=s["dh_T"])

    runs = [run(s) for s in states]
    kept = [{n: t.clone() for n, t in r[2].items()} for r in runs]
    first = []
    for call, out, _ in runs:
        call()
        first.append({n: t.clone() for n, t in out.items()})
    for _ in range(10):
        for call, _, _ in runs:
            call()
    for (_, out, ins), want, before in zip(runs, first, kept):
        assert all(torch.equal(out[n], want[n]) for n in out)
        assert all(torch.equal(ins[n], before[n]) for n in ins)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_keep_the_order_of_their_stream(captured):
    """Launches are set up while the kernels before them end; what they read and write is still in
    the stream's order, among themselves and with other kernels: a long chain in which every call
    uses what the one before it wrote, and writes what that one read, has the bits of the same chain
    with a wait after every call."""
    B, H, D, N = 3, 2, 64, 300
    f, W = moe.MOE_F32, 2 * 64
    gen = torch.Generator().manual_seed(21)
    freq = (1e4 ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()
    w = torch.rand(D, generator=gen).cuda() + 0.5
    r = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    first = dict(x=r(N, H, D), y=r(N, H, D), g=-r(N, W).abs(), h=r(N, W), h_T=r(1, W),
                 c=r((N + 63) // 64, W), dg=r(N, W), dx=r(N, H, D), dw=r(D), st=r(4, W),
                 hs=r(2, W), S=r(B, H, D, D), q=r(B, H, D).to(BF), k=r(B, H, D).to(BF),
                 v=r(B, H, D).to(BF), o=r(B, H, D).to(BF), o2=r(B, H, D).to(BF),
                 beta=torch.sigmoid(r(B, H)), gg=-r(B, H).abs())
    ws = torch.empty(moe.moe_qk_norm_rope_backward_workspace_size(N, D, H, 0), dtype=torch.uint8,
                     device="cuda")

    def chain(b, wait):
        x, y, dx = b["x"], b["y"], b["dx"]
        calls = [
            lambda: moe.moe_qk_norm_rope(N, D, D, False, f, 1e-6, pos, freq,
                                         dict(x=x, y=y, weight=w), None),
            lambda: moe.moe_glr_forward(N, W, 1, None, 1, f, b["g"], y.view(N, W), b["h_T"], b["h"],
                                        b["h_T"], b["c"]),
            lambda: moe.moe_glr_backward(N, W, 1, None, 1, f, b["g"], y.view(N, W), None, b["c"],
                                         b["h"], b["h_T"], b["dg"], dx.view(N, W), None),
            lambda: moe.moe_qk_norm_rope_backward(N, D, D, False, f, f, 1e-6, pos, freq,
                                                  dict(x=x, dy=dx, dx=y, weight=w,
                                                       dweight=b["dw"]), None, ws),
            lambda: x.add_(y, alpha=0.01),
            lambda: b["dg"].clamp_(max=0),
            lambda: moe.moe_glr_step(2, W, 1, f, b["dg"][:2], x.view(N, W)[:2], None, 4, b["st"],
                                     b["hs"]),
            lambda: moe.moe_gdr_step(B, H, D, D, b["q"], b["k"], b["v"], b["beta"], b["gg"], None, B,
                                     0.125, b["S"], b["o"]),
            lambda: moe.moe_gdr_step(B, H, D, D, b["o"], b["k"], b["v"], b["beta"], b["gg"], None, B,
                                     0.125, b["S"], b["o2"]),
            lambda: b["q"].copy_(b["o2"]).add_(1),
            lambda: b["v"].copy_(b["o"]).sub_(1),
            lambda: b["g"].copy_(b["dg"]).sub_(0.1),
        ]
        for _ in range(12):
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()

    want = {n: t.clone() for n, t in first.items()}
    chain(want, True)
    torch.cuda.synchronize()
    got = {n: t.clone() for n, t in first.items()}
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain(got, False)
        for n, t in first.items():
            got[n].copy_(t)
        graph.replay()
    else:
        chain(got, False)
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(got[n].view(torch.int16), want[n].view(torch.int16)), n


FIRST_CALL = """
import torch
from top_routing_grouped_gemm_gb300 import moe
N, H, D, B = 130, 2, 64, 3
f, dev = moe.MOE_F32, "cuda"
r = lambda *s: torch.randn(s, device=dev)
x, y, dx, w, dw = r(N, H, D), r(N, H, D), r(N, H, D), r(D), r(D)
pos = torch.arange(N, dtype=torch.int32, device=dev)
freq = 1e4 ** -(torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
ws = torch.empty(1 << 22, dtype=torch.uint8, device=dev)
g, v, h, dh, dg, dv = -r(N, 128).abs(), r(N, 128), r(N, 128), r(N, 128), r(N, 128), r(N, 128)
c, h_T, st, hs = r(3, 128), r(1, 128), r(B, 128), r(B, 128)
bf = lambda *s: r(*s).bfloat16()
q, k, vv, o, S = bf(B, H, D), bf(B, H, D), bf(B, H, D), bf(B, H, D), r(B, H, D, D)
beta, gg = torch.sigmoid(r(B, H)), -r(B, H).abs()
def calls():
    moe.moe_qk_norm_rope(N, D, D, False, f, 1e-6, pos, freq, dict(x=x, y=y, weight=w), None)
    moe.moe_qk_norm_rope_backward(N, D, D, False, f, f, 1e-6, pos, freq,
                                  dict(x=x, dy=y, dx=dx, weight=w, dweight=dw), None, ws)
    moe.moe_glr_forward(N, 128, 1, None, 1, f, g, v, None, h, h_T, c)
    moe.moe_glr_backward(N, 128, 1, None, 1, f, g, v, None, c, dh, None, dg, dv, None)
    moe.moe_glr_step(B, 128, 1, f, g[:B], v[:B], None, B, st, hs)
    moe.moe_gdr_step(B, H, D, D, q, k, vv, beta, gg, None, B, 0.125, S, o)
outs = (y, dx, dw, h, h_T, c, dg, dv, st, hs, S, o)
start = [t.clone() for t in (st, S)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
st.copy_(start[0]); S.copy_(start[1])
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
print("same")
"""


def test_first_calls_of_a_process_are_captured():
    """What the library prepares on first use (kernel attributes, the room for clusters) may be
    prepared while a stream is captured: in a process of its own, whose first calls are a graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True,
                         text=True, timeout=300)
    assert got.returncode == 0 and "same" in got.stdout, got.stderr[-2000:]
