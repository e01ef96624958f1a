"""What stands around the experts at its edges: experts out of range, infinite biases, calls from several
threads, outputs over inputs, orders and values next to a rounding.

Tolerances as in test_gpu_moe_block.py."""

import ctypes
import decimal
import threading

import numpy as np
import pytest
import torch

from oracle import moe_block as MB
from parity_util import f64
from rounding import Rounded
from test_gpu_moe_block import (BF, CODE, EPS, F32, LAST, SCALE, SIG, SOFT, U, check_w4, randn, run_select,
                                w4_case)
from top_routing_grouped_gemm_gb300 import moe

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------ 4-bit experts

def guarded(n, dtype, fill=0x5A):
    """n bytes in the middle of a larger array of bytes `fill`, and whether those are as they were."""
    around = 1 << 20
    whole = torch.full((n + 2 * around,), fill, dtype=torch.uint8, device="cuda")
    return (whole[around:around + n].view(dtype),
            lambda: bool((whole[:around] == fill).all() and (whole[around + n:] == fill).all()))


def run_w4_guarded(case, w, x, idx, gate, status=None):
    """y, whose memory and the workspace's lie between bytes that no call may change."""
    T, d, E, k, F = case[:5]
    p = moe.Problem(T, d, E, k, F)
    packed = [moe.W4Weights(*(None if t is None else t.cuda() for t in m)) for m in w]
    ws, ws_kept = guarded(moe.moe_w4_expert_ffn_workspace_size(p), torch.uint8)
    y, y_kept = guarded(T * d * 2, BF)
    y = y.view(T, d)
    moe.moe_w4_expert_ffn(p, x.cuda(), idx.cuda(), gate.cuda(), *packed, y, ws, status)
    torch.cuda.synchronize()
    assert ws_kept() and y_kept()
    return y


BAD = {"first": [0], "middle": [1], "last": [-1], "first and last": [0, -1], "all": slice(None)}


# T, d, E, k, F, group, zeros, experts used; F far larger than d, and d than F
@pytest.mark.parametrize("where", BAD)
@pytest.mark.parametrize("case", [(1, 128, 5, 4, 1152, 64, True, None), (1, 64, 3, 3, 4096, 32, False, None),
                                  (1, 2048, 6, 5, 128, 128, True, None), (1, 512, 9, 8, 512, 128, False, None),
                                  (1, 64, 1, 1, 4096, 64, False, None), (1, 64, 40, 32, 256, 32, False, None)],
                         ids=str)
def test_w4_one_token_with_experts_out_of_range(case, where):
    """They contribute nothing and are reported; the others are as ever, time after time."""
    w, x, idx, gate = w4_case(case)
    bad = torch.zeros(case[3], dtype=torch.bool)
    bad[BAD[where] if case[3] > 1 else [0]] = True
    idx[0, bad] = torch.tensor([-1, case[2], 2 ** 31 - 1, -2 ** 31] * 8, dtype=torch.int32)[:int(bad.sum())]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = run_w4_guarded(case, w, x, idx, gate, status)
    assert int(status.item()) == 6
    check_w4(case, w, x, idx, gate, y)
    if where == "all":
        assert not y.any()
    for _ in range(10):
        assert torch.equal(run_w4_guarded(case, w, x, idx, gate), y)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("T", [1, 3])
def test_w4_experts_out_of_range_read_nobodys_weights(T, value):
    """What the experts that nobody names have for scales means nothing."""
    case = (T, 512, 6, 4, 256, 64, True, None)
    w, x, idx, gate = w4_case(case)
    idx[idx == 0] = 5
    idx[:, 1] = -1
    want = run_w4_guarded(case, w, x, idx, gate)
    for m in w:
        m[1][0] = value
    assert torch.equal(run_w4_guarded(case, w, x, idx, gate), want)
    assert not want.isnan().any()


# ------------------------------------------------------------------------ routing

INF, NAN = float("inf"), float("nan")

# what a bias has, by group and expert of the group
BIASES = {
    "one +inf": {(5, 2): INF},
    "two +inf in a group": {(6, 0): INF, (6, 3): INF},
    "+inf in two groups": {(2, 1): INF, (7, 2): INF},
    "+inf and two of them": {(1, 1): INF, (4, 0): INF, (4, 3): INF},
    "three +inf in a group": {(3, 0): INF, (3, 1): INF, (3, 3): INF},
    "-inf here and there": {(0, 0): -INF, (3, 2): -INF, (3, 3): -INF},
    "groups of -inf": {(g, e): -INF for g in (0, 1, 2, 4, 5) for e in range(4)},
    "all groups but one of -inf": {(g, e): -INF for g in range(8) if g != 6 for e in range(4)},
    "nothing but -inf": {(g, e): -INF for g in range(8) for e in range(4)},
    "one of a group left": {(g, e): -INF for g in range(8) for e in range(4) if e != g % 4},
    "NaN": {(0, 1): NAN, (4, 0): NAN, (4, 1): NAN},
    "+inf, -inf and NaN": {(0, 1): -INF, (2, 0): INF, (4, 1): NAN, (7, 3): INF, (7, 1): -INF},
}


@pytest.mark.parametrize("kept", [1, 2, 3, 7])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("size", [4, 5, 32])
@pytest.mark.parametrize("what", BIASES)
def test_route_select_with_groups_and_infinite_biases(what, size, score, best, kept):
    """+inf puts an expert, and its group with it, first, -inf and NaN last; equal ones by index."""
    T, groups, k = 20, 8, 3
    case = (T, groups * size, k, score, groups, kept, best, True, True, F32)
    gen = torch.Generator().manual_seed(size)
    logits = randn(gen, *case[:2])
    bias = randn(gen, case[1]) * (0.05 if score == SIG else 0.3 / case[1])
    for (group, expert), value in BIASES[what].items():
        bias[group * size + expert] = value
    if "one of a group left" in what:
        bias.view(groups, size)[:, 4:] = -INF
    if "-inf" in what and "here" not in what and "+" not in what:
        bias.view(groups, size)[:, 4:] = bias.view(groups, size)[:, :1]
    idx, gate, _ = run_select(case, logits.cuda(), bias.cuda())
    want, ref, _ = MB.select(f64(logits), f64(bias), k, score == SIG, groups, kept, best, True, 2.5)
    assert np.array_equal(idx, want)
    assert np.allclose(gate, ref, rtol=64 * U, atol=0)


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("size", [2, 4])
def test_route_select_of_groups_of_both_infinities(size, score):
    """The best two of a group are +inf and -inf: last, whatever else there is."""
    E, T, k = 4 * size, 9, 2
    logits = randn(torch.Generator().manual_seed(size), T, E)
    bias = torch.zeros(E)
    bias[size:2 * size] = -INF
    bias[size + 1], bias[0] = INF, -0.5
    case = (T, E, k, score, 4, 3, 2, True, True, F32)
    idx, _, _ = run_select(case, logits.cuda(), bias.cuda())
    without = torch.cat([logits[:, :size], logits[:, size:2 * size] * 0 - 100, logits[:, 2 * size:]], 1)
    s = torch.sigmoid(without.double()) if score == SIG else torch.softmax(logits.double(), -1)
    c = s + torch.where(bias.isinf(), -9.0, bias.double())
    assert np.array_equal(idx, c.sort(-1, descending=True).indices[:, :k].numpy())


# ------------------------------------------------------------------------ calls from several threads

def together(calls, times):
    """Each call `times` times in a thread and on a stream of its own, all at once; its statuses."""
    start, statuses = threading.Barrier(len(calls)), [set() for _ in calls]

    def run(call, seen):
        stream = torch.cuda.Stream()
        start.wait()
        for i in range(times):
            seen.add(call(stream.cuda_stream))
            if i % 256 == 255:
                stream.synchronize()

    threads = [threading.Thread(target=run, args=a) for a in zip(calls, statuses)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return set().union(*statuses)


def ptr(t):
    return None if t is None else t.data_ptr()


def test_norms_with_and_without_gates_at_once():
    """Calls whose blocks want different amounts of shared memory, in threads beside each other."""
    N, D = 3, 256
    gen = torch.Generator().manual_seed(0)
    x, y, gate, dz = (randn(gen, N, D).cuda() for _ in range(4))
    calls, backs, outs, lib = [], [], [], moe.lib()
    for kind, a in ((moe.MOE_GATE_NONE, None), (moe.MOE_GATE_VALUE, gate)) * 2:
        z, n, dx, dy = (torch.empty_like(x) for _ in range(4))
        block = moe.moe_block_in(N, D, 1, 1, 1e-6, 0.5, kind, 1, 1, ptr(x), D, ptr(y), D, ptr(a), D, None, None)
        grads = moe.moe_block_grads(ptr(dz), D, ptr(dz), D, 1, ptr(dx), D, ptr(dy), D, None, 0, None, None)
        b, g = (ctypes.addressof(c) for c in (block, grads))
        calls.append(lambda s, b=b, z=ptr(z), n=ptr(n), keep=block: lib.moe_block_norm(b, z, D, n, D, s))
        backs.append(lambda s, b=b, g=g, keep=(block, grads): lib.moe_block_norm_backward(b, g, None, 0, s))
        outs.append((z, n, dx, dy))
    assert [c(None) for c in calls + backs] == [0] * 8
    torch.cuda.synchronize()
    want = [[t.clone() for t in o] for o in outs]
    assert together(calls, 30000) == {0}
    assert together(backs, 30000) == {0}
    assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))


def test_w4_of_two_models_at_once():
    """One token through models of few and of many columns."""
    calls, ys, lib = [], [], moe.lib()
    for d in (64, 2560) * 2:
        case = (1, d, 4, 2, 64, 32, True, None)
        w, x, idx, gate = w4_case(case)
        p = moe.Problem(*case[:5])
        packed = [moe.W4Weights(*(t.cuda() for t in m)) for m in w]
        ws = torch.empty(moe.moe_w4_expert_ffn_workspace_size(p), dtype=torch.uint8, device="cuda")
        x, idx, gate, y = x.cuda(), idx.cuda(), gate.cuda(), torch.empty((1, d), dtype=BF, device="cuda")
        shapes = (4, 64, d), (4, 64, d), (4, d, 64)
        mats = [m.c("w", s, 0) for m, s in zip(packed, shapes)]
        args = (p.c(), ptr(x), ptr(idx), ptr(gate), *mats, ptr(y), ptr(ws), ws.numel(), None)
        calls.append(lambda s, args=args, keep=(p, packed, ws, x, idx, gate): lib.moe_w4_expert_ffn(*args, s))
        ys.append(y)
    assert [c(None) for c in calls] == [0] * 4
    torch.cuda.synchronize()
    want = [y.clone() for y in ys]
    assert together(calls, 20000) == {0}
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


# ------------------------------------------------------------------------ 4-bit experts: roundings

# Sums over the codes times the values, less the zero times the sum of the values: both parts' sizes count.
# 16 products and a sum are added at once, each cut off at 2^-24 of the largest (18 halves of a step to 16
# columns of a group); a group's sum is corrected, scaled and added to the others (cols / group); the sums
# of the values, the joins of 8 warps and the last factors are 40 more.
def tight(cols, group):
    return (18 * group / 16 + cols / group + 40) * U


def code_and_zero(m):
    codes, scales, zeros = m[0].numpy(), f64(m[1]), None if m[2] is None else m[2].numpy()
    code = MB.w4_values(codes, np.ones(scales.shape), np.zeros(scales.shape, np.uint8))
    zero = np.repeat(np.full(scales.shape, 8.0) if zeros is None else zeros.astype(float),
                     code.shape[-1] // scales.shape[-1], -1)
    scale = np.repeat(scales, code.shape[-1] // scales.shape[-1], -1)
    return (code - zero) * scale, (code + zero) * scale


@pytest.mark.parametrize("small_codes", [False, True])
@pytest.mark.parametrize("case", [(1, 512, 6, 4, 256, 64, True, None), (1, 256, 3, 2, 1152, 128, False, None),
                                  (8, 384, 4, 3, 192, 32, True, None), (40, 256, 6, 2, 512, 128, True, None),
                                  (70, 192, 5, 3, 320, 64, False, None)], ids=str)
def test_w4_within_the_roundings_of_its_sums(case, small_codes):
    """The sizes of code and zero, and h in two parts (off by 2^-23, and by 2^-45 of its tile's largest)."""
    T, d, E, k, F, group, zeros = case[:7]
    w, x, idx, gate = w4_case(case, 3)
    if small_codes:  # 0 to 3, zeros 0 to 2
        w = [(m[0] & 0x33, m[1], torch.clamp(m[2], max=2) if zeros else None) for m in w]
    got = run_w4_guarded(case, w, x, idx, gate)
    W, size = zip(*(code_and_zero(m) for m in w))
    x, g, idx = f64(x), f64(gate), idx.numpy()
    value, error = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            a, b = (Rounded(W[i][e] @ x[t], tight(d, group) * (size[i][e] @ np.abs(x[t]))) for i in (0, 1))
            h = a / (1.0 + (-a).exp()) * b * g[t, j]
            most = np.repeat(np.abs(h.v).reshape(-1, 64).max(-1), 64)
            parts = 2.0 ** -23 * np.abs(h.v) + 2.0 ** -45 * most
            value[t] += W[2][e] @ h.v
            error[t] += np.abs(W[2][e]) @ h.e + size[2][e] @ (
                parts + (tight(F, group) + k * F / group * U) * np.abs(h.v))
    Rounded(value, error).close(f64(got), LAST[BF], "y")


def one_weight(E, rows, cols, group, row, col, scale):
    """Weights of which one row, or all (None), has code 15 at a column; zeros 0."""
    codes = torch.zeros((E, rows, cols // 2), dtype=torch.uint8)
    codes[:, slice(None) if row is None else row, col // 2] = 15 << col % 2 * 4
    scales = torch.full((E, rows, cols // group), scale).to(BF)
    return codes, scales, torch.zeros(scales.shape, dtype=torch.uint8)


def through_one_weight(T, col, x, scale):
    """(y, what it has to be): x's column through gate and up, h's column 70 through all rows of down."""
    d, F, group = 128, 128, 32
    case = (T, d, 2, 1, F, group, True, None)
    w = [one_weight(2, F, d, group, 70, col, scale)] * 2 + [one_weight(2, d, F, group, None, 70, 0.125)]
    y = run_w4_guarded(case, w, x, torch.ones((T, 1), dtype=torch.int32), torch.ones((T, 1)))
    a = 15 * float(torch.tensor(scale).to(BF)) * f64(x)[:, col]
    return f64(y), (a / (1 + np.exp(-a)) * a * 15 * 0.125)[:, None]


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("col", [2, 3, 38, 71, 127])
@pytest.mark.parametrize("small", [1 + 2 ** -7, 2 - 2 ** -7])
def test_w4_values_from_2_to_the_minus_27_of_a_rows_largest_on_keep_their_bits(T, col, small):
    """In columns that meet the 16-fold codes, which have the fewest bits.  A lost last bit (2^-7 of x) would
    show twice over; what is allowed is the last rounding, and 64 of fp32's."""
    x = torch.zeros((T, 128), dtype=BF)
    x[:, 0], x[:, col] = 2.0 ** 27, small
    y, want = through_one_weight(T, col, x, 1 / 16)
    assert (np.abs(y - want) <= (2.0 ** -8 / 2 + 2.0 ** -8 / 2 * 2.0 ** -7 + 64 * U) * np.abs(want)).all()


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("scale, value", [(2.0 ** 115, 2.0 ** -118), (2.0 ** -126, 2.0 ** 123),
                                          (2.0 ** -133, 2.0 ** 126)])
def test_w4_scales_from_the_smallest_to_2_to_the_115(T, scale, value):
    x = torch.zeros((T, 128), dtype=BF)
    x[:, 5] = value
    y, want = through_one_weight(T, 5, x, scale)
    assert want.all() and (np.abs(y - want) <= (2.0 ** -8 + 64 * U) * np.abs(want)).all()


# ------------------------------------------------------------------------ outputs over inputs

# N, D, stream, type; the longest rows are read from memory each time that they are wanted
IN_PLACE = [(9, 72, F32, F32), (700, 1000, BF, BF), (40, 4096, F32, BF), (30, 6152, BF, BF),
            (200, 8192, F32, BF), (5, 8200, F32, F32), (400, 8200, F32, BF), (7, 16384, BF, BF)]


def in_place_inputs(case, post):
    N, D, st, dt = case
    gen = torch.Generator().manual_seed(N + D)
    x, dz = (randn(gen, N, D).to(st).cuda() for _ in range(2))
    y, a, dn = (randn(gen, N, D).to(dt).cuda() for _ in range(3))
    wp, wn = ((1 + 0.2 * randn(gen, D)).cuda() for _ in range(2))
    return x, y, a, dz, dn, wp if post else None, wn


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("case", IN_PLACE, ids=str)
def test_block_norm_over_its_inputs(case, post):
    """z over x; n over y, and over a gate of each value."""
    N, D, st, dt = case
    x, y, a, _, _, wp, wn = in_place_inputs(case, post)
    head = (N, D, CODE[st], CODE[dt], EPS, SCALE)
    rest = (moe.MOE_GATE_VALUE, True)
    z, n = torch.empty_like(x), torch.empty_like(y)
    moe.moe_block_norm(*head, x, y, *rest, a, post, wp, wn, z, n)
    for over in ("y", "gate"):
        x2, y2, a2 = x.clone(), y.clone(), a.clone()
        n2 = y2 if over == "y" else a2
        moe.moe_block_norm(*head, x2, y2, *rest, a2, post, wp, wn, x2, n2)
        assert torch.equal(x2, z) and torch.equal(n2, n), over


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("case", IN_PLACE, ids=str)
def test_block_norm_backward_over_its_inputs(case, post):
    """dx over dz; dy over y, and over dn; a gate's gradient over the gate."""
    N, D, st, dt = case
    x, y, a, dz, dn, wp, wn = in_place_inputs(case, post)
    ws = torch.empty(moe.moe_block_norm_backward_workspace_size(N, D, 3), dtype=torch.uint8, device="cuda")

    def back(y, a, dz, dn, dx, dy, da):
        dwp, dwn = torch.empty(D, device="cuda") if post else None, torch.empty(D, device="cuda")
        moe.moe_block_norm_backward(N, D, CODE[st], CODE[dt], EPS, SCALE, x, y, moe.MOE_GATE_VALUE, True, a,
                                    post, wp, wn, dz, CODE[dt], dn, dx, dy, da, dwp, dwn, ws)
        return [dx, dy, da, dwn] + [dwp] * post

    want = back(y, a, dz, dn, torch.empty_like(x), torch.empty_like(y), torch.empty_like(a))
    for over in ("y", "dn"):
        y2, a2, dz2, dn2 = (t.clone() for t in (y, a, dz, dn))
        got = back(y2, a2, dz2, dn2, dz2, y2 if over == "y" else dn2, a2)
        assert all(torch.equal(g, w) for g, w in zip(got, want)), over


# ------------------------------------------------------------------------ nearly equal scores

def ulps(l, most, gen):
    """Logits moved by up to `most` steps of fp32."""
    step = torch.randint(-most, most + 1, l.shape, generator=gen, dtype=torch.int32)
    return (l.contiguous().view(torch.int32) + step).view(torch.float32)


def near_equal(score, T, E, near, gen):
    """Logits and a bias: the scores and biases of `near` experts of a row add up to nearly one value, the
    others' to far less."""
    value = 0.6 if score == SIG else 1 / 64
    bias = randn(gen, E) * 0.05 * value
    order = torch.rand((T, E), generator=gen).argsort(1)
    s = (value - bias.double()).repeat(T, 1)
    if score == SIG:
        l, rest = torch.logit(s), torch.full((T, 1), -1.0, dtype=torch.float64)
    else:  # shares; the others have what is left, or all of them that much more
        left = 1 - (s * (order < near)).sum(-1, keepdim=True)
        s = s + left / E if near == E else s
        l, rest = s.log(), (left / max(1, E - near)).clamp(min=1e-9).log()
    return torch.where(order < near, ulps(l.float(), 8, gen), rest.float().expand(T, E)), bias


def near_pairs(score, T, groups, size, gen):
    """Logits: the best two scores of every group have nearly one sum."""
    a = torch.rand((T, groups), generator=gen).double() - 0.5
    if score == SIG:
        b = torch.logit(1.2 - torch.sigmoid(a.float().double()))
    else:
        b = torch.log(2.0 - torch.exp(a.float().double()))
    l = torch.full((T, groups, size), -6.0) - torch.rand((T, groups, size), generator=gen)
    l[..., 1], l[..., size - 1] = a.float(), ulps(b.float(), 4, gen)
    return l.view(T, -1)


def check_order(l, bias, idx, score, groups, kept, best, k):
    """Against sums in 40 digits.  What is closer than 2^-40 may be in either order: such rows are left out,
    and there are few."""
    D, skipped = decimal.Decimal, 0
    with decimal.localcontext() as context:
        context.prec = 40
        tie = D(2) ** -40
        for t, row in enumerate(l.tolist()):
            if score == SIG:
                c = [1 / (1 + (-D(v)).exp()) for v in row]
            else:
                e = [D(v).exp() for v in row]
                total = sum(e)
                c = [v / total for v in e]
            c = c if bias is None else [v + D(b) for v, b in zip(c, bias.tolist())]
            size = len(row) // groups
            worth = [sum(sorted(c[g * size:(g + 1) * size])[::-1][:best]) for g in range(groups)]
            order = sorted(range(groups), key=lambda g: (-worth[g], g))
            near = kept < groups and worth[order[kept - 1]] - worth[order[kept]] < tie
            key = row if bias is None else c
            want = sorted((e for e in range(len(row)) if e // size in order[:kept]), key=lambda e: (-key[e], e))
            if bias is not None:
                near |= any(0 < c[a] - c[b] < tie for a, b in zip(want[:k], want[1:k + 1]))
            if near:
                skipped += 1
            else:
                assert idx[t].tolist() == want[:k], t
    assert skipped <= len(l) // 8


# experts, near ones: all of them, more than a list of 64 holds (of sigmoid scores), fewer
@pytest.mark.parametrize("E, near", [(64, 64), (512, 200), (512, 40), (300, 50)])
@pytest.mark.parametrize("groups, kept, best", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_route_select_of_some_nearly_equal_scores(score, groups, kept, best, E, near):
    T, k = 24, 8
    if score == SOFT:
        near = min(near, 50) if E > 64 else near
    case = (T, E, k, score, groups, kept, best, True, True, F32)
    l, bias = near_equal(score, T, E, near, torch.Generator().manual_seed(E + near))
    idx, _, _ = run_select(case, l.cuda(), bias.cuda())
    check_order(l, bias, idx, score, groups, kept, best, k)


@pytest.mark.parametrize("groups, size, kept", [(16, 4, 5), (8, 5, 3), (30, 32, 11), (32, 4, 31)])
@pytest.mark.parametrize("score", [SIG, SOFT])
def test_route_select_of_groups_whose_best_two_add_up_to_nearly_the_same(score, groups, size, kept):
    T, k = 24, 5
    case = (T, groups * size, k, score, groups, kept, 2, True, False, F32)
    l = near_pairs(score, T, groups, size, torch.Generator().manual_seed(groups))
    idx, _, _ = run_select(case, l.cuda(), None)
    check_order(l, None, idx, score, groups, kept, 2, k)


# ------------------------------------------------------------------------ 4-bit experts: waits that run out

@pytest.fixture
def impatient():
    """Ends the self-test of the waits whatever the test does."""
    yield
    moe.moe_selftest_w4_waits(0)


# in one strip of a team and in several, by one warp of a team and by all, with pieces at a row's end
@pytest.mark.parametrize("case", [(1, 2048, 5, 4, 1152, 32, False, None), (1, 64, 2, 1, 64, 32, False, None),
                                  (1, 2560, 3, 3, 320, 32, False, None), (3, 1152, 4, 2, 2048, 32, False, None),
                                  (40, 512, 8, 4, 640, 32, False, None)], ids=str)
def test_w4_copies_that_never_arrive_end_by_themselves_and_harm_nobody(case, impatient):
    """One copy of one warp is missing, early and late, in each product.  The launch ends and says so; what
    runs beside it and after it has its bits."""
    w, x, idx, gate = w4_case(case)
    p = moe.Problem(*case[:5])
    packed = [moe.W4Weights(m[0].cuda(), m[1].cuda()) for m in w]
    x, idx, gate = x.cuda(), idx.cuda(), gate.cuda()
    status, o_status = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    y, o_y = (torch.empty(case[:2], dtype=BF, device="cuda") for _ in range(2))
    ws, o_ws = (torch.empty(moe.moe_w4_expert_ffn_workspace_size(p), dtype=torch.uint8, device="cuda")
                for _ in range(2))
    call = lambda: moe.moe_w4_expert_ffn(p, x, idx, gate, *packed, y, ws, status)  # noqa: E731
    other = lambda: moe.moe_w4_expert_ffn(p, x, idx, gate, *packed, o_y, o_ws, o_status)  # noqa: E731
    call()
    want = y.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for down in (False, True):
        gave_up = 0
        for block, warp, copy in [(0, 0, 0), (1, 0, 0), (0, 3, 0), (2, 7, 1), (0, 0, 2), (3, 1, 3), (0, 1, 5)]:
            status.zero_()
            torch.cuda.synchronize()
            moe.moe_selftest_w4_waits(4, down, block, warp, copy)
            call()
            moe.moe_selftest_w4_waits(0)
            with torch.cuda.stream(side):
                other()
            torch.cuda.synchronize()
            assert int(status) in (0, 5) and int(o_status) == 0  # MOE_ERR_TIMEOUT where there is such a copy
            gave_up += int(status) == 5
            assert torch.equal(o_y, want) and (int(status) == 5 or torch.equal(y, want))
        assert gave_up > 0, down
    status.zero_()
    call()
    assert torch.equal(y, want) and int(status) == 0
