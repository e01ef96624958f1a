"""CPU checks of what stands around the experts: the oracle's gradients against central differences and
closed forms, and the refusals of the C ABI and of its binding, which answer before anything reaches a
GPU."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import moe_block as MB
from rounding import Rounded
from test_sequence_mixing_pins import difference
from top_routing_grouped_gemm_gb300 import build as B
from top_routing_grouped_gemm_gb300 import moe

FAKE = 0x10000  # never dereferenced: every call below fails its host checks first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


# ------------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
def test_select_gradient_against_differences(sigmoid, renormalise):
    rng = np.random.default_rng(0)
    logits, dgate = rng.normal(size=(3, 9)), rng.normal(size=(3, 4))
    idx = np.argsort(-logits, 1)[:, :4]
    idx[2, 1] = idx[2, 0]

    def value(l):
        return sum((MB._gates(l[t], idx[t], sigmoid, renormalise, 2.5)[0] * dgate[t]).sum()
                   for t in range(3))

    got = MB.select_backward(logits, idx, dgate, sigmoid, renormalise, 2.5)
    assert np.allclose(got, difference(value, logits), atol=1e-8)


def test_select_by_hand():
    # two groups of three: the best two of each give 1.1 and 1.2; the bias moves the selection only
    logits = np.log(np.array([[0.9, 0.2, 0.1, 0.6, 0.6, 0.55]]) / (1 - np.array([[0.9, 0.2, 0.1, 0.6, 0.6,
                                                                                  0.55]])))
    idx, gate, part = MB.select(logits, None, 2, True, 2, 1, 2, False, 2.0)
    assert idx.tolist() == [[3, 4]] and np.allclose(gate, 1.2)
    idx, gate, _ = MB.select(logits, np.array([0, 0.4, 0, 0, 0, 0.2]), 2, True, 2, 1, 2, True, 1.0)
    assert idx.tolist() == [[0, 1]] and np.allclose(gate, [[0.9 / 1.1, 0.2 / 1.1]])
    idx, _, _ = MB.select(logits, np.array([0, 0.4, 0, 0, 0, 0.2]), 3, True, 1, 1, 1, True, 1.0)
    assert idx.tolist() == [[0, 5, 1]]
    assert np.allclose(part.sum(), 1)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_block_norm_gradients_against_differences(sigmoid, post):
    rng = np.random.default_rng(1)
    x, y, dz, dn = (rng.normal(size=(3, 4)) for _ in range(4))
    gate, wp, wn = rng.normal(size=(3, 4)), rng.normal(size=4) + 2, rng.normal(size=4) + 2
    wp = wp if post else None

    def value(**new):
        v = dict(x=x, y=y, gate=gate, w_post=wp, w_pre=wn, **{})
        v.update(new)
        z, n = MB.block_norm(v["x"], v["y"], v["gate"], sigmoid, post, v["w_post"], v["w_pre"], 0.7, 1e-3)
        return (z * dz).sum() + (n * dn).sum()

    got = MB.block_norm_backward(x, y, gate, sigmoid, post, wp, wn, 0.7, 1e-3, dz, dn)
    for name, of, at in (("dx", "x", x), ("dy", "y", y), ("da", "gate", gate), ("dw_post", "w_post", wp),
                         ("dw_pre", "w_pre", wn)):
        if at is not None:
            assert np.allclose(got[name], difference(lambda t: value(**{of: t}), at), atol=1e-7), name


def test_w4_values_by_hand():
    codes = np.array([[[0x10, 0xF8]]], np.uint8)  # 0, 1, 8, 15
    assert MB.w4_values(codes, np.array([[[0.5]]]), None).tolist() == [[[-4, -3.5, 0, 3.5]]]
    assert MB.w4_values(codes, np.array([[[1.0, 2.0]]]), np.array([[[1, 15]]])).tolist() == [
        [[-1, 0, -14, 0]]]


def test_rounding_bounds_hold_in_fp32():
    """The bounds that the GPU tests use, against numpy's fp32."""
    rng = np.random.default_rng(2)
    a, b = (rng.normal(size=(50, 40)).astype(np.float32) for _ in range(2))
    A, Bb = Rounded(a), Rounded(b)
    ((A * Bb + A) / (Bb * Bb + 1.0)).close((a * b + a) / (b * b + np.float32(1)))
    (A * Bb).sum(1).close((a * b).sum(1))
    A.sigmoid().close(1 / (1 + np.exp(-a)))
    (A * A).sum(1).rsqrt().close(1 / np.sqrt((a * a).sum(1)))
    with pytest.raises(AssertionError):
        (A * Bb).close((a * b) * np.float32(1 + 2 ** -21))


# ------------------------------------------------------------------------ refusals of the C ABI

def select(T=8, E=64, k=4, score=1, groups=8, kept=4, best=2, renormalise=1, scale=1.0, dtype=1,
           logits=FAKE, ld=64, bias=FAKE, idx=FAKE, gate=FAKE, partials=FAKE):
    rule = moe.moe_route_rule(score, groups, kept, best, renormalise, scale)
    return moe.lib().moe_route_select(T, E, k, ctypes.addressof(rule), dtype, logits, ld, bias, idx, gate,
                                      partials, None)


def select_backward(T=8, E=64, k=4, score=1, renormalise=1, groups=8, kept=4, dtype=1, logits=FAKE, ld=64,
                    idx=FAKE, dgate=FAKE, dl=FAKE, sparse=FAKE, status=None):
    rule = moe.moe_route_rule(score, groups, kept, 2, renormalise, 1.0)
    return moe.lib().moe_route_select_backward(T, E, k, ctypes.addressof(rule), dtype, logits, ld, idx,
                                               dgate, dl, sparse, status, None)


@pytest.mark.parametrize("change, status", [
    (dict(T=0), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(score=2), INVALID),
    (dict(dtype=2), INVALID), (dict(groups=0), INVALID), (dict(groups=7), INVALID),
    (dict(kept=0), INVALID), (dict(kept=9), INVALID), (dict(ld=63), INVALID), (dict(logits=None), INVALID),
    (dict(k=33, kept=4), UNSUPPORTED), (dict(E=1032, ld=1032), UNSUPPORTED),
    (dict(E=660, groups=33, ld=660), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED),
    (dict(k=9, kept=1), INVALID), (dict(logits=FAKE + 2), UNSUPPORTED),
    (dict(idx=FAKE + 1), UNSUPPORTED), (dict(ld=(1 << 32) + 1), UNSUPPORTED),
])
def test_routing_refuses(change, status):
    assert select(**change) == status
    assert select_backward(**change) == status


@pytest.mark.parametrize("change, status", [
    (dict(best=0), INVALID), (dict(best=3), INVALID), (dict(groups=64, kept=30, best=2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(idx=None), INVALID),
    (dict(gate=None), INVALID), (dict(bias=FAKE + 2), UNSUPPORTED), (dict(gate=FAKE + 2), UNSUPPORTED),
    (dict(partials=FAKE + 1), UNSUPPORTED),
])
def test_selection_refuses(change, status):
    assert select(**change) == status


@pytest.mark.parametrize("change, status", [
    (dict(idx=None), INVALID), (dict(dgate=None), INVALID), (dict(dl=None, sparse=None), INVALID),
    (dict(score=0, renormalise=0), INVALID), (dict(dgate=FAKE + 2), UNSUPPORTED),
    (dict(sparse=FAKE + 2), UNSUPPORTED), (dict(dl=FAKE + 2), UNSUPPORTED),
    (dict(dtype=0, dl=FAKE + 1), UNSUPPORTED), (dict(status=FAKE + 1), UNSUPPORTED),
])
def test_selection_backward_refuses(change, status):
    assert select_backward(**change) == status


def test_routing_refuses_without_a_rule():
    assert moe.lib().moe_route_select(8, 64, 4, None, 1, FAKE, 64, None, FAKE, FAKE, None, None) == INVALID
    p = moe.Problem(T=64, d=128, E=16, k=4, F=128)
    call = lambda *a: moe.lib().moe_route_logits(*a, None, None)  # noqa: E731
    assert call(p.c(), FAKE, FAKE, None, None, FAKE, 1 << 40) == INVALID
    assert call(p.c(), None, FAKE, None, FAKE, FAKE, 1 << 40) == INVALID
    assert call(p.c(), FAKE + 2, FAKE, None, FAKE, FAKE, 1 << 40) == UNSUPPORTED
    assert call(p.c(), FAKE, FAKE, None, FAKE, FAKE, 16) == WORKSPACE
    assert moe.lib().moe_dispatch_logits_bwd(p.c(), FAKE, FAKE, FAKE, None, FAKE, FAKE, None) == INVALID
    assert moe.lib().moe_dispatch_logits_bwd(p.c(), FAKE + 8, FAKE, FAKE, FAKE, FAKE, FAKE,
                                             None) == UNSUPPORTED


BLOCK = dict(N=8, D=64, stream_dtype=1, dtype=0, eps=1e-6, scale=1.0, gate_kind=0, gate_sigmoid=0,
             post_norm=1, x=FAKE, ld_x=64, y=FAKE, ld_y=64, gate=None, ld_gate=0, w_post=FAKE, w_pre=FAKE)
GRADS = dict(dz=FAKE, ld_dz=64, dn=FAKE, ld_dn=64, dn_dtype=0, dx=FAKE, ld_dx=64, dy=FAKE, ld_dy=64,
             dgate=None, ld_dgate=0, dw_post=FAKE, dw_pre=FAKE)


def block(z=FAKE, ld_z=64, n=FAKE, ld_n=64, **change):
    b = moe.moe_block_in(**{**BLOCK, **change})
    return moe.lib().moe_block_norm(ctypes.addressof(b), z, ld_z, n, ld_n, None)


def block_backward(ws=FAKE, ws_bytes=1 << 40, grads=None, **change):
    b, g = moe.moe_block_in(**{**BLOCK, **change}), moe.moe_block_grads(**{**GRADS, **(grads or {})})
    return moe.lib().moe_block_norm_backward(ctypes.addressof(b), ctypes.addressof(g), ws, ws_bytes, None)


@pytest.mark.parametrize("change, status", [
    (dict(N=0), INVALID), (dict(D=0), INVALID), (dict(D=60), UNSUPPORTED), (dict(D=16392), UNSUPPORTED),
    (dict(N=(1 << 30) + 1), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(gate_kind=4), INVALID), (dict(gate_kind=-1), INVALID),
    (dict(gate_kind=1), INVALID), (dict(gate=FAKE), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(post_norm=0), INVALID), (dict(stream_dtype=2), INVALID),
    (dict(dtype=-1), INVALID), (dict(stream_dtype=0, dtype=1), UNSUPPORTED), (dict(ld_x=63), UNSUPPORTED),
    (dict(ld_x=56), INVALID), (dict(ld_y=-64), INVALID), (dict(ld_x=(1 << 32) + 8), UNSUPPORTED),
    (dict(x=FAKE + 8), UNSUPPORTED), (dict(y=FAKE + 8), UNSUPPORTED), (dict(w_post=FAKE + 4), UNSUPPORTED),
    (dict(w_pre=FAKE + 4), UNSUPPORTED), (dict(gate_kind=2, gate=FAKE + 2), UNSUPPORTED),
    (dict(gate_kind=1, gate=FAKE + 4), UNSUPPORTED), (dict(gate_kind=3, gate=FAKE, ld_gate=60), UNSUPPORTED),
    (dict(gate_kind=3, gate=FAKE, ld_gate=56), INVALID),
])
def test_block_norm_refuses(change, status):
    assert block(**change) == status
    assert block_backward(**change) == status


def test_block_norm_refuses_outputs():
    assert block(z=None) == INVALID and block(z=None, n=None) == INVALID
    assert block(n=None) == INVALID  # w_pre without n
    none = dict(y=None, post_norm=0, w_post=None)
    assert block(z=None, n=None, w_pre=None, **none) == INVALID
    assert block(z=FAKE + 4) == UNSUPPORTED and block(n=FAKE + 4) == UNSUPPORTED
    assert block(ld_z=0) == INVALID and block(ld_n=32) == INVALID and block(ld_n=68) == UNSUPPORTED
    assert moe.lib().moe_block_norm(None, FAKE, 64, FAKE, 64, None) == INVALID


@pytest.mark.parametrize("grads, status", [
    (dict(dx=None), INVALID), (dict(dz=None, dn=None), INVALID), (dict(dgate=FAKE), INVALID),
    (dict(dn_dtype=2), INVALID), (dict(dx=FAKE + 4), UNSUPPORTED), (dict(ld_dx=0), INVALID),
    (dict(ld_dy=32), INVALID), (dict(ld_dz=60), UNSUPPORTED), (dict(dy=FAKE + 2), UNSUPPORTED),
    (dict(dw_post=FAKE + 2), UNSUPPORTED), (dict(dw_pre=FAKE + 1), UNSUPPORTED),
])
def test_block_norm_backward_refuses(grads, status):
    assert block_backward(grads=grads) == status


def test_block_norm_backward_refuses_without_workspace():
    assert block_backward(ws=None) == WORKSPACE and block_backward(ws_bytes=16) == WORKSPACE
    assert block_backward(ws=FAKE + 8) == UNSUPPORTED
    assert block_backward(y=None, post_norm=0, w_post=None) == INVALID  # dy without y
    b = moe.moe_block_in(**BLOCK)
    assert moe.lib().moe_block_norm_backward(ctypes.addressof(b), None, FAKE, 1 << 40, None) == INVALID
    size = moe.moe_block_norm_backward_workspace_size
    assert size(8, 64, 0) > 0
    assert [size(0, 64, 0), size(8, 60, 0), size(8, 16392, 0), size(8, 64, 4), size(-1, 64, 1)] == [0] * 5


def w4(p=None, x=FAKE, idx=FAKE, gate=FAKE, ws=FAKE, ws_bytes=1 << 40, y=FAKE, up=None, down=None, **change):
    w = dict(codes=FAKE, scales=FAKE, group=64, has_zeros=0)
    w.update(change)
    mats = [moe.moe_w4(**{**w, **(m or {})}) for m in (None, up, down)]
    p = p or moe.Problem(T=64, d=128, E=16, k=4, F=64)
    return moe.lib().moe_w4_expert_ffn(p.c(), x, idx, gate, *(ctypes.addressof(m) for m in mats), y, ws,
                                       ws_bytes, None, None)


def problem(**change):
    return moe.Problem(**{**dict(T=64, d=128, E=16, k=4, F=64), **change})


@pytest.mark.parametrize("change, status", [
    (dict(x=None), INVALID), (dict(idx=None), INVALID), (dict(gate=None), INVALID), (dict(y=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(group=16), UNSUPPORTED),
    (dict(group=128), UNSUPPORTED),  # not a divisor of F
    (dict(up=dict(group=32)), UNSUPPORTED), (dict(up=dict(has_zeros=1)), UNSUPPORTED),
    (dict(down=dict(has_zeros=1)), UNSUPPORTED), (dict(codes=FAKE + 8), UNSUPPORTED),
    (dict(scales=FAKE + 2), UNSUPPORTED), (dict(x=FAKE + 2), UNSUPPORTED), (dict(y=FAKE + 2), UNSUPPORTED),
    (dict(idx=FAKE + 2), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
    (dict(ws=FAKE + 8), UNSUPPORTED), (dict(p=problem(T=0)), INVALID), (dict(p=problem(d=100)), UNSUPPORTED),
    (dict(p=problem(r=8)), UNSUPPORTED), (dict(p=problem(T=4097)), UNSUPPORTED),
    (dict(p=problem(E=1025)), UNSUPPORTED), (dict(p=problem(d=(1 << 20) + 64)), UNSUPPORTED),
])
def test_w4_refuses(change, status):
    assert w4(**change) == status


def test_w4_pack_refuses():
    call = lambda *a: moe.lib().moe_w4_pack(*a, None)  # noqa: E731
    ok = (2, 32, 128, 64, FAKE, FAKE, None, FAKE, FAKE)
    for at, value, status in ((0, 0, INVALID), (1, 0, INVALID), (2, -64, INVALID), (1, 24, UNSUPPORTED),
                              (2, 96, UNSUPPORTED), (3, 16, UNSUPPORTED), (4, None, INVALID),
                              (5, None, INVALID), (7, None, INVALID), (8, None, INVALID),
                              (5, FAKE + 1, UNSUPPORTED), (7, FAKE + 8, UNSUPPORTED),
                              (8, FAKE + 8, UNSUPPORTED)):
        assert call(*ok[:at], value, *ok[at + 1:]) == status, (at, value)
    assert call(2, 32, 192, 128, FAKE, FAKE, None, FAKE, FAKE) == UNSUPPORTED
    size = moe.moe_w4_expert_ffn_workspace_size
    assert size(problem()) > 0 and size(problem(r=8)) == 0 and size(problem(T=4097)) == 0


# ------------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_tensors_of_other_kinds():
    rule = moe.RouteRule(moe.MOE_SCORE_SIGMOID)
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="logits"):
        moe.moe_route_select(4, 8, 2, rule, moe.MOE_F32, cpu, None, cpu, cpu, None)
    with pytest.raises(ValueError, match="logits"):
        moe.moe_route_select_backward(4, 8, 2, rule, moe.MOE_BF16, cpu, cpu, cpu, cpu, None)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_route_select(4, 8, 2, rule, 7, cpu, None, cpu, cpu, None)
    with pytest.raises(ValueError, match="x:"):
        moe.moe_block_norm(4, 8, 1, 1, 1e-6, 1.0, cpu, cpu, 0, False, None, True, None, None, cpu, cpu)
    with pytest.raises(ValueError, match="x:"):
        moe.moe_block_norm(4, 8, 1, 1, 1e-6, 1.0, None, cpu, 0, False, None, True, None, None, cpu, cpu)
    with pytest.raises(ValueError, match="codes"):
        moe.W4Weights(torch.zeros(1, 16, 32, dtype=torch.uint8), torch.zeros(1, 16, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="codes"):
        moe.W4Weights(torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.bfloat16))


def test_limits_are_documented():
    with open(B.ROOT + "/include/moe_block.h") as f:
        text = " ".join(f.read().split())
    for words in ("E <= 1024, k <= 32, groups <= 32, T up to 2^24", "D a multiple of 8, at most 16384",
                  "T * k up to 16384"):
        assert words in text, words


@pytest.mark.parametrize("packed, structure", [("_BLOCK_IN", "moe_block_in"),
                                               ("_BLOCK_GRADS", "moe_block_grads")])
def test_structures_as_bytes(packed, structure):
    packed, structure = getattr(moe, packed), getattr(moe, structure)
    values = list(range(1, len(structure._fields_) + 1))
    assert packed.size == ctypes.sizeof(structure)
    read = structure.from_buffer_copy(packed.pack(*values))
    assert [getattr(read, name) for name, _ in structure._fields_] == values
