"""CPU checks of the operators beside the gated delta rule: the oracle's gradients against
central differences and closed forms, and the refusals of the C ABI and of its binding, which
answer before anything reaches a GPU."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import linear_attention as LA
from oracle import sequence_mixing as SM
from top_routing_grouped_gemm_gb300 import build as B
from top_routing_grouped_gemm_gb300 import moe

FAKE = 0x10000  # never dereferenced: every call below fails its host checks first
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


# ------------------------------------------------------------------------ the oracle

def difference(f, x, step=1e-6):
    """Central differences of the scalar f at x."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        out[i] = (f(hi) - f(lo)) / (2 * step)
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 6])
def test_norm_rope_gradients_are_differences(rot, interleaved):
    rng = np.random.default_rng(1)
    N, H, D = 3, 2, 6
    x, w, dy = rng.normal(size=(N, H, D)), rng.normal(size=(H, D)), rng.normal(size=(N, H, D))
    pos, freq = np.array([0, -5, 1000]), 10.0 ** -np.arange(rot // 2)
    f = lambda x, w: np.sum(dy * SM.qk_norm_rope(x, w, pos, freq, rot, interleaved, 0.1))  # noqa: E731
    dx, dw = SM.qk_norm_rope_backward(x, w, pos, freq, rot, interleaved, 0.1, dy)
    assert np.abs(dx - difference(lambda v: f(v, w), x)).max() < 1e-7
    assert np.abs(dw - difference(lambda v: f(x, v), w)).max() < 1e-7


def test_rotation_depends_on_distance_alone():
    """<R(p) q, R(p + 7) k> is the same for every p; a quarter turn swaps a pair."""
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    freq = 100.0 ** -(np.arange(8) / 8)
    dots = [np.sum(SM.qk_norm_rope(q, None, [p], freq, 16, False, 1e-9)
                   * SM.qk_norm_rope(k, None, [p + 7], freq, 16, False, 1e-9))
            for p in (0, 3, 12345, -9)]
    assert np.ptp(dots) < 1e-9
    y = SM.qk_norm_rope(np.array([[[3.0, 4.0]]]), None, [1], [math.pi / 2], 2, True, 0.0)
    assert np.allclose(y, np.array([-4.0, 3.0]) / math.sqrt(12.5))


@pytest.mark.parametrize("mix", [False, True])
def test_recurrence_gradients_are_differences(mix):
    rng = np.random.default_rng(3)
    off, D = [0, 3, 3, 7], 2
    g, x = -rng.random((8, D)), rng.normal(size=(8, D))
    h0, dh, dh_T = rng.normal(size=(3, D)), rng.normal(size=(8, D)), rng.normal(size=(3, D))
    dh[7] = 0  # a padding row

    def f(g, x, h0):
        h, h_T = SM.gated_recurrence(g, x, off, h0, mix)
        return np.sum(dh * h) + np.sum(dh_T * h_T)

    got = SM.gated_recurrence_backward(g, x, off, dh, h0, dh_T, mix)
    assert np.abs(got["dg"] - difference(lambda v: f(v, x, h0), g)).max() < 1e-7
    assert np.abs(got["dx"] - difference(lambda v: f(g, v, h0), x)).max() < 1e-7
    assert np.abs(got["dh0"] - difference(lambda v: f(g, x, v), h0)).max() < 1e-7


def test_recurrence_closed_forms():
    one = np.ones((5, 1))
    h, _ = SM.gated_recurrence(np.log(0.5) * one, one, [0, 5])
    assert np.allclose(h[:, 0], 2 - 0.5 ** np.arange(5))
    h, _ = SM.gated_recurrence(np.log(0.5) * one, one, [0, 5], mix=True)
    assert np.allclose(h[:, 0], 1 - 0.5 ** np.arange(1, 6))
    h, _ = SM.gated_recurrence(0 * one, one, [0, 2, 5])  # no decay: running sums
    assert np.allclose(h[:, 0], [1, 2, 1, 2, 3])
    x = np.arange(5.0)[:, None]
    h, h_T = SM.gated_recurrence(-np.inf * one, x, [0, 5], h0=[[9.0]])  # forgets at once
    assert np.array_equal(h, x) and h_T[0, 0] == 4


def test_steps_of_the_delta_rule_are_the_recurrence():
    """Steps from S_T go on where the whole sequence does."""
    rng = np.random.default_rng(4)
    q, k, v = (rng.normal(size=(1, 6, 1, 4)) for _ in range(3))
    beta, g = rng.random((1, 6, 1)), -rng.random((1, 6, 1))
    o, S = LA.gated_delta_rule(q, k, v, beta, g)
    now = LA.gated_delta_rule(q[:, :4], k[:, :4], v[:, :4], beta[:, :4], g[:, :4])[1]
    for t in (4, 5):
        ot, now = LA.gated_delta_rule(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1],
                                      beta[:, t:t + 1], g[:, t:t + 1], S0=now)
        assert np.allclose(ot[:, 0], o[:, t])
    assert np.allclose(now, S)


# ------------------------------------------------------------------------ refusals of the C ABI

def qk(**over):
    r = dict(x=FAKE, x_token_stride=256, x_head_stride=64, y=FAKE, y_token_stride=256,
             y_head_stride=64, weight=FAKE, weight_per_head=0, heads=4)
    r.update(over)
    return ctypes.byref(moe.moe_qk_rows(*[r[n] for n, _ in moe.moe_qk_rows._fields_]))


def qk_g(**over):
    r = dict(x=FAKE, x_token_stride=256, x_head_stride=64, dy=FAKE, dy_token_stride=256,
             dy_head_stride=64, dx=FAKE, dx_token_stride=256, dx_head_stride=64, weight=FAKE,
             dweight=FAKE, weight_per_head=0, heads=4)
    r.update(over)
    return ctypes.byref(moe.moe_qk_grads(*[r[n] for n, _ in moe.moe_qk_grads._fields_]))


ROPE_OK = dict(N=8, D=64, rot=64, inter=0, dtype=0, eps=1e-6, pos=FAKE, freq=FAKE, k=None)
ROPE_BAD = [
    (dict(N=0), INVALID), (dict(D=0), INVALID), (dict(rot=-16), INVALID),
    (dict(rot=80), INVALID), (dict(dtype=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(D=60, rot=32), UNSUPPORTED), (dict(D=264), UNSUPPORTED), (dict(rot=8), UNSUPPORTED),
]
QK_BAD = [
    (dict(x=None), INVALID), (dict(heads=0), INVALID), (dict(heads=5000), UNSUPPORTED),
    (dict(x=FAKE + 8), UNSUPPORTED), (dict(weight=FAKE + 4), UNSUPPORTED),
    (dict(x_token_stride=260), UNSUPPORTED), (dict(x_head_stride=68), UNSUPPORTED),
]
OUT_BAD = [
    (dict(p=None), INVALID), (dict(p=FAKE + 8), UNSUPPORTED), (dict(token_stride=0), INVALID),
    (dict(token_stride=192), INVALID), (dict(head_stride=0), INVALID),
    (dict(head_stride=32), INVALID), (dict(head_stride=-64), INVALID),
    (dict(token_stride=64, head_stride=448), INVALID),
]


def rope(q, backward=False, ws=FAKE, ws_bytes=1 << 30, dy_dtype=1, **over):
    a = dict(ROPE_OK, **over)
    head = (a["N"], a["D"], a["rot"], a["inter"], a["dtype"])
    if not backward:
        return moe.lib().moe_qk_norm_rope(*head, a["eps"], a["pos"], a["freq"], q, a["k"], None)
    return moe.lib().moe_qk_norm_rope_backward(*head, dy_dtype, a["eps"], a["pos"], a["freq"], q,
                                               a["k"], ws, ws_bytes, None)


@pytest.mark.parametrize("over, status", ROPE_BAD)
def test_norm_rope_refuses_sizes(over, status):
    assert rope(qk(), **over) == status
    assert rope(qk_g(), backward=True, **over) == status


@pytest.mark.parametrize("over, status", QK_BAD)
def test_norm_rope_refuses_heads(over, status):
    assert rope(qk(**over)) == status
    assert rope(qk(), k=qk(**over)) == status
    assert rope(qk_g(**over), backward=True) == status
    assert rope(qk_g(), backward=True, k=qk_g(**over)) == status


@pytest.mark.parametrize("over, status", OUT_BAD)
def test_norm_rope_refuses_outputs(over, status):
    named = lambda n: {(n if f == "p" else f"{n}_{f}"): v for f, v in over.items()}  # noqa: E731
    assert rope(qk(**named("y"))) == status
    assert rope(qk_g(**named("dx")), backward=True) == status


def test_norm_rope_refuses_the_rest():
    assert rope(None) == INVALID
    assert rope(None, backward=True) == INVALID
    assert rope(qk_g(), backward=True, dy_dtype=2) == INVALID
    assert rope(qk_g(), backward=True, dtype=1, dy_dtype=0) == INVALID
    assert rope(qk_g(dweight=FAKE + 8), backward=True) == UNSUPPORTED
    need = moe.moe_qk_norm_rope_backward_workspace_size(8, 64, 4, 0)
    assert need > 0
    assert rope(qk_g(), backward=True, ws_bytes=need - 1) == WORKSPACE
    assert rope(qk_g(), backward=True, ws=None) == WORKSPACE
    assert rope(qk_g(), backward=True, ws=FAKE + 8) == UNSUPPORTED
    assert moe.moe_qk_norm_rope_backward_workspace_size(0, 64, 4, 0) == 0
    assert moe.moe_qk_norm_rope_backward_workspace_size(8, 64, 4, 4) >= need


GLR_OK = dict(N=8, D=5, n_seq=2, off=FAKE, mode=0, dtype=0, g=FAKE, ld_g=5, x=FAKE, ld_x=5)
GLR_BAD = [
    (dict(N=0), INVALID), (dict(D=0), INVALID), (dict(n_seq=0), INVALID), (dict(g=None), INVALID),
    (dict(x=None), INVALID), (dict(mode=2), INVALID), (dict(dtype=2), INVALID),
    (dict(ld_g=4), INVALID), (dict(ld_x=4), INVALID), (dict(ld_x=-5), INVALID),
    (dict(off=None, n_seq=3), INVALID), (dict(n_seq=(1 << 24) + 1), UNSUPPORTED),
    (dict(g=FAKE + 1), UNSUPPORTED), (dict(x=FAKE + 2, dtype=1), UNSUPPORTED),
]


def glr(backward=False, out=FAKE, more=FAKE, **over):
    a = dict(GLR_OK, **over)
    head = [a[n] for n in ("N", "D", "n_seq", "off", "mode", "dtype", "g", "ld_g", "x", "ld_x")]
    if not backward:
        return moe.lib().moe_glr_forward(*head, None, out, None, None, None, None)
    return moe.lib().moe_glr_backward(*head, None, more, more, None, out, more, None, None, None)


@pytest.mark.parametrize("over, status", GLR_BAD)
def test_recurrence_refuses(over, status):
    assert glr(**over) == status
    assert glr(backward=True, **over) == status


def test_recurrence_refuses_the_rest():
    assert glr(out=None) == INVALID
    assert glr(out=FAKE + 1) == UNSUPPORTED
    assert glr(backward=True, out=None) == INVALID
    assert glr(backward=True, more=None) == INVALID
    assert glr(backward=True, more=FAKE + 1) == UNSUPPORTED
    assert glr(backward=True, ld_g=0) == INVALID  # a gradient has rows of its own


def test_steps_refuse():
    def glr_step(B=4, D=5, mode=0, dtype=0, g=FAKE, ld=5, slot=FAKE, n=4, state=FAKE, h=FAKE):
        return moe.lib().moe_glr_step(B, D, mode, dtype, g, ld, FAKE, ld, slot, n, state, h, None,
                                      None)

    for over in (dict(B=0), dict(D=0), dict(mode=3), dict(dtype=9), dict(g=None), dict(ld=4),
                 dict(n=0), dict(slot=None, n=3), dict(state=None), dict(h=None)):
        assert glr_step(**over) == INVALID, over
    for over in (dict(g=FAKE + 1), dict(h=FAKE + 1)):
        assert glr_step(**over) == UNSUPPORTED, over

    def gdr_step(B=4, H=2, dk=64, dv=128, q=FAKE, g=FAKE, slot=FAKE, n=4, S=FAKE, o=FAKE):
        return moe.lib().moe_gdr_step(B, H, dk, dv, q, FAKE, FAKE, FAKE, g, slot, n, 0.1, S, o,
                                      None, None)

    for over in (dict(B=0), dict(H=0), dict(q=None), dict(g=None), dict(n=0), dict(S=None),
                 dict(slot=None, n=3), dict(o=None)):
        assert gdr_step(**over) == INVALID, over
    for over in (dict(dk=32), dict(dv=96), dict(q=FAKE + 2), dict(S=FAKE + 4), dict(o=FAKE + 8)):
        assert gdr_step(**over) == UNSUPPORTED, over


# ------------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_tensors_that_are_not_what_the_call_says():
    """A host tensor, a wrong type, shape or stride raises before the library is called."""
    bf = torch.bfloat16
    x = torch.zeros((4, 2, 64), dtype=bf)
    freq, pos = torch.ones(32, dtype=torch.float64), torch.arange(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_qk_norm_rope(4, 64, 64, False, moe.MOE_BF16, 1e-6, pos, freq, dict(x=x, y=x),
                             None)
    z = torch.zeros((4, 8))
    with pytest.raises(ValueError):
        moe.moe_glr_forward(4, 8, 1, None, moe.MOE_GLR_ADD, moe.MOE_F32, z, z, None, z, None, None)
    with pytest.raises(ValueError):
        moe.moe_glr_step(4, 8, moe.MOE_GLR_ADD, moe.MOE_F32, z, z, None, 4, z, z)
    q, s = torch.zeros((4, 2, 64), dtype=bf), torch.zeros((4, 2))
    with pytest.raises(ValueError):
        moe.moe_gdr_step(4, 2, 64, 64, q, q, q, s, s, None, 4, 0.1, torch.zeros((4, 2, 64, 64)), q)


def test_binding_refuses_missing_tensors():
    """None where a call cannot do without a tensor raises like any other tensor that is not what
    the call says."""
    z, f = torch.zeros((4, 8)), moe.MOE_F32
    x = torch.zeros((4, 2, 64))
    freq, pos = torch.ones(32, dtype=torch.float64), torch.arange(4, dtype=torch.int32)
    calls = [lambda: moe.moe_glr_forward(4, 8, 1, None, 0, f, None, z, None, z, None, None),
             lambda: moe.moe_glr_forward(4, 8, 1, None, 0, f, z, z, None, None, None, None),
             lambda: moe.moe_glr_backward(4, 8, 1, None, 0, f, z, z, None, z[:1], z, None, None, z,
                                          None),
             lambda: moe.moe_glr_step(4, 8, 0, f, z, None, None, 4, z, z),
             lambda: moe.moe_qk_norm_rope(4, 64, 64, False, f, 1e-6, pos, freq,
                                          dict(x=None, y=x), None),
             lambda: moe.moe_qk_norm_rope(4, 64, 64, False, f, 1e-6, pos, freq,
                                          dict(x=x[:, 0], y=x), None),
             lambda: moe.moe_qk_norm_rope_backward(4, 64, 64, False, f, f, 1e-6, pos, freq,
                                                   dict(x=None, dy=x, dx=x), None, None)]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_recurrence_refuses_more_channels_than_a_launch_has_strips():
    for over in (dict(D=(1 << 20) + 1, ld_g=1 << 21, ld_x=1 << 21),
                 dict(D=1 << 30, ld_g=1 << 30, ld_x=1 << 30)):
        assert glr(**over) == UNSUPPORTED
        assert glr(backward=True, **over) == UNSUPPORTED
    assert moe.lib().moe_glr_step(4, (1 << 20) + 1, 0, 0, FAKE, 1 << 21, FAKE, 1 << 21, FAKE, 4,
                                  FAKE, FAKE, None, None) == UNSUPPORTED


def test_workspace_size_of_sizes_that_are_refused():
    big = 2 ** 31 - 1
    for N, D, q, k in ((4, 64, big, big), (4, 64, 4097, 1), (4, 64, 1, 4097), (4, 264, 1, 1),
                       (big, 64, 1, 1)):
        assert moe.moe_qk_norm_rope_backward_workspace_size(N, D, q, k) == 0
    assert moe.moe_qk_norm_rope_backward_workspace_size(1 << 30, 256, 4096, 4096) > 0


def test_packed_heads_are_the_structures():
    """The bytes that the binding hands over are the C structures, field by field."""
    for form, kind in ((moe._QK_ROWS, moe.moe_qk_rows), (moe._QK_GRADS, moe.moe_qk_grads)):
        values = tuple(range(1, len(kind._fields_) + 1))
        assert form.size == ctypes.sizeof(kind)
        assert form.pack(*values) == bytes(kind(*values))


def test_binding_refuses_heads_that_do_not_agree():
    x, y = torch.zeros((4, 2, 64)), torch.zeros((4, 3, 64))
    for r in (dict(x=x, y=y), dict(x=x, y=None), dict(x=x.transpose(1, 2), y=x),
              dict(x=x, y=x.bfloat16()), dict(x=x, y=x, weight=torch.ones(63)),
              dict(x=x, y=x, weight=torch.ones(3, 64)),
              dict(x=x, y=torch.zeros((4, 2, 128))[..., ::2])):
        with pytest.raises(ValueError):
            moe._qk_rows("q", r, torch.float32, 4, 64, -1)
        r = dict(r, dy=x, dx=r["y"])
        with pytest.raises(ValueError):
            moe._qk_grads("q", r, torch.float32, torch.float32, 4, 64, -1)
    for w, dw in ((torch.ones(64), torch.ones(2, 64)), (None, torch.ones(65))):
        with pytest.raises(ValueError):
            moe._qk_grads("q", dict(x=x, dy=x, dx=x, weight=w, dweight=dw), torch.float32,
                          torch.float32, 4, 64, -1)
    kind = moe.moe_qk_rows.from_buffer_copy(
        moe._qk_rows("q", dict(x=y[:, 1:], y=x, weight=torch.ones(2, 64)), torch.float32, 4, 64, -1))
    assert (kind.x, kind.x_token_stride, kind.x_head_stride) == (y.data_ptr() + 256, 192, 64)
    assert (kind.y_token_stride, kind.weight_per_head, kind.heads) == (128, 1, 2)
