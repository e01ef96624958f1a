"""fp64 references of the operators beside the gated delta rule (test infrastructure only): the
per-head norm with rotation by position, and the gated linear recurrence over packed sequences.

"Fine-Tuning Trillion-Parameter Sparse MoE Models: Challenges and Engineering Practices",
section 5, names normalization coefficients, gating and decay coefficients and a small state
recurrence without equations; the readings taken are the plainest ones:

    n = w x / sqrt(mean(x^2) + eps);  (y_a, y_b) = (n_a cos th - n_b sin th, n_b cos th + n_a sin th)
    h_t = exp(g_t) h_{t-1} + x_t,  or  h_t = exp(g_t) h_{t-1} + (1 - exp(g_t)) x_t

written out one token at a time.  Shapes: x [N, H, D], w [D] or [H, D] or None, positions [N],
inv_freq [rotary_dim / 2]; g, x [N, D], off [S + 1], h0 [S, D] or None.
"""

from __future__ import annotations

import numpy as np

__all__ = ["qk_norm_rope", "qk_norm_rope_backward", "gated_recurrence",
           "gated_recurrence_backward"]


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _pair_index(rotary_dim, interleaved):
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def _rotate(n, positions, inv_freq, rotary_dim, interleaved, sign):
    y = n.copy()
    if rotary_dim:
        a, b = _pair_index(rotary_dim, interleaved)
        th = sign * np.asarray(positions, dtype=np.float64)[:, None] * _f64(inv_freq)[None]
        c, s = np.cos(th)[:, None], np.sin(th)[:, None]
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
    return y


def qk_norm_rope(x, w, positions, inv_freq, rotary_dim, interleaved, eps):
    x = _f64(x)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    if w is not None:
        n = n * _f64(w)
    return _rotate(n, positions, inv_freq, rotary_dim, interleaved, 1.0)


def qk_norm_rope_backward(x, w, positions, inv_freq, rotary_dim, interleaved, eps, dy):
    """(dx, dw [H, D]) of <dy, y>: the rotation transposed, then with x^ = x / rms and
    u = w dn: dw = sum_t dn x^, dx = (u - x^ mean(u x^)) / rms."""
    x, dy = _f64(x), _f64(dy)
    rms = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    xh = x / rms
    dn = _rotate(dy, positions, inv_freq, rotary_dim, interleaved, -1.0)
    dw = np.sum(dn * xh, axis=0)
    u = dn if w is None else dn * _f64(w)
    return (u - xh * np.mean(u * xh, axis=-1, keepdims=True)) / rms, dw


def _gate(g, x, mix):
    a = np.exp(_f64(g))
    return a, (-np.expm1(_f64(g)) * _f64(x) if mix else _f64(x))


def gated_recurrence(g, x, off, h0=None, mix=False):
    """h [N, D] (padding rows zero) and h_T [S, D]."""
    a, b = _gate(g, x, mix)
    S, D = len(off) - 1, a.shape[1]
    h = np.zeros_like(a)
    h_T = np.zeros((S, D)) if h0 is None else _f64(h0).copy()
    for s in range(S):
        now = h_T[s].copy()
        for t in range(off[s], off[s + 1]):
            now = a[t] * now + b[t]
            h[t] = now
        h_T[s] = now
    return h, h_T


def gated_recurrence_backward(g, x, off, dh, h0=None, dh_T=None, mix=False):
    """Gradients of <dh, h> + <dh_T, h_T>: lam_t = dh_t + a_{t+1} lam_{t+1} (dh_T at the end),
    dx = lam or (1 - a) lam, dg = a lam h_{t-1} or a lam (h_{t-1} - x), dh0 = a lam of row 0."""
    a, _ = _gate(g, x, mix)
    x, dh = _f64(x), _f64(dh)
    S, D = len(off) - 1, a.shape[1]
    h, _ = gated_recurrence(g, x, off, h0, mix)
    dg, dx = np.zeros_like(a), np.zeros_like(a)
    dh0 = np.zeros((S, D)) if dh_T is None else _f64(dh_T).copy()
    for s in range(S):
        back = dh0[s].copy()
        for t in range(off[s + 1] - 1, off[s] - 1, -1):
            lam = dh[t] + back
            if t > off[s]:
                prev = h[t - 1]
            else:
                prev = np.zeros(D) if h0 is None else _f64(h0)[s]
            back = a[t] * lam
            dx[t] = -np.expm1(_f64(g)[t]) * lam if mix else lam
            dg[t] = back * (prev - x[t] if mix else prev)
        dh0[s] = back
    return dict(dg=dg, dx=dx, dh0=dh0)
