"""fp64 references of what stands around the experts (test infrastructure only): routing by scores
with a balance bias and groups, the norms before and after a block with its gate and residual
scale, and the experts with 4-bit weights.

"Day-Level Adaptation and LoRA Fine-Tuning of Ultra-Large-Scale Sparse MoE Models", sections 2.1
and 3.3 (routing scores, Top-k selection), "Fine-Tuning Trillion-Parameter Sparse MoE Models:
Challenges and Engineering Practices", section 5 (normalization next to the blocks); the pages
give no equations for these forms, and the plainest readings are taken.
"""

from __future__ import annotations

import numpy as np

__all__ = ["select", "select_backward", "block_norm", "block_norm_backward", "w4_values",
           "w4_expert_ffn"]


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _scores(logits, sigmoid):
    """Scores of a row, whose maximum may be -inf."""
    if sigmoid:
        with np.errstate(over="ignore"):
            return np.where(logits < 0, np.exp(np.minimum(logits, 0)) / (1 + np.exp(
                np.minimum(logits, 0))), 1 / (1 + np.exp(-np.maximum(logits, 0))))
    if logits.max() == -np.inf:
        return np.zeros_like(logits)
    with np.errstate(invalid="ignore"):  # inf - inf
        e = np.exp(logits - logits.max())
    return e / e.sum()


def _gates(row, idx, sigmoid, renormalise, scale):
    """(gates, scores over their sum or scores) of the experts idx."""
    s = _scores(row, sigmoid)[idx]
    if renormalise:
        if sigmoid and row[idx].max() < -40:  # where scores vanish
            with np.errstate(invalid="ignore"):
                s = np.exp(row[idx] - row[idx].max()) / (1 + np.exp(row[idx]))
            s = np.where(np.isnan(s), 0, s)
        elif not sigmoid and row[idx].max() > -np.inf:
            with np.errstate(invalid="ignore"):
                s = np.exp(row[idx] - row[idx].max())
        s = s / s.sum() if s.sum() > 0 else 0 * s
    return scale * s, s


def select(logits, bias, k, sigmoid, groups, kept, best, renormalise, scale):
    """(idx, gates, sums of the scores' shares over blocks of eight tokens), a token at a time."""
    logits = _f64(logits)
    logits = np.where(np.isnan(logits), -np.inf, logits)
    T, E = logits.shape
    idx, gates = np.zeros((T, k), np.int64), np.zeros((T, k))
    partials = np.zeros(((T + 7) // 8, E))
    first = lambda v, n: sorted(range(len(v)), key=lambda i: (-v[i], i))[:n]  # noqa: E731
    for t in range(T):
        s = _scores(logits[t], sigmoid)
        c = s if bias is None else s + _f64(bias)
        c = np.where(np.isnan(c), -np.inf, c)
        key = logits[t] if bias is None else c
        worth = [sum(sorted(g)[::-1][:best]) for g in c.reshape(groups, -1)]
        into = first(worth, kept) if groups > 1 else [0]
        may = [e for e in range(E) if e // (E // groups) in into]
        idx[t] = np.array(may)[first(key[may], k)]
        gates[t] = _gates(logits[t], idx[t], sigmoid, renormalise, scale)[0]
        partials[t // 8] += s / s.sum() if s.sum() > 0 else 0
    return idx, gates, partials


def select_backward(logits, idx, dgate, sigmoid, renormalise, scale):
    """Gradient of <dgate, gates> with respect to the logits; bad ids count for nothing."""
    logits = _f64(logits)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        good = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        if not good:
            continue
        e = idx[t, good]
        d = scale * _f64(dgate)[t, good]
        s = _scores(logits[t], sigmoid)
        if renormalise:
            w = _gates(logits[t], e, sigmoid, True, 1.0)[1]
            v = w * (d - (w * d).sum())
            if sigmoid:
                v = v * _scores(-logits[t], True)[e]
            np.add.at(out[t], e, v)
        elif sigmoid:
            np.add.at(out[t], e, d * s[e] * _scores(-logits[t], True)[e])
        else:
            ds = np.zeros(E)
            np.add.at(ds, e, d)
            out[t] = s * (ds - (ds * s).sum())
    return out


def block_norm(x, y, gate, gate_sigmoid, post, w_post, w_pre, scale, eps):
    """(z, n); gate: None, or an array that spreads over [N, D]."""
    z = _f64(x)
    if y is not None:
        u = _f64(y)
        if post:
            u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
            u = u if w_post is None else u * _f64(w_post)
        a = 1.0 if gate is None else _f64(gate)
        a = 1 / (1 + np.exp(-a)) if gate is not None and gate_sigmoid else a
        z = z + scale * a * u
    n = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
    return z, n if w_pre is None else n * _f64(w_pre)


def block_norm_backward(x, y, gate, gate_sigmoid, post, w_post, w_pre, scale, eps, dz, dn):
    """Gradients of <dz, z> + <dn, n>: dict of dx, dy, da (of a gate spread over [N, D]; the caller
    adds over what the gate is shared by), dw_post, dw_pre."""
    z, _ = block_norm(x, y, gate, gate_sigmoid, post, w_post, w_pre, scale, eps)

    def norm_backward(v, w, d):
        r = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
        dw = (d * v * r).sum(0)
        d = d if w is None else d * _f64(w)
        return r * d - v * r ** 3 * (d * v).mean(-1, keepdims=True), dw

    out = dict(dw_pre=np.zeros(z.shape[1]))
    total = np.zeros_like(z) if dz is None else _f64(dz)
    if dn is not None:
        through, out["dw_pre"] = norm_backward(z, w_pre, _f64(dn))
        total = total + through
    out["dx"] = total
    if y is None:
        return out
    y = _f64(y)
    a, da = 1.0, 1.0
    if gate is not None:
        a = _f64(gate)
        if gate_sigmoid:
            a = 1 / (1 + np.exp(-a))
            da = a * (1 - a)
    u = block_norm(0 * z, y, None, False, post, w_post, None, 1.0, eps)[0]
    out["da"] = scale * total * u * da
    out["dy"] = scale * total * a
    if post:
        out["dy"], out["dw_post"] = norm_backward(y, w_post, out["dy"])
    return out


def w4_values(codes, scales, zeros):
    """Weights [..., rows, cols] of codes [..., rows, cols / 2] (the lower four bits first)."""
    codes = np.asarray(codes).astype(np.int64)
    v = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.float64)
    group = v.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else np.repeat(_f64(np.asarray(zeros) & 15), group, -1)
    return (v - z) * np.repeat(_f64(scales), group, -1)


def w4_expert_ffn(x, idx, gate, w_gate, w_up, w_down):
    """y, with weights [E, F, d], [E, F, d], [E, d, F] as values; bad ids contribute nothing."""
    x, y = _f64(x), np.zeros(np.shape(x))
    E = len(w_gate)
    for t in range(len(x)):
        for j in range(idx.shape[1]):
            e = idx[t, j]
            if 0 <= e < E:
                a, b = w_gate[e] @ x[t], w_up[e] @ x[t]
                y[t] += float(gate[t, j]) * (w_down[e] @ (a / (1 + np.exp(-a)) * b))
    return y
