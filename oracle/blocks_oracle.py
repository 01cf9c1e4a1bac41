"""CPU oracle of the operators around the routed experts: plain float64 numpy, from
the definitions.

TEST INFRASTRUCTURE ONLY, like the oracles beside it: nothing on the product path
imports it.  Sequences, maps and gates are as include/moe_router.h defines them.  A
``mag`` beside a result is the same sum over absolute values, of which rounding errors
are a multiple.
"""
from __future__ import annotations

import numpy as np

from oracle.experts_oracle import combine_fwd, source_rows


def _scores(x, score_func):
    """(q, softmax, log sum exp, what d q_j takes of a difference) of one row."""
    m = np.max(x)
    e = np.exp(x - m)
    soft, lse = e / e.sum(), m + np.log(e.sum())
    if score_func == "softmax":
        return soft, soft, lse, soft
    sig = 1.0 / (1.0 + np.exp(-x))
    return sig / sig.sum(), soft, lse, sig * (1.0 - sig) / sig.sum()


def _ranges(seq, T):
    if seq is None:
        return [(0, T)]
    cut = [min(max(int(o), 0), T) for o in seq]
    return [(a, max(b, a)) for a, b in zip(cut, cut[1:])]


def balance_loss(logits, choices, score_func, coeff, z_coeff, seq=None):
    """(loss [2], counts [S, E])."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    K = np.asarray(choices).shape[1]
    ranges = _ranges(seq, T)
    counts = np.zeros((len(ranges), E), np.int64)
    n = max(ranges[-1][1] - ranges[0][0], 1)
    loss = np.zeros(2)
    for s, (a, b) in enumerate(ranges):
        sums = np.zeros(E)
        for t in range(a, b):
            q, _, lse, _ = _scores(x[t], score_func)
            sums += q
            loss[1] += z_coeff * lse * lse / n
            for e in choices[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if b > a:
            loss[0] += coeff / len(ranges) * E / (K * (b - a) ** 2) * np.dot(counts[s], sums)
    return loss, counts


def balance_loss_bwd(grad_loss, logits, counts, K, score_func, coeff, z_coeff, seq=None):
    """(grad_logits [T, E], mag)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    ranges = _ranges(seq, T)
    n = max(ranges[-1][1] - ranges[0][0], 1)
    grad, mag = np.zeros((T, E)), np.zeros((T, E))
    for s, (a, b) in enumerate(ranges):
        for t in range(a, b):
            q, soft, lse, w = _scores(x[t], score_func)
            by = grad_loss[0] * coeff / len(ranges) * E / (K * (b - a) ** 2)
            c = counts[s].astype(np.float64)
            z = grad_loss[1] * z_coeff * 2.0 * lse / n * soft
            grad[t] = by * w * (c - np.dot(c, q)) + z
            c = np.abs(c - (b - a) * K / E)  # a constant less changes nothing
            mag[t] = np.abs(by) * w * (c + np.dot(c, q)) + np.abs(z)
    return grad, mag


def quantize_rows(x):
    """(q [R, D] int, scales [R] float32)."""
    x = np.asarray(x, np.float64)
    top = np.max(np.abs(x), axis=1)
    scales = (top / 127.0).astype(np.float32)
    scales = np.where(top > 0, np.maximum(scales, np.float32(2.0 ** -126)), np.float32(0))
    q = np.zeros(x.shape, np.int64)
    for r in range(len(x)):
        if top[r] > 0:
            q[r] = np.rint(x[r] / np.float64(scales[r])).astype(np.int64)  # ties to even
    return q, scales.astype(np.float32)


def expert_matmul_w8(x, x_scales, weight, weight_scales, offsets, p2u=None, T=0):
    """(out, mag), both [P, N]; rows that no expert owns are NaN."""
    xq = np.asarray(x, np.float64)
    rows = source_rows(xq, offsets, p2u, T)
    scale = source_rows(np.asarray(x_scales, np.float64)[:, None], offsets, p2u, T)
    weight, ws = np.asarray(weight, np.float64), np.asarray(weight_scales, np.float64)
    out = np.full((rows.shape[0], weight.shape[1]), np.nan)
    mag = np.full_like(out, np.nan)
    for e in range(weight.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            out[a:b] = rows[a:b] @ weight[e].T * scale[a:b] * ws[e]
            mag[a:b] = np.abs(rows[a:b]) @ np.abs(weight[e]).T * np.abs(scale[a:b]) * np.abs(ws[e])
    return out, mag


def _wide(gate, T):
    """A gate as a [T, 1] or [T, D] factor."""
    if gate is None:
        return np.ones((T, 1))
    g = np.asarray(gate, np.float64)
    return g[:, None] if g.ndim == 1 else g


def combine_norm_fwd(expert_out, residual, u2p=None, weights=None, post_weight=None, gate=None,
                     residual_scale=1.0, pre_weight=None, eps=1e-6):
    """dict of x, normed, y, rstd [T, 2] and y_mag."""
    res = np.asarray(residual, np.float64)
    T = res.shape[0]
    if u2p is None:
        y = np.asarray(expert_out, np.float64)
        y_mag = np.abs(y)
    else:
        y, y_mag = combine_fwd(expert_out, u2p, len(u2p) // T, weights)
    rstd = np.ones((T, 2))
    h = y
    if post_weight is not None:
        rstd[:, 0] = 1.0 / np.sqrt(np.mean(y * y, axis=1) + eps)
        h = y * rstd[:, :1] * np.asarray(post_weight, np.float64)
    x = res + residual_scale * _wide(gate, T) * h
    normed = None
    if pre_weight is not None:
        rstd[:, 1] = 1.0 / np.sqrt(np.mean(x * x, axis=1) + eps)
        normed = x * rstd[:, 1:] * np.asarray(pre_weight, np.float64)
    return {"x": x, "normed": normed, "y": y, "rstd": rstd, "y_mag": y_mag}


def combine_norm_bwd(grad_sum, grad_normed, block_out, x, rstd, post_weight=None, gate=None,
                     residual_scale=1.0, pre_weight=None):
    """name -> (gradient, mag) of grad_block, grad_residual, grad_gate, grad_post_weight,
    grad_pre_weight (those that are)."""
    rows = grad_sum if grad_sum is not None else grad_normed
    T, D = rows.shape
    gx = np.zeros((T, D)) if grad_sum is None else np.asarray(grad_sum, np.float64)
    gx_mag = np.abs(gx)
    out = {}
    if pre_weight is not None:
        gn, r = np.asarray(grad_normed, np.float64), np.asarray(rstd, np.float64)[:, 1:]
        hat = np.asarray(x, np.float64) * r
        u = gn * np.asarray(pre_weight, np.float64)
        gx = gx + r * (u - hat * np.mean(u * hat, axis=1, keepdims=True))
        gx_mag = gx_mag + r * (np.abs(u) + np.abs(hat) * np.mean(np.abs(u * hat), axis=1,
                                                                  keepdims=True))
        out["grad_pre_weight"] = (gn * hat).sum(0), np.abs(gn * hat).sum(0)
    out["grad_residual"] = gx, gx_mag
    by = residual_scale * _wide(gate, T)
    gh, gh_mag = by * gx, np.abs(by) * gx_mag
    if post_weight is not None or gate is not None:
        r = np.asarray(rstd, np.float64)[:, :1] if rstd is not None else 1.0
        hat = np.asarray(block_out, np.float64) * (r if post_weight is not None else 1.0)
        w = 1.0 if post_weight is None else np.asarray(post_weight, np.float64)
        if gate is not None:
            g, m = residual_scale * gx * hat * w, np.abs(residual_scale * hat * w) * gx_mag
            out["grad_gate"] = (g.sum(1), m.sum(1)) if np.ndim(gate) == 1 else (g, m)
    if post_weight is not None:
        out["grad_post_weight"] = (gh * hat).sum(0), (gh_mag * np.abs(hat)).sum(0)
        v, v_mag = gh * w, gh_mag * np.abs(w)
        gh = r * (v - hat * np.mean(v * hat, axis=1, keepdims=True))
        gh_mag = r * (v_mag + np.abs(hat) * np.mean(v_mag * np.abs(hat), axis=1, keepdims=True))
    out["grad_block"] = gh, gh_mag
    return out
