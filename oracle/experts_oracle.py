"""CPU oracle of the expert-side operators: plain float64, from the definitions.

TEST INFRASTRUCTURE ONLY, like the router's oracle beside it: nothing on the
product path imports it.  Each function takes numpy arrays (any float type,
widened to float64) and the maps as router_expert_maps defines them: expert e
owns the permuted rows offsets[e] .. offsets[e+1]-1, and the expanded row u =
t + k T of permuted row p is permuted_to_unpermuted[p].

The ``*_magnitude`` results are the same sums over absolute values: rounding
errors of a sum in floating point are bounded by a multiple of them.
"""
from __future__ import annotations

import numpy as np


def source_rows(x, offsets, p2u, T):
    """x's rows in permuted order (those of x itself without a map); rows that
    no expert owns are zero."""
    x = np.asarray(x, dtype=np.float64)
    if p2u is None:
        return x
    out = np.zeros((len(p2u), x.shape[1]))
    for p in range(int(offsets[-1])):
        out[p] = x[int(p2u[p]) % T]
    return out


def expert_matmul(x, weight, offsets, p2u=None, T=0):
    """(out, magnitude), both [P, N]; rows that no expert owns are NaN."""
    xp = source_rows(x, offsets, p2u, T)
    weight = np.asarray(weight, dtype=np.float64)
    out = np.full((xp.shape[0], weight.shape[1]), np.nan)
    mag = np.full_like(out, np.nan)
    for e in range(weight.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            out[a:b] = xp[a:b] @ weight[e].T
            mag[a:b] = np.abs(xp[a:b]) @ np.abs(weight[e]).T
    return out, mag


def expert_matmul_bwd_input(grad_out, weight, offsets):
    """(grad_x, magnitude), both [P, D]; rows that no expert owns are NaN."""
    return expert_matmul(grad_out, np.swapaxes(np.asarray(weight, dtype=np.float64), 1, 2),
                         offsets)


def expert_matmul_bwd_weight(grad_out, x, offsets, p2u=None, T=0):
    """(grad_weight, magnitude), both [E, N, D]."""
    g = np.asarray(grad_out, dtype=np.float64)
    xp = source_rows(x, offsets, p2u, T)
    E = len(offsets) - 1
    out = np.zeros((E, g.shape[1], xp.shape[1]))
    mag = np.zeros_like(out)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        out[e] = g[a:b].T @ xp[a:b]
        mag[e] = np.abs(g[a:b]).T @ np.abs(xp[a:b])
    return out, mag


def unpack_w4(qweight, scales, zeros, group):
    """The real weights [E, N, D] behind packed nibbles: element d is the low
    half of byte d // 2 for even d, the high half for odd d."""
    q = np.asarray(qweight)
    E, N, half = q.shape
    w = np.empty((E, N, 2 * half))
    for d in range(2 * half):
        byte = q[:, :, d // 2]
        nib = (byte >> 4) if d % 2 else (byte & 15)
        z = 8.0 if zeros is None else np.asarray(zeros)[:, :, d // group].astype(np.float64)
        w[:, :, d] = (nib.astype(np.float64) - z) * np.asarray(scales, np.float64)[:, :, d // group]
    return w


def expert_matmul_w4(x, qweight, scales, zeros, group, offsets, p2u=None, T=0):
    """(out, magnitude), both [P, N]."""
    return expert_matmul(x, unpack_w4(qweight, scales, zeros, group), offsets, p2u, T)


def combine_fwd(expert_out, u2p, K, weights=None):
    """(out, magnitude), both [T, D]."""
    z = np.asarray(expert_out, dtype=np.float64)
    T = len(u2p) // K
    out = np.zeros((T, z.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for k in range(K):
            p = int(u2p[t + k * T])
            if 0 <= p < T * K:
                w = 1.0 if weights is None else float(weights[t, k])
                out[t] += w * z[p]
                mag[t] += np.abs(w * z[p])
    return out, mag


def combine_bwd(grad_out, u2p, K, expert_out=None, weights=None):
    """(grad_expert_out [T K, D] with NaN in rows no choice names, grad_weights
    [T, K] or None, magnitude of its sums)."""
    g = np.asarray(grad_out, dtype=np.float64)
    T, D = g.shape
    gz = np.full((T * K, D), np.nan)
    gw = np.zeros((T, K))
    mag = np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            p = int(u2p[t + k * T])
            if not 0 <= p < T * K:
                continue
            gz[p] = (1.0 if weights is None else float(weights[t, k])) * g[t]
            if expert_out is not None:
                z = np.asarray(expert_out[p], dtype=np.float64)
                gw[t, k] = g[t] @ z
                mag[t, k] = np.abs(g[t]) @ np.abs(z)
    return gz, (None if expert_out is None else gw), mag
