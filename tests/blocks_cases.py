"""Inputs and tolerances of the tests of the operators around the routed experts."""
import numpy as np

import oracle.blocks_oracle as B
from experts_cases import HALF_STEP, O, assert_within, normals, route

STEP = 2.0 ** -24  # half a step of fp32, relative to the value


def sequences(T, S, pad, seed, front=0):
    """Offsets [S + 1] of S sequences of random lengths (some may be empty) on the
    tokens front .. T - pad - 1."""
    cuts = np.sort(np.random.default_rng(seed).integers(front, T - pad + 1, S - 1))
    return np.concatenate([[front], cuts, [T - pad]]).astype(np.int32)


def choices(T, E, K, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    like = rng.standard_normal((T, E)) + 0.5 * rng.standard_normal((1, E))
    idx = np.argsort(-like, axis=1, kind="stable")[:, :K].astype(np.int32)
    idx[rng.random((T, K)) < drop] = -1
    return idx


def score_error(x, score_func):
    """Relative bound of a score: the hardware's exponential and reciprocal (2 ulp and 1
    ulp of 2^-23), the argument's rounding (2^-24 of up to log2(e) |x| or |x - max|,
    both ways round the sum), the division and the sum over the row's 128-column pieces
    (at most 18 + 5 + 6 additions)."""
    x = np.asarray(x, np.float64)
    if x.size == 0:
        return 0.0
    spread = float(np.max(np.abs(x - np.max(x, axis=1, keepdims=True)))) \
        if score_func == "softmax" else float(np.max(np.abs(x)))
    return (2 * (2 + 1) * 2 + 2 * 1.45 * spread + 2 + 30) * STEP


def balance_loss_tolerance(x, score_func, loss, rows_added=96):
    """Of the loss: the scores' error and as many additions to a column's sum as a team's
    rows, a block's teams and a sequence's slots make (fewer than rows_added for the sizes
    tested); the z loss takes log-sums that are off by the scores' error and two steps of
    their own value (once in the sum, once in the logarithm) each, squared."""
    e = score_error(x, score_func) + rows_added * STEP
    m = score_error(x, "softmax")
    lse = np.log(np.exp(x - x.max(1, keepdims=True)).sum(1)) + x.max(1) if x.size else np.zeros(1)
    smallest = np.sqrt(max(float(np.mean(lse * lse)), 1e-30))
    return np.array([e * abs(loss[0]),
                     abs(loss[1]) * (2 * (m / smallest + 4 * STEP) + rows_added * STEP)]) + 1e-37


def norm_tolerances(ref, case, dtype):
    """name -> bound of |result - reference| of a forward, from its formula: a sum of K
    terms is off by K half steps of its magnitude, a mean of squares by 64 (columns of a
    lane, shuffles, warps), and each norm's factor by half its mean's error."""
    y, x, rstd = ref["y"], ref["x"], ref["rstd"]
    T, K = y.shape[0], case["K"]
    half = HALF_STEP[dtype]
    dy = (K + 1) * STEP * ref["y_mag"]
    tiny = 1e-300

    def length(v):
        return np.sqrt(np.sum(v * v, axis=1, keepdims=True)) + tiny

    by = abs(case["scale"]) * np.abs(B._wide(case["gate"], T))
    r0 = 36 * STEP + length(dy) / length(y)
    w = 1.0 if case["post"] is None else np.abs(case["post"])
    h = np.abs(y) * rstd[:, :1] * w
    dh = (h * r0 if case["post"] is not None else 0.0) + 4 * STEP * h + rstd[:, :1] * w * dy
    dx = by * dh + 4 * STEP * (np.abs(x) + by * h)
    out = {"x": dx + half * (np.abs(x) + dx), "y": dy + half * (np.abs(y) + dy),
           "rstd": np.concatenate([rstd[:, :1] * r0, rstd[:, 1:] * (36 * STEP + length(dx) / length(x))],
                                  axis=1) + STEP * rstd}
    if ref["normed"] is not None:
        n = np.abs(ref["normed"])
        dn = n * (36 * STEP + length(dx) / length(x) + 4 * STEP) + \
            rstd[:, 1:] * np.abs(case["pre"]) * dx
        out["normed"] = dn + half * (n + dn)
    return out


def norm_grad_tolerance(name, ref, mag, T, dtype, gate_value):
    """Each gradient is a sum of products of up to eight factors and of row sums of 40
    additions; the weights' gradients add up to T rows (a team's, then teams in sixteenths)."""
    length = 64 + (min(T, 40 + T / 304) + 170 if name in ("grad_post_weight", "grad_pre_weight") else 0)
    s = length * STEP * mag
    rounded = name in ("grad_block", "grad_residual") or (name == "grad_gate" and gate_value)
    return s + (HALF_STEP[dtype] if rounded else 0.0) * (np.abs(ref) + s) + 1e-37


__all__ = ["B", "O", "STEP", "HALF_STEP", "assert_within", "normals", "route"]
