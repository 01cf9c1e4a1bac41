"""Inputs and tolerances of the expert-side operators' tests."""
import numpy as np

import oracle.experts_oracle as X
import oracle.router_oracle as O

# fp32 sums of L products: each addition is off by at most one step of the
# running sum (tensor cores may truncate: 2^-23 where round-to-nearest has
# 2^-24), so L additions by at most L 2^-23 times the sum of magnitudes
SUM_STEP = 2.0 ** -23
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def tolerance(ref, mag, length, out):
    """Bound of |result - ref| for a fp32 sum of ``length`` products of exact
    inputs, rounded once to ``out``."""
    s = (length + 2) * SUM_STEP * mag
    return s + HALF_STEP[out] * (np.abs(ref) + s)


def assert_within(got, ref, tol, what=""):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} values off, worst "
                           f"{np.nanmax(np.abs(got - ref) - tol):.3e} beyond the bound, first at "
                           f"{tuple(int(i[0]) for i in np.nonzero(bad))}")


def route(T, E, K, seed, spread=0.5, drop=0.0, empty=()):
    """Choices [T, K] of unequally liked experts and their maps.  ``drop``: that
    share of the choices is -1; ``empty``: experts nobody picks (their number
    leaves at least K)."""
    rng = np.random.default_rng(seed)
    like = rng.standard_normal((T, E)) + spread * rng.standard_normal((1, E))
    like[:, list(empty)] = -np.inf
    idx = np.argsort(-like, axis=1, kind="stable")[:, :K].astype(np.int32)
    if drop:
        idx[rng.random((T, K)) < drop] = -1
    w = rng.random((T, K), dtype=np.float32) + np.float32(0.1)
    choices = sorted((int(idx[t, k]), t, k) for t in range(T) for k in range(K)
                     if idx[t, k] >= 0)
    # entries of rows without a choice hold numbers that must not be used
    p2u, u2p = np.full(T * K, -7, np.int32), np.full(T * K, -1, np.int32)
    counts = np.zeros(E, np.int64)
    for p, (e, t, k) in enumerate(choices):
        p2u[p], u2p[t + k * T] = t + k * T, p
        counts[e] += 1
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return dict(idx=idx, w=w, off=off, p2u=p2u, u2p=u2p)


def normals(shape, seed, dtype, scale=1.0):
    """fp32 values, exact in ``dtype``."""
    a = (np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32)
    if dtype == "bf16":
        a = np.asarray(O.round_to_bf16(a), dtype=np.float32)
    return a


def w4_weights(E, N, D, group, zeros, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (E, N, D // 2), dtype=np.uint8)
    s = np.asarray(O.round_to_bf16(rng.uniform(0.5, 1.5, (E, N, D // group)) * 0.2 / np.sqrt(D)),
                   dtype=np.float32)
    z = rng.integers(0, 16, (E, N, D // group), dtype=np.uint8) if zeros else None
    return q, s, z


__all__ = ["X", "O", "tolerance", "assert_within", "route", "normals", "w4_weights"]
