"""The expert-side operators without a GPU: argument checks of the C ABI and of
the Python binding, and the pins of their oracle."""
import ctypes

import numpy as np
import pytest

from experts_cases import X, normals, route, w4_weights
from score_top_expert_gb300 import build as B

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its checks
BIG = 65537


@pytest.fixture(scope="module")
def L():
    B.build()
    import score_top_expert_gb300.router as r
    return r.lib()


def fwd(L, **kw):
    a = dict(x=FAKE, dt=1, w=FAKE, off=FAKE, p2u=FAKE, T=4, P=8, E=4, N=8, D=8, out=FAKE, odt=1)
    a.update(kw)
    return L.router_expert_matmul(a["x"], a["dt"], a["w"], a["off"], a["p2u"], a["T"], a["P"],
                                  a["E"], a["N"], a["D"], a["out"], a["odt"], None)


def dgrad(L, **kw):
    a = dict(g=FAKE, dt=1, w=FAKE, off=FAKE, P=8, E=4, N=8, D=8, out=FAKE, odt=1)
    a.update(kw)
    return L.router_expert_matmul_bwd_input(a["g"], a["dt"], a["w"], a["off"], a["P"], a["E"],
                                            a["N"], a["D"], a["out"], a["odt"], None)


def wgrad(L, **kw):
    a = dict(g=FAKE, dt=1, x=FAKE, off=FAKE, p2u=FAKE, T=4, P=8, E=4, N=8, D=8, out=FAKE, odt=1)
    a.update(kw)
    return L.router_expert_matmul_bwd_weight(a["g"], a["dt"], a["x"], a["off"], a["p2u"], a["T"],
                                             a["P"], a["E"], a["N"], a["D"], a["out"], a["odt"],
                                             None)


SIZES = [(dict(P=-1), -1), (dict(E=0), -1), (dict(N=0), -1), (dict(D=0), -1), (dict(dt=2), -1),
         (dict(odt=7), -1), (dict(E=2305), -2), (dict(N=BIG), -2), (dict(D=BIG), -2),
         (dict(off=None), -1), (dict(out=None), -1)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(x=None), -1), (dict(w=None), -1), (dict(T=-1), -1), (dict(T=0), -1),
    (dict(P=0, x=None, w=None, off=None, out=None), 0), (dict(P=0, T=0), 0)])
def test_matmul_rejects(L, kw, code):
    assert fwd(L, **kw) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(g=None), -1), (dict(w=None), -1), (dict(P=0, g=None, out=None), 0)])
def test_matmul_bwd_input_rejects(L, kw, code):
    assert dgrad(L, **kw) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(g=None), -1), (dict(x=None), -1), (dict(T=0), -1), (dict(T=-3), -1),
    (dict(P=0, off=None), -1), (dict(P=0, out=None), -1)])
def test_matmul_bwd_weight_rejects(L, kw, code):
    assert wgrad(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(P=-1), -1), (dict(E=0), -1), (dict(N=0), -1), (dict(D=0), -1), (dict(odt=2), -1),
    (dict(E=2305), -2), (dict(N=BIG), -2), (dict(D=128, group=48), -1), (dict(D=96, group=64), -1),
    (dict(group=0), -1), (dict(group=-32), -1), (dict(D=256, group=256), -2),
    (dict(group=16), -2), (dict(T=0), -1), (dict(x=None), -1), (dict(q=None), -1),
    (dict(s=None), -1), (dict(off=None), -1), (dict(out=None), -1),
    (dict(x=ctypes.c_void_p(0x1008)), -1), (dict(q=ctypes.c_void_p(0x1004)), -1),
    (dict(P=0, x=None), 0)])
def test_w4_rejects(L, kw, code):
    a = dict(x=FAKE, q=FAKE, s=FAKE, z=None, group=32, off=FAKE, p2u=FAKE, T=4, P=8, E=4, N=8,
             D=64, out=FAKE, odt=1)
    a.update(kw)
    assert L.router_expert_matmul_w4(a["x"], a["q"], a["s"], a["z"], a["group"], a["off"],
                                     a["p2u"], a["T"], a["P"], a["E"], a["N"], a["D"], a["out"],
                                     a["odt"], None) == code


COMBINE = [(dict(T=-1), -1), (dict(K=0), -1), (dict(D=0), -1), (dict(dt=5), -1),
           (dict(T=1 << 30, K=2), -1), (dict(K=37), -2), (dict(D=BIG), -2), (dict(ld=1), -1),
           (dict(u2p=None), -1), (dict(out=None), -1)]


@pytest.mark.parametrize("kw,code", COMBINE + [
    (dict(z=None), -1), (dict(T=0, z=None, u2p=None, out=None), 0)])
def test_combine_fwd_rejects(L, kw, code):
    a = dict(z=FAKE, dt=1, u2p=FAKE, w=FAKE, ld=2, T=4, K=2, D=8, out=FAKE)
    a.update(kw)
    assert L.router_combine_fwd(a["z"], a["dt"], a["u2p"], a["w"], a["ld"], a["T"], a["K"],
                                a["D"], a["out"], None) == code


@pytest.mark.parametrize("kw,code", COMBINE + [
    (dict(g=None), -1), (dict(z=None), -1), (dict(T=0, g=None, z=None, u2p=None, out=None), 0)])
def test_combine_bwd_rejects(L, kw, code):
    a = dict(g=FAKE, dt=1, u2p=FAKE, z=FAKE, w=FAKE, ld=2, T=4, K=2, D=8, out=FAKE, gw=FAKE)
    a.update(kw)
    assert L.router_combine_bwd(a["g"], a["dt"], a["u2p"], a["z"], a["w"], a["ld"], a["T"],
                                a["K"], a["D"], a["out"], a["gw"], None) == code


def test_binding_takes_cuda_tensors_only(L):
    torch = pytest.importorskip("torch")
    import score_top_expert_gb300.router as R
    x, w = torch.zeros(2, 8), torch.zeros(2, 8, 8)
    m = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: R.router_expert_matmul(x, w, m), lambda: R.router_combine_fwd(x, m, 1),
                 lambda: R.router_expert_matmul_bwd_input(x, w, m),
                 lambda: R.router_expert_matmul_bwd_weight(x, x, m),
                 lambda: R.router_expert_matmul_w4(x.bfloat16(), w, w, m),
                 lambda: R.router_combine_bwd(x, m, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---- pins of the oracle --------------------------------------------------------
def test_oracle_products_by_loops():
    T, E, K, N, D = 6, 4, 2, 3, 5
    m = route(T, E, K, seed=1, drop=0.2)
    x, w = normals((T, D), 1, "f32"), normals((E, N, D), 2, "f32")
    out, mag = X.expert_matmul(x, w, m["off"], m["p2u"], T)
    seen = np.zeros(T * K, bool)
    for t in range(T):
        for k in range(K):
            p, e = m["u2p"][t + k * T], m["idx"][t, k]
            if e < 0:
                assert p == -1
                continue
            seen[p] = True
            for n in range(N):
                terms = [float(w[e, n, d]) * float(x[t, d]) for d in range(D)]
                assert abs(out[p, n] - sum(terms)) < 1e-12
                assert abs(mag[p, n] - sum(map(abs, terms))) < 1e-12
    assert np.isnan(out[~seen]).all()


def test_oracle_w4_by_hand():
    # byte 0xA3: element 0 is 3, element 1 is 10
    q = np.zeros((1, 1, 16), np.uint8)
    q[0, 0, 0] = 0xA3
    w = X.unpack_w4(q, np.full((1, 1, 1), 0.5), None, 32)
    assert w[0, 0, 0] == (3 - 8) * 0.5 and w[0, 0, 1] == (10 - 8) * 0.5
    assert (w[0, 0, 2:] == -4.0).all()
    w = X.unpack_w4(q, np.full((1, 1, 1), 2.0), np.full((1, 1, 1), 3, np.uint8), 32)
    assert w[0, 0, 0] == 0.0 and w[0, 0, 1] == 14.0
    q, s, z = w4_weights(2, 3, 64, 32, True, 1)
    w = X.unpack_w4(q, s, z, 32)
    assert w.shape == (2, 3, 64) and s.shape == (2, 3, 2)


def test_oracle_gradients_by_differences():
    # L = sum(gy * combine(matmul(x, w), tw)): every gradient against central
    # differences (L is linear in each argument alone: exact up to rounding)
    T, E, K, N, D = 5, 4, 2, 3, 4
    m = route(T, E, K, seed=2, drop=0.2)
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((T, D)), rng.standard_normal((E, N, D))
    tw, gy = rng.standard_normal((T, K)), rng.standard_normal((T, N))

    def loss(x, w, tw):
        z, _ = X.expert_matmul(x, w, m["off"], m["p2u"], T)
        return float((gy * X.combine_fwd(z, m["u2p"], K, tw)[0]).sum())

    z, _ = X.expert_matmul(x, w, m["off"], m["p2u"], T)
    gz, gtw, _ = X.combine_bwd(gy, m["u2p"], K, z, tw)
    gw, _ = X.expert_matmul_bwd_weight(gz, x, m["off"], m["p2u"], T)
    gxp, _ = X.expert_matmul_bwd_input(gz, w, m["off"])
    gx, _ = X.combine_fwd(gxp, m["u2p"], K)
    h = 1e-3
    for name, args, grad in (("x", 0, gx), ("w", 1, gw), ("tw", 2, gtw)):
        base = [x, w, tw]
        for i in np.ndindex(grad.shape):
            up, dn = [b.copy() for b in base], [b.copy() for b in base]
            up[args][i] += h
            dn[args][i] -= h
            d = (loss(*up) - loss(*dn)) / (2 * h)
            assert abs(d - grad[i]) < 1e-9, (name, i)
